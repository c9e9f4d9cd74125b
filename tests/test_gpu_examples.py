"""The examples run, and check themselves, on the GPU."""
import importlib.util
import os

import pytest
import torch

from tests.parity import announce

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("argv", [[], ["--requests", "1", "--prompt", "1", "--drafts", "1"],
                                  ["--requests", "2", "--prompt", "70", "--drafts", "66", "--layers", "3"]])
def test_verify_drafts(argv):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    announce(f"verify_drafts {argv}")
    spec = importlib.util.spec_from_file_location("verify_drafts", os.path.join(ROOT, "examples", "verify_drafts.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    paths = example.main(argv)
    assert all(path[0] == 0 and path == sorted(path) for path in paths)
    if not argv:
        assert min(map(len, paths)) >= 3 and any(path != list(range(len(path))) for path in paths)
