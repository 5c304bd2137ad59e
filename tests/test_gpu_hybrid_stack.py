"""The layer operators together: examples/hybrid_stack.py serves ragged prompts and
then single tokens; the tokens must come out as they do in longer prompts."""
import importlib.util
import os

import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_stack.py")


def _example():
    spec = importlib.util.spec_from_file_location("hybrid_stack", _PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("kinds", [("decay",), ("attention",), ("kda", "decay", "attention", "decay")])
def test_tokens_one_by_one_equal_longer_prompts(kinds):
    """Both sides round every layer's activations to bf16 (2^-9 each, about ten roundings a layer that
    do not fall together): within 5 % over up to four layers."""
    need_gpu()
    one, longer = _example().run([37, 1, 130, 64], 5, kinds=kinds)
    torch.cuda.synchronize()
    assert torch.isfinite(one).all() and torch.isfinite(longer).all()
    assert float((one.float() - longer.float()).norm() / longer.float().norm()) < 0.05
