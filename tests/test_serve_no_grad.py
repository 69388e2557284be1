"""The serving operators have no backward pass, and say so."""
import pytest
import torch

from decode_megakernel_interpreter_b200 import serving as sv


def calls(grad):
    g = lambda *s, t=torch.float32: torch.zeros(s, dtype=t).requires_grad_(grad)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    bf = torch.bfloat16
    q, k = torch.zeros(2, 1, 4, 64, dtype=bf), torch.zeros(8, 2, 16, 64, dtype=bf)
    yield lambda: sv.shared_attention(g(2, 1, 4, 64, t=bf), k, k, i(2, 4), i(2))
    yield lambda: sv.shared_attention(q, g(8, 2, 16, 64, t=bf), k, i(2, 4), i(2))
    yield lambda: sv.shared_attention(q, k, g(8, 2, 16, 64, t=bf), i(2, 4), i(2))
    yield lambda: sv.token_probs(g(2, 10))
    yield lambda: sv.token_probs(torch.zeros(2, 10), g(2))
    yield lambda: sv.verify(g(2, 3, 10), None, i(2, 2), torch.zeros(2, 3))
    yield lambda: sv.verify(torch.zeros(2, 3, 10), g(2, 2, 10), i(2, 2), torch.zeros(2, 3))


def test_tensors_that_require_gradients_are_refused():
    for call in calls(True):
        with pytest.raises(ValueError, match="no backward pass"):
            call()


def test_where_no_gradient_is_recorded_they_are_taken():
    """The next refusal is that these are not CUDA tensors."""
    for call in calls(True):
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call()
    for call in calls(False):
        with pytest.raises(ValueError, match="CUDA"):
            call()
