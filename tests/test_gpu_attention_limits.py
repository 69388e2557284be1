"""Shared-prefix attention at the largest lengths: positions just below 2^31."""
import pytest
import torch

from decode_megakernel_interpreter_b200 import serving as sv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [1024, 1536])
def test_a_prefix_that_ends_just_below_2_31(page):
    """Every entry of the page list names one page, so a row's output is that over the page.

    A thread adds up the weights of its share of the prefix in 32 bits: 2^31 positions over 148 blocks are fewer than
    2^18 tiles, and as many additions, each off by 2^-24 of the sum at most: 2^-6 in all, in o as in the sum."""
    d, n = 64, (2 ** 31 - 64) // page
    if n * page >= 2 ** 31 - 64:
        n -= 1
    g = torch.Generator(device="cuda").manual_seed(0)
    k = torch.randn(1, 1, page, d, generator=g, device="cuda").bfloat16()
    v = (1 + 0.1 * torch.randn(1, 1, page, d, generator=g, device="cuda")).bfloat16()
    q = torch.randn(1, 1, 1, d, generator=g, device="cuda").bfloat16()
    length = torch.tensor([n * page], dtype=torch.int32, device="cuda")
    pages = torch.zeros(n, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert n * page > 2 ** 31 - 1984  # where a look-up of 32 boxes of 64 passes 2^31
    out, lse = sv.shared_attention(q, k, v, pages.view(1, n), length, pages, length, return_lse=True, status=status)
    assert int(status) == 0
    s = (k[0, 0].double() @ q[0, 0, 0].double()) / d ** 0.5
    want = s.softmax(0) @ v[0, 0].double()
    assert ((out[0, 0, 0].double() - want).abs() <= (2 * 2.0 ** -6 + 2.0 ** -8) * want.abs().amax()).all()
    z = torch.logsumexp(s, 0) + torch.log(torch.tensor(float(n), dtype=torch.float64))
    assert abs(float(lse) - float(z)) <= 2.0 ** -6 + 1e-4
