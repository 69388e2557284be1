"""Shared-prefix attention over many positions whose weights are small beside
the largest one: together they count."""
import pytest
import torch

from decode_megakernel_interpreter_b200 import serving as sv
from serve_ref import attention, check_attention

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("log2", [-15, -20, -24.5, -26, -28])
@pytest.mark.parametrize("kind, B, heads, n", [("prefix", 1, 1, 1 << 17), ("prefix", 1, 160, 1 << 17), ("own", 1, 1, 1 << 17),
                                               ("own", 12, 160, 1 << 17), ("prefix", 1, 1, 960)])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_small_weights(dtype, first, kind, B, heads, n, log2):
    """One position of weight 1 whose value is 0, and n of 2^log2 whose values are 1 and 2: for one head, whose
    positions are shared out over the whole GPU, and for so many that a block or a warp takes all positions of one.

    The bound is serve_ref's, and for fp16 half a step of its smallest numbers, 2^-25, for each weight: in units of
    2^-7 of the row's largest so far, which is that of all or less."""
    d, page = 64, 64
    k = torch.zeros(2, heads, page, d, device="cuda", dtype=dtype)  # page 0: the one position among small ones; page 1: small ones
    v = torch.ones(2, heads, page, d, device="cuda", dtype=dtype)
    v[..., d // 2:] = 2
    k[..., 0] = log2 * 0.6931471805599453  # (rounded to the type: the reference reads the same)
    at = 0 if first else page - 1
    k[0, :, at] = 0
    v[0, :, at] = 0
    q = torch.zeros(B, 1, heads, d, device="cuda", dtype=dtype)
    q[..., 0] = 1
    pages = [0] + [1] * (n // page)
    if not first:
        pages.reverse()
    total = len(pages) * page
    c = dict(q=q, k=k, v=v, table=ints([pages] * B), lens=ints([total] * B))
    if kind == "prefix":
        c.update(prefix_pages=ints(pages), prefix_len=ints([total]))
    got = sv.shared_attention(**c, scale=1.0, return_lse=True)
    one = dict(c, q=q[:1, :, :1], k=k[:, :1], v=v[:, :1], table=c["table"][:1], lens=c["lens"][:1])  # (all are alike)
    out, lse, tol_o, tol_l = attention(**one, scale=1.0)
    if dtype is torch.float16:
        tol_o = tol_o + total * 2.0 ** -32 * v.double().abs().amax().item()
    want = [x.expand(B, 1, heads, *x.shape[3:]) for x in (out, lse, tol_o, tol_l)]
    check_attention(got, want, (kind, first, log2))
