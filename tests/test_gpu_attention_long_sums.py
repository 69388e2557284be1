"""Shared-prefix attention where one block or one warp sums over very many
positions."""
import pytest
import torch

from decode_megakernel_interpreter_b200 import serving as sv

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kind, B, heads, n", [("prefix", 1, 160, 1 << 18), ("prefix", 1, 160, 1 << 20), ("prefix", 300, 150, 70001),
                                               ("own", 12, 160, 1 << 18), ("own", 24, 75, 100003), ("both", 12, 160, 50000)])
def test_long_sums(kind, B, heads, n, dtype, d):
    """Random positions repeated by the page list, values around 1, in as many heads as keep every block busy.

    A row's error, against 64 bits and in units of its output, all terms of one sign: half a step h of the type for the
    output and, on the tensor cores, for the weights; 2048 additions to a sum of at most 16384 positions (one for each
    16, each with its two numbers), cut off below 2^-23 of it: 2^-12; scores within 2^-15 of themselves (d + 2 products
    and the exponent's rounding: below 2^-24 (d + 2) |q||k| scale < 2^-15 here), twice; the joining of up to 64 sums and
    148 partials, 2^-15."""
    page, P = 64, 4
    g = torch.Generator(device="cuda").manual_seed(0)
    k = torch.randn(P, 1, page, d, generator=g, device="cuda").to(dtype).expand(P, heads, page, d).contiguous()
    v = (0.75 + 0.25 * torch.rand(P, 1, page, d, generator=g, device="cuda")).to(dtype).expand(P, heads, page, d).contiguous()
    q = (0.5 * torch.randn(1, 1, 1, d, generator=g, device="cuda")).to(dtype).expand(B, 1, heads, d).contiguous()
    pages = torch.arange(-(-n // page), device="cuda", dtype=torch.int32) % P
    c = dict(table=pages.repeat(B, 1), lens=ints([n] * B))
    if kind != "own":
        m = n if kind == "prefix" else n // 2
        c.update(prefix_pages=pages[:-(-m // page)].contiguous(), prefix_len=ints([m]))
    status = ints([0])
    out, lse = sv.shared_attention(q, k, v, **c, return_lse=True, status=status)
    assert int(status) == 0
    at = torch.arange(n, device="cuda")
    K, V = (x[pages[at // page].long(), 0, at % page].double() for x in (k, v))
    s = (K @ q[0, 0, 0].double()) / d ** 0.5
    want, z = s.softmax(0) @ V, torch.logsumexp(s, 0)
    h = torch.finfo(dtype).eps / 2
    tol = 2 * h + 2.0 ** -12 + 2.0 ** -14 + 2.0 ** -15
    assert ((out.double() - want).abs() <= tol * want).all(), float(((out.double() - want) / want).abs().max())
    assert ((lse.double() - z).abs() <= 2.0 ** -12 + 2.0 ** -14).all()
