"""Token probabilities and draft verification on the GPU against 64-bit plain
forms."""
import math

import numpy as np
import pytest
import torch

import decode_megakernel_interpreter_b200 as mk
from decode_megakernel_interpreter_b200 import serving as sv
from serve_ref import U32, probs, verify

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ probabilities

def check_probs(z, t, got):
    """Relative error of a probability: an exponential in powers of two of
    y = (z - m) log2(e) / T, whose argument is off by (|y| + 1) 2^-22 at most (a
    difference, two products and a sum in fp32), twice (its own and the
    slice's), the exponential's own 2^-22 twice, a sum of n terms (64 per
    thread, then trees: below 128 roundings) and three products."""
    got = got.double().cpu().numpy()
    z = z.double().cpu().numpy()
    for i in range(z.shape[0]):
        ti = 1.0 if t is None else float(t[i])
        want = probs(z[i], ti)
        if ti > 0 and want.any():
            y = np.where(np.isfinite(z[i]), (z[i].max() - z[i]) / ti * 1.4427, 0.0)
            y = np.where(want > 0, y, 0.0)
            rel = (2 * (y + 1) + 2) * 2.0 ** -22 * 0.7 + 140 * U32
            tol = want * rel + 1.2e-38  # what is below the smallest normal may become 0
        else:
            tol = np.zeros_like(want)
        assert (np.abs(got[i] - want) <= tol).all(), (i, ti, np.abs(got[i] - want).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 100, 4095, 4096, 16383, 16384, 16389, 50001, 128256])
def test_vocabularies_and_types(V, dtype):
    g = torch.Generator(device="cuda").manual_seed(V)
    z = (4 * torch.randn(3, V, generator=g, device="cuda")).to(dtype)
    t = torch.tensor([1.0, 0.3, 2.5], device="cuda")
    check_probs(z, t, sv.token_probs(z, t))
    check_probs(z, None, sv.token_probs(z))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n, V", [(40, 16384), (41, 20001), (150, 32003), (75, 50004), (38, 128256), (40, 24576), (39, 24577),
                                  (64, 49152), (38, 49153), (38, 270001)])
def test_many_rows(n, V, dtype):
    """More rows than the chip holds at a time, with every kind of row among them."""
    g = torch.Generator(device="cuda").manual_seed(V)
    z = (4 * torch.randn(n, V, generator=g, device="cuda")).to(dtype)
    t = 0.3 + 2 * torch.rand(n, generator=g, device="cuda")
    t[::7] = 0
    z[7, 5000] = z[7, 9000] = z[7].max() + 1    # greedy with a tie
    z[3, ::2] = -math.inf
    z[4] = -math.inf
    z[5, V - 1] = math.nan
    z[14, 3] = math.nan                         # greedy
    z[6, 77] = math.inf
    z[8, :V - 1] = -math.inf
    t[9] = -1
    p = sv.token_probs(z, t)
    check_probs(z[:24], t[:24], p[:24])
    check_probs(z[-3:], t[-3:], p[-3:])
    assert int(p[7].argmax()) == 5000 and (p[[4, 5, 6, 9, 14]] == 0).all() and p[8, V - 1] == 1
    if dtype is torch.float32:
        sv.token_probs(z, t, out=z)             # in place
        assert torch.equal(z, p)
        big = torch.randn(n, V + 3, generator=g, device="cuda")
        out = torch.full((n, V + 1), 7.0, device="cuda")
        sv.token_probs(big[:, 2:V + 2], t, out=out[:, :V])
        check_probs(big[:3, 2:V + 2], t[:3], out[:3, :V])
        assert (out[:, V] == 7).all()


def test_a_vocabulary_that_does_not_stay_on_chip():
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(2, 500003, generator=g, device="cuda")
    check_probs(z, None, sv.token_probs(z))
    z = torch.randn(2, 500004, generator=g, device="cuda").bfloat16()
    t = torch.tensor([0.0, 1.0], device="cuda")
    check_probs(z, t, sv.token_probs(z, t))


@pytest.mark.parametrize("V", [1000, 20000])
def test_greedy_takes_the_first_of_the_largest(V):
    z = torch.zeros(5, V, device="cuda")
    z[1, V // 2] = z[1, V - 1] = 3
    z[2, 17] = z[2, 16] = 2
    z[3] = -math.inf
    z[3, V - 1] = -1e30
    z[4] = -5
    t = torch.zeros(5, device="cuda")
    p = sv.token_probs(z, t)
    assert p.argmax(1).tolist() == [0, V // 2, 16, V - 1, 0] and (p.sum(1) == 1).all() and (p.amax(1) == 1).all()


@pytest.mark.parametrize("V", [333, 40000])
def test_masked_tokens_and_rows_without_a_distribution(V):
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(9, V, generator=g, device="cuda")
    z[0, ::2] = -math.inf                       # tokens that cannot come
    z[1, 1:] = -math.inf                        # one is left
    z[2] = -math.inf                            # none
    z[3, V - 2] = math.nan
    z[4, 5] = math.inf
    z[5, 100:] = torch.finfo(torch.float32).min
    z[6] = torch.finfo(torch.float32).min       # a mask of the type's lowest value everywhere: uniform
    z[7, 3] = 3e38
    t = torch.ones(9, device="cuda")
    p = sv.token_probs(z, t)
    check_probs(z, t, p)
    assert (p[2:5] == 0).all() and p[1, 0] == 1 and (p[0, ::2] == 0).all()
    for bad in (-1.0, math.nan, math.inf):
        t[8] = bad
        assert (sv.token_probs(z, t)[8] == 0).all()
    t[8] = 1e-30
    p = sv.token_probs(z, t)
    assert p[8].max() == 1 and int(p[8].argmax()) == int(z[8].argmax())


def test_strided_rows_and_in_place():
    g = torch.Generator(device="cuda").manual_seed(3)
    for V, pad in ((1001, 6), (20001, 2), (20000, 4)):
        big = torch.randn(4, V + pad, generator=g, device="cuda")
        z = big[:, 1:V + 1]
        keep = big.clone()
        want = sv.token_probs(z.contiguous())
        out = torch.full((4, V + 3), 7.0, device="cuda")
        sv.token_probs(z, out=out[:, :V])
        check_probs(z, None, out[:, :V])
        assert (out[:, V:] == 7).all()
        sv.token_probs(z, out=z)
        check_probs(keep[:, 1:V + 1], None, z)
        assert torch.equal(big[:, 0], keep[:, 0]) and torch.equal(big[:, V + 1:], keep[:, V + 1:])
        assert torch.allclose(z, want, rtol=1e-5, atol=0)
    one = torch.randn(1, 777, generator=g, device="cuda").expand(5, 777)  # a broadcast row
    check_probs(one, None, sv.token_probs(one))


# ------------------------------------------------------------------ verification

def drafts(B, T, V, seed, point=False, noise=0.7):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = 2 * torch.randn(B, T + 1, V, generator=g, device="cuda")
    p = torch.softmax(z, -1)
    q = torch.softmax(z[:, :T] + noise * torch.randn(B, T, V, generator=g, device="cuda"), -1) if T else None
    src = p[:, :T] if point else q
    x = torch.multinomial(src.reshape(B * T, V), 1, generator=g).reshape(B, T).int() if T else \
        torch.zeros(B, 0, dtype=torch.int32, device="cuda")
    u = torch.rand(B, T + 1, generator=g, device="cuda")
    if point:
        u[:, :T] *= p[:, :T].amax(-1)
    return p, None if point else q, x, u


def check_verify(p, q, x, u, n=None, **kw):
    tok, acc = sv.verify(p, q, x, u, n_drafted=n, **kw)
    tok, acc = tok.cpu().numpy(), acc.cpu().numpy()
    B, T = x.shape
    P, Q, X, U = p.cpu().numpy(), None if q is None else q.cpu().numpy(), x.cpu().numpy(), u.cpu().numpy()
    counts = []
    for b in range(B):
        m = T if n is None else min(max(int(n[b]), 0), T)
        a, nxt = verify(P[b, :m + 1], None if Q is None else Q[b], X[b], m, U[b])
        assert acc[b] == a, b
        assert tok[b].tolist() == X[b, :a].tolist() + [nxt] + [-1] * (T - a), b
        counts.append(a)
    return counts


@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("V", [1, 2, 5, 511, 512, 513, 4096, 32003, 128256])
def test_vocabularies(V, point):
    counts = check_verify(*drafts(7, 4, V, V, point))
    if V > 500:
        assert len(set(counts)) > 1  # some stand, some fall


@pytest.mark.parametrize("B, T", [(1, 0), (5, 0), (1, 1), (33, 3), (3, 64), (200, 2)])
def test_batches_and_lengths(B, T):
    p, q, x, u = drafts(B, T, 700, B * 100 + T)
    check_verify(p, q, x, u)
    if T:
        r = np.random.RandomState(T)
        n = torch.tensor(r.randint(0, T + 1, B), dtype=torch.int32, device="cuda")
        check_verify(p, q, x, u, n)


def test_the_sampled_token_is_the_first_past_the_sum():
    """Exact sums (multiples of 2^-10): u on a border goes to the next token, zero weights are never drawn."""
    V = 1024
    w = torch.zeros(V)
    w[[3, 4, 700, 1000]] = torch.tensor([256.0, 512.0, 128.0, 128.0]) / 1024
    p = w.repeat(6, 1, 1).cuda()
    u = torch.tensor([[0.0], [0.25], [0.2499], [0.75], [0.875], [0.9999999]], device="cuda")
    tok, acc = sv.verify(p, None, torch.zeros(6, 0, dtype=torch.int32, device="cuda"), u)
    assert tok[:, 0].tolist() == [3, 4, 3, 700, 1000, 1000] and acc.tolist() == [0] * 6


def test_residuals():
    V = 600
    p, q = torch.zeros(1, 2, V, device="cuda"), torch.zeros(1, 1, V, device="cuda")
    p[0, 0, 1], p[0, 0, 2], q[0, 0, 1], q[0, 0, 5] = 0.5, 0.5, 0.5, 0.5
    p[0, 1, 9] = 1
    one = torch.tensor([[5]], dtype=torch.int32, device="cuda")
    u = torch.tensor([[0.0, 0.9]], device="cuda")
    tok, acc = sv.verify(p, q, one, u)
    assert tok.tolist() == [[2, -1]] and acc.item() == 0        # only token 2 exceeds q
    tok, acc = sv.verify(p, q, one - 4, u)
    assert tok.tolist() == [[1, 9]] and acc.item() == 1         # token 1 stands, then row 1
    tok, acc = sv.verify(p, p[:, :1].clone(), one, u)           # q = p, a token that neither has: drawn by p
    assert tok.tolist() == [[2, -1]] and acc.item() == 0
    tok, acc = sv.verify(p, None, one - 4, torch.tensor([[0.6, 0.0]], device="cuda"))
    assert tok.tolist() == [[2, -1]] and acc.item() == 0        # without token 1
    tok, acc = sv.verify(torch.zeros_like(p), None, one, u)     # no distribution at all
    assert tok.tolist() == [[-1, -1]] and acc.item() == 0
    only = torch.zeros_like(p)
    only[0, 0, 5] = 1
    tok, acc = sv.verify(only, None, one, torch.tensor([[0.99, 0.0]], device="cuda"))
    assert tok.tolist() == [[5, -1]] and acc.item() == 1        # its next row is empty


def test_greedy_verification_keeps_what_the_target_would_choose():
    """Temperature 0 on both sides: a token stands exactly when it is the target's first largest."""
    z = torch.randn(40, 5, 300, device="cuda")
    p = sv.token_probs(z.view(-1, 300), torch.zeros(200, device="cuda")).view(40, 5, 300)
    best = z.argmax(-1).int()
    x = torch.where(torch.rand(40, 4, device="cuda") < 0.7, best[:, :4], torch.randint(0, 300, (40, 4), device="cuda").int())
    tok, acc = sv.verify(p, None, x.contiguous(), torch.rand(40, 5, device="cuda"))
    want = (x == best[:, :4]).int().cumprod(1).sum(1)
    assert torch.equal(acc.long(), want)
    assert torch.equal(tok[torch.arange(40), acc.long()], best[torch.arange(40), acc.long()])


def test_odd_values_count_as_zero():
    p, q, x, u = drafts(6, 3, 1000, 5)
    for a in (p, q):
        a[:, :, ::7] = math.nan
        a[:, :, 1::7] = math.inf
        a[:, :, 2::7] *= -1
    check_verify(p, q, x, u)


def test_bad_tokens_and_counts_are_reported():
    p, q, x, u = drafts(4, 3, 800, 9)
    for what in ("token", "negative", "count", "negative count"):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        y, n = x.clone(), None
        if what == "token":
            y[2, 0] = 800
        elif what == "negative":
            y[1, 0] = -1
        else:
            n = torch.tensor([3, 4 if what == "count" else -2, 0, 1], dtype=torch.int32, device="cuda")
        for d in (q, None):
            check_verify(p, d, y, u, n, status=st)
            assert int(st) == mk.MK_ERR_DEVICE_INPUT, what
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_verify(p, q, x, u, status=st)
    assert int(st) == 0


def test_random_numbers_out_of_range_are_clamped():
    p, q, x, u = drafts(4, 1, 900, 11)
    u[:, 1] = torch.tensor([1.0, -0.5, math.nan, 2.0], device="cuda")
    u[:, 0] = 2.0  # nothing stands
    tok, acc = sv.verify(p, None, x, u)
    assert (acc == 0).all() and ((tok[:, 0] >= 0) & (tok[:, 0] < 900)).all()


def test_strided_probabilities():
    p, q, x, u = drafts(5, 2, 1003, 13)
    P = torch.zeros(5, 4, 1009, device="cuda")
    Q = torch.zeros(3, 5, 1007, device="cuda")
    P[:, 1:, 3:1006] = p
    Q[:2, :, 1:1004] = q.transpose(0, 1)
    a, b = sv.verify(p, q, x, u)
    c, d = sv.verify(P[:, 1:, 3:1006], Q[:2, :, 1:1004].transpose(0, 1), x, u)
    assert torch.equal(a, c) and torch.equal(b, d)


def test_the_output_is_distributed_as_the_target():
    """20000 single drafts over 6 tokens: every frequency within five standard deviations of p."""
    N, V = 20000, 6
    g = torch.Generator(device="cuda").manual_seed(2)
    p = torch.tensor([0.05, 0.4, 0.0, 0.2, 0.3, 0.05], device="cuda")
    q = torch.tensor([0.3, 0.1, 0.2, 0.2, 0.1, 0.1], device="cuda")
    x = torch.multinomial(q.expand(N, V), 1, generator=g).int()
    u = torch.rand(N, 2, generator=g, device="cuda")
    tok, acc = sv.verify(p.expand(N, 2, V), q.expand(N, 1, V), x, u)
    f = torch.bincount(tok[:, 0].long(), minlength=V).double() / N
    sd = (p.double() * (1 - p.double()) / N).sqrt()
    assert ((f - p).abs() <= 5 * sd).all()


def test_streams_and_graphs():
    z = torch.randn(12, 5000, device="cuda")
    x = torch.randint(0, 5000, (4, 2), device="cuda", dtype=torch.int32)
    u = torch.rand(4, 3, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        p = sv.token_probs(z)
        tok, acc = sv.verify(p.view(4, 3, 5000), None, x, u)
    for _ in range(3):
        z.normal_()
        u.uniform_()
        x.copy_(z.view(4, 3, 5000)[:, :2].argmax(-1))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        a, b = sv.verify(sv.token_probs(z, stream=s).view(4, 3, 5000), None, x, u, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(a, tok) and torch.equal(b, acc)
        check_verify(p.view(4, 3, 5000), None, x, u)
