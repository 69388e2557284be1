"""Shared-prefix attention on the GPU against sums over single positions in 64
bits, within the bounds that serve_ref.attention derives."""
import math

import pytest
import torch

import decode_megakernel_interpreter_b200 as mk
from decode_megakernel_interpreter_b200 import serving as sv
from serve_ref import attention, check_attention

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def case(B, T, nq, nkv, d, page, prefix, lens, dtype=BF16, seed=0, width=None):
    """Inputs of one call: pages in random order, the prefix's own ones first in the list."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = torch.Generator().manual_seed(seed)
    need = [max(0, -(-max(n, 0) // page) - prefix // page) for n in lens]
    n_pre = -(-prefix // page)
    P = n_pre + sum(need) + 1
    order = torch.randperm(P, generator=r)
    width = width or max(1, max([-(-max(n, 0) // page) for n in lens] + [1]))
    table = torch.full((B, width), 1 << 30, dtype=torch.int32)  # what is not read may hold anything
    at = n_pre
    for b in range(B):
        table[b, prefix // page:prefix // page + need[b]] = order[at:at + need[b]]
        at += need[b]
    q = torch.randn((B, T, nq, d), generator=g, device="cuda").to(dtype)
    k = (1.5 * torch.randn((P, nkv, page, d), generator=g, device="cuda")).to(dtype)
    v = torch.randn((P, nkv, page, d), generator=g, device="cuda").to(dtype)
    return dict(q=q, k=k, v=v, table=table.cuda(), lens=ints(lens),
                prefix_pages=order[:n_pre].int().cuda() if n_pre else None, prefix_len=ints([prefix]) if n_pre else None)


def run(c, scale=None, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sv.shared_attention(**c, scale=scale, return_lse=True, status=status, **kw)
    return got, int(status)


def check(c, what="", scale=None):
    got, status = run(c, scale)
    assert status == 0
    check_attention(got, attention(**c, scale=scale), what)


def roomy(c, room=1100):
    """The same call with a page list that has room for a long prefix: what lies behind the prefix is not read."""
    n = -(-room // c["k"].shape[2])
    old = c["prefix_pages"]
    c["prefix_pages"] = torch.full((n,), 1 << 30, dtype=torch.int32, device="cuda")
    if old is None:
        c["prefix_len"] = ints([0])
    else:
        c["prefix_pages"][:len(old)] = old
    return c


HEADS = [(4, 2, 64), (8, 8, 64), (6, 2, 64), (8, 1, 128), (16, 1, 64), (4, 1, 128), (3, 3, 128)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("nq, nkv, d", HEADS)
def test_heads_and_types(nq, nkv, d, dtype):
    check(case(3, 1, nq, nkv, d, 16, 100, [131, 100, 170], dtype))


@pytest.mark.parametrize("prefix", [0, 1, 15, 63, 64, 65, 127, 128, 129, 255, 256, 257, 640])
def test_prefix_lengths(prefix):
    check(case(5, 1, 4, 2, 64, 16, prefix, [prefix + n for n in (1, 0, 63, 64, 65)]))


@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 100, 128, 1000])
def test_page_sizes(page):
    check(case(4, 1, 4, 2, 128, page, 130, [131, 200, 131 + 64, 259]))


@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 16])
@pytest.mark.parametrize("nq, nkv", [(2, 2), (8, 2), (16, 1)])
def test_drafted_tokens(T, nq, nkv):
    check(case(3, T, nq, nkv, 64, 16, 70, [70 + T, 70 + T + 61, 200], F16))


@pytest.mark.parametrize("B", [1, 2, 17, 64, 130])
def test_batches(B):
    lens = [40 + (7 * b) % 90 for b in range(B)]
    check(case(B, 1, 4, 2, 64, 16, 40, lens))


def test_one_long_and_many_short():
    check(case(20, 1, 2, 1, 128, 64, 3, [3 + 2000 if b == 7 else 4 for b in range(20)]))


def test_long_prefix():
    check(case(9, 2, 8, 2, 128, 64, 4001, [4003 + 5 * b for b in range(9)]))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B, T, nq, nkv, d, page, prefix", [
    (16, 1, 32, 8, 64, 64, 16000), (16, 1, 32, 8, 64, 50, 11000), (64, 1, 32, 8, 64, 16, 20011), (16, 1, 32, 8, 128, 64, 9001),
    (64, 1, 32, 8, 128, 96, 16000), (5, 8, 8, 2, 128, 32, 70001), (3, 1, 4, 4, 64, 64, 150000), (200, 1, 4, 1, 64, 64, 40000)])
def test_many_tiles_per_block(B, T, nq, nkv, d, page, prefix, dtype):
    """Prefixes of which a block takes many more tiles than it holds at a time, against 64-bit products: a row's error
    within the bound that the shorter cases derive, with the 2-norms of p v and v in the place of single elements."""
    c = case(B, T, nq, nkv, d, page, prefix, [prefix + T + 3 * (b % 9) for b in range(B)], dtype)
    h = torch.finfo(dtype).eps / 2
    for _ in range(3):  # (a race would not fail every time)
        (out, lse), status = run(c)
        assert status == 0
        for b in (0, B // 2, B - 1):
            n = int(c["lens"][b])
            at = torch.arange(n, device="cuda")
            pages = torch.where(at < prefix, c["prefix_pages"][at.clamp(max=prefix - 1) // page].long(), c["table"][b, at // page].long())
            K, V = (c[x][pages, :, at % page].double().transpose(0, 1) for x in ("k", "v"))
            for t in (0, T - 1):
                m = n - (T - 1 - t)
                q = c["q"][b, t].double().view(nkv, nq // nkv, d)
                s = torch.einsum("hgd,hnd->hgn", q, K[:, :m]) / math.sqrt(d)
                p = s.softmax(-1)
                o = torch.einsum("hgn,hnd->hgd", p, V[:, :m])
                spread = torch.einsum("hgn,hnd->hgd", p * p, V[:, :m] ** 2).sum(-1).sqrt()  # of independent roundings of p
                err = (out[b, t].double().view_as(o) - o).norm(dim=-1)
                assert (err <= h * (o.norm(dim=-1) + 4 * spread) + 1e-4 * o.norm(dim=-1)).all(), (b, t, float(err.max()))
                z = torch.logsumexp(s, -1)
                assert ((lse[b, t].double().view_as(z) - z).abs() <= 1e-4).all()


def test_only_a_prefix_and_only_own():
    check(case(3, 1, 4, 2, 64, 16, 77, [77, 77, 77]))
    check(case(3, 1, 4, 2, 64, 16, 0, [1, 64, 77]))


def test_sequences_shorter_than_the_prefix():
    """They see only their own length of it; one sees nothing."""
    check(case(6, 1, 4, 2, 64, 16, 200, [200, 199, 64, 1, 0, 230]))
    check(case(4, 4, 4, 2, 64, 16, 200, [201, 2, 0, 130]))
    check(case(40, 4, 4, 1, 64, 16, 300, [[301, 2, 0, 130][b % 4] for b in range(40)]))


def test_queries_that_see_nothing_give_zeros():
    c = case(2, 3, 4, 2, 64, 16, 0, [0, 1])
    (out, lse), status = run(c)
    assert status == 0
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    assert (out[1, :2] == 0).all() and (lse[1, :2] == -math.inf).all()
    assert torch.isfinite(lse[1, 2]).all()
    check(c)


@pytest.mark.parametrize("prefix", [0, 100])
def test_unused_rows_are_left_as_they_are(prefix):
    c = case(5, 2, 4, 2, 64, 16, prefix, [prefix + 9, -1, prefix + 70, -(2 ** 31), prefix + 2])
    out = torch.full_like(c["q"], 5.0)
    lse = torch.full((5, 2, 4), 5.0, device="cuda")
    got, status = run(c, out=out, lse=lse)
    assert status == 0
    for b in (1, 3):
        assert (out[b] == 5).all() and (lse[b] == 5).all()
    check_attention(got, attention(**c))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("T, B, nq", [(3, 2, 4), (4, 40, 8), (1, 3, 4)])
def test_masked_positions_have_no_influence(bad, T, B, nq):
    """Infinities, NaN and the type's extremes in every position that no query sees, and in those that only later
    queries see."""
    prefix, lens = 90, [95 + 13 * (b % 7) if b % 5 else 41 for b in range(B)]
    c = case(B, T, nq, 2, 64, 16, prefix, lens)
    want = attention(**c)
    used = torch.zeros(c["k"].shape[0], 16, dtype=torch.bool)
    for j in range(prefix):
        used[c["prefix_pages"][j // 16], j % 16] = True
    for b, n in enumerate(lens):
        for j in range(prefix, n):
            used[c["table"][b, j // 16], j % 16] = True
    hole = (~used).cuda()[:, None, :, None]
    for x in ("k", "v"):
        c[x].masked_fill_(hole, bad)
    got, status = run(c)
    assert status == 0
    check_attention(got, want, "unseen rows")
    if T > 1:  # the last position of a sequence, which only its last query sees
        b = 1
        j = lens[b] - 1
        c["v"][c["table"][b, j // 16], :, j % 16] = bad
        c["k"][c["table"][b, j // 16], :, j % 16] = bad
        got, _ = run(c)
        keep = torch.ones(B, T, dtype=torch.bool)
        keep[b, T - 1] = False
        w = [x.clone() for x in want]
        w[1][~keep] = math.nan  # that query itself is not held to anything
        check_attention(got, w, "a position that only the last query sees")
    else:  # rows of the prefix behind a shorter sequence
        c["v"][c["prefix_pages"][60 // 16], :, 60 % 16] = bad
        got, _ = run(c)
        w = [x.clone() for x in want]
        w[1][[b for b in range(B) if lens[b] > 60]] = math.nan
        check_attention(got, w, "a prefix row behind a shorter sequence")


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 1e-30])
def test_scales(scale):
    check(case(3, 2, 4, 2, 64, 16, 50, [60, 52, 120]), scale=scale)


def test_large_scores():
    """Scores in the hundreds: all weight on few positions."""
    c = case(3, 1, 4, 2, 64, 16, 150, [151, 200, 260])
    c["q"] *= 20
    check(c)


def test_strided_tensors():
    """q and out inside larger tensors, K/V as one layer of a pool whose rows are wider."""
    c = case(3, 2, 4, 2, 64, 16, 50, [60, 52, 120])
    big_q = torch.randn(3, 2, 4, 3, 64, device="cuda").to(BF16)
    big_q[:, :, :, 1] = c["q"]
    big_o = torch.full((2, 3, 6, 64), 9.0, device="cuda", dtype=BF16)
    wide = torch.randn(2, 2, *c["k"].shape[:3], 72, device="cuda").to(BF16)
    wide[1, 0, ..., :64], wide[1, 1, ..., :64] = c["k"], c["v"]
    want = attention(**c)
    c["q"], c["k"], c["v"] = big_q[:, :, :, 1], wide[1, 0, ..., :64], wide[1, 1, ..., :64]
    out = big_o.transpose(0, 1)[:, :, 1:5]
    got, status = run(c, out=out)
    assert status == 0 and got[0].data_ptr() == out.data_ptr()
    check_attention(got, want)
    assert (big_o[:, :, 0] == 9).all() and (big_o[:, :, 5] == 9).all()


def test_dimensions_of_size_one_with_odd_strides():
    c = case(1, 1, 4, 1, 64, 16, 50, [60])
    want = attention(**c)
    c["q"] = torch.as_strided(c["q"], c["q"].shape, (3, 5, 64, 1))
    for x in ("k", "v"):
        c[x] = torch.as_strided(c[x], c[x].shape, (c[x].stride(0), 7, 64, 1))
    got, status = run(c)
    assert status == 0
    check_attention(got, want)


def test_misaligned_tensors_are_refused():
    c = case(2, 1, 4, 2, 64, 16, 50, [60, 52])
    c["q"] = torch.zeros(2 * 4 * 64 + 4, device="cuda", dtype=BF16)[4:].view(2, 1, 4, 64)
    with pytest.raises(mk.MkError):
        run(c)


def test_bad_pages_and_lengths_are_reported():
    base = case(3, 1, 4, 2, 64, 16, 40, [50, 45, 90])
    for what in ("table", "prefix", "lens", "prefix_len", "negative prefix"):
        c = {k: v.clone() for k, v in base.items()}
        if what == "table":
            c["table"][0, 3] = c["k"].shape[0]
        elif what == "prefix":
            c["prefix_pages"][1] = -1
        elif what == "lens":
            c["lens"][1] = 2 ** 31 - 1
        elif what == "prefix_len":
            c["prefix_len"][0] = 49
        else:
            c["prefix_len"][0] = -3
        if what in ("lens", "prefix_len", "negative prefix"):  # every page of the lists is then read
            c["table"].clamp_(max=c["k"].shape[0] - 1)
        got, status = run(c)
        assert status == mk.MK_ERR_DEVICE_INPUT, what
        if what == "table":  # the others are right
            w = list(attention(**base))
            w[1] = w[1].clone()
            w[1][0] = math.nan
            check_attention(got, w)
    # a bad page is read as page 0, a length cut to the pages there are
    c = {k: v.clone() for k, v in base.items()}
    c["table"].clamp_(max=c["k"].shape[0] - 1)
    c["lens"][1] = 2 ** 31 - 1
    got, _ = run(c)
    c["lens"][1] = c["table"].shape[1] * 16
    check_attention(got, attention(**c))


def test_offsets_past_32_bits():
    c = case(3, 1, 4, 2, 128, 64, 130, [200, 131, 333])
    n = c["k"].shape[0]
    big = [torch.empty((300000, 2, 64, 128), dtype=BF16, device="cuda") for _ in range(2)]
    want = attention(**c)
    for x, y in zip(big, (c["k"], c["v"])):
        x[-n:] = y
    c["k"], c["v"] = big
    c["table"] = torch.where(c["table"] < n, c["table"] + 300000 - n, c["table"])
    c["prefix_pages"] += 300000 - n
    got, status = run(c)
    assert status == 0
    check_attention(got, want)


def test_engine_cache_layout():
    """A layer of an engine's cache: slots as pages, the prefix in one slot, own rows behind it in the others."""
    L, B, nkv, S, d, prefix = 2, 4, 2, 150, 64, 90
    kc, vc = (torch.randn(L, B, nkv, S, d, device="cuda").to(BF16) for _ in range(2))
    c = dict(q=torch.randn(3, 1, 4, d, device="cuda").to(BF16), k=kc[1], v=vc[1], table=ints([[0], [1], [3]]),
             lens=ints([91, 150, 120]), prefix_pages=ints([2]), prefix_len=ints([prefix]))
    check(c)


def test_the_same_call_gives_the_same_bits():
    c = case(9, 2, 8, 2, 64, 16, 700, [710 + 30 * b for b in range(9)])
    a = run(c)[0]
    for _ in range(3):
        b = run(c)[0]
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_streams_and_replayed_graphs():
    """A captured step replayed with other lengths, next to a second graph and eager calls on other streams."""
    cs = [case(4, 1, 4, 2, 64, 16, 60, [62, 70, 100, 61], seed=s, width=12) for s in range(2)]
    for c in cs:
        c["table"] = torch.randint(0, c["k"].shape[0], (4, 12), device="cuda", dtype=torch.int32)
    wants = []
    graphs, outs = [], []
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(sv.shared_attention(**c, return_lse=True))
            graphs.append(g)
    torch.cuda.synchronize()
    for step in range(3):
        for c in cs:
            c["lens"].copy_(ints([61 + 40 * step, 60, 180 - step, 100]))
        torch.cuda.synchronize()
        for _ in range(5):  # overlapping replays
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        eager = [sv.shared_attention(**c, return_lse=True, stream=torch.cuda.Stream()) for c in cs]
        torch.cuda.synchronize()
        for c, o, e in zip(cs, outs, eager):
            want = attention(**c)
            check_attention(o, want, "graph")
            check_attention(e, want, "stream")


# A page list with room for a long prefix is taken by other code, whatever the prefix's length.


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("nq, nkv, d", HEADS)
def test_room_heads_and_types(nq, nkv, d, dtype):
    check(roomy(case(3, 1, nq, nkv, d, 16, 100, [131, 100, 170], dtype)))


@pytest.mark.parametrize("B", [1, 5, 150])
@pytest.mark.parametrize("prefix", [0, 1, 15, 63, 64, 65, 127, 128, 129, 255, 257, 640, 1056])
def test_room_prefix_lengths(prefix, B):
    check(roomy(case(B, 1, 4, 2, 64, 16, prefix, [prefix + (1, 0, 63, 64, 65)[b % 5] for b in range(B)])))


@pytest.mark.parametrize("page", [1, 3, 16, 32, 48, 64, 96, 100, 128, 1000])
@pytest.mark.parametrize("prefix", [130, 1034])
def test_room_page_sizes(page, prefix):
    """Page sizes that are multiples of 16, 32 and 64 positions and that are not."""
    check(roomy(case(4, 1, 4, 2, 128, page, prefix, [prefix + n for n in (1, 70, 65, 129)])))


@pytest.mark.parametrize("B, T, nq", [(3, 1, 2), (3, 5, 8), (3, 16, 16), (1, 16, 16), (17, 8, 16), (130, 1, 4), (300, 2, 2)])
def test_room_rows(B, T, nq):
    """Rows that fill part of a group, one of its halves, both, and several groups."""
    check(roomy(case(B, T, nq, 1, 64, 16, 70, [70 + T + 7 * b % 90 for b in range(B)], F16)))


def test_room_sequences_shorter_than_the_prefix():
    check(roomy(case(6, 1, 4, 2, 64, 16, 200, [200, 199, 64, 1, 0, 230])))
    check(roomy(case(4, 4, 4, 2, 64, 16, 200, [201, 2, 0, 130])))
    check(roomy(case(100, 4, 4, 1, 64, 16, 300, [[301, 2, 0, 130][b % 4] for b in range(100)])))


def test_room_unused_rows_are_left_as_they_are():
    c = roomy(case(5, 2, 4, 2, 64, 16, 100, [109, -1, 170, -(2 ** 31), 102]))
    out = torch.full_like(c["q"], 5.0)
    lse = torch.full((5, 2, 4), 5.0, device="cuda")
    got, status = run(c, out=out, lse=lse)
    assert status == 0
    for b in (1, 3):
        assert (out[b] == 5).all() and (lse[b] == 5).all()
    check_attention(got, attention(**c))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("B, page", [(3, 16), (40, 16), (40, 24)])
def test_room_masked_positions_have_no_influence(bad, B, page):
    prefix, lens = 90, [95 + 13 * (b % 7) if b % 5 else 41 for b in range(B)]
    c = roomy(case(B, 1, 4, 2, 64, page, prefix, lens))
    want = attention(**c)
    used = torch.zeros(c["k"].shape[0], page, dtype=torch.bool)
    for j in range(prefix):
        used[c["prefix_pages"][j // page], j % page] = True
    for b, n in enumerate(lens):
        for j in range(prefix, n):
            used[c["table"][b, j // page], j % page] = True
    hole = (~used).cuda()[:, None, :, None]
    for x in ("k", "v"):
        c[x].masked_fill_(hole, bad)
    got, status = run(c)
    assert status == 0
    check_attention(got, want, "unseen rows")


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 1e-30])
def test_room_scales(scale):
    check(roomy(case(3, 2, 4, 2, 64, 16, 50, [60, 52, 120])), scale=scale)


def test_room_bad_pages_and_lengths_are_reported():
    base = roomy(case(3, 1, 4, 2, 64, 16, 40, [50, 45, 90]), 1040)
    for page in (-1, base["k"].shape[0]):
        for at in (0, 1, 2):  # a tile that is full and one that is not: in page lists of whole tiles all are read
            c = {k: v.clone() for k, v in base.items()}
            c["prefix_pages"][at] = page
            assert run(c)[1] == mk.MK_ERR_DEVICE_INPUT
    for n in (-3, 1041, 2 ** 31 - 1):
        c = {k: v.clone() for k, v in base.items()}
        c["prefix_pages"].clamp_(max=c["k"].shape[0] - 1)
        c["prefix_len"][0] = n
        assert run(c)[1] == mk.MK_ERR_DEVICE_INPUT
    c = {k: v.clone() for k, v in base.items()}
    c["prefix_pages"].clamp_(max=c["k"].shape[0] - 1)
    c["prefix_pages"][20] = -1
    c["prefix_len"][0] = 640
    assert run(c)[1] == mk.MK_ERR_DEVICE_INPUT


def test_room_strided_and_past_32_bits():
    c = roomy(case(30, 1, 8, 2, 128, 64, 130, [200, 131, 333] * 10))
    n = c["k"].shape[0]
    want = attention(**c)
    big = [torch.empty((300000, 2, 64, 128), dtype=BF16, device="cuda") for _ in range(2)]
    for x, y in zip(big, (c["k"], c["v"])):
        x[-n:] = y
    c["k"], c["v"] = big
    c["table"] = torch.where(c["table"] < n, c["table"] + 300000 - n, c["table"])
    c["prefix_pages"][:3] += 300000 - n
    got, status = run(c)
    assert status == 0
    check_attention(got, want)
    del big
    c = roomy(case(3, 2, 4, 2, 64, 16, 100, [131, 102, 170]))
    want = attention(**c)
    for x in ("k", "v"):  # [page][position][head] with room between rows
        y = torch.empty((c[x].shape[0], 16, 3, 80), dtype=BF16, device="cuda")
        y[:, :, :2, :64] = c[x].transpose(1, 2)
        c[x] = y[:, :, :2, :64].transpose(1, 2)
    got, status = run(c)
    assert status == 0
    check_attention(got, want)


def test_room_captured_steps():
    """A captured step replayed with prefixes and lengths of every kind."""
    c = roomy(case(20, 1, 4, 2, 64, 16, 640, [660 + b for b in range(20)], width=48))
    c["table"] = torch.randint(0, c["k"].shape[0], (20, 48), device="cuda", dtype=torch.int32)
    g = torch.cuda.CUDAGraph()
    run(c)
    with torch.cuda.graph(g):
        out = sv.shared_attention(**c, return_lse=True)
    for prefix in (640, 0, 1, 64, 500, 639):
        c["prefix_len"].fill_(prefix)
        c["lens"].copy_(ints([prefix + 3 * b for b in range(20)]))
        g.replay()
        torch.cuda.synchronize()
        check_attention(out, attention(**c), prefix)
