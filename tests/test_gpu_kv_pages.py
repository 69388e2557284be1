"""Cache pages on the GPU against a plain host cache: every word of the
bookkeeping and every row of the pool, after single calls and after long runs
of them."""
import numpy as np
import pytest
import torch

import decode_megakernel_interpreter_b200 as mk
from decode_megakernel_interpreter_b200 import serving as sv
from serve_ref import Pages

pytestmark = pytest.mark.gpu

INPUT, OOM = mk.MK_ERR_DEVICE_INPUT, mk.MK_ERR_OUT_OF_MEMORY


def ints(x):
    return torch.tensor(np.asarray(x).tolist(), dtype=torch.int32, device="cuda")


def setup(layers=2, pages=24, heads=2, page=8, d=16, n_seqs=8, max_pages=6, dtype=torch.int16, seed=0):
    """A pool of distinct numbers, its bookkeeping, and the same on the host."""
    g = np.random.RandomState(seed)
    shape = (layers, pages, heads, page, d)
    info = torch.iinfo(dtype)
    k, v = (g.randint(info.min, info.max, shape).astype(str(dtype).split(".")[1]) for _ in range(2))
    pool = sv.KvPool(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
    return pool, sv.KvState(n_seqs, pages, max_pages), Pages(k, v, n_seqs, max_pages)


def same(pool, st, host):
    host.check(st, pool.k.cpu().numpy(), pool.v.cpu().numpy())


def resize(pool, st, host, seqs, lens):
    sv.kv_resize(pool, st, ints(seqs), ints(lens))
    host.resize(seqs, lens)


def fork(pool, st, host, parents, children):
    sv.kv_fork(pool, st, ints(parents), ints(children))
    host.fork(parents, children)


def test_a_new_state_is_empty():
    pool, st, host = setup()
    same(pool, st, host)
    assert st.status() == 0


@pytest.mark.parametrize("page, d, dtype", [(1, 16, torch.int8), (8, 16, torch.int16), (7, 24, torch.int16),
                                            (16, 64, torch.int16), (33, 4, torch.int32)])
def test_grow_cut_free_fork(page, d, dtype):
    pool, st, host = setup(page=page, d=d, dtype=dtype)
    P = page
    resize(pool, st, host, [0, 3], [2 * P + 1, P])          # two pages and a bit; exactly one page
    same(pool, st, host)
    resize(pool, st, host, [0, 3], [3 * P, P + 1])          # to the page's end; past it
    same(pool, st, host)
    fork(pool, st, host, [0, 3, 0], [1, 2, 5])              # a full last page is shared, an unfilled one copied
    same(pool, st, host)
    fork(pool, st, host, [4], [6])                          # an empty parent
    same(pool, st, host)
    resize(pool, st, host, [0, 1], [2 * P + 1, 2 * P + 1])  # cut back into a shared page
    same(pool, st, host)
    resize(pool, st, host, [0, 1, 5], [3 * P + 2, 2 * P + 2, 3 * P])  # 0 and 1 grow in it: copies
    same(pool, st, host)
    resize(pool, st, host, [0, 1, 2, 3, 4, 5, 6, 7], [0] * 8)
    same(pool, st, host)
    assert len(host.free) == pool.n_pages and st.status() == 0


def test_the_last_holder_of_a_shared_page_keeps_it():
    pool, st, host = setup()
    resize(pool, st, host, [0], [16])
    fork(pool, st, host, [0, 0], [1, 2])
    resize(pool, st, host, [0, 1, 2], [13, 13, 13])
    resize(pool, st, host, [2, 0, 1], [14, 14, 15])         # all three grow on the one page
    same(pool, st, host)
    assert host.refs.count(1) == 3 and st.status() == 0


def test_capacity_and_whole_pool():
    pool, st, host = setup()
    resize(pool, st, host, [0, 1, 2, 3], [48] * 4)          # max_pages each: the pool is used up
    same(pool, st, host)
    assert host.free == []
    resize(pool, st, host, [4], [1])
    same(pool, st, host)
    assert st.status() == OOM and host.error == OOM
    fork(pool, st, host, [0], [5])                          # full pages need none
    same(pool, st, host)
    assert st.status() == 0


def test_entries_that_do_not_fit_are_skipped_in_order():
    pool, st, host = setup()
    resize(pool, st, host, [0, 1, 2], [48, 48, 40])          # 7 pages left
    resize(pool, st, host, [3, 4, 5, 6], [40, 24, 8, 16])    # 5, then 3 does not fit, then 1, then 2 does not fit
    same(pool, st, host)
    assert st.status() == OOM
    fork(pool, st, host, [0, 5, 5], [4, 6, 7])
    same(pool, st, host)
    # cut back into shared pages; then two grow there with one page left
    resize(pool, st, host, [0, 4, 5, 6, 7], [41, 41, 0, 0, 0])
    resize(pool, st, host, [7, 0, 4], [8 * len(host.free) - 8, 42, 42])
    same(pool, st, host)
    host.error = 0
    resize(pool, st, host, [7], [0])
    fork(pool, st, host, [0], [7])
    resize(pool, st, host, [7, 0], [41, 41])
    resize(pool, st, host, [1, 2, 3], [8, 48, 48])
    resize(pool, st, host, [4, 5, 6, 0, 7], [47, 48, 48, 43, 43])
    same(pool, st, host)


def test_bad_entries_are_skipped_and_reported():
    pool, st, host = setup()
    for seqs, lens in (([9, 0], [5, 5]), ([-1, 1], [5, 5]), ([2, 3], [-4, 5]), ([2, 4], [49, 5]), ([5, 5], [3, 9]),
                       ([6, 6, 7], [-1, 4, 4])):
        host.error = 0
        resize(pool, st, host, seqs, lens)
        same(pool, st, host)
        assert st.status() == INPUT == host.error
    for par, kid in (([0, 0], [9, 2]), ([12, 0], [2, 6]), ([0], [0]), ([0], [1]), ([0, 1], [5, 5])):
        host.error = 0
        fork(pool, st, host, par, kid)
        same(pool, st, host)
        assert st.status() == INPUT == host.error, (par, kid)


def test_a_damaged_bookkeeping_stays_inside_the_buffers():
    """Page numbers, counts and lengths out of range: reported, nothing outside
    the pool or the buffer is touched (canaries around both)."""
    guard = torch.full((3, 2, 24, 2, 8, 16), 7, dtype=torch.int16, device="cuda")
    words = mk.load().mk_kv_state_words(8, 6, 24)
    buf = torch.full((words + 128,), 7, dtype=torch.int32, device="cuda")
    for part in ("table", "free", "n_free", "refs", "len"):
        pool = sv.KvPool(guard[1], torch.zeros_like(guard[1]))
        st = sv.KvState(8, 24, 6, buffer=buf[64:64 + words])
        mk.load().mk_kv_init(st._ref, None)
        sv.kv_resize(pool, st, ints([0, 1, 2]), ints([20, 9, 48]))
        if part == "table":
            st.table[0, :3] = ints([99, -5, 1 << 30])
        elif part == "free":
            st.buffer[4 + 8 + 24:4 + 8 + 48] = 1 << 20
        elif part == "n_free":
            st.n_free.fill_(1000)
        elif part == "refs":
            st.refs.fill_(-3)
        else:
            st.lens[0] = 1 << 30
        sv.kv_fork(pool, st, ints([0, 1]), ints([3, 4]))
        sv.kv_resize(pool, st, ints([0, 1, 3]), ints([30, 0, 21]))
        sv.kv_compact(pool, st)
        torch.cuda.synchronize()
        assert (guard[0] == 7).all() and (guard[2] == 7).all(), part
        assert (buf[:64] == 7).all() and (buf[64 + words:] == 7).all(), part
        if part in ("table", "free", "refs", "len"):
            assert st.status() == INPUT, part


@pytest.mark.parametrize("seed", range(6))
def test_a_long_run_of_calls(seed):
    """Prompts, forks, steps, cuts, frees and compactions at random."""
    r = np.random.RandomState(seed)
    page = [1, 8, 16, 5, 8, 64][seed]
    pool, st, host = setup(pages=200, page=page, n_seqs=40, max_pages=12, d=8, seed=seed)
    cap = 12 * page
    for step in range(60):
        kind = r.randint(0, 10)
        if kind < 6:
            n = r.randint(1, 30)
            seqs = r.permutation(40)[:n]
            lens = [int(np.clip(host.len[s] + r.randint(-page - 2, 2 * page + 3), 0, cap)) if r.rand() < 0.9 else 0
                    for s in seqs]
            resize(pool, st, host, seqs.tolist(), lens)
        elif kind < 9:
            n = r.randint(1, 12)
            fork(pool, st, host, r.randint(0, 40, n).tolist(), r.randint(0, 40, n).tolist())
        else:
            sv.kv_compact(pool, st)
            host.compact()
        host.check(st)
    same(pool, st, host)


@pytest.mark.parametrize("n", [1, 33, 1024])
def test_lists_up_to_the_limit(n):
    pool, st, host = setup(pages=3000, n_seqs=2100, max_pages=3, layers=1, d=8)
    r = np.random.RandomState(n)
    seqs = r.permutation(2100)
    resize(pool, st, host, seqs[:n].tolist(), r.randint(0, 18, n).tolist())
    fork(pool, st, host, seqs[r.randint(0, n, n)].tolist(), seqs[n:2 * n].tolist())
    resize(pool, st, host, seqs[:n].tolist(), r.randint(0, 18, n).tolist())
    resize(pool, st, host, seqs[n:2 * n].tolist(), r.randint(0, 18, n).tolist())
    same(pool, st, host)


@pytest.mark.parametrize("pages, used", [(1, 1), (31, 0), (33, 33), (1000, 400), (200000, 150000)])
def test_compaction(pages, used):
    r = np.random.RandomState(pages)
    n_seqs = 64
    pool, st, host = setup(layers=1, pages=pages, heads=1, page=2, d=8, n_seqs=n_seqs, max_pages=max(1, -(-used // 40)))
    lens, left = [], used
    for s in range(n_seqs):
        k = min(left, host.max_pages)
        lens.append(2 * k - (k > 0 and s % 2))
        left -= k
    for i in range(0, n_seqs, 16):
        resize(pool, st, host, list(range(i, i + 16)), lens[i:i + 16])
    fork(pool, st, host, [0], [n_seqs - 1])
    gone = r.permutation(n_seqs - 1)[:20].tolist()
    resize(pool, st, host, gone, [0] * 20)
    sv.kv_compact(pool, st)
    host.compact()
    same(pool, st, host)
    before = st.buffer.clone()
    sv.kv_compact(pool, st)                                  # nothing left to move
    assert torch.equal(before, st.buffer) and st.status() == 0


# ------------------------------------------------------------------ copies

def copied(a, b, items, bad=()):
    k, v = b.k.cpu().numpy().copy(), b.v.cpu().numpy().copy()
    ak, av = a.k.cpu().numpy().copy(), a.v.cpu().numpy().copy()
    for i, (sp, sr, dp, dr, n) in enumerate(items):
        if i not in bad:
            k[:, dp, :, dr:dr + n] = ak[:, sp, :, sr:sr + n]
            v[:, dp, :, dr:dr + n] = av[:, sp, :, sr:sr + n]
    return k, v


def run_copy(a, b, items, bad=()):
    want = copied(a, b, items, bad)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.kv_copy(a, b, ints(items).reshape(-1, 5), status=status)
    assert np.array_equal(b.k.cpu().numpy(), want[0]) and np.array_equal(b.v.cpu().numpy(), want[1])
    assert int(status) == (INPUT if bad else 0)


@pytest.mark.parametrize("dtype, d", [(torch.int8, 16), (torch.int16, 64), (torch.int16, 128), (torch.int32, 20)])
def test_copies_between_pools_of_other_page_sizes(dtype, d):
    a = setup(pages=9, page=13, d=d, dtype=dtype, seed=1)[0]
    b = setup(pages=3, page=300, d=d, dtype=dtype, seed=2)[0]
    run_copy(a, b, [(0, 0, 2, 287, 13), (3, 5, 0, 1, 8), (3, 5, 1, 1, 1), (8, 0, 1, 100, 0), (7, 12, 1, 299, 1)])
    run_copy(b, a, [(2, 280, 5, 0, 13), (1, 17, 6, 3, 10)])
    run_copy(a, a, [(0, 0, 1, 0, 13), (0, 2, 2, 1, 4), (3, 0, 3, 6, 6)])


def test_a_slot_of_an_engine_cache():
    """Rows far beyond one warp's piece, and every slot from one."""
    b = setup(pages=4, page=1111, heads=3, d=64)[0]
    run_copy(b, b, [(0, 0, 1, 0, 1111), (0, 0, 2, 0, 1000), (0, 7, 3, 100, 1)])


def test_copies_that_would_collide_are_skipped():
    a = setup(pages=6, page=16)[0]
    b = setup(pages=6, page=16, seed=3)[0]
    run_copy(a, b, [(0, 0, 1, 0, 8), (1, 0, 1, 7, 4), (2, 0, 1, 8, 4)], bad=(1, 2))  # 1 meets 0, 2 meets 1
    run_copy(a, b, [(0, 0, 1, 0, 8)] * 3, bad=(1, 2))                                     # the same entry thrice
    run_copy(a, a, [(0, 0, 1, 0, 8), (1, 4, 2, 0, 4), (3, 0, 4, 0, 16)], bad=(0,))         # writes what entry 1 reads
    run_copy(a, a, [(0, 0, 0, 4, 8)], bad=(0,))                                            # onto itself
    run_copy(a, a, [(0, 0, 0, 8, 8), (5, 0, 5, 0, 0)])


def test_copies_out_of_range_are_skipped():
    a = setup(pages=6, page=16)[0]
    b = setup(pages=5, page=12, seed=3)[0]
    big = 2 ** 31 - 1
    for bad in ((6, 0, 0, 0, 1), (-1, 0, 0, 0, 1), (0, 0, 5, 0, 1), (0, 0, -9, 0, 1), (0, 10, 0, 0, 7), (0, 0, 0, 6, 7),
                (0, -1, 0, 0, 1), (0, 0, 0, -1, 1), (0, 0, 0, 0, -1), (0, 0, 0, 0, 13), (0, big, 0, 0, big),
                (0, 0, 0, 1, big), (0, 0, 0, big, 1)):
        run_copy(a, b, [bad, (1, 2, 3, 4, 5)], bad=(0,))


def test_a_long_list_of_copies():
    a = setup(layers=1, pages=5000, heads=1, page=4, d=8)[0]
    b = setup(layers=1, pages=5000, heads=1, page=4, d=8, seed=5)[0]
    r = np.random.RandomState(0)
    items = np.stack([r.randint(0, 5000, 16384), r.randint(0, 2, 16384), np.arange(16384) % 5000,
                      np.arange(16384) // 5000, r.randint(0, 2, 16384)], 1)
    run_copy(a, b, items.tolist())


def test_offsets_past_32_bits():
    """A pool of 9 GB per tensor: pages whose byte and element offsets need 64 bits."""
    k = torch.empty((2, 36000, 8, 64, 128), dtype=torch.int16, device="cuda")[:, :, :, :, :]
    pool = sv.KvPool(k, torch.empty((2, 36000, 8, 64, 128), dtype=torch.int16, device="cuda"))
    for x in (pool.k, pool.v):
        x[:, 7].random_()
        x[:, 35999].zero_()
    sv.kv_copy(pool, pool, ints([(7, 3, 35999, 1, 60)]))
    for x in (pool.k, pool.v):
        assert torch.equal(x[:, 35999, :, 1:61], x[:, 7, :, 3:63])
        assert (x[:, 35999, :, 0] == 0).all() and (x[:, 35999, :, 61:] == 0).all()


# ------------------------------------------------------------------ streams and graphs

def test_another_stream_and_a_captured_step():
    """Growth by one token as a graph, replayed while the list changes."""
    pool, st, host = setup()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sv.kv_resize(pool, st, ints([0, 1]), ints([9, 3]), stream=s)
    host.resize([0, 1], [9, 3])
    s.synchronize()
    host.check(st)
    sv.kv_fork(pool, st, ints([0]), ints([2]))
    host.fork([0], [2])
    seqs, lens = ints([0, 1, 2]), ints([10, 4, 10])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    before = st.buffer.clone(), pool.k.clone(), pool.v.clone()
    with torch.cuda.graph(g):
        sv.kv_resize(pool, st, seqs, lens)
    assert torch.equal(before[0], st.buffer)                 # captured, not run
    for step in range(9):
        g.replay()
        host.resize([0, 1, 2], lens.tolist())
        lens += 1
    torch.cuda.synchronize()
    same(pool, st, host)


def test_two_pools_on_two_streams():
    runs = [setup(seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for step in range(20):
        for i, ((pool, st, host), s) in enumerate(zip(runs, streams)):
            seqs, lens = [0, 1], [(step * (i + 1)) % 40, (step * 3) % 30]
            with torch.cuda.stream(s):
                sv.kv_resize(pool, st, ints(seqs), ints(lens))
            host.resize(seqs, lens)
    torch.cuda.synchronize()
    for run in runs:
        same(*run)
