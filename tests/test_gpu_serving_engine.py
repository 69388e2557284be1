"""The serving operators in an engine's own paths: a prompt prefilled once and
forked, drafted tokens checked, and decode steps over a shared prefix."""
import dataclasses

import numpy as np
import pytest
import torch

import decode_megakernel_interpreter_b200 as mk
from decode_megakernel_interpreter_b200 import harness
from decode_megakernel_interpreter_b200 import serving as sv
import synth
from gpu_common import HostSetup
from serve_ref import probs, verify

pytestmark = pytest.mark.gpu

SMALL_1B = dataclasses.replace(synth.LLAMA_1B, n_layers=2)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def engine(shape, batch, max_seq, planned=None):
    hs = HostSetup(shape, batch, max_seq)
    dev = harness.upload_model(hs.model, shape.tied)
    kc, vc = harness.upload_kv(hs.k, hs.v)
    eng = harness.make_engine(shape, dev, kc, vc, batch, max_seq)
    eng.plan(batch=planned or batch)
    return hs, eng, kc, vc


def test_fork_copies_a_prompt_to_other_sequences():
    hs, eng, kc, vc = engine(synth.TINY, 4, 80, planned=1)
    try:
        kc.normal_()
        vc.normal_()
        want = [x.clone() for x in (kc, vc)]
        for w in want:
            w[:, [0, 3], :, :41] = w[:, 2:3, :, :41]
        eng.fork(2, [0, 3], 41)
        torch.cuda.synchronize()
        assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
        for bad in (([], 4), ([2], 4), ([1, 1], 4), ([4], 4), ([1], 81), ([1], -1)):
            with pytest.raises(ValueError):
                eng.fork(2, *bad)
    finally:
        eng.close()




@pytest.mark.parametrize("shape, batch", [(synth.TINY, 1), (SMALL_1B, 16)], ids=["tiny one launch a token", "1B chunk"])
def test_speculate_keeps_what_the_engine_would_have_decoded(shape, batch):
    """Greedy: decode some tokens step by step, then offer them as drafts, whole, with a wrong one, and none."""
    ctx, seq = 24, batch - 1
    hs, eng, kc, vc = engine(shape, batch, 96)
    try:
        prompt = torch.randint(0, shape.vocab, (ctx,), dtype=torch.int32, device="cuda")
        nxt = ints([0])
        eng.prefill(seq, prompt, 0, None, nxt)
        first = int(nxt)
        kv = kc.clone(), vc.clone()
        ids, rows, tok = [], [], first
        for i in range(6):  # one token at a time
            logits = torch.empty(shape.vocab, device="cuda")
            eng.prefill(seq, ints([tok]), ctx + i, logits, nxt)
            tok = int(nxt)
            ids.append(tok)
            rows.append(logits.double().cpu().numpy())
        assert eng.status() == mk.MK_OK
        greedy = torch.zeros(1, device="cuda")
        for drafts in (ids[:5], [ids[0], ids[1], (ids[2] + 1) % shape.vocab, ids[3]], [(ids[0] + 1) % shape.vocab], []):
            kc.copy_(kv[0])
            vc.copy_(kv[1])
            n = 1 + len(drafts)
            out, acc = ints([-7] * n), ints([-7])
            eng.speculate(seq, ints([first] + drafts), ctx, torch.rand(n, device="cuda"), out, acc, temperature=greedy)
            assert eng.status() == mk.MK_OK
            a = 0
            while a < len(drafts) and drafts[a] == ids[a]:
                a += 1
            assert int(acc) == a and out.tolist() == ids[:a + 1] + [-1] * (n - a - 1)
        # with a temperature: what the rows' logits give
        g = torch.Generator(device="cuda").manual_seed(3)
        for trial in range(4):
            kc.copy_(kv[0])
            vc.copy_(kv[1])
            drafts, n = ids[:4], 5
            u = torch.rand(n, generator=g, device="cuda") * 0.3
            out, acc = ints([-7] * n), ints([-7])
            eng.speculate(seq, ints([first] + drafts), ctx, u, out, acc, temperature=torch.tensor([0.7], device="cuda"))
            p = np.stack([probs(r, np.float32(0.7)) for r in rows[:n]])
            a, new = verify(p, None, drafts, n - 1, u.cpu().numpy())
            margin = min(abs(float(u[j]) - p[j][drafts[j]]) for j in range(n - 1))
            if margin > 1e-3:
                assert int(acc) == a
                assert out.tolist()[:a] == drafts[:a] and out.tolist()[a + 1:] == [-1] * (n - a - 1)
    finally:
        eng.close()


def test_speculate_refuses_bad_calls():
    hs, eng, kc, vc = engine(synth.TINY, 1, 40)
    L = mk.load()
    try:
        t, u, o, a = ints([1] * 16), torch.rand(16, device="cuda"), ints([0] * 16), ints([0])
        call = lambda *x: L.mk_speculate(eng.h, *x)  # noqa: E731
        T, U, O, A = t.data_ptr(), u.data_ptr(), o.data_ptr(), a.data_ptr()
        for bad in ((0, None, 2, 0, None, None, U, O, A, None), (0, T, 0, 0, None, None, U, O, A, None),
                    (0, T, 17, 0, None, None, U, O, A, None), (1, T, 2, 0, None, None, U, O, A, None),
                    (0, T, 2, 39, None, None, U, O, A, None), (0, T, 2, -1, None, None, U, O, A, None),
                    (0, T, 2, 0, None, None, None, O, A, None), (0, T, 2, 0, None, None, U, None, A, None),
                    (0, T, 2, 0, None, None, U, O, None, None)):
            assert call(*bad) == mk.MK_ERR_INVALID_ARG, bad
        with pytest.raises(ValueError):
            eng.speculate(0, t, 0, u[:3], o, a)
        eng.plan(batch=1, exec_mode="per_op")
        assert call(0, T, 2, 0, None, None, U, O, A, None) == mk.MK_ERR_INVALID_ARG
    finally:
        eng.close()


def shared_setup(shape, batch, prefix, max_seq, seed=0):
    """Two engines on one set of weights: `one` decodes sequences that each hold the whole prefix, `two` sequences that
    hold only their own rows, with the prefix in sequence `batch - 1`."""
    hs = HostSetup(shape, batch, max_seq)
    hs.fill_prefix(np.full(batch, prefix + 40))
    dev = harness.upload_model(hs.model, shape.tied)
    kc, vc = harness.upload_kv(hs.k, hs.v)
    for x in (kc, vc):
        x[:, :, :, :prefix] = x[:, batch - 1:, :, :prefix]
    kc2, vc2 = kc.clone(), vc.clone()
    for x in (kc2, vc2):
        x[:, :batch - 1, :, :prefix] = float("nan")  # nothing may read these
    one = harness.make_engine(shape, dev, kc, vc, batch, max_seq)
    two = harness.make_engine(shape, dev, kc2, vc2, batch, max_seq)
    return hs, one, two


@pytest.mark.parametrize("shape, batch, prefix", [(synth.TINY, 1, 70), (SMALL_1B, 16, 300), (SMALL_1B, 16, 0),
                                                  (SMALL_1B, 5, 129), (synth.TINY, 1, 1100), (SMALL_1B, 16, 1300),
                                                  (SMALL_1B, 5, 2049)],
                         ids=["tiny", "1B", "1B without a prefix", "1B batch 5", "tiny long", "1B long", "1B batch 5 long"])
def test_decode_over_a_shared_prefix(shape, batch, prefix):
    """Logits of shared steps against those of ordinary steps on caches that hold the prefix for every sequence; steps
    of both kinds in turn."""
    max_seq = prefix + 64
    hs, one, two = shared_setup(shape, batch, prefix, max_seq)
    try:
        one.plan(batch=batch, exec_mode="per_op")
        two.plan(batch=batch, exec_mode="per_op")
        r = np.random.RandomState(1)
        pos = [prefix + int(x) for x in r.randint(0, 30, batch)]
        toks = [int(x) for x in r.randint(0, shape.vocab, batch)]
        la, lb = (torch.empty(batch, shape.vocab, device="cuda") for _ in range(2))
        na, nb = ints([0] * batch), ints([0] * batch)
        for step in range(7):
            t, p = ints(toks), ints(pos)
            one.decode_step(t, p, la, na)
            two.decode_step_shared(t, p, batch - 1, prefix, lb, nb)
            assert one.status() == mk.MK_OK and two.status() == mk.MK_OK
            a, b = la.double(), lb.double()
            # the engine's own tolerance against the oracle
            assert ((a - b).abs() <= 2e-2 + 1e-2 * a.abs()).all(), (step, float((a - b).abs().max()))
            assert torch.equal(nb.long(), lb.argmax(-1))
            toks, pos = na.tolist(), [x + 1 for x in pos]
    finally:
        one.close()
        two.close()


def test_steps_of_both_kinds_in_turn():
    """An ordinary step after shared ones starts from what ordinary steps leave behind."""
    shape, batch, prefix = SMALL_1B, 16, 100
    hs, one, two = shared_setup(shape, batch, prefix, prefix + 64)
    try:
        two._keep[1].copy_(one._keep[1])  # here the sequences do hold the prefix
        two._keep[2].copy_(one._keep[2])
        one.plan(batch=batch, exec_mode="per_op")
        two.plan(batch=batch, exec_mode="per_op")
        la, lb = (torch.empty(batch, shape.vocab, device="cuda") for _ in range(2))
        na, nb = ints([0] * batch), ints([0] * batch)
        toks, pos = list(range(batch)), [prefix + b for b in range(batch)]
        for step, kind in enumerate("o s o s s s s o o s o".split()):
            t, p = ints(toks), ints(pos)
            one.decode_step(t, p, la, na)
            if kind == "s":
                two.decode_step_shared(t, p, 3, prefix, lb, nb)
            else:
                two.decode_step(t, p, lb, nb)
            assert one.status() == mk.MK_OK and two.status() == mk.MK_OK, (step, kind)
            a, b = la.double(), lb.double()
            assert ((a - b).abs() <= 2e-2 + 1e-2 * a.abs()).all(), (step, kind)
            toks, pos = na.tolist(), [x + 1 for x in pos]
    finally:
        one.close()
        two.close()


def test_captured_steps_of_both_kinds():
    """Graphs of an ordinary and of a shared step, replayed in turn, against eager ordinary steps."""
    shape, batch, prefix = SMALL_1B, 16, 100
    hs, one, two = shared_setup(shape, batch, prefix, prefix + 64)
    try:
        two._keep[1].copy_(one._keep[1])
        two._keep[2].copy_(one._keep[2])
        one.plan(batch=batch, exec_mode="per_op")
        two.plan(batch=batch, exec_mode="per_op")
        la, lb = (torch.empty(batch, shape.vocab, device="cuda") for _ in range(2))
        na, nb = ints([0] * batch), ints([0] * batch)
        t, p = ints(list(range(batch))), ints([prefix + b for b in range(batch)])
        two.decode_step_shared(t, p, 3, prefix, lb, nb)   # (allocates its scratch)
        one.decode_step(t, p, la, na)
        assert two.status() == mk.MK_OK
        graphs = {}
        for kind in "os":
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                if kind == "s":
                    two.decode_step_shared(t, p, 3, prefix, lb, nb)
                else:
                    two.decode_step(t, p, lb, nb)
            graphs[kind] = g
        for step, kind in enumerate("o s s s s o s o o s o".split()):
            t.copy_(na)
            p += 1
            one.decode_step(t, p, la, na)
            graphs[kind].replay()
            assert one.status() == mk.MK_OK and two.status() == mk.MK_OK, (step, kind)
            a, b = la.double(), lb.double()
            assert ((a - b).abs() <= 2e-2 + 1e-2 * a.abs()).all(), (step, kind)
    finally:
        one.close()
        two.close()


def test_shared_steps_refuse_bad_calls_and_report_bad_positions():
    hs, eng, kc, vc = engine(synth.TINY, 1, 40)
    L = mk.load()
    try:
        t, p, n = ints([1]), ints([20]), ints([0])
        T, P, N = t.data_ptr(), p.data_ptr(), n.data_ptr()
        call = lambda *x: L.mk_decode_step_shared(eng.h, *x)  # noqa: E731
        assert call(T, P, 0, 10, None, N, None) == mk.MK_ERR_INVALID_ARG  # not a per-op plan
        eng.plan(batch=1, exec_mode="per_op")
        for bad in ((None, P, 0, 10, None, N, None), (T, None, 0, 10, None, N, None), (T, P, 0, 10, None, None, None),
                    (T, P, 1, 10, None, N, None), (T, P, -1, 10, None, N, None), (T, P, 0, 41, None, N, None),
                    (T, P, 0, -1, None, N, None)):
            assert call(*bad) == mk.MK_ERR_INVALID_ARG
        assert call(T, P, 0, 21, None, N, None) == mk.MK_OK
        assert eng.status() == mk.MK_ERR_DEVICE_INPUT  # position 20 lies in the prefix
        assert call(T, P, 0, 20, None, N, None) == mk.MK_OK
        assert eng.status() == mk.MK_OK
    finally:
        eng.close()


def test_serving_round():
    """Together, as a server would use them: a prompt prefilled once and forked to eight sequences, which decode over
    the shared prefix; one of them checks drafted tokens; a finished one is kept in a page pool and comes back."""
    shape, batch, prefix = SMALL_1B, 16, 90
    hs, eng, kc, vc = engine(shape, batch, 160)
    try:
        prompt = torch.randint(0, shape.vocab, (prefix,), dtype=torch.int32, device="cuda")
        nxt = ints([0])
        eng.prefill(0, prompt, 0, None, nxt)
        eng.fork(0, range(1, batch), prefix)
        eng.plan(batch=batch, exec_mode="per_op")
        toks, pos = [int(nxt)] * batch, [prefix] * batch
        lg, nx = torch.empty(batch, shape.vocab, device="cuda"), ints([0] * batch)
        for step in range(4):
            eng.decode_step_shared(ints(toks), ints(pos), 0, prefix, lg, nx)
            assert eng.status() == mk.MK_OK
            assert len(set(nx.tolist())) == 1  # the same greedy answer in every sequence
            toks, pos = nx.tolist(), [x + 1 for x in pos]
        # sequence 5 into a pool of 16-row pages, cleared, and back
        rows, page = pos[5], 16
        pool = sv.KvPool(*(torch.zeros(shape.n_layers, 20, shape.n_kv_heads, page, shape.head_dim, device="cuda",
                                       dtype=torch.bfloat16) for _ in range(2)))
        st = sv.KvState(4, 20, 12)
        sv.kv_resize(pool, st, ints([2]), ints([rows]))
        held = st.table[2].tolist()
        cache = sv.KvPool(kc, vc)
        out = [(5, i * page, held[i], 0, min(page, rows - i * page)) for i in range(-(-rows // page))]
        sv.kv_copy(cache, pool, ints(out))
        before = kc[:, 5, :, :rows].clone(), vc[:, 5, :, :rows].clone()
        kc[:, 5].zero_()
        vc[:, 5].zero_()
        sv.kv_copy(pool, cache, ints([(b, c, a, d, n) for a, d, b, c, n in out]))
        assert torch.equal(kc[:, 5, :, :rows], before[0]) and torch.equal(vc[:, 5, :, :rows], before[1])
        # the batched plan again: sequence 5 checks its own greedy continuation
        eng.plan(batch=batch)
        ids, tok = [], toks[5]
        for i in range(3):
            eng.prefill(5, ints([tok]), rows + i, None, nxt)
            tok = int(nxt)
            ids.append(tok)
        o, a = ints([0] * 4), ints([0])
        eng.speculate(5, ints([toks[5]] + ids), rows, torch.rand(4, device="cuda"), o, a,
                      temperature=torch.zeros(1, device="cuda"))
        assert eng.status() == mk.MK_OK and int(a) == 3 and o.tolist()[:3] == ids
    finally:
        eng.close()
