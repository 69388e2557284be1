"""Engine.speculate with sampling: drafters with and without probabilities, drafts refused at every place, chunks
larger than the batch.  What a call must answer is worked out in 64 bits from the logits that the engine gives for the
same tokens one at a time; the random numbers are chosen so that rounding cannot change it."""
import dataclasses

import numpy as np
import pytest
import torch

import decode_megakernel_interpreter_b200 as mk
from decode_megakernel_interpreter_b200 import harness
import synth
from gpu_common import HostSetup
from serve_ref import probs, verify

pytestmark = pytest.mark.gpu

SMALL_1B = dataclasses.replace(synth.LLAMA_1B, n_layers=2)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("with_probs", [True, False], ids=["probabilities", "lookup"])
@pytest.mark.parametrize("shape, batch, n", [(synth.TINY, 1, 5), (SMALL_1B, 16, 16), (SMALL_1B, 5, 7), (SMALL_1B, 16, 1)],
                         ids=["tiny one launch a token", "1B one chunk", "1B two chunks", "1B no drafts"])
def test_speculate_samples_as_verification_says(shape, batch, n, with_probs):
    """Logits of a chunk and of single tokens differ by less than 1e-2 T (they are 32-bit sums of the same products),
    so probabilities by 2 % of themselves and sums of them by 0.02: random numbers stay a factor of 1.5 from where a
    draft begins to stand, and in the middle of a token of weight 0.1 or more."""
    ctx, seq, V = 24, batch - 1, shape.vocab
    hs = HostSetup(shape, batch, 96)
    dev = harness.upload_model(hs.model, shape.tied)
    kc, vc = harness.upload_kv(hs.k, hs.v)
    eng = harness.make_engine(shape, dev, kc, vc, batch, 96)
    eng.plan(batch=batch)
    r = np.random.RandomState(n)
    try:
        nxt = ints([0])
        eng.prefill(seq, ints(r.randint(0, V, ctx).tolist()), 0, None, nxt)
        first = int(nxt)
        kv = kc.clone(), vc.clone()
        row, T = torch.empty(V, device="cuda"), None
        answers = set()
        for refused in sorted({0, 1, n // 2, n - 2, n - 1} & set(range(n))):  # n - 1: every draft stands
            kc.copy_(kv[0])
            vc.copy_(kv[1])
            tok, drafts, u = first, [], []
            P, Q = np.zeros((n, V)), np.zeros((n - 1, V), np.float32)
            for j in range(n):
                eng.prefill(seq, ints([tok]), ctx + j, row, nxt)
                assert eng.status() == mk.MK_OK
                if T is None:  # a temperature at which few tokens carry most of the weight
                    T = np.float32(0.12 * float(row.std()))
                P[j] = probs(row.double().cpu().numpy(), T)
                if j == n - 1:
                    break
                order = np.argsort(-P[j])
                q = r.rand(V)
                if j == refused:
                    x = int(order[3])  # the drafter is surer of it than the target
                    q[x] = 0
                    q *= 0.25 / q.sum()
                    q[x] = 0.75
                    assert P[j, x] < 0.4
                    Q[j] = q
                    u.append(0.9 if with_probs else min(0.95, 0.2 + 1.5 * P[j, x]))
                    assert u[-1] * (0.75 if with_probs else 1) > 1.5 * P[j, x]
                else:
                    x = int(order[0])
                    q[x] = 0
                    q *= 0.5 / q.sum()
                    q[x] = 0.5
                    Q[j] = q
                    u.append(min(0.97, P[j, x] / (0.5 if with_probs else 1) / 1.6))
                drafts.append(x)
                tok = x
            w = P[refused].copy()
            if refused < n - 1:
                w = np.maximum(w - Q[refused].astype(np.float64), 0) if with_probs else np.where(np.arange(V) == drafts[refused], 0, w)
            i = int(np.argsort(-w)[0 if refused % 2 else 1])
            if w[i] < 0.1:
                i = int(np.argmax(w))
            assert w[i] >= 0.1
            u.append((w[:i].sum() + w[i] / 2) / w.sum())
            u = np.array(u, np.float32)
            want = verify(P, Q if with_probs else None, drafts, n - 1, u)
            assert want == (refused, i)
            kc.copy_(kv[0])
            vc.copy_(kv[1])
            out, acc = ints([-7] * n), ints([-7])
            eng.speculate(seq, ints([first] + drafts), ctx, torch.from_numpy(u).cuda(), out, acc,
                          draft_probs=torch.from_numpy(Q).cuda() if with_probs else None,
                          temperature=torch.tensor([float(T)], device="cuda"))
            assert eng.status() == mk.MK_OK
            assert int(acc) == refused and out.tolist() == drafts[:refused] + [i] + [-1] * (n - 1 - refused), refused
            answers.add(i)
    finally:
        eng.close()
