"""Shared steps keep the precision of ordinary ones: q, the weights and the attention output as 32-bit numbers."""
import numpy as np
import pytest
import torch

import decode_megakernel_interpreter_b200 as mk
from decode_megakernel_interpreter_b200 import harness
import synth
from test_gpu_serving_engine import SMALL_1B, ints, shared_setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape, batch, prefix", [(synth.TINY, 1, 70), (synth.TINY, 1, 1100), (SMALL_1B, 16, 300),
                                                  (SMALL_1B, 16, 1300), (SMALL_1B, 5, 129)])
def test_shared_steps_against_ordinary_ones(shape, batch, prefix):
    """A sequence's logits, in the 2-norm, within 2^-11 of those of an ordinary step.

    The two kinds differ in the attention: q and the weights are two bf16 numbers each in a shared step, good to 2^-16.
    With scores of scale sum |q k| <= 6 (q of standard deviation 0.9, K/V rows of 1, 64 elements) a score is off by
    6 x 2^-16, a weight by that twice (its own and the sum's) and 2^-16 twice, so a layer's attention output by
    14 x 2^-16 of itself, and two layers' by 28 x 2^-16 < 2^-11.  The norms and products after it keep relative
    errors.  (As one bf16 number each they would be good to 2^-8 only, which gives 1e-3 and more.)"""
    assert shape.n_layers == 2
    hs, one, two = shared_setup(shape, batch, prefix, prefix + 64)
    try:
        one.plan(batch=batch, exec_mode="per_op")
        two.plan(batch=batch, exec_mode="per_op")
        r = np.random.RandomState(1)
        pos = [prefix + int(x) for x in r.randint(0, 30, batch)]
        toks = [int(x) for x in r.randint(0, shape.vocab, batch)]
        la, lb = (torch.empty(batch, shape.vocab, device="cuda") for _ in range(2))
        na, nb = ints([0] * batch), ints([0] * batch)
        for step in range(4):
            t, p = ints(toks), ints(pos)
            one.decode_step(t, p, la, na)
            two.decode_step_shared(t, p, batch - 1, prefix, lb, nb)
            assert one.status() == mk.MK_OK and two.status() == mk.MK_OK
            a, b = la.double(), lb.double()
            off = (a - b).norm(dim=1) / a.norm(dim=1)
            assert (off <= 2.0 ** -11).all(), (step, float(off.max()))
            toks, pos = na.tolist(), [x + 1 for x in pos]
    finally:
        one.close()
        two.close()


def test_a_prefix_longer_than_one_sum():
    """1.24 million positions over two K/V heads: a block's share is taken in two parts, which are added up.

    The bound is that of the shorter cases.  Keys of 2.5 times the others' size keep the weights uneven, so that an
    output is not what random values leave of one another."""
    shape, prefix, max_seq = synth.TINY, 1_240_000, 1_250_000
    dev = harness.upload_model(synth.make_model(shape), shape.tied)
    g = torch.Generator(device="cuda").manual_seed(0)
    size = (shape.n_layers, 1, shape.n_kv_heads, max_seq, shape.head_dim)
    kc, vc = (torch.randn(size, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kc *= 2.5
    one = harness.make_engine(shape, dev, kc, vc, 1, max_seq)
    two = harness.make_engine(shape, dev, kc.clone(), vc.clone(), 1, max_seq)
    try:
        one.plan(batch=1, exec_mode="per_op")
        two.plan(batch=1, exec_mode="per_op")
        la, lb = (torch.empty(1, shape.vocab, device="cuda") for _ in range(2))
        na, nb = ints([0]), ints([0])
        for step in range(3):
            t, p = ints([17 + step]), ints([prefix + 40 + step])
            one.decode_step(t, p, la, na)
            two.decode_step_shared(t, p, 0, prefix, lb, nb)
            assert one.status() == mk.MK_OK and two.status() == mk.MK_OK
            off = (la.double() - lb.double()).norm() / la.double().norm()
            assert off <= 2.0 ** -11, (step, float(off))
    finally:
        one.close()
        two.close()
