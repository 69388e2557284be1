"""Limits that the header names, where no GPU is needed to be told of them."""
import ctypes
import os

import pytest
import torch

import decode_megakernel_interpreter_b200 as mk
from decode_megakernel_interpreter_b200 import serving as sv

P = 256
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mk_serve.h")


@pytest.mark.parametrize("vocab, code", [(104857601, mk.MK_ERR_UNSUPPORTED_SHAPE), ((1 << 30) - 1, mk.MK_ERR_UNSUPPORTED_SHAPE),
                                         (1 << 30, mk.MK_ERR_INVALID_ARG)])
def test_verification_of_too_large_a_vocabulary(vocab, code):
    a = mk.mk_verify_args(batch=1, vocab=vocab, target=P, u=P, out_tokens=P, n_accepted=P, target_batch_stride=vocab,
                          target_row_stride=vocab)
    assert mk.load().mk_verify(ctypes.byref(a), None) == code
    text = open(HEADER).read()
    part = text[text.index(" * mk_verify:"):text.index("} mk_verify_args;")]
    assert "104857600" in part and "MK_ERR_UNSUPPORTED_SHAPE" in part


@pytest.mark.parametrize("layers, heads, page", [(65536, 16384, 1), (65536, 65536, 1), (4096, 1024, 1 << 18)])
def test_pools_whose_rows_cannot_be_counted(layers, heads, page):
    """Refused before anything is launched: a call must not change the bookkeeping and then fail to move the rows."""
    pool = mk.mk_kv_pool(P, P, layers, 1, heads, page, 16, 1)
    st = mk.mk_kv_state(P, 2, 1, 1)
    p, s, L = ctypes.byref(pool), ctypes.byref(st), mk.load()
    assert L.mk_kv_resize(p, s, P, P, 1, P, None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_kv_fork(p, s, P, P, 1, P, None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_kv_compact(p, s, P, None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_kv_copy(p, p, P, 1, None, P, None) == mk.MK_ERR_INVALID_ARG


def test_rows_of_tokens_that_are_not_the_drafts():
    """A longer buffer's rows would be read as if they followed one another."""
    p, u = torch.zeros(2, 3, 10), torch.zeros(2, 3)
    for shape in ((2, 3), (2, 4), (4, 1), (1, 4)):
        with pytest.raises(ValueError, match="tokens"):
            sv.verify(p, None, torch.zeros(shape, dtype=torch.int32), u)
    for shape in ((2, 2), (4,), (3, 2)):
        with pytest.raises(ValueError, match="CUDA"):  # taken, but for the device
            sv.verify(p, None, torch.zeros(shape, dtype=torch.int32), u)
