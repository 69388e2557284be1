"""Calls without work: empty lists and batches give empty outputs and change nothing; their arguments are still checked."""
import pytest
import torch

from decode_megakernel_interpreter_b200 import serving as sv

pytestmark = pytest.mark.gpu


def i(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def test_empty_page_lists():
    k = torch.randn(2, 8, 2, 16, 64, device="cuda").bfloat16()
    pool, st = sv.KvPool(k, k.clone()), sv.KvState(4, 8, 4)
    sv.kv_resize(pool, st, torch.tensor([1], dtype=torch.int32, device="cuda"), torch.tensor([40], dtype=torch.int32, device="cuda"))
    before = [x.clone() for x in (pool.k, pool.v, st.buffer)]
    sv.kv_resize(pool, st, i(0), i(0))
    sv.kv_fork(pool, st, i(0), i(0), stream=torch.cuda.Stream())
    sv.kv_copy(pool, pool, i(0, 5), status=i(1))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (pool.k, pool.v, st.buffer)))
    with pytest.raises(ValueError):
        sv.kv_resize(pool, st, i(0).long(), i(0))
    with pytest.raises(ValueError):
        sv.kv_fork(pool, st, i(0), i(1))
    with pytest.raises(ValueError):
        sv.kv_resize(pool, sv.KvState(4, 9, 4), i(0), i(0))
    with pytest.raises(ValueError):
        sv.kv_copy(pool, pool, i(0, 4))


def test_empty_batches():
    q, k = torch.zeros(0, 1, 4, 64, device="cuda").bfloat16(), torch.zeros(8, 2, 16, 64, device="cuda").bfloat16()
    out, lse = sv.shared_attention(q, k, k, i(0, 4), i(0), return_lse=True)
    assert out.shape == (0, 1, 4, 64) and out.dtype is torch.bfloat16 and lse.shape == (0, 1, 4) and lse.dtype is torch.float32
    assert sv.shared_attention(q, k, k, i(0, 4), i(0), i(2), i(1), out=q) is q
    assert sv.token_probs(torch.zeros(0, 100, device="cuda")).shape == (0, 100)
    assert sv.token_probs(torch.zeros(0, 20000, device="cuda").half(), torch.zeros(0, device="cuda")).dtype is torch.float32
    for draft in (None, torch.zeros(0, 3, 100, device="cuda")):
        tok, acc = sv.verify(torch.zeros(0, 4, 100, device="cuda"), draft, i(0, 3), torch.zeros(0, 4, device="cuda"))
        assert tok.shape == (0, 4) and acc.shape == (0,) and tok.dtype is acc.dtype is torch.int32
    with pytest.raises(ValueError):
        sv.shared_attention(q, k, k, i(1, 4), i(0))
    with pytest.raises(ValueError):
        sv.verify(torch.zeros(0, 4, 100, device="cuda"), None, i(0, 3), torch.zeros(0, 3, device="cuda"))
