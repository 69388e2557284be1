"""Lists that ask for far more pages than any pool has: the sum of what they
ask for passes 32 bits."""
import pytest
import torch

import decode_megakernel_interpreter_b200 as mk
from decode_megakernel_interpreter_b200 import serving as sv

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def want_pages(asked, n_pages):
    """(which entries fit, pages used) by list order, in whole numbers of any size."""
    used, ok = 0, []
    for x in asked:
        ok.append(used + x <= n_pages)
        used += x if ok[-1] else 0
    return ok, used


@pytest.mark.parametrize("n_seqs, max_pages", [(1024, 1 << 21), (2, 1 << 30), (3, (1 << 30) - 1)])
def test_requests_past_32_bits_do_not_fit(n_seqs, max_pages):
    """Every sequence asks for all the pages that a table row can hold (1024 x 2^21 and 2 x 2^30 are 2^31, 3 x 2^30 - 3
    is negative in 32 bits), a few for some that there are.  (Tables of 8.6 and 13 GB.)"""
    n_pages = 24
    k = torch.zeros((1, n_pages, 1, 1, 16), dtype=torch.int8, device="cuda")
    pool, st = sv.KvPool(k, k.clone()), sv.KvState(n_seqs, n_pages, max_pages)
    asked = [max_pages] * n_seqs
    sv.kv_resize(pool, st, ints(list(range(n_seqs))), ints(asked))
    assert st.status() == mk.MK_ERR_OUT_OF_MEMORY
    assert int(st.n_free) == n_pages and (st.lens == 0).all() and (st.refs == 0).all()
    asked[n_seqs // 2] = 5
    if n_seqs > 3:
        asked[7], asked[1000] = 17, 4  # 17, then 5 (at 512), leave 2: 4 do not fit
        asked[1020] = 2
    ok, used = want_pages(asked, n_pages)
    sv.kv_resize(pool, st, ints(list(range(n_seqs))), ints(asked))
    assert st.status() == mk.MK_ERR_OUT_OF_MEMORY
    assert st.lens.tolist() == [x if y else 0 for x, y in zip(asked, ok)]
    assert int(st.n_free) == n_pages - used and int(st.refs.sum()) == used
    free = st.buffer[4 + n_seqs + n_pages:][:n_pages - used].tolist()
    held = sorted(p for s, y in enumerate(ok) if y for p in st.table[s, :asked[s]].tolist())
    assert sorted(free + held) == list(range(n_pages))
