"""The serving operators' C ABI and Python front: symbols, struct mirrors and
every refusal that needs no GPU."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import decode_megakernel_interpreter_b200 as mk
from decode_megakernel_interpreter_b200 import serving as sv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mk_serve.h")
P = 256  # a non-null, aligned address for arguments that are refused before anything is read


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_every_declared_symbol_is_exported():
    lib = mk.load()
    names = set(re.findall(r"\b(mk_\w+)\s*\(", header()))
    assert {"mk_kv_init", "mk_kv_resize", "mk_kv_fork", "mk_kv_compact", "mk_kv_copy", "mk_attn_shared",
            "mk_token_probs", "mk_verify"} <= names
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("name", ["mk_kv_pool", "mk_kv_state", "mk_attn_shared_args", "mk_verify_args"])
def test_structs_follow_the_header(name):
    body = re.search(r"typedef struct \{([^}]*)\}\s*" + name + r"\s*;", header()).group(1)
    want = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        m = re.match(r"(?:const\s+)?(\w+)\s*(\*?)\s*(\w+(?:\s*,\s*\*?\w+)*)$", decl)
        want += [(f.strip(" *"), "ptr" if m.group(2) else m.group(1)) for f in m.group(3).split(",")]
    types = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float, "ptr": ctypes.c_void_p}
    assert getattr(mk, name)._fields_ == [(f, types[t]) for f, t in want]


def test_header_is_plain_c_and_sizes_agree(tmp_path):
    names = ["mk_kv_pool", "mk_kv_state", "mk_attn_shared_args", "mk_verify_args"]
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "mk_serve.h"\nint main(void) {\n' +
                   "".join(f'  printf("%zu\\n", sizeof({n}));\n' for n in names) +
                   "  return mk_kv_init(NULL, NULL) == MK_ERR_INVALID_ARG ? 0 : 1;\n}\n")
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                           str(tmp_path / "s"), mk.LIB_PATH, "-Wl,-rpath," + os.path.dirname(mk.LIB_PATH)])
    out = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0
    assert [int(x) for x in out.stdout.split()] == [ctypes.sizeof(getattr(mk, n)) for n in names]


# ------------------------------------------------------------------ cache pages

def pool(**kw):
    d = dict(k=P, v=P * 4096, n_layers=2, n_pages=8, n_kv_heads=2, page=16, head_dim=64, elem_bytes=2)
    d.update(kw)
    return mk.mk_kv_pool(*d.values())


def state(**kw):
    d = dict(words=P, n_seqs=4, max_pages=4, n_pages=8)
    d.update(kw)
    return mk.mk_kv_state(*d.values())


BAD_POOLS = [dict(k=None), dict(v=None), dict(k=P + 8), dict(n_layers=0), dict(n_pages=0), dict(n_pages=(1 << 20) + 1),
             dict(n_kv_heads=-1), dict(page=0), dict(page=(1 << 24) + 1), dict(head_dim=0), dict(head_dim=4),
             dict(elem_bytes=3)]
BAD_STATES = [dict(words=None), dict(words=P + 4), dict(n_seqs=0), dict(max_pages=0), dict(n_pages=7),
              dict(max_pages=1 << 30), dict(n_seqs=(1 << 20) + 1)]


@pytest.mark.parametrize("p, s, n, ws", [(pool(**b), state(), 1, P) for b in BAD_POOLS] +
                         [(pool(), state(**b), 1, P) for b in BAD_STATES] +
                         [(pool(), state(), 0, P), (pool(), state(), 1025, P), (pool(), state(), 1, None),
                          (pool(), state(), 1, P + 16)])
def test_page_calls_refuse_bad_arguments(p, s, n, ws):
    L = mk.load()
    p, s = ctypes.byref(p), ctypes.byref(s)
    assert L.mk_kv_resize(p, s, P, P, n, ws, None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_kv_fork(p, s, P, P, n, ws, None) == mk.MK_ERR_INVALID_ARG
    if n == 1:
        assert L.mk_kv_compact(p, s, ws, None) == mk.MK_ERR_INVALID_ARG


def test_page_calls_refuse_null_lists():
    L = mk.load()
    p, s = ctypes.byref(pool()), ctypes.byref(state())
    for a, b in ((None, P), (P, None)):
        assert L.mk_kv_resize(p, s, a, b, 1, P, None) == mk.MK_ERR_INVALID_ARG
        assert L.mk_kv_fork(p, s, a, b, 1, P, None) == mk.MK_ERR_INVALID_ARG
    assert L.mk_kv_init(None, None) == mk.MK_ERR_INVALID_ARG


@pytest.mark.parametrize("a, b, items, n, ws", [
    (pool(), pool(n_layers=3), P, 1, P), (pool(), pool(n_kv_heads=1), P, 1, P), (pool(), pool(head_dim=128), P, 1, P),
    (pool(), pool(elem_bytes=4), P, 1, P), (pool(), pool(), None, 1, P), (pool(), pool(), P, 0, P),
    (pool(), pool(), P, 16385, P), (pool(), pool(), P, 1, None), (pool(), pool(n_pages=4), P, 1, P),
    (pool(), pool(page=8), P, 1, P),          # the same memory seen in two ways
    (pool(), pool(k=P * 4096, v=P * 8192), P, 1, P),  # one pool's k is the other's v
    (pool(), pool(k=P + 16, v=P * 8192), P, 1, P)])
def test_copy_refuses_bad_arguments(a, b, items, n, ws):
    assert mk.load().mk_kv_copy(ctypes.byref(a), ctypes.byref(b), items, n, None, ws, None) == mk.MK_ERR_INVALID_ARG


def test_sizes_of_buffers():
    L = mk.load()
    assert L.mk_kv_state_words(3, 5, 7) == 4 + 3 + 14 + 15
    assert L.mk_kv_state_words(1 << 20, 1 << 11, 1) == 4 + (1 << 20) + 2 + (1 << 31)
    assert L.mk_kv_state_words(0, 1, 1) == 0
    assert L.mk_kv_workspace_bytes(0, 1) == 0
    for n_pages, n in ((1, 1), (1000, 3), (3, 1000)):
        b = L.mk_kv_workspace_bytes(n_pages, n)
        assert b % 256 == 0 and b >= 64 + 24 * max(n_pages, n)


# ------------------------------------------------------------------ attention

def attn(**kw):
    d = dict(batch=2, n_tokens=1, n_q_heads=4, n_kv_heads=2, head_dim=64, dtype=0, page=16, n_pages=8,
             n_prefix_pages=2, table_width=4, scale=0.125, q=P, k=P, v=P, out=P, lse=None, prefix_pages=P,
             prefix_len=P, table=P, lens=P, status=None, q_batch_stride=256, q_token_stride=256, q_head_stride=64,
             out_batch_stride=256, out_token_stride=256, out_head_stride=64, page_stride=2048, kv_head_stride=1024,
             row_stride=64)
    d.update(kw)
    return mk.mk_attn_shared_args(*d.values())


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(n_tokens=0), dict(n_q_heads=0), dict(n_kv_heads=0), dict(n_q_heads=5), dict(page=0),
    dict(n_pages=0), dict(n_prefix_pages=-1), dict(table_width=0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(table=None), dict(lens=None),
    dict(prefix_pages=None), dict(prefix_len=None), dict(q=P + 8), dict(k=P + 2), dict(v=P + 4), dict(out=P + 8),
    dict(q_head_stride=65), dict(row_stride=4), dict(page_stride=-8), dict(out_batch_stride=12),
    dict(table_width=1 << 27), dict(n_prefix_pages=1 << 27),
    dict(batch=1024, table_width=1 << 26)], ids=str)
def test_attention_refuses_bad_arguments(kw):
    a = attn(**kw)
    assert mk.load().mk_attn_shared(ctypes.byref(a), P, None) == mk.MK_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(head_dim=96), dict(head_dim=256), dict(dtype=2), dict(dtype=-1), dict(n_tokens=17),
                                dict(n_q_heads=34), dict(batch=1025), dict(batch=128, n_tokens=9)], ids=str)
def test_attention_refuses_shapes_that_it_lacks(kw):
    a = attn(**kw)
    assert mk.load().mk_attn_shared(ctypes.byref(a), P, None) == mk.MK_ERR_UNSUPPORTED_SHAPE
    assert mk.load().mk_attn_shared_workspace_bytes(ctypes.byref(a)) == 0


def test_attention_refuses_a_bad_workspace():
    a = attn()
    assert mk.load().mk_attn_shared(ctypes.byref(a), None, None) == mk.MK_ERR_INVALID_ARG
    assert mk.load().mk_attn_shared(ctypes.byref(a), P + 16, None) == mk.MK_ERR_INVALID_ARG
    assert mk.load().mk_attn_shared(None, P, None) == mk.MK_ERR_INVALID_ARG


# ------------------------------------------------------------------ probabilities and verification

def test_probabilities_refuse_bad_arguments():
    f = mk.load().mk_token_probs
    good = [P, 0, 100, None, P, 100, 2, 100, None]
    for i, bad in ((0, None), (1, 3), (1, -1), (2, -1), (4, None), (5, -1), (5, 99), (6, 0), (6, -1), (7, 0), (7, 1 << 30)):
        a = list(good)
        a[i] = bad
        assert f(*a) == mk.MK_ERR_INVALID_ARG, (i, bad)


def ver(**kw):
    d = dict(batch=2, max_drafted=3, vocab=100, target=P, draft=P, tokens=P, n_drafted=None, u=P, out_tokens=P,
             n_accepted=P, status=None, target_batch_stride=400, target_row_stride=100, draft_batch_stride=300,
             draft_row_stride=100)
    d.update(kw)
    return mk.mk_verify_args(*d.values())


@pytest.mark.parametrize("kw", [dict(batch=0), dict(batch=65536), dict(max_drafted=-1), dict(max_drafted=65),
                                dict(vocab=0), dict(vocab=1 << 30), dict(target=None), dict(tokens=None), dict(u=None),
                                dict(out_tokens=None), dict(n_accepted=None), dict(target_row_stride=-1),
                                dict(draft_batch_stride=-1)], ids=str)
def test_verification_refuses_bad_arguments(kw):
    a = ver(**kw)
    assert mk.load().mk_verify(ctypes.byref(a), None) == mk.MK_ERR_INVALID_ARG
    assert mk.load().mk_verify(None, None) == mk.MK_ERR_INVALID_ARG


# ------------------------------------------------------------------ the Python front

def test_python_front_refuses_what_does_not_fit():
    f = torch.zeros
    kv = f(2, 8, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.KvPool(kv, kv[:1])
    with pytest.raises(ValueError):
        sv.KvPool(kv.transpose(2, 3), kv.transpose(2, 3))
    with pytest.raises(ValueError):
        sv.KvState(0, 8, 4, buffer=f(100, dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.KvState(4, 8, 4, buffer=f(10, dtype=torch.int32))
    pl, st = sv.KvPool(kv, kv.clone()), sv.KvState(4, 8, 4, buffer=f(100, dtype=torch.int32))
    i = f(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.kv_resize(pl, st, i, i)
    with pytest.raises(ValueError):
        sv.kv_resize(pl, st, i, i[:1])
    with pytest.raises(ValueError):
        sv.kv_fork(pl, st, i, f(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.kv_resize(pl, st, i.long(), i)
    with pytest.raises(ValueError):
        sv.kv_compact(pl, sv.KvState(4, 9, 4, buffer=f(100, dtype=torch.int32)))
    with pytest.raises(ValueError):
        sv.kv_copy(pl, pl, i)
    q, k = f(2, 1, 4, 64, dtype=torch.bfloat16), kv[0]
    t, n = f(2, 4, dtype=torch.int32), f(2, dtype=torch.int32)
    for bad in (lambda: sv.shared_attention(q[0], k, k, t, n), lambda: sv.shared_attention(q, k, k[:1], t, n),
                lambda: sv.shared_attention(q.half(), k, k, t, n), lambda: sv.shared_attention(q, k, k, t[:1], n),
                lambda: sv.shared_attention(q, k, k, t, n, prefix_pages=n),
                lambda: sv.shared_attention(q, k, k, t, n, out=q.float()),
                lambda: sv.shared_attention(q, k, k, t, n, lse=f(2, 1, 4, dtype=torch.float64)),
                lambda: sv.shared_attention(q, k, k, t, n)):
        with pytest.raises(ValueError):
            bad()
    z = f(2, 10)
    for bad in (lambda: sv.token_probs(z[0]), lambda: sv.token_probs(z.double()), lambda: sv.token_probs(z, f(3)),
                lambda: sv.token_probs(z.t()), lambda: sv.token_probs(z)):
        with pytest.raises(ValueError):
            bad()
    p, u = f(2, 3, 10), f(2, 3)
    x = f(2, 2, dtype=torch.int32)
    for bad in (lambda: sv.verify(p[0], None, x, u), lambda: sv.verify(p, p, x, u), lambda: sv.verify(p, None, x, u[:, :2]),
                lambda: sv.verify(p, None, x[:1], u), lambda: sv.verify(p.double(), None, x, u),
                lambda: sv.verify(p, None, x, u)):
        with pytest.raises(ValueError):
            bad()
