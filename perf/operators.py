"""The serving operators' measured cases: cache pages (copy, fork, resize, compact), decode attention over a shared
prefix, token probabilities, and verification of drafted tokens.

Each case is run in its plain form (elementary torch operations) or through
``decode_megakernel_interpreter_b200.serving``.
"""
import numpy as np
import torch

own = False

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
DTYPES = {"bf16": BF16, "f16": F16, "f32": F32}


# ----------------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # --- cache pages
        # one prompt of 1000 tokens sampled 15 more times: shared full pages, a copied last page (1B shape)
        {"name": "fork_15_of_one_prompt", "op": "fork", "layers": 16, "kv_heads": 8, "head_dim": 64, "page": 64,
         "n_pages": 512, "n_seqs": 32, "max_pages": 64, "parents": 1, "n": 15, "len_max": 1000},
        # four suspended sequences come back from the page pool into an engine's cache slots (1B shape)
        {"name": "copy_pages_into_slots", "op": "copy", "layers": 16, "kv_heads": 8, "head_dim": 64, "page": 64,
         "n_pages": 256, "slots": 16, "slot_rows": 2048, "seqs": 4, "len_max": 2000},
        # before a decode step every running sequence grows or is cut back by a few tokens; some share a last page
        {"name": "resize_batch_16", "op": "resize", "layers": 2, "kv_heads": 2, "head_dim": 64, "page": 16,
         "n_pages": 2048, "n_seqs": 16, "max_pages": 128, "n": 16, "len_max": 1500, "delta": 9, "sharers": 4},
        # half of the pool is live, scattered; it is moved together at the low end (1B shape)
        {"name": "compact_half_full_pool", "op": "compact", "layers": 16, "kv_heads": 8, "head_dim": 64, "page": 64,
         "n_pages": 512, "n_seqs": 64, "max_pages": 64, "len_max": 480},
        # --- attention over a shared prefix
        # a short system prompt and two fresh answers of the tiny configuration: latency
        {"name": "attn_tiny", "op": "attn", "batch": 2, "tokens": 1, "q_heads": 4, "kv_heads": 2, "head_dim": 64,
         "page": 16, "prefix": 64, "own": 32, "dtype": "bf16"},
        # sixteen answers to one 8192-token document (1B shape)
        {"name": "attn_1b_b16_8k", "op": "attn", "batch": 16, "tokens": 1, "q_heads": 32, "kv_heads": 8, "head_dim": 64,
         "page": 64, "prefix": 8192, "own": 512, "dtype": "bf16"},
        # five drafted tokens of eleven sequences, pages that end inside tiles, an odd prefix
        {"name": "attn_draft5_odd", "op": "attn", "batch": 11, "tokens": 5, "q_heads": 24, "kv_heads": 8, "head_dim": 64,
         "page": 48, "prefix": 5003, "own": 701, "dtype": "f16"},
        # the largest: 64 answers over a 32768-token prefix (8B shape)
        {"name": "attn_8b_b64_32k", "op": "attn", "batch": 64, "tokens": 1, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "page": 64, "prefix": 32768, "own": 1024, "dtype": "bf16"},
        # --- token probabilities
        # one chunk of a draft check: 5 rows of the engine's logits
        {"name": "probs_5_rows", "op": "probs", "rows": 5, "vocab": 128256, "dtype": "f32"},
        # a large batch of drafted chunks
        {"name": "probs_512_rows", "op": "probs", "rows": 512, "vocab": 128256, "dtype": "f32"},
        # --- verification of drafted tokens
        # one sequence, four tokens from a drafter without probabilities (a lookup)
        {"name": "verify_lookup_b1", "op": "verify", "batch": 1, "drafted": 4, "vocab": 128256, "draft_probs": False},
        # 64 sequences, up to seven tokens each, drafted by a smaller model
        {"name": "verify_b64", "op": "verify", "batch": 64, "drafted": 7, "vocab": 128256, "draft_probs": True},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["fork", "copy", "resize", "compact", "attn", "attn", "attn", "probs", "verify", "verify"])
    heads = rng.choice([(2, 64), (8, 64), (4, 128), (8, 128)])
    if op in ("fork", "resize", "compact", "copy"):
        page = rng.choice([16, 24, 32, 64, 128])
        layers = rng.choice([1, 2, 7, 16])
        row_bytes = layers * heads[0] * heads[1] * 4
        n_pages = max(24, min(_log(rng, 64, 4096), (1 << 30) // (row_bytes * page)))
        c = {"op": op, "layers": layers, "kv_heads": heads[0], "head_dim": heads[1], "page": page, "n_pages": n_pages}
        if op == "fork":
            parents = rng.randint(1, 3)
            return {**c, "n_seqs": 40, "max_pages": n_pages, "parents": parents, "n": rng.randint(1, 16),
                    "len_max": max(1, _log(rng, 1, max(2, (n_pages - 18) * page // (2 * parents))))}
        if op == "resize":
            n = rng.randint(1, min(96, n_pages // 8))
            return {**c, "n_seqs": n + rng.randint(0, 8), "max_pages": n_pages, "n": n, "delta": rng.randint(1, 3 * page),
                    "len_max": _log(rng, 1, max(2, (n_pages // (2 * n + 16) - 3) * page)),
                    "sharers": rng.randint(1, max(1, n // 3))}
        if op == "compact":
            seqs = rng.randint(1, max(1, n_pages // 8))
            return {**c, "n_seqs": seqs, "max_pages": n_pages, "len_max": max(1, n_pages * page // (seqs + 2))}
        seqs = rng.randint(1, 8)
        rows = max(1, min(n_pages * page // (seqs + 1), (200 << 20) // (seqs * row_bytes), _log(rng, 1, 4096)))
        return {**c, "slots": seqs + rng.randint(0, 4), "slot_rows": rows + rng.randint(0, 300), "seqs": seqs, "len_max": rows}
    if op == "attn":
        nq, nkv, d = rng.choice([(4, 2, 64), (32, 8, 64), (32, 8, 128), (8, 8, 128), (16, 2, 64), (24, 8, 128)])
        tokens = rng.choice([1, 1, 1, 2, 5, 8])
        batch = max(1, _log(rng, 1, 64) // tokens)
        return {"op": op, "batch": batch, "tokens": tokens, "q_heads": nq, "kv_heads": nkv, "head_dim": d,
                "page": rng.choice([16, 40, 64, 128, 256]), "prefix": _log(rng, 1, 30000), "own": _log(rng, tokens, 1000),
                "dtype": rng.choice(["bf16", "bf16", "f16"])}
    vocab = rng.choice([4096, 32003, 50001, 128256])
    if op == "probs":
        return {"op": op, "rows": _log(rng, 1, 500), "vocab": vocab, "dtype": rng.choice(["f32", "f32", "bf16"])}
    return {"op": op, "batch": _log(rng, 1, 64), "drafted": rng.randint(1, 7), "vocab": vocab,
            "draft_probs": rng.random() < 0.7}


# ---------------------------------------------------------------------------------------------------------- the inputs

# The bookkeeping of a paged cache is one int32 buffer: [pages free, status, 0, 0], the sequences' lengths, the pages'
# reference counts, the stack of free pages (its top is the last of the first `pages free` entries), and a row of page
# numbers for each sequence (-1 where it has none).

def _views(buf, n_seqs, n_pages, max_pages):
    a, b, c = 4 + n_seqs, 4 + n_seqs + n_pages, 4 + n_seqs + 2 * n_pages
    return buf[4:a], buf[a:b], buf[b:c], buf[c:c + n_seqs * max_pages].reshape(n_seqs, max_pages)


def _bookkeeping(r, case, lens, sharers=0):
    """A bookkeeping buffer for sequences of these lengths with pages in random places; each of the `sharers` first
    sequences hands all its pages to the next one as well (which was cut back into a shared page)."""
    S, P, M, page = case["n_seqs"], case["n_pages"], case["max_pages"], case["page"]
    buf = np.zeros(4 + S + 2 * P + S * M, np.int32)
    ln, refs, free, table = _views(buf, S, P, M)
    table[:] = -1
    order = r.permutation(P)
    at = 0
    for s, n in enumerate(lens):
        k = -(-int(n) // page)
        if s % 2 and s // 2 < sharers:  # the same pages as the sequence before it
            n = ln[s - 1]
            k = -(-int(n) // page)
            table[s, :k] = table[s - 1, :k]
        else:
            table[s, :k] = order[at:at + k]
            at += k
        ln[s] = n
        np.add.at(refs, table[s, :k], 1)
    rest = order[at:]
    free[:len(rest)] = rest
    buf[0] = len(rest)
    return buf


def _pool(g, case, n_pages, page):
    shape = (case["layers"], n_pages, case["kv_heads"], page, case["head_dim"])
    return tuple(torch.randn(shape, generator=g, device="cuda", dtype=BF16) for _ in range(2))


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def prepare(case, seed):
    r = np.random.RandomState(seed % (1 << 31))
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op in ("fork", "resize", "compact"):
        s["k"], s["v"] = _pool(g, case, case["n_pages"], case["page"])
        top = max(1, case["len_max"])
        if op == "fork":
            n = case["parents"]
            lens = [max(1, top - int(r.randint(0, 1 + top // 4))) for _ in range(n)]
            s["buf"] = _ints(_bookkeeping(r, case, lens))
            s["parents"] = _ints(r.randint(0, n, case["n"]))
            s["children"] = _ints(n + r.permutation(case["n_seqs"] - n)[:case["n"]])
        elif op == "compact":
            lens = r.randint(0, top + 1, case["n_seqs"])
            while (-(-lens // case["page"])).sum() > case["n_pages"]:
                lens = lens // 2
            s["buf"] = _ints(_bookkeeping(r, case, lens))
        else:
            lens = r.randint(0, top + 1, case["n_seqs"])
            buf = _bookkeeping(r, case, lens, case["sharers"])
            ln = buf[4:4 + case["n_seqs"]]
            seqs = r.permutation(case["n_seqs"])[:case["n"]]
            new = np.clip(ln[seqs] + r.randint(-case["delta"], case["delta"] + 1, case["n"]), 0,
                          case["max_pages"] * case["page"])
            s["buf"], s["seqs"], s["lens"] = _ints(buf), _ints(seqs), _ints(new)
    elif op == "copy":
        s["k"], s["v"] = _pool(g, case, case["n_pages"], case["page"])
        s["dk"], s["dv"] = _pool(g, case, case["slots"], case["slot_rows"])
        page, items, order, at = case["page"], [], r.permutation(case["n_pages"]), 0
        for slot in r.permutation(case["slots"])[:case["seqs"]]:
            n = max(1, case["len_max"] - int(r.randint(0, 1 + case["len_max"] // 4)))
            for first in range(0, n, page):
                if at < len(order):
                    items.append((order[at], 0, slot, first, min(page, n - first)))
                    at += 1
        s["items"] = _ints(items)
    elif op == "attn":
        B, T, nq, nkv, d = (case[x] for x in ("batch", "tokens", "q_heads", "kv_heads", "head_dim"))
        t, page = DTYPES[case["dtype"]], case["page"]
        shared = -(-case["prefix"] // page)  # the prefix has pages of its own, as after a fork at its end
        pre = case["prefix"]
        lens = pre + r.randint(T, case["own"] + 1, B)
        per = [-(-int(n) // page) - pre // page for n in lens]
        width = -(-(pre + case["own"]) // page)
        n_pages = shared + sum(per)
        order = r.permutation(n_pages)
        table = np.full((B, width), -1)
        at = shared
        for b in range(B):
            table[b, :pre // page] = order[:pre // page]
            table[b, pre // page:pre // page + per[b]] = order[at:at + per[b]]
            at += per[b]
        s["q"] = torch.randn((B, T, nq, d), generator=g, device="cuda").to(t)
        s["k"] = (1.5 * torch.randn((n_pages, nkv, page, d), generator=g, device="cuda")).to(t)
        s["v"] = torch.randn((n_pages, nkv, page, d), generator=g, device="cuda").to(t)
        s["table"], s["lens"] = _ints(table), _ints(lens)
        s["prefix_pages"], s["prefix_len"] = _ints(order[:shared]), _ints([pre])
    elif op == "probs":
        s["logits"] = (3.0 * torch.randn((case["rows"], case["vocab"]), generator=g, device="cuda")).to(DTYPES[case["dtype"]])
        t = r.uniform(0.5, 1.5, case["rows"]).astype(np.float32)
        t[r.uniform(size=case["rows"]) < 0.05] = 0.0  # some requests are greedy
        s["temperature"] = torch.from_numpy(t).cuda()
    else:
        B, T, V = case["batch"], case["drafted"], case["vocab"]
        z = 3.0 * torch.randn((B, T + 1, V), generator=g, device="cuda")
        s["target"] = torch.softmax(z, -1)
        if case["draft_probs"]:
            z[:, :T] += 0.7 * torch.randn((B, T, V), generator=g, device="cuda")  # a drafter that mostly agrees
            q = torch.softmax(z[:, :T], -1)
            s["draft"] = q.contiguous()
        else:
            q = s["target"][:, :T]
            s["draft"] = None
        s["tokens"] = torch.multinomial(q.reshape(B * T, V), 1, generator=g).reshape(B, T).to(torch.int32)
        n = np.where(r.uniform(size=B) < 0.75, T, r.randint(0, T + 1, B))
        s["n"] = _ints(n)
        s["u"] = torch.rand((B, T + 1), generator=g, device="cuda")
        if not case["draft_probs"]:
            s["u"][:, :T] *= s["target"][:, :T].amax(-1)  # a lookup's tokens are accepted about as often
    return s


# ------------------------------------------------------------------------------------------------------ the plain forms

def _plain_fork(s, c):
    buf = s["buf"].clone()
    ln, refs, free, table = _views(buf, c["n_seqs"], c["n_pages"], c["max_pages"])
    par, kid, page = s["parents"].long(), s["children"].long(), c["page"]
    n = ln[par]
    full, rem = n // page, n % page
    need = rem > 0
    rank = need.cumsum(0) - 1
    new = free[(buf[0] - 1 - rank).clamp(min=0)]
    j = torch.arange(c["max_pages"], device=n.device)
    rows = table[par]
    last = rows.gather(1, full.long()[:, None].clamp(max=c["max_pages"] - 1))[:, 0]
    refs.index_add_(0, rows[j < full[:, None]].long(), torch.ones_like(rows[j < full[:, None]]))
    kids = torch.where(j < full[:, None], rows, -1)
    kids = torch.where((j == full[:, None]) & need[:, None], new[:, None], kids)
    table[kid] = kids
    ln[kid] = n
    at = need.nonzero()[:, 0]
    src, dst = last[at].long(), new[at].long()
    refs[dst] = 1
    buf[0] -= need.sum()
    keep = (torch.arange(page, device=n.device) < rem[at][:, None])[None, :, None, :, None]
    for x in (s["k"], s["v"]):
        x[:, dst] = torch.where(keep, x[:, src], x[:, dst])
    return buf, s["k"], s["v"]


def _plain_resize(s, c):
    buf = s["buf"].clone()
    ln, refs, free, table = _views(buf, c["n_seqs"], c["n_pages"], c["max_pages"])
    seqs, new, page, P = s["seqs"].long(), s["lens"], c["page"], c["n_pages"]
    old = ln[seqs]
    a, b = (new + page - 1) // page, (old + page - 1) // page
    j = torch.arange(c["max_pages"], device=new.device)
    rows = table[seqs]
    gone = (j >= a[:, None]) & (j < b[:, None])
    had = refs > 0
    refs.index_add_(0, rows[gone].long(), torch.full_like(rows[gone], -1))
    freed = (had & (refs == 0)).nonzero()[:, 0]
    free[buf[0] + torch.arange(len(freed), device=new.device)] = freed.int()
    buf[0] += len(freed)
    # a sequence that grows inside a page that others hold too gets its own copy; of several that grow on one page the
    # last holder keeps it
    last = rows.gather(1, (old // page).long()[:, None].clamp(max=c["max_pages"] - 1))[:, 0]
    grows = (new > old) & (old % page != 0)
    i = torch.arange(len(seqs), device=new.device)
    rank = ((last[:, None] == last[None]) & grows[None] & (i[None] < i[:, None])).sum(1)
    cow = grows & (refs[last.long().clamp(min=0)] - rank > 1)
    more = (a - b).clamp(min=0)
    need = cow.long() + more
    start = need.cumsum(0) - need
    own_page = free[(buf[0] - 1 - start).clamp(0, P - 1)]
    k = start[:, None] + cow[:, None] + (j - b[:, None])
    got = free[(buf[0] - 1 - k).clamp(0, P - 1)]
    add = (j >= b[:, None]) & (j < a[:, None])
    rows = torch.where(add, got, torch.where(gone, -1, rows))
    rows = torch.where(cow[:, None] & (j == (old // page)[:, None]), own_page[:, None], rows)
    table[seqs] = rows
    refs[got[add].long()] = 1
    at = cow.nonzero()[:, 0]
    src, dst = last[at].long(), own_page[at].long()
    refs[dst] = 1
    refs.index_add_(0, src, torch.full_like(last[at], -1))
    buf[0] -= need.sum()
    ln[seqs] = new
    keep = (torch.arange(page, device=new.device) < (old % page)[at][:, None])[None, :, None, :, None]
    for x in (s["k"], s["v"]):
        x[:, dst] = torch.where(keep, x[:, src], x[:, dst])
    return buf, s["k"], s["v"]


def _plain_compact(s, c):
    buf = s["buf"].clone()
    ln, refs, free, table = _views(buf, c["n_seqs"], c["n_pages"], c["max_pages"])
    P = c["n_pages"]
    live = refs > 0
    n = live.sum()
    page = torch.arange(P, device=buf.device)
    src, dst = (live & (page >= n)).nonzero()[:, 0], (~live & (page < n)).nonzero()[:, 0]
    to = page.int()
    to[src] = dst.int()
    table[:] = torch.where(table >= 0, to[table.clamp(min=0).long()], -1)
    refs[dst] = refs[src]
    refs[src] = 0
    free[:] = torch.where(page < P - n, P - 1 - page, free)
    buf[0] = P - n
    for x in (s["k"], s["v"]):
        x[:, dst] = x[:, src]
    return buf, s["k"], s["v"]


def _plain_copy(s, c):
    sp, sr, dp, dr, n = s["items"].long().unbind(1)
    r = torch.arange(int(c["page"]), device=n.device)
    keep = r < n[:, None]
    of = lambda x: x[:, None].expand_as(keep)[keep]  # noqa: E731
    src, dst = (sr[:, None] + r)[keep], (dr[:, None] + r)[keep]
    for x, y in ((s["k"], s["dk"]), (s["v"], s["dv"])):
        y.transpose(2, 3)[:, of(dp), dst] = x.transpose(2, 3)[:, of(sp), src]
    return s["dk"], s["dv"]


def _plain_attn(s, c):
    B, T, nq, nkv, d = (c[x] for x in ("batch", "tokens", "q_heads", "kv_heads", "head_dim"))
    G, page, pre, dev = nq // nkv, c["page"], c["prefix"], s["q"].device
    q = s["q"].float().reshape(B, T, nkv, G, d).permute(2, 0, 1, 3, 4)              # [kv head][b][t][g][d]
    pp = s["prefix_pages"].long()
    kp, vp = (x[pp].float().transpose(0, 1).reshape(nkv, -1, d)[:, :pre] for x in (s["k"], s["v"]))
    at = pre + torch.arange(c["own"], device=dev)
    pages = s["table"].long()[:, at // page].clamp(min=0)                            # [b][own row]
    ko, vo = (x.transpose(1, 2)[pages, at % page].float().permute(2, 0, 1, 3) for x in (s["k"], s["v"]))
    scale = d ** -0.5
    sp = (q.reshape(nkv, B * T * G, d) @ kp.transpose(1, 2)).reshape(nkv, B, T, G, -1) * scale
    so = (q.reshape(nkv, B, T * G, d) @ ko.transpose(2, 3)).reshape(nkv, B, T, G, -1) * scale
    sees = s["lens"][:, None] - (T - 1) + torch.arange(T, device=dev)                # positions that a token sees
    sees = sees[None, :, :, None, None]
    sp = sp.masked_fill(torch.arange(pre, device=dev) >= sees, float("-inf"))
    so = so.masked_fill(at >= sees, float("-inf"))
    m = torch.maximum(sp.amax(-1), so.amax(-1)).clamp(min=-3e38)
    sp, so = torch.exp(sp - m[..., None]), torch.exp(so - m[..., None])
    z = sp.sum(-1) + so.sum(-1)
    o = (sp.reshape(nkv, B * T * G, -1) @ vp).reshape(nkv, B, T, G, d)
    o = o + (so.reshape(nkv, B, T * G, -1) @ vo).reshape(nkv, B, T, G, d)
    o = torch.where(z[..., None] > 0, o / z[..., None], 0.0)
    lse = m + torch.log(z)
    return (o.permute(1, 2, 0, 3, 4).reshape(B, T, nq, d).to(s["q"].dtype),
            lse.permute(1, 2, 0, 3).reshape(B, T, nq).contiguous())


def _plain_probs(s, c):
    z = s["logits"].float()
    t = s["temperature"][:, None]
    top = z.amax(-1, keepdim=True)
    e = torch.exp((z - top) / torch.where(t > 0, t, 1.0))
    p = e / e.sum(-1, keepdim=True, dtype=torch.float64).float()
    i = torch.arange(z.shape[1], device=z.device)
    first = torch.where(z == top, i, z.shape[1]).amin(-1, keepdim=True)  # greedy: all on the first largest logit
    return torch.where(t > 0, p, (i == first).float())


def _plain_verify(s, c):
    B, T, V = c["batch"], c["drafted"], c["vocab"]
    p, q, x, n = s["target"], s["draft"], s["tokens"].long(), s["n"].long()
    dev = p.device
    px = p[:, :T].gather(2, x[..., None])[..., 0].double()
    qx = q.gather(2, x[..., None])[..., 0].double() if q is not None else torch.ones_like(px)
    j = torch.arange(T, device=dev)
    ok = (s["u"][:, :T].double() * qx < px) & (j < n[:, None])
    a = ok.long().cumprod(1).sum(1)                                                  # tokens accepted
    row = p[torch.arange(B, device=dev), a].double()
    at = a.clamp(max=T - 1)
    b = torch.arange(B, device=dev)
    if q is not None:
        less = q[b, at].double()
    else:
        less = torch.where(torch.arange(V, device=dev) == x[b, at][:, None], 1.0, 0.0).double()
    rest = torch.where((a < n)[:, None], (row - less).clamp(min=0), row)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, row)
    run_ = rest.cumsum(1)
    t = s["u"][:, T].double() * run_[:, -1]
    new = (run_ <= t[:, None]).sum(1).clamp(max=V - 1)
    out = torch.full((B, T + 1), -1, dtype=torch.int32, device=dev)
    j = torch.arange(T + 1, device=dev)
    out[:, :T] = torch.where(j[:T] < a[:, None], s["tokens"], -1)
    out = torch.where(j == a[:, None], new[:, None].int(), out)
    return out, a.int()


PLAIN = {"fork": _plain_fork, "resize": _plain_resize, "compact": _plain_compact, "copy": _plain_copy,
         "attn": _plain_attn, "probs": _plain_probs, "verify": _plain_verify}


# ------------------------------------------------------------------------------------------------------------- one pass

def _own(s, c):
    from decode_megakernel_interpreter_b200 import serving as sv

    op = c["op"]
    if op == "attn":
        return sv.shared_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["prefix_pages"], s["prefix_len"],
                                   return_lse=True)
    if op == "probs":
        return sv.token_probs(s["logits"], s["temperature"])
    if op == "verify":
        return sv.verify(s["target"], s["draft"], s["tokens"], s["u"], n_drafted=s["n"])
    if "pool" not in s:  # a server keeps the handle of its pool
        s["pool"] = sv.KvPool(s["k"], s["v"])
    if op == "copy":
        if "slots" not in s:
            s["slots"] = sv.KvPool(s["dk"], s["dv"])
        sv.kv_copy(s["pool"], s["slots"], s["items"])
        return s["dk"], s["dv"]
    state = sv.KvState(c["n_seqs"], c["n_pages"], c["max_pages"], buffer=s["buf"].clone())
    if op == "fork":
        sv.kv_fork(s["pool"], state, s["parents"], s["children"])
    elif op == "resize":
        sv.kv_resize(s["pool"], state, s["seqs"], s["lens"])
    else:
        sv.kv_compact(s["pool"], state)
    return state.buffer, s["k"], s["v"]


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return PLAIN[c["op"]](state, c)


def work(case):
    op = case["op"]
    if op in ("fork", "resize", "compact", "copy"):
        row = case["layers"] * case["kv_heads"] * case["head_dim"] * 2 * 2  # a position's K and V, all layers
        page = case["page"]
        if op == "copy":
            rows = min(case["seqs"] * case["len_max"] * 7 / 8, case["n_pages"] * page)
            return {"bytes": 2 * rows * row + 20 * rows / page, "flops": 0}
        if op == "fork":
            rows = min(page, case["len_max"]) / 2
            tables = 4 * case["len_max"] / page * (case["parents"] + 2 * case["n"])
            return {"bytes": rows * row * (case["parents"] + case["n"]) + tables + 24 * case["n"], "flops": 0}
        if op == "resize":
            rows = min(page, case["len_max"]) / 2 * min(case["sharers"], case["n"] / 2) / 2
            return {"bytes": 2 * rows * row + case["n"] * (24 + 12 * (1 + case["delta"] / page)), "flops": 0}
        live = min(1.0, case["n_seqs"] * (case["len_max"] / 2 / page + 0.5) / case["n_pages"])
        moved = case["n_pages"] * live * (1 - live)
        return {"bytes": 2 * moved * page * row + 12 * case["n_pages"], "flops": 0}
    if op == "attn":
        B, T, nq, nkv, d = (case[x] for x in ("batch", "tokens", "q_heads", "kv_heads", "head_dim"))
        mean = (case["own"] + T) / 2
        kv = (case["prefix"] + B * mean) * nkv * d * 2 * 2
        return {"bytes": kv + 2 * B * T * nq * d * 2 + 4 * B * T * nq,
                "flops": 4.0 * B * T * nq * d * (case["prefix"] + mean)}
    if op == "probs":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (4 + (2 if case["dtype"] != "f32" else 4)), "flops": 4.0 * n}
    # the accepting needs single values; the new token comes from one row of each kind
    B, T, V = case["batch"], case["drafted"], case["vocab"]
    return {"bytes": B * V * 4 * (2 if case["draft_probs"] else 1) + B * T * 20, "flops": 4.0 * B * V}


# ------------------------------------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, c = case["op"], case
    if op == "copy":
        return None  # nothing is computed
    if op in ("fork", "resize", "compact"):
        buf = s["buf"].cpu().numpy().copy()
        ln, refs, free, table = _views(buf, c["n_seqs"], c["n_pages"], c["max_pages"])
        page = c["page"]
        if op == "fork":
            for p, k in zip(s["parents"].tolist(), s["children"].tolist()):
                for j in range(int(ln[p]) // page):
                    table[k, j] = table[p, j]
                    refs[table[p, j]] += 1
                if ln[p] % page:
                    buf[0] -= 1
                    table[k, ln[p] // page] = free[buf[0]]
                    refs[free[buf[0]]] = 1
                ln[k] = ln[p]
        elif op == "resize":
            freed = []
            todo = list(zip(s["seqs"].tolist(), s["lens"].tolist()))
            for q, n in todo:
                for j in range(-(-n // page), -(-int(ln[q]) // page)):
                    refs[table[q, j]] -= 1
                    if refs[table[q, j]] == 0:
                        freed.append(int(table[q, j]))
                    table[q, j] = -1
            for x in sorted(freed):
                free[buf[0]] = x
                buf[0] += 1
            for q, n in todo:
                have = int(ln[q])
                if n > have and have % page and refs[table[q, have // page]] > 1:
                    refs[table[q, have // page]] -= 1
                    buf[0] -= 1
                    table[q, have // page] = free[buf[0]]
                    refs[free[buf[0]]] = 1
                for j in range(-(-have // page), -(-n // page)):
                    buf[0] -= 1
                    table[q, j] = free[buf[0]]
                    refs[free[buf[0]]] = 1
                ln[q] = n
        else:
            P = c["n_pages"]
            n = int((refs > 0).sum())
            holes = [x for x in range(n) if refs[x] == 0]
            moved = dict(zip([x for x in range(n, P) if refs[x] > 0], holes))
            for x, y in moved.items():
                refs[y], refs[x] = refs[x], 0
            for q in range(c["n_seqs"]):
                for j in range(c["max_pages"]):
                    table[q, j] = moved.get(int(table[q, j]), table[q, j])
            free[:P - n] = np.arange(P - 1, n - 1, -1)
            buf[0] = P - n
        return torch.from_numpy(buf), None, None
    if op == "attn":
        B, T, nq, nkv, d = (c[x] for x in ("batch", "tokens", "q_heads", "kv_heads", "head_dim"))
        out = torch.zeros((B, T, nq, d), dtype=torch.float64, device="cuda")
        lse = torch.zeros((B, T, nq), dtype=torch.float64, device="cuda")
        table, page, pre = s["table"].tolist(), c["page"], c["prefix"]
        pp = s["prefix_pages"].tolist()
        for b, n in enumerate(s["lens"].tolist()):
            pages = pp[:pre // page] + table[b][pre // page:-(-n // page)]
            kv = [x[torch.tensor(pages, device="cuda")].double().transpose(0, 1).reshape(nkv, -1, d)[:, :n].clone()
                  for x in (s["k"], s["v"])]
            if pre % page:  # the prefix's last rows stand in its own last page
                cut = (pre // page) * page
                for x, y in zip(kv, (s["k"], s["v"])):
                    x[:, cut:pre] = y[pp[-1], :, :pre - cut].double()
            qb = s["q"][b].double().reshape(T, nkv, nq // nkv, d)
            for t in range(T):
                m = n - T + 1 + t
                z = torch.einsum("hgd,hnd->hgn", qb[t], kv[0][:, :m]) / d ** 0.5
                lse[b, t] = torch.logsumexp(z, -1).reshape(-1)
                out[b, t] = torch.einsum("hgn,hnd->hgd", torch.softmax(z, -1), kv[1][:, :m]).reshape(nq, d)
        return out, lse
    if op == "probs":
        z, t = s["logits"].double(), s["temperature"].double()
        p = torch.softmax(z / torch.where(t > 0, t, 1.0)[:, None], -1)
        for i in (t == 0).nonzero()[:, 0].tolist():
            p[i] = 0
            p[i, int((z[i] == z[i].max()).nonzero()[0, 0])] = 1
        return p
    B, T = c["batch"], c["drafted"]
    tokens, count = np.full((B, T + 1), -1, np.int32), np.zeros(B, np.int32)
    x, u, n = s["tokens"].tolist(), s["u"].double().tolist(), s["n"].tolist()
    for b in range(B):
        a = 0
        while a < n[b]:
            qx = float(s["draft"][b, a, x[b][a]]) if s["draft"] is not None else 1.0
            if not u[b][a] * qx < float(s["target"][b, a, x[b][a]]):
                break
            tokens[b, a] = x[b][a]
            a += 1
        w = s["target"][b, a].cpu().numpy().astype(np.float64)
        if a < n[b]:
            if s["draft"] is not None:
                less = np.maximum(w - s["draft"][b, a].cpu().numpy(), 0.0)
            else:
                less = w.copy()
                less[x[b][a]] = 0.0
            w = less if less.any() else w
        at = np.cumsum(w)
        tokens[b, a] = int(np.argmax(at > u[b][T] * at[-1]))
        count[b] = a
    return torch.from_numpy(tokens), torch.from_numpy(count)
