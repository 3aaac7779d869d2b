"""The paged KV cache's operators as measured: attention over pages (one token a
row, verify steps, prompt chunks; causal, with an optional sliding window and
sink positions), appending rows, and managing pages (fork, copy-on-write
growth, compaction).

A cache is one pool of pages a layer, K and V each [layers][pages][KV heads]
[page size][head dim]; row s of the page table lists the pages of sequence s,
-1 where there is none, and lens[s] is its length. INT8 pools hold one code a
value and, behind all codes (at a multiple of 256 bytes), one FP32 scale a row
[layers][pages][KV heads][page size].
"""
import random

import torch

own = False

DEV = "cuda"
HEADER = 16  # words of the cache's state buffer ahead of the reference counts


# ------------------------------------------------------------------ cases
def _attend(name, n_seqs, max_len, hq, hkv, d, page, *, q_len=1, ragged=False, fmt="bf16", window=0, sinks=0):
    return {"name": name, "kind": "attend", "n_seqs": n_seqs, "q_len": q_len, "max_len": max_len, "ragged": ragged,
            "hq": hq, "hkv": hkv, "d": d, "page": page, "fmt": fmt, "window": window, "sinks": sinks}


def _append(name, n_seqs, q_len, max_len, hkv, d, page, *, ragged=False):
    return {"name": name, "kind": "append", "n_seqs": n_seqs, "q_len": q_len, "max_len": max_len, "ragged": ragged,
            "hkv": hkv, "d": d, "page": page}


def _pages(name, kind, n_seqs, max_len, layers, hkv, d, page, *, children=1):
    return {"name": name, "kind": kind, "n_seqs": n_seqs, "max_len": max_len, "children": children, "layers": layers,
            "hkv": hkv, "d": d, "page": page, "ragged": True}


def listed():
    return [
        # one sequence after 1,023 cached positions, the Llama-1B heads: the latency of a single token
        _attend("decode_1x1024_d64", 1, 1024, 32, 8, 64, 16),
        # a small server's batch of unequal lengths, the Qwen3-0.6B heads
        _attend("decode_32_ragged_d128", 32, 4096, 16, 8, 128, 64, ragged=True),
        # a full server at long contexts, the Qwen3-4B heads: the largest cache
        _attend("decode_64x32768_d128", 64, 32768, 32, 8, 128, 128),
        # long conversations kept to a window and sink positions, INT8 cache
        _attend("decode_64_window_int8", 64, 32768, 32, 8, 64, 32, ragged=True, fmt="int8", window=4096, sinks=4),
        # 16 draft tokens and the last one, checked for four sequences at once
        _attend("verify_4x17_d64", 4, 8192, 32, 8, 64, 16, q_len=17, ragged=True),
        # one long prompt from its start
        _attend("prompt_4096_d128", 1, 4096, 32, 8, 128, 64, q_len=4096),
        # a 256-token piece of a prompt behind a long context
        _attend("chunk_256_at_32768_d64", 1, 32768, 32, 8, 64, 16, q_len=256),
        # eight prompts of unequal lengths under a window with sink positions
        _attend("prompts_window_d64", 8, 2000, 32, 8, 64, 32, q_len=2000, ragged=True, window=500, sinks=4),
        # the rows of one decoding step of a batch
        _append("append_64x1_d128", 64, 1, 500, 8, 128, 16, ragged=True),
        # the rows of several prompts
        _append("append_16x2048_d64", 16, 2048, 2048, 8, 64, 64, ragged=True),
        # eight prompts, seven further samples of each: forked, then one position more for all
        _pages("fork_8x8", "fork", 8, 1000, 16, 8, 64, 16, children=7),
        # half of the sequences have ended: what is left moves to the front of the pool
        _pages("compact_64", "compact", 64, 2048, 16, 8, 64, 32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    hkv, d, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    kind = rng.random()
    if kind < 0.65:
        hq = hkv * rng.choice([1, 2, 4, 8])
        window = rng.choice([0, 0, 1])
        fmt = rng.choice(["bf16", "bf16", "int8"])
        if kind < 0.35:  # one token a row
            n_seqs = _log(rng, 1, 128)
            max_len = _log(rng, 1, min(32768, 2 ** 21 // n_seqs))
            q_len = 1
        else:  # several: the scores of the plain form bound them
            q_len = _log(rng, 2, 4096)
            n_seqs = _log(rng, 1, max(1, min(32, 4096 // q_len)))
            max_len = _log(rng, q_len, max(q_len, min(32768, 2 ** 29 // (hq * q_len * n_seqs))))
        window = _log(rng, 1, max_len) if window else 0
        return {k: v for k, v in _attend("", n_seqs, max_len, hq, hkv, d, page, q_len=q_len, ragged=rng.random() < 0.7,
                                         fmt=fmt, window=window, sinks=rng.choice([0, 1, 4, 37]) if window else 0).items()
                if k != "name"}
    if kind < 0.8:
        n_seqs = _log(rng, 1, 128)
        q_len = _log(rng, 1, min(4096, 32768 // n_seqs))
        max_len = _log(rng, q_len, max(q_len, 65536 // n_seqs))
        return {k: v for k, v in _append("", n_seqs, q_len, max_len, hkv, d, page, ragged=rng.random() < 0.7).items()
                if k != "name"}
    n_seqs = _log(rng, 2, 64)
    children = rng.randint(1, 7)
    max_len = _log(rng, 1, 65536 // n_seqs)
    return {k: v for k, v in _pages("", rng.choice(["fork", "compact"]), n_seqs, max_len, rng.randint(1, 16), hkv, d,
                                    page, children=children).items() if k != "name"}


def _lengths(c):
    """(lengths, new tokens) of the rows: fixed by the case, the same for every seed."""
    r = random.Random(c["n_seqs"] * 1000003 + c["max_len"] * 101 + c.get("q_len", 1))
    lens = [r.randint(1, c["max_len"]) if c["ragged"] else c["max_len"] for _ in range(c["n_seqs"])]
    q = [min(n, r.randint(1, c.get("q_len", 1)) if c["ragged"] else c.get("q_len", 1)) for n in lens]
    return lens, q


# ------------------------------------------------------------------ inputs
def _pool(c, layers, n_pages, gen):
    """A pool as one flat buffer, and its views: values (BF16) or codes and scales (INT8)."""
    shape = (layers, n_pages, c["hkv"], c["page"], c["d"])
    n = layers * n_pages * c["hkv"] * c["page"] * c["d"]
    if c.get("fmt") == "int8":
        off = (n + 255) // 256 * 256
        buf = torch.zeros(off + 4 * (n // c["d"]), dtype=torch.uint8, device=DEV)
        codes, scales = buf[:n].view(torch.int8).view(shape), buf[off:].view(torch.float32).view(shape[:4])
        x = torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, 40.0, generator=gen)
        codes.copy_(x.round_().clamp_(-127, 127))
        scales.uniform_(0.5 / 40, 1.5 / 40, generator=gen)  # values of about unit size
        return buf, codes, scales
    buf = torch.empty(n, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    return buf.view(torch.uint8), buf.view(shape), None


def _table(lens, page, width, n_pages, gen):
    """Each row's pages, taken from the pool in a shuffled order."""
    order = torch.randperm(n_pages, generator=gen, device=DEV, dtype=torch.int32)
    need = [-(-n // page) for n in lens]
    count = torch.tensor(need, dtype=torch.int64, device=DEV)
    j = torch.arange(width, device=DEV)
    used = j < count[:, None]
    at = (torch.cumsum(count, 0) - count)[:, None] + j
    return torch.where(used, order[torch.where(used, at, 0)], -1).to(torch.int32)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    lens, q = _lengths(c)
    if c["kind"] == "fork":  # rows n_seqs.. are the children, empty
        rows = c["n_seqs"] * (1 + c["children"])
        lens = lens + [0] * (rows - c["n_seqs"])
        extra = 2 * rows
    else:
        rows, extra = c["n_seqs"], 8
    page, layers = c["page"], c.get("layers", 1)
    width = -(-(c["max_len"] + 1) // page)
    n_pages = sum(-(-n // page) for n in lens) + extra
    s = {"case": c, "width": width, "n_pages": n_pages, "layers": layers, "rows": rows}
    s["kbuf"], s["k"], s["ks"] = _pool(c, layers, n_pages, gen)
    s["vbuf"], s["v"], s["vs"] = _pool(c, layers, n_pages, gen)
    s["tables"] = _table(lens, page, width, n_pages, gen)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    refs = torch.zeros(n_pages + 1, dtype=torch.int32, device=DEV)
    refs.scatter_add_(0, torch.where(s["tables"] >= 0, s["tables"], n_pages).flatten().long(),
                      torch.ones(rows * width, dtype=torch.int32, device=DEV))
    s["refs"] = refs[:n_pages].clone()
    if c["kind"] in ("attend", "append"):
        s["cu"] = torch.tensor([sum(q[:i]) for i in range(rows + 1)], dtype=torch.int32, device=DEV)
        s["n_tokens"], s["max_q"] = sum(q), max(q)
    if c["kind"] == "attend":
        s["q"] = torch.empty((s["n_tokens"], c["hq"], c["d"]), dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
        s["out"] = torch.empty_like(s["q"])
    if c["kind"] == "append":
        shape = (s["n_tokens"], c["hkv"], c["d"])
        s["new_k"] = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
        s["new_v"] = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    if c["kind"] == "fork":
        n, rid = c["n_seqs"], torch.arange(rows, dtype=torch.int32, device=DEV)
        s["src"] = torch.where(rid < n, -1, rid % n).to(torch.int32)
        s["back"] = torch.where(rid < n, s["lens"], 0).to(torch.int32)  # the samples end, the prompts stay
        s["grown"] = s["lens"][rid.long() % n] + 1
    if c["kind"] == "compact":  # every other sequence has ended
        ended = torch.arange(rows, device=DEV) % 2 == 0
        gone = ended[:, None] & (s["tables"] >= 0)
        s["refs"].scatter_add_(0, s["tables"].clamp(min=0).flatten().long(), -gone.flatten().to(torch.int32))
        s["tables"] = torch.where(gone, -1, s["tables"]).to(torch.int32)
        s["lens"] = torch.where(ended, 0, s["lens"]).to(torch.int32)
        s["tables0"], s["refs0"] = s["tables"].clone(), s["refs"].clone()
    if own:  # the cache object that a program keeps, over the same buffers
        import tile_scheduled_persistent_gb300 as tsp
        desc = tsp.ModelDesc(n_layers=layers, n_q_heads=c.get("hq", c["hkv"]), n_kv_heads=c["hkv"], head_dim=c["d"],
                             max_pos=width * page)
        s["cache"] = tsp.PagedKV(desc, n_pages=n_pages, page_size=page, n_seqs=rows, max_len=width * page,
                                 kv_format=tsp.KV_INT8 if c.get("fmt") == "int8" else tsp.KV_BF16,
                                 k=s["kbuf"], v=s["vbuf"], tables=s["tables"], lens=s["lens"])
        s["cache"].refs.copy_(s["refs"])
        s["refs"] = s["cache"].refs
    return s


# ------------------------------------------------------------------ plain forms
def _rows_of(s, pool, scales):
    """[rows][positions][KV heads][d] in FP32: each row's pages in order (whatever page 0 holds where there is none)."""
    x = pool[0][s["tables"].clamp(min=0).long()].float()
    if scales is not None:
        x = x * scales[0][s["tables"].clamp(min=0).long()][..., None]
    return x.permute(0, 1, 3, 2, 4).flatten(1, 2)


def _places(s):
    """Row and position of each token."""
    cu, t = s["cu"].long(), torch.arange(s["n_tokens"], device=DEV)
    row = torch.searchsorted(cu, t, right=True) - 1
    return row, s["lens"].long()[row] - cu[row + 1] + t


def _plain_attend(s):
    c = s["case"]
    hkv, g, d, n = c["hkv"], c["hq"] // c["hkv"], c["d"], s["max_q"]
    row, pos = _places(s)
    at = row * n + torch.arange(s["n_tokens"], device=DEV) - s["cu"].long()[row]  # place in the padded batch
    q = torch.zeros((s["rows"] * n, hkv, g, d), dtype=torch.float32, device=DEV)
    q[at] = s["q"].float().view(-1, hkv, g, d)
    p = torch.full((s["rows"] * n,), -1, dtype=torch.int64, device=DEV)
    p[at] = pos
    p = p.view(s["rows"], n)
    k, v = _rows_of(s, s["k"], s["ks"]), _rows_of(s, s["v"], s["vs"])
    t = torch.arange(k.shape[1], device=DEV)
    seen = t <= p[..., None]
    if c["window"]:
        seen = seen & ((t > p[..., None] - c["window"]) | (t < c["sinks"]))
    seen = seen[:, None, None]  # [rows][1][1][n][positions]
    q = q.view(s["rows"], n, hkv, g, d).permute(0, 2, 3, 1, 4)
    w = torch.matmul(q, k.permute(0, 2, 3, 1)[:, :, None]) * d ** -0.5
    w = torch.where(seen, w, -torch.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top == -torch.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    v = torch.where((t < s["lens"][:, None])[..., None, None], v, 0.0)  # nothing is read behind a sequence's end
    o = torch.matmul(w, v.permute(0, 2, 1, 3)[:, :, None]) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(s["rows"] * n, hkv * g, d)
    return o[at].to(torch.bfloat16)


def _plain_append(s):
    page = s["case"]["page"]
    row, pos = _places(s)
    where = s["tables"][row, pos // page].long()
    s["k"][0, where, :, pos % page] = s["new_k"]
    s["v"][0, where, :, pos % page] = s["new_v"]


def _plain_resize(s, new_lens):
    tables, lens, refs, page, P = s["tables"], s["lens"].long(), s["refs"], s["case"]["page"], s["n_pages"]
    rows = torch.arange(s["rows"], device=DEV)[:, None]
    new = torch.where(new_lens < 0, lens, new_lens.long())
    keep, first, j = (new + page - 1) // page, lens // page, torch.arange(s["width"], device=DEV)
    # rows that shrink let go of the pages behind their new end
    gone = (new < lens)[:, None] & (j >= keep[:, None]) & (tables >= 0)
    refs.scatter_add_(0, tables.clamp(min=0).flatten().long(), -gone.flatten().to(torch.int32))
    tables.copy_(torch.where(gone, -1, tables))
    # rows that grow: pages that are missing, and pages that others hold too
    write = (new > lens)[:, None] & (j >= first[:, None]) & (j < keep[:, None])
    page_of = tables.clamp(min=0).long()
    shared = write & (tables >= 0) & (refs[page_of] > 1)
    writers = torch.zeros(P, dtype=torch.int32, device=DEV).scatter_add_(0, page_of.flatten(), shared.flatten().to(torch.int32))
    low = torch.full((P,), s["rows"], dtype=torch.int64, device=DEV)
    low.scatter_reduce_(0, page_of.flatten(), torch.where(shared, rows, s["rows"]).flatten(), "amin")
    stays = (writers[page_of] == refs[page_of]) & (low[page_of] == rows)
    copied = shared & ~stays
    need = copied | (write & (tables < 0))
    rank = torch.cumsum(need.flatten(), 0).view_as(need) - 1
    free = torch.argsort((refs > 0).to(torch.int8), stable=True)
    fits = need.sum() <= (refs == 0).sum()
    need, copied = need & fits, copied & fits
    fresh = free[torch.where(need, rank, 0).clamp(max=P - 1)]
    refs.scatter_add_(0, page_of.flatten(), -copied.flatten().to(torch.int32))
    refs.scatter_add_(0, fresh.flatten(), need.flatten().to(torch.int32))
    # the page a row's end lies in is copied; the others are written anew
    at = first.clamp(max=s["width"] - 1)[:, None]
    moved = copied.gather(1, at)[:, 0] & (lens % page != 0)
    src = page_of.gather(1, at)[:, 0]
    dst = torch.where(moved, fresh.gather(1, at)[:, 0], src)
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    tables.copy_(torch.where(need, fresh, tables))
    s["lens"].copy_(torch.where((new > lens) & ~fits, lens, new))


def _plain_fork(s, src):
    tables, lens, page = s["tables"], s["lens"], s["case"]["page"]
    rows = torch.arange(s["rows"], device=DEV)
    frm = src.clamp(min=0).long()
    good = (src >= 0) & (frm != rows) & (src[frm] < 0) & (lens == 0) & (tables < 0).all(1)
    held = torch.arange(s["width"], device=DEV) < ((lens[frm] + page - 1) // page)[:, None]
    new = torch.where(good[:, None] & held, tables[frm], tables)
    more = good[:, None] & (new >= 0)
    s["refs"].scatter_add_(0, new.clamp(min=0).flatten().long(), more.flatten().to(torch.int32))
    tables.copy_(new)
    lens.copy_(torch.where(good, lens[frm], lens))


def _plain_compact(s):
    refs, P = s["refs"], s["n_pages"]
    ids, live = torch.arange(P, device=DEV), s["refs"] > 0
    n = live.sum()
    hole, mover = ~live & (ids < n), live & (ids >= n)
    holes = torch.argsort((~hole).to(torch.int8), stable=True)  # the i-th hole, the i-th page that moves
    movers = torch.argsort((~mover).to(torch.int8), stable=True)
    to = torch.where(mover, holes[(torch.cumsum(mover, 0) - 1).clamp(min=0)], ids)
    frm = torch.where(hole, movers[(torch.cumsum(hole, 0) - 1).clamp(min=0)], ids)
    s["k"].copy_(s["k"][:, frm])
    s["v"].copy_(s["v"][:, frm])
    s["tables"].copy_(torch.where(s["tables"] >= 0, to[s["tables"].clamp(min=0).long()], -1))
    refs.copy_(torch.where(ids < n, refs[frm], 0))


def run(state):
    s, c = state, state["case"]
    if c["kind"] == "attend":
        if own:
            s["cache"].attention(0, s["q"], s["out"], cu_tokens=s["cu"], max_tokens=s["max_q"], window=c["window"],
                                 sinks=c["sinks"])
            return s["out"]
        return _plain_attend(s)
    if c["kind"] == "append":
        if own:
            s["cache"].append(0, s["new_k"], s["new_v"], cu_tokens=s["cu"])
        else:
            _plain_append(s)
        return s["k"], s["v"]
    if c["kind"] == "fork":
        # the samples of the last pass end (none at the first), the prompts go back to their own lengths; then new
        # samples start, and each of them and the prompts take one position more
        if own:
            s["cache"].resize(s["back"])
            s["cache"].fork(s["src"])
            s["cache"].resize(s["grown"])
        else:
            _plain_resize(s, s["back"])
            _plain_fork(s, s["src"])
            _plain_resize(s, s["grown"])
        return s["tables"], s["lens"], s["refs"], s["k"], s["v"]
    # a pool with gaps again: compacting leaves the pages that it moved as they were
    s["tables"].copy_(s["tables0"])
    s["refs"].copy_(s["refs0"])
    if own:
        s["cache"].compact()
    else:
        _plain_compact(s)
    return s["tables"], s["refs"], s["k"], s["v"]


# ------------------------------------------------------------------ what a pass cannot do without
def _seen(c, lens, q):
    """(positions read, pairs of a token and a position that it sees), over the rows."""
    read = pairs = 0
    for n, m in zip(lens, q):
        w, k = c["window"], c["sinks"]
        for p in range(n - m, n):
            pairs += p + 1 if not w else min(p + 1, w) + min(k, max(0, p + 1 - w))
        lo = max(0, n - m + 1 - w) if w else 0
        read += n - lo + min(k, lo)
    return read, pairs


def work(case):
    c = case
    lens, q = _lengths(c)
    if c["kind"] == "attend":
        read, pairs = _seen(c, lens, q)
        row = 2 * (c["d"] + 4) if c["fmt"] == "int8" else 4 * c["d"]
        return {"bytes": read * c["hkv"] * row + 4 * sum(q) * c["hq"] * c["d"], "flops": 4 * c["d"] * c["hq"] * pairs}
    if c["kind"] == "append":
        return {"bytes": 8 * sum(q) * c["hkv"] * c["d"], "flops": 0}
    page, one = c["page"], c["layers"] * c["hkv"] * c["page"] * c["d"] * 8  # a page of K and of V, read and written
    tables = 8 * c["n_seqs"] * (1 + (c["children"] if c["kind"] == "fork" else 0)) * -(-(c["max_len"] + 1) // page)
    if c["kind"] == "fork":
        return {"bytes": one * sum(c["children"] for n in lens if n % page) + tables, "flops": 0}
    held = [-(-n // page) for n in lens]
    live, total = sum(held[1::2]), sum(held) + 8
    return {"bytes": one * live * (total - live) // total + tables, "flops": 0}  # pages behind the first `live` ones


# ------------------------------------------------------------------ in 64 bits, from the definition
def exact(case, seed):
    c = case
    if c["kind"] != "attend":
        return None  # rows and pages are moved, not computed
    s = prepare(case, seed)
    lens, m = _lengths(c)
    g, outs = c["hq"] // c["hkv"], []
    for i, (n, new) in enumerate(zip(lens, m)):
        ids = s["tables"][i, : -(-n // c["page"])].long()
        t0 = int(s["cu"][i])
        q = s["q"][t0:t0 + new].double()
        p = torch.arange(n - new, n, device=DEV)[:, None]
        t = torch.arange(n, device=DEV)[None]
        hidden = t > p
        if c["window"]:
            hidden |= (t <= p - c["window"]) & (t >= c["sinks"])
        row = torch.empty((new, c["hq"], c["d"]), dtype=torch.float64, device=DEV)
        for h in range(c["hkv"]):
            k, v = s["k"][0, ids, h].double(), s["v"][0, ids, h].double()
            if c["fmt"] == "int8":
                k, v = k * s["ks"][0, ids, h].double()[..., None], v * s["vs"][0, ids, h].double()[..., None]
            k, v = k.reshape(-1, c["d"])[:n], v.reshape(-1, c["d"])[:n]
            for a in range(h * g, (h + 1) * g):
                score = (q[:, a] @ k.T) / c["d"] ** 0.5
                score[hidden] = -torch.inf
                row[:, a] = torch.softmax(score, 1) @ v
        outs.append(row)
    return torch.cat(outs)
