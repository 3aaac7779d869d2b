"""The paged KV cache on the GPU: attention against the definition in 64 bits,
appended rows, and the pages' life against a sequential program; all of it
together, captured, and on another stream.

Pools are filled with NaN outside the rows' positions, so anything that reads
behind a row's end, or a masked position, shows.

Tolerance of attention: |out - ref| <= 2^-8 |ref| (the output's rounding to
BF16) + c sum_t w_t |v_t|, c = what the weights may be off by: the FP32 error of
the scores (computed by the reference) + 2^-16 (weights enter the product as a
BF16 high part and remainder) + 2^-20 (FP32 exponentials and sums). With an INT8
cache a weight times its value's scale enters as one FP16 number: half a step,
2^-11, in the place of 2^-16 (and queries, scaled to below 2, are FP16: exact but
for what lies under 2^-14 of the largest, 2^-25 absolute, which 2^-20 covers).
"""
import itertools

import numpy as np
import pytest

import paged_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tsp():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tile_scheduled_persistent_gb300 as t
    t.build()
    return t


def bf16(x):
    import torch
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def quantized(x):
    """(codes, scales) of float32 rows [..., d], as the INT8 cache states."""
    s = (np.abs(x).max(-1).astype(np.float32) / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s[..., None] > 0, np.rint(x / s[..., None]), 0).clip(-127, 127)
    return c.astype(np.int8), s


class Case:
    """A cache with rows of given lengths in shuffled pages, and queries; on the
    host, the values that it stands for."""

    def __init__(self, tsp, lens, ns, hq, hkv, d, page, int8=False, seed=0, layer=0, layers=1, pad=0, extra_pages=3,
                 max_len=None, amp=1.0):
        import torch
        r = np.random.default_rng(seed)
        self.lens, self.ns, self.hq, self.d, self.int8 = lens, ns, hq, d, int8
        width = -(-max(max(lens), 1, max_len or 0) // page)
        need = [-(-n // page) for n in lens]
        P = sum(need) + extra_pages
        desc = tsp.ModelDesc(n_layers=layers, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, max_pos=width * page)
        self.cache = c = tsp.PagedKV(desc, n_pages=P, page_size=page, n_seqs=len(lens),
                                     kv_format=tsp.KV_INT8 if int8 else tsp.KV_BF16)
        self.cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        self.n_tokens = int(self.cu[-1]) + pad
        order = r.permutation(P)
        tables = np.full((len(lens), width), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            tables[s, :n] = order[at:at + n]
            at += n
        self.tables = tables
        self.layer = layer
        (kp, ks), (vp, vs) = c.key_pool(), c.value_pool()
        shape = (P, hkv, page, d)
        self.keys, self.values = [], []
        if int8:
            hk, hv = np.full(shape, 127, np.int8), np.full(shape, -127, np.int8)
            hks, hvs = np.full(shape[:3], np.nan, np.float32), np.full(shape[:3], np.nan, np.float32)
        else:
            hk, hv = np.full(shape, np.nan, np.float32), np.full(shape, np.nan, np.float32)
        for s, n in enumerate(lens):
            k, v = (bf16(amp * r.standard_normal((n, hkv, d))).float().numpy() for _ in range(2))
            if int8:
                (kc, ksc), (vc, vsc) = quantized(k), quantized(v)
                k, v = kc * ksc[..., None].astype(np.float64), vc * vsc[..., None].astype(np.float64)
            for t in range(n):
                pg, o = tables[s, t // page], t % page
                if int8:
                    hk[pg, :, o], hks[pg, :, o], hv[pg, :, o], hvs[pg, :, o] = kc[t], ksc[t], vc[t], vsc[t]
                else:
                    hk[pg, :, o], hv[pg, :, o] = k[t], v[t]
            self.keys.append(np.asarray(k, np.float64))
            self.values.append(np.asarray(v, np.float64))
        if int8:
            kp[layer], vp[layer] = torch.from_numpy(hk), torch.from_numpy(hv)
            ks[layer], vs[layer] = torch.from_numpy(hks), torch.from_numpy(hvs)
        else:
            kp[layer], vp[layer] = bf16(hk), bf16(hv)
        c.tables.copy_(torch.from_numpy(tables))
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.refs.copy_(torch.from_numpy(np.bincount(tables[tables >= 0], minlength=P).astype(np.int32)))
        self.q = bf16(r.standard_normal((self.n_tokens, hq, d))).cuda()
        self.dcu = torch.from_numpy(self.cu).cuda()

    def run(self, window=0, sinks=0, cu=True, max_tokens=None, q=None, out=None, **kw):
        import torch
        q = self.q if q is None else q
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        self.cache.attention(self.layer, q, out, cu_tokens=self.dcu if cu else None,
                             max_tokens=max(max(self.ns), 1) if max_tokens is None else max_tokens, window=window,
                             sinks=sinks, **kw)
        return out

    def check(self, out, window=0, sinks=0, weights=None, scale=None, least=0.0):
        """weights: what a weight may be off by, before the scores' error; least: what an
        output may be off by where all of a dimension's weight lies on tiny weights."""
        if weights is None:
            weights = 2.0 ** -11 if self.int8 else 2.0 ** -16
        n = int(self.cu[-1])
        ref, spread, serr = R.attention(self.q[:n].double().cpu().numpy(), self.keys, self.values, self.lens, self.cu,
                                        self.d ** -0.5 if scale is None else scale, window, sinks)
        got = out.double().cpu().numpy()
        tol = R.BF16_HALF * np.abs(ref) + (weights + 2.0 ** -20 + serr) * spread + 1e-30 + least
        err = np.abs(got[:n] - ref)
        assert np.isfinite(got[:n]).all()
        assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:5])
        assert (got[n:] == 7.0).all()                       # padding is left as it was
        return ref


SHAPES = [  # hq, hkv, d, page, int8
    (4, 2, 64, 16, False), (8, 1, 128, 32, False), (2, 2, 128, 16, False), (6, 2, 64, 64, False),
    (16, 1, 64, 128, False), (4, 2, 64, 16, True), (8, 1, 128, 64, True), (5, 1, 128, 128, False),
    (16, 1, 128, 16, True), (3, 1, 64, 32, True),
]
SPANS = [(0, 0), (1, 0), (7, 0), (16, 4), (40, 1), (33, 20), (1000, 5), (5, 1000)]


@pytest.mark.parametrize("shape", SHAPES)
def test_one_token_a_row_over_lengths(tsp, shape):
    hq, hkv, d, page, i8 = shape
    lens = [1, 0, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 511, 0, 640]
    c = Case(tsp, lens, [1] * len(lens), hq, hkv, d, page, i8, seed=1)
    out = c.run(cu=False)
    c.check(out)
    c.cache.check()
    empty = out[1].abs().sum() + out[15].abs().sum()
    assert float(empty) == 0.0


@pytest.mark.parametrize("window,sinks", SPANS)
@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1], SHAPES[5], SHAPES[6]])
def test_one_token_a_row_under_a_window(tsp, shape, window, sinks):
    hq, hkv, d, page, i8 = shape
    lens = [1, 5, 16, 40, 41, 57, 130, 333, 700]
    c = Case(tsp, lens, [1] * len(lens), hq, hkv, d, page, i8, seed=2)
    c.check(c.run(window, sinks), window, sinks)
    c.cache.check()


@pytest.mark.parametrize("shape", SHAPES)
def test_several_tokens_a_row(tsp, shape):
    """Draft tokens and short prompts in one ragged batch, with a row of no
    tokens, one with more tokens than positions, and padding behind the last."""
    hq, hkv, d, page, i8 = shape
    lens = [40, 3, 100, 17, 0, 260, 9]
    ns = [3, 5, 1, 0, 2, 40, 9]
    c = Case(tsp, lens, ns, hq, hkv, d, page, i8, seed=3, pad=5)
    c.check(c.run(), weights=2.0 ** -8)
    c.check(c.run(11, 3), 11, 3, weights=2.0 ** -8)
    c.cache.check()


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1], SHAPES[4], SHAPES[5], SHAPES[8]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4), (1, 0)])
def test_prompts(tsp, shape, window, sinks):
    hq, hkv, d, page, i8 = shape
    lens, ns = [150, 300, 64], [150, 129, 64]
    c = Case(tsp, lens, ns, hq, hkv, d, page, i8, seed=4)
    c.check(c.run(window, sinks), window, sinks, weights=2.0 ** -8)
    c.cache.check()


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_one_long_row_is_split_and_joined(tsp, d, i8):
    c = Case(tsp, [5003], [1], 4, 1, d, 16, i8, seed=5)
    c.check(c.run(cu=False))
    c.check(c.run(cu=False, window=4000, sinks=9), 4000, 9)
    c = Case(tsp, [5003], [17], 4, 1, d, 16, i8, seed=6)
    c.check(c.run(), weights=2.0 ** -8)


def test_many_rows_some_empty(tsp):
    r = np.random.default_rng(7)
    lens = [int(x) for x in np.where(r.random(700) < 0.3, 0, r.integers(1, 90, 700))]
    c = Case(tsp, lens, [1] * 700, 2, 1, 64, 16, seed=7)
    c.check(c.run(cu=False))


@pytest.mark.parametrize("i8", [False, True])
def test_large_scores_and_far_apart_values(tsp, i8):
    """Scores of several hundred: the running maximum does its work."""
    c = Case(tsp, [300, 77], [1, 1], 4, 2, 64, 16, i8, seed=8, amp=60.0)
    c.check(c.run(cu=False))
    for d in (64, 128):
        c = Case(tsp, [300, 77], [40, 30], 4, 2, d, 16, i8, seed=8, amp=60.0)
        c.check(c.run(), weights=2.0 ** -8)


@pytest.mark.parametrize("ns", [3, 30])
def test_what_a_token_does_not_see_has_no_influence(tsp, ns):
    """Infinities and NaN in keys and values of later tokens of the same call,
    and of positions that the window hides: only tokens that see them change."""
    import torch
    lens, n = [90], [ns]
    for bad_at, window, sinks in ((89, 0, 0), (90 - ns + 1, 0, 0), (20, 30, 4), (50, 25, 0)):
        c = Case(tsp, lens, n, 4, 2, 64, 16, seed=9)
        (kp, _), (vp, _) = c.cache.key_pool(), c.cache.value_pool()
        page, o = c.tables[0, bad_at // 16], bad_at % 16
        ref = c.run(window, sinks)
        for x in (float("nan"), float("inf"), -float("inf")):
            vp[0, page, :, o, :5] = x
            kp[0, page, :, o, 3] = x
            out = c.run(window, sinks)
            for i in range(ns):
                p = 90 - ns + i
                if R.sees(p, bad_at, window, sinks):
                    continue
                err = (out[i].float() - ref[i].float()).abs()
                assert torch.isfinite(out[i].float()).all(), (i, x, bad_at)
                # twice the rounding of the output and, for prompts, of the weights
                assert (err <= 2 * (2.0 ** -8 * ref[i].float().abs() + 2.0 ** -8 * 4)).all()
    c.cache.check()


def test_values_that_are_seen_and_not_finite(tsp):
    c = Case(tsp, [90], [30], 4, 2, 64, 16, seed=10)
    vp = c.cache.value_pool()[0]
    vp[0, c.tables[0, 0], 0, 5, 7] = float("inf")
    out = c.run().float()
    assert bool((out[:, :2, 7] == float("inf")).all())
    assert bool(out[:, :2, :7].isfinite().all()) and bool(out[:, 2:].isfinite().all())


def test_strides_other_than_the_dense_ones(tsp):
    import torch
    c = Case(tsp, [40, 70], [4, 30], 8, 2, 64, 16, seed=11)
    n = c.n_tokens
    q = torch.zeros((8, n + 2, 72), dtype=torch.bfloat16, device="cuda")[:, :n, :64].transpose(0, 1)
    q.copy_(c.q)
    buf = torch.full((n, 8, 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :, 1]
    c.run(q=q, out=out)
    c.check(out, weights=2.0 ** -8)
    assert bool((buf[:, :, 0] == 7).all()) and bool((buf[:, :, 2] == 7).all())


def test_second_layer_and_scale(tsp):
    c = Case(tsp, [40, 70], [1, 1], 8, 2, 64, 16, seed=12, layer=1, layers=3)
    c.check(c.run(scale=0.3), scale=0.3)


def test_bad_tables_are_recorded_and_skipped(tsp):
    """Page ids out of range, a missing page, a length beyond the table, token
    offsets out of order: the status says so, the other rows are right."""
    c = Case(tsp, [40, 70, 33], [1, 1, 1], 4, 2, 64, 16, seed=13)
    good = c.run().clone()
    c.cache.check()
    for bad in (1 << 30, -7, c.cache.pdesc.n_pages, -1):
        keep = int(c.cache.tables[1, 2])
        c.cache.tables[1, 2] = bad
        out = c.run()
        assert c.cache.status() == -8 and c.cache.status() == 0
        assert bool((out[0] == good[0]).all()) and bool((out[2] == good[2]).all())
        assert bool(out.float().isfinite().all())
        c.cache.tables[1, 2] = keep
    c.cache.lens[1] = 10 ** 6
    out = c.run()
    assert c.cache.status() == -8 and bool((out[0] == good[0]).all()) and bool((out[2] == good[2]).all())
    c.cache.lens[1] = 70
    for cu in ([0, 2, 1, 3], [0, 1, 5, 6], [-1, 1, 2, 3]):
        import torch
        c.dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        c.run(max_tokens=2)
        assert c.cache.status() == -8


def test_checks_of_the_binding(tsp):
    import torch
    c = Case(tsp, [40, 70], [1, 1], 4, 2, 64, 16, seed=14)
    a, q, out = c.cache, c.q, torch.empty_like(c.q)
    i32 = dict(dtype=torch.int32, device="cuda")
    for f in (lambda: a.attention(0, q.float(), out), lambda: a.attention(0, q.cpu(), out),
              lambda: a.attention(0, q[:, :, :32], out), lambda: a.attention(0, q, out[:, :2]),
              lambda: a.attention(0, q, out[:1]), lambda: a.attention(0, q[:1], out[:1]),
              lambda: a.attention(0, q, out, cu_tokens=c.dcu.long()), lambda: a.attention(0, q, out, cu_tokens=c.dcu[:2]),
              lambda: a.attention(1, q, out), lambda: a.resize(torch.zeros(3, **i32)),
              lambda: a.resize(torch.zeros(2, device="cuda")), lambda: a.fork(torch.zeros(2, dtype=torch.int32)),
              lambda: a.append(0, q, q), lambda: a.append(0, q[:, :2], q[:1, :2]),
              lambda: tsp.PagedKV(tsp.ModelDesc(n_layers=1, n_kv_heads=1, head_dim=64, max_pos=16), n_pages=4,
                                  k=torch.zeros(8, device="cuda"))):
        with pytest.raises(tsp.TilesError) as e:
            f()
        assert e.value.status == -1
    with pytest.raises(tsp.TilesError) as e:
        a.attention(0, q, out, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -5


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("d,hkv,page,i8", [(64, 2, 16, False), (128, 3, 32, False), (64, 1, 64, True), (128, 8, 16, True),
                                           (64, 5, 128, True)])
def test_append_writes_rows_where_they_belong_and_nothing_else(tsp, d, hkv, page, i8):
    import torch
    lens, ns = [40, 3, 100, 17, 0, 260, 9], [3, 5, 1, 0, 2, 40, 9]
    c = Case(tsp, lens, ns, hkv, hkv, d, page, i8, seed=20, layer=1, layers=2, pad=3)
    cache, r = c.cache, np.random.default_rng(21)
    if i8:
        shift = torch.from_numpy(r.standard_normal((2, hkv, d)).astype(np.float32)).cuda()
        cache = tsp.PagedKV(tsp.ModelDesc(n_layers=2, n_kv_heads=hkv, head_dim=d, max_pos=cache.pdesc.table_width * page),
                            n_pages=cache.pdesc.n_pages, page_size=page, n_seqs=len(lens), kv_format=tsp.KV_INT8,
                            k_shift=shift, k=cache.k, v=cache.v, tables=cache.tables, lens=cache.lens)
    k, v = (bf16(r.standard_normal((hkv, c.n_tokens, d))).cuda().transpose(0, 1) for _ in range(2))
    v[4] = 0.0                                                        # an all-zero row: scale 0, codes 0
    before = [t.clone() if t is not None else None for t in (*cache.key_pool(), *cache.value_pool())]
    want = [None if t is None else t.cpu().clone() for t in before]
    for i, (s, p) in enumerate(R.places(lens, c.cu)):
        if p < 0:
            continue
        at = (1, int(c.tables[s, p // page]), slice(None), p % page)
        if not i8:
            want[0][at], want[2][at] = k[i].cpu(), v[i].cpu()
        else:
            kq, ks = quantized(k[i].float().cpu().numpy() - shift[1].cpu().numpy())
            vq, vs = quantized(v[i].float().cpu().numpy())
            want[0][at], want[1][at] = torch.from_numpy(kq), torch.from_numpy(ks)
            want[2][at], want[3][at] = torch.from_numpy(vq), torch.from_numpy(vs)
    cache.append(1, k, v, cu_tokens=c.dcu)
    cache.check()
    for got, w in zip((*cache.key_pool(), *cache.value_pool()), want):
        if w is not None:
            bits = torch.int8 if w.dtype == torch.int8 else torch.int16 if w.dtype == torch.bfloat16 else torch.int32
            assert torch.equal(got.cpu().view(bits), w.view(bits))


@pytest.mark.parametrize("n_seqs", [1, 31, 32, 33, 1000, 1100])
def test_append_finds_each_tokens_row(tsp, n_seqs):
    import torch
    r = np.random.default_rng(n_seqs)
    ns = r.integers(0, 4, n_seqs)
    ns[-1] = 1
    cache = tsp.PagedKV(tsp.ModelDesc(n_layers=1, n_kv_heads=1, head_dim=64, max_pos=16), n_pages=n_seqs, n_seqs=n_seqs)
    cache.resize(torch.from_numpy(ns.astype(np.int32)).cuda())
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    n = int(cu[-1])
    x = (torch.arange(n, device="cuda") % 256).to(torch.bfloat16)[:, None, None].expand(n, 1, 64).contiguous()
    cache.append(0, x, x, cu_tokens=torch.from_numpy(cu).cuda())
    cache.check()
    t, pool = cache.tables.cpu().numpy(), cache.key_pool()[0].float().cpu().numpy()
    for i, (s, p) in enumerate(R.places(ns, cu)):
        assert (pool[0, t[s, 0], 0, p] == i % 256).all()


def test_dense_cache_rows_move_into_pages(tsp):
    """A dense cache [n_kv][max_pos][d] by its strides."""
    import torch
    dense = bf16(np.random.default_rng(22).standard_normal((2, 50, 64))).cuda()
    cache = tsp.PagedKV(tsp.ModelDesc(n_layers=1, n_kv_heads=2, head_dim=64, max_pos=64), n_pages=5)
    cache.resize(torch.tensor([37], dtype=torch.int32, device="cuda"))
    rows = dense.transpose(0, 1)[:37]
    cache.append(0, rows, rows, cu_tokens=torch.tensor([0, 37], dtype=torch.int32, device="cuda"))
    cache.check()
    t = cache.tables[0, :3].long()
    got = cache.key_pool()[0][0, t].permute(1, 0, 2, 3).reshape(2, 48, 64)[:, :37]
    assert torch.equal(got, dense[:, :37])


# ------------------------------------------------------------------ pages
def _cache_and_model(tsp, n_pages, n_seqs, max_len, page=16, layers=2, hkv=2, d=64, i8=False):
    import torch
    desc = tsp.ModelDesc(n_layers=layers, n_kv_heads=hkv, head_dim=d, max_pos=max_len)
    cache = tsp.PagedKV(desc, n_pages=n_pages, page_size=page, n_seqs=n_seqs, kv_format=tsp.KV_INT8 if i8 else tsp.KV_BF16)
    g = torch.Generator(device="cuda").manual_seed(3)
    cache.k.random_(0, 100, generator=g)
    cache.v.random_(0, 100, generator=g)
    return cache, R.Pages(n_pages, n_seqs, cache.pdesc.table_width, page)


def _pools(cache):
    import torch
    return [t.clone().view(torch.int8 if t.dtype == torch.int8 else torch.int16 if t.dtype == torch.bfloat16 else torch.int32)
            for t in (*cache.key_pool(), *cache.value_pool()) if t is not None]


def _same(cache, model):
    assert cache.tables.cpu().tolist() == model.tables
    assert cache.lens.cpu().tolist() == model.lens
    assert cache.refs.cpu().tolist() == model.refs


def _moved(before, after, copies):
    import torch
    for b, a in zip(before, after):
        for src, dst in copies:
            b[:, dst] = b[:, src]
        assert torch.equal(b, a)


@pytest.mark.parametrize("seed,page,i8", [(0, 16, False), (1, 32, False), (2, 16, True), (3, 128, False), (4, 64, True)])
def test_pages_life_as_a_sequential_program_has_it(tsp, seed, page, i8):
    """Random resizes, forks, trims and compactions; tables, lengths, reference
    counts and the pools' bytes after each."""
    import torch
    r = np.random.default_rng(seed)
    n_seqs, max_len, n_pages = 12, 9 * page - 3, 60
    cache, m = _cache_and_model(tsp, n_pages, n_seqs, max_len, page, i8=i8)
    trimmed, failed, forked = False, 0, 0
    for step in range(60):
        before = _pools(cache)
        what = r.choice(["grow", "grow", "end", "mixed", "fork", "fork", "compact", "trim"])
        if what in ("grow", "end", "mixed"):
            new = np.array(m.lens)
            for s in range(n_seqs):
                x = r.random()
                if what != "grow" and x < 0.3:
                    new[s] = 0 if trimmed or x < 0.2 else r.integers(0, m.lens[s] + 1)
                elif what != "end" and x < 0.8:
                    new[s] = min(m.lens[s] + r.choice([1, 1, 3, page, 40]), max_len)
                else:
                    new[s] = -1
            ok = m.resize([int(x) for x in new])
            cache.resize(torch.from_numpy(new.astype(np.int32)).cuda())
            assert cache.status() == (0 if ok else -5), step
            failed += not ok
        elif what == "fork":
            src = [-1] * n_seqs
            for s in range(n_seqs):
                if m.lens[s] == 0 and r.random() < 0.7:
                    src[s] = int(r.integers(-1, n_seqs))
            src[int(r.integers(n_seqs))] = int(r.integers(-1, n_seqs + 1))   # a bad one now and then
            ok = m.fork(src)
            m.copies = []
            cache.fork(torch.tensor(src, dtype=torch.int32, device="cuda"))
            assert cache.status() == (0 if ok else -8), step
            forked += 1
        elif what == "compact":
            m.compact()
            cache.compact()
        else:
            w, k = int(r.integers(1, 4 * page)), int(r.choice([0, 3, page, page + 1]))
            m.trim(w, k)
            m.copies = []
            trimmed = True
            cache.trim(w, k)
        cache.check()
        _same(cache, m)
        _moved(before, _pools(cache), m.copies)
    assert forked and len(set(m.lens)) > 1


def test_too_few_pages_change_nothing_but_what_shrinks(tsp):
    import torch
    cache, m = _cache_and_model(tsp, 10, 4, 160)
    lens = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for new, ok in (((30, 40, 16, 0), True), ((160, -1, 0, 20), False), ((31, 41, 0, 16), True), ((-1, -1, -1, 160), False),
                    ((0, 0, 0, 160), True)):
        assert m.resize(list(new)) == ok
        cache.resize(lens(*new))
        assert cache.status() == (0 if ok else -5)
        _same(cache, m)
    cache.resize(lens(-1, 161, -1, -1))                                 # longer than a row can be
    assert cache.status() == -8
    _same(cache, m)
    cache.reset()
    assert cache.lens.sum() == 0 and cache.refs.sum() == 0 and bool((cache.tables == -1).all())


def test_forked_rows_part_when_they_grow(tsp):
    """Every holder writes: the lowest keeps the page. One does not: all writers copy."""
    import torch
    t = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for grow in ((21, 21, 21, 21), (-1, 21, 22, 40), (21, -1, 21, 21), (21, -1, -1, -1)):
        cache, m = _cache_and_model(tsp, 30, 4, 160)
        cache.resize(t(20, -1, -1, -1))
        cache.fork(t(-1, 0, 0, 0))
        m.resize([20, -1, -1, -1])
        m.fork([-1, 0, 0, 0])
        _same(cache, m)
        before = _pools(cache)
        cache.resize(t(*grow))
        m.resize(list(grow))
        _same(cache, m)
        _moved(before, _pools(cache), m.copies)
        cache.check()


@pytest.mark.parametrize("n_pages", [1, 4095, 4097, 20000])
def test_large_and_odd_pools(tsp, n_pages):
    import torch
    r = np.random.default_rng(n_pages)
    n_seqs = min(n_pages, 1500)
    cache, m = _cache_and_model(tsp, n_pages, n_seqs, 16 * 12, layers=1, hkv=1)
    lens = r.integers(0, 16 * 12, n_seqs)
    while sum(-(-int(n) // 16) for n in lens) > n_pages:
        lens //= 2
    for new in (lens, np.where(r.random(n_seqs) < 0.5, 0, -1)):
        cache.resize(torch.from_numpy(new.astype(np.int32)).cuda())
        assert m.resize([int(x) for x in new])
        _same(cache, m)
    before = _pools(cache)
    cache.compact()
    m.compact()
    _same(cache, m)
    _moved(before, _pools(cache), m.copies)


# ------------------------------------------------------------------ together
def _serve(tsp, cache, dense, steps, prompt, children, stream=None):
    """A prompt in row 0, forked to `children` further rows; then every row takes
    one token a step. dense: each row's K, V rows and queries by position.
    Returns the outputs."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = children + 1
    outs = []
    cache.resize(torch.tensor([prompt] + [-1] * children, **i32), stream=stream)
    cu = torch.tensor([0] + [prompt] * rows, **i32)
    k, v, q = dense
    cache.append(0, k[0, :prompt], v[0, :prompt], cu_tokens=cu, stream=stream)
    out = torch.empty_like(q[0, :prompt])
    cache.attention(0, q[0, :prompt], out, cu_tokens=cu, max_tokens=prompt, stream=stream)
    outs.append(out)
    cache.fork(torch.tensor([-1] + [0] * children, **i32), stream=stream)
    for i in range(steps):
        cache.resize(torch.full((rows,), prompt + i + 1, **i32), stream=stream)
        cache.append(0, k[:, prompt + i], v[:, prompt + i], stream=stream)
        out = torch.empty_like(q[:, prompt + i])
        cache.attention(0, q[:, prompt + i], out, stream=stream)
        outs.append(out)
    return outs


def _dense(rows, n, hq, hkv, d, prompt, seed):
    r = np.random.default_rng(seed)
    k, v, q = (bf16(r.standard_normal((rows, n, h, d))).cuda() for h in (hkv, hkv, hq))
    for t in (k, v, q):
        t[:, :prompt] = t[:1, :prompt]                     # the prompt is shared
    return k, v, q


def _check_serve(outs, dense, prompt, d):
    k, v, q = (t.double().cpu().numpy() for t in dense)
    rows = k.shape[0]

    def ok(out, s, p0, p1, weights):
        ref, spread, serr = R.attention(q[s, p0:p1], [k[s, :p1]], [v[s, :p1]], [p1], [0, p1 - p0], d ** -0.5)
        err = np.abs(out.double().cpu().numpy() - ref)
        assert (err <= R.BF16_HALF * np.abs(ref) + (weights + 2.0 ** -20 + serr) * spread).all()
    ok(outs[0], 0, 0, prompt, 2.0 ** -8)
    for i, out in enumerate(outs[1:]):
        for s in range(rows):
            ok(out[s:s + 1], s, prompt + i, prompt + i + 1, 2.0 ** -16)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
def test_prompt_fork_and_decode(tsp, d, page):
    prompt, steps, children = 45, 20, 3
    cache, _ = _cache_and_model(tsp, 40, children + 1, 96, page, layers=1, d=d)
    dense = _dense(children + 1, prompt + steps, 4, 2, d, prompt, 30)
    outs = _serve(tsp, cache, dense, steps, prompt, children)
    cache.check()
    _check_serve(outs, dense, prompt, d)
    # the shared prompt pages are held by all, each row's own by one
    assert cache.refs.max() == children + 1 and int(cache.refs.sum()) == (children + 1) * -(-(prompt + steps) // page)


def test_the_same_on_another_stream(tsp):
    import torch
    cache, _ = _cache_and_model(tsp, 40, 4, 96, layers=1)
    dense = _dense(4, 65, 4, 2, 64, 45, 31)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        outs = _serve(tsp, cache, dense, 20, 45, 3)
    st.synchronize()
    _check_serve(outs, dense, 45, 64)
    cache.reset()
    torch.cuda.synchronize()
    outs = _serve(tsp, cache, dense, 20, 45, 3, stream=torch.cuda.current_stream())
    _check_serve(outs, dense, 45, 64)


def test_a_captured_step_replayed(tsp):
    """resize, append and attention in one graph; its inputs change between replays."""
    import torch
    cache, _ = _cache_and_model(tsp, 60, 3, 128, layers=1)
    k, v, q = _dense(3, 100, 4, 2, 64, 0, 32)
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    sk, sv, sq = (torch.zeros_like(t[:, 0]) for t in (k, v, q))
    out = torch.empty_like(sq)

    def step():
        cache.resize(new)
        cache.append(0, sk, sv)
        cache.attention(0, sq, out)
    step()                                                  # lengths stay 0: nothing happens
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    outs = []
    for i in range(100):
        new.fill_(i + 1)
        sk.copy_(k[:, i]), sv.copy_(v[:, i]), sq.copy_(q[:, i])
        g.replay()
        outs.append(out.clone())
    cache.check()
    hk, hv, hq = (t.double().cpu().numpy() for t in (k, v, q))
    for i, s in itertools.product((0, 1, 15, 16, 17, 63, 99), range(3)):
        ref, spread, serr = R.attention(hq[s, i:i + 1], [hk[s, :i + 1]], [hv[s, :i + 1]], [i + 1], [0, 1], 0.125)
        err = np.abs(outs[i][s:s + 1].double().cpu().numpy() - ref)
        assert (err <= R.BF16_HALF * np.abs(ref) + (2.0 ** -16 + 2.0 ** -20 + serr) * spread).all(), (i, s)


def test_repeated_calls_are_bitwise_equal(tsp):
    import torch
    c = Case(tsp, [3000, 40, 700], [1, 1, 1], 4, 2, 64, 16, seed=33)
    a = c.run()
    assert all(torch.equal(a, c.run()) for _ in range(5))
    c = Case(tsp, [2000, 40, 700], [300, 40, 99], 4, 2, 64, 16, seed=34)
    a = c.run()
    assert all(torch.equal(a, c.run()) for _ in range(5))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_many_runs_are_bitwise_equal(tsp, d, i8):
    """Split, joined and whole pieces, 200 times, with a cold L2 every other time: a
    missing wait between the kernel's roles shows as a bit that changes."""
    import torch
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for lens, ns in (([5003], [17]), ([2000, 40, 700], [300, 40, 99]), ([900, 3000], [1, 1])):
        c = Case(tsp, lens, ns, 4, 1, d, 16, i8, seed=35)
        first = c.run()
        for i in range(200):
            if i % 2:
                flush.fill_(i)
            assert torch.equal(first, c.run()), i


# ------------------------------------------------------------------ windows, pages given back
@pytest.mark.parametrize("d,i8", [(64, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_attention_after_a_trim_needs_no_page_that_is_gone(tsp, d, i8, n):
    """Pages of 16 in units of up to 128 positions: the windows' first and the sinks'
    last unit reach into pages that the trim gave back."""
    import torch
    for window, sinks in ((20, 4), (33, 0), (100, 17), (49, 16)):
        lens, ns = [300, 47, 130, 301], [min(n, k) for k in (300, 47, 130, 301)]
        c = Case(tsp, lens, ns, 4, 2, d, 16, i8, seed=40)
        # what the tokens of this call see: the trim takes the rows without them
        c.cache.lens -= torch.tensor(ns, dtype=torch.int32, device="cuda")
        before = int((c.cache.tables >= 0).sum())
        c.cache.trim(window, sinks)
        c.cache.lens += torch.tensor(ns, dtype=torch.int32, device="cuda")
        assert int((c.cache.tables >= 0).sum()) < before
        c.check(c.run(window, sinks), window, sinks, weights=2.0 ** -8 if n > 2 else None)
        c.cache.check()


def test_extreme_windows_and_sinks(tsp):
    big = 2 ** 31 - 1
    for ns in ([1, 1], [9, 30]):
        c = Case(tsp, [40, 70], ns, 4, 2, 64, 16, seed=41)
        whole = c.run()
        for w, k in ((big, 0), (big, big), (10, big), (80, 3)):
            assert bool((c.run(w, k) == whole).all()), (w, k)
        c.check(c.run(1, 0), 1, 0, weights=2.0 ** -8)
    c.cache.trim(big, 0)
    c.cache.trim(1, big)
    assert int((c.cache.tables >= 0).sum()) == 3 + 5
    c.cache.check()


def test_a_captured_prompt_replayed(tsp):
    """The tensor-core form in a graph, twice in a row and beside an eager call."""
    import torch
    c = Case(tsp, [500, 90], [200, 90], 4, 2, 128, 16, seed=42)
    first = c.run()
    out = torch.zeros_like(c.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        other = c.run()
        assert torch.equal(out, first) and torch.equal(other, first)
    c.q.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    c.check(out, weights=2.0 ** -8)


def test_two_caches_on_two_streams_at_once(tsp):
    import torch
    a = Case(tsp, [3000, 2000], [64, 100], 4, 2, 64, 16, seed=43)
    b = Case(tsp, [5000, 100, 900], [1, 1, 1], 4, 2, 128, 32, seed=44)
    ra, rb = a.run(), b.run()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        with torch.cuda.stream(sa):
            oa = a.run()
        ob = torch.full_like(rb, 7.0)
        sb.wait_stream(torch.cuda.current_stream())
        b.run(out=ob, stream=sb)
        outs.append((oa, ob))
    torch.cuda.synchronize()
    assert all(torch.equal(x, ra) and torch.equal(y, rb) for x, y in outs)


@pytest.mark.parametrize("n_tokens", [1, 2])
def test_the_smallest_calls(tsp, n_tokens):
    c = Case(tsp, [n_tokens], [n_tokens], 1, 1, 64, 16, seed=45)
    c.check(c.run())
    c = Case(tsp, [n_tokens], [n_tokens], 16, 1, 128, 128, True, seed=46)
    c.check(c.run(), weights=2.0 ** -8)


@pytest.mark.parametrize("page,growth", [(16, 2000), (64, 500)])
def test_a_resize_of_more_slots_than_threads(tsp, page, growth):
    """Thousands of pages at once, shared ones among them, against the sequential program."""
    import torch
    n = 40
    cache, m = _cache_and_model(tsp, 40 * (growth // page + 4), n, growth + 200, page, layers=1, hkv=1)
    for new in ([37] * (n // 2) + [-1] * (n // 2), None, [growth + (s % 7) for s in range(n)], [s * 11 for s in range(n)],
                [growth] * n):
        if new is None:
            src = [-1] * (n // 2) + list(range(n // 2))
            m.fork(src)
            m.copies = []
            cache.fork(torch.tensor(src, dtype=torch.int32, device="cuda"))
        else:
            before = _pools(cache)
            assert m.resize(list(new))
            cache.resize(torch.tensor(new, dtype=torch.int32, device="cuda"))
            _moved(before, _pools(cache), m.copies)
        cache.check()
        _same(cache, m)


def test_more_rows_than_shared_memory_holds(tsp):
    import torch
    r = np.random.default_rng(50)
    n = 2500
    cache, m = _cache_and_model(tsp, 6000, n, 64, layers=1, hkv=1)
    for _ in range(3):
        new = [int(x) for x in r.integers(-1, 30, n)]
        assert m.resize(new)
        cache.resize(torch.tensor(new, dtype=torch.int32, device="cuda"))
        cache.check()
        _same(cache, m)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_climb_by_hundreds(tsp, d, i8):
    """Keys that grow along the sequence, so that each block's scores lie far above the
    last one's (beyond what FP32 holds relative to the first): prompts, single tokens in a
    call with prompts, and single tokens alone; and keys that all but one of shrink."""
    import torch
    for seed, factor in ((60, lambda t, n: 1.0 + 120.0 * t / n), (61, lambda t, n: 120.0 * (t == n // 3) + 0.01)):
        lens, ns = [700, 513, 90], [30, 1, 90]
        c = Case(tsp, lens, ns, 4, 2, d, 16, i8, seed=seed)
        (kp, ks), _ = c.cache.key_pool(), c.cache.value_pool()
        for s, n in enumerate(lens):
            for t in range(n):
                f = factor(t, n)
                at = (0, int(c.tables[s, t // 16]), slice(None), t % 16)
                if i8:
                    new = (ks[at].double() * f).float()
                    ks[at] = new
                    c.keys[s][t] = kp[at].double().cpu().numpy() * new.double().cpu().numpy()[:, None]
                else:
                    kp[at] = (kp[at].float() * f).to(torch.bfloat16)
                    c.keys[s][t] = kp[at].double().cpu().numpy()
        c.check(c.run(), weights=2.0 ** -8)
        c.check(c.run(300, 3), 300, 3, weights=2.0 ** -8)
        c.cache.check()


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_rise_by_any_power_of_two(tsp, d, i8):
    """One position far above all before it, by up to beyond what FP32's exponent holds, whose
    value is zero in the first half of the dimensions: there a later position 2^-20 of it
    shows. Short rows, which several blocks may share, and enough of them that most do not."""
    import torch
    rises = [0.0, 60.0, 100.0, 125.0, 126.0, 126.5, 127.0, 127.5, 128.0, 150.0, 252.0, 254.0, 500.0]
    for copies, cols in ((1, (0, 130, 300, 511)), (4, (130, 300))):
        lens, peaks = [], []
        for x in rises:
            for col in cols:
                lens += [640] * copies
                peaks += [(x, col)] * copies
        c = Case(tsp, lens, [2] * len(lens), 4, 4, d, 64, i8, seed=62)
        (kp, ks), (vp, vs) = c.cache.key_pool(), c.cache.value_pool()
        c.q.zero_()
        c.q[:, :, 0] = 1.0
        for s, (x, col) in enumerate(peaks):
            k0 = np.zeros(640)
            k0[col], k0[col + 100] = x, x - 20.0
            for t in range(640):
                c.keys[s][t, :, 0] = k0[t]
            c.values[s][col, :, : d // 2] = 0.0
            pages = torch.from_numpy(c.tables[s][:10]).cuda().long()
            at = torch.from_numpy(k0).cuda().view(10, 1, 64)
            if i8:
                kp[0, pages, :, :, 0] = torch.where(at == 0, 0, 127).to(torch.int8).expand(10, 4, 64)
                ks[0, pages] = (at / 127).float().expand(10, 4, 64)
                c.keys[s][:, :, 0] = (k0 / 127).astype(np.float32).astype(np.float64)[:, None] * 127
            else:
                kp[0, pages, :, :, 0] = at.to(torch.bfloat16).expand(10, 4, 64)
            vp[0, int(pages[col // 64]), :, col % 64, : d // 2] = 0
        # The single tokens' kernel holds a weight times its value's scale as an FP16 number of
        # steps of 2^-24, where the largest weight times a power of two below twice the largest
        # scale is 2^12: off by half a step, 2^-37 of those. Over 640 codes of 127 at most, and
        # scales of max |v| / 127: 640 * 2^-36 * max |v|, with a sum of weights of 1 or more.
        least = 640 * 2.0 ** -36 * max(np.abs(v).max() for v in c.values) if i8 else 0.0
        c.check(c.run(scale=float(np.log(2.0)), max_tokens=2), weights=2.0 ** -8, scale=np.log(2.0), least=least)
        c.check(c.run(scale=float(np.log(2.0)), max_tokens=20), weights=2.0 ** -8, scale=np.log(2.0))
        c.cache.check()


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_a_tile_of_rows_beside_an_infinity_in_a_long_cache(tsp, d, i8):
    """An infinite value that only the last token sees: the other 254 rows of its tiles are
    computed again over 32,768 positions, well within the limit of the waits."""
    import torch
    c = Case(tsp, [32768], [128], 2, 1, d, 64, i8, seed=63)
    (vp, vs) = c.cache.value_pool()
    at = (0, int(c.tables[0, 511]), 0, 63)
    if i8:
        vs[at] = float("inf")
        vp[at] = 127
    else:
        vp[at] = float("inf")
    out = c.run()
    c.cache.check()
    assert not torch.isfinite(out[127].float()).any()
    got = out.double().cpu().numpy()
    assert np.isfinite(got[:127]).all()
    for tok in (0, 60, 126):                                # at position 32,640 + tok
        ref, spread, serr = R.attention(c.q.double().cpu().numpy()[tok: tok + 1], [c.keys[0][:32641 + tok]],
                                        [c.values[0][:32641 + tok]], [32641 + tok], np.array([0, 1]), d ** -0.5)
        tol = R.BF16_HALF * np.abs(ref) + (2.0 ** -8 + 2.0 ** -20 + serr) * spread + 1e-30
        assert (np.abs(got[tok] - ref[0]) <= tol[0]).all(), tok


def test_one_cache_captured_and_on_two_streams(tsp):
    """Attention reads a cache only, so calls on it may overlap: eager ones on two streams
    and a replayed graph on a third have workspaces of their own (none is given here)."""
    import torch
    for ns in ([1] * 6, [40, 9, 30, 1, 0, 25]):
        c = Case(tsp, [700, 40, 1500, 333, 64, 2000], ns, 8, 2, 64, 16, seed=64)
        want = c.run()
        c.check(want, weights=2.0 ** -8)
        q2 = c.q.flip(0).contiguous()
        want2 = c.run(q=q2)
        streams = [torch.cuda.Stream() for _ in range(3)]
        graph, held = torch.cuda.CUDAGraph(), torch.empty_like(want)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=streams[2]):
            c.run(out=held)
        outs = [torch.empty_like(want) for _ in range(2)]
        for _ in range(20):
            held.zero_()
            torch.cuda.synchronize()
            for _ in range(4):
                with torch.cuda.stream(streams[2]):
                    graph.replay()
                for k in range(2):
                    with torch.cuda.stream(streams[k]):
                        c.run(out=outs[k], q=(c.q, q2)[k])
            torch.cuda.synchronize()
            assert torch.equal(held, want) and torch.equal(outs[0], want) and torch.equal(outs[1], want2)
        # a larger need on the same stream, then the small one again
        c.run(max_tokens=40)
        assert torch.equal(c.run(), want)
        assert len(c.cache._ws) <= 3
        c.cache.check()


@pytest.mark.parametrize("i8", [False, True])
def test_pages_behind_four_billion_elements(tsp, i8):
    """The pool's last pages, whose offsets pass 32 bits: taken, written, read by both kinds
    of attention, copied on write, and moved to the front."""
    import torch
    P, hkv, d, page, lens = 34000, 8, 128, 128, [300, 131]
    desc = tsp.ModelDesc(n_layers=1, n_q_heads=2 * hkv, n_kv_heads=hkv, head_dim=d, max_pos=512)
    c = tsp.PagedKV(desc, n_pages=P, page_size=page, n_seqs=3, kv_format=tsp.KV_INT8 if i8 else tsp.KV_BF16)
    assert (P - 40) * hkv * page * d > 2 ** 32
    c.refs[:P - 40] = 1                                     # so that only the last pages are free
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    c.resize(dev(lens + [0]))
    n = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn((n, hkv, d), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    c.append(0, k, v, cu_tokens=dev([0, lens[0], n, n]))
    assert int(c.tables.max()) < P and int(c.tables[c.tables >= 0].min()) >= P - 40
    q = torch.randn((40, 2 * hkv, d), device="cuda", generator=g).to(torch.bfloat16)
    out1, out2 = torch.zeros_like(q[:3]), torch.zeros_like(q)
    c.attention(0, q[:3], out1)
    c.attention(0, q, out2, cu_tokens=dev([0, 30, 40, 40]), max_tokens=30)
    kk, vv = k.double().cpu().numpy(), v.double().cpu().numpy()
    if i8:
        (kc, ks), (vc, vs) = quantized(k.float().cpu().numpy()), quantized(v.float().cpu().numpy())
        kk, vv = kc * ks[..., None].astype(np.float64), vc * vs[..., None].astype(np.float64)
    keys, values = [kk[:300], kk[300:]], [vv[:300], vv[300:]]
    qd = q.double().cpu().numpy()
    for out, cu, w in ((out1, [0, 1, 2], 2.0 ** -11 if i8 else 2.0 ** -16), (out2, [0, 30, 40], 2.0 ** -8)):
        ref, spread, serr = R.attention(qd[:cu[-1]], keys, values, lens, np.array(cu), d ** -0.5)
        err = np.abs(out.double().cpu().numpy()[:cu[-1]] - ref)
        assert (err <= R.BF16_HALF * np.abs(ref) + (w + 2.0 ** -20 + serr) * spread).all()
    c.fork(dev([-1, -1, 0]))
    c.resize(dev([301, -1, 301]))                           # one of the two copies the page it writes
    c.append(0, k[:2], v[:2], cu_tokens=dev([0, 1, 1, 2]))
    (kp, _), _ = c.key_pool(), c.value_pool()
    a, b = int(c.tables[0, 2]), int(c.tables[2, 2])
    assert a != b and min(a, b) >= P - 40 and torch.equal(kp[0, a, :, :44], kp[0, b, :, :44])
    before = torch.zeros_like(q[:3])
    c.attention(0, q[:3], before)
    c.refs[:P - 40] = 0
    c.compact()
    assert int(c.tables.max()) < 40
    after = torch.zeros_like(before)
    c.attention(0, q[:3], after)
    assert torch.equal(before, after)
    c.check()
