"""The paged KV cache without a GPU: layout, and every refusal that is decided
on the host (before any CUDA call)."""
import ctypes

import pytest

import tile_scheduled_persistent_gb300 as tsp

OK, INVALID, UNSUPPORTED = 0, -1, -2


@pytest.fixture(scope="module", autouse=True)
def built():
    tsp.build()


def _desc(**kw):
    d = dict(n_layers=2, n_kv_heads=2, head_dim=64, page_size=16, n_pages=10, n_seqs=3, table_width=5,
             kv_format=tsp.KV_BF16)
    d.update(kw)
    return tsp.PagedDesc(**d)


def test_layout_bf16_and_int8():
    rows = 2 * 10 * 2 * 16
    lay = tsp.paged_layout(_desc())
    assert lay["k_bytes"] == lay["v_bytes"] == rows * 64 * 2 and lay["k_scale_off"] == lay["v_scale_off"] == 0
    assert lay["state_bytes"] % 4 == 0 and lay["state_bytes"] >= 4 * (16 + 10)
    lay = tsp.paged_layout(_desc(kv_format=tsp.KV_INT8, n_pages=3, n_kv_heads=1, n_layers=1))
    assert lay["k_scale_off"] % 256 == 0 and lay["k_scale_off"] >= 3 * 16 * 64
    assert lay["k_bytes"] == lay["k_scale_off"] + 3 * 16 * 4


@pytest.mark.parametrize("bad,status", [
    (dict(n_layers=0), INVALID), (dict(n_kv_heads=0), INVALID), (dict(n_pages=0), INVALID), (dict(n_seqs=-1), INVALID),
    (dict(table_width=0), INVALID), (dict(page_size=0), INVALID), (dict(kv_format=2), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
    (dict(n_pages=1 << 30), UNSUPPORTED), (dict(table_width=1 << 28), UNSUPPORTED),
])
def test_descriptions_that_are_refused(bad, status):
    with pytest.raises(tsp.TilesError) as e:
        tsp.paged_layout(_desc(**bad))
    assert e.value.status == status


# Addresses that are never read: every call below is refused before a CUDA call.
FAKE = 1 << 20


def _view(**kw):
    v = dict(desc=_desc(), k=FAKE, v=FAKE, tables=FAKE, lens=FAKE, state=FAKE, k_shift=None)
    v.update(kw)
    return tsp.PagedCacheView(**v)


def _calls(view):
    """Every call of a cache with otherwise fine arguments."""
    L, r = tsp.lib(), ctypes.byref(view)
    return {
        "resize": lambda: L.tiles_paged_resize(r, FAKE, None), "fork": lambda: L.tiles_paged_fork(r, FAKE, None),
        "trim": lambda: L.tiles_paged_trim(r, 4, 0, None), "compact": lambda: L.tiles_paged_compact(r, None),
        "reset": lambda: L.tiles_paged_reset(r, None), "status": lambda: L.tiles_paged_status(r, None),
        "append": lambda: L.tiles_paged_append(r, 0, FAKE, 128, 64, FAKE, 128, 64, None, 3, None),
        "attention": lambda: _attention(view),
    }


def _attention(view=None, layer=0, hq=4, q=FAKE, q_t=256, q_h=64, out=FAKE, o_t=256, o_h=64, cu=FAKE, n=3, mx=1,
               scale=0.125, window=0, sinks=0, ws=FAKE, ws_bytes=1 << 40):
    view = _view() if view is None else view
    return tsp.lib().tiles_paged_attention(ctypes.byref(view), layer, hq, q, q_t, q_h, out, o_t, o_h, cu, n, mx, scale,
                                           window, sinks, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(tables=None), dict(lens=None), dict(state=None),
                                 dict(k=FAKE + 8), dict(v=FAKE + 2), dict(tables=FAKE + 1), dict(lens=FAKE + 2),
                                 dict(state=FAKE + 4), dict(k_shift=FAKE)])      # k_shift: INT8 caches only
def test_caches_that_are_refused_by_every_call(bad):
    for name, call in _calls(_view(**bad)).items():
        assert call() == INVALID, name
    for name, call in _calls(_view(desc=_desc(head_dim=80), **{})).items():
        assert call() == UNSUPPORTED, name


@pytest.mark.parametrize("bad,status", [
    (dict(layer=-1), INVALID), (dict(layer=2), INVALID), (dict(hq=0), INVALID), (dict(hq=3), INVALID),
    (dict(hq=34), UNSUPPORTED), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q=FAKE + 2), INVALID),
    (dict(out=FAKE + 8), INVALID), (dict(q_t=250), INVALID), (dict(q_h=4), INVALID), (dict(o_t=1), INVALID),
    (dict(o_h=63), INVALID), (dict(cu=FAKE + 2), INVALID), (dict(cu=None, n=4), INVALID), (dict(n=-1), INVALID),
    (dict(mx=0), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(ws=None), INVALID),
    (dict(o_t=0), INVALID), (dict(o_h=56), INVALID),                              # rows of out that overlap
    (dict(ws=FAKE + 4), INVALID), (dict(n=0), OK),                                # nothing to do: no CUDA call either
])
def test_attention_arguments(bad, status):
    assert _attention(**bad) == status


@pytest.mark.parametrize("bad", [dict(layer=2), dict(layer=-1), dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(kt=4),
                                 dict(kh=1), dict(vt=12), dict(vh=9), dict(n=-1), dict(cu=None, n=2), dict(cu=FAKE + 1)])
def test_append_arguments(bad):
    a = dict(layer=0, k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, cu=FAKE, n=3)
    a.update(bad)
    assert tsp.lib().tiles_paged_append(ctypes.byref(_view()), a["layer"], a["k"], a["kt"], a["kh"], a["v"], a["vt"],
                                        a["vh"], a["cu"], a["n"], None) == INVALID


def test_page_call_arguments():
    L, r = tsp.lib(), ctypes.byref(_view())
    assert L.tiles_paged_resize(r, None, None) == INVALID and L.tiles_paged_resize(r, FAKE + 2, None) == INVALID
    assert L.tiles_paged_fork(r, None, None) == INVALID and L.tiles_paged_fork(r, FAKE + 1, None) == INVALID
    assert L.tiles_paged_trim(r, 0, 0, None) == INVALID and L.tiles_paged_trim(r, 4, -1, None) == INVALID
    for f in ("reset", "compact", "status"):
        assert getattr(L, "tiles_paged_" + f)(None, None) == INVALID
    b = ctypes.c_int64()
    d = _desc()
    assert L.tiles_paged_workspace_bytes(ctypes.byref(d), 3, 1, ctypes.byref(b)) == INVALID
    assert L.tiles_paged_workspace_bytes(ctypes.byref(d), 4, 0, ctypes.byref(b)) == INVALID
    assert L.tiles_paged_workspace_bytes(ctypes.byref(d), 64, 1, ctypes.byref(b)) == UNSUPPORTED
    assert L.tiles_paged_workspace_bytes(None, 4, 1, ctypes.byref(b)) == INVALID
