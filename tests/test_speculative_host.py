"""CPU checks of the speculative decoding calls: workspace sizes that need no GPU, and the
refusals (a rejected call launches nothing, so plain numbers stand in for device pointers)."""

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

P = ctypes.c_void_p
OK, EINVAL, EUNSUPPORTED = 0, -1, -2


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__._cuda_build_module().build()
    import nvfp4_quantised_paged_gb300 as mod
    return mod


def desc(m, **kw):
    d = dict(pool=4096, num_pages=4, page_size=16, num_kv_heads=2, head_dim=128, dtype=0, k=1.0, v=1.0)
    d.update(kw)
    return ctypes.byref(m._CacheDesc(d["pool"], d["num_pages"], d["page_size"], d["num_kv_heads"], d["head_dim"], d["dtype"],
                                     d["k"], d["v"]))


class Rope(ctypes.Structure):
    """nvfp4kv_rope of the header."""
    _fields_ = [("cos_sin", P), ("num_positions", ctypes.c_int64), ("rot_dim", ctypes.c_int32), ("adjacent", ctypes.c_int32),
                ("num_axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 3), ("q_norm", P), ("k_norm", P),
                ("eps", ctypes.c_float)]


def rope(m, **kw):
    d = dict(cos_sin=4096, num_positions=10, rot_dim=128, adjacent=0, num_axes=1, sections=(0, 0, 0), q_norm=None, k_norm=None,
             eps=1e-6)
    d.update(kw)
    r = Rope(d["cos_sin"], d["num_positions"], d["rot_dim"], d["adjacent"], d["num_axes"])
    r.sections[:] = d["sections"]
    r.q_norm, r.k_norm, r.eps = d["q_norm"], d["k_norm"], d["eps"]
    return ctypes.addressof(r), r


def append(m, cache=None, r=None, q=4096, qs=512, qo=8192, qos=512, hq=4, k=4096, v=4096, ks=256, t=3, pos=4096, slots=4096):
    at, keep = rope(m, **(r or {}))
    return m.library().nvfp4_rope_quantize_append(cache or desc(m), at, q, qs, qo, qos, hq, k, v, ks, t, pos, slots, None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=-1), EINVAL), (dict(hq=-1), EINVAL), (dict(q=None), EINVAL), (dict(qo=None), EINVAL), (dict(q=4100), EINVAL),
    (dict(qs=504), EINVAL), (dict(qs=514), EINVAL), (dict(qos=500), EINVAL), (dict(qo=4096, qos=1024), EINVAL),
    (dict(k=None), EINVAL), (dict(v=4104), EINVAL), (dict(ks=128), EINVAL), (dict(ks=260), EINVAL), (dict(slots=None), EINVAL),
    (dict(slots=4100), EINVAL), (dict(pos=None), EINVAL), (dict(pos=4098), EINVAL), (dict(t=1 << 40), EUNSUPPORTED),
    (dict(r=dict(rot_dim=16)), EUNSUPPORTED), (dict(r=dict(rot_dim=160)), EUNSUPPORTED), (dict(r=dict(rot_dim=-32)), EUNSUPPORTED),
    (dict(r=dict(adjacent=2)), EINVAL), (dict(r=dict(num_axes=0)), EUNSUPPORTED), (dict(r=dict(num_axes=4)), EUNSUPPORTED),
    (dict(r=dict(num_axes=3, sections=(16, 24, 20))), EINVAL), (dict(r=dict(num_axes=2, sections=(30, 34, 0))), EUNSUPPORTED),
    (dict(r=dict(num_axes=2, sections=(-4, 68, 0))), EINVAL), (dict(r=dict(cos_sin=None)), EINVAL),
    (dict(r=dict(cos_sin=4100)), EINVAL), (dict(r=dict(num_positions=0)), EINVAL), (dict(r=dict(q_norm=4100)), EINVAL),
    (dict(r=dict(k_norm=4096, eps=-1.0)), EINVAL), (dict(r=dict(q_norm=4096, eps=float("nan"))), EINVAL),
])
def test_rope_append_refusals(m, kw, status):
    assert append(m, **kw) == status


def test_rope_append_refuses_the_cache_and_takes_nothing(m):
    assert append(m, cache=desc(m, head_dim=64)) == EUNSUPPORTED
    assert append(m, cache=desc(m, pool=0)) == EINVAL
    assert m.library().nvfp4_rope_quantize_append(desc(m), None, 4096, 512, 8192, 512, 4, 4096, 4096, 256, 3, 4096, 4096, None) == EINVAL
    assert append(m, t=0, q=None, k=None, v=None, slots=None, pos=None) == OK


def tree(m, cache=None, q=4096, cu=4096, total=4, batch=2, most=2, hq=4, mask=None, bt=4096, pages=2, lens=4096, scale=0.1, cap=0.0,
         window=0, slopes=None, out=8192, ws=4096, size=1 << 30, splits=1):
    return m.library().nvfp4_tree_attention(cache or desc(m), q, cu, total, batch, most, hq, mask, bt, pages, lens, scale, cap,
                                            window, slopes, out, ws, size, splits, None)


@pytest.mark.parametrize("kw,status", [
    (dict(total=-1), EINVAL), (dict(batch=-1), EINVAL), (dict(most=0), EINVAL), (dict(most=65), EUNSUPPORTED), (dict(hq=3), EINVAL),
    (dict(hq=0), EINVAL), (dict(hq=2 * 129), EUNSUPPORTED), (dict(splits=-1), EINVAL), (dict(window=-1), EINVAL),
    (dict(cap=-1.0), EINVAL), (dict(cap=float("inf")), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(q=None), EINVAL),
    (dict(q=4104), EINVAL), (dict(cu=None), EINVAL), (dict(cu=4098), EINVAL), (dict(bt=None), EINVAL), (dict(lens=None), EINVAL),
    (dict(out=None), EINVAL), (dict(out=4096), EINVAL), (dict(out=8200), EINVAL), (dict(ws=None), EINVAL), (dict(ws=4100), EINVAL),
    (dict(mask=4100), EINVAL), (dict(slopes=4098), EINVAL), (dict(pages=0), EINVAL), (dict(size=1024), EINVAL),
    (dict(pages=1 << 27), EUNSUPPORTED), (dict(batch=70000), EUNSUPPORTED), (dict(total=1 << 30), EUNSUPPORTED),
    (dict(batch=60000, pages=1 << 24), EUNSUPPORTED),
])
def test_tree_attention_refusals(m, kw, status):
    assert tree(m, **kw) == status


def test_tree_attention_refuses_fp8_and_takes_nothing(m):
    assert tree(m, cache=desc(m, dtype=1)) == EUNSUPPORTED
    assert tree(m, cache=desc(m, page_size=48)) == EUNSUPPORTED
    assert tree(m, batch=0, q=None, cu=None, out=None, ws=None) == OK
    assert tree(m, total=0, q=None, cu=None, out=None, ws=None) == OK


def test_tree_workspace(m):
    size = lambda *a, **kw: m.library().nvfp4kv_tree_workspace_bytes(desc(m, **kw), *a)  # noqa: E731
    # rows of a pair fill tiles of 16, 32, 64 or 128: partial sums of (splits + pairs) of them, and their (m, l)
    for most, rows, tiles in ((1, 16, 1), (8, 16, 1), (16, 32, 1), (17, 64, 1), (64, 128, 1)):
        slots = 7 + 3 * 2
        assert size(3, 4, most, 7) == (tiles * slots * rows * 8 + 255) // 256 * 256 + tiles * slots * rows * 512
    assert size(3, 16, 64, 7) == 4 * 13 * 128 * (8 + 512)
    for bad in ((-1, 4, 1, 1), (3, 3, 1, 1), (3, 4, 0, 1), (3, 4, 65, 1), (3, 4, 1, -1), (3, 2 * 129, 1, 1)):
        assert size(*bad) == 0
    assert size(3, 4, 1, 1, dtype=1) == 0


def accept(m, cache=None, bt=4096, pages=2, lens=4096, cu=4096, batch=2, acc=4096, most=4, num=4096, new=8192):
    return m.library().nvfp4_accept_tokens(cache or desc(m), bt, pages, lens, cu, batch, acc, most, num, new, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), EINVAL), (dict(most=0), EINVAL), (dict(most=65), EUNSUPPORTED), (dict(batch=65536), EUNSUPPORTED),
    (dict(bt=None), EINVAL), (dict(lens=None), EINVAL), (dict(cu=None), EINVAL), (dict(acc=None), EINVAL), (dict(num=None), EINVAL),
    (dict(new=None), EINVAL), (dict(new=8194), EINVAL), (dict(new=4096), EINVAL), (dict(new=4100), EINVAL), (dict(new=4092), EINVAL),
    (dict(pages=0), EINVAL), (dict(pages=1 << 27), EUNSUPPORTED),
])
def test_accept_refusals(m, kw, status):
    assert accept(m, **kw) == status


def test_accept_refuses_the_cache_and_takes_nothing(m):
    assert accept(m, cache=desc(m, num_pages=0)) == EINVAL
    assert accept(m, batch=0, bt=None, lens=None, cu=None, acc=None, num=None, new=None) == OK


def test_the_packed_rotation_is_the_struct(m):
    at, r = rope(m, cos_sin=4096, num_positions=7, rot_dim=64, adjacent=1, num_axes=3, sections=(8, 12, 12), q_norm=8192,
                 k_norm=16384, eps=0.5)
    assert m._ROPE.size == ctypes.sizeof(r)
    assert m._ROPE.pack(4096, 7, 64, 1, 3, 8, 12, 12, 8192, 16384, 0.5) == bytes(r)


# ------------------------------------------------------------------ the sources: what no output shows

def _source(name):
    with open(os.path.join(ROOT, "nvfp4_quantised_paged_gb300", "csrc", name)) as f:
        return f.read()


def test_what_the_tree_products_read_is_fenced_before_it_is_reported():
    src = _source("tree_attention.cu")
    over = src[src.index("auto hand_over"):]
    over = over[:over.index("};")]
    assert over.index("fence.proxy.async.shared::cta") < over.index("tc_wait_st") < over.index("tc_fence_before") \
        < over.index("__syncwarp") < over.index("mbar_arrive(ready)")
    # with 128 rows the scores start at the report of K: Q has to be fenced before the barrier that precedes it
    store = src[src.index("auto store_pair"):]
    assert store.index("if (W) asm volatile(\"fence.proxy.async.shared::cta") < store.index("workers_sync<N>()")
    report = src[src.index("auto report_k"):]
    assert report.index("tc_wait_st") < report.index("tc_fence_before") < report.index("mbar_arrive(k_ready(j))")


@pytest.mark.parametrize("name", ["tree_attention.cu", "rope_append.cu"])
def test_copies_in_flight_are_waited_for_at_the_end(name):
    src = _source(name)
    tail = src[src.index("no copy may still be writing when the CTA ends"):]
    assert "mbar_wait_bounded(" in tail[:400] and "nullptr" in tail[:400]
    if name == "tree_attention.cu":
        drain = src[src.index("tc_commit(drain)"):]
        assert "mbar_wait_bounded(drain" in drain[:200]
