"""CPU checks of the latent-cache and eviction calls: sizes, refusals before any
launch, and the binding's argument checks."""

import ctypes

import numpy as np
import pytest

import latent_plain as lp


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__._cuda_build_module().build()
    import nvfp4_quantised_paged_gb300 as mod
    return mod


A = ctypes.c_void_p(4096)


def _latent(m, **kw):
    d = dict(pool=4096, num_pages=4, page_size=16, latent_dim=512, rope_dim=64, global_scale=1.0)
    d.update(kw)
    return m._LatentDesc(*[d[k] for k, _ in m._LatentDesc._fields_])


def _gqa(m, **kw):
    d = dict(pool=4096, num_pages=4, page_size=16, num_kv_heads=2, head_dim=128, dtype=0, k_global_scale=1.0,
             v_global_scale=1.0)
    d.update(kw)
    return m._CacheDesc(*[d[k] for k, _ in m._CacheDesc._fields_])


def test_slab_sizes(m):
    for P in (16, 32, 64, 128):
        assert m.latent_slab_bytes(P) == 416 * P
    for bad in (8, 48, 256):
        with pytest.raises(m.NVFP4KVError):
            m.latent_slab_bytes(bad)


@pytest.mark.parametrize("kw,status", [
    (dict(page_size=48), -2), (dict(latent_dim=256), -2), (dict(rope_dim=32), -2), (dict(num_pages=0), -1),
    (dict(global_scale=0.0), -1), (dict(global_scale=float("nan")), -1), (dict(global_scale=1e-40), -1),
    (dict(pool=0), -1), (dict(pool=4097), -1),
])
def test_invalid_latent_descriptors(m, kw, status):
    lib, d = m.library(), _latent(m, **kw)
    p = ctypes.byref(d)
    assert lib.nvfp4_latent_quantize_append(p, A, 512, A, 64, 1, A, None) == status
    assert lib.nvfp4_latent_prefix_dequant(p, A, 1, A, A, 1, 16, A, A, None) == status
    assert lib.nvfp4_latent_decode_attention(p, A, A, 1, 16, A, 1, A, 0.1, A, A, 1 << 30, 1, None) == status
    assert lib.nvfp4kv_latent_decode_workspace_bytes(p, 1, 16, 1) == 0
    assert lib.nvfp4_latent_quantize_append(None, A, 512, A, 64, 1, A, None) == -1


def _refused(call, good, changes):
    for i, v, status in changes:
        args = list(good)
        args[i] = v
        assert call(*args) == status, (i, v)


def test_append_and_dequant_refusals(m):
    lib, p = m.library(), ctypes.byref(_latent(m))
    odd = ctypes.c_void_p(4104)
    _refused(lib.nvfp4_latent_quantize_append, [p, A, 576, A, 576, 1, A, None],
             [(1, None, -1), (1, odd, -1), (2, 504, -1), (2, 515, -1), (3, None, -1), (3, odd, -1), (4, 56, -1),
              (4, 65, -1), (5, -1, -1), (5, 1 << 31, -2), (6, None, -1), (6, ctypes.c_void_p(4100), -1), (5, 0, 0)])
    _refused(lib.nvfp4_latent_prefix_dequant, [p, A, 1, A, A, 1, 16, A, A, None],
             [(1, None, -1), (2, 0, -1), (3, None, -1), (4, None, -1), (5, -1, -1), (6, -1, -1), (6, 1 << 31, -2),
              (7, odd, -1), (8, odd, -1), (7, None, -1), (5, 0, 0), (6, 0, 0)])


def test_decode_refusals(m):
    lib, p = m.library(), ctypes.byref(_latent(m))
    odd = ctypes.c_void_p(4104)
    need = lib.nvfp4kv_latent_decode_workspace_bytes(p, 2, 16, 3)
    # (splits + batch) (m, l) pairs of 16 heads, and their 512 sums, each part a multiple of 256
    assert need == (5 * 16 * 8 + 255) // 256 * 256 + 5 * 16 * 512 * 4
    B = ctypes.c_void_p(8192)
    _refused(lib.nvfp4_latent_decode_attention, [p, A, A, 2, 16, A, 1, A, 0.1, B, A, need, 3, None],
             [(9, A, -1), (1, None, -1), (1, odd, -1), (2, odd, -1), (3, -1, -1), (3, 70000, -2), (4, 0, -1), (4, 129, -2),
              (5, None, -1), (6, 0, -1), (6, 1 << 27, -2), (7, None, -1), (8, float("inf"), -1),
              (8, float("nan"), -1), (9, odd, -1), (10, ctypes.c_void_p(4096 + 128), -1), (11, need - 1, -1), (12, -1, -1),
              (12, 70000, -2), (3, 0, 0)])


def test_extend_refusals(m):
    lib = m.library()
    odd = ctypes.c_void_p(4104)
    good = [A, A, A, 512, 256, A, A, 10, A, A, 512, 256, A, A, 20, 1, 20, 2, 0.1, A, None]
    _refused(lib.nvfp4_latent_extend_attention, good,
             [(0, odd, -1), (1, None, -1), (2, odd, -1), (3, 120, -1), (3, 516, -1), (4, 64, -1), (5, None, -1),
              (6, None, -1), (7, -1, -1), (7, 1 << 31, -2), (8, None, -1), (9, odd, -1), (10, 0, -1), (11, 132, -1),
              (12, None, -1), (13, None, -1), (14, -1, -1), (15, -1, -1), (15, 70000, -2), (16, -1, -1), (17, 0, -1),
              (17, 70000, -2), (18, 0.0, -1), (18, -0.1, -1), (18, float("nan"), -1), (19, None, -1),
              (14, 0, 0), (15, 0, 0), (16, 0, 0)])


def test_scores_and_evict_refusals(m):
    lib, p = m.library(), ctypes.byref(_gqa(m))
    assert lib.nvfp4kv_weights_workspace_bytes(p, 1, 3) == 0 and lib.nvfp4kv_weights_workspace_bytes(p, 1, 34) == 0
    good = [p, A, 1, 4, A, 1, A, 0.1, A, 16, A, 1 << 30, None]
    _refused(lib.nvfp4_accumulate_attention_weights, good,
             [(1, None, -1), (1, ctypes.c_void_p(4104), -1), (2, -1, -1), (3, 3, -1), (3, 34, -2), (4, None, -1),
              (5, 0, -1), (5, 1 << 27, -2), (6, None, -1), (7, float("nan"), -1), (8, None, -1), (9, 0, -1), (10, None, -1),
              (10, ctypes.c_void_p(4100), -1), (2, 0, 0)])
    B, C = ctypes.c_void_p(8192), ctypes.c_void_p(16384)
    good = [p, A, 32, 1, A, 2, A, A, 1, 8, 2, 2, B, A, C, 8, None]
    _refused(lib.nvfp4_evict, good,
             [(1, None, -1), (2, 0, -1), (3, -1, -1), (3, 40000, -2), (4, None, -1), (5, 0, -1), (5, 1 << 27, -2),
              (6, None, -1), (7, None, -1), (8, 0, -1), (9, 0, -1), (9, 3, -1), (10, -1, -1), (10, 7, -1), (11, -1, -1),
              (12, None, -1), (12, A, -1), (13, None, -1), (14, None, -1), (14, A, -1), (15, 7, -1), (3, 0, 0)])
    assert lib.nvfp4_evict(ctypes.byref(_gqa(m, page_size=48)), *good[1:]) == -2


def test_binding_refuses_host_tensors_and_wrong_shapes(m):
    import torch
    with pytest.raises(ValueError):
        m.LatentCache(4, 16, device="cpu")
    with pytest.raises(ValueError):
        m.LatentCache(4, 16, pool=torch.zeros((4, 416 * 16), dtype=torch.uint8))
    q = torch.zeros((3, 2, 192), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.latent_extend_attention(q, q[..., :128], q[..., :128], q[:, 0, :64], None, q[..., :128], q[..., :128], q[:, 0, :64],
                                  torch.zeros(2, dtype=torch.int32), 3)


def test_plain_quantiser_against_the_oracle():
    """The tests' own quantiser and the C oracle's agree on codes and scales."""
    import oracle
    oracle.build()
    rng = np.random.RandomState(3)
    x = (rng.randn(16, 512) * np.exp(rng.randn(16, 1))).astype(np.float32)
    b = (x.view(np.uint32) >> 16).astype(np.uint16)
    for g in (1.0, 0.375, 0.3712):
        pool = oracle.OraclePool(1, 16, 4, gk=g, gv=g)
        oracle.quantize_append(pool, b.reshape(16, 4, 128), b.reshape(16, 4, 128), np.arange(16, dtype=np.int64))
        codes, scales = lp.quantise(lp.bf16_to_f64(b), g)
        slab = pool.data.reshape(4, 2304)
        for h in range(4):
            packed = codes[:, h * 128::][:, :128].reshape(16, 64, 2)
            assert np.array_equal(slab[h, :1024].reshape(16, 64), packed[..., 0] | (packed[..., 1] << 4))
            assert np.array_equal(slab[h, 1024:1152].reshape(16, 8), scales[:, h * 8:h * 8 + 8])


def test_plain_eviction_order():
    s = np.array([1.0, np.nan, 3.0, 3.0, -np.inf, 0.0, -0.0, 2.0])
    assert lp.evict_plain(s, 8, 3, 0, 0).tolist() == [2, 3, 7]
    assert lp.evict_plain(s, 8, 2, 0, 1).tolist() == [0, 2]
    assert lp.evict_plain(s, 8, 5, 0, 0).tolist() == [0, 2, 3, 5, 7]
    assert lp.evict_plain(s, 8, 7, 0, 0).tolist() == [0, 2, 3, 4, 5, 6, 7]
    assert lp.evict_plain(s, 3, 5, 0, 0).tolist() == [0, 1, 2]
