"""Latent attention where sequences change often and where values are extreme, against the
64-bit formula."""

import numpy as np
import pytest
import torch

import latent_plain as lp
from test_gpu_latent import SM, _check_decode, _cuda, _f64, _filled, _rand, _slots, _table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import nvfp4_quantised_paged_gb300 as mod
    return mod


@pytest.mark.parametrize("H", [16, 32, 64])
def test_decode_of_many_short_sequences_in_one_cta(m, H):
    """A CTA that takes up a new query at almost every tile, each of another magnitude and sign:
    a tile multiplied with the query before it would show."""
    lens = [1 + (37 * i) % 150 for i in range(48)]
    cache, bt = _filled(m, lens, 16, 90 + H, 0.75)
    size = torch.tensor([(-1.0) ** i * 2.0 ** (i % 5 - 3) for i in range(48)], device="cuda")[:, None, None]
    q, qr = (_rand((48, H, 512), 1, 0.5) * size).to(torch.bfloat16), (_rand((48, H, 64), 2) * size).to(torch.bfloat16)
    for splits in (1, 2):
        out = m.latent_decode_attention(cache, q, qr, _cuda(bt), _cuda(lens), num_splits=splits)
        torch.cuda.synchronize()
        assert m.check_device_errors() == 0
        _check_decode(m, out, cache, bt, lens, 16, q, qr, 0.75)


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("s,t,r,g", [
    (1e-36, 1.0, 1.0, 1.0),
    (1e-30, 64.0, 1.0, 1.0),
    (1.0, 1.0, 1.0, 2.0**-110),
    (1.0, 4.0, 1.0, 2.0**-126),
    (0.5, 1e-36, 1e6, 1.0),
    (1e-38, 1e-4, 1e4, 1.0),
])
def test_decode_when_the_rotary_part_dwarfs_the_latent_one(m, H, s, t, r, g):
    """Latent queries (or a tensor scale) so small that their pre-scale, which the rotary part
    shares, must not push the rotary scores out of FP32."""
    P, lens = 64, [200, 300] * (1 if H == 16 else 40)      # (more tiles than SMs: larger head tiles)
    bt, pages = _table(lens, P, 5)
    cache = m.LatentCache(pages, P, global_scale=g)
    for b, n in enumerate(lens):
        x = _rand((n, 576), 50 + b % 2)
        x[:, 512:] *= r
        m.latent_quantize_append(cache, x[:, :512], x[:, 512:], _cuda(_slots(bt[b], P, n), torch.int64))
    q, qr = _rand((2, H, 512), 3, s), _rand((2, H, 64), 4, t)
    out = m.latent_decode_attention(cache, q.repeat(len(lens) // 2, 1, 1), qr.repeat(len(lens) // 2, 1, 1), _cuda(bt),
                                    _cuda(lens))
    torch.cuda.synchronize()
    assert m.check_device_errors() == 0
    _check_decode(m, out[:2], cache, bt, lens[:2], P, q, qr, g)


def _check_masked(m, out, cache, bt, n, P, q, qr, dead):
    """out [H][512] against the formula in which head h gives the tokens dead[h] a score of
    minus infinity, that is no weight."""
    c, r = lp.read_latent(cache.pool.cpu().numpy(), P, bt, n, 1.0)
    got = _f64(out)
    for h in range(q.shape[0]):
        live = ~dead[h]
        qq = np.concatenate([_f64(q[h]), _f64(qr[h])])[None]
        qq[:, 512] = 0                                     # the rotary dimension that masks adds 0 to the live ones
        rr = r.copy()
        rr[:, 0] = 0
        ref, spread, A, smax, _ = lp.attend(qq, np.concatenate([c, rr], 1)[live], c[live], SM)
        bound = lp.attention_bound(ref, spread, A, smax, lp.U_F16, n, np.abs(c).max())
        assert (np.abs(got[h] - ref[0]) <= bound[0]).all(), h


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("dead", [(0, 128), (0, 300), (128, 384), (0, 690), (300, 700)])
def test_decode_with_scores_of_minus_infinity(m, H, dead):
    """Tokens masked by a rotary value of minus infinity: whole tiles, and whole parts of a split
    sequence, then hold no score at all, before, between and behind the others."""
    P, n, B = 32, 700, (1 if H == 16 else 30)
    bt, pages = _table([n], P, 6)
    cache = m.LatentCache(pages, P)
    x = _rand((n, 576), 61)
    x[:, 512] = 0
    x[dead[0]:dead[1], 512] = -float("inf")
    m.latent_quantize_append(cache, x[:, :512], x[:, 512:], _cuda(_slots(bt[0], P, n), torch.int64))
    q, qr = _rand((1, H, 512), 7, 0.5), _rand((1, H, 64), 8)
    qr[..., 0] = 1.0
    mask = np.zeros((H, n), bool)
    mask[:, dead[0]:dead[1]] = True
    for splits in (B, 3 * B, 0):
        out = m.latent_decode_attention(cache, q.expand(B, H, 512).contiguous(), qr.expand(B, H, 64).contiguous(),
                                        _cuda(np.repeat(bt, B, 0)), _cuda([n] * B), num_splits=splits)
        torch.cuda.synchronize()
        _check_masked(m, out[-1], cache, bt[0], n, P, q[0], qr[0], mask)


@pytest.mark.parametrize("dead", [128, 256])
def test_decode_where_some_heads_mask_a_tile_and_others_do_not(m, dead):
    """A score beyond FP32's range in one head of a warpgroup, an ordinary one in its neighbour:
    the neighbour's maximum moves while the head has none yet."""
    P, n, H = 32, 400, 16
    bt, pages = _table([n], P, 9)
    cache = m.LatentCache(pages, P)
    x = _rand((n, 576), 62)
    x[:, 512] = 0
    x[:dead, 512] = -16.0
    m.latent_quantize_append(cache, x[:, :512], x[:, 512:], _cuda(_slots(bt[0], P, n), torch.int64))
    q, qr = _rand((1, H, 512), 7, 0.5), _rand((1, H, 64), 8)
    qr[:, :, 0] = 0
    qr[:, ::2, 0] = 3e38
    mask = np.zeros((H, n), bool)
    mask[::2, :dead] = True
    for splits in (1, 2, 4):
        out = m.latent_decode_attention(cache, q, qr, _cuda(bt), _cuda([n]), num_splits=splits)
        torch.cuda.synchronize()
        _check_masked(m, out[0], cache, bt[0], n, P, q[0], qr[0], mask)
