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
