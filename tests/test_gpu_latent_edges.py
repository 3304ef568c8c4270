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
