"""Eviction where few rows go or the search has little to hold on to: the number of kept rows
close to the number there are, in every selection, with guard areas around what is written.
Scores of sequences with missing pages, many units a warp."""

import pytest
import torch

import workloads
from gpu_common import fill_both
from test_gpu_eviction import _evict, _scores

pytestmark = pytest.mark.gpu
GUARD = 4096


@pytest.fixture(scope="module")
def m():
    import nvfp4_quantised_paged_gb300 as mod
    return mod


def _guarded(shape, dtype, value):
    """A buffer of `shape` inside a larger one filled with `value`; (the view, a check that the rest is untouched)."""
    n = 1
    for x in shape:
        n *= x
    whole = torch.full((n + 2 * GUARD,), value, dtype=dtype, device="cuda")

    def intact():
        return bool((whole[:GUARD] == value).all() and (whole[GUARD + n:] == value).all())
    return whole[GUARD:GUARD + n].view(shape), intact


def _run(m, lens, Hkv, keep, recent, sink, scores):
    """Every output, kept and scores as narrow as they may be, checked against the plain form (in _evict)."""
    B = len(lens)
    kept, k_ok = _guarded((B, Hkv, keep), torch.int32, -77)
    new_scores, s_ok = _guarded((B, Hkv, keep), torch.float32, -77.0)
    new_lens, l_ok = _guarded((B,), torch.int32, -77)
    _evict(m, lens, Hkv, 128, keep, recent, sink, scores, kept=kept, new_scores=new_scores, new_lens=new_lens)
    assert k_ok() and s_ok() and l_ok()


@pytest.mark.parametrize("recent,sink", [(256, 4), (0, 0)])
@pytest.mark.parametrize("more", [1, 2, 8, 16])
@pytest.mark.parametrize("keep", [2048, 4096, 8192, 32000])
def test_a_few_rows_go(m, keep, more, recent, sink):
    for seed in range(3):
        _run(m, [keep + more] * 4, 2, keep, recent, sink, _scores((4, 2, keep + more), seed))


def test_all_of_the_sampled_list_is_kept(m):
    """Trimming a cache that is a token over its budget, many segments at once: in a tenth of them the
    border falls on the lowest key between the sampled ones."""
    _run(m, [2049] * 64, 8, 2048, 256, 4, _scores((64, 8, 2049), 5))


@pytest.mark.parametrize("B,Hkv,keep", [(2, 1, 140000), (16, 8, 33000), (40, 8, 33000)])
def test_a_few_rows_of_long_segments_go(m, B, Hkv, keep):
    """Clusters of eight, four and one CTA, with more keys than a CTA's shared memory holds in the
    first and the last: one long segment, the others whole."""
    for more in (1, 2, 8, 16):
        _run(m, [keep + more] + [20] * (B - 1), Hkv, keep, 64, 4, _scores((B, Hkv, keep + more), more))


@pytest.mark.parametrize("dtype,n", [(0, 120000), (1, 120000)])
def test_scores_beside_many_missing_pages(m, dtype, n):
    """Pages out of range between good ones, in sequences so long that a warp's ring goes round
    several times: each reads as zeros, as a page of zeros does, and the pages after it are whole."""
    w = workloads.make_decode("holes", 3, [n], 16, 8, 16, extra_pages=1)
    cache, _ = fill_both(w, m, dtype=dtype)
    zero = next(iter(set(range(w.num_pages)) - set(w.block_table.flatten().tolist())))
    cache.pool[zero] = 0
    holes = torch.rand(w.block_table.shape, generator=torch.Generator().manual_seed(1)) < 0.4
    q, sl, got = w.q("cuda"), w.seq_lens.cuda(), []
    for page in (zero, w.num_pages, -1):
        scores = torch.zeros((1, 8, n), device="cuda")
        m.accumulate_attention_weights(cache, q, torch.where(holes, page, w.block_table).to(torch.int32).cuda(), sl, scores)
        torch.cuda.synchronize()
        assert m.check_device_errors() == (0 if page == zero else -4)
        got.append(scores)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
