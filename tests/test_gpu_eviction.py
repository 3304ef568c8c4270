"""Attention-weight scores and eviction on the GPU against plain 64-bit
implementations, and a decode loop that uses them together."""

import math

import numpy as np
import pytest
import torch

import latent_plain as lp
import oracle
import workloads
from gpu_common import bits, fill_both

pytestmark = pytest.mark.gpu
SM = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module")
def m():
    import nvfp4_quantised_paged_gb300 as mod
    return mod


def _k_of(w, pool, b):
    """float64 K [n][Hkv][128] of sequence b as the pool holds it (tensor scale included)."""
    n = int(w.seq_lens[b])
    cu = np.array([0, n], np.int32)
    k, _ = oracle.prefix_dequant(pool, w.block_table[b:b + 1].numpy(), np.array([n], np.int32), cu)
    return lp.bf16_to_f64(k)


# ------------------------------------------------------------------ scores

@pytest.mark.parametrize("lens,Hq,Hkv,P,dtype,gk", [
    ([1], 1, 1, 16, 0, 1.0),
    ([300, 256], 4, 1, 16, 0, 1.0),
    ([0, 63, 64, 65, 1], 16, 2, 32, 0, 1.0),
    ([1000, 17], 40, 8, 64, 0, 1.0),
    ([95, 96, 97, 192, 193], 8, 2, 16, 0, 1.0),
    ([385, 96, 95], 16, 1, 32, 1, 1.0),
    ([700, 129], 32, 2, 128, 0, 1.0),          # 16 heads a group
    ([500], 9, 1, 64, 0, 1.0),
    ([300, 40], 16, 2, 64, 1, 1.0),            # FP8 pool
    ([90, 5], 32, 2, 16, 1, 1.0),
    ([200], 8, 4, 64, 0, 0.5),
])
def test_scores_match_the_formula(m, lens, Hq, Hkv, P, dtype, gk):
    w = workloads.make_decode("weights", 5 + sum(lens), lens, Hq, Hkv, P)
    cache, pool = fill_both(w, m, dtype=dtype, gk=gk)
    q = w.q("cuda")
    S = max(lens) + 7
    old = torch.rand((len(lens), Hkv, S), generator=torch.Generator().manual_seed(1))
    scores = old.cuda()
    ws = m.alloc_weights_workspace(cache, len(lens), Hq)
    ws.fill_(0xFF)
    got = m.accumulate_attention_weights(cache, q, w.block_table.cuda(), w.seq_lens.cuda(), scores, workspace=ws)
    torch.cuda.synchronize()
    assert m.check_device_errors() == 0 and got is scores
    got, G = scores.double().cpu().numpy(), Hq // Hkv
    want, bound = old.double().numpy(), np.zeros(old.shape)
    for b, n in enumerate(lens):
        k = _k_of(w, pool, b)
        for h in range(Hkv if n else 0):
            _, _, A, smax, p = lp.attend(lp.bf16_to_f64(bits(q[b, h * G:(h + 1) * G])), k[:, h], np.zeros((n, 1)), SM)
            # each weight: e^(2 d) for its score and the denominator's, 2^-19 for the exponentials and logarithm
            d = 2.0**-16 * A + 2.0**-21 * smax
            bound[b, h, :n] = (p * (3 * d + 2.0**-19)[:, None]).sum(0)
            want[b, h, :n] += p.sum(0)
    assert (np.abs(got - want) <= bound + 2.0**-22 * np.abs(want)).all()
    for b, n in enumerate(lens):               # entries behind the sequence stay as they were
        assert np.array_equal(scores[b, :, n:].cpu().numpy(), old[b, :, n:].numpy())


@pytest.mark.parametrize("B", [140, 300])
def test_scores_of_many_sequences(m, B):
    """More sequences than a warp, and than a CTA, scans at once: each as if it were alone."""
    lens = np.random.RandomState(B).randint(0, 150, B).tolist()
    w = workloads.make_decode("weights many", B, lens, 4, 1, 16)
    cache, _ = fill_both(w, m)
    q, bt, sl = w.q("cuda"), w.block_table.cuda(), w.seq_lens.cuda()
    got = torch.zeros((B, 1, 160), device="cuda")
    m.accumulate_attention_weights(cache, q, bt, sl, got)
    torch.cuda.synchronize()
    assert m.check_device_errors() == 0
    # the number of warps that share a sequence changes the order of its denominator's sums: 2^-20
    for b in list(range(0, B, 37)) + [B - 1]:
        one = torch.zeros((1, 1, 160), device="cuda")
        m.accumulate_attention_weights(cache, q[b:b + 1].contiguous(), bt[b:b + 1].contiguous(), sl[b:b + 1].contiguous(), one)
        assert ((one[0] - got[b]).abs() <= 2.0**-20 * one[0]).all()
    assert (got[:, 0].sum(-1).cpu() - 4.0 * (torch.tensor(lens) > 0)).abs().max() < 1e-4


@pytest.mark.parametrize("scale", [-SM, 0.0, 8 * SM])
def test_scores_with_other_scales(m, scale):
    w = workloads.make_decode("weights scale", 9, [200, 77], 8, 2, 64)
    cache, pool = fill_both(w, m)
    q = w.q("cuda")
    scores = torch.zeros((2, 2, 200), device="cuda")
    m.accumulate_attention_weights(cache, q, w.block_table.cuda(), w.seq_lens.cuda(), scores, sm_scale=scale)
    torch.cuda.synchronize()
    for b, n in enumerate([200, 77]):
        k = _k_of(w, pool, b)
        for h in range(2):
            _, _, A, smax, p = lp.attend(lp.bf16_to_f64(bits(q[b, 4 * h:4 * h + 4])), k[:, h], np.zeros((n, 1)), scale)
            d = 2.0**-16 * A + 2.0**-21 * smax
            err = np.abs(scores[b, h, :n].double().cpu().numpy() - p.sum(0))
            assert (err <= (p * (3 * d + 2.0**-19)[:, None]).sum(0) + 2.0**-22 * p.sum(0)).all()


def test_scores_are_the_same_every_time_and_add_up(m):
    w = workloads.make_decode("weights twice", 3, [3000, 1, 500] * 4, 32, 8, 64)
    cache, _ = fill_both(w, m)
    q, bt, sl = w.q("cuda"), w.block_table.cuda(), w.seq_lens.cuda()
    one = torch.zeros((12, 8, 3000), device="cuda")
    m.accumulate_attention_weights(cache, q, bt, sl, one)
    for s in (None, torch.cuda.Stream()):
        again = torch.zeros_like(one)
        torch.cuda.synchronize()
        m.accumulate_attention_weights(cache, q, bt, sl, again, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(one, again)
    res, ws = torch.zeros_like(one), m.alloc_weights_workspace(cache, 12, 32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.accumulate_attention_weights(cache, q, bt, sl, res, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(res, one)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(res, one + one)
    # a token gets G weights that sum to 1 over the sequence: each head's row sums to G
    assert torch.allclose(one.double().sum(-1), torch.full((12, 8), 4.0, dtype=torch.float64, device="cuda"), atol=1e-4)


def test_scores_flag_bad_pages_and_lengths(m):
    w = workloads.make_decode("weights bad", 4, [200], 8, 2, 64)
    cache, _ = fill_both(w, m)
    q, sl = w.q("cuda"), w.seq_lens.cuda()
    bt = w.block_table.clone()
    bt[0, 1] = 99999
    scores = torch.zeros((1, 2, 200), device="cuda")
    m.accumulate_attention_weights(cache, q, bt.cuda(), sl, scores)      # the page's keys read as zeros
    torch.cuda.synchronize()
    assert m.check_device_errors() == -4
    assert torch.isfinite(scores).all() and (scores[:, :, 64:128] == scores[:, :, 64:65]).all()
    short = torch.zeros((1, 2, 150), device="cuda")
    m.accumulate_attention_weights(cache, q, w.block_table.cuda(), sl, short)   # cut to the scores there are
    torch.cuda.synchronize()
    assert m.check_device_errors() == -4
    want = torch.zeros((1, 2, 150), device="cuda")
    m.accumulate_attention_weights(cache, q, w.block_table.cuda(), torch.tensor([150], dtype=torch.int32, device="cuda"), want)
    torch.cuda.synchronize()
    assert torch.equal(short, want)


# ------------------------------------------------------------------ eviction

def _evict(m, lens, Hkv, P, keep, recent, sink, scores, dtype=0, S=None, seed=1, **kw):
    """Runs evict over random page bytes and checks everything that it writes."""
    counts = [-(-n // P) for n in lens]
    news = [-(-min(n, keep) // P) for n in lens]
    pages = sum(counts) + sum(news) + 1
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    bt, nt = -np.ones((len(lens), max(counts + [1])), np.int32), -np.ones((len(lens), max(news + [1])), np.int32)
    at = 0
    for tab, cnt in ((bt, counts), (nt, news)):
        for b, c in enumerate(cnt):
            tab[b, :c] = order[at:at + c]
            at += c
    cache = m.PagedCache(pages, P, Hkv, dtype=dtype)
    cache.pool.random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(seed))
    before = cache.pool.cpu().numpy().copy()
    old = scores.clone()
    new_lens, kept, new_scores = m.evict(cache, scores, torch.tensor(bt, device="cuda"),
                                         torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                         torch.tensor(nt, device="cuda"), keep, recent=recent, sink=sink, **kw)
    torch.cuda.synchronize()
    assert m.check_device_errors() == 0
    assert torch.equal(scores.view(torch.int32), old.view(torch.int32))
    sc = old.cpu().numpy()
    want_pool = before.copy()
    gb = 2304 if dtype == 0 else 4096

    def parts(page, h, r):
        grp = want_pool[page, h, (r // 16) * gb:(r // 16 + 1) * gb], before[page, h, (r // 16) * gb:(r // 16 + 1) * gb]
        r %= 16
        if dtype:
            return [(g[:2048].reshape(16, 128)[r], g[2048:].reshape(16, 128)[r]) for g in grp]
        return [(g[:1024].reshape(16, 64)[r], g[1024:1152].reshape(16, 8)[r], g[1152:2176].reshape(16, 64)[r],
                 g[2176:].reshape(8, 16)[:, r]) for g in grp]

    assert new_lens.tolist() == [min(n, keep) for n in lens]
    for b, n in enumerate(lens):
        for h in range(Hkv):
            rows = lp.evict_plain(sc[b, h], n, keep, recent, sink)
            k = kept[b, h].cpu().numpy()
            assert np.array_equal(k[:len(rows)], rows) and (k[len(rows):] == -1).all(), (b, h)
            ns = new_scores[b, h].cpu().numpy()
            assert np.array_equal(ns[:len(rows)].view(np.int32), sc[b, h][rows].view(np.int32))
            assert (ns[len(rows):].view(np.int32) == 0).all()
            for i, r in enumerate(rows):
                dst, src = parts(nt[b, i // P], h, i % P)[0], parts(bt[b, r // P], h, r % P)[1]
                for d, s in zip(dst, src):
                    d[...] = s
    assert np.array_equal(cache.pool.cpu().numpy(), want_pool)     # nothing else was written


def _scores(shape, seed=0):
    return torch.exp(torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * 2).cuda()


@pytest.mark.parametrize("lens,Hkv,P,keep,recent,sink,dtype", [
    ([1], 1, 16, 1, 0, 0, 0),
    ([2, 0, 1], 2, 16, 1, 1, 0, 0),
    ([100, 64, 63, 65], 2, 32, 64, 8, 4, 0),
    ([300], 8, 64, 299, 0, 0, 0),
    ([500, 17], 1, 128, 40, 40, 0, 0),          # only the recent ones
    ([500, 17], 3, 16, 40, 10, 30, 0),          # only protected ones
    ([200, 90], 2, 64, 33, 3, 2, 1),            # FP8 pool
    ([2000], 2, 64, 100, 16, 4, 0),
    ([9000, 300], 2, 64, 700, 16, 4, 0),        # more than 8,192 rows: the larger CTA
])
def test_evict_keeps_the_largest(m, lens, Hkv, P, keep, recent, sink, dtype):
    _evict(m, lens, Hkv, P, keep, recent, sink, _scores((len(lens), Hkv, max(lens) + 5), sum(lens)), dtype)


@pytest.mark.parametrize("n,keep", [(50, 20), (3000, 500), (20000, 3000), (40000, 5000), (200000, 4000)])   # each way
@pytest.mark.parametrize("kind", ["equal", "zeros", "two", "special", "rising", "falling", "narrow"])
def test_evict_ties_and_special_values(m, n, keep, kind):
    t = torch.arange(n, dtype=torch.float32)
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=g)
    if kind == "equal":
        x = torch.full((n,), 0.25)
    elif kind == "zeros":
        x = torch.where(torch.rand(n, generator=g) < 0.5, torch.zeros(n), -torch.zeros(n))
        x[::97] = 1.0
    elif kind == "two":
        x = torch.where(torch.rand(n, generator=g) < keep / n * 0.9, torch.ones(n), torch.zeros(n))
    elif kind == "special":
        x[::3] = float("nan")
        x[1::7] = float("inf")
        x[2::7] = float("-inf")
        x[3::11] = -0.0
        x[4::11] = 1e-42                       # subnormal
    elif kind == "rising":
        x = t
    elif kind == "falling":
        x = -t
    else:                                      # keys that differ in the last bits alone
        x = (1.0 + torch.randint(0, 40, (n,), generator=g) * 2.0**-23).float()
    _evict(m, [n], 1, 128, keep, min(5, keep // 4), min(2, keep // 4), x.view(1, 1, n).cuda())


@pytest.mark.parametrize("B,Hkv,n,keep", [(2, 2, 70000, 3000), (20, 8, 33000, 700), (40, 8, 33000, 90), (1, 1, 300000, 20)])
def test_evict_long_segments(m, B, Hkv, n, keep):
    """Clusters of eight, two and one CTA a segment, beside short segments; more keys than a CTA keeps."""
    lens = [n] + [100] * (B - 1)
    _evict(m, lens, Hkv, 128, keep, min(16, keep // 4), 3, _scores((B, Hkv, n + 1), B))


def test_evict_unaligned_rows_and_own_buffers(m):
    """Score rows that start off 16-byte boundaries, and buffers that the caller brings."""
    lens, Hkv, keep = [101, 77, 30], 3, 25
    sc = _scores((3, Hkv, 101), 3)
    new = dict(new_lens=torch.full((3,), -7, dtype=torch.int32, device="cuda"),
               kept=torch.full((3, Hkv, keep), -7, dtype=torch.int32, device="cuda"),
               new_scores=torch.full((3, Hkv, 31), -7.0, device="cuda"))
    _evict(m, lens, Hkv, 16, keep, 4, 1, sc, **new)


def test_evict_in_a_graph_and_on_another_stream(m):
    B, Hkv, n, keep, P = 3, 2, 700, 100, 64
    w = workloads.make_decode("evict graph", 8, [n] * B, 8, Hkv, P, extra_pages=3 * 2)
    cache, _ = fill_both(w, m)
    used = set(w.block_table.flatten().tolist())
    free = [p for p in range(w.num_pages) if p not in used][:6]
    nt = torch.tensor(free, dtype=torch.int32, device="cuda").view(3, 2)
    sc = _scores((B, Hkv, n), 2)
    bt, sl = w.block_table.cuda(), w.seq_lens.cuda()
    want = [x.clone() for x in m.evict(cache, sc, bt, sl, nt, keep, recent=5)]
    pool = cache.pool.clone()
    cache.pool[free] = 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = m.evict(cache, sc, bt, sl, nt, keep, recent=5, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(cache.pool, pool)
    outs = [torch.zeros_like(x) for x in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.evict(cache, sc, bt, sl, nt, keep, recent=5, new_lens=outs[0], kept=outs[1], new_scores=outs[2])
    cache.pool[free] = 0
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want)) and torch.equal(cache.pool, pool)


def test_evict_flags_missing_pages(m):
    w = workloads.make_decode("evict bad", 6, [200], 4, 1, 64, extra_pages=2)
    cache, _ = fill_both(w, m)
    used = set(w.block_table.flatten().tolist())
    free = [p for p in range(w.num_pages) if p not in used]
    sc = _scores((1, 1, 200), 1)
    before = cache.pool.clone()
    nt = torch.tensor([[free[0], -1]], dtype=torch.int32, device="cuda")   # rows 64 .. 99 have no page
    m.evict(cache, sc, w.block_table.cuda(), w.seq_lens.cuda(), nt, 100)
    torch.cuda.synchronize()
    assert m.check_device_errors() == -4
    changed = (cache.pool != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [free[0]]
    bad = w.block_table.clone()
    bad[0, 0] = -5                                                         # an old page that does not exist
    m.evict(cache, sc, bad.cuda(), w.seq_lens.cuda(), torch.tensor([free], dtype=torch.int32, device="cuda"), 100)
    torch.cuda.synchronize()
    assert m.check_device_errors() == -4
    m.evict(cache, sc, w.block_table.cuda(), torch.tensor([201], dtype=torch.int32, device="cuda"),
            torch.tensor([free], dtype=torch.int32, device="cuda"), 100)   # longer than its scores: cut and flagged
    torch.cuda.synchronize()
    assert m.check_device_errors() == -4


def test_pages_beyond_four_gigabytes(m):
    """Scores and eviction in the last pages of a pool of more than 2^32 bytes."""
    Hkv, P, lens, keep = 8, 128, [300, 200], 130
    w = workloads.make_decode("far", 14, lens, 16, Hkv, P, extra_pages=4)
    small, _ = fill_both(w, m)
    bt = w.block_table.clone()
    used = set(bt.flatten().tolist())
    nt = torch.tensor([p for p in range(w.num_pages) if p not in used][:4], dtype=torch.int32).view(2, 2)
    pages = (1 << 32) // (144 * P * Hkv) + 16
    big = m.PagedCache(pages, P, Hkv, pool=torch.empty((pages, Hkv, 144 * P), dtype=torch.uint8, device="cuda"))
    big.pool[pages - w.num_pages:] = small.pool.flip(0)
    q, sl, got = w.q("cuda"), w.seq_lens.cuda(), []
    for cache, far in ((small, False), (big, True)):
        t, n = [torch.where(x >= 0, pages - 1 - x, x) if far else x for x in (bt, nt)]
        sc = torch.zeros((2, Hkv, 300), device="cuda")
        m.accumulate_attention_weights(cache, q, t.cuda(), sl, sc)
        out = m.evict(cache, sc, t.cuda(), sl, n.cuda(), keep, recent=10, sink=2)
        got.append((sc, *out, cache.pool[n.flatten().long().cuda()]))
    torch.cuda.synchronize()
    assert m.check_device_errors() == 0
    assert all(torch.equal(a, b) for a, b in zip(*got))


# ------------------------------------------------------------------ together

def test_decode_score_evict_decode(m):
    """A bounded cache as a server runs it: decode steps that score the cached tokens, an
    eviction into fresh pages, more decode steps on those.  After it the cache holds exactly
    the kept tokens: decoding over it equals decoding over a cache that those were appended to."""
    Hq, Hkv, P, keep = 8, 2, 32, 48
    lens = [150, 33, 90]
    w = workloads.make_decode("bounded", 12, lens, Hq, Hkv, P, extra_pages=16)
    cache, _ = fill_both(w, m)
    used = set(w.block_table.flatten().tolist())
    free = torch.tensor([p for p in range(w.num_pages) if p not in used], dtype=torch.int32)
    bt, sl = w.block_table.cuda(), w.seq_lens.cuda()
    scores = torch.zeros((3, Hkv, 160), device="cuda")
    for step in range(3):
        q = torch.randn((3, Hq, 128), generator=torch.Generator().manual_seed(step)).to(torch.bfloat16).cuda()
        m.paged_decode_attention(cache, q, bt, sl)
        m.accumulate_attention_weights(cache, q, bt, sl, scores)
    nt = torch.full((3, 3), -1, dtype=torch.int32)
    nt[:, :2] = free[:6].view(3, 2)
    nt[:, 2] = free[6:9]                       # room for the tokens that follow
    new_lens, kept, new_scores = m.evict(cache, scores, bt, sl, nt.cuda(), keep, recent=8, sink=2)
    assert new_lens.tolist() == [48, 33, 48]
    # the same tokens appended to another cache
    ref = m.PagedCache(9, P, Hkv)
    rt = torch.arange(9, dtype=torch.int32).view(3, 3)
    for b in range(3):
        k, v = w.seq_kv(b, "cuda")
        n = int(new_lens[b])
        idx = kept[b, :, :n].long()
        kk = torch.stack([k[idx[h], h] for h in range(Hkv)], 1)
        vv = torch.stack([v[idx[h], h] for h in range(Hkv)], 1)
        t = torch.arange(n)
        m.quantize_append(ref, kk.contiguous(), vv.contiguous(), (rt[b].long()[t // P] * P + t % P).cuda())
    for step in range(2):                      # the next tokens go to the new pages in the decode call
        new_lens = new_lens + 1
        kn, vn = (torch.randn((3, Hkv, 128), generator=torch.Generator().manual_seed(70 + step + i)).to(torch.bfloat16).cuda()
                  for i in (0, 10))
        q = torch.randn((3, Hq, 128), generator=torch.Generator().manual_seed(90 + step)).to(torch.bfloat16).cuda()
        a = m.paged_decode_attention_append(cache, kn, vn, q, nt.cuda(), new_lens)
        b = m.paged_decode_attention_append(ref, kn, vn, q, rt.cuda(), new_lens)
        sa, sb = new_scores.clone(), new_scores.clone()
        m.accumulate_attention_weights(cache, q, nt.cuda(), new_lens, sa)
        m.accumulate_attention_weights(ref, q, rt.cuda(), new_lens, sb)
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(sa, sb)
    assert m.check_device_errors() == 0
