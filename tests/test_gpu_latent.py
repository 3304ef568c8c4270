"""The latent cache on the GPU against plain 64-bit implementations: quantised
append and dequant byte for byte, the absorbed decode and the expanded extend
within derived tolerances (latent_plain), and the two forms against each other."""

import math

import numpy as np
import pytest
import torch

import latent_plain as lp

pytestmark = pytest.mark.gpu
SM = 1.0 / math.sqrt(192)


@pytest.fixture(scope="module")
def m():
    import nvfp4_quantised_paged_gb300 as mod
    return mod


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed), device="cuda") * scale).to(torch.bfloat16)


def _bits(t):
    return t.contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def _f64(t):
    return t.double().cpu().numpy()


def _table(lens, P, seed, extra=0):
    counts = [-(-n // P) for n in lens]
    order = torch.randperm(sum(counts) + extra, generator=torch.Generator().manual_seed(seed)).tolist()
    bt = -np.ones((len(lens), max(counts + [1])), np.int32)
    at = 0
    for b, c in enumerate(counts):
        bt[b, :c] = order[at:at + c]
        at += c
    return bt, max(1, sum(counts) + extra)


def _cuda(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def _slots(bt_row, P, n):
    t = np.arange(n)
    return bt_row[t // P].astype(np.int64) * P + t % P


def _filled(m, lens, P, seed, g=1.0, outliers=True):
    """A cache holding random rows of every sequence; returns (cache, block table)."""
    bt, pages = _table(lens, P, seed)
    cache = m.LatentCache(pages, P, global_scale=g)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        x = torch.randn((n, 576), generator=_gen(seed * 100 + b), device="cuda")
        if outliers:
            x[:, 3::97] *= 8
        x = x.to(torch.bfloat16)
        m.latent_quantize_append(cache, x[:, :512], x[:, 512:], _cuda(_slots(bt[b], P, n), torch.int64))
    return cache, bt


# ------------------------------------------------------------------ append and dequant

@pytest.mark.parametrize("T,P,g", [(1, 16, 1.0), (3, 64, 0.75), (37, 32, 1.0), (300, 128, 0.3712), (130, 16, 117.3),
                                   (64, 64, 2.0**-70), (64, 64, 2.0**-126)])
def test_append_and_dequant_are_exact(m, T, P, g):
    x = torch.randn((T, 576), generator=_gen(T), device="cuda")
    x[:, 5::41] *= 30
    x *= float(np.float32(g))                 # values around the tensor scale
    x[0, 16:32] = 0                           # a zero block, signed zeros
    x[0, 20] = -0.0
    x = x.to(torch.bfloat16)
    pages = -(-T // P) + 2
    slots = torch.randperm(pages * P, generator=torch.Generator().manual_seed(T))[:T].numpy().astype(np.int64)
    if T > 2:
        slots[1] = -1                         # skipped
    cache = m.LatentCache(pages, P, global_scale=g)
    cache.pool.fill_(0xA5)                    # rows that no token writes stay as they are
    m.latent_quantize_append(cache, x[:, :512], x[:, 512:], _cuda(slots, torch.int64))
    torch.cuda.synchronize()
    assert m.check_device_errors() == 0
    want = np.full((pages, 416 * P), 0xA5, np.uint8)
    codes, scales = lp.quantise(_f64(x[:, :512]), g)
    lp.write_latent(want, P, slots, lp.latent_rows(codes, scales, _bits(x[:, 512:])))
    assert np.array_equal(cache.pool.cpu().numpy(), want)


def test_a_subnormal_tensor_scale_is_refused(m):
    cache = m.LatentCache(1, 64, global_scale=1e-38)
    x = _rand((64, 576), 64)
    with pytest.raises(m.NVFP4KVError):
        m.latent_quantize_append(cache, x[:, :512], x[:, 512:], torch.arange(64, device="cuda"))


def test_every_tie_and_scale_border_rounds_as_the_exact_quotient(m):
    """Blocks whose amax and values sit on and next to the rounding borders, under scales
    with short and long significands."""
    for g in (0.75, 0.625, float(np.float32(1 / 3)), 1.0):
        mags = (np.arange(128, 256)[:, None] * 2.0**np.arange(-10, 3)[None, :]).reshape(-1)   # all BF16 significands
        x = np.concatenate([mags, -mags[: 512 - mags.size % 512]])
        x = x[: x.size // 512 * 512].reshape(-1, 512)
        rng = np.random.default_rng(0)
        x = rng.permuted(x, axis=1)
        lat = torch.tensor(x, dtype=torch.bfloat16, device="cuda")
        rope = _rand((x.shape[0], 64), 1)
        cache = m.LatentCache(-(-x.shape[0] // 16), 16, global_scale=g)
        m.latent_quantize_append(cache, lat, rope, torch.arange(x.shape[0], device="cuda"))
        torch.cuda.synchronize()
        want = np.zeros(tuple(cache.pool.shape), np.uint8)
        codes, scales = lp.quantise(_f64(lat), g)
        lp.write_latent(want, 16, np.arange(x.shape[0]), lp.latent_rows(codes, scales, _bits(rope)))
        assert np.array_equal(cache.pool.cpu().numpy(), want), g


@pytest.mark.parametrize("lens,P,g", [([1], 16, 1.0), ([17, 0, 64], 32, 0.75), ([129, 300], 128, 0.3712)])
def test_prefix_dequant(m, lens, P, g):
    cache, bt = _filled(m, lens, P, 7, g)
    cu = np.concatenate([[0], np.cumsum(lens)])
    lat, rope = m.latent_prefix_dequant(cache, _cuda(bt), _cuda(lens), _cuda(cu), int(cu[-1]))
    torch.cuda.synchronize()
    assert m.check_device_errors() == 0
    pool = cache.pool.cpu().numpy()
    for b, n in enumerate(lens):
        c, r = lp.read_latent(pool, P, bt[b], n, g)
        assert np.array_equal(_f64(lat[cu[b]:cu[b + 1]]), lp.round_bf16(c))
        assert np.array_equal(_f64(rope[cu[b]:cu[b + 1]]), r)


def test_indices_out_of_range_are_skipped_and_flagged(m):
    cache = m.LatentCache(2, 16)
    x = _rand((3, 576), 1)
    m.latent_quantize_append(cache, x[:, :512], x[:, 512:], _cuda([0, 32, 5], torch.int64))   # slot 32 of 32
    torch.cuda.synchronize()
    assert m.check_device_errors() == -4
    bt, lens = _cuda([[0, 7]]), _cuda([20])
    lat = torch.full((20, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    m.latent_prefix_dequant(cache, bt, lens, _cuda([0, 20]), 20, latent_ws=lat)               # page 7 of 2
    torch.cuda.synchronize()
    assert m.check_device_errors() == -4
    assert (lat[16:] == 3.0).all()            # the rows of the missing page were not written


# ------------------------------------------------------------------ absorbed decode

def _check_decode(m, out, cache, bt, lens, P, q, qr, g, sm=SM):
    pool = cache.pool.cpu().numpy()
    got = _f64(out)
    assert np.isfinite(got).all()
    for b, n in enumerate(lens):
        if n == 0:
            assert (got[b] == 0).all()
            continue
        c, r = lp.read_latent(pool, P, bt[b], n, g)
        qq = np.concatenate([_f64(q[b]), _f64(qr[b])], 1)
        ref, spread, A, smax, _ = lp.attend(qq, np.concatenate([c, r], 1), c, sm)
        extra = 0.0 if g == 1.0 else lp.U_F16 * abs(sm) * (np.abs(_f64(q[b])) @ np.abs(c).T).max(1)
        bound = lp.attention_bound(ref, spread, A, smax, lp.U_F16, n, np.abs(c).max(), extra)
        err = np.abs(got[b] - ref)
        assert (err <= bound).all(), (b, n, (err / bound).max())


@pytest.mark.parametrize("lens,H,P,g,splits", [
    ([1], 1, 16, 1.0, 0),
    ([1, 0, 15, 16, 17], 16, 16, 1.0, 0),
    ([127, 128, 129], 32, 64, 0.75, 0),
    ([300, 700], 17, 32, 0.3712, 3),
    ([1000], 64, 128, 1.0, 0),
    ([640, 5, 0, 260], 96, 64, 0.75, 2),
    ([900, 130], 128, 32, 1.0, 1),
    ([513], 5, 16, 1.0, 7),
    ([40] * 30, 16, 16, 1.0, 0),
    ([40, 0] * 20, 40, 16, 1.0, 5),
    ([300, 129, 0, 257] * 14, 32, 16, 1.0, 0),       # more tiles than SMs: head tiles of 32
    ([300, 1, 280, 256] * 12, 64, 64, 0.75, 0),      # ... and of 64
    ([260, 300, 40] * 14, 96, 32, 1.0, 0),
    ([300, 200] * 20, 128, 128, 1.0, 0),
    ([700] * 16, 40, 32, 1.0, 9),
])
def test_decode_matches_the_formula(m, lens, H, P, g, splits):
    cache, bt = _filled(m, lens, P, 11 + H, g)
    q, qr = _rand((len(lens), H, 512), 1, 0.5), _rand((len(lens), H, 64), 2)
    ws = m.alloc_latent_decode_workspace(cache, len(lens), H, splits)
    ws.fill_(0xFF)                            # a byte read before it is written would show as a NaN
    out = m.latent_decode_attention(cache, q, qr, _cuda(bt), _cuda(lens), workspace=ws, num_splits=splits)
    torch.cuda.synchronize()
    assert m.check_device_errors() == 0
    _check_decode(m, out, cache, bt, lens, P, q, qr, g)


@pytest.mark.parametrize("B", [130, 700])
def test_decode_of_many_sequences(m, B):
    """More sequences than a warp, and than a CTA, scans at once; some empty, more splits than tiles."""
    lens = np.random.RandomState(B).randint(0, 60, B).tolist()
    cache, bt = _filled(m, [sum(lens)], 16, B)
    rows = torch.randperm(cache.num_pages, generator=torch.Generator().manual_seed(B))
    bt = np.stack([np.roll(rows.numpy(), i)[:4] for i in range(B)]).astype(np.int32)   # pages shared by several
    q, qr = _rand((B, 16, 512), 1, 0.5), _rand((B, 16, 64), 2)
    for splits in (0, 1500):
        out = m.latent_decode_attention(cache, q, qr, _cuda(bt), _cuda(lens), num_splits=splits)
        torch.cuda.synchronize()
        assert m.check_device_errors() == 0
        _check_decode(m, out, cache, bt, lens, 16, q, qr, 1.0)


@pytest.mark.parametrize("H", [16, 32, 64])
def test_decode_with_rising_scores_rescales(m, H):
    """Keys whose scores grow along the sequence move the running maximum again and again."""
    P, n = 64, 1500
    bt, pages = _table([n], P, 3)
    cache = m.LatentCache(pages, P)
    g = torch.randn(512, generator=_gen(5), device="cuda")
    ramp = torch.linspace(0, 12, n, device="cuda")[:, None]
    lat = (torch.randn((n, 512), generator=_gen(6), device="cuda") * 0.2 + ramp * g / 25).to(torch.bfloat16)
    rope = _rand((n, 64), 7, 0.1)
    m.latent_quantize_append(cache, lat, rope, _cuda(_slots(bt[0], P, n), torch.int64))
    q = (g / 4).to(torch.bfloat16).expand(1, H, 512).contiguous()
    qr = _rand((1, H, 64), 8, 0.1)
    for sm in (SM, -SM, 0.0):
        for B in (1, 20):                     # (20: more tiles than SMs, larger head tiles)
            out = m.latent_decode_attention(cache, q.expand(B, H, 512).contiguous(), qr.expand(B, H, 64).contiguous(),
                                            _cuda(np.repeat(bt, B, 0)), _cuda([n] * B), sm_scale=sm, num_splits=2 * B)
            torch.cuda.synchronize()
            _check_decode(m, out[-1:], cache, bt, [n], P, q, qr, 1.0, sm)
    for sm in (SM, -SM, 0.0):
        out = m.latent_decode_attention(cache, q, qr, _cuda(bt), _cuda([n]), sm_scale=sm, num_splits=2)
        torch.cuda.synchronize()
        _check_decode(m, out, cache, bt, [n], P, q, qr, 1.0, sm)


def test_decode_ignores_rows_behind_the_sequence(m):
    """NaN scales, infinities and NaN rotary values in rows past the length and in pages that
    the sequence does not list."""
    P, n, H = 32, 75, 16
    cache, bt = _filled(m, [n], P, 21)
    clean = cache.pool.clone()
    q, qr = _rand((1, H, 512), 1), _rand((1, H, 64), 2)
    want = m.latent_decode_attention(cache, q, qr, _cuda(bt), _cuda([n])).clone()
    dirty = clean.view(-1, 416 * P).clone()
    last = dirty[int(bt[0, n // P])].view(-1, 6656)
    r0 = n % P
    for r in range(r0, P):
        grp = last[r // 16]
        grp[4096:4608].view(16, 32)[r % 16] = 0x7F          # E4M3 NaN
        grp[4608:].view(16, 128)[r % 16] = 0xFF             # BF16 NaN
    cache.pool.copy_(dirty.view_as(cache.pool))
    out = m.latent_decode_attention(cache, q, qr, _cuda(bt), _cuda([n]))
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_decode_extreme_queries(m):
    """Query magnitudes far from 1, zero queries, a rotary part much larger than the latent one."""
    P, lens, H = 64, [200], 16
    cache, bt = _filled(m, lens, P, 31)
    for s, t in ((1e-20, 1.0), (0.0, 1.0), (1.0, 0.0), (0.0, 0.0), (1e-30, 1e-30), (0.01, 4.0)):
        q, qr = _rand((1, H, 512), 3, s), _rand((1, H, 64), 4, t)
        out = m.latent_decode_attention(cache, q, qr, _cuda(bt), _cuda(lens))
        torch.cuda.synchronize()
        _check_decode(m, out, cache, bt, lens, P, q, qr, 1.0)


def test_decode_bad_page_and_length_are_flagged(m):
    cache, bt = _filled(m, [100], 16, 41)
    q, qr = _rand((1, 16, 512), 1), _rand((1, 16, 64), 2)
    bad = bt.copy()
    bad[0, 2] = cache.num_pages               # reads as zeros
    out = m.latent_decode_attention(cache, q, qr, _cuda(bad), _cuda([100]))
    torch.cuda.synchronize()
    assert m.check_device_errors() == -4
    _check_decode(m, out, cache, bad, [100], 16, q, qr, 1.0)
    out = m.latent_decode_attention(cache, q, qr, _cuda(bt), _cuda([10**6]))      # cut to the table
    torch.cuda.synchronize()
    assert m.check_device_errors() == -4
    assert torch.equal(out, m.latent_decode_attention(cache, q, qr, _cuda(bt), _cuda([bt.shape[1] * 16])))
    assert (m.latent_decode_attention(cache, q, qr, _cuda(bt), _cuda([-3])) == 0).all()
    torch.cuda.synchronize()
    assert m.check_device_errors() == -4


def test_decode_on_other_streams_and_in_graphs(m):
    lens = [700, 33, 0, 260]
    cache, bt = _filled(m, lens, 64, 51)
    q, qr = _rand((4, 32, 512), 1), _rand((4, 32, 64), 2)
    b, n = _cuda(bt), _cuda(lens)
    want = m.latent_decode_attention(cache, q, qr, b, n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [m.latent_decode_attention(cache, q, qr, b, n, stream=side) for _ in range(4)]   # workspaces of its own each
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graphs, res = [], []
    for _ in range(2):                        # two graphs, a workspace each
        out, ws = torch.zeros_like(q), m.alloc_latent_decode_workspace(cache, 4, 32)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.latent_decode_attention(cache, q, qr, b, n, out=out, workspace=ws)
        graphs.append((g, ws))
        res.append(out)
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in res)
    assert m.check_device_errors() == 0
    n.copy_(_cuda([70, 3, 5, 0]))             # new lengths in the static buffer; row 2 lists no pages for its 5
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert m.check_device_errors() == -4
    assert torch.equal(res[0], m.latent_decode_attention(cache, q, qr, b, n))
    m.check_device_errors()


def test_pages_beyond_four_gigabytes(m):
    """The same rows in the last pages of a pool of more than 2^32 bytes: append, dequant and
    decode give what they give in a small one."""
    P, lens = 128, [300, 77]
    small, bt = _filled(m, lens, P, 71)
    pages = (1 << 32) // (416 * P) + 8
    big = m.LatentCache(pages, P, pool=torch.empty((pages, 416 * P), dtype=torch.uint8, device="cuda"))
    far = np.where(bt >= 0, pages - 1 - bt, -1).astype(np.int32)
    for old, new in zip(bt[bt >= 0], far[far >= 0]):
        big.pool[int(new)].fill_(0)
        big.pool[int(new)] = small.pool[int(old)]
    x = _rand((1, 576), 72)                   # one more token of sequence 1, into both
    for cache, table in ((small, bt), (big, far)):
        m.latent_quantize_append(cache, x[:, :512], x[:, 512:], _cuda([int(table[1, 0]) * P + 77], torch.int64))
    lens[1] += 1
    q, qr = _rand((2, 16, 512), 73, 0.5), _rand((2, 16, 64), 74)
    got = []
    for cache, table in ((small, bt), (big, far)):
        o = m.latent_decode_attention(cache, q, qr, _cuda(table), _cuda(lens))
        got.append((o, *m.latent_prefix_dequant(cache, _cuda(table), _cuda(lens), _cuda([0, 300, 378]), 378)))
    torch.cuda.synchronize()
    assert m.check_device_errors() == 0
    assert all(torch.equal(a, b) for a, b in zip(*got))


# ------------------------------------------------------------------ expanded extend

def _extend(m, pre, new, H, seed, strided=True, max_q=None):
    cp, cq = np.concatenate([[0], np.cumsum(pre)]), np.concatenate([[0], np.cumsum(new)])
    TP, TQ = int(cp[-1]), int(cq[-1])
    q = _rand((TQ, H, 192), seed)
    if strided:                               # halves of one projection output
        a, b = _rand((TP, H, 256), seed + 1), _rand((TQ, H, 256), seed + 2)
        kv = a[..., :128], a[..., 128:], b[..., :128], b[..., 128:]
    else:                                     # head-major
        kv = [_rand((H, n, 128), seed + i).transpose(0, 1) for i, n in enumerate((TP, TP, TQ, TQ))]
    r0, r1 = _rand((TP, 64), seed + 7), _rand((TQ, 64), seed + 8)
    out = m.latent_extend_attention(q, kv[0], kv[1], r0, _cuda(cp), kv[2], kv[3], r1, _cuda(cq), max_q or max(new))
    torch.cuda.synchronize()
    return out, (q, kv, r0, r1, cp, cq)


def _check_extend(out, data, sm=SM):
    q, kv, r0, r1, cp, cq = data
    got, H = _f64(out), out.shape[1]
    k0, v0, k1, v1 = (_f64(x) for x in kv)
    qd, p0, p1 = _f64(q), _f64(r0), _f64(r1)
    for r in range(len(cq) - 1):
        n, c = int(cp[r + 1] - cp[r]), int(cq[r + 1] - cq[r])
        if c == 0:
            continue
        mask = np.arange(n + c)[None, :] <= n + np.arange(c)[:, None]
        rope = np.concatenate([p0[cp[r]:cp[r + 1]], p1[cq[r]:cq[r + 1]]])
        for h in range(H):
            k = np.concatenate([k0[cp[r]:cp[r + 1], h], k1[cq[r]:cq[r + 1], h]])
            v = np.concatenate([v0[cp[r]:cp[r + 1], h], v1[cq[r]:cq[r + 1], h]])
            ref, spread, A, smax, _ = lp.attend(qd[cq[r]:cq[r + 1], h], np.concatenate([k, rope], 1), v, sm, mask)
            bound = lp.attention_bound(ref, spread, A, smax, lp.U_BF16, n + c, np.abs(v).max())
            err = np.abs(got[cq[r]:cq[r + 1], h] - ref)
            assert (err <= bound).all(), (r, h, (err / bound).max())


@pytest.mark.parametrize("pre,new,H,strided", [
    ([0], [1], 1, True),
    ([1], [1], 2, False),
    ([100, 0, 127], [17, 5, 64], 3, True),
    ([128, 300], [128, 0], 2, True),
    ([64, 500], [129, 260], 2, False),
    ([1100], [257], 1, True),                 # split over a cluster: odd tiles, a part without visible keys
    ([0, 2000], [300, 2], 1, True),
    ([1500], [600], 2, True),
    ([5] * 40, [3] * 40, 1, True),
])
def test_extend_matches_the_formula(m, pre, new, H, strided):
    out, data = _extend(m, pre, new, H, sum(pre) + sum(new), strided)
    assert m.check_device_errors() == 0
    _check_extend(out, data)


def test_extend_many_requests_of_different_shapes(m):
    rng = np.random.RandomState(4)
    pre, new = rng.randint(0, 400, 300).tolist(), rng.randint(0, 20, 300).tolist()   # more requests than are sorted
    out, data = _extend(m, pre, new, 1, 5)
    assert m.check_device_errors() == 0
    _check_extend(out, data)


def test_extend_ignores_rows_of_others(m):
    """NaN and infinities in the rows of other requests and behind the last one do not reach a
    request's output."""
    pre, new, H = [70, 90], [20, 30], 2
    cp, cq = np.concatenate([[0], np.cumsum(pre)]), np.concatenate([[0], np.cumsum(new)])
    q, a, b = _rand((60, H, 192), 1), _rand((180, H, 256), 2), _rand((60, H, 256), 3)
    r0, r1 = _rand((180, 64), 4), _rand((60, 64), 5)

    def run():
        return m.latent_extend_attention(q, a[..., :128], a[..., 128:], r0, _cuda(cp), b[..., :128], b[..., 128:], r1,
                                         _cuda(cq), 30)
    want = run().clone()
    a[70:] = float("nan")                     # the second request's prefix and the padding
    r0[70:] = float("inf")
    b[20:] = float("nan")
    r1[20:] = float("nan")
    out = run()
    torch.cuda.synchronize()
    assert m.check_device_errors() == 0
    assert torch.equal(out[:20], want[:20])


def test_extend_flags_inconsistent_lengths_and_leaves_other_rows(m):
    H = 1
    q, b, r1 = _rand((40, H, 192), 1), _rand((40, H, 256), 2), _rand((40, 64), 3)
    none, r0 = torch.zeros((0, H, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full((40, H, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    cut = m.latent_extend_attention(q, none, none, r0, _cuda([0, 0]), b[..., :128], b[..., 128:], r1, _cuda([0, 30]), 16,
                                    out=out)   # a chunk longer than the bound is cut and flagged
    torch.cuda.synchronize()
    assert m.check_device_errors() == -4
    assert (cut[16:] == 9.0).all() and (cut[:16] != 9.0).any()
    out.fill_(9.0)
    m.latent_extend_attention(q, none, none, r0, _cuda([0, 5]), b[..., :128], b[..., 128:], r1, _cuda([0, 30]), 30, out=out)
    torch.cuda.synchronize()                  # a prefix that the caller has no rows for
    assert m.check_device_errors() == -4 and (out == 9.0).all()
    m.latent_extend_attention(q, none, none, r0, _cuda([0, 0]), b[..., :128], b[..., 128:], r1, _cuda([0, 50]), 50, out=out)
    torch.cuda.synchronize()                  # rows past the chunk tensors
    assert m.check_device_errors() == -4 and (out == 9.0).all()


def test_extend_in_a_graph_and_on_another_stream(m):
    out, (q, kv, r0, r1, cp, cq) = _extend(m, [300, 40], [50, 129], 4, 9)
    args = (q, kv[0], kv[1], r0, _cuda(cp), kv[2], kv[3], r1, _cuda(cq), 129)
    side = torch.cuda.Stream()
    other = m.latent_extend_attention(*args, stream=side)
    res = torch.zeros_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.latent_extend_attention(*args, out=res)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(other, out) and torch.equal(res, out)


# ------------------------------------------------------------------ side by side

def test_calls_on_several_streams_at_once(m):
    """Decode calls of different head counts and extends on four streams, each with buffers of its
    own, give what they give alone."""
    lens = [900, 33, 400]
    cache, bt = _filled(m, lens, 64, 81)
    b, n = _cuda(bt), _cuda(lens)
    qs = {H: (_rand((3, H, 512), H, 0.5), _rand((3, H, 64), H + 1)) for H in (16, 64, 128)}
    want = {H: m.latent_decode_attention(cache, *q, b, n) for H, q in qs.items()}
    ext, (q, kv, r0, r1, cp, cq) = _extend(m, [600, 40], [50, 129], 4, 9)
    args = (q, kv[0], kv[1], r0, _cuda(cp), kv[2], kv[3], r1, _cuda(cq), 129)
    torch.cuda.synchronize()
    streams = {x: torch.cuda.Stream() for x in (16, 64, 128, "extend")}
    got = []
    for _ in range(6):
        for H in qs:
            got.append((want[H], m.latent_decode_attention(cache, *qs[H], b, n, stream=streams[H])))
        got.append((ext, m.latent_extend_attention(*args, stream=streams["extend"])))
    torch.cuda.synchronize()
    assert m.check_device_errors() == 0
    assert all(torch.equal(x, y) for x, y in got)


# ------------------------------------------------------------------ together

def test_absorbed_and_expanded_forms_agree(m):
    """Prefill and decode as a model runs them: latents appended, the prefix expanded through
    the up-projections and attended by a chunk; the chunk's last token decoded again in the
    absorbed form over the cache.  Both approximate one value, whose up-projections are exact
    here; each is held to the formula in 64 bits on the cache's own bytes."""
    H, P, n, L = 4, 32, 210, 9
    bt, pages = _table([n], P, 61)
    cache = m.LatentCache(pages, P)
    x = _rand((n, 576), 62)
    m.latent_quantize_append(cache, x[:, :512], x[:, 512:], _cuda(_slots(bt[0], P, n), torch.int64))
    wk, wv = _rand((H, 128, 512), 63, 0.05), _rand((H, 128, 512), 64, 0.05)
    lat, rope = m.latent_prefix_dequant(cache, _cuda(bt), _cuda([n]), _cuda([0, n]), n)
    k = torch.einsum("tc,hdc->thd", lat.float(), wk.float()).to(torch.bfloat16)
    v = torch.einsum("tc,hdc->thd", lat.float(), wv.float()).to(torch.bfloat16)
    q = _rand((L, H, 192), 65)
    p = n - L
    out = m.latent_extend_attention(q, k[:p], v[:p], rope[:p], _cuda([0, p]), k[p:], v[p:], rope[p:].contiguous(),
                                    _cuda([0, L]), L)
    q_abs = torch.einsum("hd,hdc->hc", q[-1, :, :128].float(), wk.float()).to(torch.bfloat16)[None]
    o = m.latent_decode_attention(cache, q_abs, q[-1:, :, 128:].contiguous(), _cuda(bt), _cuda([n]))
    torch.cuda.synchronize()
    assert m.check_device_errors() == 0
    _check_extend(out, (q, (k[:p], v[:p], k[p:], v[p:]), rope[:p], rope[p:], [0, p], [0, L]))
    _check_decode(m, o, cache, bt, [n], P, q_abs, q[-1:, :, 128:], 1.0)
    # The two forms differ in roundings to BF16 alone.  A score moves by at most d = ub sm_scale
    # (sum |q||k| + sum |q_abs||latent|) (the rounded K, the rounded absorbed query), a weight then
    # by a factor of at most e^(2d), the output by (e^(2d) - 1) 2 max|v|; the weights' own roundings
    # move it by 2 ub of a spread of at most 2 max|v|, V's and the output's by ub max|v| each, and
    # the absorbed output's by ub sum |o||w|.
    up = torch.einsum("hc,hdc->hd", o[0].float(), wv.float())
    A = (q[-1, :, :128].abs().float()[None] * k.abs().float()).sum(-1).max() + \
        torch.einsum("hc,tc->ht", q_abs[0].abs().float(), lat.abs().float()).max()
    d = lp.U_BF16 * SM * float(A)
    vmax = float(v.abs().max())
    bound = ((math.exp(2 * d) - 1) * 2 + 6 * lp.U_BF16) * vmax + lp.U_BF16 * float(
        torch.einsum("hc,hdc->hd", o[0].abs().float(), wv.abs().float()).max())
    assert float((up - out[-1].float()).abs().max()) <= bound
