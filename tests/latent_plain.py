"""Plain 64-bit implementations for the tests of the latent cache, of the
attention-weight scores and of the eviction (numpy, written from the formulas
and the page layouts of include/nvfp4kv.h), and the tolerances.

A rounding to nearest is off by at most half a step: u16 = 2^-11 for FP16, ub =
2^-8 for BF16, relative to the value.  The tolerance of an attention output

    out = sum_t w_t v_t / sum_t w_t,   w_t = 2^(s_t - m)

counts, per element, with spread = sum_t w_t |v_t - out| / sum_t w_t:

  * the kernel's score s is off by at most d = 2^-16 A + 2^-21 |s|max + r: FP32
    sums of exact products over 12 or 36 steps of 16 lose at most 2 units of 2^-23
    of the partial sums each, below 2^-16 of A = sm_scale sum_i |q_i k_i|; the
    product with the score factor and the subtraction round twice in FP32; r =
    2^-11 of the latent part of A where a tensor scale other than 1 is folded into
    the FP16 query;
  * a weight is then off by a factor of at most e^(2d) and by its rounding (u16 or
    ub; 2^-22 for the exponential), below p = 3 d + u + 2^-20 in all while d < 0.2;
    the same rounded weights form numerator and denominator, so the output moves
    by at most 2 p spread (first order p spread);
  * weights that fall below FP16's normal range (2^-21 of the largest) are off by at
    most 2^-32 of the largest: n 2^-31 max|v| covers all of them;
  * FP32 accumulation: 2^-16 (spread + |out|); the BF16 result: ub |out|.
"""

import math

import numpy as np

U_F16, U_BF16 = 2.0**-11, 2.0**-8
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
MIDS = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
E4M3 = np.array([(m * 2.0**-9 if e == 0 else (8 + m) * 2.0**(e - 10)) for e in range(16) for m in range(8)][:127])


def bf16_to_f64(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def round_bf16(x):
    """float64 -> the nearest BF16 value (ties to even), as float64 (normal range)."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def quantise(x, g):
    """[..., 16k] values -> (codes uint8 [..., 16k], scale bytes uint8 [..., k]), each the
    rounding of the exact quotient (borders compared as exact products)."""
    g = float(np.float32(g))
    b = x.reshape(x.shape[:-1] + (-1, 16))
    amax = np.abs(b).max(-1)
    grid = E4M3 * (6.0 * g)
    hi = np.clip(np.searchsorted(grid, amax), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - amax, amax - grid[lo]
    s = np.where((amax >= grid[126]) | (up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    s = np.where(amax == 0, 0, s).astype(np.uint8)
    step = (E4M3[s] * g)[..., None]
    a = np.abs(b)
    code = np.zeros(b.shape, np.uint8)
    for i, mid in enumerate(MIDS):      # a tie goes to the even code
        code[(a > mid * step) | ((a == mid * step) & (i % 2 == 1))] = i + 1
    code[np.broadcast_to(step == 0, b.shape)] = 0
    code = code | (np.signbit(b).astype(np.uint8) << 3)
    return code.reshape(x.shape), s


def latent_rows(codes, scales, rope_bits):
    """The 416 bytes of each row as (codes uint8 [T][8][32], scales uint8 [T][32], rotary uint8 [T][8][16])
    in their order in a group (the rotary chunks before their exchange)."""
    T = codes.shape[0]
    c = codes.reshape(T, 8, 32, 2)
    packed = c[..., 0] | (c[..., 1] << 4)
    blk = np.arange(32)
    pos = (blk // 2 % 2) * 16 + blk // 4 * 2 + blk % 2
    sc = np.zeros((T, 32), np.uint8)
    sc[:, pos] = scales
    return packed, sc, rope_bits.astype("<u2").view(np.uint8).reshape(T, 8, 16)


def write_latent(pool, page_size, slots, rows):
    """Puts rows (latent_rows) into pool uint8 [pages][416 P] at slots (negative: skipped)."""
    packed, sc, rope = rows
    for i, slot in enumerate(np.asarray(slots)):
        if slot < 0:
            continue
        page, r = divmod(int(slot), page_size)
        grp = pool[page, (r // 16) * 6656:(r // 16 + 1) * 6656]
        r %= 16
        grp[:4096].reshape(8, 16, 32)[:, r] = packed[i]
        grp[4096:4608].reshape(16, 32)[r] = sc[i]
        for c in range(8):
            grp[4608:].reshape(16, 8, 16)[r, c ^ (r % 8)] = rope[i, c]


def read_latent(pool, page_size, table_row, n, g):
    """float64 latents [n][512] and rotary parts [n][64] of a sequence."""
    out, rope = np.zeros((n, 512)), np.zeros((n, 64))
    blk = np.arange(32)
    pos = (blk // 2 % 2) * 16 + blk // 4 * 2 + blk % 2
    for t in range(n):
        page, r = int(table_row[t // page_size]), t % page_size
        if not 0 <= page < pool.shape[0]:
            continue
        grp = pool[page, (r // 16) * 6656:(r // 16 + 1) * 6656]
        r %= 16
        by = grp[:4096].reshape(8, 16, 32)[:, r]
        v = np.stack([E2M1[by & 15], E2M1[by >> 4]], -1).reshape(32, 16)
        out[t] = (v * E4M3[grp[4096:4608].reshape(16, 32)[r][pos]][:, None]).reshape(512) * float(np.float32(g))
        ch = grp[4608:].reshape(16, 8, 16)[r][[c ^ (r % 8) for c in range(8)]]
        rope[t] = bf16_to_f64(np.ascontiguousarray(ch).reshape(-1).view("<u2"))
    return out, rope


def attend(q, k, v, sm, mask=None):
    """float64 attention of q [R][dk] over k [n][dk], v [n][dv] (mask [R][n] of seen keys):
    (out, spread, A, |s|max)."""
    s = sm * (q @ k.T)
    A = abs(sm) * (np.abs(q) @ np.abs(k).T)
    if mask is not None:
        s, A = np.where(mask, s, -np.inf), np.where(mask, A, 0.0)
    top = s.max(1, keepdims=True)
    w = np.exp(s - top)
    w = w / w.sum(1, keepdims=True)
    out = w @ v
    spread = np.stack([(w[i][:, None] * np.abs(v - out[i])).sum(0) for i in range(q.shape[0])])
    return out, spread, A.max(1), np.abs(np.where(np.isfinite(s), s, 0)).max(1), w


def attention_bound(out, spread, A, smax, u, n, vmax, extra=0.0):
    d = 2.0**-16 * A + 2.0**-21 * smax + extra
    assert (d < 0.2).all()
    p = (3 * d + u + 2.0**-20)[:, None]
    return U_BF16 * np.abs(out) + (1 + U_BF16) * (2 * p * spread + 2.0**-16 * (spread + np.abs(out)) + n * 2.0**-31 * vmax)


def evict_plain(scores, n, keep, recent, sink):
    """Kept row indices of one segment, ascending: the rows of largest score, ties to the
    lowest index, NaN below everything."""
    if n <= keep:
        return np.arange(n)
    key = np.where(np.isnan(scores[:n]), -np.inf, scores[:n].astype(np.float64))
    rank_nan = np.isnan(scores[:n])
    t = np.arange(n)
    must = (t < sink) | (t >= n - recent)
    order = np.lexsort((t, rank_nan, -key, ~must))   # must first, then larger keys, numbers before NaN, low indices
    return np.sort(order[:keep])
