"""The operators of a speculative decoding step in 64 bits, from their formulas: head norms and
rotation, the attention of drafted tokens over the cache, and the rows that an acceptance moves.

Tolerances of the GPU tests:

  * the rotated query is FP32 rounded to BF16: half a BF16 step, 2^-8 relative, and 2^-20 of the
    pair's products for the FP32 steps before it (two products, a sum, a reciprocal root and its
    product, each 2^-24, the root 2^-22, a sum of 128 squares 2^-17 at most, which the root halves
    and which is common to the row: 2^-18 relative to the value, below a BF16 step's 2^-8 / 1000);
  * the rotated key is the exact value's rounding to BF16, so the pool's bytes are compared;
  * tree attention: each weight is rounded to FP16 (2^-11 relative), the same rounded weights in
    numerator and denominator, so the output moves by at most 2^-11 of the spread sum_t w_t |v_t -
    ref|; the score's FP32 sum of 128 products is off by at most 128 x 2^-24 = 2^-17 of sum |q_i
    k_i| sm_scale (below 32 in these tests), which is 2^-12 relative to a weight, and the exponent's
    argument, its factor and the approximate 2^x, tanh's two approximations among them, by 2^-14;
    FP32 accumulation moves the output by 2^-17 of sum_t w_t |v_t|; the output is rounded to BF16,
    2^-8 relative.  A weight below 2^-21 of the largest has an absolute error of 2^-32 of it: n 2^-32 max |v|.
"""

import math

import torch

HEAD = 128
GROUP = 2304


# ------------------------------------------------------------------------------ norms and rotation

def bf16_rounded(x):
    """64-bit numbers rounded to BF16 once, nearest even (a conversion would pass through 32 bits)."""
    step = torch.ldexp(torch.ones_like(x), torch.frexp(x).exponent.clamp(min=-125) - 8)
    return (torch.round(x / step) * step).to(torch.bfloat16)


def turned(x, weight, positions, cos_sin, eps, adjacent, sections):
    """(y, the pairs' larger products) of heads x [T][H][128] in 64 bits, not rounded."""
    x = x.double().clone()
    if weight is not None:
        x = x * weight.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    size = x.abs()
    if cos_sin is None:
        return x, size
    rot = cos_sin.shape[1]
    axis, out = 0, x.clone()
    for i in range(rot // 2):
        if sections is not None:
            axis = next(a for a in range(len(sections)) if i < sum(sections[:a + 1]))
        row = cos_sin[(positions[axis] if positions.dim() == 2 else positions).long()].double()
        c, s = row[:, i, None], row[:, rot // 2 + i, None]
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = torch.maximum(x[..., a].abs(), x[..., b].abs())
    return out, size


# ------------------------------------------------------------------------------ the cache's rows

def _e2m1(code):
    e, m = (code % 8) // 2, (code % 2).double()
    v = torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1) * (1 + 0.5 * m))
    return torch.where(code >= 8, -v, v)


def _codes(b):
    b = b.to(torch.int64)
    return _e2m1(torch.stack([b % 16, b // 16], -1).flatten(-2))


def rows_of(pool, page, pages, n):
    """K and V [kv heads][n][128] of the first n tokens in `pages`, without tensor scales, in 64 bits."""
    slabs = pool[pages[: -(-n // page)].long()].view(-1, pool.shape[1], page // 16, GROUP).transpose(0, 1)
    slabs = slabs.reshape(pool.shape[1], -1, GROUP)
    ks = slabs[..., 1024:1152].contiguous().view(torch.float8_e4m3fn).double().unflatten(-1, (16, 8))
    vs = slabs[..., 2176:].contiguous().view(torch.float8_e4m3fn).double().unflatten(-1, (8, 16)).transpose(-1, -2)
    k = _codes(slabs[..., :1024]).unflatten(-1, (16, 8, 16)) * ks[..., None]
    v = _codes(slabs[..., 1152:2176]).unflatten(-1, (16, 8, 16)) * vs[..., None]
    return k.reshape(pool.shape[1], -1, HEAD)[:, :n], v.reshape(pool.shape[1], -1, HEAD)[:, :n]


# ------------------------------------------------------------------------------ tree attention

def masks_of(parents):
    """Bit masks (Python numbers) of the drafts whose parents these are (-1: none)."""
    m = []
    for i, p in enumerate(parents):
        m.append((m[p] if p >= 0 else 0) | 1 << i)
    return m


def signed(m):
    return m - (1 << 64) if m >> 63 else m


def tree(q, k, v, masks, n, scale, cap=0.0, window=0, slopes=None, gone=()):
    """One sequence: q [d][Hq][128], k and v [kv heads][n][128], masks of the d drafts; tokens in `gone` are not seen.
    -> (out [d][Hq][128], spread, sum of w |v|)."""
    d, hq = q.shape[0], q.shape[1]
    hkv = k.shape[0]
    g, base = hq // hkv, n - d
    depth = [bin(m).count("1") - 1 for m in masks]
    place = torch.tensor(list(range(base)) + [base + x for x in depth], dtype=torch.float64)
    sees = torch.ones((d, n), dtype=torch.bool)
    for i in range(d):
        sees[i, base:] = torch.tensor([bool(masks[i] >> j & 1) for j in range(d)], dtype=torch.bool)
    away = place[None, :] - place[base:, None]
    if window:
        sees &= away > -window
    sees[:, list(gone)] = False
    out, spread, size = (torch.zeros((d, hq, HEAD), dtype=torch.float64) for _ in range(3))
    for h in range(hq):
        z = q[:, h].double() @ k[h // g].T * scale
        if cap:
            z = cap * torch.tanh(z / cap)
        if slopes is not None:
            z = z + slopes[h].double() * away
        z = z.masked_fill(~sees, -math.inf)
        w = torch.nan_to_num(torch.softmax(z, -1), nan=0.0) if not sees.any(1).all() else torch.softmax(z, -1)
        w = torch.where(sees.any(1, keepdim=True), w, 0.0)
        if torch.isnan(v[h // g]).any():     # (0 times the NaN of a token that is not seen would be one)
            out[:, h] = torch.stack([w[i][sees[i]] @ v[h // g][sees[i]] for i in range(d)])
            continue
        out[:, h] = w @ v[h // g]
        spread[:, h] = torch.einsum("dn,dnc->dc", w, (v[h // g][None] - out[:, h][:, None]).abs()) if d * n <= 20000 else \
            torch.stack([(w[i][:, None] * (v[h // g] - out[i, h]).abs()).sum(0) for i in range(d)])
        size[:, h] = w @ v[h // g].abs()
    return out, spread, size


def tree_bound(ref, spread, size, n, vmax):
    return 2.0**-8 * ref.abs() + (2.0**-11 + 2.0**-12 + 2.0**-14) * spread + 2.0**-16 * size + n * 2.0**-32 * vmax + 1e-30
