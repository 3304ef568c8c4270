"""Edges of the speculative decoding calls on the GPU: values behind the rotation, large caps, scales that are not
positive, many heads, and what stays as it was where a call flags its inputs."""

import math

import pytest
import torch

import speculative_plain as plain
from speculative_plain import HEAD
from test_gpu_speculative import gen, ints, packed, random_pool, random_tree, rotation, run_tree, sums, table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import nvfp4_quantised_paged_gb300 as mod
    return mod


def finite_rounded(y):
    """64-bit numbers rounded to BF16 once, infinities and NaN as they are."""
    fine = torch.isfinite(y)
    return torch.where(fine, plain.bf16_rounded(torch.where(fine, y, 1.0)).double(), y).to(torch.bfloat16)


# --------------------------------------------------------------------------------- rotated append

@pytest.mark.parametrize("T", [8, 6000])
@pytest.mark.parametrize("rot", [0, 32, 64])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("norms", [False, True])
def test_infinities_behind_the_rotation_stay_where_they_are(m, T, rot, adjacent, norms):
    """Infinities and NaN at rotated and at other values: y = u behind the rotation, and a norm that is infinite gives
    zeros (the rotation by angles whose cosine and sine are 0 or 1, so that every other product is exact)."""
    hq, hkv = 4, 4
    g = gen(rot + T)
    x = torch.randint(-8, 9, (T, hq + 2 * hkv, HEAD), generator=g).float()
    x[::5, 1, 127], x[1::7, 2, 100], x[2::9, 0, 70], x[3::4, 3, 3] = math.inf, math.nan, -math.inf, math.inf
    x[::3, hq, 127], x[1::7, hq + 1, 99], x[2::5, hq + 2, 66], x[3::4, hq + 3, 3] = -math.inf, math.nan, math.inf, math.inf
    half = rot // 2
    table = torch.tensor([[1.0] * half + [0.0] * half, [0.0] * half + [1.0] * half]) if rot else None
    pos = torch.randint(0, 2, (T,), generator=g, dtype=torch.int32)
    w = torch.exp2(torch.randint(-1, 2, (HEAD,), generator=g).float()).to(torch.bfloat16) if norms else None
    slots = torch.arange(T)
    pages = -(-T // 64)
    a, b = m.PagedCache(pages, 64, hkv), m.PagedCache(pages, 64, hkv)
    x = x.to(torch.bfloat16)
    q, k, v = x.cuda().split([hq, hkv, hkv], 1)
    on = lambda t: None if t is None else t.cuda()  # noqa: E731
    out = m.rope_quantize_append(a, q, k, v, pos.cuda(), on(table), slots.cuda(), q_norm=on(w), k_norm=on(w), eps=0.0,
                                 adjacent=adjacent).cpu()
    rq, _ = plain.turned(x[:, :hq], w, pos, table, 0.0, adjacent, None)
    rk, _ = plain.turned(x[:, hq:hq + hkv], w, pos, table, 0.0, adjacent, None)
    fine = torch.isfinite(rq)
    assert torch.equal(torch.isnan(out), torch.isnan(rq))
    assert torch.equal(torch.isinf(out), torch.isinf(rq))
    assert ((out.double() - rq)[fine].abs() <= (2.0**-8 + 2.0**-18) * rq[fine].abs()).all()   # half a step, and FP32's
    if not norms:
        assert torch.equal(torch.nan_to_num(out[..., rot:], nan=3.0), torch.nan_to_num(x[:, :hq, rot:], nan=3.0))
    m.quantize_append(b, packed(finite_rounded(rk)), packed(x[:, hq + hkv:]), slots.cuda())
    # (as values: where a row's norm is infinite, the order of rotation and norm decides a zero's sign)
    for ours, other in zip(*(plain.rows_of(c.pool.cpu(), 64, torch.arange(pages), T) for c in (a, b))):
        assert torch.equal(torch.isnan(ours), torch.isnan(other))
        assert torch.equal(torch.nan_to_num(ours), torch.nan_to_num(other))
    assert m.check_device_errors() == 0


@pytest.mark.parametrize("T", [9, 6000])
@pytest.mark.parametrize("rot,adjacent", [(0, False), (64, False), (64, True), (128, True)])
@pytest.mark.parametrize("norms", [False, True])
def test_zeros_keep_their_signs_in_the_pages(m, T, rot, adjacent, norms):
    hkv = 4
    g = gen(T + rot)
    x = torch.randint(-3, 4, (T, 2 * hkv, HEAD), generator=g).float()
    x = torch.where((x == 0) & (torch.rand(x.shape, generator=g) < 0.5), -x, x).to(torch.bfloat16)
    assert torch.signbit(x[x == 0]).any() and not torch.signbit(x[x == 0]).all()
    table = rotation(50, rot) if rot else None
    pos = torch.randint(0, 50, (T,), generator=g, dtype=torch.int32)
    w = (torch.randn(HEAD, generator=g) * 0.3 + 1).to(torch.bfloat16) if norms else None
    slots = torch.arange(T).cuda()
    a, b = m.PagedCache(-(-T // 64), 64, hkv), m.PagedCache(-(-T // 64), 64, hkv)
    on = lambda t: None if t is None else t.cuda()  # noqa: E731
    k, v = x.cuda().split([hkv, hkv], 1)
    m.rope_quantize_append(a, None, k, v, pos.cuda(), on(table), slots, k_norm=on(w), adjacent=adjacent)
    rk, _ = plain.turned(x[:, :hkv], w, pos, table, 1e-6, adjacent, None)
    m.quantize_append(b, packed(plain.bf16_rounded(rk)), packed(x[:, hkv:]), slots)
    assert torch.equal(a.pool, b.pool) and m.check_device_errors() == 0



@pytest.mark.parametrize("T", [9, 3000])
@pytest.mark.parametrize("size,scale,norms", [(2.0**-90, 2.0**-90, False), (2.0**-45, 1.0, True), (2.0**60, 1.0, True), (2.0**100, 2.0**98, False)])
def test_rows_far_from_one(m, T, size, scale, norms):
    """Products down to 2^-100, mean squares down to 2^-100 without an eps, and large ones: K's bytes are the formula's."""
    hq, hkv = 2, 8
    g = gen(T)
    x = (torch.randn((T, hq + 2 * hkv, HEAD), generator=g).clamp(-2.5, 2.5) * size).to(torch.bfloat16)
    table, pos = rotation(50, 64), torch.randint(0, 50, (T,), generator=g, dtype=torch.int32)
    w = (torch.rand(HEAD, generator=g) + 0.5).to(torch.bfloat16) if norms else None
    slots = torch.arange(T).cuda()
    a, b = (m.PagedCache(-(-T // 64), 64, hkv, k_global_scale=scale, v_global_scale=scale) for _ in range(2))
    on = lambda t: None if t is None else t.cuda()  # noqa: E731
    q, k, v = x.cuda().split([hq, hkv, hkv], 1)
    out = m.rope_quantize_append(a, q, k, v, pos.cuda(), table.cuda(), slots, q_norm=on(w), k_norm=on(w), eps=0.0)
    rq, top = plain.turned(x[:, :hq], w, pos, table, 0.0, False, None)
    rk, _ = plain.turned(x[:, hq:hq + hkv], w, pos, table, 0.0, False, None)
    m.quantize_append(b, packed(plain.bf16_rounded(rk)), packed(x[:, hq + hkv:]), slots)
    assert torch.equal(a.pool, b.pool) and bool((a.pool != 0).any()) and m.check_device_errors() == 0
    assert ((out.cpu().double() - rq).abs() <= 2.0**-8 * rq.abs() + 2.0**-16 * top).all()


@pytest.mark.parametrize("T", [1, 5, 6000])
def test_queries_written_between_the_rows_they_come_from(m, T):
    """An output of the same stride beside q, k and v in one row, and q itself; rows over others are refused."""
    hq, hkv = 4, 4
    g = gen(T)
    rows = torch.randn((T + 1, 2 * hq + 2 * hkv, HEAD), generator=g).to(torch.bfloat16).cuda()
    kept = rows.clone()
    q, k, v, out = rows[:T].split([hq, hkv, hkv, hq], 1)
    table, pos, slots = rotation(T, 128).cuda(), ints(list(range(T))), torch.arange(T, device="cuda")
    pages = -(-T // 64)
    a, b, c = (m.PagedCache(pages, 64, hkv) for _ in range(3))
    want = m.rope_quantize_append(a, q, k, v, pos, table, slots)
    assert m.rope_quantize_append(b, q, k, v, pos, table, slots, q_out=out).data_ptr() == out.data_ptr()
    assert torch.equal(out, want) and torch.equal(rows[:T, :-hq], kept[:T, :-hq]) and torch.equal(rows[T:], kept[T:])
    for bad in (k, v, rows[:T, 1:hq + 1], rows[:T, hq - 1:2 * hq - 1], rows[1:, :hq] if T > 1 else k, rows[1:, 2:hq + 2] if T > 1 else v):
        with pytest.raises(m.NVFP4KVError):
            m.rope_quantize_append(c, q, k, v, pos, table, slots, q_out=bad)
    assert not c.pool.any()
    m.rope_quantize_append(c, q, k, v, pos, table, slots, q_out=q)
    assert torch.equal(q, want) and torch.equal(rows[:T, hq:3 * hq], kept[:T, hq:3 * hq])
    assert torch.equal(a.pool, b.pool) and torch.equal(a.pool, c.pool) and m.check_device_errors() == 0


# --------------------------------------------------------------------------------- tree attention

@pytest.mark.parametrize("cap", [1e-42, 1e-4, 0.02, 2.0, 30.0, 50.0, 128.0, 129.0, 1e3, 2e4, 1e6, 1e30, 3e38])
@pytest.mark.parametrize("lens,drafts,hq,hkv,page", [([300, 900, 20], [1, 1, 1], 8, 2, 16), ([300, 900, 20], [5, 12, 20], 8, 2, 16),
                                                     ([600, 410], [40, 64], 8, 2, 32)])
def test_caps_of_any_size(m, cap, lens, drafts, hq, hkv, page):
    """The tolerance of the other caps: a capped score is off by 2^-20 of itself, and scores stay below 32 here, so its
    weight by 2^-15; with caps from 2^-10 to 128 by 1.3 x 2^-22 of the cap, its weight by 2^-14.6: inside the 2^-14 of the
    bound, whatever the cap."""
    run_tree(m, lens, drafts, hq, hkv, page, seed=3, cap=cap, qscale=2.0)


def test_a_cap_far_above_the_scores_is_none(m):
    """Both within their bound of the same numbers, and of each other: scores z off by z^3 / (3 cap^2) at most."""
    args = ([300, 900, 20], [5, 12, 20], 8, 2, 16)
    a = run_tree(m, *args, seed=3, qscale=2.0)
    b = run_tree(m, *args, seed=3, qscale=2.0, cap=1e6)
    # 2^-20 of scores below 32 moves a weight by 2^-15 and may round it (FP16, 2^-11) and the output (BF16, 2^-8) elsewhere
    assert ((a - b).abs() <= 2.0**-7 * a.abs() + 2.0**-10 * float(a.abs().max())).all()


def test_windows_and_counts_beyond_32_bits(m):
    """2^32 + 5 is no window of 5; the largest number that fits limits nothing."""
    g = gen(5)
    table, pages = table_of([300], 16, g)
    cache = m.PagedCache(pages, 16, 2, pool=random_pool(pages, 2, 16, 5).cuda())
    args = (cache, torch.randn((3, 8, HEAD), generator=g).to(torch.bfloat16).cuda(), sums([3]), 3, table.cuda(), ints([300]))
    for kw in (dict(window=2**32 + 5), dict(window=2**31), dict(num_splits=2**32 + 1)):
        with pytest.raises(ValueError):
            m.tree_attention(*args, **kw)
    with pytest.raises(ValueError):
        m.tree_attention(*args[:3], 2**32 + 3, *args[4:])
    assert torch.equal(m.tree_attention(*args, window=2**31 - 1), m.tree_attention(*args)) and m.check_device_errors() == 0


def check_rows(got, q, pool, page, pages, masks, n, scale=1 / math.sqrt(HEAD), **kw):
    """The drafts' outputs of one sequence against the formula, within its bound."""
    k, v = plain.rows_of(pool, page, pages, n)
    ref, spread, size = plain.tree(q, k, v, masks, n, scale, **kw)
    err = (got.cpu().double() - ref).abs()
    assert (err <= plain.tree_bound(ref, spread, size, n, float(v.abs().max()))).all()


@pytest.mark.parametrize("scale", [-0.11, 0.0, 1e-30])
@pytest.mark.parametrize("kw", [{}, dict(cap=30.0), dict(cap=1e5), dict(window=70), dict(cap=3.0, window=5, sloped=True)])
@pytest.mark.parametrize("d,hq", [(1, 8), (9, 8), (33, 16)])
def test_scales_that_are_not_positive(m, scale, kw, d, hq):
    g = gen(d)
    n, page, hkv = 310, 16, 2
    table, pages = table_of([n], page, g)
    pool = random_pool(pages, hkv, page, 9)
    q = torch.randn((d, hq, HEAD), generator=g).to(torch.bfloat16)
    masks = plain.masks_of(random_tree(d, g))
    slopes = torch.exp2(-torch.arange(1, hq + 1) * 8.0 / hq) if kw.get("sloped") else None
    cap, window = kw.get("cap", 0.0), kw.get("window", 0)
    got = m.tree_attention(m.PagedCache(pages, page, hkv, pool=pool.cuda()), q.cuda(), sums([d]), d, table.cuda(), ints([n]),
                           tree_mask=torch.tensor([plain.signed(x) for x in masks]).cuda(), sm_scale=scale, softcap=cap,
                           window=window, slopes=None if slopes is None else slopes.cuda())
    assert m.check_device_errors() == 0
    check_rows(got, q, pool, page, table[0], masks, n, scale, cap=cap, window=window, slopes=slopes)


@pytest.mark.parametrize("d", [1, 3, 64])
def test_128_query_heads_a_kv_head(m, d):
    g = gen(d)
    n, page = 200 + d, 32
    table, pages = table_of([n], page, g)
    pool = random_pool(pages, 1, page, 9)
    q = torch.randn((d, 128, HEAD), generator=g).to(torch.bfloat16)
    masks = plain.masks_of(random_tree(d, g))
    got = m.tree_attention(m.PagedCache(pages, page, 1, pool=pool.cuda()), q.cuda(), sums([d]), d, table.cuda(), ints([n]),
                           tree_mask=torch.tensor([plain.signed(x) for x in masks]).cuda())
    assert m.check_device_errors() == 0
    check_rows(got, q, pool, page, table[0], masks, n)


@pytest.mark.parametrize("hq", [2, 40])
def test_sequences_beside_one_that_does_not_fit(m, hq):
    """What each flagged sequence gives, and the others' outputs."""
    g = gen(6)
    page = 16
    table, pages = table_of([64, 64, 64], page, g)
    pool = random_pool(pages, 1, page, 1)
    cache = m.PagedCache(pages, page, 1, pool=pool.cuda())
    q = torch.randn((7, hq, HEAD), generator=g).to(torch.bfloat16)

    def run(lens, cu, bound):
        out = torch.full((7, hq, HEAD), 7.0, dtype=torch.bfloat16, device="cuda")
        m.tree_attention(cache, q.cuda(), ints(cu), bound, table.cuda(), ints(lens), out=out)
        assert m.check_device_errors() == -4
        return out

    def fine(out, b, rows, n):
        check_rows(out[rows], q[rows], pool, page, table[b], [(2 << i) - 1 for i in range(rows.stop - rows.start)], n)

    kept = lambda x: bool((x == 7.0).all())  # noqa: E731
    a, b, c, rest = slice(0, 2), slice(2, 4), slice(4, 6), slice(6, 7)
    out = run([64, 1, 60], [0, 2, 4, 6], 2)          # more drafts than tokens: zeros
    fine(out, 0, a, 64), fine(out, 2, c, 60)
    assert not out[b].any() and kept(out[rest])
    out = run([64, 70, 60], [0, 2, 4, 6], 2)         # longer than the table: cut to it
    fine(out, 0, a, 64), fine(out, 1, b, 64), fine(out, 2, c, 60)
    assert kept(out[rest])
    out = run([64, -3, 60], [0, 2, 4, 6], 2)         # a negative length: none
    fine(out, 0, a, 64), fine(out, 2, c, 60)
    assert not out[b].any() and kept(out[rest])
    out = run([64, 63, 64], [0, 2, 4, 9], 2)         # rows that there are not
    fine(out, 0, a, 64), fine(out, 1, b, 63)
    assert kept(out[4:])
    out = run([64, 63, 62], [0, 2, -1, 2], 2)        # bounds that fall, and one that begins before the first row
    fine(out, 0, a, 64)
    assert kept(out[2:])
    out = run([64, 63, 62], [0, 2, 5, 7], 2)         # more drafts than the call's bound: the first ones, as the last tokens
    fine(out, 0, a, 64), fine(out, 1, b, 63), fine(out, 2, slice(5, 7), 62)
    assert kept(out[4:5])


# --------------------------------------------------------------------------------- acceptance

@pytest.mark.parametrize("fp8", [False, True])
def test_what_an_acceptance_flags_stays_as_it_was(m, fp8):
    """The pool's bytes after calls with one inconsistent sequence or entry: the intact sequence's rows moved, no others."""
    g = gen(7)
    hkv, page = 3, 16
    dtype = m.DTYPE_FP8_E4M3 if fp8 else m.DTYPE_NVFP4
    pool = torch.randint(0, 256, (4, hkv, m.slab_bytes(dtype, page)), generator=g, dtype=torch.int32).to(torch.uint8)

    def parts(p, t):      # of token t of a sequence whose pages are p: page, bytes [heads][...]
        r, x = t % 16, p[0][p[1][t // page]]
        if fp8:
            return [x[:, r * 128:(r + 1) * 128], x[:, 2048 + r * 128:2048 + (r + 1) * 128]]
        return [x[:, r * 64:(r + 1) * 64], x[:, 1024 + r * 8:1024 + (r + 1) * 8],
                x[:, 1152 + r * 64:1152 + (r + 1) * 64], x[:, 2176 + r::16]]

    tables = [[0, 1], [2, 3]]

    def run(lens, cu, lists, counts, moved, want, bad=None):
        cache = m.PagedCache(4, page, hkv, dtype=dtype, pool=pool.clone().cuda())
        given = [list(x) for x in tables]
        if bad is not None:
            given[bad[0]][bad[1]] = bad[2]
        new = m.accept_tokens(cache, ints(given), ints(lens), ints(cu), ints(lists), ints(counts))
        assert m.check_device_errors() == -4 and new.tolist() == want
        after = pool.clone()
        for b, s, t in moved:
            for x, y in zip(parts((pool, tables[b]), s), parts((after, tables[b]), t)):
                y.copy_(x)
        assert torch.equal(cache.pool.cpu(), after)

    fit = [(1, 17, 16), (1, 19, 17)]                                             # the second sequence's, where intact
    run([20, 20], [0, 4, 8], [[2, 9, 0], [1, 3, 0]], [3, 2], [(0, 18, 16)] + fit, [17, 18])     # an entry that is no draft
    run([20, 20], [0, 4, 8], [[2, 0, 1], [1, 3, 0]], [4, 2], [(0, 18, 16), (0, 16, 17), (0, 17, 18)] + fit, [19, 18])
    run([20, 20], [0, 4, 8], [[2, 0, 1], [1, 3, 0]], [-1, 2], fit, [16, 18])                    # a negative count
    run([3, 20], [0, 4, 8], [[2, 0, 1], [1, 3, 0]], [2, 2], fit, [3, 18])                       # more drafts than tokens
    run([20, 20], [0, -4, 0], [[2, 0, 1], [1, 3, 0]], [2, 2], fit, [20, 18])                    # bounds that fall
    run([20, 20], [0, 65, 69], [[2, 0, 1], [1, 3, 0]], [2, 2], fit, [20, 18])                   # more than 64 drafts
    run([40, 20], [0, 4, 8], [[1, 0, 0], [1, 3, 0]], [1, 2], [(0, 29, 28)] + fit, [29, 18])     # longer than the table: cut
    for page_id in (4, -1, 1 << 30):
        # drafts of the first sequence on both of its pages (12 .. 19): rows from or to the one out of range stay
        run([20, 20], [0, 8, 12], [[1, 6, 3], [1, 3, 0]], [3, 2], [(0, 13, 12), (0, 15, 14)] + fit, [15, 18], bad=(0, 1, page_id))
        run([20, 20], [0, 8, 12], [[5, 6, 2], [1, 3, 0]], [3, 2], fit, [15, 18], bad=(0, 0, page_id))
