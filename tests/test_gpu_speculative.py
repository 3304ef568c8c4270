"""The cache side of speculative decoding on the GPU: rotated append, tree attention, acceptance,
each against its formula in 64 bits (tests/speculative_plain.py has the tolerances' derivation)."""

import math

import pytest
import torch

import speculative_plain as plain
from speculative_plain import GROUP, HEAD

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import nvfp4_quantised_paged_gb300 as mod
    return mod


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def random_pool(pages, heads, page, seed):
    g = gen(seed)
    pool = torch.randint(0, 256, (pages, heads, page // 16, GROUP), generator=g, dtype=torch.int32).to(torch.uint8)
    for at in (1024, 2176):
        pool[..., at:at + 128] = torch.randint(0x20, 0x32, (pages, heads, page // 16, 128), generator=g,
                                               dtype=torch.int32).to(torch.uint8)
    return pool.view(pages, heads, page // 16 * GROUP)


def table_of(lens, page, g, spare=0):
    """Shuffled pages for each sequence, -1 behind its last."""
    counts = [-(-n // page) for n in lens]
    order = torch.randperm(sum(counts) + spare, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(max(counts), 1)), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table, sum(counts) + spare


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def packed(t):
    """On the GPU with the strides that its shape has by itself (a slice of one token keeps others)."""
    return torch.empty(t.shape, dtype=t.dtype).copy_(t).cuda()


def sums(x):
    return ints([sum(x[:i]) for i in range(len(x) + 1)])


# --------------------------------------------------------------------------------- rotated append

def rotation(rows, rot, base=1e4):
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * base ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


WRITE = [  # tokens, q heads, kv heads, page, rot, adjacent, sections, norms, scale, fp8
    (1, 4, 1, 16, 128, False, None, False, 1.0, False),
    (37, 8, 2, 16, 128, False, None, True, 1.0, False),
    (300, 5, 5, 32, 128, True, None, True, 0.75, False),
    (129, 10, 2, 64, 64, False, None, False, 1.0, False),
    (65, 6, 3, 128, 64, True, None, True, 0.375, False),
    (70, 3, 1, 16, 96, False, None, True, 1.0, False),
    (33, 2, 1, 16, 32, False, None, False, 1.0, True),
    (90, 8, 1, 32, 128, False, (16, 24, 24), True, 1.0, False),
    (50, 4, 4, 16, 128, True, (4, 40, 20), False, 0.6, False),
    (41, 4, 2, 16, 64, False, (0, 32), True, 1.0, True),
    (20, 7, 1, 16, 0, False, None, True, 1.0, False),
    (999, 32, 8, 64, 128, False, None, True, 1.0, False),
    (1000, 32, 8, 64, 128, False, None, True, 1.0, False),
    (1500, 33, 7, 64, 128, True, None, True, 1.0, True),
    (1300, 40, 8, 64, 96, False, None, False, 1.0, False),
    (4097, 16, 4, 64, 128, False, None, True, 0.75, False),
]


def write_inputs(T, hq, hkv, rot, sections, norms, seed, rows=5000):
    g = gen(seed)
    x = torch.randn((T, (hq + 2 * hkv) * HEAD), generator=g)
    x = torch.where(torch.rand(x.shape, generator=g) < 0.01, x * 20, x).to(torch.bfloat16)
    axes = len(sections) if sections else 1
    pos = torch.randint(0, rows, (axes, T), generator=g, dtype=torch.int32)
    w = [(torch.randn(HEAD, generator=g) * 0.3 + 1).to(torch.bfloat16) if norms else None for _ in range(2)]
    return x, pos if sections else pos[0], rotation(rows, rot) if rot else None, w


@pytest.mark.parametrize("T,hq,hkv,page,rot,adjacent,sections,norms,scale,fp8", WRITE)
def test_rope_append(m, T, hq, hkv, page, rot, adjacent, sections, norms, scale, fp8):
    x, pos, table, (wq, wk) = write_inputs(T, hq, hkv, rot, sections, norms, T)
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=gen(5))[:T]
    slots[::7] = -1 if T > 1 else slots[0]
    dtype = m.DTYPE_FP8_E4M3 if fp8 else m.DTYPE_NVFP4
    ours, other = (m.PagedCache(pages, page, hkv, dtype=dtype, k_global_scale=scale, v_global_scale=scale) for _ in range(2))
    dev = x.cuda().unflatten(-1, (-1, HEAD))
    q, k, v = dev.split([hq, hkv, hkv], 1)
    on = lambda t: None if t is None else t.cuda()  # noqa: E731
    out = m.rope_quantize_append(ours, q, k, v, on(pos), on(table), slots.cuda(), q_norm=on(wq), k_norm=on(wk), eps=1e-5,
                                 adjacent=adjacent, sections=sections)
    hq_, hk_, hv_ = x.unflatten(-1, (-1, HEAD)).split([hq, hkv, hkv], 1)
    rq, size = plain.turned(hq_, wq, pos, table, 1e-5, adjacent, sections)
    rk, _ = plain.turned(hk_, wk, pos, table, 1e-5, adjacent, sections)
    m.quantize_append(other, packed(plain.bf16_rounded(rk)), packed(hv_), slots.cuda())
    assert m.check_device_errors() == 0
    assert torch.equal(ours.pool, other.pool)
    err = (out.cpu().double() - rq).abs()
    assert (err <= 2.0**-8 * rq.abs() + 2.0**-16 * size + 1e-30).all(), float((err / (size + 1e-30)).max())


def test_rope_append_without_queries_in_place_and_out(m):
    T, hq, hkv = 77, 4, 2
    x, pos, table, (wq, wk) = write_inputs(T, hq, hkv, 128, None, True, 9)
    slots = torch.arange(T, device="cuda")
    caches = [m.PagedCache(6, 16, hkv) for _ in range(3)]
    dev = x.cuda().unflatten(-1, (-1, HEAD))
    q, k, v = dev.split([hq, hkv, hkv], 1)
    args = (pos.cuda(), table.cuda(), slots)
    first = m.rope_quantize_append(caches[0], q, k, v, *args, q_norm=wq.cuda(), k_norm=wk.cuda())
    assert m.rope_quantize_append(caches[1], None, k, v, *args, k_norm=wk.cuda()) is None
    again = m.rope_quantize_append(caches[2], q, k, v, *args, q_norm=wq.cuda(), k_norm=wk.cuda(), q_out=q)
    assert again.data_ptr() == q.data_ptr() and torch.equal(q, first)
    assert torch.equal(caches[0].pool, caches[1].pool) and torch.equal(caches[0].pool, caches[2].pool)
    assert torch.equal(dev[:, hq:].cpu(), x.unflatten(-1, (-1, HEAD))[:, hq:])     # k and v stay
    assert m.check_device_errors() == 0


def test_rope_append_skips_what_is_out_of_range(m):
    T, hq, hkv = 9, 2, 1
    x, pos, table, _ = write_inputs(T, hq, hkv, 64, None, False, 3, rows=50)
    pos[4], pos[5] = 50, -1
    slots = torch.arange(T)
    slots[7] = 32
    cache = m.PagedCache(2, 16, hkv)
    dev = x.cuda().unflatten(-1, (-1, HEAD))
    q, k, v = dev.split([hq, hkv, hkv], 1)
    out = torch.full((T, hq, HEAD), 3.0, dtype=torch.bfloat16, device="cuda")
    m.rope_quantize_append(cache, q, k, v, pos.cuda(), table.cuda(), slots.cuda(), q_out=out)
    assert m.check_device_errors() == -4 and m.check_device_errors() == 0
    written = [bool(cache.pool[0, 0, r * 64:(r + 1) * 64].any()) for r in range(T)]
    assert written == [i not in (4, 5, 7) for i in range(T)]
    same = [bool((out[i] == 3.0).all()) for i in range(T)]
    assert same == [i in (4, 5) for i in range(T)]


@pytest.mark.parametrize("sections", [None, (8, 12, 12)])
def test_rope_append_long_skips_what_is_out_of_range(m, sections):
    """The same through the form for many tokens: negative and too large slots, positions on each axis."""
    T, hq, hkv, page = 6000, 20, 4, 64
    x, pos, table, (wq, wk) = write_inputs(T, hq, hkv, 64, sections, True, 13, rows=300)
    slots = torch.randperm(100 * page, generator=gen(1))[:T]
    bad_pos, bad_slot = list(range(3, T, 501)), list(range(5, T, 700))
    first = pos[len(sections) - 1] if sections else pos
    first[bad_pos] = torch.tensor([300, -1] * len(bad_pos))[:len(bad_pos)].int()
    slots[bad_slot] = torch.tensor([-1, 100 * page] * len(bad_slot))[:len(bad_slot)]
    a, b = m.PagedCache(100, page, hkv), m.PagedCache(100, page, hkv)
    q, k, v = x.cuda().unflatten(-1, (-1, HEAD)).split([hq, hkv, hkv], 1)
    out = torch.full((T, hq, HEAD), 3.0, dtype=torch.bfloat16, device="cuda")
    m.rope_quantize_append(a, q, k, v, pos.cuda(), table.cuda(), slots.cuda(), q_norm=wq.cuda(), k_norm=wk.cuda(),
                           sections=sections, q_out=out)
    assert m.check_device_errors() == -4 and m.check_device_errors() == 0
    fine = torch.ones(T, dtype=torch.bool)
    fine[bad_pos] = False
    assert (out[~fine.cuda()] == 3.0).all()
    some = pos[:, fine] if sections else pos[fine]
    rows = x.unflatten(-1, (-1, HEAD))[fine]
    rq, size = plain.turned(rows[:, :hq], wq, some, table, 1e-6, False, sections)
    rk, _ = plain.turned(rows[:, hq:hq + hkv], wk, some, table, 1e-6, False, sections)
    err = (out.cpu().double()[fine] - rq).abs()
    assert (err <= 2.0**-8 * rq.abs() + 2.0**-16 * size + 1e-30).all()
    kept = torch.where(slots < 100 * page, slots, torch.full_like(slots, -1))[fine]
    m.quantize_append(b, plain.bf16_rounded(rk).cuda(), packed(rows[:, hq + hkv:]), kept.cuda())
    assert torch.equal(a.pool, b.pool) and m.check_device_errors() == 0


@pytest.mark.parametrize("T", [8, 6000])
@pytest.mark.parametrize("norms", [False, True])
def test_rope_append_infinities_and_nan(m, T, norms):
    """Rows with an infinity or a NaN give what FP32 gives (the rotation by angles whose cosine and sine are 0 or 1, so
    that every other product is exact); their neighbours are not touched."""
    hq, hkv = 4, 4
    g = gen(2)
    x = torch.randint(-8, 9, (T, hq + 2 * hkv, HEAD), generator=g).float()
    x[::5, 1, 3], x[1::7, 2, 70], x[2::9, hq, 100], x[3::8, hq + 1, 5] = math.inf, math.nan, -math.inf, math.nan
    table = torch.tensor([[1.0] * 64 + [0.0] * 64, [0.0] * 64 + [1.0] * 64])
    pos = torch.randint(0, 2, (T,), generator=g, dtype=torch.int32)
    w = torch.ones(HEAD, dtype=torch.bfloat16)
    slots = torch.arange(T)
    pages = -(-T // 64)
    a, b = m.PagedCache(pages, 64, hkv), m.PagedCache(pages, 64, hkv)
    q, k, v = x.to(torch.bfloat16).cuda().split([hq, hkv, hkv], 1)
    on = w.cuda() if norms else None
    out = m.rope_quantize_append(a, q, k, v, pos.cuda(), table.cuda(), slots.cuda(), q_norm=on, k_norm=on, eps=0.0).cpu()
    y = x.double()
    if norms:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True))
    c, s = (table[pos.long(), i:i + 64].double()[:, None] for i in (0, 64))
    y = torch.cat([y[..., :64] * c - y[..., 64:] * s, y[..., 64:] * c + y[..., :64] * s], -1)
    for h in range(hq):
        fine = torch.isfinite(y[:, h])
        assert torch.equal(torch.isnan(out[:, h]), torch.isnan(y[:, h]))
        assert torch.equal(out[:, h].double()[~fine & ~torch.isnan(y[:, h])], y[:, h][~fine & ~torch.isnan(y[:, h])])
        assert ((out[:, h].double() - y[:, h])[fine].abs() <= 2.0**-8 * y[:, h][fine].abs()).all()
    rk = y[:, hq:hq + hkv]
    rounded = torch.where(torch.isfinite(rk), plain.bf16_rounded(torch.where(torch.isfinite(rk), rk, 1.0)).double(), rk)
    m.quantize_append(b, packed(rounded.to(torch.bfloat16)), packed(x[:, hq + hkv:].to(torch.bfloat16)), slots.cuda())
    # (as values: where an infinity makes a row's norm infinite, the order of rotation and norm decides a zero's sign)
    for ours, other in zip(*(plain.rows_of(c.pool.cpu(), 64, torch.arange(pages), T) for c in (a, b))):
        assert torch.equal(torch.isnan(ours), torch.isnan(other))
        assert torch.equal(torch.nan_to_num(ours), torch.nan_to_num(other))
    assert m.check_device_errors() == 0


def test_rope_append_zero_rows_and_no_tokens(m):
    cache, ref = m.PagedCache(1, 16, 1), m.PagedCache(1, 16, 1)
    z = torch.zeros((3, 1, HEAD), dtype=torch.bfloat16, device="cuda")
    w, table = torch.ones(HEAD, dtype=torch.bfloat16, device="cuda"), rotation(8, 128).cuda()
    out = m.rope_quantize_append(cache, z, z, z, ints([0, 1, 2]), table, torch.arange(3, device="cuda"), q_norm=w, k_norm=w)
    assert not out.any()
    k, _ = m.prefix_dequant(cache, ints([[0]]), ints([3]), ints([0, 3]), 3)
    assert not k.any()
    none = z[:0]
    assert m.rope_quantize_append(ref, none, none, none, ints([]), table, torch.arange(0, device="cuda")).shape == (0, 1, HEAD)
    assert m.check_device_errors() == 0


def test_rope_append_keys_next_to_rounding_borders(m):
    """Every BF16 mantissa in the pair's first value, its partner far smaller, and tables of one position: products that
    end next to a BF16 border would be quantised to another code if the product were rounded to FP32 first."""
    T = 4096
    g = gen(1)
    x = torch.randn((T, 1, HEAD), generator=g).to(torch.bfloat16)
    x[..., 64:] *= torch.exp2(torch.randint(-24, 1, (T, 1, 64), generator=g).float()).to(torch.bfloat16)
    c = torch.rand(1, 128, generator=g)
    table = torch.cat([c, torch.nextafter(c, torch.ones(1)), c.to(torch.bfloat16).float(), 1 + 0 * c])
    pos = torch.randint(0, 4, (T,), generator=g, dtype=torch.int32)
    a, b = m.PagedCache(T // 128, 128, 1), m.PagedCache(T // 128, 128, 1)
    slots = torch.arange(T, device="cuda")
    v = x.cuda()
    m.rope_quantize_append(a, None, v, v, pos.cuda(), table.cuda(), slots)
    rk, _ = plain.turned(x, None, pos, table, 0, False, None)
    m.quantize_append(b, plain.bf16_rounded(rk).cuda(), v, slots)
    assert torch.equal(a.pool, b.pool) and m.check_device_errors() == 0


# --------------------------------------------------------------------------------- tree attention

def random_tree(d, g):
    return ([-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, d)])[:d]


def run_tree(m, lens, drafts, hq, hkv, page, seed=0, parents=None, cap=0.0, window=0, slopes=None, scales=(1.0, 1.0), masks=None,
             chain=False, num_splits=0, qscale=1.0, bad_page=None, behind=None):
    g = gen(seed + 11)
    table, pages = table_of(lens, page, g, 1)
    pool = random_pool(pages, hkv, page, seed)
    total = sum(drafts)
    q = (torch.randn((total, hq, HEAD), generator=g) * qscale).to(torch.bfloat16)
    if masks is None:
        masks = [plain.masks_of(random_tree(d, g)) if not chain else [(2 << i) - 1 for i in range(d)] for d in drafts]
    given = [x for s in masks for x in s]
    if behind is not None:       # bits of drafts that there are not
        given = [x | y for x, y in zip(given, behind)]
    flat = torch.tensor([plain.signed(x) for x in given], dtype=torch.int64)
    gone = {}
    if bad_page is not None:
        b, p = bad_page
        table[b, p] = pages + 7
        gone[b] = [t for t in range(p * page, min((p + 1) * page, lens[b]))]
    cache = m.PagedCache(pages, page, hkv, k_global_scale=scales[0], v_global_scale=scales[1], pool=pool.cuda())
    scale = 0.11
    whole = torch.full((total + 3, hq, HEAD), 5.0, dtype=torch.bfloat16, device="cuda")
    out = whole[:total]
    m.tree_attention(cache, q.cuda(), sums(drafts), max(drafts), table.cuda(), ints(lens),
                     tree_mask=None if chain else flat.cuda(), sm_scale=scale, softcap=cap, window=window,
                     slopes=None if slopes is None else slopes.cuda(), out=out, num_splits=num_splits)
    status = m.check_device_errors()
    assert status == (-4 if bad_page is not None else 0)
    assert (whole[total:] == 5.0).all()
    got, at = out.cpu().double(), 0
    assert torch.isfinite(got).all()
    for b, (n, d) in enumerate(zip(lens, drafts)):
        if d == 0:
            continue
        if n == 0:
            assert not got[at:at + d].any()
            at += d
            continue
        safe = table[b].clone()
        safe[safe >= pages] = 0
        k, v = plain.rows_of(pool, page, safe, n)
        ref, spread, size = plain.tree(q[at:at + d], k * scales[0], v * scales[1], masks[b], n, scale, cap, window, slopes,
                                       gone.get(b, ()))
        err = (got[at:at + d] - ref).abs()
        bound = plain.tree_bound(ref, spread, size, n, float(v.abs().max()) * scales[1])
        worst = float((err / bound).max())
        assert worst <= 1, (b, n, d, worst)
        at += d
    return out


TREES = [  # lengths, drafts, q heads, kv heads, page
    ([77], [4], 4, 1, 16),
    ([1], [1], 1, 1, 16),
    ([5], [5], 8, 2, 16),
    ([130, 64, 128, 129], [3, 1, 16, 2], 8, 1, 64),
    ([700, 33, 512], [8, 8, 5], 8, 2, 32),
    ([300, 1000], [16, 13], 8, 2, 128),
    ([400, 70], [64, 33], 4, 4, 16),
    ([900], [64], 16, 2, 64),
    ([2000, 1500, 3], [7, 1, 3], 40, 8, 64),
    ([260], [17], 24, 1, 16),
    ([90, 0, 140], [2, 2, 2], 2, 1, 16),
    ([90, 50, 140], [2, 0, 1], 4, 2, 16),
]


@pytest.mark.parametrize("lens,drafts,hq,hkv,page", TREES)
def test_tree_attention(m, lens, drafts, hq, hkv, page):
    run_tree(m, lens, drafts, hq, hkv, page, seed=sum(lens))


@pytest.mark.parametrize("splits", [1, 2, 5, 37, 400])
def test_tree_attention_splits(m, splits):
    run_tree(m, [1300, 200, 640], [9, 4, 12], 8, 2, 64, seed=2, num_splits=splits)


@pytest.mark.parametrize("cap,window,sloped", [(5.0, 0, False), (0.0, 1, False), (0.0, 3, False), (0.0, 130, False),
                                               (0.0, 100000, False), (0.0, 0, True), (3.0, 200, True)])
@pytest.mark.parametrize("lens,drafts,hq,hkv,page", [([300, 900, 20], [5, 12, 20], 8, 2, 16), ([700], [1], 16, 1, 64),
                                                     ([600, 410], [40, 64], 8, 2, 32)])
def test_tree_attention_options(m, cap, window, sloped, lens, drafts, hq, hkv, page):
    slopes = torch.exp2(-torch.arange(1, hq + 1) * 8.0 / hq) if sloped else None
    run_tree(m, lens, drafts, hq, hkv, page, seed=len(lens), cap=cap, window=window, slopes=slopes, qscale=2.0)


def test_tree_attention_chain_and_tensor_scales(m):
    run_tree(m, [333, 200], [6, 31], 8, 2, 16, chain=True, scales=(0.7, 2.3))


def test_tree_attention_masks_that_see_nothing(m):
    # no prefix and empty masks: zeros; a draft that sees only itself; one that sees all others but not itself
    run_tree(m, [4, 64, 150], [4, 64, 3], 4, 2, 16, masks=[[0, 2, 0, 13], [0] * 63 + [(1 << 64) - 1], [0, 7, 2]])


def test_tree_attention_ignores_mask_bits_behind_the_drafts(m):
    a = run_tree(m, [100], [3], 4, 1, 16, masks=[[1, 3, 7]])
    b = run_tree(m, [100], [3], 4, 1, 16, masks=[[1, 3, 7]], behind=[1 << 40, 1 << 63, 1 << 3])
    assert torch.equal(a, b)


def test_tree_attention_pages_out_of_range_are_not_seen(m):
    run_tree(m, [300], [4], 8, 2, 16, bad_page=(0, 7))
    run_tree(m, [300], [4], 8, 2, 128, bad_page=(0, 0))


def test_tree_attention_equals_decode(m):
    """One draft a sequence, no options: the decode call's result up to both sides' rounding."""
    import gpu_common
    g = gen(4)
    lens, hq, hkv, page = [500, 64, 1, 1111], 16, 2, 64
    table, pages = table_of(lens, page, g)
    cache = m.PagedCache(pages, page, hkv, pool=random_pool(pages, hkv, page, 3).cuda())
    q = torch.randn((4, hq, HEAD), generator=g).to(torch.bfloat16).cuda()
    a = m.paged_decode_attention(cache, q, table.cuda(), ints(lens))
    b = m.tree_attention(cache, q, sums([1] * 4), 1, table.cuda(), ints(lens))
    ref, spread = [], []
    for i, n in enumerate(lens):
        k, v = plain.rows_of(cache.pool.cpu(), page, table[i], n)
        r, s, _ = plain.tree(q[i:i + 1].cpu(), k, v, [1], n, 1 / math.sqrt(HEAD))
        ref.append(r[0]), spread.append(s[0])
    for x in (a, b):
        gpu_common.check_attention(x, torch.stack(ref).numpy(), spread=torch.stack(spread).numpy())
    assert m.check_device_errors() == 0


def test_tree_attention_device_checks(m):
    """Lengths and draft counts that do not fit are flagged and cut, never followed."""
    g = gen(6)
    table, pages = table_of([64, 64, 64], 16, g)
    cache = m.PagedCache(pages, 16, 1, pool=random_pool(pages, 1, 16, 1).cuda())
    q = torch.randn((6, 2, HEAD), generator=g).to(torch.bfloat16).cuda()
    for lens, cu, bound in (([64, 1, 64], [0, 2, 4, 6], 2), ([64, 70, 64], [0, 2, 4, 6], 2), ([64, -3, 64], [0, 2, 4, 6], 2),
                            ([64, 64, 64], [0, 2, 4, 9], 2), ([64, 64, 64], [0, 4, 2, 6], 4), ([64, 64, 64], [0, 2, 4, 6], 1)):
        out = torch.full_like(q, 7.0)
        m.tree_attention(cache, q, ints(cu), bound, table.cuda(), ints(lens), out=out)
        assert m.check_device_errors() == -4, (lens, cu)
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("hq,drafts", [(4, 3), (16, 12)])
def test_tree_attention_many_sequences(m, hq, drafts):
    g = gen(8)
    lens = [int(x) for x in torch.randint(1, 60, (300,), generator=g)]
    run_tree(m, lens, [min(n, 1 + i % drafts) for i, n in enumerate(lens)], hq, 1, 16, seed=5)


def test_tree_attention_on_two_streams_at_once(m):
    """Two calls that may overlap, each with its workspace."""
    g = gen(71)
    table, pages = table_of([3000, 2500], 64, g)
    cache = m.PagedCache(pages, 64, 2, pool=random_pool(pages, 2, 64, 2).cuda())
    t, n, cu = table.cuda(), ints([3000, 2500]), sums([9, 3])
    q = [torch.randn((12, 16, HEAD), generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    want = [m.tree_attention(cache, x, cu, 9, t, n) for x in q]
    ws = [m.alloc_tree_workspace(cache, 2, 16, 9) for _ in range(2)]
    outs = [[torch.empty_like(q[0]) for _ in range(20)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for j in range(2):
            m.tree_attention(cache, q[j], cu, 9, t, n, workspace=ws[j], out=outs[j][i], stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(o, want[j]) for o in outs[j])
    assert m.check_device_errors() == 0


@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("hq", [4, 24, 64])
def test_tree_attention_nan_reaches_the_drafts_that_see_it(m, window, hq):
    """NaN scales in the rows of a draft, of a token at the window's edge, and behind the sequence."""
    g = gen(51)
    hkv, page, n, d = 2, 16, 333, 6
    base = n - d
    table, pages = table_of([n + 3], page, g)
    masks = plain.masks_of([-1, 0, 0, 1, 2, 4])
    q = torch.randn((d, hq, HEAD), generator=g).to(torch.bfloat16)

    def poisoned(tokens):
        pool = random_pool(pages, hkv, page, 4)
        grp = pool.view(pages, hkv, page // 16, GROUP)
        for t, head, block, is_k in tokens:
            row = grp[table[0, t // page].long(), head, (t % page) // 16]
            row[1024 + (t % 16) * 8 + block if is_k else 2176 + block * 16 + t % 16] = 0x7f
        return pool

    for tokens in ([(base + 2, 0, 3, False)], [(base + 4, 1, 0, False), (base + 1, 1, 7, False)], [(base + 3, 0, 5, True)],
                   [(base - 18, 0, 1, False)], [(base - 19, 1, 6, False), (base - 20, 0, 6, False)], [(7, 0, 2, False)],
                   [(n, 0, 2, False), (n + 2, 1, 2, True)]):
        pool = poisoned(tokens)
        cache = m.PagedCache(pages, page, hkv, pool=pool.cuda())
        got = m.tree_attention(cache, q.cuda(), sums([d]), d, table.cuda(), ints([n]), window=window,
                               tree_mask=torch.tensor(masks, device="cuda")).cpu()
        k, v = plain.rows_of(pool, page, table[0], n)
        ref = plain.tree(q, k, v, masks, n, 1 / math.sqrt(HEAD), window=window)[0]
        assert torch.equal(torch.isnan(got), torch.isnan(ref)), tokens
        fine = ~torch.isnan(ref)
        assert (got.double()[fine] - ref[fine]).abs().max() < 0.05 * ref[fine].abs().max(), tokens
    assert m.check_device_errors() == 0


def test_pages_beyond_four_gigabytes(m):
    g = gen(61)
    hkv, page, pages = 8, 128, 40000                 # 5.9 GB
    cache = m.PagedCache(pages, page, hkv)
    lens, drafts, hq = [300, 129], [5, 1], 16
    table = torch.tensor([[39999, 31000, 29500], [39998, 30999, -1]], dtype=torch.int32)
    small = random_pool(6, hkv, page, 2)
    for i, p in enumerate([39999, 31000, 29500, 39998, 30999]):
        cache.pool[p] = small[i].cuda()
    near = torch.tensor([[0, 1, 2], [3, 4, -1]], dtype=torch.int32)
    other = m.PagedCache(6, page, hkv, pool=small.cuda())
    q = torch.randn((6, hq, HEAD), generator=g).to(torch.bfloat16).cuda()
    x = torch.randn((6, 2 * hkv, HEAD), generator=g).to(torch.bfloat16).cuda()
    at = [(0, t) for t in range(295, 300)] + [(1, 128)]
    outs = []
    for c, t in ((cache, table), (other, near)):
        slots = torch.tensor([int(t[b, p // page]) * page + p % page for b, p in at]).cuda()
        m.rope_quantize_append(c, None, x[:, :hkv], x[:, hkv:], ints([p for _, p in at]), rotation(400, 128).cuda(), slots)
        outs.append(m.tree_attention(c, q, sums(drafts), 5, t.cuda(), ints(lens)))
        new = m.accept_tokens(c, t.cuda(), ints(lens), sums(drafts), ints([[0, 3], [0, 0]]), ints([2, 1]))
        assert new.tolist() == [297, 129]
        outs.append(m.paged_decode_attention(c, q[:2], t.cuda(), new))
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    assert m.check_device_errors() == 0


# --------------------------------------------------------------------------------- acceptance

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [16, 64])
def test_accept_moves_rows(m, page, fp8):
    g = gen(page)
    drafts, prefix = [8, 64, 1, 5, 33], [0, 250, 15, 16, 31]
    lens = [p + d for p, d in zip(prefix, drafts)]
    table, pages = table_of(lens, page, g, 1)
    hkv = 3
    dtype = m.DTYPE_FP8_E4M3 if fp8 else m.DTYPE_NVFP4
    slab = m.slab_bytes(dtype, page)
    pool = torch.randint(0, 256, (pages, hkv, slab), generator=g, dtype=torch.int32).to(torch.uint8)
    lists = [[0, 2, 3, 7], sorted(torch.randperm(64, generator=g)[:40].tolist()), [], [4, 0, 0, 3, 1], list(range(33))]
    acc = torch.full((5, 64), -1, dtype=torch.int32)
    for b, x in enumerate(lists):
        acc[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
    cache = m.PagedCache(pages, page, hkv, dtype=dtype, pool=pool.clone().cuda())
    new = m.accept_tokens(cache, table.cuda(), ints(lens), sums(drafts), acc.cuda(), ints([len(x) for x in lists]))
    assert m.check_device_errors() == 0
    assert new.tolist() == [p + len(x) for p, x in zip(prefix, lists)]

    def parts(p, t):      # the bytes of token t's rows [heads][...] in a pool
        grp = p.view(pages, hkv, page // 16, -1)[:, :, (t % page) // 16]
        r = t % 16
        if fp8:
            return [grp[..., r * 128:(r + 1) * 128], grp[..., 2048 + r * 128:2048 + (r + 1) * 128]]
        return [grp[..., r * 64:(r + 1) * 64], grp[..., 1024 + r * 8:1024 + (r + 1) * 8],
                grp[..., 1152 + r * 64:1152 + (r + 1) * 64], grp[..., 2176 + r:GROUP:16]]

    want = pool.clone()
    for b, x in enumerate(lists):
        for k, j in enumerate(x):
            s, t = prefix[b] + j, prefix[b] + k
            for a, c in zip(parts(pool, s), parts(want, t)):
                c[table[b, t // page].long()] = a[table[b, s // page].long()]
    assert torch.equal(cache.pool.cpu(), want)


def test_accept_flags_what_does_not_fit(m):
    cache = m.PagedCache(4, 16, 1)
    table, acc = ints([[0, 1], [2, 3]]), ints([[0, 1, 9], [0, 0, 0]])
    for lens, cu, counts, want in (([20, 20], [0, 4, 8], [3, 1], [18, 17]), ([20, 20], [0, 4, 8], [2, 5], [18, 19]),
                                   ([20, 3], [0, 4, 8], [0, 1], [16, 3]), ([40, 20], [0, 4, 8], [1, 0], [29, 16]),
                                   ([20, 20], [0, 4, 3], [1, 0], [17, 20]), ([20, 20], [0, 4, 8], [-1, 1], [16, 17])):
        new = m.accept_tokens(cache, table, ints(lens), ints(cu), acc, ints(counts))
        assert m.check_device_errors() == -4, (lens, cu, counts)
        assert new.tolist() == want, (lens, cu, counts)
    # a page out of range is flagged, and its rows are not moved
    new = m.accept_tokens(cache, ints([[0, 77], [2, 3]]), ints([20, 20]), sums([4, 4]), ints([[1, 2], [0, 1]]), ints([2, 2]))
    assert m.check_device_errors() == -4 and new.tolist() == [18, 18]


# --------------------------------------------------------------------------------- used together

def test_a_speculative_step_is_decoding_token_by_token(m):
    """Drafts appended with their rotation, verified, the accepted path kept: the cache's bytes are those of
    appending the accepted tokens one by one, and the outputs those of decoding them."""
    import gpu_common
    g = gen(21)
    hq, hkv, page, B = 8, 2, 16, 3
    prefix, parents = [37, 5, 64], [[-1, 0, 0, 1, 1, 2, 5], [-1, 0, 1], [-1, 0, 0, 0, 3]]
    paths = [[0, 2, 5, 6], [0, 1], [0, 3, 4]]
    drafts = [len(p) for p in parents]
    masks = [plain.masks_of(p) for p in parents]
    lens = [p + d for p, d in zip(prefix, drafts)]
    table, pages = table_of([n + 8 for n in lens], page, g)
    turn = rotation(200, 128).cuda()
    wq, wk = ((torch.randn(HEAD, generator=g) * 0.2 + 1).to(torch.bfloat16).cuda() for _ in range(2))
    spec, step = m.PagedCache(pages, page, hkv), m.PagedCache(pages, page, hkv)

    def slots_of(b, positions):
        t = torch.tensor(positions)
        return table[b, t // page].long() * page + t % page

    rows = lambda n: torch.randn((n, hq + 2 * hkv, HEAD), generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    for b in range(B):
        x = rows(prefix[b])
        for c in (spec, step):
            m.rope_quantize_append(c, None, x[:, hq:hq + hkv], x[:, hq + hkv:], ints(list(range(prefix[b]))), turn,
                                   slots_of(b, list(range(prefix[b]))).cuda(), k_norm=wk)
    new = [rows(d) for d in drafts]
    depth = [[bin(x).count("1") - 1 for x in mk] for mk in masks]
    x = torch.cat(new)
    q = m.rope_quantize_append(spec, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:],
                               ints([p + e for p, ds in zip(prefix, depth) for e in ds]), turn,
                               torch.cat([slots_of(b, list(range(prefix[b], lens[b]))) for b in range(B)]).cuda(),
                               q_norm=wq, k_norm=wk)
    out = m.tree_attention(spec, q, sums(drafts), max(drafts), table.cuda(), ints(lens),
                           tree_mask=torch.tensor([y for mk in masks for y in mk], device="cuda"))
    acc = torch.zeros((B, 4), dtype=torch.int32)
    for b, p in enumerate(paths):
        acc[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    kept = m.accept_tokens(spec, table.cuda(), ints(lens), sums(drafts), acc.cuda(), ints([len(p) for p in paths]))
    assert kept.tolist() == [p + len(x) for p, x in zip(prefix, paths)]
    first = [sum(drafts[:b]) for b in range(B)]
    for b, path in enumerate(paths):
        for e, i in enumerate(path):
            x = new[b][i:i + 1]
            at = prefix[b] + e
            qi = m.rope_quantize_append(step, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], ints([at]), turn,
                                        slots_of(b, [at]).cuda(), q_norm=wq, k_norm=wk)
            assert torch.equal(qi[0], q[first[b] + i])
            one = m.paged_decode_attention(step, qi, table[b:b + 1].cuda(), ints([at + 1]))
            k, v = plain.rows_of(step.pool.cpu(), page, table[b], at + 1)
            ref, spread, size = plain.tree(qi.cpu(), k, v, [1], at + 1, 1 / math.sqrt(HEAD))
            bound = plain.tree_bound(ref, spread, size, at + 1, float(v.abs().max()))
            assert ((out[first[b] + i].cpu().double() - ref[0]).abs() <= bound[0]).all()
            gpu_common.check_attention(one, ref.numpy(), spread=spread.numpy())
    for b in range(B):
        for which in range(2):
            a, c = (plain.rows_of(x.pool.cpu(), page, table[b], kept[b].item())[which] for x in (spec, step))
            assert torch.equal(a, c)
    assert m.check_device_errors() == 0


def test_captured_step_and_shared_workspace(m):
    """Two captured graphs of a step that share a workspace, replayed in turn with new inputs."""
    g = gen(31)
    lens, drafts, hq, hkv, page = [400, 90], [4, 4], 8, 2, 16
    table, pages = table_of(lens, page, g)
    cache = m.PagedCache(pages, page, hkv, pool=random_pool(pages, hkv, page, 2).cuda())
    q = torch.randn((8, hq, HEAD), generator=g).to(torch.bfloat16).cuda()
    q2 = torch.randn((8, hq, HEAD), generator=g).to(torch.bfloat16).cuda()
    t, n, cu = table.cuda(), ints(lens), sums(drafts)
    ws = m.alloc_tree_workspace(cache, 2, hq, 4)
    want = [m.tree_attention(cache, x, cu, 4, t, n, workspace=ws).clone() for x in (q, q2)]
    outs, graphs = [torch.empty_like(q), torch.empty_like(q)], []
    side = torch.cuda.Stream()
    for x, o in zip((q, q2), outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(gr, stream=side):
            m.tree_attention(cache, x, cu, 4, t, n, workspace=ws, out=o)
        graphs.append(gr)
    torch.cuda.synchronize()
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    q.copy_(q2)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[1]) and m.check_device_errors() == 0


def test_calls_on_another_stream(m):
    g = gen(41)
    table, pages = table_of([200], 16, g)
    cache = m.PagedCache(pages, 16, 2, pool=random_pool(pages, 2, 16, 2).cuda())
    q = torch.randn((4, 4, HEAD), generator=g).to(torch.bfloat16).cuda()
    t, n, cu = table.cuda(), ints([200]), sums([4])
    want = m.tree_attention(cache, q, cu, 4, t, n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = m.tree_attention(cache, q, cu, 4, t, n, stream=side)
        junk = torch.full((1 << 20,), 3.0, device="cuda")
        side.synchronize()
        assert torch.equal(got, want)
        del junk


def test_wrong_tensors_are_refused(m):
    """The binding's own checks: types, shapes, devices."""
    cache = m.PagedCache(2, 16, 2)
    k = torch.zeros((3, 2, HEAD), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((3, 4, HEAD), dtype=torch.bfloat16, device="cuda")
    slots, pos, turn = torch.arange(3, device="cuda"), ints([0, 1, 2]), rotation(8, 128).cuda()
    ok = dict(q=q, k=k, v=k, positions=pos, cos_sin=turn, slot_mapping=slots)
    m.rope_quantize_append(cache, **ok)
    for bad in (dict(k=k.float()), dict(k=k[:2]), dict(v=k[..., :64]), dict(q=q[:, :, ::2]), dict(q=q.cpu()), dict(positions=pos.long()),
                dict(positions=pos[:2]), dict(positions=None), dict(cos_sin=turn.double()), dict(cos_sin=turn[0]),
                dict(slot_mapping=slots.int()), dict(sections=(16, 24)), dict(sections=(16, 24, 24)), dict(cos_sin=None, sections=(64,)),
                dict(q_norm=turn[0]), dict(k_norm=k[0, 0, :64]), dict(q=None, q_out=q), dict(q_out=q[:2]),
                dict(k=torch.zeros((3, 4, HEAD), dtype=torch.bfloat16, device="cuda")[:, ::2])):
        with pytest.raises(ValueError):
            m.rope_quantize_append(cache, **{**ok, **bad})
    t, n, cu = ints([[0, 1]]), ints([20]), ints([0, 3])
    ok = dict(q=q, cu_q_lens=cu, max_q_len=3, block_table=t, seq_lens=n)
    m.tree_attention(cache, **ok)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(cu_q_lens=cu[:1]), dict(cu_q_lens=cu.long()), dict(block_table=t[0]),
                dict(seq_lens=n.long()), dict(tree_mask=ints([1, 3, 7])), dict(tree_mask=slots[:2]), dict(slopes=turn[0]),
                dict(out=k), dict(workspace=turn)):
        with pytest.raises(ValueError):
            m.tree_attention(cache, **{**ok, **bad})
    for bad in (dict(max_q_len=0), dict(max_q_len=65), dict(window=-1), dict(softcap=-1.0), dict(out=q),
                dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(m.NVFP4KVError):
            m.tree_attention(cache, **{**ok, **bad})
    ok = dict(block_table=t, seq_lens=n, cu_q_lens=cu, accepted=ints([[0, 1]]), num_accepted=ints([2]))
    m.accept_tokens(cache, **ok)
    for bad in (dict(accepted=ints([0, 1])), dict(num_accepted=ints([2, 2])), dict(cu_q_lens=n), dict(new_lens=n.long())):
        with pytest.raises(ValueError):
            m.accept_tokens(cache, **{**ok, **bad})
    with pytest.raises(m.NVFP4KVError):
        m.accept_tokens(cache, **ok, new_lens=n)
    assert m.check_device_errors() == 0
