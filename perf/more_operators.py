"""The operators of a speculative decoding step over the NVFP4 pages as they are measured: cases over their real
range, their inputs, one pass of each (the framework's calls where `own` is true, else the same operators in
elementary torch operations) and their values in 64 bits.

  write    the queries and keys of a projection normalised a head, rotated by their positions, and the keys and
           values quantised into the paged cache in the same pass, then read back as prefix_dequant hands them to
           the chunk attention
  tree     the queries of drafted tokens over the cached tokens and, of the drafts, their ancestors in the tree;
           scores capped by a tanh, limited to a window or biased by distance where the model does so
  accept   the drafts' keys and values appended, the accepted ones moved together behind the prefix, and the rows
           of the pages that hold them read back
"""

import math

import torch

own = False

HEAD = 128
GROUP = 2304                       # bytes of a 16-token group of a page
TABLE = 40960                      # positions of the rotation table


# ---------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step of a small batch: eight new tokens, latency alone
        dict(name="write 8", op="write", tokens=8, heads=32, kv_heads=8, page=16, rot=128, adjacent=False, axes=1,
             norm=False, scale=1.0),
        # a prefill with norms of the heads, bandwidth
        dict(name="write 32768 norm", op="write", tokens=32768, heads=64, kv_heads=8, page=64, rot=128, adjacent=False,
             axes=1, norm=True, scale=1.0),
        # an image's tokens with positions of three axes under calibrated tensor scales, odd count
        dict(name="write 5003 axes3", op="write", tokens=5003, heads=40, kv_heads=8, page=64, rot=128, adjacent=False,
             axes=3, norm=True, scale=0.75),
        # half of the head rotated, neighbouring values paired
        dict(name="write 2048 half", op="write", tokens=2048, heads=32, kv_heads=2, page=32, rot=64, adjacent=True,
             axes=1, norm=False, scale=1.0),
        # the smallest tree over one short sequence, 4 query heads on one kv head
        dict(name="tree b1 q4kv1 d4 n77", op="tree", batch=1, heads=4, kv_heads=1, drafts=4, tokens=77, page=16,
             cap=0.0, window=0, slopes=False),
        # a plain decode step of a model that caps its scores and sees 4,096 tokens back
        dict(name="tree b64 q64kv8 d1 n8192 cap", op="tree", batch=64, heads=64, kv_heads=8, drafts=1, tokens=8192,
             page=64, cap=50.0, window=4096, slopes=False),
        # an ordinary serving batch with trees of eight drafts
        dict(name="tree b32 q32kv8 d8 n4096", op="tree", batch=32, heads=32, kv_heads=8, drafts=8, tokens=4096, page=64,
             cap=0.0, window=0, slopes=False),
        # 32K contexts, 16 drafts of 64 query heads
        dict(name="tree b16 q64kv8 d16 n32768", op="tree", batch=16, heads=64, kv_heads=8, drafts=16, tokens=32768,
             page=64, cap=0.0, window=0, slopes=False),
        # large trees over short contexts, scores biased by distance
        dict(name="tree b4 q64kv8 d60 n2000 bias", op="tree", batch=4, heads=64, kv_heads=8, drafts=60, tokens=2000,
             page=128, cap=0.0, window=0, slopes=True),
        # one sequence's accepted path
        dict(name="accept b1 kv8 d8", op="accept", batch=1, kv_heads=8, drafts=8, prefix=300, page=16, scale=1.0),
        # a large batch with large trees
        dict(name="accept b128 kv8 d60", op="accept", batch=128, kv_heads=8, drafts=60, prefix=1000, page=64, scale=0.75),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["write", "write", "tree", "tree", "tree", "accept"])
    page, kv_heads = rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
    if op == "write":
        axes = rng.choice([1, 1, 3])
        return dict(op=op, tokens=_log(rng, 1, 32768), heads=heads, kv_heads=kv_heads, page=page,
                    rot=128 if axes == 3 else rng.choice([32, 64, 96, 128]), adjacent=rng.random() < 0.3, axes=axes,
                    norm=rng.random() < 0.5, scale=rng.choice([1.0, 0.75, 0.375]))
    if op == "tree":
        drafts = _log(rng, 1, 64)
        batch = _log(rng, 1, 64)
        top = min(65536, 4_000_000 // (batch * kv_heads), 500_000_000 // (batch * heads * drafts))
        kind = rng.choice(["", "", "cap", "window", "slopes"])
        return dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, drafts=drafts,
                    tokens=max(drafts, _log(rng, 1, max(1, top))), page=page, cap=30.0 if kind == "cap" else 0.0,
                    window=_log(rng, 1, 8192) if kind == "window" else 0, slopes=kind == "slopes")
    return dict(op=op, batch=_log(rng, 1, 128), kv_heads=kv_heads, drafts=_log(rng, 1, 64), prefix=rng.randint(0, 1000),
                page=page, scale=rng.choice([1.0, 0.75]))


def _lengths(count, longest):
    """Ragged lengths: the first is the longest, the others spread down to about a third of it."""
    return [max(1, int(longest * (1.0 - 0.66 * ((i * 0.6180339887) % 1.0)))) for i in range(count)]


def _tree_lengths(case):
    """(cached tokens, drafts among them) of each sequence; the draft counts are ragged too."""
    drafts = _lengths(case["batch"], case["drafts"])
    return [max(n, d) for n, d in zip(_lengths(case["batch"], case["tokens"]), drafts)], drafts


def _tails(case):
    """Of each sequence: prefix, drafts, and the first page that holds a draft."""
    drafts = _lengths(case["batch"], case["drafts"])
    prefix = [p - 1 for p in _lengths(case["batch"], case["prefix"] + 1)]
    return prefix, drafts, [p // case["page"] for p in prefix]


def work(case):
    op = case["op"]
    if op == "write":
        t, q, h = case["tokens"], case["heads"], case["kv_heads"]
        # projections, positions and slots in, queries and the cache's bytes out, the rotation table's rows in; the
        # cache's bytes in, BF16 rows out
        rows = min(t * case["axes"], TABLE) * case["rot"] * 4
        return dict(bytes=t * ((q + 2 * h) * 256 + 4 * case["axes"] + 8 + q * 256 + h * 144) + rows + t * h * (144 + 512),
                    flops=0)
    if op == "tree":
        n, d = _tree_lengths(case)
        seen = [min(x, case["window"] + y) if case["window"] else x for x, y in zip(n, d)]
        pairs = sum(x * y for x, y in zip(seen, d))
        return dict(bytes=sum(seen) * case["kv_heads"] * 144 + sum(d) * (case["heads"] * 512 + 8),
                    flops=4 * HEAD * case["heads"] * pairs)
    prefix, drafts, first = _tails(case)
    back = sum(p + d - f * case["page"] for p, d, f in zip(prefix, drafts, first))
    moved = sum(drafts) // 4
    # drafts in, their bytes out; the moved ones in and out; the read rows in, BF16 rows out
    return dict(bytes=case["kv_heads"] * (sum(drafts) * (512 + 144) + moved * 288 + back * (144 + 512)), flops=0)


# --------------------------------------------------------------------------------------------------- the inputs

def _random(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _normal(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def _code_bytes(n, g):
    """n bytes of two E2M1 codes each, distributed as those of normal values under a block scale near 1/3."""
    u = (torch.arange(256, dtype=torch.float64) + 0.5) / 256
    y = torch.special.ndtri(u) * 3.0
    code = torch.bucketize(y.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64))
    code = (code + 8 * (y < 0)).to(torch.int64)
    table = (code[None, :] + 16 * code[:, None]).reshape(-1).to(torch.uint8).cuda()
    return table[torch.randint(0, 65536, (n,), generator=g, device="cuda")]


def _scale_bytes(n, g):
    return torch.randint(0x28, 0x30, (n,), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)


def _tables(lengths, page, g):
    """Randomly placed pages for each sequence (-1 behind its last), and their number."""
    counts = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(counts), generator=g, device="cuda").to(torch.int32)
    at = torch.zeros(len(counts) + 1, dtype=torch.int64)
    at[1:] = torch.cumsum(torch.tensor(counts), 0)
    col = torch.arange(max(counts))
    here = col[None, :] < torch.tensor(counts)[:, None]
    index = (at[:-1, None] + col[None, :]).clamp(max=sum(counts) - 1)
    table = torch.where(here.cuda(), order[index.cuda()], torch.full((), -1, dtype=torch.int32, device="cuda"))
    return table.contiguous(), sum(counts)


def _pool(pages, kv_heads, page, g):
    groups = pages * kv_heads * (page // 16)
    pool = torch.empty((groups, GROUP), dtype=torch.uint8, device="cuda")
    for at in (0, 1024 + 128):
        pool[:, at:at + 1024] = _code_bytes(groups * 1024, g).view(groups, 1024)
        pool[:, at + 1024:at + 1152] = _scale_bytes(groups * 128, g).view(groups, 128)
    return pool.view(pages, kv_heads, page // 16 * GROUP)


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _sums(x):
    return _ints([0] + torch.cumsum(torch.tensor(x), 0).tolist())


def _trees(drafts, seed):
    """Random trees: each sequence's first draft is the root, every other one hangs on an earlier one.  The masks of
    all drafts in a row (bit j of draft i's: it sees draft j), as Python numbers, and the parents."""
    g = torch.Generator()
    g.manual_seed(int(seed) * 7919 % (1 << 62) + 3)
    masks, parents = [], []
    for d in drafts:
        u = torch.rand(d, generator=g).tolist()
        par = [-1] + [int(u[i] * i) for i in range(1, d)]
        m = []
        for i, p in enumerate(par):
            m.append((m[p] if p >= 0 else 0) | 1 << i)
        masks.append(m)
        parents.append(par)
    return masks, parents, g


def _signed(m):
    return m - (1 << 64) if m >> 63 else m


def _rotation_table(rot, base):
    """cos | sin of position p times base^(-2 i / rot), float32 [TABLE][rot]."""
    angle = torch.arange(TABLE, device="cuda", dtype=torch.float64)[:, None] \
        * base ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
    return torch.cat([torch.cos(angle), torch.sin(angle)], 1).float().contiguous()


def prepare(case, seed):
    g, op = _random(seed), case["op"]
    if op == "write":
        t, page, q, h = case["tokens"], case["page"], case["heads"], case["kv_heads"]
        # rows of a fused projection: queries, keys, values; keys with a few outliers
        rows = torch.randn((t, (q + 2 * h) * HEAD), generator=g, device="cuda")
        hit = torch.rand((t, h * HEAD), generator=g, device="cuda") < 0.01
        rows[:, q * HEAD:(q + h) * HEAD] *= torch.where(hit, 8.0, 1.0)
        table, pages = _tables([t], page, g)
        at = torch.arange(t, device="cuda")
        start = int(torch.randint(0, TABLE - t, (1,), generator=g, device="cuda"))
        pos = (start + at)[None]
        if case["axes"] == 3:      # an image behind some text: its frame, its row, its column
            pos = torch.stack([torch.full_like(at, start // 8), start // 8 + at // 89, start // 8 + at % 89])
        s = dict(case=case, rows=rows.to(torch.bfloat16), table=table, lens=_ints([t]), sums=_sums([t]),
                 slots=table[0].to(torch.int64)[at // page] * page + at % page, pos=pos.to(torch.int32).contiguous(),
                 turn=_rotation_table(case["rot"], 1e6), sections=[16, 24, 24] if case["axes"] == 3 else None,
                 pool=torch.zeros((pages, h, page * 144), dtype=torch.uint8, device="cuda"), wq=None, wk=None)
        if case["norm"]:
            s["wq"], s["wk"] = _normal((HEAD,), g, 0.2) + 1, _normal((HEAD,), g, 0.2) + 1
        return s
    if op == "tree":
        n, d = _tree_lengths(case)
        table, pages = _tables(n, case["page"], g)
        masks, _, _ = _trees(d, seed)
        return dict(case=case, pool=_pool(pages, case["kv_heads"], case["page"], g), table=table, lens=_ints(n),
                    sums=_sums(d), q=_normal((sum(d), case["heads"], HEAD), g),
                    mask=_ints([_signed(x) for m in masks for x in m], torch.int64),
                    # powers of two from 1/2 down, spread over the heads
                    slopes=torch.exp2(-8.0 * torch.arange(1, case["heads"] + 1, device="cuda") / case["heads"])
                    if case["slopes"] else None)
    prefix, drafts, first = _tails(case)
    page, h = case["page"], case["kv_heads"]
    total = [p + d for p, d in zip(prefix, drafts)]
    table, pages = _tables(total, page, g)
    _, parents, rng = _trees(drafts, seed)
    accepted, count = torch.full((len(drafts), case["drafts"]), -1, dtype=torch.int32), []
    for b, par in enumerate(parents):       # the path from the root to a draft, cut where the model disagrees
        x, path = int(torch.randint(0, len(par), (1,), generator=rng)), []
        while x >= 0:
            path.append(x)
            x = par[x]
        path = path[::-1][:int(torch.randint(1, len(path) + 1, (1,), generator=rng))]
        accepted[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
        count.append(len(path))
    seq = torch.repeat_interleave(torch.arange(len(drafts)), torch.tensor(drafts)).cuda()
    sums = _sums(drafts)
    at = torch.arange(sum(drafts), device="cuda") - sums[seq] + _ints(prefix)[seq]
    rows = torch.randn((sum(drafts), 2 * h * HEAD), generator=g, device="cuda").to(torch.bfloat16)
    tail = [t - f * page for t, f in zip(total, first)]
    width = max(-(-t // page) for t in tail)
    cols = (_ints(first, torch.int64)[:, None] + torch.arange(width, device="cuda")).clamp(max=table.shape[1] - 1)
    return dict(case=case, pool=_pool(pages, h, page, g), table=table, lens=_ints(total), sums=sums, rows=rows,
                slots=table.long()[seq, at // page] * page + at % page, accepted=accepted.cuda(), count=_ints(count),
                tail_table=torch.gather(table, 1, cols).contiguous(), tail_lens=_ints(tail), tail_sums=_sums(tail),
                tail_total=sum(tail), start=_ints([p - f * page for p, f in zip(prefix, first)]), seq=seq)


# --------------------------------------------------------------------------------------- the operators, plainly

def _e2m1(nibble):
    t = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    return t[nibble.to(torch.int64)]


def _unpack(codes):
    """Bytes of two codes -> their values, the low nibble first, along the last axis."""
    return torch.stack([_e2m1(codes & 15), _e2m1(codes >> 4)], -1).flatten(-2)


def _e4m3(x):
    return x.view(torch.float8_e4m3fn).to(torch.float32)


def _round_e4m3(x):
    step = torch.tensor([2.0**i for i in range(-9, 6)], dtype=x.dtype, device="cuda")
    step = step[(torch.frexp(x).exponent + 5).clamp(min=0, max=14).long()]
    return (torch.round(x / step) * step).clamp(max=448)


def _bf16(x):
    """64-bit numbers rounded to BF16 once (a conversion would pass through 32 bits first)."""
    step = torch.ldexp(torch.ones_like(x), torch.frexp(x).exponent.clamp(min=-125) - 8)
    out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    out.copy_(torch.round(x / step) * step)
    return out


def _quantised(x, g):
    """BF16 values as the cache holds them, in 64 bits: values next to a rounding border decide a code."""
    x = x.to(torch.float64).unflatten(-1, (HEAD // 16, 16))
    # (a division by a number would multiply with its rounded reciprocal: quotients on a border would leave it)
    scale = _round_e4m3(x.abs().amax(-1, keepdim=True) / torch.full((), 6 * g, dtype=torch.float64, device="cuda"))
    y = x.abs() / torch.where(scale > 0, scale * g, torch.ones_like(scale))
    mag = 0.5 * ((y > 0.25).double() + (y >= 0.75) + (y > 1.25) + (y >= 1.75)) + (y > 2.5).double() + (y >= 3.5) \
        + 2 * (y > 5).double()
    return _bf16((torch.copysign(mag, x) * scale * g).flatten(-2))


def _turned(x, weight, s):
    """The heads x [tokens][heads][128] normalised (where there is a weight) and rotated, rounded to BF16 once.  In 64
    bits: a key next to a border of BF16 would be quantised to another code."""
    case, x = s["case"], x.to(torch.float64)
    rot, half = case["rot"], case["rot"] // 2
    if weight is not None:
        x = x * weight.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    pair = torch.arange(half, device="cuda")
    axis = torch.bucketize(pair, torch.tensor([16, 40], device="cuda"), right=True) if case["axes"] == 3 else pair * 0
    at = s["pos"].long()[axis].T                                     # [tokens][pairs]
    cos, sin = s["turn"][at, pair].double()[:, None], s["turn"][at, half + pair].double()[:, None]
    if case["adjacent"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return _bf16(torch.cat([turned, x[..., rot:]], -1))


def _split(s):
    case = s["case"]
    return s["rows"].unflatten(-1, (-1, HEAD)).split([case["heads"], case["kv_heads"], case["kv_heads"]], 1)


def _plain_write(s):
    q, k, v = _split(s)
    g = s["case"]["scale"]
    return _turned(q, s["wq"], s), _quantised(_turned(k, s["wk"], s), g), _quantised(v, g)


def _rows(pool, page, pages, rows):
    """float32 K and V rows [...][kv heads][128] (without tensor scales) at `rows` of `pages`."""
    grp = pool.view(pool.shape[0], pool.shape[1], page // 16, GROUP).transpose(1, 2)   # [pages][groups][heads][bytes]
    j, r = rows // 16, rows % 16
    k = _unpack(grp[..., :1024].unflatten(-1, (16, 64)).permute(0, 1, 3, 2, 4)[pages, j, r])
    ks = grp[..., 1024:1152].unflatten(-1, (16, 8)).permute(0, 1, 3, 2, 4)[pages, j, r]
    v = _unpack(grp[..., 1152:2176].unflatten(-1, (16, 64)).permute(0, 1, 3, 2, 4)[pages, j, r])
    vs = grp[..., 2176:].unflatten(-1, (8, 16)).permute(0, 1, 4, 2, 3)[pages, j, r]
    return tuple((x.unflatten(-1, (8, 16)) * _e4m3(y.contiguous())[..., None]).flatten(-2) for x, y in ((k, ks), (v, vs)))


def _at(table, page, count):
    t = torch.arange(count, device="cuda")
    return table.to(torch.int64).clamp(min=0)[:, t // page], (t % page).expand(table.shape[0], count)


def _plain_tree(s):
    case = s["case"]
    page, hkv, hq = case["page"], case["kv_heads"], case["heads"]
    drafts = s["sums"][1:] - s["sums"][:-1]
    n, d, b = s["table"].shape[1] * page, case["drafts"], case["batch"]
    k, v = _rows(s["pool"], page, *_at(s["table"], page, n))
    i = torch.arange(d, device="cuda")
    real = i[None, :] < drafts[:, None]
    row = torch.where(real, s["sums"][:-1, None] + i[None, :], 0).long()
    q = s["q"][row].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4)         # [b][hkv][d][group][128]
    score = (q.flatten(2, 3) @ k.permute(0, 2, 3, 1)).unflatten(2, (d, -1)) * (1 / math.sqrt(HEAD))
    if case["cap"]:
        score = case["cap"] * torch.tanh(score / case["cap"])
    bits = (s["mask"][row][..., None] >> i) & 1                                            # [b][d][d]
    base, t = (s["lens"] - drafts)[:, None], torch.arange(n, device="cuda")[None, :]
    place = base + bits.sum(-1) - 1                                                        # positions of the drafts
    j = (t - base).clamp(min=0, max=d - 1).long()
    seen = (t < base)[:, None] | (torch.gather(bits, 2, j[:, None].expand(-1, d, -1)) == 1)
    seen = seen & (t < s["lens"][:, None])[:, None]
    where = torch.where(t < base, t.expand(b, n), torch.gather(place, 1, j))               # positions of the keys
    away = where[:, None] - place[..., None]                                               # [b][d][n]
    if case["window"]:
        seen = seen & (away > -case["window"])
    if case["slopes"]:
        score = score + s["slopes"].view(hkv, 1, -1, 1) * away[:, None, :, None].float()
    score = torch.where(seen[:, None, :, None], score, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    o = (p.flatten(2, 3) @ v.transpose(1, 2)) / p.sum(-1).flatten(2)[..., None].clamp(min=1e-30)
    return o.unflatten(2, (d, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)[real].to(torch.bfloat16)


def _plain_accept(s):
    case = s["case"]
    page, h, g = case["page"], case["kv_heads"], case["scale"]
    b, width = case["batch"], s["tail_table"].shape[1] * page
    drafts = s["sums"][1:] - s["sums"][:-1]
    k, v = _rows(s["pool"], page, *_at(s["tail_table"], page, width))
    k, v = _bf16(k.double() * g), _bf16(v.double() * g)
    new_k, new_v = (_quantised(x, g) for x in s["rows"].unflatten(-1, (2, h, HEAD)).unbind(1))
    at = torch.arange(s["rows"].shape[0], device="cuda") - s["sums"][s["seq"]] + s["start"][s["seq"]]
    k[s["seq"], at], v[s["seq"], at] = new_k, new_v
    i = torch.arange(case["drafts"], device="cuda")
    source = torch.arange(width + case["drafts"], device="cuda").repeat(b, 1)
    to = (s["start"][:, None] + i).long()
    source.scatter_(1, to, torch.where(i < s["count"][:, None], s["start"][:, None] + s["accepted"], to))
    source = source[:, :width].clamp(max=width - 1)
    seq = torch.arange(b, device="cuda")[:, None]
    here = torch.arange(width, device="cuda") < s["tail_lens"][:, None]
    return s["lens"] - drafts + s["count"], k[seq, source][here], v[seq, source][here]


# ------------------------------------------------------------------------------------ the framework's own calls

def _handle(s, kv):
    """The cache handle (and, where the call wants one, the workspace) that a user's program keeps."""
    if "handle" not in s:
        case = s["case"]
        g = case.get("scale", 1.0)
        s["handle"] = kv.PagedCache(s["pool"].shape[0], case["page"], case["kv_heads"], k_global_scale=g,
                                    v_global_scale=g, pool=s["pool"])
        if case["op"] == "tree":
            s["workspace"] = kv.alloc_tree_workspace(s["handle"], case["batch"], case["heads"], case["drafts"])
    return s["handle"]


def _own(s):
    import nvfp4_quantised_paged_gb300 as kv
    case, op = s["case"], s["case"]["op"]
    cache = _handle(s, kv)
    if op == "write":
        q, k, v = _split(s)
        turned = kv.rope_quantize_append(cache, q, k, v, s["pos"], s["turn"], s["slots"], q_norm=s["wq"], k_norm=s["wk"],
                                         eps=1e-6, adjacent=case["adjacent"], sections=s["sections"])
        return (turned,) + tuple(kv.prefix_dequant(cache, s["table"], s["lens"], s["sums"], case["tokens"]))
    if op == "tree":
        return kv.tree_attention(cache, s["q"], s["sums"], case["drafts"], s["table"], s["lens"], tree_mask=s["mask"],
                                 softcap=case["cap"], window=case["window"], slopes=s["slopes"],
                                 workspace=s["workspace"])
    k, v = s["rows"].unflatten(-1, (2, case["kv_heads"], HEAD)).unbind(1)
    kv.quantize_append(cache, k, v, s["slots"])
    lens = kv.accept_tokens(cache, s["table"], s["lens"], s["sums"], s["accepted"], s["count"])
    return (lens,) + tuple(kv.prefix_dequant(cache, s["tail_table"], s["tail_lens"], s["tail_sums"], s["tail_total"]))


def run(state):
    if own:
        return _own(state)
    return dict(write=_plain_write, tree=_plain_tree, accept=_plain_accept)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------- the values, exactly

def _x_nibbles(codes):
    c = codes.to(torch.int64)
    c = torch.stack([c % 16, c // 16], -1).flatten(-2)
    e, m = (c % 8) // 2, (c % 2).double()
    v = torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1) * (1 + 0.5 * m))
    return torch.where(c >= 8, -v, v)


def _x_scale(b):
    b = b.to(torch.int64)
    e, m = b // 8, (b % 8).double()
    return torch.where(e == 0, m * 2.0**-9, torch.exp2(e.double() - 7) * (1 + m / 8))


def _x_sequence(slabs, n):
    """K and V of n tokens of one kv head from its groups [groups][2304] in order, in 64 bits."""
    k = _x_nibbles(slabs[:, :1024]).view(-1, 16) * _x_scale(slabs[:, 1024:1152]).view(-1, 1)
    v = _x_nibbles(slabs[:, 1152:2176]).view(-1, 16, 8, 16)
    v = v * _x_scale(slabs[:, 2176:]).view(-1, 8, 16).transpose(1, 2)[..., None]
    return k.view(-1, HEAD)[:n], v.reshape(-1, HEAD)[:n]


def _x_to_bf16(x):
    """Rounded to BF16 by adding and taking off 1.5 * 2^(52 - 7 - 52) times each value's power of two."""
    power = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0**-126))))
    big = power * (1.5 * 2.0**45)
    return (x + big) - big


def _x_cached(x, g):
    """What the cache holds of 64-bit x (BF16 numbers): the nearest scale and value of the format, ties to even."""
    grid = torch.cat([torch.arange(8, device="cuda").double() * 2.0**-9]
                     + [torch.arange(8, 16, device="cuda").double() * 2.0**(e - 10) for e in range(1, 16)])[:127]
    flat = x.reshape(-1, 16)
    top, grid6 = flat.abs().amax(1), grid * (6 * g)        # borders of amax itself: exact products
    hi = torch.searchsorted(grid6, top).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid6[hi] - top, top - grid6[lo]
    k = torch.where((up < down) | ((up == down) & (hi % 2 == 0)) | (top >= grid6[126]), hi, lo)
    scale = grid[torch.where(top == 0, 0, k)]
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    mids = (levels[1:] + levels[:-1]) / 2 * g
    left, out = flat.abs(), torch.zeros_like(flat)
    for i in range(7):       # a tie goes to the even code
        border = mids[i] * scale[:, None]
        out = torch.where((left > border) | ((left == border) & (i % 2 == 1)), levels[i + 1], out)
    return (torch.where(flat < 0, -out, out) * scale[:, None] * g).view(x.shape)


def _x_write(s):
    case = s["case"]
    t, q, h, rot = case["tokens"], case["heads"], case["kv_heads"], case["rot"]
    x = s["rows"].double().view(t, q + 2 * h, HEAD)
    heads = x[:, :q + h].clone()
    if case["norm"]:
        heads[:, :q] *= s["wq"].double()
        heads[:, q:] *= s["wk"].double()
        heads /= (x[:, :q + h].square().sum(-1, keepdim=True) / HEAD + 1e-6).sqrt()
    out = heads.clone()
    for i in range(rot // 2):
        axis = 0 if case["axes"] == 1 else (0 if i < 16 else 1 if i < 40 else 2)
        p = s["pos"][axis].long()
        z = torch.complex(s["turn"][p, i].double(), s["turn"][p, rot // 2 + i].double())[:, None]
        a, b = (2 * i, 2 * i + 1) if case["adjacent"] else (i, i + rot // 2)
        z = z * torch.complex(heads[..., a].contiguous(), heads[..., b].contiguous())
        out[..., a], out[..., b] = z.real, z.imag
    return out[:, :q], _x_cached(_x_to_bf16(out[:, q:]), case["scale"]), _x_cached(x[:, q + h:], case["scale"])


def _x_tree(s):
    case = s["case"]
    page, hkv = case["page"], case["kv_heads"]
    group = case["heads"] // hkv
    grp = s["pool"].view(s["pool"].shape[0], hkv, -1, GROUP)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    sums, masks = s["sums"].tolist(), s["mask"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        d = sums[b + 1] - sums[b]
        m = [x % (1 << 64) for x in masks[sums[b]:sums[b + 1]]]
        depth = [bin(x).count("1") - 1 for x in m]
        position = _ints(list(range(n - d)) + [n - d + x for x in depth], torch.float64)
        sees = torch.ones((d, n), dtype=torch.bool)
        for i in range(d):
            sees[i, n - d:] = torch.tensor([bool(m[i] >> j & 1) for j in range(d)])
        sees = sees.cuda()
        distance = position[None, :] - position[n - d:, None]
        if case["window"]:
            sees &= distance > -case["window"]
        for h in range(hkv):
            k, v = _x_sequence(grp[s["table"][b, : -(-n // page)].long(), h].reshape(-1, GROUP), n)
            q = s["q"][sums[b]:sums[b + 1], h * group:(h + 1) * group].double().transpose(0, 1)   # [group][d][128]
            z = q @ k.T / math.sqrt(HEAD)
            if case["cap"]:
                z = torch.tanh(z / case["cap"]) * case["cap"]
            if case["slopes"]:
                z = z + s["slopes"][h * group:(h + 1) * group].double()[:, None, None] * distance
            z = z.masked_fill(~sees, -math.inf)
            out[sums[b]:sums[b + 1], h * group:(h + 1) * group] = (torch.softmax(z, -1) @ v).transpose(0, 1)
    return out


def _x_accept(s):
    case = s["case"]
    page, h, g = case["page"], case["kv_heads"], case["scale"]
    grp = s["pool"].view(s["pool"].shape[0], h, -1, GROUP)
    fresh = _x_cached(s["rows"].double(), g).view(-1, 2, h, HEAD)
    keys, values = [], []
    sums, start, count, path = s["sums"].tolist(), s["start"].tolist(), s["count"].tolist(), s["accepted"].tolist()
    for b, n in enumerate(s["tail_lens"].tolist()):
        pages = s["tail_table"][b, : -(-n // page)].long()
        x = torch.stack([torch.stack(_x_sequence(grp[pages, i].reshape(-1, GROUP), n)) for i in range(h)]) * g
        x = x.permute(2, 1, 0, 3).contiguous()                       # [rows][K, V][heads][128]
        new = fresh[sums[b]:sums[b + 1]]
        x[start[b]:start[b] + new.shape[0]] = new
        x[start[b]:start[b] + count[b]] = new[path[b][:count[b]]]
        keys.append(x[:, 0])
        values.append(x[:, 1])
    return None, torch.cat(keys), torch.cat(values)


def exact(case, seed):
    return dict(write=_x_write, tree=_x_tree, accept=_x_accept)[case["op"]](prepare(case, seed))
