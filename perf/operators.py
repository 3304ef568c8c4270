"""The latent-cache and eviction operators as they are measured: cases over their real range, their inputs, one
pass of each (the framework's calls where `own` is true, else the same operators in elementary torch operations)
and their values in 64 bits.

  latent_write    a chunk's latents quantised into the paged latent cache and read back as the BF16 workspace that
                  the expanded form multiplies with its up-projections (chunked prefill)
  latent_decode   one query a sequence over the paged latent cache, absorbed form
  latent_extend   a chunk's queries over [expanded prefix || expanded chunk], causal in the chunk
  weights         the attention weight that a decode step's queries put on every cached token, added to the scores
  evict           the tokens of largest score of each sequence and kv head, moved into new pages
"""

import math

import torch

own = False

LATENT, ROPE, HEAD = 512, 64, 128
GROUP_LATENT, GROUP_GQA = 6656, 2304      # bytes of a 16-token group of a page


# ---------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step of a small batch: 16 new tokens written, latency alone
        dict(name="write 16", op="latent_write", tokens=16, page=64, scale=1.0),
        # a prefill's 65,536 tokens through a calibrated tensor scale, bandwidth
        dict(name="write 65536", op="latent_write", tokens=65536, page=64, scale=0.75),
        # the smallest call: one short sequence, 16 heads (one of eight GPUs' share of 128)
        dict(name="decode b1 h16 n77", op="latent_decode", batch=1, heads=16, tokens=77, page=16, scale=1.0),
        # an ordinary serving batch, ragged lengths, few heads: bound by the cache's bytes
        dict(name="decode b32 h16 n8192", op="latent_decode", batch=32, heads=16, tokens=8192, page=64, scale=1.0),
        # many sequences of a few thousand tokens, 64 heads
        dict(name="decode b64 h64 n4096", op="latent_decode", batch=64, heads=64, tokens=4096, page=64, scale=0.75),
        # long contexts with all 128 heads: bound by the tensor cores
        dict(name="decode b8 h128 n32768", op="latent_decode", batch=8, heads=128, tokens=32768, page=128, scale=1.0),
        # a short chunk over a short prefix, odd sizes
        dict(name="extend r2 l17 p100", op="latent_extend", reqs=2, heads=8, chunk=17, prefix=100),
        # chunked prefill: 512-token chunks over prefixes of up to 8K tokens
        dict(name="extend r4 l512 p8192", op="latent_extend", reqs=4, heads=32, chunk=512, prefix=8192),
        # the smallest decode workload: 4 query heads on one kv head
        dict(name="weights b2 q4kv1 n300", op="weights", batch=2, heads=4, kv_heads=1, tokens=300, page=16),
        # 32K contexts, 64 query and 8 kv heads
        dict(name="weights b16 q64kv8 n32768", op="weights", batch=16, heads=64, kv_heads=8, tokens=32768, page=64),
        # a short cache cut to 64 tokens
        dict(name="evict b2 kv1 n300", op="evict", batch=2, kv_heads=1, tokens=300, page=16, keep=64, recent=16, sink=4),
        # 32K contexts cut to an eighth
        dict(name="evict b16 kv8 n32768", op="evict", batch=16, kv_heads=8, tokens=32768, page=64, keep=4096,
             recent=256, sink=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["latent_write", "latent_decode", "latent_decode", "latent_extend", "weights", "evict"])
    page = rng.choice([16, 32, 64, 128])
    if op == "latent_write":
        return dict(op=op, tokens=_log(rng, 1, 65536), page=page, scale=rng.choice([1.0, 0.75, 0.375]))
    if op == "latent_decode":
        heads = rng.choice([1, 5, 16, 24, 32, 40, 64, 96, 128])
        batch = _log(rng, 1, 64)
        top = max(64, min(131072, 33_000_000 // (batch * max(heads, 16))))
        return dict(op=op, batch=batch, heads=heads, tokens=_log(rng, 1, top), page=page,
                    scale=rng.choice([1.0, 0.75, 0.375]))
    if op == "latent_extend":
        reqs, heads = rng.randint(1, 4), rng.choice([1, 3, 8, 16, 32])
        return dict(op=op, reqs=reqs, heads=heads, chunk=_log(rng, 1, 512), prefix=_log(rng, 1, 8192))
    kv_heads = rng.choice([1, 2, 5, 8])
    batch = _log(rng, 1, 16)
    tokens = _log(rng, 1, min(65536, 4_190_000 // (batch * kv_heads)))
    if op == "weights":
        return dict(op=op, batch=batch, heads=kv_heads * rng.choice([1, 3, 4, 5, 8, 16]), kv_heads=kv_heads,
                    tokens=tokens, page=page)
    keep = _log(rng, 1, max(1, min(tokens, 8192)))
    recent = rng.randint(0, keep // 4)
    return dict(op=op, batch=batch, kv_heads=kv_heads, tokens=tokens, page=page, keep=keep, recent=recent,
                sink=rng.randint(0, min(4, keep - recent)))


def _lengths(count, longest):
    """Ragged lengths: the first is the longest, the others spread down to about a third of it."""
    return [max(1, int(longest * (1.0 - 0.66 * ((i * 0.6180339887) % 1.0)))) for i in range(count)]


def work(case):
    op = case["op"]
    if op == "latent_write":
        t = case["tokens"]
        # BF16 rows and slots in, the cache's bytes out; those bytes in, BF16 rows out
        return dict(bytes=t * (2 * 576 + 8 + 416) + t * (416 + 2 * 576), flops=0)
    if op == "latent_decode":
        n, b, h = sum(_lengths(case["batch"], case["tokens"])), case["batch"], case["heads"]
        return dict(bytes=n * 416 + b * h * 2 * (576 + 512), flops=2 * n * h * (576 + 512))
    if op == "latent_extend":
        p, r, h, c = _lengths(case["reqs"], case["prefix"]), case["reqs"], case["heads"], _lengths(case["reqs"], case["chunk"])
        rows = sum(p) + sum(c)
        pairs = sum(x * y + x * (x + 1) // 2 for x, y in zip(c, p))
        return dict(bytes=rows * (h * 2 * 256 + 128) + sum(c) * h * 2 * (192 + 128), flops=2 * pairs * h * (192 + 128))
    n = sum(_lengths(case["batch"], case["tokens"]))
    if op == "weights":
        return dict(bytes=n * case["kv_heads"] * (72 + 8) + case["batch"] * case["heads"] * 256,
                    flops=2 * n * case["heads"] * 128)
    kept = sum(min(x, case["keep"]) for x in _lengths(case["batch"], case["tokens"]))
    capacity = case["batch"] * case["kv_heads"] * case["tokens"]
    # scores in, the kept rows in and out, their indices out, the new scores out
    return dict(bytes=case["kv_heads"] * (n * 4 + kept * (144 + 144 + 4)) + 4 * capacity, flops=0)


# --------------------------------------------------------------------------------------------------- the inputs

def _random(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
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


def _tables(lengths, page, g, first=0):
    """Randomly placed pages for each sequence (-1 behind its last), and their number."""
    counts = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(counts), generator=g, device="cuda").to(torch.int32) + first
    at = torch.zeros(len(counts) + 1, dtype=torch.int64)
    at[1:] = torch.cumsum(torch.tensor(counts), 0)
    col = torch.arange(max(counts))
    here = col[None, :] < torch.tensor(counts)[:, None]
    index = (at[:-1, None] + col[None, :]).clamp(max=sum(counts) - 1)
    table = torch.where(here.cuda(), order[index.cuda()], torch.full((), -1, dtype=torch.int32, device="cuda"))
    return table.contiguous(), sum(counts)


def _latent_pool(pages, page, g):
    groups = pages * (page // 16)
    pool = torch.empty((groups, GROUP_LATENT), dtype=torch.uint8, device="cuda")
    pool[:, :4096] = _code_bytes(groups * 4096, g).view(groups, 4096)
    pool[:, 4096:4608] = _scale_bytes(groups * 512, g).view(groups, 512)
    pool[:, 4608:] = _normal((groups, 1024), g).view(torch.uint8)
    return pool.view(pages, page // 16 * GROUP_LATENT)


def _gqa_pool(pages, kv_heads, page, g):
    groups = pages * kv_heads * (page // 16)
    pool = torch.empty((groups, GROUP_GQA), dtype=torch.uint8, device="cuda")
    for at in (0, 1024 + 128):
        pool[:, at:at + 1024] = _code_bytes(groups * 1024, g).view(groups, 1024)
        pool[:, at + 1024:at + 1152] = _scale_bytes(groups * 128, g).view(groups, 128)
    return pool.view(pages, kv_heads, page // 16 * GROUP_GQA)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _sums(x):
    return _ints([sum(x[:i]) for i in range(len(x) + 1)])


def prepare(case, seed):
    g, op = _random(seed), case["op"]
    if op == "latent_write":
        t, page = case["tokens"], case["page"]
        # rows of a fused projection: 512 normalised latent values (a few outliers), then the 64 rotary ones
        rows = torch.randn((t, 576), generator=g, device="cuda")
        hit = torch.rand((t, 576), generator=g, device="cuda") < 0.01
        rows = torch.where(hit, rows * 8, rows).to(torch.bfloat16)
        table, pages = _tables([t], page, g)
        at = torch.arange(t, device="cuda")
        slots = table[0].to(torch.int64)[at // page] * page + at % page
        return dict(case=case, rows=rows, slots=slots, table=table, lens=_ints([t]), sums=_sums([t]),
                    pool=torch.zeros((pages, page * 416), dtype=torch.uint8, device="cuda"))
    if op == "latent_decode":
        lengths = _lengths(case["batch"], case["tokens"])
        table, pages = _tables(lengths, case["page"], g)
        return dict(case=case, pool=_latent_pool(pages, case["page"], g), table=table, lens=_ints(lengths),
                    q=_normal((case["batch"], case["heads"], LATENT), g, 0.7),
                    qr=_normal((case["batch"], case["heads"], ROPE), g))
    if op == "latent_extend":
        pre, new, h = _lengths(case["reqs"], case["prefix"]), _lengths(case["reqs"], case["chunk"]), case["heads"]
        # K (128 values a head without rotation) and V as the up-projection of the latents leaves them, side by side
        return dict(case=case, pre=_sums(pre), new=_sums(new), q=_normal((sum(new), h, 192), g),
                    kv_pre=_normal((sum(pre), h, 256), g), rope_pre=_normal((sum(pre), ROPE), g),
                    kv_new=_normal((sum(new), h, 256), g), rope_new=_normal((sum(new), ROPE), g))
    lengths = _lengths(case["batch"], case["tokens"])
    table, pages = _tables(lengths, case["page"], g)
    s = dict(case=case, table=table, lens=_ints(lengths))
    shape = (case["batch"], case["kv_heads"], case["tokens"])
    if op == "weights":
        s["pool"] = _gqa_pool(pages, case["kv_heads"], case["page"], g)
        s["q"] = _normal((case["batch"], case["heads"], HEAD), g)
        s["scores"] = torch.rand(shape, generator=g, device="cuda")
        return s
    new, more = _tables([min(n, case["keep"]) for n in lengths], case["page"], g, first=pages)
    s["pool"] = _gqa_pool(pages + more, case["kv_heads"], case["page"], g)
    s["new_table"], s["first_new"] = new, pages
    # heavy-tailed scores, a tenth of them exactly zero (tokens that no query looked at)
    scores = torch.exp(torch.randn(shape, generator=g, device="cuda") * 2)
    s["scores"] = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.1, torch.zeros_like(scores), scores)
    return s


# --------------------------------------------------------------------------------------- the operators, plainly

def _e2m1(nibble):
    t = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    return t[nibble.to(torch.int64)]


def _unpack(codes):
    """Bytes of two codes -> their values, the low nibble first, along the last axis."""
    return torch.stack([_e2m1(codes & 15), _e2m1(codes >> 4)], -1).flatten(-2)


def _e4m3(x):
    return x.view(torch.float8_e4m3fn).to(torch.float32)


def _latent_values(pool, page, pages, rows):
    """float32 latents (without the tensor scale) and rotary parts of the tokens at `rows` of `pages`."""
    grp = pool.view(pool.shape[0], page // 16, GROUP_LATENT)
    j, r = rows // 16, rows % 16
    codes = grp[..., :4096].unflatten(-1, (8, 16, 32)).permute(0, 1, 3, 2, 4)[pages, j, r]
    scales = grp[..., 4096:4608].unflatten(-1, (16, 2, 8, 2))[pages, j, r].transpose(-3, -2)
    values = _unpack(codes).unflatten(-1, (2, 2, 16)) * _e4m3(scales.contiguous())[..., None]
    rope = grp[..., 4608:].unflatten(-1, (16, 8, 16))[pages, j, r]
    chunk = torch.arange(8, device="cuda") ^ (r % 8)[..., None]
    rope = torch.gather(rope, -2, chunk[..., None].expand(rope.shape)).contiguous().flatten(-2)
    return values.flatten(-4), rope.view(torch.bfloat16)


def _at(table, page, count):
    t = torch.arange(count, device="cuda")
    return table.to(torch.int64).clamp(min=0)[:, t // page], (t % page).expand(table.shape[0], count)


def _round_e4m3(x):
    step = torch.tensor([2.0**i for i in range(-9, 6)], dtype=x.dtype, device="cuda")
    step = step[(torch.frexp(x).exponent + 5).clamp(min=0, max=14).long()]
    return (torch.round(x / step) * step).clamp(max=448)


def _plain_write(s):
    """The cache's definition in 64 bits: values next to a rounding border decide a code."""
    x, g = s["rows"][:, :LATENT].to(torch.float64).unflatten(-1, (32, 16)), s["case"]["scale"]
    # (a division by a number would multiply with its rounded reciprocal: quotients on a border would leave it)
    scale = _round_e4m3(x.abs().amax(-1, keepdim=True) / torch.full((), 6 * g, dtype=torch.float64, device="cuda"))
    y = x.abs() / torch.where(scale > 0, scale * g, torch.ones_like(scale))
    mag = 0.5 * ((y > 0.25).double() + (y >= 0.75) + (y > 1.25) + (y >= 1.75)) + (y > 2.5).double() + (y >= 3.5) \
        + 2 * (y > 5).double()
    values = torch.copysign(mag, x) * scale * g
    out = torch.empty((x.shape[0], LATENT), dtype=torch.bfloat16, device="cuda")
    out.copy_(values.flatten(-2))
    return out, s["rows"][:, LATENT:].clone()


def _plain_decode(s):
    case = s["case"]
    n = int(case["tokens"])
    c, kr = _latent_values(s["pool"], case["page"], *_at(s["table"], case["page"], n))
    c = c * case["scale"]
    score = s["q"].float() @ c.transpose(1, 2) + s["qr"].float() @ kr.float().transpose(1, 2)
    score = score * (1 / math.sqrt(192))
    seen = torch.arange(n, device="cuda")[None, None, :] < s["lens"][:, None, None]
    score = torch.where(seen, score, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    return ((p @ torch.where(seen.transpose(1, 2), c, 0.0)) / p.sum(-1, keepdim=True)).to(torch.bfloat16)


def _padded(x, sums, longest):
    t = torch.arange(longest, device="cuda")
    here = t[None, :] < (sums[1:] - sums[:-1])[:, None]
    return x[torch.where(here, sums[:-1, None] + t[None, :], 0).long()].float(), here


def _plain_extend(s):
    case = s["case"]
    kv0, here0 = _padded(s["kv_pre"], s["pre"], case["prefix"])
    kv1, here1 = _padded(s["kv_new"], s["new"], case["chunk"])
    r0, r1 = _padded(s["rope_pre"], s["pre"], case["prefix"])[0], _padded(s["rope_new"], s["new"], case["chunk"])[0]
    q = _padded(s["q"], s["new"], case["chunk"])[0].transpose(1, 2)
    kv, rope = torch.cat([kv0, kv1], 1).transpose(1, 2), torch.cat([r0, r1], 1)[:, None]
    score = q[..., :HEAD] @ kv[..., :HEAD].transpose(2, 3) + q[..., HEAD:] @ rope.transpose(2, 3)
    t = torch.arange(case["chunk"], device="cuda")
    seen = torch.cat([here0[:, None, :].expand(-1, case["chunk"], -1), here1[:, None, :] & (t[None, :] <= t[:, None])], 2)
    score = torch.where(seen[:, None], score * (1 / math.sqrt(192)), -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    o = (p @ kv[..., HEAD:]) / p.sum(-1, keepdim=True)
    return o.transpose(1, 2)[here1].to(torch.bfloat16)


def _gqa_groups(pool, page):
    return pool.view(pool.shape[0], pool.shape[1], page // 16, GROUP_GQA)


def _plain_weights(s):
    case = s["case"]
    n, hkv = int(case["tokens"]), case["kv_heads"]
    pages, rows = _at(s["table"], case["page"], n)
    grp = _gqa_groups(s["pool"], case["page"]).transpose(1, 2)     # [pages][groups][heads][bytes]
    codes = grp[..., :1024].unflatten(-1, (16, 64)).permute(0, 1, 3, 2, 4)[pages, rows // 16, rows % 16]
    scales = grp[..., 1024:1152].unflatten(-1, (16, 8)).permute(0, 1, 3, 2, 4)[pages, rows // 16, rows % 16]
    k = (_unpack(codes).unflatten(-1, (8, 16)) * _e4m3(scales.contiguous())[..., None]).flatten(-2)
    q = s["q"].float().unflatten(1, (hkv, case["heads"] // hkv))
    score = q @ k.permute(0, 2, 3, 1) * (1 / math.sqrt(HEAD))
    seen = torch.arange(n, device="cuda")[None, None, None, :] < s["lens"][:, None, None, None]
    score = torch.where(seen, score, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    s["scores"] += (p / p.sum(-1, keepdim=True)).sum(2)
    return s["scores"]


def _plain_evict(s):
    case = s["case"]
    n, keep = s["lens"][:, None, None], min(case["keep"], case["tokens"])
    t = torch.arange(case["tokens"], device="cuda").expand(s["scores"].shape)
    key = torch.where((t < case["sink"]) | (t >= n - case["recent"]), math.inf, s["scores"])
    key = torch.where(t < n, key, -math.inf)
    first = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    first = torch.sort(torch.where(first < n, first, 1 << 40), dim=-1).values
    there = first < (1 << 40)
    kept = torch.full(s["scores"].shape[:2] + (case["keep"],), -1, dtype=torch.int32, device="cuda")
    kept[..., :keep] = torch.where(there, first, -1)
    new_scores = torch.zeros_like(s["scores"])
    new_scores[..., :keep] = torch.where(there, torch.gather(s["scores"], -1, first.clamp(max=case["tokens"] - 1)), 0.0)
    b, h, i = torch.nonzero(there, as_tuple=True)
    src, page = first[b, h, i], case["page"]
    sp, dp = s["table"].long()[b, src // page], s["new_table"].long()[b, i // page]
    sj, sr, dj, dr = src % page // 16, src % 16, i % page // 16, i % 16
    grp = _gqa_groups(s["pool"], page)
    views = (grp[..., :1024].unflatten(-1, (16, 64)), grp[..., 1024:1152].unflatten(-1, (16, 8)),
             grp[..., 1152:2176].unflatten(-1, (16, 64)), grp[..., 2176:].unflatten(-1, (8, 16)).transpose(-1, -2))
    views[0][dp, h, dj, dr] = views[0][sp, h, sj, sr]
    views[1][dp, h, dj, dr] = views[1][sp, h, sj, sr]
    views[2][dp, h, dj, dr] = views[2][sp, h, sj, sr]
    views[3][dp, h, dj, dr] = views[3][sp, h, sj, sr]
    return torch.clamp(s["lens"], max=case["keep"]), kept, new_scores, s["pool"][s["first_new"]:]


# ------------------------------------------------------------------------------------ the framework's own calls

def _handle(s, kv):
    """The cache handle (and, where the call wants one, the workspace) that a user's program keeps."""
    if "handle" not in s:
        case = s["case"]
        if case["op"].startswith("latent"):
            s["handle"] = kv.LatentCache(s["pool"].shape[0], case["page"], global_scale=case["scale"], pool=s["pool"])
        else:
            s["handle"] = kv.PagedCache(s["pool"].shape[0], case["page"], case["kv_heads"], pool=s["pool"])
        if case["op"] == "latent_decode":
            s["workspace"] = kv.alloc_latent_decode_workspace(s["handle"], case["batch"], case["heads"])
        if case["op"] == "weights":
            s["workspace"] = kv.alloc_weights_workspace(s["handle"], case["batch"], case["heads"])
    return s["handle"]


def _own(s):
    import nvfp4_quantised_paged_gb300 as kv
    case, op = s["case"], s["case"]["op"]
    if op == "latent_write":
        cache = _handle(s, kv)
        kv.latent_quantize_append(cache, s["rows"][:, :LATENT], s["rows"][:, LATENT:], s["slots"])
        return kv.latent_prefix_dequant(cache, s["table"], s["lens"], s["sums"], case["tokens"])
    if op == "latent_decode":
        return kv.latent_decode_attention(_handle(s, kv), s["q"], s["qr"], s["table"], s["lens"],
                                          workspace=s["workspace"])
    if op == "latent_extend":
        a, b = s["kv_pre"], s["kv_new"]
        return kv.latent_extend_attention(s["q"], a[..., :HEAD], a[..., HEAD:], s["rope_pre"], s["pre"], b[..., :HEAD],
                                          b[..., HEAD:], s["rope_new"], s["new"], case["chunk"])
    if op == "weights":
        return kv.accumulate_attention_weights(_handle(s, kv), s["q"], s["table"], s["lens"], s["scores"],
                                               workspace=s["workspace"])
    new_lens, kept, scores = kv.evict(_handle(s, kv), s["scores"], s["table"], s["lens"], s["new_table"], case["keep"],
                                      recent=case["recent"], sink=case["sink"])
    return new_lens, kept, scores, s["pool"][s["first_new"]:]


def run(state):
    if own:
        return _own(state)
    return dict(latent_write=_plain_write, latent_decode=_plain_decode, latent_extend=_plain_extend,
                weights=_plain_weights, evict=_plain_evict)[state["case"]["op"]](state)


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


def _x_latent_sequence(pool, page, table, n, scale):
    """One sequence's n latents and rotary parts, page by page as the format says, in 64 bits."""
    slabs = pool[table[: -(-n // page)].long()].view(-1, GROUP_LATENT)           # its groups in order
    values = _x_nibbles(slabs[:, :4096]).view(-1, 8, 16, 64)                      # [column block][row][64]
    b = slabs[:, 4096:4608].view(-1, 16, 32)
    block = torch.arange(32, device="cuda")
    s = _x_scale(b[:, :, block // 2 % 2 * 16 + block // 4 * 2 + block % 2])       # [row][block]
    values = values.transpose(1, 2).reshape(-1, 16, 32, 16) * s[..., None] * scale
    rope = slabs[:, 4608:].contiguous().view(torch.bfloat16).double().view(-1, 16, 8, 8)
    parts = [rope[:, r, [c ^ (r % 8) for c in range(8)]].flatten(1) for r in range(16)]
    return values.reshape(-1, LATENT)[:n], torch.stack(parts, 1).view(-1, ROPE)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "latent_write":
        g = case["scale"]
        x = s["rows"][:, :LATENT].double().view(-1, 16)
        grid = torch.cat([torch.arange(8, device="cuda").double() * 2.0**-9]
                         + [torch.arange(8, 16, device="cuda").double() * 2.0**(e - 10) for e in range(1, 16)])[:127]
        top, grid6 = x.abs().amax(1), grid * (6 * g)       # borders of amax itself: exact products
        hi = torch.searchsorted(grid6, top).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        up, down = grid6[hi] - top, top - grid6[lo]
        k = torch.where((up < down) | ((up == down) & (hi % 2 == 0)) | (top >= grid6[126]), hi, lo)
        scale = grid[torch.where(top == 0, 0, k)]
        levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        mids = (levels[1:] + levels[:-1]) / 2 * g
        left, out = x.abs(), torch.zeros_like(x)
        for i in range(7):       # a tie goes to the even code
            border = mids[i] * scale[:, None]
            out = torch.where((left > border) | ((left == border) & (i % 2 == 1)), levels[i + 1], out)
        out = torch.where(x < 0, -out, out) * scale[:, None] * g
        return out.view(-1, LATENT), s["rows"][:, LATENT:].double()
    if op == "latent_decode":
        outs = []
        for b, n in enumerate(s["lens"].tolist()):
            c, r = _x_latent_sequence(s["pool"], case["page"], s["table"][b], n, case["scale"])
            z = (s["q"][b].double() @ c.T + s["qr"][b].double() @ r.T) / math.sqrt(192)
            outs.append(torch.softmax(z, -1) @ c)
        return torch.stack(outs)
    if op == "latent_extend":
        outs = []
        p, c = s["pre"].tolist(), s["new"].tolist()
        for r in range(case["reqs"]):
            kv = torch.cat([s["kv_pre"][p[r]:p[r + 1]], s["kv_new"][c[r]:c[r + 1]]]).double()
            rope = torch.cat([s["rope_pre"][p[r]:p[r + 1]], s["rope_new"][c[r]:c[r + 1]]]).double()
            q, m = s["q"][c[r]:c[r + 1]].double(), p[r + 1] - p[r]
            out = torch.empty((q.shape[0], case["heads"], HEAD), dtype=torch.float64, device="cuda")
            for h in range(case["heads"]):
                z = torch.cat([q[:, h, :HEAD], q[:, h, HEAD:]], 1) @ torch.cat([kv[:, h, :HEAD], rope], 1).T
                z = z / math.sqrt(192) + torch.full_like(z, -math.inf).triu(m + 1)
                out[:, h] = torch.softmax(z, -1) @ kv[:, h, HEAD:]
            outs.append(out)
        return torch.cat(outs)
    if op == "weights":
        total = s["scores"].double()
        grp = s["pool"].view(s["pool"].shape[0], case["kv_heads"], -1, GROUP_GQA)
        g = case["heads"] // case["kv_heads"]
        for b, n in enumerate(s["lens"].tolist()):
            for h in range(case["kv_heads"]):
                slab = grp[s["table"][b, : -(-n // case["page"])].long(), h].reshape(-1, GROUP_GQA)
                k = _x_nibbles(slab[:, :1024]).view(-1, 16) * _x_scale(slab[:, 1024:1152]).view(-1, 1)
                z = s["q"][b, h * g:(h + 1) * g].double() @ k.view(-1, HEAD)[:n].T / math.sqrt(HEAD)
                total[b, h, :n] += torch.softmax(z, -1).sum(0)
        return total
    # the moved bytes and the kept indices are whole numbers; the new scores are the old ones of the kept tokens
    new_scores = torch.zeros(s["scores"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        for h in range(case["kv_heads"]):
            x = s["scores"][b, h, :n].double()
            if n > case["keep"]:
                last, first = n - case["recent"], min(case["sink"], n)
                middle = x[first:last]
                some = case["keep"] - first - (n - last)
                pick = torch.sort(middle, descending=True, stable=True).indices[:some].sort().values
                x = torch.cat([x[:first], middle[pick], x[last:]])
            new_scores[b, h, :x.shape[0]] = x
    return None, None, new_scores, None
