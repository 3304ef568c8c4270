"""Where ordinary stores to shared memory meet the async proxy: the source's fences.

The tensor core's products and the bulk copies access shared memory through the async proxy, so
what ordinary stores put there has to be fenced by the storing threads before the other side
goes on.  A missing fence shows in no output as long as the stores happen to land in time, so
the source is read here; so is what is waited for before a CTA's memory is freed."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _source(name="latent_decode.cu"):
    with open(os.path.join(ROOT, "nvfp4_quantised_paged_gb300", "csrc", name)) as f:
        return f.read()


# ------------------------------------------------------------------ latent decode: what S^T reads

def _fenced(src, heads, half, fresh):
    """Whether the warps fence after the half's last column block, before they report it; and how many
    column blocks S^T reads from shared memory."""
    body = src[src.index("// ---- expand block"):]
    body = body[:body.index("mbar_arrive(&kv_full[i >> 1])")]
    conds = re.findall(r"if \(((?:[^()]|\([^()]*\))*)\) asm volatile\(\"fence\.proxy\.async\.shared::cta;\"", body)
    assert len(conds) == 1, conds
    smem_cbs = re.search(r"kSmemCbs = N == 64 \? (\d+) : (\d+);", src)
    cond = conds[0].replace("L::kSmemCbs", smem_cbs.group(1 if heads == 64 else 2))
    cond = cond.replace("||", " or ").replace("&&", " and ")
    return bool(eval(cond, {"i": 2 * half + 1, "fresh": fresh})), int(smem_cbs.group(1 if heads == 64 else 2))


@pytest.mark.parametrize("heads", [16, 32, 64])
def test_query_is_fenced_on_a_sequences_first_tile(heads):
    assert _fenced(_source(), heads, 0, True)[0]


@pytest.mark.parametrize("heads", [16, 32, 64])
@pytest.mark.parametrize("fresh", [False, True])
def test_blocks_that_the_scores_read_from_shared_memory_are_fenced(heads, fresh):
    for half in (0, 1):
        fenced, smem_cbs = _fenced(_source(), heads, half, fresh)
        if 4 * half < smem_cbs:          # the half's column blocks 4 half .. 4 half + 3
            assert fenced


# ------------------------------------------------------------------ scores: a missing page's zeros

def test_zeros_in_place_of_a_page_are_fenced_before_the_next_copy():
    """The ring's place of a page out of range is filled by stores, and by a bulk copy a few units later."""
    src = _source("attention_weights.cu")
    body = src[src.index("auto request = "):]
    body = body[body.index("flag_error(a.err, kErrPage)"):body.index("bulk_g2s(")]
    assert body.index("= make_uint4(0, 0, 0, 0)") < body.index("fence.proxy.async.shared::cta") < body.index("__syncwarp()")


def test_scores_wait_for_every_copy_in_flight_when_they_give_up():
    """After a wait that ran out, the units requested and not yet used, as many as the ring has stages,
    are waited for before the CTA ends: the loop's header is run here."""
    src = _source("attention_weights.cu")
    stages = int(re.search(r"kStagesW = (\d+);", src).group(1))
    body = src[src.index("if (!ok) {   // no copy"):]
    init, cond, step = re.search(r"for \((.*?);(.*?);(.*?)\) \{", body).groups()
    names = {"it.left": "left", "nx.left": "nx", "kStagesW": str(stages), "&&": "and"}
    for a, b in names.items():
        cond = cond.replace(a, b)
    for outstanding in range(1, stages + 1):
        left, waited = 10, 0
        while eval(cond, {"left": left, "nx": 10 - outstanding, "i": waited}):
            left, waited = left - 1, waited + 1
        assert waited == outstanding


# ------------------------------------------------------------------ latent extend: copies in flight

def test_extend_waits_for_its_copies_whichever_warp_gives_up():
    """The load warp may have requested everything when another warp's wait runs out: its last wait
    stands on no condition."""
    src = _source("latent_extend.cu")
    body = src[src.index("// ---------------- load warp"):src.index("// ---------------- softmax of")]
    for bar in ("k_full", "v_full"):
        before = body[:body.index("mbar_wait_bounded(&%s[t & 1]" % bar)]
        assert before.count("{") - before.count("}") == 1      # inside the loop over the blocks alone
