"""Which halves of a tile the latent decode kernel hands to the tensor core with a proxy fence.

The products read shared memory through the async proxy, so what ordinary stores put there has
to be fenced by the writing warps before they arrive.  A missing fence shows in no output as
long as the stores happen to land in time, so the condition in the source is evaluated here for
every head tile: Q, on a sequence's first tile, and the column blocks that S^T reads from
shared memory, on every tile."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _source():
    with open(os.path.join(ROOT, "nvfp4_quantised_paged_gb300", "csrc", "latent_decode.cu")) as f:
        return f.read()


def _fenced(src, heads, half, fresh):
    """Whether the last column block of the half, 2 i + par, is followed by a fence before its arrival."""
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
