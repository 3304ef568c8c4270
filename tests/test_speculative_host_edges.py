"""CPU checks of refusals of the speculative decoding calls (a refused call launches nothing, so plain numbers stand
in for device pointers; every call here is refused)."""

import pytest

from test_speculative_host import EINVAL, EUNSUPPORTED, accept, append, desc, m, tree  # noqa: F401  (m: the fixture)


@pytest.mark.parametrize("kw", [
    dict(num=8192), dict(num=8188), dict(num=8196),              # of 2 sequences: 8 bytes
    dict(cu=8192), dict(cu=8184), dict(cu=8196),                 # 12 bytes
    dict(acc=8192), dict(acc=8164), dict(acc=8196),              # 2 lists of 4: 32 bytes
    dict(bt=8192), dict(bt=8180), dict(bt=8196),                 # 2 rows of 2 pages: 16 bytes
    dict(lens=8188), dict(lens=8196),
])
def test_accept_refuses_lengths_over_what_it_reads(m, kw):  # noqa: F811
    """The new lengths are written while other warps read the lists, counts, bounds and tables."""
    assert accept(m, **kw) == EINVAL


def test_tree_attention_refuses_what_its_plan_cannot_count(m):  # noqa: F811
    """A pair's units are its tiles of 128 tokens and two more: 2^31 of them are refused.  (The workspace is too small in
    every call, which is found later: what the plan can count is refused for that.)"""
    def status(batch, heads, tiles):
        return tree(m, cache=desc(m, num_kv_heads=heads), hq=heads, total=batch, most=1, batch=batch, pages=8 * tiles, size=1)

    assert 65535 * 8 * 4096 < 2**31 <= 65535 * 8 * 4097
    assert status(65535, 8, 4094) == EINVAL
    assert status(65535, 8, 4095) == EUNSUPPORTED
    assert 65535 * 32 * 1024 < 2**31 <= 65535 * 32 * 1025
    assert status(65535, 32, 1022) == EINVAL
    assert status(65535, 32, 1023) == EUNSUPPORTED


@pytest.mark.parametrize("out", [4096, 16, 4080, 4112, 8176])
def test_tree_attention_refuses_an_output_over_its_queries(m, out):  # noqa: F811
    """4 queries of 4 heads: 4,096 bytes from address 4,096 on."""
    assert tree(m, out=out) == EINVAL


# 3 tokens of 4 query heads (1,024 bytes) and 2 kv heads (512); q, k, v are one projection's rows of 2,048 bytes from 4,096 on
ROWS = dict(q=4096, qs=1024, k=5120, v=5632, ks=1024, hq=4, t=3)


@pytest.mark.parametrize("kw", [
    dict(qo=6144, qos=1024), dict(qo=2048, qos=1024), dict(qo=4112, qos=1024), dict(qo=4080, qos=1024),     # q, shifted
    dict(qo=5120, qos=1024), dict(qo=5632, qos=1024), dict(qo=5104, qos=1024), dict(qo=6128, qos=1024),     # k, v
    dict(qo=9216, qos=512), dict(qo=4096, qos=512), dict(qo=8192, qos=2048), dict(qo=16, qos=2048),         # other strides
])
def test_rope_append_refuses_an_output_over_what_it_reads(m, kw):  # noqa: F811
    assert append(m, **{**ROWS, **kw}) == EINVAL


def test_rope_append_refuses_a_single_token_over_another(m):  # noqa: F811
    one = dict(q=4096, qs=512, k=8192, v=8704, ks=256, hq=4, t=1)
    for qo in (3088, 5104, 7184, 8688, 9200):
        assert append(m, **{**one, "qo": qo, "qos": 512}) == EINVAL


def test_numbers_beyond_32_bits_are_refused_by_the_binding(m):  # noqa: F811
    assert [m._int32(x, "window") for x in (0, -1, 2**31 - 1, -2**31, 5.0)] == [0, -1, 2**31 - 1, -2**31, 5]
    for x in (2**31, 2**32 + 5, -2**31 - 1, 1 << 70):
        with pytest.raises(ValueError, match="window"):
            m._int32(x, "window")

    class Cache:
        desc = desc(m)

    assert m.tree_workspace_bytes(Cache, 3, 4, 1, 7) == (13 * 16 * 8 + 255) // 256 * 256 + 13 * 16 * 512
    for args in ((2**32 + 3, 4, 1, 7), (3, 2**32 + 4, 1, 7), (3, 4, 2**32 + 1, 7), (3, 4, 1, 2**32 + 7)):
        with pytest.raises(ValueError):
            m.tree_workspace_bytes(Cache, *args)
