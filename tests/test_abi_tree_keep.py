"""What rra_tree_keep refuses of caches and of outputs that lie over what it reads, on the host (no GPU needed)."""

import ctypes

import pytest
import torch

from rope_gqa_paged_gb300 import _build

RRA_EINVAL, RRA_ECUDA = -1, -5
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="host-only argument checks; never given fake pointers on a GPU")


@pytest.fixture(scope="module")
def rra():
    _build.build()
    from rope_gqa_paged_gb300 import rra as binding
    return binding


AT = {n: (i + 1) << 30 for i, n in enumerate("tokens parents choices lens positions table tokens_out kept nodes_out next".split())}
POOL = 1000 * 16 * 8 * 128 * 2   # bytes of a cache of 1000 blocks of 16 tokens, 8 heads of 128, bf16
CONTIG = 4 * 8 * 500 * 128 * 2   # of 4 sequences of 500 tokens
K = 1 << 40


def keep(rra, k, v, **kw):
    a = {**AT, "mbps": 64, "bs": 16, "nblk": 1000, "max_len": 0, "B": 4, "N": 16, "dt": 1, **kw}
    arrays = [(ctypes.c_void_p * len(x))(*x) for x in (k, v)]
    return rra.lib().rra_tree_keep(a["tokens"], a["parents"], a["choices"], 1, a["lens"], a["positions"], *arrays, len(k),
                                   a["table"], a["mbps"], a["bs"], a["nblk"], a["max_len"], a["tokens_out"], a["kept"],
                                   a["nodes_out"], a["next"], a["B"], a["N"], 8, 128, a["dt"], None, None)


@pytest.mark.parametrize("size,layout", [(POOL, {}), (2 * POOL, dict(dt=0)), (CONTIG, dict(table=None, max_len=500))])
def test_caches_that_overlap(rra, size, layout):
    """Caches side by side, or the same one in several places, pass every check (there is no device to launch on);
    any other pair that shares a byte is refused, wherever the two stand."""
    def at(i):
        return K + i * size
    for k, v in (([at(0)], [at(1)]), ([at(3), at(1)], [at(0), at(2)]), ([at(0), at(0)], [at(1), at(1)]), ([at(0)], [at(0)])):
        assert keep(rra, k, v, **layout) == RRA_ECUDA, (k, v)
    for k, v in (([at(0)], [at(1) - 16]), ([at(0), at(5), at(1) - 16], [at(2), at(3), at(4)]), ([at(2), at(0)], [at(4), at(0) + 16]),
                 ([at(2)], [at(1) + 16]), ([at(0), at(0)], [at(0), at(0) + size // 2])):
        assert keep(rra, k, v, **layout) == RRA_EINVAL, (k, v)


def test_caches_of_absurd_sizes(rra):
    """Sizes whose product passes 64 bits count as all memory: two caches do not fit beside each other there."""
    kw = dict(nblk=2 ** 31 - 1, bs=1 << 29, mbps=1, B=65535)
    assert keep(rra, [K], [1 << 50], **kw) == RRA_EINVAL
    assert keep(rra, [K], [K], **kw) == RRA_ECUDA


OUTPUTS = [("tokens_out", 4 * 16 * 4), ("kept", 4 * 4), ("nodes_out", 4 * 16 * 4), ("next", 4 * 4)]


@pytest.mark.parametrize("name,size", OUTPUTS)
def test_outputs_over_the_table_or_a_cache(rra, name, size):
    """The first and the last byte of either count; beside them an output may lie."""
    caches = ([K], [K + POOL])
    for start, length in ((AT["table"], 4 * 64 * 4), (K, 2 * POOL)):
        for at in (start, start + length - 4, start - size + 4):
            assert keep(rra, *caches, **{name: at}) == RRA_EINVAL, at - start
        for at in (start - size, start + length):
            assert keep(rra, *caches, **{name: at}) == RRA_ECUDA, at - start


@pytest.mark.parametrize("name", ["tokens", "parents", "choices", "lens", "positions", "table"])
def test_inputs_over_a_cache(rra, name):
    for cache in (K, K + POOL):
        assert keep(rra, [K], [K + POOL], **{name: cache + POOL - 4}) == RRA_EINVAL
    assert keep(rra, [K], [K + POOL], **{name: K + 2 * POOL}) == RRA_ECUDA
