"""The calls on trees of drafted tokens on the host: plans, argument checks, the binding's refusals (no GPU needed)."""

import ctypes

import pytest
import torch

from rope_gqa_paged_gb300 import _build

RRA_OK, RRA_EINVAL, RRA_EUNSUPPORTED, RRA_ERANGE, RRA_EWORKSPACE = 0, -1, -2, -3, -4
host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="host-only argument checks; never given fake pointers on a GPU")


@pytest.fixture(scope="module")
def rra():
    _build.build()
    from rope_gqa_paged_gb300 import rra as binding
    return binding


PLAN = dict(B=4, N=16, Hq=32, Hkv=8, D=128, max_tokens=4096, block_size=16, num_splits=0)


def _plan(rra, **kw):
    splits, ws = ctypes.c_int(-7), ctypes.c_size_t(7)
    st = rra.lib().rra_tree_plan(*{**PLAN, **kw}.values(), ctypes.byref(splits), ctypes.byref(ws))
    return st, splits.value, ws.value


def test_plan(rra):
    st, splits, ws = _plan(rra, num_splits=5)
    assert (st, splits) == (RRA_OK, 5)
    rows, slots = 16 * 4, 5 * 2
    assert ws >= rows * slots * (128 + 2) * 4              # a row of output, a maximum and a sum per row and slot
    assert _plan(rra, num_splits=1) == (RRA_OK, 1, 0)      # one run: no partials
    assert _plan(rra, B=0)[0] == RRA_OK
    assert _plan(rra, N=1, B=1, Hq=1, Hkv=1, max_tokens=1, block_size=0) == (RRA_OK, 1, 0)
    # no more runs than the cache has key tiles, and a bounded workspace however long and many the sequences are
    assert _plan(rra, B=1, Hkv=1, Hq=1, max_tokens=256, num_splits=1000)[1] <= 4
    for kw in (dict(max_tokens=1 << 20), dict(B=4096), dict(N=128, Hq=128), dict(D=64)):
        st, splits, ws = _plan(rra, **kw)
        assert st == RRA_OK and 1 < splits <= 1024 and ws < 100 << 20, kw


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), RRA_EINVAL), (dict(N=129), RRA_EUNSUPPORTED), (dict(Hq=30), RRA_EINVAL), (dict(D=96), RRA_EUNSUPPORTED),
    (dict(block_size=4), RRA_EUNSUPPORTED), (dict(block_size=24), RRA_EUNSUPPORTED), (dict(block_size=-1), RRA_EINVAL),
    (dict(max_tokens=0), RRA_EINVAL), (dict(max_tokens=(1 << 30) + 1), RRA_ERANGE), (dict(num_splits=-1), RRA_EINVAL),
    (dict(B=65536), RRA_ERANGE), (dict(B=-1), RRA_EINVAL), (dict(Hq=8 * 65536, Hkv=1), RRA_ERANGE),
])
def test_plan_refusals(rra, kw, status):
    assert _plan(rra, **kw)[0] == status


# pointers that are never dereferenced (checks fail first), far enough apart not to overlap
AT = {n: (i + 1) << 30 for i, n in enumerate("q k_new v_new positions parents lens q_out k v table out ws".split())}
SIZES = dict(mbps=64, bs=16, nblk=1000, max_len=0)
SHAPE = dict(B=4, N=16, Hq=32, Hkv=8, D=128)


def _step(rra, **kw):
    a = {**AT, **SIZES, **SHAPE, "base": 1e4, "style": 0, "scale": 0.0, "splits": 1, "ws_bytes": 0, **kw}
    order = ("q k_new v_new positions parents lens q_out k v table mbps bs nblk max_len out B N Hq Hkv D base style scale "
             "splits ws ws_bytes").split()
    return rra.lib().rra_tree_step(*[a[k] for k in order], None, None)


def _append(rra, **kw):
    a = {**AT, **SIZES, **SHAPE, "base": 1e4, "style": 0, **kw}
    order = "q k_new v_new positions parents lens q_out k v table mbps bs nblk max_len B N Hq Hkv D base style".split()
    return rra.lib().rra_tree_append(*[a[k] for k in order], None, None)


def _attn(rra, **kw):
    a = {**AT, **SIZES, **SHAPE, "scale": 0.0, "splits": 1, "ws_bytes": 0, **kw}
    order = "q_out k v table mbps positions parents lens bs nblk max_len out B N Hq Hkv D scale splits ws ws_bytes".split()
    return rra.lib().rra_tree_attn(*[a[k] for k in order], None, None)


BOTH = [  # refused by all three
    (dict(N=0), RRA_EINVAL), (dict(N=200), RRA_EUNSUPPORTED), (dict(Hq=30), RRA_EINVAL), (dict(D=80), RRA_EUNSUPPORTED),
    (dict(bs=0), RRA_EINVAL), (dict(bs=4), RRA_EUNSUPPORTED), (dict(bs=12), RRA_EUNSUPPORTED), (dict(mbps=0), RRA_EINVAL),
    (dict(nblk=0), RRA_EINVAL), (dict(nblk=2 ** 31 - 1), RRA_ERANGE), (dict(mbps=2 ** 30), RRA_ERANGE),
    (dict(table=None, max_len=0), RRA_EINVAL), (dict(positions=None), RRA_EINVAL), (dict(parents=None), RRA_EINVAL),
    (dict(k=None), RRA_EINVAL), (dict(v=AT["v"] + 8), RRA_EINVAL), (dict(q_out=None), RRA_EINVAL),
]


@host_only
@pytest.mark.parametrize("kw,status", BOTH)
def test_refusals(rra, kw, status):
    assert _step(rra, **kw) == _append(rra, **kw) == _attn(rra, **kw) == status


@host_only
def test_refusals_of_one_call(rra):
    rows, kv = 4 * 16 * 32 * 128 * 2, 4 * 16 * 8 * 128 * 2
    for call in (_step, _append):
        for kw in (dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")), dict(style=2), dict(q=None),
                   dict(k_new=AT["k_new"] + 2), dict(v_new=None), dict(q_out=AT["q"] + rows - 16),
                   dict(q_out=AT["k_new"] + kv - 16), dict(q_out=AT["v_new"])):
            assert call(rra, **kw) == RRA_EINVAL, kw
    for call in (_step, _attn):
        for kw in (dict(scale=float("nan")), dict(out=None), dict(out=AT["q_out"] + 16), dict(splits=-1)):
            assert call(rra, **kw) == RRA_EINVAL, kw
        for kw in (dict(ws=None, ws_bytes=1 << 30), dict(ws_bytes=100), dict(ws=AT["ws"] + 8, ws_bytes=1 << 30)):
            assert call(rra, splits=0, **kw) == RRA_EWORKSPACE, kw
    for kw in (dict(q_out=AT["q"]), dict(out=AT["q"]), dict(out=AT["k_new"]), dict(out=AT["v_new"] - rows + 16)):
        assert _step(rra, **kw) == RRA_EINVAL, kw
    assert _step(rra, B=0) == _append(rra, B=0) == _attn(rra, B=0) == RRA_OK


def test_binding_refusals(rra):
    """Types and shapes are checked before any pointer is taken."""
    B, N, Hq, Hkv, D = 2, 3, 4, 2, 64
    bf = torch.bfloat16
    q = torch.zeros(B, N, Hq, D, dtype=bf)
    new = torch.zeros(B, N, Hkv, D, dtype=bf)
    k = torch.zeros(5, 16, Hkv, D, dtype=bf)
    pos, par = torch.zeros(B, dtype=torch.int32), torch.zeros(B, N, dtype=torch.int32)
    table = torch.zeros(B, 2, dtype=torch.int32)

    def step(**kw):
        a = dict(q=q, k_new=new, v_new=new, positions=pos, parents=par, q_out=q, k_cache=k, v_cache=k, out=q,
                 block_table=table, tree_lens=None)
        a.update(kw)
        rra.rra_tree_step(**a)

    for kw in (dict(q=q.float()), dict(k_cache=k.float()), dict(v_cache=k.half()), dict(out=q.float()), dict(k_new=new.float())):
        with pytest.raises(TypeError):
            step(**kw)
    for kw in (dict(q=q[0]), dict(out=q[:, :2]), dict(v_cache=k[:4]), dict(k_cache=k[..., :32], v_cache=k[..., :32]),
               dict(positions=pos.long()), dict(positions=pos[:1]), dict(parents=par[:, :2]), dict(parents=par.long()),
               dict(tree_lens=pos[:1]), dict(block_table=table.long()), dict(block_table=table[:1]), dict(block_table=None),
               dict(v_new=new[:, :2]), dict(k_new=new[..., :1, :]), dict(q_out=q[:1])):
        with pytest.raises(ValueError):
            step(**kw)
    with pytest.raises(ValueError):  # (a CPU tensor)
        step()


KEEP_AT = {n: (i + 1) << 30 for i, n in
           enumerate("tokens parents choices lens positions table tokens_out kept nodes_out next".split())}


def _keep(rra, layers=2, caches=None, **kw):
    a = {**KEEP_AT, **SIZES, "stride": 1, "B": 4, "N": 16, "Hkv": 8, "D": 128, "dt": 1, **kw}
    arrays = [(ctypes.c_void_p * max(layers, 1))(*(caches or [1 << 40] * layers)) for _ in range(2)]
    return rra.lib().rra_tree_keep(a["tokens"], a["parents"], a["choices"], a["stride"], a["lens"], a["positions"], arrays[0],
                                   arrays[1], layers, a["table"], a["mbps"], a["bs"], a["nblk"], a["max_len"],
                                   a["tokens_out"], a["kept"], a["nodes_out"], a["next"], a["B"], a["N"], a["Hkv"], a["D"],
                                   a["dt"], None, None)


@host_only
def test_keep_refusals(rra):
    n = 4 * 16 * 4
    for kw, st in ((dict(N=0), RRA_EINVAL), (dict(N=129), RRA_EUNSUPPORTED), (dict(D=32), RRA_EUNSUPPORTED),
                   (dict(dt=2), RRA_EUNSUPPORTED), (dict(layers=129), RRA_EUNSUPPORTED), (dict(layers=-1), RRA_EINVAL),
                   (dict(bs=24), RRA_EUNSUPPORTED), (dict(bs=0), RRA_EINVAL), (dict(nblk=0), RRA_EINVAL), (dict(B=-1), RRA_EINVAL),
                   (dict(B=65536), RRA_ERANGE), (dict(table=None, max_len=0), RRA_EINVAL), (dict(mbps=1 << 30), RRA_ERANGE),
                   (dict(stride=-1), RRA_EINVAL), (dict(tokens=None), RRA_EINVAL), (dict(choices=None), RRA_EINVAL),
                   (dict(positions=None), RRA_EINVAL), (dict(kept=None), RRA_EINVAL), (dict(nodes_out=None), RRA_EINVAL),
                   (dict(caches=[1 << 40, None]), RRA_EINVAL), (dict(caches=[1 << 40, (1 << 40) + 8]), RRA_EINVAL),
                   (dict(next=KEEP_AT["positions"]), RRA_EINVAL), (dict(tokens_out=KEEP_AT["tokens"]), RRA_EINVAL),
                   (dict(tokens_out=KEEP_AT["choices"] + 5 * n, stride=7), RRA_EINVAL),
                   (dict(nodes_out=KEEP_AT["tokens_out"] + n - 4), RRA_EINVAL), (dict(kept=KEEP_AT["lens"]), RRA_EINVAL)):
        assert _keep(rra, **kw) == st, kw
    assert _keep(rra, B=0) == RRA_OK


LP_AT = {n: (i + 1) << 40 for i, n in enumerate("logits tokens logprobs entropy top_lp top".split())}


def _logprobs(rra, **kw):
    a = {**LP_AT, "sb": 16000, "st": 1000, "T": 2, "k": 5, "B": 4, "N": 16, "V": 1000, "dt": 1, **kw}
    return rra.lib().rra_token_logprobs(*[a[k] for k in "logits sb st tokens T logprobs entropy k top_lp top B N V dt".split()],
                                        None, None)


@host_only
def test_logprobs_refusals(rra):
    rows = 4 * 16 * 4
    for kw, st in ((dict(dt=3), RRA_EUNSUPPORTED), (dict(T=33), RRA_EUNSUPPORTED), (dict(k=33), RRA_EUNSUPPORTED),
                   (dict(k=4, V=3), RRA_EINVAL), (dict(k=-1), RRA_EINVAL), (dict(T=-1), RRA_EINVAL), (dict(V=0), RRA_EINVAL),
                   (dict(V=(1 << 30) + 1), RRA_ERANGE), (dict(B=-1), RRA_EINVAL), (dict(N=0), RRA_EINVAL),
                   (dict(B=1 << 20, N=1 << 12), RRA_ERANGE), (dict(logits=None), RRA_EINVAL), (dict(tokens=None), RRA_EINVAL),
                   (dict(logprobs=None), RRA_EINVAL), (dict(top=None), RRA_EINVAL), (dict(top_lp=None), RRA_EINVAL),
                   (dict(logits=LP_AT["logits"] + 1), RRA_EINVAL), (dict(logits=LP_AT["logits"] + 2, dt=0), RRA_EINVAL),
                   (dict(sb=-1), RRA_EINVAL), (dict(st=-5), RRA_EINVAL), (dict(entropy=LP_AT["tokens"] + 4), RRA_EINVAL),
                   (dict(top=LP_AT["top_lp"] + 5 * rows - 4), RRA_EINVAL), (dict(logprobs=LP_AT["entropy"]), RRA_EINVAL),
                   (dict(entropy=LP_AT["logits"] + 2 * (3 * 16000 + 16 * 1000) - 4), RRA_EINVAL)):
        assert _logprobs(rra, **kw) == st, kw
    assert _logprobs(rra, B=0) == RRA_OK


def test_binding_refusals_of_the_others(rra):
    x, tok = torch.zeros(4, 100), torch.zeros(4, 2, dtype=torch.int32)
    for kw in (dict(logits=x), dict(logits=x[0]), dict(logits=x[None, None]), dict(logits=x.half())):
        with pytest.raises((ValueError, TypeError)):
            rra.rra_token_logprobs(**{"tokens": tok, **kw})
    ids, pos, k = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1, 8, 64)
    for kw in (dict(k_caches=[]), dict(v_caches=[k, k]), dict(k_caches=[k[:1]]), dict(choices=ids.long()),
               dict(v_caches=[k.bfloat16()]), dict(block_table=ids.long()), dict(k_caches=k[None, None]),
               dict(k_caches=k[None].expand(2, *k.shape), v_caches=[k, k]), dict(k_caches=k[None], v_caches=k[None, :1]), dict()):
        a = dict(draft_tokens=ids, parents=ids, choices=ids, positions=pos, k_caches=[k], v_caches=[k])
        a.update(kw)
        with pytest.raises(ValueError):
            rra.rra_tree_keep(**a)
