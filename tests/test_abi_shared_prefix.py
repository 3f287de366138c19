"""The shared-prefix attention and the draft acceptance on the host: plans, argument checks, the binding's
refusals (no GPU needed)."""

import ctypes

import pytest
import torch

from rope_gqa_paged_gb300 import _build

RRA_OK, RRA_EINVAL, RRA_EUNSUPPORTED, RRA_ERANGE, RRA_EWORKSPACE = 0, -1, -2, -3, -4
P = 4096                                       # a pointer that is never dereferenced: checks fail first
host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="host-only argument checks; never given fake pointers on a GPU")


@pytest.fixture(scope="module")
def rra():
    _build.build()
    from rope_gqa_paged_gb300 import rra as binding
    return binding


def _caller(fn, names, values):
    def call(**kw):
        args = list(values)
        for k, v in kw.items():
            args[names.index(k)] = v
        return fn(*args)
    return call


PLAN = "B gamma Hq Hkv D prefix cols bs splits chunks".split()


def _plan(rra, **kw):
    """(status, own splits, prefix chunks, workspace bytes)"""
    own, chunks, ws = ctypes.c_int(-7), ctypes.c_int(-7), ctypes.c_size_t(7)
    values = dict(zip(PLAN, (4, 1, 32, 8, 128, 512, 64, 16, 0, 0)))
    values.update(kw)
    st = rra.lib().rra_shared_prefix_plan(*[values[k] for k in PLAN], ctypes.byref(own), ctypes.byref(chunks),
                                          ctypes.byref(ws))
    return st, own.value, chunks.value, ws.value


def test_plan(rra):
    st, own, chunks, ws = _plan(rra, splits=2, chunks=3)
    assert (st, own, chunks) == (RRA_OK, 2, 3)
    rows, slots = 4 * 32, 5
    assert ws >= rows * slots * (128 + 2) * 4                       # an output row, a maximum and a sum per slot
    # one slot needs no workspace; no prefix, no chunks of it
    assert _plan(rra, prefix=0, splits=1) == (RRA_OK, 1, 0, 0)
    assert _plan(rra, prefix=0, splits=3)[1:3] == (3, 0)
    # more chunks than the prefix has key tiles, more splits than there are stages of own tokens
    st, own, chunks, _ = _plan(rra, splits=1000, chunks=1000)
    assert st == RRA_OK and chunks == 512 // 64 and own == (64 * 16 - 512) // 32
    # a split spans at most 128 blocks
    assert _plan(rra, prefix=0, cols=4096, bs=8, splits=1)[1] >= 4096 // 128
    # nothing left for own tokens, an empty batch
    assert _plan(rra, prefix=64 * 16)[0] == RRA_OK
    assert _plan(rra, B=0)[0] == RRA_OK and _plan(rra, B=0)[3] == 0
    # results may be left out
    assert rra.lib().rra_shared_prefix_plan(4, 1, 32, 8, 128, 512, 64, 16, 0, 0, None, None, None) == RRA_OK


BAD_PLANS = [
    (dict(bs=0), RRA_EINVAL), (dict(bs=-16), RRA_EINVAL), (dict(bs=24), RRA_EUNSUPPORTED), (dict(bs=4, cols=256), RRA_EUNSUPPORTED),
    (dict(gamma=0), RRA_EINVAL), (dict(gamma=17), RRA_EUNSUPPORTED), (dict(D=96), RRA_EUNSUPPORTED),
    (dict(Hq=6, Hkv=4), RRA_EINVAL), (dict(B=-1), RRA_EINVAL), (dict(B=70000), RRA_ERANGE),
    (dict(prefix=-16), RRA_EINVAL), (dict(prefix=520), RRA_EUNSUPPORTED), (dict(prefix=65 * 16), RRA_EINVAL),
    (dict(cols=0), RRA_EINVAL), (dict(splits=-1), RRA_EINVAL), (dict(chunks=-1), RRA_EINVAL),
    (dict(cols=(1 << 26) + 1), RRA_ERANGE), (dict(cols=2 ** 31 - 1, bs=1 << 30, prefix=0), RRA_ERANGE),
    (dict(B=65535, gamma=16, Hq=4096, Hkv=4096), RRA_ERANGE),
    (dict(prefix=0, cols=1 << 26, splits=1 << 28), RRA_ERANGE),
]


@pytest.mark.parametrize("kw,status", BAD_PLANS)
def test_plan_refuses(rra, kw, status):
    assert _plan(rra, **kw)[0] == status


@host_only
def test_attention_refuses_before_any_launch(rra):
    names = ("q k v prefix prefix_len table cols lens bs blocks out B gamma Hq Hkv D scale splits chunks ws ws_bytes "
             "err stream").split()
    call = _caller(rra.lib().rra_shared_prefix_attn, names,
                   [P, P, P, P, 512, P, 64, P, 16, 300, P, 4, 1, 32, 8, 128, 0.0, 1, 2, P, 1 << 30, None, None])
    assert call(B=0) == RRA_OK                                                  # empty batch: no-op
    for name in ("q", "k", "v", "table", "lens", "out", "prefix"):
        assert call(**{name: None}) == RRA_EINVAL, name
    for name in ("q", "k", "v", "out"):
        assert call(**{name: P + 8}) == RRA_EINVAL, name                       # misaligned
    assert call(blocks=0) == RRA_EINVAL
    assert call(blocks=2 ** 31 - 1) == RRA_ERANGE
    assert call(scale=float("nan")) == RRA_EINVAL and call(scale=float("inf")) == RRA_EINVAL
    assert call(ws=None) == RRA_EWORKSPACE and call(ws_bytes=1000) == RRA_EWORKSPACE
    assert call(ws=P + 4) == RRA_EWORKSPACE
    assert call(prefix_len=500) == RRA_EUNSUPPORTED
    assert call(bs=4, cols=256) == RRA_EUNSUPPORTED and call(gamma=17) == RRA_EUNSUPPORTED
    need = _plan(rra, splits=1, chunks=2)[3]
    assert call(ws_bytes=need - 1) == RRA_EWORKSPACE


@host_only
def test_step_refuses_before_any_launch(rra):
    names = ("q k_new v_new positions q_out k v prefix prefix_len table cols bs blocks out B gamma Hq Hkv D base style "
             "scale splits chunks ws ws_bytes err stream").split()
    call = _caller(rra.lib().rra_shared_prefix_step, names,
                   [P, P, P, P, P, P, P, P, 512, P, 64, 16, 300, P, 4, 1, 32, 8, 128, 10000.0, 0, 0.0, 1, 2, P, 1 << 30,
                    None, None])
    assert call(B=0) == RRA_OK
    for name in ("q", "k_new", "v_new", "positions", "q_out", "k", "v", "prefix", "table", "out"):
        assert call(**{name: None}) == RRA_EINVAL, name
    assert call(style=2) == RRA_EINVAL and call(base=0.5) == RRA_EINVAL
    assert call(ws_bytes=0) == RRA_EWORKSPACE
    assert call(prefix_len=500) == RRA_EUNSUPPORTED


@host_only
def test_acceptance_refuses_before_any_launch(rra):
    names = ("p p_sb p_st q q_sb q_st tokens lens u u_last pos tokens_out kept pos_out B gamma V dt err stream").split()
    call = _caller(rra.lib().rra_accept_draft, names,
                   [P, 500, 100, P, 400, 100, P, P, P, P, P, P, P, P, 3, 4, 100, rra.RRA_F32, None, None])
    assert call(B=0) == RRA_OK
    for name in ("p", "tokens", "u", "u_last", "tokens_out", "kept"):
        assert call(**{name: None}) == RRA_EINVAL, name
    assert call(pos=None) == RRA_EINVAL                                         # next positions of none
    assert call(B=-1) == RRA_EINVAL and call(gamma=0) == RRA_EINVAL and call(V=0) == RRA_EINVAL
    assert call(gamma=33) == RRA_EUNSUPPORTED and call(dt=7) == RRA_EUNSUPPORTED
    assert call(B=65536) == RRA_ERANGE and call(V=(1 << 30) + 1) == RRA_ERANGE
    assert call(p=P + 2) == RRA_EINVAL and call(q=P + 1) == RRA_EINVAL
    assert call(p=P + 1, dt=rra.RRA_BF16) == RRA_EINVAL
    for name in ("p_sb", "p_st", "q_sb", "q_st"):
        assert call(**{name: -1}) == RRA_EINVAL, name


BF, I32 = torch.bfloat16, torch.int32


def _attn_args():
    return dict(q=torch.zeros(2, 3, 8, 128, dtype=BF), k=torch.zeros(40, 16, 2, 128, dtype=BF),
                v=torch.zeros(40, 16, 2, 128, dtype=BF), prefix=torch.zeros(4, dtype=I32), prefix_len=64,
                table=torch.zeros(2, 8, dtype=I32), lens=torch.zeros(2, dtype=I32),
                out=torch.zeros(2, 3, 8, 128, dtype=BF))


@pytest.mark.parametrize("name,value,error", [
    ("q", torch.zeros(2, 3, 8, 128), TypeError), ("k", torch.zeros(40, 16, 2, 128), TypeError),
    ("out", torch.zeros(2, 3, 8, 128), TypeError), ("lens", torch.zeros(2, dtype=torch.int64), TypeError),
    ("table", torch.zeros(2, 8, dtype=torch.int64), TypeError), ("q", torch.zeros(8, 128, dtype=BF), ValueError),
    ("v", torch.zeros(40, 16, 1, 128, dtype=BF), ValueError), ("k", torch.zeros(40, 2, 128, dtype=BF), ValueError),
    ("out", torch.zeros(2, 8, 128, dtype=BF), ValueError), ("table", torch.zeros(3, 8, dtype=I32), ValueError),
    ("lens", torch.zeros(3, dtype=I32), ValueError), ("prefix", None, ValueError),
    ("prefix", torch.zeros(3, dtype=I32), ValueError), ("prefix", torch.zeros(4, dtype=torch.int64), ValueError),
    ("scale", 0.0, ValueError)])                                                # (the last: tensors of the CPU)
def test_binding_refuses_attention(rra, name, value, error):
    args = _attn_args()
    args[name] = value
    scale = args.pop("scale", 0.0)
    with pytest.raises(error):
        rra.rra_shared_prefix_attn(*args.values(), scale=scale)


def _draft_args():
    return dict(p=torch.zeros(3, 5, 100), x=torch.zeros(3, 4, dtype=I32), u=torch.zeros(3, 4), ul=torch.zeros(3),
                draft_probs=torch.zeros(3, 4, 100))


@pytest.mark.parametrize("name,value,error", [
    ("p", torch.zeros(3, 4, 100), ValueError), ("p", torch.zeros(3, 5, 100, dtype=torch.float16), TypeError),
    ("draft_probs", torch.zeros(3, 5, 100), ValueError), ("draft_probs", torch.zeros(3, 4, 100, dtype=BF), ValueError),
    ("p", torch.zeros(3, 5, 100), ValueError)])                                 # (the last: tensors of the CPU)
def test_binding_refuses_drafts(rra, name, value, error):
    args = _draft_args()
    args[name] = value
    with pytest.raises(error):
        rra.rra_accept_draft(args["p"], args["x"], args["u"], args["ul"], draft_probs=args["draft_probs"])


@host_only
def test_append_refuses_before_any_launch(rra):
    names = "q k_new v_new positions q_out k v prefix_len table cols bs blocks B gamma Hq Hkv D base style err stream".split()
    call = _caller(rra.lib().rra_shared_prefix_append, names,
                   [P, P, P, P, P, P, P, 512, P, 64, 16, 300, 4, 1, 32, 8, 128, 10000.0, 0, None, None])
    assert call(B=0) == RRA_OK
    for name in ("q", "k_new", "v_new", "positions", "q_out", "k", "v", "table"):
        assert call(**{name: None}) == RRA_EINVAL, name
    for name in ("q", "k_new", "v_new", "q_out", "k", "v"):
        assert call(**{name: P + 8}) == RRA_EINVAL, name                       # misaligned
    assert call(prefix_len=-16) == RRA_EINVAL and call(prefix_len=65 * 16) == RRA_EINVAL
    assert call(prefix_len=500) == RRA_EUNSUPPORTED and call(bs=4, cols=256) == RRA_EUNSUPPORTED
    assert call(bs=0) == RRA_EINVAL and call(bs=24) == RRA_EUNSUPPORTED
    assert call(gamma=0) == RRA_EINVAL and call(gamma=17) == RRA_EUNSUPPORTED and call(D=96) == RRA_EUNSUPPORTED
    assert call(cols=0, prefix_len=0) == RRA_EINVAL and call(blocks=0) == RRA_EINVAL
    assert call(style=2) == RRA_EINVAL and call(base=0.5) == RRA_EINVAL


@pytest.mark.parametrize("name,value,error", [
    ("q", torch.zeros(2, 3, 8, 128), TypeError), ("k_new", torch.zeros(2, 3, 2, 128), TypeError),
    ("k_new", torch.zeros(2, 3, 1, 128, dtype=BF), ValueError), ("v_new", torch.zeros(2, 3, 4, 128, dtype=BF), ValueError),
    ("q_out", torch.zeros(2, 8, 128, dtype=BF), ValueError), ("positions", torch.zeros(2, dtype=torch.int64), TypeError),
    ("positions", torch.zeros(3, dtype=I32), ValueError), ("q", torch.zeros(2, 3, 8, 128, dtype=BF), ValueError)])
def test_binding_refuses_append(rra, name, value, error):                       # (the last: tensors of the CPU)
    args = dict(q=torch.zeros(2, 3, 8, 128, dtype=BF), k_new=torch.zeros(2, 3, 2, 128, dtype=BF),
                v_new=torch.zeros(2, 3, 2, 128, dtype=BF), positions=torch.zeros(2, dtype=I32),
                q_out=torch.zeros(2, 3, 8, 128, dtype=BF), k=torch.zeros(40, 16, 2, 128, dtype=BF),
                v=torch.zeros(40, 16, 2, 128, dtype=BF), prefix_len=64, table=torch.zeros(2, 8, dtype=I32))
    args[name] = value
    with pytest.raises(error):
        rra.rra_shared_prefix_append(*args.values())


def test_two_call_step_hands_on_the_callers_tensors(rra, monkeypatch):
    """Nothing of the step runs outside the library: the calls get the very tensors and the stream that the caller
    gave, not results of other kernels on whichever stream is torch's current one."""
    from rope_gqa_paged_gb300 import step as step_module
    calls = []
    for name in [n for n in dir(rra) if n.startswith("rra_")]:
        monkeypatch.setattr(rra, name, lambda *a, _name=name, **kw: calls.append((_name, list(a) + list(kw.values()))))
    s = step_module.SharedPrefixStep.__new__(step_module.SharedPrefixStep)
    own = {n: torch.zeros(1) for n in "q_rot k_cache v_cache block_table out workspace err prefix_blocks".split()}
    s.__dict__.update(own, B=2, gamma=3, Hq=8, Hkv=2, D=128, prefix_len=64, num_splits=0, prefix_splits=0,
                      rope_base=10000.0, rope_style=0, scale=0.0)
    given = dict(q=torch.zeros(1), k_new=torch.zeros(1), v_new=torch.zeros(1), positions=torch.zeros(2, dtype=I32),
                 seq_lens=torch.zeros(2, dtype=I32))
    stream = object()
    s(*given.values(), stream=stream)
    known = {id(t) for t in list(own.values()) + list(given.values())}
    assert len(calls) == 2
    for name, args in calls:
        assert any(a is stream for a in args), name
        assert all(id(a) in known for a in args if isinstance(a, torch.Tensor)), name
    assert any(a is given["positions"] for a in calls[0][1]) and any(a is given["seq_lens"] for a in calls[1][1])


def test_tensor_memory_is_allocated_behind_the_wait():
    """A kernel that may start before the one ahead of it ends takes Tensor Memory only when that one is complete: the one
    ahead may still have to allocate its own, and neither would end. (Shown by the order in the source, never by running.)"""
    import glob
    import os
    import re
    found = 0
    for path in glob.glob(os.path.join(_build.CSRC, "*.cu*")):
        text = re.sub(r"//[^\n]*", "", open(path, encoding="utf-8").read())
        for kernel in re.split(r"__global__", text)[1:]:
            if "tc::tmem_alloc(" in kernel:
                found += 1
                assert 0 <= kernel.find("pdl_wait();") < kernel.index("tc::tmem_alloc("), path
    assert found >= 3


WIDE = [dict(B=16, Hkv=8, prefix=2048, own=6144), dict(B=16, Hkv=1, prefix=2048, own=6144),
        dict(B=16, Hkv=32, prefix=2048, own=6144), dict(B=64, Hkv=8, prefix=32768, own=1024),
        dict(B=512, Hkv=8, prefix=16384, own=256, bs=32), dict(B=48, gamma=4, Hkv=8, prefix=8192, own=1500),
        dict(B=21, gamma=3, Hq=42, Hkv=6, D=64, bs=8, prefix=1000, own=700), dict(B=8, Hkv=8, prefix=8192, own=100),
        dict(B=128, gamma=8, Hkv=4, prefix=4096, own=500)]


def _widths(kw):
    """The plan with tables of the sequences' width, with 2, 4 and 16 times the room for own tokens, of 131072 tokens."""
    kw = dict(kw)
    own, bs = kw.pop("own"), kw.get("bs", 16)
    for room in (own, 2 * own, 4 * own, 16 * own, 131072 - kw["prefix"]):
        yield _plan(rra_module(), cols=-(-(kw["prefix"] + room) // bs), **kw)


def rra_module():
    from rope_gqa_paged_gb300 import rra as binding
    return binding


@pytest.mark.parametrize("kw", WIDE)
def test_wide_tables_keep_the_prefix_pass(rra, kw):
    """A table may be wider than any sequence now is: the prefix is still read once, by a pass of at most twice the time (6
    us and 0.8 or 1.45 us for each of a chunk's key tiles of 64 or 128)."""
    rows = kw["B"] * kw.get("gamma", 1) * (kw.get("Hq", 32) // kw["Hkv"])
    tiles = -(-kw["prefix"] // (128 if rows > 128 or kw.get("D") == 64 else 64))

    def pass_us(chunks):
        return 6 + -(-tiles // chunks) * (1.45 if rows > 128 else 0.8)

    (st, _, chunks, _), *wide = _widths(kw)
    assert st == RRA_OK and chunks >= 1
    for st, _, n, _ in wide:
        assert st == RRA_OK and n >= 1 and pass_us(n) <= 2 * pass_us(chunks) and n <= 2 * chunks


@pytest.mark.parametrize("kw", WIDE)
def test_wide_tables_keep_units_and_workspace_in_bounds(rra, kw):
    """Room for 32 units per SM, for 8 of a sequence at least, however wide the table; the workspace with it."""
    n_rep = kw.get("Hq", 32) // kw["Hkv"]
    slices = -(-n_rep // (16 // kw.get("gamma", 1)))
    units, rows = kw["B"] * kw["Hkv"] * slices, kw["B"] * kw.get("gamma", 1) * kw.get("Hq", 32)
    for st, own, chunks, ws in _widths(kw):
        assert st == RRA_OK and 1 <= own <= max(8, 32 * 152 // units)
        assert ws <= rows * (own + chunks) * (kw.get("D", 128) + 2) * 4 + 256


@host_only
def test_acceptance_refuses_outputs_over_other_arrays(rra):
    """Every CTA of a sequence's cluster reads its inputs, one writes its outputs."""
    names = ("p p_sb p_st q q_sb q_st tokens lens u u_last pos tokens_out kept pos_out B gamma V dt err stream").split()
    apart = dict(tokens=1 << 16, lens=2 << 16, u=3 << 16, u_last=4 << 16, pos=5 << 16, tokens_out=6 << 16, kept=7 << 16,
                 pos_out=8 << 16)
    call = _caller(rra.lib().rra_accept_draft, names,
                   [P, 500, 100, P, 400, 100] + list(apart.values()) + [3, 4, 100, rra.RRA_F32, None, None])
    bytes_of = dict(tokens=48, lens=12, u=48, u_last=12, pos=12, tokens_out=60, kept=12, pos_out=12)
    for out in ("tokens_out", "kept", "pos_out"):
        for name, at in apart.items():
            if name == out:
                continue
            for shift in (0, bytes_of[name] - 4, 4 - bytes_of[out]):
                if {name, out} == {"pos", "pos_out"} and shift == 0:
                    continue
                assert call(**{out: at + shift}) == RRA_EINVAL, (out, name, shift)


def test_acceptance_checks_overlaps_last(rra):
    """Arrays side by side, and next positions in place, pass the check (shown on a call that fails at the launch or runs an
    empty batch: nothing is dereferenced on the host)."""
    if torch.cuda.is_available():
        pytest.skip("host-only argument checks; never given fake pointers on a GPU")
    names = ("p p_sb p_st q q_sb q_st tokens lens u u_last pos tokens_out kept pos_out B gamma V dt err stream").split()
    side = [65536, 65536 + 48, 65536 + 60, 65536 + 108, 65536 + 120, 65536 + 132, 65536 + 192, 65536 + 204]
    call = _caller(rra.lib().rra_accept_draft, names,
                   [P, 500, 100, P, 400, 100] + side + [3, 4, 100, rra.RRA_F32, None, None])
    ecuda = -5
    assert call() == ecuda and call(pos_out=side[4]) == ecuda
