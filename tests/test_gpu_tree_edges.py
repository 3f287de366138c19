"""The step on a tree of drafted tokens at random shapes and cuts, at far addresses, in two streams at once, and against
the numpy oracle. (Cases, tolerances: test_gpu_tree.py.)"""

import random

import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_tree import DEV, NAN, Case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    import rope_gqa_paged_gb300 as mod
    from rope_gqa_paged_gb300 import _build
    _build.build()
    return mod


@pytest.mark.parametrize("seed", range(40))
def test_random_shapes_and_cuts(R, seed):
    """The line of key tiles cut at every sort of place: inside units, at their ends, several in one run."""
    r = random.Random(seed)
    B, N, Hkv, n_rep = r.randint(1, 9), r.choice([1, 2, 5, 17, 40, 70, 128]), r.choice([1, 2, 3, 5]), r.choice([1, 2, 3, 8])
    top = r.choice([3, 130, 700, 2500])
    cached = [r.randint(0, top) for _ in range(B)]
    lens = [r.choice([0, 1, N, r.randint(1, N)]) for _ in range(B)] if r.random() < 0.6 else None
    c = Case(cached, N, Hkv * n_rep, Hkv, r.choice([64, 128]), r.choice([0, 8, 16, 64, 256]), lens,
             kind=r.choice(["random", "chain", "star", "forest"]), seed=seed)
    want, mag = c.expect()
    for splits in (0, r.randint(1, 400)):
        out, err = c.attend(R, splits)
        check(c, out, want, mag, f"seed {seed}, {splits} runs")
        assert int(err) == 0
    out, q_rot, k, v, err = c.step(R, r.choice([0, 7]))
    check(c, out, *c.expect(torch.where(torch.isnan(q_rot), 0, q_rot), k, v), f"seed {seed}, step")
    assert err == 0


@pytest.mark.parametrize("kind", ["random", "chain"])
@pytest.mark.parametrize("bs", [0, 16])
def test_against_the_oracle(R, kind, bs):
    c = Case([60, 300], 9, 8, 2, 64, bs, kind=kind, seed=21)
    c.k, c.v = torch.nan_to_num(c.k), torch.nan_to_num(c.v)

    def bits(t):
        return t.view(torch.int16).cpu().numpy().view(np.uint16)

    table = c.table.cpu().numpy() if bs else None
    q_ref, k_ref, v_ref, out_ref = oracle.tree.tree_step(bits(c.q), bits(c.k_new), bits(c.v_new), np.array(c.cached),
                                                         c.parents.cpu().numpy(), bits(c.k), bits(c.v), "bf16", table, bs)
    out, q_rot, k, v, err = c.step(R)
    assert err == 0
    for got, ref in ((q_rot, q_ref), (k, k_ref)):   # (a tie that a float64 angle puts on the other side: one bf16 step)
        ulps = np.abs(bits(got).astype(np.int32) - ref.astype(np.int32))
        assert ulps.max() <= 1
    assert np.array_equal(bits(v), v_ref)
    check(c, out, torch.from_numpy(out_ref).to(DEV), c.expect(q_rot, k, v)[1])


def test_far_contiguous_rows(R):
    """A contiguous cache of more than 2^31 elements: the last sequence's rows lie past them."""
    B, Hkv, D, max_len = 9, 8, 128, 240007
    k = torch.zeros(B, Hkv, max_len, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    g = torch.Generator(device=DEV).manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)

    N, Hq = 12, 16
    k[-1, :, :500], v[-1, :, :500] = randn(Hkv, 500, D), randn(Hkv, 500, D)
    pos = torch.full((B,), 500, dtype=torch.int32, device=DEV)
    lens = torch.tensor([0] * (B - 1) + [N], dtype=torch.int32, device=DEV)
    parents = (torch.arange(N, device=DEV) - 1).clamp(min=-1).int().expand(B, N).contiguous()
    q, kn, vn = randn(B, N, Hq, D), randn(B, N, Hkv, D), randn(B, N, Hkv, D)
    step = R.TreeStep(B, N, Hq, Hkv, D, k, v)
    out = step(q, kn, vn, pos, parents, lens)
    small = R.TreeStep(1, N, Hq, Hkv, D, k[-1:, :, :600].contiguous(), v[-1:, :, :600].contiguous())
    want = small(q[-1:].contiguous(), kn[-1:].contiguous(), vn[-1:].contiguous(), pos[:1], parents[:1])
    assert step.error_bits() == small.error_bits() == 0
    assert float((out[-1].float() - want[0].float()).abs().max()) <= 2.0 ** -7  # (the same rows, cut elsewhere: values of size 1)
    assert not out[:-1].any()
    assert torch.equal(k[-1, :, 500:512], small.k_cache[0, :, 500:512])


def test_two_streams_at_once(R):
    """Calls of both kinds of CTA (one and two row tiles) in two streams, with workspaces of their own."""
    a = Case([1500, 700, 3000], 20, 32, 8, 128, 16, seed=1)
    b = Case([900, 2100], 64, 32, 8, 128, 32, seed=2)
    wants = [c.expect() for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [c.workspace(R) for c in (a, b)]
    outs = [torch.full_like(c.q, NAN) for c in (a, b)]
    errs = [torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s, ws, out, err in zip((a, b), streams, spaces, outs, errs):
            c.attend(R, 0, ws, out, err, s)
    torch.cuda.synchronize()
    for c, out, err, (want, mag) in zip((a, b), outs, errs, wants):
        check(c, out, want, mag)
        assert int(err) == 0


def test_steps_among_other_kernels(R):
    """Back to back with the decode, prefill and shared-prefix steps on one stream, which also start early and use Tensor
    Memory: every result as alone."""
    c = Case([700, 350], 40, 32, 8, 128, 16, seed=12)
    c.k, c.v = torch.nan_to_num(c.k), torch.nan_to_num(c.v)
    tree = R.TreeStep(2, 40, 32, 8, 128, c.k.clone(), c.v.clone(), c.table)
    g = torch.Generator(device=DEV).manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)

    k1, v1 = randn(2, 1, 2048, 128), randn(2, 1, 2048, 128)
    big = R.DecodeStep(2, 128, 1, 128, k1, v1)                      # 128 heads on one KV head: tcgen05
    big_args = (randn(2, 128, 128), randn(2, 1, 128), randn(2, 1, 128), torch.tensor([1800, 77], dtype=torch.int32, device=DEV))
    k2, v2 = randn(1, 8, 512, 128), randn(1, 8, 512, 128)
    pre = R.PrefillStep(1, 300, 32, 8, 128, k2, v2)
    pre_args = (randn(1, 300, 32, 128), randn(1, 300, 8, 128), randn(1, 300, 8, 128), torch.zeros(1, dtype=torch.int32, device=DEV))
    args = (c.q, c.k_new, c.v_new, c.positions, c.parents)
    alone = []
    for step, a in ((tree, args), (big, big_args), (pre, pre_args)):
        alone.append(step(*a).clone())
        torch.cuda.synchronize()
    logits = torch.randn(2, 40, 5000, generator=g, device=DEV)
    lp = R.rra_token_logprobs(logits, None, 3)
    for _ in range(5):
        for step in (tree, big, pre, tree):
            step.out.fill_(NAN)
        for _ in range(3):
            tree(*args)
            big(*big_args)
            tree(*args)
            got = R.rra_token_logprobs(logits, None, 3)
            tree(*args)
            pre(*pre_args)
    torch.cuda.synchronize()
    for step, want in zip((tree, big, pre), alone):
        assert torch.equal(step.out, want) and step.error_bits() == 0
    for x, y in zip(got[1:], lp[1:]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("N", [20, 50])
def test_tensors_at_odd_multiples_of_16_bytes(R, N):
    c = Case([300, 77], N, 8, 2, 128, 16, seed=7)

    def moved(x):
        y = torch.empty(x.numel() + 8, dtype=x.dtype, device=DEV)[8:].reshape(x.shape)
        y.copy_(x)
        assert y.data_ptr() % 32 == 16
        return y

    c.q, c.k, c.v, c.k_new, c.v_new = (moved(x) for x in (c.q, c.k, c.v, c.k_new, c.v_new))
    out = moved(torch.full_like(c.q, NAN))
    check(c, c.attend(R, out=out)[0], *c.expect())
    q_rot = moved(torch.zeros_like(c.q))
    R.rra_tree_step(c.q, c.k_new, c.v_new, c.positions, c.parents, q_rot, c.k, c.v, out, c.table, workspace=c.workspace(R))
    check(c, out, *c.expect(q_rot))
