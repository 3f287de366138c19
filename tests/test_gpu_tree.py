"""Attention of trees of drafted tokens (rra_tree_append / rra_tree_attn / rra_tree_step) against the definition in
float64, one sequence after the other over its own tokens.

Tolerance, per output element: the weights enter the second product as bf16 (half a step: 2^-8 of
each weight, so 2^-8 sum_t w_t |v_t|), the output is stored in bf16 (2^-8 |out|), and the float32
scores (128 products of N(0,1) values: below 2^-13 of a weight), exponentials and sums add less than
2^-10 sum_t w_t |v_t|. Sequences of fewer than 256 cached tokens have their weights in two bf16 parts: without the
first of the three.
"""


import pytest
import torch

from oracle.rope import apply_rope
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAN = float("nan")


@pytest.fixture(scope="module")
def R():
    import rope_gqa_paged_gb300 as mod
    from rope_gqa_paged_gb300 import _build
    _build.build()
    return mod


def random_parents(B, N, g, kind="random"):
    at = torch.arange(N)
    if kind == "chain":
        return (at - 1).expand(B, N).int().contiguous()
    if kind == "star":
        return torch.where(at > 0, 0, -1).expand(B, N).int().contiguous()
    if kind == "forest":  # several nodes that follow the cached text itself
        p = (torch.rand(B, N, generator=g) * (at + 1)).long() - 1
        return p.int()
    return torch.where(at > 0, (torch.rand(B, N, generator=g).square() * at).long(), -1).int()


class Case:
    """Random caches with a tree behind each sequence's tokens. What no call may read is poisoned: unused blocks and
    the slots past each sequence's nodes hold NaN, table entries past them are out of range."""

    def __init__(self, cached, N, Hq, Hkv, D, bs, lens=None, kind="random", cols=None, seed=0, scale=0.0, spare=1):
        g = torch.Generator().manual_seed(seed)
        gd = torch.Generator(device=DEV).manual_seed(seed)
        B = self.B = len(cached)
        self.cached, self.N, self.Hq, self.Hkv, self.D, self.bs = list(cached), N, Hq, Hkv, D, bs
        self.n = list(lens) if lens is not None else [N] * B
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV) if lens is not None else None
        self.positions = torch.tensor(cached, dtype=torch.int32, device=DEV)
        self.parents = random_parents(B, N, g, kind).to(DEV)
        self.scale_arg, self.scale = scale, scale or D ** -0.5
        ends = [p + n for p, n in zip(cached, self.n)]

        def randn(*shape):
            return torch.randn(*shape, generator=gd, device=DEV, dtype=torch.bfloat16)

        if bs:
            need = [-(-e // bs) for e in ends]
            self.cols = cols or max(max(need), 1)
            perm = torch.randperm(sum(need) + 3, generator=g).int()
            table = torch.full((B, self.cols), -7, dtype=torch.int32)
            used = torch.zeros(sum(need) + 3, bs, dtype=torch.bool)
            at = 0
            for b, n in enumerate(need):
                table[b, :n] = perm[at:at + n]
                at += n
                for c in range(n):
                    used[int(table[b, c]), :min(bs, ends[b] - c * bs)] = True
            self.table = table.to(DEV)
            self.k, self.v = randn(len(used), bs, Hkv, D), randn(len(used), bs, Hkv, D)
            self.k[~used.to(DEV)] = NAN
            self.v[~used.to(DEV)] = NAN
            self.max_tokens = self.cols * bs
        else:
            self.table = None
            self.max_tokens = cols or max(max(ends) + spare, 1)
            self.k, self.v = randn(B, Hkv, self.max_tokens, D), randn(B, Hkv, self.max_tokens, D)
            for b, e in enumerate(ends):
                self.k[b, :, e:] = NAN
                self.v[b, :, e:] = NAN
        self.q, self.k_new, self.v_new = randn(B, N, Hq, D), randn(B, N, Hkv, D), randn(B, N, Hkv, D)

    def above(self, b):
        """Of every node: itself and its ancestors."""
        got = []
        for j, p in enumerate(self.parents[b].tolist()[:self.n[b]]):
            got.append((got[p] if p >= 0 else []) + [j])
        return got

    def rows(self, cache, b, count):
        if self.table is None:
            return cache[b, :, :count].transpose(0, 1)
        return cache[self.table[b, :-(-count // self.bs)].long()].reshape(-1, self.Hkv, self.D)[:count]

    def expect(self, q=None, k=None, v=None):
        """(out, sum of w |v|) in float64 over caches that hold the nodes."""
        q, k, v = (x if x is not None else y for x, y in ((q, self.q), (k, self.k), (v, self.v)))
        out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
        mag = torch.zeros_like(out)
        for b, p in enumerate(self.cached):
            n = self.n[b]
            if n == 0:
                continue
            K, V = self.rows(k, b, p + n).double(), self.rows(v, b, p + n).double()
            hidden = torch.ones(n, p + n, dtype=torch.bool)
            hidden[:, :p] = False
            for j, nodes in enumerate(self.above(b)):
                hidden[j, [p + x for x in nodes]] = False
            qb = q[b, :n].double().reshape(n, self.Hkv, self.Hq // self.Hkv, self.D)
            w = torch.einsum("jhrd,thd->jhrt", qb, K) * self.scale
            w = torch.softmax(w.masked_fill(hidden[:, None, None].to(DEV), -torch.inf), -1)
            out[b, :n] = torch.einsum("jhrt,thd->jhrd", w, V).reshape(n, self.Hq, self.D)
            mag[b, :n] = torch.einsum("jhrt,thd->jhrd", w, V.abs()).reshape(n, self.Hq, self.D)
        return out, mag

    def plan(self, R, num_splits=0):
        return R.rra_tree_plan(self.B, self.N, self.Hq, self.Hkv, self.D, self.max_tokens, self.bs, num_splits)

    def workspace(self, R, num_splits=0):
        need = self.plan(R, num_splits)[1]
        return torch.full((need,), 0xff, dtype=torch.uint8, device=DEV) if need else None  # (NaNs: it needs no filling)

    def attend(self, R, num_splits=0, ws=None, out=None, err=None, stream=None):
        ws = self.workspace(R, num_splits) if ws is None else ws
        err = torch.zeros(1, dtype=torch.int32, device=DEV) if err is None else err
        out = torch.full_like(self.q, NAN) if out is None else out
        R.rra_tree_attn(self.q, self.k, self.v, self.positions, self.parents, out, self.table, self.lens, self.scale_arg,
                        num_splits, ws, err, stream)
        return out, err

    def step(self, R, num_splits=0, rope_base=10000.0, rope_style=0):
        """(out, q_rot, k cache, v cache, error bits) of the fused step on copies of the caches."""
        k, v = self.k.clone(), self.v.clone()
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, q_rot = torch.full_like(self.q, NAN), torch.full_like(self.q, NAN)
        R.rra_tree_step(self.q, self.k_new, self.v_new, self.positions, self.parents, q_rot, k, v, out, self.table,
                        self.lens, rope_base, rope_style, self.scale_arg, num_splits, self.workspace(R, num_splits), err)
        return out, q_rot, k, v, int(err)


def check(case, out, want, mag, what=""):
    got = out.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    p = 2.0 ** -10 + 2.0 ** -8 * (case.positions >= 256).double()[:, None, None, None]
    tol = p * mag + 2.0 ** -8 * want.abs() + 1e-30
    bad = (got - want).abs() > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float(((got - want).abs() / tol).max()):.2f} of the tolerance at {bad.nonzero()[0].tolist()}")


SHAPES = [
    # cached tokens, N, Hq, Hkv, D, block (0: contiguous), nodes
    ([0], 1, 8, 2, 128, 16, None),
    ([5], 1, 1, 1, 64, 8, None),
    ([63, 64, 65, 127, 128, 129], 8, 8, 2, 128, 16, None),
    ([0, 1, 40, 255, 256, 300], 26, 32, 8, 128, 16, None),
    ([700, 3, 1500, 0], 13, 42, 6, 64, 8, [13, 1, 7, 0]),
    ([900, 411], 64, 32, 8, 128, 32, [64, 33]),          # 256 rows per KV head: two row tiles
    ([512], 33, 32, 8, 128, 128, None),                  # 132 rows: the second tile nearly empty
    ([300, 1000, 20], 128, 8, 2, 64, 64, [128, 100, 5]),  # most nodes, 512 rows
    ([77], 128, 16, 1, 128, 256, None),                  # 2048 rows, a block larger than a key tile
    ([100, 2000, 30, 700], 24, 16, 16, 128, 0, [24, 3, 0, 24]),
    ([10], 3, 4, 4, 64, 0, None),                        # a cache shorter than a key tile
    ([130, 3], 70, 8, 2, 128, 0, [70, 64]),
    ([5000], 5, 5, 1, 128, 16, None),
    ([16, 16, 16], 16, 32, 8, 128, 16, [0, 0, 0]),       # nothing but padding rows
]


@pytest.mark.parametrize("shape", SHAPES, ids=[f"{i}" for i in range(len(SHAPES))])
@pytest.mark.parametrize("splits", [0, 1, 3, 50])
def test_attention(R, shape, splits):
    cached, N, Hq, Hkv, D, bs, lens = shape
    c = Case(cached, N, Hq, Hkv, D, bs, lens, seed=len(cached) + N)
    out, err = c.attend(R, splits)
    want, mag = c.expect()
    check(c, out, want, mag)
    assert int(err) == 0


@pytest.mark.parametrize("kind", ["chain", "star", "forest"])
@pytest.mark.parametrize("N,D,bs", [(9, 128, 16), (64, 64, 32), (128, 128, 0)])
def test_tree_shapes(R, kind, N, D, bs):
    c = Case([0, 30, 411], N, 8, 2, D, bs, kind=kind, seed=N)
    out, err = c.attend(R)
    check(c, out, *c.expect(), kind)
    assert int(err) == 0


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("shape", [SHAPES[i] for i in (0, 3, 4, 5, 9, 11)], ids=str)
def test_step(R, shape, style):
    cached, N, Hq, Hkv, D, bs, lens = shape
    c = Case(cached, N, Hq, Hkv, D, bs, lens, seed=3)
    out, q_rot, k, v, err = c.step(R, rope_style=style)
    assert err == 0
    # expected caches and queries: node j rotated for p + depth in slot p + j; nothing else changes
    k_want, v_want = c.k.clone(), c.v.clone()
    for b, p in enumerate(c.cached):
        n = c.n[b]
        assert torch.isnan(q_rot[b, n:]).all()
        if n == 0:
            continue
        pos = [p + len(a) - 1 for a in c.above(b)]
        for x, got in ((c.q, q_rot[b, :n]), (c.k_new, c.rows(k, b, p + n)[p:])):
            ref = torch.from_numpy(apply_rope(x[b, :n].double().cpu().numpy(), torch.tensor(pos)[:, None].numpy(), 10000.0,
                                              style)).to(DEV)
            # half a bf16 step, and 2^-20 for values that a float64 angle puts on the other side of a tie
            assert ((got.double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -20) + 1e-30).all()
        for cache, new in ((k_want, c.rows(k, b, p + n)[p:]), (v_want, c.v_new[b, :n])):
            if c.table is None:
                cache[b, :, p:p + n] = new.transpose(0, 1)
            else:
                t = torch.arange(p, p + n, device=DEV)
                cache[c.table[b, t // c.bs].long(), t % c.bs] = new
    assert torch.equal(k.view(torch.int16), k_want.view(torch.int16))
    assert torch.equal(v.view(torch.int16), v_want.view(torch.int16))
    live = torch.where(torch.isnan(q_rot), 0, q_rot)
    check(c, out, *c.expect(live, k, v), "step")


def test_step_equals_two_calls(R):
    c = Case([700, 3, 1500, 40], 30, 32, 8, 128, 16, [30, 0, 11, 30], seed=8)
    out, q_rot, k, v, _ = c.step(R)
    k2, v2, q2, out2 = c.k.clone(), c.v.clone(), torch.full_like(c.q, NAN), torch.full_like(c.q, NAN)
    R.rra_tree_append(c.q, c.k_new, c.v_new, c.positions, c.parents, q2, k2, v2, c.table, c.lens)
    R.rra_tree_attn(q2, k2, v2, c.positions, c.parents, out2, c.table, c.lens, workspace=c.workspace(R))
    for a, b in ((q_rot, q2), (k, k2), (v, v2), (out, out2)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("bs", [0, 16])
def test_chain_is_the_verify_step(R, bs):
    """A chain's queries and caches are the verify step's bits, its outputs the same within both tolerances."""
    N = 6
    c = Case([100, 900], N, 32, 8, 128, bs, kind="chain", seed=5)
    out, q_rot, k, v, _ = c.step(R)
    k2, v2, q2, out2 = c.k.clone(), c.v.clone(), torch.empty_like(c.q), torch.empty_like(c.q)
    step = R.VerifyStep(2, N, 32, 8, 128, k2, v2, c.table)
    out2 = step(c.q, c.k_new, c.v_new, c.positions)
    for a, b in ((q_rot, step.q_rot), (k, k2), (v, v2)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    want, mag = c.expect(q_rot, k, v)
    check(c, out, want, mag, "tree")
    check(c, out2, want, mag, "verify")


def test_queries_in_place_and_scale(R):
    c = Case([300], 7, 8, 2, 128, 16, seed=6, scale=0.21)
    check(c, c.attend(R)[0], *c.expect(), "scale")
    k, v, q = c.k.clone(), c.v.clone(), c.q.clone()
    R.rra_tree_append(q, c.k_new, c.v_new, c.positions, c.parents, q, k, v, c.table)
    assert torch.equal(q, c.step(R)[1])


def test_device_errors(R):
    """Positions, lengths, parents and block ids out of range: flagged, and the other sequences untouched by it."""
    good = Case([40, 300, 77, 512], 12, 8, 2, 128, 16, seed=9)
    want, mag = good.expect()
    for what, bit in (("position", R.RRA_ERR_POSITION), ("negative", R.RRA_ERR_POSITION), ("huge", R.RRA_ERR_POSITION),
                      ("len", R.RRA_ERR_SEQ_LEN), ("parent", R.RRA_ERR_TREE), ("self", R.RRA_ERR_TREE),
                      ("block", R.RRA_ERR_BLOCK_ID)):
        c = Case([40, 300, 77, 512], 12, 8, 2, 128, 16, seed=9)
        if what == "position":
            c.positions[1] = c.max_tokens - 11
        elif what == "negative":
            c.positions[1] = -1
        elif what == "huge":
            c.positions[1] = 2 ** 31 - 1
        elif what == "len":
            c.lens = torch.tensor([12, 99, 12, 12], dtype=torch.int32, device=DEV)  # counts as 12
        elif what == "parent":
            c.parents[1, 3] = 7
        elif what == "self":
            c.parents[1, 3] = 3
        else:
            c.table[1, 2] = 10 ** 6
        for fused in (False, True):
            if fused:
                out, q_rot, k, v, err = c.step(R)
                w, m = good.expect(good.step(R)[1], *good.step(R)[2:4])
            else:
                out, e = c.attend(R)
                err, w, m = int(e), want, mag
            assert err == bit, (what, fused, err)
            keep = [0, 2, 3] + ([1] if what == "len" else [])
            check(_only(c, keep), out[keep], w[keep], m[keep], what)
            if bit == R.RRA_ERR_POSITION:
                assert torch.isnan(out[1]).all()
                if fused:
                    assert torch.isnan(q_rot[1]).all()
            elif bit != R.RRA_ERR_BLOCK_ID:  # (block 0 in its place may hold anything)
                assert torch.isfinite(out[1]).all()


def _only(c, keep):
    class Part:
        positions = torch.tensor([c.cached[b] for b in keep], device=DEV)
    return Part


def test_non_finite_keys_out_of_sight(R):
    """A node that a row does not attend may have any key."""
    c = Case([130], 6, 8, 2, 128, 16, kind="star", seed=2)
    at = 130 + 5
    c.k[c.table[0, at // 16].long(), at % 16] = NAN
    out, _ = c.attend(R)
    want, mag = c.expect(k=torch.nan_to_num(c.k))
    check(c, out[:, :5], want[:, :5], mag[:, :5])


def test_results_do_not_depend_on_the_batch_order_or_time(R):
    """The same call twice gives the same bits; so does a replayed graph, with a workspace that two graphs share."""
    c = Case([700, 3, 1500, 40, 90], 30, 32, 8, 128, 16, [30, 0, 11, 30, 29], seed=8)
    step = R.TreeStep(c.B, c.N, 32, 8, 128, c.k, c.v, c.table)
    first = step(c.q, c.k_new, c.v_new, c.positions, c.parents, c.lens).clone()
    assert torch.equal(first, step(c.q, c.k_new, c.v_new, c.positions, c.parents, c.lens))
    d = Case([11, 900, 20, 5, 300], 30, 32, 8, 128, 16, seed=4)
    other = R.TreeStep(c.B, c.N, 32, 8, 128, d.k, d.v, d.table)
    other.workspace = step.workspace if step.workspace.numel() >= other.workspace.numel() else other.workspace
    want = other(d.q, d.k_new, d.v_new, d.positions, d.parents).clone()
    ga = step.capture(c.q, c.k_new, c.v_new, c.positions, c.parents, c.lens)
    gb = other.capture(d.q, d.k_new, d.v_new, d.positions, d.parents, repeat=2)
    for _ in range(3):
        step.out.fill_(NAN)
        other.out.fill_(NAN)
        ga.replay()
        gb.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, first) and torch.equal(other.out, want)
    assert step.error_bits() == other.error_bits() == 0


def test_another_stream(R):
    c = Case([700, 350], 20, 32, 8, 128, 16, seed=12)
    want, mag = c.expect()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, err = c.attend(R, stream=s)
    s.synchronize()
    check(c, out, want, mag)


def test_many_sequences(R):
    """More sequences than a CTA has threads, ragged, most of them short; more units than runs of keys."""
    g = torch.Generator().manual_seed(0)
    B = 700
    cached = [int(x) for x in torch.randint(0, 90, (B,), generator=g)]
    lens = [int(x) for x in torch.randint(0, 6, (B,), generator=g)]
    c = Case(cached, 5, 4, 2, 64, 16, lens, seed=1)
    out, err = c.attend(R)
    check(c, out, *c.expect())
    assert int(err) == 0


def test_far_blocks(R):
    """Block ids whose rows lie past 2^31 elements of the pool."""
    bs, Hkv, D = 16, 8, 128
    n = 2 ** 31 // (bs * Hkv * D) + 50
    c = Case([200], 9, 16, Hkv, D, bs, seed=1)
    k = torch.zeros(n, bs, Hkv, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    ids = torch.arange(n - c.cols, n, dtype=torch.int32, device=DEV)
    k[ids.long()], v[ids.long()] = c.k[c.table[0].long()], c.v[c.table[0].long()]
    c.k, c.v, c.table = k, v, ids[None].contiguous()
    out, err = c.attend(R)
    check(c, out, *c.expect())
    out, q_rot, k2, v2, e = c.step(R)
    check(c, out, *c.expect(q_rot, k2, v2))
    assert int(err) == e == 0
