"""Shared-prefix attention (rra_shared_prefix_attn / rra_shared_prefix_step) against the definition in
float64, one sequence after the other over its own tokens.

Tolerance, per output element: the weights enter the second product as bf16 (half a step: 2^-8 of
each weight, so 2^-8 sum_t w_t |v_t|), the output is stored in bf16 (2^-8 |out|), and the float32
scores (128 products of N(0,1) values: below 2^-13 of a weight), exponentials and sums add less than
2^-10 sum_t w_t |v_t|.
"""


import pytest
import torch

import oracle
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


class Case:
    """Random pools of a batch behind a common prefix. Everything that no call may read is poisoned:
    unused blocks and the slots past each sequence's end hold NaN, table entries before the prefix's
    end and past the sequence's are out of range."""

    def __init__(self, lens, gamma, Hq, Hkv, D, bs, P, cols=None, seed=0, poison=True, scale=0.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens_list, self.gamma, self.Hq, self.Hkv, self.D, self.bs, self.P = list(lens), gamma, Hq, Hkv, D, bs, P
        self.scale = scale or D ** -0.5
        B = self.B = len(lens)
        cols = self.cols = cols or max(-(-max(list(lens) + [P]) // bs), 1)
        own = cols - P // bs
        n = P // bs + B * own + 3
        perm = torch.randperm(n, generator=g, device=DEV).int()
        self.prefix = perm[:P // bs].contiguous()
        self.table = torch.full((B, cols), -7, dtype=torch.int32, device=DEV)
        own_ids = perm[P // bs:P // bs + B * own].reshape(B, own)
        self.k = torch.randn(n, bs, Hkv, D, generator=g, device=DEV, dtype=torch.bfloat16)
        self.v = torch.randn(n, bs, Hkv, D, generator=g, device=DEV, dtype=torch.bfloat16)
        self.used = torch.zeros(n, bs, dtype=torch.bool, device=DEV)
        self.used[self.prefix.long()] = True
        for b, L in enumerate(lens):
            nb = max(-(-L // bs) - P // bs, 0)
            self.table[b, P // bs:P // bs + nb] = own_ids[b, :nb]
            for c in range(nb):
                self.used[int(own_ids[b, c]), :min(bs, L - P - c * bs)] = True
        if poison:
            self.k[~self.used] = NAN
            self.v[~self.used] = NAN
        self.q = torch.randn(B, gamma, Hq, D, generator=g, device=DEV, dtype=torch.bfloat16)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV).reshape(B)

    def full_table(self, b, L):
        nb = -(-L // self.bs)
        return torch.cat([self.prefix, self.table[b, self.P // self.bs:]])[:nb].long()

    def expect(self, q=None):
        """(out, sum of w |v|) in float64."""
        q = self.q if q is None else q
        out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
        mag = torch.zeros_like(out)
        rep = self.Hq // self.Hkv
        for b, L in enumerate(self.lens_list):
            ids = self.full_table(b, L)
            k = self.k[ids].reshape(-1, self.Hkv, self.D)[:L].double()
            v = self.v[ids].reshape(-1, self.Hkv, self.D)[:L].double()
            for j in range(self.gamma):
                n = L - self.gamma + 1 + j
                if n <= 0:
                    continue
                qj = q[b, j].double().reshape(self.Hkv, rep, self.D)
                w = torch.softmax(torch.einsum("hrd,thd->hrt", qj, k[:n]) * self.scale, -1)
                out[b, j] = torch.einsum("hrt,thd->hrd", w, v[:n]).reshape(self.Hq, self.D)
                mag[b, j] = torch.einsum("hrt,thd->hrd", w, v[:n].abs()).reshape(self.Hq, self.D)
        return out, mag

    def plan(self, R, num_splits=0, prefix_splits=0):
        return R.rra_shared_prefix_plan(self.B, self.gamma, self.Hq, self.Hkv, self.D, self.P, self.cols, self.bs,
                                        num_splits, prefix_splits)

    def run(self, R, num_splits=0, prefix_splits=0, ws=None, err=None, out=None, stream=None, q=None):
        need = self.plan(R, num_splits, prefix_splits)[2]
        if ws is None and need:
            ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV) if err is None else err
        out = torch.full_like(self.q, NAN) if out is None else out
        R.rra_shared_prefix_attn(self.q if q is None else q, self.k, self.v, self.prefix, self.P, self.table, self.lens,
                                 out, self.scale, num_splits, prefix_splits, ws, err, stream)
        return out, err


def check(out, want, mag, what=""):
    got = out.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    tol = (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -8 * want.abs() + 1e-30
    bad = (got - want).abs() > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float(((got - want).abs() / tol).max()):.2f} of the tolerance at {bad.nonzero()[0].tolist()}")


SHAPES = [  # gamma, Hq, Hkv, D, bs, P
    (1, 32, 8, 128, 16, 512), (1, 8, 8, 128, 32, 384), (1, 32, 1, 128, 16, 640), (1, 128, 1, 128, 64, 320),
    (4, 32, 8, 128, 16, 272), (3, 42, 6, 64, 8, 520), (2, 14, 2, 64, 128, 384), (16, 6, 2, 128, 8, 264),
    (5, 20, 4, 64, 16, 1040), (1, 7, 7, 64, 512, 512),
]


@pytest.mark.parametrize("gamma,Hq,Hkv,D,bs,P", SHAPES)
@pytest.mark.parametrize("splits,pre", [(0, 0), (1, 1), (3, 2), (2, 7)])
def test_shapes_and_lengths(R, gamma, Hq, Hkv, D, bs, P, splits, pre):
    """Lengths of zero, inside the prefix, at and around its end, and of several own tiles."""
    lens = [P + 300, 0, P, P + 1, 1, P - 1, gamma, P + 64, P // 2 + 3, P + gamma, P + 131]
    c = Case(lens, gamma, Hq, Hkv, D, bs, P, seed=gamma + D)
    out, err = c.run(R, splits, pre)
    assert int(err) == 0
    check(out, *c.expect(), what=f"plan {c.plan(R, splits, pre)}")
    if pre:
        assert c.plan(R, splits, pre)[1] >= 1


@pytest.mark.parametrize("pre", [0, 1, 3])
@pytest.mark.parametrize("B", [1, 2, 31, 33, 130])
def test_row_tiles(R, B, pre):
    """Rows that fill no, one or several 128-row tiles, the last one partly (4 heads a group)."""
    c = Case([300 + (37 * b) % 90 for b in range(B)], 1, 16, 4, 128, 16, 256, seed=B)
    out, err = c.run(R, 0, pre)
    assert int(err) == 0
    check(out, *c.expect())


@pytest.mark.parametrize("pre", [0, 2])
def test_without_prefix_and_without_own_tokens(R, pre):
    c = Case([5, 0, 200, 77], 2, 8, 2, 128, 16, 0, seed=3)
    out, err = c.run(R, 0, pre)
    check(out, *c.expect())
    c = Case([512, 512, 0, 100], 1, 8, 2, 128, 16, 512, cols=32, seed=4)   # capacity = prefix
    out, err = c.run(R, 0, pre)
    assert int(err) == 0
    check(out, *c.expect())


@pytest.mark.parametrize("P,pre", [(264, 1), (328, 2), (1000, 3), (2048, 0), (5000, 40)])
def test_prefix_ends_inside_a_tile(R, P, pre):
    c = Case([P + 9, P + 70, 0], 1, 32, 4, 128, 8, P, seed=P)
    check(c.run(R, 0, pre)[0], *c.expect())
    c = Case([P + 9, P + 70, 0], 1, 12, 4, 64, 8, P, seed=P)
    check(c.run(R, 0, pre)[0], *c.expect())


def test_long_prefix_in_small_blocks(R):
    """More than 2000 blocks of 8 tokens in one prefix chunk."""
    c = Case([17000, 16800], 1, 4, 1, 64, 8, 16704, seed=5)
    assert c.plan(R, 0, 1)[1] == 1
    check(c.run(R, 0, 1)[0], *c.expect())


def test_many_partials(R):
    c = Case([4100, 2500, 9], 1, 8, 2, 128, 16, 2048, seed=6)
    own, chunks, _ = c.plan(R, 33, 32)
    assert own + chunks > 60
    check(c.run(R, 33, 32)[0], *c.expect())


def test_large_scores(R):
    """Scores of several hundred: the running maximum moves from tile to tile, and whole tiles weigh nothing."""
    c = Case([900, 700, 513], 2, 16, 4, 128, 16, 512, seed=7)
    c.q *= 60
    c.k[c.prefix[-3:].long()] *= 3
    out, _ = c.run(R, 0, 2)
    want, mag = c.expect()
    # scores up to |s| ~ 4000: a float32 score is off by up to 2^-24 * 128 * 4000 / 2 = 0.015 at the very
    # worst (all partial sums at the largest score), which a weight shows as that share
    tol = (2.0 ** -8 + 2.0 ** -6) * mag + 2.0 ** -8 * want.abs()
    assert ((out.double() - want).abs() <= tol).all()


def test_same_as_the_decode_call(R):
    """The paged decode over the same tokens (each sequence's own reading of the prefix) agrees within both
    calls' tolerances."""
    c = Case([900, 700, 640, 0], 1, 32, 8, 128, 16, 640, seed=8)
    out, _ = c.run(R, 0, 2)
    table = torch.cat([c.prefix.expand(4, -1), c.table[:, 40:]], 1).contiguous()
    step = R.DecodeStep(4, 32, 8, 128, c.k, c.v, table)
    step.q_rot.copy_(c.q[:, 0])
    ref = step.attend(c.lens).double()
    _, mag = c.expect()
    assert ((out[:, 0].double() - ref).abs() <= 2 * (2.0 ** -8 + 2.0 ** -10) * mag[:, 0] + 2.0 ** -7 * ref.abs() + 1e-30).all()


def test_nothing_else_is_written(R):
    """Rows behind the batch, the pools and the workspace's counters stay as they were."""
    c = Case([600, 540, 0], 3, 8, 2, 128, 16, 512, seed=9)
    k0, v0 = c.k.clone(), c.v.clone()
    room = torch.full((c.q.numel() + 4096,), 123.0, dtype=torch.bfloat16, device=DEV)
    out = room[:c.q.numel()].view(c.q.shape)
    need = c.plan(R, 2, 3)[2]
    ws = torch.zeros(need + 256, dtype=torch.uint8, device=DEV)
    ws[need:] = 77
    c.run(R, 2, 3, ws=ws, out=out)
    check(out, *c.expect())
    assert (room[c.q.numel():] == 123.0).all() and (ws[need:] == 77).all()
    assert torch.equal(c.k.view(torch.int16), k0.view(torch.int16)) and torch.equal(c.v.view(torch.int16), v0.view(torch.int16))
    first = out.clone()
    c.run(R, 2, 3, ws=ws, out=out)                          # the counters are back at zero
    assert torch.equal(first.view(torch.int16), out.view(torch.int16))


def test_device_errors_are_flagged(R):
    c = Case([600, 540], 1, 8, 2, 128, 16, 512, seed=10, poison=False)
    c.lens[1] = c.cols * 16 + 5
    c.table[1, 32:] = c.table[0, 32:]
    _, err = c.run(R, 0, 2)
    assert int(err) & R.RRA_ERR_SEQ_LEN
    c.lens[1] = -3
    out, err = c.run(R, 0, 2)
    assert int(err) & R.RRA_ERR_SEQ_LEN and (out[1] == 0).all()
    for bad in (-1, c.k.shape[0]):
        c = Case([600, 540], 1, 8, 2, 128, 16, 512, seed=10, poison=False)
        c.prefix[5] = bad
        _, err = c.run(R, 0, 2)
        assert int(err) == R.RRA_ERR_BLOCK_ID
        c = Case([600, 540], 1, 8, 2, 128, 16, 512, seed=10, poison=False)
        c.table[0, 34] = bad
        _, err = c.run(R, 0, 2)
        assert int(err) == R.RRA_ERR_BLOCK_ID


def test_streams_and_graphs(R):
    """Captured on another stream than the inputs', two graphs with one workspace, replayed in turn with
    refilled inputs."""
    a = Case([600, 0, 777], 2, 8, 2, 128, 16, 512, seed=11)
    b = Case([900, 530], 1, 16, 2, 64, 32, 512, seed=12)
    ws = torch.zeros(max(a.plan(R)[2], b.plan(R)[2]), dtype=torch.uint8, device=DEV)
    oa, ob = torch.empty_like(a.q), torch.empty_like(b.q)
    side = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    for c, o in ((a, oa), (b, ob)):
        with torch.cuda.stream(side):
            c.run(R, ws=ws, out=o)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        with torch.cuda.graph(g, stream=side):
            R.rra_shared_prefix_attn(c.q, c.k, c.v, c.prefix, c.P, c.table, c.lens, o, workspace=ws, err_flag=err)
        graphs.append(g)
    for seed in (1, 2):
        for c, o, g in ((a, oa, graphs[0]), (b, ob, graphs[1])):
            c.q.copy_(torch.randn(c.q.shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV))
            o.fill_(NAN)
            g.replay()
            check(o, *c.expect(), what=f"seed {seed}")


def _step_case(seed, gamma, Hq, Hkv, D, bs, P, lens):
    c = Case(lens, gamma, Hq, Hkv, D, bs, P, seed=seed)
    g = torch.Generator(device=DEV).manual_seed(seed + 100)
    k_new = torch.randn(c.B, gamma, Hkv, D, generator=g, device=DEV, dtype=torch.bfloat16)
    v_new = torch.randn(c.B, gamma, Hkv, D, generator=g, device=DEV, dtype=torch.bfloat16)
    return c, k_new, v_new, (c.lens - gamma).int()


@pytest.mark.parametrize("gamma,Hq,Hkv,D,bs,P", [(1, 32, 8, 128, 16, 512), (4, 8, 2, 128, 8, 264), (3, 14, 2, 64, 32, 320)])
@pytest.mark.parametrize("style", [0, 1])
def test_step(R, gamma, Hq, Hkv, D, bs, P, style):
    """The step against the oracle's rotation and append and the float64 attention over the cache it leaves."""
    lens = [P + gamma, P + 100 + gamma, P + 64, P + 17 + gamma]
    c, k_new, v_new, pos = _step_case(20 + style, gamma, Hq, Hkv, D, bs, P, lens)
    k0, v0 = H.to_numpy(c.k), H.to_numpy(c.v)
    table = torch.cat([c.prefix.expand(c.B, -1), c.table[:, P // bs:]], 1)
    q_ref, k_ref, v_ref, _ = oracle.verify.verify_step(H.to_numpy(c.q), H.to_numpy(k_new), H.to_numpy(v_new),
                                                       pos.cpu().numpy(), k0, v0, "bf16", table.cpu().numpy(), bs,
                                                       rope_style=style)
    step = R.SharedPrefixStep(c.B, gamma, Hq, Hkv, D, c.k, c.v, c.prefix, P, c.table, rope_style=style, prefix_splits=2)
    out = step(c.q, k_new, v_new, pos).clone()
    assert step.error_bits() == 0
    H.assert_close_stored(H.to_numpy(step.q_rot), q_ref, "bf16", "q_rot")
    used = c.used.cpu().numpy()
    H.assert_close_stored(H.to_numpy(c.k)[used], k_ref[used], "bf16", "K cache")
    assert H.to_numpy(c.v)[used].tobytes() == v_ref[used].tobytes()
    check(out, *c.expect(step.q_rot), what="step")
    two = step(c.q, k_new, v_new, pos, c.lens)               # append, then attention over given lengths
    assert torch.equal(out.view(torch.int16), two.view(torch.int16))


def test_step_refuses_positions_in_the_prefix(R):
    """A token whose slot lies in the shared blocks is not written, and its sequence's output is left alone."""
    c, k_new, v_new, pos = _step_case(30, 2, 8, 2, 128, 16, 512, [600, 514, 700])
    pos[1] = 100
    table = torch.cat([c.prefix.expand(c.B, -1), c.table[:, 32:]], 1).contiguous()
    k0 = c.k.clone()
    step = R.SharedPrefixStep(3, 2, 8, 2, 128, c.k, c.v, c.prefix, 512, table, prefix_splits=2)
    step.out.fill_(5.0)
    out = step(c.q, k_new, v_new, pos)
    assert step.error_bits() == R.RRA_ERR_POSITION
    assert torch.equal(c.k[c.prefix.long()].view(torch.int16), k0[c.prefix.long()].view(torch.int16))
    assert (out[1] == 5.0).all()
    want, mag = c.expect(step.q_rot)
    check(out[[0, 2]], want[[0, 2]], mag[[0, 2]])


def test_steps_in_a_row(R):
    """Steps launched back to back, each appending what the next one attends, in a graph and eagerly: every
    output matches the attention over the final cache cut to its length."""
    P, n, gamma = 512, 24, 1
    c = Case([P + n, P + n + 40, P + n + 7], gamma, 32, 8, 128, 16, P, seed=40, poison=False)
    g = torch.Generator(device=DEV).manual_seed(41)
    qs = torch.randn(n, 3, gamma, 32, 128, generator=g, device=DEV, dtype=torch.bfloat16)
    ks = torch.randn(n, 3, gamma, 8, 128, generator=g, device=DEV, dtype=torch.bfloat16)
    vs = torch.randn(n, 3, gamma, 8, 128, generator=g, device=DEV, dtype=torch.bfloat16)
    final = c.lens.clone()
    pos = torch.stack([final - n + i for i in range(n)]).int()
    step = R.SharedPrefixStep(3, gamma, 32, 8, 128, c.k, c.v, c.prefix, P, c.table, prefix_splits=4)
    outs, rots = torch.empty_like(qs), torch.empty_like(qs)

    def loop():
        for i in range(n):
            outs[i].copy_(step(qs[i], ks[i], vs[i], pos[i]))
            rots[i].copy_(step.q_rot)

    loop()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop()
    for replay in (False, True):
        if replay:
            outs.fill_(NAN)
            graph.replay()
        assert step.error_bits() == 0
        for i in (0, 1, n // 2, n - 1):
            c.lens_list = (pos[i] + gamma).tolist()
            check(outs[i], *c.expect(rots[i]), what=f"step {i}")


def test_refusals(R):
    c = Case([600, 540], 1, 8, 2, 128, 16, 512, seed=50)
    out = torch.empty_like(c.q)
    call = R.rra_shared_prefix_attn
    with pytest.raises(R.RraError):                          # no workspace
        call(c.q, c.k, c.v, c.prefix, 512, c.table, c.lens, out, prefix_splits=2)
    with pytest.raises(R.RraError):                          # not a whole number of blocks
        call(c.q, c.k, c.v, c.prefix, 500, c.table, c.lens, out)
    with pytest.raises(ValueError):                          # too few prefix blocks
        call(c.q, c.k, c.v, c.prefix[:-1], 512, c.table, c.lens, out)
    with pytest.raises(TypeError):
        call(c.q.float(), c.k, c.v, c.prefix, 512, c.table, c.lens, out)
    with pytest.raises(TypeError):
        call(c.q, c.k, c.v, c.prefix, 512, c.table, c.lens.long(), out)
    with pytest.raises(ValueError):
        call(c.q, c.k, c.v, c.prefix, 512, c.table[:1], c.lens, out)
    with pytest.raises(ValueError):
        call(c.q, c.k.transpose(1, 2), c.v.transpose(1, 2), c.prefix, 512, c.table, c.lens, out)
    with pytest.raises(ValueError):
        call(c.q, c.k, c.v, c.prefix, 512, c.table, c.lens.cpu(), out)


def test_two_call_step_with_padding(R):
    """seq_lens given: a padding row (length 0) is zero, and its new tokens, at positions in the prefix that the
    tables do list, leave the shared blocks as they were."""
    P, gamma = 512, 3
    c, k_new, v_new, pos = _step_case(31, gamma, 8, 2, 128, 16, P, [P + 40, P + 16, P + 300])
    c.table[:, :P // 16] = c.prefix
    step = R.SharedPrefixStep(c.B, gamma, 8, 2, 128, c.k, c.v, c.prefix, P, c.table, prefix_splits=2)
    pos[1] = 0
    lens = c.lens.clone()
    lens[1] = 0
    before = c.k[c.prefix.long()].clone(), c.v[c.prefix.long()].clone()
    out = step(c.q, k_new, v_new, pos, lens)
    assert step.error_bits() == R.RRA_ERR_POSITION
    assert torch.equal(c.k[c.prefix.long()], before[0]) and torch.equal(c.v[c.prefix.long()], before[1])
    assert not out[1].any()
    c.lens_list[1], step.q_rot[1] = 0, 0
    check(out, *c.expect(step.q_rot))


def test_far_blocks(R):
    """Block ids whose bytes lie beyond 2^32, in a pool of 6.4 GB; one block twice in the prefix."""
    n, bs, Hkv, D, P = 49152, 64, 8, 128, 256
    c = Case([P + 100, P + 1, P + 70], 2, 32, Hkv, D, bs, P, seed=32, poison=False)
    small_k, small_v, ids = c.k, c.v, torch.arange(c.k.shape[0], device=DEV)
    c.k = torch.zeros(n, bs, Hkv, D, device=DEV, dtype=torch.bfloat16)
    c.v = torch.zeros(n, bs, Hkv, D, device=DEV, dtype=torch.bfloat16)
    far = n - 1 - ids * 11                     # (block 32768 of 64 x 8 x 128 values starts at byte 2^32)
    assert int(far.min()) > 32768
    c.k[far], c.v[far] = small_k, small_v
    c.prefix = far[c.prefix.long()].int()
    c.prefix[2] = c.prefix[0]
    c.table = torch.where(c.table >= 0, far[c.table.clamp(min=0).long()].int(), c.table)
    for splits, pre in ((1, 1), (3, 2), (0, 0)):
        out, err = c.run(R, splits, pre)
        assert int(err) == 0
        check(out, *c.expect(), what=f"{splits} {pre}")


@pytest.mark.parametrize("gamma,Hq,Hkv,D,bs,P,lens", [
    (16, 13, 1, 64, 1024, 1024, [1040, 1039, 0]),       # thirteen heads a group, one head per unit; one block ahead
    (1, 17, 1, 128, 2048, 4096, [4097, 6144]),          # blocks longer than a chunk
    (7, 22, 2, 128, 8, 8, [8, 15, 16, 40]),             # a prefix of one block of 8
    (1, 8, 8, 64, 16, 800, [800, 800]),                 # nothing but the prefix, as long as the tables
])
def test_odd_groups_and_blocks(R, gamma, Hq, Hkv, D, bs, P, lens):
    c = Case(lens, gamma, Hq, Hkv, D, bs, P, seed=33)
    for splits, pre in ((0, 0), (1, 1), (5, 3)):
        out, err = c.run(R, splits, pre)
        assert int(err) == 0
        check(out, *c.expect(), what=f"{splits} {pre}")


def test_calls_in_turn_on_one_workspace(R):
    """Calls of other shapes one after the other on a stream, without a wait between them, on one workspace that
    no one has filled."""
    cases = [Case([700, 0, 540], 1, 32, 8, 128, 16, 512, seed=34), Case([900] * 40, 4, 16, 2, 128, 32, 640, seed=35),
             Case([300, 260], 2, 14, 2, 64, 8, 256, seed=36)]
    plans = [(3, 2), (2, 5), (4, 0)]
    ws = torch.full((max(c.plan(R, *p)[2] for c, p in zip(cases, plans)),), 0xFF, dtype=torch.uint8, device=DEV)
    outs = [[torch.full_like(c.q, NAN) for _ in range(4)] for c in cases]
    for i in range(4):
        for c, p, o in zip(cases, plans, outs):
            c.run(R, *p, ws=ws, out=o[i])
    for c, o in zip(cases, outs):
        check(o[0], *c.expect())
        assert all(torch.equal(o[0], x) for x in o[1:])


def test_two_streams_at_once(R):
    """Calls that overlap on two streams, each with its own workspace."""
    a, b = Case([700, 540] * 8, 1, 32, 8, 128, 16, 512, seed=41), Case([2000, 1300, 0] * 5, 4, 16, 4, 128, 32, 1024, seed=42)
    plans = [(2, 2), (3, 3)]
    ws = [torch.zeros(c.plan(R, *p)[2], dtype=torch.uint8, device=DEV) for c, p in zip((a, b), plans)]
    outs = [torch.full_like(c.q, NAN) for c in (a, b)]
    streams, err = [torch.cuda.Stream(), torch.cuda.Stream()], torch.zeros(1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    for _ in range(10):
        for c, p, w, o, s in zip((a, b), plans, ws, outs, streams):
            c.run(R, *p, ws=w, err=err, out=o, stream=s)
    torch.cuda.synchronize()
    assert int(err) == 0
    for c, o in zip((a, b), outs):
        check(o, *c.expect())
