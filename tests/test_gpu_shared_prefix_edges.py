"""Shared-prefix attention at the edges of its range: rows of a few tokens, streams other than torch's current one, new
tokens at the end of the prefix, positions past any cache, kernels beside it that hold Tensor Memory, tables wider than
their sequences.

Tolerance of rows that attend at most 256 tokens, per output element: the weights enter the second product as two bf16
parts (2^-16 of each weight), the float32 scores (128 products of N(0,1) values: below 2^-13 of a weight), exponentials
and sums add less than 2^-11 sum_t w_t |v_t| with it, and the output is stored in bf16 (2^-8 |out|).
"""

import pytest
import torch

from tests.test_gpu_shared_prefix import Case, check

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAN = float("nan")


@pytest.fixture(scope="module")
def R():
    import rope_gqa_paged_gb300 as mod
    from rope_gqa_paged_gb300 import _build
    _build.build()
    return mod


def check_short(c, out, what=""):
    """Rows of at most 256 tokens within the tolerance above, the others within check()'s."""
    want, mag = c.expect()
    check(out, want, mag, what)
    n = c.lens[:, None] - c.gamma + 1 + torch.arange(c.gamma, device=DEV)
    short = (n <= 256)[..., None, None]
    tol = 2.0 ** -11 * mag + 2.0 ** -8 * want.abs() + 1e-30
    bad = ((out.double() - want).abs() > tol) & short
    assert short.any() and not bad.any(), (f"{what}: {int(bad.sum())} of {int((short & (mag > 0)).sum())} outside, worst "
                                           f"{float((((out.double() - want).abs() / tol) * short).max()):.2f}")


FEW = [2, 3, 1, 0, 4, 6, 9, 13, 33, 40, 64, 65, 100, 129, 200, 255, 256, 257, 300]


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (32, 1, 128), (14, 2, 64)])
@pytest.mark.parametrize("gamma", [1, 4])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_rows_of_few_tokens_without_a_prefix_pass(R, Hq, Hkv, D, gamma, splits):
    c = Case(FEW, gamma, Hq, Hkv, D, 16, 0, seed=60 + gamma)
    out, err = c.run(R, splits, 0)
    assert int(err) == 0
    check_short(c, out)


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (8, 8, 128), (32, 1, 128), (14, 2, 64), (64, 1, 64)])
@pytest.mark.parametrize("gamma", [1, 4])
@pytest.mark.parametrize("P,pre", [(8, 1), (64, 1), (256, 1), (256, 3), (264, 1), (264, 5), (1000, 3)])
def test_rows_of_few_tokens_in_the_prefix_pass(R, Hq, Hkv, D, gamma, P, pre):
    """One and two row tiles per CTA, rows of few tokens in one of them or in both, beside rows of many."""
    few = [n for n in FEW if n < P + 64]
    c = Case(few + [P + 70, 2, P + 400, 3], gamma, Hq, Hkv, D, 8, P, seed=P + gamma)
    out, err = c.run(R, 2, pre)
    assert int(err) == 0 and c.plan(R, 2, pre)[1] >= 1
    check_short(c, out)


def test_rows_do_not_depend_on_their_neighbours(R):
    """A row of many tokens has the same bits beside rows of few (which the prefix pass leaves out) and beside others."""
    lens = [700, 512, 600, 400]
    a = Case(lens, 1, 32, 8, 128, 16, 512, seed=70)
    out = a.run(R, 1, 1)[0]
    a.lens[1], a.lens[3] = 3, 0
    short = a.run(R, 1, 1)[0]
    for b in (0, 2):
        assert torch.equal(out[b].view(torch.int16), short[b].view(torch.int16))
    a.lens_list = a.lens.tolist()
    check_short(a, short)


def _step(R, c, seed, prefix_splits=2):
    g = torch.Generator(device=DEV).manual_seed(seed)
    new = [torch.randn(c.B, c.gamma, c.Hkv, c.D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    step = R.SharedPrefixStep(c.B, c.gamma, c.Hq, c.Hkv, c.D, c.k, c.v, c.prefix, c.P, c.table,
                              prefix_splits=prefix_splits)
    return step, new, (c.lens - c.gamma).int()


def test_two_call_step_on_another_stream(R):
    """The two calls on a stream of the caller's, while torch's current stream is busy: positions that the caller's
    stream produces at the last moment, output and caches as those of the step in one call."""
    lens = [600, 517, 730, 560]
    want, got = (Case(lens, 3, 8, 2, 128, 16, 512, seed=80, poison=False) for _ in range(2))
    one, new, pos = _step(R, want, 81)
    ref = one(want.q, *new, pos).clone()
    two, new2, _ = _step(R, got, 81)
    late, late_lens = torch.full_like(pos, 100), torch.full_like(got.lens, 515)  # (stale values: in the prefix)
    got.table[:, :32] = got.prefix
    before = got.k[got.prefix.long()].clone(), got.v[got.prefix.long()].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)                            # the current stream: busy for some 25 ms
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        late.copy_(pos)
        late_lens.copy_(got.lens)
    out = two(got.q, *new2, late, late_lens, stream=side)
    side.synchronize()
    assert one.error_bits() == two.error_bits() == 0
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    assert torch.equal(two.q_rot, one.q_rot) and torch.equal(got.k, want.k) and torch.equal(got.v, want.v)
    assert torch.equal(got.k[got.prefix.long()], before[0]) and torch.equal(got.v[got.prefix.long()], before[1])
    check(out, *got.expect(two.q_rot))


@pytest.mark.parametrize("two_calls", [False, True])
def test_new_tokens_on_both_sides_of_the_prefix_end(R, two_calls):
    """Of new tokens that start inside the prefix, those inside it are not written and the others are, in both forms."""
    c = Case([600, 512 + 1, 700], 3, 8, 2, 128, 16, 512, seed=82, poison=False)
    c.table[:, :32] = c.prefix
    step, new, pos = _step(R, c, 83)                         # (sequence 1: positions 510, 511 and 512)
    before = c.k[c.prefix.long()].clone(), c.v[c.prefix.long()].clone()
    block = int(c.table[1, 32])
    step(c.q, *new, pos, c.lens if two_calls else None)
    assert step.error_bits() == R.RRA_ERR_POSITION
    assert torch.equal(c.k[c.prefix.long()], before[0]) and torch.equal(c.v[c.prefix.long()], before[1])
    assert torch.equal(c.v[block, 0], new[1][1, 2])


@pytest.mark.parametrize("P,splits,pre", [(512, 2, 2), (512, 0, 0), (0, 1, 0), (0, 3, 0)])
@pytest.mark.parametrize("far", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 31 - 4, -2 ** 31, 2 ** 30])
def test_positions_far_out_of_range_leave_the_output(R, P, splits, pre, far):
    """Positions whose last token's would pass 2^31, with one and with several partials: flagged, the sequence's output
    as it was, the other sequences' right."""
    c = Case([P + 88, P + 60, P + 200], 3, 8, 2, 128, 16, P, seed=90, poison=False)
    g = torch.Generator(device=DEV).manual_seed(91)
    new = [torch.randn(c.B, 3, c.Hkv, c.D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    pos = (c.lens - 3).int()
    pos[1] = far
    step = R.SharedPrefixStep(c.B, 3, c.Hq, c.Hkv, c.D, c.k, c.v, c.prefix, P, c.table, num_splits=splits,
                              prefix_splits=pre)
    assert (step.splits + step.prefix_chunks == 1) == (splits == 1 and P == 0)
    k0, v0 = c.k.clone(), c.v.clone()
    step.out.fill_(5.0)
    step.q_rot.zero_()
    out = step(c.q, *new, pos)
    assert step.error_bits() == R.RRA_ERR_POSITION
    assert (out[1] == 5.0).all()
    own = c.table[1, P // 16:].long()
    assert torch.equal(c.k[own], k0[own]) and torch.equal(c.v[own], v0[own])
    want, mag = c.expect(step.q_rot)
    check(out[[0, 2]], want[[0, 2]], mag[[0, 2]])


def test_between_kernels_that_hold_tensor_memory(R):
    """Calls on one stream without a wait between them, eagerly and in a graph: a decode step of one group of 128 heads and
    a prefill (both hold all of an SM's Tensor Memory), shared-prefix calls of one and of two row tiles. Each gives what
    it gives alone."""
    g = torch.Generator(device=DEV).manual_seed(95)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)

    one, two = (Case([600, 540, 530, 700], 1, 32, 8, 128, 16, 512, seed=96), Case([900] * 40, 4, 16, 2, 128, 32, 640, seed=97))
    table = torch.arange(4 * 64, dtype=torch.int32, device=DEV).reshape(4, 64)
    dec = R.DecodeStep(4, 128, 1, 128, randn(256, 16, 1, 128), randn(256, 16, 1, 128), table)
    pre = R.PrefillStep(2, 200, 16, 2, 128, randn(2, 2, 256, 128), randn(2, 2, 256, 128))
    dec_in = (randn(4, 128, 128), randn(4, 1, 128), randn(4, 1, 128), torch.tensor([900, 1000, 7, 500], dtype=torch.int32, device=DEV))
    pre_in = (randn(2, 200, 16, 128), randn(2, 200, 2, 128), randn(2, 200, 2, 128), torch.zeros(2, dtype=torch.int32, device=DEV))
    ws = [torch.zeros(c.plan(R, 2, 2)[2], dtype=torch.uint8, device=DEV) for c in (one, two)]
    outs, err = [torch.empty_like(c.q) for c in (one, two)], torch.zeros(1, dtype=torch.int32, device=DEV)

    def shared(i):
        return (one, two)[i].run(R, 2, 2, ws=ws[i], err=err, out=outs[i])[0]

    calls = [lambda: dec(*dec_in), lambda: shared(0), lambda: pre(*pre_in), lambda: shared(1), lambda: dec(*dec_in),
             lambda: shared(1), lambda: pre(*pre_in), lambda: shared(0), lambda: shared(1)]
    alone = []
    for call in calls:
        alone.append(call().clone())
        torch.cuda.synchronize()
    got = [torch.empty_like(x) for x in alone]

    def row():
        for call, o in zip(calls, got):
            call()
        for call, o in zip(calls, got):
            o.copy_(call())

    for _ in range(5):
        row()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        row()
    for o in got:
        o.zero_()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, got))
    assert int(err) == dec.error_bits() == pre.error_bits() == 0


def widen(c, tokens):
    """The same tables with room for `tokens` tokens a sequence (entries past the sequences unset)."""
    c.table = torch.nn.functional.pad(c.table, (0, tokens // c.bs - c.cols), value=-9).contiguous()
    c.cols = tokens // c.bs


@pytest.mark.parametrize("B,gamma,Hq,Hkv,D,bs,P", [(6, 1, 32, 8, 128, 16, 512), (40, 4, 16, 2, 128, 32, 640),
                                                   (5, 3, 42, 6, 64, 8, 264), (4, 1, 32, 1, 128, 128, 1024), (7, 2, 8, 8, 64, 16, 0)])
@pytest.mark.parametrize("pre", [0, 2])
def test_width_of_the_tables(R, B, gamma, Hq, Hkv, D, bs, P, pre):
    """Tables as wide as the sequences, four times as wide, of 131072 tokens."""
    lens = [P + (gamma + 1 + 211 * b * b) % 1900 for b in range(B - 1)] + [0]
    c = Case(lens, gamma, Hq, Hkv, D, bs, P, seed=110 + B)
    want = c.expect()
    for tokens in (0, 4 * c.cols * bs, 131072):
        if tokens:
            widen(c, tokens)
        out, err = c.run(R, 0, pre)
        assert int(err) == 0
        check(out, *want, what=f"plan {c.plan(R, 0, pre)}")


@pytest.mark.parametrize("P,pre", [(0, 0), (264, 1)])
def test_chunks_of_more_blocks_than_are_held(R, P, pre):
    """So many units that eight chunks are all a sequence gets: chunks of 316 blocks of 8 tokens, whose ids are loaded some
    120 at a time."""
    lens = [P + 30 + b % 7 for b in range(79)] + [P + 20000]
    c = Case([P + 1] * 80, 1, 16, 16, 64, 8, P, cols=(P + 64) // 8, seed=120)
    own = c.table.shape[1] - P // 8
    blocks = torch.randperm(2500, device=DEV, generator=torch.Generator(device=DEV).manual_seed(121)).int()
    g = torch.Generator(device=DEV).manual_seed(122)
    n0 = c.k.shape[0]
    more = [torch.randn(2500, 8, 16, 64, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    spare = [torch.randn(n0, 8, 16, 64, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    c.k, c.v = torch.cat([spare[0], more[0]]), torch.cat([spare[1], more[1]])
    ids = torch.randperm(n0, device=DEV, generator=g).int()
    c.prefix = ids[:P // 8].contiguous()
    c.table = torch.full((80, (P + 20480) // 8), -9, dtype=torch.int32, device=DEV)
    c.table[:, P // 8:P // 8 + own] = ids[P // 8:P // 8 + 80 * own].reshape(80, own)
    c.table[79, P // 8:P // 8 + 2500] = n0 + blocks
    c.cols, c.lens_list = c.table.shape[1], lens
    c.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    splits, chunks, _ = c.plan(R, 0, pre)
    assert splits == 8 and chunks == pre
    out, err = c.run(R, 0, pre)
    assert int(err) == 0
    check(out, *c.expect())
    c.table[79, P // 8 + 2000] = c.k.shape[0]                # a bad id far behind the first that are loaded
    out, err = c.run(R, 0, pre)
    assert int(err) == R.RRA_ERR_BLOCK_ID
