"""Acceptance of drafted tokens (rra_accept_draft) against the rule in float64 on the host, and the loop it
closes with the shared-prefix step. The outputs are whole numbers: they have to be equal."""

import numpy as np
import pytest
import torch

from tests.test_gpu_shared_prefix import Case, check

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def R():
    import rope_gqa_paged_gb300 as mod
    from rope_gqa_paged_gb300 import _build
    _build.build()
    return mod


def plain(p, q, x, lens, u, u_last):
    """(tokens [B, gamma + 1], kept [B]) in float64; p, q as given (bf16 or fp32 tensors)."""
    p = p.double().cpu().numpy()
    q = None if q is None else q.double().cpu().numpy()
    x, u, u_last = x.cpu().numpy(), u.double().cpu().numpy(), u_last.double().cpu().numpy()
    B, gamma = x.shape
    V = p.shape[2]
    tokens, kept = np.full((B, gamma + 1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        m = gamma if lens is None else int(lens[b])
        n = 0
        while n < m:
            t = x[b, n]
            qx = 1.0 if q is None else q[b, n, t] if 0 <= t < V else 0.0
            if not (0 <= t < V and u[b, n] * qx < p[b, n, t]):
                break
            n += 1
        r = p[b, n].copy()
        if n < m:
            if q is None:
                if 0 <= x[b, n] < V:
                    r[x[b, n]] = 0.0
            else:
                r = np.maximum(r - q[b, n], 0.0)
            if not r.sum() > 0:
                r = p[b, n]
        c = np.cumsum(r)
        tokens[b, :n], kept[b] = x[b, :n], n
        tokens[b, n] = min(int(np.searchsorted(c, min(u_last[b], 1 - 2.0 ** -24) * c[-1], side="right")), V - 1)
    return tokens, kept


def make(B, gamma, V, dt, drafter=True, seed=0, sharp=2.0, noise=0.6):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = torch.randn(B, gamma + 1, V, generator=g, device=DEV) * sharp
    p = torch.softmax(logits, -1).to(dt)
    q, x = None, None
    if drafter:
        q = torch.softmax(logits[:, :gamma] + noise * torch.randn(B, gamma, V, generator=g, device=DEV), -1).to(dt)
    x = torch.multinomial((p[:, :gamma] if q is None else q).float().reshape(B * gamma, V), 1, generator=g)
    u = torch.rand(B, gamma, generator=g, device=DEV)
    return p, q, x.reshape(B, gamma).int(), u, torch.rand(B, generator=g, device=DEV)


def same(R, p, q, x, u, ul, lens=None, err_want=0, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tokens, kept = R.rra_accept_draft(p, x, u, ul, draft_probs=q, draft_lens=lens, err_flag=err, **kw)[:2]
    want = plain(p, q, x, lens, u, ul)
    assert int(err) == err_want
    np.testing.assert_array_equal(kept.cpu().numpy(), want[1])
    np.testing.assert_array_equal(tokens.cpu().numpy(), want[0])
    return want


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("B,gamma,V", [(3, 1, 1), (5, 2, 2), (7, 3, 31), (9, 4, 33), (40, 5, 257), (17, 32, 1000),
                                       (33, 4, 8191), (6, 7, 32000), (20, 3, 50001), (3, 2, 262147)])
def test_sizes(R, B, gamma, V, drafter, dt):
    kept = same(R, *make(B, gamma, V, dt, drafter, seed=V + gamma))[1]
    if B * gamma > 60 and drafter:
        assert 0 < kept.mean() < gamma                       # the case has kept and rejected tokens


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafter", [True, False])
@pytest.mark.parametrize("B,V", [(2, 2000003), (640, 40001), (1, 9000001)])
def test_long_runs(R, B, V, drafter, dt):
    """Parts of the vocabulary that one search of the CTA does not cover: few CTAs per sequence, or a huge one."""
    same(R, *make(B, 1, V, dt, drafter, seed=V, sharp=1.0))


@pytest.mark.parametrize("drafter", [True, False])
def test_ragged_drafts(R, drafter):
    p, q, x, u, ul = make(50, 6, 700, torch.float32, drafter, seed=1)
    same(R, p, q, x, u, ul, lens=(torch.arange(50, device=DEV) % 7).int())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rows_of_any_stride_and_alignment(R, dt):
    """Rows inside wider ones, at odd offsets, in another order, and one row broadcast to all sequences."""
    p, q, x, u, ul = make(11, 3, 1003, dt, seed=2)
    wide = torch.full((11, 4, 1003 + 38), 0.5, dtype=dt, device=DEV)
    wide[..., 1:1004] = p
    other = torch.full((3, 11, 1003 + 6), 0.5, dtype=dt, device=DEV).transpose(0, 1)
    other[..., 5:1008] = q
    same(R, wide[..., 1:1004], other[..., 5:1008], x, u, ul)
    same(R, p[:1].expand(11, -1, -1), q, x, u, ul)


def test_far_rows(R):
    """Rows more than 2^31 elements from the first."""
    V = 100000
    p, q, x, u, ul = make(2, 1, V, torch.bfloat16, seed=3)
    big = torch.empty(2, 2, V + (1 << 30), dtype=torch.bfloat16, device=DEV)[..., :V]
    big.copy_(p)
    assert big.stride(0) > 1 << 31
    same(R, big, q, x, u, ul)


def test_ends_of_the_draw(R):
    """u = 0 draws the first token that may be drawn, the largest u below 1 (and 1) the last one."""
    p, q, x, _, _ = make(4, 2, 5000, torch.float32, seed=4)
    p[:, :, 4000:] = 0
    p[:, :, :10] = 0
    u = torch.full((4, 2), 0.999, device=DEV)
    x[:] = 4500                                              # p = 0: rejected
    for ul in (0.0, 1 - 2.0 ** -24, 1.0):
        t = same(R, p, q, x, u, torch.full((4,), ul, device=DEV))[0][:, 0]
        assert (t >= 10).all() and (t < 4000).all()


def test_comparison_is_strict_and_exact(R):
    """u q = p rejects; one step of u below it keeps (24-bit u and q: the product needs 48 bits)."""
    V = 64
    q = torch.full((2, 1, V), 1 / 64, device=DEV)
    p = torch.full((2, 2, V), 1 / 64, device=DEV)
    q[:, 0, 5] = 0.7000001
    p[:, 0, 5] = 0.35
    x = torch.full((2, 1), 5, dtype=torch.int32, device=DEV)
    q5, p5 = float(q[0, 0, 5]), float(p[0, 0, 5])
    us = np.array([np.float32(p5 / q5)])
    lo = us.copy()
    while float(lo[0]) * q5 >= p5:
        lo = np.nextafter(lo, np.float32(0))
    hi = np.nextafter(lo, np.float32(1))
    assert float(hi[0]) * q5 >= p5 > float(lo[0]) * q5
    u = torch.tensor([[lo[0]], [hi[0]]], device=DEV)
    kept = same(R, p, q, x, u, torch.full((2,), 0.5, device=DEV))[1]
    assert kept.tolist() == [1, 0]
    q[:, 0, 5], p[:, 0, 5] = 0.5, 0.125
    kept = same(R, p, q, x, torch.full((2, 1), 0.25, device=DEV), torch.full((2,), 0.5, device=DEV))[1]
    assert kept.tolist() == [0, 0]


def test_nothing_left(R):
    """p below q everywhere (rows that do not sum to 1): the draw is from p; a row of zeros: the last token, flagged."""
    p, q, x, u, ul = make(6, 2, 999, torch.float32, seed=5)
    p[:, :2] = q * 0.5
    u = torch.full_like(u, 0.9)
    same(R, p, q, x, u, ul)
    p[3, 0] = 0
    t, _ = same(R, p, q, x, u, ul, err_want=R.RRA_ERR_PROBS)
    assert t[3, 0] == 998


def test_bad_values(R):
    """Tokens outside the vocabulary count as rejected, lengths outside 0..gamma are cut, both flagged; NaN and values
    outside [0, 1] count as the nearer end."""
    p, q, x, u, ul = make(6, 3, 500, torch.float32, seed=6)
    x[1, 0], x[2, 1], x[3, 2] = -1, 500, 2 ** 31 - 1
    same(R, p, q, x, u, ul, err_want=R.RRA_ERR_TOKEN)
    p, q, x, u, ul = make(6, 3, 500, torch.float32, seed=7)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = torch.tensor([-4, 9, 2, 3, 0, 1], dtype=torch.int32, device=DEV)
    tokens, kept = R.rra_accept_draft(p, x, u, ul, draft_probs=q, draft_lens=lens, err_flag=err)
    want = plain(p, q, x, lens.clamp(0, 3), u, ul)
    assert int(err) == R.RRA_ERR_SEQ_LEN
    np.testing.assert_array_equal(tokens.cpu().numpy(), want[0])
    p2, q2 = p.clone(), q.clone()
    p2[:, :, 40], p2[:, :, 41], p2[:, :, 42] = float("nan"), -3.0, float("-inf")
    q2[:, :, 43] = float("nan")
    p, q = p.clone(), q.clone()
    p[:, :, 40:43], q[:, :, 43] = 0, 0
    x[x == 43] = 44
    tokens, kept = R.rra_accept_draft(p2, x, u, ul, draft_probs=q2)
    want = plain(p, q, x, None, u, ul)
    np.testing.assert_array_equal(tokens.cpu().numpy(), want[0])


def test_emitted_tokens_follow_the_target(R):
    """100000 sequences of one drafted token: the first emitted token's frequencies are p's, within six
    standard deviations of a binomial count."""
    N, V = 50000, 6
    p1 = torch.tensor([0.4, 0.05, 0.25, 0.1, 0.0, 0.2], device=DEV)
    q1 = torch.tensor([0.1, 0.3, 0.2, 0.1, 0.1, 0.2], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(8)
    counts = np.zeros(V)
    for _ in range(2):
        x = torch.multinomial(q1.expand(N, -1), 1, generator=g).int()
        t, _ = R.rra_accept_draft(p1.expand(N, 2, V), x, torch.rand(N, 1, generator=g, device=DEV),
                                  torch.rand(N, generator=g, device=DEV), draft_probs=q1.expand(N, 1, V))
        counts += np.bincount(t[:, 0].cpu().numpy(), minlength=V)
    pn = p1.double().cpu().numpy()
    assert (np.abs(counts - 2 * N * pn) <= 6 * np.sqrt(2 * N * pn * (1 - pn)) + 1e-9).all()


def test_positions_streams_and_graphs(R):
    """Next positions (in place too); captured on a side stream, replayed with refilled inputs; two calls at once."""
    a, c = make(8, 4, 32000, torch.float32, seed=9), make(30, 2, 5001, torch.bfloat16, seed=10)
    pos = torch.arange(8, dtype=torch.int32, device=DEV) * 100
    want = plain(a[0], a[1], a[2], None, a[3], a[4])
    out = R.rra_accept_draft(a[0], a[2], a[3], a[4], draft_probs=a[1], positions=pos)
    np.testing.assert_array_equal(out[2].cpu().numpy(), pos.cpu().numpy() + want[1] + 1)
    R.rra_accept_draft(a[0], a[2], a[3], a[4], draft_probs=a[1], positions=pos, positions_out=pos)
    assert torch.equal(out[2], pos)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s1):
            ta = R.rra_accept_draft(a[0], a[2], a[3], a[4], draft_probs=a[1])
        with torch.cuda.stream(s2):
            tc = R.rra_accept_draft(c[0], c[2], c[3], c[4], draft_probs=c[1])
    torch.cuda.synchronize()
    np.testing.assert_array_equal(ta[0].cpu().numpy(), want[0])
    np.testing.assert_array_equal(tc[0].cpu().numpy(), plain(c[0], c[1], c[2], None, c[3], c[4])[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1):
        ta = R.rra_accept_draft(a[0], a[2], a[3], a[4], draft_probs=a[1])
    for seed in (11, 12):
        new = make(8, 4, 32000, torch.float32, seed=seed)
        for t, n in zip(a, new):
            t.copy_(n)
        graph.replay()
        np.testing.assert_array_equal(ta[0].cpu().numpy(), plain(*new[:3], None, *new[3:])[0])


def test_refusals(R):
    p, q, x, u, ul = make(3, 2, 100, torch.float32, seed=13)
    call = R.rra_accept_draft
    with pytest.raises(ValueError):
        call(p[:, :2], x, u, ul, draft_probs=q)
    with pytest.raises(ValueError):
        call(p, x, u, ul, draft_probs=q[..., :50])
    with pytest.raises(ValueError):
        call(p, x, u, ul, draft_probs=q.bfloat16())
    with pytest.raises(ValueError):
        call(p.transpose(1, 2).contiguous().transpose(1, 2), x, u, ul, draft_probs=q)
    with pytest.raises(ValueError):
        call(p, x.long(), u, ul, draft_probs=q)
    with pytest.raises(TypeError):
        call(p, x, u.double(), ul, draft_probs=q)
    with pytest.raises(TypeError):
        call(p.half(), x, u, ul, draft_probs=None)
    with pytest.raises(ValueError):
        call(p.cpu(), x, u, ul, draft_probs=q)
    many = make(1, 33, 50, torch.float32, seed=14)
    with pytest.raises(R.RraError):
        call(many[0], many[2], many[3], many[4], draft_probs=many[1])


def test_speculative_loop(R):
    """Rounds of a speculative decode behind a shared prompt, without reading anything back in between: the step
    over gamma drafted tokens, the target's probabilities from its output, the acceptance, the next positions.
    Each round's attention and decisions are then checked by themselves."""
    P, gamma, B, Hq, Hkv, D, V, rounds = 512, 3, 5, 8, 2, 128, 997, 6
    room = P + rounds * (gamma + 1) + 8
    c = Case([room] * B, gamma, Hq, Hkv, D, 16, P, seed=60, poison=False)
    g = torch.Generator(device=DEV).manual_seed(61)

    def randn(*s):
        return torch.randn(*s, generator=g, device=DEV)

    emb = randn(V, (Hq + 2 * Hkv) * D).bfloat16()
    head = randn(Hq * D, V) * 0.4
    step = R.SharedPrefixStep(B, gamma, Hq, Hkv, D, c.k, c.v, c.prefix, P, c.table, prefix_splits=3)
    pos = P + torch.arange(B, dtype=torch.int32, device=DEV)
    first = torch.randint(0, V, (B, 1), generator=g, device=DEV).int()
    log = []
    for _ in range(rounds):
        # the drafter: gamma - 1 tokens after the last one, from its own distributions
        q = torch.softmax(randn(B, gamma - 1, V) * 1.5, -1)
        x = torch.multinomial(q.reshape(-1, V), 1, generator=g).reshape(B, gamma - 1).int()
        tok = torch.cat([first, x], 1).long()
        qkv = emb[tok].reshape(B, gamma, Hq + 2 * Hkv, D)
        out = step(qkv[:, :, :Hq].contiguous(), qkv[:, :, Hq:Hq + Hkv].contiguous(), qkv[:, :, Hq + Hkv:].contiguous(), pos)
        p = torch.softmax(out.float().reshape(B, gamma, -1) @ head + (q.new_zeros(1)), -1)
        p[:, :gamma - 1] = 0.5 * p[:, :gamma - 1] + 0.5 * q       # a target that is near its drafter
        u, ul = torch.rand(B, gamma - 1, generator=g, device=DEV), torch.rand(B, generator=g, device=DEV)
        tokens, kept, nxt = R.rra_accept_draft(p, x, u, ul, draft_probs=q, positions=pos)
        log.append((pos, out.clone(), step.q_rot.clone(), c.k.clone(), c.v.clone(), p, q, x, u, ul, tokens, kept, nxt))
        first = tokens.gather(1, kept[:, None].long())
        pos = nxt
    assert step.error_bits() == 0
    total = 0
    for pos, out, rot, k, v, p, q, x, u, ul, tokens, kept, nxt in log:
        c.k, c.v, c.lens_list = k, v, (pos + gamma).tolist()
        check(out, *c.expect(rot))
        want = plain(p, q, x, None, u, ul)
        np.testing.assert_array_equal(tokens.cpu().numpy(), want[0])
        np.testing.assert_array_equal(nxt.cpu().numpy(), pos.cpu().numpy() + want[1] + 1)
        total += int(want[1].sum())
    assert 0 < total < rounds * B * (gamma - 1)


@pytest.mark.parametrize("V", [9, 1000, 1009, 16 * 4000 + 3, 128000])
def test_rows_that_are_no_distribution(R, V):
    """Rows that sum to 8 and more (scores passed for probabilities): some token of the vocabulary is written, and
    nothing else changes."""
    g = torch.Generator(device=DEV).manual_seed(V)
    p = torch.randn(5, 4, V, generator=g, device=DEV).abs() * 3
    p[0] = 1.0
    q = torch.zeros(5, 3, V, device=DEV)
    x = torch.randint(0, V, (5, 3), generator=g, device=DEV).int()
    lens = torch.tensor([0, 1, 2, 3, 0], dtype=torch.int32, device=DEV)       # q = 0: every drafted token is kept
    tokens = torch.full((5, 4), -77, dtype=torch.int32, device=DEV)
    p.scatter_(2, torch.cat([x, x[:, :1]], 1)[:, :, None].long(), 0.5)
    R.rra_accept_draft(p, x, torch.zeros(5, 3, device=DEV), torch.rand(5, generator=g, device=DEV), draft_probs=q,
                       draft_lens=lens, tokens_out=tokens)
    for b, n in enumerate(lens.tolist()):
        row = tokens[b].tolist()
        assert row[:n] == x[b, :n].tolist() and 0 <= row[n] < V and row[n + 1:] == [-1] * (3 - n)
