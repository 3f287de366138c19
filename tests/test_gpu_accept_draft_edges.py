"""Draft acceptance at the edges of its range: probabilities that are none at drafted tokens, draws on the borders of the
cumulative sums against exact integers."""

import numpy as np
import pytest
import torch

from tests.test_gpu_accept_draft import make, plain

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def R():
    import rope_gqa_paged_gb300 as mod
    from rope_gqa_paged_gb300 import _build
    _build.build()
    return mod


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafter", [True, False])
def test_drafted_tokens_with_bad_probabilities(R, dt, drafter):
    """NaN counts as 0 and a value outside [0, 1] as the nearer end in the comparison too, whatever the other value is."""
    bad = [NAN, -3.0, -INF, 2.0, INF, 1.5, 0.0, 1.0, -0.0, 0.25]
    pairs = [(pv, qv) for pv in bad for qv in (bad if drafter else [1.0])]
    B, gamma, V = 3 * len(pairs), 2, 300
    p, q, x, u, ul = make(B, gamma, V, dt, True, seed=11)
    u = torch.tensor([0.0, 0.5, 0.999], device=DEV).repeat_interleave(len(pairs))[:, None].expand(B, gamma).contiguous()
    x[:, 0] = 17
    p[:, 0, 17] = torch.tensor([pv for pv, _ in pairs], device=DEV).to(dt).repeat(3)
    q[:, 0, 17] = torch.tensor([qv for _, qv in pairs], device=DEV).to(dt).repeat(3)
    tokens, kept = R.rra_accept_draft(p, x, u, ul, draft_probs=q if drafter else None)
    fair = [t.nan_to_num(nan=0.0, posinf=1.0, neginf=0.0).clamp(0, 1) for t in (p, q)]
    want = plain(fair[0], fair[1] if drafter else None, x, None, u, ul)
    np.testing.assert_array_equal(kept.cpu().numpy(), want[1])
    np.testing.assert_array_equal(tokens.cpu().numpy(), want[0])
    assert 0 < (kept > 0).sum() < B


def exact_draw(p, q, skip, u):
    """The draw from max(p - q, 0) (p itself where that is nothing) in Python's integers: probabilities rounded to whole
    units, nearest even (2^-60 for float32, 2^-45 for bf16), the lowest index whose inclusive sum exceeds floor(u total)."""
    unit = 60 if p.dtype == torch.float32 else 45

    def whole(t):                                            # (a float32's product with a power of two is exact in float64)
        return np.rint(t.double().clamp(0, 1).cpu().numpy() * 2.0 ** unit).astype(np.int64)

    pi = whole(p)
    r = pi.copy() if q is None else pi - np.minimum(pi, whole(q))
    if skip is not None:
        r[skip] = 0
    if r.sum() == 0:
        r = pi
    c = np.cumsum(r << (60 - unit))
    border = (int(c[-1]) * int(float(u) * 2.0 ** 64)) >> 64
    return int(np.searchsorted(c, border, side="right")), c


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("form", ["all kept", "rejected", "looked up"])
@pytest.mark.parametrize("B", [1, 5, 19, 76, 152, 304, 700])           # clusters of 16, 16, 8, 8, 4, 2 and 1 CTAs
@pytest.mark.parametrize("V", [4096, 6007])
def test_draws_on_the_borders(R, B, V, form, dt):
    """u within two steps of a border of the cumulative sum: the same token as exact integers give."""
    g = torch.Generator(device=DEV).manual_seed(B + V)
    if V == 4096:                                            # every border is a float32
        p = torch.full((B, 2, V), 1.0 / V, device=DEV).to(dt)
        q = torch.zeros(B, 1, V, device=DEV).to(dt)
    else:                                                    # some values below a unit, some of 0
        p, q = (torch.softmax(torch.randn(B, n, V, generator=g, device=DEV) * 6, -1).to(dt) for n in (2, 1))
    x = torch.randint(0, V, (B, 1), generator=g, device=DEV).int()
    u = torch.full((B, 1), 0.999, device=DEV)
    if form == "all kept":
        u.zero_()
        p[:, 0].scatter_(1, x.long(), 1.0)
        q = None
    elif form == "rejected":
        p[:, 0].scatter_(1, x.long(), 0.0)
    else:
        q = None
        p[:, 0].clamp_(max=0.9)
    row = 1 if form == "all kept" else 0
    ul, want = np.zeros(B, np.float32), np.zeros(B, np.int64)
    rng = np.random.default_rng(B)
    for b in range(B):
        args = (p[b, row], None if q is None else q[b, 0], int(x[b, 0]) if form == "looked up" else None)
        c = exact_draw(*args, 0.0)[1]
        at = np.float32(min(int(c[rng.integers(0, V)]) / int(c[-1]), 1 - 2.0 ** -24))
        for _ in range(abs(int(rng.integers(-2, 3)))):
            at = np.nextafter(at, np.float32(rng.integers(0, 2)))
        ul[b] = min(max(at, 0.0), 1 - 2.0 ** -24)
        want[b] = exact_draw(*args, ul[b])[0]
    tokens, kept = R.rra_accept_draft(p, x, u, torch.from_numpy(ul).to(DEV), draft_probs=q)
    np.testing.assert_array_equal(kept.cpu().numpy(), np.full(B, row))
    np.testing.assert_array_equal(tokens[:, row].cpu().numpy(), want)
