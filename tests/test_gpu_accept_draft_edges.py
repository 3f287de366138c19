"""Draft acceptance at the edges of its range: probabilities that are none at drafted tokens."""

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
