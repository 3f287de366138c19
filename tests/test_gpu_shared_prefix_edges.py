"""Shared-prefix attention at the edges of its range: rows of a few tokens.

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
@pytest.mark.parametrize("P,pre", [(8, 1), (64, 1), (264, 1), (264, 5), (1000, 3)])
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
