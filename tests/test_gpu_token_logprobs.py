"""Log probabilities of tokens (rra_token_logprobs) against their definition in float64.

Tolerances, absolute, in natural logarithms. With a = x - m exact to half a float32 step (2^-24 |a|), 2^d by the
special-function unit to 2^-22 and at most n = V / 256 + 40 float32 additions one after the other (half a step each):
ln S is off by at most 2^-22 + (n + E|a|) 2^-24, where the mean of |a| under p is below ln V + 1; a log
probability adds the roundings of a, of ln S and of their difference, 2^-24 (2 |a| + 2 |ln S|). The entropy's second
term U / S is off by the same relative errors of sums, (n + 8) 2^-24 + 2^-21 of E|a|, besides.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
INF = math.inf


@pytest.fixture(scope="module")
def R():
    import rope_gqa_paged_gb300 as mod
    from rope_gqa_paged_gb300 import _build
    _build.build()
    return mod


def expect(x, tokens, k):
    """(log p of tokens, entropy, log p of the top k, their ids, m, ln S) of rows x [R, V] in float64."""
    x = x.double()
    m = x.amax(1, keepdim=True)
    log_s = (x - m).exp().sum(1, keepdim=True).log()
    lp = (x - m) - log_s
    h = -torch.where(lp > -INF, lp.exp() * lp, 0.0).sum(1)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    given = lp.gather(1, tokens.long().clamp(min=0)) if tokens is not None else None
    if given is not None:
        given = torch.where(tokens < 0, 0.0, given)
    return given, h, lp.gather(1, order), order.int(), m, log_s


def close(got, want, tol):
    same = torch.isinf(want) & (got.double() == want)
    assert (same | ((got.double() - want).abs() <= tol)).all(), float(((got.double() - want).abs() - tol).nan_to_num().max())


def check(R, x, tokens=None, k=0, rows=None, **kw):
    """x [R, V] as the kernel sees it (possibly a view); compares everything; returns the outputs."""
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lp, h, top_lp, top = R.rra_token_logprobs(x, tokens, k, err_flag=err, **kw)
    flat = x.reshape(-1, x.shape[-1])
    V = flat.shape[1]
    tok = tokens.reshape(flat.shape[0], -1) if tokens is not None else None
    w_lp, w_h, w_top_lp, w_top, m, log_s = expect(flat, tok, k)
    assert int(err) == 0
    n, mean = V / 256 + 40, math.log(V) + 1
    sums = 2.0 ** -22 + (n + mean) * 2.0 ** -24

    def tol(want):
        a = (want + log_s).abs().nan_to_num(posinf=0.0)
        return sums + 2.0 ** -24 * (2 * a + 2 * log_s.abs())

    if tokens is not None:
        assert lp.shape == tokens.shape
        close(lp.reshape(w_lp.shape), w_lp, tol(w_lp))
    else:
        assert lp is None
    close(h.reshape(-1), w_h, sums + mean * ((n + 8) * 2.0 ** -24 + 2.0 ** -21) + 2.0 ** -23 * (log_s[:, 0].abs() + w_h))
    if k:
        assert torch.equal(top.reshape(-1, k), w_top)
        close(top_lp.reshape(-1, k), w_top_lp, tol(w_top_lp))
    else:
        assert top is None and top_lp is None
    return lp, h, top_lp, top


def randn(*shape, dtype=torch.float32, seed=0, scale=2.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def tokens_of(rows, T, V, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-1, V, (rows, T), generator=g, device=DEV, dtype=torch.int32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,V", [(1, 1), (1, 2), (3, 7), (2, 33), (5, 255), (1, 257), (4, 1000), (1, 4099), (9, 8192), (1, 32000),
                                    (19, 50001), (2, 100003), (70, 20011), (700, 1031), (1300, 517), (1, 1 << 20)])
def test_rows(R, rows, V, dtype):
    k = min(V, 20)
    check(R, randn(rows, V, dtype=dtype, seed=V), tokens_of(rows, 3, V), k)


@pytest.mark.parametrize("k", [0, 1, 2, 7, 8, 9, 31, 32])
@pytest.mark.parametrize("T", [0, 1, 32])
def test_counts(R, k, T):
    V = 3001
    check(R, randn(6, V, dtype=torch.bfloat16, seed=k), tokens_of(6, T, V) if T else None, k)


def test_shapes_and_strides(R):
    """Rows at odd offsets of a larger tensor, [B, N, V] and [rows, V], one token per row, broadcast rows."""
    base = randn(6, 5, 1201)
    for dtype in (torch.float32, torch.bfloat16):
        x = base.to(dtype)
        for view in (x, x[:, 1:4, :], x[::2, ::2, 3:1000], x[:, :, 1:], x[:, 2, 7:], x.transpose(0, 1)[:, :4, 5:]):
            tok = tokens_of(view[..., 0].numel(), 1, view.shape[-1]).reshape(view.shape[:-1])
            lp = check(R, view, tok, 5)[0]
            assert lp.shape == view.shape[:-1]
    row = randn(1, 999)
    check(R, row.expand(4, 999), tokens_of(4, 2, 999), 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lowest_index(R, dtype):
    for V in (40, 1000, 50001):
        check(R, torch.zeros(3, V, device=DEV, dtype=dtype), None, 32)                        # all alike
        few = randn(5, V, seed=V).round().to(dtype)
        check(R, few, None, 32)                                                              # few values, many ties
        ramp = torch.arange(V, device=DEV, dtype=torch.float32).expand(2, V) * 1e-3
        check(R, ramp.contiguous().to(dtype), None, 32)                                       # rising: the last ones
        check(R, ramp.flip(1).contiguous().to(dtype), None, 32)
        zeros = torch.zeros(2, V, device=DEV, dtype=dtype)
        zeros[:, ::2] = -0.0                                                                  # equal to 0
        check(R, zeros, None, 9)


def test_many_values_that_reach_the_bound(R):
    """All of a thread's values above all others': more candidates than the list holds."""
    V = 120000
    for lanes in (7, 32):
        x = randn(2, V, seed=lanes)
        at = torch.arange(V, device=DEV) // 4 % 256   # the thread that reads a value, with one CTA's stride
        x[:, at < lanes] += 100.0
        check(R, x, None, 32)
        check(R, x.repeat(400, 1), None, 32)          # (one CTA per row)


def test_masked_logits(R):
    """-inf is a probability of 0, alone or nearly everywhere; lowest values of the type; given tokens that are ruled out."""
    V = 30011
    for dtype in (torch.float32, torch.bfloat16):
        for keep in (1, 3, 25, 9000):
            x = torch.full((4, V), -INF, device=DEV, dtype=dtype)
            at = torch.randperm(V, generator=torch.Generator(device=DEV).manual_seed(keep), device=DEV)[:keep]
            x[:, at] = randn(4, keep, dtype=dtype, seed=keep)
            check(R, x, tokens_of(4, 5, V), 20)
        x = randn(3, V, dtype=dtype)
        x[:, 100:20000] = torch.finfo(dtype).min
        check(R, x, tokens_of(3, 4, V), 32)
        one = torch.full((1, V), torch.finfo(dtype).min, device=DEV, dtype=dtype)   # nothing but lowest values: even
        check(R, one, tokens_of(1, 2, V), 3)
    lp, h, top_lp, top = check(R, torch.tensor([[-INF, 4.0, -INF]], device=DEV), torch.tensor([[1, 0]], dtype=torch.int32, device=DEV), 3)
    assert lp.tolist() == [[0.0, -INF]] and h.tolist() == [0.0] and top.tolist() == [[1, 0, 2]]


def test_large_and_small_values(R):
    check(R, randn(4, 5000, scale=1e30), None, 5)
    check(R, randn(4, 5000, scale=1e-30), tokens_of(4, 2, 5000), 5)
    x = randn(2, 5000)
    x[:, 77] = 3e38
    check(R, x, tokens_of(2, 3, 5000), 5)


@pytest.mark.parametrize("bad", [float("nan"), INF, -INF])
def test_rows_without_a_distribution(R, bad):
    for rows, V in ((3, 5003), (900, 300)):
        x = randn(rows, V)
        if bad == -INF:
            x[1] = bad
        else:
            x[1, V // 3] = bad
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        tok = tokens_of(rows, 2, V).clamp(min=0)
        tok[1, 1] = -1
        lp, h, top_lp, top = R.rra_token_logprobs(x, tok, 4, err_flag=err)
        assert int(err) == R.RRA_ERR_PROBS
        assert torch.isnan(lp[1, 0]) and lp[1, 1] == 0 and torch.isnan(h[1]) and torch.isnan(top_lp[1]).all()
        assert top[1].tolist() == [-1] * 4
        rest = [i for i in range(rows) if i != 1]
        assert torch.isfinite(h[rest]).all()
        check(R, x[rest], tok[rest], 4)


def test_tokens_out_of_range(R):
    x = randn(2, 100)
    tok = torch.tensor([[5, 100], [-2, -1]], dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lp = R.rra_token_logprobs(x, tok, err_flag=err)[0]
    assert int(err) == R.RRA_ERR_TOKEN
    assert torch.isfinite(lp[0, 0]) and torch.isnan(lp[0, 1]) and torch.isnan(lp[1, 0]) and lp[1, 1] == 0


def test_given_outputs_streams_and_graphs(R):
    x, tok = randn(40, 9001, dtype=torch.bfloat16), tokens_of(40, 2, 9001)
    want = R.rra_token_logprobs(x, tok, 6)
    outs = [torch.empty_like(t) for t in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    R.rra_token_logprobs(x, tok, 6, *outs, stream=s)
    s.synchronize()
    for a, b in zip(want, outs):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.rra_token_logprobs(x, tok, 6, *outs)
        R.rra_token_logprobs(x, tok, 6, *outs)
    y = randn(40, 9001, dtype=torch.bfloat16, seed=5)
    x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(R.rra_token_logprobs(y, tok, 6), outs):
        assert torch.equal(a, b)


def test_more_rows_than_a_grid_dimension(R):
    check(R, randn(70001, 40), tokens_of(70001, 1, 40), 2)


def test_empty_batch(R):
    out = R.rra_token_logprobs(torch.empty(0, 50, device=DEV), None, 3)
    assert out[1].shape == (0,) and out[3].shape == (0, 3)
