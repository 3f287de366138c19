"""The float64 oracle of the step on a tree of drafted tokens against independent statements of the same facts (CPU only),
and mistakes planted in it, each of which one of them catches."""

import numpy as np
import pytest
import torch

import oracle


def _case(layout, N=7, seed=3):
    rng = np.random.default_rng(seed)
    B, hq, hkv, d, bs, cap = 2, 8, 2, 16, 4, 24
    p0 = np.array([5, 11])
    q, kn, vn = (oracle.f64_to_bf16_bits(rng.standard_normal((B, N, h, d))) for h in (hq, hkv, hkv))
    shape = (B, hkv, cap, d) if layout == "contiguous" else (3 * cap // bs, bs, hkv, d)
    table = None if layout == "contiguous" else rng.permutation(shape[0])[:2 * (cap // bs)].reshape(2, -1).astype(np.int32)
    kc, vc = (oracle.f64_to_bf16_bits(rng.standard_normal(shape)) for _ in range(2))
    parents = np.array([[-1] + [int(rng.integers(-1, j)) for j in range(1, N)] for _ in range(B)])
    return q, kn, vn, p0, parents, kc, vc, table, bs


def pin_chain_equals_verify():
    for layout in ("contiguous", "paged"):
        for style in (0, 1):
            q, kn, vn, p0, _, kc, vc, table, bs = _case(layout)
            chain = np.tile(np.arange(-1, q.shape[1] - 1), (2, 1))
            got = oracle.tree.tree_step(q, kn, vn, p0, chain, kc, vc, "bf16", table, bs, rope_style=style)
            want = oracle.verify.verify_step(q, kn, vn, p0, kc, vc, "bf16", table, bs, rope_style=style)
            for a, b in zip(got[:3], want[:3]):
                assert np.array_equal(a, b)
            assert np.allclose(got[3], want[3], rtol=0, atol=1e-13)


def pin_every_path_equals_decoding_it():
    # node j's row is what decoding the tokens of its path one at a time gives
    for layout in ("contiguous", "paged"):
        q, kn, vn, p0, parents, kc, vc, table, bs = _case(layout)
        q_rot, k_after, v_after, out = oracle.tree.tree_step(q, kn, vn, p0, parents, kc, vc, "bf16", table, bs)
        for b in range(2):
            for j in range(q.shape[1]):
                path, x = [], j
                while x >= 0:
                    path.insert(0, x)
                    x = parents[b, x]
                k2, v2 = kc.copy(), vc.copy()
                for i, x in enumerate(path):
                    qr, k2, v2, o = oracle.decode.decode_step(q[:, x], kn[:, x], vn[:, x], p0 + i, k2, v2, "bf16", table, bs)
                assert np.array_equal(q_rot[b, j], qr[b])
                assert np.allclose(out[b, j], o[b], rtol=0, atol=1e-13), (layout, b, j)
                # ... and its key is what that leaves at the path's end, in slot p + j
                a, c = (oracle.decode.logical_kv(x, b, p0[b] + n, table, bs) for x, n in ((k_after, j + 1), (k2, len(path))))
                assert np.array_equal(a[:, p0[b] + j], c[:, p0[b] + len(path) - 1])


def pin_logprobs():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 40)) * 3
    x[1, 3:30] = -np.inf
    x[2] = np.round(x[2])
    lp, h, top = oracle.tree.token_logprobs(x, 9)
    assert np.allclose(lp, torch.log_softmax(torch.from_numpy(x), 1).numpy(), rtol=0, atol=1e-12)
    assert np.allclose(h, torch.distributions.Categorical(logits=torch.from_numpy(x).clamp(min=-1e30)).entropy().numpy(), atol=1e-12)
    for r in range(5):
        order = sorted(range(40), key=lambda v: (-x[r, v], v))[:9]
        assert top[r].tolist() == order


def pin_kept_path():
    #       0 -> 1, 2;  1 -> 3, 4;  2 -> 5;  4 -> 6
    parents, tokens = [-1, 0, 0, 1, 1, 2, 4], [9, 5, 6, 7, 7, 8, 3]
    assert oracle.tree.kept_path(tokens, parents, [5, 7, 8, 1, 3, 0, 0]) == [0, 1, 3]      # equal children: the lower one
    assert oracle.tree.kept_path(tokens, parents, [6, 7, 8, 1, 3, 0, 0]) == [0, 2, 5]
    assert oracle.tree.kept_path(tokens, parents, [4, 7, 8, 1, 3, 0, 0]) == [0]
    assert oracle.tree.kept_path([-1, -1], [-1, 0], [-1, -1]) == [0]                       # no token matches none


PINS = [pin_chain_equals_verify, pin_every_path_equals_decoding_it, pin_logprobs, pin_kept_path]


@pytest.mark.parametrize("pin", PINS, ids=lambda p: p.__name__)
def test_pin(pin):
    pin()


def _no_ancestors(parents):
    return [[j] for j in range(len(parents))]


def _all_before(parents):
    return [list(range(j + 1)) for j in range(len(parents))]


def _highest_child(tokens, parents, choices):
    path = [0]
    while True:
        below = [j for j in range(len(tokens)) if parents[j] == path[-1] and tokens[j] == choices[path[-1]]]
        if not below:
            return path
        path.append(below[-1])


def _unstable_top(x, top_k=0, old=oracle.tree.token_logprobs):
    lp, h, _ = old(x, top_k)
    return lp, h, np.argsort(np.asarray(x), axis=1, kind="stable")[:, ::-1][:, :top_k]


def _base_two(x, top_k=0, old=oracle.tree.token_logprobs):
    lp, h, top = old(x, top_k)
    return lp, h / np.log(2), top


@pytest.mark.parametrize("name,new", [("paths", _no_ancestors), ("paths", _all_before), ("kept_path", _highest_child),
                                      ("token_logprobs", _unstable_top), ("token_logprobs", _base_two)])
def test_planted_mistakes_are_caught(monkeypatch, name, new):
    monkeypatch.setattr(oracle.tree, name, new)
    failed = 0
    for pin in PINS:
        try:
            pin()
        except AssertionError:
            failed += 1
    assert failed >= 1
