"""A speculative step on a tree of drafted tokens (test infrastructure): attention, kept path, log probabilities.

[Opt-2026] §五 (speculative decoding) checks a chain of drafted tokens; here each token may have several
continuations. Sequence b has p_b cached tokens and nodes 0 .. n_b - 1; node j follows node parents[b, j] < j, or the
last cached token (-1). It sits in cache slot p_b + j, is rotated for position p_b + depth (depth: its ancestors among
the nodes), and attends the cached tokens, its ancestors and itself -- what decoding the tokens of its path one
at a time would give.
"""

from __future__ import annotations

import numpy as np

from .attention import gqa_decode_attention
from .bf16 import f64_to_storage, storage_to_f64
from .decode import logical_kv
from .kvcache import append_contiguous, append_paged
from .rope import apply_rope


def paths(parents) -> list:
    """Of every node of one tree: its ancestors, the first one first, and itself."""
    out = []
    for j, p in enumerate(np.asarray(parents).tolist()):
        out.append((out[p] if p >= 0 else []) + [j])
    return out


def rope_append_tree(q, k_new, v_new, positions, parents, k_cache, v_cache, dtype, block_table=None, block_size=0,
                     rope_base: float = 10000.0, rope_style: int = 0):
    """Rotate node j of q and k_new at p_b + depth, append rotated k and raw v at slot p_b + j, in place; returns q_rot."""
    B, N = q.shape[:2]
    slot = np.asarray(positions, dtype=np.int64)[:, None] + np.arange(N)
    depth = np.array([[len(path) - 1 for path in paths(parents[b])] for b in range(B)])
    at = np.asarray(positions, dtype=np.int64)[:, None] + depth
    q_rot = f64_to_storage(apply_rope(storage_to_f64(q, dtype), at[:, :, None], rope_base, rope_style), dtype)
    k_rot = f64_to_storage(apply_rope(storage_to_f64(k_new, dtype), at[:, :, None], rope_base, rope_style), dtype)
    for j in range(N):
        if block_table is None:
            append_contiguous(k_cache, v_cache, k_rot[:, j], v_new[:, j], slot[:, j])
        else:
            append_paged(k_cache, v_cache, block_table, block_size, k_rot[:, j], v_new[:, j], slot[:, j])
    return q_rot


def tree_attention(q_rot, k_cache, v_cache, positions, parents, dtype, block_table=None, block_size=0,
                   scale=None) -> np.ndarray:
    """out[b, j] = GQA softmax attention of q_rot[b, j] over the cached tokens and node j's path, float64."""
    B, N = q_rot.shape[:2]
    out = []
    for b in range(B):
        p = int(positions[b])
        k = storage_to_f64(logical_kv(k_cache, b, p + N, block_table, block_size), dtype)
        v = storage_to_f64(logical_kv(v_cache, b, p + N, block_table, block_size), dtype)
        rows = []
        for j, path in enumerate(paths(parents[b])):
            seen = list(range(p)) + [p + x for x in path]
            rows.append(gqa_decode_attention(storage_to_f64(q_rot[b, j], dtype), k[:, seen], v[:, seen], scale))
        out.append(np.stack(rows))
    return np.stack(out)


def tree_step(q, k_new, v_new, positions, parents, k_cache, v_cache, dtype, block_table=None, block_size=0,
              rope_base: float = 10000.0, rope_style: int = 0, scale=None):
    """RoPE + append of the nodes + their attention, on copies of the caches: (q_rot, k after, v after, out float64)."""
    kc, vc = np.array(k_cache, copy=True), np.array(v_cache, copy=True)
    q_rot = rope_append_tree(q, k_new, v_new, positions, parents, kc, vc, dtype, block_table, block_size, rope_base,
                             rope_style)
    return q_rot, kc, vc, tree_attention(q_rot, kc, vc, positions, parents, dtype, block_table, block_size, scale)


def kept_path(tokens, parents, choices) -> list:
    """The nodes of one tree that the target keeps: from node 0 on to the lowest child whose token is the node's choice."""
    path = [0]
    while True:
        x = path[-1]
        below = [j for j in range(len(tokens)) if parents[j] == x and tokens[j] == choices[x] and choices[x] >= 0]
        if not below:
            return path
        path.append(below[0])


def token_logprobs(x, top_k: int = 0):
    """Of rows of logits [R, V]: (log probabilities [R, V], entropies [R], the top_k tokens, equal ones in order), float64."""
    x = np.asarray(x, dtype=np.float64)
    m = x.max(1, keepdims=True)
    lp = x - m - np.log(np.exp(x - m).sum(1, keepdims=True))
    p = np.exp(lp)
    h = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum(1)
    return lp, h, np.argsort(-x, axis=1, kind="stable")[:, :top_k]
