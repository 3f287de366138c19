"""The accepted path of a tree of drafted tokens (rra_tree_keep) against a plain walk on the host, and the three
operators of a speculative step on a tree together."""

import pytest
import torch

from tests.test_gpu_tree import DEV, Case, random_parents

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    import rope_gqa_paged_gb300 as mod
    from rope_gqa_paged_gb300 import _build
    _build.build()
    return mod


def walk(tokens, parents, choices, n):
    path = [0] if n else []
    while path:
        x = path[-1]
        nxt = [j for j in range(n) if (parents[j] if -1 <= parents[j] < j else -1) == x and tokens[j] == choices[x] >= 0]
        if not nxt:
            return path
        path.append(nxt[0])
    return path


class Keep:
    """Random trees whose choices follow a random path, over random caches of several layers."""

    def __init__(self, cached, N, Hkv, D, bs, layers=2, lens=None, dtype=torch.bfloat16, kind="random", seed=0, vocab=50):
        g = torch.Generator().manual_seed(seed)
        B = self.B = len(cached)
        self.N, self.Hkv, self.D, self.bs, self.cached, self.n = N, Hkv, D, bs, cached, lens or [N] * B
        self.parents = random_parents(B, N, g, kind)
        self.tokens = torch.randint(0, vocab, (B, N), generator=g).int()
        self.choices = torch.randint(0, vocab, (B, N), generator=g).int()
        for b in range(B):
            for j in range(1, N):   # many a choice is one of the children's tokens
                if float(torch.rand(1, generator=g)) < 0.7 and self.parents[b, j] >= 0:
                    self.choices[b, self.parents[b, j]] = self.tokens[b, j]
        ends = [p + N for p in cached]
        if bs:
            need = [-(-e // bs) for e in ends]
            perm = torch.randperm(sum(need), generator=g).int()
            self.table = torch.full((B, max(need)), -5, dtype=torch.int32)
            at = 0
            for b, c in enumerate(need):
                self.table[b, :c] = perm[at:at + c]
                at += c
            shape = (sum(need), bs, Hkv, D)
        else:
            self.table, shape = None, (B, Hkv, max(ends) + 3, D)
        self.caches = [torch.randn(*shape, generator=g).to(dtype) for _ in range(2 * layers)]

    def args(self):
        dev = [c.to(DEV) for c in self.caches]
        half = len(dev) // 2
        return dict(draft_tokens=self.tokens.to(DEV), parents=self.parents.to(DEV), choices=self.choices.to(DEV),
                    positions=torch.tensor(self.cached, dtype=torch.int32, device=DEV), k_caches=dev[:half], v_caches=dev[half:],
                    block_table=self.table.to(DEV) if self.table is not None else None,
                    tree_lens=torch.tensor(self.n, dtype=torch.int32, device=DEV))

    def expect(self):
        paths = [walk(self.tokens[b].tolist(), self.parents[b].tolist(), self.choices[b].tolist(), self.n[b]) for b in range(self.B)]
        caches = [c.clone() for c in self.caches]

        def at(b, slot):
            if self.table is None:
                return b, slice(None), slot
            return int(self.table[b, slot // self.bs]), slot % self.bs

        for old, new in zip(self.caches, caches):
            for b, path in enumerate(paths):
                for i, x in enumerate(path):
                    new[at(b, self.cached[b] + i)] = old[at(b, self.cached[b] + x)]
        return paths, caches


def check(R, c, **kw):
    a = c.args()
    a.update(kw)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tokens, kept, nodes, positions = R.rra_tree_keep(**a, err_flag=err)
    paths, caches = c.expect()
    for b, path in enumerate(paths):
        pad = [-1] * (c.N - len(path))
        assert nodes[b].tolist() == path + pad
        assert tokens[b].tolist() == [int(c.choices[b, x]) for x in path] + pad
        assert int(kept[b]) == len(path) and int(positions[b]) == c.cached[b] + len(path)
    for got, want in zip(list(a["k_caches"]) + list(a["v_caches"]), caches):
        assert torch.equal(got.cpu(), want)
    assert int(err) == 0
    return paths


@pytest.mark.parametrize("kind", ["random", "chain", "star", "forest"])
@pytest.mark.parametrize("N,Hkv,D,bs,dtype", [(1, 2, 64, 16, torch.bfloat16), (2, 1, 64, 0, torch.bfloat16),
                                              (9, 3, 128, 4, torch.bfloat16), (33, 8, 128, 16, torch.float32),
                                              (64, 2, 64, 0, torch.float32), (128, 8, 128, 32, torch.bfloat16)])
def test_paths_and_caches(R, N, Hkv, D, bs, dtype, kind):
    paths = check(R, Keep([0, 7, 100, 31], N, Hkv, D, bs, 3, [N, (N + 1) // 2, N, 0], dtype, kind, seed=N, vocab=4))
    if N >= 9 and kind == "random":
        assert any(p != list(range(len(p))) for p in paths)     # (something moves)


def test_a_long_path_over_itself(R):
    """Slots that are written while later ones are still to be read: the path goes through every second node."""
    c = Keep([13], 120, 2, 64, 8, 1, kind="chain")
    for j in range(2, 120):
        c.parents[0, j] = j - 2
    c.parents[0, 1] = -1
    c.tokens[0] = torch.arange(120)
    c.choices[0] = torch.arange(120) + 2
    assert len(check(R, c)[0]) == 60


def test_many_layers_and_a_column_of_choices(R):
    c = Keep([40, 3], 20, 1, 64, 16, 100, seed=5, vocab=3)
    table = torch.full((2, 20, 3), -1, dtype=torch.int32, device=DEV)
    table[..., 0] = c.choices.to(DEV)
    check(R, c, choices=table[..., 0])
    wide = torch.full((2, 25), -1, dtype=torch.int32, device=DEV)
    wide[:, :20] = c.choices.to(DEV)
    check(R, c, choices=wide[:, :20])
    one = Keep([5, 9], 1, 1, 64, 0, 1)
    check(R, one, choices=one.choices.to(DEV).expand(2, 1))


def test_layers_in_one_tensor(R):
    c = Keep([40, 3, 9], 20, 2, 64, 16, 5, seed=6, vocab=3)
    a = c.args()
    stacked = [torch.stack(a["k_caches"]), torch.stack(a["v_caches"])]
    a["k_caches"], a["v_caches"] = stacked
    R.rra_tree_keep(**a)
    for got, want in zip(list(stacked[0]) + list(stacked[1]), c.expect()[1]):
        assert torch.equal(got.cpu(), want)
    mixed = c.args()
    mixed["k_caches"] = torch.stack(mixed["k_caches"])
    R.rra_tree_keep(**mixed)
    assert torch.equal(mixed["k_caches"], stacked[0]) and all(torch.equal(x, y) for x, y in zip(mixed["v_caches"], stacked[1]))


def test_choices_that_are_no_token(R):
    c = Keep([5], 4, 1, 64, 0, 1)
    c.tokens[:] = -1
    c.choices[:] = -1
    assert check(R, c) == [[0]]


def test_device_errors(R):
    for what, bit in (("position", R.RRA_ERR_POSITION), ("negative", R.RRA_ERR_POSITION), ("len", R.RRA_ERR_SEQ_LEN),
                      ("parent", R.RRA_ERR_TREE), ("block", R.RRA_ERR_BLOCK_ID)):
        c = Keep([20, 40, 60], 9, 2, 64, 16, 2, seed=2, vocab=3)
        paths, caches = c.expect()
        a = c.args()
        if what == "position":
            a["positions"][1] = 2 ** 31 - 1
        elif what == "negative":
            a["positions"][1] = -3
        elif what == "len":
            a["tree_lens"][1] = 10
        elif what == "parent":
            a["parents"][1, 5] = 5
        else:
            a["block_table"][1] = 10 ** 7
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        before = [x.clone() for x in a["k_caches"] + a["v_caches"]]
        tokens, kept, nodes, positions = R.rra_tree_keep(**a, err_flag=err)
        moved = any(i != x for i, x in enumerate(paths[1]))
        assert int(err) == bit or (what == "block" and not moved)
        for b in (0, 2):
            assert nodes[b].tolist()[:len(paths[b])] == paths[b] and int(positions[b]) == c.cached[b] + len(paths[b])
        if bit == R.RRA_ERR_POSITION:
            assert int(positions[1]) == int(a["positions"][1]) and int(kept[1]) == len(paths[1])
        if what in ("position", "negative", "block"):   # the sequence's own rows are where they were
            own = c.table[1][c.table[1] >= 0].long()
            for x, y in zip(before, a["k_caches"] + a["v_caches"]):
                assert torch.equal(x[own.to(DEV)], y[own.to(DEV)])


def test_graph_and_given_outputs(R):
    c = Keep([20, 40, 60], 16, 2, 64, 16, 2, seed=2, vocab=3)
    paths, caches = c.expect()
    a = c.args()
    outs = [torch.empty(3, 16, dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV),
            torch.empty(3, 16, dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)]
    fresh = [x.clone() for x in a["k_caches"] + a["v_caches"]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.rra_tree_keep(**a, tokens_out=outs[0], n_kept=outs[1], nodes_out=outs[2], positions_out=outs[3])
    for _ in range(2):
        for x, y in zip(a["k_caches"] + a["v_caches"], fresh):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert outs[1].tolist() == [len(p) for p in paths]
        for got, want in zip(a["k_caches"] + a["v_caches"], caches):
            assert torch.equal(got.cpu(), want)


# ------------------------------------------------------------------------------------------ the step as a whole
class TinyModel:
    """Two attention layers over caches of their own between random projections: enough of a model to decode with."""

    def __init__(self, Hq, Hkv, D, V, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.Hq, self.Hkv, self.D, self.V, self.width = Hq, Hkv, D, V, 256

        def w(*shape):
            return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float64) * shape[0] ** -0.5

        self.embed = torch.randn(V, self.width, generator=g, device=DEV, dtype=torch.float64)
        self.layers = [[w(self.width, h * D) for h in (Hq, Hkv, Hkv)] + [w(Hq * D, self.width)] for _ in range(2)]
        self.head = w(self.width, V) * 6

    def __call__(self, tokens, attend):
        """Logits of tokens [B, N]; attend(layer, q, k, v) is the cached attention."""
        x = self.embed[tokens.long().clamp(min=0)]
        B, N = tokens.shape
        for i, (wq, wk, wv, wo) in enumerate(self.layers):
            n = x / x.square().mean(-1, keepdim=True).sqrt()
            q, k, v = ((n @ m).to(torch.bfloat16).reshape(B, N, -1, self.D) for m in (wq, wk, wv))
            x = x + attend(i, q, k, v).double().reshape(B, N, -1) @ wo
        return (x / x.square().mean(-1, keepdim=True).sqrt()) @ self.head


@pytest.mark.parametrize("bs", [16, 0])
def test_speculative_steps_follow_the_model(R, bs):
    """Trees of drafted tokens, some of them right: the steps emit the model's choices, and the logits behind them are
    those of decoding the emitted tokens one at a time over caches of their own.

    Tolerance: the two attentions differ by about 2^-8 of their outputs' size per layer, so the logits (of size 6) by some
    6 * 2^-8 * 2 = 0.05, the largest of 50 x 997 differences by 5 times that; a wrong row moves them by their size."""
    B, Hq, Hkv, D, V, N, steps = 3, 8, 2, 64, 997, 12, 6
    m = TinyModel(Hq, Hkv, D, V)
    cols, prompt = 8, [5, 17, 30]
    g = torch.Generator(device=DEV).manual_seed(1)
    shape = (B * cols, bs, Hkv, D) if bs else (B, Hkv, 128, D)
    table = torch.randperm(B * cols, generator=g, device=DEV).int().reshape(B, cols) if bs else None
    ids = [torch.randint(0, V, (n + 1,), generator=g, device=DEV, dtype=torch.int32) for n in prompt]

    def caches():
        return [[torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2)] for _ in m.layers]

    def decode(kv, token, pos):  # logits after one token of each sequence
        return m(token[:, None], lambda i, q, k, v: R.VerifyStep(B, 1, Hq, Hkv, D, *kv[i], table)(q, k, v, pos))[:, 0]

    def prefill(kv):  # every prompt's tokens but the last (shorter prompts: their last token again and again, overwritten later)
        for i in range(max(prompt)):
            at = [min(i, n) for n in prompt]
            decode(kv, torch.stack([ids[b][at[b]] for b in range(B)]), torch.tensor(at, dtype=torch.int32, device=DEV))

    start, last = torch.tensor(prompt, dtype=torch.int32, device=DEV), torch.stack([t[-1] for t in ids])
    kv = caches()
    prefill(kv)
    guess, token = [], last
    for i in range(steps * 6):  # what a good drafter knows
        token = decode(kv, token, start + i).argmax(-1).int()
        guess.append(token.tolist())
    # trees: the guess along a path as far as the drafter would know it, wrong tokens elsewhere
    kv = caches()
    prefill(kv)
    trees = [R.TreeStep(B, N, Hq, Hkv, D, k, v, table) for k, v in kv]
    root, pos = last.clone(), start.clone()
    got, behind = [[] for _ in range(B)], [[] for _ in range(B)]
    gen = torch.Generator().manual_seed(7)
    most = 0
    for _ in range(steps):
        parents = random_parents(B, N, gen)
        draft = torch.randint(0, V, (B, N), generator=gen).int()
        for b in range(B):
            draft[b, 0] = root[b]
            x = 0
            for i in range(int(torch.randint(0, 5, (1,), generator=gen))):
                below = [j for j in range(N) if parents[b, j] == x]
                if not below:
                    break
                x = below[-1]
                draft[b, x] = guess[len(got[b]) + i][b]
        draft, parents = draft.to(DEV), parents.to(DEV)
        logits = m(draft, lambda i, q, k, v: trees[i](q, k, v, pos, parents)).float()
        _, _, top_lp, top = R.rra_token_logprobs(logits, None, 2)
        tokens, kept, nodes, pos = R.rra_tree_keep(draft, parents, top[..., 0], pos, [k for k, v in kv], [v for k, v in kv], table)
        for b in range(B):
            n = int(kept[b])
            most = max(most, n)
            path = nodes[b, :n].long()
            assert tokens[b, :n].tolist() == logits[b, path].argmax(-1).tolist()
            assert (top_lp[b, path, 0] - torch.log_softmax(logits[b, path].double(), -1).amax(-1)).abs().max() < 1e-4
            got[b] += tokens[b, :n].tolist()
            behind[b] += list(logits[b, path])
            root[b] = tokens[b, n - 1]
    assert most >= 3
    assert pos.tolist() == [p + len(x) for p, x in zip(prompt, got)]
    # the emitted tokens one at a time
    kv = caches()
    prefill(kv)
    token = last
    for i in range(max(len(x) for x in got)):
        logits = decode(kv, token, start + i)
        for b in range(B):
            if i < len(got[b]):
                assert float((logits[b] - behind[b][i]).abs().max()) < 0.5, (b, i)
        token = torch.tensor([x[min(i, len(x) - 1)] for x in got], dtype=torch.int32, device=DEV)
    assert all(s.error_bits() == 0 for s in trees)
