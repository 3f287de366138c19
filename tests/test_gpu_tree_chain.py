"""Steps on trees and kept paths one behind the other with no wait between them: each call starts while the one before
it still runs, and reads what that one, or one before that, has moved or written."""

import pytest
import torch

from tests.test_gpu_tree import DEV, Case, check, random_parents

pytestmark = pytest.mark.gpu

STEPS, LAYERS = 20, 2


@pytest.fixture(scope="module")
def R():
    import rope_gqa_paged_gb300 as mod
    from rope_gqa_paged_gb300 import _build
    _build.build()
    return mod


class Chain:
    """STEPS times: the layers' tree steps, then the kept path, whose positions are the next step's. All buffers are
    made beforehand, so that nothing but the library's kernels is enqueued."""

    def __init__(self, R, cached, N, Hq, Hkv, D, bs, seed):
        g = torch.Generator().manual_seed(seed)
        gd = torch.Generator(device=DEV).manual_seed(seed)
        self.R, self.B, B = R, len(cached), len(cached)

        def randn(*shape):
            return torch.randn(*shape, generator=gd, device=DEV, dtype=torch.bfloat16)

        tokens = max(cached) + STEPS * N
        if bs:
            cols = -(-tokens // bs)
            self.table = torch.randperm(B * cols, generator=g).int().reshape(B, cols).to(DEV)
            shape = (B * cols, bs, Hkv, D)
        else:
            self.table, shape, cols = None, (B, Hkv, tokens, D), 0
        self.fresh = [randn(*shape) for _ in range(2 * LAYERS)]
        self.caches = [x.clone() for x in self.fresh]
        self.inputs = [[(randn(B, N, Hq, D), randn(B, N, Hkv, D), randn(B, N, Hkv, D)) for _ in range(LAYERS)] for _ in range(STEPS)]
        self.trees = []
        for _ in range(STEPS):
            parents = random_parents(B, N, g)
            draft, choices = (torch.randint(0, 4, (B, N), generator=g).int() for _ in range(2))
            self.trees.append([x.contiguous().to(DEV) for x in (parents, draft, choices)])
        self.positions = [torch.tensor(cached, dtype=torch.int32, device=DEV)] + [torch.zeros(B, dtype=torch.int32, device=DEV)
                                                                                 for _ in range(STEPS)]
        self.out = [[torch.zeros(B, N, Hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(LAYERS)] for _ in range(STEPS)]
        self.q_rot = [torch.zeros_like(x) for x in self.out[0]]
        self.kept = [[torch.zeros(B, N, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV),
                      torch.zeros(B, N, dtype=torch.int32, device=DEV)] for _ in range(STEPS)]
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = R.rra_tree_plan(B, N, Hq, Hkv, D, cols * bs or tokens, bs)[1]
        self.ws = torch.empty(ws, dtype=torch.uint8, device=DEV) if ws else None

    def run(self, between=lambda: None):
        k, v = self.caches[:LAYERS], self.caches[LAYERS:]
        for i in range(STEPS):
            parents, draft, choices = self.trees[i]
            for layer in range(LAYERS):
                self.R.rra_tree_step(*self.inputs[i][layer], self.positions[i], parents, self.q_rot[layer], k[layer], v[layer],
                                     self.out[i][layer], self.table, workspace=self.ws, err_flag=self.err)
                between()
            tokens, kept, nodes = self.kept[i]
            self.R.rra_tree_keep(draft, parents, choices, self.positions[i], k, v, self.table, None, tokens, kept, nodes,
                                 self.positions[i + 1], self.err)
            between()

    def reset(self):
        for x, y in zip(self.caches, self.fresh):
            x.copy_(y)
        for x in [o for step in self.out for o in step] + [o for step in self.kept for o in step] + self.positions[1:]:
            x.zero_()
        torch.cuda.synchronize()

    def results(self):
        torch.cuda.synchronize()
        assert int(self.err) == 0
        return [x.clone() for x in [o for step in self.out for o in step] + [o for step in self.kept for o in step] +
                self.positions + self.caches]


CHAINS = [
    # cached tokens, N, Hq, Hkv, D, block (0: contiguous)
    ([0, 3, 40, 11], 8, 32, 8, 128, 16),        # a few key tiles: the kernels are as short as they come
    ([600], 26, 32, 8, 128, 16),                # many runs of one unit, merged
    ([500, 90, 1400, 7, 260, 33, 800], 20, 8, 2, 64, 8),
    ([700, 2100], 64, 32, 8, 128, 32),          # two row tiles
    ([300, 5, 1200], 24, 16, 16, 128, 0),       # every head its own keys, contiguous
]


@pytest.mark.parametrize("shape", CHAINS, ids=[f"{i}" for i in range(len(CHAINS))])
def test_steps_and_kept_paths_without_a_wait(R, shape):
    """Bit for bit what the same calls give with a wait behind each; and as one graph."""
    c = Chain(R, *shape, seed=len(shape[0]))
    c.reset()
    c.run(torch.cuda.synchronize)
    want = c.results()
    assert any(not torch.equal(nodes, torch.where(nodes >= 0, torch.arange(nodes.shape[1], device=DEV), -1))
               for _, _, nodes in c.kept)       # (rows move)
    for _ in range(3):
        c.reset()
        c.run()
        assert all(torch.equal(x, y) for x, y in zip(c.results(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(3):
        c.reset()
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(c.results(), want))


def test_the_batch_in_another_order(R):
    """Sequences in another order are cut at other places: each one's rows are within the tolerance all the same."""
    c = Case([700, 3, 1500, 40, 90, 2000, 256], 30, 32, 8, 128, 16, [30, 0, 11, 30, 29, 7, 30], seed=8)
    want, mag = c.expect()
    check(c, c.attend(R)[0], want, mag)
    for order in ([6, 5, 4, 3, 2, 1, 0], [2, 0, 5, 6, 1, 3, 4]):
        o = torch.tensor(order, device=DEV)
        out = torch.full_like(c.q, float("nan"))
        R.rra_tree_attn(c.q[o], c.k, c.v, c.positions[o], c.parents[o], out, c.table[o], c.lens[o], workspace=c.workspace(R))
        back = torch.empty_like(out)
        back[o] = out
        check(c, back, want, mag, str(order))
