"""rra_tree_keep on caches that layers share."""

import pytest
import torch

from tests.test_gpu_tree import DEV
from tests.test_gpu_tree_keep import Keep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    import rope_gqa_paged_gb300 as mod
    from rope_gqa_paged_gb300 import _build
    _build.build()
    return mod


@pytest.mark.parametrize("bs", [0, 16])
@pytest.mark.parametrize("share", ["pairs", "all", "keys only", "keys are values"])
def test_layers_that_share_a_cache(R, bs, share):
    """A cache that stands in the lists more than once moves once. The path goes through every second node, so that a
    row moved twice is another one's."""
    N, layers = 120, 6
    c = Keep([13, 70], N, 2, 64, bs, layers, kind="chain", seed=1)
    c.parents[:, 2:] = torch.arange(N - 2).int()
    c.parents[:, 1] = -1
    c.tokens[:] = torch.arange(N).int()
    c.choices[:] = torch.arange(N).int() + 2
    paths, caches = c.expect()
    assert [len(p) for p in paths] == [60, 60]
    a = c.args()
    own = a["k_caches"] + a["v_caches"]
    k, v = list(a["k_caches"]), list(a["v_caches"])
    if share == "pairs":               # layers 2i and 2i + 1
        k, v = [k[i - i % 2] for i in range(layers)], [v[i - i % 2] for i in range(layers)]
    elif share == "all":
        k, v = [k[0]] * layers, [v[0]] * layers
    elif share == "keys only":         # (an odd number of caches: one of keys, six of values)
        k = [k[3]] * layers
    else:
        v = k
    used = {x.data_ptr() for x in k + v}
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(20):
        for x, old in zip(own, c.caches):
            x.copy_(old)
        a.update(k_caches=k, v_caches=v)
        tokens, kept, nodes, positions = R.rra_tree_keep(**a, err_flag=err)
        for x, old, moved in zip(own, c.caches, caches):
            assert torch.equal(x.cpu(), moved if x.data_ptr() in used else old)
    assert nodes[:, :60].tolist() == paths and int(err) == 0


def test_caches_that_overlap_are_refused(R):
    c = Keep([5, 9], 4, 1, 64, 8, 2)
    a = c.args()
    pool = torch.zeros(len(a["k_caches"][0]) + 1, *a["k_caches"][0].shape[1:], dtype=torch.bfloat16, device=DEV)
    a["k_caches"][1], a["v_caches"][0] = pool[1:], pool[:-1]
    with pytest.raises(R.RraError):
        R.rra_tree_keep(**a)
    a["k_caches"][1] = pool[:-1]
    R.rra_tree_keep(**a)
