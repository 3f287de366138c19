"""Calls on a stream that is not the current one: what a call makes or copies by itself is of the call's stream, and
nothing of it waits for the current stream. In every test the current stream is kept busy meanwhile."""

import pytest
import torch

from tests.test_gpu_tree import DEV, Case
from tests.test_gpu_tree import check as check_tree
from tests.test_gpu_tree_keep import Keep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    import rope_gqa_paged_gb300 as mod
    from rope_gqa_paged_gb300 import _build
    _build.build()
    return mod


class Busy:
    """The current stream kept busy (a tenth of a second) from here on; ``still()``: whether it still is."""

    def __init__(self):
        torch.cuda._sleep(200_000_000)
        self.end = torch.cuda.Event()
        self.end.record()

    def still(self):
        return not self.end.query()


def strided(choices, kind):
    B, N = choices.shape
    if kind == "wide":      # rows further apart than N
        x = torch.full((B, N + 5), -1, dtype=torch.int32, device=DEV)[:, :N]
    elif kind == "columns":  # sequences side by side
        x = torch.full((N, B), -1, dtype=torch.int32, device=DEV).t()
    else:                    # a column of each, rows further apart
        x = torch.full((B, N + 2, 3), -1, dtype=torch.int32, device=DEV)[:, :N, 1]
    x.copy_(choices)
    return x


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("kind", ["wide", "columns", "column of wide"])
def test_choices_of_any_stride(R, kind, raw):
    """The copy of choices whose rows are not N steps apart comes before the kernel that reads it, on any stream."""
    c = Keep([40, 3, 77], 20, 2, 64, 16, 3, seed=5, vocab=3)
    paths, caches = c.expect()
    a = c.args()
    a["choices"] = strided(a["choices"], kind)
    s = torch.cuda.Stream()
    first = c.args()   # (kernels are loaded, and memory is taken, at a first call)
    R.rra_tree_keep(**{**first, "choices": strided(first["choices"], kind)}, stream=s)
    torch.cuda.synchronize()
    busy = Busy()
    tokens, kept, nodes, positions = R.rra_tree_keep(**a, stream=s.cuda_stream if raw else s)
    s.synchronize()
    assert busy.still()
    torch.cuda.synchronize()
    assert kept.tolist() == [len(p) for p in paths]
    for b, path in enumerate(paths):
        assert nodes[b, :len(path)].tolist() == path
        assert tokens[b, :len(path)].tolist() == [int(c.choices[b, x]) for x in path]
    for got, want in zip(a["k_caches"] + a["v_caches"], caches):
        assert torch.equal(got.cpu(), want)


def calls(R):
    """Of every call that makes its outputs: the call, given a stream, and what it returns on the current one."""
    g = torch.Generator(device=DEV).manual_seed(0)
    c = Keep([40, 3, 77], 20, 2, 64, 16, 1, seed=6, vocab=3)
    a = c.args()
    a["tree_lens"] = torch.ones_like(a["tree_lens"])  # (one node each: nothing moves, so the call can be repeated)
    logits = torch.randn(6, 5000, generator=g, device=DEV)
    ids = torch.randint(0, 5000, (6, 3), generator=g, device=DEV, dtype=torch.int32)
    probs = torch.softmax(torch.randn(4, 4, 1000, generator=g, device=DEV), -1)
    draft = torch.randint(0, 1000, (4, 3), generator=g, device=DEV, dtype=torch.int32)
    u = torch.rand(4, 4, generator=g, device=DEV)
    ua, us, pos = u[:, :3].contiguous(), u[:, 3].contiguous(), torch.arange(4, dtype=torch.int32, device=DEV)
    at = torch.arange(0, 90, 9, dtype=torch.int32, device=DEV)
    from rope_gqa_paged_gb300 import rra
    return {"keep": lambda s: R.rra_tree_keep(**a, stream=s),
            "logprobs": lambda s: R.rra_token_logprobs(logits, ids, 7, stream=s),
            "accept": lambda s: R.rra_accept_draft(probs, draft, ua, us, positions=pos, stream=s),
            "angles": lambda s: (rra.rra_rope_cos_sin(at, 64, stream=s),)}


@pytest.mark.parametrize("name", ["keep", "logprobs", "accept", "angles"])
def test_outputs_come_from_the_calls_stream(R, name):
    """Memory that was freed on the current stream, which has still to read it, is not what a call on another
    stream writes its outputs to."""
    call = calls(R)[name]
    want = [x.clone() for x in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(s)
    old = [torch.full_like(x, 77) for _ in range(3) for x in want]
    torch.cuda.synchronize()
    busy = Busy()
    read = [x.clone() for x in old]   # (after the busy time)
    del old                           # (back to the current stream's memory)
    got = call(s)
    s.synchronize()
    assert busy.still()
    torch.cuda.synchronize()
    assert all((x == 77).all() for x in read)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("handle", [0, 1, 2])
@pytest.mark.parametrize("name", ["keep", "logprobs", "accept", "angles"])
def test_the_default_streams_by_their_handles(R, name, handle):
    """Handles 0 and 1 are the default stream, 2 the host thread's, whatever the current one is."""
    call = calls(R)[name]
    want = [x.clone() for x in call(None)]
    call(handle)   # (memory of that stream is taken at a first call)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        busy = Busy()
        got = call(handle)
        (torch.cuda.ExternalStream(2) if handle == 2 else torch.cuda.default_stream()).synchronize()
        assert busy.still()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("name", ["keep", "logprobs", "accept"])
def test_captured_on_a_given_stream(R, name):
    call = calls(R)[name]
    want = [x.clone() for x in call(None)]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        got = call(s)
    for _ in range(2):
        for x in got:
            x.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))

def test_tree_attention_and_step(R):
    c = Case([700, 350], 20, 32, 8, 128, 16, seed=12)
    want, mag = c.expect()
    ws, err, out = c.workspace(R), torch.zeros(1, dtype=torch.int32, device=DEV), torch.full_like(c.q, float("nan"))
    step = R.TreeStep(c.B, c.N, 32, 8, 128, c.k.clone(), c.v.clone(), c.table)
    first = step(c.q, c.k_new, c.v_new, c.positions, c.parents).clone()
    step.out.fill_(float("nan"))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.attend(R, ws=ws, out=out, err=err, stream=s)
    torch.cuda.synchronize()
    out.fill_(float("nan"))
    torch.cuda.synchronize()
    busy = Busy()
    c.attend(R, ws=ws, out=out, err=err, stream=s)
    step(c.q, c.k_new, c.v_new, c.positions, c.parents, stream=s)
    s.synchronize()
    assert busy.still()
    torch.cuda.synchronize()
    check_tree(c, out, want, mag)
    assert torch.equal(step.out, first)
    assert int(err) == step.error_bits() == 0
