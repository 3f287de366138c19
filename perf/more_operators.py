"""A speculative step on a tree of drafted tokens, as its users call it: what is measured.

Three operators follow one another there: the tree's attention over the cache (``tree``), the log
probabilities of its logits with entropies and top alternatives (``logprobs``), and the accepted path, whose
keys and values move together (``keep``). ``run`` computes the plain form (torch operations in 32 or 64 bits)
while ``own`` is false, and the library's calls while it is true. A case's lengths follow from the case alone;
the seed draws the values, the trees, which sequence has which length, and the physical order of the blocks.
"""

import math

import torch

own = False

DEV = "cuda"
BASE = 10000.0  # of the rotary positions


# ------------------------------------------------------------------------------------------ cases
def _tree(name, B, N, Hq, Hkv, D, bs, lo, hi, ragged=False, pad=0):
    """B sequences of lo .. hi cached tokens, each with a tree of N nodes (`ragged`: N/2 .. N nodes; the last
    `pad` rows of the batch have none); bs 0: a contiguous cache."""
    return dict(name=name, op="tree", B=B, N=N, Hq=Hq, Hkv=Hkv, D=D, bs=bs, lo=lo, hi=hi, ragged=ragged, pad=pad)


def _logprobs(name, rows, T, V, k, dtype, masked=0.0):
    """`rows` rows of V logits, T given tokens and k alternatives each; a share `masked` of the logits is -inf."""
    return dict(name=name, op="logprobs", rows=rows, T=T, V=V, k=k, dtype=dtype, masked=masked)


def _keep(name, B, N, kept, layers, Hkv, D, bs, hi):
    """B sequences of up to hi cached tokens whose trees of N nodes keep 1 .. `kept` nodes, in the caches of `layers` layers."""
    return dict(name=name, op="keep", B=B, N=N, kept=kept, layers=layers, Hkv=Hkv, D=D, bs=bs, hi=hi)


def listed():
    return [
        # the first steps of a few short answers: latency is what counts
        _tree("tree_first_steps", 4, 8, 32, 8, 128, 16, 0, 40),
        # one user in the middle of a conversation, a tree of a common size
        _tree("tree_one_user", 1, 26, 32, 8, 128, 16, 4000, 4000),
        # one user over a long document
        _tree("tree_long_context", 1, 64, 32, 8, 128, 32, 131000, 131000),
        # a serving batch of ragged lengths, small trees: the cache's bytes are what counts
        _tree("tree_batch", 64, 16, 32, 8, 128, 16, 500, 8000),
        # larger trees, ragged, with padding rows as a captured graph of fixed batch has: the largest arithmetic
        _tree("tree_batch_large", 32, 60, 32, 8, 128, 16, 1000, 8000, ragged=True, pad=2),
        # head dim 64, seven query heads a group, blocks of 8, odd everything
        _tree("tree_odd_heads", 21, 13, 42, 6, 64, 8, 3, 2900, ragged=True, pad=1),
        # every head with keys of its own, a contiguous cache of an odd capacity
        _tree("tree_multi_head", 8, 24, 32, 32, 128, 0, 700, 4090),
        # one answer's next token with five alternatives; a small vocabulary
        _logprobs("logprobs_one", 1, 1, 32000, 5, "f32"),
        # the nodes of a batch's trees: the target's choice at each, and the log probability of one token
        _logprobs("logprobs_tree", 1024, 1, 128000, 1, "bf16"),
        # a prompt scored: an odd vocabulary, a grammar that forbids a part of it, eight alternatives
        _logprobs("logprobs_prompt", 4000, 2, 100003, 8, "f32", masked=0.3),
        # one user's path in the caches of every layer
        _keep("keep_one", 1, 26, 5, 32, 8, 128, 16, 4000),
        # a serving batch's
        _keep("keep_batch", 64, 32, 6, 32, 8, 128, 16, 120),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    x = rng.random()
    if x < 0.3:
        while True:
            c = dict(op="logprobs", rows=_log(rng, 1, 4000), T=rng.randint(1, 4), V=_log(rng, 1000, 160000),
                     k=rng.randint(1, 20), dtype=rng.choice(["f32", "bf16"]), masked=rng.choice([0.0, 0.0, 0.5, 0.99]))
            if c["rows"] * c["V"] <= 4e8:
                return c
    if x < 0.5:
        kept = rng.randint(1, 9)
        return dict(op="keep", B=_log(rng, 1, 80), N=rng.randint(2 * kept, 64), kept=kept, layers=_log(rng, 1, 40),
                    Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 128]), bs=rng.choice([0, 8, 16, 16, 32, 64]),
                    hi=rng.randint(0, 200))
    while True:
        N = _log(rng, 1, 96)
        Hkv = rng.choice([1, 2, 3, 4, 6, 8, 16])
        n_rep = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        B = _log(rng, 1, 100)
        hi = _log(rng, 1, 40000)
        c = dict(op="tree", B=B, N=N, Hq=Hkv * n_rep, Hkv=Hkv, D=rng.choice([64, 128, 128]),
                 bs=rng.choice([0, 8, 16, 16, 32, 64, 128]), lo=rng.randint(0, hi), hi=hi, ragged=rng.random() < 0.5,
                 pad=rng.randint(0, B // 4))
        w = work(c)
        cells = B * (hi + N)  # (a contiguous cache holds the longest sequence's length for every sequence)
        if (w["flops"] <= 1.1e11 and w["bytes"] <= 1.1e9 and cells * Hkv * c["D"] <= 3e8 and cells * N * c["Hq"] <= 5e8):
            return c


# The lengths of the B - pad sequences that have a tree, the nodes of their trees, the nodes that are kept.
def _cached(c):
    n = c["B"] - c["pad"]
    return [c["lo"] + (c["hi"] - c["lo"]) * i // max(1, n - 1) for i in range(n)]


def _nodes(c):
    n, low = c["B"] - c["pad"], (c["N"] + 1) // 2 if c["ragged"] else c["N"]
    return [low + (c["N"] - low) * (i * 7 % n) // max(1, n - 1) for i in range(n)]


def _kept(c):
    return [1 + (i + c["kept"] - 1) % c["kept"] for i in range(c["B"])]


def work(case):
    c = case
    if c["op"] == "tree":
        cached, nodes = _cached(c), _nodes(c)
        kv = 2 * 2 * c["Hkv"] * c["D"] * sum(cached)
        # a node: q read, rotated q and the output written, its own k and v read and written
        rows = 2 * c["D"] * (3 * c["Hq"] + 4 * c["Hkv"]) * sum(nodes)
        tables = 4 * sum(cached) // c["bs"] if c["bs"] else 0
        seen = sum(n * (p + 2) for p, n in zip(cached, nodes))  # (a node sees itself and its ancestors)
        return {"bytes": kv + rows + tables, "flops": 4 * c["D"] * c["Hq"] * seen}
    if c["op"] == "logprobs":
        e = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": c["rows"] * (c["V"] * e + 8 * c["T"] + 4 + 8 * c["k"]), "flops": 6 * c["rows"] * c["V"]}
    moved = sum(n - 1 for n in _kept(c))  # each key and value row read and written once (a copy: no arithmetic but the search's)
    return {"bytes": 2 * moved * c["layers"] * 2 * 2 * c["Hkv"] * c["D"] + 20 * c["B"] * c["N"], "flops": 3 * c["B"] * c["N"]}


# ----------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return {"tree": _prepare_tree, "logprobs": _prepare_logprobs, "keep": _prepare_keep}[case["op"]](case, gen)


def _parents(B, N, gen):
    """Random trees: node 0 the root, every other node below an earlier one, mostly an early one."""
    at = torch.arange(N, device=DEV)
    return torch.where(at > 0, (torch.rand(B, N, generator=gen, device=DEV).square() * at).long(), -1).int()


def _table(tokens, bs, gen, most=None):
    """(block table, blocks) for sequences of these many tokens: physical blocks in random order, unset past the end."""
    need = [-(-t // bs) for t in tokens]
    cols = max(1, most if most is not None else max(need))
    perm = torch.randperm(max(1, sum(need)), generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(tokens), cols), -1, dtype=torch.int32)
    table = table.to(DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, max(1, sum(need))


def _bf16(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.bfloat16)


def _prepare_tree(c, gen):
    B, N, Hq, Hkv, D, bs = (c[k] for k in ("B", "N", "Hq", "Hkv", "D", "bs"))
    order = torch.randperm(B, generator=gen, device=DEV).tolist()
    cached, nodes = [0] * B, [0] * B
    for b, p, n in zip(order, _cached(c), _nodes(c)):
        cached[b], nodes[b] = p, n
    s = dict(case=c, positions=torch.tensor(cached, dtype=torch.int32, device=DEV), parents=_parents(B, N, gen),
             lens=torch.tensor(nodes, dtype=torch.int32, device=DEV) if c["ragged"] or c["pad"] else None, table=None)
    if bs:
        s["table"], blocks = _table([p + n for p, n in zip(cached, nodes)], bs, gen)
        shape = (blocks, bs, Hkv, D)
    else:
        shape = (B, Hkv, c["hi"] + N + 1, D)
    s["k"], s["v"] = _bf16(gen, *shape), _bf16(gen, *shape)
    s["q"], s["k_new"], s["v_new"] = _bf16(gen, B, N, Hq, D), _bf16(gen, B, N, Hkv, D), _bf16(gen, B, N, Hkv, D)
    if own:  # the step's object, which a program keeps: its output, workspace and plan
        import rope_gqa_paged_gb300 as rra
        s["step"] = rra.TreeStep(B, N, Hq, Hkv, D, s["k"], s["v"], s["table"], rope_base=BASE)
        s["step"].q_rot.zero_()  # (rows past a tree's nodes are not written)
    return s


def _prepare_logprobs(c, gen):
    R, V = c["rows"], c["V"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    logits = torch.randn(R, V, generator=gen, device=DEV).mul_(2.5)
    tokens = torch.randint(0, V, (R, c["T"]), generator=gen, device=DEV, dtype=torch.int32)
    tokens[:, 0] = torch.where(torch.rand(R, generator=gen, device=DEV) < 0.7, logits.argmax(1).int(), tokens[:, 0])
    if c["masked"]:
        step = max(1, (1 << 28) // V)
        for i in range(0, R, step):
            part = logits[i:i + step]
            part.masked_fill_(torch.rand(part.shape, generator=gen, device=DEV) < c["masked"], -math.inf)
        logits[:, V // 2] = 1.0  # (a grammar leaves something)
    return dict(case=c, logits=logits.to(dt), tokens=tokens)


def _prepare_keep(c, gen):
    B, N, K, bs = c["B"], c["N"], c["kept"], c["bs"]
    order = torch.randperm(B, generator=gen, device=DEV).tolist()
    kept, cached = [0] * B, [0] * B
    for i, (b, n) in enumerate(zip(order, _kept(c))):
        kept[b], cached[b] = n, c["hi"] * (i + 1) // B
    parents = _parents(B, N, gen).cpu()
    # Tokens that differ within a tree. The path's nodes below the root lie past the slots that they move to, so
    # that a pass can be repeated on its own result.
    tokens = torch.randint(0, 1000, (B, N), generator=gen, device=DEV).cpu() * N + torch.arange(N)
    choices = torch.randint(0, 1000, (B, N), generator=gen, device=DEV).cpu() * N + torch.arange(N)  # (no child's token)
    picks = torch.rand(B, N - K, generator=gen, device=DEV).argsort(1).cpu() + K
    for b, n in enumerate(kept):
        path = [0] + sorted(picks[b, :n - 1].tolist())
        for above, node in zip(path, path[1:]):
            parents[b, node] = above
            choices[b, above] = tokens[b, node]
    s = dict(case=c, parents=parents.to(DEV), tokens=tokens.int().to(DEV), choices=choices.int().to(DEV),
             positions=torch.tensor(cached, dtype=torch.int32, device=DEV), table=None)
    if bs:
        s["table"], blocks = _table([p + N for p in cached], bs, gen)
        shape = (blocks, bs, c["Hkv"], c["D"])
    else:
        shape = (B, c["Hkv"], c["hi"] + N, c["D"])
    s["k"], s["v"] = _bf16(gen, c["layers"], *shape), _bf16(gen, c["layers"], *shape)  # every layer's cache
    return s


# -------------------------------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "logprobs": _own_logprobs, "keep": _own_keep}[op](state)
    return {"tree": _plain_tree, "logprobs": _plain_logprobs, "keep": _plain_keep}[op](state)


def _own_tree(s):
    out = s["step"](s["q"], s["k_new"], s["v_new"], s["positions"], s["parents"], s["lens"])
    return out, s["step"].q_rot, s["k"], s["v"]


def _own_logprobs(s):
    import rope_gqa_paged_gb300 as rra
    return rra.rra_token_logprobs(s["logits"], s["tokens"], top_k=s["case"]["k"])


def _own_keep(s):
    import rope_gqa_paged_gb300 as rra
    tokens, kept, nodes, positions = rra.rra_tree_keep(s["tokens"], s["parents"], s["choices"], s["positions"],
                                                       list(s["k"]), list(s["v"]), s["table"])
    return tokens, kept, nodes, positions, s["k"], s["v"]


def _ancestors(parents):
    """sees[b, i, j]: node j is node i or one of its ancestors; and the nodes' depths."""
    B, N = parents.shape
    sees = torch.zeros(B, N, N, dtype=torch.bool, device=parents.device)
    row, up = torch.arange(B, device=parents.device), parents.long()
    for i in range(N):
        if i:
            sees[:, i] = sees[row, up[:, i].clamp(min=0)] & (up[:, i] >= 0)[:, None]
        sees[:, i, i] = True
    return sees, sees.sum(2) - 1


def _rotated(x, at):
    """x [B, N, H, D] in float64, pair (i, i + D/2) turned by at[b, n] * BASE^(-2i/D)."""
    D = x.shape[-1]
    theta = BASE ** (-torch.arange(0, D, 2, device=x.device, dtype=torch.float64) / D)
    a = at.double()[..., None, None] * theta
    x = x.double()
    x1, x2 = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([x1 * a.cos() - x2 * a.sin(), x2 * a.cos() + x1 * a.sin()], -1)


def _slots(cache, table, b, at):
    """Index of the cache rows of tokens `at` of sequences `b` (tensors of one shape)."""
    if table is None:
        return b, slice(None), at
    bs = cache.shape[1]
    return table[b, at // bs].long(), at % bs


def _plain_tree(s):
    c = s["case"]
    B, N, Hq, Hkv, D, bs = (c[k] for k in ("B", "N", "Hq", "Hkv", "D", "bs"))
    p = s["positions"].long()
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), N, device=DEV)
    sees, depth = _ancestors(s["parents"])
    at = torch.arange(N, device=DEV)
    live = at < lens[:, None]
    q_rot = torch.where(live[..., None, None], _rotated(s["q"], p[:, None] + depth).to(torch.bfloat16), 0)
    b, j = live.nonzero(as_tuple=True)
    where = _slots(s["k"], s["table"], b, p[b] + j)
    s["k"][where] = _rotated(s["k_new"], p[:, None] + depth).to(torch.bfloat16)[b, j]
    s["v"][where] = s["v_new"][b, j]
    S = c["hi"] + N
    t = torch.arange(S, device=DEV)
    if s["table"] is not None:
        cols = s["table"].shape[1]
        ids = s["table"].clamp(min=0).long()
        K = s["k"][ids].reshape(B, cols * bs, Hkv, D)[:, :S]
        V = s["v"][ids].reshape(B, cols * bs, Hkv, D)[:, :S]
    else:
        K, V = s["k"][:, :, :S].transpose(1, 2), s["v"][:, :, :S].transpose(1, 2)
    S = K.shape[1]
    t = t[:S]
    rel = t - p[:, None]                                                                    # [B, S]: node of token t
    own_part = sees.gather(2, rel.clamp(0, N - 1)[:, None].expand(B, N, S)) & (rel < lens[:, None])[:, None]
    see = ((rel < 0)[:, None] | own_part) & live[..., None]                                 # [B, N, S]
    rep = Hq // Hkv
    qs = q_rot.float().reshape(B, N, Hkv, rep, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * rep, D)
    w = torch.matmul(qs, K.float().permute(0, 2, 3, 1)).reshape(B, Hkv, N, rep, S) * D ** -0.5
    w.masked_fill_(~see[:, None, :, None], -math.inf)
    m = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(torch.isinf(m), 0.0, m)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.reshape(B, Hkv, N * rep, S), V.float().permute(0, 2, 1, 3)).reshape(B, Hkv, N, rep, D)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(torch.bfloat16), q_rot, s["k"], s["v"]


def _plain_logprobs(s):
    k, V, dev = s["case"]["k"], s["case"]["V"], s["logits"].device
    parts = []
    step = max(1, (1 << 27) // V)
    for i in range(0, s["logits"].shape[0], step):
        x = s["logits"][i:i + step].float()
        m = x.amax(1, keepdim=True)
        d = x - m
        e = d.exp()
        total = e.sum(1, keepdim=True)
        log_total = total.log()
        entropy = log_total[:, 0] - (e * torch.where(e > 0, d, 0.0)).sum(1) / total[:, 0]
        given = d.gather(1, s["tokens"][i:i + step].long()) - log_total
        # the largest values, of equal ones the lowest index first: keys of whole numbers that all differ
        bits = x.view(torch.int32).long()
        bits = torch.where(x == 0, 0, bits)
        key = torch.where(bits < 0, -(bits & 0x7fffffff), bits) * (1 << 31) + (V - 1 - torch.arange(V, device=dev))
        top = V - 1 - (key.topk(k, dim=1).values & 0x7fffffff)
        parts.append((given, entropy, d.gather(1, top) - log_total, top.int()))
    return tuple(torch.cat(p) for p in zip(*parts))


def _plain_keep(s):
    B, N = s["tokens"].shape
    row, at = torch.arange(B, device=DEV), torch.arange(N, device=DEV)
    cur, alive = torch.zeros(B, dtype=torch.long, device=DEV), torch.ones(B, dtype=torch.bool, device=DEV)
    nodes = torch.full((B, N), -1, dtype=torch.long, device=DEV)
    n = torch.zeros(B, dtype=torch.long, device=DEV)
    for i in range(min(N, s["case"]["kept"] + 1)):
        nodes[:, i] = torch.where(alive, cur, -1)
        n += alive
        child = (s["parents"] == cur[:, None]) & (s["tokens"] == s["choices"][row, cur][:, None]) & alive[:, None]
        alive = child.any(1)
        cur = torch.where(child, at, N).amin(1).clamp(max=N - 1)
    kept = at < n[:, None]
    tokens = torch.where(kept, s["choices"].gather(1, nodes.clamp(min=0)), -1)
    b, i = (kept & (nodes != at)).nonzero(as_tuple=True)
    src, dst = s["positions"].long()[b] + nodes[b, i], s["positions"].long()[b] + i
    for cache in [*s["k"], *s["v"]]:
        cache[_slots(cache, s["table"], b, dst)] = cache[_slots(cache, s["table"], b, src)]
    return tokens.int(), n.int(), nodes.int(), (s["positions"] + n).int(), s["k"], s["v"]


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """The attention in 64 bits, one sequence after the other over its own rows, and the log probabilities one
    block of rows after the other (what ``keep`` returns is moved or whole numbers)."""
    c = case
    if c["op"] == "keep":
        return None
    s = prepare(case, seed)
    if c["op"] == "logprobs":
        got = []
        for i in range(0, c["rows"], 64):
            x = s["logits"][i:i + 64].double()
            lp = x - torch.logsumexp(x, 1, keepdim=True)
            h = -torch.where(lp > -math.inf, lp.exp() * lp, 0.0).sum(1)
            got.append((lp.gather(1, s["tokens"][i:i + 64].long()), h, lp.topk(c["k"], dim=1).values))
        given, entropy, top = (torch.cat(p) for p in zip(*got))
        return given, entropy, top, None
    B, N, Hq, Hkv, D = (c[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    turn = 1j * BASE ** (-2.0 * torch.arange(D // 2, device=DEV, dtype=torch.float64) / D)
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device=DEV)
    q_rot, k, v = torch.zeros_like(out), s["k"].double(), s["v"].double()
    lens = s["lens"].tolist() if s["lens"] is not None else [N] * B
    parents = s["parents"].tolist()
    for b, (p, n) in enumerate(zip(s["positions"].tolist(), lens)):
        if n == 0:
            continue
        above = []
        for j in range(n):
            above.append(([] if parents[b][j] < 0 else above[parents[b][j]]) + [j])
        depth = torch.tensor([len(a) - 1 for a in above], device=DEV, dtype=torch.float64)
        hidden = torch.ones(n, p + n, dtype=torch.bool, device=DEV)
        hidden[:, :p] = False
        hidden[[j for j in range(n) for _ in above[j]], [p + a for j in range(n) for a in above[j]]] = False

        def rotated(x):
            z = torch.complex(x[..., :D // 2].double(), x[..., D // 2:].double())
            z = z * torch.exp((p + depth)[:, None, None] * turn)
            return torch.cat([z.real, z.imag], -1)

        q_rot[b, :n] = rotated(s["q"][b, :n])
        new_k, new_v = rotated(s["k_new"][b, :n]), s["v_new"][b, :n].double()
        if s["table"] is not None:
            tok = torch.arange(p + n, device=DEV)
            where = (s["table"][b, tok // c["bs"]].long(), tok % c["bs"])
            k[where[0][p:], where[1][p:]], v[where[0][p:], where[1][p:]] = new_k, new_v
            keys, values = k[where], v[where]
        else:
            k[b, :, p:p + n], v[b, :, p:p + n] = new_k.transpose(0, 1), new_v.transpose(0, 1)
            keys, values = k[b, :, :p + n].transpose(0, 1), v[b, :, :p + n].transpose(0, 1)
        # the attention is of the stored values: rotated queries and keys as bf16 holds them
        qb = q_rot[b, :n].to(torch.bfloat16).double().reshape(n, Hkv, Hq // Hkv, D)
        w = torch.einsum("jhrd,thd->jhrt", qb, keys.to(torch.bfloat16).double()) / math.sqrt(D)
        w = torch.softmax(w.masked_fill(hidden[:, None, None, :], -math.inf), -1)
        out[b, :n] = torch.einsum("jhrt,thd->jhrd", w, values).reshape(n, Hq, D)
    return out, q_rot, k, v
