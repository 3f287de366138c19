"""The shared-prefix attention and the draft acceptance, as their users call them: what is measured.

``run`` computes the plain form (torch operations in 32 or 64 bits) while ``own`` is false, and the
library's calls while it is true. A case's lengths follow from the case alone; the seed draws the
values, which sequence has which length, and the physical order of the blocks.
"""

import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------ cases
def _attn(name, B, gamma, Hq, Hkv, D, bs, prefix, lo, hi, pad=0):
    """B sequences: `prefix` common tokens, then lo .. hi tokens of their own (the gamma new ones
    among them); the last `pad` rows of the batch are empty (length 0)."""
    return dict(name=name, op="attn", B=B, gamma=gamma, Hq=Hq, Hkv=Hkv, D=D, bs=bs, prefix=prefix, lo=lo, hi=hi, pad=pad)


def _draft(name, B, gamma, V, dtype, drafter, ragged):
    return dict(name=name, op="draft", B=B, gamma=gamma, V=V, dtype=dtype, drafter=drafter, ragged=ragged)


def listed():
    return [
        # the first tokens of four answers behind a short system prompt: latency is what counts
        _attn("decode_first_tokens", 4, 1, 32, 8, 128, 16, 512, 1, 40),
        # the repository's prefix sweep (2048 of 8192 tokens shared): grouped, multi-query, multi-head
        _attn("decode_sweep_kv8", 16, 1, 32, 8, 128, 16, 2048, 6144, 6144),
        _attn("decode_sweep_kv1", 16, 1, 32, 1, 128, 16, 2048, 6144, 6144),
        _attn("decode_sweep_kv32", 16, 1, 32, 32, 128, 16, 2048, 6144, 6144),
        # many questions about one long document
        _attn("decode_long_prompt", 64, 1, 32, 8, 128, 16, 32768, 1, 1024),
        # a large batch of short answers behind a long instruction: the largest arithmetic
        _attn("decode_large_batch", 512, 1, 32, 8, 128, 32, 16384, 1, 256),
        # four drafted tokens a sequence, ragged, with padding rows as a captured graph of fixed batch has
        _attn("verify_drafts", 48, 4, 32, 8, 128, 16, 8192, 5, 1500, pad=3),
        # head dim 64, seven query heads a group, blocks of 8, a prefix that ends inside a tile
        _attn("verify_odd_heads", 21, 3, 42, 6, 64, 8, 1000, 3, 700),
        # one user: four drafted tokens, a small vocabulary
        _draft("draft_one", 1, 4, 32000, "f32", True, False),
        # a serving batch, a large vocabulary
        _draft("draft_batch", 64, 4, 128000, "f32", True, False),
        # a drafter without probabilities (a lookup of repeated text); an odd vocabulary
        _draft("draft_lookup", 32, 3, 50001, "f32", False, True),
        # a large batch, bf16 probabilities, drafts of 0 to 7 tokens; an odd vocabulary
        _draft("draft_large", 256, 7, 100003, "bf16", True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.35:
        gamma = rng.randint(1, 8)
        return dict(op="draft", B=_log(rng, 1, 200), gamma=gamma, V=_log(rng, 500, 130000),
                    dtype=rng.choice(["f32", "bf16"]), drafter=rng.random() < 0.75, ragged=rng.random() < 0.5)
    while True:
        gamma = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        Hkv = rng.choice([1, 2, 3, 4, 6, 8, 16])
        n_rep = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        D = rng.choice([64, 128, 128])
        bs = rng.choice([8, 16, 16, 32, 64, 128])
        prefix = max(bs, _log(rng, 128, 40000) // bs * bs)
        B = _log(rng, 1, 300)
        hi = _log(rng, gamma + 1, 4000)
        lo = rng.randint(gamma, hi)
        c = dict(op="attn", B=B, gamma=gamma, Hq=Hkv * n_rep, Hkv=Hkv, D=D, bs=bs, prefix=prefix, lo=lo, hi=hi,
                 pad=rng.randint(0, B // 4))
        w = work(c)
        if w["flops"] <= 1.2e11 and w["bytes"] <= 1.6e9 and c["B"] * gamma * c["Hq"] * (prefix + hi) <= 2.5e8:
            return c


def _own_tokens(c):
    """Tokens of their own of the B - pad sequences that are not empty (evenly spread over lo .. hi)."""
    n = c["B"] - c["pad"]
    return [c["lo"] + (c["hi"] - c["lo"]) * i // max(1, n - 1) for i in range(n)]


def work(case):
    if case["op"] == "attn":
        c = case
        own_tokens = _own_tokens(c)
        kv = 2 * 2 * c["Hkv"] * c["D"] * (c["prefix"] + sum(own_tokens))
        rows = 2 * 2 * c["B"] * c["gamma"] * c["Hq"] * c["D"]
        tables = 4 * (c["prefix"] + sum(own_tokens)) // c["bs"]
        seen = sum((c["prefix"] + s - c["gamma"] + 1 + j) for s in own_tokens for j in range(c["gamma"]))
        return {"bytes": kv + rows + tables, "flops": 4 * c["D"] * c["Hq"] * seen}
    # one row of the target's probabilities, and one of the drafter's where a token is rejected
    # (the inputs are drawn so that about three tokens of four are kept)
    e = 2 if case["dtype"] == "bf16" else 4
    rows = 1 + (1 - 0.75 ** case["gamma"] if case["drafter"] else 0)
    elems = case["B"] * case["V"] * rows
    return {"bytes": int(elems * e), "flops": int(3 * elems)}


# ----------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (_prepare_attn if case["op"] == "attn" else _prepare_draft)(case, gen)


def _prepare_attn(c, gen):
    B, g, bs, P = c["B"], c["gamma"], c["bs"], c["prefix"]
    order = torch.randperm(B, generator=gen, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    own_tokens = torch.tensor(_own_tokens(c), dtype=torch.int32, device=DEV)
    lens[order[:len(own_tokens)]] = P + own_tokens if len(own_tokens) else own_tokens
    cols = -(-(P + c["hi"]) // bs)
    own_cols = cols - P // bs
    blocks = P // bs + B * own_cols
    perm = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
    prefix_blocks = perm[:P // bs].contiguous()
    table = torch.cat([prefix_blocks.expand(B, -1), perm[P // bs:].reshape(B, own_cols)], 1)
    used = torch.arange(cols, device=DEV) * bs < lens[:, None]
    table = torch.where(used, table, -1).contiguous()      # entries past a sequence's end are unset
    pool = (blocks, bs, c["Hkv"], c["D"])
    s = dict(case=c, lens=lens, prefix_blocks=prefix_blocks, table=table, max_len=cols * bs,
             q=torch.randn(B, g, c["Hq"], c["D"], generator=gen, device=DEV, dtype=torch.bfloat16),
             k=torch.randn(pool, generator=gen, device=DEV, dtype=torch.bfloat16),
             v=torch.randn(pool, generator=gen, device=DEV, dtype=torch.bfloat16))
    if own:  # what a program allocates once: the output and the split workspace
        import rope_gqa_paged_gb300 as rra
        s["out"] = torch.empty_like(s["q"])
        need = rra.rra_shared_prefix_plan(B, g, c["Hq"], c["Hkv"], c["D"], P, cols, bs)[2]
        s["workspace"] = torch.zeros(max(need, 1), dtype=torch.uint8, device=DEV)
    return s


def _prepare_draft(c, gen):
    B, g, V = c["B"], c["gamma"], c["V"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    logits = torch.randn(B, g + 1, V, generator=gen, device=DEV).mul_(2.5)
    p = torch.softmax(logits, -1).to(dt)
    if c["drafter"]:  # a drafter that is near the target
        q = torch.softmax(logits[:, :g].add_(torch.randn(B, g, V, generator=gen, device=DEV).mul_(0.55)), -1).to(dt)
        x = torch.multinomial(q.float().reshape(B * g, V), 1, generator=gen).reshape(B, g)
    else:             # looked-up tokens: mostly likely ones, each a token that the target may have said
        q = None
        x = torch.multinomial(p[:, :g].float().reshape(B * g, V).pow(2.0), 1, generator=gen).reshape(B, g)
    lens = (rand(B) * (g + 1)).int().clamp_(max=g) if c["ragged"] else None
    return dict(case=c, p=p, q=q, x=x.int().contiguous(), lens=lens, u=rand(B, g), u_last=rand(B),
                positions=torch.randint(0, 9000, (B,), generator=gen, device=DEV, dtype=torch.int32))


# -------------------------------------------------------------------------------------------- run
def run(state):
    attn = state["case"]["op"] == "attn"
    if own:
        return _own_attn(state) if attn else _own_draft(state)
    return _plain_attn(state) if attn else _plain_draft(state)


def _own_attn(s):
    import rope_gqa_paged_gb300 as rra
    rra.rra_shared_prefix_attn(s["q"], s["k"], s["v"], s["prefix_blocks"], s["case"]["prefix"], s["table"], s["lens"],
                               s["out"], workspace=s["workspace"])
    return s["out"]


def _own_draft(s):
    import rope_gqa_paged_gb300 as rra
    return rra.rra_accept_draft(s["p"], s["x"], s["u"], s["u_last"], draft_probs=s["q"], draft_lens=s["lens"],
                                positions=s["positions"])


def _plain_attn(s):
    c = s["case"]
    B, g, Hq, Hkv, D, bs, P = (c[k] for k in ("B", "gamma", "Hq", "Hkv", "D", "bs", "prefix"))
    rep, pb = Hq // Hkv, P // bs
    q = s["q"].float().reshape(B, g, Hkv, rep, D)
    n = (s["lens"][:, None] - g + 1 + torch.arange(g, device=DEV)).clamp(min=0)              # tokens row (b, j) sees
    kp = s["k"][s["prefix_blocks"]].float().reshape(P, Hkv, D)
    vp = s["v"][s["prefix_blocks"]].float().reshape(P, Hkv, D)
    s1 = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(Hkv, B * g * rep, D), kp.permute(1, 2, 0)) * D ** -0.5
    see1 = (torch.arange(P, device=DEV) < n[..., None])[None, :, :, None]                    # [1, B, g, 1, P]
    s1 = s1.reshape(Hkv, B, g, rep, P).masked_fill(~see1, -math.inf)
    tab = s["table"][:, pb:].clamp(min=0)
    ks = s["k"][tab].float().reshape(B, -1, Hkv, D)
    vs = s["v"][tab].float().reshape(B, -1, Hkv, D)
    S = ks.shape[1]
    s2 = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(Hkv, B, g * rep, D), ks.permute(2, 0, 3, 1)) * D ** -0.5
    see2 = (P + torch.arange(S, device=DEV) < n[..., None])[None, :, :, None]
    s2 = s2.reshape(Hkv, B, g, rep, S).masked_fill(~see2, -math.inf)
    m = torch.maximum(s1.amax(-1), s2.amax(-1))[..., None]
    m = torch.where(torch.isinf(m), 0.0, m)
    e1, e2 = (s1 - m).exp_(), (s2 - m).exp_()
    total = e1.sum(-1) + e2.sum(-1)
    o = torch.matmul(e1.reshape(Hkv, B * g * rep, P), vp.permute(1, 0, 2)).reshape(Hkv, B, g, rep, D)
    o = o + torch.matmul(e2.reshape(Hkv, B, g * rep, S), vs.permute(2, 0, 1, 3)).reshape(Hkv, B, g, rep, D)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    return o.permute(1, 2, 0, 3, 4).reshape(B, g, Hq, D).to(torch.bfloat16)


def _plain_draft(s):
    p, q, x = s["p"], s["q"], s["x"].long()
    B, g = x.shape
    V = p.shape[-1]
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), g, device=DEV)
    px = p[:, :g].gather(2, x[..., None])[..., 0].double()
    qx = q.gather(2, x[..., None])[..., 0].double() if q is not None else torch.ones_like(px)
    keep = (s["u"].double() * qx < px) & (torch.arange(g, device=DEV) < lens[:, None])
    n = keep.long().cumprod(1).sum(1)
    row = torch.arange(B, device=DEV)
    pn = p[row, n].double()
    at = n.clamp(max=g - 1)
    if q is not None:
        qn = q[row, at].double()
    else:
        qn = torch.zeros_like(pn).scatter_(1, x[row, at][:, None], math.inf)
    rest = torch.where((n < lens)[:, None], (pn - qn).clamp(min=0), pn)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, pn)
    cum = rest.cumsum(1)
    token = (cum <= s["u_last"].double()[:, None] * cum[:, -1:]).sum(1).clamp(max=V - 1)
    k = torch.arange(g + 1, device=DEV)
    tokens = torch.where(k < n[:, None], torch.nn.functional.pad(x, (0, 1)), torch.where(k == n[:, None], token[:, None], -1))
    return tokens.int(), n.int(), (s["positions"] + n + 1).int()


# ------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """The attention in 64 bits, one sequence after the other over its own table (a draft's outputs are whole numbers)."""
    if case["op"] != "attn":
        return None
    s = prepare(case, seed)
    c = s["case"]
    B, g, Hq, Hkv, D, bs = (c[k] for k in ("B", "gamma", "Hq", "Hkv", "D", "bs"))
    out = torch.zeros(B, g, Hq, D, dtype=torch.float64, device=DEV)
    for b, L in enumerate(s["lens"].tolist()):
        if L == 0:
            continue
        ids = s["table"][b, :-(-L // bs)].long()
        k = s["k"][ids].reshape(-1, Hkv, D)[:L].double()
        v = s["v"][ids].reshape(-1, Hkv, D)[:L].double()
        qb = s["q"][b].double().reshape(g, Hkv, Hq // Hkv, D)
        w = torch.einsum("jhrd,thd->jhrt", qb, k) / math.sqrt(D)
        hidden = torch.arange(L, device=DEV)[None, :] > L - g + torch.arange(g, device=DEV)[:, None]
        w = torch.softmax(w.masked_fill(hidden[:, None, None, :], -math.inf), -1)
        out[b] = torch.einsum("jhrt,thd->jhrd", w, v).reshape(g, Hq, D)
    return out
