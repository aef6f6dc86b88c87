"""Workloads of drafted token trees: log probabilities with alternatives, building a tree from them, masked attention of
its tokens over the paged 4-bit cache (whole or through a window with sinks), and acceptance along the tree.

Log probabilities.  z = logits / T of one row, lse = log sum exp z: logp = z[id] - lse of given tokens, the entropy
lse - sum p z, and the K tokens of the largest logits (ties to the lowest id; -1 and -inf where a row has fewer tokens
above -inf) with their logp.

Trees.  A tree has B rows.  Row 0 is the anchor, the last token already decided; every other row is a drafted token with
an earlier row as its parent.  top_ids, top_logp [N][G][K] are the K best tokens of the G positions behind the anchor,
best first.  A row of depth g + 1 takes an alternative of position g, and its score is its parent's plus that
alternative's logp (in 64 bits; the anchor's is 0).  Rows are added best first among the children whose better siblings
are rows already; ties go to the lowest parent, then to the better rank.  mask[i] has the bits of row i and its ancestors.
Rows there are no candidates for: token -1, parent -2, depth 0, mask 0.

Attention.  Row i of a sequence with `len` cached tokens has the position len + depth (in a block without a mask: len + i).
It sees the cached tokens and the own rows that its mask names (without a mask: all), and with a window of W those at
positions p with q - p < W or p < sinks.  A row that sees nothing, as one with an empty mask, is zero; one with an empty
mask sees no cached tokens either.  Cached elements are 4-bit codes with scales of 16, c * s * 2^e: s = max(2^-9,
e4m3(min(448, max|x| 2^-e / 6))), c the nearest e2m1 number to x / (s 2^e), at most 6 in magnitude.

Acceptance.  From the anchor on: the child (the lowest row of several) whose token is the target's token behind the
current row, as long as there is one.  path: the rows passed, the anchor among them, then -1; accept_len of them are
drafted; bonus is the target's token behind the last.

`run` computes the operators in plain torch, or through the package when `own` is true.
"""
import heapq
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GROUP = 16


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # One user's next token with five alternatives, as a serving API returns them.
        dict(name="logprobs_token", op="logprobs", rows=1, V=151936, dt="bf16", M=1, K=5, T=1.0, pad=0, banned=0.0),
        # The alternatives of every drafted position of a batch of 32 blocks of 16 (fp32 logits of the drafter).
        dict(name="logprobs_draft", op="logprobs", rows=480, V=151936, dt="f32", M=1, K=8, T=1.5, pad=0, banned=0.0),
        # Scoring prompts: each prompt token's log probability and the entropy behind it, rows of an odd vocabulary.
        dict(name="logprobs_prompt", op="logprobs", rows=4097, V=201087, dt="bf16", M=1, K=2, T=1.0, pad=2, banned=0.0),
        # One user's tree of 16 rows from a block of 16.
        dict(name="tree_one", op="tree", N=1, G=15, K=4, B=16),
        # Trees of 64 rows for a large batch, from the window of 32 drafted positions.
        dict(name="tree_batch", op="tree", N=256, G=32, K=16, B=64),
        # One user's tree of 16 rows over a short conversation.
        dict(name="tree_attn_one", op="attn", kind="tree", N=1, B=16, Hq=32, Hkv=8, hd=128, page=16, lo=517, hi=517,
             e=0, window=0, sinks=0),
        # A ragged batch: trees of 32 rows over fresh prompts and long documents.
        dict(name="tree_attn_batch", op="attn", kind="tree", N=32, B=32, Hq=32, Hkv=8, hd=128, page=64, lo=65, hi=8000,
             e=0, window=0, sinks=0),
        # The full layers of a model with 64 query heads of 64: trees of 16 over a few very long contexts.
        dict(name="tree_attn_long", op="attn", kind="tree", N=3, B=16, Hq=64, Hkv=8, hd=64, page=32, lo=33333,
             hi=100001, e=0, window=0, sinks=0),
        # Its sliding-window layers, token by token: the last 128 tokens and four sinks, whatever the length.
        dict(name="window_token_batch", op="attn", kind="block", N=48, B=1, Hq=64, Hkv=8, hd=64, page=64, lo=65,
             hi=16000, e=0, window=128, sinks=4),
        # Trees of 16 rows through a window of 4,096 tokens with sinks in long documents.
        dict(name="window_tree_batch", op="attn", kind="tree", N=32, B=16, Hq=32, Hkv=8, hd=128, page=64, lo=1801,
             hi=16000, e=0, window=4096, sinks=16),
        # One user's tree against the target's tokens.
        dict(name="accept_one", op="accept", N=1, G=15, K=4, B=16),
        # A large batch of trees of 64 rows.
        dict(name="accept_batch", op="accept", N=512, G=32, K=16, B=64),
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["logprobs", "logprobs", "logprobs", "tree", "attn", "attn", "attn", "attn", "accept"])
    if op == "logprobs":
        V = logint(50, 201087)
        rows = logint(1, max(1, min(30000, 800000000 // V)))
        return dict(op=op, rows=rows, V=V, dt=rng.choice(["bf16", "f32"]) if rows * V < 400000000 else "bf16",
                    M=rng.randint(1, 4), K=rng.choice([0, 1, rng.randint(2, 8), rng.randint(9, 32)]),
                    T=rng.choice([1.0, round(rng.uniform(0.3, 2.0), 3)]), pad=rng.choice([0, 0, rng.randint(1, 70)]),
                    banned=rng.choice([0.0, 0.0, 0.5, 0.999]))
    if op in ("tree", "accept"):
        return dict(op=op, N=logint(1, 256 if op == "tree" else 512), G=rng.randint(1, 32), K=rng.randint(1, 16),
                    B=rng.randint(2, 64))
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    kind = rng.choice(["tree", "tree", "block"])
    B = rng.choice([1, rng.randint(2, 16), rng.randint(17, 64)])
    # about 4e5 cached tokens and 2e9 score-rows at most
    budget = min(350000 * 8 // Hkv, 3.0e8 / (B * G * Hkv))
    N = logint(1, 64)
    hi = max(1, min(logint(1, 100000), int(budget / N)))
    window = rng.choice([0, logint(1, 8000)]) if kind == "tree" else logint(1, 8000)
    return dict(op=op, kind=kind, N=N, B=B, Hq=G * Hkv, Hkv=Hkv, hd=rng.choice([64, 128]),
                page=rng.choice([16, 32, 48, 64, 128]), lo=rng.randint(0, hi), hi=hi, e=rng.randint(-2, 2),
                window=window, sinks=rng.choice([0, rng.randint(1, 100)]) if window else 0)


def _spread(lo, hi, n):
    """n whole numbers evenly over [lo, hi] (their sum belongs to the case, their order to the seed)."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def work(case):
    op = case["op"]
    if op == "logprobs":
        size = 2 if case["dt"] == "bf16" else 4
        out = case["rows"] * (8 * case["M"] + 4 + 8 * case["K"])
        return {"bytes": case["rows"] * case["V"] * size + out, "flops": 4.0 * case["rows"] * case["V"]}
    N, B = case["N"], case["B"]
    if op == "tree":
        return {"bytes": N * (4 + case["G"] * case["K"] * 8 + B * 20 + 4), "flops": 0.0}
    if op == "accept":
        return {"bytes": N * (B * 16 + 12), "flops": 0.0}
    Hq, Hkv, hd, W, S = (case[k] for k in ("Hq", "Hkv", "hd", "window", "sinks"))
    tok = Hkv * 2 * (hd // 2 + hd // GROUP)          # bytes of one cached token
    lens = _spread(case["lo"], case["hi"], N)
    seen = [n if W == 0 else min(n, W - 1 + min(S, max(0, n - W + 1))) for n in lens]
    return {"bytes": sum(seen) * tok + N * B * ((2 * Hq + 2 * Hkv) * hd * 2 + 8),
            "flops": 4.0 * B * Hq * hd * sum(n + 1 for n in seen)}


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1 + seed * 7919)
    return g


def _ints(x, dtype=torch.int32):
    return torch.as_tensor(x, dtype=dtype).cuda()


def _logits(case, seed):
    """Logits as language models have them: a normal bulk, a few tokens well above it; ids from among them."""
    g = _gen(seed)
    rows, V = case["rows"], case["V"]
    dtype = torch.bfloat16 if case["dt"] == "bf16" else torch.float32
    buf = torch.zeros((rows, V + case["pad"]), dtype=dtype, device="cuda")
    step = max(1, (1 << 27) // V)
    for r in range(0, rows, step):
        z = torch.randn((min(step, rows - r), V), generator=g, device="cuda") * 2.5
        # (six different places of a row: a scatter to one place twice would not depend on the seed alone)
        peak = (torch.randint(0, V, (z.shape[0], 1), generator=g, device="cuda") + torch.arange(6, device="cuda") * (V // 6)) % V
        z.scatter_(1, peak, 8 + 6 * torch.rand(peak.shape, generator=g, device="cuda"))
        if case["banned"]:       # tokens that a grammar or a vocabulary mask forbids
            ban = torch.rand(z.shape, generator=g, device="cuda") < case["banned"]
            z.masked_fill_(ban, -math.inf)
        buf[r:r + z.shape[0], :V] = z
    ids = torch.randint(0, V, (rows, case["M"]), generator=g, device="cuda", dtype=torch.int32)
    return buf[:, :V], ids


def _alternatives(case, seed):
    """Anchor [N], top_ids, top_logp [N][G][K]: confident first positions, flatter ones behind them."""
    g = _gen(seed)
    N, G, K = case["N"], case["G"], case["K"]
    z = torch.randn((N, G, 64), generator=g, device="cuda") * torch.linspace(5.0, 2.0, G, device="cuda")[:, None]
    logp = torch.log_softmax(z, -1).sort(-1, descending=True)[0][:, :, :K].contiguous()
    ids = torch.rand((N, G, 1000), generator=g, device="cuda").argsort(-1)[:, :, :K] * 151 + 7
    return _ints(torch.randint(0, 151936, (N,), generator=g, device="cuda")), ids.int().contiguous(), logp


def _random_trees(case, seed):
    """parent [N][B] (numpy): random trees, in every third sequence with fewer rows than room; -2: no row."""
    rng = np.random.default_rng(seed + 17)
    N, B = case["N"], case["B"]
    parent = np.full((N, B), -2, np.int32)
    for n in range(N):
        count = B if n % 3 else int(rng.integers((B + 1) // 2, B + 1))
        parent[n, 0] = -1
        for i in range(1, count):
            # half of the rows continue the newest path, the others branch off anywhere
            parent[n, i] = i - 1 if rng.random() < 0.5 else rng.integers(0, i)
    return parent


def _masks(parent):
    """(mask int64 [N][B], depth int32 [N][B]) of parents (numpy)."""
    N, B = parent.shape
    mask, depth = np.zeros((N, B), np.uint64), np.zeros((N, B), np.int32)
    for i in range(B):
        p = parent[:, i]
        rows, up = np.arange(N), np.clip(p, 0, None)
        there = p >= -1
        mask[:, i] = np.where(there, np.where(p >= 0, mask[rows, up], np.uint64(0)) | np.uint64(1 << i), np.uint64(0))
        depth[:, i] = np.where(p >= 0, depth[rows, up] + 1, 0)
    return mask.view(np.int64), depth


def _kv_inputs(case, seed):
    """bf16 rows K, V [N][T][Hkv][hd] with outlier channels, as keys and values have them, and the tree's rows."""
    g, rng = _gen(seed), np.random.default_rng(seed)
    N, B, Hq, Hkv, hd = (case[k] for k in ("N", "B", "Hq", "Hkv", "hd"))
    T = max(1, case["hi"])
    scale = torch.exp(0.5 * torch.randn((2, Hkv, hd), generator=g, device="cuda")) * 2.0 ** case["e"]
    K, V = (torch.empty((N, T, Hkv, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for n in range(N):
        K[n] = torch.randn((T, Hkv, hd), generator=g, device="cuda") * scale[0]
        V[n] = torch.randn((T, Hkv, hd), generator=g, device="cuda") * scale[1]
    out = dict(K=K, V=V, lens=rng.permutation(np.array(_spread(case["lo"], case["hi"], N), np.int32)))
    r = lambda h: torch.randn((N, B, h, hd), generator=g, device="cuda")
    out["Q"] = r(Hq).to(torch.bfloat16)
    out["Kb"] = (r(Hkv) * scale[0]).to(torch.bfloat16)
    out["Vb"] = (r(Hkv) * scale[1]).to(torch.bfloat16)
    if case["kind"] == "tree":
        out["parent"] = _random_trees(case, seed)
    max_pages = max(1, -(-case["hi"] // case["page"]))
    out["table"] = rng.permutation(N * max_pages).reshape(N, max_pages).astype(np.int32)
    return out


def _accept_inputs(case, seed):
    """(token, parent [N][B], target [N][B]), all numpy: trees of distinct siblings, targets that agree for a while."""
    rng = np.random.default_rng(seed + 5)
    N, B = case["N"], case["B"]
    parent = _random_trees(case, seed)
    token = np.where(parent >= -1, rng.integers(0, 150000, (N, B)) // 64 * 64 + np.arange(B)[None], -1).astype(np.int32)
    target = rng.integers(0, 150000, (N, B)).astype(np.int32)
    for n in range(N):
        for i in range(B):
            kids = np.nonzero(parent[n] == i)[0]
            if kids.size and rng.random() < 0.8:
                target[n, i] = token[n, rng.choice(kids)]
    return token, parent, target


# ------------------------------------------------------------- plain forms --

def _plain_logprobs(st):
    case = st["case"]
    z_all, ids, K = st["logits"], st["ids"].long(), case["K"]
    rows, V = z_all.shape
    logp = torch.empty((rows, case["M"]), device="cuda")
    ent = torch.empty((rows,), device="cuda")
    top_id = torch.empty((rows, K), dtype=torch.int32, device="cuda")
    top_lp = torch.empty((rows, K), device="cuda")
    at = torch.arange(V, device="cuda")
    step = max(1, (1 << 27) // V)
    for r in range(0, rows, step):
        s = slice(r, min(rows, r + step))
        x = z_all[s].to(torch.float32, copy=True)
        z = x / case["T"]
        m = z.amax(-1, keepdim=True)
        e = torch.exp(z - m)
        total = e.sum(-1, keepdim=True)
        lse = m + torch.log(total)
        logp[s] = z.gather(1, ids[s]) - lse
        ent[s] = (torch.log(total) - torch.where(e > 0, e * (z - m), 0.0).sum(-1, keepdim=True) / total)[:, 0]
        for k in range(K):
            best = x.amax(-1, keepdim=True)
            i = torch.where(x == best, at, V).amin(-1, keepdim=True)
            none = best == -math.inf
            top_id[s, k] = torch.where(none, -1, i)[:, 0].int()
            top_lp[s, k] = torch.where(none, -math.inf, best / case["T"] - lse)[:, 0]
            x.scatter_(1, i, -math.inf)
    return logp, ent, top_id, top_lp


def _plain_tree(st):
    N, G, K, B = (st["case"][k] for k in ("N", "G", "K", "B"))
    ids, lp = st["top_ids"], st["top_logp"].double()
    n, row = torch.arange(N, device="cuda"), torch.arange(B, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    token, parent, depth = torch.full((N, B), -1, **i32), torch.full((N, B), -2, **i32), torch.zeros((N, B), **i32)
    mask = torch.zeros((N, B), dtype=torch.int64, device="cuda")
    token[:, 0], parent[:, 0], mask[:, 0] = st["anchor"], -1, 1
    score = torch.full((N, B), -math.inf, dtype=torch.float64, device="cuda")
    score[:, 0] = 0
    level = torch.zeros((N, B), dtype=torch.int64, device="cuda")       # depth of each row
    rank = torch.zeros((N, B), dtype=torch.int64, device="cuda")        # of each row's next child
    count = torch.ones((N,), **i32)
    for i in range(1, B):
        # the next child of each row there is
        open_ = (level < G) & (rank < K) & (mask != 0)
        pos, rk = level.clamp(max=G - 1), rank.clamp(max=K - 1)
        cand = torch.where(open_, score + lp[n[:, None], pos, rk], -math.inf)
        best = cand.amax(1)
        p = torch.where(cand == best[:, None], row, B).amin(1)          # the lowest parent of the best
        ok = best > -math.inf
        p = torch.where(ok, p, 0)
        token[:, i] = torch.where(ok, ids[n, pos[n, p], rk[n, p]], -1)
        parent[:, i] = torch.where(ok, p, -2).int()
        level[:, i] = torch.where(ok, level[n, p] + 1, 0)
        mask[:, i] = torch.where(ok, mask[n, p] | (1 << i if i < 63 else -(1 << 63)), 0)
        score[:, i] = torch.where(ok, best, -math.inf)
        rank[n, p] += ok.long()
        count += ok.int()
    return token, parent, level.int(), mask, count


def _quantise(x, e):
    """bf16 [..., hd] -> (code 0..15 uint8 [..., hd], scale fp32 [..., hd/16])."""
    g = x.float().unflatten(-1, (-1, GROUP))
    amax = g.abs().amax(-1)
    s = (amax * 2.0 ** -e / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float().clamp(min=2.0 ** -9)
    t, a = (s * 2.0 ** e).unsqueeze(-1), g.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for border, tie_up in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        code += (a >= border * t) if tie_up else (a > border * t)
    code += 8 * (g < 0)
    return code.flatten(-2), s


def _values(code, s, e):
    mag = torch.tensor(E2M1, device=code.device)[(code & 7).long()]
    v = torch.where(code > 7, -mag, mag).unflatten(-1, (-1, GROUP)) * s.unsqueeze(-1) * 2.0 ** e
    return v.flatten(-2)


def _slots(table, page, n, t):
    """Pool token index of position t of sequence n."""
    return table[n, t // page].long() * page + t % page


def _plain_attn(st):
    case, page = st["case"], st["case"]["page"]
    N, B, Hq, Hkv, hd, W = (case[k] for k in ("N", "B", "Hq", "Hkv", "hd", "window"))
    G = Hq // Hkv
    out = torch.empty((N, B, Hq, hd), dtype=torch.bfloat16, device="cuda")
    row = torch.arange(B, device="cuda")
    for n in range(N):
        L = st["lens"][n]
        t = torch.arange(L, device="cuda")
        own_seen, at, there = torch.ones((B, B), dtype=torch.bool, device="cuda"), row, row >= 0
        if st["mask"] is not None:
            own_seen = (st["mask"][n][:, None] >> row[None]) & 1 == 1
            there = st["mask"][n] != 0
            at = (own_seen.sum(1) - 1).clamp(min=0)
        q, p = L + at, torch.cat([t, L + at])
        seen = torch.cat([there[:, None].expand(B, L), own_seen], 1)
        if W:
            seen = seen & ((q[:, None] - p[None] < W) | (p[None] < case["sinks"]))
        some = torch.nonzero(seen.any(0))[:, 0]          # keys that some row sees
        cached = some[some < L]
        slots = _slots(st["table"], page, n, cached)
        k, v = (_values(st["store"][x][0][slots], st["store"][x][1][slots].float(), case["e"]) for x in "KV")
        mine = some[some >= L] - L
        k = torch.cat([k, st["Kb"][n][mine].float()]).permute(1, 2, 0)                      # [Hkv][hd][keys]
        v = torch.cat([v, st["Vb"][n][mine].float()]).permute(1, 0, 2)
        qh = st["Q"][n].float().view(B, Hkv, G, hd).permute(1, 0, 2, 3).reshape(Hkv, B * G, hd)
        bias = torch.where(seen[:, some], 0.0, -math.inf).repeat_interleave(G, 0)
        s = (qh @ k) / math.sqrt(hd) + bias
        m = s.amax(-1, keepdim=True).clamp(min=-3e38) if some.numel() else torch.zeros_like(s[..., :1])
        w = torch.exp(s - m)
        total = w.sum(-1, keepdim=True)
        o = torch.where(total > 0, (w @ v) / total, 0.0)
        out[n] = o.view(Hkv, B, G, hd).permute(1, 0, 2, 3).reshape(B, Hq, hd).to(torch.bfloat16)
    return out


def _plain_accept(st):
    token, parent, target = st["token"], st["parent"].long(), st["target"]
    N, B = token.shape
    n, row = torch.arange(N, device="cuda"), torch.arange(B, device="cuda")
    path = torch.full((N, B), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    cur, length, live = torch.zeros_like(n), torch.zeros_like(n), torch.ones_like(n, dtype=torch.bool)
    for i in range(1, B):
        hit = (parent == cur[:, None]) & (token == target[n, cur][:, None]) & (row[None] > cur[:, None])
        nxt = torch.where(hit, row, B).amin(1)
        live = live & (nxt < B)
        path[:, i] = torch.where(live, nxt, -1).int()
        cur = torch.where(live, nxt, cur)
        length += live
    return path, length.int(), target[n, cur]


# ----------------------------------------------------------- prepare and run --

def prepare(case, seed):
    st, op = dict(case=case), case["op"]
    if op == "logprobs":
        st["logits"], st["ids"] = _logits(case, seed)
        return st
    if own:
        import block_diffusion_speculative_dfl_gb300 as dfl
    if op in ("tree", "accept"):
        if own:
            st["tree"] = dfl.DraftTree(case["N"], case["B"])
        if op == "tree":
            st["anchor"], st["top_ids"], st["top_logp"] = _alternatives(case, seed)
            return st
        token, parent, target = (_ints(x) for x in _accept_inputs(case, seed))
        st.update(token=token, parent=parent, target=target)
        if own:
            st["tree"].token.copy_(token)
            st["tree"].parent.copy_(parent)
        return st
    inp = _kv_inputs(case, seed)
    N, max_pages = inp["table"].shape
    pages = N * max_pages
    st.update(Q=inp["Q"], Kb=inp["Kb"], Vb=inp["Vb"], table=_ints(inp["table"]), lens=inp["lens"].tolist())
    st["mask"] = _ints(_masks(inp["parent"])[0], torch.int64) if "parent" in inp else None
    if own:
        c = st["cache"] = dfl.PagedCache(layers=1, num_pages=pages, page=case["page"], Hkv=case["Hkv"], hd=case["hd"],
                                         N=N, max_pages=max_pages, k_exp=case["e"], v_exp=case["e"])
        c.table.copy_(st["table"])
        c.len.copy_(_ints(inp["lens"]))
        c.append(0, inp["K"], inp["V"], torch.zeros_like(c.len), c.len)
        st["out"] = torch.empty_like(inp["Q"])
        return st
    shape = (pages * case["page"], case["Hkv"])
    st["store"] = {}
    for x in "KV":
        code = torch.zeros((*shape, case["hd"]), dtype=torch.uint8, device="cuda")
        scale = torch.zeros((*shape, case["hd"] // GROUP), dtype=torch.float8_e4m3fn, device="cuda")
        for n in range(N):
            t = torch.arange(st["lens"][n], device="cuda")
            slots = _slots(st["table"], case["page"], n, t)
            c, s = _quantise(inp[x][n, :st["lens"][n]], case["e"])
            code[slots], scale[slots] = c, s.to(torch.float8_e4m3fn)
        st["store"][x] = (code, scale)
    return st


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"logprobs": _plain_logprobs, "tree": _plain_tree, "attn": _plain_attn, "accept": _plain_accept}[op](st)
    if op == "logprobs":
        import block_diffusion_speculative_dfl_gb300 as dfl
        r = dfl.token_logprobs(st["logits"], st["ids"], top=case["K"], T=case["T"])
        return r.logp, r.entropy, r.top_ids, r.top_logp
    if op == "tree":
        t = st["tree"]
        t.build(st["anchor"], st["top_ids"], st["top_logp"])
        return t.token, t.parent, t.depth, t.mask, t.count
    if op == "accept":
        t = st["tree"]
        t.accept(st["target"])
        return t.path, t.accept_len, t.bonus
    return st["cache"].attn(0, st["Q"], st["Kb"], st["Vb"], out=st["out"], mask=st["mask"], window=case["window"],
                            sinks=case["sinks"])


# -------------------------------------------------------------------- exact --

def _nearest(y, mant, emin, top):
    """y >= 0 (float64) to the nearest number of `mant` mantissa bits, exponents from emin, at most top; ties to even."""
    e = torch.floor(torch.log2(y.clamp(min=2.0 ** -300))).clamp(min=emin)
    e = torch.where(torch.exp2(e + 1) <= y, e + 1, e)
    step = torch.exp2(e - mant)
    return (torch.round(y / step) * step).clamp(max=top)


def _exact_values(x, e):
    g = x.double().unflatten(-1, (-1, GROUP)) * 2.0 ** -e
    s = _nearest(g.abs().amax(-1, keepdim=True) / 6, 3, -6, 448.0).clamp(min=2.0 ** -9)
    return (torch.sign(g) * _nearest(g.abs() / s, 1, 0, 6.0) * s * 2.0 ** e).flatten(-2)


def _exact_logprobs(case, seed):
    logits, ids = _logits(case, seed)
    rows, V = logits.shape
    out = [[], [], [], []]
    step = max(1, (1 << 26) // V)
    for r in range(0, rows, step):
        x = logits[r:r + step].double()
        lp = torch.log_softmax(x / case["T"], -1)
        out[0].append(torch.gather(lp, 1, ids[r:r + step].long()))
        out[1].append(torch.special.entr(lp.exp()).sum(-1))
        if case["K"] > V:
            x = torch.nn.functional.pad(x, (0, case["K"] - V), value=-math.inf)
            lp = torch.nn.functional.pad(lp, (0, case["K"] - V), value=-math.inf)
        best, at = torch.sort(x, dim=-1, descending=True, stable=True)
        best, at = best[:, :case["K"]], at[:, :case["K"]]
        out[2].append(torch.where(best.isinf(), -1, at).int())
        out[3].append(lp.gather(1, at))
    return tuple(torch.cat(o) for o in out)


def _exact_tree(case, seed):
    anchor, ids, lp = (x.cpu().numpy() for x in _alternatives(case, seed))
    N, G, K, B = (case[k] for k in ("N", "G", "K", "B"))
    token, parent = np.full((N, B), -1, np.int32), np.full((N, B), -2, np.int32)
    count = np.zeros(N, np.int32)
    for n in range(N):
        token[n, 0], parent[n, 0] = anchor[n], -1
        level, score = [0], [0.0]
        heap = [(-float(lp[n, 0, 0]), 0, 0)]     # (-score, parent, rank)
        while heap and len(level) < B:
            neg, p, k = heapq.heappop(heap)
            g, i = level[p], len(level)
            token[n, i], parent[n, i] = ids[n, g, k], p
            level.append(g + 1)
            score.append(-neg)
            if k + 1 < K:
                heapq.heappush(heap, (-(score[p] + float(lp[n, g, k + 1])), p, k + 1))
            if g + 1 < G:
                heapq.heappush(heap, (-(score[i] + float(lp[n, g + 1, 0])), i, 0))
        count[n] = len(level)
    mask, depth = _masks(parent)
    return _ints(token), _ints(parent), _ints(depth), _ints(mask, torch.int64), _ints(count)


def _exact_attn(case, seed):
    inp = _kv_inputs(case, seed)
    N, B, Hq, Hkv, hd, W, S = (case[k] for k in ("N", "B", "Hq", "Hkv", "hd", "window", "sinks"))
    G = Hq // Hkv
    out = torch.zeros(inp["Q"].shape, dtype=torch.float64, device="cuda")
    for n in range(N):
        L = int(inp["lens"][n])
        see = np.zeros((B, L + B), bool)
        pos = np.arange(L + B)
        if case["kind"] == "tree":
            par = inp["parent"][n]
            for i in range(B):
                line, j = [], i
                while j >= 0 and par[i] != -2:
                    line.append(j)
                    j = par[j]
                pos[L + i] = L + max(0, len(line) - 1)
                see[i, [L + j for j in line]] = True
                see[i, :L] = bool(line)
        else:
            see[:] = True
        for i in range(B):
            if W:
                see[i] &= (pos[L + i] - pos < W) | (pos < S)
        some = np.nonzero(see.any(0))[0]
        if some.size == 0:
            continue
        hidden = torch.from_numpy(~see[:, some]).cuda()
        old, new = torch.from_numpy(some[some < L]).cuda(), torch.from_numpy(some[some >= L] - L).cuda()
        for h in range(Hkv):
            k = torch.cat([_exact_values(inp["K"][n, old, h], case["e"]), inp["Kb"][n, new, h].double()])
            v = torch.cat([_exact_values(inp["V"][n, old, h], case["e"]), inp["Vb"][n, new, h].double()])
            q = inp["Q"][n, :, h * G:(h + 1) * G].double()
            s = torch.einsum("bgd,kd->bgk", q, k) / hd ** 0.5
            w = torch.softmax(s.masked_fill(hidden[:, None], -math.inf), -1).nan_to_num(0.0)
            out[n, :, h * G:(h + 1) * G] = torch.einsum("bgk,kd->bgd", w, v)
    return out


def _exact_accept(case, seed):
    token, parent, target = _accept_inputs(case, seed)
    N, B = token.shape
    path, length, bonus = np.full((N, B), -1, np.int32), np.zeros(N, np.int32), np.zeros(N, np.int32)
    for n in range(N):
        cur, done = 0, 1
        path[n, 0] = 0
        while True:
            bonus[n] = target[n, cur]
            kids = [i for i in range(cur + 1, B) if parent[n, i] == cur and token[n, i] == target[n, cur]]
            if not kids:
                break
            cur = path[n, done] = kids[0]
            done += 1
        length[n] = done - 1
    return _ints(path), _ints(length), _ints(bonus)


def exact(case, seed):
    return {"logprobs": _exact_logprobs, "tree": _exact_tree, "attn": _exact_attn, "accept": _exact_accept}[case["op"]](
        case, seed)
