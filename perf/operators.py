"""Workloads of the paged 4-bit context cache: attention over it, writing and reading it, and its page operations.

Values.  A cached element is c * s * 2^e: c one of the e2m1 numbers 0, 0.5, 1,
1.5, 2, 3, 4, 6 with a sign, s an e4m3 number shared by 16 consecutive
dimensions of one token and K/V head, e an integer of the pool (one for K, one
for V).  s = max(2^-9, e4m3(min(448, max|x| 2^-e / 6))) and c is the nearest
e2m1 number to x / (s 2^e), at most 6 in magnitude; both round to nearest even.

Pages.  A page holds `page` tokens of every K/V head.  table[n][j] is the page
of tokens j*page .. of sequence n (-1: none), len[n] the tokens it holds,
ref[p] the number of table entries naming page p (0: free).

`run` computes the operators in plain torch, or through the package when `own`
is true.
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GROUP = 16


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # One user, one token at a time, a short conversation: the smallest call.
        dict(name="attn_token_one", op="attn", N=1, B=1, Hq=32, Hkv=8, hd=128, page=16, lo=517, hi=517, e=0),
        # Token-by-token serving of a ragged batch, from fresh prompts to long documents.
        dict(name="attn_token_batch", op="attn", N=48, B=1, Hq=32, Hkv=8, hd=128, page=64, lo=65, hi=16000, e=0),
        # The Qwen3-8B-shaped drafter's block of 16 over a context around 2048.
        dict(name="attn_block_batch", op="attn", N=32, B=16, Hq=32, Hkv=8, hd=128, page=64, lo=1801, hi=2299, e=0),
        # The GPT-OSS-20B-shaped drafter's heads (64 query heads of 64) over a few very long contexts.
        dict(name="attn_block_long", op="attn", N=3, B=8, Hq=64, Hkv=8, hd=64, page=32, lo=33333, hi=100001, e=0),
        # A decoding step's new context rows, up to 16 a sequence, in the middle of pages.
        dict(name="append_step", op="append", N=32, R=16, Hkv=8, hd=128, page=64, lo=1801, hi=2299, new_lo=0, e=0),
        # Prompts arriving: thousands of rows each, read back for a contiguous cache.
        dict(name="append_prompt", op="append", N=8, R=4097, Hkv=8, hd=64, page=16, lo=0, hi=0, new_lo=1025, e=0),
        # Pages for the next tokens of a few sequences that share nothing.
        dict(name="reserve_step", op="reserve", N=8, new_hi=16, layers=1, Hkv=2, hd=64, page=16, lo=30, hi=400,
             share=1, spare=64),
        # 32 prompts forked 8 ways: every fork copies its shared last page on its first write, in 7 layers.
        dict(name="reserve_forked", op="reserve", N=256, new_hi=16, layers=7, Hkv=8, hd=128, page=64, lo=450, hi=640,
             share=8, spare=600),
        # A small batch after acceptance: rejected tokens are rolled back, one sequence ends, one forks.
        dict(name="remap_step", op="remap", N=16, Hkv=2, hd=64, page=16, lo=30, hi=2000, share=1, spare=64,
             max_pages=160),
        # Reordering 512 hypotheses of 64 long prompts.
        dict(name="remap_beams", op="remap", N=512, Hkv=8, hd=128, page=16, lo=9000, hi=16000, share=8, spare=4096,
             max_pages=1024),
        # A small fragmented pool.
        dict(name="compact_small", op="compact", N=12, layers=2, Hkv=2, hd=64, page=16, lo=30, hi=300, share=1,
             spare=120),
        # A serving pool of seven layers, a little over half in use, every page of it scattered.
        dict(name="compact_pool", op="compact", N=128, layers=7, Hkv=8, hd=128, page=32, lo=300, hi=800, share=1,
             spare=1850),
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attn", "attn", "attn", "append", "append", "reserve", "remap", "compact"])
    hd = rng.choice([64, 128])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "attn":
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 8])
        B = rng.choice([1, 1, 1, rng.randint(2, 16), rng.randint(17, 64)])
        # about 4e5 cached tokens and 2e9 score-rows at most
        budget = min(350000 * 8 // Hkv, 3.0e8 / (B * G * Hkv))
        N = logint(1, 64)
        hi = max(1, min(logint(1, 100000), int(budget / N)))
        return dict(op="attn", N=N, B=B, Hq=G * Hkv, Hkv=Hkv, hd=hd, page=page, lo=rng.randint(0, hi), hi=hi,
                    e=rng.randint(-2, 2))
    if op == "append":
        N, R, Hkv = logint(1, 48), logint(1, 4097), rng.choice([1, 2, 4, 8])
        R = max(1, min(R, 32768 // N))
        hi = rng.randint(0, 3000)
        return dict(op="append", N=N, R=R, Hkv=Hkv, hd=hd, page=page, lo=rng.randint(0, hi), hi=hi,
                    new_lo=rng.randint(0, R), e=rng.randint(-2, 2))
    if op == "reserve":
        share, layers, Hkv = rng.choice([1, 2, 4]), rng.randint(1, 7), rng.choice([1, 2, 4, 8])
        N = share * logint(1, 40)
        hi = rng.randint(1, 700)
        return dict(op="reserve", N=N, new_hi=logint(1, 100), layers=layers, Hkv=Hkv, hd=hd, page=page,
                    lo=rng.randint(0, hi), hi=hi, share=share, spare=rng.randint(0, 300))
    if op == "remap":
        share = rng.choice([1, 2, 4])
        N = share * logint(1, 100)
        hi = logint(1, 12000)
        return dict(op="remap", N=N, Hkv=2, hd=hd, page=page, lo=rng.randint(0, hi), hi=hi, share=share,
                    spare=rng.randint(0, 500), max_pages=-(-hi // page) + rng.randint(1, 50))
    N = logint(1, 60)
    hi = rng.randint(1, 600)
    return dict(op="compact", N=N, layers=rng.randint(1, 7), Hkv=rng.choice([1, 2, 4, 8]), hd=hd, page=page,
                lo=rng.randint(0, hi), hi=hi, share=rng.choice([1, 2]) if N % 2 == 0 else 1,
                spare=rng.randint(0, 800))


def _spread(lo, hi, n):
    """n whole numbers evenly over [lo, hi] (their sum belongs to the case, their order to the seed)."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _page_bytes(case):
    return case["page"] * case["Hkv"] * 2 * (case["hd"] // 2 + case["hd"] // GROUP)


def work(case):
    op, N, page = case["op"], case["N"], case["page"]
    if op in ("attn", "append"):
        Hkv, hd = case["Hkv"], case["hd"]
        tok = Hkv * 2 * (hd // 2 + hd // GROUP)      # bytes of one cached token
    if op == "attn":
        B, Hq = case["B"], case["Hq"]
        lens = _spread(case["lo"], case["hi"], N)
        keys = sum(n + B for n in lens)
        return {"bytes": sum(lens) * tok + N * B * (2 * Hq + 2 * Hkv) * hd * 2,
                "flops": 4.0 * B * Hq * hd * keys}
    if op == "append":
        rows = sum(_spread(case["new_lo"], case["R"], N))
        return {"bytes": rows * (2 * 2 * Hkv * hd * 2 + tok), "flops": 0.0}
    lens = _spread(case["lo"], case["hi"], N // case["share"])
    pages = [-(-n // page) for n in lens]
    entries = sum(pages) * case["share"]
    if op == "remap":
        return {"bytes": entries * 4 * 2 + N * 16, "flops": 0.0}
    if op == "reserve":
        tails = sum(n % page != 0 for n in lens) * case["share"] if case["share"] > 1 else 0
        copied = tails * case["layers"] * _page_bytes(case)
        return {"bytes": copied * 2 + (sum(pages) + case["spare"]) * 4 + N * 16, "flops": 0.0}
    live, total = sum(pages), sum(pages) + case["spare"]
    moved = live * (total - live) // max(1, total) * case["layers"] * _page_bytes(case)
    return {"bytes": moved * 2 + entries * 4 * 2 + total * 8, "flops": 0.0}


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1 + seed * 7919)
    return g


def _ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def _kv_inputs(case, seed):
    """bf16 rows K, V [N][T][Hkv][hd] with outlier channels, as keys and values have them."""
    g, rng = _gen(seed), np.random.default_rng(seed)
    N, Hkv, hd = case["N"], case["Hkv"], case["hd"]
    T = max(1, case["hi"] if case["op"] == "attn" else case["R"])
    scale = torch.exp(0.5 * torch.randn((2, Hkv, hd), generator=g, device="cuda")) * 2.0 ** case["e"]
    K, V = (torch.empty((N, T, Hkv, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for n in range(N):
        K[n] = torch.randn((T, Hkv, hd), generator=g, device="cuda") * scale[0]
        V[n] = torch.randn((T, Hkv, hd), generator=g, device="cuda") * scale[1]
    lens = rng.permutation(np.array(_spread(case["lo"], case["hi"], N), np.int32))
    out = dict(K=K, V=V, lens=lens)
    cap = case["hi"]
    if case["op"] == "append":
        out["new"] = rng.permutation(np.array(_spread(case["new_lo"], case["R"], N), np.int32))
        cap += case["R"]
    else:
        B, Hq = case["B"], case["Hq"]
        r = lambda h: torch.randn((N, B, h, hd), generator=g, device="cuda")
        out["Q"] = r(Hq).to(torch.bfloat16)
        out["Kb"] = (r(Hkv) * scale[0]).to(torch.bfloat16)
        out["Vb"] = (r(Hkv) * scale[1]).to(torch.bfloat16)
    max_pages = max(1, -(-cap // case["page"]))
    out["table"] = rng.permutation(N * max_pages).reshape(N, max_pages).astype(np.int32)
    return out


def _page_inputs(case, seed):
    """Tables of N sequences, `share` of which hold the same pages, in a scattered pool with free pages between."""
    rng = np.random.default_rng(seed)
    N, page, share = case["N"], case["page"], case["share"]
    groups = N // share
    lens_g = rng.permutation(np.array(_spread(case["lo"], case["hi"], groups), np.int32))
    used = -(-lens_g // page)
    total = int(used.sum()) + case["spare"]
    total = max(total, 1)
    max_pages = case.get("max_pages") or int(-(-(case["hi"] + case.get("new_hi", 0)) // page)) + 1
    ids = rng.permutation(total).astype(np.int32)
    table = np.full((N, max_pages), -1, np.int32)
    lens = np.zeros(N, np.int32)
    ref = np.zeros(total, np.int32)
    at = 0
    for i in range(groups):
        p = ids[at:at + used[i]]
        at += used[i]
        table[i * share:(i + 1) * share, :used[i]] = p
        lens[i * share:(i + 1) * share] = lens_g[i]
        ref[p] = share
    out = dict(table=table, lens=lens, ref=ref, total=total, max_pages=max_pages)
    if case["op"] == "reserve":
        out["new"] = rng.integers(1, case["new_hi"] + 1, N).astype(np.int32)
    if case["op"] == "remap":
        # most rows stay in their group, some end, some are taken over from anywhere
        parent = (np.arange(N) // share) * share + rng.integers(0, share, N)
        jump = rng.random(N)
        parent = np.where(jump < 0.1, rng.integers(0, N, N), parent)
        out["parent"] = np.where(jump > 0.95, -1, parent).astype(np.int32)
        out["keep"] = np.where(rng.random(N) < 0.5, -1, lens - rng.integers(0, 17, N).clip(0, lens)).astype(np.int32)
    return out


# ------------------------------------------------------------- plain forms --

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


def _plain_store(case, pages, dev="cuda"):
    shape = (pages * case["page"], case["Hkv"])
    return {k: (torch.zeros((*shape, case["hd"]), dtype=torch.uint8, device=dev),
                torch.zeros((*shape, case["hd"] // GROUP), dtype=torch.float8_e4m3fn, device=dev)) for k in "KV"}


def _plain_write(case, store, slots, rows, K, V):
    """slots: pool token index of each row; rows: index into K, V flattened to [rows][Hkv][hd]."""
    for k, x in (("K", K), ("V", V)):
        c, s = _quantise(x.flatten(0, 1)[rows], case["e"])
        store[k][0][slots] = c
        store[k][1][slots] = s.to(torch.float8_e4m3fn)


def _slots(table, page, n, t):
    """Pool token index of position t of sequence n."""
    return table[n, t // page].long() * page + t % page


def _plain_attn(st):
    case, page = st["case"], st["case"]["page"]
    N, B, Hq, Hkv, hd = (case[k] for k in ("N", "B", "Hq", "Hkv", "hd"))
    G = Hq // Hkv
    out = torch.empty((N, B, Hq, hd), dtype=torch.bfloat16, device="cuda")
    for n in range(N):
        slots = _slots(st["table"], page, n, torch.arange(int(st["lens"][n]), device="cuda"))
        k, v = (_values(st["store"][x][0][slots], st["store"][x][1][slots].float(), case["e"]) for x in "KV")
        k = torch.cat([k, st["Kb"][n].float()]).permute(1, 2, 0)                      # [Hkv][hd][keys]
        v = torch.cat([v, st["Vb"][n].float()]).permute(1, 0, 2)
        q = st["Q"][n].float().view(B, Hkv, G, hd).permute(1, 0, 2, 3).reshape(Hkv, B * G, hd)
        s = (q @ k) / math.sqrt(hd)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = (p @ v) / p.sum(-1, keepdim=True)
        out[n] = o.view(Hkv, B, G, hd).permute(1, 0, 2, 3).reshape(B, Hq, hd).to(torch.bfloat16)
    return out


def _plain_append(st):
    case = st["case"]
    N, R = case["N"], case["R"]
    i = torch.arange(R, device="cuda")
    n, i = torch.nonzero(i[None] < st["new"][:, None], as_tuple=True)
    t = st["start"].long()[n] + i
    slots = st["table"].long()[n, t // case["page"]] * case["page"] + t % case["page"]
    _plain_write(case, st["store"], slots, n * R + i, st["K"], st["V"])
    for k, out in (("K", st["outK"]), ("V", st["outV"])):
        v = _values(st["store"][k][0][slots], st["store"][k][1][slots].float(), case["e"])
        out.flatten(0, 1)[n * R + i] = v.to(torch.bfloat16)
    return st["outK"], st["outV"]


def _need(lens, page):
    return torch.div(lens + page - 1, page, rounding_mode="floor")


def _plain_reserve(st):
    page = st["case"]["page"]
    table, lens, ref, new, data = st["table"], st["lens"], st["ref"], st["new"], st["data"]
    N, idx = lens.numel(), torch.arange(lens.numel(), device="cuda")
    have, want = _need(lens, page).long(), _need(lens + new, page).long()
    tail = (lens // page).long().clamp(max=table.shape[1] - 1)
    shared = (new > 0) & (lens % page > 0)
    shared &= ref[table[idx, tail].long().clamp(min=0)] > 1
    need = want - have + shared
    upto = need.cumsum(0)
    free = torch.nonzero(ref == 0).flatten()
    served = (need == 0) | (upto <= free.numel())
    first = torch.where(shared, tail, have)
    # the k-th page of sequence n goes to table entry first[n] + k
    total = int((need * served).sum())
    seq = torch.repeat_interleave(idx, need * served)
    before = (upto - need)
    k = torch.arange(total, device="cuda") - torch.repeat_interleave((need * served).cumsum(0) - need * served,
                                                                      need * served)
    fresh = free[before[seq] + k]
    cow = torch.nonzero(shared & served).flatten()
    src, dst = table[cow, tail[cow]].long(), free[before[cow]]
    data[:, dst] = data[:, src]
    ref.index_add_(0, src, torch.full_like(src, -1, dtype=torch.int32))
    ref[fresh] = 1
    table[seq, first[seq] + k] = fresh.int()
    start = torch.where(served, lens, -1)
    lens += new * served
    return table, lens, ref, start, data


def _plain_remap(st):
    page = st["case"]["page"]
    table, lens, ref = st["table"], st["lens"], st["ref"]
    par = st["parent"].long()
    new_len = torch.where(par >= 0, lens[par.clamp(min=0)], 0)
    new_len = torch.where(st["keep"] >= 0, torch.minimum(new_len, st["keep"]), new_len)
    j = torch.arange(table.shape[1], device="cuda")
    new = torch.where(j[None] < _need(new_len, page)[:, None], table[par.clamp(min=0)], -1)
    for t, sign in ((table, -1), (new, 1)):
        used = t[t >= 0].long()
        ref.index_add_(0, used, torch.full_like(used, sign, dtype=torch.int32))
    table.copy_(new)
    lens.copy_(new_len)
    return table, lens, ref


def _plain_compact(st):
    table, ref, data = st["table"], st["ref"], st["data"]
    idx = torch.arange(ref.numel(), device="cuda")
    used = ref > 0
    live = used.sum()
    src = torch.nonzero(used & (idx >= live)).flatten()
    dst = torch.nonzero(~used & (idx < live)).flatten()
    moved = torch.where(used, idx, -1).int()
    moved[src] = dst.int()
    data[:, dst] = data[:, src]
    ref[dst] = ref[src]
    ref[src] = 0
    table.copy_(torch.where(table >= 0, moved[table.long().clamp(min=0)], table))
    return table, st["lens"], ref, moved, live.int().view(1), data


# ----------------------------------------------------------- prepare and run --

def prepare(case, seed):
    st = dict(case=case)
    if case["op"] in ("attn", "append"):
        inp = _kv_inputs(case, seed)
        N, max_pages = inp["table"].shape
        pages = N * max_pages
        st["table"], st["lens"] = _ints(inp["table"]), _ints(inp["lens"])
        K, V = inp["K"], inp["V"]
        if own:
            import block_diffusion_speculative_dfl_gb300 as dfl
            st["cache"] = c = dfl.PagedCache(layers=1, num_pages=pages, page=case["page"], Hkv=case["Hkv"],
                                             hd=case["hd"], N=N, max_pages=max_pages, k_exp=case["e"],
                                             v_exp=case["e"])
            c.table.copy_(st["table"])
            c.len.copy_(st["lens"])
        else:
            st["store"] = _plain_store(case, pages)
        if case["op"] == "attn":
            st.update(Q=inp["Q"], Kb=inp["Kb"], Vb=inp["Vb"])
            if own:
                st["out"] = torch.empty_like(inp["Q"])
                c.append(0, K, V, torch.zeros_like(st["lens"]), st["lens"])
            else:
                for n in range(N):
                    t = torch.arange(int(inp["lens"][n]), device="cuda")
                    _plain_write(case, st["store"], _slots(st["table"], case["page"], n, t), t, K[n:n + 1], V[n:n + 1])
                st["lens"] = inp["lens"].tolist()
        else:
            st.update(K=K, V=V, start=st["lens"], new=_ints(inp["new"]), outK=torch.zeros_like(K),
                      outV=torch.zeros_like(V))
        return st
    inp = _page_inputs(case, seed)
    N, total, max_pages = case["N"], inp["total"], inp["max_pages"]
    # the bookkeeping a pass starts from, and the buffers it works in
    st["book0"] = _ints(np.concatenate([inp["table"].ravel(), inp["lens"], inp["ref"]]))
    for k in ("new", "parent", "keep"):
        if k in inp:
            st[k] = _ints(inp[k])
    layers = case.get("layers", 1)
    if own:
        import block_diffusion_speculative_dfl_gb300 as dfl
        st["cache"] = c = dfl.PagedCache(layers=layers, num_pages=total, page=case["page"], Hkv=case["Hkv"],
                                         hd=case["hd"], N=N, max_pages=max_pages)
        data = c.data
    else:
        st["book"] = b = torch.empty_like(st["book0"])
        st["table"], st["lens"], st["ref"] = (b[:N * max_pages].view(N, max_pages),
                                              b[N * max_pages:N * max_pages + N], b[N * max_pages + N:])
        data = st["data"] = torch.empty((layers, total, _page_bytes(case)), dtype=torch.uint8, device="cuda")
    if case["op"] != "remap":
        data.copy_(_page_data(case, seed, total))
    return st


def _page_data(case, seed, total):
    return torch.randint(0, 256, (case["layers"], total, _page_bytes(case)), dtype=torch.uint8, device="cuda",
                         generator=_gen(seed))


def run(st):
    op = st["case"]["op"]
    if not own:
        if "book" in st:
            st["book"].copy_(st["book0"])
        return {"attn": _plain_attn, "append": _plain_append, "reserve": _plain_reserve, "remap": _plain_remap,
                "compact": _plain_compact}[op](st)
    c = st["cache"]
    if op == "attn":
        return c.attn(0, st["Q"], st["Kb"], st["Vb"], out=st["out"])
    if op == "append":
        c.append(0, st["K"], st["V"], st["start"], st["new"])
        return c.read(0, st["start"], st["new"], st["outK"], st["outV"])
    c.book.copy_(st["book0"])
    if op == "reserve":
        start = c.reserve(st["new"])
        return c.table, c.len, c.ref, start, c.data
    if op == "remap":
        c.remap(st["parent"], st["keep"])
        return c.table, c.len, c.ref
    moved, live = c.compact()
    return c.table, c.len, c.ref, moved, live, c.data


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


def exact(case, seed):
    op, N, page = case["op"], case["N"], case["page"]
    if op == "append":
        inp = _kv_inputs(case, seed)
        keep = torch.arange(case["R"], device="cuda")[None] < _ints(inp["new"])[:, None]
        return tuple(torch.where(keep[..., None, None], _exact_values(inp[k], case["e"]), 0.0) for k in "KV")
    if op == "attn":
        inp = _kv_inputs(case, seed)
        B, Hkv, hd = case["B"], case["Hkv"], case["hd"]
        out = torch.empty(inp["Q"].shape, dtype=torch.float64, device="cuda")
        for n in range(N):
            L = int(inp["lens"][n])
            for h in range(Hkv):
                k = torch.cat([_exact_values(inp["K"][n, :L, h], case["e"]), inp["Kb"][n, :, h].double()])
                v = torch.cat([_exact_values(inp["V"][n, :L, h], case["e"]), inp["Vb"][n, :, h].double()])
                heads = slice(h * (case["Hq"] // Hkv), (h + 1) * (case["Hq"] // Hkv))
                q = inp["Q"][n, :, heads].double()
                w = torch.softmax(torch.einsum("bgd,kd->bgk", q, k) / hd ** 0.5, -1)
                out[n, :, heads] = torch.einsum("bgk,kd->bgd", w, v)
        return out
    inp = _page_inputs(case, seed)
    table, lens, ref = inp["table"].copy(), inp["lens"].copy(), inp["ref"].copy()
    data = _page_data(case, seed, inp["total"]) if op != "remap" else None
    if op == "reserve":
        free = [p for p in range(ref.size) if ref[p] == 0]
        shared_ref, start, asked = ref.copy(), np.full(N, -1, np.int32), 0
        for n in range(N):
            m = int(inp["new"][n])
            have, want = -(-int(lens[n]) // page), -(-int(lens[n] + m) // page)
            cow = m > 0 and lens[n] % page > 0 and shared_ref[table[n, lens[n] // page]] > 1
            need = want - have + int(cow)
            asked += need
            if need and asked > len(free):
                continue
            got = free[asked - need:asked]
            if cow:
                old = table[n, have - 1]
                data[:, got[0]] = data[:, int(old)]
                ref[old] -= 1
                table[n, have - 1] = got[0]
            table[n, have:want] = got[int(cow):]
            ref[got] = 1
            start[n] = lens[n]
            lens[n] += m
        return _ints(table), _ints(lens), _ints(ref), _ints(start), data
    if op == "remap":
        new, nl = np.full_like(table, -1), np.zeros_like(lens)
        for n in range(N):
            p = inp["parent"][n]
            if p >= 0:
                nl[n] = lens[p] if inp["keep"][n] < 0 else min(lens[p], inp["keep"][n])
                c = -(-int(nl[n]) // page)
                new[n, :c] = table[p, :c]
        np.subtract.at(ref, table[table >= 0], 1)
        np.add.at(ref, new[new >= 0], 1)
        return _ints(new), _ints(nl), _ints(ref)
    live = int((ref > 0).sum())
    moved = np.full(ref.size, -1, np.int32)
    holes = iter([p for p in range(live) if ref[p] == 0])
    for p in range(ref.size):
        if ref[p] > 0:
            moved[p] = p if p < live else next(holes)
            if p >= live:
                data[:, int(moved[p])] = data[:, p]
    new_ref = np.zeros_like(ref)
    new_ref[moved[moved >= 0]] = ref[moved >= 0]
    new = np.where(table >= 0, moved[np.clip(table, 0, None)], table)
    return _ints(new), _ints(lens), _ints(new_ref), _ints(moved), _ints([live]), data
