"""fp64 restatement of the drafted-token trees: log probabilities, building, masked attention, acceptance.

Written from the definitions, one row or one sequence at a time.
"""
import heapq

import numpy as np


def token_logprobs(z, ids, K, T):
    """One row: (logp of ids, entropy, top ids, top logp); NaN for a row that is no distribution."""
    z = np.asarray(z, np.float64)
    order = [int(i) for i in np.argsort(-z, kind="stable") if not np.isnan(z[i]) and z[i] > -np.inf][:K]
    top = np.array(order + [-1] * (K - len(order)), np.int32)
    if np.isnan(z).any() or z.max() in (np.inf, -np.inf):
        nan = np.full(len(ids), np.nan)
        nan[[i for i, t in enumerate(ids) if not 0 <= t < z.size]] = -np.inf
        return nan, np.nan, top, np.where(top < 0, -np.inf, np.nan)
    m = z.max()
    d = (z - m) / T
    e = np.exp(d)
    ls = np.log(e.sum())
    with np.errstate(invalid="ignore"):
        entropy = ls - np.where(e > 0, e * d, 0.0).sum() / e.sum()
    logp = np.array([d[t] - ls if 0 <= t < z.size else -np.inf for t in ids])
    return logp, entropy, top, np.array([d[t] - ls if t >= 0 else -np.inf for t in top])


def draft_tree(anchor, ids, logp, B):
    """One sequence, ids, logp [G][K]: (token, parent, depth) lists of the rows there are."""
    G, K = len(ids), len(ids[0])
    token, parent, depth, score = [int(anchor)], [-1], [0], [0.0]
    heap = []

    def offer(p, k):
        g = depth[p]
        if g < G and k < K and np.isfinite(logp[g][k]):
            heapq.heappush(heap, (-(score[p] + float(logp[g][k])), p, k))

    offer(0, 0)
    while heap and len(token) < B:
        neg, p, k = heapq.heappop(heap)
        token.append(int(ids[depth[p]][k]))
        parent.append(p)
        depth.append(depth[p] + 1)
        score.append(-neg)
        offer(p, k + 1)
        offer(len(token) - 1, 0)
    return token, parent, depth


def ancestors(parent, i):
    """Row i and the rows above it; none where there is no row."""
    line = []
    while i >= 0 and parent[i] != -2:
        line.append(i)
        i = parent[i]
    return line


def tree_mask(parent):
    """Masks (Python ints) of parents."""
    return [sum(1 << j for j in ancestors(parent, i)) for i in range(len(parent))]


def tree_accept(token, parent, target):
    """One sequence: (path, bonus)."""
    path = [0]
    while True:
        want = target[path[-1]]
        kids = [i for i in range(path[-1] + 1, len(token)) if parent[i] == path[-1] and token[i] == want]
        if not kids:
            return path, want
        path.append(kids[0])


def sees(length, B, mask, window, sinks):
    """bool [B][length + B]: which cached tokens, then own rows, each row sees.  mask: ints, or None."""
    pos = np.arange(length + B)
    out = np.ones((B, length + B), bool)
    if mask is not None:
        bits = [[m >> j & 1 for j in range(B)] for m in mask]
        out[:, length:] = np.array(bits, bool)
        for i in range(B):
            pos[length + i] = length + max(sum(bits[i]) - 1, 0)
            out[i, :length] = sum(bits[i]) > 0
    if window:
        q = pos[length:]
        out &= (q[:, None] - pos[None] < window) | (pos[None] < sinks)
    return out


def masked_attn(q, kc, vc, kb, vb, see):
    """One sequence: q [B][Hq][hd], cached kc, vc [T][Hkv][hd], own kb, vb [B][Hkv][hd], see [B][T + B].

    Returns O [B][Hq][hd] (0 where a row sees nothing) and, for error bounds, sum p |v| and the largest |score|.
    """
    q, kc, vc, kb, vb = (np.asarray(a, np.float64) for a in (q, kc, vc, kb, vb))
    B, Hq, hd = q.shape
    G = Hq // kc.shape[1]
    O, A, smax = np.zeros((B, Hq, hd)), np.zeros((B, Hq, hd)), 0.0
    for b in range(B):
        at = np.nonzero(see[b])[0]
        if at.size == 0:
            continue
        for h in range(Hq):
            k = np.concatenate([kc[:, h // G], kb[:, h // G]])[at]
            v = np.concatenate([vc[:, h // G], vb[:, h // G]])[at]
            s = k @ q[b, h] / np.sqrt(hd)
            smax = max(smax, float(np.abs(s).max()))
            p = np.exp(s - s.max())
            p /= p.sum()
            O[b, h], A[b, h] = p @ v, p @ np.abs(v)
    return O, A, smax
