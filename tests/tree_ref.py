"""Plain 64-bit forms of the tree-draft operators, on the CPU, for the tests."""
import math

import torch


def ancestors(up, n):
    """[n, n] bool: node j is node i or above it."""
    see = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        j = i
        while j >= 0:
            see[i, j] = True
            j = up[j]
    return see


def attention(q, k_new, v_new, k_cache, v_cache, table, lens, parents=None, nodes=None, scale=None):
    """(out, lse, tol_out, tol_lse, live): float64 results, the error bounds of
    a kernel with float32 sums and, for bfloat16, weights rounded to bfloat16,
    and which rows are written.

    The bounds, with u = 2^-24 the rounding of float32: a score is a sum of D
    products, so off by at most ds = (D + 2) u scale sum |q||k|, and in units
    of log2 e by one rounding more of its own size; a weight 2^x by 2^-21
    (approximate power) + that; a sum of n terms by (n + 64) u of the sum of
    their absolute values; the output then by its own rounding."""
    B, T, Hq, D = q.shape
    Hkv, ps = k_new.shape[2], k_cache.shape[1]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    bf = q.dtype == torch.bfloat16
    u, half = 2.0 ** -24, torch.finfo(q.dtype).eps / 2
    out, tol = torch.zeros(B, T, Hq, D, dtype=torch.float64), torch.zeros(B, T, Hq, D, dtype=torch.float64)
    lse, tol_lse = torch.zeros(B, T, Hq, dtype=torch.float64), torch.zeros(B, T, Hq, dtype=torch.float64)
    live = torch.zeros(B, T, dtype=torch.bool)
    for b in range(B):
        n, m = int(lens[b]), T if nodes is None else int(nodes[b])
        if m == 0:
            continue
        live[b, :m] = True
        up = list(range(-1, T - 1)) if parents is None else parents[b].tolist()
        see = torch.cat([torch.ones(m, n, dtype=torch.bool), ancestors(up, m)], 1)
        at = torch.arange(n)
        page, row = table[b].long()[at // ps], at % ps
        for h in range(Hkv):
            K = torch.cat([k_cache[page, row, h], k_new[b, :m, h]]).double()
            V = torch.cat([v_cache[page, row, h], v_new[b, :m, h]]).double()
            for g in range(G):
                Q = q[b, :m, h * G + g].double() * scale
                x = torch.where(see, Q @ K.T, -math.inf)
                size = torch.where(see, Q.abs() @ K.abs().T, 0.0).amax(1)
                top = x.amax(1, keepdim=True)
                w = torch.exp(x - top)
                total = w.sum(1, keepdim=True)
                w = w / total
                seen_v = torch.where(see[:, :, None], V[None], 0.0)
                o = (w[:, :, None] * seen_v).sum(1)
                mass = (w[:, :, None] * seen_v.abs()).sum(1)
                ds = (D + 4) * u * size
                rel = 2 * ds + (n + m + 64) * u * 2 + 2.0 ** -20
                out[b, :m, h * G + g] = o
                tol[b, :m, h * G + g] = half * o.abs() * 1.01 + mass * (rel + (half if bf else 0.0))[:, None]
                lse[b, :m, h * G + g] = (top + total.log()).squeeze(1)
                tol_lse[b, :m, h * G + g] = rel + 4 * u * (top.abs().squeeze(1) + 1)
    return out, lse, tol, tol_lse, live


def select(logits, scores, temperature, K):
    """Per sequence the K best (score, beam, token) in float64, equal scores by
    the smaller beam and token; places without a candidate are None."""
    got = []
    B, W, V = logits.shape
    for b in range(B):
        x = torch.full((W, V), -math.inf, dtype=torch.float64)
        for w in range(W):
            if scores[b, w] > -math.inf:
                x[w] = scores[b, w].double() + torch.log_softmax(logits[b, w].double() / temperature[b].double(), -1)
        value, at = torch.sort(x.flatten(), descending=True, stable=True)
        got.append([(value[i].item(), int(at[i]) // V, int(at[i]) % V) if value[i] > -math.inf else None for i in range(K)])
    return got


def commit_path(tokens, target, up, n):
    path, cur = [0], True
    while cur:
        cur = [i for i in range(1, n) if up[i] == path[-1] and tokens[i] == target[path[-1]]][:1]
        path += cur
    return path
