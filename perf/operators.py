"""Operators of tree-shaped speculative decoding: the cases they are measured on and their plain forms.

Four operators around the draft and verification stages of this package:

  attention  attention of a tree of drafted tokens over a paged cache of keys and values (the target's pass over the drafts;
             a tree of one token is ordinary decoding)
  select     the best continuations over beams and vocabulary (how a draft tree grows by a level)
  reorder    states of the selected beams gathered by their parents
  commit     the accepted path of a verified tree, and its keys and values written into the paged cache

A case is a dict of plain values whose "op" names the operator.  With ``own`` false, ``run`` computes the plain form from
elementary torch operations; with ``own`` true it calls this package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases --

def listed():
    att = {"op": "attention", "dtype": "bf16", "page": 64, "chain": False, "ragged": False}
    sel = {"op": "select", "dtype": "bf16"}
    return [
        # one new token of one short conversation: every microsecond is latency
        dict(att, name="attention decode b1", B=1, T=1, Hq=32, Hkv=8, D=128, L=1000, page=16, chain=True),
        # a serving batch that verifies three drafted tokens in a chain, lengths spread as in a rollout
        dict(att, name="attention chain b64", B=64, T=4, Hq=16, Hkv=2, D=256, L=8192, page=32, chain=True, ragged=True),
        # the compute-heavy end: full trees of 64 nodes, eight query heads to a key head, long prompts
        dict(att, name="attention tree b8", B=8, T=64, Hq=64, Hkv=8, D=128, L=16384),
        # one very long document read by a small tree: the cache of one sequence has to feed the whole GPU
        dict(att, name="attention long b1", B=1, T=8, Hq=32, Hkv=8, D=128, L=131072, page=128),
        # a small model kept in 32 bits, an odd tree and odd lengths
        dict(att, name="attention f32 b4", dtype="f32", B=4, T=7, Hq=8, Hkv=2, D=64, L=2501, page=16, ragged=True),
        # the next level of one user's draft tree
        dict(sel, name="select b1", B=1, W=4, K=8, V=151936),
        # a batch of draft trees
        dict(sel, name="select b64", B=64, W=8, K=16, V=151936),
        # 32-bit logits of an odd vocabulary whose rows start on no vector boundary
        dict(sel, name="select f32 odd", dtype="f32", B=16, W=5, K=10, V=50257),
        # the drafter's hidden state of each beam
        {"op": "reorder", "name": "reorder hidden", "dtype": "bf16", "N0": 1, "B": 64, "W": 8, "K": 8, "N": 4096},
        # keys of the drafted tokens of each beam, all layers
        {"op": "reorder", "name": "reorder keys", "dtype": "bf16", "N0": 8, "B": 64, "W": 8, "K": 8, "N": 65536},
        # one user, a small tree, one layer
        {"op": "commit", "name": "commit b1", "dtype": "bf16", "N0": 1, "B": 1, "T": 8, "branch": 2, "Hkv": 8, "D": 128, "page": 16, "cap": 256},
        # a batch of trees, the layers of a model in one call
        {"op": "commit", "name": "commit b64", "dtype": "bf16", "N0": 16, "B": 64, "T": 32, "branch": 2, "Hkv": 8, "D": 128, "page": 16, "cap": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "select", "select", "reorder", "commit"])
    dt = "f32" if rng.random() < 0.25 else "bf16"
    if op == "attention":
        D = rng.choice([64, 128, 128, 256])
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16])
        B, T, L = _log(rng, 1, 128), _log(rng, 1, 64), _log(rng, 1, 131072)
        es = ESIZE[dt]
        most = 2.5e11 if dt == "bf16" else 4e9
        L = min(L, int(5e8 / (B * Hkv * D * 2 * es)), int(most / (4.0 * B * T * Hkv * G * D)), int(5e8 / (B * T * Hkv * G)))
        return {"op": op, "dtype": dt, "B": B, "T": T, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "L": max(L, 1),
                "page": rng.choice([16, 24, 32, 48, 64, 128, 256]), "chain": rng.random() < 0.4, "ragged": rng.random() < 0.6}
    if op == "select":
        V = rng.choice([_log(rng, 1000, 151936), _log(rng, 1000, 151936), 32000, 128256, 151936])
        W, B = rng.randint(1, 16), _log(rng, 1, 64)
        B = max(1, min(B, int(1.5e8 / (W * V * ESIZE[dt]))))
        return {"op": op, "dtype": dt, "B": B, "W": W, "K": rng.randint(1, 32), "V": V}
    if op == "reorder":
        W = rng.randint(1, 16)
        N0, B, N = rng.randint(1, 8), _log(rng, 1, 64), _log(rng, 16, 65536)
        N = max(1, min(N, int(5e8 / (N0 * B * W * ESIZE[dt]))))
        return {"op": op, "dtype": dt, "N0": N0, "B": B, "W": W, "K": rng.randint(1, W), "N": N}
    B, N0, T = _log(rng, 1, 64), rng.randint(1, 16), _log(rng, 1, 64)
    return {"op": op, "dtype": dt, "N0": N0, "B": B, "T": T, "branch": rng.randint(1, 4), "Hkv": rng.choice([1, 2, 4, 8]),
            "D": rng.choice([64, 128]), "page": rng.choice([16, 24, 64]), "cap": rng.randint(T, 128)}


def _lens(c):
    """Cached tokens of each sequence, before `prepare` shuffles them: all of L, or spread from L down to none."""
    B, L = c["B"], c["L"]
    if not c["ragged"]:
        return [L] * B
    return [L - (L * b) // max(1, B + B // 2) for b in range(B - 1)] + ([0] if B > 3 else [L])


def _depths(c):
    """Accepted drafts of each sequence in a commit case: every depth of the tree in turn."""
    deepest, i = 0, c["T"] - 1
    while i > 0:
        deepest, i = deepest + 1, (i - 1) // c["branch"]
    return [b % (deepest + 1) for b in range(c["B"])] if c["B"] > 1 else [deepest]


def work(c):
    es = ESIZE[c["dtype"]]
    if c["op"] == "attention":
        lens, B, T, D = _lens(c), c["B"], c["T"], c["D"]
        seen = T * (T + 1) / 2 if c["chain"] else T * (1 + math.log(T))
        pages = sum(-(-n // c["page"]) for n in lens)
        return {"bytes": (sum(lens) + B * T) * c["Hkv"] * D * 2 * es + 2 * B * T * c["Hq"] * D * es + 4 * (B * T * c["Hq"] + pages + B * (T + 1)),
                "flops": 4.0 * c["Hq"] * D * (T * sum(lens) + B * seen)}
    if c["op"] == "select":
        rows = c["B"] * c["W"]
        return {"bytes": rows * (c["V"] * es + 4) + 12 * c["B"] * c["K"], "flops": 3.0 * rows * c["V"]}
    if c["op"] == "reorder":
        # a parent that several beams share is read once
        read = c["W"] * (1 - (1 - 1 / c["W"]) ** c["K"])
        return {"bytes": c["N0"] * c["B"] * (read + c["K"]) * c["N"] * es + 4 * c["B"] * c["K"], "flops": 0.0}
    moved = sum(_depths(c)) + c["B"]
    return {"bytes": 4.0 * c["N0"] * moved * c["Hkv"] * c["D"] * es + 4 * c["B"] * (5 * c["T"] + 4), "flops": 0.0}


# ----------------------------------------------------------------- inputs --

def _table(rng, B, P):
    """A page table whose pages lie in the pool in no order."""
    ids = list(range(B * P + 1))
    rng.shuffle(ids)
    return torch.tensor(ids[:B * P], dtype=torch.int32, device=DEV).view(B, P)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if dt == torch.float32 else dt)

    s = {"op": c["op"]}
    if c["op"] == "attention":
        B, T, Hq, Hkv, D, ps = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
        lens = _lens(c)
        rng.shuffle(lens)
        P = max(1, -(-c["L"] // ps))
        # queries and new keys are parts of one projection, as a model has them
        qkv = normal(B, T, Hq + 2 * Hkv, D)
        qkv[:, :, :Hq] *= 2
        s.update(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:],
                 k_cache=normal(B * P + 1, ps, Hkv, D), v_cache=normal(B * P + 1, ps, Hkv, D), table=_table(rng, B, P),
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
        s["parents"], s["nodes"] = None, None
        if not c["chain"]:
            near = max(4, T // 8)
            s["parents"] = torch.tensor([[-1] + [rng.randint(max(0, i - near), i - 1) for i in range(1, T)] for _ in range(B)],
                                        dtype=torch.int32, device=DEV)
        if c["ragged"]:
            s["nodes"] = torch.tensor([rng.randint((T + 1) // 2, T) for _ in range(B)], dtype=torch.int32, device=DEV)
        s["out"] = torch.zeros(B, T, Hq, D, dtype=dt, device=DEV)
        s["lse"] = torch.zeros(B, T, Hq, device=DEV)
        s["flags"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    elif c["op"] == "select":
        B, W, V = c["B"], c["W"], c["V"]
        z = normal(B, W, V) * 2
        # a few likely words in each row, as a trained drafter gives
        at = torch.randint(V, (B, W, 24), generator=g, device=DEV)
        z.scatter_reduce_(2, at, (torch.rand(B, W, 24, generator=g, device=DEV) * 12).to(dt), "amax")
        s.update(z=z, K=min(c["K"], W * V), scores=-torch.rand(B, W, generator=g, device=DEV).mul(3).cumsum(1),
                 temperature=0.5 + torch.rand(B, generator=g, device=DEV))
        K = s["K"]
        s["tokens"], s["parents"] = (torch.zeros(B, K, dtype=torch.int32, device=DEV) for _ in range(2))
        s["best"], s["flags"] = torch.zeros(B, K, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    elif c["op"] == "reorder":
        s.update(states=normal(c["N0"], c["B"], c["W"], c["N"]),
                 parents=torch.randint(c["W"], (c["B"], c["K"]), generator=g, device=DEV, dtype=torch.int32))
        s["out"] = torch.zeros(c["N0"], c["B"], c["K"], c["N"], dtype=dt, device=DEV)
        s["flags"] = torch.zeros(c["B"], dtype=torch.int32, device=DEV)
    else:
        B, T, N0, Hkv, D, ps = c["B"], c["T"], c["N0"], c["Hkv"], c["D"], c["page"]
        P = -(-(c["cap"] + T) // ps)
        tokens = [[rng.randrange(151936) for _ in range(T)] for _ in range(B)]
        target = [[rng.randrange(151936) for _ in range(T)] for _ in range(B)]
        depths = _depths(c)
        for b in range(B):
            levels = [[0]]
            while levels[-1]:
                levels.append([i for i in range(1, T) if (i - 1) // c["branch"] in levels[-1]])
            i = rng.choice(levels[depths[b]])
            while i > 0:  # the target agrees with every draft on the way to node i
                target[b][(i - 1) // c["branch"]] = tokens[b][i]
                i = (i - 1) // c["branch"]
        as_i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        s.update(tokens=as_i32(tokens), target=as_i32(target),
                 parents=as_i32([[-1] + [(i - 1) // c["branch"] for i in range(1, T)] for _ in range(B)]),
                 k=normal(N0, B, T, Hkv, D), v=normal(N0, B, T, Hkv, D), k_cache=normal(N0, B * P + 1, ps, Hkv, D),
                 v_cache=normal(N0, B * P + 1, ps, Hkv, D), table=_table(rng, B, P),
                 lens=as_i32([rng.randint(0, c["cap"]) for _ in range(B)]))
        s["out"], s["path"] = (torch.zeros(B, T, dtype=torch.int32, device=DEV) for _ in range(2))
        s["accept"], s["new_lens"], s["flags"] = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
    return s


# ------------------------------------------------------------ plain forms --

def _ancestors(parents, B, T):
    """[B, T, T]: whether node j lies on the path from the root to node i (i itself included)."""
    if parents is None:
        return torch.ones(T, T, dtype=torch.bool, device=DEV).tril().expand(B, T, T)
    nodes = torch.arange(T, device=DEV)
    up = ((parents[:, :, None] == nodes) | (nodes[:, None] == nodes)).float()
    up = (up @ up > 0).float()   # paths of up to 2 steps, then 4, 8, 16, 32, 64
    up = (up @ up > 0).float()
    up = (up @ up > 0).float()
    up = (up @ up > 0).float()
    up = (up @ up > 0).float()
    return up @ up > 0


def _attention(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    table = s["table"].long()
    L = table.shape[1] * s["k_cache"].shape[1]
    keys = torch.cat([s["k_cache"][table].view(B, L, Hkv, D), k], 1).float()
    values = torch.cat([s["v_cache"][table].view(B, L, Hkv, D), v], 1).float()
    seen = torch.cat([(torch.arange(L, device=DEV) < s["lens"][:, None])[:, None].expand(B, T, L), _ancestors(s["parents"], B, T)], 2)
    x = torch.einsum("bthgd,bshd->bhgts", q.float().view(B, T, Hkv, Hq // Hkv, D) * D ** -0.5, keys)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.einsum("bhgts,bshd->bthgd", x.div_(total), values).reshape(B, T, Hq, D)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, T, Hq)
    if s["nodes"] is not None:  # rows behind a sequence's last node stay as they were
        live = (torch.arange(T, device=DEV) < s["nodes"][:, None])[:, :, None]
        return {"out": torch.where(live[..., None], out.to(q.dtype), s["out"]), "lse": torch.where(live, lse, s["lse"])}
    return {"out": out.to(q.dtype), "lse": lse}


def _select(s):
    z = s["z"]
    B, W, V = z.shape
    K, k = s["K"], min(s["K"], V)
    x = z.float() + 0.0  # (the two zeros are equal)
    # in one row the order is that of the logits, equal ones by index: one whole-number key for both
    bits = x.view(torch.int32)
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = (bits << 32) + (V - 1 - torch.arange(V, device=DEV))
    best = key.topk(k, 2).values
    token = V - 1 - (best & 0xFFFFFFFF)
    # log softmax in 64 bits: two beams' candidates may lie next to each other
    T = s["temperature"].double()[:, None, None]
    x = x.double() / T
    top = x.amax(2, keepdim=True)
    chosen = x.gather(2, token)
    total = (x.sub_(top)).exp_().sum(2, keepdim=True)
    score = (s["scores"].double()[:, :, None] + (chosen - top - total.log())).flatten(1)
    flat = (torch.arange(W, device=DEV)[:, None] * V + token).flatten(1)
    flat, order = flat.sort(1)
    score, which = score.gather(1, order).sort(dim=1, descending=True, stable=True)
    flat = flat.gather(1, which)[:, :K]
    return {"tokens": (flat % V).int(), "parents": (flat // V).int(), "scores": score[:, :K].float()}


def _reorder(s):
    rows = torch.arange(s["parents"].shape[0], device=DEV)[:, None]
    return {"states": s["states"][:, rows, s["parents"].long()]}


def _commit(s):
    tokens, target, parents = s["tokens"], s["target"], s["parents"].long()
    B, T = tokens.shape
    nodes = torch.arange(T, device=DEV)
    up = parents.clamp(min=0)
    match = (parents >= 0) & (tokens == target.gather(1, up))
    # of several children with the token only the first is followed
    twin = (parents[:, :, None] == parents[:, None]) & (tokens[:, :, None] == tokens[:, None]) & (nodes < nodes[:, None])
    match = (match & ~twin.any(2)) | (nodes == 0)
    above = _ancestors(s["parents"], B, T)
    taken = (match[:, None] | ~above).all(2) & above[:, :, 0]
    count = taken.sum(1)
    path = torch.where(taken, nodes, T).sort(1).values
    last = path.gather(1, count[:, None] - 1)
    drafts = torch.where(nodes < count[:, None] - 1, tokens.gather(1, path.roll(-1, 1).clamp(max=T - 1)), -1)
    out = torch.where(nodes == count[:, None] - 1, target.gather(1, last), drafts)
    ps = s["k_cache"].shape[2]
    b, j = torch.where(nodes < count[:, None])
    at = s["lens"].long()[b] + j
    page = s["table"].long()[b, at // ps]
    s["k_cache"][:, page, at % ps] = s["k"][:, b, path[b, j]]
    s["v_cache"][:, page, at % ps] = s["v"][:, b, path[b, j]]
    return {"out": out.int(), "path": torch.where(path < T, path, -1).int(), "accept": (count - 1).int(),
            "lens": (s["lens"] + count).int(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# -------------------------------------------------------------------- run --

def run(s):
    op = s["op"]
    if own:
        import mtp_speculative_decoding_row_gb300 as mtp

        if op == "attention":
            r = mtp.mtp_tree_attention(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["parents"],
                                       s["nodes"], out=mtp.TreeAttentionResult(s["out"], s["lse"], s["flags"]))
            return {"out": r.out, "lse": r.lse}
        if op == "select":
            r = mtp.mtp_beam_select(s["z"], s["scores"], s["temperature"], s["K"],
                                    out=mtp.BeamResult(s["tokens"], s["parents"], s["best"], s["flags"]))
            return {"tokens": r.tokens, "parents": r.parents, "scores": r.scores}
        if op == "reorder":
            return {"states": mtp.mtp_beam_reorder(s["states"], s["parents"], out=mtp.ReorderResult(s["out"], s["flags"])).states}
        r = mtp.mtp_tree_commit(s["tokens"], s["target"], s["parents"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"],
                                s["lens"], out=mtp.CommitResult(s["out"], s["accept"], s["path"], s["new_lens"], s["flags"]))
        return {"out": r.tokens, "path": r.path, "accept": r.accept_len, "lens": r.cache_len, "k_cache": s["k_cache"],
                "v_cache": s["v_cache"]}
    if op == "attention":
        return _attention(s)
    if op == "select":
        return _select(s)
    return _reorder(s) if op == "reorder" else _commit(s)


# ------------------------------------------------------------------ exact --

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "attention":
        out, lse = s["out"].double(), s["lse"].double()
        B, T, Hq, D = out.shape
        G, ps = Hq // c["Hkv"], c["page"]
        lens, nodes = s["lens"].tolist(), [T] * B if s["nodes"] is None else s["nodes"].tolist()
        for b in range(B):
            n, m = lens[b], nodes[b]
            pages = s["table"][b, :-(-n // ps)].long()
            up = list(range(-1, T - 1)) if s["parents"] is None else s["parents"][b].tolist()
            sees = torch.zeros(m, m, dtype=torch.bool)
            for i in range(m):
                j = i
                while j >= 0:
                    sees[i, j] = True
                    j = up[j]
            sees = torch.cat([torch.ones(m, n, dtype=torch.bool), sees], 1).to(DEV)
            for h in range(c["Hkv"]):
                K = torch.cat([s["k_cache"][pages, :, h].reshape(-1, D)[:n], s["k"][b, :m, h]]).double()
                V = torch.cat([s["v_cache"][pages, :, h].reshape(-1, D)[:n], s["v"][b, :m, h]]).double()
                x = s["q"][b, :m, h * G:(h + 1) * G].double() @ K.T / math.sqrt(D)
                x = x.masked_fill(~sees[:, None], -math.inf)
                lse[b, :m, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                out[b, :m, h * G:(h + 1) * G] = torch.softmax(x, -1) @ V
        return {"out": out, "lse": lse}
    if c["op"] == "select":
        got = {"tokens": [], "parents": [], "scores": []}
        for b in range(c["B"]):
            x = torch.log_softmax(s["z"][b].double() / s["temperature"][b].double(), -1) + s["scores"][b].double()[:, None]
            value, at = torch.sort(x.flatten(), descending=True, stable=True)
            got["tokens"].append((at[:s["K"]] % c["V"]).int())
            got["parents"].append((at[:s["K"]] // c["V"]).int())
            got["scores"].append(value[:s["K"]])
        return {k: torch.stack(v) for k, v in got.items()}
    if c["op"] == "reorder":
        parents = s["parents"].tolist()
        return {"states": torch.stack([torch.stack([s["states"][:, b, p] for p in row], 1) for b, row in enumerate(parents)], 1).double()}
    T, ps = c["T"], c["page"]
    tokens, target, up, lens, table = (s[k].tolist() for k in ("tokens", "target", "parents", "lens", "table"))
    K, V = s["k_cache"].double(), s["v_cache"].double()
    got = {"out": [], "path": [], "accept": [], "lens": []}
    for b in range(c["B"]):
        path, on = [0], True
        while on:
            on = [i for i in range(1, T) if up[b][i] == path[-1] and tokens[b][i] == target[b][path[-1]]][:1]
            path += on
        for j, i in enumerate(path):
            page, row = table[b][(lens[b] + j) // ps], (lens[b] + j) % ps
            K[:, page, row], V[:, page, row] = s["k"][:, b, i].double(), s["v"][:, b, i].double()
        more = [-1] * (T - len(path))
        got["out"].append([tokens[b][i] for i in path[1:]] + [target[b][path[-1]]] + more)
        got["path"].append(path + more)
        got["accept"].append(len(path) - 1)
        got["lens"].append(lens[b] + len(path))
    return {**{k: torch.tensor(v, dtype=torch.int32) for k, v in got.items()}, "k_cache": K, "v_cache": V}
