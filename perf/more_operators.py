"""Operators around a verification step on a paged cache: the cases they are measured on and their plain forms.

Four operators that stand beside the tree attention, the commit and the verification of this package:

  rope    rotary positions of queries and keys, and (inverse) of their gradients
  append  keys and values appended to the paged cache, rotated on the way, with the queries' rotation
  prefix  attention of the nodes of drafted trees for sequences that share long prefixes, each prefix read once for all
  adjust  penalties for repeated tokens, biases and grammar masks on the logits of a drafted chain or tree

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
    rope = {"op": "rope", "dtype": "bf16", "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "interleaved": False, "inverse": False, "far": 32768}
    app = {"op": "append", "dtype": "bf16", "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "interleaved": False}
    pre = {"op": "prefix", "dtype": "bf16", "Hq": 32, "Hkv": 8, "D": 128, "chain": True, "uneven": False}
    adj = {"op": "adjust", "dtype": "bf16", "V": 151936, "tree": False, "bias": 0, "mask": False}
    return [
        # one verification step of a serving batch: the drafted tokens of 64 sequences
        dict(rope, name="rope step b64", B=64, T=4),
        # the backward pass of a training batch: gradients of queries and keys of two texts of 8192 tokens
        dict(rope, name="rope backward", B=2, T=8192, inverse=True),
        # a small model in 32 bits with part of each head rotated, pairs side by side, at positions of a very long text
        dict(rope, name="rope f32 part", dtype="f32", B=3, T=1021, Hq=8, Hkv=2, D=96, R=64, interleaved=True, far=1000000),
        # the accepted tokens of a verification step, one to four of each sequence
        dict(app, name="append step b64", B=64, T=4, L=8192, page=16),
        # prompts of four requests, up to 8192 tokens
        dict(app, name="append prompts", B=4, T=8192, L=0, page=64),
        # four samples of one short prompt, one new token each: every microsecond is latency
        dict(pre, name="prefix b4", P=1, B=4, T=1, Lp=2000, L=100, page=16),
        # a rollout: 64 samples of one long prompt verify three drafted tokens each
        dict(pre, name="prefix rollout b64", P=1, B=64, T=4, Lp=16384, L=1024, page=64),
        # a training batch of rollouts: 16 prompts with 16 samples each, one new token
        dict(pre, name="prefix groups b256", P=16, B=256, T=1, Hq=16, Hkv=2, D=256, Lp=4096, L=1000, page=32),
        # a small model kept in 32 bits, uneven groups, trees of five nodes
        dict(pre, name="prefix f32 b24", dtype="f32", P=3, B=24, T=5, Hq=8, Hkv=2, D=64, Lp=1500, L=200, page=16, chain=False,
             uneven=True),
        # one user's verification step
        dict(adj, name="adjust b1", B=1, S=4, L=2000),
        # a serving batch with long texts and a grammar for every position
        dict(adj, name="adjust b64", B=64, S=4, L=8192, bias=8, mask=True),
        # 32-bit logits of an odd vocabulary at the nodes of small trees
        dict(adj, name="adjust f32 tree", dtype="f32", B=16, S=7, V=50257, L=1000, tree=True, bias=300, mask=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "prefix", "prefix", "adjust", "adjust"])
    dt = "f32" if rng.random() < 0.25 else "bf16"
    es = ESIZE[dt]
    if op in ("rope", "append"):
        D = rng.choice([64, 80, 96, 128, 128, 256])
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
        R = rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)])
        B, T = _log(rng, 1, 64), _log(rng, 1, 8192)
        T = max(1, min(T, int(8e7 / (B * Hkv * (G + 2) * D))))
        c = {"op": op, "dtype": dt, "B": B, "T": T, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "R": R, "interleaved": rng.random() < 0.4}
        if op == "rope":
            return dict(c, inverse=rng.random() < 0.4, far=_log(rng, 1000, 1000000))
        page = rng.choice([16, 24, 32, 64, 128])
        return dict(c, L=min(_log(rng, 1, 16384), int(4e8 / (B * Hkv * D * 2 * es))), page=page)
    if op == "prefix":
        D = rng.choice([64, 128, 128, 256])
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
        P, T = _log(rng, 1, 24), _log(rng, 1, 16)
        B = P * rng.randint(1, 16)
        Lp, L = _log(rng, 1, 65536), _log(rng, 1, 2048)
        most = 7e10 if dt == "bf16" else 4e9
        rows = B * T * Hkv * G
        Lp = max(1, min(Lp, int(4e8 / (P * Hkv * D * 2 * es)), int(most / (4.0 * rows * D)), int(2.5e8 / rows)))
        L = max(1, min(L, int(4e8 / (B * Hkv * D * 2 * es)), int(most / (4.0 * rows * D)), int(2.5e8 / rows)))
        return {"op": op, "dtype": dt, "P": P, "B": B, "T": T, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "Lp": Lp, "L": L,
                "page": rng.choice([16, 24, 32, 64, 128, 256]), "chain": rng.random() < 0.5, "uneven": rng.random() < 0.5}
    V = rng.choice([_log(rng, 1000, 151936), _log(rng, 1000, 151936), 32000, 128256, 151936])
    S, B = rng.randint(1, 16), _log(rng, 1, 64)
    B = max(1, min(B, int(7e7 / (S * V * es))))
    return {"op": op, "dtype": dt, "B": B, "S": S, "V": V, "L": _log(rng, 1, 16384), "tree": rng.random() < 0.4,
            "bias": rng.choice([0, 0, rng.randint(1, 300)]), "mask": rng.random() < 0.5}


def _lens(L, B):
    """Lengths spread from L down to none (before `prepare` shuffles them)."""
    return [L - (L * b) // max(1, B + B // 2) for b in range(B - 1)] + ([0] if B > 3 else [L])


def _news(c):
    """Appended tokens of each sequence: of a step one to T in turn, of a prompt spread as above."""
    return [1 + b % c["T"] for b in range(c["B"])] if c["T"] <= 16 else _lens(c["T"], c["B"])


def _groups(c):
    """(first sequence of each group and the end, tokens of each prefix); uneven groups include one of a single sequence and
    an unused prefix."""
    P, B = c["P"], c["B"]
    starts = [B * p // P for p in range(P + 1)]
    lens = [c["Lp"] - c["Lp"] * p // (2 * P) for p in range(P)]
    if c["uneven"] and P > 2:
        starts[1], starts[2] = 1, 1
    return starts, lens


def work(c):
    es, B = ESIZE[c["dtype"]], c["B"]
    if c["op"] == "rope":
        heads = B * c["T"] * (c["Hq"] + c["Hkv"])
        return {"bytes": 2 * heads * c["D"] * es + 4 * B * c["T"] + 2 * c["R"], "flops": 3.0 * heads * c["R"]}
    if c["op"] == "append":
        n = sum(_news(c))
        return {"bytes": n * (4 * c["Hkv"] + 2 * c["Hq"]) * c["D"] * es + 4 * (3 * B + n // c["page"]) + 2 * c["R"],
                "flops": 3.0 * n * (c["Hq"] + c["Hkv"]) * c["R"]}
    if c["op"] == "prefix":
        starts, plens = _groups(c)
        lens, T, D = _lens(c["L"], B), c["T"], c["D"]
        shared = sum(n for n, a, z in zip(plens, starts, starts[1:]) if z > a)
        met = sum(n * (z - a) for n, a, z in zip(plens, starts, starts[1:])) + sum(lens)
        seen = T * (T + 1) / 2 if c["chain"] else T * (1 + math.log(T))
        pages = sum(-(-n // c["page"]) for n in plens + lens)
        return {"bytes": (shared + sum(lens) + B * T) * c["Hkv"] * D * 2 * es + 2 * B * T * c["Hq"] * D * es +
                4 * (B * T * c["Hq"] + pages + B * (T + 1) + 2 * c["P"] + 1),
                "flops": 4.0 * c["Hq"] * D * (T * met + B * seen)}
    rows = B * c["S"]
    return {"bytes": rows * c["V"] * (2 * es + (0.125 if c["mask"] else 0.0)) + 4 * (sum(_lens(c["L"], B)) + 5 * B + 2 * rows) +
            8 * B * c["bias"], "flops": 3.0 * rows * c["V"]}


# ----------------------------------------------------------------- inputs --

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pages(rng, *counts):
    """Page tables of [rows, width] each whose pages lie in one pool in no order, and the pages of the pool."""
    n = sum(r * w for r, w in counts)
    ids = list(range(n + 1))
    rng.shuffle(ids)
    tables, at = [], 0
    for r, w in counts:
        tables.append(_i32(ids[at:at + r * w]).view(r, w))
        at += r * w
    return tables, n + 1


def _tree(rng, T):
    return [-1] + [rng.randint(max(0, i - max(4, T // 8)), i - 1) for i in range(1, T)]


def _frequencies(R, stretch):
    """Angles per token, the slow ones stretched for long texts."""
    f = 500000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    slow = ((1024.0 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)  # 0: less than one turn in 1024 tokens
    return (f * slow + f / stretch * (1 - slow)).float().to(DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[c["dtype"]]
    B = c["B"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=dt)

    s = {"op": c["op"]}
    if c["op"] in ("rope", "append"):
        T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
        # queries, keys and values are parts of one projection, as a model has them
        qkv = normal(B, T, Hq + 2 * Hkv, D)
        s.update(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:], inv_freq=_frequencies(c["R"], 8.0),
                 interleaved=c["interleaved"], factor=0.1 * math.log(8.0) + 1.0)
        s["q_out"] = torch.zeros(B, T, Hq, D, dtype=dt, device=DEV)
    if c["op"] == "rope":
        s["k_out"] = torch.zeros(B, T, Hkv, D, dtype=dt, device=DEV)
        s["positions"] = _i32([[p] for p in (rng.randint(0, c["far"]) for _ in range(B))]) + torch.arange(T, dtype=torch.int32, device=DEV)
        s["inverse"] = c["inverse"]
    elif c["op"] == "append":
        ps, news = c["page"], _news(c)
        rng.shuffle(news)
        P = -(-(c["L"] + T) // ps)
        (s["table"],), pool = _pages(rng, (B, P))
        s.update(k_cache=normal(pool, ps, Hkv, D), v_cache=normal(pool, ps, Hkv, D), lens=_i32([rng.randint(0, c["L"]) for _ in range(B)]),
                 news=_i32(news), new_lens=torch.zeros(B, dtype=torch.int32, device=DEV))
        s["flags"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    elif c["op"] == "prefix":
        T, Hq, Hkv, D, ps = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
        starts, plens = _groups(c)
        lens = _lens(c["L"], B)
        rng.shuffle(lens)
        (s["prefix_table"], s["table"]), pool = _pages(rng, (c["P"], -(-c["Lp"] // ps)), (B, -(-c["L"] // ps)))
        qkv = normal(B, T, Hq + 2 * Hkv, D)
        qkv[:, :, :Hq] *= 2
        s.update(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:], k_cache=normal(pool, ps, Hkv, D),
                 v_cache=normal(pool, ps, Hkv, D), starts=_i32(starts), plens=_i32(plens), lens=_i32(lens), groups=starts)
        s["parents"] = None if c["chain"] else _i32([_tree(rng, T) for _ in range(B)])
        s["out"] = torch.zeros(B, T, Hq, D, dtype=dt, device=DEV)
        s["lse"] = torch.zeros(B, T, Hq, device=DEV)
        s["flags"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    else:
        S, V, L, n = c["S"], c["V"], c["L"], c["bias"]
        lens = _lens(L, B)
        rng.shuffle(lens)

        def words(*shape):  # a few words make most of a text
            return (V ** torch.rand(shape, generator=g, device=DEV) - 1).int().clamp(0, V - 1)

        def uniform(lo, hi):
            return lo + (hi - lo) * torch.rand(B, generator=g, device=DEV)

        s.update(z=normal(B, S, V) * 3, history=words(B, L), lens=_i32(lens), prompts=_i32([n // 2 for n in lens]), tokens=words(B, S),
                 parents=_i32([_tree(rng, S) for _ in range(B)]) if c["tree"] else None, repetition=uniform(1, 1.5),
                 frequency=uniform(-0.2, 0.8), presence=uniform(-0.2, 0.8), bias_ids=None, bias=None, mask=None)
        if n:
            s["bias_ids"], s["bias"] = words(B, n), torch.randn(B, n, generator=g, device=DEV) * 4
        if c["mask"]:
            # at some positions the grammar allows a few words, at the others most
            W = (V + 31) // 32
            bits = torch.randint(-2 ** 31, 2 ** 31, (4, B, S, W), generator=g, device=DEV)
            few = torch.rand(B, S, 1, generator=g, device=DEV) < 0.3
            mask = torch.where(few, bits[0] & bits[1] & bits[2] & bits[3], bits[0] | bits[1] | bits[2] | bits[3])
            s["mask"] = mask.int()
        s["out"] = torch.zeros_like(s["z"])
        s["flags"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------ plain forms --

def _ancestors(parents, B, T):
    """[B, T, T]: whether node j lies on the path from the root to node i (i itself included)."""
    if parents is None:
        return torch.ones(T, T, dtype=torch.bool, device=DEV).tril().expand(B, T, T)
    nodes = torch.arange(T, device=DEV)
    up = ((parents[:, :, None] == nodes) | (nodes[:, None] == nodes)).float()
    reach = 1
    while reach < T:
        up = (up @ up > 0).float()
        reach *= 2
    return up > 0


def _rotate(x, positions, inv_freq, interleaved, factor, inverse):
    """x [B, T, H, D] rotated in its first 2 len(inv_freq) elements; angles in 64 bits, since far positions lose all of theirs
    in 32."""
    n = inv_freq.numel()
    angle = positions.double()[..., None] * inv_freq.double()
    cos, sin = (angle.cos() * factor).float()[:, :, None], (angle.sin() * (-factor if inverse else factor)).float()[:, :, None]
    y = x.float()
    a, b = (y[..., 0:2 * n:2], y[..., 1:2 * n:2]) if interleaved else (y[..., :n], y[..., n:2 * n])
    parts = [a * cos - b * sin, b * cos + a * sin]
    head = torch.stack(parts, -1).flatten(-2) if interleaved else torch.cat(parts, -1)
    return torch.cat([head, y[..., 2 * n:]], -1).to(x.dtype)


def _rope(s):
    args = s["positions"], s["inv_freq"], s["interleaved"], s["factor"], s["inverse"]
    return {"q": _rotate(s["q"], *args), "k": _rotate(s["k"], *args)}


def _append(s):
    T, ps = s["k"].shape[1], s["k_cache"].shape[1]
    at = s["lens"][:, None] + torch.arange(T, dtype=torch.int32, device=DEV)
    live = torch.arange(T, device=DEV) < s["news"][:, None]
    args = at, s["inv_freq"], s["interleaved"], s["factor"], False
    q, k = _rotate(s["q"], *args), _rotate(s["k"], *args)
    b, t = torch.where(live)
    to = at[b, t].long()
    page = s["table"][b, to // ps].long()
    s["k_cache"][page, to % ps] = k[b, t]
    s["v_cache"][page, to % ps] = s["v"][b, t]
    return {"q": torch.where(live[:, :, None, None], q, s["q_out"]), "lens": s["lens"] + s["news"], "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


def _prefix(s):
    q, k, v, ps = s["q"], s["k"], s["v"], s["k_cache"].shape[1]
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    table, ptable = s["table"].long(), s["prefix_table"].long()
    L, Lp = table.shape[1] * ps, ptable.shape[1] * ps
    qf = q.float().view(B, T, Hkv, Hq // Hkv, D) * D ** -0.5
    keys = torch.cat([s["k_cache"][table].view(B, L, Hkv, D), k], 1).float()
    values = torch.cat([s["v_cache"][table].view(B, L, Hkv, D), v], 1).float()
    seen = torch.cat([(torch.arange(L, device=DEV) < s["lens"][:, None])[:, None].expand(B, T, L), _ancestors(s["parents"], B, T)], 2)
    mine = torch.einsum("bthgd,bshd->bhgts", qf, keys).masked_fill_(~seen[:, None, None], -math.inf)
    outs, lses = [], []
    for p, (a, z) in enumerate(zip(s["groups"], s["groups"][1:])):
        if a == z:
            continue
        pk, pv = (c[ptable[p]].view(Lp, Hkv, D).float() for c in (s["k_cache"], s["v_cache"]))
        x = torch.einsum("bthgd,shd->bhgts", qf[a:z], pk)
        x.masked_fill_(torch.arange(Lp, device=DEV) >= s["plens"][p], -math.inf)
        y = mine[a:z]
        top = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
        x, y = x.sub_(top).exp_(), (y - top).exp_()
        total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
        o = torch.einsum("bhgts,shd->bthgd", x.div_(total), pv) + torch.einsum("bhgts,bshd->bthgd", y.div_(total), values[a:z])
        outs.append(o.reshape(z - a, T, Hq, D))
        lses.append((top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(z - a, T, Hq))
    return {"out": torch.cat(outs).to(q.dtype), "lse": torch.cat(lses)}


def _adjust(s):
    z = s["z"]
    B, S, V = z.shape
    L = s["history"].shape[1]
    at = torch.arange(L, device=DEV)
    live = at < s["lens"][:, None]
    ids = s["history"].long()
    zero = torch.zeros(B, V, device=DEV)
    seen = zero.scatter_add(1, ids, live.float())
    count = zero.scatter_add(1, ids, (live & (at >= s["prompts"][:, None])).float())
    path = torch.zeros(B, S, V, device=DEV).scatter_add_(2, s["tokens"].long()[:, None].expand(B, S, S),
                                                         _ancestors(s["parents"], B, S).float())
    seen, count = path + seen[:, None], path.add_(count[:, None])
    x = z.float()
    rho, freq, pres = (s[k][:, None, None] for k in ("repetition", "frequency", "presence"))
    x = torch.where(seen > 0, torch.where(x > 0, x / rho, x * rho), x)
    x = x - freq * count - pres * (count > 0)
    if s["bias"] is not None:
        x = x + torch.zeros(B, V, device=DEV).scatter_add(1, s["bias_ids"].long(), s["bias"])[:, None]
    if s["mask"] is not None:
        allowed = (s["mask"][..., None] >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
        x = x.masked_fill(allowed.flatten(2)[..., :V] == 0, -math.inf)
    return {"logits": x.to(z.dtype)}


# -------------------------------------------------------------------- run --

def run(s):
    op = s["op"]
    if own:
        import mtp_speculative_decoding_row_gb300 as mtp

        if op == "rope":
            r = mtp.mtp_rope(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=s["interleaved"], factor=s["factor"],
                             inverse=s["inverse"], out=mtp.RopeResult(s["q_out"], s["k_out"]))
            return {"q": r.q, "k": r.k}
        if op == "append":
            r = mtp.mtp_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["news"], q=s["q"],
                                     inv_freq=s["inv_freq"], interleaved=s["interleaved"], factor=s["factor"],
                                     out=mtp.AppendResult(s["new_lens"], s["q_out"], None, s["flags"]))
            return {"q": r.q, "lens": r.cache_len, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if op == "prefix":
            r = mtp.mtp_prefix_attention(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["prefix_table"], s["plens"], s["starts"],
                                         s["table"], s["lens"], s["parents"], out=mtp.TreeAttentionResult(s["out"], s["lse"], s["flags"]))
            return {"out": r.out, "lse": r.lse}
        r = mtp.mtp_adjust_logits(s["z"], s["history"], s["lens"], prompt_len=s["prompts"], tokens=s["tokens"], parents=s["parents"],
                                  repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"],
                                  bias=s["bias"], mask=s["mask"], out=mtp.AdjustResult(s["out"], s["flags"]))
        return {"logits": r.logits}
    return {"rope": _rope, "append": _append, "prefix": _prefix, "adjust": _adjust}[op](s)


# ------------------------------------------------------------------ exact --

def _turned(x, positions, inv_freq, interleaved, factor, inverse):
    """x [T, H, D] in 64 bits as complex numbers times factor e^(i angle)."""
    n = inv_freq.numel()
    x = x.double()
    pairs = x[..., :2 * n].unflatten(-1, (n, 2)) if interleaved else x[..., :2 * n].unflatten(-1, (2, n)).transpose(-1, -2)
    angle = positions.double()[:, None] * inv_freq.double()
    turn = torch.polar(torch.full_like(angle, factor), -angle if inverse else angle)
    got = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    return torch.cat([(got if interleaved else got.transpose(-1, -2)).flatten(-2), x[..., 2 * n:]], -1)


def exact(c, seed):
    s = prepare(c, seed)
    B = c["B"]
    if c["op"] == "rope":
        args = s["inv_freq"], c["interleaved"], s["factor"], c["inverse"]
        return {k: torch.stack([_turned(s[k][b], s["positions"][b], *args) for b in range(B)]) for k in ("q", "k")}
    if c["op"] == "append":
        K, V, q, ps = s["k_cache"].double(), s["v_cache"].double(), s["q_out"].double(), c["page"]
        for b, (n, m) in enumerate(zip(s["lens"].tolist(), s["news"].tolist())):
            if m == 0:
                continue
            at = torch.arange(n, n + m, device=DEV)
            args = at, s["inv_freq"], c["interleaved"], s["factor"], False
            page = s["table"][b].long()[at // ps]
            K[page, at % ps] = _turned(s["k"][b, :m], *args)
            V[page, at % ps] = s["v"][b, :m].double()
            q[b, :m] = _turned(s["q"][b, :m], *args)
        return {"q": q, "lens": s["lens"] + s["news"], "k_cache": K, "v_cache": V}
    if c["op"] == "prefix":
        out, lse = s["out"].double(), s["lse"].double()
        _, T, Hq, D = out.shape
        G, ps = Hq // c["Hkv"], c["page"]
        lens, plens, starts = s["lens"].tolist(), s["plens"].tolist(), s["groups"]
        for b in range(B):
            p = [i for i in range(c["P"]) if starts[i] <= b < starts[i + 1]][0]
            n, m = plens[p], lens[b]
            up = list(range(-1, T - 1)) if s["parents"] is None else s["parents"][b].tolist()
            sees = torch.zeros(T, T, dtype=torch.bool)
            for i in range(T):
                j = i
                while j >= 0:
                    sees[i, j] = True
                    j = up[j]
            sees = torch.cat([torch.ones(T, n + m, dtype=torch.bool), sees], 1).to(DEV)
            shared, mine = (t[:-(-k // ps)].long() for t, k in ((s["prefix_table"][p], n), (s["table"][b], m)))
            K, V = (torch.cat([x[shared].flatten(0, 1)[:n], x[mine].flatten(0, 1)[:m], y[b]]).double().transpose(0, 1)
                    for x, y in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])))
            x = s["q"][b].double().view(T, c["Hkv"], G, D).transpose(0, 1).flatten(1, 2) @ K.transpose(1, 2) / math.sqrt(D)
            x = x.view(c["Hkv"], T, G, -1).masked_fill(~sees[None, :, None], -math.inf)
            lse[b] = torch.logsumexp(x, -1).transpose(0, 1).reshape(T, Hq)
            out[b] = (torch.softmax(x, -1).flatten(1, 2) @ V).view(c["Hkv"], T, G, D).transpose(0, 1).reshape(T, Hq, D)
        return {"out": out, "lse": lse}
    S, V = c["S"], c["V"]
    got = s["z"].double()
    for b, (n, m) in enumerate(zip(s["lens"].tolist(), s["prompts"].tolist())):
        text = s["history"][b].long()
        up = list(range(-1, S - 1)) if s["parents"] is None else s["parents"][b].tolist()
        for i in range(S):
            path, j = [], i
            while j >= 0:
                path.append(j)
                j = up[j]
            path = s["tokens"][b].long()[path]
            count = torch.bincount(torch.cat([text[m:n], path]), minlength=V)
            seen = (torch.bincount(text[:m], minlength=V) + count) > 0
            x = got[b, i]
            rho = s["repetition"][b].double()
            x[seen] = torch.where(x[seen] > 0, x[seen] / rho, x[seen] * rho)
            x -= s["frequency"][b].double() * count + s["presence"][b].double() * (count > 0)
            if s["bias"] is not None:
                x.index_add_(0, s["bias_ids"][b].long(), s["bias"][b].double())
            if s["mask"] is not None:
                v = torch.arange(V, device=DEV)
                x[(s["mask"][b, i][v // 32] >> (v % 32)) & 1 == 0] = -math.inf
    return {"logits": got}
