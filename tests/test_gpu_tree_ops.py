"""The tree-draft operators on the GPU against plain 64-bit forms
(tests/tree_ref.py, which derives the tolerances of the attention)."""
import math
import random

import pytest
import torch

import mtp_speculative_decoding_row_gb300 as mtp
from tests import tree_ref

pytestmark = pytest.mark.gpu
i32, f32, bf16 = torch.int32, torch.float32, torch.bfloat16
DTYPES = {"f32": f32, "bf16": bf16}


@pytest.fixture(scope="module", autouse=True)
def library():
    from tests import gpu_util

    gpu_util.ensure_library()


# ------------------------------------------------------- tree attention --

def random_tree(rng, T, near=8):
    return [-1] + [rng.randint(max(0, i - near), i - 1) for i in range(1, T)]


def attn_case(seed, dtype, B, T, Hq, Hkv, D, ps, lens, tree="random", nodes=None, spare=2, room=0):
    """CPU inputs: pages in random order, NaN in every cache row that no
    sequence has and in the new rows of nodes that a sequence lacks."""
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[dtype]
    P = max(1, -(-max(lens) // ps)) + room
    pages = B * P + spare
    ids = list(range(pages))
    rng.shuffle(ids)
    n = lambda *s: torch.randn(*s, generator=g).to(dt)  # noqa: E731
    x = dict(q=n(B, T, Hq, D) * 2, k_new=n(B, T, Hkv, D), v_new=n(B, T, Hkv, D), k_cache=n(pages, ps, Hkv, D),
             v_cache=n(pages, ps, Hkv, D), page_table=torch.tensor(ids[:B * P], dtype=i32).view(B, P),
             cache_len=torch.tensor(lens, dtype=i32))
    x["parents"] = None if tree == "chain" else torch.tensor([random_tree(rng, T) for _ in range(B)], dtype=i32)
    if tree == "forest" and T > 1:  # two trees that both continue the text
        x["parents"][:, T // 2] = -1
    x["n_nodes"] = None if nodes is None else torch.tensor(nodes, dtype=i32)
    used = torch.zeros(pages, ps, dtype=torch.bool)
    for b in range(B):
        at = torch.arange(lens[b])
        used[x["page_table"][b].long()[at // ps], at % ps] = True
        if nodes is not None:
            x["k_new"][b, nodes[b]:] = math.nan
            x["v_new"][b, nodes[b]:] = math.nan
    x["k_cache"][~used] = math.nan
    x["v_cache"][~used] = math.inf
    return x


def on_gpu(x):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}


def check_attention(x, got, scale=None, lse=None, fill=None):
    ref, ref_lse, tol, tol_lse, live = tree_ref.attention(x["q"], x["k_new"], x["v_new"], x["k_cache"], x["v_cache"],
                                                          x["page_table"], x["cache_len"], x["parents"], x["n_nodes"], scale)
    off = (got.double().cpu() - ref).abs()
    bad = int((~(off <= tol))[live].sum())  # (a NaN is bad)
    assert bad == 0, (bad, float((off / tol.clamp(min=1e-30))[live].max()))
    if lse is not None:
        bad = int((~((lse.double().cpu() - ref_lse).abs() <= tol_lse))[live].sum())
        assert bad == 0, bad
    if fill is not None:  # rows behind the last node are as they were
        left = bool((got.cpu()[~live] == fill).all())
        assert left


def run_attention(x, with_lse=True, scale=None):
    g = on_gpu(x)
    B, T, Hq, D = x["q"].shape
    out = mtp.TreeAttentionResult(torch.full((B, T, Hq, D), 7.0, dtype=x["q"].dtype, device="cuda"),
                                  torch.full((B, T, Hq), 7.0, device="cuda") if with_lse else None,
                                  torch.full((B,), 99, dtype=i32, device="cuda"))
    r = mtp.mtp_tree_attention(**g, scale=scale, out=out)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0] * B
    check_attention(x, r.out, scale, r.lse, 7.0)
    return r


ATTN = [
    # dtype, B, T, Hq, Hkv, D, page, lens, tree, nodes
    ("bf16", 1, 1, 8, 8, 128, 16, [0], "chain", None),
    ("bf16", 1, 1, 8, 2, 128, 16, [1], "chain", None),
    ("bf16", 3, 1, 8, 1, 64, 16, [15, 16, 17], "chain", None),
    ("bf16", 4, 4, 8, 2, 128, 64, [0, 63, 64, 129], "chain", None),
    ("bf16", 2, 7, 12, 4, 64, 16, [255, 300], "random", [7, 3]),
    ("bf16", 2, 64, 8, 1, 128, 128, [127, 513], "random", None),
    ("bf16", 3, 33, 4, 4, 128, 32, [128, 0, 1000], "random", [33, 0, 17]),
    ("bf16", 2, 64, 16, 1, 64, 256, [700, 511], "forest", [64, 40]),
    ("bf16", 2, 5, 16, 2, 256, 16, [70, 190], "random", None),
    ("bf16", 1, 40, 8, 1, 256, 64, [333], "random", None),
    ("bf16", 2, 9, 4, 2, 128, 24, [241, 119], "random", None),
    ("bf16", 2, 9, 4, 2, 128, 200, [420, 200], "random", None),
    ("bf16", 2, 3, 4, 2, 64, 1, [37, 5], "random", None),
    ("bf16", 2, 3, 4, 2, 128, 13, [137, 26], "random", None),
    ("bf16", 2, 6, 6, 2, 80, 16, [100, 31], "random", None),
    ("bf16", 1, 6, 5, 1, 33, 16, [50], "random", None),
    ("bf16", 1, 2, 8, 2, 128, 16, [5003], "chain", None),
    ("bf16", 1, 64, 32, 1, 64, 64, [2000], "random", None),
    ("bf16", 2, 64, 8, 1, 256, 32, [100, 64], "random", None),      # 512 rows of one key head
    ("bf16", 1, 64, 40, 1, 64, 64, [130], "random", [61]),           # 2560 rows: ten row tiles
    ("bf16", 2, 3, 128, 2, 128, 16, [77, 300], "random", None),
    ("f32", 1, 1, 4, 2, 64, 16, [0], "chain", None),
    ("f32", 4, 7, 8, 2, 64, 16, [1, 64, 65, 400], "random", [7, 1, 0, 5]),
    ("f32", 2, 64, 4, 1, 128, 24, [200, 77], "random", None),
    ("f32", 2, 3, 3, 3, 256, 16, [33, 90], "forest", None),
    ("f32", 2, 3, 3, 1, 50, 7, [33, 90], "random", None),
    ("f32", 1, 2, 4, 1, 128, 64, [4001], "chain", None),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(v) for v in c[:7]) + "-" + c[8])
def test_tree_attention(case):
    dtype, B, T, Hq, Hkv, D, ps, lens, tree, nodes = case
    run_attention(attn_case(sum(lens) + T, dtype, B, T, Hq, Hkv, D, ps, lens, tree, nodes))


@pytest.mark.parametrize("seed", range(40))
def test_tree_attention_random(seed):
    rng = random.Random(1000 + seed)
    B, T, Hkv = rng.randint(1, 6), rng.choice([1, 2, 3, 5, 8, 16, 31, 64]), rng.choice([1, 2, 3])
    G, D = rng.choice([1, 2, 3, 8]), rng.choice([64, 128, 256, 96])
    ps = rng.choice([8, 16, 24, 32, 40, 64, 100, 128, 136, 256])
    lens = [rng.choice([0, rng.randint(1, 40), rng.randint(1, 900)]) for _ in range(B)]
    nodes = [rng.randint(0, T) for _ in range(B)] if rng.random() < 0.5 else None
    run_attention(attn_case(seed, rng.choice(["bf16", "bf16", "f32"]), B, T, G * Hkv, Hkv, D, ps, lens,
                            rng.choice(["random", "chain", "forest"]), nodes), scale=rng.choice([None, 0.3]))


def test_tree_attention_no_sequences():
    x = on_gpu(attn_case(1, "bf16", 1, 2, 4, 2, 64, 16, [5]))
    for k in ("q", "k_new", "v_new", "page_table", "cache_len", "parents"):
        x[k] = x[k][:0]
    assert mtp.mtp_tree_attention(**x).out.shape == (0, 2, 4, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_attention_strides(dtype):
    """q, k and v as parts of one projection; a cache with heads outside the
    tokens, and one with keys and values in one tensor."""
    x = attn_case(3, dtype, 3, 5, 8, 2, 128, 16, [40, 77, 200])
    g = on_gpu(x)
    plain = run_attention(x)
    qkv = torch.cat([g["q"], g["k_new"], g["v_new"]], 2)
    g.update(q=qkv[:, :, :8], k_new=qkv[:, :, 8:10], v_new=qkv[:, :, 10:])
    both = torch.stack([g["k_cache"], g["v_cache"]], 1)
    for cache in ((both[:, 0], both[:, 1]),
                  tuple(c.transpose(1, 2).contiguous().transpose(1, 2) for c in (g["k_cache"], g["v_cache"]))):
        g.update(k_cache=cache[0], v_cache=cache[1])
        assert not cache[0].is_contiguous()
        r = mtp.mtp_tree_attention(**g, with_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(r.out, plain.out) and torch.equal(r.lse, plain.lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_attention_unaligned(dtype):
    """Tensors that start off a 16-byte boundary, and odd strides."""
    x = attn_case(4, dtype, 2, 4, 4, 2, 64, 16, [40, 77])
    g = on_gpu(x)

    def shift(t, extra):
        big = torch.full((*t.shape[:-1], t.shape[-1] + extra), math.nan, dtype=t.dtype, device="cuda")
        v = big[..., 1:1 + t.shape[-1]]
        v.copy_(t)
        return v

    for k in ("q", "k_new", "v_new", "k_cache", "v_cache"):
        g[k] = shift(g[k], 3)
    r = mtp.mtp_tree_attention(**g, with_lse=True)
    torch.cuda.synchronize()
    check_attention(x, r.out, None, r.lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tree_attention_values_out_of_sight(dtype, D):
    """Infinite and NaN values of a node reach the rows that see it and no
    others."""
    T = 6
    x = attn_case(5, dtype, 2, T, 4, 2, D, 16, [30, 150])
    x["parents"] = torch.tensor([[-1, 0, 0, 1, 2, 4]] * 2, dtype=i32)
    x["v_new"][0, 2, 0, 5] = math.inf
    x["v_new"][0, 2, 1, 7] = -math.inf
    x["v_new"][1, 4, 1, 9] = math.nan
    g = on_gpu(x)
    r = mtp.mtp_tree_attention(**g)
    torch.cuda.synchronize()
    y = dict(x, v_new=torch.where(x["v_new"].isfinite(), x["v_new"], torch.zeros_like(x["v_new"])))
    clean = mtp.mtp_tree_attention(**on_gpu(y)).out.cpu()
    want = clean.clone()
    want[0, [2, 4, 5], 0:2, 5] = math.inf
    want[0, [2, 4, 5], 2:4, 7] = -math.inf
    want[1, [4, 5], 2:4, 9] = math.nan
    assert torch.equal(r.out.cpu().isnan(), want.isnan())
    assert torch.equal(torch.nan_to_num(r.out.cpu(), nan=0.0, posinf=1e30, neginf=-1e30),
                       torch.nan_to_num(want, nan=0.0, posinf=1e30, neginf=-1e30))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_attention_extreme_scores(dtype):
    """Scores far apart, of one sign, and rising along the keys: the running
    maximum moves, weights underflow."""
    x = attn_case(6, dtype, 2, 8, 4, 2, 128, 16, [700, 333])
    ramp = torch.linspace(-40, 60, 16)[None, :, None, None]
    x["k_cache"] = (x["k_cache"] * (1 + ramp.abs() / 20)).to(x["k_cache"].dtype)
    for b in range(2):  # the last cached keys point along the first query
        pos = torch.arange(int(x["cache_len"][b]))
        page, row = x["page_table"][b].long()[pos // 16], pos % 16
        grow = (pos / 40.0)[:, None, None].to(x["q"].dtype)
        x["k_cache"][page, row] += grow * x["q"][b, 0, ::2][None]
    run_attention(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [128, 100])
def test_tree_attention_flags(dtype, D):
    """Bad lengths, counts, pages and parents flag their sequence alone; its
    rows are NaN and the others' results what they are without it."""
    x = attn_case(7, dtype, 7, 5, 4, 2, D, 16, [40, 77, 100, 20, 64, 50, 300])
    good = run_attention(x)
    g = on_gpu(x)
    P = g["page_table"].shape[1]
    g["n_nodes"] = torch.full((7,), 5, dtype=i32, device="cuda")
    g["cache_len"][1] = -1
    g["cache_len"][2] = P * 16 + 1
    g["n_nodes"][3] = 6
    g["page_table"][4, 2] = x["k_cache"].shape[0]
    g["parents"][5, 3] = 3
    g["page_table"][0, 3:] = -5          # beyond the sequence's tokens: not read
    g["page_table"][6, 0] = -1
    r = mtp.mtp_tree_attention(**g, with_lse=True)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0] + [mtp.ROW_BAD_ID] * 6
    assert r.out[1:].isnan().all() and r.lse[1:].isnan().all()
    check = dict(x, **{k: x[k][:1] for k in ("q", "k_new", "v_new", "page_table", "cache_len", "parents")})
    check_attention(check, r.out[:1], None, r.lse[:1])
    assert good.out.shape == r.out.shape


def test_tree_attention_batch_of_many_and_padded():
    """More sequences than a block has threads, most of them empty slots of a
    padded batch."""
    B = 700
    rng = random.Random(8)
    lens = [rng.randint(0, 60) if rng.random() < 0.5 else 0 for _ in range(B)]
    nodes = [rng.randint(0, 2) for _ in range(B)]
    run_attention(attn_case(8, "bf16", B, 2, 2, 1, 64, 16, lens, "random", nodes))


@pytest.mark.parametrize("dtype, T, Hq, D", [("bf16", 1, 8, 64), ("bf16", 4, 64, 128), ("bf16", 9, 32, 64), ("bf16", 2, 16, 256),
                                              ("f32", 2, 16, 64)])
def test_tree_attention_many_uneven(dtype, T, Hq, D):
    """More tiles than four for every CTA, whose split counts the units too:
    runs of sequences without a cache, single tokens and longer ones."""
    rng = random.Random(D + T)
    lens = [0] * 9 + [700] + [rng.choice([0, 1, 16, 128, 129, rng.randint(200, 699)]) for _ in range(34)] + [640, 0, 0, 0]
    run_attention(attn_case(71, dtype, len(lens), T, Hq, 8, D, 32, lens))


@pytest.mark.parametrize("T, Hq, D", [(1, 8, 64), (3, 16, 128), (9, 32, 64), (2, 16, 256)])
def test_tree_attention_many_uneven_split(T, Hq, D):
    """The same with lengths that are too many tiles to be left whole."""
    rng = random.Random(T)
    lens = [0] * 5 + [2300] + [rng.choice([0, 1, 128, 129, rng.randint(500, 2299)]) for _ in range(16)] + [1408, 0]
    run_attention(attn_case(72, "bf16", len(lens), T, Hq, 8, D, 32, lens))


@pytest.mark.parametrize("dtype, T, D", [("bf16", 3, 128), ("bf16", 33, 64), ("f32", 3, 64)])
def test_tree_attention_is_repeatable(dtype, T, D):
    """The split of long sequences joins in a fixed order: the same bits every time."""
    x = on_gpu(attn_case(9, dtype, 3, T, 8, 2, D, 64, [3001, 10, 777]))
    a = mtp.mtp_tree_attention(**x).out
    for _ in range(10):
        assert torch.equal(a, mtp.mtp_tree_attention(**x).out)


@pytest.mark.parametrize("D, T, Hq, Hkv, ps", [(64, 8, 8, 2, 32), (128, 8, 16, 2, 16), (128, 40, 16, 2, 16), (64, 3, 2, 1, 128),
                                               (256, 5, 8, 2, 32), (64, 64, 12, 2, 24)])
def test_tree_attention_back_to_back(D, T, Hq, Hkv, ps):
    """Many launches behind one another, each with many short and long pieces
    per CTA: the hand-over of shared memory between copies, loads and products
    must not depend on how they are timed."""
    rng = random.Random(D + T)
    lens = [rng.choice([0, 1, ps, 200, 900]) + rng.randint(0, 50) for _ in range(60)]
    x = attn_case(13, "bf16", 60, T, Hq, Hkv, D, ps, lens, nodes=[rng.randint(1, T) for _ in range(60)])
    a = run_attention(x).out
    g = on_gpu(x)
    out = mtp.TreeAttentionResult(torch.full_like(a, 7.0), None, torch.zeros(60, dtype=i32, device="cuda"))
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(400):
        mtp.mtp_tree_attention(**g, out=out)
        wrong += (out.out != a).sum() + out.row_flags.count_nonzero()
    assert wrong.item() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_attention_graphs_and_streams(dtype):
    """Two captured graphs with lengths that change between replays, replayed
    in turn and side by side on two streams, and a call on a given stream."""
    xs = [attn_case(10 + k, dtype, 3, 4, 8, 2, 128, 16, [200 + 300 * k, 64, 1500], room=20) for k in range(2)]
    gs = [on_gpu(x) for x in xs]
    outs, graphs = [], []
    for g in gs:
        mtp.mtp_tree_attention(**g)  # loads the library's kernels
    torch.cuda.synchronize()
    for g in gs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(mtp.mtp_tree_attention(**g, with_lse=True))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        for x, g in zip(xs, gs):
            n = torch.tensor([100 * turn, 64 - turn, 1500 - 700 * turn], dtype=i32)
            x["cache_len"] = n
            g["cache_len"].copy_(n)
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for x, o in zip(xs, outs):
            y = dict(x, k_cache=torch.nan_to_num(x["k_cache"], nan=0.0), v_cache=torch.nan_to_num(x["v_cache"], posinf=0.0))
            r = mtp.mtp_tree_attention(**on_gpu(x), with_lse=True, stream=streams[0])
            torch.cuda.synchronize()
            assert torch.equal(r.out, o.out) and torch.equal(r.lse, o.lse)
            if turn > 0:  # (all rows of these lengths hold numbers)
                check_attention(y, o.out, None, o.lse)


def test_tree_attention_far_pages():
    """Pages beyond 2^32 elements of a cache of 9 GB."""
    x = attn_case(12, "bf16", 2, 4, 8, 2, 128, 16, [100, 37])
    pages = (1 << 32) // (16 * 2 * 128) + 64
    big = torch.empty(pages, 16, 2, 128, dtype=bf16, device="cuda")
    far = torch.arange(pages - x["page_table"].numel(), pages, dtype=i32).view(x["page_table"].shape)
    big[far.long().cuda()] = x["k_cache"][x["page_table"].long()].cuda()
    g = on_gpu(x)
    # keys and values from one cache: the same rows serve as both
    y = dict(x, v_cache=x["k_cache"])
    g.update(k_cache=big, v_cache=big, page_table=far.cuda())
    r = mtp.mtp_tree_attention(**g, with_lse=True)
    torch.cuda.synchronize()
    check_attention(y, r.out, None, r.lse)


# ------------------------------------------------------- beam selection --

def check_select(z, scores, T, K, r):
    """Tokens and parents equal the reference's; where two candidates' scores
    lie closer than the kernel's error their order is either one.  The error
    of a score: a sum of 2^x with |x| rounded at 2^-24 of at most 2^8 and an
    approximate power (2^-21) -- 2^-15 at the very worst, and for these logits
    (|x| < 64) below 2^-17 -- and its own rounding."""
    for b, want in enumerate(tree_ref.select(z, scores, T, K)):
        tok, par, val = r.tokens[b].tolist(), r.parents[b].tolist(), r.scores[b].tolist()
        for i, w in enumerate(want):
            if w is None:
                assert (tok[i], par[i], val[i]) == (-1, -1, -math.inf)
                continue
            tol = 2.0 ** -17 + 2.0 ** -23 * abs(w[0])
            assert abs(val[i] - w[0]) <= tol, (b, i, val[i], w)
            if (par[i], tok[i]) != (w[1], w[2]):
                near = [v for v in want if v is not None and v != w and abs(v[0] - w[0]) <= 2 * tol and v[0] != w[0]]
                assert near, (b, i, (par[i], tok[i]), w)
        live = [(p, t) for p, t in zip(par, tok) if p >= 0]
        assert len(set(live)) == len(live)


def run_select(z, scores, T, K):
    r = mtp.mtp_beam_select(z.cuda(), scores.cuda(), T.cuda(), K)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0] * z.shape[0]
    r = mtp.BeamResult(*(t.cpu() for t in r))
    check_select(z, scores, T, K, r)
    return r


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B, W, V, K", [(1, 1, 1, 1), (2, 1, 5, 5), (3, 4, 3, 12), (2, 3, 1000, 7), (2, 5, 50257, 10),
                                        (1, 4, 151936, 8), (1, 1, 32000, 64), (3, 16, 4099, 33), (1, 64, 257, 64),
                                        (2, 2, 8191, 1), (20, 8, 2048, 16), (1, 3, 20011, 64)])
def test_beam_select(dtype, B, W, V, K):
    g = torch.Generator().manual_seed(V + K)
    z = (torch.randn(B, W, V, generator=g) * 3).to(DTYPES[dtype])
    scores = -torch.rand(B, W, generator=g).cumsum(1)
    run_select(z, scores, 0.5 + torch.rand(B, generator=g), K)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [4096, 40001])
def test_beam_select_ties(dtype, V):
    """Equal logits and equal rows: the smaller beam, then the smaller token.
    Rows of one value, of few values, and the same row in every beam, at
    every alignment."""
    g = torch.Generator().manual_seed(V)
    row = torch.randint(0, 4, (V,), generator=g).float()
    z = torch.stack([torch.zeros(V), torch.zeros(V), row, row, row]).to(DTYPES[dtype])
    z = torch.stack([z, z[[2, 2, 2, 2, 2]], z[[0, 0, 0, 0, 0]]])
    r = run_select(z, torch.zeros(3, 5), torch.ones(3), 40)
    assert r.parents[1].tolist() == [0] * 40 and r.parents[2].tolist() == [0] * 40
    assert r.tokens[2].tolist() == list(range(40))
    top = torch.nonzero(z[1, 0] == 3).flatten()[:40].tolist()
    assert r.tokens[1].tolist() == top


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("order", ["up", "down", "equal then up"])
def test_beam_select_sorted_rows(dtype, order):
    """Rows in rising order pass every candidate on: the list overflows and is
    cut again and again."""
    V, K = 151936 // 2, 64
    x = torch.linspace(-20, 20, V)
    if order == "down":
        x = x.flip(0)
    if order == "equal then up":
        x[: V // 2] = -20
    z = x.to(DTYPES[dtype])[None, None].expand(40, 8, V).contiguous()
    r = mtp.mtp_beam_select(z.cuda(), torch.linspace(0, -3, 8).expand(40, 8).contiguous().cuda(), torch.ones(40).cuda(), K)
    torch.cuda.synchronize()
    check_select(z[:1], torch.linspace(0, -3, 8)[None], torch.ones(1), K, mtp.BeamResult(*(t[:1].cpu() for t in r)))
    assert (r.tokens == r.tokens[:1]).all() and (r.parents == r.parents[:1]).all() and (r.scores == r.scores[:1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_beam_select_masked_and_dead(dtype):
    """-inf logits are never selected, dead beams are not read (NaN there),
    and places without a candidate are empty."""
    g = torch.Generator().manual_seed(1)
    z = torch.randn(4, 3, 5003, generator=g).to(DTYPES[dtype])
    scores = torch.zeros(4, 3)
    z[0, :, 5:] = -math.inf                     # 15 candidates
    z[1, 1] = math.nan
    scores[1, 1] = -math.inf
    scores[2] = -math.inf                       # no live beam
    z[2] = math.inf
    z[3, 0, 1:] = -math.inf
    z[3, 1:, :2] = -math.inf
    r = run_select(z, scores, torch.ones(4), 20)
    assert (r.tokens[0] >= 0).sum() == 15 and (r.tokens[2] == -1).all() and (r.parents[1] != 1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_beam_select_flags(dtype):
    z = torch.randn(8, 2, 9001).to(DTYPES[dtype])
    scores, T = torch.zeros(8, 2), torch.ones(8)
    z[1, 1, 8999] = math.nan
    z[2, 0, 17] = math.inf
    z[3, 1] = -math.inf
    scores[4, 0] = math.nan
    scores[5, 1] = math.inf
    T[6], T[7] = 0.0, -1.0
    r = mtp.mtp_beam_select(z.cuda(), scores.cuda(), T.cuda(), 6)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0] + [mtp.ROW_NONFINITE] * 5 + [mtp.ROW_BAD_TEMP] * 2
    assert (r.tokens[1:] == -1).all() and (r.parents[1:] == -1).all() and r.scores[1:].isnan().all()
    check_select(z[:1], scores[:1], T[:1], 6, mtp.BeamResult(*(t[:1].cpu() for t in r)))
    for bad in (math.nan, math.inf):
        r = mtp.mtp_beam_select(z[:1].cuda(), scores[:1].cuda(), torch.tensor([bad]).cuda(), 6)
        assert r.row_flags.tolist() == [mtp.ROW_BAD_TEMP]


def test_beam_select_graph_and_stream():
    g = torch.Generator().manual_seed(2)
    z, scores, T = torch.randn(2, 4, 30011, generator=g).cuda(), torch.zeros(2, 4).cuda(), torch.ones(2).cuda()
    mtp.mtp_beam_select(z, scores, T, 9)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = mtp.mtp_beam_select(z, scores, T, 9)
    for seed in range(3):
        z.copy_(torch.randn(2, 4, 30011, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        check_select(z.cpu(), scores.cpu(), T.cpu(), 9, mtp.BeamResult(*(t.cpu() for t in o)))
        s = torch.cuda.Stream()
        r = mtp.mtp_beam_select(z, scores, T, 9, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, r))


# --------------------------------------------------- reorder and commit ----

@pytest.mark.parametrize("dtype", [bf16, f32, torch.uint8, torch.float64])
@pytest.mark.parametrize("N0, B, W, K, rest", [(1, 1, 1, 1, (1,)), (2, 3, 4, 4, (5, 3)), (1, 5, 8, 8, (4096,)), (3, 2, 3, 7, (1001,)),
                                               (1, 2, 5, 2, ()), (2, 300, 2, 128, (33,)), (1, 1, 2, 2, (70001,))])
def test_beam_reorder(dtype, N0, B, W, K, rest):
    g = torch.Generator().manual_seed(K)
    x = (torch.randn(N0, B, W, *rest, generator=g) * 50).to(dtype)
    up = torch.randint(0, W, (B, K), generator=g, dtype=i32)
    r = mtp.mtp_beam_reorder(x.cuda(), up.cuda())
    torch.cuda.synchronize()
    want = torch.stack([torch.stack([x[:, b, p] for p in up[b].tolist()], 1) for b in range(B)], 1)
    assert torch.equal(r.states.cpu(), want) and r.row_flags.tolist() == [0] * B


def test_beam_reorder_unaligned_and_bad_parents():
    flat = torch.arange(1 + 2 * 3 * 4 * 101, dtype=f32).to(bf16).cuda()
    x = flat[1:].view(2, 3, 4, 101)
    up = torch.tensor([[0, 3, -1], [2, 2, 2], [4, 0, 1]], dtype=i32).cuda()
    out = mtp.ReorderResult(torch.ones(2 * 3 * 3 * 101 + 3, dtype=bf16, device="cuda")[3:].view(2, 3, 3, 101),
                            torch.full((3,), 9, dtype=i32, device="cuda"))
    r = mtp.mtp_beam_reorder(x, up, out=out)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [mtp.ROW_BAD_ID, 0, mtp.ROW_BAD_ID]
    for b in range(3):
        for k, p in enumerate(up[b].tolist()):
            want = x[:, b, p] if 0 <= p < 4 else torch.zeros_like(x[:, b, 0])
            assert torch.equal(r.states[:, b, k], want)


def test_beam_reorder_flags_on_another_stream():
    """The flags are the kernel's alone: nothing that the call queues on the
    current stream, busy here, writes them later."""
    states = torch.randn(1, 2, 3, 8, device="cuda")
    parents = torch.tensor([[0, 3], [1, 2]], dtype=i32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    r = mtp.mtp_beam_reorder(states, parents, stream=side)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [mtp.ROW_BAD_ID, 0]
    assert torch.equal(r.states[0, 1], states[0, 1, 1:])


@pytest.mark.parametrize("shape", [(0, 2, 3, 4), (2, 2, 3, 0)])
def test_beam_reorder_no_bytes(shape):
    flags = torch.full((2,), 9, dtype=i32, device="cuda")
    states = torch.zeros(shape, device="cuda")
    out = mtp.ReorderResult(torch.empty_like(states), flags)
    r = mtp.mtp_beam_reorder(states, torch.zeros(2, 3, dtype=i32, device="cuda"), out=out)
    assert r.row_flags.tolist() == [0, 0]


def test_beam_reorder_overlap_is_refused():
    x = torch.zeros(1, 2, 4, 8, device="cuda")
    up = torch.zeros(2, 4, dtype=i32, device="cuda")
    with pytest.raises(mtp.MTPError):
        mtp.mtp_beam_reorder(x, up, out=mtp.ReorderResult(x, None))


def commit_case(seed, dtype, layers, B, T, Hkv, D, ps, lens, agree=0.8, nodes=None, tree="random"):
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    P = -(-(max(lens) + T) // ps)
    ids = list(range(B * P + 1))
    rng.shuffle(ids)
    n = lambda *s: torch.randn(*s, generator=g).to(DTYPES[dtype])  # noqa: E731
    tokens = [[rng.randrange(40) for _ in range(T)] for _ in range(B)]
    up = [list(range(-1, T - 1)) if tree == "chain" else random_tree(rng, T, 4) for _ in range(B)]
    target = [[rng.randrange(40) for _ in range(T)] for _ in range(B)]
    for b in range(B):
        for i in range(1, T):
            if rng.random() < agree:
                target[b][up[b][i]] = tokens[b][i]
    t = lambda v: torch.tensor(v, dtype=i32)  # noqa: E731
    return dict(tokens=t(tokens), target_tokens=t(target), parents=None if tree == "chain" else t(up), k_new=n(layers, B, T, Hkv, D),
                v_new=n(layers, B, T, Hkv, D), k_cache=n(layers, B * P + 1, ps, Hkv, D), v_cache=n(layers, B * P + 1, ps, Hkv, D),
                page_table=t(ids[:B * P]).view(B, P), cache_len=t(lens), n_nodes=None if nodes is None else t(nodes))


def check_commit(x, r, k_cache, v_cache, skip=()):
    B, T = x["tokens"].shape
    ps = x["k_cache"].shape[-3]
    K, V = x["k_cache"].clone(), x["v_cache"].clone()
    for b in range(B):
        n = T if x["n_nodes"] is None else int(x["n_nodes"][b])
        L = int(x["cache_len"][b])
        if n == 0 or b in skip:
            assert r.accept_len[b] == -1 and (r.tokens[b] == -1).all() and (r.path[b] == -1).all() and r.cache_len[b] == L
            continue
        up = list(range(-1, T - 1)) if x["parents"] is None else x["parents"][b].tolist()
        tok, tgt = x["tokens"][b].tolist(), x["target_tokens"][b].tolist()
        path = tree_ref.commit_path(tok, tgt, up, n)
        for j, i in enumerate(path):
            page, row = int(x["page_table"][b, (L + j) // ps]), (L + j) % ps
            K[..., page, row, :, :] = x["k_new"][..., b, i, :, :]
            V[..., page, row, :, :] = x["v_new"][..., b, i, :, :]
        pad = [-1] * (T - len(path))
        assert r.path[b].tolist() == path + pad
        assert r.tokens[b].tolist() == [tok[i] for i in path[1:]] + [tgt[path[-1]]] + pad
        assert r.accept_len[b] == len(path) - 1 and r.cache_len[b] == L + len(path)
    assert torch.equal(k_cache.cpu(), K) and torch.equal(v_cache.cpu(), V)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layers, B, T, Hkv, D, ps, lens, nodes, tree", [
    (1, 1, 1, 1, 8, 4, [0], None, "chain"),
    (1, 2, 8, 2, 64, 16, [15, 0], None, "random"),
    (3, 4, 33, 2, 64, 16, [1, 31, 32, 100], [33, 0, 1, 20], "random"),
    (2, 3, 64, 1, 128, 24, [5, 60, 0], None, "random"),
    (2, 2, 64, 1, 16, 8, [5, 60], None, "chain"),
    (1, 3, 6, 3, 33, 5, [4, 5, 6], None, "random"),
])
def test_tree_commit(dtype, layers, B, T, Hkv, D, ps, lens, nodes, tree):
    x = commit_case(T + B, dtype, layers, B, T, Hkv, D, ps, lens, 0.97 if tree == "chain" else 0.8, nodes, tree)
    g = on_gpu(x)
    r = mtp.mtp_tree_commit(**g)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0] * B
    check_commit(x, mtp.CommitResult(*(t.cpu() for t in r)), g["k_cache"], g["v_cache"])
    again = mtp.mtp_tree_commit(**g)  # the same call writes the same again
    torch.cuda.synchronize()
    check_commit(x, mtp.CommitResult(*(t.cpu() for t in again)), g["k_cache"], g["v_cache"])


def test_tree_commit_one_layer_and_strides():
    x = commit_case(3, "bf16", 1, 3, 9, 2, 64, 16, [3, 16, 40])
    g = on_gpu(x)
    kv = torch.stack([g["k_cache"][0], g["v_cache"][0]], 1)          # [pages, 2, page, heads, D]
    new = torch.cat([g["k_new"][0], g["v_new"][0]], 2)               # [B, T, 2 heads, D]
    y = dict(g, k_cache=kv[:, 0], v_cache=kv[:, 1], k_new=new[:, :, :2], v_new=new[:, :, 2:])
    r = mtp.mtp_tree_commit(**y)
    torch.cuda.synchronize()
    check_commit(x, mtp.CommitResult(*(t.cpu() for t in r)), kv[:, 0][None], kv[:, 1][None])


def test_tree_commit_flags():
    x = commit_case(4, "bf16", 2, 7, 6, 2, 64, 8, [10] * 7, 1.0)
    g = on_gpu(x)
    P = x["page_table"].shape[1]
    g["n_nodes"] = torch.full((7,), 6, dtype=i32, device="cuda")
    for y in (x, g):
        y["cache_len"][1] = P * 8           # full: no room for the root
        y["parents"][3, 4] = 5
        y["target_tokens"][4, 0] = -1       # a flagged draw
        y["page_table"][5, 1] = x["k_cache"].shape[1]
        y["parents"][6, 0] = 0              # node 0 has to be the root
    g["n_nodes"][2] = 7
    r = mtp.mtp_tree_commit(**g)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0] + [mtp.ROW_BAD_ID] * 6
    check_commit(x, mtp.CommitResult(*(t.cpu() for t in r)), g["k_cache"], g["v_cache"], skip=range(1, 7))


# ------------------------------------------------------------- together ----

def test_draft_attend_verify_commit():
    """Greedy decoding of a small model with drafted trees gives the tokens of
    plain decoding: the drafter's tree is grown by beam selection, the target
    attends from every node over the paged cache, its arg max after every node
    (draft_sample at T = 0) verifies the tree, and the commit extends the
    cache."""
    torch.manual_seed(0)
    B, V, Hq, Hkv, D, ps, W, steps = 3, 64, 4, 2, 64, 16, 3, 30
    dev = "cuda"
    E = torch.randn(V, Hq * D) * 0.7
    Wq, Wk, Wv = (torch.randn(Hq * D, n * D) * (Hq * D) ** -0.5 for n in (Hq, Hkv, Hkv))
    Wo = torch.randn(Hq * D, Hq * D) * (Hq * D) ** -0.5 * 3
    start = [[3], [17, 4, 4, 9], [50] * 20]

    def greedy(text):
        text = list(text)
        e, wq, wk, wv, wo = (t.double() for t in (E, Wq, Wk, Wv, Wo))
        for _ in range(steps):
            x = e[text]
            k, v = (x @ wk).view(-1, Hkv, D), (x @ wv).view(-1, Hkv, D)
            q = (x[-1] @ wq).view(Hkv, Hq // Hkv, D)
            a = torch.softmax(torch.einsum("hgd,shd->hgs", q, k) * D ** -0.5, -1)
            o = torch.einsum("hgs,shd->hgd", a, v).reshape(-1)
            text.append(int(((o @ wo + 0.3 * x[-1]) @ e.T).argmax()))
        return text

    want = [greedy(t) for t in start]
    # a drafter that knows which words followed which, and some noise: often right
    follow = torch.randn(V, V)
    for t in want:
        for a, b in zip(t, t[1:]):
            follow[a, b] += 4
    follow = follow.to(dev)
    E, Wq, Wk, Wv, Wo = (t.to(dev) for t in (E, Wq, Wk, Wv, Wo))
    pages = B * 8 + 1
    kc, vc = torch.zeros(pages, ps, Hkv, D, device=dev), torch.zeros(pages, ps, Hkv, D, device=dev)
    table = torch.randperm(pages)[:B * 8].view(B, 8).to(i32).to(dev)
    lens = torch.zeros(B, dtype=i32, device=dev)
    for b, t in enumerate(start):  # the prompt but its last token is in the cache
        for i, w in enumerate(t[:-1]):
            kc[table[b, i // ps].long(), i % ps] = (E[w] @ Wk).view(Hkv, D)
            vc[table[b, i // ps].long(), i % ps] = (E[w] @ Wv).view(Hkv, D)
        lens[b] = len(t) - 1
    root = torch.tensor([t[-1] for t in start], dtype=i32, device=dev)
    text = [list(t) for t in start]
    one = torch.ones(B, device=dev)
    passes = accepted = 0
    while min(len(t) - len(s) for t, s in zip(text, start)) < steps:
        # level 0: the root; two more levels of W beams each
        tokens, parents = [root[:, None]], [torch.full((B, 1), -1, dtype=i32, device=dev)]
        state, scores, ids = E[root.long()][None, :, None], torch.zeros(B, 1, device=dev), torch.zeros(B, 1, dtype=i32, device=dev)
        for level in range(2):
            last = tokens[-1].long()
            s = mtp.mtp_beam_select(follow[last].contiguous(), scores, one, W)
            up = torch.gather(ids, 1, s.parents.long())
            state = mtp.mtp_beam_reorder(state.contiguous(), s.parents).states
            assert torch.equal(state[0], torch.gather(E[last], 1, s.parents.long()[:, :, None].expand(-1, -1, Hq * D)))
            state = E[s.tokens.long()][None]
            scores, ids = s.scores, torch.arange(1 + level * W, 1 + (level + 1) * W, dtype=i32, device=dev).expand(B, W)
            tokens.append(s.tokens)
            parents.append(up)
        tokens, parents = torch.cat(tokens, 1), torch.cat(parents, 1)
        T = tokens.shape[1]
        x = E[tokens.long()]
        q, k, v = (x @ Wq).view(B, T, Hq, D), (x @ Wk).view(B, T, Hkv, D), (x @ Wv).view(B, T, Hkv, D)
        o = mtp.mtp_tree_attention(q, k, v, kc, vc, table, lens, parents).out
        logits = (o.view(B, T, -1) @ Wo + 0.3 * x) @ E.T
        draw = mtp.mtp_draft_sample(logits.view(B * T, V).contiguous(), torch.zeros(B * T, device=dev),
                                    torch.zeros(B * T, device=dev)).ids.view(B, T)
        r = mtp.mtp_tree_commit(tokens, draw, parents, k, v, kc, vc, table, lens)
        lens = r.cache_len
        for b in range(B):
            n = int(r.accept_len[b])
            text[b] += r.tokens[b, :n + 1].tolist()
            accepted += n
        root = torch.gather(r.tokens, 1, r.accept_len[:, None].long())[:, 0].contiguous()
        passes += 1
    for t, w in zip(text, want):
        assert t[:len(w)] == w
    assert accepted > 0
