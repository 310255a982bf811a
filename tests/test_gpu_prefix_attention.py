"""Attention with shared prefixes on the GPU against the plain 64-bit form of
tree attention (tests/tree_ref.py, which derives the tolerances) over each
sequence's prefix and own tokens in one text."""
import math
import random

import pytest
import torch

import mtp_speculative_decoding_row_gb300 as mtp
from tests import tree_ref

pytestmark = pytest.mark.gpu
i32, f32, bf16 = torch.int32, torch.float32, torch.bfloat16
DTYPES = {"f32": f32, "bf16": bf16}
PER_SEQUENCE = ("q", "k_new", "v_new", "page_table", "cache_len", "parents", "n_nodes")


@pytest.fixture(scope="module", autouse=True)
def library():
    from tests import gpu_util

    gpu_util.ensure_library()


def prefix_case(seed, dtype, sizes, plens, T, Hq, Hkv, D, ps, lens, tree="random", nodes=None, room=0):
    """CPU inputs: prefix p of plens[p] tokens has sizes[p] sequences.  Pages in
    random order, NaN in every cache row that nothing has and in the new rows of
    nodes that a sequence lacks."""
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[dtype]
    B, P = sum(sizes), len(sizes)
    W, Wp = (max(1, -(-max(n, default=0) // ps)) + room for n in (lens, plens))
    pages = B * W + P * Wp + 2
    ids = list(range(pages))
    rng.shuffle(ids)
    n = lambda *s: torch.randn(*s, generator=g).to(dt)  # noqa: E731
    starts = [sum(sizes[:p]) for p in range(P + 1)]
    x = dict(q=n(B, T, Hq, D) * 2, k_new=n(B, T, Hkv, D), v_new=n(B, T, Hkv, D), k_cache=n(pages, ps, Hkv, D), v_cache=n(pages, ps, Hkv, D),
             prefix_table=torch.tensor(ids[B * W:B * W + P * Wp], dtype=i32).view(P, Wp), prefix_len=torch.tensor(plens, dtype=i32),
             group_start=torch.tensor(starts, dtype=i32), page_table=torch.tensor(ids[:B * W], dtype=i32).view(B, W),
             cache_len=torch.tensor(lens, dtype=i32))
    x["parents"] = None if tree == "chain" else torch.tensor([[-1] + [rng.randint(max(-1, i - 8), i - 1) for i in range(1, T)] for _ in range(B)],
                                                             dtype=i32).view(B, T)
    x["n_nodes"] = None if nodes is None else torch.tensor(nodes, dtype=i32)
    used = torch.zeros(pages, ps, dtype=torch.bool)
    for table, counts in ((x["page_table"], lens), (x["prefix_table"], plens)):
        for b, c in enumerate(counts):
            at = torch.arange(c)
            used[table[b].long()[at // ps], at % ps] = True
    if nodes is not None:
        for b in range(B):
            x["k_new"][b, nodes[b]:] = math.nan
            x["v_new"][b, nodes[b]:] = math.nan
    x["k_cache"][~used] = math.nan
    x["v_cache"][~used] = math.inf
    return x


def one_text(x):
    """The arguments of tree_ref.attention: every token a page of its own, the prefix's before the sequence's."""
    ps = x["k_cache"].shape[1]
    starts = x["group_start"].tolist()
    rows = []
    for b in range(x["q"].shape[0]):
        p = [i for i in range(len(starts) - 1) if starts[i] <= b < starts[i + 1]][0]
        row = []
        for table, n in ((x["prefix_table"][p], int(x["prefix_len"][p])), (x["page_table"][b], int(x["cache_len"][b]))):
            at = torch.arange(n)
            row.append(table.long()[at // ps] * ps + at % ps)
        rows.append(torch.cat(row))
    table = torch.zeros(len(rows), max(max(len(r) for r in rows), 1), dtype=i32)
    for b, r in enumerate(rows):
        table[b, :len(r)] = r
    return (x["q"], x["k_new"], x["v_new"], x["k_cache"].flatten(0, 1)[:, None], x["v_cache"].flatten(0, 1)[:, None], table,
            torch.tensor([len(r) for r in rows]), x["parents"], x["n_nodes"])


def on_gpu(x):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in x.items()}


def check(x, out, lse, scale=None, fill=None):
    ref, ref_lse, tol, tol_lse, live = tree_ref.attention(*one_text(x), scale)
    off = (out.double().cpu() - ref).abs()
    bad = int((~(off <= tol))[live].sum())  # (a NaN is bad)
    assert bad == 0, (bad, float((off / tol.clamp(min=1e-30))[live].max()))
    if lse is not None:
        bad = int((~((lse.double().cpu() - ref_lse).abs() <= tol_lse))[live].sum())
        assert bad == 0, bad
    if fill is not None:
        assert bool((out.cpu()[~live] == fill).all())


def run(x, scale=None):
    g = on_gpu(x)
    B, T, Hq, D = x["q"].shape
    out = mtp.TreeAttentionResult(torch.full((B, T, Hq, D), 7.0, dtype=x["q"].dtype, device="cuda"), torch.full((B, T, Hq), 7.0, device="cuda"),
                                  torch.full((B,), 99, dtype=i32, device="cuda"))
    r = mtp.mtp_prefix_attention(**g, scale=scale, out=out)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [0] * B
    check(x, r.out, r.lse, scale, 7.0)
    return r


CASES = [
    # dtype, sizes, plens, T, Hq, Hkv, D, page, lens, tree, nodes
    ("bf16", [1], [1], 1, 1, 1, 64, 16, [0], "chain", None),
    ("bf16", [4], [100], 1, 8, 2, 128, 16, [0, 1, 16, 50], "chain", None),
    ("bf16", [3], [0], 2, 8, 2, 128, 16, [5, 0, 40], "chain", None),
    ("bf16", [2, 0, 5, 1], [130, 50, 0, 257], 3, 8, 2, 64, 32, [3, 70, 0, 0, 1, 33, 64, 200], "random", None),
    ("bf16", [40], [700], 4, 8, 2, 128, 64, [0] * 20 + [65] * 20, "chain", None),               # 640 rows of a head: three row tiles
    ("bf16", [9, 11], [513, 90], 3, 10, 2, 128, 24, [7] * 20, "random", [3, 0, 1, 2] * 5),     # tiles that end inside a token's heads
    ("bf16", [5, 3], [300, 1000], 2, 8, 4, 256, 16, [17, 0, 3, 90, 40, 12, 64, 65], "random", None),
    ("bf16", [16], [333], 5, 16, 2, 256, 64, [20] * 16, "random", None),
    ("bf16", [2, 2], [2000, 3000], 1, 32, 8, 128, 16, [10, 20, 30, 40], "chain", None),
    ("bf16", [1] * 12, list(range(0, 1200, 100)), 2, 4, 2, 128, 16, [9] * 12, "random", None),
    ("bf16", [33], [1], 1, 7, 1, 128, 200, [1] * 33, "chain", None),
    ("bf16", [7, 1], [150, 420], 3, 6, 3, 80, 16, [31, 0, 5, 6, 7, 8, 9, 10], "random", None),  # no tensor cores
    ("bf16", [3], [137], 2, 4, 2, 64, 13, [13, 26, 0], "random", None),
    ("bf16", [2], [40], 64, 8, 1, 64, 16, [12, 100], "random", [64, 33]),
    ("bf16", [1, 60], [90, 400], 1, 4, 1, 64, 16, [5] * 61, "chain", None),                    # one prefix has nearly all sequences
    ("bf16", [3, 4], [300, 77], 4, 16, 2, 128, 64, [0, 1, 130, 128, 400, 5, 60], "random", [4, 0, 2, 4, 1, 3, 4]),  # 32 rows of a key head
    ("bf16", [1, 2, 1], [700, 300, 15], 2, 8, 2, 256, 32, [3, 0, 129, 1000], "random", None),
    ("bf16", [1, 1], [5000, 129], 3, 10, 2, 128, 16, [2000, 33], "chain", None),
    ("bf16", [2], [5000], 5, 3, 1, 256, 128, [900, 127], "random", [5, 4]),
    ("bf16", [1] * 70, [40] * 70, 1, 4, 1, 128, 8, [3] * 70, "chain", None),
    ("f32", [4], [100], 1, 8, 2, 64, 16, [0, 1, 16, 50], "chain", None),
    ("f32", [2, 0, 5, 1], [130, 50, 0, 257], 3, 8, 2, 128, 32, [3, 70, 0, 0, 1, 33, 64, 200], "random", [3, 3, 1, 0, 2, 3, 3, 2]),
    ("f32", [13], [999], 3, 9, 3, 50, 7, [8] * 13, "random", None),
    ("f32", [2, 3], [65, 64], 2, 3, 1, 256, 16, [1, 2, 3, 4, 5], "random", None),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:8]).replace(" ", ""))
def test_prefix_attention(case):
    dtype, sizes, plens, T, Hq, Hkv, D, ps, lens, tree, nodes = case
    run(prefix_case(sum(plens) + T, dtype, sizes, plens, T, Hq, Hkv, D, ps, lens, tree, nodes))


@pytest.mark.parametrize("seed", range(40))
def test_prefix_attention_random(seed):
    rng = random.Random(7000 + seed)
    sizes = [rng.choice([0, 1, 2, rng.randint(1, 20)]) for _ in range(rng.randint(1, 5))]
    sizes[rng.randrange(len(sizes))] += 1
    B, T, Hkv = sum(sizes), rng.choice([1, 1, 2, 4, 7, 20]), rng.choice([1, 2, 3])
    G, D = rng.choice([1, 2, 3, 5, 8]), rng.choice([64, 128, 128, 256, 96])
    plens = [rng.choice([0, rng.randint(1, 200), rng.randint(1, 1500)]) for _ in sizes]
    lens = [rng.choice([0, rng.randint(1, 40), rng.randint(1, 300)]) for _ in range(B)]
    nodes = [rng.randint(0, T) for _ in range(B)] if rng.random() < 0.5 else None
    run(prefix_case(seed, rng.choice(["bf16", "bf16", "f32"]), sizes, plens, T, G * Hkv, Hkv, D, rng.choice([8, 16, 24, 64, 100, 128, 256]), lens,
                    rng.choice(["random", "chain"]), nodes), scale=rng.choice([None, 0.3]))


@pytest.mark.parametrize("dtype, D", [("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_prefix_attention_is_tree_attention(dtype, D):
    """Without prefixes the results are those of tree attention over the same
    tokens, and a prefix in pages before a sequence's own gives the same text."""
    x = prefix_case(20, dtype, [6], [0], 3, 8, 2, D, 16, [0, 5, 100, 64, 33, 700])
    r = run(x)
    g = on_gpu({k: x[k] for k in PER_SEQUENCE + ("k_cache", "v_cache")})
    t = mtp.mtp_tree_attention(**g, with_lse=True)
    eps = torch.finfo(r.out.dtype).eps
    assert (r.out.double() - t.out.double()).abs().max() <= 8 * eps * t.out.double().abs().max()
    y = prefix_case(21, dtype, [3], [48], 3, 8, 2, D, 16, [20, 0, 64])
    r = run(y)
    both = torch.cat([y["prefix_table"].expand(3, -1), y["page_table"]], 1).contiguous()
    g = on_gpu(dict({k: y[k] for k in PER_SEQUENCE + ("k_cache", "v_cache")}, page_table=both, cache_len=y["cache_len"] + 48))
    t = mtp.mtp_tree_attention(**g, with_lse=True)
    assert (r.out.double() - t.out.double()).abs().max() <= 8 * eps * t.out.double().abs().max()


@pytest.mark.parametrize("dtype, D", [("bf16", 128), ("bf16", 64), ("f32", 100)])
def test_prefix_attention_strides(dtype, D):
    """q, k and v as parts of one projection, sequences and tokens in another
    order in memory, heads of the cache outside its tokens, odd addresses."""
    x = prefix_case(22, dtype, [4, 3], [200, 77], 3, 8, 2, D, 16, [40, 0, 7, 100, 16, 3, 90])
    a = run(x)
    g = on_gpu(x)
    qkv = torch.cat([g["q"], g["k_new"], g["v_new"]], 2)
    for order in (qkv, qkv.transpose(0, 1).contiguous().transpose(0, 1)):
        g.update(q=order[:, :, :8], k_new=order[:, :, 8:10], v_new=order[:, :, 10:])
        for c in ("k_cache", "v_cache"):
            g[c] = x[c].cuda().transpose(1, 2).contiguous().transpose(1, 2)
        r = mtp.mtp_prefix_attention(**g, with_lse=True)
        assert torch.equal(r.out, a.out) and torch.equal(r.lse, a.lse)
    odd = torch.zeros(*x["q"].shape[:3], D + 3, dtype=x["q"].dtype, device="cuda")[..., 1:D + 1]
    g["q"] = odd.copy_(x["q"])
    r = mtp.mtp_prefix_attention(**g, with_lse=True)
    check(x, r.out, r.lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [128, 100])
def test_prefix_attention_flags(dtype, D):
    """Bad lengths, counts, pages and parents of a sequence flag it alone, those of
    a prefix its sequences; all their rows are NaN, the others as without them."""
    sizes, plens = [3, 2, 2, 1, 2], [200, 90, 64, 300, 40]
    x = prefix_case(23, dtype, sizes, plens, 4, 4, 2, D, 16, [40, 77, 100, 20, 64, 50, 30, 8, 9, 10])
    good = run(x)
    g = on_gpu(x)
    g["n_nodes"] = torch.full((10,), 4, dtype=i32, device="cuda")
    g["cache_len"][1] = -1
    g["n_nodes"][2] = 5
    g["prefix_len"][1] = x["prefix_table"].shape[1] * 16 + 1          # sequences 3 and 4
    g["prefix_table"][2, 3] = -1                                      # the last page of 5's and 6's prefix
    g["prefix_table"][4, 3:] = -5                                     # beyond the prefix: not read
    g["parents"][7, 2] = 2
    r = mtp.mtp_prefix_attention(**g, with_lse=True)
    torch.cuda.synchronize()
    bad = [1, 2, 3, 4, 5, 6, 7]
    assert r.row_flags.tolist() == [mtp.ROW_BAD_ID if b in bad else 0 for b in range(10)]
    assert r.out[bad].isnan().all() and r.lse[bad].isnan().all()
    fine = [0, 8, 9]
    assert torch.equal(r.out[fine], good.out[fine]) and torch.equal(r.lse[fine], good.lse[fine])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("starts", [[1, 3, 6], [0, 3, 5], [0, 7, 6], [0, -2, 6], [-1, 3, 6], [6, 0, 6], [0, 4, 2 ** 31 - 1], [-2 ** 31, 0, 6]])
def test_prefix_attention_bad_groups(dtype, starts):
    x = on_gpu(prefix_case(24, dtype, [3, 3], [100, 200], 2, 4, 2, 64, 16, [5, 6, 7, 8, 9, 0]))
    x["group_start"] = torch.tensor(starts, dtype=i32, device="cuda")
    r = mtp.mtp_prefix_attention(**x, with_lse=True)
    torch.cuda.synchronize()
    assert r.row_flags.tolist() == [mtp.ROW_BAD_ID] * 6 and r.out.isnan().all() and r.lse.isnan().all()


@pytest.mark.parametrize("dtype, D, Hq", [("bf16", 128, 8), ("bf16", 128, 20), ("bf16", 256, 8), ("f32", 64, 8)])
def test_prefix_attention_repeatable_back_to_back(dtype, D, Hq):
    """The same bits every time, many launches behind one another."""
    rng = random.Random(D)
    sizes = [rng.randint(0, 12) for _ in range(7)] + [1]
    x = prefix_case(25, dtype, sizes, [rng.choice([0, 1, 130, 700, 1500]) for _ in sizes], 3, Hq, 2, D, 32,
                    [rng.choice([0, 1, 60, 200]) for _ in range(sum(sizes))])
    a = run(x)
    g = on_gpu(x)
    out = mtp.TreeAttentionResult(torch.zeros_like(a.out), torch.zeros_like(a.lse), torch.zeros_like(a.row_flags))
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        mtp.mtp_prefix_attention(**g, out=out)
        wrong += (out.out != a.out).sum() + (out.lse != a.lse).sum() + out.row_flags.count_nonzero()
    assert wrong.item() == 0


@pytest.mark.parametrize("D, T, Hq", [(128, 2, 4), (128, 3, 20), (256, 2, 8), (64, 2, 8), (128, 20, 8)])
def test_prefix_attention_values_out_of_sight(D, T, Hq):
    """Infinite and NaN values of a node reach the rows that see it and no others."""
    x = prefix_case(27, "bf16", [1, 1], [150, 30], T, Hq, 2, D, 16, [30, 150])
    x["parents"] = torch.tensor([[-1] + [max(0, i - 2) for i in range(1, T)]] * 2, dtype=i32)
    x["v_new"][0, 1, 0, 5], x["v_new"][0, 1, 1, D - 1], x["v_new"][1, 0, 1, 9] = math.inf, -math.inf, math.nan
    r = mtp.mtp_prefix_attention(**on_gpu(x)).out.cpu()
    y = dict(x, v_new=torch.where(x["v_new"].isfinite(), x["v_new"], torch.zeros_like(x["v_new"])))
    want = mtp.mtp_prefix_attention(**on_gpu(y)).out.cpu()
    assert want.isfinite().all()
    for b, node, h, d, value in ((0, 1, 0, 5, math.inf), (0, 1, 1, D - 1, -math.inf), (1, 0, 1, 9, math.nan)):
        for i in range(T):
            j = i
            while j > node:
                j = int(x["parents"][b, j])
            if j == node:
                want[b, i, h * (Hq // 2):(h + 1) * (Hq // 2), d] = value
    assert torch.equal(r.isnan(), want.isnan())
    assert torch.equal(torch.nan_to_num(r, nan=0.0), torch.nan_to_num(want, nan=0.0))


@pytest.mark.parametrize("dtype, D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64)])
def test_prefix_attention_extreme_scores(dtype, D):
    """The largest scores in the prefix for some rows, in the sequence's own
    tokens for others, far apart: weights of either side underflow."""
    x = prefix_case(26, dtype, [4], [300], 2, 4, 2, D, 16, [100, 100, 0, 33])
    pos = torch.arange(300)
    x["k_cache"][x["prefix_table"][0].long()[pos // 16], pos % 16] += (pos / 20.0)[:, None, None].to(x["q"].dtype) * x["q"][0, 0, ::2][None]
    at = torch.arange(100)
    x["k_cache"][x["page_table"][1].long()[at // 16], at % 16] += (at / 4.0)[:, None, None].to(x["q"].dtype) * x["q"][1, 1, ::2][None]
    run(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_attention_graphs_and_streams(dtype):
    """Two captured graphs whose lengths and groups change between replays, side by
    side on two streams, and calls on a given stream."""
    xs = [prefix_case(30 + k, dtype, [3, 4], [900, 300 + k], 3, 8, 2, 128, 16, [0, 20, 64, 100, 7, 9, 33], room=3) for k in range(2)]
    for x in xs:
        x["k_cache"].nan_to_num_(nan=0.5)
        x["v_cache"].nan_to_num_(posinf=0.5)
    gs = [on_gpu(x) for x in xs]
    for g in gs:
        mtp.mtp_prefix_attention(**g)  # loads the library's kernels
    torch.cuda.synchronize()
    outs, graphs = [], []
    for g in gs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(mtp.mtp_prefix_attention(**g, with_lse=True))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        for x, g in zip(xs, gs):
            for name, v in (("prefix_len", [900 - 400 * turn, 10 * turn]), ("group_start", [0, 3 + 2 * turn, 7]),
                            ("cache_len", [turn, 20, 64 - turn, 100, 7, 9, 33 * turn])):
                x[name] = torch.tensor(v, dtype=i32)
                g[name].copy_(x[name])
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for x, g, o in zip(xs, gs, outs):
            r = mtp.mtp_prefix_attention(**g, with_lse=True, stream=streams[0])
            torch.cuda.synchronize()
            assert torch.equal(r.out, o.out) and torch.equal(r.lse, o.lse) and not o.row_flags.any()
            check(x, o.out, o.lse)


def test_prefix_attention_no_sequences():
    x = on_gpu(prefix_case(31, "bf16", [1], [5], 2, 4, 2, 64, 16, [5]))
    for k in PER_SEQUENCE:
        x[k] = None if x[k] is None else x[k][:0]
    x["group_start"].zero_()
    assert mtp.mtp_prefix_attention(**x).out.shape == (0, 2, 4, 64)


@pytest.mark.parametrize("sizes, T, Hq, D", [([40], 2, 8, 128), ([8, 8], 2, 8, 128), ([1, 2], 2, 4, 64), ([6, 3], 3, 8, 256), ([1, 1], 2, 4, 128),
                                                 ([1, 1], 2, 8, 256)])
def test_prefix_attention_a_wait_that_runs_out_is_reported(sizes, T, Hq, D):
    """In every mode: a CTA of either kernel whose loader leaves out a signal gives
    up after its time.  Each row is NaN or right, exactly the sequences with NaN
    rows are flagged, and the next call is right."""
    B = sum(sizes)
    x = prefix_case(32, "bf16", sizes, [1500] * len(sizes), T, Hq, 2, D, 32, [100] * B, "chain")
    good = run(x)
    g = on_gpu(x)
    for cta in (0, 1, 7, 40):
        with mtp.tuning(fault_wait_us=2000, fault_skip_position=1 + cta):
            r = mtp.mtp_prefix_attention(**g, with_lse=True)
            torch.cuda.synchronize()
        lost = r.out.isnan().flatten(1).any(1)
        assert r.row_flags.tolist() == [mtp.ROW_TIMEOUT if n else 0 for n in lost.tolist()]
        assert r.out[lost].isnan().all() and torch.equal(r.out[~lost], good.out[~lost])
        if cta == 0:
            assert lost.any()
        assert torch.equal(mtp.mtp_prefix_attention(**g).out, good.out)


def few_keys(x):
    """out, its bound and what weights rounded once to bfloat16 would give, in 64
    bits, of sequences whose every node sees its whole text (T = 1).

    A weight is off by 2^-16 (two roundings of 2^-8) and by its score's error,
    which a product of D terms in float32 keeps below D 2^-23 of the terms' sum; the
    weights' sum likewise.  The output is rounded once, by 2^-8 of itself."""
    q, k, v, kc, vc, table, lens, _, _ = one_text(x)
    B, _, Hq, D = q.shape
    G = Hq // k.shape[2]
    ref, tol, once = (torch.zeros(B, 1, Hq, D, dtype=torch.float64) for _ in range(3))
    for b in range(B):
        rows = table[b, :int(lens[b])].long()
        keys, values = (torch.cat([c[rows, 0], n[b]]).double().repeat_interleave(G, 1) for c, n in ((kc, k), (vc, v)))
        terms = q[b, 0].double()[None] * keys * D ** -0.5
        s = terms.sum(-1)
        e = D * 2.0 ** -23 * terms.abs().sum(-1).max()
        p = (s - s[0]).exp()
        w = p / p.sum(0)
        ref[b, 0] = (w[..., None] * values).sum(0)
        tol[b, 0] = 2.0 ** -8 * ref[b, 0].abs() + (2.0 ** -16 + 2 * e + 2.0 ** -20) * (w[..., None] * values.abs()).sum(0) + 2.0 ** -130
        once[b, 0] = (p.to(bf16).double()[..., None] * values).sum(0) / p.sum(0)[:, None]
    return ref, tol, once


@pytest.mark.parametrize("D, Hq", [(128, 4), (128, 20), (256, 8)])
def test_prefix_attention_weights_of_two_parts(D, Hq):
    x = prefix_case(5, "bf16", [1, 1], [5, 9], 1, Hq, 1, D, 16, [3, 0], "chain")
    ref, tol, once = few_keys(x)
    assert bool(((once - ref).abs() > tol).any())  # the bound tells one rounding of the weights
    out = run(x).out.double().cpu()
    assert bool(((out - ref).abs() <= tol).all()), float(((out - ref).abs() / tol).max())
