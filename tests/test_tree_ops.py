"""Refusals of the tree-draft operators, without a GPU: the binding's checks
of its arguments and the C ABI's answers."""
import ctypes
import os
import subprocess

import pytest
import torch

import mtp_speculative_decoding_row_gb300 as mtp
from mtp_speculative_decoding_row_gb300 import build as mtp_build
from mtp_speculative_decoding_row_gb300 import tree

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
i32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    mtp_build.build()


@pytest.fixture(autouse=True)
def no_launch(monkeypatch, request):
    if "lib" in request.fixturenames:
        return

    def no_library(*a, **k):
        raise AssertionError("the library must not be called")

    monkeypatch.setattr(mtp, "load_library", no_library)


@pytest.fixture
def lib():
    mtp_build.build()
    return mtp.load_library()


def attn_args(**new):
    B, T, Hq, Hkv, D = 2, 3, 4, 2, 64
    a = dict(q=torch.zeros(B, T, Hq, D), k_new=torch.zeros(B, T, Hkv, D), v_new=torch.zeros(B, T, Hkv, D),
             k_cache=torch.zeros(5, 16, Hkv, D), v_cache=torch.zeros(5, 16, Hkv, D), page_table=torch.zeros(B, 2, dtype=i32),
             cache_len=torch.zeros(B, dtype=i32))
    a.update(new)
    return a


@pytest.mark.parametrize("new, error, text", [
    (dict(q=torch.zeros(2, 3, 4, 64, dtype=torch.float16)), TypeError, "float32 or bfloat16"),
    (dict(k_new=torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)), TypeError, "k_new"),
    (dict(k_new=torch.zeros(2, 3, 3, 64)), ValueError, "heads"),
    (dict(v_new=torch.zeros(2, 3, 1, 64)), ValueError, "v_new"),
    (dict(v_cache=torch.zeros(5, 8, 2, 64)), ValueError, "v_cache"),
    (dict(k_cache=torch.zeros(5, 16, 64, 2).transpose(2, 3)), ValueError, "k_cache"),
    (dict(page_table=torch.zeros(3, 2, dtype=i32)), ValueError, "page_table"),
    (dict(page_table=torch.zeros(2, 2, dtype=torch.int64)), TypeError, "page_table"),
    (dict(cache_len=torch.zeros(3, dtype=i32)), ValueError, "cache_len"),
    (dict(parents=torch.zeros(2, 4, dtype=i32)), ValueError, "parents"),
    (dict(n_nodes=torch.zeros(2, 1, dtype=i32)), ValueError, "n_nodes"),
    (dict(scale=0.0), ValueError, "scale"),
    (dict(scale=float("nan")), ValueError, "scale"),
    (dict(q=torch.zeros(2, 65, 4, 64)), ValueError, "nodes"),
    (dict(q=torch.zeros(2, 3, 4, 257)), ValueError, "elements"),
    (dict(q=torch.zeros(6, 4, 64)), ValueError, "dimensions"),
    (dict(out=mtp.TreeAttentionResult(torch.zeros(2, 3, 4, 32), None, None)), ValueError, "out.out"),
    (dict(out=mtp.TreeAttentionResult(torch.zeros(2, 3, 4, 64), torch.zeros(2, 4, 3), None)), ValueError, "out.lse"),
    ({}, ValueError, "CUDA"),
])
def test_tree_attention_refusals(new, error, text):
    with pytest.raises(error, match=text):
        mtp.mtp_tree_attention(**attn_args(**new))


def test_tree_attention_most_heads_of_one_key_head():
    a = attn_args(q=torch.zeros(2, 3, 4097, 8), k_new=torch.zeros(2, 3, 1, 8), v_new=torch.zeros(2, 3, 1, 8),
                  k_cache=torch.zeros(5, 16, 1, 8), v_cache=torch.zeros(5, 16, 1, 8))
    with pytest.raises(ValueError, match="up to 4096"):
        mtp.mtp_tree_attention(**a)


@pytest.mark.parametrize("new, error, text", [
    (dict(logits=torch.zeros(2, 3, 10, dtype=torch.float64)), TypeError, "float32 or bfloat16"),
    (dict(logits=torch.zeros(2, 30)), ValueError, "dimensions"),
    (dict(scores=torch.zeros(2, 4)), ValueError, "scores"),
    (dict(scores=torch.zeros(2, 3, dtype=torch.bfloat16)), TypeError, "scores"),
    (dict(temperature=torch.ones(3)), ValueError, "temperature"),
    (dict(K=0), ValueError, "K must"),
    (dict(K=31), ValueError, "K must"),
    (dict(logits=torch.zeros(1, 65, 10)), ValueError, "beams"),
    (dict(logits=torch.zeros(2, 10, 3).transpose(1, 2)), ValueError, "CUDA|contiguous"),
    ({}, ValueError, "CUDA"),
])
def test_beam_select_refusals(new, error, text):
    a = dict(logits=torch.zeros(2, 3, 10), scores=torch.zeros(2, 3), temperature=torch.ones(2), K=4)
    a.update(new)
    with pytest.raises(error, match=text):
        mtp.mtp_beam_select(**a)


def test_beam_select_more_than_the_most():
    with pytest.raises(ValueError, match="K must"):
        mtp.mtp_beam_select(torch.zeros(1, 2, 100), torch.zeros(1, 2), torch.ones(1), 65)


@pytest.mark.parametrize("states, parents, text", [
    (torch.zeros(2, 3), torch.zeros(3, 1, dtype=i32), "states"),
    (torch.zeros(1, 2, 3, 4), torch.zeros(3, 1, dtype=i32), "parents"),
    (torch.zeros(1, 2, 3, 4), torch.zeros(2, 0, dtype=i32), "at least one"),
    (torch.zeros(1, 2, 4, 3).transpose(2, 3), torch.zeros(2, 1, dtype=i32), "contiguous"),
    (torch.zeros(1, 2, 3, 4), torch.zeros(2, 1, dtype=i32), "CUDA"),
])
def test_beam_reorder_refusals(states, parents, text):
    with pytest.raises(ValueError, match=text):
        mtp.mtp_beam_reorder(states, parents)


def commit_args(**new):
    B, T = 2, 4
    a = dict(tokens=torch.zeros(B, T, dtype=i32), target_tokens=torch.zeros(B, T, dtype=i32), k_new=torch.zeros(1, B, T, 2, 8),
             v_new=torch.zeros(1, B, T, 2, 8), k_cache=torch.zeros(1, 5, 16, 2, 8), v_cache=torch.zeros(1, 5, 16, 2, 8),
             page_table=torch.zeros(B, 2, dtype=i32), cache_len=torch.zeros(B, dtype=i32))
    a.update(new)
    return a


@pytest.mark.parametrize("new, error, text", [
    (dict(tokens=torch.zeros(2, 4)), TypeError, "tokens"),
    (dict(tokens=torch.zeros(2, 65, dtype=i32)), ValueError, "nodes"),
    (dict(target_tokens=torch.zeros(2, 3, dtype=i32)), ValueError, "target_tokens"),
    (dict(parents=torch.zeros(2, 5, dtype=i32)), ValueError, "parents"),
    (dict(k_new=None), ValueError, "k_new"),
    (dict(v_new=torch.zeros(1, 2, 4, 2, 9)), ValueError, "v_new"),
    (dict(k_cache=torch.zeros(2, 5, 16, 2, 8)), ValueError, "k_cache"),
    (dict(v_cache=torch.zeros(1, 5, 16, 8, 2).transpose(3, 4)), ValueError, "v_cache"),
    (dict(cache_len=torch.zeros(2, dtype=torch.int64)), TypeError, "cache_len"),
    ({}, ValueError, "CUDA"),
])
def test_tree_commit_refusals(new, error, text):
    with pytest.raises(error, match=text):
        mtp.mtp_tree_commit(**commit_args(**new))


def test_structs_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include "mtp_rs.h"\n#include <stddef.h>\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu %zu %d %d %d", '
                   'sizeof(mtp_tree_attention_args), sizeof(mtp_tree_commit_args), offsetof(mtp_tree_attention_args, scale), '
                   'offsetof(mtp_tree_commit_args, max_pages), MTP_MAX_NODES, MTP_MAX_BEAMS, MTP_MAX_SELECT); return 0; }')
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")])
    got = [int(x) for x in subprocess.check_output([str(tmp_path / "s")]).split()]
    assert got[0] == tree._ATTN.size and got[1] == tree._COMMIT.size
    assert got[2] == tree._ATTN.size - 4 and got[3] == tree._COMMIT.size - 8
    assert got[4:] == [tree.MAX_NODES, tree.MAX_BEAMS, tree.MAX_SELECT]


def attn_struct(ptr=1 << 20, ws=1 << 30, dtype=1, B=2, T=3, Hq=4, Hkv=2, D=64, pages=5, ps=16, mp=2, scale=1.0, q=None, out=None):
    p = [ptr] * 13
    p[0] = ptr if q is None else q
    p[9] = ptr if out is None else out
    return tree._ATTN.pack(*p, ws, *([64] * 15), dtype, B, T, Hq, Hkv, D, pages, ps, mp, scale)


def test_host_validation_of_tree_attention(lib):
    f = lib.mtp_tree_attention
    assert f(None, None) == 1
    assert f(attn_struct(dtype=2), None) == 2
    for bad in (dict(B=-1), dict(T=0), dict(T=65), dict(Hq=5), dict(Hkv=0), dict(D=0), dict(D=257), dict(pages=0), dict(ps=0),
                dict(mp=0), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(ps=1 << 16, mp=1 << 16),
                dict(q=0), dict(out=0)):
        assert f(attn_struct(**bad), None) == 1, bad
        if not ("q" in bad or "out" in bad):
            assert lib.mtp_tree_attention_workspace(attn_struct(**bad)) == -1
    assert f(attn_struct(q=(1 << 20) + 1), None) == 3
    assert f(attn_struct(B=0, ptr=0), None) == 0


def test_host_validation_of_beam_select(lib):
    P = ctypes.c_void_p
    ok, odd = 1 << 20, (1 << 20) + 8

    def call(z=ok, dtype=1, s=ok, B=2, W=4, V=100, K=8, out=ok, ws=ok):
        return lib.mtp_beam_select(P(z), dtype, P(s), P(ok), B, W, V, K, P(out), P(ok), P(ok), None, P(ws), 1 << 40, None)

    assert call(dtype=5) == 2
    for bad in (dict(B=-1), dict(W=0), dict(W=65), dict(V=0), dict(V=(1 << 24) + 1), dict(K=0), dict(K=65), dict(W=1, V=7, K=8),
                dict(z=0), dict(s=0), dict(out=0), dict(ws=0)):
        assert call(**bad) == 1, bad
    assert call(z=odd) == 3 and call(ws=odd) == 3
    assert call(B=0, z=0) == 0
    assert lib.mtp_beam_select_workspace(1, 2, 0, 100, 8) == -1


def test_host_validation_of_beam_reorder(lib):
    P = ctypes.c_void_p

    def call(src=1 << 20, up=1 << 10, N0=1, B=2, W=4, K=4, row=64, dst=1 << 24):
        return lib.mtp_beam_reorder(P(src), P(up), N0, B, W, K, row, P(dst), None, None)

    for bad in (dict(N0=-1), dict(B=-1), dict(W=0), dict(K=0), dict(row=-1), dict(src=0), dict(up=0), dict(dst=0),
                dict(dst=(1 << 20) + 511), dict(dst=(1 << 20) - 511), dict(N0=1 << 20, B=1 << 20)):
        assert call(**bad) == 1, bad
    assert call(B=0, src=0) == 0 and call(N0=0, src=0) == 0 and call(row=0, src=0) == 0


def test_host_validation_of_tree_commit(lib):
    def call(ptr=1 << 20, dtype=1, layers=1, B=2, T=3, Hkv=2, D=64, pages=5, ps=16, mp=2, tokens=None, k_new=None):
        p = [ptr] * 15
        p[0] = ptr if tokens is None else tokens
        p[6] = ptr if k_new is None else k_new
        return lib.mtp_tree_commit(tree._COMMIT.pack(*p, *([64] * 16), dtype, layers, B, T, Hkv, D, pages, ps, mp), None)

    assert lib.mtp_tree_commit(None, None) == 1
    assert call(dtype=9) == 2
    for bad in (dict(layers=-1), dict(layers=40000), dict(B=-1), dict(T=0), dict(T=65), dict(Hkv=0), dict(D=0), dict(pages=0),
                dict(ps=0), dict(mp=0), dict(tokens=0), dict(k_new=0), dict(ps=1 << 16, mp=1 << 16)):
        assert call(**bad) == 1, bad
    assert call(k_new=(1 << 20) + 1) == 3
    assert call(B=0, ptr=0) == 0


def test_tree_commit_most_elements(lib):
    """A path's words are counted in 32 bits."""
    p = [1 << 20] * 15

    def call(T, Hkv, D, B):
        return lib.mtp_tree_commit(tree._COMMIT.pack(*p, *([64] * 16), 1, 1, B, T, Hkv, D, 5, 16, 2), None)

    assert call(64, 65536, 512, 2) == 1
    assert call(64, 65536, 4096, 2) == 1
    assert call(64, 65536, 256, 0) == 0
