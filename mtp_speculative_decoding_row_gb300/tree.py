"""Binding of the tree-draft operators (see "Tree-shaped drafts" in
``include/mtp_rs.h``): attention of a drafted tree over a paged cache, beam
selection, beam reordering and the commit of an accepted path.

Argument marshalling only, like the package's other entry points.  These calls
sit between the small launches of a decoding loop, so the checks are kept
short: each tensor is looked at once, and the two calls with many arguments
pass them as one packed struct.
"""
from __future__ import annotations

import functools
import struct
from typing import NamedTuple, Optional

import mtp_speculative_decoding_row_gb300 as _m

MAX_NODES, MAX_BEAMS, MAX_SELECT = 64, 64, 64

_ATTN = struct.Struct("@13Pq15q9if")
_COMMIT = struct.Struct("@15P16q9i4x")  # (as the C structs lie in memory)


class TreeAttentionResult(NamedTuple):
    out: "object"        # [B, T, Hq, D], the inputs' dtype
    lse: "object"        # [B, T, Hq] float32 or None: ln of the softmax's sum
    row_flags: "object"  # [B] int32


class BeamResult(NamedTuple):
    tokens: "object"     # [B, K] int32, best first (-1: none)
    parents: "object"    # [B, K] int32: the beam each continues (-1: none)
    scores: "object"     # [B, K] float32
    row_flags: "object"  # [B] int32


class ReorderResult(NamedTuple):
    states: "object"     # [N0, B, K, ...]
    row_flags: "object"  # [B] int32


class CommitResult(NamedTuple):
    tokens: "object"      # [B, T] int32: accepted drafts, then the target's token, -1 padded
    accept_len: "object"  # [B] int32: accepted drafts (-1 if flagged or without nodes)
    path: "object"        # [B, T] int32: accepted nodes, the root first, -1 padded
    cache_len: "object"   # [B] int32: cached tokens after the call
    row_flags: "object"   # [B] int32


def _shape(t, name, dtype, shape, index):
    """The pointer of a contiguous tensor of this dtype and shape on device `index`."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the device of the other tensors")
    return t.data_ptr()


def _strided(t, name, dtype, shape, index):
    """As _shape, but only the last dimension has to be contiguous: (pointer, strides of the others)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    s = t.stride()
    if s[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the device of the other tensors")
    return t.data_ptr(), s[:-1]


def _dims(t, name, n):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {tuple(t.shape)}")
    return t.shape


class _on:
    """The device of a call made current, where it is not."""

    __slots__ = ("guard",)

    def __init__(self, torch, index, name):
        if index < 0:
            raise ValueError(f"{name} must be a CUDA tensor")
        self.guard = None if torch.cuda.current_device() == index else torch.cuda.device(index)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _launch_stream(torch, dev, stream, *mine):
    """The raw stream of a call; tensors allocated for it here are tied to a
    stream that is not the current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev.index)
    for t in mine:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


@functools.lru_cache(maxsize=1024)
def _attn_workspace(index, *sizes):
    n = _m.load_library().mtp_tree_attention_workspace(_ATTN.pack(*([0] * 14), *([0] * 15), *sizes, 1.0))
    if n < 0:
        raise _m.MTPError("mtp_tree_attention_workspace", _m.MTP_ERR_INVALID_ARG)
    return n


def mtp_tree_attention(q, k_new, v_new, k_cache, v_cache, page_table, cache_len, parents=None, n_nodes=None, *,
                       scale: Optional[float] = None, with_lse: bool = False, out: Optional[TreeAttentionResult] = None,
                       stream=None) -> TreeAttentionResult:
    """Attention of the T nodes of a drafted tree over the cached tokens and
    the nodes on their own path (see mtp_tree_attention in include/mtp_rs.h).

    q [B, T, Hq, D], k_new and v_new [B, T, Hkv, D], k_cache and v_cache
    [num_pages, page_size, Hkv, D] (float32 or bfloat16; any strides but a
    contiguous last dimension), page_table [B, max_pages], cache_len [B],
    parents [B, T] (None: a chain), n_nodes [B] (None: T), int32.  `scale`
    defaults to D ** -0.5.  Returns out [B, T, Hq, D], lse [B, T, Hq] (with
    with_lse, or where `out` has it) and row_flags [B]; rows of nodes >=
    n_nodes are left as they were (undefined in outputs allocated here)."""
    torch = _m._torch()
    B, T, Hq, D = _dims(q, "q", 4)
    Hkv = _dims(k_new, "k_new", 4)[2]
    pages, page_size = _dims(k_cache, "k_cache", 4)[:2]
    max_pages = _dims(page_table, "page_table", 2)[1]
    dt, dev = q.dtype, q.device
    code = _m._dtype_code(q)
    i32 = torch.int32
    if Hkv < 1 or Hq % Hkv != 0 or Hq < 1:
        raise ValueError(f"q has {Hq} heads: not a multiple of the {Hkv} of k_new")
    if not 1 <= T <= MAX_NODES:
        raise ValueError(f"trees have 1 to {MAX_NODES} nodes, got {T}")
    if not 1 <= D <= 256:
        raise ValueError(f"heads have 1 to 256 elements, got {D}")
    if scale is None:
        scale = D ** -0.5
    elif not 0.0 < scale < 1e30:
        raise ValueError(f"scale must be positive, got {scale}")
    index = q.get_device()
    if out is not None:
        pl = _shape(out.lse, "out.lse", torch.float32, (B, T, Hq), index) if out.lse is not None else 0
        pf = _shape(out.row_flags, "out.row_flags", i32, (B,), index) if out.row_flags is not None else 0
        po = _shape(out.out, "out.out", dt, (B, T, Hq, D), index)
        if with_lse and not pl:
            raise ValueError("mtp_tree_attention: with_lse needs out.lse")
    pq, sq = _strided(q, "q", dt, (B, T, Hq, D), index)
    pk, sk = _strided(k_new, "k_new", dt, (B, T, Hkv, D), index)
    pv, sv = _strided(v_new, "v_new", dt, (B, T, Hkv, D), index)
    pkc, skc = _strided(k_cache, "k_cache", dt, (pages, page_size, Hkv, D), index)
    pvc, svc = _strided(v_cache, "v_cache", dt, (pages, page_size, Hkv, D), index)
    pt = _shape(page_table, "page_table", i32, (B, max_pages), index)
    pc = _shape(cache_len, "cache_len", i32, (B,), index)
    pp = _shape(parents, "parents", i32, (B, T), index) if parents is not None else 0
    pn = _shape(n_nodes, "n_nodes", i32, (B,), index) if n_nodes is not None else 0
    with _on(torch, index, "q"):
        mine = ()
        if out is None:
            out = TreeAttentionResult(torch.empty((B, T, Hq, D), dtype=dt, device=dev),
                                      torch.empty((B, T, Hq), dtype=torch.float32, device=dev) if with_lse else None,
                                      torch.empty((B,), dtype=i32, device=dev))
            mine = out
            po, pf = out.out.data_ptr(), out.row_flags.data_ptr()
            pl = out.lse.data_ptr() if with_lse else 0
        sizes = (code, B, T, Hq, Hkv, D, pages, page_size, max_pages)
        nbytes = _attn_workspace(index, *sizes)
        ws = torch.empty((nbytes,), dtype=torch.uint8, device=dev)
        raw = _launch_stream(torch, dev, stream, ws, *mine)
        rc = _m.load_library().mtp_tree_attention(
            _ATTN.pack(pq, pk, pv, pkc, pvc, pt, pc, pp, pn, po, pl, pf, ws.data_ptr(), nbytes, *sq, *sk, *sv, *skc, *svc, *sizes,
                       scale), raw)
    if rc:
        raise _m.MTPError("mtp_tree_attention", rc)
    return out


@functools.lru_cache(maxsize=1024)
def _beam_workspace(index, code, B, W, V, K):
    n = _m.load_library().mtp_beam_select_workspace(code, B, W, V, K)
    if n < 0:
        raise _m.MTPError("mtp_beam_select_workspace", _m.MTP_ERR_INVALID_ARG)
    return n


def mtp_beam_select(logits, scores, temperature, K: int, *, out: Optional[BeamResult] = None, stream=None) -> BeamResult:
    """The K best continuations of each sequence's W beams (see
    mtp_beam_select in include/mtp_rs.h): logits [B, W, V] (float32 or
    bfloat16), scores [B, W] float32 (-inf: a dead beam), temperature [B]
    float32.  Returns tokens, parents and scores [B, K], best first."""
    torch = _m._torch()
    B, W, V = _dims(logits, "logits", 3)
    code = _m._dtype_code(logits)
    dev, i32, f32 = logits.device, torch.int32, torch.float32
    if not 1 <= W <= MAX_BEAMS:
        raise ValueError(f"1 to {MAX_BEAMS} beams, got {W}")
    if not 1 <= K <= MAX_SELECT or K > W * V:
        raise ValueError(f"K must be 1 to {MAX_SELECT} and at most W V, got {K}")
    index = logits.get_device()
    if out is not None:
        po = (_shape(out.tokens, "out.tokens", i32, (B, K), index), _shape(out.parents, "out.parents", i32, (B, K), index),
              _shape(out.scores, "out.scores", f32, (B, K), index),
              _shape(out.row_flags, "out.row_flags", i32, (B,), index) if out.row_flags is not None else 0)
    pz = _shape(logits, "logits", logits.dtype, (B, W, V), index)
    ps = _shape(scores, "scores", f32, (B, W), index)
    pt = _shape(temperature, "temperature", f32, (B,), index)
    with _on(torch, index, "logits"):
        mine = ()
        if out is None:
            out = BeamResult(torch.empty((B, K), dtype=i32, device=dev), torch.empty((B, K), dtype=i32, device=dev),
                             torch.empty((B, K), dtype=f32, device=dev), torch.empty((B,), dtype=i32, device=dev))
            mine = out
            po = tuple(t.data_ptr() for t in out)
        nbytes = _beam_workspace(index, code, B, W, V, K)
        ws = torch.empty((nbytes,), dtype=torch.uint8, device=dev)
        raw = _launch_stream(torch, dev, stream, ws, *mine)
        rc = _m.load_library().mtp_beam_select(pz, code, ps, pt, B, W, V, K, *po, ws.data_ptr(), nbytes, raw)
    if rc:
        raise _m.MTPError("mtp_beam_select", rc)
    return out


def mtp_beam_reorder(states, parents, *, out: Optional[ReorderResult] = None, stream=None) -> ReorderResult:
    """States of the selected beams (see mtp_beam_reorder in
    include/mtp_rs.h): states [N0, B, W, ...] of any dtype, parents [B, K]
    int32; returns states [N0, B, K, ...] with out[n, b, k] = states[n, b,
    parents[b, k]], zeros for a parent outside [0, W)."""
    torch = _m._torch()
    if states.dim() < 3:
        raise ValueError(f"states must be [N0, B, W, ...], got {tuple(states.shape)}")
    N0, B, W = states.shape[:3]
    K = _dims(parents, "parents", 2)[1]
    dev, dt, i32 = states.device, states.dtype, torch.int32
    if W < 1 or K < 1:
        raise ValueError(f"at least one beam and one place are needed, got W = {W}, K = {K}")
    index = states.get_device()
    shape = (N0, B, K, *states.shape[3:])
    if out is not None:
        pd = _shape(out.states, "out.states", dt, shape, index)
        pf = _shape(out.row_flags, "out.row_flags", i32, (B,), index) if out.row_flags is not None else 0
    ps = _shape(states, "states", dt, states.shape, index)
    pp = _shape(parents, "parents", i32, (B, K), index)
    row = states.element_size()
    for n in shape[3:]:
        row *= n
    with _on(torch, index, "states"):
        mine = ()
        if out is None:
            out = ReorderResult(torch.empty(shape, dtype=dt, device=dev), torch.zeros((B,), dtype=i32, device=dev))
            mine = out
            pd, pf = out.states.data_ptr(), out.row_flags.data_ptr()
        raw = _launch_stream(torch, dev, stream, *mine)
        rc = _m.load_library().mtp_beam_reorder(ps, pp, N0, B, W, K, row, pd, pf, raw)
    if rc:
        raise _m.MTPError("mtp_beam_reorder", rc)
    return out


def mtp_tree_commit(tokens, target_tokens, parents=None, k_new=None, v_new=None, k_cache=None, v_cache=None, page_table=None,
                    cache_len=None, n_nodes=None, *, out: Optional[CommitResult] = None, stream=None) -> CommitResult:
    """Walk a drafted tree along the target's tokens and write the keys and
    values of the accepted path behind the cached tokens (see mtp_tree_commit
    in include/mtp_rs.h).

    tokens, target_tokens, parents [B, T] int32 (parents None: a chain; node 0
    is the root), k_new and v_new [layers, B, T, Hkv, D], k_cache and v_cache
    [layers, num_pages, page_size, Hkv, D] (without the layers' dimension for
    one layer; written in place), page_table [B, max_pages], cache_len [B],
    n_nodes [B] (None: T)."""
    torch = _m._torch()
    i32 = torch.int32
    B, T = _dims(tokens, "tokens", 2)
    if not 1 <= T <= MAX_NODES:
        raise ValueError(f"trees have 1 to {MAX_NODES} nodes, got {T}")
    for t, name in ((k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"), (v_cache, "v_cache"), (page_table, "page_table"),
                    (cache_len, "cache_len")):
        if t is None:
            raise ValueError(f"{name} is required")
    dt = k_new.dtype
    code = _m._dtype_code(k_new)
    if k_new.dim() == 4:
        k_new, v_new, k_cache, v_cache = k_new[None], v_new[None], k_cache[None], v_cache[None]
    layers, _, _, Hkv, D = _dims(k_new, "k_new", 5)
    pages, page_size = _dims(k_cache, "k_cache", 5)[1:3]
    max_pages = _dims(page_table, "page_table", 2)[1]
    index, dev = tokens.get_device(), tokens.device
    if out is not None:
        po = (_shape(out.tokens, "out.tokens", i32, (B, T), index), _shape(out.accept_len, "out.accept_len", i32, (B,), index),
              _shape(out.path, "out.path", i32, (B, T), index), _shape(out.cache_len, "out.cache_len", i32, (B,), index),
              _shape(out.row_flags, "out.row_flags", i32, (B,), index) if out.row_flags is not None else 0)
    pt = _shape(tokens, "tokens", i32, (B, T), index)
    pg = _shape(target_tokens, "target_tokens", i32, (B, T), index)
    pp = _shape(parents, "parents", i32, (B, T), index) if parents is not None else 0
    pn = _shape(n_nodes, "n_nodes", i32, (B,), index) if n_nodes is not None else 0
    pk, sk = _strided(k_new, "k_new", dt, (layers, B, T, Hkv, D), index)
    pv, sv = _strided(v_new, "v_new", dt, (layers, B, T, Hkv, D), index)
    pkc, skc = _strided(k_cache, "k_cache", dt, (layers, pages, page_size, Hkv, D), index)
    pvc, svc = _strided(v_cache, "v_cache", dt, (layers, pages, page_size, Hkv, D), index)
    pta = _shape(page_table, "page_table", i32, (B, max_pages), index)
    pc = _shape(cache_len, "cache_len", i32, (B,), index)
    if out is not None and po[3] == pc and B:
        raise ValueError("out.cache_len must not be cache_len itself")
    with _on(torch, index, "tokens"):
        mine = ()
        if out is None:
            e = lambda *s: torch.empty(s, dtype=i32, device=dev)  # noqa: E731
            out = mine = CommitResult(e(B, T), e(B), e(B, T), e(B), e(B))
            po = tuple(t.data_ptr() for t in out)
        raw = _launch_stream(torch, dev, stream, *mine)
        rc = _m.load_library().mtp_tree_commit(
            _COMMIT.pack(pt, pg, pp, pn, pta, pc, pk, pv, pkc, pvc, po[0], po[1], po[2], po[3], po[4], *sk, *sv, *skc, *svc, code,
                         layers, B, T, Hkv, D, pages, page_size, max_pages), raw)
    if rc:
        raise _m.MTPError("mtp_tree_commit", rc)
    return out
