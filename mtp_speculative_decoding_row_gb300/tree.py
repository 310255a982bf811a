"""Binding of the tree-draft operators (see "Tree-shaped drafts" in
``include/mtp_rs.h``): attention of a drafted tree over a paged cache, beam
selection, beam reordering and the commit of an accepted path.

Argument marshalling only, like the package's other entry points.  These calls
sit between the small launches of a decoding loop, so the checks of their
tensors and the call of the library are native (``csrc/binding.cpp``); here
missing outputs are allocated and the stream is chosen.
"""
from __future__ import annotations

import os
import struct
from typing import NamedTuple, Optional

import mtp_speculative_decoding_row_gb300 as _m

MAX_NODES, MAX_BEAMS, MAX_SELECT = 64, 64, 64

# the C structs as they lie in memory (for callers of the C ABI through ctypes)
_ATTN = struct.Struct("@13Pq15q9if")
_COMMIT = struct.Struct("@15P16q9i4x")

_NOT_BOUND = -1
_native = None


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


def _binding():
    """The native marshalling module; raises if it was not built."""
    global _native
    if _native is None:
        _m._torch()  # (its libraries come first)
        if not os.path.exists(_m._build.BINDING):
            raise ImportError(f"{_m._build.BINDING} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
        from . import _binding as native

        _native = native
    return _native


def _bind(lib) -> None:
    """Tell the marshalling module where the functions of `lib` are."""
    import ctypes

    names = ("mtp_tree_attention", "mtp_tree_attention_workspace", "mtp_beam_select", "mtp_beam_select_workspace",
             "mtp_beam_reorder", "mtp_tree_commit", "mtp_prefix_attention", "mtp_prefix_attention_workspace", "mtp_rope",
             "mtp_cache_append", "mtp_adjust_logits")
    _binding().bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names))


def unbind() -> None:
    """Another library was loaded: the next call looks its functions up."""
    if _native is not None:
        _native.bind(*[0] * 11)


def _call(name, args):
    rc = getattr(_binding(), name)(*args)
    if rc == _NOT_BOUND:
        _bind(_m.load_library())
        rc = getattr(_binding(), name)(*args)
    if rc:
        raise _m.MTPError("mtp_" + name, rc)


class _on:
    """The device and the stream of a call made current, where they are not.

    What is allocated inside -- outputs here, the workspace natively -- then
    belongs to the stream that it is used on: memory of the caller's current
    stream may still be written by work queued there before it was freed."""

    __slots__ = ("guard", "caller")

    def __init__(self, torch, index, stream):
        self.guard = self.caller = None
        if stream is not None and index >= 0:
            if stream.device.index != index:
                raise ValueError(f"stream must be on the device of the tensors, cuda:{index}, not {stream.device}")
            self.caller = torch.cuda.current_stream(index)
            self.guard = torch.cuda.stream(stream)
        elif index >= 0 and torch._C._cuda_getDevice() != index:
            self.guard = torch.cuda.device(index)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def raw(self, torch, index, mine):
        """The raw stream of the call.  Outputs allocated for it here will be
        read, and may be freed, on the caller's stream: they are tied to both."""
        if self.caller is not None:
            for t in mine:
                if t is not None:
                    t.record_stream(self.caller)
        return torch._C._cuda_getCurrentRawStream(index) if index >= 0 else 0


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
    index = q.get_device()
    if out is not None and with_lse and out.lse is None:
        raise ValueError("mtp_tree_attention: with_lse needs out.lse")
    with _on(torch, index, stream) as on:
        mine = ()
        if out is None:
            if q.dim() != 4:
                raise ValueError(f"q must have 4 dimensions, got {tuple(q.shape)}")
            dev = q.device
            out = mine = TreeAttentionResult(torch.empty(q.shape, dtype=q.dtype, device=dev),
                                             torch.empty(q.shape[:3], dtype=torch.float32, device=dev) if with_lse else None,
                                             torch.empty(q.shape[:1], dtype=torch.int32, device=dev))
        _call("tree_attention",
              (q, k_new, v_new, k_cache, v_cache, page_table, cache_len, parents, n_nodes,
               q.shape[-1] ** -0.5 if scale is None else scale, out.out, out.lse, out.row_flags, on.raw(torch, index, mine)))
    return out


def mtp_prefix_attention(q, k_new, v_new, k_cache, v_cache, prefix_table, prefix_len, group_start, page_table, cache_len, parents=None,
                         n_nodes=None, *, scale: Optional[float] = None, with_lse: bool = False,
                         out: Optional[TreeAttentionResult] = None, stream=None) -> TreeAttentionResult:
    """mtp_tree_attention for sequences that share prefixes, each prefix read
    once for all of its sequences (see mtp_prefix_attention in
    include/mtp_rs.h).

    prefix_table [P, max_prefix_pages] and prefix_len [P] int32 are the pages
    and tokens of the prefixes; sequences group_start[p] .. group_start[p + 1] - 1
    (group_start [P + 1] int32, from 0 to B) continue prefix p with their own
    cache_len tokens in the pages of page_table.  The rest is as in
    mtp_tree_attention; all rows of a flagged sequence are NaN."""
    torch = _m._torch()
    index = q.get_device()
    if out is not None and with_lse and out.lse is None:
        raise ValueError("mtp_prefix_attention: with_lse needs out.lse")
    with _on(torch, index, stream) as on:
        mine = ()
        if out is None:
            if q.dim() != 4:
                raise ValueError(f"q must have 4 dimensions, got {tuple(q.shape)}")
            dev = q.device
            out = mine = TreeAttentionResult(torch.empty(q.shape, dtype=q.dtype, device=dev),
                                             torch.empty(q.shape[:3], dtype=torch.float32, device=dev) if with_lse else None,
                                             torch.empty(q.shape[:1], dtype=torch.int32, device=dev))
        _call("prefix_attention",
              (q, k_new, v_new, k_cache, v_cache, prefix_table, prefix_len, group_start, page_table, cache_len, parents, n_nodes,
               q.shape[-1] ** -0.5 if scale is None else scale, out.out, out.lse, out.row_flags, on.raw(torch, index, mine)))
    return out


def mtp_beam_select(logits, scores, temperature, K: int, *, out: Optional[BeamResult] = None, stream=None) -> BeamResult:
    """The K best continuations of each sequence's W beams (see
    mtp_beam_select in include/mtp_rs.h): logits [B, W, V] (float32 or
    bfloat16, contiguous, starting on 16 bytes), scores [B, W] float32 (-inf: a
    dead beam), temperature [B] float32.  Returns tokens, parents and scores [B, K], best first."""
    torch = _m._torch()
    index = logits.get_device()
    with _on(torch, index, stream) as on:
        mine = ()
        if out is None:
            B, dev, i32 = logits.shape[0], logits.device, torch.int32
            k = max(int(K), 0)
            out = mine = BeamResult(torch.empty((B, k), dtype=i32, device=dev), torch.empty((B, k), dtype=i32, device=dev),
                                    torch.empty((B, k), dtype=torch.float32, device=dev), torch.empty((B,), dtype=i32, device=dev))
        _call("beam_select", (logits, scores, temperature, K, out.tokens, out.parents, out.scores, out.row_flags,
                              on.raw(torch, index, mine)))
    return out


def mtp_beam_reorder(states, parents, *, out: Optional[ReorderResult] = None, stream=None) -> ReorderResult:
    """States of the selected beams (see mtp_beam_reorder in
    include/mtp_rs.h): states [N0, B, W, ...] of any dtype, parents [B, K]
    int32; returns states [N0, B, K, ...] with out[n, b, k] = states[n, b,
    parents[b, k]], zeros for a parent outside [0, W)."""
    torch = _m._torch()
    index = states.get_device()
    with _on(torch, index, stream) as on:
        mine = ()
        if out is None:
            if states.dim() < 3 or parents.dim() != 2:
                raise ValueError(f"states must be [N0, B, W, ...] and parents [B, K], got {tuple(states.shape)} and "
                                 f"{tuple(parents.shape)}")
            dev = states.device
            out = mine = ReorderResult(
                torch.empty((*states.shape[:2], parents.shape[1], *states.shape[3:]), dtype=states.dtype, device=dev),
                torch.empty((states.shape[1],), dtype=torch.int32, device=dev))
        _call("beam_reorder", (states, parents, out.states, out.row_flags, on.raw(torch, index, mine)))
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
    n_nodes [B] (None: T).  Without keys, values, caches and table the tree is
    verified alone: nothing is written but the outputs, whose cache_len counts
    from `cache_len` or (None) from 0."""
    torch = _m._torch()
    index = tokens.get_device()
    with _on(torch, index, stream) as on:
        mine = ()
        if out is None:
            if tokens.dim() != 2:
                raise ValueError(f"tokens must have 2 dimensions, got {tuple(tokens.shape)}")
            e = lambda s: torch.empty(s, dtype=torch.int32, device=tokens.device)  # noqa: E731
            n = tokens.shape[:1]
            out = mine = CommitResult(e(tokens.shape), e(n), e(tokens.shape), e(n), e(n))
        _call("tree_commit",
              (tokens, target_tokens, parents, k_new, v_new, k_cache, v_cache, page_table, cache_len, n_nodes, out.tokens,
               out.accept_len, out.path, out.cache_len, out.row_flags, on.raw(torch, index, mine)))
    return out
