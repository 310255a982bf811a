// tree_attention.cuh -- what the tree-attention kernels share: how the key
// tiles of a batch are dealt out to the CTAs, the ancestor masks of a tree,
// the checks of a sequence, and the slots that partial results go to.
//
// The queries of one (sequence b, key head h) are the T nodes x G query heads
// that share the head: row r = t * G + g.  They read the same keys, so a unit
// of work is (b, h): ceil(len_b / ktile) tiles of cached keys, then one tile
// of the T new keys.  Rows beyond one tile of BM rows go to `mtiles` CTAs
// that walk the same key tiles at the same time, so the keys come from HBM
// once and from L2 for the others.
//
// Lengths live on the device and differ between sequences, so the split is
// made there: the tiles of all units in a row, (b, h) after (b, h), make a
// list of W tiles, and group g of CTAs takes tiles [W g / NG, W (g + 1) / NG)
// of it.  Every CTA then has the same number of tiles to within one, whatever
// the lengths are, and a launch fits any lengths (a captured graph too).  A
// unit that lies in several groups' ranges is joined afterwards from its
// parts' running maxima, sums and unnormalised rows, in the order of the
// groups: the result does not depend on which CTA ran first.
#pragma once

#include "common.cuh"
#include "tree.h"

namespace mtp {

// Cached tokens of sequence b; 0 for a length that the page table cannot hold
// (the sequence is flagged).
__device__ __forceinline__ int attn_len(const TreeAttnArgs &A, int b, bool &bad) {
    const int n = __ldg(A.len + b);
    bad = n < 0 || n > static_cast<long long>(A.max_pages) * A.page_size;
    return bad ? 0 : n;
}

__device__ __forceinline__ int attn_nodes(const TreeAttnArgs &A, int b, bool &bad) {
    if (!A.nodes) {
        bad = false;
        return A.T;
    }
    const int n = __ldg(A.nodes + b);
    bad = n < 0 || n > A.T;
    return bad ? 0 : n;
}

// Tiles of cached keys of a sequence of `len` tokens.  Tiles follow one another
// every ktile keys -- whole pages, or equal parts of one -- except where pages
// are larger than a tile and no multiple of it (per_page > 0): there every
// page is cut into per_page tiles of its own, the last of them short.
__device__ __forceinline__ int attn_prefix_tiles(const TreeAttnArgs &A, int len) {
    if (A.per_page == 0) return (len + A.ktile - 1) / A.ktile;
    const int full = len / A.page_size, rest = len - full * A.page_size;
    return full * A.per_page + (rest + A.ktile - 1) / A.ktile;
}

// First key position of tile t, and the keys of it that the sequence has.
__device__ __forceinline__ void attn_tile(const TreeAttnArgs &A, int len, int t, int &pos, int &valid) {
    if (A.per_page == 0) {
        pos = t * A.ktile;
        valid = min(A.ktile, len - pos);
    } else {
        const int page = t / A.per_page, off = (t - page * A.per_page) * A.ktile;
        pos = page * A.page_size + off;
        valid = min(min(A.ktile, A.page_size - off), len - pos);
    }
}

// One part of a unit that a CTA works on: tiles [t0, t1) of unit (b, h); tile
// index `prefix` is the tile of the new keys.
struct AttnPiece {
    int b, h, len, prefix, t0, t1;
    bool first;  // the first piece of the group's range
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == prefix + 1; }
};

__device__ __forceinline__ long long attn_lo(long long W, int g, int groups) { return W * g / groups; }

// The walk over a group's pieces.  start() finds the first one (all threads
// of the block call it; `scan` is shared memory of NT / 32 long longs, two at least), next()
// steps on.
struct AttnWalk {
    long long W = 0, lo = 0, hi = 0, at = 0;  // all tiles, this group's range, the next tile
    int groups = 0;                           // groups that have tiles: no range of theirs is empty
    int b = 0, h = 0, tile = 0;               // where `at` is
    int len = 0, prefix = 0;

    template <int NT>
    __device__ __forceinline__ void start(const TreeAttnArgs &A, int g, long long *scan) {
        const int tid = threadIdx.x;
        const int per = (A.B + NT - 1) / NT;
        const int b0 = min(A.B, tid * per), b1 = min(A.B, b0 + per);
        long long sum = 0;
        bool bad;
        for (int i = b0; i < b1; ++i) sum += static_cast<long long>(attn_prefix_tiles(A, attn_len(A, i, bad)) + 1) * A.Hkv;
        // inclusive scan of the threads' sums
        const int lane = tid & 31, warp = tid >> 5;
        long long inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(FULL, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        long long before = 0, total = 0;
        for (int w = 0; w < NT / 32; ++w) {
            if (w < warp) before += scan[w];
            total += scan[w];
        }
        __syncthreads();
        W = total;
        groups = W < A.groups ? static_cast<int>(W) : A.groups;
        lo = attn_lo(W, min(g, groups), groups);
        hi = attn_lo(W, min(g + 1, groups), groups);
        at = lo;
        const long long from = before + inc - sum;
        if (lo < hi && lo >= from && lo < from + sum) {
            long long x = lo - from;
            for (int i = b0; i < b1; ++i) {
                const int n = attn_len(A, i, bad), p = attn_prefix_tiles(A, n);
                const long long unit = static_cast<long long>(p + 1) * A.Hkv;
                if (x < unit) {
                    scan[0] = i;
                    scan[1] = x;
                    break;
                }
                x -= unit;
            }
        }
        __syncthreads();
        if (lo < hi) {
            b = static_cast<int>(scan[0]);
            len = attn_len(A, b, bad);
            prefix = attn_prefix_tiles(A, len);
            h = static_cast<int>(scan[1] / (prefix + 1));
            tile = static_cast<int>(scan[1] - static_cast<long long>(h) * (prefix + 1));
        } else {
            b = h = tile = len = prefix = 0;
        }
        __syncthreads();
    }

    // The next piece, or false at the end of the range.
    __device__ __forceinline__ bool next(const TreeAttnArgs &A, AttnPiece &p) {
        if (at >= hi) return false;
        p.b = b;
        p.h = h;
        p.len = len;
        p.prefix = prefix;
        p.first = at == lo;
        p.t0 = tile;
        const long long left = hi - at;
        p.t1 = static_cast<int>(tile + left < prefix + 1 ? tile + left : prefix + 1);
        at += p.t1 - p.t0;
        tile = p.t1;
        if (tile == prefix + 1 && at < hi) {
            tile = 0;
            if (++h == A.Hkv) {
                h = 0;
                ++b;
                bool bad;
                len = attn_len(A, b, bad);
                prefix = attn_prefix_tiles(A, len);
            }
        }
        return true;
    }
};

// Slot of a piece that is not a whole unit: a piece that begins its group's
// range takes slot 0, a piece that ends it slot 1.
__device__ __forceinline__ size_t attn_slot(const TreeAttnArgs &A, int group, int mtile, bool first) {
    return (static_cast<size_t>(group) * A.mtiles + mtile) * 2 + (first ? 0 : 1);
}

// Tell the join about the unit that begins in this group and goes on in the
// next ones (at most one does): {b, h, parts, slot of the first part}.
__device__ __forceinline__ void attn_write_desc(const TreeAttnArgs &A, int g, const AttnWalk &w, bool any,
                                                const AttnPiece &last) {
    int *d = A.desc + static_cast<size_t>(g) * ATTN_DESC;
    if (!any || last.t0 != 0 || last.t1 == last.prefix + 1) {
        d[2] = 0;
        return;
    }
    const long long end = w.hi + (last.prefix + 1 - last.t1);  // one past the unit's last tile
    int n = 1;
    while (g + n < w.groups && attn_lo(w.W, g + n, w.groups) < end) ++n;
    d[0] = last.b;
    d[1] = last.h;
    d[3] = last.first ? 0 : 1;
    d[2] = n;
}

// Ancestor mask of node i (itself included); sets bad for a parent that is
// not a node before i.  A null `up` is a chain: node i sees nodes 0 .. i.
__device__ __forceinline__ uint64_t attn_mask(const int32_t *up, int i, bool &bad) {
    if (!up) return (2ull << i) - 1ull;
    uint64_t m = 0;
    int j = i;
    for (int step = 0; step < MAX_NODES && j >= 0; ++step) {
        m |= 1ull << j;
        const int p = __ldg(up + j);
        if (p >= j || p < -1) {
            bad = true;
            break;
        }
        j = p;
    }
    return m;
}

// Flags that one thread of `nt` finds in its share of sequence b's page table.
__device__ __forceinline__ int attn_check_pages(const TreeAttnArgs &A, int b, int len, int t, int nt) {
    const int n = (len + A.page_size - 1) / A.page_size;
    const int32_t *row = A.table + static_cast<size_t>(b) * A.max_pages;
    int bad = 0;
#pragma unroll 8
    for (int i = t; i < n; i += nt) {
        const int p = __ldg(row + i);
        bad |= (p < 0 || p >= A.num_pages) ? F_BAD_ID : 0;
    }
    return bad;
}

// The page of key position pos, in bounds whatever the table holds.
__device__ __forceinline__ int attn_page(const TreeAttnArgs &A, int b, int page) {
    const int p = __ldg(A.table + static_cast<size_t>(b) * A.max_pages + page);
    return p < 0 || p >= A.num_pages ? 0 : p;
}

}  // namespace mtp
