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
// groups: the result does not depend on which CTA ran first.  Where no unit can
// have more than a few tiles, whole units are dealt out instead and nothing is
// joined: the second launch takes as long as several tiles.
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

// The node of query row r = node G + head: r / G by multiplication (r < 64 G and
// G <= 4096, so r G < 2^32 and the quotient is exact).
__device__ __forceinline__ int node_of(const TreeAttnArgs &A, int r) {
    return static_cast<int>(__umulhi(static_cast<uint32_t>(r), A.g_inverse)) + (A.G == 1 ? r : 0);
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

// Groups that have tiles: none of their ranges is empty.
__device__ __forceinline__ int attn_groups(const TreeAttnArgs &A, long long W) {
    return W < A.groups ? static_cast<int>(W) : A.groups;
}
// The first tile of group g's range (a 64-bit division only where it is needed).
__device__ __forceinline__ long long attn_lo(long long W, int g, int groups) {
    if (W == groups) return g;
    const unsigned long long x = static_cast<unsigned long long>(W) * g;
    return x >> 32 ? static_cast<long long>(x / groups) : static_cast<uint32_t>(x) / static_cast<uint32_t>(groups);
}

// The walk over a group's pieces.  start() finds the first one, in every warp
// by itself (a lane takes a stretch of the sequences): a barrier would cost
// more than the second reading of a few lengths.
struct AttnWalk {
    long long hi = 0, at = 0;    // the end of this group's range, the next tile
    int b = 0, h = 0, tile = 0;  // where `at` is
    int len = 0, prefix = 0;
    int extra = 0;               // a unit ends with so many tiles that are none (see start)
    bool begins = true;          // no piece was taken yet

    // Returns the number of all tiles (of all units where they are not split;
    // hi and at count units then).
    __device__ __forceinline__ long long start(const TreeAttnArgs &A, int g) {
        if (A.whole) {
            const long long units = static_cast<long long>(A.B) * A.Hkv;
            at = attn_lo(units, min(g, A.groups), A.groups);
            hi = attn_lo(units, min(g + 1, A.groups), A.groups);
            b = static_cast<int>(at / A.Hkv);
            h = static_cast<int>(at - static_cast<long long>(b) * A.Hkv);
            if (at < hi) read(A);
            return units;
        }
        const int lane = threadIdx.x & 31;
        const int per = (A.B + 31) / 32;
        const int b0 = min(A.B, lane * per), b1 = min(A.B, b0 + per);
        long long sum = 0;
        bool bad;
#pragma unroll 4
        for (int i = b0; i < b1; ++i) {
            len = attn_len(A, i, bad);
            prefix = attn_prefix_tiles(A, len);
            sum += prefix + 1;
        }
        sum *= A.Hkv;
        long long inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(FULL, inc, d);
            if (lane >= d) inc += o;
        }
        // On the tensor cores the start and end of a piece take the time of
        // about three tiles: where there are tiles enough, that is counted.  (A
        // sequence without a cache is Hkv pieces of one tile each, which one
        // group would get otherwise.  16 sequences of 1333 to 4000 tokens and
        // an empty one: 59 -> 45 us.  In the other kernel a piece costs little
        // beside its tiles: 1000 tokens of 32 sequences took 152 us without
        // and 177 us with three tiles.)
        const long long real = __shfl_sync(FULL, inc, 31);
        if (real >= 4ll * A.groups) extra = A.extra;
        const long long W = real + static_cast<long long>(A.B) * A.Hkv * extra;
        inc += static_cast<long long>(b1) * A.Hkv * extra;
        sum += static_cast<long long>(b1 - b0) * A.Hkv * extra;
        const int groups = attn_groups(A, W);
        const long long lo = attn_lo(W, min(g, groups), groups);
        hi = attn_lo(W, min(g + 1, groups), groups);
        at = lo;
        const long long from = inc - sum;
        const uint32_t own = __ballot_sync(FULL, lo < hi && lo >= from && lo < inc);
        if (own == 0) return W;  // no tiles for this group
        long long x = lo - from;
        int i = b0;
        if ((own >> lane) & 1u) {
            for (;; ++i) {
                if (per > 1) {  // (one sequence to a lane: they are here)
                    len = attn_len(A, i, bad);
                    prefix = attn_prefix_tiles(A, len);
                }
                const long long unit = static_cast<long long>(prefix + 1 + extra) * A.Hkv;
                if (x < unit) break;  // (x lies in this lane's stretch)
                x -= unit;
            }
        }
        const int src = __ffs(own) - 1;
        b = __shfl_sync(FULL, i, src);
        len = __shfl_sync(FULL, len, src);
        prefix = __shfl_sync(FULL, prefix, src);
        const int first = __shfl_sync(FULL, static_cast<int>(x), src);  // < Hkv (prefix + 1 + extra)
        h = first / (prefix + 1 + extra);
        tile = first - h * (prefix + 1 + extra);
        if (tile > prefix) {  // the range begins behind a unit's tiles
            at += prefix + 1 + extra - tile;
            step(A);
        }
        return W;
    }

    __device__ __forceinline__ void read(const TreeAttnArgs &A) {
        bool bad;
        len = attn_len(A, b, bad);
        prefix = attn_prefix_tiles(A, len);
    }

    // On to the next unit, if the range has it.
    __device__ __forceinline__ void step(const TreeAttnArgs &A) {
        if (at >= hi) return;
        tile = 0;
        if (++h == A.Hkv) {
            h = 0;
            ++b;
            read(A);
        }
    }

    // The next piece, or false at the end of the range.
    __device__ __forceinline__ bool next(const TreeAttnArgs &A, AttnPiece &p) {
        if (at >= hi) return false;
        p.b = b;
        p.h = h;
        p.len = len;
        p.prefix = prefix;
        p.first = begins;
        begins = false;
        p.t0 = tile;
        if (A.whole) {
            p.t1 = prefix + 1;
            if (++at < hi && ++h == A.Hkv) {
                h = 0;
                ++b;
                read(A);
            }
            return true;
        }
        const long long left = hi - at;
        p.t1 = static_cast<int>(tile + left < prefix + 1 ? tile + left : prefix + 1);
        at += p.t1 - p.t0;
        tile = p.t1;
        if (tile == prefix + 1) {
            at += extra;
            step(A);
        }
        return true;
    }
};

// Slot of a piece that is not a whole unit: a piece that begins its group's
// range takes slot 0, a piece that ends it slot 1.
__device__ __forceinline__ size_t attn_slot(const TreeAttnArgs &A, int group, int mtile, bool first) {
    return (static_cast<size_t>(group) * A.mtiles + mtile) * 2 + (first ? 0 : 1);
}

// Programmatic launches: what the kernels before this one in the stream wrote
// may be read after pdl_wait(); the next kernel's CTAs may be set up from
// pdl_next() on (they wait in turn).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Tell the join about the unit that begins in this group and goes on in the
// next ones (at most one does): {b, h, parts, slot of the first part}.
__device__ __forceinline__ void attn_write_desc(const TreeAttnArgs &A, int g, long long W, long long hi,
                                                const AttnPiece &last) {
    if (A.whole) return;
    int *d = A.desc + static_cast<size_t>(g) * ATTN_DESC;
    if (last.t0 != 0 || last.t1 == 0 || last.t1 == last.prefix + 1) {  // (t1 = 0: the group had no piece)
        d[2] = 0;
        return;
    }
    const long long end = hi + (last.prefix + 1 - last.t1);  // one past the unit's last tile (the range ended inside of the unit)
    const int groups = attn_groups(A, W);
    int n = 1;
    while (g + n < groups && attn_lo(W, g + n, groups) < end) ++n;
    d[0] = last.b;
    d[1] = last.h;
    d[3] = last.first ? 0 : 1;
    d[2] = n;
}

// Ancestor masks of a tree's n nodes (a node's own bit included) into `mask`,
// by one warp, two nodes to a lane; a null `up` is a chain.  Each round a node
// takes over the mask of the farthest ancestor it knows of and that one's own,
// so six rounds reach any of 64 -- not a chain of loads as deep as the tree.
// Returns F_BAD_ID (in some lane) for a parent that is not a node before its
// child.  `above` is scratch of MAX_NODES ints.
__device__ __forceinline__ int attn_masks(const int32_t *up, int n, uint64_t *mask, int *above) {
    const int lane = threadIdx.x & 31;
    int flag = 0;
    if (!up) {
        for (int i = lane; i < n; i += 32) mask[i] = (2ull << i) - 1ull;
        __syncwarp();
        return 0;
    }
    for (int i = lane; i < n; i += 32) {
        int p = __ldg(up + i);
        if (p >= i || p < -1) {
            flag = F_BAD_ID;
            p = -1;
        }
        above[i] = p;
        mask[i] = 1ull << i;
    }
    __syncwarp();
    for (int reach = 1; reach < n; reach <<= 1) {
        uint64_t m[2];
        int a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = lane + 32 * e, p = i < n ? above[i] : -1;
            m[e] = p < 0 ? 0ull : mask[p];
            a[e] = p < 0 ? -1 : above[p];
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = lane + 32 * e;
            if (i < n) {
                mask[i] |= m[e];
                above[i] = a[e];
            }
        }
        __syncwarp();
    }
    return flag;
}

// Flags that one thread of `nt` finds in its share of sequence b's page table.
__device__ __forceinline__ int attn_check_pages(const TreeAttnArgs &A, int b, int len, int t, int nt) {
    const int n = (static_cast<uint32_t>(len) + A.page_size - 1) / A.page_size;  // (the sum may pass 2^31)
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
