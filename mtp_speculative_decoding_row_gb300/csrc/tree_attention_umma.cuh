// tree_attention_umma.cuh -- tree attention on the tensor cores: bfloat16
// storage, head sizes 64, 128 and 256, caches that tiled copies can address
// (tree_attention.cuh has the split of the work over CTAs).
//
// One CTA per SM works through its list of key tiles.  A tile is BN keys of
// one (sequence, key head); the CTA's query rows (nodes x query heads of the
// group) stay in shared memory for the piece.
//   warp 0      copies key and value tiles page by page into a ring of slots
//               (cp.async.bulk.tensor, 128-byte swizzle)
//   warps 1, 2  issue S = Q K^T into a score buffer of TMEM and, when the
//               weights are back, O += P V with P read from TMEM; a warp for
//               each group of softmax warps, so that neither waits for the
//               other's weights
//   warp 3      loads the new keys and values and the ancestor masks of a
//               piece, and checks its page table
//   warps 4 ..  softmax: a thread has one row of a score tile, so the running
//               maximum and sum need no exchange.  Weights go back to TMEM as
//               bfloat16 over the scores they came from.  The same warps copy
//               the next piece's queries while this one is worked on.
// The softmax of a tile takes longer than its copy or its products, so two
// score tiles are worked on at a time by two groups of four warps, each with
// its own accumulator in TMEM:
//   ROWS   more than 128 query rows: one group has rows 0 - 127, the other
//          128 - 255, and a key tile is copied once for both
//   KEYS   33 to 128 rows: the groups take turns at the key tiles; at the end
//          of a piece their maxima, sums and outputs are joined
//   FEW    up to 32 rows: as KEYS, but those rows would lie in the lanes of one
//          warp and leave three idle, so each warp of a group gets the scores
//          of a quarter of the keys (64 sequences of 768 tokens, 16 rows: 74 ->
//          68 us; one of 131072, 32 rows: 3 % less).  They exchange the
//          maximum of each tile; weights go through shared memory, because in
//          TMEM a warp reaches its own lanes only
//   ONE    heads of 256: TMEM holds one accumulator, so one group works, with
//          two score buffers (the products of tile j + 1 run under the softmax
//          of tile j); warp 1 issues the products with the keys, warp 2 those
//          with the values
// Measured, replayed in a graph: one token after 1000 12.4 us (latency: two
// launches and a chain of dependent loads); 64 sequences of up to 8192, heads of
// 256, 132 us, and one of 131072, 96 us (memory, at 0.81 of a copy's rate);
// trees of 64 nodes over 8 sequences of 16384, 260 us (the softmax warps; 0.55 of
// the tensor cores' rate).
//
// The output accumulator is rescaled only when a row's maximum has risen by
// more than 2^8 since the last time: until then the weights are taken
// relative to the older maximum, which changes nothing but their scale.
//
// Rounding: scores, statistics and outputs are float32; the weights are
// rounded to bfloat16 because the tensor core takes both operands of P V in
// one type, and the values are bfloat16.  Their sum is taken before rounding.
//
// PREFIX: the same of shared prefixes (mtp_prefix_attention): no new keys, the
// rows of a piece are those of a tile of all the sequences that have the prefix,
// and every result is a part that another kernel joins with the sequence's own.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "tree_attention.cuh"
#include "umma.cuh"

namespace mtp {
namespace {

constexpr int LOADERS = 32;
constexpr float RESCALE = 8.f;  // rescale when the maximum rose by this many powers of two
constexpr int MAX_SLOTS = 14;
enum Mode { ONE = 0, KEYS = 1, ROWS = 2, FEW = 3 };

template <int D, int MODE>
struct Cfg {
    static constexpr int NT = MODE == ONE ? 256 : 384;
    static constexpr int BN = D == 256 ? 64 : 128;
    static constexpr int CH = D / 64;                      // 64-element blocks of a row
    static constexpr bool TURNS = MODE == KEYS || MODE == FEW;  // the groups take turns at the key tiles
    static constexpr uint32_t P = MODE == FEW ? 16384 : 0; // weights in shared memory: 32 rows for each group
    static constexpr int GROUPS = MODE == ONE ? 1 : 2;     // of softmax warps
    static constexpr uint32_t SLOT = BN * D * 2;           // a key or value tile
    static constexpr uint32_t S_COL = 128;                 // score buffers at columns 0 and 128
    static constexpr uint32_t O_COL = 256;                 // accumulators at 256 and 256 + D
};

// What the loader says about a piece lies in a ring of four.
template <class Walk>
struct Control {
    uint64_t full[2 * MAX_SLOTS], empty[MAX_SLOTS], s_full[2], p_half[2], p_full[2], o_done[2], q_full[2], q_empty[2];
    uint64_t grant[8];            // two slots of the ring are the loader's to fill (at most slots / 2 at a time)
    uint64_t masks[4], ready[4], done[4];  // a piece's masks are there; all that the loader found out is; it has been read
    uint64_t tops[2];             // FEW: the maxima of a tile's quarters are there
    uint64_t stats, joined;       // KEYS: both groups' statistics are there; both have read the accumulators
    uint64_t mask[4][MAX_NODES];
    uint64_t poison[4];
    int flag[4];
    int above[MAX_NODES];
    long long W;
    Walk begin;
    float top[2][2][4][32];       // FEW: group, even and odd tiles, quarter, row
    float m[2][128], l[2][128];   // KEYS: the groups' statistics
    uint32_t tmem;
    int dead;
};

// A ring position: the slot and how often the ring has gone round.  A slot has
// two barriers for "full", for even and odd laps: in KEYS mode a reader passes
// over the other group's slots without waiting for them, and could take the
// lap before last for its own if there were one barrier with a parity bit.
// (When it looks at a slot in lap k it has read a slot that was filled after
// this one in lap k - 1, and that fill had waited for lap k - 2 to be read.)
struct Ring {
    int slots;
    int slot = 0, lap = 0;
    __device__ __forceinline__ explicit Ring(int n) : slots(n) {}
    __device__ __forceinline__ void step() {
        if (++slot == slots) {
            slot = 0;
            ++lap;
        }
    }
    __device__ __forceinline__ int full() const { return 2 * slot + (lap & 1); }  // index of the barrier
    __device__ __forceinline__ uint32_t phase() const { return (lap >> 1) & 1; }  // its parity
};

// Wait for an mbarrier's phase, A.wait_us at most (2 s but for tests).  The first
// tries are inline, the rest is one function for all of the kernel's waits:
// every byte of code counts here (see softmax_part).  Lanes may differ in what
// they get back, so it is put to the vote before it decides where a warp goes.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, uint32_t us) { return mbar_wait_spin(bar, parity, us * 1000ull); }
__device__ __forceinline__ bool wait_for(const TreeAttnArgs &A, uint32_t bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || wait_long(bar, parity, A.wait_us);
}

__device__ __forceinline__ int round16(int n) { return (n + 15) & ~15; }

// The largest of three (NaN only if all are).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Weights of one block of 32 scores, two to a register; their sum goes to acc.
__device__ __forceinline__ void weights(const uint32_t (&s)[32], uint64_t K2, uint64_t N2, uint64_t (&acc)[2], uint32_t (&p)[16]) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        float a, b;
        f2unpack(f2fma(f2pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), K2, N2), a, b);
        a = ex2(a);
        b = ex2(b);
        acc[(i >> 1) & 1] = f2add(acc[(i >> 1) & 1], f2pack(a, b));
        p[i / 2] = bf16x2(a, b);
    }
}

// The same, stored as bfloat16 in 16 columns at p_addr.
__device__ __forceinline__ void weigh_block(const uint32_t (&s)[32], uint64_t K2, uint64_t N2, uint64_t (&acc)[2], uint32_t p_addr) {
    uint32_t p[16];
    weights(s, K2, N2, acc, p);
    tmem_st16(p_addr, p);
}

// The maximum of one block; with `masked`, of the columns in `see`, and -inf
// is written over the others.
__device__ __forceinline__ void max_block(uint32_t (&s)[32], float (&t)[4], bool masked, uint32_t see, uint32_t s_addr) {
    if (masked) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!((see >> i) & 1u)) s[i] = 0xff800000u;
        __syncwarp();
        tmem_st32(s_addr, s);
    }
#pragma unroll
    for (int i = 0; i < 32; i += 2)
        t[(i >> 1) & 3] = max3(t[(i >> 1) & 3], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
}

// The row's reference maximum for a tile whose largest score is `top` (in
// units of log2 e); the accumulator (if this warp has one) is rescaled where it
// has to be.
__device__ __forceinline__ void rescale(const TreeAttnArgs &A, float top, bool first, float &m, float &l, uint32_t o_addr, int ocols, uint32_t o_bar,
                                        uint32_t o_phase, bool &ok, bool has = true) {
    if (first) {
        m = top;
        l = 0.f;
        return;
    }
    const bool up = top > m + RESCALE;
    if (!__any_sync(FULL, up)) return;
    const float f = up ? ex2(m - top) : 1.f;
    if (up) m = top;
    l *= f;
    if (!has) return;
    ok = wait_for(A, o_bar, o_phase) && ok;  // the products before this tile
    __syncwarp();
    tmem_fence_after_sync();
#pragma unroll 1
    for (int c = 0; c < ocols; c += 32) {
        uint32_t o[32];
        __syncwarp();
        tmem_ld32(o_addr + c, o);
        tmem_wait_ld32(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st32(o_addr + c, o);
        tmem_wait_st();
    }
}

// The weights stored so far may be read by a product.
__device__ __forceinline__ void publish(uint32_t bar) {
    tmem_wait_st();
    tmem_fence_before_sync();
    mbar_arrive(bar);
}

__device__ __forceinline__ float sum4(const uint64_t (&acc)[2]) {
    float a0, a1, b0, b1;
    f2unpack(acc[0], a0, a1);
    f2unpack(acc[1], b0, b1);
    return (a0 + a1) + (b0 + b1);
}

// Softmax of a score tile of CH blocks of 32 columns, all of which the row
// sees.  Two blocks are in registers at a time; of four, the last two are read
// a second time for their weights while those of the first two are worked on
// (168 registers a thread do not hold 128 scores and what else is needed).
// Block c's weights go to columns 16 c .. of the tile, over scores that have
// been read.  The first half of them is announced as soon as it is there: the
// product over those keys runs while the other half is made (trees of 64
// nodes: 290 -> 275 us).
template <int CH>
__device__ __forceinline__ void softmax_full(const TreeAttnArgs &A, uint32_t s_addr, uint32_t o_addr, int ocols, float scale, bool first, float &m,
                                             float &l, uint32_t o_bar, uint32_t o_phase, uint32_t half_bar, bool &ok) {
    uint32_t s[2][32];
    float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    __syncwarp();  // TMEM accesses are warp-wide, and the lanes may have left a wait one by one
    if (CH == 4) {
        tmem_ld32(s_addr + 64, s[0]);
        tmem_ld32(s_addr + 96, s[1]);
        tmem_wait_ld32(s);
        max_block(s[0], t, false, 0u, 0u);
        max_block(s[1], t, false, 0u, 0u);
    }
    tmem_ld32(s_addr, s[0]);
    tmem_ld32(s_addr + 32, s[1]);
    tmem_wait_ld32(s);
    max_block(s[0], t, false, 0u, 0u);
    max_block(s[1], t, false, 0u, 0u);
    rescale(A, max3(t[0], t[1], fmaxf(t[2], t[3])) * scale, first, m, l, o_addr, ocols, o_bar, o_phase, ok);
    const uint64_t K2 = f2pack(scale, scale), N2 = m == -INFINITY ? f2pack(0.f, 0.f) : f2pack(-m, -m);
    uint64_t acc[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
    __syncwarp();
    weigh_block(s[0], K2, N2, acc, s_addr);
    if (CH == 4) tmem_ld32(s_addr + 64, s[0]);
    if (CH == 2) publish(half_bar);
    weigh_block(s[1], K2, N2, acc, s_addr + 16);
    if (CH == 4) {
        publish(half_bar);
        tmem_wait_ld32(s[0]);
        tmem_ld32(s_addr + 96, s[1]);
        weigh_block(s[0], K2, N2, acc, s_addr + 32);
        tmem_wait_ld32(s[1]);
        weigh_block(s[1], K2, N2, acc, s_addr + 48);
    }
    l += sum4(acc);
    tmem_wait_st();
}

// The same for the other tiles, of `blocks` blocks: the row sees the columns
// in lo (the first 64) and hi.  One short loop for all of them: the warps of
// an SM run five different programs at once, and unrolled by kind of tile they
// did not fit in its instruction cache.
__device__ __forceinline__ void softmax_part(const TreeAttnArgs &A, uint32_t s_addr, uint32_t o_addr, int ocols, float scale, int blocks, uint64_t lo,
                                             uint64_t hi, bool first, float &m, float &l, uint32_t o_bar, uint32_t o_phase,
                                             bool &ok) {
    uint32_t s[32];
    float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
    for (int c = 0; c < blocks; ++c) {
        __syncwarp();
        tmem_ld32(s_addr + 32 * c, s);
        tmem_wait_ld32(s);
        max_block(s, t, true, static_cast<uint32_t>((c < 2 ? lo : hi) >> (32 * (c & 1))), s_addr + 32 * c);
    }
    tmem_wait_st();
    rescale(A, max3(t[0], t[1], fmaxf(t[2], t[3])) * scale, first, m, l, o_addr, ocols, o_bar, o_phase, ok);
    const uint64_t K2 = f2pack(scale, scale), N2 = m == -INFINITY ? f2pack(0.f, 0.f) : f2pack(-m, -m);
    uint64_t acc[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
#pragma unroll 1
    for (int c = 0; c < blocks; ++c) {
        __syncwarp();
        tmem_ld32(s_addr + 32 * c, s);
        tmem_wait_ld32(s);
        weigh_block(s, K2, N2, acc, s_addr + 16 * c);
    }
    l += sum4(acc);
    tmem_wait_st();
}

// FEW: a quarter of a score tile of at most 32 rows, by one of a group's four
// warps.  `any`: there are keys in it, of which the row sees those in `see`.
// The four share the row's maximum; each keeps the sum of its own weights.
// Weights go to shared memory at p (128-byte rows, swizzled).
__device__ __forceinline__ void softmax_quarter(const TreeAttnArgs &A, uint32_t s_addr, uint32_t o_addr, int ocols, float scale, int quarter, bool any,
                                                uint32_t see, bool live, bool first, float &m, float &l, uint32_t o_bar,
                                                uint32_t o_phase, bool used, float (&tops)[4][32], uint32_t top_bar,
                                                uint32_t top_phase, unsigned char *p, int prows, bool &ok) {
    const int lane = threadIdx.x & 31;
    uint32_t s[32];
    float top = -INFINITY;
    if (any) {
        float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        __syncwarp();
        tmem_ld32(s_addr, s);
        tmem_wait_ld32(s);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!((see >> i) & 1u)) s[i] = 0xff800000u;
        max_block(s, t, false, 0u, 0u);
        if (live) top = max3(t[0], t[1], fmaxf(t[2], t[3])) * scale;
    }
    tops[quarter][lane] = top;
    __syncwarp();
    if (lane == 0) mbar_arrive(top_bar);
    ok = wait_for(A, top_bar, top_phase) && ok;
    top = fmaxf(max3(tops[0][lane], tops[1][lane], tops[2][lane]), tops[3][lane]);
    rescale(A, top, first, m, l, o_addr, ocols, o_bar, o_phase, ok, quarter == 0);
    if (any) {
        const uint64_t K2 = f2pack(scale, scale), N2 = m == -INFINITY ? f2pack(0.f, 0.f) : f2pack(-m, -m);
        uint64_t acc[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
        uint32_t w[16];
        weights(s, K2, N2, acc, w);
        l += sum4(acc);
        // (the product that read the weights before these is done: its scores'
        // successors are here)
        if (used) ok = wait_for(A, o_bar, o_phase) && ok;
        if (lane < prows && ok) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4 *>(p + (quarter >> 1) * 4096 + sw128(lane, (quarter & 1) * 4 + j)) =
                    make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        }
        fence_proxy_async();
    }
}

// Values that are not finite, of the nodes in `seen`, added to columns c0 .. c1
// of one finished row (`part`: of a partial result): the products took them as
// zeros.
__device__ __noinline__ void add_far_values(float *part, bf16_t *out, const bf16_t *v, int64_t stride, uint64_t seen, int c0, int c1) {
    for (; seen; seen &= seen - 1) {
        const bf16_t *row = v + (__ffsll(static_cast<long long>(seen)) - 1) * stride;
        for (int c = c0; c < c1; ++c) {
            const float x = __uint_as_float(static_cast<uint32_t>(row[c].bits) << 16);
            if (fabsf(x) < INFINITY) continue;
            if (part)
                part[c] += x;
            else
                out[c].bits = static_cast<uint16_t>(bf16x2(__uint_as_float(static_cast<uint32_t>(out[c].bits) << 16) + x, 0.f));
        }
    }
}

// The new keys or values of n nodes into a slot, by one warp.  Of the keys no
// more than the sequence's nodes is looked at; the values behind them are zero,
// and so is one that is not finite (its rows get it later): those nodes' bits are
// returned.
template <int D, int BN>
__device__ __forceinline__ uint64_t load_new(const TreeAttnArgs &A, unsigned char *dst, bool kv, int b, int h, int n) {
    const int lane = threadIdx.x & 31;
    uint64_t poison = 0;
    const bf16_t *src = static_cast<const bf16_t *>(kv ? A.v_new : A.k_new);
    const int64_t *st = kv ? A.vs : A.ks;
    src += b * st[0] + h * st[2];
    const int fill = (kv ? round16(n > 0 ? n : 1) : n) * (D / 8);
#pragma unroll 1
    for (int i0 = lane; i0 < fill; i0 += 32 * 4) {
        uint4 y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = (i0 + 32 * e) / (D / 8), u = (i0 + 32 * e) % (D / 8);
            y[e] = j < n ? __ldg(reinterpret_cast<const uint4 *>(src + j * st[1]) + u) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = (i0 + 32 * e) / (D / 8), u = (i0 + 32 * e) % (D / 8);
            if (i0 + 32 * e >= fill) break;
            if (kv) {
                uint32_t w[4] = {y[e].x, y[e].y, y[e].z, y[e].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const bool lo = (w[q] & 0x7f80u) == 0x7f80u, hi = (w[q] & 0x7f800000u) == 0x7f800000u;
                    if (lo || hi) poison |= 1ull << j;
                    w[q] = (lo ? 0u : w[q] & 0xffffu) | (hi ? 0u : w[q] & 0xffff0000u);
                }
                y[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *reinterpret_cast<uint4 *>(dst + (u >> 3) * (BN * 128) + sw128(j, u & 7)) = y[e];
        }
    }
    return poison;
}

// Start copies of `rows` query rows from row `row` on, by `threads` threads, this
// being number i.
template <int D>
__device__ __noinline__ void copy_queries(const bf16_t *q, const TreeAttnArgs &A, int row, int rows, uint32_t dst, int i, int threads) {
    constexpr int VECS = D / 8;
#pragma unroll 1
    for (; i < rows * VECS; i += threads) {
        const int r = i / VECS, u = i % VECS, t = node_of(A, row + r);
        cp_async16(dst + (u >> 3) * A.qrows * 128 + sw128(r, u & 7), q + t * A.qs[1] + (row + r - t * A.G) * A.qs[2] + 8 * u);
    }
}

// The same of rows `row` .. of a prefix's piece: row r of its tile is a head of
// token `token + d` of the prefix's sequences, T tokens each.
template <int D>
__device__ __noinline__ void copy_prefix_queries(const TreeAttnArgs &A, const PrefixPiece &p, int row, int rows, uint32_t dst, int i, int threads) {
    constexpr int VECS = D / 8;
    const int seq0 = A.T == 1 ? p.token : p.token / A.T, t0 = p.token - seq0 * A.T, u = i % VECS;  // (threads is a multiple of VECS)
    const bf16_t *q = static_cast<const bf16_t *>(A.q) + (p.start + seq0) * A.qs[0] + static_cast<int64_t>(p.h) * A.G * A.qs[2] + 8 * u;
    dst += (u >> 3) * A.qrows * 128;
#pragma unroll 4
    for (int r = i / VECS; r < rows; r += threads / VECS) {
        const int d = node_of(A, p.rest + row + r), t = t0 + d;
        const int s = A.T == 1 ? t : static_cast<int>(__umulhi(static_cast<uint32_t>(t), A.t_inverse));  // (t < T + 257, T <= 64: exact)
        cp_async16(dst + sw128(r, u & 7), q + s * A.qs[0] + (t - s * A.T) * A.qs[1] + (p.rest + row + r - d * A.G) * A.qs[2]);
    }
}

// The flags of a sequence are stored by the loader of one CTA, the one that has
// the first tile of its first head and row tile.
__device__ __forceinline__ bool flags_owner(const AttnPiece &p, int mtile) { return p.h == 0 && mtile == 0 && p.t0 == 0; }
__device__ __forceinline__ bool flags_owner(const PrefixPiece &p, int) { return p.h == 0 && p.mt == 0 && p.t0 == 0; }

// A CTA that has given up may belong to another head, tile or row tile of the
// sequence, and its report must not be lost whichever of the two comes first.
// So it leaves the call's number in A.late[b] before it adds its bit to the flags,
// and the owner looks there after its store: with a full fence between the two
// on either side, one of them sees the other.  (A workspace holds anything; the
// number is 64 random bits, another for each call.  A replayed graph has one
// number for all replays: the owner takes away what it has seen, and a report
// that came after it may show once more in the next replay.)
__device__ __forceinline__ void put_flag(const TreeAttnArgs &A, int b, int flag) {
    *const_cast<volatile int32_t *>(A.flags + b) = flag;
    __threadfence();
    volatile unsigned long long *late = A.late + b;
    if (*late == A.number) {
        atomicOr(A.flags + b, F_TIMEOUT);
        *late = 0ull;
    }
}

// By all threads of a CTA that has given up: its rows become NaN -- of a unit
// that it shares with others its part's sum, from which the join makes NaN --
// and its sequences are flagged.
template <class Walk>
__device__ __noinline__ void give_up(const TreeAttnArgs &A, const Walk &begin, int group, int mtile, int row0, int rows, int tid, int nt) {
    constexpr bool PREFIX = std::is_same<Walk, PrefixWalk>::value;
    Walk w = begin;
    typename Walk::Piece p;
    while (w.next(A, p)) {
        int live;
        if constexpr (PREFIX) {
            live = p.rows;
        } else {
            bool bad;
            const int n = attn_nodes(A, p.b, bad);
            live = min(rows, (bad ? A.rows : n * A.G) - row0);
        }
        if (p.whole()) {
            for (int r = 0; r < live; ++r) {
                if (A.row_o) {  // (of a prefix always)
                    if (tid == 0) {
                        A.row_m[unit_row(A, p) + row0 + r] = -INFINITY;
                        A.row_l[unit_row(A, p) + row0 + r] = NAN;
                    }
                } else {
                    const int node = node_of(A, row0 + r), hq = p.h * A.G + row0 + r - node * A.G;
                    const size_t at = (static_cast<size_t>(p.b) * A.T + node) * A.Hq + hq;
                    for (int c = tid; c < A.D; c += nt) static_cast<uint16_t *>(A.out)[at * A.D + c] = 0x7fffu;
                    if (A.lse && tid == 0) A.lse[at] = NAN;
                }
            }
        } else {
            float *slot = A.part + attn_slot(A, group, mtile, p.first) * attn_slot_floats(A.bm, A.D);
            for (int r = tid; r < live; r += nt) {
                slot[r] = -INFINITY;
                slot[A.bm + r] = NAN;
            }
        }
        if (A.flags && tid == 0) {
            atomicExch(A.late + p.b, A.number);
            __threadfence();
            if (flags_owner(p, mtile))
                *const_cast<volatile int32_t *>(A.flags + p.b) = F_TIMEOUT;  // (in place of a flag that may never have been stored)
            else
                atomicOr(A.flags + p.b, F_TIMEOUT);
        }
    }
}

template <int D, int MODE, bool PREFIX>
__global__ void __launch_bounds__(Cfg<D, MODE>::NT, 1)
    attn_umma_impl(const __grid_constant__ TreeAttnArgs A, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
    using C = Cfg<D, MODE>;
    using Walk = typename std::conditional<PREFIX, PrefixWalk, AttnWalk>::type;
    using Piece = typename Walk::Piece;
    constexpr int NT = C::NT, BM = MODE == ROWS ? 256 : 128;
    // FEW: weights; queries (blocks of 64 elements x qrows rows, once or twice), ring, control
    extern __shared__ __align__(1024) unsigned char smem[];
    const int qbufs = MODE == ROWS ? 2 : A.qbufs;  // ROWS: one for each group
    const uint32_t qblock = A.qrows * 128, qbytes = qblock * C::CH * qbufs;
    unsigned char *queries = smem + C::P;
    Control<Walk> &ctl = *reinterpret_cast<Control<Walk> *>(queries + qbytes + C::SLOT * A.slots);
    unsigned char *ring = queries + qbytes;
    const uint32_t sq = smem_addr(queries), ring0 = sq + qbytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = blockIdx.x / A.mtiles, mtile = blockIdx.x - group * A.mtiles;
    // this CTA's rows; of a prefix every piece has rows of its own
    const int row0 = PREFIX ? 0 : mtile * BM, rows = PREFIX ? 0 : min(BM, A.rows - row0);
    auto rows_of = [&](const Piece &p) {
        if constexpr (PREFIX)
            return p.rows;
        else
            return rows;
    };

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < A.slots; ++i) {
            mbar_init(smem_addr(&ctl.full[2 * i]), 1);
            mbar_init(smem_addr(&ctl.full[2 * i + 1]), 1);
            mbar_init(smem_addr(&ctl.empty[i]), MODE == ROWS ? 2 : 1);  // products that read a slot
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl.s_full[i]), 1);
            mbar_init(smem_addr(&ctl.p_half[i]), 128);
            mbar_init(smem_addr(&ctl.p_full[i]), MODE == FEW ? 4 : 128);
            mbar_init(smem_addr(&ctl.tops[i]), 4);
            mbar_init(smem_addr(&ctl.o_done[i]), 1);
            mbar_init(smem_addr(&ctl.q_full[i]), C::TURNS ? 256 : 128);  // ROWS: a group's own rows
            mbar_init(smem_addr(&ctl.q_empty[i]), C::TURNS ? 2 : 1);
        }
        for (int i = 0; i < 8; ++i) mbar_init(smem_addr(&ctl.grant[i]), 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_addr(&ctl.masks[i]), LOADERS);
            mbar_init(smem_addr(&ctl.ready[i]), LOADERS);
            mbar_init(smem_addr(&ctl.done[i]), 128 * C::GROUPS);
        }
        mbar_init(smem_addr(&ctl.stats), 256);
        mbar_init(smem_addr(&ctl.joined), 256);
        ctl.dead = 0;
        fence_mbar_init();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(&ctl.tmem, TMEM_COLS);
    }
    // Rows of the query tile that no query fills.  (The product reads 128 rows
    // of each block whatever qrows is: what lies behind them gives rows that
    // nobody looks at.)
    for (int buf = 0; buf < qbufs; ++buf) {
        const int used = PREFIX ? 0 : MODE == ROWS ? max(0, min(rows - 128 * buf, 128)) : rows;
        for (int i = tid; i < (A.qrows - used) * (D / 8); i += NT) {
            const int r = used + i / (D / 8), u = i % (D / 8);
            *reinterpret_cast<uint4 *>(queries + (buf * C::CH + (u >> 3)) * qblock + sw128(r, u & 7)) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    fence_proxy_async();
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tmem = ctl.tmem;
    // (what was done so far reads nothing that another kernel writes; the kernel of
    // the prefixes has waited for all before it, and wrote nothing that is read here)
    if (PREFIX || !A.overlap) pdl_wait();
    pdl_next();
    Walk walk;
    {
        const long long W = walk.start(A, group, attn_limit<PREFIX>(A));
        if (tid == 0) {  // for the end
            ctl.W = W;
            ctl.begin = walk;
        }
    }
    bool ok = (sq & 1023u) == 0u;    // the swizzle counts on it
    Piece pc;

    if (warp == 0) {
        // ---------------------------------------------------- copies ----
        Ring r(A.slots);
        int grants = 0;
        const int boxrows = min(C::BN, A.page_size);
        while (ok && walk.next(A, pc)) {
            for (int t = pc.t0; t < pc.t1 && ok; ++t) {
                if (!PREFIX && t == pc.prefix) {  // the loaders fill these two slots once they are free
                    for (int i = 0; i < 2; ++i) {
                        if (r.lap) ok = wait_for(A, smem_addr(&ctl.empty[r.slot]), (r.lap - 1) & 1) && ok;
                        r.step();
                    }
                    ok = __all_sync(FULL, ok);
                    if (lane == 0 && ok) mbar_arrive(smem_addr(&ctl.grant[grants & 7]));
                    ++grants;
                    continue;
                }
                int pos, valid;
                attn_tile(A, pc.len, t, pos, valid);
                const int page0 = pos / A.page_size, off = pos - page0 * A.page_size;
                const int pages = A.page_size >= C::BN ? 1 : (valid + A.page_size - 1) / A.page_size;
                const int mine = lane < pages ? attn_page(A, pc.b, page0 + lane) : 0;  // at most BN / 8 pages
                for (int kv = 0; kv < 2; ++kv) {
                    // (the first use of every slot needs no wait)
                    if (r.lap) ok = wait_for(A, smem_addr(&ctl.empty[r.slot]), (r.lap - 1) & 1) && ok;
                    ok = __all_sync(FULL, ok);
                    if (!ok) break;
                    const uint32_t full = smem_addr(&ctl.full[r.full()]), dst = ring0 + r.slot * C::SLOT;
                    const void *map = kv ? static_cast<const void *>(&vmap) : static_cast<const void *>(&kmap);
                    if (elect_one()) mbar_arrive_expect_tx(full, pages * C::CH * boxrows * 128);
                    __syncwarp();
                    for (int p = 0; p < pages; ++p) {
                        const int id = __shfl_sync(FULL, mine, p);
                        if (elect_one()) {
#pragma unroll
                            for (int c = 0; c < C::CH; ++c)
                                tma_load_4d(dst + c * (C::BN * 128) + p * boxrows * 128, map, c * 64, off, pc.h, id, full);
                        }
                        __syncwarp();
                    }
                    r.step();
                }
            }
        }
    } else if (warp < 3) {
        // -------------------------------------------------- products ----
        Ring r(A.slots);
        const int g = MODE == ONE ? 0 : warp - 1;  // the group of softmax warps
        int qi = MODE == ROWS ? g : 0;
        uint32_t q_phase = 0;
        int count = 0, other = 0;  // uses of the group's score buffer (ONE: of both buffers)
        // O += P V of a tile: its buffer, the use of it, its slot of the ring
        auto pv = [&](int buf, int use, const Ring &at, int steps, bool first) {
            if (MODE != FEW) ok = wait_for(A, smem_addr(&ctl.p_half[buf]), (use - 1) & 1) && ok;
            ok = wait_for(A, smem_addr(&ctl.full[at.full()]), at.phase()) && ok;
            ok = __all_sync(FULL, ok);
            if (!ok) return;
            tmem_fence_after_sync();
            constexpr int HALF = C::BN / 32;  // steps of 16 keys in half a tile
            const uint64_t v = umma_desc(ring0 + at.slot * C::SLOT, C::BN * 128);
            const uint32_t o = tmem + C::O_COL + (MODE == ONE ? 0 : g * D), p = tmem + buf * C::S_COL;
            const uint64_t shared_p = umma_desc(sq - C::P + g * 8192);
            auto step = [&](int k) {
                if (MODE == FEW)
                    umma_ss(o, shared_p + (((k >> 2) * 4096 + (k & 3) * 32) >> 4), v + k * (2048 >> 4), umma_idesc(D, true), !(first && k == 0));
                else
                    umma_ts(o, p + 8 * k, v + k * (2048 >> 4), umma_idesc(D, true), !(first && k == 0));
            };
            if (MODE != FEW && elect_one()) {
#pragma unroll
                for (int k = 0; k < HALF; ++k)
                    if (k < steps) step(k);
            }
            __syncwarp();
            ok = wait_for(A, smem_addr(&ctl.p_full[buf]), (use - 1) & 1) && ok;
            ok = __all_sync(FULL, ok);
            if (!ok) return;
            tmem_fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int k = MODE == FEW ? 0 : HALF; k < 2 * HALF; ++k)
                    if (k < steps) step(k);
                umma_commit(smem_addr(&ctl.o_done[buf]));
                umma_commit(smem_addr(&ctl.empty[at.slot]));
            }
            __syncwarp();
        };
        // S = Q K^T of the first `keys` keys of a tile.  FEW: quarter by quarter,
        // the queries' first row 32 rows further down the tile each time, so that
        // each quarter's scores end in the lanes of another warp.  (The rows
        // before and behind the queries give scores that nobody looks at.)
        auto qk = [&](int buf, int slot, int keys) {
            tmem_fence_after_sync();
            if (elect_one()) {
                const uint64_t qdesc = umma_desc(sq + qi * C::CH * qblock);
                const uint64_t k = umma_desc(ring0 + slot * C::SLOT);
#pragma unroll 1
                for (int part = 0; part < (MODE == FEW ? keys : 1); part += 32) {
                    const uint32_t idesc = umma_idesc(MODE == FEW ? min(32, keys - part) : keys, false);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        umma_ss(tmem + buf * C::S_COL + part, qdesc + (((i >> 2) * qblock + (i & 3) * 32) >> 4) - part * 128 / 16,
                                k + (((i >> 2) * (C::BN * 128) + (i & 3) * 32 + part * 128) >> 4), idesc, i > 0);
                }
                umma_commit(smem_addr(&ctl.s_full[buf]));
                umma_commit(smem_addr(&ctl.empty[slot]));
            }
            __syncwarp();
        };
        while (ok && walk.next(A, pc)) {
            bool bad;
            const int n = PREFIX ? 0 : attn_nodes(A, pc.b, bad);
            if (MODE != ONE || warp == 1) {
                ok = wait_for(A, smem_addr(&ctl.q_full[qi]), q_phase) && ok;
                ok = __all_sync(FULL, ok);
            }
            // the tile whose weights' product is still to be issued
            bool have = false, old_first = false;
            int old_steps = 0;
            Ring old(A.slots);
            for (int t = pc.t0; t < pc.t1 && ok; ++t) {
                const Ring kr = r;
                r.step();
                const Ring vr = r;
                r.step();
                if (C::TURNS && ((t - pc.t0) & 1) != g) continue;
                int pos, valid;
                if (!PREFIX && t == pc.prefix)
                    valid = n > 0 ? n : 1;
                else
                    attn_tile(A, pc.len, t, pos, valid);
                const int buf = MODE == ONE ? (t - pc.t0) & 1 : g;
                int &uses = MODE == ONE && buf ? other : count;
                if (MODE == ONE && warp == 2) {  // the values' products
                    ++uses;
                    pv(buf, uses, vr, round16(valid) / 16, t == pc.t0);
                    continue;
                }
                // the buffer's last weights have to be used before new scores go there
                if (MODE == ONE) {
                    if (uses > 0) ok = wait_for(A, smem_addr(&ctl.o_done[buf]), (uses - 1) & 1) && ok;
                } else if (have) {
                    pv(buf, uses, old, old_steps, old_first);
                }
                ok = wait_for(A, smem_addr(&ctl.full[kr.full()]), kr.phase()) && ok;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                qk(buf, kr.slot, !PREFIX && t == pc.prefix ? round16(valid) : C::BN);
                ++uses;
                have = true;
                old_first = C::TURNS ? t - pc.t0 < 2 : t == pc.t0;
                old = vr;
                old_steps = round16(valid) / 16;
            }
            if (MODE == ONE && warp == 2) {
                ok = __all_sync(FULL, ok);
                continue;
            }
            // all scores of the piece are on their way: its queries may go
            if (elect_one()) {
                if (have)
                    umma_commit(smem_addr(&ctl.q_empty[qi]));
                else
                    mbar_arrive(smem_addr(&ctl.q_empty[qi]));
            }
            __syncwarp();
            if (MODE != ROWS && A.qbufs == 2) {
                q_phase ^= static_cast<uint32_t>(qi);
                qi ^= 1;
            } else {
                q_phase ^= 1u;
            }
            if (MODE != ONE && ok && have) pv(g, count, old, old_steps, old_first);
        }
    } else if (PREFIX && warp == 3) {
        // --------------------------------------------- page tables ----
        // (one piece of a prefix looks at its pages and speaks for all: the join
        // makes the rows of a flagged prefix NaN)
        if (blockIdx.x == 0) prefix_check_starts(A);
        for (int np = 0; ok && walk.next(A, pc); ++np) {
            if (np >= 4) {
                ok = wait_for(A, smem_addr(&ctl.done[np & 3]), ((np >> 2) - 1) & 1) && ok;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
            }
            if (np > 0 || A.fault_cta != static_cast<int>(blockIdx.x) + 1) mbar_arrive(smem_addr(&ctl.ready[np & 3]));
            if (flags_owner(pc, 0)) {
                const int flag = __reduce_or_sync(FULL, attn_check_pages(A, pc.b, pc.len, lane, LOADERS));
                if (lane == 0) put_flag(A, pc.b, flag);
            }
        }
    } else if (!PREFIX && warp == 3) {
        // --------------------------------------- new keys and values ----
        Ring r(A.slots);
        int grants = 0;
        for (int np = 0; ok && walk.next(A, pc); ++np) {
            const int b = pc.b, h = pc.h;
            bool bad_len, bad_nodes;
            attn_len(A, b, bad_len);
            const int n = attn_nodes(A, b, bad_nodes);
            if (np >= 4) {
                ok = wait_for(A, smem_addr(&ctl.done[np & 3]), ((np >> 2) - 1) & 1) && ok;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
            }
            int flag = (bad_len || bad_nodes) ? F_BAD_ID : 0;
            flag |= attn_masks(A.parents ? A.parents + static_cast<size_t>(b) * A.T : nullptr, n, ctl.mask[np & 3], ctl.above);
            mbar_arrive(smem_addr(&ctl.masks[np & 3]));
            for (int t = pc.t0; t < min(pc.t1, pc.prefix); ++t) {
                r.step();
                r.step();
            }
            uint64_t poison = 0;
            if (pc.t1 > pc.prefix) {
                ok = wait_for(A, smem_addr(&ctl.grant[grants & 7]), (grants >> 3) & 1) && ok;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                ++grants;
                for (int kv = 0; kv < 2; ++kv) {
                    poison |= load_new<D, C::BN>(A, ring + r.slot * C::SLOT, kv != 0, b, h, n);
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&ctl.full[r.full()]));
                    r.step();
                }
            }
            flag |= attn_check_pages(A, b, pc.len, lane, LOADERS);
            flag = __reduce_or_sync(FULL, flag);
            const uint32_t plo = __reduce_or_sync(FULL, static_cast<uint32_t>(poison));
            const uint32_t phi = __reduce_or_sync(FULL, static_cast<uint32_t>(poison >> 32));
            if (lane == 0) {
                ctl.flag[np & 3] = flag;
                ctl.poison[np & 3] = (static_cast<uint64_t>(phi) << 32) | plo;
            }
            if (np > 0 || A.fault_cta != static_cast<int>(blockIdx.x) + 1) mbar_arrive(smem_addr(&ctl.ready[np & 3]));
            if (A.flags && lane == 0 && flags_owner(pc, mtile)) put_flag(A, b, flag);
        }
    } else if (warp >= 4) {
        // --------------------------------------------------- softmax ----
        const int wg = (warp - 4) >> 2;                 // group of four warps
        const int wt = (tid - 128) & 127;               // this thread's row
        const int part = warp & 3;                      // its 32 TMEM lanes
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * part) << 16);
        const int quarter = wt >> 5;                     // FEW: of the keys of a tile
        const int lrow = MODE == FEW ? lane : wt + (MODE == ROWS ? 128 * wg : 0);  // row of the CTA's tile
        bool live = lrow < rows;
        bool busy = MODE == FEW ? quarter == 0 : lrow - lane < rows;  // the warp has rows of the accumulator
        const int rr = row0 + lrow, node = PREFIX ? 0 : node_of(A, rr);
        const uint32_t o_addr = lanes + C::O_COL + (MODE == ONE ? 0 : wg * D);
        Ring r(A.slots);
        int count0 = 0, count1 = 0;                     // uses of the group's score buffer (ONE: of both)
        uint32_t join_phase = 0, top_phase = 0;
        // The queries of piece `np`: copies into shared memory are started, by the
        // threads that arrive on q_full, once the scores of the piece before that
        // were in this buffer are done.
        const int depth = MODE == ROWS ? 1 : A.qbufs;
        auto copy_q = [&](const Piece &p, int np) {
            const int qi = MODE == ROWS ? wg : np & (depth - 1);
            if (np >= depth) ok = wait_for(A, smem_addr(&ctl.q_empty[qi]), (np / depth - 1) & 1) && ok;
            const int q0 = MODE == ROWS ? 128 * wg : 0;
            ok = __all_sync(FULL, ok);
            if (!ok) return;
            if constexpr (PREFIX)
                copy_prefix_queries<D>(A, p, q0, min(p.rows - q0, 128), sq + qi * C::CH * qblock, C::TURNS ? tid - 128 : wt,
                                       C::TURNS ? 256 : 128);
            else
                copy_queries<D>(static_cast<const bf16_t *>(A.q) + p.b * A.qs[0] + static_cast<int64_t>(p.h) * A.G * A.qs[2], A,
                                row0 + q0, min(rows - q0, 128), sq + qi * C::CH * qblock, C::TURNS ? tid - 128 : wt,
                                C::TURNS ? 256 : 128);
        };
        // (the turn before the first piece only loads its queries)
        Piece next = {};
        bool more = true;
        for (int np = -1; ok && more; ++np) {
            pc = next;
            more = walk.next(A, next);
            // with two buffers the next queries are copied during this piece
            const bool early = np < 0 || depth == 2;
            if (more && early) copy_q(next, np + 1);
            const int b = pc.b, h = pc.h;
            bool bad = false;
            const int n = PREFIX ? 0 : attn_nodes(A, b, bad);
            if (PREFIX) {
                live = lrow < rows_of(pc);
                busy = MODE == FEW ? quarter == 0 : lrow - lane < rows_of(pc);
            }
            float m = -INFINITY, l = 0.f;
            bool first = true;
            for (int t = pc.t0; t < pc.t1 && ok; ++t) {
                r.step();  // the keys' slot
                const Ring vr = r;
                r.step();
                if (C::TURNS && ((t - pc.t0) & 1) != wg) continue;
                const int buf = MODE == ONE ? (t - pc.t0) & 1 : wg;
                const int use = MODE == ONE && buf ? count1 : count0;
                const uint32_t s_addr = lanes + buf * C::S_COL;
                ok = wait_for(A, smem_addr(&ctl.s_full[buf]), use & 1) && ok;
                tmem_fence_after_sync();
                // the product before this one into the accumulator
                const uint32_t o_bar = smem_addr(&ctl.o_done[MODE == ONE ? buf ^ 1 : wg]);
                const uint32_t o_phase = ((MODE == ONE ? buf ? count0 : count1 : count0) - 1) & 1;
                int valid = C::BN;
                uint64_t lo = ~0ull, hi = ~0ull;
                const bool tree = !PREFIX && t == pc.prefix;
                if (tree) {
                    ok = wait_for(A, smem_addr(&ctl.masks[np & 3]), (np >> 2) & 1) && ok;
                    lo = live && node < n ? ctl.mask[np & 3][node] : 0ull;
                } else {
                    int pos;
                    attn_tile(A, pc.len, t, pos, valid);
                    if (valid < 64) lo = (1ull << valid) - 1ull;
                    hi = valid > 64 ? (valid < 128 ? (1ull << (valid - 64)) - 1ull : ~0ull) : 0ull;
                }
                bool half = true;  // the first half was announced
                if (MODE == FEW) {
                    softmax_quarter(A, s_addr + 32 * quarter, o_addr, D, A.scale_log2, quarter, 32 * quarter < (tree ? max(n, 1) : valid),
                                    static_cast<uint32_t>((quarter < 2 ? lo : hi) >> (32 * (quarter & 1))), live, first, m, l, o_bar,
                                    o_phase, use > 0, ctl.top[wg][top_phase], smem_addr(&ctl.tops[wg]), top_phase,
                                    smem + wg * 8192, A.qrows, ok);
                    top_phase ^= 1u;
                } else if (busy && !tree && valid == C::BN)
                    softmax_full<C::BN / 32>(A, s_addr, o_addr, D, A.scale_log2, first, m, l, o_bar, o_phase,
                                             smem_addr(&ctl.p_half[buf]), ok);
                else {
                    half = false;
                    if (busy)
                        softmax_part(A, s_addr, o_addr, D, A.scale_log2, tree ? max(n + 31, 32) >> 5 : (valid + 31) >> 5, lo, hi, first,
                                     m, l, o_bar, o_phase, ok);
                }
                if (!tree && (valid & 15)) {
                    // What lies behind the last key meets a weight of 0: it has
                    // to be a number.  (ROWS: each group sees to it for its own
                    // product; both write the same.)
                    const int end = round16(valid);
                    ok = wait_for(A, smem_addr(&ctl.full[vr.full()]), vr.phase()) && ok;
                    for (int i = wt; i < (end - valid) * (D / 8); i += 128) {
                        const int j = valid + i / (D / 8), u = i % (D / 8);
                        *reinterpret_cast<uint4 *>(ring + vr.slot * C::SLOT + (u >> 3) * (C::BN * 128) + sw128(j, u & 7)) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async();
                }
                first = false;
                tmem_fence_before_sync();
                if (MODE == FEW) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&ctl.p_full[buf]));
                } else {
                    if (!half) mbar_arrive(smem_addr(&ctl.p_half[buf]));
                    mbar_arrive(smem_addr(&ctl.p_full[buf]));
                }
                if (MODE == ONE && buf)
                    ++count1;
                else
                    ++count0;
                ok = __all_sync(FULL, ok);
            }
            if (!ok) break;
            if (more) {
                if (!early) copy_q(next, np + 1);
                cp_async_wait_all();
                fence_proxy_async();
                mbar_arrive(smem_addr(&ctl.q_full[MODE == ROWS ? wg : (np + 1) & (depth - 1)]));
                if (!ok) break;
            }
            if (np < 0) continue;
            // ------------------------------------------------ results ----
            ok = wait_for(A, smem_addr(&ctl.ready[np & 3]), (np >> 2) & 1) && ok;
            if (!first) {
                const int buf = MODE == ONE ? (pc.t1 - 1 - pc.t0) & 1 : wg;
                const int use = MODE == ONE && buf ? count1 : count0;
                ok = wait_for(A, smem_addr(&ctl.o_done[buf]), (use - 1) & 1) && ok;
            }
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            // KEYS: o = f0 o0 + f1 o1, each group for half of the columns
            float f0 = 1.f, f1 = 0.f;
            const bool two = C::TURNS && pc.t1 - pc.t0 > 1;  // the second group had tiles
            if (two || MODE == FEW) {
                ctl.m[wg][wt] = m;
                ctl.l[wg][wt] = l;
            }
            tmem_fence_before_sync();
            if (C::TURNS) {
                mbar_arrive(smem_addr(&ctl.stats));
                ok = wait_for(A, smem_addr(&ctl.stats), join_phase) && ok;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
            }
            tmem_fence_after_sync();
            // the sum over a group's weights (FEW: the four warps' sums)
            auto sum_of = [&](int of) {
                const float *x = ctl.l[of];
                return MODE == FEW ? (x[lane] + x[lane + 32]) + (x[lane + 64] + x[lane + 96]) : x[wt];
            };
            if (MODE == FEW && !two) l = sum_of(0);
            if (two) {
                const float m0 = ctl.m[0][wt], m1 = ctl.m[1][wt];
                m = fmaxf(m0, m1);
                const float ref = m == -INFINITY ? 0.f : m;
                f0 = ex2(m0 - ref);
                f1 = ex2(m1 - ref);
                l = f0 * sum_of(0) + f1 * sum_of(1);
            }
            uint64_t seen = 0;
            size_t at = 0;
            if constexpr (!PREFIX) {
                const int flag = ctl.flag[np & 3];
                if (pc.t1 == pc.prefix + 1 && live && node < n) seen = ctl.mask[np & 3][node] & ctl.poison[np & 3];
                if (flag) l = NAN;
                at = (static_cast<size_t>(b) * A.T + node) * A.Hq + h * A.G + rr - node * A.G;
            }
            const bool mine = live && (PREFIX || bad || node < n);
            // the finished row, or a part of it: of a whole unit by rows, else in a slot
            const bool whole = pc.whole(), done = !PREFIX && whole && !A.row_o;
            float *slot = A.part + attn_slot(A, group, mtile, pc.first) * attn_slot_floats(BM, D);
            const size_t place = unit_row(A, pc) + row0 + lrow;
            float *part_o = whole ? A.row_o + place * D : slot + 2 * BM + static_cast<size_t>(lrow) * D;
            const float inv = 1.f / l;
            // columns of this group (a piece of one tile: the first group had it, and has all)
            const int c0 = two ? wg * (D / 2) : 0, c1 = two ? c0 + D / 2 : C::TURNS && wg == 1 ? 0 : D;
            if (busy) {
#pragma unroll 1
                for (int c = c0; c < c1; c += 32) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_ld32((two ? lanes + C::O_COL : o_addr) + c, o);
                    if (two) {
                        uint32_t o1[32];
                        tmem_ld32(lanes + C::O_COL + D + c, o1);
                        tmem_wait_ld32(o);
                        tmem_wait_ld32(o1);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(fmaf(f1, __uint_as_float(o1[i]), f0 * __uint_as_float(o[i])));
                    } else {
                        tmem_wait_ld32(o);
                    }
                    if (!mine) continue;
                    if (done) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<bf16_t *>(A.out) + at * D + c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(o[8 * i + e]) * inv;
                            dst[i] = make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
                        }
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(part_o + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
                if (mine && seen)
                    add_far_values(done ? nullptr : part_o,
                                   static_cast<bf16_t *>(A.out) + at * D, static_cast<const bf16_t *>(A.v_new) + b * A.vs[0] + h * A.vs[2],
                                   A.vs[1], seen, c0, c1);
                if (mine && c0 == 0 && c1 > 0) {
                    if (!done) {
                        *(whole ? A.row_m + place : slot + lrow) = m;
                        *(whole ? A.row_l + place : slot + BM + lrow) = l;
                    } else if (A.lse) {
                        A.lse[at] = (m + log2f(l)) * LN2;
                    }
                }
            }
            tmem_fence_before_sync();
            mbar_arrive(smem_addr(&ctl.done[np & 3]));
            if (C::TURNS) {  // the next piece's products may write the accumulators
                mbar_arrive(smem_addr(&ctl.joined));
                ok = wait_for(A, smem_addr(&ctl.joined), join_phase) && ok;
                join_phase ^= 1u;
                ok = __all_sync(FULL, ok);
            }
        }
    }
    // ---------------------------------------------------------- the end ----
    __syncwarp();
    if (!ok) ctl.dead = 1;
    __syncthreads();
    if (ctl.dead) {
        // a wait gave up: let copies and products in flight end before the
        // shared and tensor memory goes
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 10000000ull) __nanosleep(1000);
        give_up(A, ctl.begin, group, mtile, row0, rows, tid, NT);
    }
    if (mtile == 0 && tid == 0) attn_report(A, group, ctl.W, ctl.begin);
    if (!PREFIX && A.overlap && blockIdx.x == 0) pdl_wait();  // the join waits for this kernel, and so for the one before
    tmem_fence_after_sync();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <bool PREFIX, typename F>
auto pick(int D, int mode, F f) {
    if (D == 256) return f(Cfg<256, ONE>{}, attn_umma_impl<256, ONE, PREFIX>);
    if (D == 128)
        return mode == ROWS   ? f(Cfg<128, ROWS>{}, attn_umma_impl<128, ROWS, PREFIX>)
               : mode == KEYS ? f(Cfg<128, KEYS>{}, attn_umma_impl<128, KEYS, PREFIX>)
                              : f(Cfg<128, FEW>{}, attn_umma_impl<128, FEW, PREFIX>);
    return mode == ROWS   ? f(Cfg<64, ROWS>{}, attn_umma_impl<64, ROWS, PREFIX>)
           : mode == KEYS ? f(Cfg<64, KEYS>{}, attn_umma_impl<64, KEYS, PREFIX>)
                          : f(Cfg<64, FEW>{}, attn_umma_impl<64, FEW, PREFIX>);
}

// Two buffers of queries where they fit beside at least six slots of the ring
// (or as many as go in with one buffer).
template <bool PREFIX>
UmmaPlan umma_plan(int D, int rows, long long most) {
    using Ctl = Control<typename std::conditional<PREFIX, PrefixWalk, AttnWalk>::type>;
    UmmaPlan p;
    const int mode = D == 256 ? ONE : rows > 128 ? ROWS : rows > 32 ? KEYS : FEW;
    p.bm = mode == ROWS ? 256 : 128;
    p.tile_rows = mode == FEW ? 32 : p.bm;
    const int tile = mode == FEW && PREFIX ? 32 : 128;
    p.qrows = most >= tile ? tile : (static_cast<int>(most) + 7) / 8 * 8;
    uint32_t q = static_cast<uint32_t>(p.qrows) * D * 2 * (mode == ROWS ? 2 : 1);
    const uint32_t slot = static_cast<uint32_t>(attn_umma_bn(D)) * D * 2;
    const uint32_t p_bytes = mode == FEW ? Cfg<64, FEW>::P : 0;
    auto fit = [&](uint32_t queries) {
        const int n = static_cast<int>((UMMA_SMEM - sizeof(Ctl) - p_bytes - queries) / slot);
        return n < MAX_SLOTS ? n : MAX_SLOTS;
    };
    p.slots = fit(q);
    p.qbufs = 1;
    if (mode != ROWS && (fit(2 * q) >= 6 || fit(2 * q) == p.slots)) {
        p.qbufs = 2;
        p.slots = fit(2 * q);
        q *= 2;
    }
    // the product reads 128 rows of every block of queries
    p.smem = p_bytes + q + p.slots * slot + static_cast<uint32_t>(sizeof(Ctl));
    p.bn = attn_umma_bn(D);
    p.cost = mode == ROWS ? 230 : mode == ONE ? 170 : mode == KEYS ? 150 : 110;
    p.func = pick<PREFIX>(D, mode, [](auto, auto f) { return reinterpret_cast<const void *>(f); });
    p.threads = pick<PREFIX>(D, mode, [](auto c, auto) { return decltype(c)::NT; });
    return p;
}

}  // namespace
}  // namespace mtp
