// tree_attention_umma.cu -- tree attention on the tensor cores: bfloat16
// storage, head sizes 64, 128 and 256, caches that tiled copies can address
// (tree_attention.cuh has the split of the work over CTAs).
//
// One CTA per SM works through its list of key tiles.  A tile is BN keys of
// one (sequence, key head); the CTA's query rows (nodes x query heads of the
// group) stay in shared memory for the piece.
//   warp 0      copies key and value tiles page by page into a ring of slots
//               (cp.async.bulk.tensor, 128-byte swizzle)
//   warp 1      one lane issues S = Q K^T into a score buffer of TMEM and,
//               when the weights are back, O += P V with P read from TMEM
//   warps 2, 3  load the queries, the new keys and values and the ancestor
//               masks of a piece, and check its page table
//   warps 4 ..  softmax: a thread has one row of a score tile, so the running
//               maximum and sum need no exchange.  Weights go back to TMEM as
//               bfloat16 over the scores they came from.
// The softmax of a tile takes longer than its copy or its products, so two
// score tiles are worked on at a time by two groups of four warps, each with
// its own accumulator in TMEM:
//   ROWS   more than 128 query rows: one group has rows 0 - 127, the other
//          128 - 255, and a key tile is copied once for both
//   KEYS   up to 128 rows: the groups take turns at the key tiles; at the end
//          of a piece their maxima, sums and outputs are joined
//   ONE    heads of 256: TMEM holds one accumulator, so one group works, with
//          two score buffers (the products of tile j + 1 run under the softmax
//          of tile j)
// The output accumulator is rescaled only when a row's maximum has risen by
// more than 2^8 since the last time: until then the weights are taken
// relative to the older maximum, which changes nothing but their scale.
//
// Rounding: scores, statistics and outputs are float32; the weights are
// rounded to bfloat16 because the tensor core takes both operands of P V in
// one type, and the values are bfloat16.  Their sum is taken before rounding.
#include <cuda.h>

#include "tree_attention.cuh"
#include "umma.cuh"

namespace mtp {
namespace {

constexpr int LOADERS = 64;
constexpr float RESCALE = 8.f;  // rescale when the maximum rose by this many powers of two
constexpr int MAX_SLOTS = 14;
enum Mode { ONE = 0, KEYS = 1, ROWS = 2 };

template <int D, int MODE>
struct Cfg {
    static constexpr int NT = MODE == ONE ? 256 : 384;
    static constexpr int BN = D == 256 ? 64 : 128;
    static constexpr int CH = D / 64;                      // 64-element blocks of a row
    static constexpr uint32_t SLOT = BN * D * 2;           // a key or value tile
    static constexpr uint32_t S_COL = 128;                 // score buffers at columns 0 and 128
    static constexpr uint32_t O_COL = 256;                 // accumulators at 256 and 256 + D
};

// What the loaders say about a piece lies in a ring of four: the products are
// at most two tiles, and so two pieces, ahead of the softmax, and the loaders
// one piece ahead of the products.
struct Control {
    uint64_t full[MAX_SLOTS], empty[MAX_SLOTS], s_full[2], p_full[2], o_done[2], q_full, q_empty, tree;
    uint64_t grant[8];            // two slots of the ring are the loaders' to fill (at most slots / 2 at a time)
    uint64_t masks[4], ready[4];  // a piece's masks are there; all that the loaders found out is
    uint64_t stats, joined;       // KEYS: both groups' statistics are there; both have read the accumulators
    uint64_t mask[4][MAX_NODES];
    uint64_t poison[4][2];
    int flag[4][2];
    long long scan[12];
    AttnWalk begin;
    float m[2][128], l[2][128];   // KEYS: the groups' statistics
    uint32_t tmem;
    int dead;
};

// A ring position: slot index and the parity of its current use.
struct Ring {
    int slots;
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ explicit Ring(int n) : slots(n) {}
    __device__ __forceinline__ void step() {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ int round16(int n) { return (n + 15) & ~15; }

// The largest of three (NaN only if all are).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// -inf in the columns of block c that the row does not see.
template <bool TREE>
__device__ __forceinline__ void mask_block(uint32_t (&s)[32], int c, int valid, uint64_t see) {
    if (TREE) {
        const uint32_t w = static_cast<uint32_t>(see >> (32 * c));
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!((w >> i) & 1u)) s[i] = 0xff800000u;
    } else if (valid < 32 * (c + 1)) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (32 * c + i >= valid) s[i] = 0xff800000u;
    }
}

// Softmax of one score tile: CH blocks of 32 columns, of which a row sees the
// first `valid` or, of a tree tile, those in `see`.  The scores are read from
// TMEM twice, once for the maximum and once for the weights, the next block
// while one is worked on: a row's 128 scores never lie in registers at once.
template <int CH, bool TREE>
__device__ __forceinline__ void softmax_tile(uint32_t s_addr, uint32_t o_addr, int ocols, float scale, int valid, uint64_t see,
                                             bool first, float &m, float &l, uint32_t o_bar, uint32_t o_phase, bool &ok) {
    uint32_t s[2][32];
    float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    __syncwarp();  // TMEM accesses are warp-wide, and the lanes may have left a wait one by one
    tmem_ld32(s_addr, s[0]);
    tmem_wait_ld32(s[0]);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (c + 1 < CH) tmem_ld32(s_addr + 32 * (c + 1), s[(c + 1) & 1]);
        uint32_t(&x)[32] = s[c & 1];
        mask_block<TREE>(x, c, valid, see);
#pragma unroll
        for (int i = 0; i < 32; i += 2) t[(i >> 1) & 3] = max3(t[(i >> 1) & 3], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
        if (c + 1 < CH) tmem_wait_ld32(s[(c + 1) & 1]);
    }
    const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * scale;
    if (first) {
        m = top;
        l = 0.f;
    } else {
        const bool up = top > m + RESCALE;
        if (__any_sync(FULL, up)) {
            ok = mbar_wait_bounded(o_bar, o_phase) && ok;  // the products before this tile
            __syncwarp();
            tmem_fence_after_sync();
            const float f = up ? ex2(m - top) : 1.f;
            if (up) m = top;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < ocols; c += 32) {
                __syncwarp();
                tmem_ld32(o_addr + c, s[0]);
                tmem_wait_ld32(s[0]);
#pragma unroll
                for (int i = 0; i < 32; ++i) s[0][i] = __float_as_uint(__uint_as_float(s[0][i]) * f);
                tmem_st32(o_addr + c, s[0]);
                tmem_wait_st();
            }
        }
    }
    const uint64_t K2 = f2pack(scale, scale), N2 = m == -INFINITY ? f2pack(0.f, 0.f) : f2pack(-m, -m);
    uint64_t acc[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
    __syncwarp();
    tmem_ld32(s_addr, s[0]);
    tmem_wait_ld32(s[0]);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if (c + 1 < CH) tmem_ld32(s_addr + 32 * (c + 1), s[(c + 1) & 1]);
        uint32_t(&x)[32] = s[c & 1];
        mask_block<TREE>(x, c, valid, see);
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            float a, b;
            f2unpack(f2fma(f2pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), K2, N2), a, b);
            a = ex2(a);
            b = ex2(b);
            acc[(i >> 1) & 1] = f2add(acc[(i >> 1) & 1], f2pack(a, b));
            p[i / 2] = bf16x2(a, b);
        }
        // block c's weights lie over scores of blocks <= c
        tmem_st16(s_addr + 16 * c, p);
        if (c + 1 < CH) tmem_wait_ld32(s[(c + 1) & 1]);
    }
    float a0, a1, b0, b1;
    f2unpack(acc[0], a0, a1);
    f2unpack(acc[1], b0, b1);
    l += (a0 + a1) + (b0 + b1);
    tmem_wait_st();
}

template <int D, int MODE>
__global__ void __launch_bounds__(Cfg<D, MODE>::NT, 1)
    attn_umma_impl(const __grid_constant__ TreeAttnArgs A, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
    using C = Cfg<D, MODE>;
    constexpr int NT = C::NT, BM = MODE == ROWS ? 256 : 128;
    // queries (blocks of 64 elements x qrows rows; in ROWS mode twice), ring, control
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t qblock = A.qrows * 128, qbytes = qblock * C::CH * (MODE == ROWS ? 2 : 1);
    Control &ctl = *reinterpret_cast<Control *>(smem + qbytes + C::SLOT * A.slots);
    unsigned char *ring = smem + qbytes;
    const uint32_t sq = smem_addr(smem), ring0 = sq + qbytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = blockIdx.x / A.mtiles, mtile = blockIdx.x - group * A.mtiles;
    const int row0 = mtile * BM, rows = min(BM, A.rows - row0);

    AttnWalk walk;
    walk.start<NT>(A, group, ctl.scan);
    if (walk.at >= walk.hi) {  // no tiles for this group
        if (mtile == 0 && tid == 0) A.desc[static_cast<size_t>(group) * ATTN_DESC + 2] = 0;
        return;
    }
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < A.slots; ++i) {
            mbar_init(smem_addr(&ctl.full[i]), 1);
            mbar_init(smem_addr(&ctl.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl.s_full[i]), 1);
            mbar_init(smem_addr(&ctl.p_full[i]), 128);
            mbar_init(smem_addr(&ctl.o_done[i]), 1);
        }
        for (int i = 0; i < 8; ++i) mbar_init(smem_addr(&ctl.grant[i]), 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_addr(&ctl.masks[i]), LOADERS);
            mbar_init(smem_addr(&ctl.ready[i]), LOADERS);
        }
        mbar_init(smem_addr(&ctl.q_full), LOADERS);
        mbar_init(smem_addr(&ctl.q_empty), 1);
        mbar_init(smem_addr(&ctl.tree), LOADERS);
        mbar_init(smem_addr(&ctl.stats), 256);
        mbar_init(smem_addr(&ctl.joined), 256);
        ctl.dead = 0;
        fence_mbar_init();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    if (warp == 1) tmem_alloc(&ctl.tmem, TMEM_COLS);
    // Rows of the query tile that no query fills.  (The product reads 128 rows
    // of each block whatever qrows is: what lies behind them gives rows that
    // nobody looks at.)
    for (int i = tid; i < (A.qrows * (MODE == ROWS ? 2 : 1) - rows) * (D / 8); i += NT) {
        const int r = rows + i / (D / 8), u = i % (D / 8);
        *reinterpret_cast<uint4 *>(smem + ((r >> 7) * C::CH + (u >> 3)) * qblock + sw128(r & 127, u & 7)) =
            make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async();
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tmem = ctl.tmem;
    if (tid == 0) ctl.begin = walk;  // read at the end, by the same thread
    bool ok = (sq & 1023u) == 0u;    // the swizzle counts on it
    AttnPiece pc;

    if (warp == 0) {
        // ---------------------------------------------------- copies ----
        Ring r(A.slots);
        int grants = 0;
        uint32_t lap = 0;  // the first use of every slot needs no wait
        const int boxrows = A.per_page ? C::BN : A.page_size;
        while (ok && walk.next(A, pc)) {
            for (int t = pc.t0; t < pc.t1 && ok; ++t) {
                if (t == pc.prefix) {  // the loaders fill these two slots once they are free
                    for (int i = 0; i < 2; ++i) {
                        if (lap) ok = mbar_wait_bounded(smem_addr(&ctl.empty[r.slot]), r.phase ^ 1u) && ok;
                        r.step();
                        if (r.slot == 0) lap = 1;
                    }
                    ok = __all_sync(FULL, ok);
                    if (lane == 0 && ok) mbar_arrive(smem_addr(&ctl.grant[grants & 7]));
                    ++grants;
                    continue;
                }
                int pos, valid;
                attn_tile(A, pc.len, t, pos, valid);
                const int page0 = pos / A.page_size, off = pos - page0 * A.page_size;
                const int pages = A.per_page ? 1 : (valid + A.page_size - 1) / A.page_size;
                const int mine = lane < pages ? attn_page(A, pc.b, page0 + lane) : 0;  // at most BN / 8 pages
                for (int kv = 0; kv < 2; ++kv) {
                    if (lap) ok = mbar_wait_bounded(smem_addr(&ctl.empty[r.slot]), r.phase ^ 1u) && ok;
                    ok = __all_sync(FULL, ok);
                    if (!ok) break;
                    const uint32_t full = smem_addr(&ctl.full[r.slot]), dst = ring0 + r.slot * C::SLOT;
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
                    if (r.slot == 0) lap = 1;
                }
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------------- products ----
        Ring r(A.slots);
        uint32_t q_phase = 0;
        int count[2] = {0, 0};  // score tiles of each group of warps (ONE: of each buffer)
        int n_tiles = 0;
        // the weights' product that is still to be issued, for each of the two
        bool have[2] = {false, false}, first[2] = {}, release[2] = {};
        int steps[2] = {}, slot[2] = {};
        uint32_t phase[2] = {};
        auto pv = [&](int s) {
            ok = mbar_wait_bounded(smem_addr(&ctl.p_full[s]), (count[s] - 1) & 1) && ok;
            ok = mbar_wait_bounded(smem_addr(&ctl.full[slot[s]]), phase[s]) && ok;
            ok = __all_sync(FULL, ok);
            have[s] = false;
            if (!ok) return;
            tmem_fence_after_sync();
            if (elect_one()) {
                const uint32_t v = ring0 + slot[s] * C::SLOT, o = tmem + C::O_COL + (MODE == ONE ? 0 : s * D);
                for (int k = 0; k < steps[s]; ++k)
                    umma_ts(o, tmem + s * C::S_COL + 8 * k, umma_desc(v + k * 2048, C::BN * 128), umma_idesc(D, true),
                            !(first[s] && k == 0));
                if (release[s]) umma_commit(smem_addr(&ctl.empty[slot[s]]));
                umma_commit(smem_addr(&ctl.o_done[s]));
            }
            __syncwarp();
        };
        while (ok && walk.next(A, pc)) {
            bool bad;
            const int n = attn_nodes(A, pc.b, bad);
            ok = mbar_wait_bounded(smem_addr(&ctl.q_full), q_phase) && ok;
            q_phase ^= 1u;
            for (int t = pc.t0; t < pc.t1 && ok; ++t) {
                int pos, valid;
                if (t == pc.prefix)
                    valid = n > 0 ? n : 1;
                else
                    attn_tile(A, pc.len, t, pos, valid);
                const int k_slot = r.slot;
                const uint32_t k_phase = r.phase;
                r.step();
#pragma unroll
                for (int half = 0; half < (MODE == ROWS ? 2 : 1); ++half) {
                    const int s = MODE == ROWS ? half : MODE == KEYS ? (t - pc.t0) & 1 : n_tiles & 1;
                    // the group's last weights first: they lie where the scores go.
                    // (ONE: the other buffer is free; its last product follows the
                    // scores unless the keys are not there yet.)
                    if (MODE != ONE && have[s]) pv(s);
                    if (MODE == ONE && have[s ^ 1] &&
                        !__all_sync(FULL, mbar_test_wait(smem_addr(&ctl.full[k_slot]), k_phase)))
                        pv(s ^ 1);
                    ok = mbar_wait_bounded(smem_addr(&ctl.full[k_slot]), k_phase) && ok;
                    ok = __all_sync(FULL, ok);
                    if (!ok) break;
                    tmem_fence_after_sync();
                    if (elect_one()) {
                        const uint32_t k = ring0 + k_slot * C::SLOT, q = sq + (MODE == ROWS ? s * C::CH * qblock : 0);
                        const uint32_t idesc = umma_idesc(t == pc.prefix ? round16(valid) : C::BN, false);
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
                            umma_ss(tmem + s * C::S_COL, umma_desc(q + (i >> 2) * qblock + (i & 3) * 32),
                                    umma_desc(k + (i >> 2) * (C::BN * 128) + (i & 3) * 32), idesc, i > 0);
                        if (MODE != ROWS || s == 1) {
                            umma_commit(smem_addr(&ctl.empty[k_slot]));
                            if (t + 1 == pc.t1) umma_commit(smem_addr(&ctl.q_empty));
                        }
                        umma_commit(smem_addr(&ctl.s_full[s]));
                    }
                    __syncwarp();
                    if (MODE == ONE && have[s ^ 1]) pv(s ^ 1);
                    have[s] = true;
                    first[s] = MODE == KEYS ? t - pc.t0 < 2 : t == pc.t0;
                    release[s] = MODE != ROWS || s == 1;
                    steps[s] = round16(valid) / 16;
                    slot[s] = r.slot;
                    phase[s] = r.phase;
                    ++count[s];
                }
                r.step();
                ++n_tiles;
            }
            // the piece's last weights, the older ones first
            const int older = MODE == KEYS ? (pc.t1 - pc.t0) & 1 : 0;
            if (ok && have[older]) pv(older);
            if (ok && have[older ^ 1]) pv(older ^ 1);
        }
    } else if (warp < 4) {
        // ------------------------------------- queries and new tokens ----
        const int lt = tid - 64;
        Ring r(A.slots);
        uint32_t q_phase = 0, tree_phase = 0;
        int grants = 0;
        const bf16_t *gq = static_cast<const bf16_t *>(A.q);
        const int vecs = rows * (D / 8);
        for (int np = 0; ok && walk.next(A, pc); ++np) {
            const int b = pc.b, h = pc.h;
            bool bad_len, bad_nodes;
            attn_len(A, b, bad_len);
            const int n = attn_nodes(A, b, bad_nodes);
            auto q_vec = [&](int i) {
                const int rr = row0 + i / (D / 8), u = i % (D / 8), t = rr / A.G, g = rr - t * A.G;
                return __ldg(reinterpret_cast<const uint4 *>(gq + b * A.qs[0] + t * A.qs[1] +
                                                             (static_cast<int64_t>(h) * A.G + g) * A.qs[2]) +
                             u);
            };
            auto q_put = [&](int i, const uint4 &x) {
                const int rr = i / (D / 8), u = i % (D / 8);
                *reinterpret_cast<uint4 *>(smem + ((rr >> 7) * C::CH + (u >> 3)) * qblock + sw128(rr & 127, u & 7)) = x;
            };
            constexpr int AHEAD = 8;  // vectors of a thread that are under way while the last piece ends
            uint4 x[AHEAD];
#pragma unroll
            for (int e = 0; e < AHEAD; ++e)
                if (lt + e * LOADERS < vecs) x[e] = q_vec(lt + e * LOADERS);
            if (np > 0) {
                ok = mbar_wait_bounded(smem_addr(&ctl.q_empty), q_phase) && ok;
                q_phase ^= 1u;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
            }
#pragma unroll
            for (int e = 0; e < AHEAD; ++e)
                if (lt + e * LOADERS < vecs) q_put(lt + e * LOADERS, x[e]);
#pragma unroll 4
            for (int i = lt + AHEAD * LOADERS; i < vecs; i += LOADERS) q_put(i, q_vec(i));
            int flag = (bad_len || bad_nodes) ? F_BAD_ID : 0;
            if (lt < n) {
                bool bad_up = false;
                ctl.mask[np & 3][lt] = attn_mask(A.parents ? A.parents + static_cast<size_t>(b) * A.T : nullptr, lt, bad_up);
                if (bad_up) flag |= F_BAD_ID;
            }
            fence_proxy_async();
            mbar_arrive(smem_addr(&ctl.q_full));
            mbar_arrive(smem_addr(&ctl.masks[np & 3]));
            uint64_t poison = 0;
            for (int t = pc.t0; t < pc.t1; ++t) {
                for (int kv = 0; kv < 2; ++kv) {
                    if (t == pc.prefix) {
                        if (kv == 0) {
                            ok = mbar_wait_bounded(smem_addr(&ctl.grant[grants & 7]), (grants >> 3) & 1) && ok;
                            ++grants;
                        }
                        unsigned char *dst = ring + r.slot * C::SLOT;
                        const bf16_t *src = static_cast<const bf16_t *>(kv ? A.v_new : A.k_new);
                        const int64_t *st = kv ? A.vs : A.ks;
                        // of the keys no more than the sequence's nodes is
                        // looked at; the values behind them are zero, and so
                        // is one that is not finite (its rows get it later)
                        const int fill = kv ? round16(n > 0 ? n : 1) : n;
                        if (ok) {
#pragma unroll 4
                            for (int i = lt; i < fill * (D / 8); i += LOADERS) {
                                const int j = i / (D / 8), u = i % (D / 8);
                                uint4 y = make_uint4(0u, 0u, 0u, 0u);
                                if (j < n) y = __ldg(reinterpret_cast<const uint4 *>(src + b * st[0] + j * st[1] + h * st[2]) + u);
                                if (kv) {
                                    uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const bool lo = (w[e] & 0x7f80u) == 0x7f80u, hi = (w[e] & 0x7f800000u) == 0x7f800000u;
                                        if (lo || hi) poison |= 1ull << j;
                                        w[e] = (lo ? 0u : w[e] & 0xffffu) | (hi ? 0u : w[e] & 0xffff0000u);
                                    }
                                    y = make_uint4(w[0], w[1], w[2], w[3]);
                                }
                                *reinterpret_cast<uint4 *>(dst + (u >> 3) * (C::BN * 128) + sw128(j, u & 7)) = y;
                            }
                        }
                        fence_proxy_async();
                        // everyone waits: a thread that went on would arrive
                        // a second time in the same phase
                        mbar_arrive(smem_addr(&ctl.tree));
                        ok = mbar_wait_bounded(smem_addr(&ctl.tree), tree_phase) && ok;
                        tree_phase ^= 1u;
                        if (lt == 0) mbar_arrive(smem_addr(&ctl.full[r.slot]));
                    }
                    r.step();
                }
            }
            flag |= attn_check_pages(A, b, pc.len, lt, LOADERS);
            flag = __reduce_or_sync(FULL, flag);
            if (lane == 0) ctl.flag[np & 3][warp - 2] = flag;
            const uint32_t plo = __reduce_or_sync(FULL, static_cast<uint32_t>(poison));
            const uint32_t phi = __reduce_or_sync(FULL, static_cast<uint32_t>(poison >> 32));
            if (lane == 0) ctl.poison[np & 3][warp - 2] = (static_cast<uint64_t>(phi) << 32) | plo;
            mbar_arrive(smem_addr(&ctl.ready[np & 3]));
            ok = __all_sync(FULL, ok);
        }
    } else {
        // --------------------------------------------------- softmax ----
        const int wg = (warp - 4) >> 2;                 // group of four warps
        const int wt = (tid - 128) & 127;               // this thread's row
        const int part = warp & 3;                      // its 32 TMEM lanes
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * part) << 16);
        const int lrow = wt + (MODE == ROWS ? 128 * wg : 0);  // row of the CTA's tile
        const bool live = lrow < rows;
        const bool busy = lrow - lane < rows;           // the warp has rows
        const int rr = row0 + lrow, node = rr / A.G;
        const uint32_t o_addr = lanes + C::O_COL + (MODE == ONE ? 0 : wg * D);
        Ring r(A.slots);
        int count = 0;                                  // score tiles of this group
        uint32_t join_phase = 0;
        for (int np = 0; ok && walk.next(A, pc); ++np) {
            const int b = pc.b, h = pc.h;
            bool bad;
            const int n = attn_nodes(A, b, bad);
            float m = -INFINITY, l = 0.f;
            bool first = true;
            for (int t = pc.t0; t < pc.t1 && ok; ++t) {
                r.step();  // the keys' slot
                const int v_slot = r.slot;
                const uint32_t v_phase = r.phase;
                r.step();
                if (MODE == KEYS && ((t - pc.t0) & 1) != wg) continue;
                const int buf = MODE == ONE ? count & 1 : wg;
                const uint32_t phase = MODE == ONE ? (count >> 1) & 1 : count & 1;
                const uint32_t s_addr = lanes + buf * C::S_COL;
                ok = mbar_wait_bounded(smem_addr(&ctl.s_full[buf]), phase) && ok;
                tmem_fence_after_sync();
                // the product before this one into the accumulator
                const uint32_t o_bar = smem_addr(&ctl.o_done[MODE == ONE ? buf ^ 1 : wg]);
                const uint32_t o_phase = MODE == ONE ? ((count - 1) >> 1) & 1 : (count - 1) & 1;
                if (t == pc.prefix) {
                    ok = mbar_wait_bounded(smem_addr(&ctl.masks[np & 3]), (np >> 2) & 1) && ok;
                    const uint64_t see = live && node < n ? ctl.mask[np & 3][node] : 0ull;
                    if (busy) {
                        if (n <= 32)
                            softmax_tile<1, true>(s_addr, o_addr, D, A.scale_log2, 0, see, first, m, l, o_bar, o_phase, ok);
                        else
                            softmax_tile<2, true>(s_addr, o_addr, D, A.scale_log2, 0, see, first, m, l, o_bar, o_phase, ok);
                    }
                } else {
                    int pos, valid;
                    attn_tile(A, pc.len, t, pos, valid);
                    if (busy)
                        softmax_tile<C::BN / 32, false>(s_addr, o_addr, D, A.scale_log2, valid, 0ull, first, m, l, o_bar, o_phase,
                                                        ok);
                    const int end = round16(valid);
                    // What lies behind the last key meets a weight of 0: it has
                    // to be a number.  (ROWS: the first group's product is the
                    // first to read it, and the first group writes it.)
                    if (valid < end && (MODE != ROWS || wg == 0)) {
                        ok = mbar_wait_bounded(smem_addr(&ctl.full[v_slot]), v_phase) && ok;
                        for (int i = wt; i < (end - valid) * (D / 8); i += 128) {
                            const int j = valid + i / (D / 8), u = i % (D / 8);
                            *reinterpret_cast<uint4 *>(ring + v_slot * C::SLOT + (u >> 3) * (C::BN * 128) + sw128(j, u & 7)) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async();
                    }
                }
                first = false;
                tmem_fence_before_sync();
                mbar_arrive(smem_addr(&ctl.p_full[buf]));
                ++count;
                ok = __all_sync(FULL, ok);
            }
            // ------------------------------------------------ results ----
            ok = mbar_wait_bounded(smem_addr(&ctl.ready[np & 3]), (np >> 2) & 1) && ok;
            if (!first) {
                const int buf = MODE == ONE ? (count - 1) & 1 : wg;
                ok = mbar_wait_bounded(smem_addr(&ctl.o_done[buf]), MODE == ONE ? ((count - 1) >> 1) & 1 : (count - 1) & 1) && ok;
            }
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            // KEYS: o = f0 o0 + f1 o1, each group for half of the columns
            float f0 = 1.f, f1 = 0.f;
            const bool two = MODE == KEYS && pc.t1 - pc.t0 > 1;  // the second group had tiles
            if (two) {
                ctl.m[wg][wt] = m;
                ctl.l[wg][wt] = l;
            }
            tmem_fence_before_sync();
            if (MODE == KEYS) {
                mbar_arrive(smem_addr(&ctl.stats));
                ok = mbar_wait_bounded(smem_addr(&ctl.stats), join_phase) && ok;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
            }
            tmem_fence_after_sync();
            if (two) {
                const float m0 = ctl.m[0][wt], m1 = ctl.m[1][wt];
                m = fmaxf(m0, m1);
                const float ref = m == -INFINITY ? 0.f : m;
                f0 = ex2(m0 - ref);
                f1 = ex2(m1 - ref);
                l = f0 * ctl.l[0][wt] + f1 * ctl.l[1][wt];
            }
            const int flag = ctl.flag[np & 3][0] | ctl.flag[np & 3][1];
            if (A.flags && tid == 128 && h == 0 && mtile == 0) A.flags[b] = flag;
            const uint64_t seen = pc.t1 == pc.prefix + 1 && live && node < n
                                      ? ctl.mask[np & 3][node] & (ctl.poison[np & 3][0] | ctl.poison[np & 3][1])
                                      : 0ull;
            if (flag) l = NAN;
            const bool whole = pc.whole();
            const bool mine = live && (bad || node < n);
            const int hq = h * A.G + rr - node * A.G;
            const size_t at = (static_cast<size_t>(b) * A.T + node) * A.Hq + hq;
            float *slot = A.part + attn_slot(A, group, mtile, pc.first) * attn_slot_floats(BM, D);
            const float inv = 1.f / l;
            // columns of this group (a piece of one tile: the first group had it, and has all)
            const int c0 = two ? wg * (D / 2) : 0, c1 = two ? c0 + D / 2 : MODE == KEYS && wg == 1 ? 0 : D;
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
                    if (seen) {  // values that are not finite, of nodes that this row sees
                        const bf16_t *v = static_cast<const bf16_t *>(A.v_new) + b * A.vs[0] + h * A.vs[2];
                        for (int j = 0; j < n; ++j) {
                            if (!((seen >> j) & 1ull)) continue;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float x = __uint_as_float(static_cast<uint32_t>(v[j * A.vs[1] + c + i].bits) << 16);
                                if (!(fabsf(x) < INFINITY)) o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
                            }
                        }
                    }
                    if (!mine) continue;
                    if (whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<bf16_t *>(A.out) + at * D + c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(o[8 * i + e]) * inv;
                            dst[i] = make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
                        }
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(slot + 2 * BM + static_cast<size_t>(lrow) * D + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
                if (mine && c0 == 0 && c1 > 0) {
                    if (!whole) {
                        slot[lrow] = m;
                        slot[BM + lrow] = l;
                    } else if (A.lse) {
                        A.lse[at] = (m + log2f(l)) * LN2;
                    }
                }
            }
            tmem_fence_before_sync();
            if (MODE == KEYS) {  // the next piece's products may write the accumulators
                mbar_arrive(smem_addr(&ctl.joined));
                ok = mbar_wait_bounded(smem_addr(&ctl.joined), join_phase) && ok;
                join_phase ^= 1u;
                ok = __all_sync(FULL, ok);
            }
        }
        __syncwarp();
    }
    // ---------------------------------------------------------- the end ----
    __syncwarp();
    if (!ok) ctl.dead = 1;
    __syncthreads();
    if (ctl.dead) {
        // a wait gave up: let copies and products in flight end before the
        // shared and tensor memory goes, and flag every sequence of the range
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 10000000ull) __nanosleep(1000);
    }
    if (mtile == 0 && tid == 0) {
        AttnWalk w = ctl.begin;
        AttnPiece last = {};
        while (w.next(A, pc)) {
            last = pc;
            if (ctl.dead && A.flags) atomicOr(A.flags + pc.b, F_TIMEOUT);
        }
        attn_write_desc(A, group, w, true, last);
    }
    tmem_fence_after_sync();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

}  // namespace

namespace {
template <typename F>
auto pick(int D, int mode, F f) {
    return D == 64    ? mode == ROWS ? f(Cfg<64, ROWS>{}, attn_umma_impl<64, ROWS>) : f(Cfg<64, KEYS>{}, attn_umma_impl<64, KEYS>)
           : D == 128 ? mode == ROWS ? f(Cfg<128, ROWS>{}, attn_umma_impl<128, ROWS>) : f(Cfg<128, KEYS>{}, attn_umma_impl<128, KEYS>)
                      : f(Cfg<256, ONE>{}, attn_umma_impl<256, ONE>);
}
}  // namespace

int attn_umma_bn(int D) { return D == 256 ? 64 : 128; }

UmmaPlan attn_umma_plan(int D, int rows) {
    UmmaPlan p;
    const int mode = D == 256 ? ONE : rows > 128 ? ROWS : KEYS;
    p.bm = mode == ROWS ? 256 : 128;
    p.qrows = rows >= 128 ? 128 : (rows + 7) / 8 * 8;
    const uint32_t q = static_cast<uint32_t>(p.qrows) * D * 2 * (mode == ROWS ? 2 : 1);
    const uint32_t slot = static_cast<uint32_t>(attn_umma_bn(D)) * D * 2;
    p.slots = static_cast<int>((UMMA_SMEM - sizeof(Control) - q) / slot);
    if (p.slots > MAX_SLOTS) p.slots = MAX_SLOTS;
    // the product reads 128 rows of every block of queries
    p.smem = q + p.slots * slot + static_cast<uint32_t>(sizeof(Control));
    p.func = pick(D, mode, [](auto, auto f) { return reinterpret_cast<const void *>(f); });
    p.threads = pick(D, mode, [](auto c, auto) { return decltype(c)::NT; });
    return p;
}

}  // namespace mtp
