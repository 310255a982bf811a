// tree_attention_umma.cu -- tree attention on the tensor cores: bfloat16
// storage, head sizes 64, 128 and 256, caches that tiled copies can address
// (tree_attention.cuh has the split of the work over CTAs).
//
// One CTA per SM works through its list of key tiles.  A tile is BN keys of
// one (sequence, key head); the CTA's 128 query rows (nodes x query heads of
// the group) stay in shared memory for the piece.
//   warp 0      copies key and value tiles page by page into a ring of slots
//               (cp.async.bulk.tensor, 128-byte swizzle)
//   warp 1      one lane issues S = Q K^T into one of two TMEM buffers, then
//               O += P V of the tile before, P read from TMEM: the products of
//               tile j + 1 are in the pipe while the softmax of tile j runs
//   warps 2, 3  load the queries, the new keys and values and the ancestor
//               masks of a piece, and check its page table
//   warps 4 - 7 softmax: a thread has one row, so the running maximum and sum
//               need no exchange.  Weights go back to TMEM as bfloat16 over
//               the scores they came from.
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

constexpr int NT = UMMA_THREADS;
constexpr int LOADERS = 64;
constexpr float RESCALE = 8.f;  // rescale when the maximum rose by this many powers of two

template <int D>
struct Cfg {
    static constexpr int BN = D == 256 ? 64 : 128;
    static constexpr int CH = D / 64;                      // 64-element blocks of a row
    static constexpr uint32_t QBYTES = 128 * D * 2;
    static constexpr uint32_t SLOT = BN * D * 2;           // a key or value tile
    static constexpr int SLOTS = D == 64 ? 12 : D == 128 ? 6 : 5;
    static constexpr uint32_t S_COL = 128;                 // score buffers at columns 0 and 128
    static constexpr uint32_t O_COL = 256;
};

// What the loaders say about a piece lies in a ring of four: the products are
// at most two tiles, and so two pieces, ahead of the softmax, and the loaders
// one piece ahead of the products.
struct Control {
    uint64_t full[12], empty[12], s_full[2], p_full[2], o_done[2], q_full, q_empty, tree;
    uint64_t grant[8];            // two slots of the ring are the loaders' to fill (at most SLOTS / 2 at a time)
    uint64_t masks[4], ready[4];  // a piece's masks are there; all that the loaders found out is
    uint64_t mask[4][MAX_NODES];
    uint64_t poison[4][2];
    int flag[4][2];
    long long scan[NT / 32];
    AttnWalk begin;
    uint32_t tmem;
    int dead;
};

template <int D>
constexpr uint32_t smem_bytes() {
    return Cfg<D>::QBYTES + Cfg<D>::SLOT * Cfg<D>::SLOTS + sizeof(Control);
}

// A ring position: slot index and the parity of its current use.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ int round16(int n) { return (n + 15) & ~15; }

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
        for (int i = 0; i < 32; ++i) t[i & 3] = fmaxf(t[i & 3], __uint_as_float(x[i]));
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

template <int D>
__global__ void __launch_bounds__(NT, 1)
    attn_umma_impl(const __grid_constant__ TreeAttnArgs A, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Control &ctl = *reinterpret_cast<Control *>(smem + C::QBYTES + C::SLOT * C::SLOTS);
    const uint32_t sq = smem_addr(smem), ring0 = sq + C::QBYTES;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = blockIdx.x / A.mtiles, mtile = blockIdx.x - group * A.mtiles;
    const int row0 = mtile * 128, rows = min(128, A.rows - row0);

    AttnWalk walk;
    walk.start<NT>(A, group, ctl.scan);
    if (walk.at >= walk.hi) {  // no tiles for this group
        if (mtile == 0 && tid == 0) A.desc[static_cast<size_t>(group) * ATTN_DESC + 2] = 0;
        return;
    }
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < C::SLOTS; ++i) {
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
        ctl.dead = 0;
        fence_mbar_init();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    if (warp == 1) tmem_alloc(&ctl.tmem, TMEM_COLS);
    // rows of the query tile that no query fills
    for (int i = tid; i < (128 - rows) * (D / 8); i += NT) {
        const int r = rows + i / (D / 8), u = i % (D / 8);
        *reinterpret_cast<uint4 *>(smem + (u >> 3) * (128 * 128) + sw128(r, u & 7)) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async();
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tmem = ctl.tmem;
    if (tid == 0) ctl.begin = walk;  // read at the end, by the same thread
    bool ok = (sq & 1023u) == 0u;  // the swizzle counts on it
    AttnPiece pc;

    if (warp == 0) {
        // ---------------------------------------------------- copies ----
        Ring<C::SLOTS> r;
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
        Ring<C::SLOTS> r;
        uint32_t q_phase = 0;
        int n_tiles = 0;             // tiles so far: score buffer and its parity
        bool have = false;           // a tile whose P V is still to be issued
        bool pv_first = false;
        int pv_steps = 0, pv_slot = 0;
        uint32_t pv_phase = 0;
        auto pv = [&]() {
            const int j = n_tiles - 1, buf = j & 1;
            ok = mbar_wait_bounded(smem_addr(&ctl.p_full[buf]), (j >> 1) & 1) && ok;
            ok = mbar_wait_bounded(smem_addr(&ctl.full[pv_slot]), pv_phase) && ok;
            ok = __all_sync(FULL, ok);
            if (!ok) return;
            tmem_fence_after_sync();
            if (elect_one()) {
                const uint32_t v = ring0 + pv_slot * C::SLOT;
                for (int k = 0; k < pv_steps; ++k)
                    umma_ts(tmem + C::O_COL, tmem + buf * C::S_COL + 8 * k, umma_desc(v + k * 2048, C::BN * 128),
                            umma_idesc(D, true), !(pv_first && k == 0));
                umma_commit(smem_addr(&ctl.empty[pv_slot]));
                umma_commit(smem_addr(&ctl.o_done[buf]));
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
                ok = mbar_wait_bounded(smem_addr(&ctl.full[r.slot]), r.phase) && ok;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                tmem_fence_after_sync();
                if (elect_one()) {
                    // the products before this one in the pipe have read the
                    // weights that lay in this buffer
                    const uint32_t s = tmem + (n_tiles & 1) * C::S_COL, k = ring0 + r.slot * C::SLOT;
                    const uint32_t idesc = umma_idesc(t == pc.prefix ? round16(valid) : C::BN, false);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        umma_ss(s, umma_desc(sq + (i >> 2) * (128 * 128) + (i & 3) * 32),
                                umma_desc(k + (i >> 2) * (C::BN * 128) + (i & 3) * 32), idesc, i > 0);
                    umma_commit(smem_addr(&ctl.empty[r.slot]));
                    umma_commit(smem_addr(&ctl.s_full[n_tiles & 1]));
                    if (t + 1 == pc.t1) umma_commit(smem_addr(&ctl.q_empty));
                }
                __syncwarp();
                r.step();
                if (have) pv();
                have = true;
                pv_first = t == pc.t0;
                pv_steps = round16(valid) / 16;
                pv_slot = r.slot;
                pv_phase = r.phase;
                r.step();
                ++n_tiles;
            }
        }
        if (ok && have) pv();
    } else if (warp < 4) {
        // ------------------------------------- queries and new tokens ----
        const int lt = tid - 64;
        Ring<C::SLOTS> r;
        uint32_t q_phase = 0, tree_phase = 0;
        int grants = 0;
        const bf16_t *gq = static_cast<const bf16_t *>(A.q);
        for (int np = 0; ok && walk.next(A, pc); ++np) {
            const int b = pc.b, h = pc.h;
            bool bad_len, bad_nodes;
            attn_len(A, b, bad_len);
            const int n = attn_nodes(A, b, bad_nodes);
            if (np > 0) {
                ok = mbar_wait_bounded(smem_addr(&ctl.q_empty), q_phase) && ok;
                q_phase ^= 1u;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
            }
#pragma unroll 4
            for (int i = lt; i < rows * (D / 8); i += LOADERS) {
                const int rr = i / (D / 8), u = i % (D / 8);
                const int t = (row0 + rr) / A.G, g = row0 + rr - t * A.G;
                const uint4 x = __ldg(reinterpret_cast<const uint4 *>(gq + b * A.qs[0] + t * A.qs[1] +
                                                                      (static_cast<int64_t>(h) * A.G + g) * A.qs[2]) +
                                      u);
                *reinterpret_cast<uint4 *>(smem + (u >> 3) * (128 * 128) + sw128(rr, u & 7)) = x;
            }
            int flag = (bad_len || bad_nodes) ? F_BAD_ID : 0;
            if (lt < n) {
                bool bad_up = false;
                ctl.mask[np & 3][lt] = attn_mask(A.parents ? A.parents + static_cast<size_t>(b) * A.T : nullptr, lt, bad_up);
                if (bad_up) flag |= F_BAD_ID;
            }
            fence_proxy_async();
            mbar_arrive(smem_addr(&ctl.q_full));
            mbar_arrive(smem_addr(&ctl.masks[np & 3]));
            flag |= attn_check_pages(A, b, pc.len, lt, LOADERS);
            flag = __reduce_or_sync(FULL, flag);
            if (lane == 0) ctl.flag[np & 3][warp - 2] = flag;
            uint64_t poison = 0;
            for (int t = pc.t0; t < pc.t1; ++t) {
                for (int kv = 0; kv < 2; ++kv) {
                    if (t == pc.prefix) {
                        if (kv == 0) {
                            ok = mbar_wait_bounded(smem_addr(&ctl.grant[grants & 7]), (grants >> 3) & 1) && ok;
                            ++grants;
                        }
                        unsigned char *dst = smem + C::QBYTES + r.slot * C::SLOT;
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
                                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                                if (j < n) x = __ldg(reinterpret_cast<const uint4 *>(src + b * st[0] + j * st[1] + h * st[2]) + u);
                                if (kv) {
                                    uint32_t *w = &x.x;
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const bool lo = (w[e] & 0x7f80u) == 0x7f80u, hi = (w[e] & 0x7f800000u) == 0x7f800000u;
                                        if (lo || hi) poison |= 1ull << j;
                                        w[e] = (lo ? 0u : w[e] & 0xffffu) | (hi ? 0u : w[e] & 0xffff0000u);
                                    }
                                }
                                *reinterpret_cast<uint4 *>(dst + (u >> 3) * (C::BN * 128) + sw128(j, u & 7)) = x;
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
            const uint32_t plo = __reduce_or_sync(FULL, static_cast<uint32_t>(poison));
            const uint32_t phi = __reduce_or_sync(FULL, static_cast<uint32_t>(poison >> 32));
            if (lane == 0) ctl.poison[np & 3][warp - 2] = (static_cast<uint64_t>(phi) << 32) | plo;
            mbar_arrive(smem_addr(&ctl.ready[np & 3]));
            ok = __all_sync(FULL, ok);
        }
    } else {
        // --------------------------------------------------- softmax ----
        const int wt = tid - 128;                       // this thread's row
        const int part = warp - 4;                      // its 32 TMEM lanes
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * part) << 16);
        const bool busy = 32 * part < rows;             // the warp has rows
        const int rr = row0 + wt, node = rr / A.G;
        Ring<C::SLOTS> r;
        int n_tiles = 0;
        for (int np = 0; ok && walk.next(A, pc); ++np) {
            const int b = pc.b, h = pc.h;
            bool bad;
            const int n = attn_nodes(A, b, bad);
            float m = -INFINITY, l = 0.f;
            for (int t = pc.t0; t < pc.t1 && ok; ++t) {
                const int buf = n_tiles & 1;
                const uint32_t s_addr = lanes + buf * C::S_COL;
                r.step();  // the keys' slot
                const int v_slot = r.slot;
                const uint32_t v_phase = r.phase;
                r.step();
                ok = mbar_wait_bounded(smem_addr(&ctl.s_full[buf]), (n_tiles >> 1) & 1) && ok;
                tmem_fence_after_sync();
                const uint32_t o_bar = smem_addr(&ctl.o_done[buf ^ 1]), o_phase = ((n_tiles - 1) >> 1) & 1;
                if (t == pc.prefix) {
                    ok = mbar_wait_bounded(smem_addr(&ctl.masks[np & 3]), (np >> 2) & 1) && ok;
                    const uint64_t see = wt < rows && node < n ? ctl.mask[np & 3][node] : 0ull;
                    if (busy) {
                        if (n <= 32)
                            softmax_tile<1, true>(s_addr, lanes + C::O_COL, D, A.scale_log2, 0, see, t == pc.t0, m, l,
                                                  o_bar, o_phase, ok);
                        else
                            softmax_tile<2, true>(s_addr, lanes + C::O_COL, D, A.scale_log2, 0, see, t == pc.t0, m, l,
                                                  o_bar, o_phase, ok);
                    }
                } else {
                    int pos, valid;
                    attn_tile(A, pc.len, t, pos, valid);
                    if (busy)
                        softmax_tile<C::BN / 32, false>(s_addr, lanes + C::O_COL, D, A.scale_log2, valid, 0ull, t == pc.t0, m, l,
                                                        o_bar, o_phase, ok);
                    const int end = round16(valid);
                    if (valid < end) {  // what lies behind the last key meets a weight of 0: it has to be a number
                        ok = mbar_wait_bounded(smem_addr(&ctl.full[v_slot]), v_phase) && ok;
                        for (int i = wt; i < (end - valid) * (D / 8); i += 128) {
                            const int j = valid + i / (D / 8), u = i % (D / 8);
                            *reinterpret_cast<uint4 *>(smem + C::QBYTES + v_slot * C::SLOT + (u >> 3) * (C::BN * 128) +
                                                       sw128(j, u & 7)) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async();
                    }
                }
                tmem_fence_before_sync();
                mbar_arrive(smem_addr(&ctl.p_full[buf]));
                ++n_tiles;
                ok = __all_sync(FULL, ok);
            }
            // ------------------------------------------------ results ----
            ok = mbar_wait_bounded(smem_addr(&ctl.ready[np & 3]), (np >> 2) & 1) && ok;
            ok = mbar_wait_bounded(smem_addr(&ctl.o_done[(n_tiles - 1) & 1]), ((n_tiles - 1) >> 1) & 1) && ok;
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            tmem_fence_after_sync();
            const int flag = ctl.flag[np & 3][0] | ctl.flag[np & 3][1];
            if (A.flags && wt == 0 && h == 0 && mtile == 0) A.flags[b] = flag;
            const uint64_t seen = pc.t1 == pc.prefix + 1 && wt < rows && node < n
                                      ? ctl.mask[np & 3][node] & (ctl.poison[np & 3][0] | ctl.poison[np & 3][1])
                                      : 0ull;
            if (flag) l = NAN;
            const bool whole = pc.whole();
            const bool mine = wt < rows && (bad || node < n);
            const int hq = h * A.G + rr - node * A.G;
            const size_t at = (static_cast<size_t>(b) * A.T + node) * A.Hq + hq;
            float *slot = A.part + attn_slot(A, group, mtile, pc.first) * attn_slot_floats(128, D);
            const float inv = 1.f / l;
            if (busy) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_ld32(lanes + C::O_COL + c, o);
                    tmem_wait_ld32(o);
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
                        uint4 *dst = reinterpret_cast<uint4 *>(slot + 2 * 128 + static_cast<size_t>(wt) * D + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
                if (mine && whole && A.lse) A.lse[at] = (m + log2f(l)) * LN2;
                if (mine && !whole) {
                    slot[wt] = m;
                    slot[128 + wt] = l;
                }
            }
            tmem_fence_before_sync();
        }
    }
    // ---------------------------------------------------------- the end ----
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
    if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
}

}  // namespace

const void *attn_umma_func(int D) {
    return D == 64    ? reinterpret_cast<const void *>(attn_umma_impl<64>)
           : D == 128 ? reinterpret_cast<const void *>(attn_umma_impl<128>)
                      : reinterpret_cast<const void *>(attn_umma_impl<256>);
}
uint32_t attn_umma_smem(int D) { return D == 64 ? smem_bytes<64>() : D == 128 ? smem_bytes<128>() : smem_bytes<256>(); }
int attn_umma_bn(int D) { return D == 256 ? Cfg<256>::BN : Cfg<128>::BN; }

}  // namespace mtp
