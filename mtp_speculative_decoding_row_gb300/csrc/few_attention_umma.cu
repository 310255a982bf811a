// few_attention_umma.cu -- the tensor-core kernels of mtp_prefix_attention for few
// query rows (a sequence's own tokens, and prefixes of few sequences): up to 32
// with heads of 128, up to 16 with heads of 256 (three tiles of 64 KB fit beside
// those).
//
// With few rows a product whose 128 rows are queries leaves most of them empty
// and a softmax warp's lanes with them.  Here the operands change places: the
// 128 keys of a tile are the rows,
//   S^T = K Q^T   [128 keys, R],   O^T = V^T P^T   [D, R],   R = 16 or 32,
// so that each thread of one group of four warps has one key with its scores
// against all R rows in registers, and the products cost an eighth.  Nothing of a
// tile is then summed over lanes: a thread keeps the sums of its own keys'
// weights until a piece ends, and of the maxima the threads only vote whether
// a score lies far above its row's reference; where one does the maxima are found
// by halving exchanges.  Weights lie in shared memory as bfloat16 (in TMEM a product's
// second operand cannot lie).
//   warp 0      copies key and value tiles, as in the other kernel
//   warp 1      issues the products; those with the keys of tile j + 1 before
//               those with the values of tile j, so that the tensor cores' and
//               the softmax's latencies overlap
//   warp 2      masks, new values, page tables
//   warp 3      queries, new keys
//   warps 4..7  softmax, results
// Two score buffers, two of weights and two accumulators: the next piece begins
// while the last one's results are written.
//
// Precision is float32 but for the weights, which are bfloat16 in the products as
// in the other kernel, or the sum of two such numbers (to 2^-16).  Memory
// bounds it where it has the GPU (64 sequences of 1024 tokens, 16 rows, heads of
// 128: 37 us from the first copy on, 7.2 TB/s with what the L2 cache still has; the
// other kernel 55): a tile of 64 KB each us and SM, the ring's 192 KB over the
// copies' latency.  What a unit costs beside its tiles, some 3 us, is latency (the
// new keys' loads, the last products, the first scores) and code that the
// instruction cache no longer holds.
#include "tree_attention_umma.cuh"

namespace mtp {
namespace {

// A row's reference rises when a score lies 2^30 above it: the weights are then
// at most 2^30, their sums far below float32's largest, and what float32 cannot
// hold below a reference that low is nothing beside the largest weight.
constexpr float RISE = 30.f;

// PARTS: bfloat16 numbers that a weight is the sum of.
template <int D, int R, int PARTS>
struct Few {
    static constexpr int NT = 256, BN = 128;
    static constexpr int CH = D / 64, HALVES = D / 128;
    static constexpr uint32_t SLOT = BN * D * 2;
    static constexpr uint32_t PLANE = R * 256, PB = PLANE * PARTS;  // weights of a tile
    static constexpr uint32_t S_COL = 32, O_COL = 64;       // score buffers at 0, 32; accumulators from 64 on, 32 columns each half
};

template <class Walk, int R>
struct FewControl {
    uint64_t full[2 * MAX_SLOTS], empty[MAX_SLOTS], s_full[2], s_empty[2], p_full[2], o_done[2], o_free[2], q_full[2], q_empty[2];
    uint64_t grant[8], masks[4], ready[4], done[4];  // as in the other kernel
    uint64_t vote, tops, sums, begun;                // the softmax warps' exchanges
    uint64_t mask[4][R];  // (no more nodes than rows)
    uint64_t poison[4];
    int above[R];
    long long W;
    Walk begin;
    alignas(16) int votes[2][4];
    alignas(16) float top[2][R][4], sum[2][R][4];  // row, warp
    alignas(16) float first[2][R];                  // scores of a piece's first key
    uint32_t tmem;
    int dead;
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
          "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}
// R columns of this lane; valid on return.
__device__ __forceinline__ void load_cols(uint32_t taddr, uint32_t (&v)[16]) {
    tmem_ld16(taddr, v);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ void load_cols(uint32_t taddr, uint32_t (&v)[32]) {
    tmem_ld32(taddr, v);
    tmem_wait_ld32(v);
}
__device__ __forceinline__ void store_cols(uint32_t taddr, const uint32_t (&v)[16]) { tmem_st16(taddr, v); }
__device__ __forceinline__ void store_cols(uint32_t taddr, const uint32_t (&v)[32]) { tmem_st32(taddr, v); }

// Instruction descriptor with A MN-major: the rows of V^T lie along a key's values.
constexpr uint32_t idesc_turned(uint32_t n) { return umma_idesc(n, false) | (1u << 15); }

// v[r] of all lanes joined for each row r: half of the rows are handed to the
// lane 16 on, a quarter to that 8 on, ..  Lane i ends with row i (R = 32) or
// i / 2 (R = 16) in v[0].
template <int R, bool SUM>
__device__ __forceinline__ float join_rows(float (&v)[R]) {
    const int lane = threadIdx.x & 31;
    auto op = [](float a, float b) { return SUM ? a + b : fmaxf(a, b); };
    int d = 16;
#pragma unroll
    for (int n = R / 2; n >= 1; n /= 2) {
        const bool up = (lane & d) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = op(keep, __shfl_xor_sync(FULL, give, d));
        }
        d /= 2;
    }
    if (R == 16) v[0] = op(v[0], __shfl_xor_sync(FULL, v[0], 1));
    return v[0];
}

template <int D, int R, int PARTS, bool PREFIX>
__global__ void __launch_bounds__(Few<D, R, PARTS>::NT, 1)
    attn_few_impl(const __grid_constant__ TreeAttnArgs A, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using C = Few<D, R, PARTS>;
    using Walk = typename std::conditional<PREFIX, PrefixWalk, AttnWalk>::type;
    using Piece = typename Walk::Piece;
    constexpr int NT = C::NT;
    // weights (two buffers of two blocks of 64 keys x R rows), queries (blocks of
    // 64 elements x R rows, once or twice), ring, control
    extern __shared__ __align__(1024) unsigned char smem[];
    constexpr uint32_t QBLOCK = R * 128, QBYTES = QBLOCK * C::CH * 2;
    unsigned char *queries = smem + 2 * C::PB, *ring = queries + QBYTES;
    using Ctl = FewControl<Walk, R>;
    Ctl &ctl = *reinterpret_cast<Ctl *>(ring + C::SLOT * A.slots);
    const uint32_t sp = smem_addr(smem), sq = smem_addr(queries), ring0 = smem_addr(ring);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = blockIdx.x;

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < A.slots; ++i) {
            mbar_init(smem_addr(&ctl.full[2 * i]), 1);
            mbar_init(smem_addr(&ctl.full[2 * i + 1]), 1);
            mbar_init(smem_addr(&ctl.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl.s_full[i]), 1);
            mbar_init(smem_addr(&ctl.s_empty[i]), 4);
            mbar_init(smem_addr(&ctl.p_full[i]), 4);
            mbar_init(smem_addr(&ctl.o_done[i]), 1);
            mbar_init(smem_addr(&ctl.o_free[i]), 4);
            mbar_init(smem_addr(&ctl.q_full[i]), 32);
            mbar_init(smem_addr(&ctl.q_empty[i]), 1);
        }
        for (int i = 0; i < 8; ++i) mbar_init(smem_addr(&ctl.grant[i]), 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_addr(&ctl.masks[i]), LOADERS);
            mbar_init(smem_addr(&ctl.ready[i]), LOADERS);
            mbar_init(smem_addr(&ctl.done[i]), 128);
        }
        mbar_init(smem_addr(&ctl.vote), 4);
        mbar_init(smem_addr(&ctl.tops), 4);
        mbar_init(smem_addr(&ctl.sums), 4);
        mbar_init(smem_addr(&ctl.begun), 4);
        ctl.dead = 0;
        fence_mbar_init();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(&ctl.tmem, TMEM_COLS);
    }
    for (uint32_t i = tid; i < QBYTES / 16; i += NT) reinterpret_cast<uint4 *>(queries)[i] = make_uint4(0u, 0u, 0u, 0u);  // rows that no query fills
    fence_proxy_async();
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tmem = ctl.tmem;
    if (PREFIX || !A.overlap) pdl_wait();
    pdl_next();
    Walk walk;
    {
        const long long W = walk.start(A, group, attn_limit<PREFIX>(A));
        if (tid == 0) {
            ctl.W = W;
            ctl.begin = walk;
        }
    }
    bool ok = (sq & 1023u) == 0u;  // the swizzle counts on it
    Piece pc;

    if (warp == 0) {
        // ---------------------------------------------------- copies ----
        Ring r(A.slots);
        int grants = 0;
        const int boxrows = min(C::BN, A.page_size);
        while (ok && walk.next(A, pc)) {
            for (int t = pc.t0; t < pc.t1 && ok; ++t) {
                if (!PREFIX && t == pc.prefix) {
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
                const int mine = lane < pages ? attn_page(A, pc.b, page0 + lane) : 0;
                for (int kv = 0; kv < 2; ++kv) {
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
    } else if (warp == 1) {
        // -------------------------------------------------- products ----
        Ring r(A.slots), old(A.slots);
        bool have = false;  // the product with the values of tile `count - 1` is still to be issued
        int count = 0, np = 0, steps = 0, acc = 0;
        bool fresh = false;
        auto pv = [&]() {
            const int c = count - 1, buf = c & 1;
            if (fresh && acc >= 2) ok = wait_for(A, smem_addr(&ctl.o_free[acc & 1]), ((acc >> 1) - 1) & 1) && ok;
            ok = wait_for(A, smem_addr(&ctl.p_full[buf]), (c >> 1) & 1) && ok;
            ok = wait_for(A, smem_addr(&ctl.full[old.full()]), old.phase()) && ok;
            ok = __all_sync(FULL, ok);
            if (!ok) return;
            tmem_fence_after_sync();
            if (elect_one()) {
                const uint64_t v = umma_desc(ring0 + old.slot * C::SLOT, C::BN * 128), p = umma_desc(sp + buf * C::PB);
#pragma unroll
                for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
                    for (int k = 0; k < C::BN / 16; ++k)
                        if (k < steps)
#pragma unroll
                            for (int part = 0; part < PARTS; ++part)
                                umma_ss(tmem + C::O_COL + ((acc & 1) * C::HALVES + h) * 32, v + ((h * 2 * (C::BN * 128) + k * 2048) >> 4),
                                        p + ((part * C::PLANE + (k >> 2) * (R * 128) + (k & 3) * 32) >> 4), idesc_turned(R),
                                        !(fresh && k == 0 && part == 0));
                umma_commit(smem_addr(&ctl.o_done[buf]));
                umma_commit(smem_addr(&ctl.empty[old.slot]));
            }
            __syncwarp();
            have = false;
        };
        for (; ok && walk.next(A, pc); ++np) {
            bool bad;
            const int n = PREFIX ? 0 : attn_nodes(A, pc.b, bad);
            const int qi = (np & 1);
            ok = wait_for(A, smem_addr(&ctl.q_full[qi]), (np >> 1) & 1) && ok;
            ok = __all_sync(FULL, ok);
            for (int t = pc.t0; t < pc.t1 && ok; ++t) {
                const Ring kr = r;
                r.step();
                const Ring vr = r;
                r.step();
                int pos, valid;
                if (!PREFIX && t == pc.prefix)
                    valid = n > 0 ? n : 1;
                else
                    attn_tile(A, pc.len, t, pos, valid);
                const int buf = count & 1;
                if (count >= 2) ok = wait_for(A, smem_addr(&ctl.s_empty[buf]), ((count >> 1) - 1) & 1) && ok;
                ok = wait_for(A, smem_addr(&ctl.full[kr.full()]), kr.phase()) && ok;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                tmem_fence_after_sync();
                if (elect_one()) {
                    const uint64_t q = umma_desc(sq + qi * C::CH * QBLOCK), k = umma_desc(ring0 + kr.slot * C::SLOT);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        umma_ss(tmem + buf * C::S_COL, k + (((i >> 2) * (C::BN * 128) + (i & 3) * 32) >> 4),
                                q + (((i >> 2) * QBLOCK + (i & 3) * 32) >> 4), umma_idesc(R, false), i > 0);
                    umma_commit(smem_addr(&ctl.s_full[buf]));
                    umma_commit(smem_addr(&ctl.empty[kr.slot]));
                }
                __syncwarp();
                if (have) pv();
                if (!ok) break;
                ++count;
                have = true;
                old = vr;
                steps = round16(valid) / 16;
                fresh = t == pc.t0;
                acc = np;
            }
            if (elect_one()) umma_commit(smem_addr(&ctl.q_empty[qi]));
            __syncwarp();
            if (ok && have) pv();  // (the piece's results wait for it)
        }
    } else if (warp == 2 || warp == 3) {
        // ---- warp 2: masks, new values, pages; warp 3: queries, new keys ----
        // (One piece of a sequence or prefix looks at its pages and speaks for all:
        // the join makes the rows of what is flagged NaN.)
        Ring r(A.slots);
        int grants = 0;
        // Queries of piece `np`, into the buffer that the piece before the last had.
        auto copy_q = [&](const Piece &p, int np) {
            const int qi = np & 1;
            if (np >= 2) ok = wait_for(A, smem_addr(&ctl.q_empty[qi]), ((np >> 1) - 1) & 1) && ok;
            ok = __all_sync(FULL, ok);
            if (!ok) return;
            if constexpr (PREFIX)
                copy_prefix_queries<D>(A, p, 0, p.rows, sq + qi * C::CH * QBLOCK, lane, 32);
            else
                copy_queries<D>(static_cast<const bf16_t *>(A.q) + p.b * A.qs[0] + static_cast<int64_t>(p.h) * A.G * A.qs[2], A, 0, A.rows,
                                sq + qi * C::CH * QBLOCK, lane, 32);
            cp_async_wait_all();
            fence_proxy_async();
            mbar_arrive(smem_addr(&ctl.q_full[qi]));
        };
        if (PREFIX && warp == 2 && blockIdx.x == 0) prefix_check_starts(A);
        Piece next;
        bool more = walk.next(A, next);
        if (warp == 3 && more) copy_q(next, 0);
        for (int np = 0; ok && more; ++np) {
            pc = next;
            more = walk.next(A, next);
            if (warp == 3 && more) copy_q(next, np + 1);
            if (!ok) break;
            if (warp == 2 && np >= 4) {
                ok = wait_for(A, smem_addr(&ctl.done[np & 3]), ((np >> 2) - 1) & 1) && ok;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
            }
            int flag = 0;
            if constexpr (!PREFIX) {
                const int b = pc.b, h = pc.h;
                bool bad_len, bad_nodes;
                attn_len(A, b, bad_len);
                const int n = attn_nodes(A, b, bad_nodes);
                if (bad_len || bad_nodes) flag = F_BAD_ID;
                if (warp == 2) {
                    flag |= attn_masks(A.parents ? A.parents + static_cast<size_t>(b) * A.T : nullptr, n, ctl.mask[np & 3], ctl.above);
                    mbar_arrive(smem_addr(&ctl.masks[np & 3]));
                }
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
                        if (kv == (warp == 2)) {
                            poison = load_new<D, C::BN>(A, ring + r.slot * C::SLOT, kv != 0, b, h, n);
                            fence_proxy_async();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(smem_addr(&ctl.full[r.full()]));
                        }
                        r.step();
                    }
                }
                const uint32_t plo = __reduce_or_sync(FULL, static_cast<uint32_t>(poison));
                const uint32_t phi = __reduce_or_sync(FULL, static_cast<uint32_t>(poison >> 32));
                if (warp == 2 && lane == 0) ctl.poison[np & 3] = (static_cast<uint64_t>(phi) << 32) | plo;
            }
            if (warp == 3) continue;
            if (np > 0 || A.fault_cta != static_cast<int>(blockIdx.x) + 1) mbar_arrive(smem_addr(&ctl.ready[np & 3]));
            if (flags_owner(pc, 0)) {
                flag |= attn_check_pages(A, pc.b, pc.len, lane, LOADERS);
                flag = __reduce_or_sync(FULL, flag);
                if (lane == 0) put_flag(A, pc.b, flag);
            }
        }
    } else if (warp >= 4) {
        // --------------------------------------------------- softmax ----
        const int w = warp - 4, wt = tid - 128;  // wt: this thread's key of a tile, and its element of the head
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        Ring r(A.slots);
        int count = 0;                           // tiles so far
        uint32_t votes = 0, exchanges = 0, begun = 0;
        for (int np = 0; ok && walk.next(A, pc); ++np) {
            bool bad = false;
            const int n = PREFIX ? 0 : attn_nodes(A, pc.b, bad);
            int live;  // rows of the piece
            if constexpr (PREFIX)
                live = pc.rows;
            else
                live = bad ? A.rows : n * A.G;
            float m[R], l[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
            }
            bool first = true;
            for (int t = pc.t0; t < pc.t1 && ok; ++t, ++count) {
                r.step();  // the keys' slot
                const Ring vr = r;
                r.step();
                const int buf = count & 1;
                // which rows see this thread's key
                int valid = C::BN;
                uint32_t see = ~0u;
                const bool tree = !PREFIX && t == pc.prefix;
                if (tree) {
                    ok = wait_for(A, smem_addr(&ctl.masks[np & 3]), (np >> 2) & 1) && ok;
                    see = 0;
                    if (wt < n)
#pragma unroll 4
                        for (int i = 0; i < min(R, live); ++i)
                            see |= static_cast<uint32_t>((ctl.mask[np & 3][node_of(A, i)] >> wt) & 1ull) << i;
                } else {
                    int pos;
                    attn_tile(A, pc.len, t, pos, valid);
                    if (wt >= valid) see = 0;
                }
                ok = wait_for(A, smem_addr(&ctl.s_full[buf]), (count >> 1) & 1) && ok;
                ok = __all_sync(FULL, ok);
                tmem_fence_after_sync();
                uint32_t s[R];
                load_cols(lanes + buf * C::S_COL, s);
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ctl.s_empty[buf]));
#pragma unroll
                for (int i = 0; i < R; ++i) s[i] = (see >> i) & 1u ? __float_as_uint(__uint_as_float(s[i]) * A.scale_log2) : 0xff800000u;
                if (first && !tree) {
                    // any key's score serves as a reference until one lies far above it:
                    // those of the first key, which all rows see
                    if (wt == 0)
#pragma unroll
                        for (int i = 0; i < R; i += 4)
                            *reinterpret_cast<uint4 *>(&ctl.first[np & 1][i]) = make_uint4(s[i], s[i + 1], s[i + 2], s[i + 3]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&ctl.begun));
                    ok = wait_for(A, smem_addr(&ctl.begun), begun & 1) && ok;
                    ++begun;
#pragma unroll
                    for (int i = 0; i < R; i += 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(&ctl.first[np & 1][i]);
                        m[i] = x.x;
                        m[i + 1] = x.y;
                        m[i + 2] = x.z;
                        m[i + 3] = x.w;
                    }
                }
                float over = -INFINITY;
#pragma unroll
                for (int i = 0; i < R; ++i) over = fmaxf(over, __uint_as_float(s[i]) - m[i]);  // (a NaN is passed over, as a maximum does)
                // does any row's reference have to rise?
                const bool up = __any_sync(FULL, over > RISE);
                if (lane == 0) {
                    ctl.votes[votes & 1][w] = up;
                    mbar_arrive(smem_addr(&ctl.vote));
                }
                ok = wait_for(A, smem_addr(&ctl.vote), votes & 1) && ok;
                const int4 all = *reinterpret_cast<const int4 *>(ctl.votes[votes & 1]);
                ++votes;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                if (all.x | all.y | all.z | all.w) {
                    float f[R];
#pragma unroll
                    for (int i = 0; i < R; ++i) f[i] = __uint_as_float(s[i]);
                    const float top = join_rows<R, false>(f);
                    if (R == 32 || (lane & 1) == 0) ctl.top[exchanges & 1][R == 32 ? lane : lane >> 1][w] = top;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&ctl.tops));
                    ok = wait_for(A, smem_addr(&ctl.tops), exchanges & 1) && ok;
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float4 x = *reinterpret_cast<const float4 *>(ctl.top[exchanges & 1][i]);
                        const float y = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
                        f[i] = 1.f;
                        if (y > m[i] + RISE || (m[i] == -INFINITY && y > m[i])) {
                            f[i] = m[i] == -INFINITY ? 0.f : ex2(m[i] - y);
                            m[i] = y;
                        }
                        l[i] *= f[i];
                    }
                    ++exchanges;
                    if (!first) {  // the accumulator of the tiles before this one
                        ok = wait_for(A, smem_addr(&ctl.o_done[buf ^ 1]), ((count - 1) >> 1) & 1) && ok;
                        ok = __all_sync(FULL, ok);
                        if (!ok) break;
                        tmem_fence_after_sync();
#pragma unroll
                        for (int h = 0; h < C::HALVES; ++h) {
                            uint32_t o[R];
                            const uint32_t at = lanes + C::O_COL + ((np & 1) * C::HALVES + h) * 32;
                            load_cols(at, o);
#pragma unroll
                            for (int i = 0; i < R; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f[i]);
                            store_cols(at, o);
                        }
                        tmem_wait_st();
                    }
                }
                first = false;
                // the product that read the weights before these is done
                if (count >= 2) ok = wait_for(A, smem_addr(&ctl.o_done[buf]), ((count >> 1) - 1) & 1) && ok;
                ok = __all_sync(FULL, ok);
                if (!ok) break;
                unsigned char *p = smem + buf * C::PB + (wt >> 6) * (R * 128) + (wt & 7) * 2;
#pragma unroll
                for (int i = 0; i < R; i += 2) {
                    const float x = __uint_as_float(s[i]), y = __uint_as_float(s[i + 1]);
                    const float a = ex2(x - (m[i] == -INFINITY ? 0.f : m[i])), c = ex2(y - (m[i + 1] == -INFINITY ? 0.f : m[i + 1]));
                    l[i] += a;
                    l[i + 1] += c;
                    const uint32_t both = bf16x2(a, c);
                    *reinterpret_cast<uint16_t *>(p + sw128(i, (wt >> 3) & 7)) = static_cast<uint16_t>(both);
                    *reinterpret_cast<uint16_t *>(p + sw128(i + 1, (wt >> 3) & 7)) = static_cast<uint16_t>(both >> 16);
                    if constexpr (PARTS == 2) {  // what the rounding left
                        const uint32_t rest = bf16x2(a - __uint_as_float(both << 16), c - __uint_as_float(both & 0xffff0000u));
                        *reinterpret_cast<uint16_t *>(p + C::PLANE + sw128(i, (wt >> 3) & 7)) = static_cast<uint16_t>(rest);
                        *reinterpret_cast<uint16_t *>(p + C::PLANE + sw128(i + 1, (wt >> 3) & 7)) = static_cast<uint16_t>(rest >> 16);
                    }
                }
                if (!tree && (valid & 15)) {
                    // what lies behind the last key meets a weight of 0: it has to be a number
                    const int end = round16(valid);
                    ok = wait_for(A, smem_addr(&ctl.full[vr.full()]), vr.phase()) && ok;
                    for (int i = wt; i < (end - valid) * (D / 8); i += 128) {
                        const int j = valid + i / (D / 8), u = i % (D / 8);
                        *reinterpret_cast<uint4 *>(ring + vr.slot * C::SLOT + (u >> 3) * (C::BN * 128) + sw128(j, u & 7)) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async();
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ctl.p_full[buf]));
                ok = __all_sync(FULL, ok);
            }
            if (!ok) break;
            // ------------------------------------------------ results ----
            const float mine = join_rows<R, true>(l);
            if (R == 32 || (lane & 1) == 0) ctl.sum[np & 1][R == 32 ? lane : lane >> 1][w] = mine;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ctl.sums));
            if (w == 0) ok = wait_for(A, smem_addr(&ctl.sums), np & 1) && ok;
            ok = wait_for(A, smem_addr(&ctl.ready[np & 3]), (np >> 2) & 1) && ok;
            ok = wait_for(A, smem_addr(&ctl.o_done[(count - 1) & 1]), ((count - 1) >> 1) & 1) && ok;
            ok = __all_sync(FULL, ok);
            if (!ok) break;
            tmem_fence_after_sync();
            const bool whole = pc.whole();
            float *slot = A.part + attn_slot(A, group, 0, pc.first) * attn_slot_floats(R, D);
            const size_t place = unit_row(A, pc);
            float *part_m = whole ? A.row_m + place : slot, *part_l = whole ? A.row_l + place : slot + R;
            float *part_o = whole ? A.row_o + place * D : slot + 2 * R;
            uint64_t poison = 0;
            if constexpr (!PREFIX)
                if (pc.t1 == pc.prefix + 1) poison = ctl.poison[np & 3];
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h) {
                uint32_t o[R];
                __syncwarp();
                load_cols(lanes + C::O_COL + ((np & 1) * C::HALVES + h) * 32, o);
                const int d = h * 128 + wt;
                for (uint64_t q = poison; q; q &= q - 1) {  // values that are not finite, which the products took as zeros
                    const int node = __ffsll(static_cast<long long>(q)) - 1;
                    const bf16_t *v = static_cast<const bf16_t *>(A.v_new) + pc.b * A.vs[0] + node * A.vs[1] + pc.h * A.vs[2];
                    const float x = __uint_as_float(static_cast<uint32_t>(v[d].bits) << 16);
                    if (fabsf(x) < INFINITY) continue;
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        if (i < live && ((ctl.mask[np & 3][node_of(A, i)] >> node) & 1ull)) o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
                }
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (i < live) part_o[i * D + d] = __uint_as_float(o[i]);
            }
            if (w == 0) {
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (lane == i) top = m[i];
                if (lane < live && lane < R) {
                    const float4 x = *reinterpret_cast<const float4 *>(ctl.sum[np & 1][lane]);
                    part_m[lane] = top;
                    part_l[lane] = (x.x + x.y) + (x.z + x.w);
                }
            }
            tmem_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ctl.o_free[np & 1]));
            mbar_arrive(smem_addr(&ctl.done[np & 3]));
        }
    }
    // ---------------------------------------------------------- the end ----
    __syncwarp();
    if (!ok) ctl.dead = 1;
    __syncthreads();
    if (ctl.dead) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 10000000ull) __nanosleep(1000);
        give_up(A, ctl.begin, group, 0, 0, PREFIX ? 0 : A.rows, tid, NT);
    }
    if (tid == 0) attn_report(A, group, ctl.W, ctl.begin);
    if (!PREFIX && A.overlap && blockIdx.x == 0) pdl_wait();
    tmem_fence_after_sync();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <int D, int R, int PARTS, bool PREFIX>
UmmaPlan plan_of() {
    using C = Few<D, R, PARTS>;
    using Ctl = FewControl<typename std::conditional<PREFIX, PrefixWalk, AttnWalk>::type, R>;
    UmmaPlan p;
    constexpr uint32_t fixed = 2 * C::PB + 2 * R * D * 2 + sizeof(Ctl);
    constexpr int fit = static_cast<int>((UMMA_SMEM - fixed) / C::SLOT);
    static_assert(fit >= 3, "a tile's keys and values and the next tile's keys");
    p.func = reinterpret_cast<const void *>(attn_few_impl<D, R, PARTS, PREFIX>);
    p.threads = C::NT;
    p.bm = p.tile_rows = p.qrows = R;
    p.qbufs = 2;
    p.slots = fit < MAX_SLOTS ? fit : MAX_SLOTS;
    p.bn = C::BN;
    p.cost = D == 256 ? 250 : 100;
    p.smem = fixed + p.slots * C::SLOT;
    return p;
}

}  // namespace

// Of the prefixes always with weights of two parts.  The sequences' own tokens
// have them where the prefixes' kernel is this one, too: beside one that rounds
// its weights to bfloat16 a row is no more exact for them (64 samples of 16384
// tokens: 143 us with two parts, 135 with one, error 0.0023 both times; four
// samples of 2000 tokens: 23.6 and 22.9 us, errors 0.0017 and 0.0023 to 0.0026).
UmmaPlan few_umma_plan(int D, int rows, bool prefix, bool precise) {
    if (D == 128)
        return rows <= 16 ? (prefix    ? plan_of<128, 16, 2, true>()
                             : precise ? plan_of<128, 16, 2, false>()
                                       : plan_of<128, 16, 1, false>())
                          : (prefix    ? plan_of<128, 32, 2, true>()
                             : precise ? plan_of<128, 32, 2, false>()
                                       : plan_of<128, 32, 1, false>());
    return prefix ? plan_of<256, 16, 2, true>() : precise ? plan_of<256, 16, 2, false>() : plan_of<256, 16, 1, false>();
}

}  // namespace mtp
