// tree_attention_simt.cu -- tree attention on the FP32 pipes, and the join of
// units whose keys several CTAs share (tree_attention.cuh has the split).
//
// This kernel takes what the tensor-core kernel does not: float32 storage
// (whose products a bf16 or tf32 tensor product would round), head sizes
// other than 64, 128 and 256, and caches whose pages or strides a tiled copy
// cannot address.  One CTA holds 32 query rows and walks tiles of 64 keys:
// keys and values in shared memory as float32, scores and outputs in
// registers, the running maximum m and sum l of the softmax per row
//   m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m'),
//   o' = o 2^(m - m') + sum_j 2^(s_j - m') v_j       (s in units of log2 e),
// all in float32.  Each sum is made of shorter ones -- a score of two halves, an
// output of its tiles' sums -- which halves the error (one token after 122070:
// 1.3e-6 -> 6e-7 of the output) and costs 3 % (68 -> 70 us below).  A warp has four rows from their scores to their output, so
// only the tile itself needs barriers.  The next tile's keys are on their way
// while this one's weights and outputs are formed, its values while the next
// scores are: one tile of shared memory each, so that two CTAs fit an SM (64
// ragged sequences of up to 2500 tokens, 16 rows, float32: 89 -> 68 us, 70 with
// the shorter sums; 128 without the four rows to a warp and the values four at a time).  What bounds
// it: half of the issue slots, and as many empty while warps wait for shared
// memory and for each other (28 rows); memory runs at 14 % of its rate.
#include <type_traits>

#include "tree_attention.cuh"

namespace mtp {
namespace {

constexpr int BM = SIMT_BM, BN = SIMT_BN, NT = SIMT_THREADS;

template <typename T>
__device__ __forceinline__ float ld1(const void *p, int64_t i);
template <>
__device__ __forceinline__ float ld1<float>(const void *p, int64_t i) {
    return __ldg(static_cast<const float *>(p) + i);
}
template <>
__device__ __forceinline__ float ld1<bf16_t>(const void *p, int64_t i) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const unsigned short *>(p) + i)) << 16);
}

// One row of D elements at p + off into shared memory, zero beyond D: each of
// `nl` threads of a row (index l) copies every nl-th vector.
template <typename T, int DP>
__device__ __forceinline__ void row_to_smem(float *dst, const void *p, int64_t off, int D, int l, int nl, bool vec) {
    constexpr int VEC = Store<T>::VEC;
    if (vec) {  // D is a multiple of VEC and every row starts on 16 bytes
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(p) + off * Store<T>::ES);
        for (int c = l; c < DP / VEC; c += nl) {
            float z[VEC];
            Store<T>::unpack(c * VEC < D ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u), z);
#pragma unroll
            for (int e = 0; e < VEC; e += 4)
                *reinterpret_cast<float4 *>(dst + c * VEC + e) = make_float4(z[e], z[e + 1], z[e + 2], z[e + 3]);
        }
    } else {
        for (int c = l; c < DP; c += nl) dst[c] = c < D ? ld1<T>(p, off + c) : 0.f;
    }
}

// The same of a key or value: in float32 whole vectors are copied
// asynchronously (a group is to be committed and waited for).
template <typename T, int DP>
__device__ __forceinline__ void row_async(float *dst, const void *p, int64_t off, int D, int l, int nl, bool vec) {
    if constexpr (Store<T>::ES == 4) {
        if (vec) {
            for (int c = l; c < DP / 4; c += nl)
                if (4 * c < D)
                    cp_async16(smem_addr(dst + 4 * c), static_cast<const float *>(p) + off + 4 * c);
                else
                    *reinterpret_cast<float4 *>(dst + 4 * c) = make_float4(0.f, 0.f, 0.f, 0.f);
            return;
        }
    }
    row_to_smem<T, DP>(dst, p, off, D, l, nl, vec);
}

__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(bf16_t *p, float x) {
    // round to nearest even; a NaN keeps its sign and becomes quiet
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(p->bits) : "f"(x));
}

// PREFIX: the keys of shared prefixes, as in the tensor-core kernel.
template <typename T, int DC, bool PREFIX>
__global__ void __launch_bounds__(NT) attn_simt_impl(const __grid_constant__ TreeAttnArgs A) {
    using Walk = typename std::conditional<PREFIX, PrefixWalk, AttnWalk>::type;
    using Piece = typename Walk::Piece;
    constexpr int DP = DC * 64, KS = DP + 4;  // key row stride: rows of a float4 column in different banks
    extern __shared__ __align__(16) unsigned char smem[];
    float *sq = reinterpret_cast<float *>(smem);  // [BM][KS]
    float *sk = sq + BM * KS;                     // [BN][KS]
    float *sv = sk + BN * KS;                     // [BN][DP]
    float *sp = sv + BN * DP;                     // [BM][BN + 4]
    float *sm = sp + BM * (BN + 4);               // [BM] maximum
    float *sl = sm + BM;                          // [BM] sum
    float *sf = sl + BM;                          // [BM] factor of the old rows
    uint64_t *smask = reinterpret_cast<uint64_t *>(sf + BM);  // [MAX_NODES]
    __shared__ int s_flag, s_above[MAX_NODES];
    __shared__ __align__(16) unsigned char s_begin[sizeof(Walk)];

    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int group = blockIdx.x / A.mtiles, mtile = blockIdx.x - group * A.mtiles;
    const int row0 = PREFIX ? 0 : mtile * BM;
    const bool vec = A.vec != 0;

    if (PREFIX || !A.overlap) pdl_wait();
    pdl_next();
    Walk walk;
    const long long W = walk.start(A, group, attn_limit<PREFIX>(A));
    if (tid == 0) *reinterpret_cast<Walk *>(s_begin) = walk;  // for the end
    if (PREFIX && blockIdx.x == 0 && tid < 32) prefix_check_starts(A);
    Piece pc;
    while (walk.next(A, pc)) {
        const int b = pc.b, h = pc.h;
        bool bad_len, bad_nodes = false;
        attn_len(A, b, bad_len);
        int n = 0, rows, rows_n;  // nodes; rows of the tile; rows that are written
        if constexpr (PREFIX) {
            rows = rows_n = pc.rows;
        } else {
            n = attn_nodes(A, b, bad_nodes);
            rows = min(BM, A.rows - row0);
            rows_n = bad_nodes ? A.rows : n * A.G;
        }
        const bool works = 4 * (tid >> 5) < rows;  // a warp has rows 4 w .. 4 w + 3 from the scores to the output
        if (tid == 0) s_flag = (bad_len || bad_nodes) ? F_BAD_ID : 0;
        __syncthreads();
        // This thread's part of the keys or of the values of tile t, one row for
        // four threads; `pid`: the row's page.
        auto page_of = [&](int t) {
            const int pos = t * BN + (tid >> 2);
            return t < pc.t1 && t < pc.prefix && pos < pc.len ? attn_page(A, b, pos / A.page_size) : 0;
        };
        auto fetch = [&](bool values, int t, int pid) {
            const int j = tid >> 2;
            const bool fresh = !PREFIX && t == pc.prefix;
            if (t < pc.t1 && j < (fresh ? n : min(BN, pc.len - t * BN))) {
                const int off = (t * BN + j) % A.page_size;
                const int64_t *cs = values ? A.vcs : A.kcs, *ns = values ? A.vs : A.ks;
                const int64_t from = fresh ? b * ns[0] + j * ns[1] + h * ns[2] : pid * cs[0] + off * cs[1] + h * cs[2];
                const void *src = fresh ? (values ? A.v_new : A.k_new) : (values ? A.v_cache : A.k_cache);
                row_async<T, DP>(values ? sv + j * DP : sk + j * KS, src, from, A.D, tid & 3, 4, vec);
            }
            cp_async_commit();
        };
        int pid = page_of(pc.t0);
        fetch(false, pc.t0, pid);
        fetch(true, pc.t0, pid);
        int bad = 0;
        if constexpr (PREFIX) {
            if (h == 0 && pc.mt == 0 && pc.t0 == 0) bad = attn_check_pages(A, b, pc.len, tid, NT);
        } else {
            bad = attn_check_pages(A, b, pc.len, tid, NT);
        }
        if (!PREFIX && tid < 32) bad |= attn_masks(A.parents ? A.parents + static_cast<size_t>(b) * A.T : nullptr, n, smask, s_above);
        if (bad) atomicOr(&s_flag, bad);
        {
            const int r = tid >> 3;  // 8 threads a row
            int64_t from = 0;
            if constexpr (PREFIX) {
                const int d = node_of(A, pc.rest + r), tok = pc.token + d, s = tok / A.T;
                from = (pc.start + s) * A.qs[0] + (tok - s * A.T) * A.qs[1] + (static_cast<int64_t>(h) * A.G + (pc.rest + r - d * A.G)) * A.qs[2];
            } else {
                const int t = (row0 + r) / A.G, g = row0 + r - t * A.G;
                from = b * A.qs[0] + t * A.qs[1] + (static_cast<int64_t>(h) * A.G + g) * A.qs[2];
            }
            if (r < rows)
                row_to_smem<T, DP>(sq + r * KS, A.q, from, A.D, tid & 7, 8, vec);
            else
                for (int c = tid & 7; c < DP; c += 8) sq[r * KS + c] = 0.f;
        }
        if (tid < BM) {
            sm[tid] = -INFINITY;
            sl[tid] = 0.f;
        }
        float acc[2][DC * 4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < DC * 4; ++c) acc[i][c] = 0.f;

        for (int t = pc.t0; t < pc.t1; ++t) {
            const bool tree = !PREFIX && t == pc.prefix;
            const int valid = tree ? n : min(BN, pc.len - t * BN);
            pid = page_of(t + 1);
            cp_async_wait<1>();  // the keys
            __syncthreads();
            if (works) {
                // scores of rows 2 ty, 2 ty + 1 against keys tx + 16 i
                float s[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[i][c] = 0.f;
                const float *q0 = sq + 2 * ty * KS;
                // each half of the elements on its own: shorter sums lose less
                float half[2][4] = {};
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
#pragma unroll 4
                    for (int d = part * (DP / 2); d < (part + 1) * (DP / 2); d += 4) {
                        const float4 a0 = *reinterpret_cast<const float4 *>(q0 + d);
                        const float4 a1 = *reinterpret_cast<const float4 *>(q0 + KS + d);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float4 k = *reinterpret_cast<const float4 *>(sk + (tx + 16 * c) * KS + d);
                            s[0][c] = fmaf(a0.x, k.x, fmaf(a0.y, k.y, fmaf(a0.z, k.z, fmaf(a0.w, k.w, s[0][c]))));
                            s[1][c] = fmaf(a1.x, k.x, fmaf(a1.y, k.y, fmaf(a1.z, k.z, fmaf(a1.w, k.w, s[1][c]))));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float x = s[i][c];
                            s[i][c] = part ? half[i][c] + x : 0.f;
                            half[i][c] = x;
                        }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 2 * ty + i;
                    const uint64_t see = tree && r < rows && (row0 + r) / A.G < n ? smask[(row0 + r) / A.G] : 0ull;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int j = tx + 16 * c;
                        const bool on = tree ? ((see >> j) & 1ull) != 0 : j < valid;
                        sp[r * (BN + 4) + j] = on ? s[i][c] : -INFINITY;
                    }
                }
            }
            cp_async_wait<0>();  // the values
            __syncthreads();
            fetch(false, t + 1, pid);  // the next keys: on their way from here on
            if (works) {
                {  // softmax: 8 threads a row
                    const int r = tid >> 3, l = tid & 7;
                    float *p = sp + r * (BN + 4);
                    float x[8], top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] = p[l + 8 * i];
                        top = max_nan(top, x[i]);
                    }
#pragma unroll
                    for (int d = 1; d < 8; d <<= 1) top = max_nan(top, __shfl_xor_sync(FULL, top, d));
                    const float m0 = sm[r], m1 = max_nan(m0, top);
                    // (the reference is the rounded product, in the weights and in the
                    // factor of the old ones alike: the exact product in one of the two
                    // would put them 2^-24 of a score's size apart at every new maximum)
                    const float ref = m1 == -INFINITY ? 0.f : __fmul_rn(m1, A.scale_log2);
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] = exp2f(fmaf(x[i], A.scale_log2, -ref));
                        p[l + 8 * i] = x[i];
                        sum += x[i];
                    }
#pragma unroll
                    for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(FULL, sum, d);
                    __syncwarp();
                    if (l == 0) {
                        const float f = m0 == -INFINITY ? 0.f : exp2f(__fsub_rn(__fmul_rn(m0, A.scale_log2), ref));
                        sf[r] = f;
                        sl[r] = sl[r] * f + sum;
                        sm[r] = m1;
                    }
                }
                __syncwarp();
                {  // outputs of rows 2 ty, 2 ty + 1, columns 64 c + 4 tx ..
                    const float f0 = sf[2 * ty], f1 = sf[2 * ty + 1];
                    uint64_t see0 = ~0ull, see1 = ~0ull;
                    if (tree) {  // a node that a row does not see never reaches it, not even as 0 times infinity
                        const int r = row0 + 2 * ty, t0 = r / A.G, t1 = (r + 1) / A.G;
                        see0 = 2 * ty < rows && t0 < n ? smask[t0] : 0ull;
                        see1 = 2 * ty + 1 < rows && t1 < n ? smask[t1] : 0ull;
                    }
                    // a tile's sums on their own first: one sum over all keys of a long
                    // text would lose twice what the shorter ones do
                    float add[2][DC * 4];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int c = 0; c < DC * 4; ++c) add[i][c] = 0.f;
                    const float *p0 = sp + 2 * ty * (BN + 4), *p1 = p0 + BN + 4;
                    int j = 0;
                    if (!tree) {  // four keys at a time
#pragma unroll 2
                        for (; j + 4 <= valid; j += 4) {
                            const float4 wa = *reinterpret_cast<const float4 *>(p0 + j), wb = *reinterpret_cast<const float4 *>(p1 + j);
                            const float w0[4] = {wa.x, wa.y, wa.z, wa.w}, w1[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
#pragma unroll
                                for (int c = 0; c < DC; ++c) {
                                    const float4 v = *reinterpret_cast<const float4 *>(sv + (j + e) * DP + 64 * c + 4 * tx);
                                    add[0][4 * c] = fmaf(w0[e], v.x, add[0][4 * c]);
                                    add[0][4 * c + 1] = fmaf(w0[e], v.y, add[0][4 * c + 1]);
                                    add[0][4 * c + 2] = fmaf(w0[e], v.z, add[0][4 * c + 2]);
                                    add[0][4 * c + 3] = fmaf(w0[e], v.w, add[0][4 * c + 3]);
                                    add[1][4 * c] = fmaf(w1[e], v.x, add[1][4 * c]);
                                    add[1][4 * c + 1] = fmaf(w1[e], v.y, add[1][4 * c + 1]);
                                    add[1][4 * c + 2] = fmaf(w1[e], v.z, add[1][4 * c + 2]);
                                    add[1][4 * c + 3] = fmaf(w1[e], v.w, add[1][4 * c + 3]);
                                }
                        }
                    }
                    for (; j < valid; ++j) {
                        const float w0 = p0[j], w1 = p1[j];
                        const bool on0 = (see0 >> j) & 1ull, on1 = (see1 >> j) & 1ull;
#pragma unroll
                        for (int c = 0; c < DC; ++c) {
                            const float4 v = *reinterpret_cast<const float4 *>(sv + j * DP + 64 * c + 4 * tx);
                            if (on0) {
                                add[0][4 * c] = fmaf(w0, v.x, add[0][4 * c]);
                                add[0][4 * c + 1] = fmaf(w0, v.y, add[0][4 * c + 1]);
                                add[0][4 * c + 2] = fmaf(w0, v.z, add[0][4 * c + 2]);
                                add[0][4 * c + 3] = fmaf(w0, v.w, add[0][4 * c + 3]);
                            }
                            if (on1) {
                                add[1][4 * c] = fmaf(w1, v.x, add[1][4 * c]);
                                add[1][4 * c + 1] = fmaf(w1, v.y, add[1][4 * c + 1]);
                                add[1][4 * c + 2] = fmaf(w1, v.z, add[1][4 * c + 2]);
                                add[1][4 * c + 3] = fmaf(w1, v.w, add[1][4 * c + 3]);
                            }
                        }
                    }
#pragma unroll
                    for (int c = 0; c < DC * 4; ++c) {
                        acc[0][c] = fmaf(acc[0][c], f0, add[0][c]);
                        acc[1][c] = fmaf(acc[1][c], f1, add[1][c]);
                    }
                }
            }
            __syncthreads();
            fetch(true, t + 1, pid);
        }

        const int flag = s_flag;
        if constexpr (PREFIX) {
            if (tid == 0 && h == 0 && pc.mt == 0 && pc.t0 == 0) A.flags[b] = flag;
        } else {
            if (A.flags && tid == 0 && h == 0 && mtile == 0) A.flags[b] = flag;
        }
        const bool whole = pc.whole();
        float *slot = whole ? nullptr : A.part + attn_slot(A, group, mtile, pc.first) * attn_slot_floats(BM, A.D);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 2 * ty + i;
            if (row0 + r >= rows_n || r >= rows) continue;
            const float l = flag ? NAN : sl[r];
            if (!PREFIX && whole && !A.row_o) {
                const int t = (row0 + r) / A.G, hq = h * A.G + row0 + r - t * A.G;
                const size_t at = (static_cast<size_t>(b) * A.T + t) * A.Hq + hq;
                const float inv = 1.f / l;
                T *o = static_cast<T *>(A.out) + at * A.D;
#pragma unroll
                for (int c = 0; c < DC * 4; ++c) {
                    const int d = 64 * (c >> 2) + 4 * tx + (c & 3);
                    if (d < A.D) put(o + d, acc[i][c] * inv);
                }
                if (A.lse && tx == 0) A.lse[at] = (sm[r] * A.scale_log2 + log2f(l)) * LN2;
            } else {
                const size_t place = unit_row(A, pc) + row0 + r;
                float *o = whole ? A.row_o + place * A.D : slot + 2 * BM + static_cast<size_t>(r) * A.D;
#pragma unroll
                for (int c = 0; c < DC * 4; ++c) {
                    const int d = 64 * (c >> 2) + 4 * tx + (c & 3);
                    if (d < A.D) o[d] = acc[i][c];
                }
                if (tx == 0) {
                    *(whole ? A.row_m + place : slot + r) = sm[r] * A.scale_log2;
                    *(whole ? A.row_l + place : slot + BM + r) = l;
                }
            }
        }
        __syncthreads();
    }
    if (mtile == 0 && tid == 0) attn_report(A, group, W, *reinterpret_cast<const Walk *>(s_begin));
    if (!PREFIX && A.overlap && blockIdx.x == 0) pdl_wait();  // the join waits for this kernel, and so for the one before
}

// Join one unit that begins in group blockIdx.x / mtiles and goes on in the
// next groups: with m the largest of the parts' maxima, o = sum_i 2^(m_i - m)
// o_i / sum_i 2^(m_i - m) l_i, the parts in the order of their keys.  A warp
// takes one row and lane i the columns 4 i ..; the maxima and sums of 32 parts
// are loaded by the 32 lanes at once and handed round, and the rows of several
// parts are on their way at a time: what bounds this kernel is the time of a
// load, not their number (a row of 20 parts read one after the other took 30
// us).  bfloat16 has many rows of few parts: four at a time, few registers and
// many warps on an SM (trees of 64 nodes: with four 262 us, with eight 267, with
// sixteen 278).  float32 has more and smaller CTAs, so more parts: sixteen (4 sequences
// of 2501: 22.0 us with four, 20.3 with eight, 19.6 with sixteen).

template <typename T, int NQ>
__global__ void __launch_bounds__(JOIN_THREADS, Store<T>::ES == 4 ? 5 : 10) attn_join_impl(const __grid_constant__ TreeAttnArgs A) {
    constexpr int AHEAD = Store<T>::ES == 4 ? 16 / NQ : 4;
    pdl_wait();
    pdl_next();
    const int group = blockIdx.x / A.mtiles, mtile = blockIdx.x - group * A.mtiles;
    const int4 d = *reinterpret_cast<const int4 *>(A.desc + static_cast<size_t>(group) * ATTN_DESC);
    const int b = d.x, h = d.y, parts = d.z;
    if (parts == 0) return;
    bool bad;
    const int n = attn_nodes(A, b, bad);
    const int r = blockIdx.y * JOIN_ROWS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r >= min(A.bm, (bad ? A.rows : n * A.G) - mtile * A.bm)) return;
    const size_t slot_floats = attn_slot_floats(A.bm, A.D);
    const float *first = A.part + attn_slot(A, group, mtile, d.w == 0) * slot_floats;
    const float *next = A.part + attn_slot(A, group + 1, mtile, true) * slot_floats;
    const size_t step = 2 * slot_floats * A.mtiles;
    auto part = [&](int k) { return k == 0 ? first : next + (k - 1) * step; };
    float top = -INFINITY;
    for (int k = lane; k < parts; k += 32) top = max_nan(top, part(k)[r]);
#pragma unroll
    for (int e = 1; e < 32; e <<= 1) top = max_nan(top, __shfl_xor_sync(FULL, top, e));
    const float ref = top == -INFINITY ? 0.f : top;
    float l = 0.f, o[NQ][4] = {};
    const bool quads = A.D % 4 == 0;  // (rows of part results start on 16 bytes then)
    for (int k0 = 0; k0 < parts; k0 += 32) {
        float w = 0.f;
        if (k0 + lane < parts) {
            const float *s = part(k0 + lane);
            w = exp2f(s[r] - ref);
            l = fmaf(w, s[A.bm + r], l);
        }
        const int here = min(32, parts - k0);
        for (int i0 = 0; i0 < here; i0 += AHEAD) {
            float4 x[AHEAD][NQ];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    const int c = 4 * lane + 128 * q;
                    x[i][q] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i0 + i >= here || c >= A.D) continue;
                    const float *s = part(k0 + i0 + i) + 2 * A.bm + static_cast<size_t>(r) * A.D + c;
                    if (quads)
                        x[i][q] = *reinterpret_cast<const float4 *>(s);
                    else
                        x[i][q] = make_float4(s[0], c + 1 < A.D ? s[1] : 0.f, c + 2 < A.D ? s[2] : 0.f, c + 3 < A.D ? s[3] : 0.f);
                }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const float wi = __shfl_sync(FULL, w, (i0 + i) & 31);
                if (i0 + i >= here) continue;
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    o[q][0] = fmaf(wi, x[i][q].x, o[q][0]);
                    o[q][1] = fmaf(wi, x[i][q].y, o[q][1]);
                    o[q][2] = fmaf(wi, x[i][q].z, o[q][2]);
                    o[q][3] = fmaf(wi, x[i][q].w, o[q][3]);
                }
            }
        }
    }
    l = warp_allsum(l);
    const int row = mtile * A.bm + r, t = row / A.G, hq = h * A.G + row - t * A.G;
    const size_t at = (static_cast<size_t>(b) * A.T + t) * A.Hq + hq;
    const float inv = 1.f / l;
    T *out = static_cast<T *>(A.out) + at * A.D;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = 4 * lane + 128 * q + e;
            if (c < A.D) put(out + c, o[q][e] * inv);
        }
    if (A.lse && lane == 0) A.lse[at] = (ref + log2f(l)) * LN2;
}

// Join of a sequence's own parts (A) with those of its prefix (S), both from
// the kernels above: eight lanes take one row of the output, find the row's two
// units and join their parts in their order, the prefix's first.  What bounds it
// is a chain of loads (units and flags, then references, sums and rows): with a
// warp to a row 8192 rows were two and a half rounds of it, now they are one.
template <typename T, int NQ>
__global__ void __launch_bounds__(JOIN_THREADS) prefix_join_impl(const __grid_constant__ TreeAttnArgs A, const __grid_constant__ TreeAttnArgs S) {
    constexpr int LANES = 8, AHEAD = NQ <= 4 ? 2 : 1;
    pdl_next();
    const int lane = threadIdx.x & (LANES - 1), shift = threadIdx.x & 24;  // in the row's lanes; theirs in the warp
    // (the call's rows are counted in 31 bits)
    const uint32_t rows = static_cast<uint32_t>(A.B) * A.T * A.Hq, mine = (blockIdx.x * JOIN_THREADS + threadIdx.x) / LANES;
    const bool there = mine < rows;
    const uint32_t row_out = there ? mine : rows - 1, token = row_out / A.Hq;
    const size_t at = row_out;
    const int hq = static_cast<int>(row_out - token * A.Hq), b = static_cast<int>(token / A.T), t = static_cast<int>(token - static_cast<uint32_t>(b) * A.T);
    const int h = hq / A.G, g = hq - h * A.G;
    // The call's inputs were there before its first kernel: they are read before
    // the second is done.
    bool bad_nodes;
    const int n = attn_nodes(A, b, bad_nodes);
    // the sequence's prefix: the last that starts at or before it, 8 guesses at a time
    int lo = 0, hi = S.B;
    while (__any_sync(FULL, hi - lo > 1)) {
        const int stride = (hi - lo + LANES - 1) / LANES, i = lo + lane * stride;
        const uint32_t under = (__ballot_sync(FULL, i < hi && __ldg(S.starts + i) <= b) >> shift) & 255u;
        const int last = under ? 31 - __clz(under) : 0;
        hi = min(hi, lo + (last + 1) * stride);
        lo += last * stride;
    }
    // (in bounds whatever the starts hold)
    int group;
    const int p = lo, first = prefix_group(S, p, group);
    bool bad_len;
    const int plen = attn_len(S, p, bad_len);
    const bool inside = b >= first && b < first + group, shared = plen > 0 && inside;
    const int row = t * A.G + g;
    const size_t own_at = static_cast<size_t>(b) * A.Hkv + h;
    int mt = 0, prow = 0;
    size_t pre_at = 0;
    if (shared) {
        const uint32_t r = static_cast<uint32_t>(b - first) * A.rows + row;
        mt = static_cast<int>(r / static_cast<uint32_t>(S.tile_rows));
        prow = static_cast<int>(r - static_cast<uint32_t>(mt) * S.tile_rows);
        pre_at = prefix_unit(S, p, static_cast<uint32_t>(first) * A.rows, mt, h);
    }
    pdl_wait();
    const int2 own_unit = A.units[own_at], pre_unit = shared ? S.units[pre_at] : make_int2(0, 0);
    int flag = A.flags[b] | (*S.bad_starts || bad_len || !inside ? F_BAD_ID : 0);
    if (shared) flag |= S.flags[p];
    if (there && t == 0 && hq == 0 && A.flags_out && lane == 0) A.flags_out[b] = flag;
    const bool live = there && t < (bad_nodes ? A.T : n);
    T *out = static_cast<T *>(A.out) + at * A.D;
    if (live && flag) {
        for (int c = lane; c < A.D; c += LANES) put(out + c, NAN);
        if (A.lse && lane == 0) A.lse[at] = NAN;
    }
    // a row's parts: of a whole unit one, by rows; else one in a slot of each group
    struct Parts {
        const float *m, *o;    // the first part's maximum and row
        long long l;           // from the maximum to the sum
        long long next, step;  // from the first part to the second, if there is one; from each to the next
        int n;
    };
    auto parts_of = [&](const TreeAttnArgs &X, int2 u, size_t place, int mtile, int r) {
        Parts q = {};
        if (u.x == 0) {
            q.m = X.row_m + place;
            q.l = X.row_l - X.row_m;
            q.o = X.row_o + place * X.D;
            q.n = 1;
            return q;
        }
        const long long slot = static_cast<long long>(attn_slot_floats(X.bm, X.D));
        const int group = u.y >> 1;
        const float *start = X.part + attn_slot(X, group, mtile, (u.y & 1) == 0) * slot;
        q.m = start + r;
        q.l = X.bm;
        q.o = start + 2 * X.bm + static_cast<long long>(r) * X.D;
        q.next = X.part + attn_slot(X, group + 1, mtile, true) * slot - start;
        q.step = 2 * slot * X.mtiles;
        q.n = u.x;
        return q;
    };
    Parts own = {}, pre = {};
    if (live && !flag) {
        own = parts_of(A, own_unit, own_at * A.rows + row, row / A.bm, row % A.bm);
        if (shared) pre = parts_of(S, pre_unit, pre_at * S.tile_rows + prow, 0, prow);
    }
    const int parts = pre.n + own.n;
    auto far = [&](const Parts &q, int k) { return k == 0 ? 0ll : q.next + (k - 1) * q.step; };
    auto m_of = [&](int k) { return k < pre.n ? pre.m + far(pre, k) : own.m + far(own, k - pre.n); };
    auto o_of = [&](int k) { return k < pre.n ? pre.o + far(pre, k) : own.o + far(own, k - pre.n); };
    // Weights of eight parts at a time, relative to the largest reference so far;
    // the rows of the first parts are on their way while those are found.
    float top = -INFINITY, l = 0.f, o[NQ][4] = {};
    const bool quads = A.D % 4 == 0;
    for (int k0 = 0; __any_sync(FULL, k0 < parts); k0 += LANES) {
        float4 x[AHEAD][NQ];
        auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const float *from = k0 + i0 + i < parts ? o_of(k0 + i0 + i) : nullptr;
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    const int c = 4 * lane + 4 * LANES * q;
                    x[i][q] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (!from || c >= A.D) continue;
                    const float *s = from + c;
                    if (quads)
                        x[i][q] = *reinterpret_cast<const float4 *>(s);
                    else
                        x[i][q] = make_float4(s[0], c + 1 < A.D ? s[1] : 0.f, c + 2 < A.D ? s[2] : 0.f, c + 3 < A.D ? s[3] : 0.f);
                }
            }
        };
        float m = -INFINITY, sum = 0.f;
        if (k0 + lane < parts) {
            const float *at_m = m_of(k0 + lane);
            m = at_m[0];
            sum = at_m[k0 + lane < pre.n ? pre.l : own.l];
        }
        load(0);
        float here = m;
#pragma unroll
        for (int e = 1; e < LANES; e <<= 1) here = max_nan(here, __shfl_xor_sync(FULL, here, e));
        here = max_nan(here, top);
        const float ref = here == -INFINITY ? 0.f : here, old = top == -INFINITY ? 0.f : exp2f(top - ref);
        top = here;
        const float w = k0 + lane < parts ? exp2f(m - ref) : 0.f;
        l = fmaf(w, sum, l * old);
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[q][e] *= old;
#pragma unroll
        for (int i0 = 0; i0 < LANES; i0 += AHEAD) {
            if (!__any_sync(FULL, k0 + i0 < parts)) break;
            if (i0 > 0) load(i0);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const float wi = __shfl_sync(FULL, w, i0 + i, LANES);
                if (k0 + i0 + i >= parts) continue;
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    o[q][0] = fmaf(wi, x[i][q].x, o[q][0]);
                    o[q][1] = fmaf(wi, x[i][q].y, o[q][1]);
                    o[q][2] = fmaf(wi, x[i][q].z, o[q][2]);
                    o[q][3] = fmaf(wi, x[i][q].w, o[q][3]);
                }
            }
        }
    }
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int e = 1; e < LANES; e <<= 1) l += __shfl_xor_sync(FULL, l, e);
    if (!live || flag) return;
    const float inv = 1.f / l;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        const int c = 4 * lane + 4 * LANES * q;
        if (c >= A.D) break;
        if (A.wide_out) {
            if constexpr (Store<T>::ES == 4)
                *reinterpret_cast<float4 *>(out + c) = make_float4(o[q][0] * inv, o[q][1] * inv, o[q][2] * inv, o[q][3] * inv);
            else {
                uint2 y;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y.x) : "f"(o[q][1] * inv), "f"(o[q][0] * inv));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y.y) : "f"(o[q][3] * inv), "f"(o[q][2] * inv));
                *reinterpret_cast<uint2 *>(out + c) = y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < A.D) put(out + c + e, o[q][e] * inv);
        }
    }
    if (A.lse && lane == 0) A.lse[at] = (ref + log2f(l)) * LN2;
}

}  // namespace

uint32_t attn_simt_smem(int D) {
    const int dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
    const size_t f = static_cast<size_t>(BM) * (dp + 4) + BN * (dp + 4) + BN * dp + BM * (BN + 4) + 3 * BM;
    return static_cast<uint32_t>(f * 4 + MAX_NODES * 8);
}

namespace {
template <typename T, bool PREFIX>
const void *pick(int D) {
    return D <= 64    ? reinterpret_cast<const void *>(attn_simt_impl<T, 1, PREFIX>)
           : D <= 128 ? reinterpret_cast<const void *>(attn_simt_impl<T, 2, PREFIX>)
                      : reinterpret_cast<const void *>(attn_simt_impl<T, 4, PREFIX>);
}
}  // namespace

const void *attn_simt_func(int dtype, int D, bool prefix) {
    if (dtype == 0) return prefix ? pick<float, true>(D) : pick<float, false>(D);
    return prefix ? pick<bf16_t, true>(D) : pick<bf16_t, false>(D);
}

namespace {
template <typename T>
const void *pick_join(int D) {
    return D <= 64    ? reinterpret_cast<const void *>(prefix_join_impl<T, 2>)
           : D <= 128 ? reinterpret_cast<const void *>(prefix_join_impl<T, 4>)
                      : reinterpret_cast<const void *>(prefix_join_impl<T, 8>);
}
}  // namespace

const void *prefix_join_func(int dtype, int D) { return dtype == 0 ? pick_join<float>(D) : pick_join<bf16_t>(D); }

const void *attn_join_func(int dtype, int D) {
    if (D <= 128)
        return dtype == 0 ? reinterpret_cast<const void *>(attn_join_impl<float, 1>)
                          : reinterpret_cast<const void *>(attn_join_impl<bf16_t, 1>);
    return dtype == 0 ? reinterpret_cast<const void *>(attn_join_impl<float, 2>)
                      : reinterpret_cast<const void *>(attn_join_impl<bf16_t, 2>);
}

}  // namespace mtp
