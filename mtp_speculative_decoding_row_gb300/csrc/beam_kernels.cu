// beam_kernels.cu -- the best K continuations of a sequence's W beams over a
// vocabulary of V: score(w, v) = scores[w] + ln softmax(z_w / T)(v), the K
// largest, equal ones by the smaller (w, v).
//
// Every logit is read once.  A row is cut into parts, one CTA each; a part
// yields its maximum, its sum of 2^((z - max) k) with k = log2(e) / T, and
// its own K best logits (within a row the order of the scores is that of the
// logits).  A second launch turns the parts' candidates into scores in
// float64 -- candidates of two beams may lie closer than float32 tells apart
// -- and merges the sorted lists.
//
// A part keeps its candidates in shared memory as 64-bit keys: the logit's
// bits in an order-preserving form, then the complement of the index, so one
// integer comparison orders by value and then by smaller index.  The K-th
// largest of the threads' maxima over the first 4 vectors each bounds the
// K-th best from below; what follows is compared with that bound vector by
// vector (one comparison for 8 bf16 logits), and few pass.  When the list is
// full it is cut to its K best and the bound rises.
//
// Rows may start on any element.  A vector is always elements [8 j, 8 j + 8)
// (4 j of float32) of the row, put together from two aligned loads where the
// row is not aligned, so the order of the sums -- and with it the last bit of
// a normaliser -- does not depend on where a row lies: equal rows get equal
// scores and their ties go to the smaller beam.
#include "common.cuh"
#include "tree.h"

namespace mtp {
namespace {

constexpr int NT = BEAM_THREADS;
constexpr int UN = 4;        // vectors of a thread per round
constexpr int CAP = 2048;    // candidates held by a part

// Order-preserving bits of a float (the two zeros are equal).
__device__ __forceinline__ uint32_t order_bits(float z) {
    const uint32_t u = __float_as_uint(z + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_float(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ uint64_t make_key(float z, int v) {
    return (static_cast<uint64_t>(order_bits(z)) << 32) | static_cast<uint32_t>(~v);
}

// 16 bytes at byte `sh` of the 32 bytes a, b.
__device__ __forceinline__ uint4 realign(const uint4 &a, const uint4 &b, uint32_t sh) {
    const uint32_t bs = (sh & 3u) * 8u;
    switch (sh >> 2) {
        case 0:
            return make_uint4(__funnelshift_r(a.x, a.y, bs), __funnelshift_r(a.y, a.z, bs), __funnelshift_r(a.z, a.w, bs),
                              __funnelshift_r(a.w, b.x, bs));
        case 1:
            return make_uint4(__funnelshift_r(a.y, a.z, bs), __funnelshift_r(a.z, a.w, bs), __funnelshift_r(a.w, b.x, bs),
                              __funnelshift_r(b.x, b.y, bs));
        case 2:
            return make_uint4(__funnelshift_r(a.z, a.w, bs), __funnelshift_r(a.w, b.x, bs), __funnelshift_r(b.x, b.y, bs),
                              __funnelshift_r(b.y, b.z, bs));
        default:
            return make_uint4(__funnelshift_r(a.w, b.x, bs), __funnelshift_r(b.x, b.y, bs), __funnelshift_r(b.y, b.z, bs),
                              __funnelshift_r(b.z, b.w, bs));
    }
}

template <typename T>
__device__ __forceinline__ uint4 minus_inf_vec() {
    const uint32_t w = Store<T>::ES == 2 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(w, w, w, w);
}

// Vector j of a row (elements j VEC ..), -inf beyond the row's V elements.
template <typename T>
__device__ __forceinline__ uint4 row_vec(const unsigned char *row, uint32_t sh, int j, int V) {
    constexpr int VEC = Store<T>::VEC, ES = Store<T>::ES;
    if ((j + 1) * VEC <= V) {
        const uint4 *a = reinterpret_cast<const uint4 *>(row - sh) + j;
        if (sh == 0) return __ldg(a);
        return realign(__ldg(a), __ldg(a + 1), sh);  // the row's bytes reach into the second load
    }
    uint32_t w[4] = {minus_inf_vec<T>().x, minus_inf_vec<T>().x, minus_inf_vec<T>().x, minus_inf_vec<T>().x};
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        if (j * VEC + e >= V) break;
        if (ES == 4)
            w[e] = __ldg(reinterpret_cast<const uint32_t *>(row) + j * VEC + e);
        else {
            const uint32_t x = __ldg(reinterpret_cast<const unsigned short *>(row) + j * VEC + e);
            w[e / 2] = (e & 1) ? (w[e / 2] & 0x0000ffffu) | (x << 16) : (w[e / 2] & 0xffff0000u) | x;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Keys of the vectors in `raw` that beat `bound` go into the list; `dup` > 0:
// except those among its first `dup` entries (a round that is done again).
template <typename T>
__device__ __forceinline__ void offer(const uint4 (&raw)[UN], const int (&at)[UN], uint64_t bound, uint64_t *list, int *count,
                                      int dup) {
    constexpr int VEC = Store<T>::VEC;
    const float zb = order_float(static_cast<uint32_t>(bound >> 32));
#pragma unroll
    for (int u = 0; u < UN; ++u) {
        if (!(Store<T>::vmax(raw[u]) >= zb)) continue;
        float z[VEC];
        Store<T>::unpack(raw[u], z);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (!(z[e] >= zb) || z[e] == -INFINITY) continue;
            const uint64_t key = make_key(z[e], at[u] * VEC + e);
            if (key < bound) continue;
            bool seen = false;
            for (int i = 0; i < dup; ++i) seen |= list[i] == key;
            if (seen) continue;
            const int i = atomicAdd(count, 1);
            if (i < CAP) list[i] = key;
        }
    }
}

// Cut list[0 .. n) to its `keep` largest, sorted: each key's rank is the
// number of larger ones (keys differ).  All threads call it.
__device__ __forceinline__ int cut(uint64_t *list, int n, int keep, uint64_t *tmp) {
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += NT) {
        const uint64_t key = list[i];
        int rank = 0;
        int j = 0;
        for (; j + 4 <= n && rank < keep; j += 4)
            rank += (list[j] > key) + (list[j + 1] > key) + (list[j + 2] > key) + (list[j + 3] > key);
        if (j + 4 > n)
            for (; j < n; ++j) rank += list[j] > key;
        if (rank < keep) tmp[rank] = key;
    }
    __syncthreads();
    const int m = min(n, keep);
    for (int i = threadIdx.x; i < m; i += NT) list[i] = tmp[i];
    __syncthreads();
    return m;
}

template <typename T>
__global__ void __launch_bounds__(NT) beam_part_impl(const __grid_constant__ BeamArgs A) {
    constexpr int VEC = Store<T>::VEC, ES = Store<T>::ES;
    __shared__ uint64_t list[CAP];
    __shared__ uint64_t tmp[BEAM_MAX_K];
    __shared__ uint64_t tops[NT];
    __shared__ int s_count, s_bad;
    __shared__ float s_m[NT / 32];
    __shared__ double s_s[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / A.parts, part = blockIdx.x - row * A.parts;
    const int b = row / A.W;
    const size_t slot = static_cast<size_t>(row) * A.parts + part;
    float *cz = A.cand_z + slot * A.KL;
    int *cv = A.cand_v + slot * A.KL;
    const float temp = __ldg(A.temp + b), score = __ldg(A.scores + row);
    if (!(temp > 0.f) || temp == INFINITY || !(score < INFINITY) || score == -INFINITY) {
        // a dead beam, or a sequence that the join flags: its logits are not read
        if (tid == 0) {
            A.part_max[slot] = -INFINITY;
            A.part_sum[slot] = 0.0;
            A.part_flag[slot] = 0;
        }
        for (int i = tid; i < A.KL; i += NT) cv[i] = -1;
        return;
    }
    // k in two floats: a row's sum is corrected for the rounding of k (below)
    const double kd = 1.4426950408889634 / static_cast<double>(temp);
    const float k = static_cast<float>(kd), dk = static_cast<float>(kd - static_cast<double>(k));
    const unsigned char *base = static_cast<const unsigned char *>(A.logits) + static_cast<size_t>(row) * A.V * ES;
    const uint32_t sh = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(base) & 15u);
    const int j0 = part * (A.part_elems / VEC);
    const int j1 = min((A.V + VEC - 1) / VEC, j0 + A.part_elems / VEC);
    if (tid == 0) s_count = s_bad = 0;

    // sums of e_i = 2^(z_i k - mk) and of e_i z_i, where mk = m k rounded
    float m = -INFINITY, mk = 0.f, s = 0.f, s1 = 0.f;
    const uint64_t K2 = f2pack(k, k);
    uint64_t bound = static_cast<uint64_t>(order_bits(-INFINITY)) << 32;
    int count = 0;
    for (int j = j0; j < j1; j += NT * UN) {
        uint4 raw[UN];
        int at[UN];
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            at[u] = j + u * NT + tid;
            raw[u] = at[u] < j1 ? row_vec<T>(base, sh, at[u], A.V) : minus_inf_vec<T>();
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) top = max_nan(top, Store<T>::vmax(raw[u]));
        if (!(top <= m)) {  // a new maximum of this thread, or NaN
            if (!(top < INFINITY)) {
                s_bad = 1;  // the join flags the sequence; nothing of this thread counts
#pragma unroll
                for (int u = 0; u < UN; ++u) raw[u] = minus_inf_vec<T>();
                top = -INFINITY;
            } else {
                const float f = m == -INFINITY ? 0.f : ex2(mk - top * k);
                m = top;
                mk = top * k;
                s *= f;
                s1 *= f;
            }
        }
        if (m > -INFINITY) {
            const uint64_t N2 = f2pack(-mk, -mk);
            uint64_t acc = f2pack(0.f, 0.f), acc1 = acc;
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    // -inf becomes the lowest finite number: e = 0 then, and e z = 0
                    uint64_t z2;
                    if (ES == 2)
                        z2 = bf16pair_f2(bmax2_nan(w[e], 0xff7fff7fu));
                    else
                        z2 = f2pack(fmaxf(__uint_as_float(w[2 * e & 3]), -3.0e38f), fmaxf(__uint_as_float(w[(2 * e + 1) & 3]), -3.0e38f));
                    float d0, d1;
                    f2unpack(f2fma(z2, K2, N2), d0, d1);
                    const uint64_t e2 = f2pack(ex2(d0), ex2(d1));
                    acc = f2add(acc, e2);
                    acc1 = f2fma(e2, z2, acc1);
                }
            }
            float a0, a1;
            f2unpack(acc, a0, a1);
            s += a0 + a1;
            f2unpack(acc1, a0, a1);
            s1 += a0 + a1;
        }
        if (j == j0) {
            // the KL-th largest of the threads' maxima: KL logits are at least as large
            const uint64_t mine = (static_cast<uint64_t>(order_bits(top)) << 32) | static_cast<uint32_t>(tid);
            tops[tid] = mine;
            __syncthreads();
            int rank = 0;
            for (int i = 0; i < NT; ++i) rank += tops[i] > mine;
            if (rank == A.KL - 1) tmp[0] = static_cast<uint64_t>(order_bits(top)) << 32;
            __syncthreads();
            bound = tmp[0];
        }
        // offer this round's logits; cut the list and do the round again when it overflows
        for (int dup = 0;;) {
            offer<T>(raw, at, bound, list, &s_count, dup);
            __syncthreads();
            count = s_count;
            __syncthreads();
            if (count <= CAP) break;
            dup = cut(list, CAP, A.KL, tmp);
            bound = list[dup - 1];
            if (tid == 0) s_count = dup;
            __syncthreads();
        }
    }
    __syncthreads();
    const int n = cut(list, count, A.KL, tmp);
    for (int i = tid; i < A.KL; i += NT) {
        cz[i] = i < n ? order_float(static_cast<uint32_t>(list[i] >> 32)) : -INFINITY;
        cv[i] = i < n ? static_cast<int>(~static_cast<uint32_t>(list[i])) : -1;
    }
    float top = warp_allmax(m);
    if (lane == 0) s_m[warp] = top;
    __syncthreads();
    top = -INFINITY;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) top = fmaxf(top, s_m[w]);
    // 2^((z_i - m) kd) = e_i 2^(z_i dk + mk - m kd), and the second factor is
    // 1 + (z_i dk + mk - m kd) ln 2 to within its square (1e-12)
    float sum = 0.f;
    if (m > -INFINITY) {
        const float off = -fmaf(m, k, -mk) - m * dk;
        sum = fmaf(LN2, fmaf(off, s, dk * s1), s) * ex2((m - top) * k);
    }
    sum = warp_allsum(sum);
    if (lane == 0) s_s[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        double t = 0.0;
        for (int w = 0; w < NT / 32; ++w) t += s_s[w];
        A.part_max[slot] = top;
        A.part_sum[slot] = t;
        A.part_flag[slot] = s_bad;
    }
}

// Order-preserving integer of a double (float64 comparisons are slow here).
__device__ __forceinline__ long long order_double(double x) {
    const long long u = __double_as_longlong(x + 0.0);
    return u < 0 ? u ^ 0x7fffffffffffffffll : u;
}

// One CTA per sequence: thread i holds the head of sorted list i = (beam,
// part); each round takes the best head (equal scores: the smaller list, and
// so the smaller beam and index) and moves its list on.
__global__ void __launch_bounds__(NT) beam_join_impl(const __grid_constant__ BeamArgs A) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float s_max[BEAM_MAX_W];
    __shared__ double s_off[BEAM_MAX_W];  // scores[w] - ln sum
    __shared__ int s_flag;
    __shared__ long long s_key[2][NT / 32];
    __shared__ int s_who[2][NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
    const int lists = A.W * A.parts;
    const float temp = __ldg(A.temp + b);
    const bool bad_temp = !(temp > 0.f) || temp == INFINITY;
    if (tid == 0) s_flag = bad_temp ? F_BAD_TEMP : 0;
    __syncthreads();
    if (tid < A.W) {
        const int row = b * A.W + tid;
        const float score = __ldg(A.scores + row);
        const size_t p0 = static_cast<size_t>(row) * A.parts;
        float top = -INFINITY;
        int bad = 0;
        for (int p = 0; p < A.parts; ++p) {
            top = fmaxf(top, A.part_max[p0 + p]);
            bad |= A.part_flag[p0 + p];
        }
        const float k = LOG2E / temp;
        double sum = 0.0;
        for (int p = 0; p < A.parts; ++p)
            if (A.part_max[p0 + p] > -INFINITY) sum += A.part_sum[p0 + p] * ex2((A.part_max[p0 + p] - top) * k);
        s_max[tid] = top;
        // a dead beam has no candidates; a live one with no finite logit is an error
        const bool dead = score == -INFINITY;
        s_off[tid] = dead || top == -INFINITY ? 0.0 : static_cast<double>(score) - log(sum);
        if (!bad_temp && (bad || !(score < INFINITY) || (!dead && top == -INFINITY))) atomicOr(&s_flag, F_NONFINITE);
    }
    __syncthreads();
    const int flag = s_flag;
    if (A.flags && tid == 0) A.flags[b] = flag;
    int32_t *tokens = A.tokens + static_cast<size_t>(b) * A.K, *parents = A.parents + static_cast<size_t>(b) * A.K;
    float *best = A.best + static_cast<size_t>(b) * A.K;
    if (flag) {
        for (int i = tid; i < A.K; i += NT) {
            tokens[i] = parents[i] = -1;
            best[i] = NAN;
        }
        return;
    }
    constexpr long long NONE = -0x7fffffffffffffffll - 1;
    const double inv_t = 1.0 / static_cast<double>(temp);
    const int w = tid / A.parts;
    const size_t at = (static_cast<size_t>(b) * lists + tid) * A.KL;
    int pos = 0, v = -1;
    double x = 0.0;
    long long key = NONE;
    auto load = [&]() {
        key = NONE;
        if (tid >= lists || pos >= A.KL) return;
        v = A.cand_v[at + pos];
        if (v < 0) return;
        x = s_off[w] + static_cast<double>(A.cand_z[at + pos] - s_max[w]) * inv_t;
        key = order_double(x);
    };
    load();
    for (int i = 0; i < A.K; ++i) {
        long long top = key;
        int who = tid;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_down_sync(FULL, top, d);
            const int ow = __shfl_down_sync(FULL, who, d);
            if (lane + d < 32 && o > top) {  // the lower lane keeps a tie
                top = o;
                who = ow;
            }
        }
        if (lane == 0) {
            s_key[i & 1][warp] = top;
            s_who[i & 1][warp] = who;
        }
        __syncthreads();
        top = NONE;
        who = -1;
#pragma unroll
        for (int u = 0; u < NT / 32; ++u)
            if (s_key[i & 1][u] > top) {
                top = s_key[i & 1][u];
                who = s_who[i & 1][u];
            }
        if (who == tid) {
            tokens[i] = v;
            parents[i] = w;
            best[i] = static_cast<float>(x);
            ++pos;
            load();
        }
        if (who < 0 && tid == 0) {  // fewer candidates than K: the rest is empty
            tokens[i] = parents[i] = -1;
            best[i] = -INFINITY;
        }
    }
}

}  // namespace

const void *beam_part_func(int dtype) {
    return dtype == 0 ? reinterpret_cast<const void *>(beam_part_impl<float>)
                      : reinterpret_cast<const void *>(beam_part_impl<bf16_t>);
}

const void *beam_join_func() { return reinterpret_cast<const void *>(beam_join_impl); }

}  // namespace mtp
