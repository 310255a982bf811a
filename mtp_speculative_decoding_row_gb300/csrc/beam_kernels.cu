// beam_kernels.cu -- the best K continuations of a sequence's W beams over a
// vocabulary of V: score(w, v) = scores[w] + ln softmax(z_w / T)(v), the K
// largest, equal ones by the smaller (w, v).
//
// Every logit is read once.  A row is cut into parts, one CTA each; a part
// yields its maximum, its sum of 2^((z - max) k) with k = log2(e) / T, and
// its own K best logits (within a row the order of the scores is that of the
// logits).  A second launch turns the parts' candidates into scores -- each
// logit's difference to its row's maximum, over T, less the logarithm of the
// float32 sum, in float64, because candidates may lie closer than float32 tells
// apart -- and merges the sorted lists.
//
// Candidates are 64-bit keys: the logit's bits in an order-preserving form,
// then the complement of the index, so one integer comparison orders by value
// and then by smaller index.  The K-th largest of the threads' running maxima
// bounds the K-th best from below; vectors are compared with that bound four
// at a time, and the indices of the few that pass are put aside: looking at
// them at once, in the midst of the loop, took a third of the kernel's time.
// The bound is taken again whenever three times as much of the row has been
// seen; a candidate costs as much as 500 elements of the sums (with the first
// bound alone the kernel took 81 us at 512 rows of 151936).  Each warp keeps a
// list of its own; one that is full is cut to its K best, and the bound rises
// for all warps.
//
// 512 rows of 151936 bfloat16 logits (64 sequences, 8 beams, K = 16) take 64
// us, 2.4 TB/s; one sequence of 4 rows 14.6 us.  Nothing of the first kernel is at
// its limit: about 10 instructions a logit, 56 % of the issue slots, memory at 37
// %, the rest waits for a round's loads and the bound's barriers; few rows are
// bound by the chain of steps in both kernels.
//
// Rows may start on any element.  A vector is always elements [8 j, 8 j + 8)
// (4 j of float32) of the row, put together from two aligned loads where the
// row is not aligned, so the order of the sums -- and with it the last bit of
// a normaliser -- does not depend on where a row lies: equal rows get equal
// scores and their ties go to the smaller beam.
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "tree.h"

namespace mtp {
namespace {

constexpr int NT = BEAM_THREADS;
constexpr int UN = 4;        // vectors of a thread per round
constexpr int NW = NT / 32;
constexpr int CAP = 384;     // candidates held by a warp: BEAM_MAX_K and a warp's vectors of 8 at least
constexpr int QUEUE = 256;   // vectors put aside by a warp: two rounds' at least
constexpr int SMEM_CAND = 2048;  // candidates that the join holds in shared memory

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

// Vector j of a row (elements j VEC ..), all of it in the row.
template <typename T>
__device__ __forceinline__ uint4 row_vec(const unsigned char *row, uint32_t sh, int j) {
    const uint4 *a = reinterpret_cast<const uint4 *>(row - sh) + j;
    if (sh == 0) return __ldg(a);
    return realign(__ldg(a), __ldg(a + 1), sh);  // the row's bytes reach into the second load
}

// The row's last vector, -inf beyond its V elements.
template <typename T>
__device__ __noinline__ uint4 row_tail(const unsigned char *row, int j, int V) {
    constexpr int VEC = Store<T>::VEC, ES = Store<T>::ES;
    uint32_t w[4] = {minus_inf_vec<T>().x, minus_inf_vec<T>().x, minus_inf_vec<T>().x, minus_inf_vec<T>().x};
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        if (j * VEC + e >= V) break;
        if (ES == 4)
            w[e & 3] = __ldg(reinterpret_cast<const uint32_t *>(row) + j * VEC + e);
        else {
            const uint32_t x = __ldg(reinterpret_cast<const unsigned short *>(row) + j * VEC + e);
            w[e / 2] = (e & 1) ? (w[e / 2] & 0x0000ffffu) | (x << 16) : (w[e / 2] & 0xffff0000u) | x;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The `keep` largest of list[0 .. n), sorted, to the front of the list: each
// key's rank is the number of larger ones (keys differ).  Warp-wide; `tmp`
// holds `keep` keys.
__device__ __forceinline__ int cut(uint64_t *list, int n, int keep, uint64_t *tmp) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    for (int i = lane; i < n; i += 32) {
        const uint64_t key = list[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += list[j] > key;
        if (rank < keep) tmp[rank] = key;
    }
    __syncwarp();
    const int m = min(n, keep);
    for (int i = lane; i < m; i += 32) list[i] = tmp[i];
    __syncwarp();
    return m;
}

// Look at the `queued` vectors that a warp has put aside, all of them in its
// part: their elements that reach the bound join the warp's list of `count`.
// Returns the list's new length; a cut raises *s_bound.
template <typename T>
__device__ __noinline__ int drain(const unsigned char *row, uint32_t sh, int whole, int V, const int *queue, int queued, uint64_t *list,
                                  int count, int keep, uint64_t *tmp, unsigned long long *s_bound) {
    constexpr int VEC = Store<T>::VEC;
    const int lane = threadIdx.x & 31;
    __syncwarp();
    for (int i0 = 0; i0 < queued; i0 += 32) {
        uint64_t bound = __shfl_sync(FULL, *static_cast<volatile unsigned long long *>(s_bound), 0);
        if (count + 32 * VEC > CAP) {
            count = cut(list, count, keep, tmp);
            if (count == keep) {
                bound = max(bound, list[keep - 1]);
                if (lane == 0) atomicMax(s_bound, static_cast<unsigned long long>(bound));
            }
        }
        const int at = i0 + lane < queued ? queue[i0 + lane] : -1;
        const uint4 raw = at < 0 ? minus_inf_vec<T>() : at < whole ? row_vec<T>(row, sh, at) : row_tail<T>(row, at, V);
        float z[VEC];
        Store<T>::unpack(raw, z);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const uint64_t key = make_key(z[e], at * VEC + e);
            const bool take = key >= bound && z[e] > -INFINITY;  // (not of a round that had a NaN: it may lie in this vector)
            const uint32_t in = __ballot_sync(FULL, take);
            if (take) list[count + __popc(in & ((1u << lane) - 1u))] = key;
            count += __popc(in);
        }
        __syncwarp();
    }
    return count;
}

// A lower bound of the keep-th largest of the block's values (for bfloat16 the
// value itself) raises *s_bound: its leading bits one by one, by counting the
// values that reach them.
template <int BITS>
__device__ __forceinline__ void raise_bound(float value, int keep, unsigned long long *s_bound) {
    const uint32_t mine = order_bits(value);
    uint32_t at = 0;
#pragma unroll 1
    for (uint32_t bit = 0x80000000u; bit >= (1u << (32 - BITS)); bit >>= 1)
        if (__syncthreads_count(mine >= (at | bit)) >= keep) at |= bit;
    // (not below -inf: what lies there is no number)
    if (threadIdx.x == 0) atomicMax(s_bound, static_cast<unsigned long long>(max(at, order_bits(-INFINITY))) << 32);
    __syncthreads();
}

// k = log2(e) / T; the largest float where that is beyond it (a difference of
// two logits is then 0 or far beyond any weight, whichever of the two k is).
__device__ __forceinline__ float exponent_scale(float temp) { return fminf(LOG2E / temp, FLT_MAX); }

template <typename T>
__global__ void __launch_bounds__(NT, BEAM_PER_SM) beam_part_impl(const __grid_constant__ BeamArgs A) {
    constexpr int VEC = Store<T>::VEC, ES = Store<T>::ES;
    __shared__ uint64_t lists[NW][CAP];
    __shared__ uint64_t tmps[NW][BEAM_MAX_K];
    __shared__ int queue[NW][QUEUE];
    __shared__ unsigned long long s_bound;
    __shared__ int s_bad, s_n[NW];
    __shared__ float s_m[NW];
    __shared__ float s_s[NW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / A.parts, part = blockIdx.x - row * A.parts;
    const int b = row / A.W;
    const size_t slot = static_cast<size_t>(row) * A.parts + part;
    float *cz = A.cand_z + slot * A.KL;
    int *cv = A.cand_v + slot * A.KL;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const float temp = __ldg(A.temp + b), score = __ldg(A.scores + row);
    if (!(temp > 0.f) || temp == INFINITY || !(score < INFINITY) || score == -INFINITY) {
        // a dead beam, or a sequence that the join flags: its logits are not read
        if (tid == 0) {
            A.part_max[slot] = -INFINITY;
            A.part_sum[slot] = 0.f;
            A.part_flag[slot] = 0;
        }
        for (int i = tid; i < A.KL; i += NT) cv[i] = -1;
        return;
    }
    // log2(e) / T in two floats, k + dk: a row's sum is corrected for the
    // rounding of k (below).  log2(e) = LOG2E + LOG2E_LO.
    constexpr float LOG2E_LO = 1.9259629911266175e-8f;
    const float k = exponent_scale(temp), dk = k < FLT_MAX ? (fmaf(-k, temp, LOG2E) + LOG2E_LO) / temp : 0.f;
    const unsigned char *base = static_cast<const unsigned char *>(A.logits) + static_cast<size_t>(row) * A.V * ES;
    const uint32_t sh = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(base) & 15u);
    const int j0 = part * (A.part_elems / VEC);
    const int j1 = min((A.V + VEC - 1) / VEC, j0 + A.part_elems / VEC);
    const int whole = min(A.V / VEC, j1);  // vectors without a tail
    if (tid == 0) {
        s_bound = 0;
        s_bad = 0;
    }

    // s: the sum of e_i = 2^((z_i - m) k): the difference first, so that the
    // exponents that weigh are small and exact to 2^-23 of themselves at any
    // temperature (z_i k - m k loses what a low temperature leaves of it: m k has
    // half a unit of error at 2^24).  se and s1: the sums of e_i and of e_i (z_i
    // - m) over every fourth vector; their ratio says where the row's weight
    // lies, which is all that the correction for dk needs to know (it is below
    // 3e-7 of a score to begin with).
    float m = -INFINITY, s = 0.f, se = 0.f, s1 = 0.f;
    int count = 0, queued = 0, again = j0;
    // one round: vectors j + tid, j + tid + NT, .. of the row
    auto round = [&](int j, uint4 (&raw)[UN]) {
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < UN; ++u) top = max_nan(top, Store<T>::vmax(raw[u]));
        if (!(top <= m)) {  // a new maximum of this thread, or NaN
            if (!(top < INFINITY)) {
                s_bad = 1;  // the join flags the sequence; nothing of this round counts
#pragma unroll
                for (int u = 0; u < UN; ++u) raw[u] = minus_inf_vec<T>();
                top = -INFINITY;
            } else {
                const float gap = m - top, f = ex2(gap * k);  // (m = -inf at first: f = 0)
                s1 = f > 0.f ? f * fmaf(se, gap, s1) : 0.f;
                m = top;
                s *= f;
                se *= f;
            }
        }
        if (m > -INFINITY) {
            // (four sums, in plain instructions: packed pairs cost more in moves
            // than they save)
            float a[4] = {0.f, 0.f, 0.f, 0.f}, a1 = 0.f;
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                float z[VEC];
                Store<T>::unpack(raw[u], z);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float d = z[e] - m, x = ex2(d * k);
                    a[e & 3] += x;
                    if (u == 0) a1 = fmaf(x, fmaxf(d, -FLT_MAX), a1);  // (-inf: 0 times a finite number)
                }
                if (u == 0) se += (a[0] + a[1]) + (a[2] + a[3]);
            }
            s += (a[0] + a[1]) + (a[2] + a[3]);
            s1 += a1;
        }
        if (j >= again) {
            raise_bound<ES == 2 ? 16 : 20>(m, A.KL, &s_bound);
            again = j + 2 * (j - j0) + 2 * NT * UN;
        }
        // (a bound that is read late is a lower bound all the same)
        const uint64_t bound = __shfl_sync(FULL, *static_cast<volatile unsigned long long *>(&s_bound), 0);
        // Vectors of -inf alone are never put aside: they hold no candidate, and
        // what stands in for vectors behind the part's end is such a one (drain()
        // would read the next part's logits for it, candidates of two parts then).
        const float zb = fmaxf(order_float(static_cast<uint32_t>(bound >> 32)), -FLT_MAX);
        if (__any_sync(FULL, top >= zb)) {
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const bool take = Store<T>::vmax(raw[u]) >= zb;
                const uint32_t in = __ballot_sync(FULL, take);
                if (take) queue[warp][queued + __popc(in & ((1u << lane) - 1u))] = j + u * NT + tid;
                queued += __popc(in);
            }
            if (queued > QUEUE - 32 * UN) {
                count = drain<T>(base, sh, whole, A.V, queue[warp], queued, lists[warp], count, A.KL, tmps[warp], &s_bound);
                queued = 0;
            }
        }
    };
    // vectors of a round; whole rounds of aligned rows need no test
    const uint4 *fast = reinterpret_cast<const uint4 *>(base) + tid;
    auto fetch = [&](int j, uint4 (&raw)[UN]) {
        if (sh == 0 && j + NT * UN <= whole) {
#pragma unroll
            for (int u = 0; u < UN; ++u) raw[u] = __ldg(fast + j + u * NT);
        } else {
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const int at = j + u * NT + tid;
                raw[u] = at < whole ? row_vec<T>(base, sh, at) : at < j1 ? row_tail<T>(base, at, A.V) : minus_inf_vec<T>();
            }
        }
    };
    // the next round's vectors are on their way while one is worked on
    constexpr int STEP = NT * UN;
    uint4 one[UN], two[UN];
    fetch(j0, one);
    __syncthreads();  // s_bad and s_bound are set (a thread that met a NaN before could be overwritten)
    for (int j = j0; j < j1; j += 2 * STEP) {
        if (j + STEP < j1) fetch(j + STEP, two);
        round(j, one);
        if (j + STEP >= j1) break;
        if (j + 2 * STEP < j1) fetch(j + 2 * STEP, one);
        round(j + STEP, two);
    }
    count = drain<T>(base, sh, whole, A.V, queue[warp], queued, lists[warp], count, A.KL, tmps[warp], &s_bound);
    if (count > 2 * BEAM_MAX_K) count = cut(lists[warp], count, A.KL, tmps[warp]);
    if (lane == 0) s_n[warp] = count;
    float top = warp_allmax(m);
    if (lane == 0) s_m[warp] = top;
    __syncthreads();
    // the warps' lists to one: a key's place is the number of larger ones
    int ends[NW], total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) ends[w] = total += s_n[w];
    for (int i = tid; i < total; i += NT) {
        int w = 0;
        for (; i >= ends[w]; ++w) {
        }
        const uint64_t key = lists[w][i - (ends[w] - s_n[w])];
        int rank = 0;
        for (int o = 0; o < NW && rank < A.KL; ++o)
#pragma unroll 4
            for (int e = 0; e < s_n[o]; ++e) rank += lists[o][e] > key;
        if (rank < A.KL) {
            cz[rank] = order_float(static_cast<uint32_t>(key >> 32));
            cv[rank] = static_cast<int>(~static_cast<uint32_t>(key));
        }
    }
    for (int i = total + tid; i < A.KL; i += NT) cv[i] = -1;
    top = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, s_m[w]);
    // The thread's share of sum_i 2^((z_i - top) (k + dk)) is s 2^((m - top) k)
    // 2^(((m - top) + d) dk), d the mean of z_i - m over its weight (the spread of
    // z_i dk about its mean changes the sum by its square: 1e-12).  A share below
    // 2^-200 is none.
    float sum = 0.f;
    const float gap = (m - top) * k;
    if (gap > -200.f) sum = s * ex2(fmaf((m - top) + (se > 0.f ? s1 / se : 0.f), dk, gap));
    sum = warp_allsum(sum);
    if (lane == 0) s_s[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        float t = 0.f;
        for (int w = 0; w < NW; ++w) t += s_s[w];
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

// One CTA per sequence.  All threads turn the lists' candidates into scores;
// then one warp merges the sorted lists (beam after beam, part after part),
// eight of them to a lane: each round takes the best head -- equal scores: the
// smaller list, and so the smaller beam and index -- and moves its list on.
// A round is a few warp-wide reductions, with no barrier and no load from
// global memory.  Where float64 may not tell the scores of two different logits
// of a beam apart (a temperature of 10^12, logits of 10^-12 below one of 10),
// equal scores are looked at by beam, logit and list.  (Doing so always: one
// sequence of 4 rows 16.3 us instead of 15.3.)  No more registers than the first
// kernel has: a CTA fits in as soon as one of that kernel's has ended (with 88 of
// them 64 sequences of 8 rows took 66.5 us instead of 64.5).
__global__ void __launch_bounds__(NT, BEAM_PER_SM) beam_join_impl(const __grid_constant__ BeamArgs A) {
    constexpr long long NONE = -0x7fffffffffffffffll - 1;
    constexpr int PER = NT / 32;  // lists of a lane
    __shared__ float s_max[BEAM_MAX_W];
    __shared__ double s_off[BEAM_MAX_W];  // scores[w] - ln sum
    __shared__ int s_flag;
    __shared__ long long s_key[SMEM_CAND];
    __shared__ int s_v[SMEM_CAND];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
    const int lists = A.W * A.parts;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const float temp = __ldg(A.temp + b);
    const bool bad_temp = !(temp > 0.f) || temp == INFINITY;
    const double inv_t = 1.0 / static_cast<double>(temp);
    if (tid == 0) s_flag = bad_temp ? F_BAD_TEMP : 0;
    __syncthreads();
    const size_t cand0 = static_cast<size_t>(b) * lists * A.KL;
    const int n = lists * A.KL;
    const bool shared = n <= SMEM_CAND;
    float z0 = 0.f;  // the first candidate of this thread is on its way during the statistics
    int v0 = -1;
    if (shared && tid < n) {
        z0 = A.cand_z[cand0 + tid];
        v0 = A.cand_v[cand0 + tid];
    }
    for (int w = warp; w < A.W; w += NW) {  // a warp per beam, a lane per part
        const int row = b * A.W + w;
        const float score = __ldg(A.scores + row);
        const size_t p0 = static_cast<size_t>(row) * A.parts;
        const float k = exponent_scale(temp);
        float top = -INFINITY, sum = 0.f;
        int bad = 0;
        for (int p = lane; p < A.parts; p += 32) {
            const float m = A.part_max[p0 + p], s = A.part_sum[p0 + p];
            bad |= A.part_flag[p0 + p];
            const float up = fmaxf(top, m);
            if (up > -INFINITY) sum = sum * ex2((top - up) * k) + s * ex2((m - up) * k);
            top = up;
        }
        const float all = warp_allmax(top);
        sum = warp_allsum(top > -INFINITY ? sum * ex2((top - all) * k) : 0.f);
        bad = __reduce_or_sync(FULL, bad);
        if (lane == 0) {
            // a dead beam has no candidates; a live one with no finite logit is an error
            const bool dead = score == -INFINITY;
            s_max[w] = all;
            s_off[w] = dead || all == -INFINITY ? 0.0 : static_cast<double>(score) - log(static_cast<double>(sum));
            if (!bad_temp && (bad || !(score < INFINITY) || (!dead && all == -INFINITY))) atomicOr(&s_flag, F_NONFINITE);
        }
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
    const int beam_cand = A.parts * A.KL;
    auto key_of = [&](int i, float z, int v) {
        const int w = i / beam_cand;
        // (the difference in float64 too: in float32 neighbouring logits fall together beside a large one)
        return v < 0 ? NONE : order_double(s_off[w] + (static_cast<double>(z) - static_cast<double>(s_max[w])) * inv_t);
    };
    // Different logits lie at least 2^-24 of the larger one apart, and a score is
    // formed by three roundings of 2^-53 of it or of s_off: where |z| / T is below
    // 2^-26 of these, two scores may be one number.  (By the exponents: float64
    // arithmetic is slow here.)
    const int exp_t = static_cast<int>(__float_as_uint(temp) >> 23);
    auto coarse = [&](int i, long long key, float z) {
        const int exp_z = static_cast<int>((__float_as_uint(z) >> 23) & 0xffu);
        const int of_key = static_cast<int>((key < 0 ? ~key : key) >> 52), of_off = (__double2hiint(s_off[i / beam_cand]) >> 20) & 0x7ff;
        return key != NONE && z != 0.f && (exp_z == 0 ? -24 : exp_z) - max(exp_t, 1) < max(of_key, of_off) - 1023 - 24;
    };
    bool careful = !shared;
    if (shared) {
        for (int i = tid; i < n; i += NT) {
            if (i != tid) {
                z0 = A.cand_z[cand0 + i];
                v0 = A.cand_v[cand0 + i];
            }
            const long long key = key_of(i, z0, v0);
            careful |= coarse(i, key, z0);
            s_key[i] = key;
            s_v[i] = v0;
        }
        careful = __syncthreads_or(careful);
    }
    if (warp != 0) return;
    long long head[PER];
    int pos[PER];
    auto load = [&](int list, int at) {
        if (list >= lists || at >= A.KL) return NONE;
        const int i = list * A.KL + at;
        return shared ? s_key[i] : key_of(i, A.cand_z[cand0 + i], A.cand_v[cand0 + i]);
    };
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        head[q] = load(lane * PER + q, 0);
        pos[q] = 0;
    }
    auto merge = [&](auto looks) {
        for (int i = 0; i < A.K; ++i) {
            long long mine = head[0];
            int q0 = 0;
#pragma unroll
            for (int q = 1; q < PER; ++q)
                if (head[q] > mine) {
                    mine = head[q];
                    q0 = q;
                }
            const uint64_t u = static_cast<uint64_t>(mine) ^ 0x8000000000000000ull;
            const uint32_t hi = static_cast<uint32_t>(u >> 32), lo = static_cast<uint32_t>(u);
            const uint32_t top = __reduce_max_sync(FULL, hi);
            const uint32_t low = __reduce_max_sync(FULL, hi == top ? lo : 0u);
            const uint32_t same = __ballot_sync(FULL, hi == top && lo == low);
            int who = __ffs(same) - 1;
            if constexpr (decltype(looks)::value) {
                // of the smallest beam with this score the largest logit
                const int beam = __shfl_sync(FULL, (lane * PER + q0) / A.parts, who);
                uint32_t zb = 0u;
                if ((same >> lane) & 1u && mine != NONE) {
#pragma unroll
                    for (int q = 0; q < PER; ++q) {
                        const int list = lane * PER + q;
                        if (head[q] != mine || list / A.parts != beam) continue;
                        const uint32_t o = order_bits(A.cand_z[cand0 + list * A.KL + pos[q]]);
                        if (o > zb) {
                            zb = o;
                            q0 = q;
                        }
                    }
                }
                const uint32_t most = __reduce_max_sync(FULL, zb);
                who = __ffs(__ballot_sync(FULL, zb == most)) - 1;
            }
            if (lane != who) continue;
            if (mine == NONE) {  // fewer candidates than K: the rest is empty
                tokens[i] = parents[i] = -1;
                best[i] = -INFINITY;
                continue;
            }
            const int list = lane * PER + q0;
            int at = 0;
#pragma unroll
            for (int q = 0; q < PER; ++q)
                if (q == q0) at = pos[q]++;
            const int c = list * A.KL + at;
            tokens[i] = shared ? s_v[c] : A.cand_v[cand0 + c];
            parents[i] = list / A.parts;
            best[i] = static_cast<float>(__longlong_as_double(mine < 0 ? mine ^ 0x7fffffffffffffffll : mine));
            const long long next = load(list, at + 1);
#pragma unroll
            for (int q = 0; q < PER; ++q)
                if (q == q0) head[q] = next;
        }
    };
    if (careful)
        merge(std::true_type{});
    else
        merge(std::false_type{});
}

}  // namespace

const void *beam_part_func(int dtype) {
    return dtype == 0 ? reinterpret_cast<const void *>(beam_part_impl<float>)
                      : reinterpret_cast<const void *>(beam_part_impl<bf16_t>);
}

const void *beam_join_func() { return reinterpret_cast<const void *>(beam_join_impl); }

}  // namespace mtp
