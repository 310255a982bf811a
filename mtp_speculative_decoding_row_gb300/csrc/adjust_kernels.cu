// adjust_kernels.cu -- logits of a drafted chain or tree with the penalties for
// repeated tokens, biases and grammar masks of their sequence.
//
// For row s of a sequence, with c(v) the occurrences of v in the generated part
// of the text and on the path to node s, and [seen] whether v is in the text or
// on the path at all:
//   x = z > 0 ? z / rho : z rho   where seen, else z
//   x = x - freq c - pres [c > 0] + sum of v's biases
//   x = -inf                      where the mask has no bit.
//
// One pass: memory bounds it, every logit is read and written once.  A block has
// a slice of the vocabulary and some rows of one sequence.  It counts the
// slice's tokens of the text in shared memory (integers: the order of the atomic
// additions changes nothing), with one bit for each entry that needs more than
// its mask, and then streams the rows: a vector whose bits are clear is copied.
// Rows differ in their paths only; the few tokens of the drafts are looked up
// in the path's list where they occur, so that the counts serve all rows.
#include "common.cuh"
#include "step.h"

namespace mtp {
namespace {

constexpr int NT = ADJ_THREADS;
// An entry of the table: in the text's first part; a drafted token; has a
// bias; occurrences in the rest of the text.
constexpr uint32_t PROMPT = 1u, DRAFT = 2u, BIAS = 4u, ONE = 8u;

__device__ __forceinline__ uint32_t bf16_of(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[Store<T>::VEC]) {
    if constexpr (Store<T>::ES == 4)
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    else
        return make_uint4(bf16_of(x[0], x[1]), bf16_of(x[2], x[3]), bf16_of(x[4], x[5]), bf16_of(x[6], x[7]));
}

template <typename T>
__device__ __forceinline__ float load1(const unsigned char *p) {
    if constexpr (Store<T>::ES == 4)
        return *reinterpret_cast<const float *>(p);
    else
        return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(p)) << 16);
}
template <typename T>
__device__ __forceinline__ void store1(unsigned char *p, float x) {
    if constexpr (Store<T>::ES == 4)
        *reinterpret_cast<float *>(p) = x;
    else
        *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(bf16_of(x, 0.f));
}

struct Shared {
    int token[ADJ_MAX_ROWS];      // of the nodes; -1: none
    uint64_t path[ADJ_MAX_ROWS];  // nodes on the way to a node, itself included
    int above[ADJ_MAX_ROWS];
    int biases;                   // of this slice
    int flag;
};

// Bits v .. v + 31 of a row of words that are zero from word `n` on.
__device__ __forceinline__ uint32_t bits_at(const uint32_t *w, int v, int n) {
    const int i = v >> 5, r = v & 31;
    const uint32_t lo = w[i];
    if (r == 0) return lo;
    return __funnelshift_r(lo, i + 1 < n ? w[i + 1] : 0u, r);
}

template <typename T>
__global__ void __launch_bounds__(NT) adjust_impl(const __grid_constant__ AdjArgs A) {
    constexpr int VEC = Store<T>::VEC, ES = Store<T>::ES, AHEAD = 4;
    extern __shared__ __align__(16) uint32_t smem[];
    uint32_t *table = smem;                   // [slice]
    uint32_t *touched = table + A.slice;      // [slice / 32] bits: look at the entry
    int *bias_id = reinterpret_cast<int *>(touched + A.slice / 32);     // [n_bias] of this slice, in their order
    float *bias_sum = reinterpret_cast<float *>(bias_id + A.n_bias);    // [n_bias] sum of all biases of the id
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.y, s0 = blockIdx.z * A.rows;
    const int lo = blockIdx.x * A.slice, hi = min(A.V, lo + A.slice);  // this block's tokens
    if (tid == 0) sh.flag = 0;
    for (int i = tid; i < (A.slice + A.slice / 32) / 4; i += NT) reinterpret_cast<uint4 *>(table)[i] = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- what the sequence has; every block finds the same flag ----
    int flag = 0;
    int n = A.nodes ? __ldg(A.nodes + b) : A.S, len = A.len ? __ldg(A.len + b) : 0, prompt = A.prompt ? __ldg(A.prompt + b) : 0;
    if (n < 0 || n > A.S) {
        flag |= F_BAD_ID;
        n = A.S;
    }
    if (len < 0 || len > A.L) {
        flag |= F_BAD_ID;
        len = 0;
    }
    if (prompt < 0 || prompt > len) flag |= F_BAD_ID;
    const float rho = A.rho ? __ldg(A.rho + b) : 1.f, freq = A.freq ? __ldg(A.freq + b) : 0.f, pres = A.pres ? __ldg(A.pres + b) : 0.f;
    if (!(rho > 0.f && rho < INFINITY && fabsf(freq) < INFINITY && fabsf(pres) < INFINITY)) flag |= F_NONFINITE;
    if (A.tokens && tid < 32) {
        for (int i = lane; i < A.S; i += 32) {
            const int t = i < n ? __ldg(A.tokens + static_cast<size_t>(b) * A.S + i) : -1;
            if (t >= A.V) flag |= F_BAD_ID;
            sh.token[i] = t;
            int p = i - 1;
            if (A.parents && i < n) {
                p = __ldg(A.parents + static_cast<size_t>(b) * A.S + i);
                if (p >= i || p < -1) {
                    flag |= F_BAD_ID;
                    p = -1;
                }
            }
            sh.above[i] = p;
            sh.path[i] = 1ull << i;
        }
        __syncwarp();
        // in each round a node takes over what its farthest known ancestor knows
        for (int reach = 1; reach < n; reach <<= 1) {
            uint64_t m[2];
            int a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = lane + 32 * e, p = i < A.S ? sh.above[i] : -1;
                m[e] = p < 0 ? 0ull : sh.path[p];
                a[e] = p < 0 ? -1 : sh.above[p];
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = lane + 32 * e;
                if (i < A.S) {
                    sh.path[i] |= m[e];
                    sh.above[i] = a[e];
                }
            }
            __syncwarp();
        }
    }
    __syncthreads();  // the table is clear

    auto touch = [&](int i, uint32_t add) {
        atomicAdd(table + i, add);
        atomicOr(touched + (i >> 5), 1u << (i & 31));
    };
    // ---- the text ----
    {
        const int32_t *text = A.history + static_cast<size_t>(b) * A.L;
        auto see = [&](int id, int at) {
            if (id >= A.V) flag |= F_BAD_ID;
            if (id >= lo && id < hi) {
                if (at < prompt) {
                    atomicOr(table + (id - lo), PROMPT);
                    atomicOr(touched + ((id - lo) >> 5), 1u << ((id - lo) & 31));
                } else {
                    touch(id - lo, ONE);
                }
            }
        };
        int done = 0;
        if (A.vec_history) {
            const int vecs = len / 4;
#pragma unroll 4
            for (int i = tid; i < vecs; i += NT) {
                const int4 x = __ldg(reinterpret_cast<const int4 *>(text) + i);
                see(x.x, 4 * i);
                see(x.y, 4 * i + 1);
                see(x.z, 4 * i + 2);
                see(x.w, 4 * i + 3);
            }
            done = 4 * vecs;
        }
#pragma unroll 4
        for (int i = done + tid; i < len; i += NT) see(__ldg(text + i), i);
    }
    // ---- drafted tokens, biases ----
    if (A.tokens && tid < n) {
        const int id = sh.token[tid];
        if (id >= lo && id < hi) {
            atomicOr(table + (id - lo), DRAFT);
            atomicOr(touched + ((id - lo) >> 5), 1u << ((id - lo) & 31));
        }
    }
    if (A.n_bias > 0) {
        const int32_t *ids = A.bias_ids + static_cast<size_t>(b) * A.n_bias;
        const float *bias = A.bias + static_cast<size_t>(b) * A.n_bias;
        if (tid < 32) {  // in their order, so that a sum of several has one value
            int found = 0;
            for (int i0 = 0; i0 < A.n_bias; i0 += 32) {
                const int id = i0 + lane < A.n_bias ? __ldg(ids + i0 + lane) : -1;
                if (id >= A.V) flag |= F_BAD_ID;
                const bool in = id >= lo && id < hi;
                const uint32_t who = __ballot_sync(FULL, in);
                if (in) {
                    const int at = found + __popc(who & ((1u << lane) - 1u));
                    bias_id[at] = id;
                    bias_sum[at] = __ldg(bias + i0 + lane);
                    atomicOr(table + (id - lo), BIAS);
                    atomicOr(touched + ((id - lo) >> 5), 1u << ((id - lo) & 31));
                }
                found += __popc(who);
            }
            if (lane == 0) sh.biases = found;
        }
        __syncthreads();
        float sum[ADJ_MAX_BIAS / NT];
#pragma unroll
        for (int e = 0; e < ADJ_MAX_BIAS / NT; ++e) {
            const int j = tid + e * NT;
            sum[e] = 0.f;
            if (j < sh.biases)
                for (int i = 0; i < sh.biases; ++i)
                    if (bias_id[i] == bias_id[j]) sum[e] += bias_sum[i];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < ADJ_MAX_BIAS / NT; ++e)
            if (tid + e * NT < sh.biases) bias_sum[tid + e * NT] = sum[e];
    }
    if (flag) atomicOr(&sh.flag, flag);
    __syncthreads();
    flag = sh.flag;
    if (A.flags && tid == 0 && blockIdx.x == 0 && blockIdx.z == 0) A.flags[b] = flag;

    // ---- the rows ----
    auto adjust = [&](float x, int v, int s) {
        const uint32_t e = table[v - lo];
        uint32_t count = e / ONE;
        if (e & DRAFT)
            for (int i = 0; i <= s; ++i) count += ((sh.path[s] >> i) & 1ull) && sh.token[i] == v ? 1u : 0u;
        if (count > 0 || (e & PROMPT)) x = x > 0.f ? __fdiv_rn(x, rho) : x * rho;
        if (count > 0) x = fmaf(-freq, static_cast<float>(count), x) - pres;
        if (e & BIAS)
            for (int i = 0; i < sh.biases; ++i)
                if (bias_id[i] == v) {
                    x += bias_sum[i];
                    break;
                }
        return x;
    };
    const int words = (A.V + 31) / 32;
    const bool in_place = A.out == A.z;
    for (int s = s0; s < min(n, s0 + A.rows); ++s) {
        const size_t row = (static_cast<size_t>(b) * A.S + s) * A.V;
        const unsigned char *z = A.z + row * ES;
        unsigned char *out = A.out + row * ES;
        const uint32_t *mask = A.mask ? A.mask + b * A.mask_s[0] + s * A.mask_s[1] : nullptr;
        auto allowed = [&](int v) {  // bits of entries v, v + 1, ..
            if (!mask) return ~0u;
            const int i = v >> 5, r = v & 31;
            const uint32_t w = __ldg(mask + i);
            return r + VEC <= 32 ? w >> r : __funnelshift_r(w, i + 1 < words ? __ldg(mask + i + 1) : 0u, r);
        };
        // vectors of the row that lie in the slice, wherever the row starts
        const int first = min(hi, lo + static_cast<int>((VEC - (row + lo) % VEC) % VEC)), vecs = (hi - first) / VEC;
        constexpr uint32_t ALL = (1u << VEC) - 1u;
        for (int i0 = tid; i0 < vecs; i0 += NT * AHEAD) {
            uint4 x[AHEAD];
            uint32_t may[AHEAD];
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const int i = i0 + a * NT;
                if (i >= vecs) break;
                x[a] = *reinterpret_cast<const uint4 *>(z + static_cast<size_t>(first + i * VEC) * ES);
                may[a] = allowed(first + i * VEC) & ALL;
            }
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const int i = i0 + a * NT, v = first + i * VEC;
                if (i >= vecs) break;
                const uint32_t look = bits_at(touched, v - lo, A.slice / 32) & ALL;
                if (flag) {
                    float y[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) y[e] = NAN;
                    x[a] = pack<T>(y);
                } else if (look || may[a] != ALL) {
                    float y[VEC];
                    Store<T>::unpack(x[a], y);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        if ((look >> e) & 1u) y[e] = adjust(y[e], v + e, s);
                        if (!((may[a] >> e) & 1u)) y[e] = -INFINITY;
                    }
                    x[a] = pack<T>(y);
                } else if (in_place) {
                    continue;
                }
                *reinterpret_cast<uint4 *>(out + static_cast<size_t>(v) * ES) = x[a];
            }
        }
        // the entries before the first vector and behind the last
        const int head = first - lo, tail = hi - first - vecs * VEC;
        if (tid < head + tail) {
            const int v = tid < head ? lo + tid : hi - tail + (tid - head);
            float y = load1<T>(z + static_cast<size_t>(v) * ES);
            if ((touched[(v - lo) >> 5] >> (v & 31)) & 1u) y = adjust(y, v, s);
            if (!(allowed(v) & 1u)) y = -INFINITY;
            store1<T>(out + static_cast<size_t>(v) * ES, flag ? NAN : y);
        }
    }
}

}  // namespace

const void *adj_func(int dtype) {
    return dtype == 0 ? reinterpret_cast<const void *>(adjust_impl<float>) : reinterpret_cast<const void *>(adjust_impl<bf16_t>);
}

uint32_t adj_smem(int slice, int n_bias) { return static_cast<uint32_t>(slice) * 4 + slice / 8 + n_bias * 8; }

}  // namespace mtp
