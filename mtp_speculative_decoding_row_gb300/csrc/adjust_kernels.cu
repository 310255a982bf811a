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
// Memory bounds it: every logit is read and written once.  A block has a slice
// of the vocabulary and some rows of one sequence.  It streams the rows through
// their masks, counts the slice's tokens of the text in shared memory (integers:
// the order of the atomic additions changes nothing), lists the entries that
// anything but the mask changes, and writes those once more, a thread to an
// entry.  A text's words crowd in few places: dealt out from a list they keep
// all threads busy, where looking for them beside the streamed vectors left one
// block with nearly all the work (64 x 4 rows, 8192 tokens: 118 us).  Rows
// differ in their paths only; the few drafted tokens are looked up in the path
// where they occur, so that one count serves all rows.
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
    int listed;
    int flag;
};

template <typename T>
__global__ void __launch_bounds__(NT) adjust_impl(const __grid_constant__ AdjArgs A) {
    constexpr int VEC = Store<T>::VEC, ES = Store<T>::ES, AHEAD = 4, EARLY = 2, ROWS = 4;
    constexpr uint32_t ALL = (1u << VEC) - 1u;
    extern __shared__ __align__(16) uint32_t smem[];
    uint32_t *table = smem;                                             // [slice]
    uint16_t *list = reinterpret_cast<uint16_t *>(table + A.slice);     // [slice] entries that are not 0
    int *bias_id = reinterpret_cast<int *>(list + A.slice);             // [n_bias] of this slice, in their order
    float *bias_of = reinterpret_cast<float *>(bias_id + A.n_bias);     // [n_bias]
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.x, s0 = blockIdx.z * A.rows;
    const int lo = blockIdx.y * A.slice, hi = min(A.V, lo + A.slice);  // this block's tokens
    if (tid == 0) sh.flag = sh.listed = 0;
    for (int i = tid; i < A.slice / 4; i += NT) reinterpret_cast<uint4 *>(table)[i] = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- what the sequence has; every block finds the same flag ----
    const int32_t *text = A.history + static_cast<size_t>(b) * A.L;
    int4 early[EARLY];  // the text's first tokens are on their way while the rows go by
#pragma unroll
    for (int e = 0; e < EARLY; ++e) {
        const int i = tid + e * NT;
        early[e] = A.vec_history && 4 * i < A.L ? __ldg(reinterpret_cast<const int4 *>(text) + i) : make_int4(-1, -1, -1, -1);
    }
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
    const int s1 = min(n, s0 + A.rows);

    // ---- the rows through their masks ----
    const int words = (A.V + 31) / 32;
    const bool in_place = A.out == A.z;
    auto mask_of = [&](int s) { return A.mask ? A.mask + b * A.mask_s[0] + s * A.mask_s[1] : nullptr; };
    auto allowed = [&](const uint32_t *mask, int v) {  // bits of entries v, v + 1, .. v + VEC - 1
        if (!mask) return ~0u;
        const int i = v >> 5, r = v & 31;
        const uint32_t w = __ldg(mask + i);
        return r + VEC <= 32 ? w >> r : __funnelshift_r(w, i + 1 < words ? __ldg(mask + i + 1) : 0u, r);
    };
    auto row_of = [&](int s) { return (static_cast<size_t>(b) * A.S + s) * A.V; };
    if (!in_place || A.mask) {
        for (int s = s0; s < s1; ++s) {
            const size_t row = row_of(s);
            const unsigned char *z = A.z + row * ES;
            unsigned char *out = A.out + row * ES;
            const uint32_t *mask = mask_of(s);
            // vectors of the row that lie in the slice, wherever the row starts
            const int first = min(hi, lo + static_cast<int>((VEC - (row + lo) % VEC) % VEC)), vecs = (hi - first) / VEC;
            for (int i0 = tid; i0 < vecs; i0 += NT * AHEAD) {
                uint4 x[AHEAD];
                uint32_t may[AHEAD];
#pragma unroll
                for (int a = 0; a < AHEAD; ++a) {
                    const int i = i0 + a * NT;
                    if (i >= vecs) break;
                    x[a] = *reinterpret_cast<const uint4 *>(z + static_cast<size_t>(first + i * VEC) * ES);
                    may[a] = allowed(mask, first + i * VEC) & ALL;
                }
#pragma unroll
                for (int a = 0; a < AHEAD; ++a) {
                    const int i = i0 + a * NT;
                    if (i >= vecs) break;
                    if (may[a] != ALL) {
                        float y[VEC];
                        Store<T>::unpack(x[a], y);
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            if (!((may[a] >> e) & 1u)) y[e] = -INFINITY;
                        x[a] = pack<T>(y);
                    } else if (in_place) {
                        continue;
                    }
                    *reinterpret_cast<uint4 *>(out + static_cast<size_t>(first + i * VEC) * ES) = x[a];
                }
            }
            // the entries before the first vector and behind the last
            const int head = first - lo, tail = hi - first - vecs * VEC;
            if (tid < head + tail) {
                const int v = tid < head ? lo + tid : hi - tail + (tid - head);
                store1<T>(out + static_cast<size_t>(v) * ES, allowed(mask, v) & 1u ? load1<T>(z + static_cast<size_t>(v) * ES) : -INFINITY);
            }
        }
    }

    // ---- the tree ----
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
    __syncthreads();  // the table is clear, the tokens are there

    // ---- the text, drafted tokens, biases ----
    {
        auto see = [&](int id, int at) {
            if (at >= len) return;
            if (id >= A.V) flag |= F_BAD_ID;
            if (id < lo || id >= hi) return;
            if (at < prompt)
                atomicOr(table + (id - lo), PROMPT);
            else
                atomicAdd(table + (id - lo), ONE);
        };
        auto four = [&](const int4 &x, int at) {
            see(x.x, at);
            see(x.y, at + 1);
            see(x.z, at + 2);
            see(x.w, at + 3);
        };
        if (A.vec_history) {
#pragma unroll
            for (int e = 0; e < EARLY; ++e) four(early[e], 4 * (tid + e * NT));
#pragma unroll 4
            for (int i = tid + EARLY * NT; 4 * i < len; i += NT) four(__ldg(reinterpret_cast<const int4 *>(text) + i), 4 * i);
        } else {
#pragma unroll 4
            for (int i = tid; i < len; i += NT) see(__ldg(text + i), i);
        }
    }
    if (A.tokens && tid < n) {
        const int id = sh.token[tid];
        if (id >= lo && id < hi) atomicOr(table + (id - lo), DRAFT);
    }
    if (A.n_bias > 0 && tid < 32) {  // in their order, so that a sum of several has one value
        const int32_t *ids = A.bias_ids + static_cast<size_t>(b) * A.n_bias;
        const float *bias = A.bias + static_cast<size_t>(b) * A.n_bias;
        int found = 0;
        for (int i0 = 0; i0 < A.n_bias; i0 += 32) {
            const int id = i0 + lane < A.n_bias ? __ldg(ids + i0 + lane) : -1;
            if (id >= A.V) flag |= F_BAD_ID;
            const bool in = id >= lo && id < hi;
            const uint32_t who = __ballot_sync(FULL, in);
            if (in) {
                const int at = found + __popc(who & ((1u << lane) - 1u));
                bias_id[at] = id;
                bias_of[at] = __ldg(bias + i0 + lane);
                atomicOr(table + (id - lo), BIAS);
            }
            found += __popc(who);
        }
        if (lane == 0) sh.biases = found;
    }
    if (flag) atomicOr(&sh.flag, flag);
    __syncthreads();
    flag = sh.flag;
    if (A.flags && tid == 0 && blockIdx.y == 0 && blockIdx.z == 0) A.flags[b] = flag;
    if (flag) {
        for (int s = s0; s < s1; ++s)
            for (int v = lo + tid; v < hi; v += NT) store1<T>(A.out + (row_of(s) + v) * ES, NAN);
        return;
    }

    // ---- the entries that change ----
    for (int i0 = tid - lane; i0 < hi - lo; i0 += NT) {
        const bool on = i0 + lane < hi - lo && table[i0 + lane] != 0u;
        const uint32_t who = __ballot_sync(FULL, on);
        int at = 0;
        if (lane == 0 && who) at = atomicAdd(&sh.listed, __popc(who));
        at = __shfl_sync(FULL, at, 0);
        if (on) list[at + __popc(who & ((1u << lane) - 1u))] = static_cast<uint16_t>(i0 + lane);
    }
    __syncthreads();
    const int listed = sh.listed, turns = (s1 - s0 + ROWS - 1) / ROWS;
    for (int j = tid; j < listed * turns; j += NT) {
        const int turn = j / listed, at = list[j - turn * listed], v = lo + at, r0 = s0 + turn * ROWS;
        const uint32_t e = table[at];
        float x[ROWS];
        uint32_t may[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (r0 + r >= s1) break;
            x[r] = load1<T>(A.z + (row_of(r0 + r) + v) * ES);
            const uint32_t *mask = mask_of(r0 + r);
            may[r] = mask ? (__ldg(mask + (v >> 5)) >> (v & 31)) & 1u : 1u;
        }
        float bias = 0.f;
        if (e & BIAS)
            for (int i = 0; i < sh.biases; ++i)
                if (bias_id[i] == v) bias += bias_of[i];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int s = r0 + r;
            if (s >= s1) break;
            uint32_t count = e / ONE;
            if (e & DRAFT) {
                const uint64_t path = sh.path[s];
                for (int i = 0; i <= s; ++i) count += ((path >> i) & 1ull) && sh.token[i] == v ? 1u : 0u;
            }
            float y = x[r];
            if (count > 0 || (e & PROMPT)) y = y > 0.f ? __fdiv_rn(y, rho) : y * rho;
            if (count > 0) y = fmaf(-freq, static_cast<float>(count), y) - pres;
            if (e & BIAS) y += bias;
            if (may[r]) store1<T>(A.out + (row_of(s) + v) * ES, y);
        }
    }
}

}  // namespace

const void *adj_func(int dtype) {
    return dtype == 0 ? reinterpret_cast<const void *>(adjust_impl<float>) : reinterpret_cast<const void *>(adjust_impl<bf16_t>);
}

uint32_t adj_smem(int slice, int n_bias) { return static_cast<uint32_t>(slice) * 6 + n_bias * 8; }

}  // namespace mtp
