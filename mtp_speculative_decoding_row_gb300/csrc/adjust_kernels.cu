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
// Memory bounds the rows: every logit is read and written once, by a kernel that
// streams them through their masks (64 x 4 rows of 151936: 25 us, 28 with masks;
// floor 23).  A second one, a block to a slice of the vocabulary of one sequence,
// counts the slice's tokens of the text in shared memory (integers: the order of
// the atomic additions changes nothing) and lists the entries that anything but
// the mask changes, then, when the first is done, rewrites those, a thread to an
// entry.  A text's words crowd in few places: dealt out from a list they keep all
// threads busy (texts of 8192 tokens: 118 us where each streamed vector looked for
// its own, 54 so).  What bounds the second: its blocks' instructions -- each goes
// through the whole text of its sequence -- and the blocks of the first slices,
// where most words are.  Both in one kernel, with the rows in shared memory, took
// 71 us: a text was then counted four times as often.  Rows differ in their paths
// only; the few drafted tokens are looked up in the path where they occur, so that
// one count serves all rows.
#include "common.cuh"
#include "step.h"

namespace mtp {
namespace {

constexpr int NT = ADJ_THREADS, CT = ADJ_COUNT_THREADS;
// An entry of the table: in the text's first part; drafted or biased (look at
// the lists); occurrences in the rest of the text.  In 16 bits where the text is
// short enough for 14 bits of those: half the shared memory, so that all blocks
// of 64 sequences run at one time, beside the streaming kernel.
constexpr uint32_t PROMPT = 1u, LOOK = 2u, ONE = 4u;

template <bool SMALL>
struct Table {
    uint32_t *words;
    __device__ __forceinline__ void add(int i, uint32_t x) const {
        if (SMALL)
            atomicAdd(words + (i >> 1), x << (16 * (i & 1)));
        else
            atomicAdd(words + i, x);
    }
    __device__ __forceinline__ void set(int i, uint32_t bits) const {
        if (SMALL)
            atomicOr(words + (i >> 1), bits << (16 * (i & 1)));
        else
            atomicOr(words + i, bits);
    }
    __device__ __forceinline__ uint32_t get(int i) const { return SMALL ? reinterpret_cast<const uint16_t *>(words)[i] : words[i]; }
};

__device__ __forceinline__ uint32_t bf16_of(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// -inf in place of the elements whose bit is clear, the others bit for bit.
template <typename T>
__device__ __forceinline__ void masked(uint4 &x, uint32_t may) {
    if constexpr (Store<T>::ES == 4) {
        if (!(may & 1u)) x.x = 0xff800000u;
        if (!(may & 2u)) x.y = 0xff800000u;
        if (!(may & 4u)) x.z = 0xff800000u;
        if (!(may & 8u)) x.w = 0xff800000u;
    } else {
        auto two = [](uint32_t w, uint32_t bits) {
            const uint32_t keep = (bits & 1u) * 0xffffu | (bits & 2u) * 0x7fff8000u;
            return (w & keep) | (0xff80ff80u & ~keep);
        };
        x.x = two(x.x, may);
        x.y = two(x.y, may >> 2);
        x.z = two(x.z, may >> 4);
        x.w = two(x.w, may >> 6);
    }
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

// Nodes that sequence b has (all rows where the count is none: they become NaN).
__device__ __forceinline__ int nodes_of(const AdjArgs &A, int b, int &flag) {
    const int n = A.nodes ? __ldg(A.nodes + b) : A.S;
    if (n >= 0 && n <= A.S) return n;
    flag |= F_BAD_ID;
    return A.S;
}

// Bits of entries v, v + 1, .. v + VEC - 1 of a row's mask.
template <int VEC>
__device__ __forceinline__ uint32_t allowed(const uint32_t *mask, int v, int words) {
    if (!mask) return ~0u;
    const int i = v >> 5, r = v & 31;
    const uint32_t w = __ldg(mask + i);
    return r + VEC <= 32 ? w >> r : __funnelshift_r(w, i + 1 < words ? __ldg(mask + i + 1) : 0u, r);
}

// Row blockIdx.x through its mask: a block takes NT * AHEAD vectors, wherever the
// row starts, and the first one the entries before and behind them.
template <typename T, int AHEAD>
__global__ void __launch_bounds__(NT, 8) mask_impl(const __grid_constant__ AdjArgs A) {
    constexpr int VEC = Store<T>::VEC, ES = Store<T>::ES;
    constexpr uint32_t ALL = (1u << VEC) - 1u;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, b = blockIdx.x / A.S, s = blockIdx.x - b * A.S, words = (A.V + 31) / 32;
    const bool in_place = A.out == A.z;
    const uint32_t *mask = A.mask ? A.mask + b * A.mask_s[0] + s * A.mask_s[1] : nullptr;
    const size_t row = static_cast<size_t>(blockIdx.x) * A.V;
    const unsigned char *z = A.z + row * ES;
    unsigned char *out = A.out + row * ES;
    const int first = min(A.V, static_cast<int>((VEC - row % VEC) % VEC)), vecs = (A.V - first) / VEC, i0 = blockIdx.y * (NT * AHEAD) + tid;
    uint4 x[AHEAD];
    uint32_t may[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
        const int i = i0 + a * NT;
        if (i >= vecs) break;
        x[a] = *reinterpret_cast<const uint4 *>(z + static_cast<size_t>(first + i * VEC) * ES);
        may[a] = allowed<VEC>(mask, first + i * VEC, words);
    }
    int flag = 0;
    const int n = nodes_of(A, b, flag);  // (the loads are on their way)
    if (A.alone) {  // no second kernel follows
        if (A.flags && s == 0 && blockIdx.y == 0 && tid == 0) A.flags[b] = flag;
        if (flag) {
            for (int v = blockIdx.y * (NT * AHEAD) * VEC + tid; v < min(A.V, (static_cast<int>(blockIdx.y) + 1) * (NT * AHEAD) * VEC); v += NT)
                store1<T>(out + static_cast<size_t>(v) * ES, NAN);
            return;
        }
    }
    if (s >= n) return;
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
        const int i = i0 + a * NT;
        if (i >= vecs) break;
        if ((may[a] & ALL) != ALL)
            masked<T>(x[a], may[a]);
        else if (in_place)
            continue;
        *reinterpret_cast<uint4 *>(out + static_cast<size_t>(first + i * VEC) * ES) = x[a];
    }
    if (blockIdx.y != 0) return;
    const int tail = A.V - first - vecs * VEC;
    if (tid < first + tail) {
        const int v = tid < first ? tid : A.V - tail + (tid - first);
        store1<T>(out + static_cast<size_t>(v) * ES, allowed<1>(mask, v, words) & 1u ? load1<T>(z + static_cast<size_t>(v) * ES) : -INFINITY);
    }
}

template <typename T, bool SMALL>
__global__ void __launch_bounds__(CT, 4) adjust_impl(const __grid_constant__ AdjArgs A) {
    constexpr int ES = Store<T>::ES, ROWS = 4;
    extern __shared__ __align__(16) uint32_t smem[];
    constexpr int PER = SMALL ? 8 : 4;                                  // entries of 16 bytes
    const Table<SMALL> table = {smem};                                  // [slice]
    uint16_t *list = reinterpret_cast<uint16_t *>(smem + A.slice / PER * 4);  // [listed_most] entries that are not 0
    int *bias_id = reinterpret_cast<int *>(list + A.listed_most);       // [bias_room] of this slice, in their order, then -1
    float *bias_of = reinterpret_cast<float *>(bias_id + A.bias_room);  // [bias_room]
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.x;
    const int lo = blockIdx.y * A.slice, hi = min(A.V, lo + A.slice);  // this block's tokens
    if (tid == 0) sh.flag = sh.listed = sh.biases = 0;
    for (int i = tid; i < A.slice / PER; i += CT) reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    // (the first kernel has waited for those before it and writes nothing that is
    // read before it is done)
    if (!A.overlap) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- what the sequence has; every block finds the same flag ----
    int flag = 0;
    const int n = nodes_of(A, b, flag);
    int len = A.len ? __ldg(A.len + b) : 0, prompt = A.prompt ? __ldg(A.prompt + b) : 0;
    if (len < 0 || len > A.L) {
        flag |= F_BAD_ID;
        len = 0;
    }
    if (prompt < 0 || prompt > len) flag |= F_BAD_ID;
    const float rho = A.rho ? __ldg(A.rho + b) : 1.f, freq = A.freq ? __ldg(A.freq + b) : 0.f, pres = A.pres ? __ldg(A.pres + b) : 0.f;
    if (!(rho > 0.f && rho < INFINITY && fabsf(freq) < INFINITY && fabsf(pres) < INFINITY)) flag |= F_NONFINITE;
    auto row_of = [&](int s) { return (static_cast<size_t>(b) * A.S + s) * A.V; };

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
    for (int i = tid; i < A.n_bias; i += CT) {
        bias_id[i] = __ldg(A.bias_ids + static_cast<size_t>(b) * A.n_bias + i);
        bias_of[i] = __ldg(A.bias + static_cast<size_t>(b) * A.n_bias + i);
    }
    __syncthreads();  // the table is clear, the tokens and biases are there

    // ---- the text, drafted tokens, biases ----
    {
        int most = -1;
        const int32_t *text = A.history + static_cast<size_t>(b) * A.L;
        auto see = [&](int id, int at) {
            most = max(most, id);
            if (static_cast<uint32_t>(id) - static_cast<uint32_t>(lo) >= static_cast<uint32_t>(hi - lo)) return;
            if (at < prompt)
                table.set(id - lo, PROMPT);
            else
                table.add(id - lo, ONE);
        };
        const int vecs = A.vec_history ? len / 4 : 0;
#pragma unroll 4
        for (int i = tid; i < vecs; i += CT) {
            const int4 x = __ldg(reinterpret_cast<const int4 *>(text) + i);
            see(x.x, 4 * i);
            see(x.y, 4 * i + 1);
            see(x.z, 4 * i + 2);
            see(x.w, 4 * i + 3);
        }
#pragma unroll 4
        for (int i = 4 * vecs + tid; i < len; i += CT) see(__ldg(text + i), i);
        if (most >= A.V) flag |= F_BAD_ID;
    }
    if (A.tokens && tid < n) {
        const int id = sh.token[tid];
        if (id >= lo && id < hi) table.set(id - lo, LOOK);
    }
    if (A.n_bias > 0 && tid < 32) {  // this slice's, in their order, so that a sum of several has one value
        int found = 0;
        for (int i0 = 0; i0 < A.n_bias; i0 += 32) {
            const bool there = i0 + lane < A.n_bias;
            const int id = there ? bias_id[i0 + lane] : -1;
            const float value = there ? bias_of[i0 + lane] : 0.f;
            if (id >= A.V) flag |= F_BAD_ID;
            const bool in = id >= lo && id < hi;
            const uint32_t who = __ballot_sync(FULL, in);
            if (in) {
                const int at = found + __popc(who & ((1u << lane) - 1u));
                bias_id[at] = id;
                bias_of[at] = value;
                table.set(id - lo, LOOK);
            }
            __syncwarp();
            found += __popc(who);
        }
        if (lane < 4 && found + lane < A.bias_room) bias_id[found + lane] = -1;  // (read four at a time)
        if (lane == 0) sh.biases = found;
    }
    if (flag) atomicOr(&sh.flag, flag);
    __syncthreads();
    flag = sh.flag;
    if (A.flags && tid == 0 && blockIdx.y == 0) A.flags[b] = flag;
    if (flag) {
        if (A.overlap) asm volatile("griddepcontrol.wait;" ::: "memory");
        for (int s = 0; s < n; ++s)
            for (int v = lo + tid; v < hi; v += CT) store1<T>(A.out + (row_of(s) + v) * ES, NAN);
        return;
    }

    // ---- the entries that change ----
    for (int i = tid; i < A.slice / PER; i += CT) {  // (a slice is a multiple of PER times the threads of a warp)
        const uint4 e = reinterpret_cast<const uint4 *>(smem)[i];
        if (!__any_sync(FULL, (e.x | e.y | e.z | e.w) != 0u)) continue;
        const uint32_t w[4] = {e.x, e.y, e.z, e.w};
        int mine = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) mine += SMALL ? ((w[k] & 0xffffu) != 0u) + (w[k] >> 16 != 0u) : w[k] != 0u;
        int before = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(FULL, before, d);
            if (lane >= d) before += o;
        }
        int at = 0;
        if (lane == 31) at = atomicAdd(&sh.listed, before);
        at = __shfl_sync(FULL, at, 31) + before - mine;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (SMALL) {
                if (w[k] & 0xffffu) list[at++] = static_cast<uint16_t>(PER * i + 2 * k);
                if (w[k] >> 16) list[at++] = static_cast<uint16_t>(PER * i + 2 * k + 1);
            } else if (w[k]) {
                list[at++] = static_cast<uint16_t>(PER * i + k);
            }
        }
    }
    __syncthreads();
    if (A.overlap) asm volatile("griddepcontrol.wait;" ::: "memory");
    const int listed = sh.listed, turns = (n + ROWS - 1) / ROWS;
    for (int j = tid; j < listed * turns; j += CT) {
        const int turn = j / listed, at = list[j - turn * listed], v = lo + at, r0 = turn * ROWS;
        const uint32_t e = table.get(at);
        float x[ROWS];  // as they are behind their masks
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (r0 + r < n) x[r] = load1<T>(A.out + (row_of(r0 + r) + v) * ES);
        float bias = 0.f;
        bool biased = false;
        if (e & LOOK)
            for (int i = 0; i < sh.biases; i += 4) {
                const int4 id = *reinterpret_cast<const int4 *>(bias_id + i);
                if (id.x != v && id.y != v && id.z != v && id.w != v) continue;
                biased = true;
                if (id.x == v) bias += bias_of[i];
                if (id.y == v) bias += bias_of[i + 1];
                if (id.z == v) bias += bias_of[i + 2];
                if (id.w == v) bias += bias_of[i + 3];
            }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int s = r0 + r;
            if (s >= n) break;
            uint32_t count = e / ONE;
            if ((e & LOOK) && A.tokens) {
                const uint64_t path = sh.path[s];
                for (int i = 0; i <= s; ++i) count += ((path >> i) & 1ull) && sh.token[i] == v ? 1u : 0u;
            }
            float y = x[r];
            if (y == -INFINITY) {  // masked, or what no finite change would change
                const uint32_t *mask = A.mask ? A.mask + b * A.mask_s[0] + s * A.mask_s[1] : nullptr;
                if (bias < INFINITY || !(allowed<1>(mask, v, 0) & 1u)) continue;
            }
            if (count > 0 || (e & PROMPT)) y = y > 0.f ? __fdiv_rn(y, rho) : y * rho;
            if (count > 0) y = fmaf(-freq, static_cast<float>(count), y) - pres;
            if (biased) y += bias;
            store1<T>(A.out + (row_of(s) + v) * ES, y);
        }
    }
}

}  // namespace

const void *adj_func(int dtype, bool small) {
    if (dtype == 0) return small ? reinterpret_cast<const void *>(adjust_impl<float, true>) : reinterpret_cast<const void *>(adjust_impl<float, false>);
    return small ? reinterpret_cast<const void *>(adjust_impl<bf16_t, true>) : reinterpret_cast<const void *>(adjust_impl<bf16_t, false>);
}

const void *mask_func(int dtype, bool few) {
    if (dtype == 0) return few ? reinterpret_cast<const void *>(mask_impl<float, 1>) : reinterpret_cast<const void *>(mask_impl<float, 4>);
    return few ? reinterpret_cast<const void *>(mask_impl<bf16_t, 1>) : reinterpret_cast<const void *>(mask_impl<bf16_t, 4>);
}

uint32_t adj_smem(int slice, int listed, int biases, bool small) {
    return static_cast<uint32_t>(slice) * (small ? 2 : 4) + static_cast<uint32_t>(listed) * 2 + static_cast<uint32_t>(biases) * 8;
}

}  // namespace mtp
