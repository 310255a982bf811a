// rope_kernels.cu -- rotary positions of queries and keys, and the same on the
// way into the paged cache.
//
// Pair i of a head, (a, b) = (x_i, x_{n+i}) or (x_{2i}, x_{2i+1}), becomes
//   f (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq[i],
// with sin t negated for the inverse (the transpose, so the gradient).
//
// The angle is reduced in whole numbers: inv_freq / 2 pi is a 64-bit fraction
// of a turn, and its product with the position, modulo 2^64, is the angle
// modulo one turn -- to 2^-32 turns at any 32-bit position and frequencies of up to
// one radian, where a product in float32 is off by whole radians from position 10^7 on.
//
// A block takes a few tokens of one sequence.  Its threads first start the
// loads of their first elements, then compute each of the tokens' n angles
// once, into shared memory, where all heads read them.
//
// Memory bounds it: 16384 tokens of 32 and 8 heads of 128 (bfloat16) 54 us, 6.2
// TB/s, 0.92 of a copy's rate; appended with their values and rotated queries 86
// us for 20,481 tokens, 0.86.  256 tokens take 3 us: the launch, and where they are
// appended three loads that wait for one another (length, page, row).
#include "common.cuh"
#include "step.h"

namespace mtp {
namespace {

// inv_freq / 2 pi as a 64-bit fraction of a turn (modulo 1).
__device__ __forceinline__ uint64_t turns_of(float w) {
    const uint32_t bits = __float_as_uint(w);
    const int e = static_cast<int>((bits >> 23) & 255u);
    const uint64_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
    const uint64_t K = 0xa2f9836e4e441529ull;  // 2^66 / 2 pi
    // |w| = m 2^(max(e, 1) - 150), so |w| / 2 pi = m K 2^-(s + 64) turns
    const int s = 152 - (e ? e : 1);
    const uint64_t hi = __umul64hi(m, K), lo = m * K;
    uint64_t f = 0;
    if (s <= 0)
        f = s > -64 ? lo << -s : 0ull;
    else if (s < 64)
        f = (hi << (64 - s)) | (lo >> s);
    else if (s < 128)
        f = hi >> (s - 64);
    return bits >> 31 ? 0ull - f : f;
}

// (cos, sin) of position * w, times f (sin also times `sign`).
__device__ __forceinline__ float2 angle(float w, int position, float f, float sign) {
    const uint64_t p = turns_of(w) * static_cast<uint64_t>(static_cast<int64_t>(position));
    const uint32_t quarter = static_cast<uint32_t>((p + (1ull << 61)) >> 62);
    // what is left of the quarter turn: [-1/8, 1/8) turns, in half turns
    const float x = __ll2float_rn(static_cast<int64_t>(p - (static_cast<uint64_t>(quarter) << 62))) * 0x1p-63f;
    float s, c;
    sincospif(x, &s, &c);
    const float cs = quarter & 1u ? s : c, sn = quarter & 1u ? c : s;
    const float cc = ((quarter + 1u) & 2u) ? -cs : cs, ss = (quarter & 2u) ? -sn : sn;
    if (!(fabsf(w) < INFINITY)) return make_float2(NAN, NAN);
    return make_float2(cc * f, ss * f * sign);
}

// VEC elements at once: 16 bytes, or one element.
template <typename T, int VEC>
struct Piece {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[VEC]) { Store<T>::unpack(r, x); }
    static __device__ __forceinline__ Raw pack(const float (&x)[VEC]) {
        if constexpr (Store<T>::ES == 4)
            return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
            return make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};
template <>
struct Piece<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[1]) { x[0] = r; }
    static __device__ __forceinline__ Raw pack(const float (&x)[1]) { return x[0]; }
};
template <>
struct Piece<bf16_t, 1> {
    using Raw = uint16_t;
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[1]) { x[0] = __uint_as_float(static_cast<uint32_t>(r) << 16); }
    static __device__ __forceinline__ Raw pack(const float (&x)[1]) {
        uint16_t r;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x[0]));
        return r;
    }
};

constexpr long long NO_ROW = -(1ll << 62);

// A head is `rot_units` units that rotate two pieces and units that copy one.
// Item i of a block is head i % H of token i / H, heads of q first, then of k,
// then of v; a thread has the same unit of every (threads / units)-th item.
template <typename T, int VEC, bool PAIRS, bool APPEND>
__global__ void __launch_bounds__(ROT_THREADS) rot_impl(const __grid_constant__ RotArgs A) {
    using P = Piece<T, VEC>;
    using Raw = typename P::Raw;
    constexpr int ES = Store<T>::ES;
    extern __shared__ __align__(16) float2 angles[];  // [tokens][n], see `place`
    __shared__ long long s_k[ROT_MAX_TOKENS], s_v[ROT_MAX_TOKENS];
    const int tid = threadIdx.x;
    const int b = blockIdx.x / A.chunks, t0 = (blockIdx.x - b * A.chunks) * A.tokens;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int nt = A.T, len = 0, flag = 0;
    if (APPEND) {
        len = __ldg(A.len + b);
        nt = A.count ? __ldg(A.count + b) : A.T;
        const long long room = static_cast<long long>(A.max_pages) * A.page_size;
        if (nt < 0 || nt > A.T || len < 0 || static_cast<long long>(len) + nt > room) {
            flag = F_BAD_ID;
            nt = 0;
        }
        if (t0 == 0) {  // this block speaks for the sequence
            if (nt > 0) {
                const int p0 = len / A.page_size, p1 = static_cast<int>((static_cast<uint32_t>(len) + nt - 1) / A.page_size);
#pragma unroll 4
                for (int i = p0 + tid; i <= p1; i += ROT_THREADS) {
                    const int p = __ldg(A.table + static_cast<size_t>(b) * A.max_pages + i);
                    if (p < 0 || p >= A.num_pages) flag = F_BAD_ID;
                }
            }
            flag = __syncthreads_or(flag) ? F_BAD_ID : 0;
            if (tid == 0) {
                A.new_len[b] = flag ? len : len + nt;
                if (A.flags) A.flags[b] = flag;
            }
        }
    }
    nt = min(nt - t0, A.tokens);  // of this block
    if (nt <= 0) return;
    const int H = A.hq + A.hk + A.hv, items = nt * H;
    const int u = tid % A.units, par = ROT_THREADS / A.units;
    int i = tid / A.units;
    if (i >= par) i = items;  // (threads that are left over)
    const bool rot = u < A.rot_units;
    // elements of the unit's first piece, and how far its second one is
    const int off = rot ? (PAIRS ? 2 * u * VEC : u * VEC) : 2 * A.n + (u - A.rot_units) * VEC, more = PAIRS ? VEC : A.n;

    auto source = [&](int item, int &token, int &head) {
        token = item / H;
        head = item - token * H;
        const long long t = t0 + token;
        if (head < A.hq) return A.q + b * A.qs[0] + t * A.qs[1] + head * A.qs[2];
        if (head < A.hq + A.hk) return A.k + b * A.ks[0] + t * A.ks[1] + (head - A.hq) * A.ks[2];
        return A.v + b * A.vs[0] + t * A.vs[1] + (head - A.hq - A.hk) * A.vs[2];
    };
    Raw x0 = {}, x1 = {};
    int token = 0, head = 0;
    auto fetch = [&]() {
        const unsigned char *p = source(i, token, head) + off * ES;
        x0 = *reinterpret_cast<const Raw *>(p);
        if (rot) x1 = *reinterpret_cast<const Raw *>(p + more * ES);
    };
    if (i < items) fetch();

    // the angles: those of one unit lie `rot_units` vectors of two apart, so that
    // neighbouring units read neighbouring vectors
    auto place = [&](int tok, int c) {
        if (VEC == 1) return tok * A.n + c;
        const int unit = c / VEC, e = c % VEC;
        return tok * A.n + 2 * ((e >> 1) * A.rot_units + unit) + (e & 1);
    };
    for (int j = tid; j < nt * A.n; j += ROT_THREADS) {
        const int tok = j / A.n, c = j - tok * A.n;
        const int pos = A.pos ? __ldg(A.pos + b * A.ps[0] + (t0 + tok) * A.ps[1]) : len + t0 + tok;
        angles[place(tok, c)] = angle(__ldg(A.inv_freq + c), pos, A.factor, A.sign);
    }
    if (APPEND && tid < nt) {
        const int at = len + t0 + tid, page = __ldg(A.table + static_cast<size_t>(b) * A.max_pages + at / A.page_size);
        const bool ok = page >= 0 && page < A.num_pages;
        const long long row = at % A.page_size;
        s_k[tid] = ok ? page * A.kcs[0] + row * A.kcs[1] : NO_ROW;
        s_v[tid] = ok ? page * A.vcs[0] + row * A.vcs[1] : NO_ROW;
    }
    __syncthreads();
    while (i < items) {
        Raw y0 = x0, y1 = x1;
        const int tok = token, h = head;
        const bool turns = rot && h < A.hq + A.hk;
        i += par;
        if (i < items) fetch();  // the next item is on its way
        if (turns) {
            float a[VEC], c[VEC];
            P::unpack(y0, a);
            P::unpack(y1, c);
            float2 t[VEC];
            if constexpr (VEC == 1) {
                t[0] = angles[tok * A.n + u];
            } else {
                const float4 *from = reinterpret_cast<const float4 *>(angles + tok * A.n) + u;
#pragma unroll
                for (int e = 0; e < VEC; e += 2) {
                    const float4 w = from[(e >> 1) * A.rot_units];
                    t[e] = make_float2(w.x, w.y);
                    t[e + 1] = make_float2(w.z, w.w);
                }
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                // half layout: (a[e], c[e]); pairs: neighbours among a, then c
                float &lo = !PAIRS || VEC == 1 ? a[e] : 2 * e < VEC ? a[(2 * e) % VEC] : c[(2 * e) % VEC];
                float &hi = !PAIRS || VEC == 1 ? c[e] : 2 * e < VEC ? a[(2 * e + 1) % VEC] : c[(2 * e + 1) % VEC];
                const float l = lo, r = hi;
                lo = l * t[e].x - r * t[e].y;
                hi = r * t[e].x + l * t[e].y;
            }
            y0 = P::pack(a);
            y1 = P::pack(c);
        }
        auto put = [&](unsigned char *p) {
            p += off * ES;
            *reinterpret_cast<Raw *>(p) = y0;
            if (rot) *reinterpret_cast<Raw *>(p + more * ES) = y1;
        };
        const long long t = t0 + tok;
        if (h < A.hq) {
            put(A.q_out + b * A.qos[0] + t * A.qos[1] + h * A.qos[2]);
        } else if (h < A.hq + A.hk) {
            const int g = h - A.hq;
            if (A.k_out) put(A.k_out + b * A.kos[0] + t * A.kos[1] + g * A.kos[2]);
            if (APPEND && s_k[tok] != NO_ROW) put(A.k_cache + s_k[tok] + g * A.kcs[2]);
        } else if (APPEND && s_v[tok] != NO_ROW) {
            put(A.v_cache + s_v[tok] + (h - A.hq - A.hk) * A.vcs[2]);
        }
    }
}

template <typename T>
const void *pick(bool vec, bool pairs, bool append) {
    constexpr int V = Store<T>::VEC;
    if (vec)
        return append ? (pairs ? reinterpret_cast<const void *>(rot_impl<T, V, true, true>) : reinterpret_cast<const void *>(rot_impl<T, V, false, true>))
                      : (pairs ? reinterpret_cast<const void *>(rot_impl<T, V, true, false>) : reinterpret_cast<const void *>(rot_impl<T, V, false, false>));
    return append ? (pairs ? reinterpret_cast<const void *>(rot_impl<T, 1, true, true>) : reinterpret_cast<const void *>(rot_impl<T, 1, false, true>))
                  : (pairs ? reinterpret_cast<const void *>(rot_impl<T, 1, true, false>) : reinterpret_cast<const void *>(rot_impl<T, 1, false, false>));
}

}  // namespace

const void *rot_func(int dtype, bool vec, bool interleaved, bool append) {
    return dtype == 0 ? pick<float>(vec, interleaved, append) : pick<bf16_t>(vec, interleaved, append);
}

uint32_t rot_smem(const RotArgs &A) { return static_cast<uint32_t>(A.tokens) * A.n * sizeof(float2); }

}  // namespace mtp
