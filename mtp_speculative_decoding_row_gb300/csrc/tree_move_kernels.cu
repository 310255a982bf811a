// tree_move_kernels.cu -- states of selected beams gathered by their parents,
// and the accepted path of a verified tree with its keys and values written
// into the paged cache.  Both move bytes: the element type only sets how wide
// a copy may be.  Replayed in a graph (a call through the binding takes two
// microseconds more): memory bounds a large reorder (887 MB read and written in
// 126 us, at the rate of a plain copy), latency the small ones (64 x 8 rows of 8
// KB: 2.4 us) and the commit (one sequence 3.1 us; 64 sequences of 16 layers
// 8.3 us, floor 4.3; with all 64 nodes of a chain accepted 110 us, 4.9 TB/s).
#include "common.cuh"
#include "tree.h"

namespace mtp {
namespace {

template <int WIDTH>
struct Word;
template <>
struct Word<16> {
    using type = uint4;
    static __device__ __forceinline__ type zero() { return make_uint4(0u, 0u, 0u, 0u); }
};
template <>
struct Word<4> {
    using type = uint32_t;
    static __device__ __forceinline__ type zero() { return 0u; }
};
template <>
struct Word<2> {
    using type = unsigned short;
    static __device__ __forceinline__ type zero() { return 0; }
};
template <>
struct Word<1> {
    using type = unsigned char;
    static __device__ __forceinline__ type zero() { return 0; }
};

// ------------------------------------------------------------- reorder ----

constexpr int RT = REORDER_THREADS, RU = REORDER_UNROLL;

// dst[n, b, k] = src[n, b, parents[b, k]]: block (x, y) copies words x RT RU
// .. of row y = (n B + b) K + k (rows beyond the grid's y extent in steps).
template <int WIDTH>
__global__ void __launch_bounds__(RT) reorder_impl(const __grid_constant__ ReorderArgs A) {
    using W = typename Word<WIDTH>::type;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long rows = static_cast<long long>(A.N0) * A.B * A.K, words = A.bytes / WIDTH;
    for (long long y = blockIdx.y; y < rows; y += gridDim.y) {
        const long long nb = y / A.K;
        const int b = static_cast<int>(nb % A.B);
        const int p = __ldg(A.parents + b * static_cast<long long>(A.K) + (y - nb * A.K));
        const bool ok = p >= 0 && p < A.W;
        const W *src = reinterpret_cast<const W *>(A.src + (nb * A.W + (ok ? p : 0)) * A.bytes);
        W *dst = reinterpret_cast<W *>(A.dst + y * A.bytes);
        const long long i0 = static_cast<long long>(blockIdx.x) * (RT * RU) + threadIdx.x;
        W v[RU];
#pragma unroll
        for (int u = 0; u < RU; ++u) v[u] = ok && i0 + u * RT < words ? __ldg(src + i0 + u * RT) : Word<WIDTH>::zero();
#pragma unroll
        for (int u = 0; u < RU; ++u)
            if (i0 + u * RT < words) dst[i0 + u * RT] = v[u];
        if (A.flags && blockIdx.x == 0 && y < static_cast<long long>(A.B) * A.K && y - nb * A.K == 0 && threadIdx.x == 0) {
            int flag = 0;
            for (int i = 0; i < A.K; ++i) {
                const int q = __ldg(A.parents + b * static_cast<long long>(A.K) + i);
                if (q < 0 || q >= A.W) flag = F_BAD_ID;
            }
            A.flags[b] = flag;
        }
    }
}

// -------------------------------------------------------------- commit ----

// Block (b, y): y = 2 layer + (0 keys, 1 values).  Its first warp walks the
// tree of sequence b -- two nodes to a lane; from node c on to its first child
// whose token is the target's token after c -- and then all threads copy the
// path's rows of this layer.  Every block of a sequence walks for itself: the
// walk is a few votes per step, less than a second launch.
template <int WIDTH>
__global__ void __launch_bounds__(COMMIT_THREADS) commit_impl(const __grid_constant__ CommitArgs A) {
    using W = typename Word<WIDTH>::type;
    __shared__ int s_target[MAX_NODES], s_token[MAX_NODES], s_path[MAX_NODES], s_page[MAX_NODES], s_off[MAX_NODES];
    __shared__ int s_count, s_flag;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int T = A.T;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int n = A.nodes ? __ldg(A.nodes + b) : T;
    const int len = A.len ? __ldg(A.len + b) : 0;
    int flag = 0;
    if (n < 0 || n > T) {
        flag = F_BAD_ID;
        n = 0;
    }
    if (len < 0 || (A.table && len > static_cast<long long>(A.max_pages) * A.page_size)) flag = F_BAD_ID;
    const size_t o = static_cast<size_t>(b) * T;
    if (tid < 32) {
        // everything that the walk needs, two nodes to a lane, loaded at once:
        // what bounds a block is the number of loads that wait for another
        int up[2], mine[2];
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = tid + 32 * e;
            up[e] = -2;
            mine[e] = 0;
            if (i < n) {
                mine[e] = __ldg(A.tokens + o + i);
                up[e] = A.parents ? __ldg(A.parents + o + i) : i - 1;
                s_target[i] = __ldg(A.target + o + i);
                s_token[i] = mine[e];
                bad |= up[e] >= i || up[e] < -1 || (i == 0 && up[e] != -1);
            }
        }
        // where tokens len, len + 1, .. go (as far as the table reaches)
        int page[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const long long pos = static_cast<long long>(len) + tid + 32 * e;
            page[e] = -1;
            if (A.table && flag == 0 && tid + 32 * e < n && pos < static_cast<long long>(A.max_pages) * A.page_size) {
                const int at = static_cast<int>(pos) / A.page_size;
                page[e] = __ldg(A.table + static_cast<size_t>(b) * A.max_pages + at);
                s_page[tid + 32 * e] = page[e];
                s_off[tid + 32 * e] = static_cast<int>(pos) - at * A.page_size;
            }
        }
        if (__any_sync(FULL, bad)) flag |= F_BAD_ID;
        __syncwarp();
        int count = 0;
        if (n > 0 && !flag) {
            int cur = 0;
            for (count = 1;; ++count) {
                if (tid == 0) s_path[count - 1] = cur;
                const int want = s_target[cur];
                if (want < 0) flag |= F_BAD_ID;  // no token (a flagged draw)
                const uint32_t lo = __ballot_sync(FULL, up[0] == cur && mine[0] == want);
                const uint32_t hi = __ballot_sync(FULL, up[1] == cur && mine[1] == want);
                if (!(lo | hi)) break;
                cur = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);  // a child comes after its parent: at most T steps
            }
            // no room for the path, or a page that is none
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (A.table && tid + 32 * e < count && (page[e] < 0 || page[e] >= A.num_pages)) flag |= F_BAD_ID;
        }
        flag = __reduce_or_sync(FULL, flag);
        if (flag) count = 0;
        if (tid == 0) {
            s_count = count;
            s_flag = flag;
        }
    }
    __syncthreads();
    const int count = s_count;
    if (blockIdx.y == 0) {
        for (int j = tid; j < T; j += COMMIT_THREADS) {
            A.path[o + j] = j < count ? s_path[j] : -1;
            A.out[o + j] = j + 1 < count ? s_token[s_path[j + 1]] : j + 1 == count ? s_target[s_path[j]] : -1;
        }
        if (tid == 0) {
            A.accept[b] = count - 1;
            A.new_len[b] = len + count;
            if (A.flags) A.flags[b] = s_flag;
        }
    }
    if (A.N0 == 0) return;
    const int layer = blockIdx.y >> 1;
    const bool val = blockIdx.y & 1;
    const long long *ns = val ? A.vs : A.ks, *cs = val ? A.vcs : A.kcs;
    const unsigned char *src = (val ? A.v_new : A.k_new) + layer * ns[0] + b * ns[1];
    unsigned char *dst = (val ? A.v_cache : A.k_cache) + layer * cs[0];
    const int words = A.row_bytes / WIDTH, per = A.Hkv * words;
    for (int i = tid; i < count * per; i += COMMIT_THREADS) {
        const int j = i / per, r = i - j * per, h = r / words, c = r - h * words;
        const W x = __ldg(reinterpret_cast<const W *>(src + s_path[j] * ns[2] + h * ns[3]) + c);
        *(reinterpret_cast<W *>(dst + s_page[j] * cs[1] + s_off[j] * cs[2] + h * cs[3]) + c) = x;
    }
}

}  // namespace

const void *reorder_func(int width) {
    return width == 16  ? reinterpret_cast<const void *>(reorder_impl<16>)
           : width == 4 ? reinterpret_cast<const void *>(reorder_impl<4>)
           : width == 2 ? reinterpret_cast<const void *>(reorder_impl<2>)
                        : reinterpret_cast<const void *>(reorder_impl<1>);
}

const void *commit_func(int width) {
    return width == 16  ? reinterpret_cast<const void *>(commit_impl<16>)
           : width == 4 ? reinterpret_cast<const void *>(commit_impl<4>)
                        : reinterpret_cast<const void *>(commit_impl<2>);
}

}  // namespace mtp
