// tree_api.cu -- the C ABI of the tree-decoding operators (include/mtp_rs.h):
// argument validation, launch plans and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <cstdint>
#include <mutex>
#include <vector>

#include "mtp_rs.h"
#include "tree.h"

namespace {

using namespace mtp;

constexpr uint32_t kMaxSmem = 232448;  // 227 KB per CTA
constexpr float kLog2e = 1.4426950408889634f;

struct FuncInfo {
    int device;
    const void *func;
    uint32_t smem;
    int per_sm;  // resident CTAs per SM
};
struct DeviceInfo {
    int device, sms;
};
std::mutex g_mu;
std::vector<FuncInfo> g_funcs;
std::vector<DeviceInfo> g_devices;

bool device_sms(int &dev, int &sms) {
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    std::lock_guard<std::mutex> lk(g_mu);
    for (auto &d : g_devices)
        if (d.device == dev) {
            sms = d.sms;
            return true;
        }
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    try {
        g_devices.push_back({dev, sms});
    } catch (...) {  // out of memory: asked again next time
    }
    return true;
}

// Resident CTAs per SM of a kernel, its shared-memory limit raised first.
int resident(int dev, const void *func, uint32_t smem, int threads) {
    std::lock_guard<std::mutex> lk(g_mu);
    for (auto &f : g_funcs)
        if (f.device == dev && f.func == func && f.smem == smem) return f.per_sm;
    int n = 0;
    // the limit is the kernel's largest, not this call's size: calls of one
    // kernel differ in it
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, func) != cudaSuccess ||
        cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kMaxSmem - at.sharedSizeBytes)) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, func, threads, smem) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
    }
    try {
        g_funcs.push_back({dev, func, smem, n});
    } catch (...) {
    }
    return n;
}

// Every kernel here waits for the launches before it itself
// (griddepcontrol.wait) before it touches memory, and lets the next one's CTAs
// be set up early, so all are launched programmatically.
int launch(const void *func, dim3 grid, int threads, uint32_t smem, const void *args, mtp_stream_t stream,
           const void *map1 = nullptr, const void *map2 = nullptr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *kargs[] = {const_cast<void *>(args), const_cast<void *>(map1), const_cast<void *>(map2)};
    return cudaLaunchKernelExC(&cfg, func, kargs) == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

bool good_dtype(int d) { return d == MTP_DTYPE_F32 || d == MTP_DTYPE_BF16; }

// ------------------------------------------------------- tree attention --

struct AttnPlan {
    const void *func = nullptr;
    uint32_t smem = 0;
    int threads = 0, bm = 0, ktile = 0, per_page = 0, rows = 0, mtiles = 0, groups = 0, qrows = 0, qbufs = 1, slots = 0;
    long long max_tiles = 0;  // of one unit, the new keys' tile included
    size_t part_bytes = 0, desc_bytes = 0, late_bytes = 0;
    bool whole = false;       // units are not split
    bool joins() const { return !whole && max_tiles > 1 && groups > 1; }
    size_t bytes() const { return desc_bytes + late_bytes + (joins() ? part_bytes : 0); }
};

int attn_sizes(const mtp_tree_attention_args &a) {
    if (!good_dtype(a.dtype)) return MTP_ERR_UNSUPPORTED_DTYPE;
    if (a.B < 0 || a.T < 1 || a.T > MTP_MAX_NODES || a.Hkv < 1 || a.Hq < 1 || a.Hq % a.Hkv != 0 || a.Hq / a.Hkv > 4096 || a.D < 1 || a.D > 256 ||
        a.num_pages < 1 || a.page_size < 1 || a.max_pages < 1 || !(a.scale > 0.f) || a.scale > 1e30f)
        return MTP_ERR_INVALID_ARG;
    if (static_cast<long long>(a.max_pages) * a.page_size > 0x7fff0000ll || a.B > (1 << 20) || a.Hq > (1 << 16))
        return MTP_ERR_INVALID_ARG;
    return MTP_OK;
}

// Whether the tensor-core kernel takes these sizes: bfloat16, its head sizes,
// and pages whose rows are whole groups of the swizzle (8) or at least a tile.
bool umma_sizes(const mtp_tree_attention_args &a) {
    return a.dtype == MTP_DTYPE_BF16 && (a.D == 64 || a.D == 128 || a.D == 256) &&
           (a.page_size % 8 == 0 || a.page_size >= attn_umma_bn(a.D));
}

int attn_plan(const mtp_tree_attention_args &a, bool umma, AttnPlan &p) {
    int dev, sms;
    if (!device_sms(dev, sms)) return MTP_ERR_CUDA;
    const long long cap = static_cast<long long>(a.max_pages) * a.page_size;
    p.rows = a.T * (a.Hq / a.Hkv);
    if (umma) {
        const UmmaPlan u = attn_umma_plan(a.D, p.rows);
        p.func = u.func;
        p.smem = u.smem;
        p.threads = u.threads;
        p.bm = u.bm;
        p.qrows = u.qrows;
        p.qbufs = u.qbufs;
        p.slots = u.slots;
        const int bn = attn_umma_bn(a.D);
        p.per_page = a.page_size > bn && a.page_size % bn != 0 ? (a.page_size + bn - 1) / bn : 0;
        p.ktile = a.page_size >= bn ? bn : bn / a.page_size * a.page_size;
    } else {
        p.func = attn_simt_func(a.dtype, a.D);
        p.smem = attn_simt_smem(a.D);
        p.threads = SIMT_THREADS;
        p.bm = SIMT_BM;
        p.ktile = SIMT_BN;
    }
    const int per_sm = resident(dev, p.func, p.smem, p.threads);
    if (per_sm < 1) return MTP_ERR_NO_DEVICE;
    p.mtiles = (p.rows + p.bm - 1) / p.bm;
    p.max_tiles = 1 + (p.per_page ? static_cast<long long>(a.max_pages) * p.per_page : (cap + p.ktile - 1) / p.ktile);
    if (p.max_tiles * a.Hkv > 0x7fffffffll) return MTP_ERR_INVALID_ARG;  // tiles of a sequence are counted in 32 bits
    long long groups = static_cast<long long>(sms) * per_sm / p.mtiles;
    // Units are not split where that costs less.  Whole, the CTAs take them in
    // `waves` of max_tiles; split, all have the same number of tiles, and a
    // join and the ends of the pieces take as long as about six tiles on the
    // tensor cores, two of the other kernel.  (Whole against split: one token
    // after 256 8.3 and 13 us; 128 units of 1000 tokens 17 and 26 us, 512 of
    // 1000 65 and 73; all with a page table cut to the text.)  The lengths are not
    // known here, only the table's width: beyond 16 tiles, or four waves, one
    // long unit could cost more than it saves, so with a wide table short texts
    // are split as well.
    const long long units = static_cast<long long>(a.Hkv) * (a.B > 0 ? a.B : 1);
    const long long waves = (units + groups - 1) / (groups > 0 ? groups : 1);
    p.whole = umma ? p.max_tiles <= 16 && waves <= 4 && (waves * groups - units) * p.max_tiles <= 6 * groups
                   : p.max_tiles <= 2 && waves <= 2;
    const long long all = p.whole ? units : p.max_tiles * units;
    if (groups > all) groups = all;
    p.groups = static_cast<int>(groups < 1 ? 1 : groups);
    p.part_bytes = attn_slot_floats(p.bm, a.D) * 4 * 2 * p.groups * p.mtiles;
    p.part_bytes = (p.part_bytes + 15) / 16 * 16;
    p.desc_bytes = static_cast<size_t>(p.groups) * ATTN_DESC * sizeof(int32_t);
    p.late_bytes = umma ? (static_cast<size_t>(a.B) * 8 + 15) / 16 * 16 : 0;
    return MTP_OK;
}

// 64 bits that no other call has and that no memory holds by chance (the mixing
// is the finaliser of the SplitMix64 generator).
unsigned long long call_number() {
    static std::atomic<unsigned long long> count{
        static_cast<unsigned long long>(std::chrono::high_resolution_clock::now().time_since_epoch().count()) ^
        (static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(&g_mu)) << 20)};
    unsigned long long x = count.fetch_add(0x9e3779b97f4a7c15ull, std::memory_order_relaxed);
    x = (x ^ (x >> 30)) * 0xbf58476d1ce4e5b9ull;
    x = (x ^ (x >> 27)) * 0x94d049bb133111ebull;
    return x ^ (x >> 31);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// A paged cache as a 4-dimensional tensor (D, token, head, page), copied in
// boxes of 64 elements x `rows` tokens.  False where the addresses or strides
// cannot be described: the other kernel takes the call.
bool cache_map(CUtensorMap *map, const mtp_tree_attention_args &a, const void *base, const int64_t *s, int rows) {
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.D), static_cast<cuuint64_t>(a.page_size),
                                static_cast<cuuint64_t>(a.Hkv), static_cast<cuuint64_t>(a.num_pages)};
    const int64_t by[3] = {s[1], s[2], s[0]};
    cuuint64_t strides[3];
    for (int i = 0; i < 3; ++i) {
        const int64_t bytes = dims[i + 1] > 1 ? by[i] * 2 : static_cast<int64_t>(a.D) * 2;
        if (bytes <= 0 || bytes % 16 != 0 || bytes >= (1ll << 40)) return false;
        strides[i] = static_cast<cuuint64_t>(bytes);
    }
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1}, ones[4] = {1, 1, 1, 1};
    const EncodeTiled f = encode_tiled();
    return f && f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool vec_ok(const void *p, const int64_t *s, int es) {
    const int64_t v = 16 / es;
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && s[0] % v == 0 && s[1] % v == 0 && s[2] % v == 0;
}

}  // namespace

extern "C" int64_t mtp_tree_attention_workspace(const mtp_tree_attention_args *args) {
    if (!args || attn_sizes(*args) != MTP_OK) return -1;
    AttnPlan p;
    if (attn_plan(*args, false, p) != MTP_OK) return -1;
    size_t bytes = p.bytes();
    if (umma_sizes(*args)) {
        AttnPlan u;
        if (attn_plan(*args, true, u) != MTP_OK) return -1;
        if (u.bytes() > bytes) bytes = u.bytes();
    }
    return static_cast<int64_t>(bytes);
}

extern "C" int mtp_tree_attention(const mtp_tree_attention_args *args, mtp_stream_t stream) {
    if (!args) return MTP_ERR_INVALID_ARG;
    const mtp_tree_attention_args &a = *args;
    const int rc = attn_sizes(a);
    if (rc != MTP_OK) return rc;
    if (a.B == 0) return MTP_OK;
    if (!a.q || !a.k_new || !a.v_new || !a.k_cache || !a.v_cache || !a.page_table || !a.cache_len || !a.out || !a.workspace)
        return MTP_ERR_INVALID_ARG;
    const int es = a.dtype == MTP_DTYPE_F32 ? 4 : 2;
    const uintptr_t low = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k_new) |
                          reinterpret_cast<uintptr_t>(a.v_new) | reinterpret_cast<uintptr_t>(a.k_cache) |
                          reinterpret_cast<uintptr_t>(a.v_cache) | reinterpret_cast<uintptr_t>(a.out);
    if (low % es != 0 || reinterpret_cast<uintptr_t>(a.workspace) % 16 != 0) return MTP_ERR_MISALIGNED;
    TreeAttnArgs A = {};
    A.q = a.q;
    A.k_new = a.k_new;
    A.v_new = a.v_new;
    A.k_cache = a.k_cache;
    A.v_cache = a.v_cache;
    A.table = a.page_table;
    A.len = a.cache_len;
    A.parents = a.parents;
    A.nodes = a.n_nodes;
    A.out = a.out;
    A.lse = a.lse;
    A.flags = a.row_flags;
    // the stride of a dimension of one says nothing
    const int nq[3] = {a.B, a.T, a.Hq}, nk[3] = {a.B, a.T, a.Hkv}, nc[3] = {a.num_pages, a.page_size, a.Hkv};
    for (int i = 0; i < 3; ++i) {
        A.qs[i] = nq[i] > 1 ? a.q_stride[i] : 0;
        A.ks[i] = nk[i] > 1 ? a.k_new_stride[i] : 0;
        A.vs[i] = nk[i] > 1 ? a.v_new_stride[i] : 0;
        A.kcs[i] = nc[i] > 1 ? a.k_cache_stride[i] : 0;
        A.vcs[i] = nc[i] > 1 ? a.v_cache_stride[i] : 0;
    }
    A.B = a.B;
    A.T = a.T;
    A.Hq = a.Hq;
    A.Hkv = a.Hkv;
    A.D = a.D;
    A.G = a.Hq / a.Hkv;
    A.g_inverse = A.G == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + A.G - 1) / A.G);
    A.num_pages = a.num_pages;
    A.page_size = a.page_size;
    A.max_pages = a.max_pages;
    A.scale_log2 = a.scale * kLog2e;
    A.vec = a.D % (16 / es) == 0 && vec_ok(a.q, A.qs, es) && vec_ok(a.k_new, A.ks, es) && vec_ok(a.v_new, A.vs, es) &&
            vec_ok(a.k_cache, A.kcs, es) && vec_ok(a.v_cache, A.vcs, es);
    // the tensor cores wherever sizes and alignment allow: at one query row
    // of 128 they still keep up with the memory (a tile's products take 0.7
    // us, its bytes 1.5 us)
    CUtensorMap kmap, vmap;
    const int bn = attn_umma_bn(a.D), boxrows = a.page_size < bn ? a.page_size : bn;
    const bool umma = umma_sizes(a) && A.vec && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
                      cache_map(&kmap, a, a.k_cache, A.kcs, boxrows) && cache_map(&vmap, a, a.v_cache, A.vcs, boxrows);
    AttnPlan p;
    const int pc = attn_plan(a, umma, p);
    if (pc != MTP_OK) return pc;
    if (a.workspace_bytes < static_cast<int64_t>(p.bytes())) return MTP_ERR_INVALID_ARG;
    A.desc = static_cast<int32_t *>(a.workspace);
    A.late = reinterpret_cast<unsigned long long *>(static_cast<unsigned char *>(a.workspace) + p.desc_bytes);
    A.part = reinterpret_cast<float *>(static_cast<unsigned char *>(a.workspace) + p.desc_bytes + p.late_bytes);
    if (umma) {
        mtp_tuning tuning;
        (void)mtp_get_tuning(&tuning);
        A.number = call_number();
        A.wait_us = tuning.fault_wait_us > 0 ? static_cast<uint32_t>(tuning.fault_wait_us) : 2000000u;
        A.fault_cta = tuning.fault_skip_position;
    }
    A.rows = p.rows;
    A.mtiles = p.mtiles;
    A.groups = p.groups;
    A.bm = p.bm;
    A.whole = p.whole;
    A.ktile = p.ktile;
    A.extra = umma ? UMMA_EXTRA : 0;
    A.qrows = p.qrows;
    A.qbufs = p.qbufs;
    A.slots = p.slots;
    A.per_page = p.per_page;
    const int e = launch(p.func, dim3(p.groups * p.mtiles), p.threads, p.smem, &A, stream, &kmap, &vmap);
    if (e != MTP_OK || !p.joins()) return e;
    return launch(attn_join_func(a.dtype, a.D), dim3(p.groups * p.mtiles, ((p.rows < p.bm ? p.rows : p.bm) + JOIN_ROWS - 1) / JOIN_ROWS), JOIN_THREADS, 0, &A, stream);
}

// ------------------------------------------------------- beam selection --

namespace {

struct BeamPlan {
    int KL = 0, parts = 0, part_elems = 0;
    size_t n = 0;  // parts of all rows
    size_t bytes() const { return n * (12 + static_cast<size_t>(KL) * 8); }
};

int beam_sizes(int dtype, int B, int W, int V, int K) {
    if (!good_dtype(dtype)) return MTP_ERR_UNSUPPORTED_DTYPE;
    if (B < 0 || W < 1 || W > MTP_MAX_BEAMS || V < 1 || V > (1 << 24) || K < 1 || K > MTP_MAX_SELECT || B > (1 << 20))
        return MTP_ERR_INVALID_ARG;
    if (K > static_cast<long long>(W) * V) return MTP_ERR_INVALID_ARG;
    return MTP_OK;
}

int beam_plan(int dtype, int B, int W, int V, int K, BeamPlan &p) {
    int dev, sms;
    if (!device_sms(dev, sms)) return MTP_ERR_CUDA;
    const int vec = dtype == MTP_DTYPE_F32 ? 4 : 8;
    const int per_sm = resident(dev, beam_part_func(dtype), 0, BEAM_THREADS);
    if (per_sm < 1) return MTP_ERR_NO_DEVICE;
    // Parts of at least one round of a CTA each, and no more lists than the
    // join has threads.  Few rows: as many parts as fill the GPU once.  Many:
    // the number of parts (up to 8) that leaves the least of the last wave
    // idle; a part costs about three and a half rounds beside its own.
    const long long rows = static_cast<long long>(B > 0 ? B : 1) * W;
    const long long vecs = (V + vec - 1) / vec, round = BEAM_THREADS * 4, slots = static_cast<long long>(sms) * per_sm;
    long long most = (vecs + round - 1) / round;
    if (most > BEAM_THREADS / W) most = BEAM_THREADS / W;
    if (most < 1) most = 1;
    long long parts = slots / rows;
    if (parts < 8) {
        double best = 0.0;
        long long pick = 1;
        for (long long c = 1; c <= 8 && c <= most; ++c) {
            const long long waves = (rows * c + slots - 1) / slots;
            const double cost = static_cast<double>(waves) * (static_cast<double>(vecs) / (c * round) + 3.5);
            if (c == 1 || cost < best) {
                best = cost;
                pick = c;
            }
        }
        parts = pick;
    }
    if (parts > most) parts = most;
    const long long each = (vecs + parts - 1) / parts;
    p.parts = static_cast<int>((vecs + each - 1) / each);
    p.part_elems = static_cast<int>(each * vec);
    p.KL = K < V ? K : V;
    p.n = static_cast<size_t>(rows) * p.parts;
    return MTP_OK;
}

}  // namespace

extern "C" int64_t mtp_beam_select_workspace(mtp_dtype dtype, int B, int W, int V, int K) {
    if (beam_sizes(dtype, B, W, V, K) != MTP_OK) return -1;
    BeamPlan p;
    if (beam_plan(dtype, B, W, V, K, p) != MTP_OK) return -1;
    return static_cast<int64_t>(p.bytes());
}

extern "C" int mtp_beam_select(const void *logits, mtp_dtype dtype, const float *scores, const float *temperature, int B, int W,
                               int V, int K, int32_t *tokens, int32_t *parents, float *out_scores, int32_t *row_flags,
                               void *workspace, int64_t workspace_bytes, mtp_stream_t stream) {
    const int rc = beam_sizes(dtype, B, W, V, K);
    if (rc != MTP_OK) return rc;
    if (B == 0) return MTP_OK;
    if (!logits || !scores || !temperature || !tokens || !parents || !out_scores || !workspace) return MTP_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(workspace)) % 16 != 0) return MTP_ERR_MISALIGNED;
    BeamPlan p;
    const int pc = beam_plan(dtype, B, W, V, K, p);
    if (pc != MTP_OK) return pc;
    if (workspace_bytes < static_cast<int64_t>(p.bytes())) return MTP_ERR_INVALID_ARG;
    BeamArgs A = {};
    A.logits = logits;
    A.scores = scores;
    A.temp = temperature;
    A.B = B;
    A.W = W;
    A.V = V;
    A.K = K;
    A.KL = p.KL;
    A.parts = p.parts;
    A.part_elems = p.part_elems;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    A.part_sum = reinterpret_cast<float *>(ws);
    A.part_max = reinterpret_cast<float *>(ws + p.n * 4);
    A.part_flag = reinterpret_cast<int *>(ws + p.n * 8);
    A.cand_z = reinterpret_cast<float *>(ws + p.n * 12);
    A.cand_v = reinterpret_cast<int *>(ws + p.n * 12 + p.n * p.KL * 4);
    A.tokens = tokens;
    A.parents = parents;
    A.best = out_scores;
    A.flags = row_flags;
    const int e = launch(beam_part_func(dtype), dim3(static_cast<unsigned>(p.n)), BEAM_THREADS, 0, &A, stream);
    if (e != MTP_OK) return e;
    return launch(beam_join_func(), dim3(B), BEAM_THREADS, 0, &A, stream);
}

// --------------------------------------------------- reorder and commit ----

namespace {
struct Ints {  // n 32-bit integers at p, or none
    const int32_t *p;
    long long n;
    bool overlaps(const Ints &o) const {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        return p && o.p && a < b + static_cast<uintptr_t>(o.n) * 4 && b < a + static_cast<uintptr_t>(n) * 4;
    }
};
}  // namespace

extern "C" int mtp_beam_reorder(const void *states, const int32_t *parents, int N0, int B, int W, int K, int64_t row_bytes,
                                void *out, int32_t *row_flags, mtp_stream_t stream) {
    if (N0 < 0 || B < 0 || W < 1 || K < 1 || row_bytes < 0 || row_bytes > (1ll << 40)) return MTP_ERR_INVALID_ARG;
    const long long rows = static_cast<long long>(N0) * B * K;
    if (static_cast<long long>(N0) * B > (1ll << 31) / K) return MTP_ERR_INVALID_ARG;
    if (rows == 0 || row_bytes == 0) {  // nothing is moved: nothing is flagged
        if (row_flags && B > 0 &&
            cudaMemsetAsync(row_flags, 0, static_cast<size_t>(B) * sizeof(int32_t), reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
            return MTP_ERR_CUDA;
        return MTP_OK;
    }
    if (!states || !parents || !out) return MTP_ERR_INVALID_ARG;
    const uintptr_t s0 = reinterpret_cast<uintptr_t>(states), d0 = reinterpret_cast<uintptr_t>(out);
    const uintptr_t s1 = s0 + static_cast<uintptr_t>(N0) * B * W * row_bytes, d1 = d0 + static_cast<uintptr_t>(rows) * row_bytes;
    if (s0 < d1 && d0 < s1) return MTP_ERR_INVALID_ARG;  // a row may be read after it was written
    const uintptr_t low = s0 | d0 | static_cast<uintptr_t>(row_bytes);
    const int width = low % 16 == 0 ? 16 : low % 4 == 0 ? 4 : low % 2 == 0 ? 2 : 1;
    ReorderArgs A = {static_cast<const unsigned char *>(states), static_cast<unsigned char *>(out), parents, row_flags, N0, B, W,
                     K, row_bytes};
    const long long blocks = (row_bytes / width + REORDER_BLOCK - 1) / REORDER_BLOCK;
    if (blocks > 0x7fffffffll) return MTP_ERR_INVALID_ARG;
    return launch(reorder_func(width), dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(rows < 65535 ? rows : 65535)),
                  REORDER_THREADS, 0, &A, stream);
}

extern "C" int mtp_tree_commit(const mtp_tree_commit_args *args, mtp_stream_t stream) {
    if (!args) return MTP_ERR_INVALID_ARG;
    const mtp_tree_commit_args &a = *args;
    if (!good_dtype(a.dtype)) return MTP_ERR_UNSUPPORTED_DTYPE;
    if (a.layers < 0 || a.layers > 32767 || a.B < 0 || a.T < 1 || a.T > MTP_MAX_NODES) return MTP_ERR_INVALID_ARG;
    if ((a.layers > 0 || a.page_table) && (a.num_pages < 1 || a.page_size < 1 || a.max_pages < 1 ||
                                           static_cast<long long>(a.max_pages) * a.page_size > 0x7fff0000ll))
        return MTP_ERR_INVALID_ARG;
    if (a.layers > 0 && (a.Hkv < 1 || a.D < 1 || a.D > 4096 || a.Hkv > 65536)) return MTP_ERR_INVALID_ARG;
    if (a.layers > 0 && static_cast<long long>(a.T) * a.Hkv * a.D > (1ll << 30)) return MTP_ERR_INVALID_ARG;  // words of a path, in 32 bits
    if (a.B == 0) return MTP_OK;
    if (!a.tokens || !a.target_tokens || !a.out_tokens || !a.accept_len || !a.path || !a.new_len ||
        (a.layers > 0 && (!a.page_table || !a.cache_len || !a.k_new || !a.v_new || !a.k_cache || !a.v_cache)))
        return MTP_ERR_INVALID_ARG;
    const int es = a.dtype == MTP_DTYPE_F32 ? 4 : 2;
    CommitArgs A = {};
    A.tokens = a.tokens;
    A.target = a.target_tokens;
    A.parents = a.parents;
    A.nodes = a.n_nodes;
    A.table = a.page_table;
    A.len = a.cache_len;
    A.k_new = static_cast<const unsigned char *>(a.k_new);
    A.v_new = static_cast<const unsigned char *>(a.v_new);
    A.k_cache = static_cast<unsigned char *>(a.k_cache);
    A.v_cache = static_cast<unsigned char *>(a.v_cache);
    A.N0 = a.layers;
    A.B = a.B;
    A.T = a.T;
    A.Hkv = a.Hkv;
    A.row_bytes = a.D * es;
    A.num_pages = a.num_pages;
    A.page_size = a.page_size;
    A.max_pages = a.max_pages;
    A.out = a.out_tokens;
    A.accept = a.accept_len;
    A.path = a.path;
    A.new_len = a.new_len;
    A.flags = a.row_flags;
    uintptr_t low = 0;
    if (a.layers > 0) {
        low = reinterpret_cast<uintptr_t>(a.k_new) | reinterpret_cast<uintptr_t>(a.v_new) | reinterpret_cast<uintptr_t>(a.k_cache) |
              reinterpret_cast<uintptr_t>(a.v_cache);
        if (low % es != 0) return MTP_ERR_MISALIGNED;
        const int nn[4] = {a.layers, a.B, a.T, a.Hkv}, nc[4] = {a.layers, a.num_pages, a.page_size, a.Hkv};
        for (int i = 0; i < 4; ++i) {  // the stride of a dimension of one says nothing
            A.ks[i] = nn[i] > 1 ? a.k_new_stride[i] * es : 0;
            A.vs[i] = nn[i] > 1 ? a.v_new_stride[i] * es : 0;
            A.kcs[i] = nc[i] > 1 ? a.k_cache_stride[i] * es : 0;
            A.vcs[i] = nc[i] > 1 ? a.v_cache_stride[i] * es : 0;
            low |= static_cast<uintptr_t>(A.ks[i] | A.vs[i] | A.kcs[i] | A.vcs[i]);
        }
        low |= static_cast<uintptr_t>(A.row_bytes);
    }
    // every block of a sequence reads its inputs, one of them writes the outputs
    const long long each = a.B, nodes = each * a.T, table = each * a.max_pages;
    const Ints in[] = {{a.tokens, nodes}, {a.target_tokens, nodes}, {a.parents, nodes}, {a.n_nodes, each}, {a.page_table, table}, {a.cache_len, each}};
    const Ints out[] = {{a.out_tokens, nodes}, {a.path, nodes}, {a.accept_len, each}, {a.new_len, each}, {a.row_flags, each}};
    for (const Ints &o : out)
        for (const Ints &i : in)
            if (o.overlaps(i)) return MTP_ERR_INVALID_ARG;
    const int width = low % 16 == 0 ? 16 : low % 4 == 0 ? 4 : 2;
    return launch(commit_func(width), dim3(a.B, a.layers > 0 ? 2 * a.layers : 1), COMMIT_THREADS, 0, &A, stream);
}
