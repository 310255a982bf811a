// step_api.cu -- the C ABI of the rotary positions, the cache append and the
// adjustment of logits (include/mtp_rs.h): argument validation and launches.
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "mtp_rs.h"
#include "step.h"

namespace {

using namespace mtp;

// A tensor [n0, n1, n2, row] of `row` contiguous bytes: its byte strides (of a
// dimension of one: 0, it says nothing) and the memory between its first and
// last byte.
struct Span {
    uintptr_t lo = 0, hi = 0;
    bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
};
struct Rows {
    Span span;
    bool gaps = true;  // no stride of 0: no two indices are one place
    uintptr_t low = 0; // the bits of the address and the strides
    int n[3] = {};     // sizes; 1 where the stride is 0
    long long s[3] = {}, row = 0;
    // False for a stride or a tensor that no memory has (|stride| < 2^40 elements
    // times the dimension within 2^62 bytes).
    bool set(const void *p, const int64_t *stride, const int (&size)[3], long long bytes, int es, long long *out) {
        span.lo = reinterpret_cast<uintptr_t>(p);
        unsigned long long reach = 0;
        low = span.lo;
        row = bytes;
        for (int i = 0; i < 3; ++i) {
            out[i] = 0;
            n[i] = 1;
            if (size[i] <= 1) continue;
            if (stride[i] < 0 || stride[i] >= (1ll << 40)) return false;
            out[i] = s[i] = stride[i] * es;
            if (out[i] == 0)
                gaps = false;
            else
                n[i] = size[i];
            low |= static_cast<uintptr_t>(out[i]);
            const unsigned long long far = static_cast<unsigned long long>(out[i]) * (size[i] - 1);
            if (out[i] > 0 && far / out[i] != static_cast<unsigned long long>(size[i] - 1)) return false;
            reach += far;
            if (far >= (1ull << 61) || reach >= (1ull << 61)) return false;
        }
        span.hi = span.lo + reach + row;
        return true;
    }
};

bool same(const long long (&a)[3], const long long (&b)[3]) { return a[0] == b[0] && a[1] == b[1] && a[2] == b[2]; }

// Whether a row at `off` bytes meets one at a sum of d_i s[i], -back[i] <= d_i <=
// ahead[i], strides falling: of each d_i only those matter that leave what the
// other strides reach.
bool reaches(long long off, const long long *s, const long long *back, const long long *ahead, int i, long long row) {
    if (i == 3) return -row < off && off < row;
    long long left = row, right = row;  // off lies in (-left, right) of the rest
    for (int j = i + 1; j < 3; ++j) {
        left += back[j] * s[j];
        right += ahead[j] * s[j];
    }
    if (s[i] == 0) return reaches(off, s, back, ahead, i + 1, row);
    long long lo = -back[i], hi = ahead[i];
    while (lo <= hi && off - lo * s[i] >= right) {  // too far ahead: d has to be larger
        const long long step = (off - lo * s[i] - right) / s[i] + 1;
        lo += step;
    }
    while (lo <= hi && off - hi * s[i] <= -left) {
        const long long step = (-left - (off - hi * s[i])) / s[i] + 1;
        hi -= step;
    }
    if (hi - lo > 3) return true;  // strides that do not nest: taken for a meeting
    for (long long d = lo; d <= hi; ++d)
        if (reaches(off - d * s[i], s, back, ahead, i + 1, row)) return true;
    return false;
}

// Whether two tensors have a byte in common.  Parts of one tensor, of the same
// strides, may lie between one another's rows; of other strides they are taken to
// meet where their ranges do.
bool meet(const Rows &a, const Rows &b) {
    if (!a.span.meets(b.span)) return false;
    long long s[3], back[3], ahead[3];
    for (int i = 0; i < 3; ++i) {
        if (a.n[i] > 1 && b.n[i] > 1 && a.s[i] != b.s[i]) return true;
        s[i] = a.n[i] > 1 ? a.s[i] : b.n[i] > 1 ? b.s[i] : 0;
        back[i] = b.n[i] - 1;  // the place of a less that of b: (index of a - index of b) strides
        ahead[i] = a.n[i] - 1;
    }
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (s[j] < s[j + 1]) {
                const long long t[3] = {s[j], back[j], ahead[j]};
                s[j] = s[j + 1], back[j] = back[j + 1], ahead[j] = ahead[j + 1];
                s[j + 1] = t[0], back[j + 1] = t[1], ahead[j + 1] = t[2];
            }
    return reaches(static_cast<long long>(b.span.lo - a.span.lo), s, back, ahead, 0, a.row);
}

// `out` of a tensor `in`, of the same shape: in place, or apart from it; and
// apart from `other`, another input of the call (which may lie between the rows of
// an output that is in place, but is read by other threads than write it).
bool out_of(const Rows &out, const long long (&os)[3], const Rows &in, const long long (&is)[3], const Rows *other) {
    if (!out.gaps) return false;
    if (out.span.lo == in.span.lo && same(os, is)) return !(other && meet(out, *other));
    return !out.span.meets(in.span) && !(other && out.span.meets(other->span));
}

Span ints(const int32_t *p, long long n) {
    Span s;
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = p ? s.lo + static_cast<uintptr_t>(n) * 4 : s.lo;
    return s;
}

constexpr int kMostHeads = 65536;

int rot_launch(RotArgs &A, int dtype, uintptr_t low, bool interleaved, bool append, mtp_stream_t stream) {
    int dev, sms;
    if (!device_sms(dev, sms)) return MTP_ERR_CUDA;
    const int es = dtype == MTP_DTYPE_F32 ? 4 : 2, width = 16 / es;
    const bool vec = low % 16 == 0 && A.n % width == 0 && A.D % width == 0;
    const int piece = vec ? width : 1;
    A.rot_units = A.n / piece;
    A.units = A.rot_units + (A.D - 2 * A.n) / piece;
    // Tokens of a block, which share its start (heads of 128, bfloat16, captured
    // calls in turn).  Few tokens, few to a block, so that no SM is idle: of 40 heads
    // 256 tokens take 2.9, 3.1 and 4.0 us with one, two and four (160 appended ones
    // 3.8, 4.2 and 5.2), 512 tokens 4.0, 3.5 and 4.1.  Then four (1024: 5.7, 5.7
    // and 4.9; 16384: 71, 58 and 54, eight 55), though 2048 in two waves take 9.0
    // and with two 7.4.  Eight where there are many and their heads few (16384 of 9
    // heads: four 19.8, eight 17.5; but 4096 6.4 and 7.3).
    const long long all = static_cast<long long>(A.B) * A.T, units = 4ll * (A.hq + A.hk + A.hv) * A.units;
    A.tokens = all <= 2ll * sms ? 1 : all <= 4ll * sms ? 2 : units < 4 * ROT_THREADS && all > 32ll * sms ? 8 : 4;
    if (A.tokens > A.T) A.tokens = A.T;
    A.chunks = static_cast<int>((static_cast<long long>(A.T) + A.tokens - 1) / A.tokens);
    const long long blocks = static_cast<long long>(A.B) * A.chunks;
    if (blocks > 0x7fffffffll) return MTP_ERR_INVALID_ARG;
    return launch(rot_func(dtype, vec, interleaved, append), dim3(static_cast<unsigned>(blocks)), ROT_THREADS, rot_smem(A), &A, stream);
}

bool aligned(const Rows &r, int es) { return r.span.lo % es == 0; }

}  // namespace

extern "C" int mtp_rope(const mtp_rope_args *args, mtp_stream_t stream) {
    if (!args) return MTP_ERR_INVALID_ARG;
    const mtp_rope_args &a = *args;
    if (!good_dtype(a.dtype)) return MTP_ERR_UNSUPPORTED_DTYPE;
    if (a.B < 0 || a.T < 0 || a.Hq < 0 || a.Hkv < 0 || a.Hq > kMostHeads || a.Hkv > kMostHeads || a.D < 1 || a.D > 256 || a.pairs < 0 ||
        2 * static_cast<long long>(a.pairs) > a.D || !(a.factor - a.factor == 0.f))
        return MTP_ERR_INVALID_ARG;
    if (a.B == 0 || a.T == 0 || (a.Hq == 0 && a.Hkv == 0)) return MTP_OK;
    if ((a.Hq > 0 && (!a.q || !a.q_out)) || (a.Hkv > 0 && (!a.k || !a.k_out)) || !a.positions || (a.pairs > 0 && !a.inv_freq))
        return MTP_ERR_INVALID_ARG;
    const int es = a.dtype == MTP_DTYPE_F32 ? 4 : 2;
    const long long row = static_cast<long long>(a.D) * es;
    RotArgs A = {};
    const int nq[3] = {a.B, a.T, a.Hq}, nk[3] = {a.B, a.T, a.Hkv};
    Rows q, k, qo, ko;
    uintptr_t low = 0;
    if (a.Hq > 0) {
        if (!q.set(a.q, a.q_stride, nq, row, es, A.qs) || !qo.set(a.q_out, a.q_out_stride, nq, row, es, A.qos)) return MTP_ERR_INVALID_ARG;
        low |= q.low | qo.low;
    }
    if (a.Hkv > 0) {
        if (!k.set(a.k, a.k_stride, nk, row, es, A.ks) || !ko.set(a.k_out, a.k_out_stride, nk, row, es, A.kos)) return MTP_ERR_INVALID_ARG;
        low |= k.low | ko.low;
    }
    if ((a.Hq > 0 && !out_of(qo, A.qos, q, A.qs, a.Hkv > 0 ? &k : nullptr)) || (a.Hkv > 0 && !out_of(ko, A.kos, k, A.ks, a.Hq > 0 ? &q : nullptr)))
        return MTP_ERR_INVALID_ARG;
    if (a.Hq > 0 && a.Hkv > 0 && meet(qo, ko)) return MTP_ERR_INVALID_ARG;
    if (low % es != 0) return MTP_ERR_MISALIGNED;
    A.q = static_cast<const unsigned char *>(a.q);
    A.k = static_cast<const unsigned char *>(a.k);
    A.q_out = static_cast<unsigned char *>(a.q_out);
    A.k_out = static_cast<unsigned char *>(a.k_out);
    A.pos = a.positions;
    A.ps[0] = a.B > 1 ? a.pos_stride[0] : 0;
    A.ps[1] = a.T > 1 ? a.pos_stride[1] : 0;
    A.inv_freq = a.inv_freq;
    A.B = a.B;
    A.T = a.T;
    A.D = a.D;
    A.n = a.pairs;
    A.hq = a.Hq;
    A.hk = a.Hkv;
    A.factor = a.factor;
    A.sign = a.inverse ? -1.f : 1.f;
    return rot_launch(A, a.dtype, low, a.interleaved != 0, false, stream);
}

extern "C" int mtp_cache_append(const mtp_cache_append_args *args, mtp_stream_t stream) {
    if (!args) return MTP_ERR_INVALID_ARG;
    const mtp_cache_append_args &a = *args;
    if (!good_dtype(a.dtype)) return MTP_ERR_UNSUPPORTED_DTYPE;
    if (a.B < 0 || a.T < 1 || a.Hq < 0 || a.Hkv < 1 || a.Hq > kMostHeads || a.Hkv > kMostHeads || a.D < 1 || a.D > 256 || a.pairs < 0 ||
        2 * static_cast<long long>(a.pairs) > a.D || !(a.factor - a.factor == 0.f) || a.num_pages < 1 || a.page_size < 1 || a.max_pages < 1 ||
        static_cast<long long>(a.max_pages) * a.page_size > 0x7fff0000ll)
        return MTP_ERR_INVALID_ARG;
    if (a.B == 0) return MTP_OK;
    if (!a.k || !a.v || !a.k_cache || !a.v_cache || !a.page_table || !a.cache_len || !a.new_len || (a.Hq > 0 && (!a.q || !a.q_out)) ||
        (a.pairs > 0 && !a.inv_freq))
        return MTP_ERR_INVALID_ARG;
    const int es = a.dtype == MTP_DTYPE_F32 ? 4 : 2;
    const long long row = static_cast<long long>(a.D) * es;
    RotArgs A = {};
    const int nq[3] = {a.B, a.T, a.Hq}, nk[3] = {a.B, a.T, a.Hkv}, nc[3] = {a.num_pages, a.page_size, a.Hkv};
    Rows q, k, v, qo, ko, kc, vc;
    if (!k.set(a.k, a.k_stride, nk, row, es, A.ks) || !v.set(a.v, a.v_stride, nk, row, es, A.vs) ||
        !kc.set(a.k_cache, a.k_cache_stride, nc, row, es, A.kcs) || !vc.set(a.v_cache, a.v_cache_stride, nc, row, es, A.vcs))
        return MTP_ERR_INVALID_ARG;
    uintptr_t low = k.low | v.low | kc.low | vc.low;
    if (!kc.gaps || !vc.gaps || meet(kc, vc) || kc.span.meets(k.span) || kc.span.meets(v.span) || vc.span.meets(k.span) || vc.span.meets(v.span))
        return MTP_ERR_INVALID_ARG;
    if (a.Hq > 0) {
        if (!q.set(a.q, a.q_stride, nq, row, es, A.qs) || !qo.set(a.q_out, a.q_out_stride, nq, row, es, A.qos)) return MTP_ERR_INVALID_ARG;
        low |= q.low | qo.low;
        if (!out_of(qo, A.qos, q, A.qs, &k) || kc.span.meets(q.span) || vc.span.meets(q.span) || kc.span.meets(qo.span) || vc.span.meets(qo.span))
            return MTP_ERR_INVALID_ARG;
        if (qo.span.lo == q.span.lo ? meet(qo, v) : qo.span.meets(v.span)) return MTP_ERR_INVALID_ARG;
    }
    if (a.k_out) {
        if (!ko.set(a.k_out, a.k_out_stride, nk, row, es, A.kos)) return MTP_ERR_INVALID_ARG;
        low |= ko.low;
        if (!out_of(ko, A.kos, k, A.ks, a.Hq > 0 ? &q : nullptr) || kc.span.meets(ko.span) || vc.span.meets(ko.span)) return MTP_ERR_INVALID_ARG;
        if (ko.span.lo == k.span.lo ? meet(ko, v) : ko.span.meets(v.span)) return MTP_ERR_INVALID_ARG;
        if (a.Hq > 0 && meet(qo, ko)) return MTP_ERR_INVALID_ARG;
    }
    if (low % es != 0) return MTP_ERR_MISALIGNED;
    // every block of a sequence reads its lengths and pages, one writes the outputs
    const Span in[] = {ints(a.cache_len, a.B), ints(a.n_new, a.B), ints(a.page_table, static_cast<long long>(a.B) * a.max_pages)};
    for (const Span &o : {ints(a.new_len, a.B), ints(a.row_flags, a.B)})
        for (const Span &i : in)
            if (o.meets(i)) return MTP_ERR_INVALID_ARG;
    A.q = static_cast<const unsigned char *>(a.q);
    A.k = static_cast<const unsigned char *>(a.k);
    A.v = static_cast<const unsigned char *>(a.v);
    A.q_out = static_cast<unsigned char *>(a.q_out);
    A.k_out = static_cast<unsigned char *>(a.k_out);
    A.k_cache = static_cast<unsigned char *>(a.k_cache);
    A.v_cache = static_cast<unsigned char *>(a.v_cache);
    A.pos = a.positions;
    A.ps[0] = a.B > 1 ? a.pos_stride[0] : 0;
    A.ps[1] = a.T > 1 ? a.pos_stride[1] : 0;
    A.inv_freq = a.inv_freq;
    A.table = a.page_table;
    A.len = a.cache_len;
    A.count = a.n_new;
    A.new_len = a.new_len;
    A.flags = a.row_flags;
    A.B = a.B;
    A.T = a.T;
    A.D = a.D;
    A.n = a.pairs;
    A.hq = a.Hq;
    A.hk = a.Hkv;
    A.hv = a.Hkv;
    A.num_pages = a.num_pages;
    A.page_size = a.page_size;
    A.max_pages = a.max_pages;
    A.factor = a.factor;
    A.sign = 1.f;
    return rot_launch(A, a.dtype, low, a.interleaved != 0, true, stream);
}

extern "C" int mtp_adjust_logits(const mtp_adjust_args *args, mtp_stream_t stream) {
    if (!args) return MTP_ERR_INVALID_ARG;
    const mtp_adjust_args &a = *args;
    if (!good_dtype(a.dtype)) return MTP_ERR_UNSUPPORTED_DTYPE;
    if (a.B < 0 || a.B > (1 << 20) || a.S < 1 || a.S > MTP_MAX_NODES || a.V < 1 || a.V > (1 << 24) || a.L < 0 || a.L > (1 << 28) || a.n_bias < 0 ||
        a.n_bias > MTP_MAX_BIAS)
        return MTP_ERR_INVALID_ARG;
    if (a.B == 0) return MTP_OK;
    if (!a.logits || !a.out || (a.L > 0 && (!a.history || !a.history_len)) || (a.prompt_len && !a.history_len) || (a.parents && !a.tokens) ||
        (a.n_bias > 0 && (!a.bias_ids || !a.bias)))
        return MTP_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.out)) % 16 != 0) return MTP_ERR_MISALIGNED;
    const int es = a.dtype == MTP_DTYPE_F32 ? 4 : 2;
    const uintptr_t z = reinterpret_cast<uintptr_t>(a.logits), o = reinterpret_cast<uintptr_t>(a.out);
    const uintptr_t bytes = static_cast<uintptr_t>(a.B) * a.S * a.V * es;
    if (z != o && z < o + bytes && o < z + bytes) return MTP_ERR_INVALID_ARG;
    if (a.mask && (a.mask_stride[0] < 0 || a.mask_stride[1] < 0)) return MTP_ERR_INVALID_ARG;
    int dev, sms;
    if (!device_sms(dev, sms)) return MTP_ERR_CUDA;
    AdjArgs A = {};
    A.z = static_cast<const unsigned char *>(a.logits);
    A.out = static_cast<unsigned char *>(a.out);
    A.L = a.history ? a.L : 0;
    A.history = a.history;
    A.len = a.history_len;
    A.prompt = a.prompt_len;
    A.tokens = a.tokens;
    A.parents = a.parents;
    A.nodes = a.n_nodes;
    A.rho = a.repetition;
    A.freq = a.frequency;
    A.pres = a.presence;
    A.bias_ids = a.bias_ids;
    A.bias = a.bias;
    A.n_bias = a.n_bias;
    A.mask = reinterpret_cast<const uint32_t *>(a.mask);
    A.mask_s[0] = a.B > 1 ? a.mask_stride[0] : 0;
    A.mask_s[1] = a.S > 1 ? a.mask_stride[1] : 0;
    A.flags = a.row_flags;
    A.B = a.B;
    A.S = a.S;
    A.V = a.V;
    A.vec_history = reinterpret_cast<uintptr_t>(a.history) % 16 == 0 && a.L % 4 == 0;
    // Slices as large as leaves a block for every place on the GPU: each reads the
    // text, and those that wait for a place count nothing beside the first kernel.
    // (64 sequences, 4 rows of 151936, in slices of 8192, two rounds of blocks,
    // and of 16,896, one: drafts and biases 36 and 28 us, with texts of 8192 tokens
    // 52 and 54.)
    const bool small = A.L <= ADJ_SMALL;
    const void *adjust = adj_func(a.dtype, small);
    const int most = small ? ADJ_SMALL_SLICE : ADJ_SLICE;
    A.bias_room = a.n_bias > 0 ? (a.n_bias + 7) / 4 * 4 : 0;
    // (raises the kernel's limit of shared memory, too)
    const int per_sm = resident(dev, adjust, adj_smem(most, most, MTP_MAX_BIAS + 4, small), ADJ_COUNT_THREADS);
    if (per_sm < 1) return MTP_ERR_NO_DEVICE;
    const long long places = static_cast<long long>(sms) * (2048 / ADJ_COUNT_THREADS);
    long long parts = places / a.B;
    parts = parts < 1 ? 1 : parts;
    const long long each = (a.V + parts - 1) / parts;
    A.slice = static_cast<int>(each < 1024 ? 1024 : each > most ? most : (each + 255) / 256 * 256);
    if (A.slice > most) A.slice = most;
    const long long events = (static_cast<long long>(A.L) + (a.tokens ? a.S : 0) + a.n_bias + 7) / 8 * 8;
    A.listed_most = static_cast<int>(events < A.slice ? events : A.slice);
    if (z != o || a.mask) {  // (in place and without a mask nothing is streamed)
        const long long rows = static_cast<long long>(a.B) * a.S, vecs = (static_cast<long long>(a.V) * es + 15) / 16;
        const bool few = rows * ((vecs + 4 * ADJ_THREADS - 1) / (4 * ADJ_THREADS)) < 4 * sms;
        A.alone = !a.history && !a.tokens && a.n_bias == 0 && !a.repetition && !a.frequency && !a.presence;
        const long long each = ADJ_THREADS * (few ? 1 : 4);
        const int rc = launch(mask_func(a.dtype, few), dim3(static_cast<unsigned>(rows), static_cast<unsigned>((vecs + each - 1) / each)),
                              ADJ_THREADS, 0, &A, stream);
        if (rc != MTP_OK || A.alone) return rc;
        A.overlap = 1;
    }
    // (the sequences next to one another: the first slices, of the most frequent
    // words, start first)
    return launch(adjust, dim3(a.B, (a.V + A.slice - 1) / A.slice), ADJ_COUNT_THREADS, adj_smem(A.slice, A.listed_most, A.bias_room, small), &A, stream);
}
