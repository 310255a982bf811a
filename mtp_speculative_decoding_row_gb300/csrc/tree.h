// tree.h -- internal interface of the tree-decoding operators: tree attention
// over a paged cache, beam selection, beam reordering and tree commit.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mtp {

constexpr int MAX_NODES = 64;  // drafted nodes per tree: one 64-bit ancestor mask per node

// ------------------------------------------------------- tree attention --

struct TreeAttnArgs {
    const void *q, *k_new, *v_new, *k_cache, *v_cache;
    const int32_t *table;    // [B, max_pages]
    const int32_t *len;      // [B]
    const int32_t *parents;  // [B, T] or null (a chain)
    const int32_t *nodes;    // [B] or null (T)
    void *out;               // [B, T, Hq, D]
    float *lse;              // [B, T, Hq] or null
    int32_t *flags;          // [B] or null
    float *part;             // partial results, two slots per CTA (attn_slot_floats each)
    int32_t *desc;           // ATTN_DESC ints per group: the unit to join (see tree_attention.cuh)
    int64_t qs[3], ks[3], vs[3], kcs[3], vcs[3];  // element strides: (b, t, h) and (page, token, head)
    int B, T, Hq, Hkv, D, G;
    uint32_t g_inverse;      // ceil(2^32 / G); 0 for G = 1
    int num_pages, page_size, max_pages;
    int rows;                // T * G: query rows of one (sequence, key head)
    int mtiles;              // row tiles of BM rows
    int groups;              // CTAs / mtiles: each group of CTAs walks one range of key tiles
    int whole;               // units are not split: the groups share them out, not the tiles
    int extra;               // what a unit counts for beside its tiles, in tiles (see AttnWalk)
    int bm;                  // query rows of one tile
    int ktile;               // keys of one tile
    int per_page;            // tiles of one page where pages are larger than a tile and no multiple of it, else 0
    int qrows, qbufs, slots; // tensor-core kernel: query rows in shared memory (a multiple of 8), buffers for them, slots of its ring
    float scale_log2;        // scale * log2(e)
    int vec;                 // SIMT kernel: 16-byte loads are aligned
    // tensor-core kernel: how a wait that gave up is reported (see put_flag)
    unsigned long long *late;   // [B], workspace
    unsigned long long number;  // the call's
    uint32_t wait_us;           // limit of every wait
    int fault_cta;              // 1 + a CTA whose loader leaves out a signal (tests), else 0
};

constexpr int ATTN_DESC = 4;

// Floats of one partial slot: running maximum and sum of each row, then the
// unnormalised output rows.
__host__ __device__ inline size_t attn_slot_floats(int bm, int d) { return static_cast<size_t>(bm) * (d + 2); }

// SIMT kernel (csrc/tree_attention_simt.cu).
constexpr int SIMT_BM = 32, SIMT_BN = 64, SIMT_THREADS = 256;
const void *attn_simt_func(int dtype, int D);
uint32_t attn_simt_smem(int D);
// Tensor-core kernel (csrc/tree_attention_umma.cu): bfloat16, D 64, 128, 256.
constexpr uint32_t UMMA_SMEM = 232448;  // 227 KB per CTA
constexpr int UMMA_EXTRA = 3;
struct UmmaPlan {
    const void *func;
    int threads, bm, qrows, qbufs, slots;
    uint32_t smem;
};
UmmaPlan attn_umma_plan(int D, int rows);
int attn_umma_bn(int D);  // keys of a tile
const void *attn_join_func(int dtype, int D);
constexpr int JOIN_ROWS = 4, JOIN_THREADS = 128;  // rows of a block, a warp each

// ------------------------------------------------------- beam selection --

constexpr int BEAM_MAX_K = 64;     // continuations selected per sequence
constexpr int BEAM_MAX_W = 64;     // beams of a sequence

struct BeamArgs {
    const void *logits;   // [B, W, V]
    const float *scores;  // [B, W]
    const float *temp;    // [B]
    int B, W, V, K;
    int KL;               // candidates kept of each part: min(K, V)
    int parts;            // parts each row is cut into
    int part_elems;       // elements of one part (a multiple of the 16-byte vector)
    float *part_max;      // [B * W, parts] maximum of z
    float *part_sum;      // [B * W, parts] sum of 2^((z - max) k)
    int *part_flag;       // [B * W, parts]
    float *cand_z;        // [B * W, parts, KL] candidates, best first
    int *cand_v;          // their vocabulary indices (-1: none)
    int32_t *tokens, *parents;  // [B, K]
    float *best;                // [B, K]
    int32_t *flags;             // [B] or null
};

constexpr int BEAM_THREADS = 256, BEAM_PER_SM = 4;
const void *beam_part_func(int dtype);
const void *beam_join_func();

// ------------------------------------------------- reorder and commit ----

struct ReorderArgs {
    const unsigned char *src;  // [N0, B, W, bytes]
    unsigned char *dst;        // [N0, B, K, bytes]
    const int32_t *parents;    // [B, K]
    int32_t *flags;            // [B] or null
    int N0, B, W, K;
    long long bytes;           // of one row
};
const void *reorder_func(int width);  // word size: 16, 4, 2 or 1 bytes
constexpr int REORDER_THREADS = 256, REORDER_UNROLL = 4, REORDER_BLOCK = REORDER_THREADS * REORDER_UNROLL;  // words of a block

struct CommitArgs {
    const int32_t *tokens, *target, *parents, *nodes;  // [B, T]; nodes [B] or null
    const int32_t *table, *len;  // null where no cache is written: no pages to look at, lengths from 0
    const unsigned char *k_new, *v_new;
    unsigned char *k_cache, *v_cache;
    // byte strides: new (layer, b, t, h), cache (layer, page, token, head)
    long long ks[4], vs[4], kcs[4], vcs[4];
    int N0, B, T, Hkv;
    int row_bytes;  // bytes of one head's key or value
    int num_pages, page_size, max_pages;
    int32_t *out, *accept, *path, *new_len, *flags;
};
const void *commit_func(int width);  // word size: 16, 4 or 2 bytes
constexpr int COMMIT_THREADS = 128;

}  // namespace mtp
