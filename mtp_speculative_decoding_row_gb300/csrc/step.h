// step.h -- internal interface of the operators around a verification step:
// rotary positions, appending to the paged cache, and the adjustment of logits.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mtp {

// --------------------------------------------------- rope and append ----

struct RotArgs {
    const unsigned char *q, *k, *v;  // [B, T, heads, D]; v of an append only
    unsigned char *q_out, *k_out;    // null: not written
    unsigned char *k_cache, *v_cache;
    long long qs[3], ks[3], vs[3], qos[3], kos[3];  // byte strides: b, t, head
    long long kcs[3], vcs[3];                       // page, token, head
    const int32_t *pos;     // [B, T] (element strides ps), or null: cache length + t
    long long ps[2];
    const float *inv_freq;  // [n]
    const int32_t *table, *len, *count;  // append: [B, max_pages], [B], [B] or null (T)
    int32_t *new_len, *flags;            // append: [B]; [B] or null
    int B, T, D, n;         // n pairs of each head are rotated
    int hq, hk, hv;         // heads of q, k and v that the call deals with
    int num_pages, page_size, max_pages;
    int tokens;             // of a block
    int chunks;             // blocks of a sequence
    int rot_units, units;   // of a head: units that rotate, all of them
    float factor, sign;     // of the rotation; -1 for the inverse
};
constexpr int ROT_THREADS = 256, ROT_MAX_TOKENS = 8;
const void *rot_func(int dtype, bool vec, bool interleaved, bool append);
uint32_t rot_smem(const RotArgs &A);

// ----------------------------------------------------- adjust logits ----

constexpr int ADJ_THREADS = 256, ADJ_COUNT_THREADS = 512, ADJ_MAX_ROWS = 64;

struct AdjArgs {
    const unsigned char *z;  // [B, S, V]
    unsigned char *out;      // the same, or z itself
    const int32_t *history;  // [B, L] or null
    const int32_t *len, *prompt;                // [B]; [B] or null (0)
    const int32_t *tokens, *parents, *nodes;    // [B, S] or null; [B, S] or null (a chain); [B] or null (S)
    const float *rho, *freq, *pres;             // [B] or null (1, 0, 0)
    const int32_t *bias_ids;                    // [B, n_bias] or null
    const float *bias;
    const uint32_t *mask;                       // words, rows of mask_s[0] (b) and mask_s[1] (s) words, or null
    long long mask_s[2];
    int32_t *flags;
    int B, S, V, L, n_bias;
    int slice;               // vocabulary entries of a block (a multiple of 256)
    int listed_most;         // entries of a slice that can change (a multiple of 8)
    int bias_room;           // n_bias and four more, a multiple of 4; 0 for none
    int alone;               // nothing but masks: the first kernel is the only one
    int overlap;             // launched behind the kernel of the masks, beside which it may run
    int vec_history;         // 16-byte loads of the history are aligned
};
const void *adj_func(int dtype, bool small);  // small: tables of 16 bits, texts of up to ADJ_SMALL tokens
const void *mask_func(int dtype, bool few);  // few: a block takes a quarter of the vectors
constexpr int ADJ_SMALL = 16383, ADJ_SLICE = 8192, ADJ_SMALL_SLICE = 20480;
uint32_t adj_smem(int slice, int listed, int biases, bool small);

}  // namespace mtp
