// seq_internal.h -- private declarations of the sequence operators (layer
// norm, rotary positions, attention): parameter blocks and launchers.
#pragma once

#include "dc1d_internal.h"

namespace dc1d {

// ---- layer norm over axis 1 -----------------------------------------------
//
// x [B][C][L] (L = 1: rows of C).  w, b may be null.  mean, rstd [B][L].
struct LayerNormArgs {
    const void *x, *w, *b, *g;  // g: the output's gradient (backward)
    void *y;                    // forward: y; backward: x's gradient (may be null)
    float *mean, *rstd;         // forward: written unless null; backward: read
    void *gw, *gb;              // backward: may be null
    int dtype;
    int64_t B, L;
    int C;
    float eps, inv_c;           // inv_c: 1 / C
    float *ws;                  // backward: the parameter gradients' partial sums
};
hipError_t launch_layer_norm(const LayerNormArgs &a, int num_cus, hipStream_t stream);
size_t layer_norm_backward_workspace(int64_t B, int C, int64_t L, int dtype, bool want_params, int num_cus);
hipError_t launch_layer_norm_backward(const LayerNormArgs &a, int num_cus, hipStream_t stream);

// ---- rotary positions -------------------------------------------------------

struct Strides3 {
    int64_t b, l, h;  // elements; the last dimension is contiguous
};
struct RotaryTensor {
    const void *x;
    void *y;
    Strides3 xs, ys;
    int H;
};
struct RotaryArgs {
    RotaryTensor t[2];  // queries and keys; t[1].H == 0: none
    const float *cos, *sin;  // [P][R]
    const int *pos;          // [B or 1][L][A]
    int64_t pos_b;           // elements between batches (0: shared)
    int dtype, B, L, D, R, A, P;
    int first[4];            // the first pair of each axis' section (R past the last)
    int interleaved;
    float sign;              // -1: the inverse rotation
};
hipError_t launch_rotary(const RotaryArgs &a, hipStream_t stream);

// ---- attention ----------------------------------------------------------------

// Query row r of a key head: position r / G, query head (head * G) + r % G,
// so that neighbouring rows share their keys and a tile of rows spans few
// positions.
struct AttnArgs {
    const void *q, *k, *v, *g;  // g: the output's gradient (backward)
    const void *o;              // backward: the forward's output
    void *out;                  // forward
    float *lse;                 // [B][Hq][Lq]; forward: written unless null, backward: read
    void *gq, *gk, *gv;
    Strides3 qs, ks, vs, os, gs, gqs, gks, gvs;
    const int *kv_lens, *q_start;  // [B] or null
    int dtype, B, Lq, Lk, Hq, Hkv, G, D;
    int64_t rows;               // Lq * G
    FastDiv by_G;
    int causal, window;         // window 0: none
    float scale;
    bool vec;                   // 16-byte pieces of every row are aligned
    int splits;                 // forward: parts of the keys; backward: parts of the rows
    int part_tiles;             // forward: tiles of 32 keys in a part
    float *part;                // the parts' partial sums
    float *delta;               // backward: sum_d g out, [B][Hkv][rows]
};

struct AttnPlan {
    const char *name;
    bool by_keys;  // the waves of a workgroup share its rows and split its keys
    int splits, part_tiles;
    int64_t blocks;
    size_t ws_bytes;
};
AttnPlan plan_attention(const AttnArgs &a, int num_cus);
hipError_t launch_attention(AttnArgs a, const AttnPlan &pl, void *ws, hipStream_t stream);

struct AttnBwdPlan {
    int splits;
    size_t ws_bytes, delta_bytes;
};
AttnBwdPlan plan_attention_backward(const AttnArgs &a, int num_cus);
hipError_t launch_attention_backward(AttnArgs a, const AttnBwdPlan &pl, void *ws, hipStream_t stream);

}  // namespace dc1d
