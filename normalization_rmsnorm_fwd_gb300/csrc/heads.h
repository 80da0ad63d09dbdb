// heads.h -- parameter blocks and launches of the query / key kernels
// (heads_*.cu, rope.cu), shared with the host ABI (api_heads.cu).
#pragma once

#include "crmsnorm.h"
#include "launch.h"

namespace crmsn {

// [T, H, D] with a token stride and a head stride (elements).
struct HeadView {
    const uint16_t *p;
    int64_t ld, hs;
    int H;
};

// One layer of the cache: base, and strides of a page, a slot in it, a head.
struct CacheView {
    void *p;
    int64_t ps, ss, hs;
};

struct QkParams {
    HeadView in[3];              // q, k, v (v only for the append)
    HeadView out[2];             // q_out, k_out (k_out only without a cache)
    const void *w[2];            // wq, wk (both NULL: no norm)
    int w32;
    float bias, eps, inv_d;      // inv_d = 1 / D
    const float *cs;             // [cs_rows][>= R]: cosines, then sines
    int64_t ldcs;
    int cs_rows, R, pairs;
    int T, D;
    // append
    CacheView cache[2];
    int kind;                    // CRMSN_CACHE_*
    const float *scale[2];
    const void *slots;
    int slot64;
    int64_t num_slots;
    int page_size;
    // launch
    int heads;                   // rows per token: Hq + Hk (+ Hk)
    int lg;                      // log2 of the lanes of a row
    int chunks, steps;           // tasks per token, steps per task
#ifdef CRMSN_DEBUG
    DebugRanges dbg;
#endif
};

struct QkBwdParams {
    HeadView g[2], x[2], dx[2];  // of q and of k
    const void *w[2];
    int w32;
    float bias, eps, inv_d;
    const float *cs;
    int64_t ldcs;
    int cs_rows, R, pairs;
    int T, D;
    float *dw[2];
    float *part;                 // [nblk[0] + nblk[1]][D] partial dw rows
    int nblk[2];                 // CTAs of q and of k
    int lg;
    int chunks[2], steps[2];
#ifdef CRMSN_DEBUG
    DebugRanges dbg;
#endif
};

struct RopeParams {
    const void *pos;
    int pos64;
    int64_t ldp;                 // elements between axes
    int axes, mixed;
    int sections[4];             // columns of each axis
    const float *freq;
    float scaling;
    int64_t T;
    int half;                    // R / 2
    float *out;
    int64_t ldo;
#ifdef CRMSN_DEBUG
    DebugRanges dbg;
#endif
};

// Most CTAs per SM of the backward (its workspace holds one row for each).
constexpr int kQkBwdCtasPerSm = 4;

// norm: with weights; fast: the 16-byte form (D a multiple of 8, R of 16,
// aligned tensors).
cudaError_t launch_qk_fwd(QkParams p, bool norm, bool append, bool fast, int sms, cudaStream_t s);
cudaError_t launch_qk_bwd(QkBwdParams p, bool norm, bool fast, int sms, cudaStream_t s);
cudaError_t launch_rope(const RopeParams &p, bool vec, int sms, cudaStream_t s);

}  // namespace crmsn
