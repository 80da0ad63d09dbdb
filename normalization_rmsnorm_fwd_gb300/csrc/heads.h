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

// How a tensor's position moves with a step: `step` elements, and `wrap` more
// where the step passes a token's last head.
struct Stride {
    int64_t step, wrap;
};

// The share of one tensor in a launch.  Warp w of it takes rows
// w run rps + i rps (i < run; rps rows at once), then the same `inc` rows on,
// and so forth: neighbouring warps read neighbouring memory at any time.
struct Share {
    int blocks;                  // CTAs
    int run;                     // steps of a run: kRun or 1
    int64_t rows;                // T * heads
    int64_t inc;                 // rows from a run to the warp's next
    // Inside a run [0] and to the next run [1]: tokens (dtc: modulo the rows
    // of cos_sin) and heads of a step, and the tensors' strides.
    int dt[2], dtc[2], dh[2];
    Stride in[2], in2[2], out[2];
};
// Steps of a run, and of a copy group of the rings.
constexpr int kRun = 2;

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
    int lanes;                   // lanes of a row
    int l1;                      // copies of a partly rotated row through L1 (split_sectors)
    Share share[3];
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
    float *part;                 // [CTAs of q, then of k][D] partial dw rows
    int lanes, l1;
    Share share[2];
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

// CTAs per SM of the forward and the append: 128 threads of at most 80
// registers, 16 KB of ring each.  The general code of an append with norms
// spills in 80 and has 102 (D = 80, 32 + 4 heads, T = 16000 48.5 -> 40.0 us).
constexpr int qk_fwd_ctas_per_sm(bool append, bool norm, bool general) { return append && norm && general ? 5 : 6; }
// Head sizes with code of their own (16-byte form).
inline bool own_code(int vec, int D) { return vec == 8 && (D == 64 || D == 128 || D == 192 || D == 256); }
// Most CTAs per SM of the backward (its workspace holds one row for each).
constexpr int kQkBwdCtasPerSm = 4;

// Deals `ctas` CTAs of `warps` warps out to n tensors of heads[i] heads
// (heads.cu) by their rows times the cost of a row: at least one CTA to each
// and no more than its rows fill; runs: runs of kRun steps where there are
// enough.
void deal(Share *s, const int *heads, const int *cost, int n, int64_t T, int cs_rows, int rows_per_step, int warps,
          int ctas, bool runs);
void set_strides(Stride (&d)[2], const Share &s, int H, int64_t ld, int64_t hs);

// Whether a row's two pieces (heads.cuh) meet inside a 32-byte sector.
bool split_sectors(int R, int D, const HeadView *v, int n);

// norm: with weights; vec: elements of an access, 8, 4 or 2 (row_lanes() at
// most 32), or 0: the element-wise form.
cudaError_t launch_qk_fwd(QkParams p, bool norm, bool append, int vec, int sms, cudaStream_t s);
cudaError_t launch_qk_bwd(QkBwdParams p, bool norm, int vec, int sms, cudaStream_t s);
// The kernels of one translation unit each (compiled in parallel).
cudaError_t run_qk_fwd(const QkParams &p, bool norm, dim3 grid, cudaStream_t s);
cudaError_t run_qk_append(const QkParams &p, bool norm, dim3 grid, cudaStream_t s);
cudaError_t run_qk_narrow(const QkParams &p, bool norm, bool append, int vec, dim3 grid, cudaStream_t s);
cudaError_t run_qk_bwd(const QkBwdParams &p, bool norm, dim3 grid, cudaStream_t s);
cudaError_t run_qk_bwd_narrow(const QkBwdParams &p, bool norm, int vec, dim3 grid, cudaStream_t s);
cudaError_t launch_rope(const RopeParams &p, bool vec, int sms, cudaStream_t s);

}  // namespace crmsn
