// attn.h -- parameter block and launches of the attention kernels
// (attn_*.cu), shared with the host ABI (api_attn.cu).
#pragma once

#include "heads.h"

namespace crmsn {

// Division of 0 <= x < 2^31 by a divisor known on the host: with
// l = ceil(log2 d) and mul = floor(2^(31+l) / d) + 1, mul d exceeds 2^(31+l)
// by at most 2^l, so x mul >> (31 + l) is the exact quotient.
struct FastDiv {
    uint32_t mul;
    int shift, d;
    FastDiv() = default;
    explicit FastDiv(int d_) : mul(0), shift(31), d(d_)
    {
        while (((int64_t)1 << (shift - 31)) < d) ++shift;
        mul = (uint32_t)((((uint64_t)1 << shift) / (uint64_t)d) + 1);
    }
    __host__ __device__ __forceinline__ int div(int x) const
    {
        return (int)(((uint64_t)(uint32_t)x * mul) >> shift);
    }
};

// Keys or values: a paged cache (strides of a page, a slot in it, a head), or
// [T, Hk, D] with ss the token stride.
struct KvView {
    const uint8_t *p;
    int64_t ps, ss, hs;          // elements
};

struct AttnParams {
    HeadView q, out;
    KvView kv[2];                // keys, values
    int kind;                    // CRMSN_CACHE_* of the keys and values
    const float *scale[2];       // FP8 caches: device scales of keys, values
    const int *table;            // page numbers (NULL: keys are the sequence's own tokens)
    int64_t ldt;
    int num_pages;
    FastDiv page;
    int max_keys;                // table_pages * page_size
    const int *lens;             // keys of each sequence (paged)
    const int *starts;           // first token of each sequence, or NULL: n each
    int n;
    int T, B, D, Hk;
    FastDiv group;               // query heads of a key head
    int causal, window;          // window 0: none
    int whole;                   // tiles are dealt whole (kShortKeys)
    float qk_scale;              // scale * log2(e)
    float *lse;
    uint8_t *ws;
#ifdef CRMSN_DEBUG
    DebugRanges dbg;
    int wait_tries;              // of a wait inside a kernel (0: as ever)
#endif
};

// Head sizes that the fast forms hold: D rounded up to one of these.
constexpr int kAttnMaxDim = 256;
inline int attn_padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : D <= 192 ? 192 : 256; }

// The workspace: a header for each CTA, then two parts for each CTA (the end
// of the tile that it finds begun, the beginning of the one that it leaves).
// A part of `rows` rows: their maxima and sums, then rows x DP sums of values.
struct AttnHeader {
    int64_t first, last, units;  // units of the tile's blocks; of all tiles of a head
    int groups, tile;            // groups that share them; 1: begins inside this tile
    int b, h, tok, ntok;         // sequence, key head, first token and tokens of the tile
    int pad[4];
};
static_assert(sizeof(AttnHeader) == 64, "one header");
constexpr int kAttnMaxCtas = 1024;
constexpr int64_t kAttnParts = (int64_t)kAttnMaxCtas * (int64_t)sizeof(AttnHeader);
// Groups of Hk CTAs that a device runs at once.  (One: no tile is shared, and
// neither headers nor parts are written.)
inline int attn_groups(int sms, int Hk)
{
    const int n = (sms < kAttnMaxCtas ? sms : kAttnMaxCtas) / Hk;
    return n < 1 ? 1 : n;
}
inline int64_t attn_part_floats(int rows, int DP) { return (int64_t)rows * (2 + DP); }

// Sequences of at most this many keys are dealt out by whole tiles, without a
// count of their blocks and without a second kernel.  Dealt whole against shared
// out, device us, heads of 128 in BF16 (by the call a lone short sequence takes
// 13.9 us against 19 to 20, for one launch and one allocation less):
//                             128 keys     384        640       1024       2048
//   1 token, 32 + 8 heads    4.6   6.2   7.3  7.7  10.0  7.9  13.8  8.5  24   10
//   16 of them               4.9   6.7   7.7 12.3  10.4 15.1  14.4 17.8  28   32
//   128 of them               23    24    49   53    69   72   100  100  184  179
//   16 of them, 16 + 16      7.5   9.3    13   17    18   22    29   32   51   52
//   a prompt, 32 + 8         9.4  14.4  12.5 19.2  16.0 26.8  20.9 34.0   62   58
//   8 prompts               10.6  15.4    29   39    56   68   104  106  344  275
// Only the lone token loses on the device from about 400 keys on, 2 us at the
// threshold; all others gain to 1024 and lose by 2048.
constexpr int kShortKeys = CRMSN_ATTENTION_SHORT;

// Joins the parts of the tiles that several CTAs shared (attn_combine.cu).
cudaError_t launch_attn_combine(const AttnParams &p, int rows, int DP, int groups, cudaStream_t s);

// At most 16 rows (tokens times heads of a group) of each sequence, the same
// number of tokens for all (attn_decode.cu).
constexpr int kDecodeRows = 16;
cudaError_t launch_attn_decode(const AttnParams &p, int sms, cudaStream_t s);

// Everything else of those head sizes and layouts, on the tensor cores
// (attn_tile_*.cu): attn_tile_rows() rows of a sequence and key head at once.
inline int attn_tile_rows(int DP) { return DP > 192 ? 128 : 256; }
cudaError_t launch_attn_tile_bf16(const AttnParams &p, int sms, cudaStream_t s);
cudaError_t launch_attn_tile_e4m3(const AttnParams &p, int sms, cudaStream_t s);
cudaError_t launch_attn_tile_e5m2(const AttnParams &p, int sms, cudaStream_t s);
// CTAs of the current device whose waits ran out since the last call; waits for the device's legacy stream.
cudaError_t take_given_up_bf16(unsigned int &n);
cudaError_t take_given_up_e4m3(unsigned int &n);
cudaError_t take_given_up_e5m2(unsigned int &n);

// One warp for each row (attn_row.cu): any layout and head size.
cudaError_t launch_attn_row(const AttnParams &p, int sms, cudaStream_t s);

}  // namespace crmsn
