// attn_tile.cuh -- attention on the tensor cores: chunks, prompts, and every
// batch that attn_decode.cu does not take.
//
// A tile is NT x 128 rows of one sequence and key head: consecutive tokens
// times the query heads of the key head, so that grouped heads share the tile's
// keys.  Its keys come in blocks of BN.  For each block and each 128 rows
//   S = Q K^T (tcgen05, FP32 in tensor memory),  P = 2^(c S - c M) (registers),
//   O += P V  (tcgen05, P read from tensor memory, where it replaces S).
//
// 16 warps: 0-3 and 4-7 work out the weights of the two halves of a tile, one
// row a thread, so that a row's maximum and sum never leave the thread; 8-11
// copy keys and values (FP8: convert what 14 and 15 copy); 12 issues the
// products; 13 walks through the CTA's work and tells the others piece by piece.
// While one half's weights are worked out, the tensor cores run the other half's
// products: S of the next block follows O of this one at once.  Heads of 256
// leave no room for two halves in tensor memory (O takes 256 of its 512
// columns); there one half has two S, and S of the next block runs ahead of O
// of this one.
//
// The reference M of a row's weights is a maximum of before; it moves only when
// the true one has passed it by 2^kLag, as moving it means reading and writing O.
// A weight is then at most 2^8 (FP16: 2^kWeightTop), its rounding relative as ever.
//
// Keys and values: 16-byte asynchronous copies (any page size; what lies behind
// the last key becomes zeros), into the swizzled layout that the products read;
// FP8 codes to slots of their own, from where they become FP16 (exact).  The
// blocks of a tile, and the tiles that a CTA works through, form one stream:
// loads run ahead across the ends of tiles, and so do the next tile's queries.
//
// Work is shared out by blocks (share_work): CTAs that meet inside a tile write
// parts, which attn_combine.cu joins.
//
// What it takes (GB300, 32 + 8 heads of 128), call after call: 16384 tokens
// 1556 us, 1413 TFLOP/s, 72 % of the rate of a large BF16 product alone and 82 %
// of its rate under the power cap, which holds here too (1750 to 1900 MHz; after
// a pause, at 2070 MHz, 1430 us); 2048 tokens over 32768 keys in pages of 64,
// 806 us (736).  What bounds it: the products of two halves over 128 keys take
// 2048 cycles, their round longer: a half's scores, 270 cycles for their maximum,
// 1200 for the weights and its products do not fit behind the other half's
// products (an earlier form took 3000, and 1389 of 1501 us with nothing to load).
// A piece's end costs some 4000 cycles, mostly instructions that arrive from the
// L2 cache: this kernel's code is larger than the SM keeps, and shorter loops at
// a tile's end were faster than unrolled ones.  Halves in turn and a reference
// that may lag are published techniques for these tensor cores.  Tried and left: the halves of a tile of
// 128 rows taking every other block (no faster: 222 against 215 us for one chunk
// among single tokens), results staged in shared memory (a stage of keys less).
#pragma once

#include "attn.cuh"
#include "tcgen05.cuh"

namespace crmsn {

template <int KIND, int DP>
struct TileShape {
    static constexpr bool FP8 = KIND != KV_BF16;
    static constexpr int NT = DP > 192 ? 1 : 2;              // halves of 128 rows
    static constexpr int NS = 3 - NT;                        // S of a half
    static constexpr int BN = DP > 128 ? 64 : 128;           // keys of a block
    static constexpr int ROWS = NT * 128;
    static constexpr int QBYTES = 128 * DP * 2;              // queries of a half
    static constexpr int STAGE = BN * DP * 2;                // keys or values of a block
    static constexpr int STAGES = DP == 64 ? (FP8 ? 5 : 8) : (FP8 ? 3 : 5);
    static constexpr int RAW = FP8 ? BN * DP : 0;            // FP8 codes of a block
    static constexpr int RAWS = FP8 ? (DP == 64 ? 8 : 4) : 0;
    static constexpr int SMEM = 1024 + NT * QBYTES + STAGES * STAGE + RAWS * RAW;
    static constexpr int OCOL = DP == 256 ? 256 : NT * NS * BN;   // columns of S, then of O
    // Registers of a thread: of the 128 at launch the copying and the issuing
    // warps give up what the weights' warps need.  The loops that the compiler
    // makes of it differ from step to step and not in one direction (BF16, by the
    // call: 16384 tokens 1577, 1966, 1610, 1670 us at 144, 152, 160, 168, 24 packed
    // prompts 460, 565, 476, 483; FP8, whose copying warps convert: a chunk among
    // single tokens 200, 200, 221 at 144, 152, 160).
    static constexpr int REGS = FP8 ? 152 : 144, OTHER_REGS = 256 - REGS;
    static_assert(OCOL + NT * DP <= 512, "tensor memory");
    static constexpr int STATIC = 2048;                      // for what is not dynamic
    static_assert(SMEM + STATIC <= 227 * 1024, "shared memory");
};
constexpr int kLag = 8;              // binary digits by which a row's reference may lag behind its maximum
constexpr int kTileThreads = 512;
constexpr int kTileColumns = 512;

// Sum of floor((b + a i) / 2^lb) over 0 <= i < n; a > 0, b >= 0.  The terms
// themselves add up to n b + a n (n - 1) / 2.  What the divisions leave over is
// their remainders: these repeat after P = 2^lb / g terms, g the greatest power
// of two in a and 2^lb, and are in some order the numbers below 2^lb that are b
// modulo g; so whole periods are known, and the rest, at most 127 terms, are
// added one by one.
__device__ __forceinline__ int64_t quotient_sum(int64_t n, int lb, int a, int64_t b)
{
    if (n <= 0) return 0;
    const int lg = min(__ffs(a) - 1, lb), mask = (1 << lb) - 1;
    const int64_t P = 1 << (lb - lg);
    int64_t over = (n >> (lb - lg)) * (P * (b & ((1 << lg) - 1)) + ((P * (P - 1) / 2) << lg));
    int x = (int)(b & mask), some = 0;
    for (int i = (int)(n & (P - 1)); i > 0; --i) {
        some += x;
        x = (x + a) & mask;
    }
    over += some;
    return (n * b + a * (n * (n - 1) / 2) - over) >> lb;
}

// What a tile costs beside its blocks (its queries' and results' ways, the
// first scores that nothing overlaps), in blocks.
constexpr int kTileCost = 2;
// Tiles of a sequence up to which their blocks are added one by one: shorter
// than the closed form, whose code must arrive first.
constexpr int kFewTiles = 4;

// The tiles of a sequence: TT tokens each.  Tile t takes the blocks [k0, k1),
// at least one.
template <int BN>
__device__ __forceinline__ void tile_blocks(const AttnParams &p, const Seq &s, int TT, int t, int &k0, int &k1)
{
    const int last = min((t + 1) * TT, s.n) - 1;
    k0 = key_lo(p, s, t * TT) / BN;
    k1 = max((key_hi(p, s, last) + BN - 1) / BN, k0 + 1);
}
// Blocks of BN (a power of two) keys of the first t of a sequence's nt tiles, in closed form.
// (Not inlined: it is called three times, and the start of a small call is
// the time that its code takes to arrive.)
static __device__ __noinline__ int64_t blocks_before(int BN, int n, int m, int causal, int window, int TT, int nt, int t)
{
    if (t <= 0) return 0;
    const int lb = __ffs(BN) - 1, all = (m + BN - 1) >> lb;
    if (!causal) return (int64_t)t * max(all, 1);
    const int64_t off = (int64_t)m - n;
    int64_t sum = 0;
    const bool last = t == nt;       // that tile may be short: its keys end with the sequence's
    if (last) --t;
    // Tiles whose tokens all stand before the first key: one block each.
    const int64_t z = off < 0 ? min(quotient(-off, TT), (int64_t)t) : 0;
    sum += z + quotient_sum(t - z, lb, TT, off + (z + 1) * TT + BN - 1);
    const int64_t gap = window - 1 - off;            // the first tiles' windows reach the first key
    if (window) {
        const int64_t y = max(z, gap > 0 ? quotient(gap + TT - 1, TT) : (int64_t)0);
        if (y < t) sum -= quotient_sum(t - y, lb, TT, off + 1 - window + y * TT);
    }
    if (last) {
        const int64_t lo = window ? max(off + (int64_t)t * TT + 1 - window, (int64_t)0) : 0, k0 = lo >> lb;
        sum += max((int64_t)all, k0 + 1) - k0;
    }
    return sum;
}

// A CTA's work is a run of units: a tile is kTileCost units, then one for each
// block.  A CTA whose units end inside the former has no part of the tile, one
// whose units begin there has all of its first blocks.  The walk:
struct Walk {
    int b, t, nt;
    Seq s;
    int k, end, k0, k1;              // blocks [k, end) of a tile that has [k0, k1)
    int64_t left;                    // units from block k on; tiles, where they are dealt whole
};
__device__ __forceinline__ void walk_end(const AttnParams &p, Walk &c)
{
    c.end = p.whole ? c.k1 : (int)min((int64_t)c.k1, c.k + c.left);
}
// To the next tile, by a whole warp; false: there is no more work.  Sequences
// without tokens are passed over 32 at a time (one by one they cost 100 ns each).
template <int BN>
__device__ __forceinline__ bool walk_on(const AttnParams &p, int TT, Walk &c)
{
    c.left -= p.whole ? 1 : c.end - c.k + kTileCost;
    if (c.left <= 0) return false;
    if (++c.t == c.nt) {
        c.t = 0;
        ++c.b;
        if (p.starts) {              // work is left: there is a sequence with tokens
            const int lane = threadIdx.x & 31;
            for (; c.b + 1 < p.B; c.b += 32) {
                const int b = min(c.b + lane, p.B - 1);
                const uint32_t some = __ballot_sync(0xffffffffu, sequence(p, b).n > 0);
                if (some) {
                    c.b += __ffs(some) - 1;
                    break;
                }
            }
            c.b = min(c.b, p.B - 1);
        }
        c.s = sequence(p, c.b);
        c.nt = (c.s.n + TT - 1) / TT;
    }
    tile_blocks<BN>(p, c.s, TT, c.t, c.k0, c.k1);
    c.k = c.k0;
    walk_end(p, c);
    return true;
}
// What the other warps are told of a piece.
struct __align__(16) Piece {
    int b, tok, ntok;                // sequence, first token and tokens of the tile
    Seq s;
    int k, end;                      // blocks [k, end)
    int flags;
    int hi, lo;                      // keys [lo, hi) that the tile's rows see
    int pad;
};
enum { PIECE_BEGINS = 1, PIECE_ENDS = 2, PIECE_NONE = 4 };   // the tile's first block, its last; no piece: the end
constexpr int kPieces = 8;

// CTAs whose waits ran out since this was last read (by their element kind).
static __device__ unsigned int g_given_up;
static cudaError_t take_given_up(unsigned int &n)
{
    const unsigned int zero = 0;
    if (cudaError_t e = cudaMemcpyFromSymbol(&n, g_given_up, sizeof n)) return e;
    return n ? cudaMemcpyToSymbol(g_given_up, &zero, sizeof zero) : cudaSuccess;
}

// A wait ran out: some pieces were not worked out, or not told at all.  NaN for
// all of the CTA's rows, sums of logarithms and parts.
template <int KIND, int DP>
__device__ __noinline__ void give_up(const AttnParams &p, const Walk &begin)
{
    using S = TileShape<KIND, DP>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = p.group.d, TT = S::ROWS / G, h = (int)blockIdx.x % p.Hk;
    if (threadIdx.x == 0) atomicAdd(&g_given_up, 1u);
    Walk c = begin;
    do {
        const int tok = c.s.first + c.t * TT, rows = min(TT, c.s.n - c.t * TT) * G;
        for (int r = warp; r < rows; r += 8) {
            if (c.k == c.k0 && c.end == c.k1) {
                const int i = p.group.div(r), hq = h * G + r - i * G;
                uint16_t *const out = const_cast<uint16_t *>(p.out.p) + (int64_t)(tok + i) * p.out.ld + hq * p.out.hs;
                for (int d = 2 * lane; d < p.D; d += 64)
                    if (dbg_global(out + d, 4, true)) *reinterpret_cast<uint32_t *>(out + d) = 0x7fff7fffu;
                if (p.lse && lane == 0) st_f32(p.lse + (int64_t)(tok + i) * p.out.H + hq, NAN);
            } else if (lane < 2) {
                st_f32(part_of(p.ws, blockIdx.x, c.k == c.k0, S::ROWS, DP) + 2 * r + lane, NAN);
            }
        }
    } while (walk_on<S::BN>(p, TT, c));
}

// The rows of the pieces that are whole tiles, once more where a result is not
// finite: 32 rows a warp.
template <int KIND, int DP>
__device__ __noinline__ void look_again(const AttnParams &p, const Walk &begin)
{
    using S = TileShape<KIND, DP>;
    const int lane = threadIdx.x & 31, first = (threadIdx.x >> 5) * 32, G = p.group.d, TT = S::ROWS / G, h = (int)blockIdx.x % p.Hk;
    Walk c = begin;
    do {
        const int tok = c.s.first + c.t * TT, ntok = min(TT, c.s.n - c.t * TT), rows = ntok * G;
        if (c.k == c.k0 && c.end == c.k1 && first < rows) {
            const int row = min(first + lane, rows - 1), i = p.group.div(row), t = tok + i, hq = h * G + row - i * G;
            const bool suspect = first + lane < rows && not_finite(p.out.p + (int64_t)t * p.out.ld + hq * p.out.hs, p.D);
            if (__any_sync(0xffffffffu, suspect)) work_out_again<KIND, DP / 32>(p, c.b, h, tok, ntok, t, hq, suspect);
        }
    } while (walk_on<S::BN>(p, TT, c));
}

// What is left to do behind all pieces, by the warps of the weights (those that
// have not given their registers away): state 2, 3: a wait ran out; 1: some
// result is not finite.  (One call: with two the 16384-token prompt took 1637 us
// instead of 1622, as the loops before are compiled differently.)
template <int KIND, int DP>
__device__ __noinline__ void last_look(const AttnParams &p, const Walk &begin, int state)
{
    if (state & 2) give_up<KIND, DP>(p, begin);
    else look_again<KIND, DP>(p, begin);
}

template <int KIND, int DP>
struct TileKernel {
    using S = TileShape<KIND, DP>;
    static constexpr int NT = S::NT, NS = S::NS, BN = S::BN, STAGES = S::STAGES;
    static constexpr bool FP8 = S::FP8;

    struct Shared {
        WorkScratch scratch;
        Piece piece[kPieces];
        uint64_t full[STAGES], empty[STAGES], landed[STAGES], raw_full[S::RAWS + 1], raw_empty[S::RAWS + 1], q[NT], s[NT * NS], w[NT * NS][2], o[NT], last, told[kPieces], heard[kPieces];
        uint32_t tmem;
        volatile int failed, odd;    // a wait ran out; some result is not finite
        Walk begin;
    };
    static_assert(sizeof(Shared) <= S::STATIC, "shared memory");

    const AttnParams &p;
    Shared &sm;
    uint8_t *const base;             // queries, stages, codes
    uint32_t tmem;
    int TT;
    const int groups, group, h;      // of Hk CTAs each, this CTA's, its head

    static __device__ __forceinline__ uint32_t at(const uint64_t *bar) { return smem_addr(bar); }
    // How often a wait tries.  (The debug build can be told to give up early.)
    __device__ __forceinline__ int tries() const
    {
#ifdef CRMSN_DEBUG
        if (p.wait_tries > 0) return p.wait_tries;
#endif
        return kWaitTries;
    }
    __device__ __forceinline__ bool wait(const uint64_t *bar, uint32_t parity)
    {
        return bar_wait(at(bar), parity, &sm.failed, tries());
    }
    // The same for a whole warp that goes on together.
    __device__ __forceinline__ bool wait_all(const uint64_t *bar, uint32_t parity)
    {
        return __all_sync(0xffffffffu, wait(bar, parity));
    }
    // This warp's writes to shared or to tensor memory are done, for the products.
    static __device__ __forceinline__ void ready(const uint64_t *bar)
    {
        fence_async();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) bar_arrive(at(bar));
    }
    static __device__ __forceinline__ void ready_tmem(const uint64_t *bar)
    {
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) bar_arrive(at(bar));
    }
    __device__ __forceinline__ uint8_t *queries(int half) const { return base + half * S::QBYTES; }
    __device__ __forceinline__ uint8_t *stage(int i) const { return base + NT * S::QBYTES + i * S::STAGE; }
    __device__ __forceinline__ int rows_of(const Piece &c) const { return c.ntok * p.group.d; }
    __device__ __forceinline__ bool used(const Piece &c, int half) const { return rows_of(c) > half * 128; }

    static __device__ __forceinline__ void put16(uint8_t *at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
    {
        if (dbg_shared(at, 16)) *reinterpret_cast<uint4 *>(at) = make_uint4(a, b, c, d);
    }

    // ------------------------------------------------------------- pieces --
    // A reader's place in the pieces.
    struct Place {
        int i;
        uint32_t parity;
    };
    // The next piece, read by a whole warp; false: no more, or a wait ran out.
    __device__ __forceinline__ bool next(Place &at_, Piece &c)
    {
        if (!wait_all(&sm.told[at_.i], at_.parity)) return false;
        const int4 *src = reinterpret_cast<const int4 *>(&sm.piece[at_.i]);
        int4 *dst = reinterpret_cast<int4 *>(&c);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(Piece) / 16); ++i) dst[i] = src[i];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) bar_arrive(at(&sm.heard[at_.i]));
        if (++at_.i == kPieces) {
            at_.i = 0;
            at_.parity ^= 1;
        }
        return !(c.flags & PIECE_NONE);
    }
    __device__ __forceinline__ void tell(int i, const Walk &c, bool more)
    {
        Piece &d = sm.piece[i];
        d.b = c.b;
        d.tok = c.t * TT;
        d.ntok = min(TT, c.s.n - c.t * TT);
        d.s = c.s;
        d.k = c.k;
        d.end = c.end;
        d.flags = (c.k == c.k0 ? PIECE_BEGINS : 0) | (c.end == c.k1 ? PIECE_ENDS : 0) | (more ? 0 : PIECE_NONE);
        d.hi = key_hi(p, c.s, d.tok + d.ntok - 1);
        d.lo = key_lo(p, c.s, d.tok);
        bar_arrive(at(&sm.told[i]));
    }
    // Warp 13: the pieces behind the first.
    __device__ __forceinline__ void tell_loop(Walk c)
    {
        int i = 1;
        uint32_t parity = 1;
        for (;;) {
            const bool more = walk_on<BN>(p, TT, c);
            if (!wait_all(&sm.heard[i], parity)) return;
            if ((threadIdx.x & 31) == 0) tell(i, c, more);
            __syncwarp();
            if (!more) return;
            if (++i == kPieces) {
                i = 0;
                parity ^= 1;
            }
        }
    }

    // ------------------------------------------------------------- copies --
    // Warps 8-11: warp w the rows w BN / 4 ... of every block; lane l finds
    // where key l of them lies.
    struct Rows {
        int64_t off[2];
        bool ok;
    };
    __device__ __forceinline__ Rows find_rows(const Piece &c, int first) const
    {
        Rows r{{0, 0}, false};
        const int j = c.k * BN + first + (int)(threadIdx.x & 31) % (BN / 4);
        if (j < c.hi && j >= c.lo) {
            int page, row;
            locate(p, c.b, c.s, j, page, row);
            if (page >= 0) {
                r.ok = true;
                r.off[0] = kv_offset(p.kv[0], page, row, h);
                r.off[1] = kv_offset(p.kv[1], page, row, h);
            }
        }
        return r;
    }
    // Copies the keys (which = 0) or values of BN / 4 rows from `first` on: to
    // their places in a stage (BF16), or as codes, row behind row.
    __device__ __forceinline__ void copy_rows(const Rows &r, int first, int which, uint32_t dst) const
    {
        constexpr int CH = DP * (FP8 ? 1 : 2) / 16, RW = BN / 4, N = RW * CH / 32;
        static_assert(RW * CH % 32 == 0, "whole instructions");
        const int lane = threadIdx.x & 31;
        const uint8_t *src = p.kv[which].p;
        const int64_t mine = which ? r.off[1] : r.off[0];
        const int have = p.D * (FP8 ? 1 : 2);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = i * 32 + lane, row = e / CH, chunk = e % CH;
            const int64_t o = __shfl_sync(0xffffffffu, mine, row);
            const bool ok = __shfl_sync(0xffffffffu, r.ok, row) && chunk * 16 < have;
            const uint32_t to = dst + (FP8 ? (uint32_t)((first + row) * CH + chunk) * 16u : matrix_at(first + row, chunk, BN * 128));
            copy16(to, src + o * (FP8 ? 1 : 2) + chunk * 16, ok);
        }
    }
    // A quarter of the codes of a block to FP16 in a stage.  (All loads before the
    // first store: one after another, each waits for the other's latency.)
    __device__ __forceinline__ void convert(const uint8_t *codes, uint8_t *dst) const
    {
        constexpr int CH = DP / 16, RW = BN / 4, N = RW * CH / 32;
        const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
        uint4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint8_t *from = codes + (warp * N + i) * 512 + lane * 16;
            v[i] = make_uint4(0, 0, 0, 0);
            if (dbg_shared(from, 16)) v[i] = *reinterpret_cast<const uint4 *>(from);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = i * 32 + lane, row = warp * RW + e / CH, chunk = e % CH;
            uint32_t h[8];
            f16_codes<KIND>(v[i].x, h[0], h[1]);
            f16_codes<KIND>(v[i].y, h[2], h[3]);
            f16_codes<KIND>(v[i].z, h[4], h[5]);
            f16_codes<KIND>(v[i].w, h[6], h[7]);
            put16(dst + matrix_at(row, 2 * chunk, BN * 128), h[0], h[1], h[2], h[3]);
            put16(dst + matrix_at(row, 2 * chunk + 1, BN * 128), h[4], h[5], h[6], h[7]);
        }
    }

    // BF16: blocks in the order K0 V0 K1 V1 ...  Copies and announcements wait
    // for nothing but their own condition: an empty stage, copies that have
    // landed.  (Each thread's copies are seen by the products after its own fence
    // behind their landing.)
    __device__ __forceinline__ void copy_loop()
    {
        int in = 0, out = 0, pending = 0;                     // stages to fill, to announce
        uint32_t empty = 1, landed = 0;                       // parities: all stages are empty at first
        Place place{0, 0};
        Piece c;
        bool more = next(place, c);
        int which = 0;
        const int first = (int)((threadIdx.x >> 5) & 3) * (BN / 4);
        Rows r = find_rows(c, first);
        for (int idle = 0; more || pending;) {
            if (more && __all_sync(0xffffffffu, bar_test(at(&sm.empty[in]), empty))) {
                copy_rows(r, first, which, smem_addr(stage(in)));
                bar_arrive_copies(at(&sm.landed[in]));
                ++pending;
                if (++in == STAGES) {
                    in = 0;
                    empty ^= 1;
                }
                which ^= 1;
                if (which == 0) {
                    if (++c.k == c.end) more = next(place, c);
                    if (more) r = find_rows(c, first);
                }
                idle = 0;
            }
            if (pending && __all_sync(0xffffffffu, bar_test(at(&sm.landed[out]), landed))) {
                ready(&sm.full[out]);
                if (++out == STAGES) {
                    out = 0;
                    landed ^= 1;
                }
                --pending;
                idle = 0;
            }
            if (++idle > 256 && (__any_sync(0xffffffffu, sm.failed) || idle > tries())) {
                sm.failed = 1;
                return;
            }
        }
    }

    // FP8: warps 14 and 15 copy the codes, half of a block each, as far ahead as
    // there are slots; warps 8-11 turn what has landed into FP16.  (One warp doing
    // both in turn had neither under way for long: 1500 cycles a block.)
    __device__ __forceinline__ void code_loop()
    {
        constexpr int RAWS = S::RAWS > 0 ? S::RAWS : 1;
        uint8_t *const raw = stage(STAGES);
        const int first = (int)((threadIdx.x >> 5) & 1) * (BN / 2);
        Place place{0, 0};
        Piece c;
        int in = 0;
        uint32_t parity = 1;
        while (next(place, c)) {
#pragma unroll 1
            for (; c.k < c.end; ++c.k) {
                const Rows r[2] = {find_rows(c, first), find_rows(c, first + BN / 4)};
#pragma unroll 1
                for (int which = 0; which < 2; ++which) {
                    if (!wait_all(&sm.raw_empty[in], parity)) return;
                    copy_rows(r[0], first, which, smem_addr(raw + in * S::RAW));
                    copy_rows(r[1], first + BN / 4, which, smem_addr(raw + in * S::RAW));
                    bar_arrive_copies(at(&sm.raw_full[in]));
                    if (++in == RAWS) {
                        in = 0;
                        parity ^= 1;
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void convert_loop()
    {
        constexpr int RAWS = S::RAWS > 0 ? S::RAWS : 1;
        uint8_t *const raw = stage(STAGES);
        Place place{0, 0};
        Piece c;
        int slot = 0, to = 0;
        uint32_t landed = 0, empty = 1;
        while (next(place, c)) {
#pragma unroll 1
            for (int i = 2 * (c.end - c.k); i > 0; --i) {
                if (!wait_all(&sm.raw_full[slot], landed) || !wait_all(&sm.empty[to], empty)) return;
                convert(raw + slot * S::RAW, stage(to));
                __syncwarp();
                if ((threadIdx.x & 31) == 0) bar_arrive(at(&sm.raw_empty[slot]));
                ready(&sm.full[to]);
                if (++slot == RAWS) {
                    slot = 0;
                    landed ^= 1;
                }
                if (++to == STAGES) {
                    to = 0;
                    empty ^= 1;
                }
            }
        }
    }

    // ----------------------------------------------------------- products --
    static constexpr uint32_t kScores = product_desc(!FP8, false, 128, BN);
    static constexpr uint32_t kValues = product_desc(!FP8, true, 128, DP);

    __device__ __forceinline__ uint32_t s_col(int half, int buf) const { return tmem + (uint32_t)(half * NS + buf) * BN; }
    __device__ __forceinline__ uint32_t o_col(int half) const { return tmem + (uint32_t)(S::OCOL + half * DP); }
    __device__ __forceinline__ void scores(int half, int buf, int st) const
    {
        const uint32_t q = matrix_low(smem_addr(queries(half)), 16), k = matrix_low(smem_addr(stage(st)), 16);
        const uint32_t d = s_col(half, buf);
#pragma unroll
        for (int i = 0; i < DP / 16; ++i)
            product_ss(d, matrix_desc(q + (i / 4) * (128 * 128 / 16) + (i % 4) * 2),
                       matrix_desc(k + (i / 4) * (BN * 128 / 16) + (i % 4) * 2), kScores, i > 0);
    }
    // The products of the first or second half of a block's keys.
    __device__ __forceinline__ void values(int half, int buf, int st, int part, bool add) const
    {
        constexpr int N = BN / 32;
        const uint32_t v = matrix_low(smem_addr(stage(st)), BN * 128) + part * N * (2048 / 16);
        const uint32_t d = o_col(half), w = s_col(half, buf) + part * N * 8;
#pragma unroll
        for (int i = 0; i < N; ++i) product_ts(d, w + i * 8, matrix_desc(v + i * (2048 / 16)), kValues, add || part || i > 0);
    }

    // Warp 12, all lanes together; one issues.
    __device__ __forceinline__ void issue_loop()
    {
        Place place{0, 0};
        Piece c;
        const bool one = elect_one();
        int st = 0;                                           // stage of the next block in the stream
        uint32_t full = 0;
        uint32_t q_par[NT], w_cnt[NT];                        // parities; blocks of a half so far
        for (int h = 0; h < NT; ++h) q_par[h] = w_cnt[h] = 0;
        const auto later = [&](int n, int &i, uint32_t &par) {
            i = st + n;
            par = full;
            if (i >= STAGES) {
                i -= STAGES;
                par ^= 1;
            }
        };
        while (next(place, c)) {
            const int blocks = uniform(c.end - c.k);
            const bool both = NT == 2 && uniform((int)used(c, NT - 1));
            const int halves = both ? 2 : 1;
            if (!wait_all(&sm.full[st], full)) return;
#pragma unroll
            for (int h = 0; h < NT; ++h) {
                if (h == 1 && !both) break;
                if (!wait_all(&sm.q[h], q_par[h])) return;
                q_par[h] ^= 1;
                tc_fence_after();
                if (one) {
                    const int buf = NS == 2 ? w_cnt[h] & 1 : 0;
                    scores(h, buf, st);
                    products_done(at(&sm.s[h * NS + buf]));
                    if (h + 1 == halves) products_done(at(&sm.empty[st]));
                }
            }
            for (int i = 0; i < blocks; ++i) {
                int kst, vst;
                uint32_t kpar, vpar;
                later(1, vst, vpar);
                later(2, kst, kpar);
                const bool more = i + 1 < blocks;
                if (NS == 2) {
                    const int buf = w_cnt[0] & 1;
                    if (more) {
                        if (!wait_all(&sm.full[kst], kpar)) return;
                        tc_fence_after();
                        if (one) {
                            scores(0, buf ^ 1, kst);
                            products_done(at(&sm.s[buf ^ 1]));
                            products_done(at(&sm.empty[kst]));
                        }
                    }
                    if (!wait_all(&sm.full[vst], vpar)) return;
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        if (!wait_all(&sm.w[buf][part], (w_cnt[0] >> 1) & 1)) return;
                        tc_fence_after();
                        if (one) values(0, buf, vst, part, i > 0);
                    }
                    if (one) {
                        products_done(at(&sm.o[0]));
                        products_done(at(&sm.empty[vst]));
                    }
                    ++w_cnt[0];
                } else {
                    if (!wait_all(&sm.full[vst], vpar)) return;
#pragma unroll
                    for (int h = 0; h < NT; ++h) {
                        if (h == 1 && !both) break;
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            if (!wait_all(&sm.w[h][part], w_cnt[h] & 1)) return;
                            tc_fence_after();
                            if (one) values(h, 0, vst, part, i > 0);
                        }
                        if (more && h == 0 && !wait_all(&sm.full[kst], kpar)) return;
                        tc_fence_after();
                        if (one) {
                            products_done(at(&sm.o[h]));
                            if (h + 1 == halves) products_done(at(&sm.empty[vst]));
                            if (more) {
                                scores(h, 0, kst);
                                products_done(at(&sm.s[h]));
                                if (h + 1 == halves) products_done(at(&sm.empty[kst]));
                            }
                        }
                        ++w_cnt[h];
                    }
                }
                later(2, st, full);
            }
        }
    }

    // ------------------------------------------------------------ weights --
    // Warps 4 half ... 4 half + 3: row threadIdx.x % 128 of the half.
    // The row's token and query head; rows behind the last: the last token's.
    struct Row {
        int tok, head;
        bool valid;
    };
    __device__ __forceinline__ Row row_of(const Piece &c, int half) const
    {
        const int r = half * 128 + (threadIdx.x & 127), rows = rows_of(c);
        Row w;
        w.valid = r < rows;
        const int rr = w.valid ? r : rows - 1, i = p.group.div(rr);
        w.tok = c.tok + i;
        w.head = h * p.group.d + rr - i * p.group.d;
        return w;
    }

    // A warp's 32 rows of queries: LANES lanes a row, RPI rows an instruction.
    static constexpr int CH = DP / 8, LANES = CH <= 8 ? 8 : CH <= 16 ? 16 : 32, RPI = 32 / LANES, NI = 32 / RPI;

    // Asynchronous copies of a tile's queries to their place.
    __device__ __forceinline__ void copy_queries(const Piece &c, int half) const
    {
        const Row w = row_of(c, half);
        const int64_t mine = (int64_t)(c.s.first + w.tok) * p.q.ld + w.head * p.q.hs;
        const int lane = threadIdx.x & 31, first = threadIdx.x & 96, chunk = lane % LANES;
        const uint32_t dst = smem_addr(queries(half));
#pragma unroll 8
        for (int i = 0; i < NI; ++i) {
            const int row = i * RPI + lane / LANES;
            const int64_t o = __shfl_sync(0xffffffffu, mine, row);
            const bool ok = __shfl_sync(0xffffffffu, w.valid, row) && chunk * 8 < p.D;
            if (chunk < CH) copy16(dst + matrix_at(first + row, chunk, 128 * 128), p.q.p + o + chunk * 8, ok);
        }
        copy_commit();
    }
    // They have arrived (FP8: and become FP16, each thread what it copied).
    // Returns the exponent by which this lane's row was scaled.  sign: score_sign.
    __device__ __forceinline__ int queries_here(int half, uint32_t sign) const
    {
        copy_wait<0>();
        int mine = 0;
        if constexpr (FP8) {
            const int lane = threadIdx.x & 31, first = threadIdx.x & 96, chunk = lane % LANES;
            uint8_t *const base_q = queries(half);
#pragma unroll 2
            for (int i = 0; i < NI; ++i) {
                uint8_t *const at = base_q + matrix_at(first + i * RPI + lane / LANES, chunk < CH ? chunk : 0, 128 * 128);
                uint4 v = make_uint4(0, 0, 0, 0);
                if (chunk < CH && dbg_shared(at, 16)) v = *reinterpret_cast<const uint4 *>(at);
                float top = 0.f;
                for (const uint32_t x : {v.x, v.y, v.z, v.w}) top = fmaxf(top, fmaxf(fabsf(bf_lo(x)), fabsf(bf_hi(x))));
#pragma unroll
                for (int o = 1; o < LANES; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int e = row_exponent(top), there = __shfl_sync(0xffffffffu, e, (lane % RPI) * LANES);
                if (lane / RPI == i) mine = there;
                const auto f16 = [&](uint32_t x) { return pack_f16(scaled(bf_lo(x), e), scaled(bf_hi(x), e)) ^ sign; };
                if (chunk < CH) put16(at, f16(v.x), f16(v.y), f16(v.z), f16(v.w));
            }
        }
        ready(&sm.q[half]);
        return mine;
    }

    // Four lanes, a row each of four chunks (w: 4 words a chunk), exchange them
    // in two butterfly steps: lane l gets chunk l & 3 of the four rows.  So four
    // lanes store 64 bytes of a row together: stores of a row a lane occupy the
    // memory pipe for 32 lines each, four times as long.
    static __device__ __forceinline__ void turn_quads(uint32_t (&w)[16])
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int step = 1; step < 4; step *= 2) {
            const bool up = lane & step;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int a = step == 1 ? i / 4 * 8 + i % 4 : i, b = a + 4 * step;    // chunks 0, 1 and 2, 3; then 0, 2 and 1, 3
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[a] : w[b], step);
                if (up) w[a] = got;
                else w[b] = got;
            }
        }
    }

    // Bits [lo, hi) of a word.
    static __device__ __forceinline__ uint32_t bits(int lo, int hi)
    {
        const uint32_t up = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1u;
        return lo <= 0 ? up : lo >= 32 ? 0u : up & ~((1u << lo) - 1u);
    }

    // What weights are relative to (kWeightTop), with M a raw score.
    static __device__ __forceinline__ float reference(float M, float scale)
    {
        return FP8 ? fmaf(M, scale, (float)(kLag - kWeightTop)) : M * scale;
    }

    // Ends at once where a wait ran out (give_up follows).
    __device__ __forceinline__ void weight_loop(int half)
    {
        const uint32_t lanes = (uint32_t)((threadIdx.x >> 5) & 3) << 21;       // lane 32 (warp % 4), in bits 16 up
        const float vs = FP8 ? ld_f32_ro(p.scale[1]) : 1.f;
        const float c_all = FP8 ? p.qk_scale * ld_f32_ro(p.scale[0]) : p.qk_scale;
        Place place{0, 0};
        Piece c, nx;
        bool any = next(place, nx), have = false, copied = false;
        Row row;
        int e = 0;
        float scale = 0.f, M = 0.f, L = 0.f;                  // M: the reference, a raw score
        uint32_t cnt = 0;                                     // blocks so far
        for (;;) {
            // The next tile's queries first (its scores are worked out meanwhile), then this one's results.
            while (any && !used(nx, half)) any = next(place, nx);
            if (any) {
                if (!copied) copy_queries(nx, half);
                e = queries_here(half, FP8 ? score_sign(c_all) : 0u);
            }
            if (have) {
                if (!wait_all(&sm.o[half], (cnt - 1) & 1)) return;
                tc_fence_after();
                finish(c, half, row, reference(M, scale), L, vs, lanes);
            }
            if (!any) return;
            c = nx;
            have = true;
            copied = false;
            row = row_of(c, half);
            scale = FP8 ? score_factor(c_all, e) : c_all;
            M = -INFINITY;
            L = 0.f;
            int hk = key_hi(p, c.s, row.tok) - c.k * BN, lk = key_lo(p, c.s, row.tok) - c.k * BN;    // seen: [lk, hk) of the block
            bool begun = false;
            for (int n = c.end - c.k; n > 0; --n, ++cnt, hk -= BN, lk -= BN) {
                const int buf = NS == 2 ? cnt & 1 : 0;
                const uint32_t sc = s_col(half, buf) + lanes;
                const bool edge = __any_sync(0xffffffffu, hk < BN || lk > 0);
                if (!wait_all(&sm.s[half * NS + buf], NS == 2 ? (cnt >> 1) & 1 : cnt & 1)) return;
                tc_fence_after();
                // The last scores are here: the next tile's queries may take the place of these.
                if (__builtin_expect(n == 1, 0)) {
                    // (One piece ahead and no further: later ones may wait for what this half still owes.)
                    any = next(place, nx);
                    copied = any && used(nx, half);
                    if (copied) copy_queries(nx, half);
                }
                // Scores that the row does not see leave tensor memory as -infinity.
                if (__builtin_expect(edge, 0)) {
#pragma unroll 1
                    for (int i = 0; i < BN / 32; ++i) {
                        uint32_t x[32];
                        if (__all_sync(0xffffffffu, hk >= 32 * i + 32 && lk <= 32 * i)) continue;
                        tmem_ld32(sc + 32 * i, x);
                        tmem_wait_ld();
                        const uint32_t see = bits(lk - 32 * i, hk - 32 * i);
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] = see >> j & 1u ? x[j] : 0xff800000u;
                        tmem_st32(sc + 32 * i, x);
                    }
                    tmem_wait_st();
                }
                // The maximum.  Scores are read twice: tensor memory gives 32 columns in a few tens of cycles, and
                // a block of them held in registers would leave none.
                float top[4] = {M, M, M, M};
#pragma unroll
                for (int i = 0; i < BN / 64; ++i) {
                    uint32_t x[64];
                    tmem_ld32(sc + 64 * i, x);
                    tmem_ld32(sc + 64 * i + 32, x + 32);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 64; j += 2)
                        top[j / 2 % 4] = fmaxf(top[j / 2 % 4], fmaxf(__uint_as_float(x[j]), __uint_as_float(x[j + 1])));
                }
                const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                // A new reference changes O, the products of the block before done.  (One S: they were issued before
                // its products, and are done with them.)
                if (NS == 2 && cnt > 0) {
                    if (!wait_all(&sm.o[half], (cnt - 1) & 1)) return;
                    tc_fence_after();
                }
                if (__builtin_expect(__any_sync(0xffffffffu, (most - M) * scale > kLag || M == -INFINITY), 0)) {
                    const float keep = M == -INFINITY || most == M ? 1.f : exp2_fast((M - most) * scale);
                    L *= keep;
                    if (begun && __any_sync(0xffffffffu, keep != 1.f)) {
#pragma unroll 1
                        for (int i = 0; i < DP / 32; ++i) {
                            uint32_t y[32];
                            tmem_ld32(o_col(half) + lanes + 32 * i, y);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * keep);
                            tmem_st32(o_col(half) + lanes + 32 * i, y);
                        }
                        tmem_wait_st();
                    }
                    M = most;
                }
                begun = true;
                const float ref = M == -INFINITY ? 0.f : -reference(M, scale);
                F2 sum = f2(0.f), sum1 = f2(0.f);
                // The weights of 32 keys take 16 columns: they replace scores that have been read.  The next 32 scores
                // are on their way meanwhile.
                uint32_t x[2][32];
                tmem_ld32(sc, x[0]);
#pragma unroll
                for (int i = 0; i < BN / 32; ++i) {
                    uint32_t w[16];
                    tmem_wait_ld();
                    if (i + 1 < BN / 32) tmem_ld32(sc + 32 * (i + 1), x[(i + 1) & 1]);
                    const uint32_t *y = x[i & 1];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const F2 a = f2_fma(f2(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1])), f2(scale), f2(ref));
                        const F2 b = f2(exp2_fast(a.x), exp2_fast(a.y));
                        if (j & 1) sum1 = f2_add(sum1, b);
                        else sum = f2_add(sum, b);
                        w[j] = FP8 ? pack_f16(b.x, b.y) : pack_bf16(b.x, b.y);
                    }
                    tmem_st16(sc + 16 * i, w);
                    if (i == BN / 64 - 1) ready_tmem(&sm.w[half * NS + buf][0]);
                }
                sum = f2_add(sum, sum1);
                L += sum.x + sum.y;
                ready_tmem(&sm.w[half * NS + buf][1]);
            }
        }
    }

    // A row's result, or part.
    __device__ __forceinline__ void finish(const Piece &c, int half, const Row &row, float M, float L, float vs, uint32_t lanes) const
    {
        const int64_t t = c.s.first + row.tok;
        const int r = threadIdx.x & 127;
        // This code runs once for each tile, from a cold instruction cache: a short loop is faster than a long one
        // unrolled.  16 columns at a time are two chunks of a result, four of a part.
        const bool whole = (c.flags & (PIECE_BEGINS | PIECE_ENDS)) == (PIECE_BEGINS | PIECE_ENDS);
        const float inv = vs / L;
        F2 odd = f2(0.f);                                     // NaN: some value is not finite
        uint8_t *to;
        int have = DP * 4;
        if (whole) {
            to = reinterpret_cast<uint8_t *>(const_cast<uint16_t *>(p.out.p) + t * p.out.ld + row.head * p.out.hs);
            have = p.D * 2;
            if (row.valid && p.lse) st_f32(p.lse + t * p.out.H + row.head, L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718f);
        } else {
            float *part = part_of(p.ws, blockIdx.x, c.flags & PIECE_BEGINS, S::ROWS, DP);
            if (row.valid) {
                st_f32(part + 2 * (half * 128 + r), M);
                st_f32(part + 2 * (half * 128 + r) + 1, L);
            }
            to = reinterpret_cast<uint8_t *>(part + 2 * S::ROWS + (int64_t)(half * 128 + r) * DP);
        }
        // 64 bytes of the four rows of this lane's quad at a time.
        uint8_t *quad[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            quad[j] = reinterpret_cast<uint8_t *>(__shfl_sync(0xffffffffu, (unsigned long long)(row.valid ? to : nullptr), (r & 28) + j));
        int done = (r & 3) * 16;                              // this lane's first byte of them
#pragma unroll 1
        for (int n = 0; n < DP / 16; ++n, done += 64) {
            uint32_t w[16];
            tmem_ld16(o_col(half) + lanes + 16 * n, w);
            tmem_wait_ld();
            if (whole) {
                // The next 16 columns too: 32 results.
                uint32_t y[16];
                tmem_ld16(o_col(half) + lanes + 16 * ++n, y);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint32_t *x = j < 8 ? w + 2 * j : y + 2 * (j - 8);
                    F2 v = f2_mul(f2(__uint_as_float(x[0]), __uint_as_float(x[1])), f2(inv));
                    if (L == 0.f) v = f2(0.f);                // whatever 0 times the values was
                    odd = f2_fma(v, f2(0.f), odd);
                    w[j] = bf16_f2(v);
                }
            }
            turn_quads(w);
            if (done < have)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (quad[j] && dbg_global(quad[j] + done, 16, true))
                        *reinterpret_cast<uint4 *>(quad[j] + done) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        }
        const bool again = whole && row.valid && !(odd.x == 0.f && odd.y == 0.f) && L > 0.f && L < INFINITY;
        if (again) sm.odd = 1;
        tc_fence_before();
    }

    // -------------------------------------------------------------- start --
    __device__ __forceinline__ void go()
    {
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
        // What needs no input, before the kernel ahead has ended.
        if (tid == 0) {
            for (int i = 0; i < STAGES; ++i) {
                bar_init(at(&sm.full[i]), 4);
                bar_init(at(&sm.empty[i]), 1);
                bar_init(at(&sm.landed[i]), 128);
            }
            for (int i = 0; i < NT; ++i) {
                bar_init(at(&sm.q[i]), 4);
                bar_init(at(&sm.o[i]), 1);
            }
            for (int i = 0; i < NT * NS; ++i) {
                bar_init(at(&sm.s[i]), 1);
                bar_init(at(&sm.w[i][0]), 4);
                bar_init(at(&sm.w[i][1]), 4);
            }
            for (int i = 0; i < kPieces; ++i) {
                bar_init(at(&sm.told[i]), 1);
                bar_init(at(&sm.heard[i]), 4 * NT + (FP8 ? 7 : 5));
            }
            for (int i = 0; i < S::RAWS; ++i) {
                bar_init(at(&sm.raw_full[i]), 64);
                bar_init(at(&sm.raw_empty[i]), 4);
            }
            bar_init(at(&sm.last), 1);
            sm.failed = sm.odd = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        if (warp == 12) tmem_alloc(smem_addr(&sm.tmem), kTileColumns);
        tc_fence_before();
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;");
        TT = S::ROWS / p.group.d;
        Walk c;
        bool work;
        if (p.whole && p.starts) {
            // Tiles as units.
            const Work w = share_work<kTileThreads>(
                p.B, group, sm.scratch, [&](int b, int64_t &u, int64_t &t) { u = t = (sequence(p, b).n + TT - 1) / TT; },
                [&](int64_t tiles, int64_t) { return (int)min((int64_t)groups, tiles); });
            work = group < w.groups;
            if (work) {
                c.b = w.b;
                c.t = (int)w.rest;
                c.s = sequence(p, c.b);
                c.nt = (c.s.n + TT - 1) / TT;
                tile_blocks<BN>(p, c.s, TT, c.t, c.k0, c.k1);
                c.k = c.k0;
                c.left = w.u1 - w.u0;
            }
        } else if (p.whole) {
            const int nt = (p.n + TT - 1) / TT;
            const int64_t tiles = (int64_t)p.B * nt;
            const int n = (int)min((int64_t)groups, tiles);
            __syncthreads();
            work = group < n;
            if (work) {
                const int64_t first = first_unit(tiles, n, group);
                c.b = (int)quotient(first, nt);
                c.t = (int)(first - (int64_t)c.b * nt);
                c.nt = nt;
                c.s = sequence(p, c.b);
                tile_blocks<BN>(p, c.s, TT, c.t, c.k0, c.k1);
                c.k = c.k0;
                c.left = first_unit(tiles, n, group + 1) - first;
            }
        } else {
            work = share(c, lane);
        }
        if (work) run_work(c, warp, lane);
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 12) tmem_free(tmem, kTileColumns);
    }

    // By the units of all tiles: where this CTA's begin; false: it has none.
    __device__ __forceinline__ bool share(Walk &c, int lane)
    {
        const Work work = share_work<kTileThreads>(
            p.B, group, sm.scratch,
            [&](int b, int64_t &u, int64_t &t) {
                const Seq s = sequence(p, b);
                const int nt = (s.n + TT - 1) / TT;
                u = (int64_t)nt * kTileCost;
                t = nt;
                if (nt > kFewTiles) {
                    u += blocks_before(BN, s.n, s.m, p.causal, p.window, TT, nt, nt);
                } else {
                    for (int i = 0; i < nt; ++i) {
                        int k0, k1;
                        tile_blocks<BN>(p, s, TT, i, k0, k1);
                        u += k1 - k0;
                    }
                }
            },
            // A group for each tile; tiles are shared out further while that leaves a group four units (more than
            // kTileCost: every group has a block).
            [&](int64_t units, int64_t tiles) { return (int)min((int64_t)groups, max(tiles, units / 4)); });
        if (group >= work.groups) {
            if (threadIdx.x == 0 && groups > 1) st_header(p.ws, blockIdx.x, AttnHeader{});
            return false;
        }
        c.b = work.b;
        c.s = sequence(p, c.b);
        c.nt = (c.s.n + TT - 1) / TT;
        // The tile of unit `rest`: the last with no more units before it.
        const int64_t rest = work.rest;
        int64_t before;
        if (c.nt <= 32) {
            // A lane for each tile.
            int k0 = 0, k1 = -kTileCost;
            if (lane < c.nt) tile_blocks<BN>(p, c.s, TT, lane, k0, k1);
            const int64_t mine = k1 - k0 + kTileCost;
            int64_t upto = mine;
            for (int o = 1; o < 32; o *= 2) {
                const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            c.t = min(__popc(__ballot_sync(0xffffffffu, upto <= rest)), c.nt - 1);
            before = __shfl_sync(0xffffffffu, upto - mine, c.t);
        } else {
            const auto units_before = [&](int t) {
                return blocks_before(BN, c.s.n, c.s.m, p.causal, p.window, TT, c.nt, t) + (int64_t)t * kTileCost;
            };
            int lo = 0, hi = c.nt;               // 32 places at a time
            while (hi - lo > 1) {
                const int by = (hi - lo + 31) / 32, t = lo + lane * by;
                const bool in = t < hi && units_before(t) <= rest;
                const int n = __popc(__ballot_sync(0xffffffffu, in)) - 1;
                lo += n * by;
                hi = min(hi, lo + by);
            }
            c.t = lo;
            before = units_before(lo);
        }
        tile_blocks<BN>(p, c.s, TT, c.t, c.k0, c.k1);
        const int in = (int)(rest - before) - kTileCost;      // blocks before u0, or less than none
        c.k = c.k0 + max(in, 0);
        c.left = work.u1 - work.u0 + min(in, 0);
        if (threadIdx.x == 0 && groups > 1) {
            AttnHeader hd{};
            hd.first = work.u0 - in;                          // the tile's first block
            hd.last = hd.first + (c.k1 - c.k0);
            hd.units = work.units;
            hd.groups = work.groups;
            hd.tile = c.k > c.k0;
            hd.b = c.b;
            hd.h = h;
            hd.tok = c.s.first + c.t * TT;
            hd.ntok = min(TT, c.s.n - c.t * TT);
            st_header(p.ws, blockIdx.x, hd);
        }
        return true;
    }

    // All threads, after a barrier behind the start's own work.
    __device__ __forceinline__ void run_work(Walk &c, int warp, int lane)
    {
        tc_fence_after();
        tmem = uniform(sm.tmem);
        walk_end(p, c);
        if (threadIdx.x == 0) {
            sm.begin = c;
            tell(0, c, true);
        }
        __syncwarp();
        if (warp < 8) {
            more_registers<S::REGS>();
            if (warp < 4 * NT) weight_loop(warp >> 2);
            copy_wait_all();
            asm volatile("bar.sync 1, 256;" ::: "memory");    // all results are written
            if (const int state = sm.failed * 2 | sm.odd) last_look<KIND, DP>(p, sm.begin, state);
        } else {
            fewer_registers<S::OTHER_REGS>();
            if (warp < 12) {
                if constexpr (FP8) convert_loop();
                else copy_loop();
                copy_wait_all();
            } else if (warp == 12) {
                issue_loop();
                __syncwarp();
                // Products in flight end before their memory goes, whatever became of the waits.
                if (elect_one()) {
                    products_done(at(&sm.last));
                    for (int i = 0; i < kWaitTries && !bar_try(at(&sm.last), 0); ++i) {}
                }
                __syncwarp();
            } else if (warp == 13) {
                tell_loop(c);
            } else if (FP8) {
                code_loop();
                copy_wait_all();
            }
        }
    }
};

template <int KIND, int DP>
__global__ void __launch_bounds__(kTileThreads, 1) k_attn_tile(const __grid_constant__ AttnParams p)
{
    extern __shared__ __align__(1024) uint8_t tile_smem[];
    __shared__ typename TileKernel<KIND, DP>::Shared sm;
    CRMSN_DEBUG_ENTER(p.dbg);
    uint8_t *const base = tile_smem + (1024 - (smem_addr(tile_smem) & 1023)) % 1024;
    const int group = (int)blockIdx.x / p.Hk;
    TileKernel<KIND, DP> k{p, sm, base, 0, 0, (int)gridDim.x / p.Hk, group, (int)blockIdx.x - group * p.Hk};
    k.go();
}

template <int KIND, int DP>
cudaError_t run_attn_tile(const AttnParams &p, int sms, cudaStream_t s)
{
    using S = TileShape<KIND, DP>;
    static std::atomic<int> opted[kOptInDevices];
    if (cudaError_t e = opt_in_smem(k_attn_tile<KIND, DP>, S::SMEM, opted)) return e;
    const int groups = attn_groups(sms, p.Hk);
    if (cudaError_t e = launch_pdl(k_attn_tile<KIND, DP>, dim3(groups * p.Hk), dim3(kTileThreads), S::SMEM, s, p)) return e;
    return p.whole ? cudaSuccess : launch_attn_combine(p, S::ROWS, DP, groups, s);
}

}  // namespace crmsn
