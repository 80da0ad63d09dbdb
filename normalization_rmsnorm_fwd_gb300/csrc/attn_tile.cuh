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
// copy keys and values; one thread of warp 12 issues the products.  While one
// half's weights are worked out, the tensor cores run the other half's
// products: S of the next block follows O of this one at once.  Heads of 256
// leave no room for two halves in tensor memory (O takes 256 of its 512
// columns); there one half has two S, and S of the next block runs ahead of O
// of this one.
//
// The reference M of a row's weights is a maximum of before; it moves only when
// the true one has passed it by 2^8, as moving it means reading and writing O.
// A weight is then at most 2^8, its rounding relative as ever.
//
// Keys and values: 16-byte asynchronous copies by the copying warps (any page
// size; what lies behind the last key becomes zeros), into the swizzled layout
// that the products read.  FP8 caches: each thread copies into slots of its own
// and turns what arrived into FP16.  The blocks of a tile, and the tiles that a
// CTA works through, form one stream: loads run ahead across the ends of tiles.
//
// Work is shared out by blocks (share_work): CTAs that meet inside a tile write
// parts, which attn_combine.cu joins.
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
    static_assert(OCOL + NT * DP <= 512, "tensor memory");
    static_assert(SMEM + 1600 <= 227 * 1024, "shared memory");
};
constexpr int kTileThreads = 512;
constexpr int kTileColumns = 512;
// Registers of a thread: of the 128 at launch the copying and the issuing
// warps give up what the weights' warps need.
constexpr int kWeightRegs = 184, kOtherRegs = 72;
static_assert(2 * kWeightRegs + 2 * kOtherRegs <= 4 * 128, "registers of the launch");

// sum of floor((a i + b) / m) over 0 <= i < n (the classic Euclid-like
// reduction of a count of lattice points under a line).
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b)
{
    int64_t sum = 0;
    while (n > 0) {
        sum += n * (n - 1) / 2 * (a / m) + n * (b / m);
        a %= m;
        b %= m;
        const int64_t y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const int64_t t = m;
        m = a;
        a = t;
    }
    return sum;
}

// The tiles of a sequence: TT tokens each.  Tile t takes the blocks [k0, k1),
// at least one.
template <int BN>
__device__ __forceinline__ void tile_blocks(const AttnParams &p, const Seq &s, int TT, int t, int &k0, int &k1)
{
    const int last = min((t + 1) * TT, s.n) - 1;
    k0 = key_lo(p, s, t * TT) / BN;
    k1 = max((key_hi(p, s, last) + BN - 1) / BN, k0 + 1);
}
// Blocks of the first t of a sequence's nt tiles, in closed form.
template <int BN>
__device__ __forceinline__ int64_t blocks_before(const AttnParams &p, const Seq &s, int TT, int nt, int t)
{
    if (t <= 0) return 0;
    if (!p.causal) return (int64_t)t * max((s.m + BN - 1) / BN, 1);
    int64_t sum = 0;
    if (t == nt) {                   // the last tile may be short
        int k0, k1;
        tile_blocks<BN>(p, s, TT, nt - 1, k0, k1);
        sum = k1 - k0;
        --t;
    }
    const int64_t off = (int64_t)s.m - s.n;
    // Tiles whose tokens all stand before the first key: one block each.
    const int64_t z = off < 0 ? min(-off / TT, (int64_t)t) : 0;
    sum += z;
    sum += floor_sum(t - z, BN, TT, off + (z + 1) * TT + BN - 1);
    if (p.window) {
        const int64_t gap = p.window - 1 - off;      // first tiles whose window reaches the first key
        const int64_t y = max(z, gap > 0 ? (gap + TT - 1) / TT : (int64_t)0);
        if (y < t) sum -= floor_sum(t - y, BN, TT, off + 1 - p.window + y * TT);
    }
    return sum;
}

// A piece of a CTA's work: blocks [k, end) of a tile that has [k0, k1).
struct Piece {
    int b, h, t, nt;
    Seq s;
    int k, end, k0, k1;
    int64_t left;                    // units from block k on
};
template <int BN>
__device__ __forceinline__ void piece_ends(Piece &c)
{
    c.end = (int)min((int64_t)c.k1, c.k + c.left);
}
// The next piece; false: there is none.
template <int BN>
__device__ __forceinline__ bool next_piece(const AttnParams &p, int TT, Piece &c)
{
    c.left -= c.end - c.k;
    if (c.left <= 0) return false;
    if (++c.t == c.nt) {
        c.t = 0;
        if (++c.h == p.Hk) {
            c.h = 0;
            do {                     // work is left: there is a sequence with tokens
                ++c.b;
                c.s = sequence(p, c.b);
            } while (c.s.n == 0 && c.b + 1 < p.B);
            c.nt = (c.s.n + TT - 1) / TT;
        }
    }
    tile_blocks<BN>(p, c.s, TT, c.t, c.k0, c.k1);
    c.k = c.k0;
    piece_ends<BN>(c);
    return true;
}

template <int KIND, int DP>
struct TileKernel {
    using S = TileShape<KIND, DP>;
    static constexpr int NT = S::NT, NS = S::NS, BN = S::BN, STAGES = S::STAGES;
    static constexpr bool FP8 = S::FP8;

    struct Shared {
        WorkScratch scratch;
        uint64_t full[STAGES], empty[STAGES], q[NT], s[NT * NS], w[NT * NS], o[NT], last;
        uint32_t tmem;
        volatile int failed;
    };

    const AttnParams &p;
    Shared &sm;
    uint8_t *const base;             // queries, stages, codes
    uint32_t tmem;
    int TT;

    static __device__ __forceinline__ uint32_t at(const uint64_t *bar) { return smem_addr(bar); }
    __device__ __forceinline__ bool wait(const uint64_t *bar, uint32_t parity) { return bar_wait(at(bar), parity, &sm.failed); }
    // The same for a whole warp that goes on together.
    __device__ __forceinline__ bool wait_all(const uint64_t *bar, uint32_t parity)
    {
        return __all_sync(0xffffffffu, wait(bar, parity));
    }
    __device__ __forceinline__ uint8_t *queries(int half) const { return base + half * S::QBYTES; }
    __device__ __forceinline__ uint8_t *stage(int i) const { return base + NT * S::QBYTES + i * S::STAGE; }
    __device__ __forceinline__ int rows_of(const Piece &c) const
    {
        return min(TT, c.s.n - c.t * TT) * p.group.d;
    }
    __device__ __forceinline__ bool used(const Piece &c, int half) const { return rows_of(c) > half * 128; }

    static __device__ __forceinline__ void put16(uint8_t *at, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
    {
        if (dbg_shared(at, 16)) *reinterpret_cast<uint4 *>(at) = make_uint4(a, b, c, d);
    }

    // ------------------------------------------------------------- copies --
    // Warps 8-11: warp w the rows w BN / 4 ... of every block; lane l finds
    // where key l of them lies.
    struct Rows {
        int64_t off[2];
        bool ok;
    };
    __device__ __forceinline__ Rows find_rows(const Piece &c, int k, int hi, int lo) const
    {
        const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
        Rows r{{0, 0}, false};
        const int j = k * BN + warp * (BN / 4) + lane % (BN / 4);
        if (j < hi && j >= lo) {
            int page, row;
            locate(p, c.b, c.s, j, page, row);
            if (page >= 0) {
                r.ok = true;
                r.off[0] = kv_offset(p.kv[0], page, row, c.h);
                r.off[1] = kv_offset(p.kv[1], page, row, c.h);
            }
        }
        return r;
    }
    // Copies the keys (which = 0) or values of the rows: to their places in a
    // stage (BF16), or as codes to this thread's slots.
    __device__ __forceinline__ void copy_rows(const Rows &r, int which, uint32_t dst) const
    {
        constexpr int CH = DP * (FP8 ? 1 : 2) / 16, RW = BN / 4, N = RW * CH / 32;
        static_assert(RW * CH % 32 == 0, "whole instructions");
        const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
        const uint8_t *src = p.kv[which].p;
        const int64_t mine = which ? r.off[1] : r.off[0];
        const int have = p.D * (FP8 ? 1 : 2);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = i * 32 + lane, row = e / CH, chunk = e % CH;
            const int64_t o = __shfl_sync(0xffffffffu, mine, row);
            const bool ok = __shfl_sync(0xffffffffu, r.ok, row) && chunk * 16 < have;
            const uint32_t to = FP8 ? dst + (uint32_t)(i * 128 + warp * 32 + lane) * 16u
                                    : dst + matrix_at(warp * RW + row, chunk, BN * 128);
            copy16(to, src + o * (FP8 ? 1 : 2) + chunk * 16, ok);
        }
    }
    // This thread's codes, arrived, to FP16 in a stage.
    __device__ __forceinline__ void convert(const uint8_t *codes, uint8_t *dst) const
    {
        constexpr int CH = DP / 16, RW = BN / 4, N = RW * CH / 32;
        const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = i * 32 + lane, row = warp * RW + e / CH, chunk = e % CH;
            const uint8_t *from = codes + (i * 128 + warp * 32 + lane) * 16;
            const uint4 v = dbg_shared(from, 16) ? *reinterpret_cast<const uint4 *>(from) : make_uint4(0, 0, 0, 0);
            put16(dst + matrix_at(row, 2 * chunk, BN * 128), f16_fp8<KIND>(v.x), f16_fp8<KIND>(v.x >> 16), f16_fp8<KIND>(v.y),
                  f16_fp8<KIND>(v.y >> 16));
            put16(dst + matrix_at(row, 2 * chunk + 1, BN * 128), f16_fp8<KIND>(v.z), f16_fp8<KIND>(v.z >> 16), f16_fp8<KIND>(v.w),
                  f16_fp8<KIND>(v.w >> 16));
        }
    }

    // BF16: blocks in the order K0 V0 K1 V1 ..., their arrival announced up to
    // AHEAD blocks later, or as soon as there is no free stage.
    __device__ __forceinline__ void copy_loop(Piece c)
    {
        constexpr int AHEAD = 3;
        int in = 0, out = 0, pending = 0;                     // stages to fill, to announce
        uint32_t parity = 1;                                  // of `in`'s emptiness: free at first
        const auto announce = [&]() {
            fence_async();
            bar_arrive(at(&sm.full[out]));
            out = out + 1 == STAGES ? 0 : out + 1;
            --pending;
        };
        do {
            const int TTt = c.t * TT, last = min(TTt + TT, c.s.n) - 1;
            const int hi = key_hi(p, c.s, last), lo = key_lo(p, c.s, TTt);
            for (int k = c.k; k < c.end; ++k) {
                const Rows r = find_rows(c, k, hi, lo);
                for (int which = 0; which < 2; ++which) {
                    if (!__all_sync(0xffffffffu, bar_try(at(&sm.empty[in]), parity))) {
                        copy_wait<0>();
                        while (pending) announce();
                        if (!wait_all(&sm.empty[in], parity)) return;
                    }
                    copy_rows(r, which, smem_addr(stage(in)));
                    copy_commit();
                    ++pending;
                    if (++in == STAGES) {
                        in = 0;
                        parity ^= 1;
                    }
                    if (pending > AHEAD) {
                        copy_wait<AHEAD>();
                        announce();
                    }
                }
            }
        } while (next_piece<BN>(p, TT, c));
        copy_wait<0>();
        while (pending) announce();
    }

    // FP8: the codes run RAWS - 1 blocks ahead.
    __device__ __forceinline__ void convert_loop(Piece c)
    {
        constexpr int RAWS = S::RAWS > 0 ? S::RAWS : 1;
        uint8_t *const raw = stage(STAGES);
        Piece src = c;
        int64_t total = 2 * c.left, copied = 0;
        int hi = 0, lo = 0, slot_in = 0;
        Rows r{};
        bool fresh = true;
        const auto copy_next = [&]() {
            if (copied < total) {
                const int which = (int)(copied & 1);
                if (which == 0) {
                    if (fresh) {
                        const int first = src.t * TT, last = min(first + TT, src.s.n) - 1;
                        hi = key_hi(p, src.s, last);
                        lo = key_lo(p, src.s, first);
                        fresh = false;
                    }
                    r = find_rows(src, src.k, hi, lo);
                }
                copy_rows(r, which, smem_addr(raw + slot_in * S::RAW));
                if (which == 1) {
                    // One block further: a piece of its own for the cursor.
                    ++src.k;
                    --src.left;
                    if (src.k == src.end && src.left > 0) {
                        next_piece<BN>(p, TT, src);
                        fresh = true;
                    }
                }
            }
            copy_commit();
            ++copied;
            slot_in = slot_in + 1 == RAWS ? 0 : slot_in + 1;
        };
        for (int i = 0; i < RAWS - 1; ++i) copy_next();
        int slot = 0, to = 0;
        uint32_t parity = 1;
        for (int64_t i = 0; i < total; ++i) {
            copy_next();                                      // into the slot converted last
            copy_wait<RAWS - 1>();
            if (!wait_all(&sm.empty[to], parity)) break;
            convert(raw + slot * S::RAW, stage(to));
            fence_async();
            bar_arrive(at(&sm.full[to]));
            slot = slot + 1 == RAWS ? 0 : slot + 1;
            if (++to == STAGES) {
                to = 0;
                parity ^= 1;
            }
        }
        copy_wait<0>();
    }

    // ----------------------------------------------------------- products --
    static constexpr uint32_t kScores = product_desc(!FP8, false, 128, BN);
    static constexpr uint32_t kValues = product_desc(!FP8, true, 128, DP);

    __device__ __forceinline__ uint32_t s_col(int half, int buf) const { return tmem + (uint32_t)(half * NS + buf) * BN; }
    __device__ __forceinline__ uint32_t o_col(int half) const { return tmem + (uint32_t)(S::OCOL + half * DP); }
    __device__ __forceinline__ void scores(int half, int buf, int st) const
    {
        const uint32_t q = smem_addr(queries(half)), k = smem_addr(stage(st));
#pragma unroll
        for (int i = 0; i < DP / 16; ++i)
            product_ss(s_col(half, buf), matrix_desc(q + (i / 4) * (128 * 128) + (i % 4) * 32, 16),
                       matrix_desc(k + (i / 4) * (BN * 128) + (i % 4) * 32, 16), kScores, i > 0);
    }
    __device__ __forceinline__ void values(int half, int buf, int st, bool add) const
    {
        const uint32_t v = smem_addr(stage(st));
#pragma unroll
        for (int i = 0; i < BN / 16; ++i)
            product_ts(o_col(half), s_col(half, buf) + i * 8, matrix_desc(v + i * 2048, BN * 128), kValues, add || i > 0);
    }

    __device__ __forceinline__ void issue_loop(Piece c)
    {
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
        do {
            const int blocks = c.end - c.k;
            bool use[NT];
            for (int h = 0; h < NT; ++h) use[h] = used(c, h);
            for (int h = 0; h < NT; ++h)
                if (use[h]) {
                    if (!wait(&sm.q[h], q_par[h])) return;
                    q_par[h] ^= 1;
                }
            if (!wait(&sm.full[st], full)) return;
            tc_fence_after();
            for (int h = 0; h < NT; ++h)
                if (use[h]) {
                    const int buf = NS == 2 ? w_cnt[h] & 1 : 0;
                    scores(h, buf, st);
                    products_done(at(&sm.s[h * NS + buf]));
                }
            products_done(at(&sm.empty[st]));
            for (int i = 0; i < blocks; ++i) {
                int kst, vst;
                uint32_t kpar, vpar;
                later(1, vst, vpar);
                later(2, kst, kpar);
                const bool more = i + 1 < blocks;
                if (NS == 2) {
                    if (more) {
                        if (!wait(&sm.full[kst], kpar)) return;
                        tc_fence_after();
                        const int buf = (w_cnt[0] + 1) & 1;
                        scores(0, buf, kst);
                        products_done(at(&sm.s[buf]));
                        products_done(at(&sm.empty[kst]));
                    }
                    const int buf = w_cnt[0] & 1;
                    if (!wait(&sm.full[vst], vpar) || !wait(&sm.w[buf], (w_cnt[0] >> 1) & 1)) return;
                    tc_fence_after();
                    values(0, buf, vst, i > 0);
                    products_done(at(&sm.o[0]));
                    products_done(at(&sm.empty[vst]));
                    ++w_cnt[0];
                } else {
                    bool k_here = false;
                    if (!wait(&sm.full[vst], vpar)) return;
                    for (int h = 0; h < NT; ++h) {
                        if (!use[h]) continue;
                        if (!wait(&sm.w[h], w_cnt[h] & 1)) return;
                        tc_fence_after();
                        values(h, 0, vst, i > 0);
                        products_done(at(&sm.o[h]));
                        if (h == NT - 1 || !use[NT - 1]) products_done(at(&sm.empty[vst]));
                        if (more) {
                            if (!k_here && !wait(&sm.full[kst], kpar)) return;
                            k_here = true;
                            tc_fence_after();
                            scores(h, 0, kst);
                            products_done(at(&sm.s[h]));
                        }
                        ++w_cnt[h];
                    }
                    if (more) products_done(at(&sm.empty[kst]));
                }
                later(2, st, full);
            }
        } while (next_piece<BN>(p, TT, c));
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
        w.tok = c.t * TT + i;
        w.head = c.h * p.group.d + rr - i * p.group.d;
        return w;
    }
    // The row's queries to shared memory; returns the exponent by which they
    // were scaled (FP8).
    __device__ __forceinline__ int load_queries(const Piece &c, int half) const
    {
        const Row w = row_of(c, half);
        const uint16_t *src = p.q.p + (int64_t)(c.s.first + w.tok) * p.q.ld + w.head * p.q.hs;
        uint8_t *dst = queries(half);
        const int r = threadIdx.x & 127;
        const auto load = [&](int chunk) {
            if (!w.valid || chunk * 8 >= p.D || !dbg_global(src + chunk * 8, 16, false)) return make_uint4(0, 0, 0, 0);
            return __ldg(reinterpret_cast<const uint4 *>(src + chunk * 8));
        };
        int e = 0;
        if constexpr (FP8) {
            float top = 0.f;
#pragma unroll 8
            for (int k = 0; k < DP / 8; ++k) {
                const uint4 v = load(k);
                for (const uint32_t x : {v.x, v.y, v.z, v.w}) top = fmaxf(top, fmaxf(fabsf(bf_lo(x)), fabsf(bf_hi(x))));
            }
            e = row_exponent(top);
        }
#pragma unroll 8
        for (int k = 0; k < DP / 8; ++k) {
            uint4 v = load(k);
            if constexpr (FP8) {
                const auto half_of = [&](uint32_t x) { return pack_f16(scaled(bf_lo(x), e), scaled(bf_hi(x), e)); };
                v = make_uint4(half_of(v.x), half_of(v.y), half_of(v.z), half_of(v.w));
            }
            put16(dst + matrix_at(r, k, 128 * 128), v.x, v.y, v.z, v.w);
        }
        fence_async();
        bar_arrive(at(&sm.q[half]));
        return e;
    }

    __device__ __forceinline__ void weight_loop(Piece c, int half)
    {
        const uint32_t lanes = (uint32_t)((threadIdx.x >> 5) & 3) << 21;       // lane 32 (warp % 4), in bits 16 up
        const float vs = FP8 ? ld_f32_ro(p.scale[1]) : 1.f;
        const float c_all = FP8 ? p.qk_scale * ld_f32_ro(p.scale[0]) : p.qk_scale;
        bool any = true;
        while (!used(c, half) && (any = next_piece<BN>(p, TT, c))) {}
        if (!any) return;
        int e = load_queries(c, half);
        uint32_t cnt = 0;                                     // blocks so far
        bool good = true;
        while (any) {
            const Row row = row_of(c, half);
            const int hi = key_hi(p, c.s, row.tok), lo = key_lo(p, c.s, row.tok);
            const float scale = FP8 ? scaled(c_all, -e) : c_all;
            float M = -INFINITY;                              // reference, as a raw score
            float L = 0.f;
            for (int k = c.k; k < c.end && good; ++k, ++cnt) {
                const int buf = NS == 2 ? cnt & 1 : 0;
                const uint32_t sc = s_col(half, buf) + lanes;
                good = wait_all(&sm.s[half * NS + buf], NS == 2 ? (cnt >> 1) & 1 : cnt & 1);
                if (!good) break;
                tc_fence_after();
                uint32_t x[BN];
#pragma unroll
                for (int i = 0; i < BN / 32; ++i) tmem_ld32(sc + 32 * i, x + 32 * i);
                tmem_wait_ld();
                const int hk = hi - k * BN, lk = lo - k * BN;
                if (__any_sync(0xffffffffu, hk < BN || lk > 0)) {
#pragma unroll
                    for (int j = 0; j < BN; ++j)
                        if (j >= hk || j < lk) x[j] = 0xff800000u;
                }
                float top = -INFINITY, top1 = -INFINITY, top2 = -INFINITY, top3 = -INFINITY;
#pragma unroll
                for (int j = 0; j < BN; j += 8) {
                    top = fmaxf(top, fmaxf(__uint_as_float(x[j]), __uint_as_float(x[j + 1])));
                    top1 = fmaxf(top1, fmaxf(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])));
                    top2 = fmaxf(top2, fmaxf(__uint_as_float(x[j + 4]), __uint_as_float(x[j + 5])));
                    top3 = fmaxf(top3, fmaxf(__uint_as_float(x[j + 6]), __uint_as_float(x[j + 7])));
                }
                top = fmaxf(M, fmaxf(fmaxf(top, top1), fmaxf(top2, top3)));
                // O of the block before is done; it is what a new reference changes.
                if (cnt > 0) {
                    good = wait_all(&sm.o[half], (cnt - 1) & 1);
                    if (!good) break;
                    tc_fence_after();
                }
                if (__any_sync(0xffffffffu, (top - M) * scale > 8.f || M == -INFINITY)) {
                    const float keep = M == -INFINITY || top == M ? 1.f : exp2_fast((M - top) * scale);
                    L *= keep;
                    if (k > c.k && __any_sync(0xffffffffu, keep != 1.f)) {
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
                    M = top;
                }
                const float ref = M == -INFINITY ? 0.f : -M * scale;
                F2 sum = f2(0.f), sum1 = f2(0.f);
#pragma unroll
                for (int i = 0; i < BN / 32; ++i) {
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const F2 a = f2_fma(f2(__uint_as_float(x[32 * i + 2 * j]), __uint_as_float(x[32 * i + 2 * j + 1])), f2(scale),
                                            f2(ref));
                        const F2 b = f2(exp2_fast(a.x), exp2_fast(a.y));
                        if (j & 1) sum1 = f2_add(sum1, b);
                        else sum = f2_add(sum, b);
                        w[j] = FP8 ? pack_f16(b.x, b.y) : pack_bf16(b.x, b.y);
                    }
                    tmem_st16(sc + 16 * i, w);
                }
                sum = f2_add(sum, sum1);
                L += sum.x + sum.y;
                tmem_wait_st();
                tc_fence_before();
                bar_arrive(at(&sm.w[half * NS + buf]));
            }
            // The scores are read: the next tile's queries may come.
            Piece nx = c;
            int e1 = 0;
            while ((any = next_piece<BN>(p, TT, nx)) && !used(nx, half)) {}
            if (any && good) e1 = load_queries(nx, half);
            if (good) good = wait_all(&sm.o[half], (cnt - 1) & 1);
            tc_fence_after();
            finish(c, half, row, M * scale, L, vs, lanes, good);
            c = nx;
            e = e1;
        }
    }

    // A row's result, or part.  good = false: a wait ran out, and the row is NaN.
    __device__ __forceinline__ void finish(const Piece &c, int half, const Row &row, float M, float L, float vs, uint32_t lanes,
                                           bool good)
    {
        const int64_t t = c.s.first + row.tok;
        const bool whole = c.k == c.k0 && c.end == c.k1;
        if (!good) L = NAN;
        if (whole) {
            const float inv = L == 0.f ? 0.f : vs / L;
            uint16_t *out = const_cast<uint16_t *>(p.out.p) + t * p.out.ld + row.head * p.out.hs;
            bool odd = false;
#pragma unroll 1
            for (int i = 0; i < DP / 32; ++i) {
                uint32_t y[32];
                tmem_ld32(o_col(half) + lanes + 32 * i, y);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 8) {
                    uint32_t z[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const F2 v = f2_mul(f2(__uint_as_float(y[j + 2 * n]), __uint_as_float(y[j + 2 * n + 1])), f2(inv));
                        odd = odd || (row.valid && (suspect(v.x, L) || suspect(v.y, L)));
                        z[n] = bf16_f2(v);
                    }
                    if (row.valid && 32 * i + j < p.D) st_u32x4(out + 32 * i + j, z[0], z[1], z[2], z[3]);
                }
            }
            if (row.valid && p.lse) st_f32(p.lse + t * p.out.H + row.head, L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718f);
            uint32_t again = __ballot_sync(0xffffffffu, odd);
            __syncwarp();
            while (again) {
                const int l = __ffs(again) - 1;
                again &= again - 1;
                attend_row<KIND, DP / 32>(p, c.b, c.s, __shfl_sync(0xffffffffu, row.tok, l), __shfl_sync(0xffffffffu, row.head, l),
                                          false);
            }
        } else {
            float *part = part_of(p.ws, blockIdx.x, c.k == c.k0, S::ROWS, DP);
            const int r = half * 128 + (threadIdx.x & 127);
            if (row.valid) {
                st_f32(part + 2 * r, good ? M : 0.f);
                st_f32(part + 2 * r + 1, L);
            }
            part += 2 * S::ROWS + (int64_t)r * DP;
#pragma unroll 1
            for (int i = 0; i < DP / 32; ++i) {
                uint32_t y[32];
                tmem_ld32(o_col(half) + lanes + 32 * i, y);
                tmem_wait_ld();
                if (row.valid)
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        st_f32x4(part + 32 * i + j, __uint_as_float(y[j]), __uint_as_float(y[j + 1]), __uint_as_float(y[j + 2]),
                                 __uint_as_float(y[j + 3]));
            }
        }
        tc_fence_before();
    }

    // -------------------------------------------------------------- start --
    __device__ __forceinline__ void go()
    {
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
        TT = S::ROWS / p.group.d;
        const Work work = share_work<kTileThreads>(
            p.B, p.Hk, sm.scratch,
            [&](int b, int64_t &u, int64_t &t) {
                const Seq s = sequence(p, b);
                const int nt = (s.n + TT - 1) / TT;
                u = blocks_before<BN>(p, s, TT, nt, nt);
                t = nt;
            },
            // A CTA for each tile; tiles are shared out further while that leaves a CTA four blocks.
            [&](int64_t units, int64_t tiles) { return (int)min((int64_t)gridDim.x, max(tiles, units / 4)); });
        if ((int)blockIdx.x >= work.ctas) {
            if (tid == 0) st_header(p.ws, blockIdx.x, AttnHeader{});
            return;
        }
        Piece c;
        c.b = work.b;
        c.s = sequence(p, c.b);
        c.nt = (c.s.n + TT - 1) / TT;
        const int64_t whole = blocks_before<BN>(p, c.s, TT, c.nt, c.nt);
        c.h = (int)(work.rest / whole);
        const int64_t rest = work.rest - c.h * whole;
        // The tile of block `rest`: the last with blocks_before(t) <= rest, 32 places at a time.
        int lo = 0, hi = c.nt;
        while (hi - lo > 1) {
            const int by = (hi - lo + 31) / 32, t = lo + lane * by;
            const bool before = t < hi && blocks_before<BN>(p, c.s, TT, c.nt, t) <= rest;
            const int n = __popc(__ballot_sync(0xffffffffu, before)) - 1;
            lo += n * by;
            hi = min(hi, lo + by);
        }
        c.t = lo;
        tile_blocks<BN>(p, c.s, TT, c.t, c.k0, c.k1);
        c.k = c.k0 + (int)(rest - blocks_before<BN>(p, c.s, TT, c.nt, c.t));
        c.left = work.u1 - work.u0;
        piece_ends<BN>(c);
        if (tid == 0) {
            AttnHeader hd{};
            hd.first = work.u0 - (c.k - c.k0);
            hd.last = hd.first + (c.k1 - c.k0);
            hd.units = work.units;
            hd.ctas = work.ctas;
            hd.tile = c.k > c.k0;
            hd.b = c.b;
            hd.h = c.h;
            hd.tok = c.s.first + c.t * TT;
            hd.ntok = min(TT, c.s.n - c.t * TT);
            st_header(p.ws, blockIdx.x, hd);
            for (int i = 0; i < STAGES; ++i) {
                bar_init(at(&sm.full[i]), 128);
                bar_init(at(&sm.empty[i]), 1);
            }
            for (int i = 0; i < NT; ++i) {
                bar_init(at(&sm.q[i]), 128);
                bar_init(at(&sm.o[i]), 1);
            }
            for (int i = 0; i < NT * NS; ++i) {
                bar_init(at(&sm.s[i]), 1);
                bar_init(at(&sm.w[i]), 128);
            }
            bar_init(at(&sm.last), 1);
            sm.failed = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        if (warp == 12) tmem_alloc(smem_addr(&sm.tmem), kTileColumns);
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        tmem = sm.tmem;
        if (warp < 8) {
            more_registers<kWeightRegs>();
            if (warp < 4 * NT) weight_loop(c, warp >> 2);
        } else {
            fewer_registers<kOtherRegs>();
            if (warp < 12) {
                if constexpr (FP8) convert_loop(c);
                else copy_loop(c);
                copy_wait<0>();
            } else if (warp == 12) {
                if (lane == 0) {
                    issue_loop(c);
                    if (sm.failed) {                          // products in flight end before their memory goes
                        products_done(at(&sm.last));
                        for (int i = 0; i < kWaitTries && !bar_try(at(&sm.last), 0); ++i) {}
                    }
                }
                __syncwarp();
            }
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 12) tmem_free(tmem, kTileColumns);
    }
};

template <int KIND, int DP>
__global__ void __launch_bounds__(kTileThreads, 1) k_attn_tile(const __grid_constant__ AttnParams p)
{
    extern __shared__ __align__(1024) uint8_t tile_smem[];
    __shared__ typename TileKernel<KIND, DP>::Shared sm;
    CRMSN_DEBUG_ENTER(p.dbg);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    uint8_t *const base = tile_smem + (1024 - (smem_addr(tile_smem) & 1023)) % 1024;
    TileKernel<KIND, DP> k{p, sm, base, 0, 0};
    k.go();
}

template <int KIND, int DP>
cudaError_t run_attn_tile(const AttnParams &p, int sms, cudaStream_t s)
{
    using S = TileShape<KIND, DP>;
    static std::atomic<int> opted[kOptInDevices];
    if (cudaError_t e = opt_in_smem(k_attn_tile<KIND, DP>, S::SMEM, opted)) return e;
    const int ctas = sms < kAttnMaxCtas ? sms : kAttnMaxCtas;
    if (cudaError_t e = launch_pdl(k_attn_tile<KIND, DP>, dim3(ctas), dim3(kTileThreads), S::SMEM, s, p)) return e;
    return launch_attn_combine(p, S::ROWS, DP, ctas, s);
}

}  // namespace crmsn
