// attn_decode.cu -- attention of few rows over many keys: the tokens of a
// sequence times the query heads of a key head are at most 16 rows, one side
// of a matrix instruction (mma.m16n8k16).
//
// What bounds it is the cache's way from memory: 2 D elements a key and head,
// read once, for 64 operations an element at 16 rows.  So each warp is a
// pipeline of its own: it copies its KB keys and their values asynchronously
// into a ring of slots in shared memory, works through them with its own
// running maximum, sum and values, and meets the CTA's other warps only at the
// end of a tile (the keys of one sequence and head), whose parts are then
// joined.  The ring runs on across the ends of tiles.  The keys are shared out
// evenly over the CTAs (attn.cuh).  128 sequences of up to 8192 keys, 32 + 8
// heads of 128 in BF16: 368 us, 6.7 TB/s, 98 % of the copy rate.  FP8: half the
// bytes for the same instructions; 2 x 131071 keys in E4M3 take 102 us (78 %),
// with the issue slots 44 % and the arithmetic pipe 40 % busy and two warps a
// scheduler to hide it behind.
//
// Layouts.  Slots hold rows of DP elements with their 16-byte chunks permuted
// (swz) so that the rows of a matrix fragment lie in different banks.  BF16:
// ldmatrix for keys, its transposed form for values.  FP8: products in FP16,
// which holds every code exactly.  A thread's four neighbouring bytes of a key
// serve as the elements k, k+1, k+8, k+9 of its fragment; the queries are
// loaded in the same order.  For the values, transposed 16-bit units bring two
// neighbouring columns of two keys, which go to two products, of the even and
// of the odd columns.
#include "attn.cuh"

namespace crmsn {
namespace {

template <int KIND, int DP>
struct Shape {
    static constexpr int ES = KIND == KV_BF16 ? 2 : 1;
    static constexpr int W = DP > 128 ? 4 : 8;               // warps
    static constexpr int KB = KIND == KV_BF16 && DP > 64 ? 16 : 32;   // keys of a slot
    static constexpr int UNIT = W * KB;                      // keys of a unit
    static constexpr int PITCH = DP * ES, CH = PITCH / 16;   // bytes and chunks of a row
    static constexpr int SLOT = KB * PITCH;
    static constexpr int JOIN = W * kDecodeRows * (DP * 4 + 8);   // parts of the warps
    static constexpr int FIT = (227 * 1024 - 1536 - JOIN) / (W * SLOT);
    static constexpr int NS = FIT < 12 ? FIT : 12;           // slots of a warp
    static constexpr int SMEM = JOIN + W * NS * SLOT;
    static_assert(NS >= 4, "two keys and two values in flight");
};

template <int CH>
__device__ __forceinline__ int swz(int row, int chunk)
{
    return CH % 8 == 0 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
}

// Column d of a row of the joined parts: groups of eight permuted, so that the
// rows of a fragment lie in different banks.
__device__ __forceinline__ int turn(int row, int d) { return d ^ ((row & 7) << 3); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <int KIND>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (KIND == KV_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Units of sequence s: blocks [k0, k1) of UNIT keys, at least one.
template <int UNIT>
__device__ __forceinline__ void units_of(const AttnParams &p, const Seq &s, int &k0, int &k1)
{
    k0 = key_lo(p, s, 0) / UNIT;
    k1 = max((s.m + UNIT - 1) / UNIT, k0 + 1);
}

// A place in the line of units.
struct Cursor {
    int b, k, k0, k1;
    Seq s;
};
struct Begin {
    Cursor at;
    int items;
};
template <int UNIT>
__device__ __forceinline__ void step(const AttnParams &p, Cursor &c)
{
    if (++c.k < c.k1) return;
    if (++c.b < p.B) {
        c.s = sequence(p, c.b);
        units_of<UNIT>(p, c.s, c.k0, c.k1);
    }
    c.k = c.k0;
}

// The rows of the tiles that the CTA had whole, once more where a result is not
// finite: a warp for each tile.
template <int KIND, int DP>
__device__ __noinline__ void look_again(const AttnParams &p, const Begin &begin)
{
    using S = Shape<KIND, DP>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = p.group.d, R = p.n * G, h = (int)blockIdx.x % p.Hk;
    Cursor c = begin.at;
    int items = begin.items;
    for (int tile = 0;; ++tile) {
        const int n = min(c.k1 - c.k, items);
        if (n == c.k1 - c.k0 && tile % S::W == warp) {
            const int row = lane < R ? lane : 0, i = p.group.div(row), t = c.s.first + i, hq = h * G + row - i * G;
            const bool suspect = lane < R && not_finite(p.out.p + (int64_t)t * p.out.ld + hq * p.out.hs, p.D);
            if (__any_sync(0xffffffffu, suspect)) work_out_again<KIND, DP / 32>(p, c.b, h, c.s.first, p.n, t, hq, suspect);
        }
        items -= n;
        if (items <= 0) return;
        c.k = c.k1 - 1;
        step<S::UNIT>(p, c);
    }
}

template <int KIND, int DP>
__global__ void __launch_bounds__(Shape<KIND, DP>::W * 32, 1) k_attn_decode(const __grid_constant__ AttnParams p)
{
    using S = Shape<KIND, DP>;
    constexpr int W = S::W, KB = S::KB, NS = S::NS, CH = S::CH, UNIT = S::UNIT;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ WorkScratch scratch;
    __shared__ int odd;                                       // some result is not finite
    __shared__ Begin begin;
    float *const join_o = reinterpret_cast<float *>(smem);                        // [W][16][DP], permuted (turn)
    float *const join_ml = join_o + W * kDecodeRows * DP;                 // [W][16][2]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t *const ring = smem + S::JOIN + warp * NS * S::SLOT;
    const uint32_t ring_at = smem_addr(ring);
    CRMSN_DEBUG_ENTER(p.dbg);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int G = p.group.d, R = p.n * G;
    Cursor at;                        // of the work
    int items;
    int64_t tile_first = 0, u0 = 0;   // units where the current tile begins, where this CTA does
    const int groups = (int)gridDim.x / p.Hk, group = (int)blockIdx.x / p.Hk, h = (int)blockIdx.x - group * p.Hk;
    if (tid == 0) odd = 0;
    if (p.whole) {
        const int n = min(groups, p.B);
        if (group >= n) return;
        at.b = (int)first_unit(p.B, n, group);
        const int end = (int)first_unit(p.B, n, group + 1);
        at.s = sequence(p, at.b);
        units_of<UNIT>(p, at.s, at.k0, at.k1);
        at.k = at.k0;
        items = 0;
        for (int b = at.b + lane; b < end; b += 32) {
            int k0, k1;
            units_of<UNIT>(p, sequence(p, b), k0, k1);
            items += k1 - k0;
        }
        for (int o = 16; o > 0; o >>= 1) items += __shfl_xor_sync(0xffffffffu, items, o);
    } else {
        const Work work = share_work<W * 32>(
            p.B, group, scratch,
            [&](int b, int64_t &u, int64_t &t) {
                int k0, k1;
                units_of<UNIT>(p, sequence(p, b), k0, k1);
                u = k1 - k0;
                t = 1;
            },
            [&](int64_t units, int64_t) { return (int)min((int64_t)groups, units); });
        if (group >= work.groups) {
            if (tid == 0 && groups > 1) st_header(p.ws, blockIdx.x, AttnHeader{});
            return;
        }
        items = (int)(work.u1 - work.u0);
        u0 = work.u0;
        at.b = work.b;
        at.s = sequence(p, at.b);
        units_of<UNIT>(p, at.s, at.k0, at.k1);
        at.k = at.k0 + (int)work.rest;
        tile_first = u0 - (at.k - at.k0);
        if (tid == 0 && groups > 1) {
            AttnHeader hd{};
            hd.first = tile_first;
            hd.last = tile_first + (at.k1 - at.k0);
            hd.units = work.units;
            hd.groups = work.groups;
            hd.tile = at.k > at.k0;
            hd.b = at.b;
            hd.h = h;
            hd.tok = at.s.first;
            hd.ntok = p.n;
            st_header(p.ws, blockIdx.x, hd);
        }
    }

    if (tid == 0) begin = {at, items};
    // ---- copies: slot 2 i holds the keys, slot 2 i + 1 the values of item i
    Cursor src = at;
    int copied = 0, slot_in = 0;      // slots copied, and where the next goes
    int64_t off[2];                   // of this lane's key of the item: keys, values
    bool ok = false;
    const auto copy_slot = [&]() {
        const int which = copied & 1;
        if (copied < 2 * items) {
            if (which == 0) {
                const int j = src.k * UNIT + warp * KB + lane % KB;
                ok = j < src.s.m && j >= key_lo(p, src.s, 0);
                off[0] = off[1] = 0;
                if (ok) {
                    int page, row;
                    locate(p, src.b, src.s, j, page, row);
                    ok = page >= 0;
                    if (ok) {
                        off[0] = kv_offset(p.kv[0], page, row, h);
                        off[1] = kv_offset(p.kv[1], page, row, h);
                    }
                }
                step<UNIT>(p, src);
            }
            const uint8_t *base = p.kv[which].p;
            const int64_t mine = which ? off[1] : off[0];
            const uint32_t dst = ring_at + slot_in * S::SLOT;
            constexpr int ROWS = CH >= 32 ? 1 : 32 / CH;      // rows of an instruction (CH = 12, 24: idle lanes)
            const int sub = lane / CH, chunk = lane % CH;
#pragma unroll
            for (int r = 0; r < KB; r += ROWS) {
                const int row = r + sub;
                const bool in = sub < ROWS && row < KB;
                const int64_t o = __shfl_sync(0xffffffffu, mine, row & 31);
                const bool good = __shfl_sync(0xffffffffu, ok, row & 31);
                if (in)
                    copy16(dst + row * S::PITCH + swz<CH>(row, chunk) * 16, base + o * S::ES + chunk * 16,
                           good && chunk * 16 < p.D * S::ES);
            }
        }
        copy_commit();
        ++copied;
        slot_in = slot_in + 1 == NS ? 0 : slot_in + 1;
    };
    for (int i = 0; i < NS - 1; ++i) copy_slot();

    // ---- a tile's state
    const int g = lane >> 2, q4 = lane & 3;                   // rows g and g + 8, columns 2 q4, 2 q4 + 1
    const int tok0 = p.group.div(g), tok1 = p.group.div(g + 8);
    // Queries as fragments: in registers, or, where O leaves none, in this warp's place for its part of the join, which
    // is free until the tile ends.
    constexpr bool QS = DP >= 192;
    uint32_t q_regs[QS ? 1 : DP / 16][4];
    uint4 *const q_place = reinterpret_cast<uint4 *>(join_o + warp * kDecodeRows * DP) + lane;
    constexpr float UP = KIND == KV_BF16 ? 0.f : kWeightTop;  // weights are 2^(x - (m - UP))
    float o[DP / 8][4], m0, m1, l0, l1, c0, c1, vs = 1.f, ks = 1.f;
    int hi0, hi1, lo0, lo1, hi_all = 0, lo_all = 0;
    if (KIND != KV_BF16) {
        ks = ld_f32_ro(p.scale[0]);
        vs = ld_f32_ro(p.scale[1]);
    }
    const auto load_queries = [&]() {
        uint32_t qa[DP / 16][4];
        c0 = c1 = p.qk_scale * ks;
        const bool in0 = g < R, in1 = g + 8 < R;
        const uint16_t *r0 = p.q.p + (at.s.first + (in0 ? tok0 : 0)) * p.q.ld + (h * G + (in0 ? g - tok0 * G : 0)) * p.q.hs;
        const uint16_t *r1 = p.q.p + (at.s.first + (in1 ? tok1 : 0)) * p.q.ld + (h * G + (in1 ? g + 8 - tok1 * G : 0)) * p.q.hs;
        const auto pair = [&](const uint16_t *r, bool in, int d) -> uint32_t {
            if (!in || d >= p.D || !dbg_global(r + d, 4, false)) return 0u;
            return __ldg(reinterpret_cast<const uint32_t *>(r + d));
        };
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            const int d0 = 16 * k + (KIND == KV_BF16 ? 2 : 4) * q4, d1 = d0 + (KIND == KV_BF16 ? 8 : 2);
            qa[k][0] = pair(r0, in0, d0);
            qa[k][1] = pair(r1, in1, d0);
            qa[k][2] = pair(r0, in0, d1);
            qa[k][3] = pair(r1, in1, d1);
        }
        if constexpr (KIND != KV_BF16) {
            float a0 = 0.f, a1 = 0.f;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float v = fmaxf(fabsf(bf_lo(qa[k][i])), fabsf(bf_hi(qa[k][i])));
                    if (i & 1) a1 = fmaxf(a1, v);
                    else a0 = fmaxf(a0, v);
                }
            for (int w = 1; w < 4; w *= 2) {
                a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, w));
                a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, w));
            }
            const int e0 = row_exponent(a0), e1 = row_exponent(a1);
            const uint32_t sign = score_sign(c0);
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = i & 1 ? e1 : e0;
                    qa[k][i] = pack_f16(scaled(bf_lo(qa[k][i]), e), scaled(bf_hi(qa[k][i]), e)) ^ sign;
                }
            c0 = score_factor(c0, e0);
            c1 = score_factor(c1, e1);
        }
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            if constexpr (QS) {
                if (dbg_shared(q_place + 32 * k, 16)) q_place[32 * k] = make_uint4(qa[k][0], qa[k][1], qa[k][2], qa[k][3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) q_regs[k][i] = qa[k][i];
            }
        }
#pragma unroll
        for (int k = 0; k < DP / 8; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
        hi0 = key_hi(p, at.s, tok0);
        hi1 = key_hi(p, at.s, tok1);
        lo0 = key_lo(p, at.s, tok0);
        lo1 = key_lo(p, at.s, tok1);
        hi_all = key_hi(p, at.s, 0);                          // keys that all rows see
        lo_all = key_lo(p, at.s, p.n - 1);
    };
    load_queries();

    // ---- the items
    int slot = 0;
    for (int item = 0; item < items; ++item) {
        const int j0 = at.k * UNIT + warp * KB;
        float x[KB / 8][4];
        copy_wait<NS - 2>();
        __syncwarp();
        const uint32_t keys = ring_at + slot * S::SLOT;
        const uint8_t *keys_p = ring + slot * S::SLOT;
#pragma unroll
        for (int b = 0; b < KB / 8; ++b) x[b][0] = x[b][1] = x[b][2] = x[b][3] = 0.f;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
            uint32_t qa[4];
            if constexpr (QS) {
                const uint4 v = q_place[32 * k];
                qa[0] = v.x;
                qa[1] = v.y;
                qa[2] = v.z;
                qa[3] = v.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) qa[i] = q_regs[k][i];
            }
            if constexpr (KIND == KV_BF16) {
#pragma unroll
                for (int b = 0; b < KB / 16; ++b) {
                    const int row = 16 * b + (lane & 7) + ((lane >> 4) << 3), chunk = 2 * k + ((lane >> 3) & 1);
                    uint32_t f[4];
                    ldsm4(f, keys + row * S::PITCH + swz<CH>(row, chunk) * 16);
                    mma<KIND>(x[2 * b], qa, f[0], f[1]);
                    mma<KIND>(x[2 * b + 1], qa, f[2], f[3]);
                }
            } else {
#pragma unroll
                for (int b = 0; b < KB / 8; ++b) {
                    const int row = 8 * b + g;
                    const uint32_t codes = *reinterpret_cast<const uint32_t *>(keys_p + row * S::PITCH + swz<CH>(row, k) * 16 + 4 * q4);
                    uint32_t b0, b1;
                    f16_codes<KIND>(codes, b0, b1);
                    mma<KIND>(x[b], qa, b0, b1);
                }
            }
        }
        __syncwarp();                 // all lanes have read the slot before the last
        slot = slot + 1 == NS ? 0 : slot + 1;
        copy_slot();
        if (j0 + KB > hi_all || j0 < lo_all) {
#pragma unroll
            for (int b = 0; b < KB / 8; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int j = j0 + 8 * b + 2 * q4 + i;
                    if (j >= hi0 || j < lo0) x[b][i] = -INFINITY;
                    if (j >= hi1 || j < lo1) x[b][2 + i] = -INFINITY;
                }
        }
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int b = 0; b < KB / 8; ++b) {
            t0 = fmaxf(t0, fmaxf(x[b][0], x[b][1]));
            t1 = fmaxf(t1, fmaxf(x[b][2], x[b][3]));
        }
        for (int w = 1; w < 4; w *= 2) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, w));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, w));
        }
        t0 = fmaxf(m0, t0 * c0);
        t1 = fmaxf(m1, t1 * c1);
        if (__any_sync(0xffffffffu, t0 > m0 || t1 > m1)) {
            const float a0 = t0 > m0 ? exp2_fast(m0 - t0) : 1.f, a1 = t1 > m1 ? exp2_fast(m1 - t1) : 1.f;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int k = 0; k < DP / 8; ++k) {
                o[k][0] *= a0;
                o[k][1] *= a0;
                o[k][2] *= a1;
                o[k][3] *= a1;
            }
            m0 = t0;
            m1 = t1;
        }
        const float z0 = m0 == -INFINITY ? 0.f : m0 - UP, z1 = m1 == -INFINITY ? 0.f : m1 - UP;
        uint32_t pa[KB / 16][4];      // the weights: BF16 (FP8 caches: FP16) operands of the product with the values
#pragma unroll
        for (int b = 0; b < KB / 8; ++b) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = exp2_fast(fmaf(x[b][i], i < 2 ? c0 : c1, i < 2 ? -z0 : -z1));
            l0 += w[0] + w[1];
            l1 += w[2] + w[3];
            pa[b / 2][(b & 1) * 2] = KIND == KV_BF16 ? pack_bf16(w[0], w[1]) : pack_f16(w[0], w[1]);
            pa[b / 2][(b & 1) * 2 + 1] = KIND == KV_BF16 ? pack_bf16(w[2], w[3]) : pack_f16(w[2], w[3]);
        }
        copy_wait<NS - 2>();
        __syncwarp();
        const uint32_t values = ring_at + slot * S::SLOT;
#pragma unroll
        for (int b = 0; b < KB / 16; ++b) {
            if constexpr (KIND == KV_BF16) {
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const int row = 16 * b + (lane & 15), chunk = 2 * k + (lane >> 4);
                    uint32_t f[4];
                    ldsm4_t(f, values + row * S::PITCH + swz<CH>(row, chunk) * 16);
                    mma<KIND>(o[2 * k], pa[b], f[0], f[1]);
                    mma<KIND>(o[2 * k + 1], pa[b], f[2], f[3]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < DP / 32; ++k) {
                    const int row = 16 * b + (lane & 15), chunk = 2 * k + (lane >> 4);
                    uint32_t f[4];
                    ldsm4_t(f, values + row * S::PITCH + swz<CH>(row, chunk) * 16);
                    uint32_t even[4], odd[4];             // columns of two keys
#pragma unroll
                    for (int i = 0; i < 4; ++i) f16_codes<KIND>(__byte_perm(f[i], 0, 0x3120), even[i], odd[i]);
                    // Products 4 k, 4 k + 1: even and odd columns of chunk 2 k; 4 k + 2, 4 k + 3: of chunk 2 k + 1.
                    mma<KIND>(o[4 * k], pa[b], even[0], even[1]);
                    mma<KIND>(o[4 * k + 1], pa[b], odd[0], odd[1]);
                    mma<KIND>(o[4 * k + 2], pa[b], even[2], even[3]);
                    mma<KIND>(o[4 * k + 3], pa[b], odd[2], odd[3]);
                }
            }
        }
        __syncwarp();
        slot = slot + 1 == NS ? 0 : slot + 1;
        copy_slot();

        const bool tile_ends = at.k + 1 == at.k1;
        if (!tile_ends && item + 1 < items) {
            ++at.k;
            continue;
        }
        // ---- the tile's end, or this CTA's: join the warps
        for (int w = 1; w < 4; w *= 2) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, w);
            l1 += __shfl_xor_sync(0xffffffffu, l1, w);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = g + 8 * half;
            if (row >= R) continue;
            float *dst = join_o + (warp * kDecodeRows + row) * DP;
#pragma unroll
            for (int k = 0; k < DP / 8; ++k) {
                const float a = o[k][2 * half], b = o[k][2 * half + 1];
                if constexpr (KIND == KV_BF16) {
                    *reinterpret_cast<float2 *>(dst + turn(row, 8 * k + 2 * q4)) = make_float2(a, b);
                } else {
                    const int d = 16 * (k / 2) + 4 * q4 + (k & 1);    // columns 2 n + parity of a chunk
                    dst[turn(row, d)] = a;
                    dst[turn(row, d + 2)] = b;
                }
            }
            if (q4 == 0) {
                float *ml = join_ml + (warp * kDecodeRows + row) * 2;
                ml[0] = (half ? m1 : m0) - UP;
                ml[1] = half ? l1 : l0;
            }
        }
        __syncthreads();
        const bool whole = tile_first >= u0 && tile_ends;
        float *const part = whole ? nullptr : part_of(p.ws, blockIdx.x, tile_first >= u0, kDecodeRows, DP);
        for (int e = tid; e < R * (DP / 4); e += W * 32) {
            const int row = e / (DP / 4), d = (e - row * (DP / 4)) * 4;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < W; ++w) M = fmaxf(M, join_ml[(w * kDecodeRows + row) * 2]);
            const float z = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            F2 a = f2(0.f), b = f2(0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float2 ml = *reinterpret_cast<const float2 *>(join_ml + (w * kDecodeRows + row) * 2);
                const float4 v = *reinterpret_cast<const float4 *>(join_o + (w * kDecodeRows + row) * DP + turn(row, d));
                const float s = exp2f(ml.x - z);
                L = fmaf(ml.y, s, L);
                a = f2_fma(f2(v.x, v.y), f2(s), a);
                b = f2_fma(f2(v.z, v.w), f2(s), b);
            }
            if (whole) {
                const int i = p.group.div(row), hq = h * G + row - i * G;
                const int64_t t = at.s.first + i;
                const float inv = vs / L;
                a = L == 0.f ? f2(0.f) : f2_mul(a, f2(inv));  // no key: zeros, whatever 0 times the values was
                b = L == 0.f ? f2(0.f) : f2_mul(b, f2(inv));
                if (d < p.D) {
                    if (suspect(a.x, L) || suspect(a.y, L) || suspect(b.x, L) || suspect(b.y, L)) odd = 1;
                    st_u32x2(const_cast<uint16_t *>(p.out.p) + t * p.out.ld + hq * p.out.hs + d, bf16_f2(a), bf16_f2(b));
                }
                if (d == 0 && p.lse)
                    st_f32(p.lse + t * p.out.H + hq, L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718f);
            } else {
                if (d == 0) {
                    st_f32(part + 2 * row, M);
                    st_f32(part + 2 * row + 1, L);
                }
                st_f32x4(part + 2 * kDecodeRows + row * DP + d, a.x, a.y, b.x, b.y);
            }
        }
        __syncthreads();
        // Wide heads: the places are kept in memory, which leaves registers to the products.  (64 sequences of 3000 keys, 16 +
        // 4 heads, E5M2: 102.7 us at D = 192 and 116.6 at 256, in registers 110.5 and 124.8.)
        if constexpr (QS) asm volatile("" :: "l"(&at), "l"(&src) : "memory");
        if (item + 1 < items) {
            tile_first += at.k1 - at.k0;
            step<UNIT>(p, at);
            load_queries();
        }
    }
    copy_wait<0>();
    if (odd) look_again<KIND, DP>(p, begin);                  // (the barrier behind the last tile's results)
}

template <int KIND, int DP>
cudaError_t run(const AttnParams &p, int sms, cudaStream_t s)
{
    using S = Shape<KIND, DP>;
    static std::atomic<int> opted[kOptInDevices];
    if (cudaError_t e = opt_in_smem(k_attn_decode<KIND, DP>, S::SMEM, opted)) return e;
    const int groups = attn_groups(sms, p.Hk);
    if (cudaError_t e = launch_pdl(k_attn_decode<KIND, DP>, dim3(groups * p.Hk), dim3(S::W * 32), S::SMEM, s, p)) return e;
    return p.whole ? cudaSuccess : launch_attn_combine(p, kDecodeRows, DP, groups, s);
}

template <int KIND>
cudaError_t run(const AttnParams &p, int sms, cudaStream_t s)
{
    switch (attn_padded(p.D)) {
        case 64: return run<KIND, 64>(p, sms, s);
        case 128: return run<KIND, 128>(p, sms, s);
        case 192: return run<KIND, 192>(p, sms, s);
        default: return run<KIND, 256>(p, sms, s);
    }
}

}  // namespace

cudaError_t launch_attn_decode(const AttnParams &p, int sms, cudaStream_t s)
{
    switch (p.kind) {
        case KV_BF16: return run<KV_BF16>(p, sms, s);
        case KV_E4M3: return run<KV_E4M3>(p, sms, s);
        default: return run<KV_E5M2>(p, sms, s);
    }
}

}  // namespace crmsn
