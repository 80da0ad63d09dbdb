// api_attn.cu -- the C ABI of the attention functions declared in
// include/crmsnorm.h: argument checks and the choice of the kernel.  Nothing
// here allocates, synchronises or throws; every check happens before the first
// launch.
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "api_tensors.h"
#include "attn.h"

using namespace crmsn;

namespace {

constexpr int64_t kMaxSequences = 1 << 20, kMaxGroup = 128;
constexpr float kLog2e = 1.44269504f;

// What both functions check first; on CRMSN_OK with no tokens there is nothing
// to launch.
crmsn_status check_common(const crmsn_attention &a)
{
    if (a.T < 0 || a.T > kMaxTokens || a.B < 0 || a.B > kMaxSequences) return CRMSN_ERR_SHAPE;
    if (a.Hk < 1 || a.Hq < 1 || a.Hq > kMaxHeads || a.Hq % a.Hk || a.Hq / a.Hk > kMaxGroup) return CRMSN_ERR_SHAPE;
    if (a.D < 1) return CRMSN_ERR_SHAPE;
    if (a.D > CRMSN_MAX_HEAD_DIM || (a.D & 1)) return CRMSN_ERR_UNSUPPORTED_H;
    if (!a.starts && (a.B ? a.T % a.B : a.T)) return CRMSN_ERR_SHAPE;
    if (!std::isfinite(a.scale * kLog2e) || !(a.scale > 0.f) || a.window < 0 || (a.window && !a.causal)) return CRMSN_ERR_ARG;
    if (a.T == 0 || a.B == 0) return CRMSN_OK;
    const Heads q = heads(a.q, a.Hq), out = heads(a.out, a.Hq);
    if (crmsn_status s = check_heads(q, a.T, a.D)) return s;
    if (crmsn_status s = check_heads(out, a.T, a.D)) return s;
    if (!al(a.starts, 4) || !al(a.lse, 4)) return CRMSN_ERR_ALIGNMENT;
    return CRMSN_OK;
}

// Whether a call whose sequences can have at most `keys` keys needs no workspace.
bool is_short(int64_t keys) { return keys <= kShortKeys; }

crmsn_status check_workspace(const crmsn_attention &a, int64_t keys)
{
    if (is_short(keys)) return CRMSN_OK;
    if (!a.workspace) return CRMSN_ERR_NULL;
    return a.workspace_bytes == 0 || a.workspace_bytes > (uint64_t)1 << 40 ? CRMSN_ERR_WORKSPACE : CRMSN_OK;
}

Region starts_region(const crmsn_attention &a) { return vec_region(a.starts, a.B + 1, 4); }
Region lse_region(const crmsn_attention &a) { return vec_region(a.lse, a.T * a.Hq, 4, true); }
Region ws_region(const crmsn_attention &a, int64_t keys)
{
    return vec_region(is_short(keys) ? nullptr : a.workspace, (int64_t)a.workspace_bytes, 1, true);
}

// The device, its SM count and the workspace, after everything else.
crmsn_status check_device(const crmsn_attention &a, int64_t keys, int &sms)
{
    int dev;
    if (crmsn_status s = device_sms(dev, sms)) return s;
    if (is_short(keys)) return CRMSN_OK;
    if (!al(a.workspace, 256) || a.workspace_bytes < attention_workspace_bytes(a.D, dev)) return CRMSN_ERR_WORKSPACE;
    return CRMSN_OK;
}

void set_common(AttnParams &p, const crmsn_attention &a, int64_t keys)
{
    p.whole = is_short(keys);
    p.q = view(heads(a.q, a.Hq));
    p.out = view(heads(a.out, a.Hq));
    p.starts = a.starts;
    p.n = a.starts ? 0 : (int)(a.T / a.B);
    p.T = (int)a.T;
    p.B = (int)a.B;
    p.D = (int)a.D;
    p.Hk = (int)a.Hk;
    p.group = FastDiv((int)(a.Hq / a.Hk));
    p.causal = a.causal != 0;
    p.window = a.window < kMaxTokens ? (int)a.window : 0;      // no sequence is longer
    p.qk_scale = a.scale * kLog2e;
    p.lse = a.lse;
    p.ws = static_cast<uint8_t *>(a.workspace);
#ifdef CRMSN_DEBUG
    const char *tries = std::getenv("CRMSN_DEBUG_WAIT_TRIES");
    p.wait_tries = tries ? std::atoi(tries) : 0;
#endif
}

// What the tiled kernels want: 16-byte accesses and a head that they hold.
bool tiled(const crmsn_attention &a, int es)
{
    return a.D <= kAttnMaxDim && a.D % (16 / es) == 0 && heads_vec(heads(a.q, a.Hq), a.T, 8) &&
           heads_vec(heads(a.out, a.Hq), a.T, 8);
}

crmsn_status launch(const AttnParams &p, bool fast, int sms, cudaStream_t stream)
{
    if (!fast) return launched(launch_attn_row(p, sms, stream));
    if (!p.starts && (int64_t)p.n * p.group.d <= kDecodeRows) return launched(launch_attn_decode(p, sms, stream));
    switch (p.kind) {
        case CRMSN_CACHE_BF16: return launched(launch_attn_tile_bf16(p, sms, stream));
        case CRMSN_CACHE_E4M3: return launched(launch_attn_tile_e4m3(p, sms, stream));
        default: return launched(launch_attn_tile_e5m2(p, sms, stream));
    }
}

}  // namespace

// ======================================================================
extern "C" {

size_t attention_workspace_bytes(int64_t D, int device)
{
    if (D < 2 || D > CRMSN_MAX_HEAD_DIM || (D & 1)) return 0;
    const int sms = sm_count(device);
    if (sms <= 0) return 0;
    const int ctas = sms < kAttnMaxCtas ? sms : kAttnMaxCtas;
    const int DP = attn_padded((int)D);
    const int64_t parts = D <= kAttnMaxDim ? 2 * ctas * attn_part_floats(attn_tile_rows(DP), DP) : 0;
    return (size_t)(kAttnParts + parts * (int64_t)sizeof(float) + 255) / 256 * 256;
}

crmsn_status attention_status(uint64_t *blocks)
{
    if (blocks) *blocks = 0;
    if (cudaError_t e = cudaDeviceSynchronize()) return launched(e);
    uint64_t sum = 0;
    for (const auto take : {take_given_up_bf16, take_given_up_e4m3, take_given_up_e5m2}) {
        unsigned int n = 0;
        if (cudaError_t e = take(n)) return launched(e);
        sum += n;
    }
    if (blocks) *blocks = sum;
    return sum ? CRMSN_ERR_DEVICE_TIMEOUT : CRMSN_OK;
}

crmsn_status prompt_attention(const crmsn_prompt_attention_call *call, cudaStream_t stream)
{
    if (!call) return CRMSN_ERR_NULL;
    const crmsn_attention &a = call->attention;
    if (crmsn_status s = check_common(a)) return s;
    if (a.T == 0 || a.B == 0) return CRMSN_OK;
    const Heads k = heads(call->k, a.Hk), v = heads(call->v, a.Hk);
    const int64_t keys = a.starts ? a.T : a.T / a.B;
    if (crmsn_status s = check_workspace(a, keys)) return s;
    if (crmsn_status s = check_heads(k, a.T, a.D)) return s;
    if (crmsn_status s = check_heads(v, a.T, a.D)) return s;
    const Region ts[] = {
        heads_region(heads(a.q, a.Hq), a.T, a.D), heads_region(k, a.T, a.D), heads_region(v, a.T, a.D), starts_region(a),
        heads_region(heads(a.out, a.Hq), a.T, a.D, true), lse_region(a), ws_region(a, keys),
    };
    if (crmsn_status s = check_alias(ts, 7)) return s;
    int sms;
    if (crmsn_status s = check_device(a, keys, sms)) return s;
    AttnParams p{};
    CRMSN_SET_DEBUG(p, ts);
    set_common(p, a, keys);
    p.kv[0] = {static_cast<const uint8_t *>(k.p), 0, k.ld, k.hs};
    p.kv[1] = {static_cast<const uint8_t *>(v.p), 0, v.ld, v.hs};
    p.kind = CRMSN_CACHE_BF16;
    p.page = FastDiv(1);
    return launch(p, tiled(a, 2) && heads_vec(k, a.T, 8) && heads_vec(v, a.T, 8), sms, stream);
}

crmsn_status paged_attention(const crmsn_paged_attention_call *call, cudaStream_t stream)
{
    if (!call) return CRMSN_ERR_NULL;
    const crmsn_paged_attention_call &c = *call;
    const crmsn_attention &a = c.attention;
    if (crmsn_status s = check_common(a)) return s;
    if (c.cache_kind != CRMSN_CACHE_BF16 && c.cache_kind != CRMSN_CACHE_E4M3 && c.cache_kind != CRMSN_CACHE_E5M2)
        return CRMSN_ERR_DTYPE;
    if (c.num_pages < 0 || c.page_size < 1 || c.page_size > 0x7fffffff || c.num_pages > 0x7fffffff / c.page_size ||
        c.table_pages < 0 || c.table_pages > kMaxTokens / c.page_size)
        return CRMSN_ERR_SHAPE;
    if (a.T == 0 || a.B == 0) return CRMSN_OK;
    if (c.table_pages > 0 && a.B > 1 && (c.ld_table < 0 || c.ld_table > kMaxStride)) return CRMSN_ERR_SHAPE;
    const bool fp8 = c.cache_kind != CRMSN_CACHE_BF16;
    const int es = fp8 ? 1 : 2;
    const int64_t keys = c.table_pages * c.page_size;
    if (crmsn_status s = check_workspace(a, keys)) return s;
    if (!c.lens || (c.table_pages > 0 && !c.page_table) || (fp8 && (!c.k_scale || !c.v_scale))) return CRMSN_ERR_NULL;
    if (!al(c.lens, 4) || !al(c.page_table, 4) || (fp8 && (!al(c.k_scale, 4) || !al(c.v_scale, 4))))
        return CRMSN_ERR_ALIGNMENT;
    const int64_t P = c.num_pages, S = c.page_size;
    if (P > 0) {
        if (crmsn_status s = check_cache(c.k_cache, c.kps, c.kss, c.khs, es, P, S, a.Hk, a.D)) return s;
        if (crmsn_status s = check_cache(c.v_cache, c.vps, c.vss, c.vhs, es, P, S, a.Hk, a.D)) return s;
    }
    const int64_t pages = P > 0 ? P : 1;
    // A table that the kernels can load from even where no sequence has a page.
    const int32_t *const table = c.table_pages > 0 ? c.page_table : c.lens;
    const Region ts[] = {
        heads_region(heads(a.q, a.Hq), a.T, a.D),
        cache_region(P > 0 ? c.k_cache : nullptr, c.kps, c.kss, c.khs, es, pages, S, a.Hk, a.D, false),
        cache_region(P > 0 ? c.v_cache : nullptr, c.vps, c.vss, c.vhs, es, pages, S, a.Hk, a.D, false),
        {c.table_pages > 0 ? c.page_table : nullptr, 4, c.table_pages, {a.B, 1, 1}, {a.B > 1 ? c.ld_table : 0, 0, 0}, false, -1},
        vec_region(c.lens, a.B, 4), vec_region(fp8 ? c.k_scale : nullptr, 1, 4), vec_region(fp8 ? c.v_scale : nullptr, 1, 4),
        starts_region(a), heads_region(heads(a.out, a.Hq), a.T, a.D, true), lse_region(a), ws_region(a, keys),
    };
    if (crmsn_status s = check_alias(ts, 11)) return s;
    int sms;
    if (crmsn_status s = check_device(a, keys, sms)) return s;
    AttnParams p{};
    CRMSN_SET_DEBUG(p, ts);
    set_common(p, a, keys);
    p.kv[0] = {static_cast<const uint8_t *>(c.k_cache), c.kps, c.kss, c.khs};
    p.kv[1] = {static_cast<const uint8_t *>(c.v_cache), c.vps, c.vss, c.vhs};
    p.kind = c.cache_kind;
    p.scale[0] = c.k_scale;
    p.scale[1] = c.v_scale;
    p.table = table;
    p.ldt = c.ld_table;
    p.num_pages = (int)P;
    p.page = FastDiv((int)S);
    p.max_keys = (int)keys;
    p.lens = c.lens;
    const int v = 16 / es;
    return launch(p, tiled(a, es) && (P == 0 || (cache_vec(c.k_cache, c.kps, c.kss, c.khs, es, P, S, a.Hk, v) &&
                                                 cache_vec(c.v_cache, c.vps, c.vss, c.vhs, es, P, S, a.Hk, v))), sms, stream);
}

}  // extern "C"
