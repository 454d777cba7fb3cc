// C ABI of libkvq: argument validation on the host, then launches.  No call
// allocates memory, throws or aborts; every failure is a kvq_status plus a
// thread-local message.
#include <stdarg.h>
#include <stdio.h>

#include <atomic>
#include <string>

#include <algorithm>

#include "kvq_internal.h"
#include "rows.h"

extern "C" cudaError_t kvq_internal_status_quant(cudaStream_t, uint32_t*);
extern "C" cudaError_t kvq_internal_status_prefill(cudaStream_t, uint32_t*);
extern "C" cudaError_t kvq_internal_status_prefill_bwd(cudaStream_t, uint32_t*);
extern "C" cudaError_t kvq_internal_status_select(cudaStream_t, uint32_t*);
extern "C" cudaError_t kvq_internal_status_decode(cudaStream_t, uint32_t*);
extern "C" cudaError_t kvq_internal_status_policy(cudaStream_t, uint32_t*);
extern "C" cudaError_t kvq_internal_status_block8(cudaStream_t, uint32_t*);
extern "C" cudaError_t kvq_internal_status_block8_attn(cudaStream_t, uint32_t*);

namespace kvq {

static thread_local std::string g_last_error;

void set_error(const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
}

int device_sms(int* device) {
    static std::atomic<int> known[64];
    int dev = -1, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        dev = -1;
    }
    if (device) *device = dev;
    if (dev < 0) return 152;
    if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 152;
    }
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

}  // namespace kvq

using kvq::set_error;

#define KVQ_REQUIRE(cond, code, ...) \
    do {                             \
        if (!(cond)) {               \
            set_error(__VA_ARGS__);  \
            return code;             \
        }                            \
    } while (0)

static bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static kvq_status cuda_status(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return KVQ_OK;
    set_error("%s: %s", what, cudaGetErrorString(e));
    return KVQ_ECUDA;
}

static bool valid_bits(int b) { return b == 2 || b == 4 || b == 8; }
static bool valid_group(int g) { return g == 16 || g == 32 || g == 64 || g == 128; }

extern "C" {

int kvq_version(void) { return 100; }

const char* kvq_last_error(void) { return kvq::g_last_error.c_str(); }

kvq_status kv_quant_pack(const void* x, kvq_dtype dt, int B, int H, int T, int D,
                         const int32_t* gather_idx, int n, int bits, int group, kvq_axis axis,
                         uint32_t* codes, uint16_t* scale, uint16_t* zero, void* stream) {
    KVQ_REQUIRE(B >= 0 && H >= 0 && T >= 0 && n >= 0, KVQ_EINVAL, "kv_quant_pack: negative size");
    if (n == 0 || B == 0 || H == 0) return KVQ_OK;     // nothing to pack
    KVQ_REQUIRE(x && codes && scale && zero, KVQ_EINVAL, "kv_quant_pack: null pointer");
    KVQ_REQUIRE(dt == KVQ_F16 || dt == KVQ_BF16, KVQ_EINVAL, "kv_quant_pack: dtype must be f16 or bf16");
    KVQ_REQUIRE(B >= 0 && H >= 0 && T >= 0 && n >= 0, KVQ_EINVAL, "kv_quant_pack: negative size");
    KVQ_REQUIRE(valid_bits(bits), KVQ_EINVAL, "kv_quant_pack: bits must be 2, 4 or 8 (got %d)", bits);
    KVQ_REQUIRE(valid_group(group), KVQ_EINVAL, "kv_quant_pack: group must be 16/32/64/128 (got %d)", group);
    KVQ_REQUIRE(D > 0 && D <= 1024 && D % 32 == 0, KVQ_EINVAL, "kv_quant_pack: D must be a multiple of 32 in [32, 1024]");
    KVQ_REQUIRE(axis == KVQ_AXIS_CHANNEL || axis == KVQ_AXIS_TOKEN, KVQ_EINVAL, "kv_quant_pack: bad axis");
    KVQ_REQUIRE(gather_idx || n <= T, KVQ_EINVAL, "kv_quant_pack: n > T without a gather list");
    if (axis == KVQ_AXIS_CHANNEL)
        KVQ_REQUIRE(n % group == 0, KVQ_EINVAL, "kv_quant_pack: CHANNEL axis needs n %% group == 0 (n=%d, G=%d)", n, group);
    else
        KVQ_REQUIRE(D % group == 0, KVQ_EINVAL, "kv_quant_pack: TOKEN axis needs D %% group == 0");
    KVQ_REQUIRE(aligned(codes, 4) && aligned(scale, 2) && aligned(zero, 2) && aligned(x, 2),
                KVQ_EINVAL, "kv_quant_pack: misaligned pointer");
    return cuda_status(kvq::launch_quant_pack(x, dt, B * H, T, D, gather_idx, n, bits, group, axis,
                                              codes, scale, zero, (cudaStream_t)stream),
                       "kv_quant_pack launch");
}

kvq_status prefill_attn_scores(const void* q, const void* k, const void* v, kvq_dtype dt, int B,
                               int Hq, int Hkv, int T, int D, float sm_scale, int causal, void* o,
                               float* lse, float* colscore, void* ws, size_t ws_bytes,
                               void* stream) {
    (void)ws;
    (void)ws_bytes;
    KVQ_REQUIRE(q && k && v && o && lse, KVQ_EINVAL, "prefill_attn_scores: null pointer");
    KVQ_REQUIRE(dt == KVQ_F16 || dt == KVQ_BF16, KVQ_EINVAL, "prefill_attn_scores: dtype must be f16 or bf16");
    KVQ_REQUIRE(B > 0 && Hq > 0 && Hkv > 0 && T > 0, KVQ_EINVAL, "prefill_attn_scores: sizes must be positive");
    KVQ_REQUIRE(Hq % Hkv == 0, KVQ_EINVAL, "prefill_attn_scores: Hq %% Hkv != 0");
    KVQ_REQUIRE(D == 64 || D == 128, KVQ_EUNSUPPORTED, "prefill_attn_scores: head dim %d unsupported (64 or 128)", D);
    KVQ_REQUIRE(causal == 1, KVQ_EUNSUPPORTED, "prefill_attn_scores: only causal attention");
    KVQ_REQUIRE((long long)B * Hq <= 65535LL * 1024 && T <= (1 << 30), KVQ_EINVAL, "prefill_attn_scores: too large");
    KVQ_REQUIRE((T + 127) / 128 <= 65535, KVQ_EUNSUPPORTED,
                "prefill_attn_scores: T = %d needs more than 65535 tiles of 128 rows", T);
    KVQ_REQUIRE(aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(o, 16) && aligned(lse, 4),
                KVQ_EINVAL, "prefill_attn_scores: q/k/v/o must be 16-byte aligned");
    KVQ_REQUIRE(sm_scale > 0.0f, KVQ_EINVAL, "prefill_attn_scores: sm_scale must be positive");
    return kvq::run_prefill(q, k, v, dt, B, Hq, Hkv, T, D, sm_scale, o, lse, colscore, 0,
                            (cudaStream_t)stream);
}

kvq_status prefill_window_scores(const void* q, const void* k, kvq_dtype dt, int B, int Hq, int Hkv, int T,
                                 int D, float sm_scale, const float* lse, int w_obs, float* colscore,
                                 void* stream) {
    KVQ_REQUIRE(q && k && lse && colscore, KVQ_EINVAL, "prefill_window_scores: null pointer");
    KVQ_REQUIRE(dt == KVQ_F16 || dt == KVQ_BF16, KVQ_EINVAL, "prefill_window_scores: dtype must be f16 or bf16");
    KVQ_REQUIRE(B > 0 && Hq > 0 && Hkv > 0 && T > 0, KVQ_EINVAL, "prefill_window_scores: sizes must be positive");
    KVQ_REQUIRE(Hq % Hkv == 0, KVQ_EINVAL, "prefill_window_scores: Hq %% Hkv != 0");
    KVQ_REQUIRE(D == 64 || D == 128, KVQ_EUNSUPPORTED, "prefill_window_scores: head dim %d unsupported (64 or 128)", D);
    KVQ_REQUIRE(w_obs >= 1 && w_obs <= T, KVQ_EINVAL, "prefill_window_scores: w_obs must be in [1, T]");
    KVQ_REQUIRE((long long)B * Hq <= 65535LL * 1024 && T <= (1 << 30), KVQ_EINVAL, "prefill_window_scores: too large");
    KVQ_REQUIRE((T + 127) / 128 <= 65535, KVQ_EUNSUPPORTED,
                "prefill_window_scores: T = %d needs more than 65535 tiles of 128 rows", T);
    KVQ_REQUIRE(aligned(q, 16) && aligned(k, 16) && aligned(lse, 4) && aligned(colscore, 4), KVQ_EINVAL,
                "prefill_window_scores: q/k must be 16-byte aligned");
    KVQ_REQUIRE(sm_scale > 0.0f, KVQ_EINVAL, "prefill_window_scores: sm_scale must be positive");
    // pass 2 alone over the last w_obs queries (k stands in for the unused value map)
    return kvq::run_prefill(q, k, k, dt, B, Hq, Hkv, T, D, sm_scale, nullptr, const_cast<float*>(lse),
                            colscore, T - w_obs, (cudaStream_t)stream);
}

kvq_status kvq_score_reduce(const float* colscore, int B, int Hq, int Hkv, int T, int mode,
                            float* out, void* stream) {
    KVQ_REQUIRE(colscore && out, KVQ_EINVAL, "kvq_score_reduce: null pointer");
    KVQ_REQUIRE(B >= 0 && Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && T >= 0, KVQ_EINVAL,
                "kvq_score_reduce: bad sizes");
    KVQ_REQUIRE(mode == 0 || mode == 1, KVQ_EINVAL, "kvq_score_reduce: mode must be 0 or 1");
    return cuda_status(kvq::launch_score_reduce(colscore, B, Hq, Hkv, T, mode, out, (cudaStream_t)stream),
                       "kvq_score_reduce launch");
}

kvq_status select_tokens(const float* score, int B, int H, int T, const int32_t* k_hh, int kmax,
                         int w_recent, int32_t* idx_out, int32_t* n_out, void* ws,
                         size_t ws_bytes, void* stream) {
    (void)ws;
    (void)ws_bytes;
    KVQ_REQUIRE(score && k_hh && idx_out && n_out, KVQ_EINVAL, "select_tokens: null pointer");
    KVQ_REQUIRE(B >= 0 && H >= 0 && T >= 0 && T <= 65536, KVQ_EINVAL, "select_tokens: T must be in [0, 65536]");
    KVQ_REQUIRE(w_recent >= 0 && w_recent <= T, KVQ_EINVAL, "select_tokens: w_recent must be in [0, T]");
    KVQ_REQUIRE(kmax >= 0, KVQ_EINVAL, "select_tokens: kmax must be >= 0");
    KVQ_REQUIRE(B * H <= 2147483647 / 2, KVQ_EINVAL, "select_tokens: too many units");
    return cuda_status(kvq::launch_select(score, B * H, T, k_hh, kmax, w_recent, idx_out, n_out,
                                          (cudaStream_t)stream),
                       "select_tokens launch");
}

static kvq_status check_cache(const kvq_cache* c, const char* who) {
    KVQ_REQUIRE(c, KVQ_EINVAL, "%s: null cache", who);
    KVQ_REQUIRE(c->B > 0 && c->Hq > 0 && c->Hkv > 0 && c->Hq % c->Hkv == 0, KVQ_EINVAL,
                "%s: bad B/Hq/Hkv", who);
    KVQ_REQUIRE(c->Hq / c->Hkv <= 8, KVQ_EUNSUPPORTED, "%s: more than 8 query heads per KV head", who);
    KVQ_REQUIRE(c->D == 64 || c->D == 128, KVQ_EUNSUPPORTED, "%s: head dim must be 64 or 128", who);
    KVQ_REQUIRE(valid_group(c->G) && c->D % c->G == 0, KVQ_EINVAL, "%s: bad group size", who);
    KVQ_REQUIRE(c->dtype == KVQ_F16 || c->dtype == KVQ_BF16, KVQ_EINVAL, "%s: bad dtype", who);
    KVQ_REQUIRE(c->policy >= KVQ_POLICY_MINIKV && c->policy <= KVQ_POLICY_MIKV, KVQ_EINVAL, "%s: bad policy", who);
    KVQ_REQUIRE(c->n_tiers >= 1 && c->n_tiers <= KVQ_MAX_TIERS, KVQ_EINVAL, "%s: n_tiers must be 1 or 2", who);
    for (int t = 0; t < c->n_tiers; ++t) {
        const kvq_tier& tr = c->tier[t];
        KVQ_REQUIRE(valid_bits(tr.k_bits) && valid_bits(tr.v_bits), KVQ_EINVAL, "%s: tier %d bits", who, t);
        KVQ_REQUIRE(tr.k_axis == KVQ_AXIS_CHANNEL || tr.k_axis == KVQ_AXIS_TOKEN, KVQ_EINVAL, "%s: tier %d axis", who, t);
        KVQ_REQUIRE(tr.cap >= 0 && tr.cap % 32 == 0, KVQ_EINVAL, "%s: tier %d cap must be a multiple of 32", who, t);
        KVQ_REQUIRE(aligned(tr.k_codes, 16) && aligned(tr.k_scale, 16) && aligned(tr.k_zero, 16) &&
                        aligned(tr.v_codes, 16) && aligned(tr.v_scale, 16) && aligned(tr.v_zero, 16),
                    KVQ_EINVAL, "%s: tier %d arrays must be 16-byte aligned", who, t);
        if (tr.k_axis == KVQ_AXIS_CHANNEL)
            KVQ_REQUIRE(tr.cap % c->G == 0, KVQ_EINVAL, "%s: tier %d cap must be a multiple of G", who, t);
        KVQ_REQUIRE(tr.k_codes && tr.k_scale && tr.k_zero && tr.v_codes && tr.v_scale && tr.v_zero &&
                        tr.token_id && tr.count,
                    KVQ_EINVAL, "%s: tier %d null pointer", who, t);
        // formats the decode kernel is built for
        const bool ok_combo =
            (tr.k_axis == KVQ_AXIS_CHANNEL && tr.k_bits == 2 && tr.v_bits == 2) ||
            (c->D == 128 && tr.k_axis == KVQ_AXIS_TOKEN &&
             ((tr.k_bits == 8 && tr.v_bits == 4) || (tr.k_bits == 4 && tr.v_bits == 8) ||
              (tr.k_bits == 4 && tr.v_bits == 2) ||
              (tr.k_bits == 4 && tr.v_bits == 4) || (tr.k_bits == 2 && tr.v_bits == 2)));
        KVQ_REQUIRE(ok_combo, KVQ_EUNSUPPORTED, "%s: tier %d format K%dV%d axis %d not built", who, t,
                    tr.k_bits, tr.v_bits, tr.k_axis);
        // the decode kernels take groups of 32 (channels of a value or per-token key, tokens of
        // a per-channel key); the MiniKV single-head path (one query head per KV head, D = 128,
        // 2-bit keys and values) also takes groups of 16
        const bool g16 = c->G == 16 && tr.k_axis == KVQ_AXIS_CHANNEL && tr.k_bits == 2 && tr.v_bits == 2 &&
                         c->D == 128 && c->Hq == c->Hkv;
        KVQ_REQUIRE(c->G == 32 || g16, KVQ_EUNSUPPORTED,
                    "%s: tier %d: G = %d is built for 2-bit MiniKV tiers with D = 128 and Hq == Hkv only", who, t,
                    c->G);
        if (tr.page_table) {
            KVQ_REQUIRE(c->policy == KVQ_POLICY_DIFFKV, KVQ_EUNSUPPORTED, "%s: tier %d: only DiffKV tiers are paged",
                        who, t);
            KVQ_REQUIRE(tr.page_owner && tr.free_ring && tr.ring_ctr && tr.n_pages > 0 && tr.max_pages > 0,
                        KVQ_EINVAL, "%s: tier %d: page pool arrays missing", who, t);
            KVQ_REQUIRE((long long)tr.max_pages * KVQ_PAGE_TOKENS == tr.cap, KVQ_EINVAL,
                        "%s: tier %d: a paged tier's cap must be max_pages * %d", who, t, KVQ_PAGE_TOKENS);
            KVQ_REQUIRE((long long)c->B * c->Hkv * tr.max_pages <= (1LL << 31) - 1, KVQ_EINVAL,
                        "%s: tier %d: page table too large", who, t);
        }
    }
    KVQ_REQUIRE(c->res_cap > 0 && c->res_k && c->res_v && c->res_token_id && c->res_start && c->res_len &&
                    c->seq_len,
                KVQ_EINVAL, "%s: residual arrays missing", who);
    if (c->policy == KVQ_POLICY_MINIKV) {
        KVQ_REQUIRE(c->tier[0].k_axis == KVQ_AXIS_CHANNEL, KVQ_EINVAL, "%s: MiniKV keys are per channel", who);
        KVQ_REQUIRE(c->res_cap >= c->nr + c->G, KVQ_EINVAL, "%s: MiniKV needs res_cap >= nr + G", who);
    } else {
        KVQ_REQUIRE(c->n_tiers == 2, KVQ_EINVAL, "%s: DiffKV/MiKV need two tiers", who);
        KVQ_REQUIRE(c->tier[0].k_axis == KVQ_AXIS_TOKEN && c->tier[1].k_axis == KVQ_AXIS_TOKEN, KVQ_EINVAL,
                    "%s: DiffKV/MiKV tiers use per-token keys", who);
        KVQ_REQUIRE(c->res_cap >= c->nr + 1, KVQ_EINVAL, "%s: res_cap must be >= nr + 1", who);
    }
    if (c->policy == KVQ_POLICY_DIFFKV)
        KVQ_REQUIRE(c->win_acc && c->alpha, KVQ_EINVAL, "%s: DiffKV state arrays missing", who);
    if (c->policy == KVQ_POLICY_MIKV) {
        KVQ_REQUIRE(c->cum_score && c->score_cap > 0, KVQ_EINVAL, "%s: MiKV score array missing", who);
        KVQ_REQUIRE(c->hi_den >= 1, KVQ_EINVAL, "%s: hi_den must be >= 1", who);
        KVQ_REQUIRE(c->tier[0].cap <= 48000, KVQ_EUNSUPPORTED, "%s: INT4 tier capacity above 48000", who);
    }
    return KVQ_OK;
}

size_t kvq_decode_workspace_bytes(const kvq_cache* c) {
    if (check_cache(c, "kvq_decode_workspace_bytes") != KVQ_OK) return (size_t)-1;
    return kvq::decode_workspace_bytes(*c);
}

int kvq_decode_launches(const kvq_cache* c) {
    if (check_cache(c, "kvq_decode_launches") != KVQ_OK) return -1;
    const int n = kvq::decode_launches(*c);
    if (n < 0) set_error("kvq_decode_launches: the device occupancy query failed");
    return n;
}

kvq_status decode_attn_qkv(const void* q, const void* k_new, const void* v_new, kvq_cache* c,
                           float sm_scale, void* o, float* lse_out, void* ws, size_t ws_bytes,
                           void* stream) {
    kvq_status st = check_cache(c, "decode_attn_qkv");
    if (st != KVQ_OK) return st;
    KVQ_REQUIRE(q && k_new && v_new && o, KVQ_EINVAL, "decode_attn_qkv: null pointer");
    KVQ_REQUIRE(aligned(k_new, 16) && aligned(v_new, 16) && aligned(c->res_k, 16) && aligned(c->res_v, 16),
                KVQ_EINVAL, "decode_attn_qkv: k_new, v_new and the residual ring must be 16-byte aligned");
    const size_t need = kvq::decode_workspace_bytes(*c);
    KVQ_REQUIRE(need == 0 || (ws && ws_bytes >= need), KVQ_EWORKSPACE,
                "decode_attn_qkv: workspace of %zu bytes needed, %zu given", need, ws_bytes);
    KVQ_REQUIRE(need == 0 || aligned(ws, 256), KVQ_EINVAL, "decode_attn_qkv: workspace must be 256-byte aligned");
    KVQ_REQUIRE(sm_scale > 0.0f, KVQ_EINVAL, "decode_attn_qkv: sm_scale must be positive");
    return cuda_status(kvq::launch_decode(q, k_new, v_new, *c, sm_scale, o, lse_out, ws,
                                          (cudaStream_t)stream),
                       "decode_attn_qkv launch");
}

kvq_status decode_attn_qkv_static(const void* q, const void* k_new, const void* v_new, kvq_cache* c,
                                  float sm_scale, void* o, float* lse_out, void* stream) {
    kvq_status st = check_cache(c, "decode_attn_qkv_static");
    if (st != KVQ_OK) return st;
    KVQ_REQUIRE(q && k_new && v_new && o, KVQ_EINVAL, "decode_attn_qkv_static: null pointer");
    KVQ_REQUIRE(aligned(k_new, 16) && aligned(v_new, 16) && aligned(c->res_k, 16) && aligned(c->res_v, 16),
                KVQ_EINVAL, "decode_attn_qkv_static: k_new, v_new and the residual ring must be 16-byte aligned");
    KVQ_REQUIRE(sm_scale > 0.0f, KVQ_EINVAL, "decode_attn_qkv_static: sm_scale must be positive");
    const size_t need = kvq::decode_workspace_bytes(*c);
    KVQ_REQUIRE(need <= (size_t)KVQ_STATIC_SCRATCH_BYTES, KVQ_EWORKSPACE,
                "decode_attn_qkv_static: this cache needs %zu bytes of scratch, more than the %u bytes "
                "built into the library; use decode_attn_qkv with a caller workspace",
                need, (unsigned)KVQ_STATIC_SCRATCH_BYTES);
    void* ws = nullptr;
    kvq_status s2 = cuda_status(kvq::static_decode_scratch(&ws), "decode_attn_qkv_static scratch lookup");
    if (s2 != KVQ_OK) return s2;
    return cuda_status(kvq::launch_decode(q, k_new, v_new, *c, sm_scale, o, lse_out, ws,
                                          (cudaStream_t)stream),
                       "decode_attn_qkv_static launch");
}

kvq_status requant_demote(kvq_cache* c, kvq_policy mode, const kvq_policy_params* p, int step,
                          void* stream) {
    kvq_status st = check_cache(c, "requant_demote");
    if (st != KVQ_OK) return st;
    KVQ_REQUIRE((int)mode == c->policy, KVQ_EINVAL, "requant_demote: mode differs from the cache policy");
    KVQ_REQUIRE(step >= 0, KVQ_EINVAL, "requant_demote: step must be >= 0");
    if (step == 0) {
        KVQ_REQUIRE(p && p->k_src && p->v_src && p->T > 0, KVQ_EINVAL, "requant_demote: build inputs missing");
        if (mode == KVQ_POLICY_MINIKV) {
            KVQ_REQUIRE(p->sel_idx && p->n_sel >= 0 && p->n_sel <= p->T, KVQ_EINVAL, "requant_demote: sel_idx/n_sel");
            const int n = p->n_sel, nr = c->nr, G = c->G;
            const int r0 = n <= nr ? n : nr + (n - nr) % G;
            KVQ_REQUIRE(n - r0 <= c->tier[0].cap, KVQ_EINVAL, "requant_demote: tier 0 capacity %d < %d packed tokens",
                        c->tier[0].cap, n - r0);
            KVQ_REQUIRE(r0 < c->res_cap, KVQ_EINVAL, "requant_demote: residual capacity too small");
        } else {
            KVQ_REQUIRE(p->colscore, KVQ_EINVAL, "requant_demote: colscore missing");
            KVQ_REQUIRE(p->T > c->nr, KVQ_EINVAL, "requant_demote: T must exceed the window/residual");
            KVQ_REQUIRE(p->T <= c->score_cap || mode == KVQ_POLICY_DIFFKV, KVQ_EINVAL, "requant_demote: score_cap < T");
            if (mode == KVQ_POLICY_DIFFKV) {
                // n_high / n_low live on the device: tier capacities are checked there
                KVQ_REQUIRE(p->n_high && p->n_low, KVQ_EINVAL, "requant_demote: n_high/n_low missing");
            } else {
                KVQ_REQUIRE(c->tier[0].cap + 0 >= (p->T - c->nr) / c->hi_den && c->tier[1].cap >= p->T - c->nr - (p->T - c->nr) / c->hi_den,
                            KVQ_EINVAL, "requant_demote: tier capacity too small");
            }
        }
    }
    return kvq::run_policy(*c, mode, p, step, (cudaStream_t)stream);
}

static bool any_paged(const kvq_cache* c) {
    for (int t = 0; t < c->n_tiers; ++t)
        if (c->tier[t].page_table) return true;
    return false;
}

kvq_status kvq_pages_init(kvq_cache* c, void* stream) {
    kvq_status st = check_cache(c, "kvq_pages_init");
    if (st != KVQ_OK) return st;
    KVQ_REQUIRE(any_paged(c), KVQ_EINVAL, "kvq_pages_init: the cache has no paged tier");
    return kvq::run_pages_init(*c, (cudaStream_t)stream);
}

kvq_status kvq_pages_release(kvq_cache* c, const int32_t* release_mask, void* stream) {
    kvq_status st = check_cache(c, "kvq_pages_release");
    if (st != KVQ_OK) return st;
    KVQ_REQUIRE(release_mask, KVQ_EINVAL, "kvq_pages_release: null mask");
    return kvq::run_pages_release(*c, release_mask, (cudaStream_t)stream);
}

kvq_status minikv_prefill_build(kvq_cache* c, const void* k, const void* v, int T, const float* score,
                                const int32_t* k_hh, int kmax, int w_recent, int32_t* idx_out, void* stream) {
    kvq_status st = check_cache(c, "minikv_prefill_build");
    if (st != KVQ_OK) return st;
    KVQ_REQUIRE(c->policy == KVQ_POLICY_MINIKV, KVQ_EINVAL, "minikv_prefill_build: not a MiniKV cache");
    KVQ_REQUIRE(k && v && score && k_hh, KVQ_EINVAL, "minikv_prefill_build: null pointer");
    KVQ_REQUIRE(c->G == 32, KVQ_EUNSUPPORTED, "minikv_prefill_build: built for G = 32 (requant_demote takes G = 16)");
    KVQ_REQUIRE(aligned(k, 16) && aligned(v, 16) && aligned(c->res_k, 16) && aligned(c->res_v, 16), KVQ_EINVAL,
                "minikv_prefill_build: k, v and the residual ring must be 16-byte aligned");
    KVQ_REQUIRE(T > 0 && T <= 65536, KVQ_EINVAL, "minikv_prefill_build: T must be in [1, 65536]");
    KVQ_REQUIRE(w_recent >= 0 && w_recent <= T && kmax >= 0, KVQ_EINVAL, "minikv_prefill_build: bad kmax / w_recent");
    KVQ_REQUIRE((long long)kmax + w_recent <= 51200, KVQ_EUNSUPPORTED,
                "minikv_prefill_build: kmax + w_recent = %lld positions exceed the 200 KB on-chip list",
                (long long)kmax + w_recent);
    const int nmax = std::min(kmax, T - w_recent) + w_recent;
    KVQ_REQUIRE(std::max(0, nmax - c->nr) <= c->tier[0].cap, KVQ_EINVAL,
                "minikv_prefill_build: tier 0 capacity %d < %d packed tokens", c->tier[0].cap,
                std::max(0, nmax - c->nr));
    return kvq::run_minikv_fused_build(*c, k, v, T, score, k_hh, kmax, w_recent, idx_out, (cudaStream_t)stream);
}

// ---------------------------------------------------------------- 8-bit block cache

static kvq_status check_block8(const kvq_block8* c, const char* who) {
    KVQ_REQUIRE(c, KVQ_EINVAL, "%s: null cache", who);
    KVQ_REQUIRE(c->B > 0 && c->Hq > 0 && c->Hkv > 0 && c->Hq % c->Hkv == 0, KVQ_EINVAL, "%s: bad B/Hq/Hkv", who);
    KVQ_REQUIRE(c->Hq / c->Hkv <= KVQ_BLOCK8_MAX_GROUP, KVQ_EUNSUPPORTED, "%s: more than %d query heads per KV head",
                who, KVQ_BLOCK8_MAX_GROUP);
    KVQ_REQUIRE(c->D == 64 || c->D == 128, KVQ_EUNSUPPORTED, "%s: head dim %d unsupported (64 or 128)", who, c->D);
    KVQ_REQUIRE(c->dtype == KVQ_F16 || c->dtype == KVQ_BF16, KVQ_EINVAL, "%s: dtype must be f16 or bf16", who);
    KVQ_REQUIRE(c->code == KVQ_CODE_E4M3 || c->code == KVQ_CODE_INT8, KVQ_EINVAL, "%s: code must be e4m3 or int8", who);
    KVQ_REQUIRE(c->block == 16 || c->block == 32 || c->block == 64 || c->block == 128, KVQ_EINVAL,
                "%s: block must be 16, 32, 64 or 128 tokens (got %d)", who, c->block);
    KVQ_REQUIRE(c->max_blocks > 0 && c->n_blocks > 0, KVQ_EINVAL, "%s: max_blocks and n_blocks must be positive", who);
    // counts, token numbers and work items (16 tokens each, for every query) are 32-bit
    KVQ_REQUIRE((long long)c->max_blocks * c->block <= (1LL << 30), KVQ_EUNSUPPORTED, "%s: more than 2^30 tokens per unit",
                who);
    KVQ_REQUIRE((long long)c->B * c->Hq <= (1LL << 24) &&
                    (long long)c->B * c->Hkv <= ((1LL << 35) / KVQ_BLOCK8_MAX_Q) / ((long long)c->max_blocks * c->block),
                KVQ_EUNSUPPORTED, "%s: cache too large", who);
    KVQ_REQUIRE((long long)c->n_blocks * c->block <= (1LL << 35), KVQ_EUNSUPPORTED, "%s: pool too large", who);
    KVQ_REQUIRE(c->k_codes && c->v_codes && c->k_scale && c->v_scale && c->k_bound && c->bound_scale && c->tail_k &&
                    c->tail_v && c->table && c->count && c->seq_len && c->block_pos && c->acc,
                KVQ_EINVAL, "%s: null array", who);
    KVQ_REQUIRE(aligned(c->k_codes, 16) && aligned(c->v_codes, 16) && aligned(c->k_bound, 16) && aligned(c->tail_k, 16) &&
                    aligned(c->tail_v, 16),
                KVQ_EINVAL, "%s: codes, bounds and tails must be 16-byte aligned", who);
    KVQ_REQUIRE(aligned(c->k_scale, 4) && aligned(c->v_scale, 4) && aligned(c->bound_scale, 4) && aligned(c->table, 4) &&
                    aligned(c->count, 4) && aligned(c->seq_len, 4) && aligned(c->block_pos, 4) && aligned(c->acc, 4),
                KVQ_EINVAL, "%s: misaligned array", who);
    return KVQ_OK;
}

// Element strides {b, h, t} of x [B, H, n, D]; NULL means contiguous.
static kvq_status row_strides(const void* x, const int64_t* given, int H, int n, int D, const char* who, int64_t* out) {
    KVQ_REQUIRE(x, KVQ_EINVAL, "%s: null pointer", who);
    KVQ_REQUIRE(aligned(x, 16), KVQ_EINVAL, "%s: activations must be 16-byte aligned", who);
    const int64_t dense[3] = {(int64_t)H * n * D, (int64_t)n * D, D};
    for (int i = 0; i < 3; ++i) {
        out[i] = given ? given[i] : dense[i];
        KVQ_REQUIRE(out[i] >= 0 && out[i] % 8 == 0, KVQ_EINVAL, "%s: strides must be >= 0 and multiples of 8 elements",
                    who);
    }
    return KVQ_OK;
}

kvq_status block8_reset(kvq_block8* c, const int32_t* mask, void* stream) {
    kvq_status st = check_block8(c, "block8_reset");
    if (st != KVQ_OK) return st;
    return cuda_status(kvq::launch_block8_reset(*c, mask, (cudaStream_t)stream), "block8_reset launch");
}

kvq_status block8_append(kvq_block8* c, const void* k, const int64_t* k_strides, const void* v,
                         const int64_t* v_strides, int n, const int32_t* n_new, const float* colscore,
                         void* stream) {
    kvq_status st = check_block8(c, "block8_append");
    if (st != KVQ_OK) return st;
    KVQ_REQUIRE(n >= 0, KVQ_EINVAL, "block8_append: negative size");
    if (n == 0) return KVQ_OK;
    KVQ_REQUIRE(n <= c->max_blocks * c->block, KVQ_EINVAL, "block8_append: n = %d tokens exceed the table's %d", n,
                c->max_blocks * c->block);
    int64_t ks[3], vs[3];
    if ((st = row_strides(k, k_strides, c->Hkv, n, c->D, "block8_append", ks)) != KVQ_OK) return st;
    if ((st = row_strides(v, v_strides, c->Hkv, n, c->D, "block8_append", vs)) != KVQ_OK) return st;
    return cuda_status(kvq::launch_block8_append(*c, k, ks, v, vs, n, n_new, colscore, (cudaStream_t)stream),
                       "block8_append launch");
}

static kvq_status check_queries(const kvq_block8* c, int n_q, const char* who) {
    kvq_status st = check_block8(c, who);
    if (st != KVQ_OK) return st;
    KVQ_REQUIRE(n_q >= 1, KVQ_EINVAL, "%s: n_q must be positive", who);
    KVQ_REQUIRE(n_q <= KVQ_BLOCK8_MAX_Q, KVQ_EUNSUPPORTED, "%s: more than %d queries per sequence", who,
                KVQ_BLOCK8_MAX_Q);
    return KVQ_OK;
}

static kvq_status check_ws(const void* ws, size_t given, size_t need, const char* who) {
    KVQ_REQUIRE(need == 0 || (ws && given >= need), KVQ_EWORKSPACE, "%s: workspace of %zu bytes needed, %zu given", who,
                need, ws ? given : (size_t)0);
    KVQ_REQUIRE(need == 0 || aligned(ws, 256), KVQ_EINVAL, "%s: workspace must be 256-byte aligned", who);
    return KVQ_OK;
}

// What a call writes shares no memory with what it reads nor with what else it writes (row 0: not there).  Bit 10 i + j of
// `same`: output i may be input j, which it replaces row for row.
static kvq_status check_apart(const kvq::Rows* out, int n_out, const kvq::Rows* in, int n_in, uint64_t same,
                              const char* who) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; out[i].row && j < n_in; ++j)
            KVQ_REQUIRE(in[j].row == 0 || (same >> (10 * i + j) & 1) || !kvq::rows_meet(out[i], in[j]), KVQ_EINVAL,
                        "%s: an output or the workspace overlaps an input", who);
        for (int j = 0; out[i].row && j < i; ++j)
            KVQ_REQUIRE(out[j].row == 0 || !kvq::rows_meet(out[i], out[j]), KVQ_EINVAL,
                        "%s: outputs or the workspace overlap one another", who);
    }
    return KVQ_OK;
}

// Rows of n_sel list entries (0: no lists).  What one call works through, 16 tokens for up to 32 rows
// at a time (at least 8), is counted in 32 bits.
static kvq_status check_list(const kvq_block8* c, int n_q, int n_sel, const char* who) {
    KVQ_REQUIRE(n_sel <= (1 << 20), KVQ_EUNSUPPORTED, "%s: n_sel = %d is too large", who, n_sel);
    const long long g = c->Hq / c->Hkv, rows = n_sel ? g : g * n_q, sets = (long long)c->B * c->Hkv * (n_sel ? n_q : 1);
    const long long cells = (long long)(n_sel && n_sel < c->max_blocks ? n_sel : c->max_blocks) * (c->block / 16);
    KVQ_REQUIRE(cells <= (1LL << 30) / (sets * ((rows + 31) / 32)), KVQ_EUNSUPPORTED,
                "%s: too many tokens for one call (%lld units or lists of %lld x 16)", who, sets, cells);
    return KVQ_OK;
}

size_t block8_attn_workspace_bytes(const kvq_block8* c, int n_q, int n_sel, int accumulate) {
    const char* who = "block8_attn_workspace_bytes";
    if (check_queries(c, n_q, who) != KVQ_OK) return (size_t)-1;
    if (n_sel < 0) {
        set_error("%s: n_sel must be >= 0", who);
        return (size_t)-1;
    }
    if (check_list(c, n_q, n_sel, who) != KVQ_OK) return (size_t)-1;
    return kvq::block8_attn_bytes(*c, n_q, n_sel, accumulate);
}

kvq_status block8_attn(const void* q, const int64_t* q_strides, int n_q, const int32_t* n_new, kvq_block8* c,
                       float sm_scale, const int32_t* blocks, const int32_t* list_len, int n_sel,
                       int accumulate, void* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
    kvq_status st = check_queries(c, n_q, "block8_attn");
    if (st != KVQ_OK) return st;
    int64_t qs[3];
    if ((st = row_strides(q, q_strides, c->Hq, n_q, c->D, "block8_attn", qs)) != KVQ_OK) return st;
    KVQ_REQUIRE(o && aligned(o, 16) && aligned(lse, 4), KVQ_EINVAL, "block8_attn: o must be given and 16-byte aligned");
    KVQ_REQUIRE(sm_scale > 0.0f, KVQ_EINVAL, "block8_attn: sm_scale must be positive");
    if (blocks) {
        KVQ_REQUIRE(list_len && n_sel >= 1, KVQ_EINVAL, "block8_attn: a block list needs list_len and n_sel >= 1");
    } else {
        KVQ_REQUIRE(!list_len && n_sel == 0, KVQ_EINVAL, "block8_attn: list_len or n_sel without a block list");
    }
    if ((st = check_list(c, n_q, n_sel, "block8_attn")) != KVQ_OK) return st;
    if ((st = check_ws(ws, ws_bytes, kvq::block8_attn_bytes(*c, n_q, n_sel, accumulate), "block8_attn")) != KVQ_OK)
        return st;
    return cuda_status(kvq::launch_block8_attn(q, qs, n_q, n_new, *c, sm_scale, blocks, list_len, n_sel, accumulate, o,
                                               lse, ws, (cudaStream_t)stream),
                       "block8_attn launch");
}

size_t block8_select_workspace_bytes(const kvq_block8* c, int n_q) {
    if (check_queries(c, n_q, "block8_select_workspace_bytes") != KVQ_OK) return (size_t)-1;
    return kvq::block8_select_bytes(*c, n_q);
}

kvq_status block8_select(const void* q, const int64_t* q_strides, int n_q, const int32_t* n_new, kvq_block8* c,
                         int n_sel, int n_first, int n_last, int32_t* idx_out, int32_t* n_out, void* ws,
                         size_t ws_bytes, void* stream) {
    kvq_status st = check_queries(c, n_q, "block8_select");
    if (st != KVQ_OK) return st;
    int64_t qs[3];
    if ((st = row_strides(q, q_strides, c->Hq, n_q, c->D, "block8_select", qs)) != KVQ_OK) return st;
    KVQ_REQUIRE(idx_out && n_out, KVQ_EINVAL, "block8_select: null output");
    KVQ_REQUIRE(n_sel >= 1 && n_first >= 0 && n_last >= 0 && n_first <= n_sel && n_last <= n_sel - n_first, KVQ_EINVAL,
                "block8_select: n_sel >= 1, n_first, n_last >= 0 and n_first + n_last <= n_sel are needed");
    KVQ_REQUIRE(c->max_blocks <= (1 << 20), KVQ_EUNSUPPORTED, "block8_select: more than 2^20 blocks per unit");
    if ((st = check_list(c, n_q, n_sel, "block8_select")) != KVQ_OK) return st;
    if ((st = check_ws(ws, ws_bytes, kvq::block8_select_bytes(*c, n_q), "block8_select")) != KVQ_OK) return st;
    return cuda_status(kvq::launch_block8_select(q, qs, n_q, n_new, *c, n_sel, n_first, n_last, idx_out, n_out, ws,
                                                 (cudaStream_t)stream),
                       "block8_select launch");
}

kvq_status block8_evict(kvq_block8* c, const int32_t* keep, int n_first, int n_last, int32_t* n_evicted,
                        void* stream) {
    kvq_status st = check_block8(c, "block8_evict");
    if (st != KVQ_OK) return st;
    KVQ_REQUIRE(keep, KVQ_EINVAL, "block8_evict: null keep");
    KVQ_REQUIRE(n_first >= 0 && n_last >= 1 && n_first <= c->max_blocks && n_last <= c->max_blocks, KVQ_EINVAL,
                "block8_evict: n_first >= 0 and n_last >= 1 (the open block stays), at most max_blocks");
    KVQ_REQUIRE(c->max_blocks <= 51200, KVQ_EUNSUPPORTED, "block8_evict: more than 51200 blocks per unit");
    return cuda_status(kvq::launch_block8_evict(*c, keep, n_first, n_last, n_evicted, (cudaStream_t)stream),
                       "block8_evict launch");
}

// ---------------------------------------------------------------- gradient of prefill attention

static kvq_status check_prefill_bwd(int B, int Hq, int Hkv, int T, const char* who) {
    KVQ_REQUIRE(B > 0 && Hq > 0 && Hkv > 0 && T > 0, KVQ_EINVAL, "%s: sizes must be positive", who);
    KVQ_REQUIRE(Hq % Hkv == 0, KVQ_EINVAL, "%s: Hq %% Hkv != 0", who);
    // a CTA per head and tile of 128 tokens
    KVQ_REQUIRE(T <= (1 << 24) && (long long)B * Hq <= (1LL << 30) / ((T + 127) / 128), KVQ_EUNSUPPORTED, "%s: too large",
                who);
    return KVQ_OK;
}

size_t prefill_attn_bwd_workspace_bytes(int B, int Hq, int Hkv, int T) {
    if (check_prefill_bwd(B, Hq, Hkv, T, "prefill_attn_bwd_workspace_bytes") != KVQ_OK) return (size_t)-1;
    return kvq::prefill_bwd_bytes(B, Hq, Hkv, T);
}

kvq_status prefill_attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* go, kvq_dtype dt,
                            int B, int Hq, int Hkv, int T, int D, float sm_scale, int causal, const float* lse,
                            const float* glse, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
    const char* who = "prefill_attn_bwd";
    KVQ_REQUIRE(q && k && v && o && go && lse && dq && dk && dv, KVQ_EINVAL, "%s: null pointer", who);
    KVQ_REQUIRE(dt == KVQ_F16 || dt == KVQ_BF16, KVQ_EINVAL, "%s: dtype must be f16 or bf16", who);
    kvq_status st = check_prefill_bwd(B, Hq, Hkv, T, who);
    if (st != KVQ_OK) return st;
    KVQ_REQUIRE(D == 64 || D == 128, KVQ_EUNSUPPORTED, "%s: head dim %d unsupported (64 or 128)", who, D);
    KVQ_REQUIRE(causal == 1, KVQ_EUNSUPPORTED, "%s: only causal attention", who);
    KVQ_REQUIRE(aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(o, 16) && aligned(go, 16) &&
                    aligned(dq, 16) && aligned(dk, 16) && aligned(dv, 16) && aligned(lse, 4) && aligned(glse, 4),
                KVQ_EINVAL, "%s: q/k/v/o/go/dq/dk/dv must be 16-byte aligned", who);
    KVQ_REQUIRE(sm_scale > 0.0f && sm_scale < 1e30f, KVQ_EINVAL, "%s: sm_scale must be positive and finite", who);
    const size_t need = kvq::prefill_bwd_bytes(B, Hq, Hkv, T);
    if ((st = check_ws(ws, ws_bytes, need, who)) != KVQ_OK) return st;
    // the two kernels of the call run side by side: neither may write what the other still reads
    const int64_t lse_bytes = (int64_t)B * Hq * T * 4, q_bytes = lse_bytes / 2 * D, kv_bytes = (int64_t)B * Hkv * T * D * 2;
    const kvq::Rows in[] = {{q, q_bytes}, {k, kv_bytes}, {v, kv_bytes}, {o, q_bytes}, {go, q_bytes}, {lse, lse_bytes},
                            {glse, glse ? lse_bytes : 0}};
    const kvq::Rows out[] = {{dq, q_bytes}, {dk, kv_bytes}, {dv, kv_bytes}, {ws, (int64_t)need}};
    if ((st = check_apart(out, 4, in, 7, 0, who)) != KVQ_OK) return st;
    kvq::PrefillBwdCall c = {};
    c.dt = dt, c.B = B, c.Hq = Hq, c.Hkv = Hkv, c.T = T, c.D = D, c.q = q, c.k = k, c.v = v, c.o = o, c.go = go;
    c.lse = lse, c.glse = glse, c.sm_scale = sm_scale, c.dq = dq, c.dk = dk, c.dv = dv, c.ws = ws;
    return kvq::run_prefill_bwd(c, (cudaStream_t)stream);
}

// ---------------------------------------------------------------- norm and rotation per head

static kvq_status check_rope(const kvq_rope* r, kvq_dtype dt, int B, int T, int Hq, int Hkv, int D, float eps,
                             const char* who) {
    KVQ_REQUIRE(r, KVQ_EINVAL, "%s: null rope", who);
    KVQ_REQUIRE(dt == KVQ_F16 || dt == KVQ_BF16, KVQ_EINVAL, "%s: dtype must be f16 or bf16", who);
    KVQ_REQUIRE(B >= 0 && T >= 0 && Hq > 0 && Hkv > 0 && Hq % Hkv == 0, KVQ_EINVAL, "%s: bad B/T/Hq/Hkv", who);
    KVQ_REQUIRE(D == 64 || D == 128, KVQ_EUNSUPPORTED, "%s: head dim %d unsupported (64 or 128)", who, D);
    KVQ_REQUIRE(Hq <= (1 << 20) && (long long)B * T <= (1LL << 30), KVQ_EUNSUPPORTED, "%s: too large", who);
    KVQ_REQUIRE(r->rot >= 0 && r->rot <= D && r->rot % 16 == 0, KVQ_EINVAL,
                "%s: rot = %d must be a multiple of 16 in [0, D]", who, r->rot);
    KVQ_REQUIRE(r->interleaved == 0 || r->interleaved == 1, KVQ_EINVAL, "%s: interleaved must be 0 or 1", who);
    KVQ_REQUIRE(r->n_axes >= 1 && r->n_axes <= KVQ_ROPE_MAX_AXES, KVQ_EINVAL, "%s: n_axes must be 1 to %d", who,
                KVQ_ROPE_MAX_AXES);
    for (int i = 0; i < r->rot / 2; ++i)
        KVQ_REQUIRE(r->axis[i] < r->n_axes, KVQ_EINVAL, "%s: pair %d has axis %d of %d", who, i, r->axis[i], r->n_axes);
    KVQ_REQUIRE(eps >= 0.0f && eps < 1e30f, KVQ_EINVAL, "%s: eps must be >= 0 and finite", who);
    return KVQ_OK;
}

// Strides {b, t, head} of rows [B, T, H, D]; that of an axis of one entry counts for nothing.
static kvq_status head_strides(const void* x, const int64_t* given, int B, int T, int H, int D, const char* who,
                               int64_t* out) {
    KVQ_REQUIRE(x, KVQ_EINVAL, "%s: null pointer", who);
    KVQ_REQUIRE(aligned(x, 16), KVQ_EINVAL, "%s: activations must be 16-byte aligned", who);
    const int64_t dense[3] = {(int64_t)T * H * D, (int64_t)H * D, D};
    const int size[3] = {B, T, H};
    for (int i = 0; i < 3; ++i) {
        out[i] = size[i] == 1 ? 0 : given ? given[i] : dense[i];
        KVQ_REQUIRE(out[i] >= 0 && out[i] % 8 == 0, KVQ_EINVAL, "%s: strides must be >= 0 and multiples of 8 elements",
                    who);
    }
    return KVQ_OK;
}

// Rows [B, T, H, D] of 16-bit elements (strides of head_strides()); x NULL: none.
static kvq::Rows head_rows(const void* x, int B, int T, int H, int D, const int64_t* st) {
    if (!x) return {};
    return kvq::Rows(x, 2 * D, {B, T, H}, {2 * st[0], 2 * st[1], 2 * st[2]});
}

// Bit `bit` where rows [B, T, H, D] at x with strides st are those at y with strides sy (NULL: contiguous [B, H, T, D]).
// A row's lanes read it before they write it and no others do, so such an output may replace its input.
static uint64_t same_rows(int bit, const void* x, const int64_t* st, const void* y, const int64_t* sy, int B, int T, int H,
                          int D) {
    const int64_t dense[3] = {(int64_t)H * T * D, D, (int64_t)T * D};
    const int size[3] = {B, T, H};
    for (int i = 0; i < 3; ++i)
        if (x != y || (size[i] != 1 && st[i] != (sy ? sy : dense)[i])) return 0;
    return 1ull << bit;
}

kvq_status qk_norm_rope(const kvq_rope* rope, kvq_dtype dt, int B, int T, int Hq, int Hkv, int D, const void* q,
                        const void* k, const void* v, const int64_t* strides, const int32_t* pos, const void* q_weight,
                        const void* k_weight, int weight_f32, float eps, void* q_out, void* k_out, void* v_out,
                        void* stream) {
    const char* who = "qk_norm_rope";
    kvq_status st = check_rope(rope, dt, B, T, Hq, Hkv, D, eps, who);
    if (st != KVQ_OK || B == 0 || T == 0) return st;
    kvq::RopeCall c = {};
    c.rope = rope, c.dt = dt, c.B = B, c.T = T, c.Hq = Hq, c.Hkv = Hkv, c.D = D, c.q = q, c.k = k, c.v = v;
    c.pos = pos, c.qw = q_weight, c.kw = k_weight, c.w_f32 = weight_f32 != 0, c.eps = eps;
    c.qo = q_out, c.ko = k_out, c.vo = v_out;
    if ((st = head_strides(q, strides, B, T, Hq, D, who, c.strides[0])) != KVQ_OK) return st;
    if ((st = head_strides(k, strides ? strides + 3 : nullptr, B, T, Hkv, D, who, c.strides[1])) != KVQ_OK) return st;
    if (v && (st = head_strides(v, strides ? strides + 6 : nullptr, B, T, Hkv, D, who, c.strides[2])) != KVQ_OK) return st;
    KVQ_REQUIRE(q_out && k_out && (v_out || !v) && (pos || rope->rot == 0), KVQ_EINVAL, "%s: null pointer", who);
    KVQ_REQUIRE(aligned(q_out, 16) && aligned(k_out, 16) && aligned(v_out, 16) && aligned(q_weight, 16) &&
                    aligned(k_weight, 16) && aligned(pos, 4),
                KVQ_EINVAL, "%s: misaligned pointer", who);
    const int64_t tokens = (int64_t)B * T, pos_bytes = rope->rot ? 4 * tokens * rope->n_axes : 0;
    const int64_t q_bytes = 2 * tokens * Hq * D, kv_bytes = 2 * tokens * Hkv * D, w_bytes = (weight_f32 ? 4 : 2) * D;
    const kvq::Rows in[] = {head_rows(q, B, T, Hq, D, c.strides[0]), head_rows(k, B, T, Hkv, D, c.strides[1]),
                            head_rows(v, B, T, Hkv, D, c.strides[2]), {pos, pos_bytes},
                            {q_weight, q_weight ? w_bytes : 0}, {k_weight, k_weight ? w_bytes : 0}};
    const kvq::Rows out[] = {{q_out, q_bytes}, {k_out, kv_bytes}, {v_out, v ? kv_bytes : 0}};
    const uint64_t same = same_rows(0, q, c.strides[0], q_out, nullptr, B, T, Hq, D) |
                          same_rows(11, k, c.strides[1], k_out, nullptr, B, T, Hkv, D) |
                          (v ? same_rows(22, v, c.strides[2], v_out, nullptr, B, T, Hkv, D) : 0);
    if ((st = check_apart(out, 3, in, 6, same, who)) != KVQ_OK) return st;
    return cuda_status(kvq::launch_rope(c, (cudaStream_t)stream), "qk_norm_rope launch");
}

size_t qk_norm_rope_bwd_workspace_bytes(int B, int T, int D, int norm) {
    if (B < 0 || T < 0 || (D != 64 && D != 128)) {
        set_error("qk_norm_rope_bwd_workspace_bytes: bad sizes");
        return (size_t)-1;
    }
    return norm ? (size_t)kvq::rope_bwd_ctas(B, T) * D * sizeof(float) : 0;
}

kvq_status qk_norm_rope_bwd(const kvq_rope* rope, kvq_dtype dt, int B, int T, int Hq, int Hkv, int D, const void* dq,
                            const void* dk, const void* dv, const void* q, const void* k, const int64_t* strides,
                            const int32_t* pos, const void* q_weight, const void* k_weight, int weight_f32, float eps,
                            void* gq, void* gk, void* gv, const int64_t* g_strides, float* gq_weight, float* gk_weight,
                            void* ws, size_t ws_bytes, void* stream) {
    const char* who = "qk_norm_rope_bwd";
    kvq_status st = check_rope(rope, dt, B, T, Hq, Hkv, D, eps, who);
    if (st != KVQ_OK) return st;
    KVQ_REQUIRE((gq_weight || !q_weight) && (gk_weight || !k_weight), KVQ_EINVAL, "%s: null weight gradient", who);
    KVQ_REQUIRE(aligned(gq_weight, 4) && aligned(gk_weight, 4), KVQ_EINVAL, "%s: misaligned pointer", who);
    if (B == 0 || T == 0) {         // sums of nothing
        cudaError_t e = q_weight ? cudaMemsetAsync(gq_weight, 0, D * sizeof(float), (cudaStream_t)stream) : cudaSuccess;
        if (e == cudaSuccess && k_weight) e = cudaMemsetAsync(gk_weight, 0, D * sizeof(float), (cudaStream_t)stream);
        return cuda_status(e, who);
    }
    kvq::RopeCall c = {};
    c.rope = rope, c.dt = dt, c.B = B, c.T = T, c.Hq = Hq, c.Hkv = Hkv, c.D = D;
    c.q = q_weight ? q : nullptr, c.k = k_weight ? k : nullptr;
    c.pos = pos, c.qw = q_weight, c.kw = k_weight, c.w_f32 = weight_f32 != 0, c.eps = eps;
    c.qo = const_cast<void*>(dq), c.ko = const_cast<void*>(dk), c.vo = const_cast<void*>(dv);
    c.gq = gq, c.gk = gk, c.gv = gv, c.gqw = gq_weight, c.gkw = gk_weight, c.ws = ws;
    if (q_weight && (st = head_strides(q, strides, B, T, Hq, D, who, c.strides[0])) != KVQ_OK) return st;
    if (k_weight && (st = head_strides(k, strides ? strides + 3 : nullptr, B, T, Hkv, D, who, c.strides[1])) != KVQ_OK)
        return st;
    if ((st = head_strides(gq, g_strides, B, T, Hq, D, who, c.gstrides[0])) != KVQ_OK) return st;
    if ((st = head_strides(gk, g_strides ? g_strides + 3 : nullptr, B, T, Hkv, D, who, c.gstrides[1])) != KVQ_OK) return st;
    if (dv && (st = head_strides(gv, g_strides ? g_strides + 6 : nullptr, B, T, Hkv, D, who, c.gstrides[2])) != KVQ_OK)
        return st;
    for (int i = 0; i < 9; ++i) {
        const int size = i % 3 == 0 ? B : i % 3 == 1 ? T : i == 2 ? Hq : Hkv;
        KVQ_REQUIRE(size == 1 || c.gstrides[i / 3][i % 3] > 0 || (i >= 6 && !dv), KVQ_EINVAL,
                    "%s: rows of a gradient must not overlap", who);
    }
    KVQ_REQUIRE(dq && dk && (pos || rope->rot == 0), KVQ_EINVAL, "%s: null pointer", who);
    KVQ_REQUIRE(aligned(dq, 16) && aligned(dk, 16) && aligned(dv, 16) && aligned(q_weight, 16) && aligned(k_weight, 16) &&
                    aligned(pos, 4),
                KVQ_EINVAL, "%s: misaligned pointer", who);
    const size_t need = qk_norm_rope_bwd_workspace_bytes(B, T, D, q_weight || k_weight);
    if ((st = check_ws(ws, ws_bytes, need, who)) != KVQ_OK) return st;
    const int64_t tokens = (int64_t)B * T, pos_bytes = rope->rot ? 4 * tokens * rope->n_axes : 0;
    const int64_t q_bytes = 2 * tokens * Hq * D, kv_bytes = 2 * tokens * Hkv * D, w_bytes = (weight_f32 ? 4 : 2) * D;
    const kvq::Rows in[] = {{dq, q_bytes}, {dk, kv_bytes}, {dv, dv ? kv_bytes : 0},
                            head_rows(c.q, B, T, Hq, D, c.strides[0]), head_rows(c.k, B, T, Hkv, D, c.strides[1]),
                            {pos, pos_bytes}, {q_weight, q_weight ? w_bytes : 0}, {k_weight, k_weight ? w_bytes : 0}};
    const kvq::Rows out[] = {head_rows(gq, B, T, Hq, D, c.gstrides[0]), head_rows(gk, B, T, Hkv, D, c.gstrides[1]),
                             head_rows(dv ? gv : nullptr, B, T, Hkv, D, c.gstrides[2]), {gq_weight, q_weight ? 4 * D : 0},
                             {gk_weight, k_weight ? 4 * D : 0}, {ws, (int64_t)need}};
    for (int i = 0; i < 3; ++i)
        KVQ_REQUIRE(out[i].nested(), KVQ_EINVAL, "%s: rows of a gradient must not overlap", who);
    const uint64_t same = same_rows(0, gq, c.gstrides[0], dq, nullptr, B, T, Hq, D) |
                          same_rows(3, gq, c.gstrides[0], c.q, c.strides[0], B, T, Hq, D) |
                          same_rows(11, gk, c.gstrides[1], dk, nullptr, B, T, Hkv, D) |
                          same_rows(14, gk, c.gstrides[1], c.k, c.strides[1], B, T, Hkv, D) |
                          (dv ? same_rows(22, gv, c.gstrides[2], dv, nullptr, B, T, Hkv, D) : 0);
    if ((st = check_apart(out, 6, in, 8, same, who)) != KVQ_OK) return st;
    return cuda_status(kvq::launch_rope_bwd(c, (cudaStream_t)stream), "qk_norm_rope_bwd launch");
}

size_t kvq_tier_bytes(int units, int D, int G, int k_bits, int v_bits, int k_axis, int cap,
                      size_t out[8]) {
    if (units <= 0 || D <= 0 || !valid_group(G) || D % G || !valid_bits(k_bits) || !valid_bits(v_bits) || cap < 0)
        return 0;
    if (k_axis == KVQ_AXIS_CHANNEL && cap % G) return 0;
    size_t u = (size_t)units;
    size_t kc = k_axis == KVQ_AXIS_CHANNEL ? u * (size_t)cap * k_bits / 32 * D * 4 : u * cap * (size_t)(D * k_bits / 32) * 4;
    size_t ks = k_axis == KVQ_AXIS_CHANNEL ? u * (size_t)(cap / G) * D * 2 : u * cap * (size_t)(D / G) * 2;
    size_t vc = u * cap * (size_t)(D * v_bits / 32) * 4;
    size_t vs = u * cap * (size_t)(D / G) * 2;
    size_t sizes[8] = {kc, ks, ks, vc, vs, vs, u * cap * 4, u * 4};
    size_t tot = 0;
    for (int i = 0; i < 8; ++i) {
        if (out) out[i] = sizes[i];
        tot += sizes[i];
    }
    return tot;
}

kvq_status kvq_debug_withhold_copy(int on) {
    kvq::set_withhold_copy(on);
    return KVQ_OK;
}

kvq_status kvq_device_status(void* stream, uint32_t* out) {
    KVQ_REQUIRE(out, KVQ_EINVAL, "kvq_device_status: null out");
    cudaStream_t s = (cudaStream_t)stream;
    uint32_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    cudaError_t e = kvq_internal_status_quant(s, &v[0]);
    if (e == cudaSuccess) e = kvq_internal_status_prefill(s, &v[1]);
    if (e == cudaSuccess) e = kvq_internal_status_select(s, &v[2]);
    if (e == cudaSuccess) e = kvq_internal_status_decode(s, &v[3]);
    if (e == cudaSuccess) e = kvq_internal_status_policy(s, &v[4]);
    if (e == cudaSuccess) e = kvq_internal_status_block8(s, &v[5]);
    if (e == cudaSuccess) e = kvq_internal_status_block8_attn(s, &v[6]);
    if (e == cudaSuccess) e = kvq_internal_status_prefill_bwd(s, &v[7]);
    if (e != cudaSuccess) return cuda_status(e, "kvq_device_status");
    uint32_t all = v[0] | v[1] | v[2] | v[3] | v[4] | v[5] | v[6] | v[7];
    *out = (all & 1u) ? (uint32_t)KVQ_ETIMEOUT : ((all & 2u) ? (uint32_t)KVQ_EDEVICE : 0u);
    return KVQ_OK;
}

}  // extern "C"
