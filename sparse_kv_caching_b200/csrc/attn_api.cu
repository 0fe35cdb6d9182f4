// C ABI of the exact attention calls (declared in include/lola.h): argument
// checks and the kernels' arguments.
#include <cmath>
#include <cstdint>

#include "attn.h"
#include "lola.h"

using lola::report;

namespace {

bool misaligned(const void* p) { return ((uintptr_t)p & 15u) != 0; }

int bad_stride(const char* what, long long stride, long long size, int esize, bool zero_ok) {
    if (size <= 1) return LOLA_OK;                       // never used
    if (stride < 0 || stride * esize % 16 || stride >= (1LL << 36) || (stride == 0 && !zero_ok))
        return report(LOLA_ERR_INVALID_ARG, "%s stride %lld: not a non-negative multiple of 16 bytes%s", what, stride,
                      stride == 0 ? " (0 is not allowed here)" : "");
    return LOLA_OK;
}

int check_config(const lola_attn_config* c) {
    if (!c) return report(LOLA_ERR_INVALID_ARG, "null config");
    if (c->B < 1 || c->T < 1 || c->Hq < 1 || c->Hkv < 1 || c->Hq % c->Hkv || c->B > 65535 || c->Hkv > 65535)
        return report(LOLA_ERR_INVALID_ARG, "bad heads, batch or tokens: B=%d T=%d Hq=%d Hkv=%d", c->B, c->T, c->Hq,
                      c->Hkv);
    if ((double)c->B * c->T * c->Hq >= 2147483648.0)
        return report(LOLA_ERR_UNSUPPORTED, "B * T * Hq = %g is not below 2^31", (double)c->B * c->T * c->Hq);
    if (c->P < 0 || c->L < 0) return report(LOLA_ERR_INVALID_ARG, "negative key count: P=%d L=%d", c->P, c->L);
    if ((double)c->P + c->L >= 2147000000.0)
        return report(LOLA_ERR_UNSUPPORTED, "P + L = %g keys", (double)c->P + c->L);
    if (c->d != 64 && c->d != 128) return report(LOLA_ERR_UNSUPPORTED, "d=%d (64 or 128)", c->d);
    if (c->dtype != LOLA_DTYPE_F32 && c->dtype != LOLA_DTYPE_BF16)
        return report(LOLA_ERR_INVALID_ARG, "dtype=%d", c->dtype);
    if (!(c->scale > 0.f) || !std::isfinite(c->scale * 1.4426950408889634f))
        return report(LOLA_ERR_INVALID_ARG, "scale=%g must be positive and finite", (double)c->scale);
    const int e = c->dtype == LOLA_DTYPE_BF16 ? 2 : 4;
    const struct { const char* what; long long stride, size; bool zero_ok; } st[] = {
        {"q batch", c->q_stride[0], c->B, true},    {"q token", c->q_stride[1], c->T, true},
        {"q head", c->q_stride[2], c->Hq, true},    {"k_prefix token", c->kp_stride[0], c->P, false},
        {"k_prefix head", c->kp_stride[1], c->P > 0 ? c->Hkv : 1, true},
        {"v_prefix token", c->vp_stride[0], c->P, false},
        {"v_prefix head", c->vp_stride[1], c->P > 0 ? c->Hkv : 1, true},
        {"k batch", c->k_stride[0], c->L > 0 ? c->B : 1, true}, {"k token", c->k_stride[1], c->L, false},
        {"k head", c->k_stride[2], c->L > 0 ? c->Hkv : 1, true},
        {"v batch", c->v_stride[0], c->L > 0 ? c->B : 1, true}, {"v token", c->v_stride[1], c->L, false},
        {"v head", c->v_stride[2], c->L > 0 ? c->Hkv : 1, true}};
    for (const auto& x : st)
        if (int rc = bad_stride(x.what, x.stride, x.size, e, x.zero_ok)) return rc;
    return LOLA_OK;
}

lola::AttnArgs make_args(const lola_attn_config* c, int causal) {
    lola::AttnArgs a{};
    a.qb = c->q_stride[0]; a.qs = c->q_stride[1]; a.qh = c->q_stride[2];
    a.shared = {nullptr, nullptr, 0, c->kp_stride[0], c->kp_stride[1], 0, c->vp_stride[0], c->vp_stride[1], c->P};
    a.own = {nullptr, nullptr, c->k_stride[0], c->k_stride[1], c->k_stride[2], c->v_stride[0], c->v_stride[1],
             c->v_stride[2], c->L};
    a.causal = causal;
    a.B = c->B; a.T = c->T; a.Hq = c->Hq; a.Hkv = c->Hkv; a.Gq = c->Hq / c->Hkv; a.d = c->d; a.dtype = c->dtype;
    a.scale_log2 = c->scale * 1.4426950408889634f;
    return a;
}

// SMs of the current device (asked of the driver once); without a device (size queries on a host that
// has none) those of a B200.
int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 148;
    }
    if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 148;
    }
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

// One encoder output for all sequences, all of it read: the keys are shared.
bool keys_shared(const lola_attn_config* c) {
    return c->P == 0 && c->B > 1 && c->L > 0 && c->k_stride[0] == 0 && c->v_stride[0] == 0;
}
lola_attn_config as_shared(const lola_attn_config& c) {
    lola_attn_config x = c;
    x.P = c.L;
    x.L = 0;
    x.kp_stride[0] = c.k_stride[1]; x.kp_stride[1] = c.k_stride[2];
    x.vp_stride[0] = c.v_stride[1]; x.vp_stride[1] = c.v_stride[2];
    return x;
}

int run(const lola_attn_config* c, int causal, const void* q, const void* kp, const void* vp, const void* k,
        const void* v, const int* len, void* y, float* lse, void* workspace, size_t bytes, void* stream) {
    if (int rc = check_config(c)) return rc;
    if (!q || !y || (c->P > 0 && (!kp || !vp)) || (c->L > 0 && (!k || !v)))
        return report(LOLA_ERR_INVALID_ARG, "null argument");
    if (misaligned(q) || misaligned(y) || (c->P > 0 && (misaligned(kp) || misaligned(vp))) ||
        (c->L > 0 && (misaligned(k) || misaligned(v))))
        return report(LOLA_ERR_INVALID_ARG, "q, k, v and y must be 16-byte aligned");
    if (((uintptr_t)len | (uintptr_t)lse) & 3)
        return report(LOLA_ERR_INVALID_ARG, "lengths and lse must be 4-byte aligned");
    const int sms = sm_count();
    lola::AttnArgs a = make_args(c, causal);
    const size_t need = lola::plan_attn(a, sms);
    if (need && (!workspace || ((uintptr_t)workspace & 255)))
        return report(LOLA_ERR_INVALID_ARG, "workspace must be a 256-byte aligned pointer");
    if (bytes < need) return report(LOLA_ERR_BUF_TOO_SMALL, "workspace has %zu bytes, needs %zu", bytes, need);
    a.q = q;
    a.y = y;
    a.lse = lse;
    a.shared.k = kp; a.shared.v = vp;
    a.own.k = k; a.own.v = v;
    a.own_len = len;
    lola::place_attn(a, workspace);
    int launches = 0;
    const cudaError_t e = lola::launch_attn(a, sms, &launches, (cudaStream_t)stream);
    if (e != cudaSuccess) return report(LOLA_ERR_CUDA, "attention kernel: %s", cudaGetErrorString(e));
    lola::count_launches(launches);
    return LOLA_OK;
}

}  // namespace

extern "C" {

int lola_attn_workspace(const lola_attn_config* cfg, size_t* bytes) {
    if (int rc = check_config(cfg)) return rc;
    if (!bytes) return report(LOLA_ERR_INVALID_ARG, "null bytes pointer");
    // (the causal limit does not enter the plan: one size serves both calls)
    lola::AttnArgs a = make_args(cfg, 0);
    const int sms = sm_count();
    *bytes = lola::plan_attn(a, sms);
    if (keys_shared(cfg)) {
        const lola_attn_config x = as_shared(*cfg);
        a = make_args(&x, 0);
        const size_t n = lola::plan_attn(a, sms);
        if (n > *bytes) *bytes = n;
    }
    return LOLA_OK;
}

int lola_cross_attention(const lola_attn_config* cfg, const void* q, const void* k, const void* v, const int* kv_len,
                         void* y, float* lse, void* workspace, size_t bytes, void* stream) {
    if (cfg && cfg->P != 0) return report(LOLA_ERR_INVALID_ARG, "P=%d: cross attention has no shared prefix", cfg->P);
    if (int rc = check_config(cfg)) return rc;
    if (!kv_len && keys_shared(cfg)) {
        const lola_attn_config x = as_shared(*cfg);
        return run(&x, 0, q, k, v, nullptr, nullptr, nullptr, y, lse, workspace, bytes, stream);
    }
    return run(cfg, 0, q, nullptr, nullptr, k, v, kv_len, y, lse, workspace, bytes, stream);
}

int lola_prefix_attention(const lola_attn_config* cfg, const void* q, const void* k_prefix, const void* v_prefix,
                          const void* k, const void* v, const int* own_len, void* y, float* lse, void* workspace,
                          size_t bytes, void* stream) {
    return run(cfg, 1, q, k_prefix, v_prefix, k, v, own_len, y, lse, workspace, bytes, stream);
}

int lola_attn_check(void* stream) {
    int word = 0;
    const cudaError_t e = lola::attn_error_word(&word, (cudaStream_t)stream);
    if (e != cudaSuccess) return report(LOLA_ERR_CUDA, "reading the attention error word: %s", cudaGetErrorString(e));
    if (word)
        return report(LOLA_ERR_TIMEOUT, "a bounded device-side wait of an attention call gave up since the last check; "
                      "the results of the calls since then are not valid");
    return LOLA_OK;
}

}  // extern "C"
