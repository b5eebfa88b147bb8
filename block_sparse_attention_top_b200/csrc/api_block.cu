// C ABI of the block operators: argument validation and launches of the cross
// attention and of the norms (kernels in cross_*.cu and norm.cu).
#include "bsa_internal.cuh"

using namespace bsa;

namespace {

bool misaligned(const void* p, size_t a) { return ((uintptr_t)p) % a != 0; }

// The plan's device is the current one.
bool on_device(const bsa_plan* p) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == p->device;
}

int check_workspace(const void* ws, size_t bytes, size_t need) {
    if (need == 0) return BSA_OK;
    return !ws || bytes < need || misaligned(ws, kAlign) ? BSA_EWORKSPACE : BSA_OK;
}

bool overlaps_null(int64_t extent, const void* p) { return extent > 0 && !p; }

constexpr int64_t kMaxStates = 1ll << 30;
constexpr int64_t kMaxStride = 1ll << 39;     // in elements: a tensor map's strides are below 2^40 bytes

// Extents [B, rows, heads] with their strides: dense defaults filled in, limits checked.
int fill_strides(const int64_t* in, int64_t* out, int64_t B, int64_t rows, int64_t heads, int d) {
    const int64_t dense[3] = {rows * heads * d, heads * d, d}, ext[3] = {B, rows, heads};
    for (int i = 0; i < 3; ++i) {
        out[i] = in && ext[i] > 1 ? in[i] : dense[i];
        if (ext[i] <= 1) out[i] = d;                       // never multiplied by a non-zero index
        if (ext[i] > 1 && out[i] <= 0) return BSA_EUNSUPPORTED;
        if (out[i] % 8 != 0 || out[i] >= kMaxStride) return BSA_EUNSUPPORTED;
    }
    return BSA_OK;
}

int cross_args(const bsa_plan* p, const void* q, const void* k, const void* v, int64_t M, int Hkv,
               const int64_t* strides, const int32_t* kv_len, const uint8_t* key_mask, CrossArgs* a) {
    if (!p || !q || M < 0 || Hkv < 1 || overlaps_null(M, k) || overlaps_null(M, v)) return BSA_EINVAL;
    if (p->H % Hkv != 0) return BSA_EINVAL;
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(kv_len, 4)) return BSA_EINVAL;
    if (M > kMaxStates || (int64_t)p->B * p->H * p->N > INT32_MAX || (int64_t)p->B * M * Hkv > INT32_MAX)
        return BSA_EUNSUPPORTED;
    a->q = q; a->k = k; a->v = v; a->M = M; a->Hkv = Hkv;
    a->kv_len = kv_len; a->key_mask = key_mask;
    if (int rc = fill_strides(strides, a->st, p->B, p->N, p->H, p->d)) return rc;
    if (int rc = fill_strides(strides ? strides + 3 : nullptr, a->st + 3, p->B, M, Hkv, p->d)) return rc;
    if (int rc = fill_strides(strides ? strides + 6 : nullptr, a->st + 6, p->B, M, Hkv, p->d)) return rc;
    return BSA_OK;
}

bool norm_kind(int k) { return k == BSA_NORM_NONE || k == BSA_NORM_LAYER || k == BSA_NORM_RMS; }

constexpr int kMaxChannels = 16384;

int norm_args(const bsa_plan* p, const bsa_norm_args* a) {
    if (!p || !a || a->C < 1 || a->groups < 1 || p->N % a->groups != 0) return BSA_EINVAL;
    if (a->dtype != BSA_BF16 && a->dtype != BSA_F32) return BSA_EINVAL;
    if (!norm_kind(a->norm) || !norm_kind(a->post_norm) || !(a->eps > 0.f)) return BSA_EINVAL;
    const void* par[6] = {a->gate, a->scale, a->shift, a->weight, a->bias, a->post_weight};
    for (const void* q : par)
        if (misaligned(q, 16)) return BSA_EINVAL;
    if (a->C > kMaxChannels || (int64_t)p->B * p->N > INT32_MAX) return BSA_EUNSUPPORTED;
    return BSA_OK;
}

// The gradients of the parameters leave in 16-byte stores where the width allows.
bool misaligned(const NormGrads& g) {
    const void* out[6] = {g.dgate, g.dscale, g.dshift, g.dweight, g.dbias, g.dpost_weight};
    for (const void* q : out)
        if (misaligned(q, 16)) return true;
    return false;
}

int status(cudaError_t e) { return e == cudaSuccess ? BSA_OK : BSA_ECUDA; }

}  // namespace

extern "C" {

size_t bsa_cross_attn_workspace_size(const bsa_plan* p, int64_t M, int Hkv, int backward) {
    if (!p || M < 0 || M > kMaxStates || Hkv < 1 || p->H % Hkv != 0) return 0;
    return cross_ws_bytes(*p, M, Hkv, backward != 0);
}

int bsa_cross_attn(const bsa_plan* p, const void* q, const void* k, const void* v, int64_t M, int Hkv,
                   const int64_t* strides, const int32_t* kv_len, const uint8_t* key_mask, void* o, float* lse,
                   void* ws, size_t ws_bytes, void* stream) {
    CrossArgs a;
    if (int rc = cross_args(p, q, k, v, M, Hkv, strides, kv_len, key_mask, &a)) return rc;
    if (!o || misaligned(o, 16) || misaligned(lse, 4) || !on_device(p)) return BSA_EINVAL;
    if (int rc = check_workspace(ws, ws_bytes, cross_ws_bytes(*p, M, Hkv, false))) return rc;
    return status(launch_cross(*p, a, o, lse, (cudaStream_t)stream));
}

int bsa_cross_attn_bwd(const bsa_plan* p, const void* q, const void* k, const void* v, int64_t M, int Hkv,
                       const int64_t* strides, const int32_t* kv_len, const uint8_t* key_mask, const void* o,
                       const float* lse, const void* d_o, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                       void* stream) {
    CrossArgs a;
    if (int rc = cross_args(p, q, k, v, M, Hkv, strides, kv_len, key_mask, &a)) return rc;
    if (!o || !lse || !d_o || !dq || overlaps_null(M, dk) || overlaps_null(M, dv)) return BSA_EINVAL;
    if (misaligned(o, 16) || misaligned(lse, 4) || misaligned(d_o, 16) || misaligned(dq, 16) || misaligned(dk, 16) ||
        misaligned(dv, 16) || !on_device(p))
        return BSA_EINVAL;
    if (int rc = check_workspace(ws, ws_bytes, cross_ws_bytes(*p, M, Hkv, true))) return rc;
    return status(launch_cross_bwd(*p, a, o, lse, d_o, dq, dk, dv, ws, (cudaStream_t)stream));
}

int bsa_norm_modulate(const bsa_plan* p, const bsa_norm_args* a, const void* x, void* h, void* stream) {
    if (int rc = norm_args(p, a)) return rc;
    if (!x || !h || a->norm == BSA_NORM_NONE || a->post_norm != BSA_NORM_NONE) return BSA_EINVAL;
    if (misaligned(x, 16) || misaligned(h, 16) || !on_device(p)) return BSA_EINVAL;
    return status(launch_norm(*p, *a, x, nullptr, nullptr, h, (cudaStream_t)stream));
}

int bsa_residual_norm(const bsa_plan* p, const bsa_norm_args* a, const void* x, const void* y, void* x_out, void* h,
                      void* stream) {
    if (int rc = norm_args(p, a)) return rc;
    if (!x || !y || !x_out || (h != nullptr) != (a->norm != BSA_NORM_NONE)) return BSA_EINVAL;
    if (misaligned(x, 16) || misaligned(y, 16) || misaligned(x_out, 16) || misaligned(h, 16) || !on_device(p))
        return BSA_EINVAL;
    return status(launch_norm(*p, *a, x, y, x_out, h, (cudaStream_t)stream));
}

size_t bsa_norm_bwd_workspace_size(const bsa_plan* p, const bsa_norm_args* a) {
    return norm_args(p, a) ? 0 : norm_bwd_ws_bytes(*p, *a);
}

int bsa_norm_modulate_bwd(const bsa_plan* p, const bsa_norm_args* a, const void* dh, const void* x, void* dx,
                          float* dscale, float* dshift, float* dweight, float* dbias, void* ws, size_t ws_bytes,
                          void* stream) {
    if (int rc = norm_args(p, a)) return rc;
    if (!dh || !x || !dx || a->norm == BSA_NORM_NONE || a->post_norm != BSA_NORM_NONE) return BSA_EINVAL;
    const NormGrads g{nullptr, dscale, dshift, dweight, dbias, nullptr};
    if (misaligned(dh, 16) || misaligned(x, 16) || misaligned(dx, 16) || misaligned(g) || !on_device(p))
        return BSA_EINVAL;
    if (int rc = check_workspace(ws, ws_bytes, norm_bwd_ws_bytes(*p, *a))) return rc;
    return status(launch_norm_bwd(*p, *a, g, dh, nullptr, x, nullptr, dx, nullptr, ws, (cudaStream_t)stream));
}

int bsa_residual_norm_bwd(const bsa_plan* p, const bsa_norm_args* a, const void* dh, const void* dx_out,
                          const void* x_out, const void* y, void* dx, void* dy, float* dgate, float* dscale,
                          float* dshift, float* dweight, float* dbias, float* dpost_weight, void* ws, size_t ws_bytes,
                          void* stream) {
    if (int rc = norm_args(p, a)) return rc;
    if (!y || !dx || !dy || (!dh && !dx_out) || (dh != nullptr) != (a->norm != BSA_NORM_NONE) || (dh && !x_out))
        return BSA_EINVAL;
    const NormGrads g{dgate, dscale, dshift, dweight, dbias, dpost_weight};
    if (misaligned(dh, 16) || misaligned(dx_out, 16) || misaligned(x_out, 16) || misaligned(y, 16) ||
        misaligned(dx, 16) || misaligned(dy, 16) || misaligned(g) || !on_device(p))
        return BSA_EINVAL;
    if (int rc = check_workspace(ws, ws_bytes, norm_bwd_ws_bytes(*p, *a))) return rc;
    return status(launch_norm_bwd(*p, *a, g, dh, dx_out, x_out, y, dx, dy, ws, (cudaStream_t)stream));
}

}  // extern "C"
