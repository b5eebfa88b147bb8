// Cross attention to an encoder's states and its gradient (formulas in bsa.h),
// one warp per query row or key, fp32 throughout.
#include <cuda_bf16.h>

#include "cross_common.cuh"

namespace bsa {
namespace {

struct CrossP {
    const __nv_bfloat16 *q, *k, *v;
    int64_t st[9];
    const int32_t* kv_len;
    const uint8_t* key_mask;
    int64_t N, M;
    int B, H, Hkv;
    float scale;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ int64_t key_count(const CrossP& p, int b) {
    if (!p.kv_len) return p.M;
    const int64_t n = p.kv_len[b];
    return n < 0 ? 0 : (n > p.M ? p.M : n);
}
__device__ __forceinline__ bool key_on(const CrossP& p, int b, int64_t j) {
    return !p.key_mask || p.key_mask[(int64_t)b * p.M + j];
}
template <int C>
__device__ __forceinline__ void load_row(const __nv_bfloat16* r, int lane, float* v) {
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = __bfloat162float(r[lane * C + c]);
}
template <int C>
__device__ __forceinline__ float dot(const float* a, const float* b) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) s += a[c] * b[c];
    return warp_sum(s);
}
template <int C>
__device__ __forceinline__ void store_row(__nv_bfloat16* r, int lane, const float* v, float f) {
#pragma unroll
    for (int c = 0; c < C; ++c) r[lane * C + c] = __float2bfloat16_rn(v[c] * f);
}

template <int D>
__global__ void k_cross_rows(const CrossP p, __nv_bfloat16* o, float* lse) {
    constexpr int C = D / 32;
    const int lane = threadIdx.x % 32;
    const int64_t r = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;     // (b, n, h)
    if (r >= p.B * p.N * p.H) return;
    const int h = (int)(r % p.H), hk = h / (p.H / p.Hkv);
    const int64_t n = r / p.H % p.N;
    const int b = (int)(r / p.H / p.N);
    float q[C], acc[C] = {}, t[C];
    load_row<C>(p.q + b * p.st[0] + n * p.st[1] + h * p.st[2], lane, q);
    const __nv_bfloat16* k = p.k + b * p.st[3] + hk * p.st[5];
    const __nv_bfloat16* v = p.v + b * p.st[6] + hk * p.st[8];
    float m = -INFINITY, l = 0.f;
    const int64_t cnt = key_count(p, b);
    for (int64_t j = 0; j < cnt; ++j) {
        if (!key_on(p, b, j)) continue;
        load_row<C>(k + j * p.st[4], lane, t);
        const float s = dot<C>(q, t) * p.scale;
        const float mn = fmaxf(m, s), a = m == mn ? 1.f : expf(m - mn), w = s == mn ? 1.f : expf(s - mn);
        load_row<C>(v + j * p.st[7], lane, t);
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = acc[c] * a + w * t[c];
        l = l * a + w;
        m = mn;
    }
    store_row<C>(o + r * D, lane, acc, l > 0.f ? 1.f / l : 0.f);
    if (lse && lane == 0) lse[((int64_t)b * p.H + h) * p.N + n] = l > 0.f ? m + logf(l) : -INFINITY;
}

// dQ of one row; D = rowsum(dO * O) is left in `dsum` for the key side.
template <int D>
__global__ void k_cross_dq(const CrossP p, const __nv_bfloat16* o, const float* lse, const __nv_bfloat16* d_o,
                           __nv_bfloat16* dq, float* dsum) {
    constexpr int C = D / 32;
    const int lane = threadIdx.x % 32;
    const int64_t r = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    if (r >= p.B * p.N * p.H) return;
    const int h = (int)(r % p.H), hk = h / (p.H / p.Hkv);
    const int64_t n = r / p.H % p.N;
    const int b = (int)(r / p.H / p.N);
    float q[C], g[C], acc[C] = {}, t[C];
    load_row<C>(p.q + b * p.st[0] + n * p.st[1] + h * p.st[2], lane, q);
    load_row<C>(d_o + r * D, lane, g);
    load_row<C>(o + r * D, lane, t);
    const float dd = dot<C>(g, t);
    const int64_t li = ((int64_t)b * p.H + h) * p.N + n;
    if (lane == 0) dsum[li] = dd;
    const float L = lse[li];
    const __nv_bfloat16* k = p.k + b * p.st[3] + hk * p.st[5];
    const __nv_bfloat16* v = p.v + b * p.st[6] + hk * p.st[8];
    const int64_t cnt = key_count(p, b);
    for (int64_t j = 0; j < cnt; ++j) {
        if (!key_on(p, b, j)) continue;
        load_row<C>(v + j * p.st[7], lane, t);
        const float dp = dot<C>(g, t);
        load_row<C>(k + j * p.st[4], lane, t);
        const float w = expf(dot<C>(q, t) * p.scale - L) * (dp - dd);
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] += w * t[c];
    }
    store_row<C>(dq + r * D, lane, acc, p.scale);
}

template <int D>
__global__ void k_cross_dkv(const CrossP p, const float* lse, const __nv_bfloat16* d_o, const float* dsum,
                            __nv_bfloat16* dk, __nv_bfloat16* dv) {
    constexpr int C = D / 32;
    const int lane = threadIdx.x % 32, G = p.H / p.Hkv;
    const int64_t r = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;     // (b, j, hk)
    if (r >= p.B * p.M * p.Hkv) return;
    const int hk = (int)(r % p.Hkv);
    const int64_t j = r / p.Hkv % p.M;
    const int b = (int)(r / p.Hkv / p.M);
    float kk[C], vv[C], ak[C] = {}, av[C] = {}, q[C], g[C];
    if (j < key_count(p, b) && key_on(p, b, j)) {
        load_row<C>(p.k + b * p.st[3] + j * p.st[4] + hk * p.st[5], lane, kk);
        load_row<C>(p.v + b * p.st[6] + j * p.st[7] + hk * p.st[8], lane, vv);
        for (int h = hk * G; h < (hk + 1) * G; ++h)
            for (int64_t n = 0; n < p.N; ++n) {
                load_row<C>(p.q + b * p.st[0] + n * p.st[1] + h * p.st[2], lane, q);
                load_row<C>(d_o + ((b * p.N + n) * p.H + h) * D, lane, g);
                const int64_t li = ((int64_t)b * p.H + h) * p.N + n;
                const float w = expf(dot<C>(q, kk) * p.scale - lse[li]);
                const float ds = w * (dot<C>(g, vv) - dsum[li]);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    av[c] += w * g[c];
                    ak[c] += ds * q[c];
                }
            }
    }
    store_row<C>(dk + r * D, lane, ak, p.scale);
    store_row<C>(dv + r * D, lane, av, 1.f);
}

CrossP cross_params(const bsa_plan& p, const CrossArgs& a) {
    CrossP c;
    c.q = (const __nv_bfloat16*)a.q; c.k = (const __nv_bfloat16*)a.k; c.v = (const __nv_bfloat16*)a.v;
    for (int i = 0; i < 9; ++i) c.st[i] = a.st[i];
    c.kv_len = a.kv_len; c.key_mask = a.key_mask;
    c.N = p.N; c.M = a.M; c.B = p.B; c.H = p.H; c.Hkv = a.Hkv;
    c.scale = 1.f / sqrtf((float)p.d);
    return c;
}

constexpr int kRowWarps = 8;
unsigned row_grid(int64_t rows) { return (unsigned)((rows + kRowWarps - 1) / kRowWarps); }

}  // namespace

size_t cross_ws_bytes(const bsa_plan& p, int64_t M, int Hkv, bool backward) {
    return backward ? cross_bwd_ws_bytes(p, M, Hkv) : 0;
}

cudaError_t launch_cross(const bsa_plan& p, const CrossArgs& a, void* o, float* lse, void*, cudaStream_t s) {
    if (a.M > 0 && p.N * (p.H / a.Hkv) <= 64 && (int64_t)p.B * a.Hkv <= 65535) return launch_cross_few(p, a, o, lse, s);
    if (a.M > 0) return launch_cross_fwd_tc(p, a, o, lse, s);
    const CrossP c = cross_params(p, a);
    auto kern = p.d == 128 ? k_cross_rows<128> : k_cross_rows<64>;
    kern<<<row_grid(p.B * p.N * p.H), 32 * kRowWarps, 0, s>>>(c, (__nv_bfloat16*)o, lse);
    return cudaGetLastError();
}

cudaError_t launch_cross_bwd(const bsa_plan& p, const CrossArgs& a, const void* o, const float* lse, const void* d_o,
                             void* dq, void* dk, void* dv, void* ws, cudaStream_t s) {
    if (a.M > 0) return launch_cross_bwd_tc(p, a, o, lse, d_o, dq, dk, dv, ws, s);
    const CrossP c = cross_params(p, a);
    const __nv_bfloat16* g = (const __nv_bfloat16*)d_o;
    auto kq = p.d == 128 ? k_cross_dq<128> : k_cross_dq<64>;
    kq<<<row_grid(p.B * p.N * p.H), 32 * kRowWarps, 0, s>>>(c, (const __nv_bfloat16*)o, lse, g, (__nv_bfloat16*)dq,
                                                           (float*)ws);
    if (cudaError_t e = cudaGetLastError()) return e;
    if (a.M == 0) return cudaSuccess;
    auto kk = p.d == 128 ? k_cross_dkv<128> : k_cross_dkv<64>;
    kk<<<row_grid(p.B * a.M * a.Hkv), 32 * kRowWarps, 0, s>>>(c, lse, g, (const float*)ws, (__nv_bfloat16*)dk,
                                                             (__nv_bfloat16*)dv);
    return cudaGetLastError();
}

}  // namespace bsa
