// Norms at the boundaries of a transformer block, fused with modulation, gate
// and residual sum, and their gradients (formulas in bsa.h).
//
// Forward: one pass.  A row's channels live in registers (16 per thread), so
// x and y are read once and x_out and h written once; the kernel is bound by
// HBM.  Rows of at most 512 channels take one warp each, longer rows one CTA
// each.  Mean and variance are two register passes in fp32 (the variance from
// the centred values, so a large mean costs no digits).
//
// Backward: a CTA walks a contiguous range of rows and keeps the column sums
// of the group it is in (A = sum dh * xhat, S = sum dh, T = sum g * yhat) in
// registers.  With the group's parameters constant over the group, every
// parameter gradient follows from the three:
//   dshift = S, dscale = weight A + bias S, dgate = post_weight T,
//   dweight = sum_f (1 + scale_f) A_f, dbias = sum_f (1 + scale_f) S_f,
//   dpost_weight = sum_f gate_f T_f.
// A group that lies inside one CTA's range is written at once; the pieces of
// a group that spans CTAs, and the CTAs' weight sums, go to the workspace and
// a second kernel adds them in CTA order, so the result is the same every
// time.
#include <algorithm>

#include <cuda_bf16.h>

#include "bsa_internal.cuh"

namespace bsa {
namespace {

constexpr int kCols = 16;            // channels a thread holds

template <int VEC>
__device__ __forceinline__ void load_cols(const __nv_bfloat16* p, float* v) {
    if constexpr (VEC == 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        v[0] = __bfloat162float(*p);
    }
}
template <int VEC>
__device__ __forceinline__ void load_cols(const float* p, float* v) {
    if constexpr (VEC == 8) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        v[0] = *p;
    }
}
template <int VEC>
__device__ __forceinline__ void store_cols(__nv_bfloat16* p, const float* v) {
    if constexpr (VEC == 8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&t);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        *p = __float2bfloat16_rn(v[0]);
    }
}
template <int VEC>
__device__ __forceinline__ void store_cols(float* p, const float* v) {
    if constexpr (VEC == 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *p = v[0];
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of K values over a row's threads: a warp (kWarpRow) or the whole CTA.
// Every thread gets the same bits.
template <bool kWarpRow, int K>
__device__ __forceinline__ void row_sum(float* v, float* red) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
    if constexpr (!kWarpRow) {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) red[k * 32 + warp] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = warp_sum(lane < warps ? red[k * 32 + lane] : 0.f);
        __syncthreads();
    }
}

struct NormP {
    int C;
    int64_t rows, group_rows;        // B * N; N / groups
    int norm, post;
    float eps, res_scale, inv_c;
    const float *gate, *scale, *shift, *weight, *bias, *post_weight;
};

// In-register normalisation of a row; columns past C hold 0 before and
// garbage-free 0 after.  Returns 1 / deviation.
template <int VEC, bool kWarpRow>
__device__ __forceinline__ float normalise(float* v, int kind, const NormP& p, int stride, int first, float* red) {
    float mean = 0.f;
    if (kind == BSA_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kCols; ++i) s += v[i];
        row_sum<kWarpRow, 1>(&s, red);
        mean = s * p.inv_c;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < kCols / VEC; ++k) {
        const bool in = (first + k * stride) * VEC < p.C;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float& x = v[k * VEC + e];
            x = in ? x - mean : 0.f;
            q += x * x;
        }
    }
    row_sum<kWarpRow, 1>(&q, red);
    const float r = rsqrtf(q * p.inv_c + p.eps);
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] *= r;
    return r;
}

template <typename TX, int VEC, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 128 : 1024)
k_norm(const NormP p, const TX* x, const __nv_bfloat16* y, TX* x_out, __nv_bfloat16* h) {
    __shared__ float red[32];
    const int64_t row = kWarpRow ? (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32 : (int64_t)blockIdx.x;
    if (kWarpRow && row >= p.rows) return;
    const int first = kWarpRow ? threadIdx.x % 32 : threadIdx.x, stride = kWarpRow ? 32 : blockDim.x;
    const int64_t base = row * p.C, gbase = row / p.group_rows * p.C;
    float v[kCols];
    float t[VEC];
#pragma unroll
    for (int k = 0; k < kCols / VEC; ++k) {
        const int c = (first + k * stride) * VEC;
        if (c < p.C) {
            load_cols<VEC>(x + base + c, v + k * VEC);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[k * VEC + e] = 0.f;
        }
    }
    if (y) {
        float u[kCols];
#pragma unroll
        for (int k = 0; k < kCols / VEC; ++k) {
            const int c = (first + k * stride) * VEC;
            if (c < p.C) {
                load_cols<VEC>(y + base + c, u + k * VEC);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) u[k * VEC + e] = 0.f;
            }
        }
        if (p.post != BSA_NORM_NONE) normalise<VEC, kWarpRow>(u, p.post, p, stride, first, red);
#pragma unroll
        for (int k = 0; k < kCols / VEC; ++k) {
            const int c = (first + k * stride) * VEC;
            if (c < p.C) {
                float* uk = u + k * VEC;
                if (p.post_weight) {
                    load_cols<VEC>(p.post_weight + c, t);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) uk[e] *= t[e];
                }
                if (p.gate) {
                    load_cols<VEC>(p.gate + gbase + c, t);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) uk[e] *= t[e];
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[k * VEC + e] = p.res_scale * v[k * VEC + e] + uk[e];
                store_cols<VEC>(x_out + base + c, v + k * VEC);
            }
        }
    }
    if (p.norm == BSA_NORM_NONE) return;
    normalise<VEC, kWarpRow>(v, p.norm, p, stride, first, red);
#pragma unroll
    for (int k = 0; k < kCols / VEC; ++k) {
        const int c = (first + k * stride) * VEC;
        if (c < p.C) {
            float* vk = v + k * VEC;
            if (p.weight) {
                load_cols<VEC>(p.weight + c, t);
#pragma unroll
                for (int e = 0; e < VEC; ++e) vk[e] *= t[e];
            }
            if (p.bias) {
                load_cols<VEC>(p.bias + c, t);
#pragma unroll
                for (int e = 0; e < VEC; ++e) vk[e] += t[e];
            }
            if (p.scale) {
                load_cols<VEC>(p.scale + gbase + c, t);
#pragma unroll
                for (int e = 0; e < VEC; ++e) vk[e] *= 1.f + t[e];
            }
            if (p.shift) {
                load_cols<VEC>(p.shift + gbase + c, t);
#pragma unroll
                for (int e = 0; e < VEC; ++e) vk[e] += t[e];
            }
            store_cols<VEC>(h + base + c, vk);
        }
    }
}

// ------------------------------------------------------------------ backward
// Rows of CTA i of n: [i * rows / n, (i + 1) * rows / n).
struct Ranges {
    int64_t rows;
    int n;
    __host__ __device__ int64_t begin(int i) const { return rows / n * i + (rows % n < i ? rows % n : i); }
};

struct GradP {
    float *dgate, *dscale, *dshift, *dweight, *dbias, *dpost;
    float* piece;                    // [n][2][3][C]: a CTA's first and last pieces of split groups
    float* wsum;                     // [n][3][C]: a CTA's sums for dweight, dbias, dpost_weight
};

// kThreads: upper bound of the CTA size (the register budget follows from it)
template <typename TX, int VEC, int kThreads>
__global__ void __launch_bounds__(kThreads)
k_norm_bwd(const NormP p, const GradP g, const Ranges rg, const __nv_bfloat16* dh, const TX* dx_out,
                           const TX* x_out, const __nv_bfloat16* y, TX* dx, __nv_bfloat16* dy) {
    __shared__ float red[64];
    const int first = threadIdx.x, stride = blockDim.x;
    const int64_t r0 = rg.begin(blockIdx.x), r1 = rg.begin(blockIdx.x + 1);
    float sa[kCols] = {}, ss[kCols] = {}, st[kCols] = {};     // A, S, T of the current group
    float wa[kCols] = {}, wb[kCols] = {}, wp[kCols] = {};     // the CTA's weight sums
    float t[VEC];
    for (int64_t row = r0; row < r1; ++row) {
        const int64_t base = row * p.C, grp = row / p.group_rows, gbase = grp * p.C;
        float d[kCols];                                       // total gradient of x_out
#pragma unroll
        for (int k = 0; k < kCols / VEC; ++k) {
            const int c = (first + k * stride) * VEC;
            if (c < p.C && dx_out) {
                load_cols<VEC>(dx_out + base + c, d + k * VEC);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) d[k * VEC + e] = 0.f;
            }
        }
        if (dh) {
            float xh[kCols], gr[kCols];
#pragma unroll
            for (int k = 0; k < kCols / VEC; ++k) {
                const int c = (first + k * stride) * VEC;
                if (c < p.C) {
                    load_cols<VEC>(x_out + base + c, xh + k * VEC);
                    load_cols<VEC>(dh + base + c, gr + k * VEC);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) xh[k * VEC + e] = gr[k * VEC + e] = 0.f;
                }
            }
            const float r = normalise<VEC, false>(xh, p.norm, p, stride, first, red);
            float two[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kCols / VEC; ++k) {
                const int c = (first + k * stride) * VEC;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    sa[k * VEC + e] += gr[k * VEC + e] * xh[k * VEC + e];
                    ss[k * VEC + e] += gr[k * VEC + e];
                }
                if (c < p.C) {
                    if (p.weight) {
                        load_cols<VEC>(p.weight + c, t);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) gr[k * VEC + e] *= t[e];
                    }
                    if (p.scale) {
                        load_cols<VEC>(p.scale + gbase + c, t);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) gr[k * VEC + e] *= 1.f + t[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    two[0] += gr[k * VEC + e];
                    two[1] += gr[k * VEC + e] * xh[k * VEC + e];
                }
            }
            row_sum<false, 2>(two, red);
            const float m0 = p.norm == BSA_NORM_LAYER ? two[0] * p.inv_c : 0.f, m1 = two[1] * p.inv_c;
#pragma unroll
            for (int i = 0; i < kCols; ++i) d[i] += r * (gr[i] - m0 - xh[i] * m1);
        }
        if (y) {
            float yh[kCols], gy[kCols];
#pragma unroll
            for (int k = 0; k < kCols / VEC; ++k) {
                const int c = (first + k * stride) * VEC;
                if (c < p.C) {
                    load_cols<VEC>(y + base + c, yh + k * VEC);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) yh[k * VEC + e] = 0.f;
                }
            }
            float ry = 1.f;
            if (p.post != BSA_NORM_NONE) ry = normalise<VEC, false>(yh, p.post, p, stride, first, red);
            float two[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kCols / VEC; ++k) {
                const int c = (first + k * stride) * VEC;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int i = k * VEC + e;
                    gy[i] = c < p.C ? d[i] : 0.f;
                    st[i] += gy[i] * yh[i];
                }
                if (c < p.C) {
                    if (p.gate) {
                        load_cols<VEC>(p.gate + gbase + c, t);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) gy[k * VEC + e] *= t[e];
                    }
                    if (p.post_weight) {
                        load_cols<VEC>(p.post_weight + c, t);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) gy[k * VEC + e] *= t[e];
                    }
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    two[0] += gy[k * VEC + e];
                    two[1] += gy[k * VEC + e] * yh[k * VEC + e];
                }
            }
            if (p.post != BSA_NORM_NONE) {
                row_sum<false, 2>(two, red);
                const float m0 = p.post == BSA_NORM_LAYER ? two[0] * p.inv_c : 0.f, m1 = two[1] * p.inv_c;
#pragma unroll
                for (int i = 0; i < kCols; ++i) gy[i] = ry * (gy[i] - m0 - yh[i] * m1);
            }
#pragma unroll
            for (int k = 0; k < kCols / VEC; ++k) {
                const int c = (first + k * stride) * VEC;
                if (c < p.C) store_cols<VEC>(dy + base + c, gy + k * VEC);
            }
        }
        const float rs = y ? p.res_scale : 1.f;
#pragma unroll
        for (int k = 0; k < kCols / VEC; ++k) {
            const int c = (first + k * stride) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) d[k * VEC + e] *= rs;
            if (c < p.C) store_cols<VEC>(dx + base + c, d + k * VEC);
        }
        // the group ends here, or this CTA's share of it does
        const bool group_end = (row + 1) % p.group_rows == 0;
        if (!group_end && row + 1 < r1) continue;
        const bool whole = group_end && grp * p.group_rows >= r0;
        const int slot = grp * p.group_rows < r0 ? 0 : 1;     // a piece that began earlier, or one that goes on
#pragma unroll
        for (int k = 0; k < kCols / VEC; ++k) {
            const int c = (first + k * stride) * VEC;
            if (c >= p.C) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int i = k * VEC + e, ch = c + e;
                const float sc = p.scale ? 1.f + p.scale[gbase + ch] : 1.f;
                wa[i] += sc * sa[i];
                wb[i] += sc * ss[i];
                wp[i] += p.gate ? p.gate[gbase + ch] * st[i] : st[i];
                if (whole) {
                    if (g.dscale)
                        g.dscale[gbase + ch] = (p.weight ? p.weight[ch] : 1.f) * sa[i] + (p.bias ? p.bias[ch] : 0.f) * ss[i];
                    if (g.dshift) g.dshift[gbase + ch] = ss[i];
                    if (g.dgate) g.dgate[gbase + ch] = (p.post_weight ? p.post_weight[ch] : 1.f) * st[i];
                } else {
                    float* o = g.piece + ((int64_t)blockIdx.x * 2 + slot) * 3 * p.C + ch;
                    o[0] = sa[i];
                    o[p.C] = ss[i];
                    o[2 * p.C] = st[i];
                }
                sa[i] = ss[i] = st[i] = 0.f;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kCols / VEC; ++k) {
        const int c = (first + k * stride) * VEC;
        if (c >= p.C) continue;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float* o = g.wsum + (int64_t)blockIdx.x * 3 * p.C + c + e;
            o[0] = wa[k * VEC + e];
            o[p.C] = wb[k * VEC + e];
            o[2 * p.C] = wp[k * VEC + e];
        }
    }
}

// Adds the pieces.  blockIdx.y = 0: the weight sums of all CTAs; y > 0: the
// group that holds the first row of CTA y, if it began in an earlier CTA and
// CTA y - 1 is not inside it as well (each split group once).
__global__ void k_norm_bwd_join(const NormP p, const GradP g, const Ranges rg) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= p.C) return;
    if (blockIdx.y == 0) {
        float a = 0.f, b = 0.f, w = 0.f;
        for (int i = 0; i < rg.n; ++i) {
            const float* s = g.wsum + (int64_t)i * 3 * p.C + c;
            a += s[0];
            b += s[p.C];
            w += s[2 * p.C];
        }
        if (g.dweight) g.dweight[c] = a;
        if (g.dbias) g.dbias[c] = b;
        if (g.dpost) g.dpost[c] = w;
        return;
    }
    const int cta = blockIdx.y;
    const int64_t grp = rg.begin(cta) / p.group_rows, lo = grp * p.group_rows, hi = lo + p.group_rows;
    if (lo >= rg.begin(cta) || lo < rg.begin(cta - 1)) return;     // not split here, or an earlier CTA's to join
    float a = 0.f, s = 0.f, t = 0.f;
    for (int i = cta - 1; i < rg.n && rg.begin(i) < hi; ++i) {
        const int slot = lo < rg.begin(i) ? 0 : 1;
        const float* q = g.piece + ((int64_t)i * 2 + slot) * 3 * p.C + c;
        a += q[0];
        s += q[p.C];
        t += q[2 * p.C];
    }
    const int64_t gc = grp * p.C + c;
    if (g.dscale) g.dscale[gc] = (p.weight ? p.weight[c] : 1.f) * a + (p.bias ? p.bias[c] : 0.f) * s;
    if (g.dshift) g.dshift[gc] = s;
    if (g.dgate) g.dgate[gc] = (p.post_weight ? p.post_weight[c] : 1.f) * t;
}

NormP norm_params(const bsa_plan& p, const bsa_norm_args& a) {
    NormP n;
    n.C = a.C;
    n.rows = (int64_t)p.B * p.N;
    n.group_rows = p.N / a.groups;
    n.norm = a.norm;
    n.post = a.post_norm;
    n.eps = a.eps;
    n.res_scale = a.res_scale;
    n.inv_c = 1.f / (float)a.C;
    n.gate = a.gate; n.scale = a.scale; n.shift = a.shift;
    n.weight = a.weight; n.bias = a.bias; n.post_weight = a.post_weight;
    return n;
}

// Threads that hold a row of C channels, 16 each.
int row_threads(int C) { return ((C + kCols - 1) / kCols + 31) / 32 * 32; }

int bwd_ctas(const bsa_plan& p) { return (int)std::min<int64_t>((int64_t)p.num_sms * 2, (int64_t)p.B * p.N); }

template <typename TX, int VEC>
cudaError_t fwd(const NormP& n, const void* x, const void* y, void* x_out, void* h, cudaStream_t s) {
    const TX* xi = (const TX*)x;
    const __nv_bfloat16* yi = (const __nv_bfloat16*)y;
    if (n.C <= 32 * kCols) {
        constexpr int kWarps = 4;
        k_norm<TX, VEC, true><<<(unsigned)((n.rows + kWarps - 1) / kWarps), 32 * kWarps, 0, s>>>(
            n, xi, yi, (TX*)x_out, (__nv_bfloat16*)h);
    } else {
        k_norm<TX, VEC, false><<<(unsigned)n.rows, row_threads(n.C), 0, s>>>(n, xi, yi, (TX*)x_out, (__nv_bfloat16*)h);
    }
    return cudaGetLastError();
}

template <typename TX, int VEC>
cudaError_t bwd(const NormP& n, const GradP& g, const Ranges& rg, const void* dh, const void* dx_out, const void* x_out,
                const void* y, void* dx, void* dy, cudaStream_t s) {
    const int threads = row_threads(n.C);
    auto kern = threads <= 384 ? k_norm_bwd<TX, VEC, 384> : k_norm_bwd<TX, VEC, 1024>;
    kern<<<rg.n, threads, 0, s>>>(n, g, rg, (const __nv_bfloat16*)dh, (const TX*)dx_out, (const TX*)x_out,
                                  (const __nv_bfloat16*)y, (TX*)dx, (__nv_bfloat16*)dy);
    if (cudaError_t e = cudaGetLastError()) return e;
    k_norm_bwd_join<<<dim3((n.C + 127) / 128, rg.n), 128, 0, s>>>(n, g, rg);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const bsa_plan& p, const bsa_norm_args& a, const void* x, const void* y, void* x_out, void* h,
                        cudaStream_t s) {
    const NormP n = norm_params(p, a);
    const bool wide = a.C % 8 == 0;
    if (a.dtype == BSA_BF16)
        return wide ? fwd<__nv_bfloat16, 8>(n, x, y, x_out, h, s) : fwd<__nv_bfloat16, 1>(n, x, y, x_out, h, s);
    return wide ? fwd<float, 8>(n, x, y, x_out, h, s) : fwd<float, 1>(n, x, y, x_out, h, s);
}

size_t norm_bwd_ws_bytes(const bsa_plan& p, const bsa_norm_args& a) {
    return align_up((size_t)bwd_ctas(p) * 9 * a.C * sizeof(float));
}

cudaError_t launch_norm_bwd(const bsa_plan& p, const bsa_norm_args& a, const NormGrads& out, const void* dh,
                            const void* dx_out, const void* x_out, const void* y, void* dx, void* dy, void* ws,
                            cudaStream_t s) {
    const NormP n = norm_params(p, a);
    const Ranges rg{n.rows, bwd_ctas(p)};
    GradP g;
    g.dgate = out.dgate; g.dscale = out.dscale; g.dshift = out.dshift;
    g.dweight = out.dweight; g.dbias = out.dbias; g.dpost = out.dpost_weight;
    g.piece = (float*)ws;
    g.wsum = g.piece + (size_t)rg.n * 6 * a.C;
    const bool wide = a.C % 8 == 0;
    if (a.dtype == BSA_BF16)
        return wide ? bwd<__nv_bfloat16, 8>(n, g, rg, dh, dx_out, x_out, y, dx, dy, s)
                    : bwd<__nv_bfloat16, 1>(n, g, rg, dh, dx_out, x_out, y, dx, dy, s);
    return wide ? bwd<float, 8>(n, g, rg, dh, dx_out, x_out, y, dx, dy, s)
                : bwd<float, 1>(n, g, rg, dh, dx_out, x_out, y, dx, dy, s);
}

}  // namespace bsa
