// Norms at the boundaries of a transformer block, fused with modulation, gate
// and residual sum, and their gradients (formulas in bsa.h).
//
// Forward: one pass.  A row's channels live in registers (16 per thread), so
// x and y are read once and x_out and h written once; the kernel is bound by
// HBM.  Rows of at most 512 channels take one warp each.  Longer rows take a
// CTA each; the CTAs stay and walk the rows, and every thread fetches its own
// 16-byte pieces of the next rows by cp.async into a ring in shared memory
// that only it reads, so loads stay in flight over the row's reductions
// without a barrier.  Mean and variance are two register passes in fp32 (the
// variance from the centred values, so a large mean costs no digits).
//
// Backward: a CTA walks a contiguous range of rows (same ring) and keeps the
// column sums of the group it is in (A = sum dh * xhat, S = sum dh,
// T = sum g * yhat) in registers.  With the group's parameters constant over
// the group, every parameter gradient follows from the three:
//   dshift = S, dscale = weight A + bias S, dgate = post_weight T,
//   dweight = sum_f (1 + scale_f) A_f, dbias = sum_f (1 + scale_f) S_f,
//   dpost_weight = sum_f gate_f T_f.
// A group that lies inside one CTA's range is written at once; the pieces of
// a group that spans CTAs, and the CTAs' weight sums, go to the workspace and
// a second kernel adds them in a fixed order, so the result is the same every
// time.  Where every token is a group of its own, the registers hold the
// weight sums instead and each row writes its group's gradients.
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

// Sums of K values over a row's threads: a warp (kWarpRow) or the whole CTA, through red[K][32].  Every thread gets
// the same bits.  One barrier: a caller's next sum uses another `red`, or comes two barriers later.
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
    }
}

struct NormP {
    int C;
    int64_t rows, group_rows;        // B * N; N / groups
    int norm, post;
    float eps, res_scale, c, inv_c;      // c = C
    const float *gate, *scale, *shift, *weight, *bias, *post_weight;
};

// A thread's channels: kCols / VEC runs of VEC, run k at (first + k * stride) * VEC.
template <int VEC>
struct Cols {
    int C, first, stride;
    __device__ __forceinline__ int at(int k) const { return (first + k * stride) * VEC; }
    __device__ __forceinline__ bool in(int k) const { return at(k) < C; }
};

template <int VEC, typename T>
__device__ __forceinline__ void load_row(const T* p, const Cols<VEC>& c, float* v) {
#pragma unroll
    for (int k = 0; k < kCols / VEC; ++k) {
        if (c.in(k)) {
            load_cols<VEC>(p + c.at(k), v + k * VEC);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[k * VEC + e] = 0.f;
        }
    }
}

__device__ __forceinline__ void fetch16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void fetch_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory"); }

// A thread's slots of one row of type T in a ring stage: 16-byte pieces, piece i at [i][thread].
template <typename T>
constexpr int row_pieces() { return kCols * (int)sizeof(T) / 16; }
template <typename T>
__device__ __forceinline__ void fetch_row(unsigned char* slot, const T* p, const Cols<8>& c) {
    constexpr int kPer = 8 * sizeof(T) / 16;
#pragma unroll
    for (int k = 0; k < kCols / 8; ++k)
        if (c.in(k))
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                fetch16((uint32_t)__cvta_generic_to_shared(slot + ((k * kPer + i) * blockDim.x + threadIdx.x) * 16),
                        reinterpret_cast<const char*>(p + c.at(k)) + 16 * i);
}
template <typename T>
__device__ __forceinline__ void slot_row(const unsigned char* slot, const Cols<8>& c, float* v) {
    constexpr int kPer = 8 * sizeof(T) / 16;
#pragma unroll
    for (int k = 0; k < kCols / 8; ++k) {
        if (c.in(k)) {
            if constexpr (sizeof(T) == 2) {
                load_cols<8>(reinterpret_cast<const __nv_bfloat16*>(slot + (k * blockDim.x + threadIdx.x) * 16), v + 8 * k);
            } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const float4 a = *reinterpret_cast<const float4*>(slot + ((k * kPer + i) * blockDim.x + threadIdx.x) * 16);
                    v[8 * k + 4 * i] = a.x;
                    v[8 * k + 4 * i + 1] = a.y;
                    v[8 * k + 4 * i + 2] = a.z;
                    v[8 * k + 4 * i + 3] = a.w;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * k + e] = 0.f;
        }
    }
}

// v -= mean of the row (layer norm); channels past C become 0.
template <int VEC>
__device__ __forceinline__ void centre(float* v, float mean, const Cols<VEC>& c) {
#pragma unroll
    for (int k = 0; k < kCols / VEC; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[k * VEC + e] = c.in(k) ? v[k * VEC + e] - mean : 0.f;
}
__device__ __forceinline__ float sum_of(const float* v) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) s += v[i];
    return s;
}
__device__ __forceinline__ float square_of(const float* v) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) s += v[i] * v[i];
    return s;
}
// v = v op p over a thread's channels
template <int VEC, typename F>
__device__ __forceinline__ void with_param(float* v, const float* p, const Cols<VEC>& c, F f) {
    if (!p) return;
#pragma unroll
    for (int k = 0; k < kCols / VEC; ++k)
        if (c.in(k)) {
            float t[VEC];
            load_cols<VEC>(p + c.at(k), t);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[k * VEC + e] = f(v[k * VEC + e], t[e]);
        }
}
template <int VEC, typename T>
__device__ __forceinline__ void store_row(T* p, const Cols<VEC>& c, const float* v) {
#pragma unroll
    for (int k = 0; k < kCols / VEC; ++k)
        if (c.in(k)) store_cols<VEC>(p + c.at(k), v + k * VEC);
}
__device__ __forceinline__ float times(float a, float b) { return a * b; }
__device__ __forceinline__ float times1(float a, float b) { return a * (1.f + b); }
__device__ __forceinline__ float plus(float a, float b) { return a + b; }

// In-register normalisation; red: [2][32].
template <int VEC, bool kWarpRow>
__device__ __forceinline__ void normalise(float* v, int kind, const NormP& p, const Cols<VEC>& c, float* red) {
    if (kind == BSA_NORM_LAYER) {
        float s = sum_of(v);
        row_sum<kWarpRow, 1>(&s, red);
        centre(v, s / p.c, c);            // a division: the mean of equal values is that value
    }
    float q = square_of(v);
    row_sum<kWarpRow, 1>(&q, red + 32);
    const float r = rsqrtf(q * p.inv_c + p.eps);
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] *= r;
}

// A group's parameters folded into three coefficients a channel: x_out = r x + g post(y), h = a xhat + b.
struct Coef {
    float g[kCols], a[kCols], b[kCols];
};
template <int VEC>
__device__ __forceinline__ void load_coef(Coef& k, const NormP& p, int64_t grp, const Cols<VEC>& c, bool has_y) {
    const int64_t gbase = grp * p.C;
    if (has_y) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) k.g[i] = 1.f;
        with_param(k.g, p.post_weight, c, times);
        if (p.gate) with_param(k.g, p.gate + gbase, c, times);
    }
    if (p.norm == BSA_NORM_NONE) return;
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
        k.a[i] = 1.f;
        k.b[i] = 0.f;
    }
    with_param(k.a, p.weight, c, times);
    with_param(k.b, p.bias, c, plus);
    if (p.scale) {
        with_param(k.a, p.scale + gbase, c, times1);
        if (p.bias) with_param(k.b, p.scale + gbase, c, times1);
    }
    if (p.shift) with_param(k.b, p.shift + gbase, c, plus);
}

// One row: v holds x, u holds y (if any).
template <typename TX, int VEC, bool kWarpRow>
__device__ __forceinline__ void norm_row(const NormP& p, int64_t row, const Cols<VEC>& c, float* v, float* u, bool has_y,
                                         const Coef& k, TX* x_out, __nv_bfloat16* h, float* red) {
    const int64_t base = row * p.C;
    if (has_y) {
        if (p.post != BSA_NORM_NONE) normalise<VEC, kWarpRow>(u, p.post, p, c, red);
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[i] = fmaf(k.g[i], u[i], p.res_scale * v[i]);
        store_row(x_out + base, c, v);
    }
    if (p.norm == BSA_NORM_NONE) return;
    normalise<VEC, kWarpRow>(v, p.norm, p, c, red + 64);
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] = fmaf(k.a[i], v[i], k.b[i]);
    store_row(h + base, c, v);
}

// A warp to a row (C <= 512).
template <typename TX, int VEC>
__global__ void __launch_bounds__(128)
k_norm_warp(const NormP p, const TX* x, const __nv_bfloat16* y, TX* x_out, __nv_bfloat16* h) {
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    if (row >= p.rows) return;
    const Cols<VEC> c{p.C, (int)threadIdx.x % 32, 32};
    float v[kCols], u[kCols];
    load_row<VEC>(x + row * p.C, c, v);
    if (y) load_row<VEC>(y + row * p.C, c, u);
    Coef k;
    load_coef(k, p, row / p.group_rows, c, y != nullptr);
    norm_row<TX, VEC, true>(p, row, c, v, u, y != nullptr, k, x_out, h, nullptr);
}

// Rows of CTA i of n: the first rows % n CTAs have one more.
struct Ranges {
    int64_t rows;
    int n;
    __host__ __device__ int64_t begin(int i) const { return rows / n * i + (rows % n < i ? rows % n : i); }
    __device__ int owner(int64_t row) const {
        const int64_t q = rows / n, big = rows % n * (q + 1);
        return (int)(row < big ? row / (q + 1) : rows % n + (row - big) / q);
    }
};

// A CTA to a row, a range of rows to a CTA, the coefficients of the group in registers.
template <typename TX, int VEC, int kStages, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads <= 320 ? 2 : 1)
k_norm_cta(const NormP p, const Ranges rg, const TX* x, const __nv_bfloat16* y, TX* x_out, __nv_bfloat16* h) {
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ float red[2][4 * 32];                     // rows alternate: a barrier lies between two uses
    const Cols<VEC> c{p.C, (int)threadIdx.x, (int)blockDim.x};
    const int x_bytes = row_pieces<TX>() * 16 * blockDim.x, stage = x_bytes + (y ? row_pieces<__nv_bfloat16>() * 16 * blockDim.x : 0);
    const int64_t r0 = rg.begin(blockIdx.x), r1 = rg.begin(blockIdx.x + 1);
    auto fetch = [&](int64_t row, int st) {
        if constexpr (VEC == 8) {
            if (row < r1) {
                fetch_row(ring + st * stage, x + row * p.C, c);
                if (y) fetch_row(ring + st * stage + x_bytes, y + row * p.C, c);
            }
            fetch_commit();
        }
    };
    for (int i = 0; i < kStages - 1; ++i) fetch(r0 + i, i);
    Coef coef;
    int64_t grp = r0 / p.group_rows, left = 0;           // rows of the group still to come
    for (int64_t row = r0; row < r1; ++row) {
        const int n = (int)(row - r0);
        if (left == 0) {
            grp = row / p.group_rows;
            left = (grp + 1) * p.group_rows - row;
            load_coef(coef, p, grp, c, y != nullptr);
        }
        --left;
        fetch(row + kStages - 1, (n + kStages - 1) % kStages);
        float v[kCols], u[kCols];
        if constexpr (VEC == 8) {
            fetch_wait<kStages - 1>();
            const unsigned char* s = ring + n % kStages * stage;
            slot_row<TX>(s, c, v);
            if (y) slot_row<__nv_bfloat16>(s + x_bytes, c, u);
        } else {
            load_row<VEC>(x + row * p.C, c, v);
            if (y) load_row<VEC>(y + row * p.C, c, u);
        }
        norm_row<TX, VEC, false>(p, row, c, v, u, y != nullptr, coef, x_out, h, red[n & 1]);
    }
}

// ------------------------------------------------------------------ backward
struct GradP {
    float *dgate, *dscale, *dshift, *dweight, *dbias, *dpost;
    float* piece;                    // [n][2][3][C]: a CTA's first and last pieces of split groups
    float* wsum;                     // [n][3][C]: a CTA's sums for dweight, dbias, dpost_weight
};

constexpr int kBwdStages = 3, kRingThreads = 384;

// kThreads: upper bound of the CTA size (the register budget follows from it); kToken: every token is a group
template <typename TX, int VEC, int kThreads, bool kToken>
__global__ void __launch_bounds__(kThreads, 1)
k_norm_bwd(const NormP p, const GradP g, const Ranges rg, const __nv_bfloat16* dh, const TX* dx_out,
           const TX* x_out, const __nv_bfloat16* y, TX* dx, __nv_bfloat16* dy) {
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ float red[2][8 * 32];                     // rows alternate
    constexpr bool kRing = VEC == 8 && kThreads <= kRingThreads;      // longer rows: the ring would not fit
    const Cols<VEC> c{p.C, (int)threadIdx.x, (int)blockDim.x};
    const int64_t r0 = rg.begin(blockIdx.x), r1 = rg.begin(blockIdx.x + 1);
    const int xb = row_pieces<TX>() * 16 * blockDim.x, hb = row_pieces<__nv_bfloat16>() * 16 * blockDim.x;
    const int off_h = dh ? xb : 0, off_d = off_h + (dh ? hb : 0), off_y = off_d + (dx_out ? xb : 0),
              stage = off_y + (y ? hb : 0);
    auto fetch = [&](int64_t row, int st) {
        if constexpr (kRing) {
            if (row < r1) {
                unsigned char* s = ring + st * stage;
                if (dh) {
                    fetch_row(s, x_out + row * p.C, c);
                    fetch_row(s + off_h, dh + row * p.C, c);
                }
                if (dx_out) fetch_row(s + off_d, dx_out + row * p.C, c);
                if (y) fetch_row(s + off_y, y + row * p.C, c);
            }
            fetch_commit();
        }
    };
    // kToken: dweight, dbias, dpost_weight sums of the CTA; else A, S, T of the current group
    float sa[kCols] = {}, ss[kCols] = {}, st[kCols] = {};
    bool flushed = false;
    for (int i = 0; i < kBwdStages - 1; ++i) fetch(r0 + i, i);
    int n = 0;
    for (int64_t row = r0; row < r1; ++row, ++n) {
        fetch(row + kBwdStages - 1, (n + kBwdStages - 1) % kBwdStages);
        if constexpr (kRing) fetch_wait<kBwdStages - 1>();
        const unsigned char* slot = ring + n % kBwdStages * stage;
        float* rd = red[n & 1];
        const int64_t base = row * p.C, grp = row / p.group_rows, gbase = grp * p.C;
        auto get_x = [&](const TX* t, int off, float* v) {
            if constexpr (kRing) slot_row<TX>(slot + off, c, v); else load_row<VEC>(t + base, c, v);
        };
        auto get_h = [&](const __nv_bfloat16* t, int off, float* v) {
            if constexpr (kRing) slot_row<__nv_bfloat16>(slot + off, c, v); else load_row<VEC>(t + base, c, v);
        };
        // xh: x, centred, normalised; yh likewise
        float xh[kCols], yh[kCols];
        float rx = 1.f, ry = 1.f;
        if (dh) get_x(x_out, 0, xh);
        if (y) get_h(y, off_y, yh);
        float mean[2] = {0.f, 0.f};
        const bool lx = dh && p.norm == BSA_NORM_LAYER, ly = y && p.post == BSA_NORM_LAYER;
        if (lx || ly) {
            if (lx) mean[0] = sum_of(xh);
            if (ly) mean[1] = sum_of(yh);
            row_sum<false, 2>(mean, rd);
            if (lx) centre(xh, mean[0] / p.c, c);
            if (ly) centre(yh, mean[1] / p.c, c);
        }
        float d[kCols];                                  // total gradient of x_out
        if (dx_out) {
            get_x(dx_out, off_d, d);
        } else {
#pragma unroll
            for (int i = 0; i < kCols; ++i) d[i] = 0.f;
        }
        float four[4] = {0.f, 0.f, 0.f, 0.f};            // sum xc^2, sum g, sum g xc, sum yc^2
        float gr[kCols];
        if (dh) {
            get_h(dh, off_h, gr);
            with_param(gr, p.weight, c, times);
            if (p.scale) with_param(gr, p.scale + gbase, c, times1);
            four[0] = square_of(xh);
            four[1] = sum_of(gr);
#pragma unroll
            for (int i = 0; i < kCols; ++i) four[2] += gr[i] * xh[i];
        }
        if (y && p.post != BSA_NORM_NONE) four[3] = square_of(yh);
        if (dh || (y && p.post != BSA_NORM_NONE)) row_sum<false, 4>(four, rd + 64);
        if (dh) {
            rx = rsqrtf(four[0] * p.inv_c + p.eps);
            const float m0 = p.norm == BSA_NORM_LAYER ? four[1] * p.inv_c : 0.f, m1 = four[2] * rx * p.inv_c;
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
                xh[i] *= rx;
                d[i] += rx * (gr[i] - m0 - xh[i] * m1);
            }
            get_h(dh, off_h, gr);
            if constexpr (kToken) {
                if (g.dshift) store_row(g.dshift + gbase, c, gr);
                if (g.dscale) {
                    float t[kCols];
#pragma unroll
                    for (int i = 0; i < kCols; ++i) t[i] = xh[i];
                    with_param(t, p.weight, c, times);
                    with_param(t, p.bias, c, plus);
#pragma unroll
                    for (int i = 0; i < kCols; ++i) t[i] *= gr[i];
                    store_row(g.dscale + gbase, c, t);
                }
                if (p.scale) with_param(gr, p.scale + gbase, c, times1);
            }
#pragma unroll
            for (int i = 0; i < kCols; ++i) {
                sa[i] += gr[i] * xh[i];
                ss[i] += gr[i];
            }
        }
        if (y) {
            if (p.post != BSA_NORM_NONE) {
                ry = rsqrtf(four[3] * p.inv_c + p.eps);
#pragma unroll
                for (int i = 0; i < kCols; ++i) yh[i] *= ry;
            }
            float gy[kCols];
#pragma unroll
            for (int k = 0; k < kCols / VEC; ++k)
#pragma unroll
                for (int e = 0; e < VEC; ++e) gy[k * VEC + e] = c.in(k) ? d[k * VEC + e] : 0.f;
            if constexpr (kToken) {
                if (g.dgate) {
                    float t[kCols];
#pragma unroll
                    for (int i = 0; i < kCols; ++i) t[i] = yh[i];
                    with_param(t, p.post_weight, c, times);
#pragma unroll
                    for (int i = 0; i < kCols; ++i) t[i] *= gy[i];
                    store_row(g.dgate + gbase, c, t);
                }
                if (p.gate) with_param(gy, p.gate + gbase, c, times);
#pragma unroll
                for (int i = 0; i < kCols; ++i) st[i] += gy[i] * yh[i];
            } else {
#pragma unroll
                for (int i = 0; i < kCols; ++i) st[i] += gy[i] * yh[i];
                if (p.gate) with_param(gy, p.gate + gbase, c, times);
            }
            with_param(gy, p.post_weight, c, times);
            if (p.post != BSA_NORM_NONE) {
                float two[2] = {sum_of(gy), 0.f};
#pragma unroll
                for (int i = 0; i < kCols; ++i) two[1] += gy[i] * yh[i];
                row_sum<false, 2>(two, rd + 192);
                const float m0 = p.post == BSA_NORM_LAYER ? two[0] * p.inv_c : 0.f, m1 = two[1] * p.inv_c;
#pragma unroll
                for (int i = 0; i < kCols; ++i) gy[i] = ry * (gy[i] - m0 - yh[i] * m1);
            }
            store_row(dy + base, c, gy);
#pragma unroll
            for (int i = 0; i < kCols; ++i) d[i] *= p.res_scale;
        }
        store_row(dx + base, c, d);
        if constexpr (!kToken) {
            // the group ends here, or this CTA's share of it does
            const bool group_end = (row + 1) % p.group_rows == 0;
            if (!group_end && row + 1 < r1) continue;
            const bool whole = group_end && grp * p.group_rows >= r0;
            const int piece = grp * p.group_rows < r0 ? 0 : 1;        // one that began earlier, or one that goes on
#pragma unroll
            for (int k = 0; k < kCols / VEC; ++k) {
                if (!c.in(k)) continue;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int i = k * VEC + e, ch = c.at(k) + e;
                    const float sc = p.scale ? 1.f + p.scale[gbase + ch] : 1.f, gt = p.gate ? p.gate[gbase + ch] : 1.f;
                    float* w = g.wsum + (int64_t)blockIdx.x * 3 * p.C + ch;
                    w[0] = (flushed ? w[0] : 0.f) + sc * sa[i];
                    w[p.C] = (flushed ? w[p.C] : 0.f) + sc * ss[i];
                    w[2 * p.C] = (flushed ? w[2 * p.C] : 0.f) + gt * st[i];
                    if (whole) {
                        if (g.dscale)
                            g.dscale[gbase + ch] =
                                (p.weight ? p.weight[ch] : 1.f) * sa[i] + (p.bias ? p.bias[ch] : 0.f) * ss[i];
                        if (g.dshift) g.dshift[gbase + ch] = ss[i];
                        if (g.dgate) g.dgate[gbase + ch] = (p.post_weight ? p.post_weight[ch] : 1.f) * st[i];
                    } else {
                        float* o = g.piece + ((int64_t)blockIdx.x * 2 + piece) * 3 * p.C + ch;
                        o[0] = sa[i];
                        o[p.C] = ss[i];
                        o[2 * p.C] = st[i];
                    }
                    sa[i] = ss[i] = st[i] = 0.f;
                }
            }
            flushed = true;
        }
    }
    if constexpr (kToken) {
        float* w = g.wsum + (int64_t)blockIdx.x * 3 * p.C;
#pragma unroll
        for (int k = 0; k < kCols / VEC; ++k)
            if (c.in(k))
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    w[c.at(k) + e] = sa[k * VEC + e];
                    w[p.C + c.at(k) + e] = ss[k * VEC + e];
                    w[2 * p.C + c.at(k) + e] = st[k * VEC + e];
                }
    }
}

// Adds the pieces, 32 channels to a CTA and 32 strided shares to a channel, then the shares in order.  blockIdx.y = 0:
// the weight sums of all CTAs; the other y walk the groups and join those that span CTAs.
constexpr int kShares = 32;
__global__ void __launch_bounds__(32 * kShares)
k_norm_bwd_join(const NormP p, const GradP g, const Ranges rg, int64_t groups) {
    __shared__ float part[3][kShares][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    auto join = [&](const float* src, int64_t stride, int first, int count, float* out) {
        float s[3] = {0.f, 0.f, 0.f};
        if (c < p.C)
            for (int i = threadIdx.y; i < count; i += kShares) {
                // a split group's pieces: slot 1 of the CTA it begins in, slot 0 of the others
                const float* q = src + (first + i) * stride + (stride == 6 * (int64_t)p.C && i == 0 ? 3 * (int64_t)p.C : 0) + c;
                s[0] += q[0];
                s[1] += q[p.C];
                s[2] += q[2 * (int64_t)p.C];
            }
#pragma unroll
        for (int k = 0; k < 3; ++k) part[k][threadIdx.y][threadIdx.x] = s[k];
        __syncthreads();
        if (threadIdx.y < 3) {
            float a = 0.f;
            for (int i = 0; i < kShares; ++i) a += part[threadIdx.y][i][threadIdx.x];
            part[threadIdx.y][0][threadIdx.x] = a;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) out[k] = part[k][0][threadIdx.x];
        __syncthreads();
    };
    float s[3];
    if (blockIdx.y == 0) {
        join(g.wsum, 3 * (int64_t)p.C, 0, rg.n, s);
        if (c < p.C && threadIdx.y == 0) {
            if (g.dweight) g.dweight[c] = s[0];
            if (g.dbias) g.dbias[c] = s[1];
            if (g.dpost) g.dpost[c] = s[2];
        }
        return;
    }
    for (int64_t grp = blockIdx.y - 1; grp < groups; grp += gridDim.y - 1) {
        const int64_t lo = grp * p.group_rows;
        const int a = rg.owner(lo), b = rg.owner(lo + p.group_rows - 1);
        if (a == b) continue;
        join(g.piece, 6 * (int64_t)p.C, a, b - a + 1, s);
        if (c < p.C && threadIdx.y == 0) {
            const int64_t gc = grp * p.C + c;
            if (g.dscale) g.dscale[gc] = (p.weight ? p.weight[c] : 1.f) * s[0] + (p.bias ? p.bias[c] : 0.f) * s[1];
            if (g.dshift) g.dshift[gc] = s[1];
            if (g.dgate) g.dgate[gc] = (p.post_weight ? p.post_weight[c] : 1.f) * s[2];
        }
    }
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
    n.c = (float)a.C;
    n.inv_c = 1.f / n.c;
    n.gate = a.gate; n.scale = a.scale; n.shift = a.shift;
    n.weight = a.weight; n.bias = a.bias; n.post_weight = a.post_weight;
    return n;
}

// Threads that hold a row of C channels, 16 each.
int row_threads(int C) { return ((C + kCols - 1) / kCols + 31) / 32 * 32; }

constexpr int kSmemPerSm = 227 * 1024, kRegsPerSm = 65536;
// CTAs of `threads` with `regs` registers a thread and `smem` bytes that an SM holds.
int ctas_per_sm(int threads, int regs, int smem) {
    return std::max(1, std::min({2048 / threads, 32, kRegsPerSm / (threads * regs), kSmemPerSm / (smem + 2048)}));
}

// The gradient's CTAs (its workspace depends on them): as many as fit, 8 rows at least to each.
constexpr int kBwdRegs = 168;
int bwd_stage_bytes(const bsa_norm_args& a) {
    return a.C % 8 == 0 && row_threads(a.C) <= kRingThreads ? row_threads(a.C) * kCols * (2 * (a.dtype == BSA_BF16 ? 2 : 4) + 4) : 0;
}
int bwd_ctas(const bsa_plan& p, const bsa_norm_args& a) {
    const int threads = row_threads(a.C);
    const int per = ctas_per_sm(threads, threads <= kRingThreads ? kBwdRegs : 64, kBwdStages * bwd_stage_bytes(a));
    return (int)std::min<int64_t>((int64_t)p.num_sms * per, ((int64_t)p.B * p.N + 7) / 8);
}

template <typename TX, int VEC>
cudaError_t fwd(const bsa_plan& p, const NormP& n, const void* x, const void* y, void* x_out, void* h, cudaStream_t s) {
    const TX* xi = (const TX*)x;
    const __nv_bfloat16* yi = (const __nv_bfloat16*)y;
    if (n.C <= 32 * kCols) {
        constexpr int kWarps = 4;
        k_norm_warp<TX, VEC><<<(unsigned)((n.rows + kWarps - 1) / kWarps), 32 * kWarps, 0, s>>>(
            n, xi, yi, (TX*)x_out, (__nv_bfloat16*)h);
        return cudaGetLastError();
    }
    const int threads = row_threads(n.C);
    // a ring of three rows, of two where three would leave an SM with one CTA
    const int row_bytes = threads * kCols * (int)(sizeof(TX) + (y ? 2 : 0));
    const bool three = 3 * row_bytes <= 96 * 1024;
    const int smem = VEC == 8 ? (three ? 3 : 2) * row_bytes : 0;
    auto kern = threads <= 320 ? (three || VEC == 1 ? k_norm_cta<TX, VEC, 3, 320> : k_norm_cta<TX, VEC, 2, 320>)
                               : (three || VEC == 1 ? k_norm_cta<TX, VEC, 3, 1024> : k_norm_cta<TX, VEC, 2, 1024>);
    if (smem > 48 * 1024)
        if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
    const Ranges rg{n.rows, (int)std::min<int64_t>(n.rows, (int64_t)p.num_sms * ctas_per_sm(threads, threads <= 320 ? 102 : 64, smem))};
    kern<<<rg.n, threads, smem, s>>>(n, rg, xi, yi, (TX*)x_out, (__nv_bfloat16*)h);
    return cudaGetLastError();
}

template <typename TX, int VEC>
cudaError_t bwd(const bsa_norm_args& a, const NormP& n, const GradP& g, const Ranges& rg, const void* dh,
                const void* dx_out, const void* x_out, const void* y, void* dx, void* dy, cudaStream_t s) {
    const int threads = row_threads(n.C);
    const bool token = n.group_rows == 1;
    auto kern = threads <= kRingThreads ? (token ? k_norm_bwd<TX, VEC, kRingThreads, true> : k_norm_bwd<TX, VEC, kRingThreads, false>)
                               : (token ? k_norm_bwd<TX, VEC, 1024, true> : k_norm_bwd<TX, VEC, 1024, false>);
    const int smem = kBwdStages * bwd_stage_bytes(a);
    if (smem > 48 * 1024)
        if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
    kern<<<rg.n, threads, smem, s>>>(n, g, rg, (const __nv_bfloat16*)dh, (const TX*)dx_out, (const TX*)x_out,
                                     (const __nv_bfloat16*)y, (TX*)dx, (__nv_bfloat16*)dy);
    if (cudaError_t e = cudaGetLastError()) return e;
    const int64_t groups = token ? 0 : n.rows / n.group_rows;
    k_norm_bwd_join<<<dim3((n.C + 31) / 32, 1 + (unsigned)std::min<int64_t>(groups, 1024)), dim3(32, kShares), 0, s>>>(
        n, g, rg, groups);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const bsa_plan& p, const bsa_norm_args& a, const void* x, const void* y, void* x_out, void* h,
                        cudaStream_t s) {
    const NormP n = norm_params(p, a);
    const bool wide = a.C % 8 == 0;
    if (a.dtype == BSA_BF16)
        return wide ? fwd<__nv_bfloat16, 8>(p, n, x, y, x_out, h, s) : fwd<__nv_bfloat16, 1>(p, n, x, y, x_out, h, s);
    return wide ? fwd<float, 8>(p, n, x, y, x_out, h, s) : fwd<float, 1>(p, n, x, y, x_out, h, s);
}

size_t norm_bwd_ws_bytes(const bsa_plan& p, const bsa_norm_args& a) {
    return align_up((size_t)bwd_ctas(p, a) * 9 * a.C * sizeof(float));
}

cudaError_t launch_norm_bwd(const bsa_plan& p, const bsa_norm_args& a, const NormGrads& out, const void* dh,
                            const void* dx_out, const void* x_out, const void* y, void* dx, void* dy, void* ws,
                            cudaStream_t s) {
    const NormP n = norm_params(p, a);
    const Ranges rg{n.rows, bwd_ctas(p, a)};
    GradP g;
    g.dgate = out.dgate; g.dscale = out.dscale; g.dshift = out.dshift;
    g.dweight = out.dweight; g.dbias = out.dbias; g.dpost = out.dpost_weight;
    g.piece = (float*)ws;
    g.wsum = g.piece + (size_t)rg.n * 6 * a.C;
    const bool wide = a.C % 8 == 0;
    if (a.dtype == BSA_BF16)
        return wide ? bwd<__nv_bfloat16, 8>(a, n, g, rg, dh, dx_out, x_out, y, dx, dy, s)
                    : bwd<__nv_bfloat16, 1>(a, n, g, rg, dh, dx_out, x_out, y, dx, dy, s);
    return wide ? bwd<float, 8>(a, n, g, rg, dh, dx_out, x_out, y, dx, dy, s)
                : bwd<float, 1>(a, n, g, rg, dh, dx_out, x_out, y, dx, dy, s);
}

}  // namespace bsa
