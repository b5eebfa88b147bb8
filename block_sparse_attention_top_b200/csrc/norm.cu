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
#include "cross_common.cuh"

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

// A thread's channels: runs of VEC, run k at (first + k * stride) * VEC.
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

// Rows off the 16-byte grid do not come through a ring: their 128-byte lines are brought to L2 two rows ahead, a line to a
// thread (32 760 fp32 rows of 1219 channels, norms on both sides: 251 -> 242 us; in the backward kernel it cost 3 % at
// 2958 such rows).  (A thread holds at most 64 bytes of the row.)
template <typename T>
__device__ __forceinline__ void prefetch_row(const T* p, int C) {
    if (threadIdx.x * 128 < C * sizeof(T))
        asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(p) + threadIdx.x * 128));
}

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
        } else if (row < r1) {
            prefetch_row(x + row * p.C, p.C);
            if (y) prefetch_row(y + row * p.C, p.C);
        }
    };
    for (int i = 0; i < kStages - 1; ++i) fetch(r0 + i, i);
    Coef coef;
    int64_t grp = r0 / p.group_rows, left = 0;           // rows of the group still to come
    for (int64_t row = r0; row < r1; ++row) {
        const int n = (int)(row - r0);
        float v[kCols], u[kCols];
        if (left == 0) {
            grp = row / p.group_rows;
            left = (grp + 1) * p.group_rows - row;
            load_coef(coef, p, grp, c, y != nullptr);
        }
        --left;
        fetch(row + kStages - 1, (n + kStages - 1) % kStages);
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

// Sums of 4 G values over a CTA with one barrier, through red[4 G][32] (zero where no warp writes).  Four values take
// six shuffles to a warp's sums (each step halves what a lane still carries), and behind the barrier one 16-byte load
// and three shuffles add 32 warps' sums of all four.
template <int G>
__device__ __forceinline__ void cta_sums(float* v, float* red) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const bool h16 = lane & 16, h8 = lane & 8;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float* w = v + 4 * g;
        float a0 = h16 ? w[2] : w[0], a1 = h16 ? w[3] : w[1];
        a0 += __shfl_xor_sync(0xffffffffu, h16 ? w[0] : w[2], 16);
        a1 += __shfl_xor_sync(0xffffffffu, h16 ? w[1] : w[3], 16);
        float c = (h8 ? a1 : a0) + __shfl_xor_sync(0xffffffffu, h8 ? a0 : a1, 8);
        c += __shfl_xor_sync(0xffffffffu, c, 4);
        c += __shfl_xor_sync(0xffffffffu, c, 2);
        c += __shfl_xor_sync(0xffffffffu, c, 1);
        if ((lane & 7) == 0) red[(4 * g + lane / 8) * 32 + warp] = c;
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const float4 f = *reinterpret_cast<const float4*>(red + (4 * g + lane / 8) * 32 + 4 * (lane & 7));
        float s = (f.x + f.y) + (f.z + f.w);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        s += __shfl_xor_sync(0xffffffffu, s, 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * g + k] = __shfl_sync(0xffffffffu, s, 8 * k);
    }
}

// Channels a thread holds in the backward kernel: 8, or 16 where a row would need more than 1024 threads.
constexpr int bwd_cols(int C) { return C <= 8 * 1024 ? 8 : 16; }
constexpr int kBwdStages = 3;

// kToken: every token is a group; kPost: the branch is normalised; kRing: rows come through the ring
template <typename TX, int VEC, int NC, int kThreads, bool kToken, bool kPost, bool kRing>
__global__ void __launch_bounds__(kThreads, 1)
k_norm_bwd(const NormP p, const GradP g, const Ranges rg, const __nv_bfloat16* dh, const TX* dx_out,
           const TX* x_out, const __nv_bfloat16* y, TX* dx, __nv_bfloat16* dy) {
    constexpr int R = NC / VEC;                          // runs
    constexpr int G = kPost ? 2 : 1;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ __align__(16) float red[2][(G + 1) * 4 * 32];          // rows alternate
    for (int i = threadIdx.x; i < 2 * (G + 1) * 4 * 32; i += blockDim.x) red[0][i] = 0.f;
    __syncthreads();
    const Cols<VEC> c{p.C, (int)threadIdx.x, (int)blockDim.x};
    const int64_t r0 = rg.begin(blockIdx.x), r1 = rg.begin(blockIdx.x + 1);
    const bool lx = dh && p.norm == BSA_NORM_LAYER, ly = kPost && p.post == BSA_NORM_LAYER;

    // ---- loads of a row's channels
    const int xb = NC * (int)sizeof(TX) * blockDim.x, hb = NC * 2 * blockDim.x;
    const int off_h = dh ? xb : 0, off_d = off_h + (dh ? hb : 0), off_y = off_d + (dx_out ? xb : 0),
              stage = off_y + (y ? hb : 0);
    auto fetch_one = [&](unsigned char* slot, const auto* t) {
        constexpr int kPer = 8 * sizeof(*t) / 16;
#pragma unroll
        for (int k = 0; k < NC / 8; ++k)
            if (c.in(k))
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    fetch16((uint32_t)__cvta_generic_to_shared(slot + ((k * kPer + i) * blockDim.x + threadIdx.x) * 16),
                            reinterpret_cast<const char*>(t + c.at(k)) + 16 * i);
    };
    auto fetch = [&](int64_t row, int st) {
        if constexpr (kRing) {
            if (row < r1) {
                unsigned char* s = ring + st * stage;
                const int64_t base = row * p.C;
                if (dh) {
                    fetch_one(s, x_out + base);
                    fetch_one(s + off_h, dh + base);
                }
                if (dx_out) fetch_one(s + off_d, dx_out + base);
                if (y) fetch_one(s + off_y, y + base);
            }
            fetch_commit();
        }
    };
    // channels of one array of the row in ring stage `st` (or at `t`)
    auto get = [&](const auto* t, int st, int off, float* v) {
        constexpr int kPer = 8 * sizeof(*t) / 16;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (!c.in(k)) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[k * VEC + e] = 0.f;
            } else if constexpr (kRing) {
                const unsigned char* s = ring + st * stage + off + (k * kPer * blockDim.x + threadIdx.x) * 16;
                if constexpr (sizeof(*t) == 2) {
                    load_cols<8>(reinterpret_cast<const __nv_bfloat16*>(s), v + 8 * k);
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 f = *reinterpret_cast<const float4*>(s + i * blockDim.x * 16);
                        v[8 * k + 4 * i] = f.x;
                        v[8 * k + 4 * i + 1] = f.y;
                        v[8 * k + 4 * i + 2] = f.z;
                        v[8 * k + 4 * i + 3] = f.w;
                    }
                }
            } else {
                load_cols<VEC>(t + c.at(k), v + k * VEC);
            }
        }
    };
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < NC; ++i) f(i);
    };
    auto param = [&](float* v, const float* q, auto f) {
        if (!q) return;
#pragma unroll
        for (int k = 0; k < R; ++k)
            if (c.in(k)) {
                float t[VEC];
                load_cols<VEC>(q + c.at(k), t);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[k * VEC + e] = f(v[k * VEC + e], t[e]);
            }
    };
    auto store = [&](auto* t, const float* v) {
#pragma unroll
        for (int k = 0; k < R; ++k)
            if (c.in(k)) store_cols<VEC>(t + c.at(k), v + k * VEC);
    };
    // The arithmetic of a row is in pairs of channels (f32x2): it issues half as many instructions, which bound the
    // kernel (72 % of issue slots at 5120 channels with single ones).
    auto pairs = [&](auto f) {
#pragma unroll
        for (int i = 0; i < NC; i += 2) f(i);
    };
    auto total = [&](const float* v) {
        float s0 = 0.f, s1 = 0.f;
        pairs([&](int i) { tc::fadd2(s0, s1, s0, s1, v[i], v[i + 1]); });
        return s0 + s1;
    };
    auto centred = [&](float* v, float mean) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if constexpr (VEC == 8) {
                if (c.in(k))                             // channels past C hold 0
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        tc::fadd2(v[8 * k + e], v[8 * k + e + 1], v[8 * k + e], v[8 * k + e + 1], -mean, -mean);
            } else {
                v[k] = c.in(k) ? v[k] - mean : 0.f;
            }
        }
    };

    // kToken: dweight, dbias, dpost_weight sums of the CTA; else A, S, T of the current group
    float sa[NC] = {}, ss[NC] = {}, st_[NC] = {};
    float ca[NC], cg[NC];                                // weight (1 + scale), gate post_weight of the group
    bool flushed = false;
    int64_t left = 0, gbase = 0;                         // rows of the group still to come; its parameters
    for (int i = 0; i < kBwdStages - 1; ++i) fetch(r0 + i, i);
    // the first row's sums for its means; every later row's travel with the sums of the row before it
    float sums[4 * G];
    for (int i = 0; i < 4 * G; ++i) sums[i] = 0.f;
    if (lx || ly) {
        if constexpr (kRing) fetch_wait<kBwdStages - 2>();
        float t[NC];
        if (lx) {
            get(x_out + r0 * p.C, 0, 0, t);
            sums[3] = total(t);
        }
        if constexpr (kPost)
            if (ly) {
                get(y + r0 * p.C, 0, off_y, t);
                sums[5] = total(t);
            }
        cta_sums<G>(sums, red[1]);
    }
    int st = 0;
    for (int64_t row = r0; row < r1; ++row) {
        const int nx = st + 1 == kBwdStages ? 0 : st + 1;            // the next row's stage
        fetch(row + kBwdStages - 1, nx + 1 == kBwdStages ? 0 : nx + 1);
        float* rd = red[(row - r0) & 1];
        const int64_t base = row * p.C;
        if (left == 0) {
            const int64_t grp = row / p.group_rows;
            left = (grp + 1) * p.group_rows - row;
            gbase = grp * p.C;
            each([&](int i) { ca[i] = cg[i] = 1.f; });
            param(ca, p.weight, times);
            if (p.scale) param(ca, p.scale + gbase, times1);
            param(cg, p.post_weight, times);
            if (p.gate) param(cg, p.gate + gbase, times);
        }
        --left;
        const float mean_x = sums[3] / p.c, mean_y = kPost ? sums[4 * G - 3] / p.c : 0.f;
        if constexpr (kRing) fetch_wait<kBwdStages - 2>();           // this row and the next
        // xh: x centred, then normalised; yh likewise
        float xh[NC], gh[NC], yh[NC], d[NC];
        for (int i = 0; i < 4 * G; ++i) sums[i] = 0.f;               // sum xc^2, g, g xc, next x | yc^2, next y
        if (dh) {
            get(x_out + base, st, 0, xh);
            get(dh + base, st, off_h, gh);
            if (lx) centred(xh, mean_x);
            float q0 = 0.f, q1 = 0.f, s0 = 0.f, s1 = 0.f, x0 = 0.f, x1 = 0.f;
            pairs([&](int i) {
                float g0, g1;
                cross::fmul2(g0, g1, gh[i], gh[i + 1], ca[i], ca[i + 1]);
                tc::ffma2(q0, q1, xh[i], xh[i + 1], xh[i], xh[i + 1], q0, q1);
                tc::fadd2(s0, s1, s0, s1, g0, g1);
                tc::ffma2(x0, x1, g0, g1, xh[i], xh[i + 1], x0, x1);
            });
            sums[0] = q0 + q1;
            sums[1] = s0 + s1;
            sums[2] = x0 + x1;
            if (lx && row + 1 < r1) {
                get(x_out + base + p.C, nx, 0, d);
                sums[3] = total(d);
            }
        }
        if (y) get(y + base, st, off_y, yh);
        if constexpr (kPost) {
            if (ly) centred(yh, mean_y);
            float q0 = 0.f, q1 = 0.f;
            pairs([&](int i) { tc::ffma2(q0, q1, yh[i], yh[i + 1], yh[i], yh[i + 1], q0, q1); });
            sums[4] = q0 + q1;
            if (ly && row + 1 < r1) {
                get(y + base + p.C, nx, off_y, d);
                sums[5] = total(d);
            }
        }
        if (dx_out) {
            get(dx_out + base, st, off_d, d);
        } else {
            each([&](int i) { d[i] = 0.f; });
        }
        if (dh || kPost) cta_sums<G>(sums, rd);
        if (dh) {
            const float rx = rsqrtf(sums[0] * p.inv_c + p.eps);
            const float m0 = p.norm == BSA_NORM_LAYER ? sums[1] * p.inv_c : 0.f, m1 = sums[2] * rx * p.inv_c;
            pairs([&](int i) {
                float t0, t1;
                cross::fmul2(xh[i], xh[i + 1], xh[i], xh[i + 1], rx, rx);
                tc::ffma2(t0, t1, gh[i], gh[i + 1], ca[i], ca[i + 1], -m0, -m0);
                tc::ffma2(t0, t1, xh[i], xh[i + 1], -m1, -m1, t0, t1);
                tc::ffma2(d[i], d[i + 1], rx, rx, t0, t1, d[i], d[i + 1]);
            });
            if constexpr (kToken) {
                if (g.dshift) store(g.dshift + gbase, gh);
                if (g.dscale) {
                    float t[NC];
                    each([&](int i) { t[i] = xh[i]; });
                    param(t, p.weight, times);
                    param(t, p.bias, plus);
                    each([&](int i) { t[i] *= gh[i]; });
                    store(g.dscale + gbase, t);
                }
                if (p.scale) param(gh, p.scale + gbase, times1);
            }
            pairs([&](int i) {
                tc::ffma2(sa[i], sa[i + 1], gh[i], gh[i + 1], xh[i], xh[i + 1], sa[i], sa[i + 1]);
                tc::fadd2(ss[i], ss[i + 1], ss[i], ss[i + 1], gh[i], gh[i + 1]);
            });
        }
        if (y) {
            float ry = 1.f;
            if constexpr (kPost) {
                ry = rsqrtf(sums[4] * p.inv_c + p.eps);
                pairs([&](int i) { cross::fmul2(yh[i], yh[i + 1], yh[i], yh[i + 1], ry, ry); });
            }
            if constexpr (kToken) {
                float t[NC];
                if (g.dgate) {
                    each([&](int i) { t[i] = yh[i]; });
                    param(t, p.post_weight, times);
                    each([&](int i) { t[i] *= d[i]; });
                    store(g.dgate + gbase, t);
                }
                each([&](int i) { t[i] = d[i]; });
                if (p.gate) param(t, p.gate + gbase, times);
                each([&](int i) { st_[i] += t[i] * yh[i]; });
            } else {
                pairs([&](int i) { tc::ffma2(st_[i], st_[i + 1], d[i], d[i + 1], yh[i], yh[i + 1], st_[i], st_[i + 1]); });
            }
            if constexpr (kPost) {
                // channels past C: cg is 1 there, yh 0
                float two[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < R; ++k)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float gy = c.in(k) ? d[k * VEC + e] * cg[k * VEC + e] : 0.f;
                        two[0] += gy;
                        two[1] += gy * yh[k * VEC + e];
                    }
                cta_sums<1>(two, rd + G * 4 * 32);
                const float m0 = p.post == BSA_NORM_LAYER ? two[0] * p.inv_c : 0.f, m1 = two[1] * p.inv_c;
                each([&](int i) { yh[i] = ry * (d[i] * cg[i] - m0 - yh[i] * m1); });
            } else {
                pairs([&](int i) { cross::fmul2(yh[i], yh[i + 1], d[i], d[i + 1], cg[i], cg[i + 1]); });
            }
            store(dy + base, yh);
            if (p.res_scale != 1.f)
                pairs([&](int i) { cross::fmul2(d[i], d[i + 1], d[i], d[i + 1], p.res_scale, p.res_scale); });
        }
        store(dx + base, d);
        st = nx;
        if constexpr (!kToken) {
            // the group ends here, or this CTA's share of it does
            if (left > 0 && row + 1 < r1) continue;
            const int64_t first = row + 1 + left - p.group_rows;      // the group's first row
            const bool whole = left == 0 && first >= r0;
            const int piece = first < r0 ? 0 : 1;                     // one that began earlier, or one that goes on
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (!c.in(k)) continue;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int i = k * VEC + e, ch = c.at(k) + e;
                    const float sc = p.scale ? 1.f + p.scale[gbase + ch] : 1.f, gt = p.gate ? p.gate[gbase + ch] : 1.f;
                    float* w = g.wsum + (int64_t)blockIdx.x * 3 * p.C + ch;
                    w[0] = (flushed ? w[0] : 0.f) + sc * sa[i];
                    w[p.C] = (flushed ? w[p.C] : 0.f) + sc * ss[i];
                    w[2 * p.C] = (flushed ? w[2 * p.C] : 0.f) + gt * st_[i];
                    if (whole) {
                        if (g.dscale)
                            g.dscale[gbase + ch] =
                                (p.weight ? p.weight[ch] : 1.f) * sa[i] + (p.bias ? p.bias[ch] : 0.f) * ss[i];
                        if (g.dshift) g.dshift[gbase + ch] = ss[i];
                        if (g.dgate) g.dgate[gbase + ch] = (p.post_weight ? p.post_weight[ch] : 1.f) * st_[i];
                    } else {
                        float* o = g.piece + ((int64_t)blockIdx.x * 2 + piece) * 3 * p.C + ch;
                        o[0] = sa[i];
                        o[p.C] = ss[i];
                        o[2 * p.C] = st_[i];
                    }
                    sa[i] = ss[i] = st_[i] = 0.f;
                }
            }
            flushed = true;
        }
    }
    if constexpr (kToken) {
        float* w = g.wsum + (int64_t)blockIdx.x * 3 * p.C;
#pragma unroll
        for (int k = 0; k < R; ++k)
            if (c.in(k))
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    w[c.at(k) + e] = sa[k * VEC + e];
                    w[p.C + c.at(k) + e] = ss[k * VEC + e];
                    w[2 * p.C + c.at(k) + e] = st_[k * VEC + e];
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
#pragma unroll 4
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

// Parameters that have no part in a call are null from here on, whatever the caller's struct holds there: gate and
// post_weight without a branch y, the affine and the modulation without an h.
NormP norm_params(const bsa_plan& p, const bsa_norm_args& a, bool has_y) {
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
    const bool has_h = a.norm != BSA_NORM_NONE;
    n.gate = has_y ? a.gate : nullptr;
    n.post_weight = has_y ? a.post_weight : nullptr;
    n.scale = has_h ? a.scale : nullptr;
    n.shift = has_h ? a.shift : nullptr;
    n.weight = has_h ? a.weight : nullptr;
    n.bias = has_h ? a.bias : nullptr;
    return n;
}

// Threads that hold a row of C channels, 16 each.
int row_threads(int C) { return ((C + kCols - 1) / kCols + 31) / 32 * 32; }

constexpr int kSmemPerSm = 227 * 1024, kRegsPerSm = 65536;
constexpr int kRingBytes = 200 * 1024;   // the largest ring of any variant
template <typename K>
cudaError_t allow_ring(K kern, int smem) { return allow_smem(kern, smem, kRingBytes); }

// CTAs of `threads` with `regs` registers a thread and `smem` bytes that an SM holds.
int ctas_per_sm(int threads, int regs, int smem) {
    return std::max(1, std::min({2048 / threads, 32, kRegsPerSm / (threads * regs), kSmemPerSm / (smem + 2048)}));
}

// The gradient's CTAs (its workspace depends on them): as many as fit, 8 rows at least to each.
int bwd_threads(int C) { return ((C + bwd_cols(C) - 1) / bwd_cols(C) + 31) / 32 * 32; }
// bytes of a ring stage, 0: no ring (rows off the 16-byte grid; more than 8192 channels, 5632 in fp32)
int bwd_stage_bytes(const bsa_norm_args& a) {
    const int bytes = bwd_threads(a.C) * bwd_cols(a.C) * (2 * (a.dtype == BSA_BF16 ? 2 : 4) + 4);
    return a.C % 8 == 0 && bwd_cols(a.C) == 8 && kBwdStages * bytes <= kRingBytes ? bytes : 0;
}
int bwd_ctas(const bsa_plan& p, const bsa_norm_args& a) {
    const int threads = bwd_threads(a.C);
    const int per = ctas_per_sm(threads, threads <= 512 ? 128 : threads <= 640 ? 96 : 64, kBwdStages * bwd_stage_bytes(a));
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
    // A ring of three rows, of two where three do not fit: fp32 rows with a branch of more than 704 threads (11 264 channels).
    const int row_bytes = threads * kCols * (int)(sizeof(TX) + (y ? 2 : 0));
    const bool three = 3 * row_bytes <= kRingBytes;
    const int smem = VEC == 8 ? (three ? 3 : 2) * row_bytes : 0;
    // Up to 640 threads a CTA to an SM with 96 registers a thread is faster than two with 64, which spill (50 400 bf16 rows
    // of 6144 channels 573 against 657 us, of 8192 654 against 869; fp32 rows of 8192 1176 against 1580).  Scalar loads
    // keep the two CTAs for their warps; since their lines are prefetched it makes little difference (5308 channels,
    // 75 600 bf16 rows 2.98 ms against 3.01 with one; 25 200 fp32 rows 1.01 against 0.93).
    const bool roomy = VEC == 8 && threads <= 640;
    auto kern = k_norm_cta<TX, VEC, 3, 1024>;
    if constexpr (VEC == 8) {
        static_assert(3 * 640 * kCols * (sizeof(TX) + 2) <= kRingBytes, "up to 640 threads have three rows");
        if (threads <= 320) kern = k_norm_cta<TX, VEC, 3, 320>;
        else if (roomy) kern = k_norm_cta<TX, VEC, 3, 640>;
        if constexpr (sizeof(TX) == 4)
            if (!three) kern = k_norm_cta<TX, VEC, 2, 1024>;
    } else if (threads <= 320) {
        kern = k_norm_cta<TX, VEC, 3, 320>;
    }
    if (cudaError_t e = allow_ring(kern, smem)) return e;
    const Ranges rg{n.rows, (int)std::min<int64_t>(n.rows, (int64_t)p.num_sms * ctas_per_sm(threads, threads <= 320 || roomy ? 102 : 64, smem))};
    kern<<<rg.n, threads, smem, s>>>(n, rg, xi, yi, (TX*)x_out, (__nv_bfloat16*)h);
    return cudaGetLastError();
}

struct BwdCall {
    NormP n;
    GradP g;
    Ranges rg;
    const void *dh, *dx_out, *x_out, *y;
    void *dx, *dy;
    int threads, stage;
    cudaStream_t s;
};

template <typename TX, int VEC, int NC, int kThreads, bool kToken, bool kPost, bool kRing>
cudaError_t bwd_t(const BwdCall& b) {
    auto kern = k_norm_bwd<TX, VEC, NC, kThreads, kToken, kPost, kRing>;
    const int smem = kRing ? kBwdStages * b.stage : 0;
    if (cudaError_t e = allow_ring(kern, smem)) return e;
    kern<<<b.rg.n, b.threads, smem, b.s>>>(b.n, b.g, b.rg, (const __nv_bfloat16*)b.dh, (const TX*)b.dx_out,
                                           (const TX*)b.x_out, (const __nv_bfloat16*)b.y, (TX*)b.dx, (__nv_bfloat16*)b.dy);
    return cudaGetLastError();
}
template <typename TX, int VEC, int NC, int kThreads, bool kRing>
cudaError_t bwd_opts(const BwdCall& b) {
    const bool token = b.n.group_rows == 1, post = b.y && b.n.post != BSA_NORM_NONE;
    if (token) return post ? bwd_t<TX, VEC, NC, kThreads, true, true, kRing>(b) : bwd_t<TX, VEC, NC, kThreads, true, false, kRing>(b);
    return post ? bwd_t<TX, VEC, NC, kThreads, false, true, kRing>(b) : bwd_t<TX, VEC, NC, kThreads, false, false, kRing>(b);
}
template <typename TX>
cudaError_t bwd(const BwdCall& b) {
    if (b.n.C % 8 == 0 && b.stage > 0) {
        if (b.threads <= 512) return bwd_opts<TX, 8, 8, 512, true>(b);
        if (b.threads <= 640) return bwd_opts<TX, 8, 8, 640, true>(b);
        return bwd_opts<TX, 8, 8, 1024, true>(b);
    }
    if (bwd_cols(b.n.C) == 16)
        return b.n.C % 8 == 0 ? bwd_opts<TX, 8, 16, 1024, false>(b) : bwd_opts<TX, 1, 16, 1024, false>(b);
    if constexpr (sizeof(TX) == 4)                       // (a bf16 row of up to 8192 channels always has a ring)
        if (b.n.C % 8 == 0) return bwd_opts<TX, 8, 8, 1024, false>(b);
    return b.threads <= 512 ? bwd_opts<TX, 1, 8, 512, false>(b) : bwd_opts<TX, 1, 8, 1024, false>(b);
}

}  // namespace

cudaError_t launch_norm(const bsa_plan& p, const bsa_norm_args& a, const void* x, const void* y, void* x_out, void* h,
                        cudaStream_t s) {
    const NormP n = norm_params(p, a, y != nullptr);
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
    const NormP n = norm_params(p, a, y != nullptr);
    const Ranges rg{n.rows, bwd_ctas(p, a)};
    GradP g;
    g.dgate = out.dgate; g.dscale = out.dscale; g.dshift = out.dshift;
    g.dweight = out.dweight; g.dbias = out.dbias; g.dpost = out.dpost_weight;
    g.piece = (float*)ws;
    g.wsum = g.piece + (size_t)rg.n * 6 * a.C;
    const BwdCall b{n, g, rg, dh, dx_out, x_out, y, dx, dy, bwd_threads(a.C), bwd_stage_bytes(a), s};
    cudaError_t e = a.dtype == BSA_BF16 ? bwd<__nv_bfloat16>(b) : bwd<float>(b);
    if (e != cudaSuccess) return e;
    // No h: its scale and shift have no part in the result.  The kernel writes a token's own gradients where it has a dh;
    // those of larger groups come out of its sums, which are 0.
    if (!dh && n.group_rows == 1)
        for (float* d : {g.dscale, g.dshift})
            if (d && (e = cudaMemsetAsync(d, 0, (size_t)n.rows * n.C * sizeof(float), s)) != cudaSuccess) return e;
    const int64_t groups = n.group_rows == 1 ? 0 : n.rows / n.group_rows;
    k_norm_bwd_join<<<dim3((n.C + 31) / 32, 1 + (unsigned)std::min<int64_t>(groups, 1024)), dim3(32, kShares), 0, s>>>(
        n, g, rg, groups);
    return cudaGetLastError();
}

}  // namespace bsa
