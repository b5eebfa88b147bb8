// Cross attention of few query rows (a new token, or a handful): the work is
// reading K and V once, so it is split over the states and joined.
//
// The query rows that share a key head (H / Hkv heads times N tokens) make
// tiles of 16; a cluster of up to 8 CTAs shares a row tile's states, and each
// of a CTA's 4 warps takes every fourth block of 16 states of its share, with
// a ring of its own that cp.async fills two blocks ahead: no barrier between
// warps until the end, and 128 KB in flight per SM.  Products are mma.sync
// m16n8k16 (bf16, fp32 sums); bound by HBM, they do not need more.  Partial
// results (maximum, sum, O) join in shared memory, first a CTA's warps, then
// over distributed shared memory the cluster's CTAs, in a fixed order; nothing
// goes through a workspace.
//
// Measured: a token of each of 4 sequences, 40 query heads on 8 key heads of
// 128, 32 760 states each: 93 us, 5.78 TB/s (a copy makes 6.55).  With lengths
// from a third of that to all of it 59-77 us: every sequence has as many
// CTAs, so the longest one decides.
#include <algorithm>

#include <cooperative_groups.h>

#include "cross_common.cuh"

namespace bsa {
namespace {

namespace cg = cooperative_groups;
using namespace tc;
using namespace cross;

constexpr int kRows = 16, kBlkKeys = 16, kWarps = 4, kStages = 3;
constexpr int kMaxSplit = 8;         // CTAs of a cluster

struct FewP {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16* o;
    float* lse;
    Keys keys;
    int64_t st[9];
    int N, H, Hkv, G;
    float scale_log2;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
    const int n = real ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
struct FewSmem {
    static constexpr int kBlock = kBlkKeys * D * 2;                 // K or V of 16 states
    static constexpr int kWarpBytes = kStages * 2 * kBlock;
    static constexpr int kBytes = kWarps * kWarpBytes;
    // after the loop: O [4 warps][16][D], then m, l [4 warps][16]; joined: O [16][D], m, l [16]
    static constexpr int offM = kWarps * kRows * D * 4;
    static constexpr int offJoin = offM + 2 * kWarps * kRows * 4;
    static_assert(offJoin + kRows * (D + 2) * 4 <= kBytes, "the join reuses the rings");
};

template <int D>
__global__ void __launch_bounds__(32 * kWarps, 2)
k_cross_few(const FewP p) {
    using L = FewSmem<D>;
    extern __shared__ __align__(128) unsigned char smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int split = cluster.block_rank(), splits = cluster.num_blocks();
    const int row0 = blockIdx.y * kRows, rows = p.G * p.N;
    const int b = blockIdx.z / p.Hkv, hk = blockIdx.z % p.Hkv;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int len = p.keys.count(b), blocks = (len + kBlkKeys - 1) / kBlkKeys;
    const int beg = (int)((int64_t)blocks * split / splits), end = (int)((int64_t)blocks * (split + 1) / splits);

    // row r is token r / G of head hk * G + r % G
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = row0 + lane / 4 + 8 * i;
        const __nv_bfloat16* qr = p.q + b * p.st[0] + (int64_t)(r / p.G) * p.st[1] + (int64_t)(hk * p.G + r % p.G) * p.st[2];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int c = kk * 16 + (lane % 4) * 2;
            qf[kk][i] = r < rows ? *reinterpret_cast<const uint32_t*>(qr + c) : 0u;
            qf[kk][2 + i] = r < rows ? *reinterpret_cast<const uint32_t*>(qr + c + 8) : 0u;
        }
    }
    const __nv_bfloat16* kb = p.k + b * p.st[3] + hk * p.st[5];
    const __nv_bfloat16* vb = p.v + b * p.st[6] + hk * p.st[8];
    const uint32_t ring = smem_u32(smem) + warp * L::kWarpBytes;
    // K and V of state block t into stage st; states past the length become zeros.  Chunk c of row r lies at c ^ (r & 7).
    auto load = [&](int t, int st) {
        const uint32_t dst = ring + st * 2 * L::kBlock;
#pragma unroll
        for (int i = 0; i < kBlkKeys * D / 8 / 32; ++i) {
            const int e = i * 32 + lane, r = e / (D / 8), c = e % (D / 8), j = t * kBlkKeys + r;
            const bool real = j < len;
            const uint32_t at = r * D * 2 + ((c ^ (r & 7)) * 16);
            cp_async16(dst + at, kb + (int64_t)(real ? j : 0) * p.st[4] + c * 8, real);
            cp_async16(dst + L::kBlock + at, vb + (int64_t)(real ? j : 0) * p.st[7] + c * 8, real);
        }
    };
    float o[D / 8][4] = {};
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int t_load = beg + warp, s_load = 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (t_load < end) load(t_load, s_load);
        asm volatile("cp.async.commit_group;" ::: "memory");
        t_load += kWarps;
        s_load = (s_load + 1) % kStages;
    }
    int st = 0;
    for (int t = beg + warp; t < end; t += kWarps) {
        if (t_load < end) load(t_load, s_load);
        asm volatile("cp.async.commit_group;" ::: "memory");
        t_load += kWarps;
        s_load = (s_load + 1) % kStages;
        // states of this block that count
        const int j0 = t * kBlkKeys;
        uint32_t on = len - j0 >= kBlkKeys ? 0xffffu : (1u << (len - j0)) - 1u;
        if (p.keys.key_mask) {
            const int j = j0 + (lane & 15);
            on &= __ballot_sync(0xffffffffu, j < len && p.keys.key_mask[(int64_t)b * p.keys.M + j] != 0);
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        const uint32_t ks = ring + st * 2 * L::kBlock, vs = ks + L::kBlock;
        st = (st + 1) % kStages;
        if (on == 0) continue;
        float s[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int r = (lane & 7) + ((lane >> 4) & 1) * 8, c = kk * 2 + ((lane >> 3) & 1);
            uint32_t f[4];
            ldsm4(ks + r * D * 2 + ((c ^ (r & 7)) * 16), f);
            mma16816(s[0], qf[kk], f[0], f[1]);
            mma16816(s[1], qf[kk], f[2], f[3]);
        }
        if (on != 0xffffu) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(on >> (n * 8 + (lane % 4) * 2 + (e & 1)) & 1)) s[n][e] = -INFINITY;
            // 0 * NaN is NaN: rows of V that do not count become zeros
            for (int r = 0; r < kBlkKeys; ++r)
                if (!(on >> r & 1) && lane < D / 8)
                    *reinterpret_cast<uint4*>(smem + (vs - smem_u32(smem)) + r * D * 2 + lane * 16) = make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
        uint32_t pf[4];
        bool moved = false;
        float alpha[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float mx = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[i], mx * p.scale_log2), base = mn == -INFINITY ? 0.f : mn;
            alpha[i] = mn == m[i] ? 1.f : ex2_mufu(m[i] - mn);
            moved |= mn != m[i];
            m[i] = mn;
            float w[4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) w[2 * n + e] = ex2_mufu(fmaf(s[n][2 * i + e], p.scale_log2, -base));
            l[i] = l[i] * alpha[i] + ((w[0] + w[1]) + (w[2] + w[3]));
            pf[i] = pack_bf16(w[0], w[1]);
            pf[2 + i] = pack_bf16(w[2], w[3]);
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                o[c][0] *= alpha[0];
                o[c][1] *= alpha[0];
                o[c][2] *= alpha[1];
                o[c][3] *= alpha[1];
            }
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            const int r = (lane & 7) + ((lane >> 3) & 1) * 8, ch = c * 2 + (lane >> 4);
            uint32_t f[4];
            ldsm4_t(vs + r * D * 2 + ((ch ^ (r & 7)) * 16), f);
            mma16816(o[2 * c], pf, f[0], f[1]);
            mma16816(o[2 * c + 1], pf, f[2], f[3]);
        }
        __syncwarp();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();                                                  // the rings become the join's space

    float* so = reinterpret_cast<float*>(smem);
    float* sm = reinterpret_cast<float*>(smem + L::offM);             // m, then l
    float* jo = reinterpret_cast<float*>(smem + L::offJoin);
    float* jm = jo + kRows * D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        const int r = lane / 4 + 8 * i;
        if (lane % 4 == 0) {
            sm[warp * kRows + r] = m[i];
            sm[kWarps * kRows + warp * kRows + r] = l[i];
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
            *reinterpret_cast<float2*>(so + (warp * kRows + r) * D + c * 8 + (lane % 4) * 2) =
                make_float2(o[c][2 * i], o[c][2 * i + 1]);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kRows * D; e += 32 * kWarps) {
        const int r = e / D;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm[w * kRows + r]);
        float a = 0.f, ll = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = sm[w * kRows + r], f = mw == -INFINITY ? 0.f : ex2_mufu(mw - mm);
            a += f * so[w * kRows * D + e];
            ll += f * sm[kWarps * kRows + w * kRows + r];
        }
        jo[e] = a;
        if (e % D == 0) {
            jm[r] = mm;
            jm[kRows + r] = ll;
        }
    }
    cluster.sync();
    const int share = kRows * D / splits + 1;
    for (int e = split * share + threadIdx.x; e < min((split + 1) * share, kRows * D); e += 32 * kWarps) {
        const int r = e / D, row = row0 + r;
        if (row >= rows) break;
        float mm = -INFINITY;
        for (int c = 0; c < splits; ++c) mm = fmaxf(mm, cluster.map_shared_rank(jm, c)[r]);
        float a = 0.f, ll = 0.f;
        for (int c = 0; c < splits; ++c) {
            const float* om = cluster.map_shared_rank(jm, c);
            const float f = om[r] == -INFINITY ? 0.f : ex2_mufu(om[r] - mm);
            a += f * cluster.map_shared_rank(jo, c)[e];
            ll += f * om[kRows + r];
        }
        const int n = row / p.G, h = hk * p.G + row % p.G;
        p.o[(((int64_t)b * p.N + n) * p.H + h) * D + e % D] = __float2bfloat16_rn(ll == 0.f ? 0.f : a / ll);
        if (p.lse && e % D == 0)
            p.lse[((int64_t)b * p.H + h) * p.N + n] = ll == 0.f ? -INFINITY : 0.69314718055994531f * (mm + log2f(ll));
    }
    cluster.sync();                                                   // no CTA leaves while another reads its results
}

template <int D>
cudaError_t launch_d(const FewP& prm, int splits, dim3 grid, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(k_cross_few<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewSmem<D>::kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = FewSmem<D>::kBytes;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_cross_few<D>, prm);
}

}  // namespace

cudaError_t launch_cross_few(const bsa_plan& p, const CrossArgs& a, void* o, float* lse, cudaStream_t s) {
    FewP prm;
    prm.q = (const __nv_bfloat16*)a.q; prm.k = (const __nv_bfloat16*)a.k; prm.v = (const __nv_bfloat16*)a.v;
    prm.o = (__nv_bfloat16*)o;
    prm.lse = lse;
    prm.keys = Keys{a.kv_len, a.key_mask, (int)a.M};
    for (int i = 0; i < 9; ++i) prm.st[i] = a.st[i];
    prm.N = (int)p.N; prm.H = p.H; prm.Hkv = a.Hkv; prm.G = p.H / a.Hkv;
    prm.scale_log2 = 1.4426950408889634f / sqrtf((float)p.d);
    const int tiles = (int)((p.N * prm.G + kRows - 1) / kRows), heads = p.B * a.Hkv;
    // two CTAs to an SM; a share of at least two blocks to a warp
    int splits = 1;
    while (splits < kMaxSplit && (int64_t)heads * tiles * splits * 2 <= 2 * p.num_sms &&
           a.M >= (int64_t)splits * 2 * kWarps * 2 * kBlkKeys)
        splits *= 2;
    const dim3 grid((unsigned)splits, (unsigned)tiles, (unsigned)heads);
    return p.d == 128 ? launch_d<128>(prm, splits, grid, s) : launch_d<64>(prm, splits, grid, s);
}

}  // namespace bsa
