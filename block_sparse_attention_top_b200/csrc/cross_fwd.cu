// Cross attention forward on the tensor cores (formula in bsa.h).
//
// One CTA per SM walks items of two 128-row query tiles of one head; both
// tiles use the same key tiles (128 keys), so K and V cross L2 once for 256
// query rows.  Q, K and V come by TMA straight from the caller's strided
// tensors, O leaves by TMA.
//
//   warps 0-3, 4-7  softmax of query tile 0, 1: a thread owns a row of S, its
//                   running maximum and sum; it also stores the row of O
//   warp 8          one thread issues every MMA:  ... PV0(t) QK0(t+1) PV1(t) QK1(t+1) ...
//   warp 9          one thread loads Q tiles and the K ring
//   warp 10         loads the V ring; in a tile with states that do not count
//                   it overwrites their rows with zeros (0 * NaN is NaN)
//
// TMEM: S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [384,384+D).  P_g (bf16)
// overwrites the first half of S_g: a thread has loaded its whole row of S
// before it stores P, and QK_g(t+1) is issued behind PV_g(t), which reads P.
// While one group exponentiates, the tensor cores work for the other.  When
// S_g(t) is complete so is PV_g(t-1), which was issued before it, so a group
// may rescale O_g without another barrier; it does so only when the maximum
// grows by more than 2^8.  Walking on from item to item, the MMA thread issues
// the next item's first QK_g behind this item's last PV_g, so the groups store
// O while the next scores are made.
//
// Waits are bounded as in attn_pp.cu.
#include <algorithm>

#include "cross_common.cuh"

namespace bsa {
namespace {

using namespace tc;
using namespace cross;

constexpr int kMmaWarp = 8, kKWarp = 9, kVWarp = 10;
constexpr int kThreads = 12 * 32;
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;   // tile g at + g * 128

template <int D>
struct Smem {
    static constexpr int kSlab = kTile * 128;                  // 128 rows x 64 columns
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kStages = D == 128 ? 2 : 4;           // of K and of V
    static constexpr int offQ = 0;
    static constexpr int offK = offQ + 2 * kTileBytes;
    static constexpr int offV = offK + kStages * kTileBytes;
    static constexpr int offOut = offV + kStages * kTileBytes; // 8 warps x 32 rows x 64 columns
    static constexpr int offBar = offOut + 8 * 4096;
    static constexpr int offMisc = offBar + 32 * 8;
    static constexpr int kAlloc = offMisc + 64 + 1024;         // room to align the base to 1024 B
};

struct FwdP {
    Keys keys;
    float* lse;
    int32_t* err;
    int N, H, G, tiles, per_item, units, items;   // units: items of one head
    float scale_log2;
    unsigned long long wait_ns;
};

struct Item {
    int b, h, tile, ng, len, nt;
};

__device__ __forceinline__ bool item_at(const FwdP& p, int k, Item& it) {
    const int idx = k * gridDim.x + blockIdx.x;
    if (idx >= p.items) return false;
    const int bh = idx / p.units;
    it.b = bh / p.H;
    it.h = bh % p.H;
    it.tile = (idx - bh * p.units) * p.per_item;
    it.ng = min(p.per_item, p.tiles - it.tile);
    it.len = p.keys.count(it.b);
    it.nt = (it.len + kTile - 1) / kTile;
    return true;
}

// The key tiles of this CTA's items, in the order every role walks them.
struct Walk {
    Item it;
    int k = 0, t = 0;
    bool ok;
    __device__ __forceinline__ void seek(const FwdP& p) {
        while ((ok = item_at(p, k, it)) && it.nt == 0) ++k;
    }
    __device__ __forceinline__ void open(const FwdP& p) { seek(p); }
    __device__ __forceinline__ void next(const FwdP& p) {
        if (++t < it.nt) return;
        t = 0;
        ++k;
        seek(p);
    }
};

template <int D, uint32_t kEvery>
__global__ void __launch_bounds__(kThreads, 1)
k_cross_fwd(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
            const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const FwdP prm) {
    using L = Smem<D>;
    enum {
        Q_FULL = 0, Q_EMPTY = 2, S_FULL = 4, P_FULL = 6, O_DONE = 8, V_RAW = 10, DRAIN = 11, K_FULL = 12,
        K_EMPTY = K_FULL + L::kStages, V_FULL = K_EMPTY + L::kStages, V_EMPTY = V_FULL + L::kStages,
        kBars = V_EMPTY + L::kStages
    };
    static_assert(kBars <= 32, "barrier slots");
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + L::offBar + 8u * (uint32_t)i; };
    volatile WaitCtl* ctl = reinterpret_cast<volatile WaitCtl*>(smem + L::offMisc);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::offMisc + 16);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        ctl->abort = 0;
        ctl->limit_ns = prm.wait_ns;
        for (int i = 0; i < kBars; ++i) mbar_init(bar(i), i == P_FULL || i == P_FULL + 1 ? 128 : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == kKWarp) {
        // ------------------------------------------------------- Q tiles and K ring
        if (lane == 0) {
            uint32_t u = 0, nq[2] = {0, 0};
            bool ok = true;
            Walk w;
            for (w.open(prm); w.ok && ok; w.next(prm), ++u) {
                if (w.t == 0)
                    for (int g = 0; g < w.it.ng && ok; ++g) {
                        if (nq[g] > 0 && !(ok = mbar_wait<kEvery>(bar(Q_EMPTY + g), (nq[g] - 1) & 1, ctl))) break;
                        mbar_expect_tx(bar(Q_FULL + g), L::kTileBytes);
                        for (int s = 0; s < D / 64; ++s)
                            tma_load_4d(sbase + L::offQ + g * L::kTileBytes + s * L::kSlab, &tmQ, s * 64,
                                        (w.it.tile + g) * kTile, w.it.h, w.it.b, bar(Q_FULL + g));
                        ++nq[g];
                    }
                if (!ok) break;
                const int st = u % L::kStages;
                if (u >= L::kStages && !(ok = mbar_wait<kEvery>(bar(K_EMPTY + st), (u / L::kStages - 1) & 1, ctl))) break;
                mbar_expect_tx(bar(K_FULL + st), L::kTileBytes);
                for (int s = 0; s < D / 64; ++s)
                    tma_load_4d(sbase + L::offK + st * L::kTileBytes + s * L::kSlab, &tmK, s * 64, w.t * kTile,
                                w.it.h / prm.G, w.it.b, bar(K_FULL + st));
            }
            if (!ok) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -1); }
            // every tile this thread issued lands before the CTA exits
            for (uint32_t st = 0; st < L::kStages; ++st)
                if (u > st) mbar_drain(bar(K_FULL + st), ((u - 1 - st) / L::kStages) & 1);
            for (int g = 0; g < 2; ++g)
                if (nq[g] > 0) mbar_drain(bar(Q_FULL + g), (nq[g] - 1) & 1);
        }
    } else if (warp == kVWarp) {
        // ------------------------------------------------------------------ V ring
        uint32_t u = 0, raw = 0;
        bool ok = true;
        Walk w;
        for (w.open(prm); w.ok; w.next(prm), ++u) {
            const int st = u % L::kStages;
            if (u >= L::kStages && !(ok = warp_wait<kEvery>(bar(V_EMPTY + st), (u / L::kStages - 1) & 1, ctl))) break;
            uint32_t bits[4];
            const bool all = prm.keys.bits(w.it.b, w.it.len, w.t * kTile, lane, bits);
            // rows past M are zero already: the copy fills them
            const bool fix = !all && (prm.keys.key_mask || w.it.len < prm.keys.M);
            const uint32_t full = bar(fix ? V_RAW : V_FULL + st);
            const uint32_t dst = sbase + L::offV + st * L::kTileBytes;
            if (lane == 0) {
                mbar_expect_tx(full, L::kTileBytes);
                for (int s = 0; s < D / 64; ++s)
                    tma_load_4d(dst + s * L::kSlab, &tmV, s * 64, w.t * kTile, w.it.h / prm.G, w.it.b, full);
            }
            if (fix) {
                const bool landed = warp_wait<kEvery>(full, raw & 1, ctl);
                if (!landed) {
                    mbar_drain(full, raw & 1);
                    ok = false;
                    break;
                }
                ++raw;
                for (int i = 0; i < kTile; ++i)                  // a row of a slab: 8 lanes of 16 bytes
                    if (!(bits[i / 32] >> (i % 32) & 1) && lane < D / 8)
                        *reinterpret_cast<uint4*>(smem + (dst - sbase) + (lane / 8) * L::kSlab + i * 128 +
                                                  (lane % 8) * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(V_FULL + st));
            }
        }
        if (!ok && lane == 0) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -2); }
        for (uint32_t st = 0; st < L::kStages; ++st)
            if (u > st) mbar_drain(bar(V_FULL + st), ((u - 1 - st) / L::kStages) & 1);
    } else if (warp == kMmaWarp) {
        // --------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc_qk = instr_desc(kTile, 0), idesc_pv = instr_desc(D, 1);
            uint32_t uk = 0, uv = 0, nq[2] = {0, 0}, np[2] = {0, 0};
            bool ok = true;
            // S_g = Q_g K^T of step w, whose K tile is number uk
            auto qk = [&](const Walk& w, int g) {
                if (w.t == 0) {
                    if (!mbar_wait<kEvery>(bar(Q_FULL + g), nq[g] & 1, ctl)) return false;
                    ++nq[g];
                }
                const int st = uk % L::kStages;
                if (!mbar_wait<kEvery>(bar(K_FULL + st), (uk / L::kStages) & 1, ctl)) return false;
                fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk / 4) * L::kSlab + (kk % 4) * 32;
                    mma_ss(tmem + kColS + g * 128, smem_desc(sbase + L::offQ + g * L::kTileBytes + off, 16, 1024),
                           smem_desc(sbase + L::offK + st * L::kTileBytes + off, 16, 1024), idesc_qk, kk > 0);
                }
                commit(bar(S_FULL + g));
                if (w.t == w.it.nt - 1) commit(bar(Q_EMPTY + g));
                return true;
            };
            Walk cur, nxt;
            cur.open(prm);
            if (cur.ok) {
                for (int g = 0; g < cur.it.ng && ok; ++g) ok = qk(cur, g);
                if (ok) commit(bar(K_EMPTY + uk % L::kStages));
                ++uk;
            }
            while (cur.ok && ok) {
                nxt = cur;
                nxt.next(prm);
                const int st = uv % L::kStages;
                for (int g = 0; g < 2 && ok; ++g) {
                    if (g < cur.it.ng) {
                        if (!(ok = mbar_wait<kEvery>(bar(P_FULL + g), np[g] & 1, ctl))) break;
                        ++np[g];
                        if (!(ok = mbar_wait<kEvery>(bar(V_FULL + st), (uv / L::kStages) & 1, ctl))) break;
                        fence_after();
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            mma_ts(tmem + kColO + g * 128, tmem + kColS + g * 128 + kk * 8,
                                   smem_desc(sbase + L::offV + st * L::kTileBytes + kk * 16 * 128, L::kSlab, 1024),
                                   idesc_pv, cur.t > 0 || kk > 0);
                        if (cur.t == cur.it.nt - 1) commit(bar(O_DONE + g));
                    }
                    if (nxt.ok && g < nxt.it.ng) ok = qk(nxt, g);
                }
                if (!ok) break;
                commit(bar(V_EMPTY + st));
                ++uv;
                if (nxt.ok) {
                    commit(bar(K_EMPTY + uk % L::kStages));
                    ++uk;
                }
                cur = nxt;
            }
            if (!ok) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -3); }
            commit(bar(DRAIN));                          // everything issued completes before TMEM is freed
            mbar_drain(bar(DRAIN), 0);
        }
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------------ softmax
        const int g = warp / 4, quad = warp & 3;
        const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
        const uint32_t ts = tmem + lane_base + kColS + g * 128, to = tmem + lane_base + kColO + g * 128;
        unsigned char* stage = smem + L::offOut + warp * 4096;
        const uint32_t stage_u32 = sbase + L::offOut + warp * 4096;
        uint32_t ns = 0, no = 0;
        bool ok = true;
        Item it;
        for (int k = 0; ok && item_at(prm, k, it); ++k) {
            if (g >= it.ng) continue;
            const int row0 = (it.tile + g) * kTile + 32 * quad;       // first query row of this warp
            float m = -INFINITY, l = 0.f;
            for (int t = 0; t < it.nt; ++t, ++ns) {
                uint32_t bits[4];
                const bool all = prm.keys.bits(it.b, it.len, t * kTile, lane, bits);
                if (!(ok = warp_wait<kEvery>(bar(S_FULL + g), ns & 1, ctl))) break;
                fence_after();
                uint32_t sv[kTile];
#pragma unroll
                for (int c = 0; c < kTile / 32; ++c) tmem_ld32(ts + c * 32, sv + 32 * c);
                tmem_wait_ld();
                if (!all) {
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        if (!(bits[c / 32] >> (c % 32) & 1)) sv[c] = __float_as_uint(-INFINITY);
                }
                const float mx = row_max<kTile>(sv, -INFINITY) * prm.scale_log2;
                // lazy maximum: P stays below 2^8
                const bool grow = t > 0 && mx > m + 8.f;
                const float alpha = grow ? ex2_mufu(m - mx) : 1.f;
                if (t == 0 || grow) m = mx;
                const float neg_m = m == -INFINITY ? 0.f : -m;        // no valid state so far
                float acc[8] = {};
                uint32_t pk[kTile / 2];
#pragma unroll
                for (int c = 0; c < kTile; c += 2) {
                    float x0, x1;
                    ffma2(x0, x1, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]), prm.scale_log2, prm.scale_log2,
                          neg_m, neg_m);
                    const float p0 = ex2_mufu(x0), p1 = ex2_mufu(x1);
                    const int u = (c / 2) & 3;
                    fadd2(acc[2 * u], acc[2 * u + 1], acc[2 * u], acc[2 * u + 1], p0, p1);
                    pk[c / 2] = pack_bf16(p0, p1);
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(to + c * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32(to + c * 32, o);
                    }
                }
#pragma unroll
                for (int c = 0; c < kTile / 64; ++c) tmem_st32(ts + c * 32, pk + 32 * c);
                l = l * alpha + (((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7])));
                tmem_wait_st();
                fence_before();
                mbar_arrive(bar(P_FULL + g));
            }
            if (!ok) break;
            // epilogue: O / l (zeros for a row without a valid state) through shared memory
            if (it.nt > 0) {
                if (!(ok = warp_wait<kEvery>(bar(O_DONE + g), no & 1, ctl))) break;
                ++no;
                fence_after();
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int n = row0 + lane;
            if (prm.lse && n < prm.N)
                prm.lse[((int64_t)it.b * prm.H + it.h) * prm.N + n] =
                    l == 0.f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
#pragma unroll
            for (int s = 0; s < D / 64; ++s) {
                uint32_t o[64];
                if (it.nt > 0) {
                    tmem_ld32(to + s * 64, o);
                    tmem_ld32(to + s * 64 + 32, o + 32);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 64; ++e) o[e] = 0u;
                }
                if (lane == 0) bulk_wait_read();                      // the slab before this one has left
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint4 v;
                    v.x = pack_bf16(__uint_as_float(o[8 * c + 0]) * inv, __uint_as_float(o[8 * c + 1]) * inv);
                    v.y = pack_bf16(__uint_as_float(o[8 * c + 2]) * inv, __uint_as_float(o[8 * c + 3]) * inv);
                    v.z = pack_bf16(__uint_as_float(o[8 * c + 4]) * inv, __uint_as_float(o[8 * c + 5]) * inv);
                    v.w = pack_bf16(__uint_as_float(o[8 * c + 6]) * inv, __uint_as_float(o[8 * c + 7]) * inv);
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) * 16)) = v;
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0 && row0 < prm.N) {
                    tma_store_4d(&tmO, stage_u32, s * 64, row0, it.h, it.b);
                    bulk_commit();
                }
            }
            fence_before();                                           // O was read: ordered before P of the next item
        }
        if (!ok) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -4); }
        tmem_wait_st();
        tmem_wait_ld();
        if (lane == 0) bulk_wait();
    }

    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int D, uint32_t kEvery>
cudaError_t launch_t(const bsa_plan& p, const CrossArgs& a, const FwdP& prm, void* o, cudaStream_t s) {
    using L = Smem<D>;
    CUtensorMap mq, mk, mv, mo;
    int64_t so[3];
    dense_strides(so, p.N, p.H, D);
    if (!make_map_4d(&mq, a.q, p.B, p.N, p.H, D, a.st, kTile) || !make_map_4d(&mk, a.k, p.B, a.M, a.Hkv, D, a.st + 3, kTile) ||
        !make_map_4d(&mv, a.v, p.B, a.M, a.Hkv, D, a.st + 6, kTile) || !make_map_4d(&mo, o, p.B, p.N, p.H, D, so, 32))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(k_cross_fwd<D, kEvery>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
    if (e != cudaSuccess) return e;
    k_cross_fwd<D, kEvery><<<std::min(p.num_sms, prm.items), kThreads, L::kAlloc, s>>>(mq, mk, mv, mo, prm);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const bsa_plan& p, const CrossArgs& a, const FwdP& prm, void* o, cudaStream_t s) {
    // a wait limit below a millisecond: the variant that checks it at every probe
    return prm.wait_ns < 1000000ull ? launch_t<D, 0>(p, a, prm, o, s) : launch_t<D, 1023>(p, a, prm, o, s);
}

}  // namespace

cudaError_t launch_cross_fwd_tc(const bsa_plan& p, const CrossArgs& a, void* o, float* lse, cudaStream_t s) {
    FwdP prm;
    prm.keys = Keys{a.kv_len, a.key_mask, (int)a.M};
    prm.lse = lse;
    prm.err = p.d_err;
    prm.N = (int)p.N;
    prm.H = p.H;
    prm.G = p.H / a.Hkv;
    prm.tiles = (int)((p.N + kTile - 1) / kTile);
    // two tiles to an item unless that leaves SMs without one
    prm.per_item = (int64_t)p.B * p.H * ((prm.tiles + 1) / 2) >= p.num_sms ? 2 : 1;
    prm.units = (prm.tiles + prm.per_item - 1) / prm.per_item;
    prm.items = p.B * p.H * prm.units;
    prm.scale_log2 = 1.4426950408889634f / sqrtf((float)p.d);
    prm.wait_ns = p.wait_ns;
    return p.d == 128 ? launch_d<128>(p, a, prm, o, s) : launch_d<64>(p, a, prm, o, s);
}

}  // namespace bsa
