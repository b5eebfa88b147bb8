// Cross attention forward on the tensor cores (formula in bsa.h).
//
// One CTA per SM walks items of two 128-row query tiles of one head; both
// tiles use the same key tiles (64 keys), so K and V cross L2 once for 256
// query rows.  Q, K and V come by TMA straight from the caller's strided
// tensors, O leaves by TMA.
//
//   warps 0-3, 4-7  softmax of query tile 0, 1: a thread owns a row of S, its
//                   running maximum and sum
//   warps 8-11      O / l to global memory, while the softmax warps are in the
//                   next item
//   warps 12, 13    MMAs of query tile 0, 1:  PV(t) QK(t+2)
//   warp 14         one thread loads Q tiles and the K ring
//   warp 15         loads the V ring; in a tile with states that do not count
//                   it overwrites their rows with zeros (0 * NaN is NaN)
//
// TMEM: two score buffers of 64 columns for each query tile, S0 [0,128)
// S1 [128,256), and O0 [256,256+D) O1 [384,384+D).  P(t) in bf16 overwrites the
// first half of S(t), columns its thread has read before.  The scores of tile
// t+1 are made while the softmax warps work on tile t, so those never wait for
// the tensor cores.  (With one buffer of 128 keys a group waited for PV and QK
// between tiles: 4200 cycles for 128 keys of both query tiles.)
// O_g is rescaled only when the maximum grows by more than 2^8; the softmax
// warp then waits for PV(t-1).
//
// Bound by the hand-offs between the softmax warps and the tensor cores: a
// step of 64 keys of both query tiles takes about 2 700 cycles (1.44 us),
// where its products take 1 280 and its exponentials 1 024 (one MUFU result a
// score; a share of them as polynomials on the FMA pipe cost 7 % more time).
// Measured, over several boxes: 75 600 tokens, 40 heads of 128, 512 states
// 0.92-0.96 ms, 823-861 TFLOP/s, 50-52 % of a bf16 GEMM's rate (the simple
// fp32 kernel that this one replaced took 129 ms); 32 760 tokens, 12 heads,
// 257 states 91-94 us.  Code size counts: each role is one loop body, not one
// per tile or parity.
//
// Waits are bounded as in attn_pp.cu.
#include <algorithm>

#include "cross_common.cuh"

namespace bsa {
namespace {

using namespace tc;
using namespace cross;

constexpr int kOutWarp = 8, kMmaWarp = 12, kKWarp = 14, kVWarp = 15;
constexpr int kThreads = 16 * 32;
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;   // tile g at + g * 128

template <int D>
struct Smem {
    static constexpr int kSlabQ = kTile * 128, kSlab = kKeys * 128;    // rows x 64 columns
    static constexpr int kQBytes = kTile * D * 2, kTileBytes = kKeys * D * 2;
    static constexpr int kStages = 4;                          // of K and of V
    static constexpr int offQ = 0;
    static constexpr int offK = offQ + 2 * kQBytes;
    static constexpr int offV = offK + kStages * kTileBytes;
    static constexpr int offOut = offV + kStages * kTileBytes; // 4 warps x 32 rows x 64 columns
    static constexpr int kOutBytes = 4096;
    // float l, m [4 items][2 tiles][128].  The softmax warps end item i + 2 once PV of item i has been issued (items of
    // one key tile), and its O may still be waiting for the output warps then: three items at a time.
    static constexpr int offSum = offOut + 4 * kOutBytes;
    static constexpr int kSumItems = 4;
    static constexpr int offBar = offSum + kSumItems * 2 * 2 * kTile * 4;
    static constexpr int offMisc = offBar + 40 * 8;
    static constexpr int kAlloc = offMisc + 64 + 1024;         // room to align the base to 1024 B
};

struct FwdP {
    Keys keys;
    float* lse;
    int32_t* err;
    int N, H, tiles, per_item, items;
    Div units, heads, G;             // items of one head; query heads; query heads of a key head
    float scale_log2;
    unsigned long long wait_ns;
};

struct Item {
    int b, h, tile, ng, len, nt;
};

__device__ __forceinline__ bool item_at(const FwdP& p, int k, Item& it) {
    const int idx = k * gridDim.x + blockIdx.x;
    if (idx >= p.items) return false;
    uint32_t rest = (uint32_t)idx;
    uint32_t bh = p.units.split(rest);
    it.tile = (int)rest * p.per_item;
    it.b = (int)p.heads.split(bh);
    it.h = (int)bh;
    it.ng = min(p.per_item, p.tiles - it.tile);
    it.len = p.keys.count(it.b);
    it.nt = (it.len + kKeys - 1) / kKeys;
    return true;
}

// The key tiles of this CTA's items, in the order every role walks them.
struct Walk {
    Item it;
    int k = -1, t = 0;
    bool ok = true;
    __device__ __forceinline__ Walk() { it.nt = 0; }
    __device__ __forceinline__ bool next(const FwdP& p) {
        if (++t < it.nt) return true;
        t = 0;
        do {
            ++k;
            ok = item_at(p, k, it);
        } while (ok && it.nt == 0);
        return ok;
    }
};

// 32 scores to 32 probabilities (16 bf16 pairs); adds them to acc.  (A polynomial on the FMA pipe for an eighth or a
// quarter of them measured 1 and 4 % slower: MUFU is busy a third of the time.)
__device__ __forceinline__ void exp_chunk(const uint32_t* x, float scale, float neg_m, float* acc, uint32_t* pk) {
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        float x0, x1;
        ffma2(x0, x1, __uint_as_float(x[c]), __uint_as_float(x[c + 1]), scale, scale, neg_m, neg_m);
        const float p0 = ex2_mufu(x0), p1 = ex2_mufu(x1);
        const int u = (c / 2) & 1;
        fadd2(acc[2 * u], acc[2 * u + 1], acc[2 * u], acc[2 * u + 1], p0, p1);
        pk[c / 2] = pack_bf16(p0, p1);
    }
}

// -inf where a state does not count
__device__ __forceinline__ void mask_cols(uint32_t* s, uint32_t bits) {
#pragma unroll
    for (int c = 0; c < 32; ++c)
        if (!(bits >> c & 1)) s[c] = __float_as_uint(-INFINITY);
}

template <int D, uint32_t kEvery>
__global__ void __launch_bounds__(kThreads, 1)
k_cross_fwd(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
            const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, const FwdP prm) {
    using L = Smem<D>;
    enum {
        Q_FULL = 0, Q_EMPTY = 2, S_FULL = 4, P_FULL = 8, PV_DONE = 12, O_DONE = 14, O_FREE = 16, DRAIN = 18, K_FULL = 20,
        K_EMPTY = K_FULL + L::kStages, V_FULL = K_EMPTY + L::kStages, V_EMPTY = V_FULL + L::kStages,
        V_RAW = V_EMPTY + L::kStages, kBars = V_RAW + L::kStages
    };
    static_assert(kBars <= 40, "barrier slots");
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + L::offBar + 8u * (uint32_t)i; };
    volatile WaitCtl* ctl = reinterpret_cast<volatile WaitCtl*>(smem + L::offMisc);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::offMisc + 16);
    float* sums = reinterpret_cast<float*>(smem + L::offSum);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        ctl->abort = 0;
        ctl->limit_ns = prm.wait_ns;
        for (int i = 0; i < kBars; ++i) {
            uint32_t count = 1;
            if ((i >= P_FULL && i < P_FULL + 4) || (i >= O_FREE && i < O_FREE + 2)) count = 4;      // warps
            if ((i >= K_EMPTY && i < V_FULL) || (i >= V_EMPTY && i < V_RAW)) count = 2;    // MMA threads
            mbar_init(bar(i), count);
        }
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
            for (; w.next(prm); ++u) {
                const int st = u % L::kStages;
                if (u >= L::kStages && !(ok = mbar_sleep<kEvery>(bar(K_EMPTY + st), (u / L::kStages - 1) & 1, ctl))) break;
                mbar_expect_tx(bar(K_FULL + st), L::kTileBytes);
                for (int s = 0; s < D / 64; ++s)
                    tma_load_4d(sbase + L::offK + st * L::kTileBytes + s * L::kSlab, &tmK, s * 64, w.t * kKeys,
                                (int)prm.G.quot(w.it.h), w.it.b, bar(K_FULL + st));
                if (w.t == 0)
                    for (int g = 0; g < w.it.ng && ok; ++g) {
                        if (nq[g] > 0 && !(ok = mbar_sleep<kEvery>(bar(Q_EMPTY + g), (nq[g] - 1) & 1, ctl))) break;
                        mbar_expect_tx(bar(Q_FULL + g), L::kQBytes);
                        for (int s = 0; s < D / 64; ++s)
                            tma_load_4d(sbase + L::offQ + g * L::kQBytes + s * L::kSlabQ, &tmQ, s * 64,
                                        (w.it.tile + g) * kTile, w.it.h, w.it.b, bar(Q_FULL + g));
                        ++nq[g];
                    }
                if (!ok) { ++u; break; }
                // The next item's Q, on its way to L2 while this item runs: a slab behind every K tile but the first
                // few, since a later load waits for the copies issued before it.
                Item n;
                if (w.t >= 2 && w.t < 2 + 2 * (D / 64) && item_at(prm, w.k + 1, n)) {
                    const int g = (w.t - 2) / (D / 64), s = (w.t - 2) % (D / 64);
                    if (g < n.ng) prefetch_4d(&tmQ, s * 64, (n.tile + g) * kTile, n.h, n.b);
                }
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
        struct {
            Walk w;
            const FwdP& p;
            __device__ __forceinline__ bool next() { return w.next(p); }
            __device__ __forceinline__ int b() const { return w.it.b; }
            __device__ __forceinline__ int head() const { return (int)p.G.quot(w.it.h); }
            __device__ __forceinline__ int len() const { return w.it.len; }
            __device__ __forceinline__ int t() const { return w.t; }
        } walk{Walk(), prm};
        if (!fill_ring<D, kKeys, L::kStages, 2, kEvery>(walk, prm.keys, &tmV, smem + L::offV, bar(V_FULL), bar(V_EMPTY), bar(V_RAW),
                                                ctl) && lane == 0) {
            ctl->abort = 1;
            record_error(prm.err, BSA_EDEVICE, -2);
        }
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        // -------------------------------------------------------------- MMA issuers
        // The whole warp walks and waits, so that descriptors stay in uniform registers; one lane issues.
        constexpr uint32_t idesc_qk = instr_desc(kKeys, 0), idesc_pv = instr_desc(D, 1);
        const int g = __shfl_sync(0xffffffffu, warp, 0) - kMmaWarp;
        const uint32_t ts = tmem + kColS + g * 128, to = tmem + kColO + g * 128;
        const uint32_t q_tile = sbase + L::offQ + g * L::kQBytes;
        uint32_t uk = 0, uv = 0, sk = 0, sp = 0, nq = 0, no = 0;   // ring tiles; this group's S, P, Q, O
        bool ok = true;
        // K tile uk of step w, and Q_g with an item's first, have landed
        auto qk_ready = [&](const Walk& w) {
            return warp_wait<kEvery>(bar(K_FULL + uk % L::kStages), (uk / L::kStages) & 1, ctl) &&
                   (w.t > 0 || g >= w.it.ng || warp_wait<kEvery>(bar(Q_FULL + g), nq++ & 1, ctl));
        };
        const uint64_t dq = smem_desc(q_tile, 16, 1024), dk = smem_desc(sbase + L::offK, 16, 1024),
                       dv = smem_desc(sbase + L::offV, L::kSlab, 1024);
        Walk cur, ahead;                                 // ahead: the step whose scores are made next
        cur.next(prm);
        ahead.next(prm);
        for (int made = 0; made > 0 || ahead.ok;) {      // scores made and not yet used
            const bool pv = made == 2 || !ahead.ok, more = ahead.ok;
            const int sv = uv % L::kStages, sq = uk % L::kStages;
            const bool pv_g = pv && g < cur.it.ng, qk_g = more && g < ahead.it.ng;
            // everything but P first
            if (more && !(ok = qk_ready(ahead))) break;
            if (pv && !(ok = warp_wait<kEvery>(bar(V_FULL + sv), (uv / L::kStages) & 1, ctl))) break;
            if (pv_g) {
                // the item before this one has been read out of O_g
                if (cur.t == 0 && no++ > 0 && !(ok = warp_wait<kEvery>(bar(O_FREE + g), no & 1, ctl))) break;
                if (!(ok = warp_wait<kEvery>(bar(P_FULL + 2 * g + (sp & 1)), (sp >> 1) & 1, ctl))) break;
            }
            fence_after();
            if (elect_one()) {
                if (pv_g) {
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk)
                        mma_ts(to, ts + (sp & 1) * kKeys + kk * 8, desc_at(dv, sv * L::kTileBytes + kk * 16 * 128), idesc_pv,
                               cur.t > 0 || kk > 0);
                    commit(bar(PV_DONE + g));
                    commit(bar(V_EMPTY + sv));
                    if (cur.t == cur.it.nt - 1) commit(bar(O_DONE + g));
                } else if (pv) {
                    mbar_arrive(bar(V_EMPTY + sv));
                }
                if (qk_g) {                              // S[sk & 1] = Q_g K^T
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ss(ts + (sk & 1) * kKeys, desc_at(dq, (kk / 4) * L::kSlabQ + (kk % 4) * 32),
                               desc_at(dk, sq * L::kTileBytes + (kk / 4) * L::kSlab + (kk % 4) * 32), idesc_qk, kk > 0);
                    commit(bar(S_FULL + 2 * g + (sk & 1)));
                    commit(bar(K_EMPTY + sq));
                    if (ahead.t == ahead.it.nt - 1) commit(bar(Q_EMPTY + g));
                } else if (more) {                       // a step without this query tile passes the stage on
                    mbar_arrive(bar(K_EMPTY + sq));
                }
            }
            __syncwarp();
            if (pv) {
                sp += pv_g;
                ++uv;
                --made;
                cur.next(prm);
            }
            if (more) {
                sk += qk_g;
                ++uk;
                ++made;
                ahead.next(prm);
            }
        }
        if (!ok && lane == 0) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -3); }
        if (elect_one()) {
            commit(bar(DRAIN + g));                      // everything issued completes before TMEM is freed
            mbar_drain(bar(DRAIN + g), 0);
        }
        __syncwarp();
    } else if (warp < kOutWarp) {
        // ------------------------------------------------------------------ softmax
        const int g = warp / 4, quad = warp & 3;
        const uint32_t lane_base = (uint32_t)(32 * quad) << 16;
        const uint32_t ts = tmem + lane_base + kColS + g * 128, to = tmem + lane_base + kColO + g * 128;
        uint32_t ns = 0, done = 0;
        bool ok = true;
        Item it;
        for (int k = 0; ok && item_at(prm, k, it); ++k) {
            if (g >= it.ng || it.nt == 0) continue;
            float m = -INFINITY, l = 0.f;
            for (int t = 0; t < it.nt; ++t, ++ns) {
                const uint32_t tsb = ts + (ns & 1) * kKeys;
                uint32_t bits[2];
                const bool all = prm.keys.bits(it.b, it.len, t * kKeys, lane, bits);
                if (!(ok = warp_wait<kEvery>(bar(S_FULL + 2 * g + (ns & 1)), (ns >> 1) & 1, ctl))) break;
                fence_after();
                uint32_t sv[kKeys];
                tmem_ld32(tsb, sv);
                tmem_ld32(tsb + 32, sv + 32);
                tmem_wait_ld();
                if (!all) {
                    mask_cols(sv, bits[0]);
                    mask_cols(sv + 32, bits[1]);
                }
                const float mx = row_max<kKeys>(sv, -INFINITY) * prm.scale_log2;
                // lazy maximum: P stays below 2^8
                const bool grow = t > 0 && mx > m + 8.f;
                const float alpha = grow ? ex2_mufu(m - mx) : 1.f;
                if (t == 0 || grow) m = mx;
                const float neg_m = m == -INFINITY ? 0.f : -m;        // no valid state so far
                float acc[4] = {};
                uint32_t pk[kKeys / 2];
                exp_chunk(sv, prm.scale_log2, neg_m, acc, pk);
                tmem_st16(tsb, pk);
                exp_chunk(sv + 32, prm.scale_log2, neg_m, acc, pk + 16);
                tmem_st16(tsb + 16, pk + 16);
                l = l * alpha + ((acc[0] + acc[1]) + (acc[2] + acc[3]));
                if (__any_sync(0xffffffffu, grow)) {
                    // PV(t-1) is the tile before this one; PV(t-2) was complete before S(t) was, so the parity is exact
                    if (!(ok = warp_wait<kEvery>(bar(PV_DONE + g), (ns - 1) & 1, ctl))) break;
                    fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        tmem_ld32(to + c, sv);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) sv[e] = __float_as_uint(__uint_as_float(sv[e]) * alpha);
                        tmem_st32(to + c, sv);
                    }
                }
                if (t == it.nt - 1) {                                 // for the output warps
                    float* slot = sums + ((done % L::kSumItems) * 2 + g) * 2 * kTile + 32 * quad + lane;
                    slot[0] = l;
                    slot[kTile] = m;
                    ++done;
                }
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(P_FULL + 2 * g + (ns & 1)));
            }
        }
        if (!ok) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -4); }
        __syncwarp();
        tmem_wait_st();
        tmem_wait_ld();
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------------- output
        const int quad = warp & 3;
        const uint32_t to = tmem + ((uint32_t)(32 * quad) << 16) + kColO;
        unsigned char* stage = smem + L::offOut + quad * L::kOutBytes;
        uint32_t done[2] = {0, 0};
        bool ok = true;
        Item it;
        for (int k = 0; ok && item_at(prm, k, it); ++k)
            for (int g = 0; g < it.ng; ++g) {
                const int row0 = (it.tile + g) * kTile + 32 * quad, n = row0 + lane;
                float l = 0.f, m = -INFINITY;
                if (it.nt > 0) {
                    // the last PV is complete, so its P and with it l and m were written before
                    if (!(ok = warp_sleep<kEvery>(bar(O_DONE + g), done[g] & 1, ctl))) break;
                    fence_after();
                    const float* slot = sums + ((done[g] % L::kSumItems) * 2 + g) * 2 * kTile + 32 * quad + lane;
                    l = slot[0];
                    m = slot[kTile];
                    ++done[g];
                }
                // No valid state: zeros.  Told by the sum, which is at least about 1 otherwise; the maximum drops NaN, and
                // a row of NaN must stay NaN.
                const bool empty = l == 0.f;
                const float inv = empty ? 0.f : 1.f / l;
                if (prm.lse && n < prm.N)
                    prm.lse[((int64_t)it.b * prm.H + it.h) * prm.N + n] =
                        empty ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
#pragma unroll 1
                for (int s = 0; s < D / 64; ++s) {
                    uint32_t o[64];
                    __syncwarp();                                     // tmem_ld takes the whole warp
                    if (it.nt > 0) {
                        tmem_ld32(to + g * 128 + s * 64, o);
                        tmem_ld32(to + g * 128 + s * 64 + 32, o + 32);
                        tmem_wait_ld();
                        if (s == D / 64 - 1) {                        // O_g may take the next item
                            fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar(O_FREE + g));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 64; ++e) o[e] = 0u;
                    }
                    if (lane == 0) bulk_wait_read();                  // the slab before this one has left
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
                        tma_store_4d(&tmO, smem_u32(stage), s * 64, row0, it.h, it.b);
                        bulk_commit();
                    }
                }
            }
        if (!ok) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -5); }
        __syncwarp();
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
    if (!make_map_4d(&mq, a.q, p.B, p.N, p.H, D, a.st, kTile) || !make_map_4d(&mk, a.k, p.B, a.M, a.Hkv, D, a.st + 3, kKeys) ||
        !make_map_4d(&mv, a.v, p.B, a.M, a.Hkv, D, a.st + 6, kKeys) || !make_map_4d(&mo, o, p.B, p.N, p.H, D, so, 32))
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
    prm.heads = Div(p.H);
    prm.G = Div(p.H / a.Hkv);
    prm.tiles = (int)((p.N + kTile - 1) / kTile);
    // two tiles to an item unless that leaves SMs without one
    prm.per_item = (int64_t)p.B * p.H * ((prm.tiles + 1) / 2) >= p.num_sms ? 2 : 1;
    const int units = (prm.tiles + prm.per_item - 1) / prm.per_item;
    prm.units = Div(units);
    prm.items = p.B * p.H * units;
    prm.scale_log2 = 1.4426950408889634f / sqrtf((float)p.d);
    prm.wait_ns = p.wait_ns;
    return p.d == 128 ? launch_d<128>(p, a, prm, o, s) : launch_d<64>(p, a, prm, o, s);
}

}  // namespace bsa
