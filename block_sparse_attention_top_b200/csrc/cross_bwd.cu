// Gradient of the cross attention on the tensor cores (formulas in bsa.h).
//
// Two passes, each of which keeps its sums in TMEM and needs no atomics, so
// the same inputs give the same bits:
//   k_cross_dq   a CTA owns a query tile and walks the keys:
//                S = Q K^T, dP = dO V^T, dS = P * (dP - D), dQ += dS K;
//   k_cross_dkv  a CTA owns a key tile and walks a share of the query tokens:
//                S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.
// Making S and dP twice costs two more products than one pass would, 7 for 5,
// but one pass would have to add dQ tiles (fp32, once for every key tile) in
// memory: more traffic than the two products take time, and an order that
// depends on scheduling.  A third kernel adds the key side's shares in order.
//
// Both passes work in tiles of 64 on the side they walk, with two buffers of
// S and dP in TMEM.  Each of the softmax warps 0-3 and 4-7 takes half of every
// tile's columns, a thread per row of the owned side (lse and D are given);
// P and dS (bf16) overwrite the columns that their thread has read, so the A
// operand of a product is two runs of 16 columns.
// The tensor cores make S and dP of tile u+2 behind the products that read
// tile u.  (Taking turns, each group a whole tile, the softmax of a tile took
// 1500 cycles, longer than the tensor cores' 1400 for the tile between.)
//
// D comes from the bf16 O, off by up to 2^-8 of the terms it sums; where a few
// states hold nearly all of P that error is as large as dP - D itself.  For
// the exact D a row of dS sums to 0, so the sum that is left is the error:
// k_cross_dq takes it out of its own dS where all states fit one tile, and
// always out of the D that k_cross_dkv reads.
//
// Bound by the softmax warps' and the tensor cores' taking turns on a tile.
// Measured with 32 760 tokens, 12 heads of 128, 512 states: k_cross_dq 185 us,
// k_cross_dkv 200, the sum of shares 8 (five products at a GEMM's rate:
// 156 us).  Both kernels were held back by their code first: at 120 KB the
// instruction caches were busy 87 % of the time, at 33 KB 2 %.
//
// Waits are bounded as in attn_pp.cu.
#include <algorithm>

#include "cross_common.cuh"

namespace bsa {
namespace {

using namespace tc;
using namespace cross;

constexpr int kRowWarp = 8, kMmaWarp = 12, kPollWarp = 13;
constexpr int kThreads = 16 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

// Address of 16-byte chunk c of row r in a tile of 64-column slabs with 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int r, int c, int slab_bytes) {
    return (uint32_t)((c / 8) * slab_bytes + r * 128 + (((c % 8) ^ (r & 7)) * 16));
}
__device__ __forceinline__ float dot8(uint4 a, uint4 b) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s += __uint_as_float(x[i] << 16) * __uint_as_float(y[i] << 16) +
             __uint_as_float(x[i] & 0xffff0000u) * __uint_as_float(y[i] & 0xffff0000u);
    return s;
}

// Shared prologue: barriers, TMEM.  Shared epilogue: TMEM.
template <int kBars, typename Count>
__device__ __forceinline__ uint32_t begin_cta(uint32_t bar0, volatile WaitCtl* ctl, uint32_t* tmem_slot,
                                              unsigned long long wait_ns, Count count) {
    if (threadIdx.x == 0) {
        ctl->abort = 0;
        ctl->limit_ns = wait_ns;
        for (int i = 0; i < kBars; ++i) mbar_init(bar0 + 8 * i, count(i));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x / 32 == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    return *tmem_slot;
}
__device__ __forceinline__ void end_cta(uint32_t tmem) {
    fence_before();
    __syncthreads();
    fence_after();
    if (threadIdx.x / 32 == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------------ query side
// warps 0-7 softmax, 8-11 rows (the next item's Q, dO and D, then dQ to
// memory), 12 MMA, 13 polls for it, 14 K ring, 15 V ring.  Q and dO go to TMEM (tcgen05.cp), so that S and dP
// read only K and V from shared memory.
struct DqP {
    Keys keys;
    const __nv_bfloat16 *o, *d_o;
    const float* lse;
    float* dsum;
    int32_t* err;
    int N, H, items;
    Div tiles, heads, G;             // query tiles of a head; query heads; query heads of a key head
    float scale, scale_log2;
    unsigned long long wait_ns;
};

template <int D>
struct DqSmem {
    static constexpr int kSlabQ = kTile * 128, kSlab = kKeys * 128;
    static constexpr int kQBytes = kTile * D * 2, kTileBytes = kKeys * D * 2;
    static constexpr int kStages = 4, kStagesV = 3;                // a K tile is used once more than a V tile
    static constexpr int offQ = 0;                                 // Q, dO
    static constexpr int offK = offQ + 2 * kQBytes;
    static constexpr int offV = offK + kStages * kTileBytes;
    static constexpr int kOutBytes = 32 * D * 2;
    static constexpr int offOut = offV + kStagesV * kTileBytes;    // 4 warps x 32 rows x D columns
    static constexpr int offRows = offOut + 4 * kOutBytes;         // float lse, D [2 items][128]
    static constexpr int offHalves = offRows + 2 * 2 * kTile * 4;  // float sums of dS [2 items][2 halves][128]
    static constexpr int offBar = offHalves + 2 * 2 * kTile * 4;
    static constexpr int offMisc = offBar + 48 * 8;
    static constexpr int kAlloc = offMisc + 64 + 1024;
    static constexpr uint32_t colS = 0, colDP = 128, colQ = 256, colDO = 256 + D / 2, colDQ = 384;
};

struct DqItem {
    int b, h, tile, len, nt;
};
__device__ __forceinline__ bool item_at(const DqP& p, int k, DqItem& it) {
    const int idx = k * gridDim.x + blockIdx.x;
    if (idx >= p.items) return false;
    uint32_t tile = (uint32_t)idx, h = p.tiles.split(tile);
    it.tile = (int)tile;
    it.b = (int)p.heads.split(h);
    it.h = (int)h;
    it.len = p.keys.count(it.b);
    it.nt = (it.len + kKeys - 1) / kKeys;
    return true;
}
struct DqWalk {
    DqItem it;
    int k = -1, t = 0, nth = -1;     // nth: which of the items with keys
    bool ok = true;
    __device__ __forceinline__ DqWalk() { it.nt = 0; }
    __device__ __forceinline__ bool next(const DqP& p) {
        if (++t < it.nt) return true;
        return next_item(p);
    }
    __device__ __forceinline__ bool next_item(const DqP& p) {
        t = 0;
        do {
            ++k;
            ok = item_at(p, k, it);
        } while (ok && it.nt == 0);
        ++nth;
        return ok;
    }
    __device__ __forceinline__ bool last() const { return t == it.nt - 1; }
};

template <int D, uint32_t kEvery>
__global__ void __launch_bounds__(kThreads, 1)
k_cross_dq(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
           const __grid_constant__ CUtensorMap tmDQ, const DqP prm) {
    using L = DqSmem<D>;
    enum {
        QD_FULL = 0, QD_EMPTY, AB_FREE, S_FULL, DS_FULL = S_FULL + 2, ROWS_FULL = DS_FULL + 2, ROWS_EMPTY = ROWS_FULL + 2,
        DQ_DONE = ROWS_EMPTY + 2, DQ_FREE, DRAIN, K_FULL, K_EMPTY = K_FULL + L::kStages,
        V_FULL = K_EMPTY + L::kStages, V_EMPTY = V_FULL + L::kStagesV, K_RAW = V_EMPTY + L::kStagesV,
        kBars = K_RAW + L::kStages
    };
    static_assert(kBars <= 48, "barrier slots");
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + L::offBar + 8u * (uint32_t)i; };
    volatile WaitCtl* ctl = reinterpret_cast<volatile WaitCtl*>(smem + L::offMisc);
    float* row_vals = reinterpret_cast<float*>(smem + L::offRows);
    float* halves = reinterpret_cast<float*>(smem + L::offHalves);
    const uint32_t tmem = begin_cta<kBars>(bar(0), ctl, reinterpret_cast<uint32_t*>(smem + L::offMisc + 16), prm.wait_ns,
                                           [](int i) -> uint32_t {
                                               if ((i >= DS_FULL && i < DS_FULL + 2) || (i >= ROWS_EMPTY && i < ROWS_EMPTY + 2)) return 8;
                                               if ((i >= ROWS_FULL && i < ROWS_FULL + 2) || i == DQ_FREE) return 4;
                                               return 1;
                                           });
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    bool ok = true;
    auto wait_full = [&](uint32_t b, uint32_t parity) { return warp_wait<kEvery>(b, parity, ctl); };

    if (warp == kMmaWarp) {
        constexpr uint32_t idesc_s = instr_desc(kKeys, 0), idesc_dq = instr_desc(D, 1);
        const uint64_t dk = smem_desc(sbase + L::offK, 16, 1024), dv = smem_desc(sbase + L::offV, 16, 1024),
                       dk_mn = smem_desc(sbase + L::offK, L::kSlab, 1024), dqd = smem_desc(sbase + L::offQ, 16, 1024);
        uint32_t ua = 0, uc = 0;                                  // steps: scores made, dQ added
        // ahead: the step whose scores are made next, at most in the item after cur's: an item's Q and dO come while the
        // one before it is added up, so the second item after cur's waits for cur's dQ
        DqWalk cur, ahead;
        bool use = true, more = true;
        for (int made = 0;;) {                                    // scores made and not yet used
            if (more) ahead.next(prm);
            if (use) cur.next(prm);
            if (made == 0 && !ahead.ok) break;
            use = made == 2 || !ahead.ok;
            more = ahead.ok && ahead.nth - cur.nth < 2;
            if (!(ok = meet(true))) break;
            fence_after();
            if (elect_one()) {
                if (use) {
                    const uint32_t st = uc % L::kStages;
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk)
                        mma_ts(tmem + L::colDQ, tmem + L::colS + (uc & 1) * kKeys + (kk / 2) * 32 + (kk % 2) * 8,
                               desc_at(dk_mn, st * L::kTileBytes + kk * 16 * 128), idesc_dq, cur.t > 0 || kk > 0);
                    commit(bar(K_EMPTY + st));
                    if (cur.last()) commit(bar(DQ_DONE));
                }
                if (more) {
                    const uint32_t st = ua % L::kStages, sv = ua % L::kStagesV, buf = (ua & 1) * kKeys;
                    if (ahead.t == 0) {                           // the item's Q and dO to TMEM
#pragma unroll 1
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = (kk / 4) * L::kSlabQ + (kk % 4) * 32;
                            cp_128x256b(tmem + L::colQ + kk * 8, desc_at(dqd, off));
                            cp_128x256b(tmem + L::colDO + kk * 8, desc_at(dqd, L::kQBytes + off));
                        }
                        commit(bar(QD_EMPTY));
                    }
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk / 4) * L::kSlab + (kk % 4) * 32;
                        mma_ts(tmem + L::colS + buf, tmem + L::colQ + kk * 8, desc_at(dk, st * L::kTileBytes + off), idesc_s,
                               kk > 0);
                        mma_ts(tmem + L::colDP + buf, tmem + L::colDO + kk * 8, desc_at(dv, sv * L::kTileBytes + off),
                               idesc_s, kk > 0);
                    }
                    commit(bar(S_FULL + (ua & 1)));
                    commit(bar(V_EMPTY + sv));
                    if (ahead.last()) commit(bar(AB_FREE));
                }
            }
            __syncwarp();
            uc += use;
            ua += more;
            made += (int)more - (int)use;
        }
        if (elect_one()) {
            commit(bar(DRAIN));
            mbar_drain(bar(DRAIN), 0);
        }
        __syncwarp();
    } else if (warp == kPollWarp) {
        // what each of the MMA warp's steps waits for
        uint32_t ua = 0, uc = 0, items_a = 0, items_c = 0;
        DqWalk cur, ahead;
        bool use = true, more = true;
        for (int made = 0;;) {
            if (more) ahead.next(prm);
            if (use) cur.next(prm);
            if (made == 0 && !ahead.ok) break;
            use = made == 2 || !ahead.ok;
            more = ahead.ok && ahead.nth - cur.nth < 2;
            bool go = true;
            if (more) {
                go = warp_wait<kEvery>(bar(K_FULL + ua % L::kStages), (ua / L::kStages) & 1, ctl) &&
                     warp_wait<kEvery>(bar(V_FULL + ua % L::kStagesV), (ua / L::kStagesV) & 1, ctl);
                // Q and dO have landed, and the item before has made its last scores (a copy into TMEM is not ordered
                // behind the products that read the same columns)
                if (ahead.t == 0) {
                    go = go && (items_a == 0 || warp_wait<kEvery>(bar(AB_FREE), (items_a - 1) & 1, ctl)) &&
                         warp_wait<kEvery>(bar(QD_FULL), items_a & 1, ctl);
                    ++items_a;
                }
                ++ua;
            }
            if (use) {
                // dQ of the item before this one has been read
                if (cur.t == 0 && items_c++ > 0) go = go && warp_wait<kEvery>(bar(DQ_FREE), items_c & 1, ctl);
                go = go && warp_wait<kEvery>(bar(DS_FULL + (uc & 1)), (uc >> 1) & 1, ctl);
                ++uc;
            }
            if (!(ok = meet(go))) break;
            made += (int)more - (int)use;
        }
        if (!ok && lane == 0) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -3); }
    } else if (warp == kPollWarp + 1) {
        // K ring: dQ += dS K, so rows of states that do not count are zeroed.  S of tile u + 2 is made before tile u is
        // used up, hence the lag of one.
        struct {
            DqWalk w;
            const DqP& p;
            __device__ __forceinline__ bool next() { return w.next(p); }
            __device__ __forceinline__ int b() const { return w.it.b; }
            __device__ __forceinline__ int head() const { return (int)p.G.quot(w.it.h); }
            __device__ __forceinline__ int len() const { return w.it.len; }
            __device__ __forceinline__ int t() const { return w.t; }
        } walk{DqWalk(), prm};
        if (!fill_ring<D, kKeys, L::kStages, 1, kEvery>(walk, prm.keys, &tmK, smem + L::offK, bar(K_FULL), bar(K_EMPTY), bar(K_RAW),
                                                ctl) && lane == 0) {
            ctl->abort = 1;
            record_error(prm.err, BSA_EDEVICE, -1);
        }
    } else if (warp == kPollWarp + 2) {
        if (lane == 0) {
            uint32_t u = 0;
            DqWalk w;
            for (; w.next(prm); ++u) {
                const int st = u % L::kStagesV;
                if (u >= L::kStagesV && !(ok = mbar_sleep<kEvery>(bar(V_EMPTY + st), (u / L::kStagesV - 1) & 1, ctl))) break;
                mbar_expect_tx(bar(V_FULL + st), L::kTileBytes);
                for (int s = 0; s < D / 64; ++s)
                    tma_load_4d(sbase + L::offV + st * L::kTileBytes + s * L::kSlab, &tmV, s * 64, w.t * kKeys,
                                (int)prm.G.quot(w.it.h), w.it.b, bar(V_FULL + st));
            }
            if (!ok) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -2); }
            for (uint32_t st = 0; st < L::kStagesV; ++st)
                if (u > st) mbar_drain(bar(V_FULL + st), ((u - 1 - st) / L::kStagesV) & 1);
        }
    } else if (warp < kRowWarp) {
        // ------------------------------------------------------------------ softmax
        const int g = warp / 4, quad = warp & 3;                  // columns [32 g, 32 g + 32) of every tile
        const uint32_t ts0 = tmem + ((uint32_t)(32 * quad) << 16) + L::colS + g * 32;
        uint32_t u = 0, ni = 0;
        DqItem it;
        // Both warps of a row leave together: one that has given up says so at the other's next exchange, and every
        // item has exactly one.
        auto give_up = [&] {
            meet(false, 2 + quad);
            ok = false;
        };
        for (int k = 0; ok && item_at(prm, k, it); ++k) {
            if (it.nt == 0) continue;
            if (!wait_full(bar(ROWS_FULL + (ni & 1)), (ni >> 1) & 1)) {
                give_up();
                break;
            }
            const float* rv = row_vals + (ni & 1) * 2 * kTile + 32 * quad + lane;
            const float neg_lse = -rv[0];
            float neg_d = -rv[kTile], sum = 0.f;                      // sum: of this half's dS so far
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(ROWS_EMPTY + (ni & 1)));
            float* mine = halves + ((ni & 1) * 2 + g) * kTile + 32 * quad + lane;
            const float* theirs = halves + ((ni & 1) * 2 + 1 - g) * kTile + 32 * quad + lane;
            ++ni;
            // D from the rounded o is off by what dS sums to over all states (0 for the exact D)
            auto correct = [&] {
                *mine = sum;
                if (!meet(true, 2 + quad)) return false;
                neg_d -= sum + *theirs;
                return true;
            };
            for (int t = 0; t < it.nt && ok; ++t, ++u) {
                const uint32_t ts = ts0 + (u & 1) * kKeys, tp = ts - L::colS + L::colDP;
                uint32_t bits[2];
                prm.keys.bits(it.b, it.len, t * kKeys, lane, bits);
                const uint32_t word = g ? bits[1] : bits[0];
                if (!wait_full(bar(S_FULL + (u & 1)), (u >> 1) & 1)) {
                    give_up();
                    break;
                }
                fence_after();
                uint32_t sv[32], dv[32], pk[16];
                tmem_ld32(ts, sv);
                tmem_ld32(tp, dv);
                tmem_wait_ld();
                if (word != 0xffffffffu) {                            // P = 0, dS = 0
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        sv[e] = word >> e & 1 ? sv[e] : __float_as_uint(-INFINITY);
                        dv[e] = word >> e & 1 ? dv[e] : 0u;
                    }
                }
                // one tile holds all states: its dS with the corrected D
#pragma unroll 1
                for (int pass = it.nt == 1 ? 0 : 1; pass < 2; ++pass) {
                    float acc[4] = {};
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float x0, x1, d0, d1;
                        ffma2(x0, x1, __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]), prm.scale_log2, prm.scale_log2,
                              neg_lse, neg_lse);
                        fadd2(d0, d1, __uint_as_float(dv[e]), __uint_as_float(dv[e + 1]), neg_d, neg_d);
                        const float p0 = ex2_mufu(x0), p1 = ex2_mufu(x1);
                        fmul2(d0, d1, d0, d1, p0, p1);
                        fadd2(acc[e & 2], acc[(e & 2) + 1], acc[e & 2], acc[(e & 2) + 1], d0, d1);
                        pk[e / 2] = pack_bf16(d0, d1);
                    }
                    sum += (acc[0] + acc[1]) + (acc[2] + acc[3]);
                    if (pass == 0 && !(ok = correct())) break;
                }
                if (!ok) break;
                tmem_st16(ts, pk);
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(DS_FULL + (u & 1)));
            }
            if (!ok || (it.nt > 1 && !(ok = correct()))) break;
            const int n = it.tile * kTile + 32 * quad + lane;
            if (g == 0 && n < prm.N) prm.dsum[((int64_t)it.b * prm.H + it.h) * prm.N + n] = -neg_d;
        }
        if (!ok) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -4); }
        __syncwarp();
        tmem_wait_st();
        tmem_wait_ld();
    } else {
        // --------------------------------------------- rows: D ahead of the item, dQ behind it
        const int quad = warp & 3, r = 32 * quad + lane;
        const uint32_t tq = tmem + ((uint32_t)(32 * quad) << 16) + L::colDQ;
        unsigned char* stage = smem + L::offOut + quad * L::kOutBytes;
        uint32_t nr = 0, nd = 0, nl = 0;
        // Q and dO of an item, once the copies of the one before have read theirs
        auto load = [&](const DqItem& it) {
            if (warp != kRowWarp) return true;
            if (nl > 0 && !warp_sleep<kEvery>(bar(QD_EMPTY), (nl - 1) & 1, ctl)) return false;
            ++nl;
            if (lane == 0) {
                mbar_expect_tx(bar(QD_FULL), 2 * L::kQBytes);
                for (int s = 0; s < D / 64; ++s) {
                    tma_load_4d(sbase + L::offQ + s * L::kSlabQ, &tmQ, s * 64, it.tile * kTile, it.h, it.b, bar(QD_FULL));
                    tma_load_4d(sbase + L::offQ + L::kQBytes + s * L::kSlabQ, &tmDO, s * 64, it.tile * kTile, it.h, it.b,
                                bar(QD_FULL));
                }
            }
            __syncwarp();
            return true;
        };
        auto rows = [&](const DqItem& it) {
            if (nr >= 2 && !warp_sleep<kEvery>(bar(ROWS_EMPTY + (nr & 1)), ((nr >> 1) - 1) & 1, ctl)) return false;
            // D of the warp's 32 rows: D / 8 lanes to a row, 16 bytes of O and dO a lane
            constexpr int kLanes = D / 8, kPer = 32 / kLanes;
            const int sub = lane / kLanes, c = lane % kLanes, n0 = it.tile * kTile + 32 * quad;
            const int64_t at = (((int64_t)it.b * prm.N + n0) * prm.H + it.h) * D + c * 8;
            // four rows of each group of kLanes lanes at a time; the sums over a row's lanes carry half as many values
            // after each of the first two steps
            float d = 0.f;
#pragma unroll 1
            for (int i0 = 0; i0 < kLanes; i0 += 4) {
                float t[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rr = (i0 + i) * kPer + sub;
                    const int64_t e = at + (int64_t)rr * prm.H * D;
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    const bool in = n0 + rr < prm.N;
                    t[i] = dot8(in ? __ldg(reinterpret_cast<const uint4*>(prm.o + e)) : zero,
                                in ? __ldg(reinterpret_cast<const uint4*>(prm.d_o + e)) : zero);
                }
                const bool u2 = c & (kLanes / 2), u1 = c & (kLanes / 4);
                const float a = (u2 ? t[2] : t[0]) + __shfl_xor_sync(0xffffffffu, u2 ? t[0] : t[2], kLanes / 2);
                const float b = (u2 ? t[3] : t[1]) + __shfl_xor_sync(0xffffffffu, u2 ? t[1] : t[3], kLanes / 2);
                float v = (u1 ? b : a) + __shfl_xor_sync(0xffffffffu, u1 ? a : b, kLanes / 4);
#pragma unroll
                for (int x = kLanes / 8; x > 0; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
                // row (i0 + i) kPer + sub is in lane sub kLanes + i kLanes / 4: to the lane of its number
                const float got = __shfl_sync(0xffffffffu, v, (lane % kPer) * kLanes + (lane / kPer) % 4 * (kLanes / 4));
                if (lane / (4 * kPer) == i0 / 4) d = got;
            }
            float lse2 = 0.f;
            const int n = n0 + lane;
            if (n < prm.N) {
                const int64_t i = ((int64_t)it.b * prm.H + it.h) * prm.N + n;
                const float l = prm.lse[i];
                lse2 = l * kLog2e;
                if (l == -INFINITY) lse2 = d = 0.f;                   // no valid state: P = 0, and dS = 0 whatever dO holds
            }
            float* rv = row_vals + (nr & 1) * 2 * kTile + r;
            rv[0] = lse2;
            rv[kTile] = d;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(ROWS_FULL + (nr & 1)));
            ++nr;
            return true;
        };
        DqWalk pre;
        DqItem it;
        // k = -1: the first item's rows only
        for (int k = -1; k < 0 || item_at(prm, k, it); ++k) {
            if (k < 0 || it.nt > 0) {
                // the next item's D before this one's dQ
                if (pre.ok && pre.next_item(prm) && !(ok = load(pre.it) && rows(pre.it))) break;
                if (k < 0) continue;
                if (!(ok = warp_sleep<kEvery>(bar(DQ_DONE), nd & 1, ctl))) break;
                ++nd;
                fence_after();
            }
            const int row0 = it.tile * kTile + 32 * quad;
            if (lane == 0) bulk_wait_read();                          // the rows before these have left
            __syncwarp();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                if (it.nt > 0) {
                    tmem_ld32(tq + c * 32, v);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0u;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint4 w;
                    w.x = pack_bf16(__uint_as_float(v[8 * e + 0]) * prm.scale, __uint_as_float(v[8 * e + 1]) * prm.scale);
                    w.y = pack_bf16(__uint_as_float(v[8 * e + 2]) * prm.scale, __uint_as_float(v[8 * e + 3]) * prm.scale);
                    w.z = pack_bf16(__uint_as_float(v[8 * e + 4]) * prm.scale, __uint_as_float(v[8 * e + 5]) * prm.scale);
                    w.w = pack_bf16(__uint_as_float(v[8 * e + 6]) * prm.scale, __uint_as_float(v[8 * e + 7]) * prm.scale);
                    *reinterpret_cast<uint4*>(stage + swizzled(lane, 4 * c + e, 4096)) = w;
                }
            }
            fence_before();
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                if (it.nt > 0) mbar_arrive(bar(DQ_FREE));             // dQ may take the next item
                if (row0 < prm.N) {
                    for (int s = 0; s < D / 64; ++s)
                        tma_store_4d(&tmDQ, smem_u32(stage) + s * 4096, s * 64, row0, it.h, it.b);
                    bulk_commit();
                }
            }
        }
        if (!ok) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -5); }
        if (nl > 0) mbar_drain(bar(QD_FULL), (nl - 1) & 1);           // what this warp loaded has landed
        __syncwarp();
        tmem_wait_ld();
        if (lane == 0) bulk_wait();
    }
    end_cta(tmem);
}

// -------------------------------------------------------------------- key side
// warps 0-7 softmax, 8-11 dK and dV to memory, 12 MMA, 13 polls for it, 14 Q /
// dO ring with the rows' lse and D, 15 K and V.  An item: a key tile of one key head and a share
// of the (query head, 64-token) steps that read it.
struct DkvP {
    Keys keys;
    const float *lse, *dsum;
    float* part;                     // [2: dK, dV][chunks][B, M, Hkv, D], or null: dk, dv hold the result
    __nv_bfloat16 *dk, *dv;
    int32_t* err;
    int N, H, G, Hkv, chunks, nq, items;
    int share, extra;                // steps of a share, of which the first `extra` have one more
    Div key_tiles, shares, key_heads, nqd;
    int64_t part_stride;             // floats of one chunk: B * M * Hkv * D
    float scale, scale_log2;
    unsigned long long wait_ns;
};

template <int D>
struct DkvSmem {
    static constexpr int kSlab = kKeys * 128, kSlabK = kTile * 128;
    static constexpr int kTileBytes = kKeys * D * 2, kKBytes = kTile * D * 2;
    static constexpr int kStages = 4;
    static constexpr int offK = 0;                                 // K, V
    static constexpr int offQ = offK + 2 * kKBytes;                // stages of Q, dO
    static constexpr int offRows = offQ + kStages * 2 * kTileBytes;   // stages of float lse, D [64]
    static constexpr int offBar = offRows + kStages * 2 * kKeys * 4;
    static constexpr int offMisc = offBar + 32 * 8;
    static constexpr int kAlloc = offMisc + 64 + 1024;
    static constexpr uint32_t colS = 0, colDP = 128, colDV = 256, colDK = 384;
};

struct DkvItem {
    int b, hk, kt, chunk, len, beg, end;      // steps [beg, end); none if the tile has no valid state
};
__device__ __forceinline__ bool item_at(const DkvP& p, int k, DkvItem& it) {
    const int idx = k * gridDim.x + blockIdx.x;
    if (idx >= p.items) return false;
    uint32_t kt = (uint32_t)idx, c = p.key_tiles.split(kt), hk = p.shares.split(c);
    it.kt = (int)kt;
    it.chunk = (int)c;
    it.b = (int)p.key_heads.split(hk);
    it.hk = (int)hk;
    it.len = p.keys.count(it.b);
    it.beg = p.share * it.chunk + min(it.chunk, p.extra);
    it.end = it.kt * kTile < it.len ? it.beg + p.share + (it.chunk < p.extra) : it.beg;
    return true;
}
struct DkvWalk {
    DkvItem it;
    int k = -1, s = 0;
    bool ok = true;
    __device__ __forceinline__ DkvWalk() { it.beg = it.end = 0; }
    __device__ __forceinline__ bool next(const DkvP& p) {
        if (++s < it.end) return true;
        return next_item(p);
    }
    __device__ __forceinline__ bool next_item(const DkvP& p) {
        do {
            ++k;
            ok = item_at(p, k, it);
        } while (ok && it.end == it.beg);
        s = it.beg;
        return ok;
    }
    __device__ __forceinline__ bool first() const { return s == it.beg; }
    __device__ __forceinline__ bool last() const { return s == it.end - 1; }
};

template <int D, uint32_t kEvery>
__global__ void __launch_bounds__(kThreads, 1)
k_cross_dkv(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
            const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO, const DkvP prm) {
    using L = DkvSmem<D>;
    enum {
        KV_FULL = 0, KV_EMPTY, S_FULL, PD_FULL = S_FULL + 2, ACC_DONE = PD_FULL + 2, ACC_FREE, DRAIN, ST_FULL,
        ST_EMPTY = ST_FULL + L::kStages, kBars = ST_EMPTY + L::kStages
    };
    static_assert(kBars <= 32, "barrier slots");
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + L::offBar + 8u * (uint32_t)i; };
    volatile WaitCtl* ctl = reinterpret_cast<volatile WaitCtl*>(smem + L::offMisc);
    float* row_vals = reinterpret_cast<float*>(smem + L::offRows);
    const uint32_t tmem = begin_cta<kBars>(bar(0), ctl, reinterpret_cast<uint32_t*>(smem + L::offMisc + 16), prm.wait_ns,
                                           [](int i) -> uint32_t {
                                               return i >= PD_FULL && i < PD_FULL + 2 ? 8 : i == ACC_FREE ? 4 : 1;
                                           });
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    bool ok = true;

    if (warp == kMmaWarp) {
        constexpr uint32_t idesc_s = instr_desc(kKeys, 0), idesc_g = instr_desc(D, 1);
        const uint64_t dk = smem_desc(sbase + L::offK, 16, 1024), dq = smem_desc(sbase + L::offQ, 16, 1024),
                       dq_mn = smem_desc(sbase + L::offQ, L::kSlab, 1024);
        uint32_t ua = 0, uc = 0;
        DkvWalk cur, ahead;
        bool use = true, more = true;
        for (int made = 0;;) {
            if (more) ahead.next(prm);
            if (use) cur.next(prm);
            if (made == 0 && !ahead.ok) break;
            use = made == 2 || !ahead.ok;
            more = ahead.ok;
            if (!(ok = meet(true))) break;
            fence_after();
            if (elect_one()) {
                if (use) {
                    const uint32_t st = uc % L::kStages, q = st * 2 * L::kTileBytes, buf = (uc & 1) * kKeys;
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk) {
                        mma_ts(tmem + L::colDV, tmem + L::colS + buf + (kk / 2) * 32 + (kk % 2) * 8,
                               desc_at(dq_mn, q + L::kTileBytes + kk * 16 * 128), idesc_g, !cur.first() || kk > 0);
                        mma_ts(tmem + L::colDK, tmem + L::colDP + buf + (kk / 2) * 32 + (kk % 2) * 8, desc_at(dq_mn, q + kk * 16 * 128), idesc_g,
                               !cur.first() || kk > 0);
                    }
                    commit(bar(ST_EMPTY + st));
                    if (cur.last()) commit(bar(ACC_DONE));
                }
                if (more) {
                    const uint32_t buf = (ua & 1) * kKeys, q = ua % L::kStages * 2 * L::kTileBytes;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t ok_ = (kk / 4) * L::kSlabK + (kk % 4) * 32, oq = q + (kk / 4) * L::kSlab + (kk % 4) * 32;
                        mma_ss(tmem + L::colS + buf, desc_at(dk, ok_), desc_at(dq, oq), idesc_s, kk > 0);
                        mma_ss(tmem + L::colDP + buf, desc_at(dk, L::kKBytes + ok_), desc_at(dq, L::kTileBytes + oq), idesc_s,
                               kk > 0);
                    }
                    commit(bar(S_FULL + (ua & 1)));
                    if (ahead.last()) commit(bar(KV_EMPTY));
                }
            }
            __syncwarp();
            uc += use;
            ua += more;
            made += (int)more - (int)use;
        }
        if (elect_one()) {
            commit(bar(DRAIN));
            mbar_drain(bar(DRAIN), 0);
        }
        __syncwarp();
    } else if (warp == kPollWarp) {
        uint32_t ua = 0, uc = 0, items_a = 0, items_c = 0;
        DkvWalk cur, ahead;
        bool use = true, more = true;
        for (int made = 0;;) {
            if (more) ahead.next(prm);
            if (use) cur.next(prm);
            if (made == 0 && !ahead.ok) break;
            use = made == 2 || !ahead.ok;
            more = ahead.ok;
            bool go = true;
            if (more) {
                go = warp_wait<kEvery>(bar(ST_FULL + ua % L::kStages), (ua / L::kStages) & 1, ctl);
                if (ahead.first()) go = go && warp_wait<kEvery>(bar(KV_FULL), items_a++ & 1, ctl);
                ++ua;
            }
            if (use) {
                // dK and dV of the item before this one have been read
                if (cur.first() && items_c++ > 0) go = go && warp_wait<kEvery>(bar(ACC_FREE), items_c & 1, ctl);
                go = go && warp_wait<kEvery>(bar(PD_FULL + (uc & 1)), (uc >> 1) & 1, ctl);
                ++uc;
            }
            if (!(ok = meet(go))) break;
            made += (int)more - (int)use;
        }
        if (!ok && lane == 0) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -3); }
    } else if (warp == kPollWarp + 1) {
        uint32_t u = 0;
        DkvWalk w;
        for (; w.next(prm); ++u) {
            const int st = u % L::kStages;
            uint32_t tile = (uint32_t)w.s;
            const int h = w.it.hk * prm.G + (int)prm.nqd.split(tile), q0 = (int)tile * kKeys;
            float l[2], d[2];                            // rows past N: lse = inf, so P is 0
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = q0 + 32 * i + lane;
                const int64_t at = ((int64_t)w.it.b * prm.H + h) * prm.N + n;
                l[i] = n < prm.N ? prm.lse[at] * kLog2e : INFINITY;
                d[i] = n < prm.N ? prm.dsum[at] : 0.f;
            }
            if (u >= L::kStages && !(ok = warp_sleep<kEvery>(bar(ST_EMPTY + st), (u / L::kStages - 1) & 1, ctl))) break;
            float* rv = row_vals + st * 2 * kKeys + lane;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                rv[32 * i] = l[i] == -INFINITY ? -INFINITY : -l[i];   // negated: addends
                rv[kKeys + 32 * i] = -d[i];
            }
            __syncwarp();
            if (lane == 0) {
                const uint32_t dst = sbase + L::offQ + st * 2 * L::kTileBytes;
                mbar_expect_tx(bar(ST_FULL + st), 2 * L::kTileBytes);
                for (int s = 0; s < D / 64; ++s) {
                    tma_load_4d(dst + s * L::kSlab, &tmQ, s * 64, q0, h, w.it.b, bar(ST_FULL + st));
                    tma_load_4d(dst + L::kTileBytes + s * L::kSlab, &tmDO, s * 64, q0, h, w.it.b, bar(ST_FULL + st));
                }
            }
        }
        if (!ok && lane == 0) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -1); }
        for (uint32_t st = 0; st < L::kStages; ++st)
            if (u > st) mbar_drain(bar(ST_FULL + st), ((u - 1 - st) / L::kStages) & 1);
    } else if (warp == kPollWarp + 2) {
        if (lane == 0) {
            uint32_t n = 0;
            DkvWalk w;
            for (; w.next_item(prm); ++n) {
                if (n > 0 && !(ok = mbar_sleep<kEvery>(bar(KV_EMPTY), (n - 1) & 1, ctl))) break;
                mbar_expect_tx(bar(KV_FULL), 2 * L::kKBytes);
                for (int s = 0; s < D / 64; ++s) {
                    tma_load_4d(sbase + L::offK + s * L::kSlabK, &tmK, s * 64, w.it.kt * kTile, w.it.hk, w.it.b, bar(KV_FULL));
                    tma_load_4d(sbase + L::offK + L::kKBytes + s * L::kSlabK, &tmV, s * 64, w.it.kt * kTile, w.it.hk, w.it.b,
                                bar(KV_FULL));
                }
            }
            if (!ok) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -2); }
            if (n > 0) mbar_drain(bar(KV_FULL), (n - 1) & 1);
        }
    } else if (warp < kRowWarp) {
        // ------------------------------------------------------------------ softmax
        const int g = warp / 4, quad = warp & 3;                      // columns [32 g, 32 g + 32) of every tile
        const uint32_t ts0 = tmem + ((uint32_t)(32 * quad) << 16) + L::colS + g * 32;
        uint32_t u = 0;
        DkvWalk w;
        while (ok && w.next_item(prm)) {
            const int j = w.it.kt * kTile + 32 * quad + lane;         // this thread's key
            const bool on = prm.keys.counts(w.it.b, w.it.len, j);
            for (int s = w.it.beg; s < w.it.end; ++s, ++u) {
                const int st = u % L::kStages;
                const uint32_t ts = ts0 + (u & 1) * kKeys, tp = ts - L::colS + L::colDP;
                if (!(ok = warp_wait<kEvery>(bar(ST_FULL + st), (u / L::kStages) & 1, ctl))) break;
                if (!(ok = warp_wait<kEvery>(bar(S_FULL + (u & 1)), (u >> 1) & 1, ctl))) break;
                fence_after();
                const float* rv = row_vals + st * 2 * kKeys + g * 32;
                uint32_t sv[32], dv[32], pk[16], dk[16];
                tmem_ld32(ts, sv);
                tmem_ld32(tp, dv);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 l4 = *reinterpret_cast<const float4*>(rv + e);
                    const float4 d4 = *reinterpret_cast<const float4*>(rv + kKeys + e);
                    const float l[4] = {l4.x, l4.y, l4.z, l4.w}, d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                    for (int f = 0; f < 4; f += 2) {
                        float x0, x1, d0, d1;
                        ffma2(x0, x1, __uint_as_float(sv[e + f]), __uint_as_float(sv[e + f + 1]), prm.scale_log2,
                              prm.scale_log2, l[f], l[f + 1]);
                        fadd2(d0, d1, __uint_as_float(dv[e + f]), __uint_as_float(dv[e + f + 1]), d[f], d[f + 1]);
                        const float p0 = ex2_mufu(x0), p1 = ex2_mufu(x1);
                        fmul2(d0, d1, d0, d1, p0, p1);
                        pk[(e + f) / 2] = on ? pack_bf16(p0, p1) : 0u;
                        dk[(e + f) / 2] = on ? pack_bf16(d0, d1) : 0u;
                    }
                }
                tmem_st16(ts, pk);
                tmem_st16(tp, dk);
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(PD_FULL + (u & 1)));
            }
        }
        if (!ok) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -4); }
        __syncwarp();
        tmem_wait_st();
        tmem_wait_ld();
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------ dK, dV of an item
        const int quad = warp & 3;
        const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
        uint32_t nd = 0;
        DkvItem it;
        for (int k = 0; ok && item_at(prm, k, it); ++k) {
            const bool work = it.end > it.beg;
            if (!work && prm.part) continue;                          // the sum leaves this tile out
            const int j = it.kt * kTile + 32 * quad + lane;
            if (work) {
                if (!(ok = warp_sleep<kEvery>(bar(ACC_DONE), nd & 1, ctl))) break;
                ++nd;
                fence_after();
            }
            const int64_t at = (((int64_t)it.b * prm.keys.M + j) * prm.Hkv + it.hk) * D;
            // 0 * NaN is NaN: a state that does not count gets its zeros here (of shares: in their sum)
            const bool on = work && prm.keys.counts(it.b, it.len, j);
#pragma unroll 1
            for (int c = 0; c < 2 * D / 32; ++c) {
                const bool is_v = c < D / 32;
                const int col = (is_v ? c : c - D / 32) * 32;
                uint32_t v[32];
                if (work) {
                    tmem_ld32(tl + (is_v ? L::colDV : L::colDK) + col, v);
                    tmem_wait_ld();
                }
                if (!on)
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0u;
                if (j >= prm.keys.M) {
                    // nothing to write
                } else if (prm.part) {
                    float4* dst = reinterpret_cast<float4*>(prm.part + ((is_v ? prm.chunks : 0) + it.chunk) * prm.part_stride +
                                                            at + col);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                             __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
                } else {
                    const float f = is_v ? 1.f : prm.scale;
                    uint4* dst = reinterpret_cast<uint4*>((is_v ? prm.dv : prm.dk) + at + col);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint4 w;
                        w.x = pack_bf16(__uint_as_float(v[8 * e + 0]) * f, __uint_as_float(v[8 * e + 1]) * f);
                        w.y = pack_bf16(__uint_as_float(v[8 * e + 2]) * f, __uint_as_float(v[8 * e + 3]) * f);
                        w.z = pack_bf16(__uint_as_float(v[8 * e + 4]) * f, __uint_as_float(v[8 * e + 5]) * f);
                        w.w = pack_bf16(__uint_as_float(v[8 * e + 6]) * f, __uint_as_float(v[8 * e + 7]) * f);
                        dst[e] = w;
                    }
                }
                __syncwarp();                                         // lanes past M: the next tmem_ld takes the whole warp
            }
            if (work) {
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ACC_FREE));
            }
        }
        if (!ok) { ctl->abort = 1; record_error(prm.err, BSA_EDEVICE, -5); }
        __syncwarp();
        tmem_wait_ld();
    }
    end_cta(tmem);
}

// dK (scaled) and dV from the shares, in share order; states that do not count get zeros (no share has written the tiles
// behind a length).
__global__ void k_cross_dkv_sum(const DkvP prm, int D) {
    const int64_t i4 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i4 * 4 >= prm.part_stride) return;
    const bool is_v = blockIdx.y != 0;
    const int64_t row = i4 * 4 / ((int64_t)prm.Hkv * D), b = row / prm.keys.M;
    const int j = (int)(row - b * prm.keys.M);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (prm.keys.counts((int)b, prm.keys.count((int)b), j)) {
        const float* src = prm.part + (is_v ? prm.chunks * prm.part_stride : 0) + i4 * 4;
        for (int c = 0; c < prm.chunks; ++c) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(src + c * prm.part_stride));
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    }
    const float f = is_v ? 1.f : prm.scale;
    reinterpret_cast<uint2*>(is_v ? prm.dv : prm.dk)[i4] = make_uint2(pack_bf16(s.x * f, s.y * f), pack_bf16(s.z * f, s.w * f));
}

// Shares of the query steps for one key tile: enough items to fill the SMs evenly, each share at least 8 steps.
int share_count(const bsa_plan& p, int64_t M, int Hkv) {
    const int64_t tiles = (int64_t)p.B * Hkv * ((M + kTile - 1) / kTile);
    const int64_t steps = (int64_t)(p.H / Hkv) * ((p.N + kKeys - 1) / kKeys);
    int best = 1;
    double best_cost = 1e300;
    for (int c = 1; c <= 64 && (c == 1 || steps / c >= 8); ++c) {
        const int64_t waves = (tiles * c + p.num_sms - 1) / p.num_sms;
        // in steps of one SM: a share, its start and end (about 3 steps), and a little for the sum's traffic
        const double cost = (double)waves * ((double)steps / c + 3.0) + (c > 1 ? 0.02 * tiles * c : 0.0);
        if (cost < best_cost) {
            best_cost = cost;
            best = c;
        }
    }
    return best;
}

template <int D, uint32_t kEvery>
cudaError_t launch_t(const bsa_plan& p, const CrossArgs& a, const DqP& pq, const DkvP& pk, const void* d_o, void* dq,
                     cudaStream_t s) {
    CUtensorMap mq, mk, mv, mg, mo;
    int64_t so[3];
    dense_strides(so, p.N, p.H, D);
    if (!make_map_4d(&mq, a.q, p.B, p.N, p.H, D, a.st, kTile) || !make_map_4d(&mk, a.k, p.B, a.M, a.Hkv, D, a.st + 3, kKeys) ||
        !make_map_4d(&mv, a.v, p.B, a.M, a.Hkv, D, a.st + 6, kKeys) || !make_map_4d(&mg, d_o, p.B, p.N, p.H, D, so, kTile) ||
        !make_map_4d(&mo, dq, p.B, p.N, p.H, D, so, 32))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(k_cross_dq<D, kEvery>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         DqSmem<D>::kAlloc);
    if (e != cudaSuccess) return e;
    k_cross_dq<D, kEvery><<<std::min(p.num_sms, pq.items), kThreads, DqSmem<D>::kAlloc, s>>>(mq, mk, mv, mg, mo, pq);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;

    if (!make_map_4d(&mq, a.q, p.B, p.N, p.H, D, a.st, kKeys) || !make_map_4d(&mk, a.k, p.B, a.M, a.Hkv, D, a.st + 3, kTile) ||
        !make_map_4d(&mv, a.v, p.B, a.M, a.Hkv, D, a.st + 6, kTile) || !make_map_4d(&mg, d_o, p.B, p.N, p.H, D, so, kKeys))
        return cudaErrorInvalidValue;
    e = cudaFuncSetAttribute(k_cross_dkv<D, kEvery>, cudaFuncAttributeMaxDynamicSharedMemorySize, DkvSmem<D>::kAlloc);
    if (e != cudaSuccess) return e;
    k_cross_dkv<D, kEvery><<<std::min(p.num_sms, pk.items), kThreads, DkvSmem<D>::kAlloc, s>>>(mq, mk, mv, mg, pk);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (pk.part) {
        k_cross_dkv_sum<<<dim3((unsigned)((pk.part_stride / 4 + 255) / 256), 2), 256, 0, s>>>(pk, D);
        e = cudaGetLastError();
    }
    return e;
}

template <int D>
cudaError_t launch_d(const bsa_plan& p, const CrossArgs& a, const DqP& pq, const DkvP& pk, const void* d_o, void* dq,
                     cudaStream_t s) {
    // a wait limit below a millisecond: the variant that checks it at every probe
    return p.wait_ns < 1000000ull ? launch_t<D, 0>(p, a, pq, pk, d_o, dq, s) : launch_t<D, 1023>(p, a, pq, pk, d_o, dq, s);
}

size_t dsum_bytes(const bsa_plan& p) { return align_up((size_t)p.B * p.H * p.N * sizeof(float)); }

}  // namespace

size_t cross_bwd_ws_bytes(const bsa_plan& p, int64_t M, int Hkv) {
    const int c = M > 0 ? share_count(p, M, Hkv) : 1;
    const size_t part = (size_t)p.B * M * Hkv * p.d * sizeof(float);
    return dsum_bytes(p) + (c > 1 ? align_up(2 * c * part) : 0);
}

cudaError_t launch_cross_bwd_tc(const bsa_plan& p, const CrossArgs& a, const void* o, const float* lse, const void* d_o,
                                void* dq, void* dk, void* dv, void* ws, cudaStream_t s) {
    DqP pq;
    pq.keys = Keys{a.kv_len, a.key_mask, (int)a.M};
    pq.o = (const __nv_bfloat16*)o;
    pq.d_o = (const __nv_bfloat16*)d_o;
    pq.lse = lse;
    pq.dsum = (float*)ws;
    pq.err = p.d_err;
    pq.N = (int)p.N;
    pq.H = p.H;
    pq.heads = Div(p.H);
    pq.G = Div(p.H / a.Hkv);
    const int tiles = (int)((p.N + kTile - 1) / kTile);
    pq.tiles = Div(tiles);
    pq.items = p.B * p.H * tiles;
    pq.scale = 1.f / sqrtf((float)p.d);
    pq.scale_log2 = kLog2e * pq.scale;
    pq.wait_ns = p.wait_ns;
    DkvP pk;
    pk.keys = pq.keys;
    pk.lse = lse;
    pk.dsum = pq.dsum;
    pk.chunks = share_count(p, a.M, a.Hkv);
    pk.part = pk.chunks > 1 ? (float*)((char*)ws + dsum_bytes(p)) : nullptr;
    pk.dk = (__nv_bfloat16*)dk;
    pk.dv = (__nv_bfloat16*)dv;
    pk.err = p.d_err;
    pk.N = pq.N; pk.H = p.H; pk.G = p.H / a.Hkv; pk.Hkv = a.Hkv;
    const int key_tiles = (int)((a.M + kTile - 1) / kTile);
    pk.nq = (int)((p.N + kKeys - 1) / kKeys);
    pk.share = (int)((int64_t)pk.G * pk.nq / pk.chunks);
    pk.extra = (int)((int64_t)pk.G * pk.nq % pk.chunks);
    pk.key_tiles = Div(key_tiles);
    pk.shares = Div(pk.chunks);
    pk.key_heads = Div(a.Hkv);
    pk.nqd = Div(pk.nq);
    pk.items = p.B * a.Hkv * key_tiles * pk.chunks;
    pk.part_stride = (int64_t)p.B * a.M * a.Hkv * p.d;
    pk.scale = pq.scale; pk.scale_log2 = pq.scale_log2;
    pk.wait_ns = p.wait_ns;
    return p.d == 128 ? launch_d<128>(p, a, pq, pk, d_o, dq, s) : launch_d<64>(p, a, pq, pk, d_o, dq, s);
}

}  // namespace bsa
