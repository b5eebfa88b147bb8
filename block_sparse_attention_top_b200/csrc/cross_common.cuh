// Shared by the cross-attention kernels: parameters, valid-state masks, 4-D
// tensor maps over [B, rows, heads, d] tensors and their TMA copies.  (The norms
// take fmul2 from here.)
#pragma once

#include <cuda_bf16.h>

#include "bsa_internal.cuh"
#include "tc_common.cuh"

namespace bsa {
namespace cross {

constexpr int kTile = 128;           // query rows of a tensor-core tile
constexpr int kKeys = 64;            // keys of one

// n / d by a multiplication, n < 2^31: the walks over work items divide in every role, and a division's code in each
// place adds up (these kernels are sensitive to code size: 16 warps in seven roles share the instruction caches, and
// at 94 KB of code instruction fetches took most of the time).
struct Div {
    uint32_t d, m, s;
    Div() = default;
    explicit Div(int64_t by) : d((uint32_t)by), m(0), s(0) {
        if (d > 1) {
            while ((1ull << s) < d) ++s;
            m = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
            --s;
        }
    }
    __device__ __forceinline__ uint32_t quot(uint32_t n) const { return m ? __umulhi(n, m) >> s : n; }
    // quotient, and n becomes the remainder
    __device__ __forceinline__ uint32_t split(uint32_t& n) const {
        const uint32_t q = quot(n);
        n -= q * d;
        return q;
    }
};

// Valid states of batch entry b.
struct Keys {
    const int32_t* kv_len;           // [B] or null
    const uint8_t* key_mask;         // [B, M] or null
    int M;
    __device__ __forceinline__ int count(int b) const {
        if (!kv_len) return M;
        const int n = __ldg(kv_len + b);
        return n < 0 ? 0 : (n > M ? M : n);
    }
    // State j of batch entry b, whose length is len, counts.
    __device__ __forceinline__ bool counts(int b, int len, int j) const {
        return j < len && (!key_mask || __ldg(key_mask + (int64_t)b * M + j) != 0);
    }
    // Warp-collective: bit i of w[i / 32] = key base + i counts (kKeys of them); true if all do.
    __device__ __forceinline__ bool bits(int b, int len, int base, int lane, uint32_t* w) const {
        if (!key_mask) {
            const int n = len - base;
            w[0] = n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
            w[1] = n >= 64 ? 0xffffffffu : (n <= 32 ? 0u : (1u << (n - 32)) - 1u);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = base + 32 * i + lane;
                w[i] = __ballot_sync(0xffffffffu, counts(b, len, j));
            }
        }
        return (w[0] & w[1]) == 0xffffffffu;
    }
};

// Zeros in the rows of a K or V tile in shared memory whose state does not count (D / 8 lanes to a row).
template <int D, int kRows>
__device__ __forceinline__ void zero_rows(unsigned char* tile, const uint32_t* bits, int lane) {
    constexpr int kLanes = D / 8, kPer = 32 / kLanes;
    const int c = lane % kLanes, r = lane / kLanes;
    unsigned char* at = tile + (c / 8) * kRows * 128 + r * 128 + (c % 8) * 16;
#pragma unroll
    for (int w = 0; w < kRows / 32; ++w) {               // (bits stay in registers)
        const uint32_t off = ~bits[w] >> r;
#pragma unroll 4
        for (int i = 0; i < 32; i += kPer)
            if (off >> i & 1) *reinterpret_cast<uint4*>(at + (w * 32 + i) * 128) = make_uint4(0, 0, 0, 0);
    }
}

// One lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Packed fp32 pairs beside tc::ffma2 and tc::fadd2: d = a * b.
__device__ __forceinline__ void fmul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// A descriptor `bytes` further on (a multiple of 16, inside the shared memory window).
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }

// A meeting of two warps at a named barrier that tells both whether both are well, so that neither waits for one that
// has given up.  The MMA warp learns this way (barrier 1) from a polling warp that its operands are ready: a warp that
// has issued MMAs stalls on its next shared-memory access until the tensor cores have taken them, and a mbarrier probe
// is one; the named barrier is not.
__device__ __forceinline__ bool meet(bool ok, int id = 1) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok), "r"(id)
        : "memory");
    return r != 0;
}

// A bounded wait that lets the hardware suspend the thread between probes: for the roles that wait most of the
// time (loads, output), whose spinning would take issue slots from the softmax warps.
template <uint32_t kEvery>
__device__ __noinline__ bool mbar_sleep(uint32_t bar, uint32_t parity, volatile tc::WaitCtl* ctl) {
    const unsigned long long t0 = tc::globaltimer();
    for (uint32_t n = 1;; ++n) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 10000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (kEvery == 0 || (n & 15) == 0) {
            if (ctl->abort) return false;
            if (tc::globaltimer() - t0 >= ctl->limit_ns) return false;
        }
    }
}
template <uint32_t kEvery>
__device__ __forceinline__ bool warp_sleep(uint32_t bar, uint32_t parity, volatile tc::WaitCtl* ctl) {
    return __all_sync(0xffffffffu, tc::mbar_test(bar, parity) || mbar_sleep<kEvery>(bar, parity, ctl));
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c, int row, int head, int b,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(row), "r"(head), "r"(b), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void prefetch_4d(const CUtensorMap* map, int c, int row, int head, int b) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global [%0, {%1, %2, %3, %4}];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(row), "r"(head), "r"(b)
                 : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int c, int row, int head, int b) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(c), "r"(row), "r"(head), "r"(b)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The source of every committed store may be overwritten.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A warp fills a ring of K or V tiles (kRows rows).  In a tile with states that do not count their rows are
// overwritten with zeros once the copy has landed (0 * NaN is NaN); kLag (1 or 2) later copies are under way by then.  A
// tile must be needed only after the stage of the tile kStages - kLag before it has been emptied.  Rows past M are zero
// already: the copy fills them.  next() moves to the next tile; b(), head(), len(), t() describe it.
// full, empty, raw: the first of kStages barriers each.  Returns false if a wait ran out.
template <int D, int kRows, int kStages, int kLag, uint32_t kEvery, typename Walk>
__device__ __forceinline__ bool fill_ring(Walk& w, const Keys& keys, const CUtensorMap* map, unsigned char* tiles,
                                          uint32_t full, uint32_t empty, uint32_t raw, volatile tc::WaitCtl* ctl) {
    constexpr int kTileBytes = kRows * D * 2;
    const int lane = threadIdx.x % 32;
    struct Fix {
        bool on = false;
        int st;
        uint32_t bits[kRows / 32];
    } f1, f0;                                            // of the tile before the last (kLag 2), and the last
    uint32_t u = 0, phases = 0;                          // bit st: parity of raw[st]
    int lost = -1;                                       // stage whose copy ran out of time
    bool ok = true;
    auto mend = [&](Fix& f) {
        if (!f.on) return true;
        const bool landed = tc::warp_wait<kEvery>(raw + 8 * f.st, phases >> f.st & 1, ctl);
        if (!landed) tc::mbar_drain(raw + 8 * f.st, phases >> f.st & 1);
        phases ^= 1u << f.st;
        f.on = false;
        if (!landed) {
            lost = f.st;
            return false;
        }
        zero_rows<D, kRows>(tiles + f.st * kTileBytes, f.bits, lane);
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(full + 8 * f.st);
        return true;
    };
    bool more = true;
    for (int after = 0; after < kLag;) {                 // kLag rounds past the last tile
        if (more) more = w.next();
        Fix f;
        if (more) {
            const int st = u % kStages;
            if (u >= kStages && !(ok = warp_sleep<kEvery>(empty + 8 * st, (u / kStages - 1) & 1, ctl))) break;
            bool all = true;
#pragma unroll
            for (int i = 0; i < kRows / kKeys; ++i)
                all &= keys.bits(w.b(), w.len(), w.t() * kRows + i * kKeys, lane, f.bits + 2 * i);
            f.on = !all && (keys.key_mask || w.len() < keys.M);
            f.st = st;
            if (lane == 0) {
                const uint32_t bar = (f.on ? raw : full) + 8 * st;
                tc::mbar_expect_tx(bar, kTileBytes);
                for (int s = 0; s < D / 64; ++s)
                    tma_load_4d(tc::smem_u32(tiles) + st * kTileBytes + s * kRows * 128, map, s * 64, w.t() * kRows, w.head(),
                                w.b(), bar);
            }
            ++u;
        } else {
            ++after;
        }
        Fix& oldest = kLag == 2 ? f1 : f0;
        if (!(ok = mend(oldest))) {
            oldest = f;
            break;
        }
        if (kLag == 2) f1 = f0;
        f0 = f;
    }
    // every copy lands before the CTA exits; stages that were never made full are not waited for
    if (!ok) {
        if (f1.on) tc::mbar_drain(raw + 8 * f1.st, phases >> f1.st & 1);
        if (f0.on) tc::mbar_drain(raw + 8 * f0.st, phases >> f0.st & 1);
    }
    for (uint32_t st = 0; st < kStages; ++st) {
        const bool waits = !ok && ((f1.on && f1.st == (int)st) || (f0.on && f0.st == (int)st) || lost == (int)st);
        const uint32_t loads = u > st ? (u - 1 - st) / kStages + 1 : 0;
        if (loads > (uint32_t)waits) tc::mbar_drain(full + 8 * st, (loads - waits - 1) & 1);
    }
    return ok;
}

// bf16 [B, rows, heads, d] with element strides (batch, row, head) as a map of
// [d, rows, heads, B], box [64, box_rows, 1, 1] with 128-byte swizzle.
inline bool make_map_4d(CUtensorMap* m, const void* base, int64_t B, int64_t rows, int64_t heads, int d,
                        const int64_t* st, int box_rows) {
    auto enc = tc::get_encode();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)heads, (cuuint64_t)B};
    cuuint64_t strides[3] = {(cuuint64_t)st[1] * 2, (cuuint64_t)st[2] * 2, (cuuint64_t)st[0] * 2};
    cuuint32_t box[4] = {64u, (cuuint32_t)box_rows, 1u, 1u};
    cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline void dense_strides(int64_t* st, int64_t rows, int64_t heads, int d) {
    st[0] = rows * heads * d;
    st[1] = heads * d;
    st[2] = d;
}

}  // namespace cross

// cross_fwd.cu: M > 0
cudaError_t launch_cross_fwd_tc(const bsa_plan& p, const CrossArgs& a, void* o, float* lse, cudaStream_t s);

// cross_few.cu: few query rows, M > 0
cudaError_t launch_cross_few(const bsa_plan& p, const CrossArgs& a, void* o, float* lse, cudaStream_t s);
// cross_bwd.cu: M > 0
size_t cross_bwd_ws_bytes(const bsa_plan& p, int64_t M, int Hkv);
cudaError_t launch_cross_bwd_tc(const bsa_plan& p, const CrossArgs& a, const void* o, const float* lse, const void* d_o,
                                void* dq, void* dk, void* dv, void* ws, cudaStream_t s);

}  // namespace bsa
