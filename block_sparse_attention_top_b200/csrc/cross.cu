// Cross attention to an encoder's states and its gradient (formulas in bsa.h):
// which kernel takes a call.  cross_fwd.cu works through query tiles on the
// tensor cores, cross_few.cu splits the states of a few query rows,
// cross_bwd.cu is the gradient.
#include "cross_common.cuh"

namespace bsa {
namespace {

__global__ void k_fill(float* p, int64_t n, float v) {
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) p[i] = v;
}

size_t q_bytes(const bsa_plan& p) { return (size_t)p.B * p.N * p.H * p.d * 2; }

// The split kernel reads K and V once for every 16 query rows of a key head, the tensor-core kernel works through an
// item's states one after the other.  Measured (d 128, 12 heads; tensor-core against split): 51 rows, 512 states 14.8 /
// 14.7 us; 128 rows, 512 states 14.6 / 18.8; 128 rows, 4096 states 61.9 / 41.5; 256 rows, 4096 states 62 / 70; 4 x 8
// key heads of 5 query heads: 60 rows, 512 states 21.1 / 18.8; 125 rows, 512 states 21.3 / 23.0; 125 rows, 4096 states
// 117 / 70; 255 rows, 4096 states 117 / 134.
bool few_rows(const bsa_plan& p, const CrossArgs& a) {
    const int64_t heads = (int64_t)p.B * a.Hkv, rows = p.N * (p.H / a.Hkv);
    if (heads > 65535) return false;                     // its grid
    if (rows <= 64) return true;
    const int64_t waves = ((int64_t)p.B * p.H * ((p.N + 127) / 128) + p.num_sms - 1) / p.num_sms;
    return a.M >= 4096 && rows <= 1024 && heads * ((rows + 15) / 16) <= p.num_sms * waves;
}

}  // namespace

size_t cross_ws_bytes(const bsa_plan& p, int64_t M, int Hkv, bool backward) {
    return backward ? cross_bwd_ws_bytes(p, M, Hkv) : 0;
}

cudaError_t launch_cross(const bsa_plan& p, const CrossArgs& a, void* o, float* lse, cudaStream_t s) {
    if (a.M > 0) return few_rows(p, a) ? launch_cross_few(p, a, o, lse, s) : launch_cross_fwd_tc(p, a, o, lse, s);
    cudaError_t e = cudaMemsetAsync(o, 0, q_bytes(p), s);
    if (e != cudaSuccess || !lse) return e;
    k_fill<<<p.num_sms, 256, 0, s>>>(lse, (int64_t)p.B * p.H * p.N, -INFINITY);
    return cudaGetLastError();
}

cudaError_t launch_cross_bwd(const bsa_plan& p, const CrossArgs& a, const void* o, const float* lse, const void* d_o,
                             void* dq, void* dk, void* dv, void* ws, cudaStream_t s) {
    if (a.M > 0) return launch_cross_bwd_tc(p, a, o, lse, d_o, dq, dk, dv, ws, s);
    return cudaMemsetAsync(dq, 0, q_bytes(p), s);
}

}  // namespace bsa
