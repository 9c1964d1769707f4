// The sum of the shares that CTAs have formed of per-channel gradients.
#include "m3_common.cuh"
#include "m3_internal.h"
#include "m3_sm100.cuh"

namespace m3 {
namespace {

struct Sums {
    const float* part;
    int shares, nouts;
    int64_t C;
    float* out[4];
};

// One column's shares are added in order by 32 threads, then those by a tree.
__global__ void __launch_bounds__(1024) sum_shares_kernel(const Sums p) {
    __shared__ float s[32][33];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int64_t n = p.nouts * p.C, c = static_cast<int64_t>(blockIdx.x) * 32 + cx;
    sm100::grid_dep_wait();     // may have started while the shares were formed
    float sum = 0.f;
    if (c < n)
#pragma unroll 4
        for (int k = ry; k < p.shares; k += 32) sum += __ldcg(p.part + k * n + c);
    s[ry][cx] = sum;
    __syncthreads();
    sum = warp_sum(s[cx][ry]);      // warp ry takes column ry
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + ry;
    if (cx == 0 && col < n) {
        const int o = static_cast<int>(col / p.C);
        if (p.out[o]) p.out[o][col - o * p.C] = sum;
    }
}

}  // namespace

cudaError_t launch_sum_shares(const float* part, int shares, int64_t C, float* const* outs, int nouts,
                              cudaStream_t s) {
    Sums p{part, shares, nouts, C, {}};
    for (int i = 0; i < nouts; ++i) p.out[i] = outs[i];
    return launch_after_rms(sum_shares_kernel, static_cast<unsigned>((nouts * C + 31) / 32), 1024, 0, s, p);
}

}  // namespace m3
