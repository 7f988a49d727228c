// grouped_mm.cu -- products of rows with the matrix of their group, for experts of another form
// than the SwiGLU pair of the two stages: out[r] = x[r] . w[g(r)]^T (or . w[g(r)]), its gradients
// (the same call on dy for dx; dw[g] = dy_g^T x_g), and the MXFP8 form. The products run on the
// grouped-GEMM kernel (gemm_kernel.cuh, plain modes); the group sizes are read on the device.
#include "gemm_kernel.cuh"

namespace moe {

namespace {

// The groups' rows from the caller's offsets, one thread a group: counts, starts and the prefix
// of 256-row tiles that the units are numbered by. Offsets that decrease or leave [0, R] would
// send a product out of its operands: then no group has rows, and the error word says so.
__global__ void __launch_bounds__(1024)
grouped_tiles_kernel(const int32_t *__restrict__ offsets, int G, int R, int32_t *__restrict__ counts,
                     int32_t *__restrict__ starts, int32_t *__restrict__ mt_prefix, int32_t *__restrict__ err) {
    __shared__ int warp_sum[32];
    griddep_wait();
    const int g = threadIdx.x, lane = g & 31, warp = g >> 5;
    int a = 0, b = 0;
    if (g < G) {
        a = offsets[g];
        b = offsets[g + 1];
    }
    const bool bad = __syncthreads_or(a < 0 || b < a || b > R);
    const int n = bad ? 0 : b - a;
    int sum = (n + kUnitM - 1) / kUnitM;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    if (g < G) {
        for (int w = 0; w < warp; ++w) sum += warp_sum[w];
        counts[g] = n;
        starts[g] = bad ? 0 : a;
        mt_prefix[g + 1] = sum;
    }
    if (g == 0) {
        mt_prefix[0] = 0;
        if (bad) atomicOr(err, MOE_DEVERR_BAD_OFFSETS);
    }
}

}  // namespace

cudaError_t setup_grouped_mm_kernels() {
    cudaError_t e = set_gemm_smem<kRows>();
    if (e == cudaSuccess) e = set_gemm_smem<kRowsT>();
    if (e == cudaSuccess) e = set_gemm_smem<kRowsWgrad>();
    if (e == cudaSuccess) e = set_gemm_smem<kRowsMx>();
    return e;
}

cudaError_t launch_grouped_tiles(const int32_t *offsets, int G, int R, int32_t *counts, int32_t *starts,
                                 int32_t *mt_prefix, int32_t *err, cudaStream_t st) {
    const cudaError_t e = launch_dep(grouped_tiles_kernel, dim3(1), dim3((G + 31) / 32 * 32), 0, st, offsets, G, R,
                                     counts, starts, mt_prefix, err);
    note_launches(1);
    return e;
}

cudaError_t launch_grouped_mm(const GemmLaunch &p, GroupedKind kind, cudaStream_t st) {
    GemmArgs g = grouped_args(p);
    int64_t units;              // at most: the rows' tiles are known on the device alone
    if (kind == GroupedKind::wgrad) {
        units = static_cast<int64_t>(g.E) * g.m_tiles * g.n_tiles;
        g.total_units = static_cast<int>(units);
    } else {
        units = (static_cast<int64_t>(p.R) / kUnitM + (p.R < p.E ? p.R : p.E)) * g.n_tiles;
    }
    const int grid = units < p.num_sms ? static_cast<int>(units) : p.num_sms;
    if (grid <= 0) return cudaSuccess;
    switch (kind) {
        case GroupedKind::rows: return launch_tc_gemm<kRows>(maps_of(p), g, grid, st);
        case GroupedKind::rows_t: return launch_tc_gemm<kRowsT>(maps_of(p), g, grid, st);
        case GroupedKind::wgrad: return launch_tc_gemm<kRowsWgrad>(maps_of(p), g, grid, st);
        case GroupedKind::rows_mx: return launch_tc_gemm<kRowsMx>(maps_of(p), g, grid, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
