// rows.cu -- the row movements of expert parallelism across devices (MegaMoE
// guide, opening section: dispatch_grouped_gemm fuses the token dispatch
// all-to-all, grouped_gemm_combine the combine all-to-all). With the exchange
// done by the caller's collective, the device work on each side is a copy of
// the token rows into routed order (the send buffer of the dispatch; on one
// device, the A rows of stage 1) and, after the return exchange, the k-way sum
// of the returned rows (the combine).
#include "internal.cuh"

namespace moe {

namespace {

// The dispatch copy: rows[row_of[t k + j], :] = x[t, :] for every slot (t, j)
// with row_of >= 0 (dropped slots have none), and with row_w also
// row_w[row_of[s]] = topk_w[s]. One warp per token (grid-stride over tokens):
// the token's row is read once, eight 16-byte chunks per lane at a time, and
// stored to each of its k routed rows, so x is read T H times rather than
// T k H times (a gather by routed row would load the row once per slot).
__global__ void __launch_bounds__(256)
dispatch_rows_kernel(const __nv_bfloat16 *__restrict__ x, const int32_t *__restrict__ row_of, int T, int k,
                     int64_t H, __nv_bfloat16 *__restrict__ rows, const float *__restrict__ topk_w,
                     float *__restrict__ row_w) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    const int chunks = static_cast<int>(H / 8);
    for (int64_t t = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5); t < T; t += warps) {
        const int my_row = lane < k ? __ldg(&row_of[t * k + lane]) : -1;
        if (row_w != nullptr && my_row >= 0) row_w[my_row] = topk_w[t * k + lane];
        const uint4 *src = reinterpret_cast<const uint4 *>(x + t * H);
        for (int cb = 0; cb < chunks; cb += 256) {    // the same passes on every lane (shuffles below)
            const int c0 = cb + lane;
            uint4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = (c0 + 32 * j < chunks) ? __ldg(src + c0 + 32 * j) : make_uint4(0u, 0u, 0u, 0u);
            for (int j2 = 0; j2 < k; ++j2) {
                const int r = __shfl_sync(0xffffffffu, my_row, j2);
                if (r < 0) continue;                       // a dropped slot (the same for the whole warp)
                uint4 *dst = reinterpret_cast<uint4 *>(rows + static_cast<int64_t>(r) * H);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c0 + 32 * j < chunks) dst[c0 + 32 * j] = v[j];
            }
        }
    }
}

// The MXFP8 dispatch of rows quantized in token order (as the norm in front of the layer writes
// them). The first `copy_blocks` blocks copy codes, a warp a token: its row is read once and stored
// to its routed rows. The others gather the scale words of one k-block, a thread a routed row.
__global__ void __launch_bounds__(256)
mx_dispatch_kernel(const uint8_t *__restrict__ x_codes, const uint32_t *__restrict__ x_scales,
                   const int32_t *__restrict__ row_of, const int32_t *__restrict__ perm_slot,
                   const int32_t *__restrict__ routed, int k, int64_t T, int64_t cols, int copy_blocks,
                   uint8_t *__restrict__ codes, uint32_t *__restrict__ scales) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    if (static_cast<int>(blockIdx.x) < copy_blocks) {
        const int64_t n = cols / 16;
        const int64_t warps = static_cast<int64_t>(copy_blocks) * 8;
        for (int64_t t = blockIdx.x * 8ll + (threadIdx.x >> 5); t < T; t += warps) {
            const int my_row = lane < k ? row_of[t * k + lane] : -1;          // k <= 32
            const uint4 *src = reinterpret_cast<const uint4 *>(x_codes + t * cols);
            for (int64_t c0 = 0; c0 < n; c0 += 128) {
                uint4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c0 + 32 * i + lane < n) v[i] = __ldg(src + c0 + 32 * i + lane);
                for (int j = 0; j < k; ++j) {
                    const int r = __shfl_sync(0xffffffffu, my_row, j);
                    if (r < 0) continue;
                    uint4 *dst = reinterpret_cast<uint4 *>(codes + static_cast<int64_t>(r) * cols);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c0 + 32 * i + lane < n) dst[c0 + 32 * i + lane] = v[i];
                }
            }
        }
        return;
    }
    const int64_t R = *routed, kbs = cols / 128;
    const int64_t in_rows = (T + 3) & ~3ll, out_rows = (T * k + 3) & ~3ll;
    const int64_t blocks = (R + 255) / 256, step = gridDim.x - copy_blocks;
    for (int64_t b = blockIdx.x - copy_blocks; b < blocks * kbs; b += step) {
        const int64_t kb = b / blocks, r = (b - kb * blocks) * 256 + threadIdx.x;
        if (r < R) scales[kb * out_rows + r] = __ldg(x_scales + kb * in_rows + perm_slot[r] / k);
    }
}

}  // namespace

cudaError_t launch_mx_dispatch(const uint8_t *x_codes, const uint32_t *x_scales, const int32_t *row_of,
                               const int32_t *perm_slot, const int32_t *routed, int k, int64_t T, int64_t cols,
                               uint8_t *codes, uint32_t *scales, cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    int64_t copy = (T + 7) / 8, words = (T * k + 255) / 256 * (cols / 128);
    if (copy > 152 * 8) copy = 152 * 8;
    if (words > 152 * 8) words = 152 * 8;
    const cudaError_t e = launch_dep(mx_dispatch_kernel, dim3(static_cast<unsigned>(copy + words)), dim3(256), 0, st,
                                     x_codes, x_scales, row_of, perm_slot, routed, k, T, cols, static_cast<int>(copy),
                                     codes, scales);
    note_launches(1);
    return e;
}

cudaError_t launch_dispatch_rows(const __nv_bfloat16 *x, const int32_t *row_of, int64_t T, int k, int64_t H,
                                 __nv_bfloat16 *rows, const float *topk_w, float *row_w, cudaStream_t st) {
    if (T == 0 || H == 0) return cudaSuccess;
    int64_t grid = (T + 7) / 8;                     // eight tokens (warps) per block
    if (grid > 152 * 8) grid = 152 * 8;
    const cudaError_t e = launch_dep(dispatch_rows_kernel, dim3(static_cast<int>(grid)), dim3(256), 0, st, x, row_of,
                                     static_cast<int>(T), k, H, rows, topk_w, row_w);
    note_launches(1);
    return e;
}

}  // namespace moe
