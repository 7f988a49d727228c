// norm_bwd.cu -- gradients of the root-mean-square norm. With z = h rstd and g = dy w:
//   dx = rstd (g - z mean(g z)) + dh;   dw = sum over the rows of dy z
// dx is the gradient of both x and the residual, which h is the sum of; dh what reaches h by the
// stream itself. A row is read once and held in registers between the sum and dx. Every thread
// keeps the same columns for all rows of its block and adds their part of dw in registers (at most
// kNormRowsPerBlock rows in fp32); a second launch adds the blocks' parts, in one order.
#include "norm.cuh"

namespace moe {

namespace {

template <typename T, int TPR, int V, int ACCESS>
__global__ void __launch_bounds__(Lane<T, TPR, V, ACCESS>::THREADS)
rms_norm_bwd_kernel(const NormBackwardLaunch p) {
    using L = Lane<T, TPR, V, ACCESS>;
    constexpr int N = L::N;
    __shared__ float part[2][TPR / 32];
    extern __shared__ float columns[];                      // rows of warps: the block's sums, [H]
    griddep_wait();
    const L lane(p.H);
    const float inv_h = 1.f / static_cast<float>(p.H);
    float dw[V][N];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < N; ++j) dw[v][j] = 0.f;
    int turn = 0;
    // the rows of this block: whole warps leave the loop together
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * L::ROWS + threadIdx.x / TPR; t < p.T;
         t += static_cast<int64_t>(gridDim.x) * L::ROWS, turn ^= 1) {
        const T *dyr = static_cast<const T *>(p.dy) + t * p.H, *hr = static_cast<const T *>(p.h) + t * p.ld_h;
        Vec<T> dy[V], h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dy[v] = lane.template load<false>(dyr, v);
            h[v] = lane.load(hr, v);
        }
        const float rstd = p.rstd[t];
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float w[N];
            lane.weight(p.weight, p.w_f32, v, w);
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float z = to_float(h[v].v[j]) * rstd, d = to_float(dy[v].v[j]);
                dw[v][j] = fmaf(d, z, dw[v][j]);
                s = fmaf(d * w[j], z, s);
            }
            sum += s;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        if constexpr (TPR > 32) {
            // two sets of sums in turn: a warp may be a row ahead of the others, never two
            if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = sum;
            __syncthreads();
            sum = 0.f;
#pragma unroll
            for (int w = 0; w < TPR / 32; ++w) sum += part[turn][w];
        }
        const float mean = sum * inv_h;
        T *dxr = static_cast<T *>(p.dx) + t * p.H;
        const T *dhr = static_cast<const T *>(p.dh) + t * p.H;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float w[N];
            lane.weight(p.weight, p.w_f32, v, w);
            Vec<T> more, dx;
            more.raw = make_uint4(0u, 0u, 0u, 0u);
            if (p.dh != nullptr) more = lane.template load<false>(dhr, v);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float z = to_float(h[v].v[j]) * rstd;
                dx.v[j] = from_float<T>(fmaf(rstd, fmaf(-z, mean, to_float(dy[v].v[j]) * w[j]), to_float(more.v[j])));
            }
            lane.store(dxr, v, dx);
        }
    }
    float *out = p.part + static_cast<int64_t>(blockIdx.x) * p.H;
    if constexpr (L::ROWS > 1) {
        // the warps' sums, one warp after the other
        for (int w = 0; w < L::ROWS; ++w) {
            if (threadIdx.x / TPR == w) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (lane.has(v, j)) {
                            float &c = columns[lane.column(v, j)];
                            c = w == 0 ? dw[v][j] : c + dw[v][j];
                        }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < p.H; c += L::THREADS) out[c] = columns[c];
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (lane.has(v, j)) out[lane.column(v, j)] = dw[v][j];
    }
}

// dweight[c] = the sum of the blocks' parts, 32 columns a block; 32 rows at a time in fp32, then fp64.
template <typename W>
__global__ void __launch_bounds__(1024)
rms_norm_dw_kernel(const float *__restrict__ part, int blocks, int H, W *__restrict__ dweight) {
    __shared__ double sums[32][33];
    griddep_wait();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + x;
    double total = 0.0;
    if (c < H) {
        for (int b0 = y; b0 < blocks; b0 += 32 * 32) {
            float s = 0.f;
#pragma unroll 8
            for (int k = 0; k < 32; ++k) {
                const int b = b0 + 32 * k;
                if (b < blocks) s += part[static_cast<int64_t>(b) * H + c];
            }
            total += s;
        }
    }
    sums[y][x] = total;
    __syncthreads();
    if (y == 0 && c < H) {
#pragma unroll 4
        for (int k = 1; k < 32; ++k) total += sums[k][x];
        dweight[c] = from_float<W>(static_cast<float>(total));
    }
}

template <typename T>
cudaError_t launch_of(const NormBackwardLaunch &p, cudaStream_t st) {
    return with_lane<T>(p.H, p.access, [&](auto lane) {
        using L = decltype(lane);
        return launch_dep(rms_norm_bwd_kernel<T, L::TPR, L::V, L::ACCESS>, dim3(static_cast<unsigned>(p.blocks)),
                          dim3(L::THREADS), L::ROWS > 1 ? 4 * static_cast<size_t>(p.H) : 0, st, p);
    });
}

template <typename W>
cudaError_t launch_dw(const NormBackwardLaunch &p, cudaStream_t st) {
    return launch_dep(rms_norm_dw_kernel<W>, dim3((p.H + 31) / 32), dim3(1024), 0, st, static_cast<const float *>(p.part),
                      static_cast<int>(p.blocks), p.H, static_cast<W *>(p.dweight));
}

}  // namespace

// Blocks of the backward: up to two an SM, and no block has more than kNormRowsPerBlock rows a thread.
int64_t rms_norm_bwd_blocks(int64_t T) {
    const int64_t few = T < 304 ? T : 304, many = (T + kNormRowsPerBlock - 1) / kNormRowsPerBlock;
    return few > many ? few : many;
}

cudaError_t launch_rms_norm_backward(const NormBackwardLaunch &p, cudaStream_t st) {
    cudaError_t e = p.T == 0                    ? cudaSuccess
                    : p.dtype == MOE_DTYPE_F32  ? launch_of<float>(p, st)
                    : p.dtype == MOE_DTYPE_BF16 ? launch_of<__nv_bfloat16>(p, st)
                                                : launch_of<__half>(p, st);
    if (e != cudaSuccess) return e;
    e = p.w_f32                       ? launch_dw<float>(p, st)
        : p.dtype == MOE_DTYPE_BF16 ? launch_dw<__nv_bfloat16>(p, st)
                                      : launch_dw<__half>(p, st);
    note_launches(p.T == 0 ? 1 : 2);
    return e;
}

}  // namespace moe
