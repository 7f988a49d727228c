// norm_bwd.cu -- gradients of the root-mean-square norm. With z = h rstd and g = dy w:
//   dx = rstd (g - z mean(g z)) + dh;   dw = sum over the rows of dy z
// dx is the gradient of both x and the residual, which h is the sum of; dh what reaches h by the
// stream itself. A row is read once and held in registers between the sum and dx. Every thread
// keeps the same columns for all rows of its block and adds their part of dw in registers (at most
// kNormRowsPerBlock rows in fp32); a second launch adds the blocks' parts, in one order.
//
// HBM bounds it. A block goes from row to row, so that while it adds one up nothing of the next
// would be on its way: whole rows are fetched a row ahead with cp.async, every thread into a place
// of its own (nothing but itself waits for it).
#include "norm.cuh"

namespace moe {

namespace {

constexpr int kMostShared = 200 * 1024;
constexpr int kAhead = 2;                                   // rows of a block in shared memory
// Rows are fetched ahead where they are whole vectors (h, where it lies at odd places, is not) and
// kAhead of them fit, which fp32 rows of more than 1024 vectors do not.
template <typename L>
constexpr bool kFetchAhead = L::ALIGNED && kAhead * 3 * L::V * L::MOST * 16 <= kMostShared;

__device__ __forceinline__ void cp_async16(uint4 *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src) : "memory");
}

template <typename L>
__global__ void __launch_bounds__(L::MOST, L::WARP ? 3 : L::MOST == 256 ? 2 : 1)
rms_norm_bwd_kernel(const NormBackwardLaunch p) {
    using T = typename L::T;
    constexpr int N = L::N, V = L::V;
    constexpr bool AHEAD = kFetchAhead<L>;
    __shared__ float part[2][32];
    extern __shared__ uint4 fetched[];                      // [kAhead][dy, h, dh][V][threads]
    griddep_wait();
    const L lane(p.H);
    const int threads = blockDim.x;
    const float inv_h = 1.f / static_cast<float>(p.H);
    const int64_t step = static_cast<int64_t>(gridDim.x) * L::ROWS;
    const int operands = p.dh != nullptr ? 3 : 2;
    auto place = [&](int s, int o, int v) { return fetched + ((s * operands + o) * V + v) * threads + threadIdx.x; };
    auto fetch = [&](int64_t t, int s) {
        const T *src[3] = {static_cast<const T *>(p.dy) + t * p.H, static_cast<const T *>(p.h) + t * p.ld_h,
                           static_cast<const T *>(p.dh) + t * p.H};
#pragma unroll
        for (int o = 0; o < 3; ++o)
            if (o < operands && (o != 1 || L::ACCESS == kWhole))
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (lane.has(v)) cp_async16(place(s, o, v), src[o] + lane.column(v, 0));
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&](int s, int o, int v) {
        Vec<T> r;
        r.raw = lane.has(v) ? *place(s, o, v) : make_uint4(0u, 0u, 0u, 0u);
        return r;
    };
    float dw[V][N];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < N; ++j) dw[v][j] = 0.f;
    // the rows of this block (a warp's leave the loop by themselves)
    int64_t t = static_cast<int64_t>(blockIdx.x) * L::ROWS + lane.row();
    if (AHEAD && t < p.T) fetch(t, 0);
    for (int turn = 0; t < p.T; t += step, turn ^= 1) {
        Vec<T> h[V];
        float g[V][N];                                      // the weights, then dy w
        // (read before the row's values are waited for)
#pragma unroll
        for (int v = 0; v < V; ++v) lane.weight(p.weight, p.w_f32, v, g[v]);
        const float rstd = p.rstd[t];
        if constexpr (AHEAD) {
            // (a branch, behind which the compiler does not move the reads above)
            if (t + step < p.T) {
                fetch(t + step, turn ^ 1);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
        }
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Vec<T> dy;
            if constexpr (AHEAD) dy = take(turn, 0, v);
            else dy = lane.load(static_cast<const T *>(p.dy) + t * p.H, v);
            if constexpr (AHEAD && L::ACCESS == kWhole) h[v] = take(turn, 1, v);
            else h[v] = lane.template load<true>(static_cast<const T *>(p.h) + t * p.ld_h, v, t == 0 || t == p.T - 1);
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float z = to_float(h[v].v[j]) * rstd, d = to_float(dy.v[j]);
                dw[v][j] = fmaf(d, z, dw[v][j]);
                g[v][j] *= d;
                s = fmaf(g[v][j], z, s);
            }
            sum += s;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
        if constexpr (!L::WARP) {
            // two sets of sums in turn: a warp may be a row ahead of the others, never two
            if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = sum;
            __syncthreads();
            sum = 0.f;
            for (int w = 0; w < threads / 32; ++w) sum += part[turn][w];
        }
        const float mean = sum * inv_h;
        T *dxr = static_cast<T *>(p.dx) + t * p.H;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Vec<T> more, dx;
            more.raw = make_uint4(0u, 0u, 0u, 0u);
            if (p.dh != nullptr) {
                if constexpr (AHEAD) more = take(turn, 2, v);
                else more = lane.load(static_cast<const T *>(p.dh) + t * p.H, v);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float z = to_float(h[v].v[j]) * rstd;
                dx.v[j] = from_float<T>(fmaf(rstd, fmaf(-z, mean, g[v][j]), to_float(more.v[j])));
            }
            lane.store(dxr, v, dx);
        }
    }
    float *out = p.part + static_cast<int64_t>(blockIdx.x) * p.H;
    if constexpr (L::WARP) {
        // the warps' sums, one warp after the other
        float *columns = reinterpret_cast<float *>(fetched);
        __syncthreads();                                    // no warp takes rows any more
        for (int w = 0; w < L::ROWS; ++w) {
            if (lane.row() == w) {
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
        for (int c = threadIdx.x; c < p.H; c += threads) out[c] = columns[c];
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (lane.has(v, j)) out[lane.column(v, j)] = dw[v][j];
    }
}

// dweight[c] = the sum of the blocks' parts, 16 columns a block: a thread takes a column and every 64th
// part, 10 of them in a row, and a warp adds the 64 sums of two columns.
constexpr int kDwCols = 16;
template <typename W>
__global__ void __launch_bounds__(1024, 2)
rms_norm_dw_kernel(const float *__restrict__ part, int blocks, int H, W *__restrict__ dweight) {
    __shared__ float sums[64][kDwCols + 1];
    griddep_wait();
    const int x = threadIdx.x % kDwCols, y = threadIdx.x / kDwCols;
    const int c0 = blockIdx.x * kDwCols;
    float total = 0.f;
    if (c0 + x < H) {
        const float *p = part + static_cast<int64_t>(y) * H + c0 + x;
        const int64_t step = 64 * static_cast<int64_t>(H);
#pragma unroll 1
        for (int b0 = y; b0 < blocks; b0 += 64 * 10, p += 10 * step) {
            float v[10];
#pragma unroll
            for (int k = 0; k < 10; ++k) v[k] = b0 + 64 * k < blocks ? __ldg(p + k * step) : 0.f;
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < 10; ++k) s += v[k];
            total += s;
        }
    }
    sums[y][x] = total;
    __syncthreads();
    const int lane = threadIdx.x & 31, c = threadIdx.x >> 5;
    if (c >= kDwCols) return;
    total = sums[lane][c] + sums[lane + 32][c];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(kAll, total, d);
    if (lane == 0 && c0 + c < H) dweight[c0 + c] = from_float<W>(total);
}

template <typename T>
cudaError_t launch_of(const NormBackwardLaunch &p, cudaStream_t st) {
    return with_plan<T>(p.H, p.access, [&](auto plan) {
        using L = typename decltype(plan)::L;
        const size_t ahead = kFetchAhead<L> ? 16 * static_cast<size_t>(kAhead * (p.dh != nullptr ? 3 : 2) * L::V) * plan.threads : 0;
        const size_t sums = L::WARP ? 4 * static_cast<size_t>(p.H) : 0;
        return launch_dep(rms_norm_bwd_kernel<L>, dim3(static_cast<unsigned>(p.blocks)), dim3(plan.threads),
                          ahead > sums ? ahead : sums, st, p);
    });
}

template <typename W>
cudaError_t launch_dw(const NormBackwardLaunch &p, cudaStream_t st) {
    return launch_dep(rms_norm_dw_kernel<W>, dim3((p.H + kDwCols - 1) / kDwCols), dim3(1024), 0, st, static_cast<const float *>(p.part),
                      static_cast<int>(p.blocks), p.H, static_cast<W *>(p.dweight));
}

}  // namespace

// Blocks of the backward, by the width alone: each has a part of dw to write and to be added (bf16: 4096 rows of
// 2048 in four blocks an SM 17 us, in eight 21; 16384 of 1024 34, and 27). That is what an SM holds of bf16 rows of
// 520 to 8192 columns in whole vectors, for which alone it was measured; of a warp a row, of odd widths up to 1024, of bf16 rows
// beyond 8192 and of fp32 rows of 4096 with dh an SM holds about half of them, and the rest are a second wave. Few
// rows get a block each, also where a block could take eight: blocks without rows write parts of 0. No block has
// more than kNormRowsPerBlock rows a thread.
int64_t rms_norm_bwd_blocks(int64_t T, int64_t H) {
    const int64_t wave = 152 * (H <= 512 ? 6 : H <= 1024 ? 8 : H <= 4096 ? 4 : 2);
    const int64_t few = T < wave ? T : wave, many = (T + kNormRowsPerBlock - 1) / kNormRowsPerBlock;
    return few > many ? few : many;
}

// Shared memory of wide rows is above a launch's default.
cudaError_t setup_norm_kernels() {
    cudaError_t e = cudaSuccess;
    auto of = [&](auto type) {
        for (int64_t H : {8, 512, 1024, 2048, 4096, 8192, 16384})
            for (int access : {kWhole, kLoadsOne})
                if (e == cudaSuccess) e = with_plan<decltype(type)>(H, access, [](auto plan) {
                    return cudaFuncSetAttribute(rms_norm_bwd_kernel<typename decltype(plan)::L>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
                });
    };
    of(0.f);
    of(__nv_bfloat16());
    of(__half());
    return e;
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
