// grouped_mm.cu -- products of rows with the matrix of their group, for experts of another form
// than the SwiGLU pair of the two stages: out[r] = x[r] . w[g(r)]^T (or . w[g(r)]), its gradients
// (the same call on dy for dx; dw[g] = dy_g^T x_g), and the MXFP8 form. They run on pairs of SMs
// (pair_gemm.cuh), a few rows on the kernel below; the group sizes are read on the device.
#include "pair_gemm.cuh"

namespace moe {

namespace {

// The weight gradients' tensor maps, a thread a group: those of a and b with as many rows as end at the
// group's last one, so that rows behind it are read as zeros. (Of bad offsets nothing is computed.)
__global__ void __launch_bounds__(256)
grouped_maps_kernel(const __grid_constant__ CUtensorMap a, const __grid_constant__ CUtensorMap b,
                    const int32_t *__restrict__ offsets, int G, int R, CUtensorMap *__restrict__ maps) {
    griddep_wait();
    const int g = blockIdx.x * 256 + threadIdx.x;
    if (g >= G) return;
    const int end = max(1, min(R, offsets[g + 1]));
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        const uint4 *src = reinterpret_cast<const uint4 *>(o == 0 ? &a : &b);
        uint4 *dst = reinterpret_cast<uint4 *>(maps + 2 * g + o);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(CUtensorMap) / 16); ++i) dst[i] = src[i];
        asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;"
                     ::"l"(__cvta_generic_to_global(dst)), "r"(end) : "memory");
    }
    asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
}

// ---------------------------------------------------------------- a few rows
//
// With a few rows in all the products only stream matrices: out[r, n] = x[r, :] . w[g, n, :] for 16
// columns n a block, its eight warps a slice of K each, so that even one row's N columns keep every SM
// reading. A warp multiplies 16 x 32 of w by 32 x 8 of x^T (8 rows of x) with two m16n8k16 products:
// tensor cores of the older kind, whose operands come from registers, and so straight from the rows of
// w: K is added in any order, so lane (i, q) takes the 16 bytes w[i, 8 q ..] of a 32-wide step whole,
// and of x's row i the same ones, and lets the product take the eight pairs for the k it likes. The
// warps' sums are added in order.
//
// HBM bounds it: 8 rows through 8 of 32 matrices of 4096 x 7168 (470 MB) 68 to 71 us by the run, 6.6 to
// 6.9 TB/s where a copy has 6.8; on the kernel of many rows 94, since a 128-row tile of one row streams
// its 256 matrix rows in pieces of 128 bytes, and 128 of 152 SMs have a tile. One row of 4096 x 4096:
// 6.9 us, and 35.

constexpr int kFewWarps = 8;

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct GroupedFew {
    const uint16_t *x, *w;
    const int32_t *offsets;
    uint16_t *out;
    int32_t *err;
    int64_t ld_x, ld_out;
    int R, G, K, N;
    int nan_on_bad;
};

// Weights are read once: no place in L1 for them.
__device__ __forceinline__ uint4 ld_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// TILES: tiles of 16 columns of a block; two halve the reads of x.
template <int TILES, bool F16>
__global__ void __launch_bounds__(32 * kFewWarps)
grouped_few_kernel(const GroupedFew p) {
    constexpr int kFewSteps = 4 / TILES;                    // 32-wide steps of K in flight, beside as many in use
    constexpr int COLS = 16 * TILES;
    __shared__ float sums[kFewWarps][COLS][9];
    __shared__ int found[2];
    griddep_wait();
    // the group of row blockIdx.y; blocks of its first row, and of every eighth from there, have work
    const int r0 = blockIdx.y;
    bool bad = false;
    if (threadIdx.x == 0) found[0] = -1;
    __syncthreads();
    for (int g = threadIdx.x; g < p.G; g += 32 * kFewWarps) {
        const int a = p.offsets[g], b = p.offsets[g + 1];
        bad |= a < 0 || b < a || b > p.R;
        if (a <= r0 && r0 < b && (r0 - a) % 8 == 0) {
            found[0] = g;
            found[1] = b;
        }
    }
    if (__syncthreads_or(bad)) {
        if (blockIdx.x == 0 && r0 == 0 && threadIdx.x == 0) atomicOr(p.err, MOE_DEVERR_BAD_OFFSETS);
        const int n = blockIdx.x * COLS + 2 * threadIdx.x;  // of bad offsets every row and column has its block
        if (p.nan_on_bad && 2 * threadIdx.x < COLS && n < p.N)
            *reinterpret_cast<uint32_t *>(p.out + r0 * p.ld_out + n) = nan_16x2(F16);
        return;
    }
    const int g = found[0];
    if (g < 0) return;
    const int m = min(8, found[1] - r0);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = lane >> 2, q = lane & 3;
    const int n0 = blockIdx.x * COLS;
    // rows past N are not read: zeros
    bool has[2 * TILES];
    const uint16_t *w0[2 * TILES];
#pragma unroll
    for (int t = 0; t < 2 * TILES; ++t) {
        has[t] = n0 + 8 * t + i < p.N;
        w0[t] = p.w + (static_cast<int64_t>(g) * p.N + n0 + (has[t] ? 8 * t + i : 0)) * p.K + 8 * q;
    }
    const bool hasx = i < m;
    const uint16_t *x0 = p.x + (r0 + (hasx ? i : 0)) * p.ld_x + 8 * q;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    float c[TILES][4];
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[t][e] = 0.f;

    // the warps take kFewSteps steps in turn
    uint4 a[2][kFewSteps][2 * TILES], b[2][kFewSteps];
    constexpr int kSpan = 32 * kFewSteps;
    auto read = [&](int s, int k0) {
#pragma unroll
        for (int u = 0; u < kFewSteps; ++u) {
            const int k = k0 + 32 * u;
            const bool in = k + 8 * q < p.K;
#pragma unroll
            for (int t = 0; t < 2 * TILES; ++t) a[s][u][t] = in && has[t] ? ld_stream(w0[t] + k) : zero;
            b[s][u] = in && hasx ? __ldg(reinterpret_cast<const uint4 *>(x0 + k)) : zero;
        }
    };
    auto multiply = [&](int s) {
#pragma unroll
        for (int u = 0; u < kFewSteps; ++u) {
            const uint4 &v = b[s][u];
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                const uint4 &l = a[s][u][2 * t], &h = a[s][u][2 * t + 1];
                mma_16816<F16>(c[t], l.x, h.x, l.y, h.y, v.x, v.y);
                mma_16816<F16>(c[t], l.z, h.z, l.w, h.w, v.z, v.w);
            }
        }
    };
    int k = warp * kSpan;
    if (k < p.K) {
        read(0, k);
        while (true) {
            const int k1 = k + kFewWarps * kSpan, k2 = k1 + kFewWarps * kSpan;
            if (k1 < p.K) read(1, k1);
            multiply(0);
            if (k1 >= p.K) break;
            if (k2 < p.K) read(0, k2);
            multiply(1);
            if (k2 >= p.K) break;
            k = k2;
        }
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[warp][16 * t + i + (e >= 2 ? 8 : 0)][2 * q + (e & 1)] = c[t][e];
    __syncthreads();
    const int n = threadIdx.x % COLS, row = threadIdx.x / COLS;
    if (row < m && n0 + n < p.N) {
        float v = 0.f;
#pragma unroll
        for (int t = 0; t < kFewWarps; ++t) v += sums[t][n][row];
        uint16_t *dst = p.out + (r0 + row) * p.ld_out + n0 + n;
        if constexpr (F16) *reinterpret_cast<__half *>(dst) = __float2half_rn(v);
        else *reinterpret_cast<__nv_bfloat16 *>(dst) = __float2bfloat16_rn(v);
    }
}

}  // namespace

cudaError_t launch_grouped_few(const void *x, const void *w, const int32_t *offsets, void *out, int32_t *err, int64_t ld_x,
                               int64_t ld_out, int R, int G, int K, int N, bool f16, bool nan_on_bad, cudaStream_t st) {
    GroupedFew p{static_cast<const uint16_t *>(x), static_cast<const uint16_t *>(w), offsets, static_cast<uint16_t *>(out),
                 err, ld_x, ld_out, R, G, K, N, nan_on_bad};
    // groups of several rows: fewer reads of x (8 rows of one group, 4096 x 11008: 19.9 us, and 22.4 with
    // 16 columns); of one: more blocks (8 of 32 matrices of 4096 x 7168: 68.0 us, and 73.7 with 32)
    const int cols = R > 2 * G ? 32 : 16;
    const dim3 grid((N + cols - 1) / cols, R), block(32 * kFewWarps);
    const cudaError_t e =
        cols == 32 ? launch_dep(f16 ? grouped_few_kernel<2, true> : grouped_few_kernel<2, false>, grid, block, 0, st, p)
                   : launch_dep(f16 ? grouped_few_kernel<1, true> : grouped_few_kernel<1, false>, grid, block, 0, st, p);
    note_launches(1);
    return e;
}

namespace {

template <int MODE, int MOST>
cudaError_t setup_pair(int *clusters) {
    cudaError_t e = cudaFuncSetAttribute(pair_gemm_kernel<MODE, MOST>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kPairSmemBytes<MODE, MOST>));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kPairThreads<MODE>);
    cfg.dynamicSmemBytes = kPairSmemBytes<MODE, MOST>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, pair_gemm_kernel<MODE, MOST>, &cfg);
    if (e == cudaSuccess && n < *clusters) *clusters = n;
    return e;
}

template <int MODE, int MOST>
cudaError_t launch_pair_of(const PairMapsOf<MODE> &maps, const PairArgs &p, int clusters, cudaStream_t st) {
    return launch_dep(pair_gemm_kernel<MODE, MOST>, dim3(2 * clusters), dim3(kPairThreads<MODE>),
                      kPairSmemBytes<MODE, MOST>, st, maps, p);
}

}  // namespace

cudaError_t setup_pair_kernels(int *clusters) {
    cudaError_t e = setup_pair<kPairWgrad, 256>(clusters);
    if (e == cudaSuccess) e = setup_pair<kPairMx, 64>(clusters);
    if (e == cudaSuccess) e = setup_pair<kPairMx, 192>(clusters);
    if (e == cudaSuccess) e = setup_pair<kPairMx, 224>(clusters);
    if (e == cudaSuccess) e = setup_pair<kPairRows, 64>(clusters);
    if (e == cudaSuccess) e = setup_pair<kPairRows, 256>(clusters);
    if (e == cudaSuccess) e = setup_pair<kPairRowsT, 64>(clusters);
    if (e == cudaSuccess) e = setup_pair<kPairRowsT, 256>(clusters);
    return e;
}

cudaError_t launch_pair(const PairLaunch &l, GroupedKind kind, cudaStream_t st) {
    PairArgs p{};
    p.offsets = l.offsets;
    p.err = l.err;
    p.out = static_cast<uint16_t *>(l.out);
    p.ld_out = l.ld_out;
    p.R = l.R;
    p.G = l.G;
    p.K = l.K;
    p.N = l.N;
    p.n_tiles = (l.N + 255) / 256;
    p.k_tiles = (l.K + 255) / 256;
    p.f16 = l.f16;
    p.nan_on_bad = l.nan_on_bad;
    p.a_one = l.a_one;
    p.b_one = l.b_one;
    p.group_maps = static_cast<const CUtensorMap *>(l.group_maps);
    if (kind == GroupedKind::wgrad) {
        const cudaError_t e = launch_dep(grouped_maps_kernel, dim3((l.G + 255) / 256), dim3(256), 0, st, *l.tm_a, *l.tm_b,
                                         l.offsets, l.G, l.R, static_cast<CUtensorMap *>(l.group_maps));
        if (e != cudaSuccess) return e;
        note_launches(1);
    }
    const PairMaps maps{*l.tm_a, *l.tm_b, *(l.tm_b_wide != nullptr ? l.tm_b_wide : l.tm_b)};
    const int most = kind == GroupedKind::wgrad ? 256 : grouped_most(l.R, l.G, kind == GroupedKind::rows_mx);
    const int64_t tiles = kind == GroupedKind::wgrad ? grouped_matrix_tiles(l.G, l.K, l.N) : grouped_row_tiles(l.R, l.G, l.N, most);
    const int clusters = tiles < l.clusters ? static_cast<int>(tiles) : l.clusters;
    cudaError_t e = cudaErrorInvalidValue;
    if (kind == GroupedKind::wgrad) e = launch_pair_of<kPairWgrad, 256>(maps, p, clusters, st);
    else if (kind == GroupedKind::rows) e = most == 64 ? launch_pair_of<kPairRows, 64>(maps, p, clusters, st)
                                                       : launch_pair_of<kPairRows, 256>(maps, p, clusters, st);
    else if (kind == GroupedKind::rows_mx) {
        const PairMxMaps mx{maps, *l.tm_sfa, *l.tm_sfb};
        e = most == 64 ? launch_pair_of<kPairMx, 64>(mx, p, clusters, st)
            : most == 192 ? launch_pair_of<kPairMx, 192>(mx, p, clusters, st) : launch_pair_of<kPairMx, 224>(mx, p, clusters, st);
    }
    else if (kind == GroupedKind::rows_t) e = most == 64 ? launch_pair_of<kPairRowsT, 64>(maps, p, clusters, st)
                                                         : launch_pair_of<kPairRowsT, 256>(maps, p, clusters, st);
    note_launches(1);
    return e;
}

}  // namespace moe
