// norm.cuh -- shared by the root-mean-square norm's forward (norm.cu) and backward (norm_bwd.cu).
//
// A row is held by TPR threads (a warp, or a block) in registers, as V "vectors" of 16 bytes a
// thread. Aligned rows: vector v of thread i is the row's vector v TPR + i, one 16-byte access. Where only rows that are
// read lie at odd places (kLoadsOne), the same vector is read element by element. Other rows (odd
// widths): a vector's elements lie TPR apart, so that a warp's accesses are consecutive elements.
#pragma once

#include "internal.cuh"
#include "mx.cuh"

namespace moe {

namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

// A value rounded to nearest.
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

template <typename T> constexpr int kVec = 16 / static_cast<int>(sizeof(T));     // elements of a vector

template <typename T>
union Vec {
    uint4 raw;
    T v[kVec<T>];
};

// The threads of a row and their vectors.
template <typename T_, int TPR_, int V_, int ACCESS_>
struct Lane {
    using T = T_;
    static constexpr int TPR = TPR_, V = V_, N = kVec<T_>, ACCESS = ACCESS_;
    static constexpr bool ALIGNED = ACCESS != kOne;
    static constexpr int ROWS = TPR == 32 ? 8 : 1;          // rows of a block
    static constexpr int THREADS = TPR * ROWS;
    int i;                                                  // the thread within its row
    int H;
    __host__ __device__ explicit Lane(int h) : i(0), H(h) {
#ifdef __CUDA_ARCH__
        i = threadIdx.x % TPR;
#endif
    }
    __device__ int column(int v, int j) const { return ALIGNED ? (v * TPR + i) * N + j : (v * N + j) * TPR + i; }
    __device__ bool has(int v, int j = 0) const { return column(v, j) < H; }
    // vector v of a row (0 past its end); `at_odds`: of one that may lie at an odd place
    template <bool at_odds = true>
    __device__ __forceinline__ Vec<T> load(const T *row, int v) const {
        Vec<T> r;
        r.raw = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (ACCESS == kWhole || (ALIGNED && !at_odds)) {
            if (has(v)) r.raw = *reinterpret_cast<const uint4 *>(row + column(v, 0));
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (has(v, j)) r.v[j] = row[column(v, j)];
        }
        return r;
    }
    __device__ __forceinline__ void store(T *row, int v, const Vec<T> &r) const {
        if constexpr (ALIGNED) {
            if (has(v)) *reinterpret_cast<uint4 *>(row + column(v, 0)) = r.raw;
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (has(v, j)) row[column(v, j)] = r.v[j];
        }
    }
    // the weights of vector v in fp32, of the row's type or fp32 (0 past the end)
    __device__ __forceinline__ void weight(const void *w, bool f32, int v, float (&out)[N]) const {
        if (f32 || sizeof(T) == 4) {
            const float *p = static_cast<const float *>(w);
            if constexpr (ALIGNED) {
#pragma unroll
                for (int q = 0; q < N / 4; ++q) {
                    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (has(v)) f = __ldg(reinterpret_cast<const float4 *>(p + column(v, 0)) + q);
                    out[4 * q] = f.x;
                    out[4 * q + 1] = f.y;
                    out[4 * q + 2] = f.z;
                    out[4 * q + 3] = f.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) out[j] = has(v, j) ? __ldg(p + column(v, j)) : 0.f;
            }
        } else {
            const Vec<T> r = load<false>(static_cast<const T *>(w), v);
#pragma unroll
            for (int j = 0; j < N; ++j) out[j] = to_float(r.v[j]);
        }
    }
};

// Calls f with the lane type of a row of H <= 16384 elements: the fewest threads that hold it in at
// most four vectors each; a warp up to 128 vectors, eight rows a block.
template <typename T, typename F>
cudaError_t with_lane(int64_t H, int access, F f) {
    const int64_t vecs = (H + kVec<T> - 1) / kVec<T>;
    if (access == kLoadsOne) {
        if (vecs <= 128) return f(Lane<T, 32, 4, kLoadsOne>(0));
        if (vecs <= 1024) return f(Lane<T, 256, 4, kLoadsOne>(0));
        return f(Lane<T, 1024, 4, kLoadsOne>(0));
    }
    if (access == kOne) {
        if (vecs <= 128) return f(Lane<T, 32, 4, kOne>(0));
        if (vecs <= 1024) return f(Lane<T, 256, 4, kOne>(0));
        return f(Lane<T, 1024, 4, kOne>(0));
    }
    if (vecs <= 32) return f(Lane<T, 32, 1, kWhole>(0));
    if (vecs <= 64) return f(Lane<T, 32, 2, kWhole>(0));
    if (vecs <= 128) return f(Lane<T, 32, 4, kWhole>(0));
    if (vecs <= 256) return f(Lane<T, 128, 2, kWhole>(0));
    if (vecs <= 512) return f(Lane<T, 128, 4, kWhole>(0));
    if (vecs <= 1024) return f(Lane<T, 256, 4, kWhole>(0));
    if (vecs <= 2048) return f(Lane<T, 512, 4, kWhole>(0));
    return f(Lane<T, 1024, 4, kWhole>(0));
}

}  // namespace

}  // namespace moe
