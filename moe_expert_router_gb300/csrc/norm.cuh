// norm.cuh -- shared by the root-mean-square norm's forward (norm.cu) and backward (norm_bwd.cu).
//
// A row is held in registers by a warp (up to 64 vectors; eight rows a block) or by a block of as
// many warps as it fills, as V "vectors" of 16 bytes a thread. Aligned rows: vector v of thread i is
// the row's vector v threads + i, one 16-byte access. Where only rows that are read lie at odd places
// (kLoadsOne), it is shifted out of the two aligned vectors around it. Other rows (odd widths): a vector's
// elements lie `threads` apart, so that a warp's accesses are consecutive elements.
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

// The threads of a row and their vectors. MOST: threads of a block at most.
template <typename T_, int V_, int ACCESS_, bool WARP_, int MOST_>
struct Lane {
    using T = T_;
    static constexpr int V = V_, N = kVec<T_>, ACCESS = ACCESS_, MOST = MOST_;
    static constexpr bool ALIGNED = ACCESS != kOne, WARP = WARP_;
    static constexpr int ROWS = WARP ? 8 : 1;               // rows of a block
    int tpr, i, H;                                          // the row's threads, and this one among them
    __device__ explicit Lane(int h) : tpr(WARP ? 32 : blockDim.x), i(WARP ? threadIdx.x % 32 : threadIdx.x), H(h) {}
    __device__ int row() const { return WARP ? static_cast<int>(threadIdx.x / 32) : 0; }
    __device__ int column(int v, int j) const { return ALIGNED ? (v * tpr + i) * N + j : (v * N + j) * tpr + i; }
    __device__ bool has(int v, int j = 0) const { return column(v, j) < H; }
    // vector v of a row (0 past its end); `at_odds`: of one that may lie at an odd place, and `edge`: of
    // the first or last such row
    template <bool at_odds = false>
    __device__ __forceinline__ Vec<T> load(const T *row, int v, bool edge = true) const {
        Vec<T> r;
        r.raw = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (ACCESS == kWhole || (ALIGNED && !at_odds)) {
            if (has(v)) r.raw = *reinterpret_cast<const uint4 *>(row + column(v, 0));
        } else if constexpr (ALIGNED) {
            if (!has(v)) return r;
            const T *at = row + column(v, 0);
            if (edge) {
#pragma unroll
                for (int j = 0; j < N; ++j) r.v[j] = at[j];
            } else {
                // the two aligned vectors around it, shifted (both lie between the first row and the last)
                const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at)) & 15u;
                const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(at) - off);
                const uint4 a = p[0], b = p[1];
                uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int k = 0; k < 6; ++k) w[k] = (off & 8u) ? w[k + 2] : w[k];
#pragma unroll
                for (int k = 0; k < 5; ++k) w[k] = (off & 4u) ? w[k + 1] : w[k];
                const uint32_t bits = (off & 3u) * 8u;
                r.raw = make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                                   __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
            }
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
            const Vec<T> r = load(static_cast<const T *>(w), v);
#pragma unroll
            for (int j = 0; j < N; ++j) out[j] = to_float(r.v[j]);
        }
    }
};

// A lane type and its block, as a value that a launch takes its kernel from.
template <typename T, int V, int ACCESS, bool WARP, int MOST>
struct Plan {
    using L = Lane<T, V, ACCESS, WARP, MOST>;
    int threads;
};

// Calls f with the plan for a row of H <= 16384 elements. Vectors: four a thread are enough accesses
// at once, and few warps to add up. Single elements: one vector's worth a thread, since each is an
// access of its own.
template <typename T, typename F>
cudaError_t with_plan(int64_t H, int access, F f) {
    const int vecs = static_cast<int>((H + kVec<T> - 1) / kVec<T>);
    constexpr int kWide = sizeof(T) == 4 ? 1024 : 512;
    auto threads = [&](int v) { return ((vecs + v - 1) / v + 31) / 32 * 32; };
    if (access == kWhole) {
        if (vecs <= 32) return f(Plan<T, 1, kWhole, true, 256>{256});
        if (vecs <= 64) return f(Plan<T, 2, kWhole, true, 256>{256});
        if (vecs <= 256) return f(Plan<T, 2, kWhole, false, 256>{threads(2)});
        if (vecs <= 1024) return f(Plan<T, 4, kWhole, false, 256>{threads(4)});
        return f(Plan<T, 4, kWhole, false, kWide>{threads(4)});
    }
    if (access == kLoadsOne) {
        if (vecs <= 64) return f(Plan<T, 2, kLoadsOne, true, 256>{256});
        if (vecs <= 1024) return f(Plan<T, 4, kLoadsOne, false, 256>{threads(4)});
        return f(Plan<T, 4, kLoadsOne, false, kWide>{threads(4)});
    }
    if (vecs <= 32) return f(Plan<T, 1, kOne, true, 256>{256});
    if (vecs <= 256) return f(Plan<T, 1, kOne, false, 256>{threads(1)});
    if (vecs <= 1024) return f(Plan<T, 1, kOne, false, 1024>{threads(1)});
    return f(Plan<T, 4, kOne, false, kWide>{threads(4)});
}

}  // namespace

}  // namespace moe
