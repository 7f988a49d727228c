// multi_tensor.cu -- the end of a training step, over lists of tensors of any sizes
// and types: the global gradient norm, clipping by it, and the AdamW update.
//
//   norm = sqrt(sum x^2), sum |x| or max |x| over every element of every tensor
//   f    = min(1, max_norm / (norm + 1e-6)),  x <- f x
//   AdamW, a parameter's step t:  g = f grad,  m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2
//                   p <- p - lr (wd p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps))
//
// Lists reach the device in the kernels' arguments (pointers, sizes and types), so a
// call copies nothing, keeps nothing and can be captured into a graph. The tensors'
// 16-byte vectors are numbered through the whole list (with some more for each tensor,
// what turning to one costs) and cut into equal runs, a whole number of them for each
// resident block; block b takes runs b, b + grid, ...: the same sums on every call. Runs
// of 128 KB on whole memory lines: 16 KB ones reached 6.15 TB/s in AdamW, 128 KB ones 6.5,
// and runs cut at any vector 5.8.
//
// All three are bound by HBM (of 6.78 TB/s for a plain copy, over 2.8e9 bf16 gradients: the
// norm 0.78 ms, 7.2 TB/s; clipping's second pass 1.79 ms, 6.3 TB/s; AdamW over 5.5e8 bf16
// parameters with fp32 masters 2.38 ms, 6.5 TB/s). The norm reads each element once. Clipping reads and
// writes each once more, from the last run backwards, so that it starts on what the
// norm has left in L2, and does nothing where f is 1. AdamW takes f as it reads the
// gradients, which saves that pass.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include "internal.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kSms = 152;
constexpr int kMaxGrid = kSms * 4;
constexpr int kNormPerSm = 3, kClipPerSm = 3, kAdamPerSm = 2;   // resident blocks
constexpr int64_t kTurn = 256;              // units that turning to a tensor counts for
constexpr int64_t kGrain = 256;             // tensors and runs start on a multiple of these: whole lines of memory
constexpr int64_t kLeast = 1024, kMost = 8192; // units of a run

struct Runs {
    int64_t size, total;                    // units of a run, of the list
    int n;                                  // tensors
};
template <int N>
struct Table {                              // one pointer a tensor
    void *ptr[N];
    int64_t numel[N], unit[N];              // unit: its first one
    uint8_t dtype[N];
    Runs runs;
};
template <int N>
struct AdamTable {
    void *p[N], *g[N], *m[N], *v[N], *x[N];
    int64_t numel[N], unit[N];
    int32_t which[N];                       // its place in the call's list
    uint8_t p_dtype[N], g_dtype[N];
    uint8_t head[N];                        // elements before the first vector of four, kScalar: none
    Runs runs;
};
constexpr uint8_t kScalar = 255;
// a list is launched with the shortest argument block that holds it (1.7, 6.5 or 25 KB: the host
// writes it at every launch, some 3 us for the longest)
constexpr int kShort = 64, kMiddle = 256, kLong = 1000;
constexpr int kAdamShort = 64, kAdamMiddle = 192, kAdamLong = 500;
static_assert(sizeof(Table<kLong>) < 32000 && sizeof(AdamTable<kAdamLong>) < 32000, "kernel arguments");

// A tensor as elements before the first 16-byte vector, vectors, and elements after.
struct Span {
    int64_t head, vecs;
};
__host__ __device__ __forceinline__ Span span_of(const void *ptr, int64_t numel, int size) {
    Span s;
    s.head = static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(ptr) & 15)) & 15) / size;
    if (s.head > numel) s.head = numel;
    s.vecs = (numel - s.head) / (16 / size);
    return s;
}
// The tensor that holds a unit.
__device__ __forceinline__ int find_tensor(const int64_t *unit, int n, int64_t u) {
    int lo = 0, hi = n - 1;                 // the last tensor with unit <= u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (unit[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
__host__ __device__ __forceinline__ int size_of(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

__device__ __forceinline__ float widen(uint32_t bits16, int dtype) {
    return dtype == MOE_DTYPE_BF16 ? __uint_as_float(bits16 << 16)
                                   : __half2float(__ushort_as_half(static_cast<unsigned short>(bits16)));
}
__device__ __forceinline__ uint32_t narrow(float v, int dtype) {
    return dtype == MOE_DTYPE_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ float load_elem(const void *p, int dtype, int64_t i) {
    return dtype == MOE_DTYPE_F32 ? static_cast<const float *>(p)[i]
                                  : widen(static_cast<const unsigned short *>(p)[i], dtype);
}
__device__ __forceinline__ void store_elem(void *p, int dtype, int64_t i, float v) {
    if (dtype == MOE_DTYPE_F32) static_cast<float *>(p)[i] = v;
    else static_cast<unsigned short *>(p)[i] = static_cast<unsigned short>(narrow(v, dtype));
}

// Running value of the norm. Squares are added in fp32 over 64 elements (in four chains:
// 18 roundings at most, which the root halves) and folded into 64 bits: all in 64 bits,
// 1.25 TFLOP/s would hold the norm to a fifth of what memory gives. Where those 64 left fp32's comfortable range (all below 1e-12, or
// some above 1e15) they are added again, scaled by a power of two.
template <int kType>
struct Sum {
    double acc = 0.0;
    uint32_t top = 0;                       // max |x| as bits: NaN is above everything
    __device__ __forceinline__ void fold(const float *x, int n) {
        if constexpr (kType == MOE_NORM_INF) {
#pragma unroll
            for (int i = 0; i < n; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
        } else {
            float q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < n; ++i) {
                if constexpr (kType == MOE_NORM_2) q[i & 3] = fmaf(x[i], x[i], q[i & 3]);
                else q[i & 3] += fabsf(x[i]);
            }
            const float s = (q[0] + q[1]) + (q[2] + q[3]);
            if (s > 1e-24f && s < 1e30f) acc += static_cast<double>(s);
            else if (s != 0.0f || kType == MOE_NORM_2) acc += scaled(x, n, s);
        }
    }
    __device__ __forceinline__ double scaled(const float *x, int n, float s) const {
        const float f = s < 1.0f ? 0x1p96f : 0x1p-96f;
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float y = x[i] * f;
            q += kType == MOE_NORM_2 ? y * y : fabsf(y);
        }
        const double back = s < 1.0f ? 0x1p-96 : 0x1p96;
        return static_cast<double>(q) * (kType == MOE_NORM_2 ? back * back : back);
    }
    __device__ __forceinline__ void join(double v) {
        if constexpr (kType == MOE_NORM_INF) top = max(top, __float_as_uint(static_cast<float>(v)));
        else acc += v;
    }
    __device__ __forceinline__ double get() const {
        return kType == MOE_NORM_INF ? static_cast<double>(__uint_as_float(top)) : acc;
    }
};

// The norm from its sum.
template <int kType>
__device__ __forceinline__ float finish(double v) {
    if (kType != MOE_NORM_2) return static_cast<float>(v);
    if (!(v > 1e-30 && v < 1e38)) return static_cast<float>(sqrt(v));
    // the root in 32 bits, and one step towards that of the 64-bit sum: rounded once, not two and a half
    // times, since clipping multiplies everything by it
    const float r = sqrtf(static_cast<float>(v));
    return r + static_cast<float>(fma(-static_cast<double>(r), static_cast<double>(r), v)) * (0.5f / r);
}

// The block's sum or maximum, in every thread. One warp adds, from shared memory: a 64-bit
// addition takes a warp some 60 cycles, and eight warps that reduce each their own and then
// all the same eight values wait 3 us for them. kFinish: the norm from them.
template <int kType, bool kFinish>
__device__ __forceinline__ double block_value(const Sum<kType> &s) {
    __shared__ double part[kThreads];
    __shared__ double value;
    __syncthreads();
    part[threadIdx.x] = kType == MOE_NORM_INF ? static_cast<double>(__uint_as_float(s.top)) : s.acc;
    __syncthreads();
    if (threadIdx.x < 32) {
        Sum<kType> t;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) t.join(part[threadIdx.x + 32 * i]);
        if constexpr (kType == MOE_NORM_INF) {
            t.top = __reduce_max_sync(0xffffffffu, t.top);
        } else {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) t.acc += __shfl_xor_sync(0xffffffffu, t.acc, off);
        }
        if (threadIdx.x == 0) value = kFinish ? static_cast<double>(finish<kType>(t.get())) : t.get();
    }
    __syncthreads();
    return value;
}

constexpr int kBatch = 8;                   // 16-byte loads of a thread in flight

// A block's part of the norm: its runs.
template <int kType, int N>
__device__ __forceinline__ void sum_runs(const Table<N> &tab, Sum<kType> &sum) {
    for (int64_t u0 = blockIdx.x * tab.runs.size; u0 < tab.runs.total; u0 += gridDim.x * tab.runs.size) {
        const int64_t u1 = min(tab.runs.total, u0 + tab.runs.size);
        for (int i = find_tensor(tab.unit, tab.runs.n, u0); i < tab.runs.n && tab.unit[i] < u1; ++i) {
            const int dtype = tab.dtype[i], size = size_of(dtype);
            const int64_t numel = tab.numel[i];
            const Span s = span_of(tab.ptr[i], numel, size);
            const int64_t lo = max(u0 - tab.unit[i], static_cast<int64_t>(0)), end = u1 - tab.unit[i], hi = min(end, s.vecs);
            const uint4 *body = reinterpret_cast<const uint4 *>(static_cast<const char *>(tab.ptr[i]) + s.head * size);
            for (int64_t v = lo + threadIdx.x; v < hi; v += kThreads * kBatch) {
                uint4 r[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    r[j] = v + j * kThreads < hi ? __ldcg(body + v + j * kThreads) : make_uint4(0u, 0u, 0u, 0u);
                if (dtype == MOE_DTYPE_F32) {
                    float x[4 * kBatch];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        x[4 * j] = __uint_as_float(r[j].x);
                        x[4 * j + 1] = __uint_as_float(r[j].y);
                        x[4 * j + 2] = __uint_as_float(r[j].z);
                        x[4 * j + 3] = __uint_as_float(r[j].w);
                    }
                    sum.fold(x, 4 * kBatch);
                } else {
                    float x[8 * kBatch];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) {
                        const uint32_t w[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            x[8 * j + 2 * q] = widen(w[q] & 0xffffu, dtype);
                            x[8 * j + 2 * q + 1] = widen(w[q] >> 16, dtype);
                        }
                    }
                    sum.fold(x, 8 * kBatch);
                }
            }
            if (lo <= s.vecs && s.vecs < end) {          // the unit after the vectors: the odd elements
                const int64_t gap = s.vecs * (16 / size);
                for (int64_t e = threadIdx.x; e < numel - gap; e += kThreads) {
                    const float x[1] = {load_elem(tab.ptr[i], dtype, e < s.head ? e : e + gap)};
                    sum.fold(x, 1);
                }
            }
        }
    }
}

template <int kType, int N>
__global__ void __launch_bounds__(kThreads, kNormPerSm)
norm_kernel(const __grid_constant__ Table<N> tab, double *__restrict__ part, int32_t *__restrict__ step) {
    griddep_wait();
    if (step != nullptr && blockIdx.x == 0 && threadIdx.x == 0) ++*step;   // AdamW's, which comes next
    Sum<kType> sum;
    sum_runs<kType>(tab, sum);
    const double v = block_value<kType, false>(sum);
    if (threadIdx.x == 0) part[blockIdx.x] = v;
}

// The norm from the blocks' values, in order; the same in every block that asks.
template <int kType>
__device__ __forceinline__ float total_norm(const double *__restrict__ part, int n) {
    Sum<kType> s;
    for (int i = threadIdx.x; i < n; i += kThreads) s.join(__ldcg(part + i));
    return static_cast<float>(block_value<kType, true>(s));
}

// max_norm / (norm + 1e-6), at most 1; NaN stays NaN
__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
    const float f = max_norm / (norm + 1e-6f);
    return f > 1.0f ? 1.0f : f;
}

template <int kType>
__global__ void __launch_bounds__(kThreads)
norm_total_kernel(const double *__restrict__ part, int n, float *__restrict__ norm) {
    griddep_wait();
    const float v = total_norm<kType>(part, n);
    if (threadIdx.x == 0) *norm = v;
}

// A block's part of the scaling: its runs, from the last backwards.
template <int N>
__device__ __forceinline__ void scale_runs(const Table<N> &tab, float f) {
    const int64_t runs = (tab.runs.total + tab.runs.size - 1) / tab.runs.size;
    for (int64_t c = runs - 1 - static_cast<int64_t>(blockIdx.x); c >= 0; c -= gridDim.x) {
        const int64_t u0 = c * tab.runs.size, u1 = min(tab.runs.total, u0 + tab.runs.size);
        for (int i = find_tensor(tab.unit, tab.runs.n, u1 - 1); i >= 0; --i) {
            const int dtype = tab.dtype[i], size = size_of(dtype);
            const int64_t numel = tab.numel[i];
            const Span s = span_of(tab.ptr[i], numel, size);
            const int64_t lo = max(u0 - tab.unit[i], static_cast<int64_t>(0)), end = u1 - tab.unit[i], hi = min(end, s.vecs);
            uint4 *body = reinterpret_cast<uint4 *>(static_cast<char *>(tab.ptr[i]) + s.head * size);
            for (int64_t v = hi - 1 - static_cast<int64_t>(threadIdx.x); v >= lo; v -= kThreads * kBatch) {
                uint4 r[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (v - j * kThreads >= lo) r[j] = body[v - j * kThreads];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (v - j * kThreads < lo) continue;
                    uint32_t w[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (dtype == MOE_DTYPE_F32)
                            w[q] = __float_as_uint(__uint_as_float(w[q]) * f);
                        else
                            w[q] = narrow(widen(w[q] & 0xffffu, dtype) * f, dtype) |
                                   narrow(widen(w[q] >> 16, dtype) * f, dtype) << 16;
                    }
                    body[v - j * kThreads] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (lo <= s.vecs && s.vecs < end) {
                const int64_t gap = s.vecs * (16 / size);
                for (int64_t k = threadIdx.x; k < numel - gap; k += kThreads) {
                    const int64_t e = k < s.head ? k : k + gap;
                    store_elem(tab.ptr[i], dtype, e, load_elem(tab.ptr[i], dtype, e) * f);
                }
            }
            if (tab.unit[i] <= u0) break;
        }
    }
}

template <int kType, int N>
__global__ void __launch_bounds__(kThreads, kClipPerSm)
clip_kernel(const __grid_constant__ Table<N> tab, const double *__restrict__ part, int n_part, float max_norm,
            float *__restrict__ norm) {
    griddep_wait();
    const float total = total_norm<kType>(part, n_part);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    const float f = clip_factor(total, max_norm);
    if (f == 1.0f) return;                  // x * 1 = x
    scale_runs(tab, f);
}

// A short list of no more than kSmall units in one launch: a cluster of eight blocks, which
// exchange their sums through shared memory. It saves the host a launch, for which eight SMs take
// longer than fifty. Three bf16 tensors clipped, us a call one after another (us on the device),
// one launch against two: 30 K elements 9.3 (5.2), 10.9 (7.1); 0.2 M 9.5 (9.4), 11.0 (7.3); 0.3 M,
// 38 K units, 10.4 (10.4), 11.2 (7.1); 0.4 M, 51 K units, 12.6 (12.5), 11.0 (7.9). fp32, with half
// the elements to a unit, and the norm alone take less on the device, and one launch pays up to
// 300 K units. (In a replayed graph, where the device alone counts, two pay from 0.1 M on.)
constexpr int kCluster = 8;
constexpr int64_t kSmall = 32768;

template <int kType, bool kClip>
__global__ void __launch_bounds__(kThreads)
small_kernel(const __grid_constant__ Table<kShort> tab, float max_norm, float *__restrict__ norm) {
    griddep_wait();
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ double mine;
    Sum<kType> sum;
    sum_runs<kType>(tab, sum);
    const double v = block_value<kType, false>(sum);
    if (threadIdx.x == 0) mine = v;
    cluster.sync();
    __shared__ float norm_shared;
    if (threadIdx.x == 0) {
        Sum<kType> all;
#pragma unroll
        for (int i = 0; i < kCluster; ++i) all.join(*cluster.map_shared_rank(&mine, i));
        norm_shared = finish<kType>(all.get());
    }
    cluster.sync();                         // the sums are read while their blocks last
    const float total = norm_shared;
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    if constexpr (kClip) {
        const float f = clip_factor(total, max_norm);
        if (f != 1.0f) scale_runs(tab, f);
    }
}

// Where AdamW needs no norm, the count of its step alone.
__global__ void adamw_count_kernel(int32_t *__restrict__ step) {
    griddep_wait();
    ++*step;
}

// What a step is made of; step[0] has been counted up. `undo`: the last launch of a step, which
// takes the count back where the step is skipped.
struct AdamConst {
    float beta1, beta2, rest1, rest2;       // rest: 1 - beta, rounded from 64 bits (of a rounded 0.999 it is off by 1.3e-5)
    float eps, weight_decay, max_norm;
    double ln_beta1, ln_beta2;
    const double *part;
    int n_part, skip_nonfinite, undo;
    const float *lr;
    int32_t *step;
    const int32_t *missed;
    float *norm;
};
struct Hyper {
    float factor, lr, inv_c1, inv_c2;
    int skip;
};

// 1 / (1 - b^t) for both b. 1 - b^t = -expm1(t ln b): ln b comes from the host in 64 bits, and
// expm1 keeps fp32's digits where b^t is near 1.
__device__ __forceinline__ float2 corrections(const AdamConst &k, int t) {
    return make_float2(-1.0f / expm1f(static_cast<float>(t * k.ln_beta1)), -1.0f / expm1f(static_cast<float>(t * k.ln_beta2)));
}

// The step's numbers, in every block, through its shared memory; where parameters have missed
// steps (`own`: one a tensor of the table), their corrections by their own counts.
template <int N>
__device__ __forceinline__ void begin_step(const AdamConst &k, const AdamTable<N> &tab, Hyper &h, float2 *own) {
    const float total = k.n_part > 0 ? total_norm<MOE_NORM_2>(k.part, k.n_part) : 0.0f;
    if (threadIdx.x == 0) {
        h.skip = k.skip_nonfinite && !isfinite(total);
        h.factor = k.n_part > 0 && k.max_norm > 0.0f ? clip_factor(total, k.max_norm) : 1.0f;
        const int t = *k.step;
        h.lr = *k.lr;
        const float2 c = corrections(k, t);
        h.inv_c1 = c.x;
        h.inv_c2 = c.y;
        if (blockIdx.x == 0) {
            if (k.n_part > 0 && k.norm != nullptr) *k.norm = total;
            if (h.skip && k.undo) *k.step = t - 1;
        }
    }
    if (k.missed != nullptr) {
        const int t = *k.step;
        for (int i = threadIdx.x; i < tab.runs.n; i += kThreads) own[i] = corrections(k, max(1, t - k.missed[tab.which[i]]));
    }
    __syncthreads();
}

__device__ __forceinline__ void adam_element(const Hyper &h, const AdamConst &c, float grad, float &m, float &v, float &p) {
    const float g = grad * h.factor;
    m = c.beta1 * m + c.rest1 * g;
    v = c.beta2 * v + c.rest2 * g * g;
    const float u = m * h.inv_c1 / (sqrtf(v * h.inv_c2) + c.eps);
    p = p - h.lr * (c.weight_decay * p + u);
}

// Four elements as they lie in memory: 16 bytes of fp32, 8 of a 16-bit type (in x, y).
__device__ __forceinline__ uint4 load_four(const void *p, int dtype, int64_t i) {
    if (dtype == MOE_DTYPE_F32) return __ldcs(reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i));
    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const unsigned short *>(p) + i));
    return make_uint4(v.x, v.y, 0u, 0u);
}
__device__ __forceinline__ uint32_t load_bits(const void *p, int dtype, int64_t i) {
    return dtype == MOE_DTYPE_F32 ? __ldcs(static_cast<const unsigned int *>(p) + i)
                                  : __ldcs(static_cast<const unsigned short *>(p) + i);
}
__device__ __forceinline__ float bits_float(uint32_t r, int dtype) {
    return dtype == MOE_DTYPE_F32 ? __uint_as_float(r) : widen(r, dtype);
}
__device__ __forceinline__ float4 four_floats(const uint4 &r, int dtype) {
    if (dtype == MOE_DTYPE_F32)
        return make_float4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w));
    return make_float4(widen(r.x & 0xffffu, dtype), widen(r.x >> 16, dtype), widen(r.y & 0xffffu, dtype),
                       widen(r.y >> 16, dtype));
}

// 28 bytes an element with bf16 parameters and gradients and fp32 masters, and some 20
// operations: bound by HBM, so by the loads in flight. A thread has two groups of four
// elements of every operand under way before it computes (112 bytes); operands are
// converted after all loads are issued. Where a parameter's operands are never aligned
// together, it is eight single elements of each.
template <int N>
__global__ void __launch_bounds__(kThreads, kAdamPerSm)
adamw_kernel(const __grid_constant__ AdamTable<N> tab, const __grid_constant__ AdamConst k) {
    griddep_wait();
    __shared__ Hyper shared;
    __shared__ float2 own[N];
    begin_step(k, tab, shared, own);
    Hyper h = shared;
    if (h.skip) return;
    for (int64_t u0 = blockIdx.x * tab.runs.size; u0 < tab.runs.total; u0 += gridDim.x * tab.runs.size) {
        const int64_t u1 = min(tab.runs.total, u0 + tab.runs.size);
        for (int i = find_tensor(tab.unit, tab.runs.n, u0); i < tab.runs.n && tab.unit[i] < u1; ++i) {
            const int pt = tab.p_dtype[i], gt = tab.g_dtype[i];
            if (k.missed != nullptr) {
                h.inv_c1 = own[i].x;
                h.inv_c2 = own[i].y;
            }
            float *m = static_cast<float *>(tab.m[i]), *v = static_cast<float *>(tab.v[i]);
            float *x = static_cast<float *>(tab.x[i]);
            const void *pin = x != nullptr ? x : tab.p[i];
            const int xt = x != nullptr ? MOE_DTYPE_F32 : pt;
            const int64_t numel = tab.numel[i];
            const bool scalar = tab.head[i] == kScalar;
            const int64_t head = scalar ? 0 : min(numel, static_cast<int64_t>(tab.head[i]));
            const int64_t vecs = (numel - head) / 4;
            const int64_t lo = max(u0 - tab.unit[i], static_cast<int64_t>(0)), last = u1 - tab.unit[i];
            const int64_t begin = head + 4 * lo, end = head + 4 * min(last, vecs);
            if (scalar) {
                constexpr int kU = 8;
                for (int64_t e = begin + threadIdx.x; e < end; e += kThreads * kU) {
                    uint32_t rg[kU], rp[kU];
                    float rm[kU], rv[kU];
#pragma unroll
                    for (int j = 0; j < kU; ++j) {
                        const int64_t a = e + j * kThreads;
                        if (a >= end) break;
                        rg[j] = load_bits(tab.g[i], gt, a);
                        rm[j] = __ldcs(m + a);
                        rv[j] = __ldcs(v + a);
                        rp[j] = load_bits(pin, xt, a);
                    }
#pragma unroll
                    for (int j = 0; j < kU; ++j) {
                        const int64_t a = e + j * kThreads;
                        if (a >= end) break;
                        float p = bits_float(rp[j], xt);
                        adam_element(h, k, bits_float(rg[j], gt), rm[j], rv[j], p);
                        __stcs(m + a, rm[j]);
                        __stcs(v + a, rv[j]);
                        if (x != nullptr) __stcs(x + a, p);
                        store_elem(tab.p[i], pt, a, p);
                    }
                }
            } else {
                constexpr int kU = 2;
                for (int64_t e = begin + threadIdx.x * 4; e < end; e += kThreads * 4 * kU) {
                    uint4 rg[kU], rp[kU];
                    float4 rm[kU], rv[kU];
#pragma unroll
                    for (int j = 0; j < kU; ++j) {
                        const int64_t a = e + j * kThreads * 4;
                        if (a >= end) break;
                        rg[j] = load_four(tab.g[i], gt, a);
                        rm[j] = __ldcs(reinterpret_cast<const float4 *>(m + a));
                        rv[j] = __ldcs(reinterpret_cast<const float4 *>(v + a));
                        rp[j] = load_four(pin, xt, a);
                    }
#pragma unroll
                    for (int j = 0; j < kU; ++j) {
                        const int64_t a = e + j * kThreads * 4;
                        if (a >= end) break;
                        const float4 g = four_floats(rg[j], gt);
                        float4 p = four_floats(rp[j], xt);
                        adam_element(h, k, g.x, rm[j].x, rv[j].x, p.x);
                        adam_element(h, k, g.y, rm[j].y, rv[j].y, p.y);
                        adam_element(h, k, g.z, rm[j].z, rv[j].z, p.z);
                        adam_element(h, k, g.w, rm[j].w, rv[j].w, p.w);
                        __stcs(reinterpret_cast<float4 *>(m + a), rm[j]);
                        __stcs(reinterpret_cast<float4 *>(v + a), rv[j]);
                        if (x != nullptr) __stcs(reinterpret_cast<float4 *>(x + a), p);
                        if (pt == MOE_DTYPE_F32) {
                            __stcs(reinterpret_cast<float4 *>(static_cast<float *>(tab.p[i]) + a), p);
                        } else {
                            const uint2 o =
                                make_uint2(narrow(p.x, pt) | narrow(p.y, pt) << 16, narrow(p.z, pt) | narrow(p.w, pt) << 16);
                            __stcs(reinterpret_cast<uint2 *>(static_cast<unsigned short *>(tab.p[i]) + a), o);
                        }
                    }
                }
            }
            if (lo <= vecs && vecs < last && threadIdx.x < numel - 4 * vecs) {   // the odd elements, at most six
                const int64_t e = threadIdx.x < head ? threadIdx.x : threadIdx.x + 4 * vecs;
                float mv = m[e], vv = v[e], pv = load_elem(pin, xt, e);
                adam_element(h, k, load_elem(tab.g[i], gt, e), mv, vv, pv);
                m[e] = mv;
                v[e] = vv;
                if (x != nullptr) x[e] = pv;
                store_elem(tab.p[i], pt, e, pv);
            }
        }
    }
}

int64_t grains(int64_t units) { return (units + kGrain - 1) / kGrain * kGrain; }

// Equal runs of `total` units, as many a block as keep them under kMost; returns the number
// of blocks.
int make_runs(Runs &r, int n, int64_t total, int resident) {
    int64_t blocks = (total + kLeast - 1) / kLeast;
    blocks = blocks < 1 ? 1 : blocks > resident ? resident : blocks;
    const int64_t each = (total + blocks * kMost - 1) / (blocks * kMost);
    r.n = n;
    r.total = total;
    r.size = each > 0 ? grains((total + blocks * each - 1) / (blocks * each)) : kGrain;
    return static_cast<int>(blocks);
}

// The next at most N tensors of a list that are not empty, from `at` on; returns their units.
template <int N>
int64_t fill_table(const TensorList &l, int &at, Table<N> &t, int &n) {
    int64_t total = 0;
    n = 0;
    for (; at < l.n && n < N; ++at) {
        if (l.numel[at] == 0) continue;
        t.ptr[n] = const_cast<void *>(l.ptr[at]);
        t.numel[n] = l.numel[at];
        t.dtype[n] = static_cast<uint8_t>(l.dtype[at]);
        t.unit[n] = total;
        total += grains(span_of(l.ptr[at], l.numel[at], size_of(l.dtype[at])).vecs + 1 + kTurn);
        ++n;
    }
    return total;
}

// The list as tables of at most N tensors: f(table, blocks) for each.
template <int N, typename F>
cudaError_t for_tables(const TensorList &l, int most, F f) {
    static_assert(std::is_trivially_copyable<Table<N>>::value, "passed as an argument");
    int at = 0;
    do {
        Table<N> t;
        int n = 0;
        const int64_t total = fill_table(l, at, t, n);
        const int blocks = make_runs(t.runs, n, total, most);
        const cudaError_t e = f(t, blocks);
        if (e != cudaSuccess) return e;
    } while (at < l.n);
    return cudaSuccess;
}

// A short and small list in one launch; false: it is not one.
template <int kType, bool kClip>
bool launch_small(const TensorList &l, float max_norm, float *norm, cudaStream_t st, cudaError_t *err) {
    if (l.n > kShort) return false;
    Table<kShort> t;
    int at = 0, n = 0;
    const int64_t total = fill_table(l, at, t, n);
    if (total > kSmall) return false;
    t.runs.n = n;
    t.runs.total = total;
    t.runs.size = total > 0 ? grains((total + kCluster - 1) / kCluster) : kGrain;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    *err = cudaLaunchKernelEx(&cfg, small_kernel<kType, kClip>, t, max_norm, norm);
    note_launches(1);
    return true;
}

double *partials(void *ws) { return static_cast<double *>(ws); }

template <int kType, int N>
cudaError_t norm_parts(const TensorList &l, void *ws, int32_t *step, int *n_part, cudaStream_t st) {
    *n_part = 0;
    return for_tables<N>(l, kSms * kNormPerSm, [&](const Table<N> &t, int grid) {
        const cudaError_t e = launch_dep(norm_kernel<kType, N>, dim3(grid), dim3(kThreads), 0, st, t, partials(ws) + *n_part,
                                         *n_part == 0 ? step : static_cast<int32_t *>(nullptr));
        note_launches(1);
        *n_part += grid;
        return e;
    });
}

template <int kType, int N>
cudaError_t clip_parts(const TensorList &l, float max_norm, float *norm, void *ws, int n_part, cudaStream_t st) {
    return for_tables<N>(l, kSms * kClipPerSm, [&](const Table<N> &t, int grid) {
        const cudaError_t e = launch_dep(clip_kernel<kType, N>, dim3(grid), dim3(kThreads), 0, st, t,
                                         static_cast<const double *>(partials(ws)), n_part, max_norm, norm);
        note_launches(1);
        return e;
    });
}

template <int kType>
cudaError_t norm_typed(const TensorList &l, void *ws, int32_t *step, int *n_part, cudaStream_t st) {
    if (l.n <= kShort) return norm_parts<kType, kShort>(l, ws, step, n_part, st);
    if (l.n <= kMiddle) return norm_parts<kType, kMiddle>(l, ws, step, n_part, st);
    return norm_parts<kType, kLong>(l, ws, step, n_part, st);
}

template <typename F>
cudaError_t with_norm_type(int type, F f) {
    if (type == MOE_NORM_1) return f(std::integral_constant<int, MOE_NORM_1>{});
    if (type == MOE_NORM_2) return f(std::integral_constant<int, MOE_NORM_2>{});
    return f(std::integral_constant<int, MOE_NORM_INF>{});
}

// Elements until every operand of a parameter is aligned for groups of four, kScalar where
// they never are together.
uint8_t vector_head(const AdamwLaunch &p, int i) {
    auto aligned = [](const void *q, int32_t dtype, int h) {
        const uintptr_t size = dtype == MOE_DTYPE_F32 ? 4 : 2;
        return (reinterpret_cast<uintptr_t>(q) + h * size) % (4 * size) == 0;
    };
    for (int h = 0; h < 4; ++h) {
        if (aligned(p.params.ptr[i], p.params.dtype[i], h) && aligned(p.grads.ptr[i], p.grads.dtype[i], h) &&
            aligned(p.exp_avg[i], MOE_DTYPE_F32, h) && aligned(p.exp_avg_sq[i], MOE_DTYPE_F32, h) &&
            (p.masters == nullptr || p.masters[i] == nullptr || aligned(p.masters[i], MOE_DTYPE_F32, h)))
            return static_cast<uint8_t>(h);
    }
    return kScalar;
}

template <int N>
cudaError_t adamw_tables(const AdamwLaunch &p, AdamConst k, cudaStream_t st) {
    int at = 0;
    do {
        AdamTable<N> t;
        int n = 0;
        int64_t total = 0;
        for (; at < p.params.n && n < N; ++at) {
            const int64_t numel = p.params.numel[at];
            if (numel == 0) continue;
            t.p[n] = const_cast<void *>(p.params.ptr[at]);
            t.g[n] = const_cast<void *>(p.grads.ptr[at]);
            t.m[n] = p.exp_avg[at];
            t.v[n] = p.exp_avg_sq[at];
            t.x[n] = p.masters != nullptr ? p.masters[at] : nullptr;
            t.numel[n] = numel;
            t.which[n] = at;
            t.p_dtype[n] = static_cast<uint8_t>(p.params.dtype[at]);
            t.g_dtype[n] = static_cast<uint8_t>(p.grads.dtype[at]);
            t.head[n] = vector_head(p, at);
            t.unit[n] = total;
            total += grains(numel / 4 + 1 + kTurn);
            ++n;
        }
        while (at < p.params.n && p.params.numel[at] == 0) ++at;
        k.undo = at == p.params.n;
        const int blocks = make_runs(t.runs, n, total, kSms * kAdamPerSm);
        const cudaError_t e = launch_dep(adamw_kernel<N>, dim3(blocks), dim3(kThreads), 0, st, t, k);
        note_launches(1);
        if (e != cudaSuccess) return e;
    } while (at < p.params.n);
    return cudaSuccess;
}

}  // namespace

size_t multi_tensor_ws_bytes(int64_t n) {
    const int64_t tables = n <= kLong ? 1 : (n + kLong - 1) / kLong;
    return static_cast<size_t>(tables) * kMaxGrid * sizeof(double);
}

cudaError_t launch_grad_norm(const TensorList &grads, int norm_type, float *norm, void *ws, cudaStream_t st) {
    return with_norm_type(norm_type, [&](auto type) {
        constexpr int kType = decltype(type)::value;
        int n_part = 0;
        cudaError_t e;
        if (launch_small<kType, false>(grads, 0.0f, norm, st, &e)) return e;
        e = norm_typed<kType>(grads, ws, nullptr, &n_part, st);
        if (e != cudaSuccess) return e;
        e = launch_dep(norm_total_kernel<kType>, dim3(1), dim3(kThreads), 0, st,
                       static_cast<const double *>(partials(ws)), n_part, norm);
        note_launches(1);
        return e;
    });
}

cudaError_t launch_clip_grads(const TensorList &grads, int norm_type, float max_norm, float *norm, void *ws,
                              cudaStream_t st) {
    return with_norm_type(norm_type, [&](auto type) {
        constexpr int kType = decltype(type)::value;
        int n_part = 0;
        cudaError_t e;
        if (launch_small<kType, true>(grads, max_norm, norm, st, &e)) return e;
        e = norm_typed<kType>(grads, ws, nullptr, &n_part, st);
        if (e != cudaSuccess) return e;
        if (grads.n <= kShort) return clip_parts<kType, kShort>(grads, max_norm, norm, ws, n_part, st);
        if (grads.n <= kMiddle) return clip_parts<kType, kMiddle>(grads, max_norm, norm, ws, n_part, st);
        return clip_parts<kType, kLong>(grads, max_norm, norm, ws, n_part, st);
    });
}

cudaError_t launch_adamw(const AdamwLaunch &p, cudaStream_t st) {
    AdamConst k = {};
    k.beta1 = static_cast<float>(p.beta1);
    k.beta2 = static_cast<float>(p.beta2);
    k.rest1 = static_cast<float>(1.0 - p.beta1);
    k.rest2 = static_cast<float>(1.0 - p.beta2);
    k.eps = p.eps;
    k.weight_decay = p.weight_decay;
    k.max_norm = p.max_norm;
    k.ln_beta1 = log(p.beta1);
    k.ln_beta2 = log(p.beta2);
    k.part = partials(p.ws);
    k.skip_nonfinite = p.skip_nonfinite;
    k.lr = p.lr;
    k.step = p.step;
    k.missed = p.missed;
    k.norm = p.norm;
    cudaError_t e;
    if (p.norm != nullptr || p.max_norm > 0.0f || p.skip_nonfinite) {
        e = norm_typed<MOE_NORM_2>(p.grads, p.ws, p.step, &k.n_part, st);
    } else {
        e = launch_dep(adamw_count_kernel, dim3(1), dim3(1), 0, st, p.step);
        note_launches(1);
    }
    if (e != cudaSuccess) return e;
    if (p.params.n <= kAdamShort) return adamw_tables<kAdamShort>(p, k, st);
    if (p.params.n <= kAdamMiddle) return adamw_tables<kAdamMiddle>(p, k, st);
    return adamw_tables<kAdamLong>(p, k, st);
}

}  // namespace moe
