// norm.cu -- the norm in front of the expert layer: the residual stream takes a branch's output,
// and its root-mean-square norm goes on, in the stream's type and, where the MXFP8 path reads it,
// as E4M3 codes with scales too:
//   h = x + r;  y = h / sqrt(mean h^2 + eps) w;  codes, scales = MXFP8(y)
// One pass: a row stays in registers between the sum of its squares and its outputs, so x and r
// are read once and h, y and the codes written once, which is all the memory traffic there is
// (what bounds the kernel).
//
// y is the exact quotient rounded once (its codes are then the ones that moe_mx_quantize gives for
// y): squares are added in pairs of fp32 numbers, sum and what its roundings lost (Knuth's TwoSum;
// Dekker 1971, "A floating-point technique for extending the available precision"), 1 / sqrt is
// one Newton step on such a pair, and an element whose fp32 product lies within its error of a
// border between two values of the 16-bit type, one in some thousand, is rounded from the product
// to 48 bits (with its neighbour alone, not its vector: 8192 rows of 7168 fp16 with MXFP8 111 us, and 101). What
// fp32's ends cut, of rows near its largest number, say, is rounded from 64 bits. Two elements go through each
// fp32 instruction (f32x2).
#include "norm.cuh"

namespace moe {

namespace {

// ---------------------------------------------------------------- pairs of fp32 numbers

using F2 = unsigned long long;              // two fp32 values in one 64-bit register

__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 split(F2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 sub2(F2 a, F2 b) { return fma2(b, f2(-1.f, -1.f), a); }

struct Sum2 {                               // two running sums and what their roundings lost
    F2 s, c;
};
__device__ __forceinline__ void add_square(Sum2 &a, F2 h, bool exact) {
    const F2 q = mul2(h, h);                // exact for 16-bit values
    const F2 t = add2(a.s, q);
    const F2 b = sub2(t, a.s);
    a.c = add2(a.c, add2(sub2(a.s, sub2(t, b)), sub2(q, b)));
    if (!exact) a.c = add2(a.c, fma2(h, h, sub2(0ull, q)));
    a.s = t;
}

struct Pair {                               // hi + lo, lo far below hi's last bit
    float hi, lo;
};
__device__ __forceinline__ Pair join(Pair a, Pair b) {
    const float t = __fadd_rn(a.hi, b.hi);
    const float v = __fsub_rn(t, a.hi);
    const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(t, v)), __fsub_rn(b.hi, v));
    return {t, __fadd_rn(__fadd_rn(a.lo, b.lo), e)};
}
// hi + lo with hi the nearest fp32 number to the sum (|hi| >= |lo|)
__device__ __forceinline__ Pair normal(float hi, float lo) {
    const float s = __fadd_rn(hi, lo);
    return {s, __fsub_rn(lo, __fsub_rn(s, hi))};
}

// kUp times 1 / rms, for a sum of H squares of scale h (a power of two). Rows near fp32's largest number have 1 / rms
// below its normal ones, and their elements may lie far below them: at 2^64 as large all of it keeps its digits.
// (1 / rms is 2^50 at most, and products, z of sqrt(H) at most, have room for y up to 2^64.)
constexpr float kUp = 1.8446744073709552e19f, kDown = 5.421010862427522e-20f;   // 2^64, 2^-64
__device__ __forceinline__ Pair inverse_root(Pair sum, float scale, const NormLaunch &p) {
    if (!(sum.hi < __int_as_float(0x7f800000))) return {1.f / sum.hi, 0.f};     // infinity: 0; NaN
    const Pair a = join(sum, {p.h_eps_hi * scale * scale, p.h_eps_lo * scale * scale});
    const Pair n = normal(a.hi, a.lo);
    const float r = rsqrtf(n.hi);
    const float t = __fmul_rn(r, r), tl = fmaf(r, r, -t);
    const float q = __fmul_rn(n.hi, t), ql = fmaf(n.hi, t, -q);
    // 1 - A r^2, then r (1 + e / 2 + 3 e^2 / 8)
    float e = __fsub_rn(__fsub_rn(1.f, q), ql);
    e = fmaf(-n.hi, tl, e);
    e = fmaf(-n.lo, t, e);
    const float rl = __fmul_rn(r, fmaf(__fmul_rn(0.375f, e), e, 0.5f * e));
    const float m = __fmul_rn(r, p.root_h_hi);
    const float ml = fmaf(r, p.root_h_hi, -m);
    const Pair root = normal(m, fmaf(r, p.root_h_lo, fmaf(rl, p.root_h_hi, ml)));
    return {root.hi * (scale * kUp), root.lo * (scale * kUp)};
}

// Where z = h r or y = z w is not between these, they or their low parts may have lost digits to fp32's ends.
constexpr float kLeast = 1.4551915228366852e-11f, kMost = 1.7014118346046923e38f;   // 2^-36, 2^127
__device__ __forceinline__ bool inside(float z, float y) { return fminf(fabsf(z), fabsf(y)) >= kLeast && fabsf(y) < kMost; }

// The smallest and the largest magnitude of three numbers.
__device__ __forceinline__ float least(float a, float b, float c) {
    float r;
    asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float most(float a, float b, float c) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// h r / kUp w rounded once. (h r is taken first: it stays below kUp sqrt(H), where h w may leave fp32's range.) A
// value of more digits is cut to fp32 with its last bit set where digits follow (round to odd): from there it rounds on
// to 16 bits as it would itself.
template <typename T>
__device__ __noinline__ T rounded_once(float h, float w, Pair r) {
    const float z = __fmul_rn(h, r.hi), y = __fmul_rn(z, w);
    if (!inside(z, y)) {                                    // in 64 bits
        if (h == 0.f || w == 0.f) return from_float<T>(y);
        const double v = static_cast<double>(h) * ((static_cast<double>(r.hi) + r.lo) * kDown) * w;
        if constexpr (sizeof(T) == 4) {
            return __double2float_rn(v);
        } else {
            const float f = __double2float_rz(v);
            return from_float<T>(static_cast<double>(f) != v ? __uint_as_float(__float_as_uint(f) | 1u) : f);
        }
    }
    // from some 48 bits
    const float zl = fmaf(h, r.lo, fmaf(h, r.hi, -z));
    const Pair n = normal(y, fmaf(zl, w, fmaf(z, w, -y)));
    if constexpr (sizeof(T) == 4) return n.hi * kDown;
    uint32_t b = __float_as_uint(n.hi);
    if ((b & 1u) == 0u && (n.lo < 0.f || n.lo > 0.f)) b += (n.lo > 0.f) == (n.hi > 0.f) ? 1u : 0xffffffffu;
    return from_float<T>(__uint_as_float(b) * kDown);
}

__device__ __forceinline__ uint32_t pack2(float2 v, __nv_bfloat16) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t pack2(float2 v, __half) {
    const __half2 r = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// ---------------------------------------------------------------- the kernel

// Blocks of the most threads that an SM has room for: left to itself the compiler takes more registers
// (8192 rows of 7168 with MXFP8 122 us, and 92 by this; 4096 rows of 16384 120, and 95; four blocks of a warp a
// row: 65536 rows of 512 54, and 50).
template <typename L>
constexpr int kNormBlocks = L::WARP ? 4 : L::MOST == 256 ? 3 : (L::MOST == 512 ? 2 : 1);

template <typename L>
__global__ void __launch_bounds__(L::MOST, kNormBlocks<L>)
rms_norm_kernel(const NormLaunch p) {
    using T = typename L::T;
    constexpr int N = L::N, V = L::V;
    __shared__ Pair part[32];
    griddep_wait();
    const L lane(p.H);
    const int64_t t = static_cast<int64_t>(blockIdx.x) * L::ROWS + lane.row();
    if (L::ROWS > 1 && t >= p.T) return;                    // whole warps
    const bool edge = t == 0 || t == p.T - 1;
    const T *x = static_cast<const T *>(p.x) + t * p.ld_x;
    Vec<T> h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = lane.template load<true>(x, v, edge);
    if (p.residual != nullptr) {
        const T *r = static_cast<const T *>(p.residual) + t * p.ld_r;
        Vec<T> b[V];
#pragma unroll
        for (int v = 0; v < V; ++v) b[v] = lane.template load<true>(r, v, edge);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < N; ++j) h[v].v[j] = from_float<T>(to_float(h[v].v[j]) + to_float(b[v].v[j]));
    }
    Pair all;
    float scale = 1.f;
#pragma unroll 1
    while (true) {
        Sum2 sum = {0ull, 0ull};
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < N; j += 2)
                add_square(sum, mul2(f2(to_float(h[v].v[j]), to_float(h[v].v[j + 1])), f2(scale, scale)), sizeof(T) == 2);
        const float2 s = split(sum.s), c = split(sum.c);
        all = join({s.x, c.x}, {s.y, c.y});
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            all = join(all, {__shfl_xor_sync(kAll, all.hi, d), __shfl_xor_sync(kAll, all.lo, d)});
        if constexpr (!L::WARP) {
            // every warp adds the warps' sums, in one order
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = all;
            __syncthreads();
            constexpr int WARPS = L::MOST / 32;
            const int w = threadIdx.x & (WARPS - 1);
            all = w < lane.tpr / 32 ? part[w] : Pair{0.f, 0.f};
#pragma unroll
            for (int d = WARPS / 2; d > 0; d >>= 1)
                all = join(all, {__shfl_xor_sync(kAll, all.hi, d), __shfl_xor_sync(kAll, all.lo, d)});
        }
        // a sum that its inverse's digits are lost of, or that left fp32: again, of values 2^-80 as large
        // (the row's threads agree; infinities and NaN stay what they are)
        if (all.hi < 1.2676506e30f || scale != 1.f) break;
        scale = 8.271806125530277e-25f;
        if constexpr (!L::WARP) __syncthreads();
    }
    const Pair r = inverse_root(all, scale, p);
    if (p.rstd != nullptr && lane.i == 0) p.rstd[t] = r.hi * kDown;
    const bool store_h = p.h != nullptr;
    T *ho = static_cast<T *>(p.h) + t * p.H, *yo = static_cast<T *>(p.y) + t * p.H;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (store_h) lane.store(ho, v, h[v]);
        float w[N];
        lane.weight(p.weight, p.w_f32, v, w);
        Vec<T> y;
        if constexpr (sizeof(T) == 4) {
            float low = kMost, top = 0.f, last = 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float z = __fmul_rn(h[v].v[j], r.hi), zl = fmaf(h[v].v[j], r.lo, fmaf(h[v].v[j], r.hi, -z));
                const float o = __fmul_rn(z, w[j]);
                y.v[j] = (o + fmaf(zl, w[j], fmaf(z, w[j], -o))) * kDown;
                low = least(low, z, o);
                if (j & 1) top = most(top, o, last);
                last = o;
            }
            if (low < kLeast || !(top < kMost)) {           // mostly a product of 0, which has no digits to lose
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float z = __fmul_rn(h[v].v[j], r.hi);
                    if (!inside(z, __fmul_rn(z, w[j])) && h[v].v[j] != 0.f && w[j] != 0.f) y.v[j] = rounded_once<T>(h[v].v[j], w[j], r);
                }
            }
        } else {
            uint32_t *out = reinterpret_cast<uint32_t *>(&y.raw);
            uint32_t apart[N / 2], any = 0u;
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                const F2 q = mul2(mul2(f2(to_float(h[v].v[j]), to_float(h[v].v[j + 1])), f2(r.hi, r.hi)), f2(w[j], w[j + 1]));
                // q is good to 3 2^-24: where both ends of its error round alike, so does the product. The upper end is
                // 4 2^-24 up, the lower 9 2^-24 below that; of a q that left fp32, infinity, the lower is NaN.
                constexpr float kHi = kDown * 1.0000002384185791015625f, kLo = kDown * -5.364418029785156e-07f;
                const F2 hi = mul2(q, f2(kHi, kHi)), lo = fma2(q, f2(kLo, kLo), hi);
                out[j / 2] = pack2(split(hi), T());
                any |= apart[j / 2] = out[j / 2] ^ pack2(split(lo), T());
            }
            if (any != 0u) {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (apart[j / 2] != 0u) y.v[j] = rounded_once<T>(to_float(h[v].v[j]), w[j], r);
            }
        }
        if (p.y != nullptr) lane.store(yo, v, y);
        if constexpr (L::ALIGNED) {
            if (p.codes != nullptr) {                       // H is a multiple of 128: whole groups of lanes
                constexpr int B = 32 / N;                   // lanes of a block of 32 columns
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < N; ++j) top = fmaxf(top, fabsf(to_float(y.v[j])));
#pragma unroll
                for (int d = 1; d < B; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
                const uint32_t code = mx_scale_code(top);
                const float inv = mx_inv_scale(code);
                uint32_t q[N / 4];
#pragma unroll
                for (int j = 0; j < N / 4; ++j)
                    q[j] = e4m3x2(to_float(y.v[4 * j]) * inv, to_float(y.v[4 * j + 1]) * inv) |
                           (e4m3x2(to_float(y.v[4 * j + 2]) * inv, to_float(y.v[4 * j + 3]) * inv) << 16);
                // the four blocks of a 128-column word
                const int col = lane.column(v, 0);
                uint32_t word = code << (8 * ((col >> 5) & 3));
                word |= __shfl_xor_sync(kAll, word, B);
                word |= __shfl_xor_sync(kAll, word, 2 * B);
                if (lane.has(v)) {
                    uint8_t *dst = p.codes + t * p.H + col;
                    if constexpr (N == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(q[0], q[1]);
                    else *reinterpret_cast<uint32_t *>(dst) = q[0];
                    if ((col & 127) == 0) p.scales[static_cast<int64_t>(col >> 7) * p.sf_rows + t] = word;
                }
            }
        }
    }
}

template <typename T>
cudaError_t launch_of(const NormLaunch &p, cudaStream_t st) {
    return with_plan<T>(p.H, p.access, [&](auto plan) {
        using L = typename decltype(plan)::L;
        const int64_t blocks = (p.T + L::ROWS - 1) / L::ROWS;
        return launch_dep(rms_norm_kernel<L>, dim3(static_cast<unsigned>(blocks)), dim3(plan.threads), 0, st, p);
    });
}

}  // namespace

cudaError_t launch_rms_norm(const NormLaunch &p, cudaStream_t st) {
    const cudaError_t e = p.dtype == MOE_DTYPE_F32    ? launch_of<float>(p, st)
                          : p.dtype == MOE_DTYPE_BF16 ? launch_of<__nv_bfloat16>(p, st)
                                                      : launch_of<__half>(p, st);
    note_launches(1);
    return e;
}

}  // namespace moe
