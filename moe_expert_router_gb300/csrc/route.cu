// route.cu -- the trainable router: selection from given logits with its balance
// terms, the backward of both, and the update of the selection bias.
//
// Forward, for token t with logits l (fp32, bf16 or fp16, converted to fp32):
//   expert e is off when l[e] = -inf; a token is live when its mask is set and not
//   all experts are off
//   s   = softmax(l) or sigmoid(l)
//   key = l without a selection bias (s increases with l), else s + bias
//   K   = the k best keys of the kept groups, ties to the lower index
//   w   = s_K / (sum_K s + 1e-20) * scale, or s_K * scale
// and for sequence b (n_b live tokens, c_be slots on expert e)
//   balance = 1/S' sum_b sum_e E c_be / (k n_b) P_be,  P_be = 1/n_b sum_t s[t,e] / (sum s[t,:] + 1e-20)
//   z       = 1/N sum_t log(sum_e exp(l[t,e]))^2
//
// A token is held by G lanes of a warp, each keeping V experts in registers: up to eight
// consecutive ones, so that index order is lane order.
// The k best are found in one of three ways:
//   16-bit logits, no bias: key and index share one word. k <= 8: every lane sorts its
//     keys, and the eight best of two lanes are merged log2 G times; larger k: k rounds
//     of a maximum over the lanes and a clearing, without a branch.
//   other keys, G >= 16: the few that can be chosen are gathered, one a lane, and ranked.
//   else: k rounds of a maximum, a ballot, and the winning lane looking up its next best.
//
// Keys that pass through exp carry an error of some 1e-7, and two experts nearer than
// that would be chosen by rounding. Neighbouring chosen keys, the last of them and whatever
// stands behind it, and the group sums at the border, are compared with the bound of that
// error; experts of the same logit and bias are a tie, whatever the error. The rare token
// below it (one in some thousand) is decided in 64 bits, on the experts that matter, one a
// lane: the 64-bit pipe takes some 60 cycles for an instruction, so that scoring every expert
// there cost such a token 20 us.
//
// Bound by instructions, not by memory: 131072 tokens of 128 bf16 experts (34 MB, 5 us of
// HBM) take 58 us at 335 warp instructions a token and 0.61 issued a cycle, with 24 warps
// an SM; their backward (67 MB) 39 us at 238. At 8192 tokens of 256 experts in groups (22
// us, 11.5 us for the backward) the latency of a block's three passes is what is left.
//
// Statistics are sums without float atomics: a block keeps its tokens' score sums
// in registers and its counts in shared memory, and writes them to a slot of its
// own at the end of each sequence it meets (slot = block + sequence: consecutive
// (block, sequence) pairs never share one); route_reduce_kernel adds the slots of a
// sequence in a fixed order, so every output has the same bits on every call. They are held in
// 32 bits: a thread adds no more than 64 tokens in a row (a block has no more passes), a block
// its rows at its end, and the slots, and the sequences in the losses, with the rounding of each
// addition kept, so that the error stays at some 2^-24 x 120 at worst however many tokens there
// are (with one block's tokens added one by one, 134 million of them were 8e-5 off).
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include "internal.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

// Threads of a block; with 32 experts a lane fewer, for their shared memory.
template <int V>
constexpr int kBlock = V > 16 ? 128 : 256;
constexpr int kMaxK = 32;
constexpr int kMaxGroups = 32;
constexpr float kEps = 1e-20f;
// Bounds of the relative error of a 32-bit score, in units of 2^-24. Sigmoid: exp (2 ulp),
// an addition, a reciprocal (1 ulp). Softmax with V experts a lane: the sum's V + 5 additions,
// two exps' worth, a division and a product (the rounding of l - max is at most 2^-24 of the
// row's largest score, and is added apart).
constexpr float kUlp = 6e-8f;
constexpr float kSigmoidErr = 8.0f * kUlp;
template <int V>
__device__ constexpr float softmax_err() { return (V + 12) * kUlp; }
// Weights, shares and gradients are made of the same 32-bit scores (64-bit ones would cost what
// the 64-bit selection costs, for every token): 6e-8 to 1.6e-7 off, where 64-bit scores rounded
// at the end are 5e-8 to 1.2e-7 off. The approximate forms are within those bounds: ex2 (2 ulp),
// rcp (1 ulp), a quotient of 2 ulp, and for a token's log(sum) an absolute 4e-7 (lg2's 2^-21.4 near
// 1, 3 ulp above): the accurate log took 131072 tokens of 128 experts from 108 to 112 us.

__device__ __forceinline__ float from_bits16(uint32_t v, int dtype) {
    if (dtype == MOE_DTYPE_BF16) return __uint_as_float(v << 16);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(v)));
}

__device__ __forceinline__ float load_one(const void *p, int dtype, int64_t i) {
    if (dtype == MOE_DTYPE_F32) return __ldg(static_cast<const float *>(p) + i);
    return from_bits16(__ldg(static_cast<const unsigned short *>(p) + i), dtype);
}

// A lane's experts: e0 + at<V>(i). Up to eight are consecutive; more (of a whole warp then) come
// in fours, each four next to the neighbouring lane's, so that the warp's 16-byte accesses to
// global and shared memory are consecutive (in one run a lane they met in the same banks, and
// E = 832 took 2.2 times as long). There index order is not lane order, and ties compare indices.
template <int V>
__host__ __device__ constexpr int at(int i) { return V <= 8 ? i : (i >> 2) * 128 + (i & 3); }
template <int V>
__device__ __forceinline__ int first_expert(int sub) { return sub * (V <= 8 ? V : 4); }

// The lane's experts of the row at element `row`; -inf past E. `vec`: the rows
// are 16-byte aligned.
template <int V>
__device__ __forceinline__ void load_experts(const void *p, int dtype, int vec, int64_t row, int e0, int E,
                                             float (&l)[V]) {
    if constexpr (V <= 8) {
        if (!vec || e0 + V > E) {
#pragma unroll
            for (int i = 0; i < V; ++i) l[i] = e0 + i < E ? load_one(p, dtype, row + e0 + i) : -INFINITY;
            return;
        }
    }
    // fours, and for 16-bit types the eight of V = 8 at once
    if (dtype == MOE_DTYPE_F32) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const int e = e0 + at<V>(i);
            if (V > 8 && !(vec && e + 4 <= E)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) l[i + j] = e + j < E ? load_one(p, dtype, row + e + j) : -INFINITY;
                continue;
            }
            const float4 x = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + row + e));
            l[i] = x.x;
            l[i + 1] = x.y;
            l[i + 2] = x.z;
            l[i + 3] = x.w;
        }
        return;
    }
    const unsigned short *h = static_cast<const unsigned short *>(p) + row + e0;
    uint2 x[V / 4];
    if constexpr (V == 8) {
        const uint4 y = __ldg(reinterpret_cast<const uint4 *>(h));
        x[0] = make_uint2(y.x, y.y);
        x[1] = make_uint2(y.z, y.w);
    } else {
        const unsigned off = dtype == MOE_DTYPE_BF16 ? 0xff80u : 0xfc00u;      // -inf
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const int e = at<V>(4 * i);
            if (V <= 8 || (vec && e0 + e + 4 <= E)) {
                x[i] = __ldg(reinterpret_cast<const uint2 *>(h + e));
            } else {
                unsigned w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = e0 + e + j < E ? __ldg(h + e + j) : off;
                x[i] = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
            }
        }
    }
    if (dtype == MOE_DTYPE_BF16) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            l[4 * i] = __uint_as_float(x[i].x << 16);
            l[4 * i + 1] = __uint_as_float(x[i].x & 0xffff0000u);
            l[4 * i + 2] = __uint_as_float(x[i].y << 16);
            l[4 * i + 3] = __uint_as_float(x[i].y & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&x[i].x));
            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&x[i].y));
            l[4 * i] = a.x;
            l[4 * i + 1] = a.y;
            l[4 * i + 2] = b.x;
            l[4 * i + 3] = b.y;
        }
    }
}

// 2^x (2 ulp). softmax's exp(l - top) is taken as 2^((l - top) log2 e), whose exponent has
// two roundings: 2^-23 |x| 2^x of the row's largest score, less than 2^-24 of it.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float rcp_fast(float x) {       // 1 ulp
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN where either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// A float's bits in the order of signed compares. -0 and 0 tie; NaN takes -inf's key, the
// lowest, which an expert that is off has. Keys below kFirst are not chosen.
__device__ __forceinline__ int order_key(float v) {
    const int u = __float_as_int(fmaxf(v + 0.0f, -INFINITY));
    return u ^ ((u >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_value(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }
constexpr int kFirst = static_cast<int>(0x80800000u);      // of the lowest finite value
constexpr int kGone = static_cast<int>(0x80000000u);

template <int G, typename F, typename X>
__device__ __forceinline__ X lanes_reduce(unsigned mask, X v, F f) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v = f(v, __shfl_xor_sync(mask, v, off));
    return v;
}
template <int G>
__device__ __forceinline__ unsigned lanes_or(unsigned mask, unsigned v) {
    if constexpr (G == 32) return __reduce_or_sync(0xffffffffu, v);
    return lanes_reduce<G>(mask, v, [](unsigned a, unsigned b) { return a | b; });
}
template <int G>
__device__ __forceinline__ float lanes_sum(unsigned mask, float v) {
    return lanes_reduce<G>(mask, v, [](float a, float b) { return a + b; });
}
template <int G>
__device__ __forceinline__ float lanes_max(unsigned mask, float v) {
    return lanes_reduce<G>(mask, v, [](float a, float b) { return fmaxf(a, b); });
}
template <int G>
__device__ __forceinline__ int lanes_max_key(unsigned mask, int v) {
    if constexpr (G == 32) return __reduce_max_sync(0xffffffffu, v);
    return lanes_reduce<G>(mask, v, [](int a, int b) { return max(a, b); });
}
template <int G>
__device__ __forceinline__ uint32_t lanes_max_u32(unsigned mask, uint32_t v) {
    if constexpr (G == 32) return __reduce_max_sync(0xffffffffu, v);
    return lanes_reduce<G>(mask, v, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// Eight keys in descending order: a bitonic sequence's last half, and a whole network.
__device__ __forceinline__ void order_pair(int (&k)[8], int a, int b) {
    const int hi = max(k[a], k[b]), lo = min(k[a], k[b]);
    k[a] = hi;
    k[b] = lo;
}
__device__ __forceinline__ void bitonic_merge8(int (&k)[8]) {
#pragma unroll
    for (int d = 4; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((i & d) == 0) order_pair(k, i, i + d);
}
__device__ __forceinline__ void sort8(int (&k)[8]) {
    // Batcher's odd-even merge sort, 19 comparisons
    constexpr int kPairs[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                                   {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
    for (int i = 0; i < 19; ++i) order_pair(k, kPairs[i][0], kPairs[i][1]);
}

constexpr uint32_t kIndexBits = 0x1fffu;
constexpr int kIndexMax = 1023;

// A sum with the roundings of its additions beside it.
__device__ __forceinline__ void add_exact(float2 &sum, float v) {
    const float s = sum.x + v, b = s - sum.x;
    sum.y += (sum.x - (s - b)) + (v - b);
    sum.x = s;
}
__device__ __forceinline__ float total_of(const float2 &sum) { return isfinite(sum.x) ? sum.x + sum.y : sum.x; }

// The scratch of a block's tokens.
template <int G, int V>
struct Slots {
    static constexpr int kRows = kBlock<V> / G;
    int idx[kRows][kMaxK + 1];
    float s[kRows][kMaxK + 1];
    int key[kRows][kMaxK + 1];
    double group[kRows][kMaxGroups];
};

// A double's bits in an order that unsigned compares keep (64-bit floating-point
// instructions, compares among them, take some 60 cycles a warp here).
__device__ __forceinline__ uint64_t order_key64(double v) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return v != v ? 0u : ((u >> 63) ? ~u : (u | 0x8000000000000000ull));
}

template <int G>
__device__ __forceinline__ uint64_t lanes_max_u64(unsigned mask, uint64_t v) {
    const uint32_t hi = lanes_max_u32<G>(mask, static_cast<uint32_t>(v >> 32));
    const uint32_t lo = lanes_max_u32<G>(mask, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}

// In what follows a lane's experts are unrolled where they are few; the rest is in local memory.

// A token's scores in 64 bits: what softmax needs of the whole row, then one expert's.
struct WideScore {
    double top, inv;                                 // softmax only
    __device__ __forceinline__ double operator()(bool softmax, double l) const {
        return softmax ? exp(l - top) * inv : 1.0 / (1.0 + exp(-l));
    }
};
template <int G, int V>
__device__ __forceinline__ WideScore wide_score(const RouteLaunch &p, int64_t row, int e0, unsigned gmask) {
    WideScore w = {0.0, 1.0};
    if (p.score_fn != MOE_SCORE_SOFTMAX) return w;
    float top = -INFINITY;
#pragma unroll (V <= 8 ? V : 1)
    for (int i = 0; i < V; ++i)
        if (e0 + at<V>(i) < p.E) top = fmaxf(top, load_one(p.logits, p.dtype, row + e0 + at<V>(i)));
    w.top = lanes_max<G>(gmask, top);
    double z = 0.0;
#pragma unroll (V <= 8 ? V : 1)
    for (int i = 0; i < V; ++i)
        if (e0 + at<V>(i) < p.E) z += exp(static_cast<double>(load_one(p.logits, p.dtype, row + e0 + at<V>(i))) - w.top);
    for (int off = G / 2; off > 0; off >>= 1) z += __shfl_xor_sync(gmask, z, off);
    w.inv = 1.0 / z;
    return w;
}

// Selection in 64 bits among the experts marked in `cand` (at most G of the token's, all
// that can be among its k best): one expert a lane, and its rank is the number of better ones.
template <int G, int V>
__device__ __noinline__ void select_near(const RouteLaunch &p, int64_t row, int sub, unsigned gmask, unsigned cand,
                                         int *out_idx, float *out_s) {
    const int e0 = first_expert<V>(sub), lane = threadIdx.x & 31;
    const WideScore score = wide_score<G, V>(p, row, e0, gmask);
    int n = 0;
#pragma unroll (V <= 8 ? V : 1)
    for (int i = 0; i < V; ++i) {
        const unsigned b = __ballot_sync(gmask, (cand >> i) & 1u) & gmask;
        if ((cand >> i) & 1u) out_idx[n + __popc(b & ((1u << lane) - 1u))] = e0 + at<V>(i);
        n += __popc(b);
    }
    __syncwarp(gmask);
    const int e = sub < n ? out_idx[sub] : 0x7fffffff;
    __syncwarp(gmask);
    uint64_t key = 0;
    float s32 = 0.0f;
    if (sub < n) {
        const double s = score(p.score_fn == MOE_SCORE_SOFTMAX, load_one(p.logits, p.dtype, row + e));
        s32 = static_cast<float>(s);
        key = order_key64(s + static_cast<double>(__ldg(p.sel_bias + e)));
    }
    int rank = 0;
    for (int c = 0; c < n; ++c) {
        const uint64_t ok = __shfl_sync(gmask, key, c, G);
        const int oe = __shfl_sync(gmask, e, c, G);
        rank += ok > key || (ok == key && oe < e);
    }
    if (sub < n && rank < p.k) {
        out_idx[rank] = e;
        out_s[rank] = s32;
    }
    __syncwarp(gmask);
}

// The groups that stay of those in `near`, whose sums differ by less than the error of 32-bit
// ones: the experts that can be among a near group's best (no more than the error `err1` below
// its last) are scored in 64 bits, one a lane. sel_row: the token's selection scores, -inf where
// off. Returns the near groups that stay, `room` of them; ~0 where there are more such experts
// than lanes. Without a bias softmax's sums need no normaliser; they are taken about `top`, the
// row's largest logit, as everywhere else: a finite logit may be any distance below another (a
// mask of -1e4), and about any but the largest its exponential leaves fp64.
template <int G, int V>
__device__ __noinline__ unsigned resolve_groups(const RouteLaunch &p, int64_t row, const float *sel_row, int sub,
                                                unsigned gmask, unsigned near, int room, float err1, bool biased, float top,
                                                int *list, double *group) {
    const int lane = threadIdx.x & 31, e0 = first_expert<V>(sub);
    const int gs = p.E / p.n_group;
    const bool softmax = p.score_fn == MOE_SCORE_SOFTMAX;
    int n = 0;
    for (unsigned left = near; left != 0; left &= left - 1u) {
        const int g = __ffs(left) - 1;
        auto inside = [&](int i) {                   // the lane's i-th expert is one of the group's
            const int e = e0 + at<V>(i);
            return e >= g * gs && e < (g + 1) * gs;
        };
        // the group's group_topn-th best, ties counted
        int floor = 0x7fffffff;
        for (int taken = 0; taken < p.group_topn;) {
            int best = kGone;
            for (int i = 0; i < V; ++i) {
                const int k = inside(i) ? order_key(sel_row[e0 + at<V>(i)]) : kGone;
                if (k < floor && k > best) best = k;
            }
            const int m = lanes_max_key<G>(gmask, best);
            if (m < kFirst) break;
            int same = 0;
            for (int i = 0; i < V; ++i) same += inside(i) && order_key(sel_row[e0 + at<V>(i)]) == m;
            taken += lanes_reduce<G>(gmask, same, [](int a, int b) { return a + b; });
            floor = m;
        }
        const float least = key_value(floor) - 2.0f * err1;
        for (int i = 0; i < V; ++i) {
            const int e = e0 + at<V>(i);
            const bool in = inside(i) && sel_row[e] > -INFINITY && sel_row[e] >= least;
            const unsigned who = __ballot_sync(gmask, in) & gmask;
            const int place = n + __popc(who & ((1u << lane) - 1u));
            if (in && place < G) list[place] = e;
            n += __popc(who);
        }
    }
    if (n > G) return ~0u;
    __syncwarp(gmask);
    const int e = sub < n ? list[sub] : -1;
    WideScore score = {0.0, 1.0};
    if (softmax && biased) {
        score = wide_score<G, V>(p, row, e0, gmask);
    } else if (softmax) {
        score.top = top;
    }
    double v = 0.0;
    uint64_t key = 0;
    int own = -1;                                    // group
    if (e >= 0) {
        v = score(softmax, load_one(p.logits, p.dtype, row + e));
        if (biased) v += static_cast<double>(__ldg(p.sel_bias + e));
        key = order_key64(v);
        own = e / gs;
    }
    int rank = 0;
    for (int c = 0; c < n; ++c) {
        const uint64_t ok = __shfl_sync(gmask, key, c, G);
        const int og = __shfl_sync(gmask, own, c, G);
        rank += og == own && (ok > key || (ok == key && c < sub));
    }
    const double part = rank < p.group_topn ? v : 0.0;
    double total = 0.0;
    for (int c = 0; c < n; ++c) {
        const double x = __shfl_sync(gmask, part, c, G);
        if (__shfl_sync(gmask, own, c, G) == own) total += x;
    }
    if (e >= 0) group[own] = total;                  // the same number from each of its lanes
    __syncwarp(gmask);
    unsigned stay = 0;
    for (unsigned left = near; left != 0; left &= left - 1u) {
        const int g = __ffs(left) - 1;
        int before = 0;
        for (unsigned other = near; other != 0; other &= other - 1u) {
            const int o = __ffs(other) - 1;
            before += group[o] > group[g] || (group[o] == group[g] && o < g);
        }
        if (before < room) stay |= 1u << g;
    }
    __syncwarp(gmask);
    return stay;
}

// One token's whole selection in 64 bits: the groups in `sure` stay, of those in `near`
// the best stay as far as topk_group allows, then k rounds.
template <int G, int V>
__device__ __noinline__ void select_wide(const RouteLaunch &p, int64_t row, int sub, unsigned gmask, unsigned sure,
                                         unsigned near, bool by_score, int *out_idx, float *out_s, double *group) {
    const int e0 = first_expert<V>(sub);
    const WideScore score = wide_score<G, V>(p, row, e0, gmask);
    const bool softmax = p.score_fn == MOE_SCORE_SOFTMAX;
    const int gs = p.E / p.n_group, g_first = e0 / gs, bound = (g_first + 1) * gs;
    auto group_of = [&](int e) { return V <= 8 && gs >= V ? g_first + (e >= bound) : e / gs; };
    double sel[V];
    uint64_t key[V];
    unsigned open = 0;                               // experts that may still be chosen
#pragma unroll (V <= 8 ? V : 1)
    for (int i = 0; i < V; ++i) {
        key[i] = 0;
        if (e0 + at<V>(i) >= p.E || !(((sure | near) >> group_of(e0 + at<V>(i))) & 1u)) continue;
        const float l = load_one(p.logits, p.dtype, row + e0 + at<V>(i));
        if (l == -INFINITY) continue;
        sel[i] = score(softmax, l) + (p.sel_bias != nullptr ? static_cast<double>(__ldg(p.sel_bias + e0 + at<V>(i))) : 0.0);
        if (!(sel[i] > -INFINITY)) continue;
        open |= 1u << i;
        key[i] = order_key64(sel[i]);
    }
    if (near != 0) {
        for (unsigned left = near; left != 0; left &= left - 1u) {
            const int g = __ffs(left) - 1;
            unsigned taken = 0;
            double total = -INFINITY;
            for (int n = 0; n < p.group_topn; ++n) {
                uint64_t b = 0;
#pragma unroll (V <= 8 ? V : 1)
                for (int i = 0; i < V; ++i)
                    if (((open & ~taken) >> i) & 1u && group_of(e0 + at<V>(i)) == g && key[i] > b) b = key[i];
                const uint64_t m = lanes_max_u64<G>(gmask, b);
                if (m == 0) break;
                const unsigned who = __ballot_sync(gmask, b == m) & gmask;
                const int from = __ffs(who) - 1;
                double v = 0.0;
                if ((threadIdx.x & 31) == from) {
                    int pick = 0;
#pragma unroll (V <= 8 ? V : 1)
                    for (int i = V - 1; i >= 0; --i)
                        if (((open & ~taken) >> i) & 1u && group_of(e0 + at<V>(i)) == g && key[i] == m) pick = i;
                    taken |= 1u << pick;
                    v = sel[pick];
                }
                v = __shfl_sync(gmask, v, from);
                total = n == 0 ? v : total + v;
            }
            if (sub == 0) group[g] = total;
        }
        __syncwarp(gmask);
        const int room = p.topk_group - __popc(sure);
#pragma unroll (V <= 8 ? V : 1)
        for (int i = 0; i < V; ++i) {
            if (!((open >> i) & 1u)) continue;
            const int g = group_of(e0 + at<V>(i));
            if (!((near >> g) & 1u)) continue;
            int before = 0;
            for (unsigned left = near; left != 0; left &= left - 1u) {
                const int o = __ffs(left) - 1;
                before += group[o] > group[g] || (group[o] == group[g] && o < g);
            }
            if (before >= room) {
                open &= ~(1u << i);
                key[i] = 0;
            }
        }
        __syncwarp(gmask);
    }
    if (!by_score)                                   // the score's order is the logit's
#pragma unroll (V <= 8 ? V : 1)
        for (int i = 0; i < V; ++i)
            if ((open >> i) & 1u) key[i] = order_key64(load_one(p.logits, p.dtype, row + e0 + at<V>(i)));
    for (int j = 0; j < p.k; ++j) {
        uint64_t b = 0;
#pragma unroll (V <= 8 ? V : 1)
        for (int i = 0; i < V; ++i) b = max(b, key[i]);
        const uint64_t m = lanes_max_u64<G>(gmask, b);
        // the lowest index among equal keys
        int mine = -1;
#pragma unroll (V <= 8 ? V : 1)
        for (int i = V - 1; i >= 0; --i)
            if (m != 0 && key[i] == m) mine = i;
        const int e = mine < 0 ? -0x7fffffff : -(e0 + at<V>(mine));
        const int best = lanes_max_key<G>(gmask, e);
        if (mine >= 0 && e == best) {
            key[mine] = 0;
            out_idx[j] = -best;
        } else if (best == -0x7fffffff && sub == 0) {
            out_idx[j] = -1;
        }
    }
    __syncwarp(gmask);
    for (int j = sub; j < p.k; j += G) {
        const int e = out_idx[j];
        out_s[j] = e >= 0 ? static_cast<float>(score(softmax, load_one(p.logits, p.dtype, row + e))) : 0.0f;
    }
    __syncwarp(gmask);
}

// Sums of the groups' group_topn best of sel_row, a power of two of lanes to each group.
template <int G>
__device__ __forceinline__ void search_groups(const RouteLaunch &p, const float *sel_row, float *sums, int sub,
                                              unsigned gmask) {
    const int gs = p.E / p.n_group;
    int per = G;                                     // lanes of a group
    while (per > 1 && per * p.n_group > G) per >>= 1;
    const int part = sub & (per - 1);
    for (int g0 = 0; g0 < p.n_group; g0 += G / per) {
        const int g = g0 + sub / per;
        const float *row = sel_row + g * gs;
        // a lane's experts part, part + per, ... from a start that spreads the banks
        const int n = g < p.n_group && part < gs ? (gs - part + per - 1) / per : 0;
        int i = n > 0 ? g % n : 0;
        float total = -INFINITY;
        if (p.group_topn <= 2) {
            float a = -INFINITY, b = -INFINITY;      // the two best, a >= b
            for (int c = 0; c < n; ++c) {
                const float v = row[part + per * i];
                b = fmaxf(b, min_nan(a, v));       // as in kept_groups
                a = fmaxf(a, v);
                i = i + 1 == n ? 0 : i + 1;
            }
            for (int off = per >> 1; off > 0; off >>= 1) {
                const float oa = __shfl_xor_sync(gmask, a, off), ob = __shfl_xor_sync(gmask, b, off);
                b = fmaxf(fminf(a, oa), fmaxf(b, ob));
                a = fmaxf(a, oa);
            }
            total = p.group_topn == 2 && b > -INFINITY ? a + b : a;
        } else {
            float pv = INFINITY;
            int pi = -1;
            for (int r = 0; r < p.group_topn; ++r) {
                float bv = -INFINITY;
                int bi = 0x7fffffff;
                for (int c = 0; c < n; ++c) {
                    const int e = part + per * c;
                    const float v = row[e];
                    if ((v < pv || (v == pv && e > pi)) && v > bv) {
                        bv = v;
                        bi = e;
                    }
                }
                for (int off = per >> 1; off > 0; off >>= 1) {
                    const float ov = __shfl_xor_sync(gmask, bv, off);
                    const int oi = __shfl_xor_sync(gmask, bi, off);
                    if (ov > bv || (ov == bv && oi < bi)) {
                        bv = ov;
                        bi = oi;
                    }
                }
                if (bi != 0x7fffffff) total = total == -INFINITY ? bv : total + bv;
                pv = bi == 0x7fffffff ? -INFINITY : bv;
                pi = bi;
            }
        }
        if (part == 0 && g < p.n_group) sums[g] = total;
    }
}

// The groups of one token that stay, as bits; v: the lane's selection scores (-inf: off). NaN is as
// good as off: in the second best it goes through a minimum that hands it on, into a maximum that
// does not (a minimum without it would be the best, taken twice).
// Where a group is a power of two of whole lanes (`group_lanes`, from the host) and is known
// by its best one or two, those are found in registers. Else a group is searched in `sel_row`
// by a power of two of lanes, each taking every so many of its experts. `near`: the groups
// that could be on either side, where the last kept and the first dropped sum differ by no
// more than `err`, the error of two sums; 0 where none could.
template <int G, int V>
__device__ __forceinline__ unsigned kept_groups(const RouteLaunch &p, const float (&vals)[V], float *sel_row, float *sums,
                                                int sub, unsigned gmask, float err, unsigned &near) {
    if (p.group_lanes != 0) {
        float a = -INFINITY, b = -INFINITY;          // the two best, a >= b
#pragma unroll
        for (int i = 0; i < V; ++i) {
            b = fmaxf(b, min_nan(a, vals[i]));
            a = fmaxf(a, vals[i]);
        }
        for (int off = 1; off < p.group_lanes; off <<= 1) {
            const float oa = __shfl_xor_sync(gmask, a, off), ob = __shfl_xor_sync(gmask, b, off);
            b = fmaxf(fminf(a, oa), fmaxf(b, ob));
            a = fmaxf(a, oa);
        }
        const int g = sub / p.group_lanes;
        if (g * p.group_lanes == sub && g < p.n_group) sums[g] = p.group_topn == 2 && b > -INFINITY ? a + b : a;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) sel_row[first_expert<V>(sub) + at<V>(i)] = vals[i];
        __syncwarp();
        search_groups<G>(p, sel_row, sums, sub, gmask);
    }
    __syncwarp();
    unsigned kept = 0;
    for (int g = sub; g < p.n_group; g += G) {
        const float mine = sums[g];
        int before = 0;
#pragma unroll 4
        for (int o = 0; o < p.n_group; ++o) before += sums[o] > mine || (sums[o] == mine && o < g);
        if (before < p.topk_group) kept |= 1u << g;
        // the sums at the border
        if (before == p.topk_group - 1) sums[kMaxGroups] = mine;
        if (before == p.topk_group) sums[kMaxGroups + 1] = mine;
    }
    kept = lanes_or<G>(gmask, kept);
    __syncwarp();
    const float in = sums[kMaxGroups], out = sums[kMaxGroups + 1];
    near = 0;
    if (out > -INFINITY && in - out <= err) {
        // a sum above out + err outranks every dropped group, one below in - err no kept one
        for (int g = sub; g < p.n_group; g += G)
            if (sums[g] <= out + err && sums[g] >= in - err) near |= 1u << g;
        near = lanes_or<G>(gmask, near);
        __syncwarp(gmask);
    }
    return kept;
}

// Tokens [per_block b, per_block (b + 1)) in block b, as many at a time as it has rows of lanes.
// kShort: 16-bit logits without a selection bias. An fp32 of such a value has its low 13
// bits clear, which hold the expert's index instead: one 32-bit key tells both, no two are
// equal, and a round is a maximum and a clearing without a branch.
template <int G, int V, bool kStats, bool kShort>
__global__ void __launch_bounds__(kBlock<V>, V <= 8 ? 3 : V == 16 ? 2 : 1)
route_kernel(const RouteLaunch p) {
    constexpr int kThreads = kBlock<V>, kRows = kThreads / G;
    // score sums of a lane's experts: in registers, or where those run out in shared memory
    constexpr bool kShared = V > 16;
    constexpr int kOwn = kMaxK / G;                  // slots of a lane
    __shared__ Slots<G, V> slots;
    __shared__ __align__(16) float buf[kRows * G * V];
    __shared__ __align__(16) float sums_buf[kStats && kShared ? kRows * G * V : 1];
    __shared__ int hist[kStats ? G * V : 1];
    __shared__ float red_z[kRows];
    __shared__ int red_n[kRows];
    griddep_wait();
    const int row = threadIdx.x / G, sub = threadIdx.x % G;
    const int lane = threadIdx.x & 31;
    const unsigned gmask = G == 32 ? 0xffffffffu : ((1u << G) - 1u) << (lane / G * G);
    const int e0 = first_expert<V>(sub);
    const int t_begin = blockIdx.x * p.per_block;
    const int t_end = min(p.T, t_begin + p.per_block);
    const bool grouped = p.n_group > 1 && p.topk_group < p.n_group;
    const bool softmax = p.score_fn == MOE_SCORE_SOFTMAX;
    const bool biased = !kShort && p.sel_bias != nullptr;
    const int gs = p.E / p.n_group;
    constexpr int kRuns = V <= 8 ? 1 : V / 4, kRun = V / kRuns;   // runs of consecutive experts
    int run_group[kRuns];
#pragma unroll
    for (int r = 0; r < kRuns; ++r) run_group[r] = grouped ? (e0 + at<V>(r * kRun)) / gs : 0;
    float *own_row = buf + row * G * V;
    // a lane's biases stay in registers where there are few
    constexpr int kHeld = V <= 8 ? V : 1;
    float held[kHeld], bias_max = 0.0f;              // the largest that is finite
    bool nonzero = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float b = biased && e0 + at<V>(i) < p.E ? __ldg(p.sel_bias + e0 + at<V>(i)) : 0.0f;
        if (V <= 8) held[i % kHeld] = b;
        nonzero |= !(b == 0.0f);
        if (fabsf(b) < INFINITY) bias_max = fmaxf(bias_max, fabsf(b));
    }
    auto bias = [&](int i) {
        if (V <= 8) return held[i % kHeld];
        return biased && e0 + at<V>(i) < p.E ? __ldg(p.sel_bias + e0 + at<V>(i)) : 0.0f;
    };
    if (biased) {
        bias_max = lanes_max<G>(gmask, bias_max);
        nonzero = (__ballot_sync(0xffffffffu, nonzero) & gmask) != 0;
    }
    // with no bias, or none but zeros, the order is the logits' own, without a rounding; so is
    // that of groups known by their best expert
    const bool by_score = biased && nonzero;
    const bool best_only = !by_score && p.group_topn == 1;
    int seq = 0;
    float acc[kShared ? 1 : V];
    float *own_sums = sums_buf + (kStats && kShared ? row * G * V + e0 : 0);      // at<V>(i)
    auto add = [&](int i, float v) {
        if (kShared) own_sums[at<V>(i)] += v;
        else acc[kShared ? 0 : i] += v;
    };
    float z_acc = 0.0f;
    int n_acc = 0;
    if constexpr (kStats) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (kShared) own_sums[at<V>(i)] = 0.0f;
            else acc[kShared ? 0 : i] = 0.0f;
        }
        for (int e = threadIdx.x; e < G * V; e += kThreads) hist[e] = 0;
        for (int b = 1; b < p.S; b += kThreads) {
            const int i = b + static_cast<int>(threadIdx.x);
            seq += __syncthreads_count(i < p.S && __ldg(p.seq_offsets + i) <= t_begin);
        }
        __syncthreads();
    }
    int t = t_begin;
    while (t < t_end) {
        int seg_end = t_end;
        if constexpr (kStats) {
            while (seq < p.S - 1 && __ldg(p.seq_offsets + seq + 1) <= t) ++seq;
            if (seq < p.S - 1) seg_end = min(t_end, __ldg(p.seq_offsets + seq + 1));
        }
        for (int base = t; base < seg_end; base += kRows) {
            const int tok = base + row;
            const bool inside = tok < seg_end;
            const bool given = inside && (p.mask == nullptr || __ldg(p.mask + tok) != 0);
            const int64_t lrow = static_cast<int64_t>(tok) * p.ld;
            float l[V], s[V];
            if (given) {
                load_experts<V>(p.logits, p.dtype, p.vec, lrow, e0, p.E, l);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) l[i] = -INFINITY;
            }
            // the row's largest logit, NaN where one is; -inf: the token is not live
            float top = l[0];
#pragma unroll
            for (int i = 1; i < V; ++i) top = max_nan(top, l[i]);
            if (softmax || kStats)
                top = lanes_reduce<G>(gmask, top, [](float a, float b) { return max_nan(a, b); });
            const bool live = !(top == -INFINITY);
            // scores (exp(-inf) = 0 puts out the experts that are off)
            float s_max = 1.0f;                      // no score is above it
            if (softmax) {
                float ssum = 0.0f;
                const float shift = live ? top : 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s[i] = exp2_fast((l[i] - shift) * kLog2e);
                    ssum += s[i];
                }
                ssum = lanes_sum<G>(gmask, ssum);
                s_max = 1.0f / (live ? ssum : 1.0f);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s[i] *= s_max;
                    if constexpr (kStats) add(i, s[i]);
                }
                if (kStats && live && sub == 0) {
                    const float lse = top + __logf(ssum);
                    z_acc += lse * lse;
                }
            } else {
                float ex = 0.0f, ssum = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float e = expf(-l[i]);
                    s[i] = rcp_fast(1.0f + e);
                    if constexpr (kStats) {
                        ssum += s[i];
                        ex += rcp_fast(e);           // exp(l)
                    }
                }
                if constexpr (kStats) {
                    float shift = 0.0f;
                    if (!(top < 80.0f && top > -60.0f)) {
                        // exp(l) leaves fp32: about the maximum, as softmax does
                        shift = live ? top : 0.0f;
                        ex = 0.0f;
#pragma unroll
                        for (int i = 0; i < V; ++i) ex += expf(l[i] - shift);
                    }
                    ssum = lanes_sum<G>(gmask, ssum);
                    ex = lanes_sum<G>(gmask, ex);
                    if (live && sub == 0) {
                        const float lse = shift + __logf(ex);
                        z_acc += lse * lse;
                    }
                    const float share = live ? 1.0f / (ssum + kEps) : 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) add(i, s[i] * share);
                }
            }
            if (kStats) n_acc += live && sub == 0;
            // keys
            const float rel = softmax ? softmax_err<V>() : kSigmoidErr;
            int key[V];
            unsigned kept = 0xffffffffu, near_groups = 0;
            bool near = false;                       // nearer than the error of a 32-bit key
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float by = l[i] == -INFINITY ? -INFINITY : s[i] + bias(i);
                key[i] = order_key(by_score ? by : l[i]);
                if (kShort) key[i] = (key[i] & ~static_cast<int>(kIndexBits)) | (kIndexMax - (e0 + at<V>(i)));
            }
            if (grouped) {
                float v[V];
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = best_only || l[i] == -INFINITY ? l[i] : s[i] + bias(i);
                const float n = static_cast<float>(p.group_topn);
                kept = kept_groups<G, V>(p, v, own_row, reinterpret_cast<float *>(slots.group[row]), sub, gmask,
                                         best_only ? -1.0f : 2.0f * n * (rel * s_max + kUlp * (2.0f + n) * (s_max + bias_max)),
                                         near_groups);
                if (near_groups != 0) {
#pragma unroll
                    for (int i = 0; i < V; ++i) own_row[e0 + at<V>(i)] = v[i];
                    __syncwarp(gmask);
                    const unsigned sure = kept & ~near_groups;
                    const unsigned stay = resolve_groups<G, V>(p, lrow, own_row, sub, gmask, near_groups,
                                                               p.topk_group - __popc(sure),
                                                               rel * s_max + 2.0f * kUlp * (s_max + bias_max), by_score, top,
                                                               slots.idx[row], slots.group[row]);
                    if (stay != ~0u) {
                        kept = sure | stay;
                        near_groups = 0;
                    }
                }
#pragma unroll
                for (int r = 0; r < kRuns; ++r) {
                    int g = run_group[r], next = (g + 1) * gs;
#pragma unroll
                    for (int i = r * kRun; i < (r + 1) * kRun; ++i) {
                        if (e0 + at<V>(i) == next) {
                            ++g;
                            next += gs;
                        }
                        if (!((kept >> (g & 31)) & 1u)) key[i] = kGone;
                    }
                }
                __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < V; ++i) own_row[e0 + at<V>(i)] = s[i];
            int best = key[0];
#pragma unroll
            for (int i = 1; i < V; ++i) best = max(best, key[i]);
            float sv[kOwn];
            int ev[kOwn];
            if constexpr (kShort) {
#pragma unroll
                for (int q = 0; q < kOwn; ++q) ev[q] = -1;
                bool done = false;
                if constexpr (V == 8) {
                    if (p.k <= 8) {
                        done = true;
                        // every lane's keys in order, then the eight best of two lanes at a time: 200
                        // instructions for 16 lanes against 310 of eight rounds
                        sort8(key);
#pragma unroll
                        for (int off = 1; off < G; off <<= 1) {
                            int other[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(gmask, key[i], off);
#pragma unroll
                            for (int i = 0; i < 8; ++i) key[i] = max(key[i], other[7 - i]);
                            bitonic_merge8(key);
                        }
                        int m = kGone;
#pragma unroll
                        for (int i = 0; i < 8; ++i) m = sub == i ? key[i] : m;
                        if (sub < p.k && m >= kFirst) ev[0] = kIndexMax - (m & static_cast<int>(kIndexBits));
                    }
                }
                for (int j = 0; j < p.k && !done; ++j) {
                    const int m = lanes_max_key<G>(gmask, best);
#pragma unroll
                    for (int q = 0; q < kOwn; ++q)
                        if (j == sub + q * G && m >= kFirst) ev[q] = kIndexMax - (m & static_cast<int>(kIndexBits));
                    key[0] = key[0] == m ? kGone : key[0];
                    best = key[0];
#pragma unroll
                    for (int i = 1; i < V; ++i) {
                        key[i] = key[i] == m ? kGone : key[i];
                        best = max(best, key[i]);
                    }
                }
                if (grouped) {                       // where the selection in 64 bits starts from
#pragma unroll
                    for (int q = 0; q < kOwn; ++q)
                        if (sub + q * G < p.k) slots.idx[row][sub + q * G] = ev[q];
                }
                __syncwarp();
            } else {
                // one more than k where the last chosen key is compared with the next
                const int rounds = p.k + (by_score ? 1 : 0);
                // No more than the experts at or above the rounds-th largest of the lanes' best can
                // be chosen: some ten for eight of 256. Where there are no more than lanes, each is
                // ranked by a lane of its own against the others, at a third of the rounds' work.
                int n = G + 1;
                if (G >= 16 && rounds <= G) {
                    int lane_best = best, floor = kGone;
                    for (int j = 0; j < rounds; ++j) {
                        floor = lanes_max_key<G>(gmask, lane_best);
                        if (lane_best == floor) lane_best = kGone;
                    }
                    floor = max(floor, kFirst);
                    auto gather = [&] {
                        n = 0;
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const bool in = key[i] >= floor;
                            const unsigned who = __ballot_sync(0xffffffffu, in) & gmask;
                            const int place = n + __popc(who & ((1u << lane) - 1u));
                            if (in && place < G) {
                                slots.idx[row][place] = e0 + at<V>(i);
                                slots.key[row][place] = key[i];
                            }
                            n += __popc(who);
                        }
                    };
                    gather();
                    if (!__all_sync(0xffffffffu, n <= G)) {
                        // too many (more chosen experts than a quarter of the lanes, as a rule): a
                        // floor with no fewer than `rounds` above it and no more than lanes, by halving
                        if (n > G) {
                            int low = floor, high = lanes_max_key<G>(gmask, best);
                            while (static_cast<unsigned>(high) - static_cast<unsigned>(low) > 1u) {
                                const int mid =
                                    low + static_cast<int>((static_cast<unsigned>(high) - static_cast<unsigned>(low)) >> 1);
                                int c = 0;
#pragma unroll
                                for (int i = 0; i < V; ++i) c += key[i] >= mid;
                                c = lanes_reduce<G>(gmask, c, [](int a, int b) { return a + b; });
                                if (c > G) low = mid;
                                else high = mid;
                                if (c >= rounds && c <= G) {
                                    floor = mid;
                                    break;
                                }
                            }
                        }
                        __syncwarp();                // votes order no memory: the first places before the second
                        gather();
                    }
                }
                if (__all_sync(0xffffffffu, n <= G)) {
                    __syncwarp();
                    int e = -1, k = kGone, rank = sub;
                    if (sub < n) {
                        e = slots.idx[row][sub];
                        k = slots.key[row][sub];
                        rank = 0;
                        for (int o = 0; o < n; ++o) {
                            const int ok = slots.key[row][o];
                            rank += ok > k || (ok == k && slots.idx[row][o] < e);
                        }
                    }
                    __syncwarp();
                    if (rank < rounds) {             // lanes past the candidates: slots left over
                        slots.idx[row][rank] = e;
                        slots.key[row][rank] = k;
                    }
                } else {
                    for (int j = 0; j < rounds; ++j) {
                        const int m = lanes_max_key<G>(gmask, best);
                        int mine = -1;               // the lane's first with that key
#pragma unroll
                        for (int i = V - 1; i >= 0; --i)
                            if (key[i] == m) mine = i;
                        bool wins;
                        if constexpr (V <= 8) {
                            const unsigned who = __ballot_sync(0xffffffffu, best == m) & gmask;
                            wins = lane == __ffs(who) - 1;
                        } else {
                            const int e = mine < 0 ? -0x7fffffff : -(e0 + at<V>(mine));
                            wins = lanes_max_key<G>(gmask, e) == e && mine >= 0;
                        }
                        if (wins) {
                            if (m >= kFirst) {
                                best = kGone;
#pragma unroll
                                for (int i = 0; i < V; ++i) {
                                    if (i == mine) key[i] = kGone;
                                    best = max(best, key[i]);
                                }
                            }
                            slots.idx[row][j] = m >= kFirst ? e0 + at<V>(mine) : -1;
                            slots.key[row][j] = m;
                        }
                    }
                }
                __syncwarp();
#pragma unroll
                for (int q = 0; q < kOwn; ++q) ev[q] = sub + q * G < p.k ? slots.idx[row][sub + q * G] : -1;
            }
#pragma unroll
            for (int q = 0; q < kOwn; ++q) sv[q] = ev[q] >= 0 ? own_row[ev[q]] : 0.0f;
            bool tied = false;                       // the last chosen and the first not chosen are a tie
            if (by_score) {
#pragma unroll
                for (int q = 0; q < kOwn; ++q) {
                    // this slot's key against the next one's (the last one's: the first not chosen)
                    const int b = ev[q] >= 0 ? slots.idx[row][sub + q * G + 1] : -1;
                    if (b < 0) continue;
                    const float x = key_value(slots.key[row][sub + q * G]), y = key_value(slots.key[row][sub + q * G + 1]);
                    // beyond the last there may be others whose score, and so its error, is larger
                    const bool border = sub + q * G == p.k - 1;
                    const float both = border ? 2.0f * s_max : sv[q] + own_row[b];
                    if (x - y <= rel * both + kUlp * (2.0f * (fabsf(x) + fabsf(y)) + s_max)) {
                        // not near: a tie of the same logit and bias
                        const bool same = load_one(p.logits, p.dtype, lrow + ev[q]) == load_one(p.logits, p.dtype, lrow + b) &&
                                          __ldg(p.sel_bias + ev[q]) == __ldg(p.sel_bias + b);
                        near |= !same;
                        tied |= same && border;
                    }
                }
            }
            // the vote is the whole warp's: it stands before any branch that a token takes alone
            bool any_near = (__ballot_sync(0xffffffffu, near || tied || near_groups != 0) & gmask) != 0;
            if (any_near && by_score && near_groups == 0) {
                // behind a tie at the border stand experts that were compared with none: any of another
                // logit or bias within the error of the tie's key
                if ((__ballot_sync(gmask, tied) & gmask) != 0) {
                    const int b = slots.idx[row][p.k];
                    const float x = key_value(slots.key[row][p.k]), bl = load_one(p.logits, p.dtype, lrow + b);
                    const float bb = __ldg(p.sel_bias + b), err = 2.0f * rel * s_max + kUlp * (4.0f * fabsf(x) + s_max);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float v = own_row[e0 + at<V>(i)] + bias(i);
                        near |= l[i] != -INFINITY && fabsf(v - x) <= err && !(l[i] == bl && bias(i) == bb) &&
                                (!grouped || (kept >> ((e0 + at<V>(i)) / gs)) & 1u);
                    }
                }
                any_near = (__ballot_sync(gmask, near) & gmask) != 0;
            }
            if (any_near) {
                // candidates: no more than the error below the first key that was not chosen
                unsigned cand = 0;
                int n = G + 1;
                if (near_groups == 0) {
                    const int b = slots.idx[row][p.k];
                    const float last = b >= 0 ? key_value(slots.key[row][p.k]) : -INFINITY;
                    const float floor = last - 2.0f * (rel * s_max + 2.0f * kUlp * (s_max + bias_max));
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float v = own_row[e0 + at<V>(i)] + bias(i);
                        if (l[i] != -INFINITY && v > -INFINITY && v >= floor && (!grouped || (kept >> ((e0 + at<V>(i)) / gs)) & 1u)) cand |= 1u << i;
                    }
                    n = lanes_reduce<G>(gmask, __popc(cand), [](int a, int b) { return a + b; });
                }
                __syncwarp(gmask);                   // the slots are read before others are written there
                if (n <= G)
                    select_near<G, V>(p, lrow, sub, gmask, cand, slots.idx[row], slots.s[row]);
                else
                    select_wide<G, V>(p, lrow, sub, gmask, kept & ~near_groups, near_groups, by_score, slots.idx[row], slots.s[row],
                                      slots.group[row]);
#pragma unroll
                for (int q = 0; q < kOwn; ++q) {
                    const int j = sub + q * G;
                    ev[q] = j < p.k ? slots.idx[row][j] : -1;
                    sv[q] = ev[q] >= 0 ? slots.s[row][j] : 0.0f;
                }
            }
            // weights
            float chosen = 1.0f;
            if (p.normalize) {
                chosen = 0.0f;
#pragma unroll
                for (int q = 0; q < kOwn; ++q) chosen += sv[q];
                chosen = lanes_sum<G>(gmask, chosen) + kEps;
            }
            if (inside) {
#pragma unroll
                for (int q = 0; q < kOwn; ++q) {
                    const int j = sub + q * G;
                    if (j >= p.k) break;
                    p.topk_idx[static_cast<int64_t>(tok) * p.k + j] = ev[q];
                    p.topk_w[static_cast<int64_t>(tok) * p.k + j] = sv[q] / chosen * p.scale;
                    if (kStats && ev[q] >= 0) atomicAdd(&hist[ev[q]], 1);
                }
            }
            __syncwarp();
        }
        if constexpr (kStats) {
            // this block's sums of the sequence, rows in order
            __syncthreads();
#pragma unroll
            for (int i = 0; i < V; ++i) {
                own_row[e0 + at<V>(i)] = kShared ? own_sums[at<V>(i)] : acc[kShared ? 0 : i];
                if (kShared) own_sums[at<V>(i)] = 0.0f;
                else acc[kShared ? 0 : i] = 0.0f;
            }
            if (sub == 0) {
                red_z[row] = z_acc;
                red_n[row] = n_acc;
            }
            z_acc = 0.0f;
            n_acc = 0;
            __syncthreads();
            const int64_t slot = static_cast<int64_t>(blockIdx.x) + seq;
            const int ld = route_stride(p.E);        // no more than G V; past E the sums are 0
            for (int e = threadIdx.x; e < ld; e += kThreads) {
                float v = 0.0f;
#pragma unroll
                for (int r = 0; r < kRows; ++r) v += buf[r * G * V + e];
                p.part_score[slot * ld + e] = v;
                p.part_count[slot * ld + e] = hist[e];
                hist[e] = 0;
            }
            if (threadIdx.x == 0) {
                float zz = 0.0f;
                int n = 0;
                for (int r = 0; r < kRows; ++r) {
                    zz += red_z[r];
                    n += red_n[r];
                }
                p.part_z[slot] = zz;
                p.part_n[slot] = n;
            }
            __syncthreads();
        }
        t = seg_end;
    }
}

// Counts, live tokens and the two terms from the slots. Block (32-expert chunk,
// sequences blockIdx.y, + gridDim.y, ...): 64 rows of 8 threads, four experts a thread, walk
// the sequence's slots, eight loads of each array in flight; the last block to finish adds
// the sequences' terms in order.
constexpr int kReduceThreads = 512, kReduceWarps = kReduceThreads / 32;

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
__device__ __forceinline__ int warp_total(int v) { return __reduce_add_sync(0xffffffffu, v); }

__global__ void __launch_bounds__(kReduceThreads)
route_reduce_kernel(const RouteLaunch p) {
    griddep_wait();
    __shared__ __align__(16) float sh_s[kReduceWarps][32];
    __shared__ __align__(16) int sh_c[kReduceWarps][32];
    __shared__ float sh_z[kReduceWarps];
    __shared__ int sh_n[kReduceWarps], sh_used[kReduceWarps];
    __shared__ int last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = threadIdx.x >> 3;                // 0 .. 63
    const int e4 = blockIdx.x * 32 + (threadIdx.x & 7) * 4;
    constexpr int kRows = kReduceThreads / 8, kBatch = 8;
    const int ld = route_stride(p.E);
    for (int q = blockIdx.y; q < p.S; q += gridDim.y) {
        const int a = q > 0 ? max(0, min(p.T, __ldg(p.seq_offsets + q))) : 0;
        const int z = q < p.S - 1 ? max(0, min(p.T, __ldg(p.seq_offsets + q + 1))) : p.T;
        const int b0 = a / p.per_block, b1 = z > a ? (z - 1) / p.per_block : b0 - 1;
        float2 s4[4], z2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) s4[i] = z2;
        int4 c = make_int4(0, 0, 0, 0);
        int n = 0;
        for (int b = b0 + threadIdx.x; b <= b1; b += kReduceThreads) {
            n += __ldcg(p.part_n + b + q);
            add_exact(z2, __ldcg(p.part_z + b + q));
        }
        if (e4 < ld) {
            for (int b = b0 + row; b <= b1; b += kRows * kBatch) {
                float4 sv[kBatch];
                int4 cv[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    sv[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    cv[j] = make_int4(0, 0, 0, 0);
                    if (b + j * kRows <= b1) {
                        const int64_t at = (static_cast<int64_t>(b) + j * kRows + q) * ld + e4;
                        sv[j] = __ldcg(reinterpret_cast<const float4 *>(p.part_score + at));
                        cv[j] = __ldcg(reinterpret_cast<const int4 *>(p.part_count + at));
                    }
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    add_exact(s4[0], sv[j].x);
                    add_exact(s4[1], sv[j].y);
                    add_exact(s4[2], sv[j].z);
                    add_exact(s4[3], sv[j].w);
                    c.x += cv[j].x;
                    c.y += cv[j].y;
                    c.z += cv[j].z;
                    c.w += cv[j].w;
                }
            }
        }
        float4 s = make_float4(total_of(s4[0]), total_of(s4[1]), total_of(s4[2]), total_of(s4[3]));
        float zs = total_of(z2);
        // the warp's four rows, then the warps in order
#pragma unroll
        for (int off = 8; off <= 16; off <<= 1) {
            s.x += __shfl_xor_sync(0xffffffffu, s.x, off);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, off);
            s.z += __shfl_xor_sync(0xffffffffu, s.z, off);
            s.w += __shfl_xor_sync(0xffffffffu, s.w, off);
            c.x += __shfl_xor_sync(0xffffffffu, c.x, off);
            c.y += __shfl_xor_sync(0xffffffffu, c.y, off);
            c.z += __shfl_xor_sync(0xffffffffu, c.z, off);
            c.w += __shfl_xor_sync(0xffffffffu, c.w, off);
        }
        n = warp_total(n);
        zs = warp_total(zs);
        __syncthreads();                             // the last sequence's values are used
        if (lane < 8) {
            *reinterpret_cast<float4 *>(&sh_s[warp][lane * 4]) = s;
            *reinterpret_cast<int4 *>(&sh_c[warp][lane * 4]) = c;
        }
        if (lane == 0) {
            sh_z[warp] = zs;
            sh_n[warp] = n;
        }
        __syncthreads();
        if (warp == 0) {
            const int e = blockIdx.x * 32 + lane;
            float sum = 0.0f;
            int count = 0;
            zs = 0.0f;
            n = 0;
#pragma unroll
            for (int r = 0; r < kReduceWarps; ++r) {
                sum += sh_s[r][lane];
                count += sh_c[r][lane];
                zs += sh_z[r];
                n += sh_n[r];
            }
            if (e < p.E) p.counts[static_cast<int64_t>(q) * p.E + e] = count;
            else sum = 0.0f;
            const float nf = static_cast<float>(max(n, 1));
            const float term = warp_total((sum / nf) * (static_cast<float>(count) / (nf * static_cast<float>(p.k))));
            if (lane == 0) {
                p.part_balance[static_cast<int64_t>(q) * gridDim.x + blockIdx.x] = term;
                if (blockIdx.x == 0) {
                    p.seq_tokens[q] = n;
                    p.seq_z[q] = zs;
                }
            }
        }
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
        last = atomicAdd(p.ticket, 1) == static_cast<int>(gridDim.x * gridDim.y) - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    float2 bal2 = make_float2(0.0f, 0.0f), zs2 = bal2;
    int n = 0, used = 0;
    const int64_t terms = static_cast<int64_t>(p.S) * gridDim.x;
    for (int64_t i = threadIdx.x; i < terms; i += kReduceThreads) add_exact(bal2, __ldcg(p.part_balance + i));
    for (int q = threadIdx.x; q < p.S; q += kReduceThreads) {
        const int m = __ldcg(p.seq_tokens + q);
        n += m;
        used += m > 0;
        add_exact(zs2, __ldcg(p.seq_z + q));
    }
    float bal = warp_total(total_of(bal2)), zs = warp_total(total_of(zs2));
    n = warp_total(n);
    used = warp_total(used);
    if (lane == 0) {
        sh_s[warp][0] = bal;
        sh_z[warp] = zs;
        sh_n[warp] = n;
        sh_used[warp] = used;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        bal = 0.0f;
        zs = 0.0f;
        n = 0;
        used = 0;
        for (int r = 0; r < kReduceWarps; ++r) {
            bal += sh_s[r][0];
            zs += sh_z[r];
            n += sh_n[r];
            used += sh_used[r];
        }
        p.seq_tokens[p.S] = n;
        p.seq_tokens[p.S + 1] = used;
        p.losses[0] = static_cast<float>(p.E) * bal / static_cast<float>(max(used, 1));
        p.losses[1] = zs / static_cast<float>(max(n, 1));
    }
}

// Gradient of the logits. With gw the weights' gradient at the chosen scores (taken
// through their normalisation), a_e = dbalance E c_be / (S' k n_b^2) that of the
// shares and Z = sum s + 1e-20:
//   softmax: dl = s (g - sum s g),  g = gw (chosen) + a
//   sigmoid: dl = s (1 - s) (gw (chosen) + (a - sum s a / Z) / Z)
// and dl += dz 2/N lse softmax(l). One pass: a token's logits are read, its scores
// recomputed, its gradient written.
template <int G, int V>
__global__ void __launch_bounds__(kBlock<V>, V <= 8 ? 4 : V == 16 ? 2 : 1)
route_backward_kernel(const RouteBackwardLaunch p) {
    constexpr int kThreads = kBlock<V>, kRows = kThreads / G;
    constexpr int kOwn = kMaxK / G;                  // slots of a lane
    __shared__ __align__(16) float s_buf[kRows * G * V], g_buf[kRows * G * V];
    // a's row of the sequence: in registers where a lane has few experts
    constexpr bool kShared = V > 8;
    __shared__ float a_buf[kShared ? G * V : 1];
    griddep_wait();
    const int row = threadIdx.x / G, sub = threadIdx.x % G;
    const int lane = threadIdx.x & 31;
    const unsigned gmask = G == 32 ? 0xffffffffu : ((1u << G) - 1u) << (lane / G * G);
    const int e0 = first_expert<V>(sub);
    const int t_begin = blockIdx.x * p.per_block;
    const int t_end = min(p.T, t_begin + p.per_block);
    const bool terms = p.dlosses != nullptr;
    const bool softmax = p.score_fn == MOE_SCORE_SOFTMAX;
    float dbal = 0.0f, dz = 0.0f;
    int seq = 0;
    if (terms) {
        dbal = __ldg(p.dlosses);
        dz = 2.0f * __ldg(p.dlosses + 1) / static_cast<float>(max(1, __ldg(p.seq_tokens + p.S)));
        for (int b = 1; b < p.S; b += kThreads) {
            const int i = b + static_cast<int>(threadIdx.x);
            seq += __syncthreads_count(i < p.S && __ldg(p.seq_offsets + i) <= t_begin);
        }
    }
    float *s_row = s_buf + row * G * V, *g_row = g_buf + row * G * V;
    auto fours = [&](float *of, int i) { return reinterpret_cast<float4 *>(of + e0 + at<V>(4 * i)); };
#pragma unroll
    for (int i = 0; i < V / 4; ++i) *fours(g_row, i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    int t = t_begin;
    while (t < t_end) {
        int seg_end = t_end;
        float f = 0.0f;
        float held[kShared ? 1 : V];
        auto a = [&](int i) { return kShared ? a_buf[e0 + at<V>(i)] : held[kShared ? 0 : i]; };
        if (terms) {
            while (seq < p.S - 1 && __ldg(p.seq_offsets + seq + 1) <= t) ++seq;
            if (seq < p.S - 1) seg_end = min(t_end, __ldg(p.seq_offsets + seq + 1));
            const float n = static_cast<float>(max(1, __ldg(p.seq_tokens + seq)));
            const float used = static_cast<float>(max(1, __ldg(p.seq_tokens + p.S + 1)));
            f = dbal / used * (static_cast<float>(p.E) / n) / (n * static_cast<float>(p.k));
        }
        auto of = [&](int e) {
            return terms && e < p.E ? f * static_cast<float>(__ldg(p.counts + static_cast<int64_t>(seq) * p.E + e)) : 0.0f;
        };
        if constexpr (kShared) {
            __syncthreads();                         // the last sequence's are used
            for (int e = threadIdx.x; e < G * V; e += kThreads) a_buf[e] = of(e);
            __syncthreads();
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) held[i] = of(e0 + at<V>(i));
        }
        for (int base = t; base < seg_end; base += kRows) {
            const int tok = base + row;
            const bool inside = tok < seg_end;
            const bool given = inside && (p.mask == nullptr || __ldg(p.mask + tok) != 0);
            float l[V], s[V];
            int ce[kOwn];                            // lane j has slots j, j + G, ...
            float cw[kOwn];
#pragma unroll
            for (int q = 0; q < kOwn; ++q) {
                ce[q] = -1;
                cw[q] = 0.0f;
                if (q * G >= p.k) continue;
                const int j = sub + q * G;
                if (given && j < p.k) {
                    const int64_t at = static_cast<int64_t>(tok) * p.k + j;
                    ce[q] = __ldg(p.topk_idx + at);
                    cw[q] = __ldg(p.dtopk_w + at);
                }
            }
            if (given) {
                load_experts<V>(p.logits, p.dtype, p.vec, static_cast<int64_t>(tok) * p.ld, e0, p.E, l);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) l[i] = -INFINITY;
            }
            unsigned off = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) off |= l[i] == -INFINITY ? 1u << i : 0u;
            float zc = 0.0f, Z = 0.0f;               // z's coefficient at s; sigmoid: the sum of scores
            float z[V];                              // sigmoid: the z term
            if (softmax || dz != 0.0f) {
                float top = l[0];
#pragma unroll
                for (int i = 1; i < V; ++i) top = max_nan(top, l[i]);
                top = lanes_reduce<G>(gmask, top, [](float a, float b) { return max_nan(a, b); });
                const bool live = !(top == -INFINITY);
                const float shift = live ? top : 0.0f;
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s[i] = exp2_fast((l[i] - shift) * kLog2e);
                    sum += s[i];
                }
                sum = lanes_sum<G>(gmask, sum);
                const float inv = live ? __fdividef(1.0f, sum) : 0.0f;
                zc = live ? dz * (top + __logf(sum)) : 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] *= inv;
            }
            float sum = 0.0f;                        // sum s a; softmax: sum s g
            if (softmax) {
#pragma unroll
                for (int i = 0; i < V / 4; ++i) *fours(s_row, i) = make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
            } else {
                // the scores go to s_row; s[] keeps their derivative s (1 - s). 1 - s is exp(-l) s: subtracted, it
                // would keep s's last digit only (6 % off at l = 16, nothing from 17 on). Where exp(-l) is infinite
                // and s 0, that product is NaN, of which the minimum makes 1.
#pragma unroll
                for (int i = 0; i < V / 4; ++i) {
                    float four[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int c = 4 * i + j;
                        z[c] = dz != 0.0f ? zc * s[c] : 0.0f;
                        const float e = expf(-l[c]);
                        four[j] = rcp_fast(1.0f + e);
                        Z += four[j];
                        if (terms) sum += four[j] * a(c);
                        s[c] = four[j] * fminf(e * four[j], 1.0f);
                    }
                    *fours(s_row, i) = make_float4(four[0], four[1], four[2], four[3]);
                }
            }
            __syncwarp();
            // the weights' gradient, taken to the chosen scores
            float cs[kOwn], chosen = 0.0f, dot = 0.0f, to_score = p.scale;
#pragma unroll
            for (int q = 0; q < kOwn; ++q) {
                cs[q] = 0.0f;
                if (q * G >= p.k) continue;
                if (ce[q] >= p.E) ce[q] = -1;
                if (ce[q] >= 0) cs[q] = s_row[ce[q]];
                else cw[q] = 0.0f;                   // the weight of a slot left over is a constant: whatever its gradient
                chosen += cs[q];
            }
            float rest = 0.0f;                       // sum s g over the chosen: the denominator's 1e-20 has that part
            if (p.normalize) {
                chosen = lanes_sum<G>(gmask, chosen);
                const float inv = 1.0f / (chosen + kEps);
#pragma unroll
                for (int q = 0; q < kOwn; ++q) dot += cs[q] * inv * cw[q];
                dot = lanes_sum<G>(gmask, dot);
                const float eps_share = chosen + kEps != chosen ? kEps * inv : 0.0f;
                if (eps_share != 0.0f) rest = p.scale * dot * eps_share;
                // one weight alone is the constant scale but for that part
                to_score = p.scale * inv * (p.k > 1 ? 1.0f : eps_share);
                if (p.k == 1) dot = 0.0f;
            }
#pragma unroll
            for (int q = 0; q < kOwn; ++q)
                if (q * G < p.k && ce[q] >= 0) g_row[ce[q]] = to_score * (cw[q] - dot);
            __syncwarp();
            float g[V];
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const float4 x = *fours(g_row, i);
                g[4 * i] = x.x;
                g[4 * i + 1] = x.y;
                g[4 * i + 2] = x.z;
                g[4 * i + 3] = x.w;
                *fours(g_row, i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            // through the score function
            if (softmax) {
                // with normalised weights the chosen scores' part of sum s g is `rest`
                if (terms || !p.normalize) {
#pragma unroll
                    for (int i = 0; i < V; ++i) sum += s[i] * (p.normalize ? a(i) : g[i] + a(i));
                    sum = lanes_sum<G>(gmask, sum);
                }
                sum += rest;
                const float minus = zc - sum;
#pragma unroll
                for (int i = 0; i < V; ++i) g[i] = s[i] * (g[i] + (a(i) + minus));
            } else {
                float invZ = 0.0f;
                if (terms) {
                    sum = lanes_sum<G>(gmask, sum);
                    Z = lanes_sum<G>(gmask, Z);
                    invZ = 1.0f / (Z + kEps);        // a token that is not live has s = 0 and a finite factor
                    sum *= invZ;
                }
#pragma unroll
                for (int i = 0; i < V; ++i) g[i] = s[i] * (g[i] + (a(i) - sum) * invZ) + z[i];
            }
            // an expert that is off has s = 0, but NaN beside a NaN
#pragma unroll
            for (int i = 0; i < V; ++i) g[i] = (off >> i) & 1u ? 0.0f : g[i];
            if (inside) {
                const int64_t out = static_cast<int64_t>(tok) * p.E + e0;
                if (p.dtype == MOE_DTYPE_F32) {
                    float *q = static_cast<float *>(p.dlogits) + out;
#pragma unroll
                    for (int i = 0; i < V; i += 4) {
                        if (p.vec_out && e0 + at<V>(i) + 4 <= p.E) {
                            *reinterpret_cast<float4 *>(q + at<V>(i)) = make_float4(g[i], g[i + 1], g[i + 2], g[i + 3]);
                        } else {
#pragma unroll
                            for (int j = i; j < i + 4; ++j)
                                if (e0 + at<V>(j) < p.E) q[at<V>(j)] = g[j];
                        }
                    }
                } else {
                    uint32_t pk[V / 2];
                    if (p.dtype == MOE_DTYPE_BF16) {
#pragma unroll
                        for (int i = 0; i < V / 2; ++i) pk[i] = pack_bf16x2(g[2 * i], g[2 * i + 1]);
                    } else {
#pragma unroll
                        for (int i = 0; i < V / 2; ++i) {
                            const __half2 h = __floats2half2_rn(g[2 * i], g[2 * i + 1]);
                            pk[i] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                    }
                    unsigned short *q = static_cast<unsigned short *>(p.dlogits) + out;
                    if (V == 8 && p.vec_out && e0 + V <= p.E) {
                        *reinterpret_cast<uint4 *>(q) = make_uint4(pk[0], pk[1], pk[2 % (V / 2)], pk[3 % (V / 2)]);
                    } else {
#pragma unroll
                        for (int i = 0; i < V; i += 4) {
                            if (p.vec_out && e0 + at<V>(i) + 4 <= p.E) {
                                *reinterpret_cast<uint2 *>(q + at<V>(i)) = make_uint2(pk[i / 2], pk[i / 2 + 1]);
                            } else {
#pragma unroll
                                for (int j = i; j < i + 4; ++j)
                                    if (e0 + at<V>(j) < p.E)
                                        q[at<V>(j)] = static_cast<unsigned short>(pk[j / 2] >> (16 * (j & 1)));
                            }
                        }
                    }
                }
            }
        }
        t = seg_end;
    }
}

// Selection bias, a cluster of four blocks to a layer: b_e += rate sign(sum_e' c_e' - E c_e),
// the counts added over the sequences as integers. Block r of the cluster has a quarter of the
// experts; a thread adds W experts' counts (four, where rows are whole 16-byte vectors) over
// its rows, eight loads in flight. Only the blocks' totals are exchanged, through their shared
// memory. One block for a layer is bound by its SM's reads (7.2 us for 58 layers of 128
// sequences and 256 experts).
constexpr int kBiasThreads = 256, kBiasBlocks = 4;

template <int W>
__global__ void __launch_bounds__(kBiasThreads)
bias_update_kernel(float *__restrict__ bias, const int32_t *__restrict__ counts, int S, int E, int quarter, float rate) {
    griddep_wait();
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ long long part[W][kBiasThreads];
    __shared__ long long warp_part[kBiasThreads / 32];
    __shared__ long long block_total;
    const int layer = blockIdx.x / kBiasBlocks;
    const int e_first = static_cast<int>(cluster.block_rank()) * quarter;
    const int mine = max(0, min(quarter, E - e_first));      // experts of this block
    const int width = quarter / W;                           // threads of a row
    const int rows = min(min(kBiasThreads / width, 32), S);
    const int r = threadIdx.x / width, c = threadIdx.x - r * width;
    const int32_t *from = counts + static_cast<int64_t>(layer) * S * E + e_first + c * W;
    long long n[W];
#pragma unroll
    for (int w = 0; w < W; ++w) n[w] = 0;
    if (r < rows && c * W < mine) {
        constexpr int kBatch = 8;
        for (int q = r; q < S; q += rows * kBatch) {
            int v[kBatch][W];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const bool in = q + j * rows < S;
                const int32_t *at = from + static_cast<int64_t>(in ? q + j * rows : q) * E;
                if constexpr (W == 4) {
                    const int4 x = in ? __ldg(reinterpret_cast<const int4 *>(at)) : make_int4(0, 0, 0, 0);
                    v[j][0] = x.x;
                    v[j][1] = x.y;
                    v[j][2] = x.z;
                    v[j][3] = x.w;
                } else {
                    v[j][0] = in ? __ldg(at) : 0;
                }
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
#pragma unroll
                for (int w = 0; w < W; ++w) n[w] += v[j][w];
        }
    }
    long long all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        part[w][threadIdx.x] = n[w];
        all += n[w];
    }
    for (int off = 16; off > 0; off >>= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
    if ((threadIdx.x & 31) == 0) warp_part[threadIdx.x >> 5] = all;
    __syncthreads();
    if (threadIdx.x == 0) {
        long long t = 0;
#pragma unroll
        for (int i = 0; i < kBiasThreads / 32; ++i) t += warp_part[i];
        block_total = t;
    }
    cluster.sync();
    long long total = 0;
#pragma unroll
    for (int i = 0; i < kBiasBlocks; ++i) total += *cluster.map_shared_rank(&block_total, i);
    if (threadIdx.x < mine) {
        long long own = 0;
        for (int i = 0; i < rows; ++i) own += part[threadIdx.x % W][i * width + threadIdx.x / W];
        const long long d = total - static_cast<long long>(E) * own;
        float *b = bias + static_cast<int64_t>(layer) * E + e_first + threadIdx.x;
        *b += d > 0 ? rate : d < 0 ? -rate : 0.0f;
    }
    cluster.sync();                                          // the totals are read while their blocks last
}

// (lanes of a token, experts of a lane) for E experts.
template <typename F>
cudaError_t with_layout(int E, F f) {
    if (E <= 32) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
    if (E <= 64) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{});
    if (E <= 128) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
    if (E <= 256) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 8>{});
    if (E <= 512) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 32>{});
}

int rows_of(int E) { return E <= 64 ? 32 : E <= 128 ? 16 : E <= 512 ? 8 : 4; }

}  // namespace

RouteTiles route_tiles(int64_t T, int64_t E) {
    const int64_t rows = rows_of(static_cast<int>(E));
    const int64_t passes = (T + rows - 1) / rows;
    int64_t each = (passes + route_max_blocks(E) - 1) / route_max_blocks(E);
    if (each > kRouteMaxPasses) each = kRouteMaxPasses;
    RouteTiles r;
    r.per_block = each * rows;
    r.blocks = (passes + each - 1) / each;
    return r;
}

cudaError_t launch_route(const RouteLaunch &launch, cudaStream_t st) {
    RouteLaunch p = launch;
    const RouteTiles tiles = route_tiles(p.T, p.E);
    cudaError_t err = with_layout(p.E, [&](auto g, auto v) {
        constexpr int G = decltype(g)::value, V = decltype(v)::value;
        const int gs = p.E / p.n_group, lanes = gs / V;
        p.group_lanes = V <= 8 && p.group_topn <= 2 && gs % V == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
        const dim3 grid(static_cast<unsigned>(tiles.blocks));
        const bool brief = p.dtype != MOE_DTYPE_F32 && p.sel_bias == nullptr;
        if (p.losses != nullptr)
            return brief ? launch_dep(route_kernel<G, V, true, true>, grid, dim3(kBlock<V>), 0, st, p)
                         : launch_dep(route_kernel<G, V, true, false>, grid, dim3(kBlock<V>), 0, st, p);
        return brief ? launch_dep(route_kernel<G, V, false, true>, grid, dim3(kBlock<V>), 0, st, p)
                     : launch_dep(route_kernel<G, V, false, false>, grid, dim3(kBlock<V>), 0, st, p);
    });
    note_launches(1);
    if (err != cudaSuccess || p.losses == nullptr) return err;
    const int chunks = (p.E + 31) / 32;
    const int seqs = p.S < 1024 ? p.S : 1024;
    err = launch_dep(route_reduce_kernel, dim3(chunks, seqs), dim3(kReduceThreads), 0, st, p);
    note_launches(1);
    return err;
}

cudaError_t launch_route_backward(const RouteBackwardLaunch &p, cudaStream_t st) {
    const RouteTiles tiles = route_tiles(p.T, p.E);
    const cudaError_t err = with_layout(p.E, [&](auto g, auto v) {
        constexpr int G = decltype(g)::value, V = decltype(v)::value;
        return launch_dep(route_backward_kernel<G, V>, dim3(static_cast<unsigned>(tiles.blocks)), dim3(kBlock<V>), 0, st, p);
    });
    note_launches(1);
    return err;
}

cudaError_t launch_bias_update(float *bias, const int32_t *counts, int L, int S, int E, float rate, cudaStream_t st) {
    const bool whole = E % 4 == 0 && reinterpret_cast<uintptr_t>(counts) % 16 == 0;
    const int quarter = (E + 4 * kBiasBlocks - 1) / (4 * kBiasBlocks) * 4;    // experts of a block, at most 256
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L * kBiasBlocks);
    cfg.blockDim = dim3(kBiasThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kBiasBlocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t err = whole ? cudaLaunchKernelEx(&cfg, bias_update_kernel<4>, bias, counts, S, E, quarter, rate)
                                  : cudaLaunchKernelEx(&cfg, bias_update_kernel<1>, bias, counts, S, E, quarter, rate);
    note_launches(1);
    return err;
}

}  // namespace moe
