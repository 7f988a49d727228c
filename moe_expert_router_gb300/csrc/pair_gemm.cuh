// pair_gemm.cuh -- the grouped products on pairs of SMs: a cluster of two CTAs multiplies one tile
// of 256 x 256 with cta_group::2 MMAs, each holding half of both operands and 128 rows of the
// accumulator. At the bytes per flop of the one-CTA kernel's 256 x 256 unit (32 KB a CTA for a
// 64-deep k-block of 128 x 256) that leaves half of tensor memory free, so the accumulator is
// doubled and a tile's epilogue runs under the next tile's MMAs: what the weight gradients, whose
// tiles add up a group's few rows only, spend half of their time on otherwise.
//
//   kPairRows   out[r, n] = x[r, :] . w[g, n, :]     w [G, N, K], K-major
//   kPairRowsT  out[r, n] = x[r, :] . w[g, :, n]     w [G, K, N], MN-major
//   kPairWgrad  dw[g, n, k] = sum over g's rows of a[r, n] b[r, k]
//   kPairMx     kPairRows on MXFP8 operands
//
// In the first two the matrix is the MMA's A (256 columns n of out as its M) and the rows are its B:
// N is any multiple of 32, so a tile takes little more tensor time than its rows need, and a group's rows
// are cut into equal tiles (384 rows: two of 192). A lane of tensor memory is then a column of out
// and the accumulator's columns are rows: the epilogue's stores of one row are 64 consecutive bytes
// of a warp. In the third both operands are read MN-major over the group's rows. Its last k-block may
// reach behind them, into rows of the next group, which may hold NaN: every group has tensor maps of
// its own that end where it does, so that the copy engine fills zeros there (grouped_maps_kernel).
// (Warps that zeroed those rows in shared memory cost 112 of 330 us for 24576 rows of 64 groups,
// 2048 x 2816: the MMAs waited for them at every tile's end.)
//
// kPairMx runs the block-scaled MMAs on E4M3 codes, 128 deep a stage. The scale words (one of a row and
// k-block) come with TMA, those of two or four k-blocks at a time, and four more warps of each CTA put them into its
// tensor memory: those of its own half of the matrix's columns, and of all rows of x.
//
// Roles of a CTA: warp 0 loads its halves with TMA onto the leader's barriers; warp 1 of the leader
// issues the MMAs; warps 2 .. 9 are the epilogue. Tiles are dealt to the clusters in turn. Every CTA
// reads the group offsets itself.
#pragma once

#include <type_traits>

#include "gemm_kernel.cuh"

namespace moe {

namespace {

enum PairMode : int { kPairRows = 0, kPairRowsT = 1, kPairWgrad = 2, kPairMx = 3 };

constexpr int kPairHalf = 128 * BK * 2;     // bytes of a CTA's half of one operand's k-block
constexpr int kPairBoxRows = 32;            // rows of x in one copy: of these, or of all that a CTA can have
constexpr int kMaxGroups = 1024;
constexpr uint64_t kBlockLimitNs = 2000;    // of a k-block, in a wait for a whole sum

template <int MODE> constexpr int kPairThreads = 64 + EPI_THREADS + (MODE == kPairMx ? HELPER_THREADS : 0);
template <int MODE> constexpr bool kPairAMn = MODE == kPairRowsT || MODE == kPairWgrad;
template <int MODE> constexpr bool kPairBMn = MODE == kPairWgrad;

// Shared memory for tiles of at most MOST rows of x (kPairWgrad: 256). Their bytes of a k-block in a CTA, of
// x beside the matrix's 16 KB, leave room for ten stages or six: with few rows a tile only streams its
// matrix, and more of it in flight counts (1024 rows of 64 groups, 4096 x 1536: 128 us, and 134 with six).
template <int MOST> constexpr int kPairB = MOST / 2 * BK * 2;
template <int MOST> constexpr int kPairStagesOf = MOST == 64 ? 10 : MOST == 192 ? 7 : 6;
// kPairMx: the scale words of some k-blocks in shared memory, of 128 matrix rows and, from a row whose number
// is a multiple of 4, of MOST rows of x; in tensor memory 16 columns a k-block behind each accumulator, of four
// k-blocks where these leave 64 columns, of two where they leave 32.
constexpr int kSfSlots = 3;
template <int MOST> constexpr int kSfDeepOf = MOST > 192 ? 2 : 4;
template <int MOST> constexpr int kPairSfB = kSfDeepOf<MOST> * 512;
template <int MOST> constexpr int kPairSfBytes = kPairSfB<MOST> + kSfDeepOf<MOST> * 4 * (MOST + 4);     // of a copy
template <int MODE, int MOST> constexpr int kPairSf = MODE == kPairMx ? (kPairSfBytes<MOST> + 127) / 128 * 128 : 16;
template <int MODE, int MOST>
struct __align__(1024) PairSmem {
    static constexpr int kPairStages = kPairStagesOf<MOST>;
    uint8_t a[kPairStages][kPairHalf];
    uint8_t b[kPairStages][kPairB<MOST>];
    uint8_t box[MODE == kPairWgrad ? EPI_WARPS : 1][32 * 64];       // kPairWgrad: a warp's 32 x 32 output box
    uint8_t sf[kSfSlots][kPairSf<MODE, MOST>];              // kPairMx: scale words
    uint64_t sf_full[kSfSlots];             // ... have landed
    uint64_t sf_read[kSfSlots];             // ... have been read
    uint64_t sf_ready[2];                   // the leader's: ... are in tensor memory of both CTAs
    uint64_t sf_free[2];                    // ... the MMAs have used them
    uint64_t full[kPairStages];             // the leader's: both CTAs' halves have landed
    uint64_t empty[kPairStages];            // the MMAs have read the stage
    uint64_t acc_full[2];
    uint64_t acc_empty[2];                  // the leader's: every epilogue warp of both CTAs has read it
    uint64_t drain;
    int start[kMaxGroups + 1];              // the groups' first rows
    int tiles[kMaxGroups + 1];              // prefix of their row tiles
    int scan[32];
    uint32_t none;                          // kPairWgrad: what a group without rows has, two of it
    uint32_t tmem_base;
    int abort;
};
template <int MODE, int MOST> constexpr size_t kPairSmemBytes = sizeof(PairSmem<MODE, MOST>) + 1024;

struct PairArgs {
    const int32_t *offsets;
    int32_t *err;
    uint16_t *out;
    int64_t ld_out;
    int R, G;
    int K;                  // rows: the reduction; kPairWgrad: columns of dw
    int N;                  // columns of out; kPairWgrad: rows of dw
    int n_tiles, k_tiles;
    int f16;
    int nan_on_bad;         // bad offsets: out becomes NaN
    int a_one, b_one;       // MN-major operands: both 64-column atoms in one copy
    const CUtensorMap *group_maps;  // kPairWgrad: a's and b's of each group
};
struct PairMaps {
    CUtensorMap a, b;
    CUtensorMap b_wide;     // rows: x in boxes of MOST / 2 rows
};
struct PairMxMaps : PairMaps {
    CUtensorMap sfa, sfb;   // scale words of the matrices, and of x
};
template <int MODE> using PairMapsOf = std::conditional_t<MODE == kPairMx, PairMxMaps, PairMaps>;

// Two NaN of the operands' type.
__device__ __forceinline__ uint32_t nan_16x2(bool f16) { return f16 ? 0x7e007e00u : 0x7fc07fc0u; }

// ---------------------------------------------------------------- cluster and pair instructions

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The leader's copy of a shared-memory object of this CTA.
__device__ __forceinline__ uint32_t leader_addr(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}
// Arrives on a barrier of either CTA. What it tells of (reads of tensor memory, which tcgen05.wait::ld has
// seen completed) needs no release at the cluster's scope, which waits until this SM's stores to global
// memory have been seen. (With it, in every k-block, the kernel took 2.4 times as long; at the
// accumulators' release the weight gradients of 32 groups of 256 rows, 7168 x 4096, 591 us, and 439 without.)
__device__ __forceinline__ void mbar_arrive_peer(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Loads into this CTA's shared memory that complete on a barrier of either CTA of the pair.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z,
                                             uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
// Both 64-column atoms of a matrix's k-block: inner coordinate 0, then k, atom and group.
__device__ __forceinline__ void pair_load_4d(uint32_t dst, const CUtensorMap *map, int32_t y, int32_t z, int32_t g,
                                             uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(g), "r"(bar) : "memory");
}
// Before the first use of a tensor map that a kernel wrote.
__device__ __forceinline__ void tensormap_acquire(const CUtensorMap *map) {
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void pair_mma_mx(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc) : "memory");
}
// One lane of a warp that runs together: always the same one. (In code that one lane runs by this choice the
// compiler knows so, and the operands of copies and MMAs stay in uniform registers. By `lane == 0` four MMAs and a
// commit took 565 .. 780 cycles to issue: 1024 rows of 64 groups, 4096 x 1536, 141 us, and 130 by this; MXFP8 91
// and 76.)
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// A place in a ring of N slots, and the parity of its turn.
template <int N> struct Ring {
    int s = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) {
            s = 0;
            turn ^= 1u;
        }
    }
};
// A matrix descriptor `bytes` further on.
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) {
    return (desc & 0xffffffff00000000ull) | (static_cast<uint32_t>(desc) + (bytes >> 4));
}
// Arrives on `bar` in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
}

// ---------------------------------------------------------------- epilogue pieces

// Two fp32 values rounded to the operands' type.
__device__ __forceinline__ uint32_t pack_16x2(float lo, float hi, bool f16) {
    if (f16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    return pack_bf16x2(lo, hi);
}

// 64 accumulator columns, packed: both loads in flight before the one wait.
__device__ __forceinline__ void pair_piece2(uint32_t tacc, bool f16, uint32_t (&pk0)[16], uint32_t (&pk1)[16]) {
    uint32_t v0[32], v1[32];
    tmem_ld32(tacc, v0);
    tmem_ld32(tacc + 32, v1);
    tmem_wait_ld();
    tmem_reg_fence(v0);
    tmem_reg_fence(v1);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        pk0[i] = pack_16x2(__uint_as_float(v0[2 * i]), __uint_as_float(v0[2 * i + 1]), f16);
        pk1[i] = pack_16x2(__uint_as_float(v1[2 * i]), __uint_as_float(v1[2 * i + 1]), f16);
    }
}

// ---------------------------------------------------------------- tiles

struct PairTile {
    int g, n0;              // group, first column of out (row of dw)
    int row0, rows;         // rows of x (of this tile), or of the group
    int k0;                 // kPairWgrad: first column of dw
    int nkb;                // k-blocks
};

template <int MODE, int MOST>
__device__ __forceinline__ PairTile pair_tile(int u, const PairSmem<MODE, MOST> &sm, const PairArgs &p) {
    PairTile t;
    if constexpr (MODE == kPairWgrad) {
        const int per = p.n_tiles * p.k_tiles;
        t.g = u / per;
        const int rem = u - t.g * per;
        const int n = rem / p.k_tiles;
        t.n0 = n * 256;
        t.k0 = (rem - n * p.k_tiles) * 256;
        t.row0 = sm.start[t.g];
        t.rows = sm.start[t.g + 1] - t.row0;
        t.nkb = (t.rows + BK - 1) / BK;
    } else {
        int lo = 0, hi = p.G;               // tiles of group g: [tiles[g], tiles[g + 1]) * n_tiles
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sm.tiles[mid] * p.n_tiles <= u) lo = mid; else hi = mid;
        }
        const int mine = sm.tiles[lo + 1] - sm.tiles[lo];
        const int local = u - sm.tiles[lo] * p.n_tiles;
        const int n = local / mine, m = local - n * mine;
        const int rows = sm.start[lo + 1] - sm.start[lo];
        const int each = ((rows + mine - 1) / mine + 31) & ~31;
        t.g = lo;
        t.n0 = n * 256;
        t.k0 = 0;
        t.row0 = sm.start[lo] + m * each;
        t.rows = min(each, rows - m * each);
        t.nkb = MODE == kPairMx ? p.K / 128 : (p.K + BK - 1) / BK;
    }
    return t;
}

// kPairWgrad: this CTA's halves of 64 rows of a and b from `row` on.
__device__ __forceinline__ void pair_load_rows(uint32_t sa, uint32_t sb, const CUtensorMap *ma, const CUtensorMap *mb,
                                               const PairArgs &p, const PairTile &t, uint32_t rank, int row, uint32_t bar) {
    const int n = t.n0 + 128 * static_cast<int>(rank), k = t.k0 + 128 * static_cast<int>(rank);
    if (p.a_one) {
        pair_load_3d(sa, ma, 0, row, n / 64, bar);
    } else {
        pair_load_2d(sa, ma, n, row, bar);
        pair_load_2d(sa + MN_ATOM_BYTES, ma, n + 64, row, bar);
    }
    if (p.b_one) {
        pair_load_3d(sb, mb, 0, row, k / 64, bar);
    } else {
        pair_load_2d(sb, mb, k, row, bar);
        pair_load_2d(sb + MN_ATOM_BYTES, mb, k + 64, row, bar);
    }
}

// ---------------------------------------------------------------- the kernel

template <int MODE, int MOST>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads<MODE>, 1)
pair_gemm_kernel(const __grid_constant__ PairMapsOf<MODE> maps, const PairArgs p) {
    griddep_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    using Smem = PairSmem<MODE, MOST>;
    constexpr int kPairStages = Smem::kPairStages, kSfDeep = kSfDeepOf<MOST>;
    static_assert(kPairSmemBytes<MODE, MOST> <= 227 * 1024, "shared memory of a CTA");
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw + ((1024u - (raw & 1023u)) & 1023u));
    volatile int *abort_flag = &sm.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(smem_addr(&sm.full[s]), 1);
            mbar_init(smem_addr(&sm.empty[s]), 1);
        }
        for (int s = 0; MODE == kPairMx && s < kSfSlots; ++s) {
            mbar_init(smem_addr(&sm.sf_full[s]), 1);
            mbar_init(smem_addr(&sm.sf_read[s]), HELPER_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&sm.acc_full[b]), 1);
            mbar_init(smem_addr(&sm.acc_empty[b]), 2 * EPI_WARPS);
            if constexpr (MODE == kPairMx) {
                mbar_init(smem_addr(&sm.sf_ready[b]), 2 * HELPER_WARPS);
                mbar_init(smem_addr(&sm.sf_free[b]), 1);
            }
        }
        mbar_init(smem_addr(&sm.drain), 1);
        sm.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.a);
        tma_prefetch_desc(&maps.b);
        tma_prefetch_desc(&maps.b_wide);
        if constexpr (MODE == kPairMx) {
            tma_prefetch_desc(&maps.sfa);
            tma_prefetch_desc(&maps.sfb);
        }
    }
    if (warp == 1) pair_tmem_alloc(smem_addr(&sm.tmem_base), 512);
    tc_fence_before();
    griddep_wait();

    // The groups' rows and the prefix of their tiles. Offsets that decrease or leave [0, R] would send a
    // product out of its operands: then no group has rows, and the error word says so.
    constexpr int PER = 4;                  // groups a thread
    static_assert(PER * kPairThreads<MODE> >= kMaxGroups, "every group has a thread");
    int first[PER], count[PER], sum = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int g = threadIdx.x * PER + i;
        first[i] = g < p.G ? p.offsets[g] : 0;
        const int end = g < p.G ? p.offsets[g + 1] : 0;
        bad |= g < p.G && (first[i] < 0 || end < first[i] || end > p.R);
        count[i] = end - first[i];
        sum += (count[i] + MOST - 1) / MOST;
    }
    bad = __syncthreads_or(bad);
    if (bad) sum = 0;
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += sm.scan[w];
    int before = incl - sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int g = threadIdx.x * PER + i;
        if (g < p.G) {
            sm.start[g] = bad ? 0 : first[i];
            if (g == p.G - 1) sm.start[p.G] = bad ? 0 : first[i] + count[i];
            sm.tiles[g] = before;
            before += bad ? 0 : (count[i] + MOST - 1) / MOST;
            if (g == p.G - 1) sm.tiles[p.G] = before;
        }
    }
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, MOE_DEVERR_BAD_OFFSETS);
    if (threadIdx.x == 0) sm.none = bad && p.nan_on_bad ? nan_16x2(p.f16) : 0u;
    if (MODE != kPairWgrad && bad && p.nan_on_bad) {        // (no tile writes out then)
        const int cols = p.N / 2;                           // pairs of columns: rows are 16-byte aligned
        const int64_t step = static_cast<int64_t>(gridDim.x) * kPairThreads<MODE>;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPairThreads<MODE> + threadIdx.x; i < static_cast<int64_t>(p.R) * cols; i += step)
            *reinterpret_cast<uint32_t *>(p.out + i / cols * p.ld_out + i % cols * 2) = nan_16x2(p.f16);
    }
    __syncthreads();
    cluster_sync();                         // both CTAs' barriers and tensor memory are set up
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    const int total = MODE == kPairWgrad ? p.G * p.n_tiles * p.k_tiles : sm.tiles[p.G] * p.n_tiles;

    if (warp == 0) {
        // ------------------------------------------------ loads
        if (elect_one()) {
            int seen = -1;
            bool ok = true;
            Ring<kPairStages> at;
            Ring<kSfSlots> sf;
            for (int u = cluster; ok && u < total; u += clusters) {
                const PairTile t = pair_tile<MODE, MOST>(u, sm, p);
                const CUtensorMap *ma = &maps.a, *mb = &maps.b;
                if constexpr (MODE == kPairWgrad) {
                    ma = p.group_maps + 2 * t.g;
                    mb = ma + 1;
                    if (t.g != seen) {
                        tensormap_acquire(ma);
                        tensormap_acquire(mb);
                        seen = t.g;
                    }
                }
                // the tile's rows in this CTA (half of the MMA's N), in one copy or in copies of 32
                const int half = MODE == kPairWgrad ? 128 : ((t.rows + 31) & ~31) / 2;
                const bool wide = half > 64;
                const uint32_t bytes =
                    kPairHalf + (wide ? MOST / 2 : (half + kPairBoxRows - 1) / kPairBoxRows * kPairBoxRows) * BK * 2;
                const int n = t.n0 + 128 * static_cast<int>(rank);
                const int r = t.row0 + half * static_cast<int>(rank);
                for (int kb = 0; kb < t.nkb; ++kb, at.next()) {
                    if constexpr (MODE == kPairMx) {
                        if (kb % kSfDeep == 0) {
                            const uint32_t sff = smem_addr(&sm.sf_full[sf.s]), dst = smem_addr(sm.sf[sf.s]);
                            ok = mbar_wait(smem_addr(&sm.sf_read[sf.s]), sf.turn ^ 1u, abort_flag, p.err);
                            if (!ok) break;
                            mbar_arrive_expect_tx(sff, kPairSfBytes<MOST>);
                            tma_load_2d(dst, &maps.sfa, t.g * p.N + n, kb, sff);
                            tma_load_2d(dst + kPairSfB<MOST>, &maps.sfb, t.row0 & ~3, kb, sff);
                            sf.next();
                        }
                    }
                    ok = mbar_wait(smem_addr(&sm.empty[at.s]), at.turn ^ 1u, abort_flag, p.err);
                    if (!ok) break;
                    const uint32_t sa = smem_addr(sm.a[at.s]), sb = smem_addr(sm.b[at.s]);
                    // (the leader expects both CTAs' bytes: an arrival of the other with release at the
                    // cluster's scope in every k-block made the kernel 2.4 times slower)
                    const uint32_t bar = leader_addr(smem_addr(&sm.full[at.s]));
                    if (rank == 0) mbar_arrive_expect_tx(smem_addr(&sm.full[at.s]), 2 * bytes);
                    const int kx = kb * (MODE == kPairMx ? 128 : BK);
                    if constexpr (MODE == kPairRows || MODE == kPairMx) {
                        pair_load_2d(sa, &maps.a, kx, t.g * p.N + n, bar);
                    } else if constexpr (MODE == kPairRowsT) {
                        if (p.a_one) {
                            pair_load_4d(sa, &maps.a, kx, n / 64, t.g, bar);
                        } else {
                            pair_load_3d(sa, &maps.a, n, kx, t.g, bar);
                            pair_load_3d(sa + MN_ATOM_BYTES, &maps.a, n + 64, kx, t.g, bar);
                        }
                    } else {
                        pair_load_rows(sa, sb, ma, mb, p, t, rank, t.row0 + kx, bar);
                    }
                    if constexpr (MODE != kPairWgrad) {
                        if (MOST > 64 && wide) {
                            pair_load_2d(sb, &maps.b_wide, kx, r, bar);
                        } else {
                            for (int i = 0; i < half; i += kPairBoxRows)
                                pair_load_2d(sb + i * BK * 2, &maps.b, kx, r + i, bar);
                        }
                    }
                }
            }
            // the last arrivals on this CTA's barriers have come before it ends: `empty` completes once for each
            // turn, and of a slot that was never filled the turn before the first counts as complete
            for (int i = 0; ok && i < kPairStages; ++i, at.next())
                ok = mbar_wait(smem_addr(&sm.empty[at.s]), at.turn ^ 1u, abort_flag, p.err);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMAs, of both CTAs by the leader
        if (rank == 0 && elect_one()) {
            int n_done = 0;
            bool ok = true, any = false;
            Ring<kPairStages> at;
            Ring<2> sf;
            const uint32_t full0 = smem_addr(sm.full), empty0 = smem_addr(sm.empty);
            const uint64_t a0 = operand_desc<kPairAMn<MODE>>(smem_addr(sm.a), 0);
            const uint64_t b0 = operand_desc<kPairBMn<MODE>>(smem_addr(sm.b), 0);
            for (int u = cluster; ok && u < total; u += clusters, ++n_done) {
                const PairTile t = pair_tile<MODE, MOST>(u, sm, p);
                const int buf = n_done & 1;
                ok = mbar_wait(smem_addr(&sm.acc_empty[buf]), ((n_done >> 1) & 1) ^ 1u, abort_flag, p.err);
                if (!ok) break;
                tc_fence_after();
                const int n_mma = MODE == kPairWgrad ? 256 : (t.rows + 31) & ~31;
                uint32_t idesc = MODE == kPairMx ? idesc_mxf8(256, n_mma, 0)
                                                 : idesc_bf16_f32(256, n_mma) | (kPairAMn<MODE> ? (1u << 15) : 0u) |
                                                       (kPairBMn<MODE> ? (1u << 16) : 0u);
                if (MODE != kPairMx && p.f16) idesc &= ~((1u << 7) | (1u << 10));   // operand formats 0, fp16, for 1, bf16
                const uint32_t acc = tmem + buf * 256;
                constexpr int DEEP = MODE == kPairMx ? kSfDeep : 1;
                for (int kb0 = 0; ok && kb0 < t.nkb; kb0 += DEEP) {
                    if constexpr (MODE == kPairMx) {
                        ok = mbar_wait(smem_addr(&sm.sf_ready[sf.s]), sf.turn, abort_flag, p.err);
                        if (!ok) break;
                        tc_fence_after();
                    }
#pragma unroll
                    for (int d = 0; d < DEEP; ++d) {
                        if (d > 0 && kb0 + d >= t.nkb) break;
                        ok = mbar_wait(full0 + 8 * at.s, at.turn, abort_flag, p.err);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t da = desc_at(a0, kPairHalf * at.s), db = desc_at(b0, kPairB<MOST> * at.s);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint32_t more = d > 0 || kk > 0 ? 1u : kb0 > 0;
                            if constexpr (MODE == kPairMx) {        // K = 32 each: byte kk of the scale words
                                const uint32_t words = tmem + 256 * sf.s + MOST + 16 * d;
                                pair_mma_mx(acc, desc_at(da, 32 * kk), desc_at(db, 32 * kk), idesc | idesc_mxf8(0, 0, kk), words,
                                            words + 8, more);
                            } else {
                                pair_mma(acc, desc_at(da, kk * (kPairAMn<MODE> ? UMMA_K * 128 : UMMA_K * 2)),
                                         desc_at(db, kk * (kPairBMn<MODE> ? UMMA_K * 128 : UMMA_K * 2)), idesc, more);
                            }
                        }
                        pair_commit(empty0 + 8 * at.s);
                        any = true;
                        at.next();
                    }
                    if constexpr (MODE == kPairMx) {
                        if (ok) pair_commit(smem_addr(&sm.sf_free[sf.s]));
                        sf.next();
                    }
                }
                if (!ok) break;
                pair_commit(smem_addr(&sm.acc_full[buf]));      // at once without k-blocks: the epilogue writes zeros
            }
            if (!ok && any) {
                pair_commit(smem_addr(&sm.drain));
                drain_wait(smem_addr(&sm.drain), 0);
            }
        }
        __syncwarp();
    } else if (warp < 2 + EPI_WARPS) {
        // ------------------------------------------------ epilogue
        const int quad = warp & 3, side = (warp - 2) >> 2;      // lanes of tensor memory, half of the columns
        const uint32_t tacc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 128 * side;
        const uint32_t buf_addr = smem_addr(sm.box[MODE == kPairWgrad ? warp - 2 : 0]);
        const bool f16 = p.f16 != 0;
        int n_done = 0;
        for (int u = cluster; u < total; u += clusters, ++n_done) {
            const PairTile t = pair_tile<MODE, MOST>(u, sm, p);
            const int buf = n_done & 1;
            bool ok = true;
            // (the one wait that lasts as long as a tile's sum: a k-block takes some 0.25 us, so that a second is over
            // after 240 million rows of a group, or columns of K)
            if (lane == 0)
                ok = mbar_wait(smem_addr(&sm.acc_full[buf]), (n_done >> 1) & 1, abort_flag, p.err,
                               kWaitLimitNs + kBlockLimitNs * static_cast<uint64_t>(t.nkb));
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            tc_fence_after();
            const int n = t.n0 + 128 * static_cast<int>(rank) + 32 * quad;      // the warp's first lane
            const uint32_t released = leader_addr(smem_addr(&sm.acc_empty[buf]));
            if constexpr (MODE != kPairWgrad) {
                uint16_t *dst = p.out + t.row0 * p.ld_out + n + lane;
                const bool live = n + lane < p.N;
                const int end = min(t.rows, 128 * side + 128);
#pragma unroll 1
                for (int c = 128 * side; c < end; c += 64) {
                    uint32_t v[2][32];
                    tmem_ld32(tacc + 256 * buf + (c - 128 * side), v[0]);
                    if (c + 32 < end) tmem_ld32(tacc + 256 * buf + (c + 32 - 128 * side), v[1]);
                    tmem_wait_ld();
                    tmem_reg_fence(v[0]);
                    tmem_reg_fence(v[1]);
                    if (c + 64 >= end) {                    // read out: free for the tile after next
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_peer(released);
                    }
                    if (live) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint16_t *at = dst + (c + 32 * q) * p.ld_out;
                            const int m = t.rows - c - 32 * q;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (i < m) *at = static_cast<uint16_t>(pack_16x2(__uint_as_float(v[q][i]), 0.f, f16));
                                at += p.ld_out;
                            }
                        }
                    }
                }
                if (end <= 128 * side) {                    // no rows on this side
                    __syncwarp();
                    if (lane == 0) mbar_arrive_peer(released);
                }
            } else {
                // the warp's 128 columns in registers first, so that the accumulator is free for the tile
                // after next while they are stored
                const int k = t.k0 + 128 * side;
                const bool work = k < p.K && n < p.N;
                uint32_t pk[4][16];
                if (work && t.rows > 0) {
                    pair_piece2(tacc + 256 * buf, f16, pk[0], pk[1]);
                    pair_piece2(tacc + 256 * buf + 64, f16, pk[2], pk[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 64; ++i) pk[i >> 4][i & 15] = sm.none;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_peer(released);
                if (!work) continue;
                // turned in shared memory, so that a store covers 64 bytes of eight rows
                const int row = lane >> 2, chunk = lane & 3;
                uint16_t *dst = p.out + (static_cast<int64_t>(t.g) * p.N + n + row) * p.K + k + 8 * chunk;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    stage_row32(buf_addr, lane, pk[c]);
                    __syncwarp();
                    uint4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = ld_shared_v4(buf_addr + swizzled_chunk<64>(8 * i + row, chunk));
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n + 8 * i + row < p.N && k + 32 * c + 8 * chunk < p.K)
                            *reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(8 * i) * p.K + 32 * c) = v[i];
                }
            }
        }
    } else {
        // ------------------------------------------------ scale words into tensor memory (kPairMx)
        if constexpr (MODE == kPairMx) {
            const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
            int sf = 0;
            bool ok = true;
            for (int u = cluster; ok && u < total; u += clusters) {
                const PairTile t = pair_tile<MODE, MOST>(u, sm, p);
                const int rem = t.row0 & 3;                 // the copy began at a multiple of 4
                for (int kb = 0; kb < t.nkb; kb += kSfDeep, ++sf) {
                    const int q = sf % kSfSlots;
                    const uint32_t sff = smem_addr(&sm.sf_full[q]), at = smem_addr(sm.sf[q]);
                    const uint32_t parity = (sf / kSfSlots) & 1;
                    if (lane == 0)
                        ok = mbar_wait(sff, parity, abort_flag, p.err) &&
                             mbar_wait(smem_addr(&sm.sf_free[sf & 1]), ((sf >> 1) & 1) ^ 1u, abort_flag, p.err);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    (void)mbar_try_wait(sff, parity);       // every lane sees the phase
                    tc_fence_after();
                    // column j of a k-block: rows 32 j + lane of the matrix, and from column 8 on of x. (Rows behind
                    // the tile's have any scale: their products are not stored.)
#pragma unroll
                    for (int d = 0; d < kSfDeep; ++d) {
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (j < 4) w[j] = ld_shared_u32(at + 512 * d + 4 * (32 * j + lane));
                            else if (j >= 8 && j - 8 < MOST / 32)
                                w[j] = ld_shared_u32(at + kPairSfB<MOST> + 4 * (d * (MOST + 4) + rem + 32 * (j - 8) + lane));
                            else w[j] = 0u;
                        }
                        tmem_st16(mine + 256 * (sf & 1) + MOST + 16 * d, w);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_addr(&sm.sf_read[q]));
                        mbar_arrive_peer(leader_addr(smem_addr(&sm.sf_ready[sf & 1])));
                    }
                }
            }
            // the last arrivals on this CTA's barriers have come before it ends
            for (int i = max(0, sf - 2); ok && lane == 0 && i < sf; ++i)
                ok = mbar_wait(smem_addr(&sm.sf_free[i & 1]), (i >> 1) & 1, abort_flag, p.err);
            __syncwarp();
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();                         // nothing of the pair reads this CTA's memory or barriers any more
    if (sm.abort) {
        // copies in flight may not land in memory that another block has by then
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < kDrainLimitNs) __nanosleep(100000);
    }
    if (warp == 1) {
        tc_fence_after();
        pair_tmem_dealloc(tmem, 512);
    }
}

}  // namespace

}  // namespace moe
