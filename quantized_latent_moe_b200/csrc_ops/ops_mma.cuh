// ops_mma.cuh -- products on the 5th-generation tensor cores: dense or grouped
// by expert with ragged sizes, 8-bit codes (kind::i8, int32 accumulators) or
// bf16 / fp16 (kind::f16, fp32 accumulators).
//
// The weights are the MMA's M operand (128 channels a tile) and the rows of
// activations its N operand, so that a ragged group costs its rows rounded up
// to 16, not to 128, and each weight tile is read from HBM once for up to 256
// rows.  One persistent CTA per SM; units are (expert, channel tile, row tile),
// row tiles innermost, and CTA b takes units b, b + grid, ..., so that the CTAs
// read neighbouring weights and the row tiles of one weight tile share it in L2.
//
// Warp 0 issues tensor-map copies (both operands in 128-byte K steps, 128-byte
// swizzle) into a ring of stages, warp 1 issues the MMAs into one of two TMEM
// accumulators, warps 4..11 drain the other: a warp reads the 32 TMEM lanes
// (channels) it may, 32 rows at a time, rescales, and writes.  Rows of a copied
// box that belong to the next group, or lie past the matrix (zeros), only meet
// accumulator columns that are not written.
//
// Bound by the weights' HBM traffic where groups are small, by L2 to shared memory
// and the tensor cores (and power) where rows are many.  Measured on B200: 256 rows
// over 128 experts of 2048 x 1792 codes 75 us (6.3 TB/s), 16384 rows 92 to 97 us
// (5.8 TB/s; bf16, 1792 x 1024: 96 us), dense 8192 x 4096 x 4096 codes 87 us (3.2
// POP/s, of 4.54 that MMAs alone reach), 2048 x 1792 x 4096 16.2 us: 9.5 us and 0.51
// per 128 of K.
#pragma once

#include <cuda.h>

#include "../csrc/elq_device.cuh"
#include "ops_gemv.cuh"

namespace elqops {

using elq::fence_barrier_init;
using elq::global_timer_ns;
using elq::mbar_arrive_expect_tx;
using elq::mbar_init;
using elq::mbar_try_wait;
using elq::mbar_try_wait_hint;
using elq::smem_addr;

// Set by a product whose bounded wait ran out; read and cleared in one step by
// k_status, so that no other stream's is lost between the two.
__device__ int g_ops_err;
__device__ int g_ops_said;      // what k_status read

inline __global__ void k_status() { g_ops_said = atomicExch(&g_ops_err, 0); }

constexpr uint64_t kOpsWaitNs = 2000000000ull;     // 2 s per bounded device wait (a test's are shorter)
constexpr uint64_t kOpsDrainNs = 100000000ull;     // 0.1 s for what is in flight after one ran out
constexpr int kMmaThreads = 384;
constexpr int kMmaEpiWarps = 8;
constexpr int kMmaStagesMax = 16;
constexpr int kTileCh = 128;                        // channels of a tile
constexpr int kStepBytes = 128;                     // bytes of K a stage holds
constexpr int kABytes = kTileCh * kStepBytes;
constexpr int kBoxRows = 32;                        // rows of one activation copy
constexpr int kBoxBytes = kBoxRows * kStepBytes;
constexpr int kMmaHdr = 512 + kMmaEpiWarps * 32 * 4;
constexpr int kMmaSmemMax = 227 * 1024;

struct alignas(64) MmaArgs {
    CUtensorMap tw;             // weights [E][N][K], box 128 bytes x 128 channels
    CUtensorMap tx;             // activations [M][K], box 128 bytes x 32 rows
    const int32_t* offsets;     // NULL: one group of all M rows
    int M, E, N, Kb;
    int bn;                     // most rows of a tile: a multiple of 32 a CTA, <= 256
    int stages;
    int split;                  // k_split: CTAs of a tile
    int stall;                  // 0; a test's: 1 the first CTA's copies stop one K step short, 2 no accumulator is given back
    uint64_t wait_ns;           // limit of a device wait
    uint32_t idesc;             // instruction descriptor without its N field
    const float* sx;
    const float* sw;
    const float* bias;
    void* y;
    int y_type;
    int64_t ldy;
};

// ---- tcgen05 primitives --------------------------------------------------------

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
    if constexpr (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

template <int KIND, int CG>
__device__ __forceinline__ void umma(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
    if constexpr (KIND == KIND_I8 && CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
            : "memory");
    else if constexpr (KIND == KIND_I8)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
            : "memory");
    else if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
            : "memory");
}
// An arrival on this CTA's barrier when all MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void umma_commit_here(uint64_t* bar) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                     : "memory");
}
// The same, in a pair on both CTAs' barriers at this offset.
template <int CG>
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
    if constexpr (CG == 1)
        umma_commit_here<1>(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_addr(bar)),
            "h"((uint16_t)3)
            : "memory");
}
// One lane of the warp.  Chosen by elect.sync, not by its number: the compiler then
// knows that a single thread issues what follows, and keeps the MMAs' operands in
// uniform registers (a loop of MMAs of 32 rows issues one every 22 ns, behind
// `lane == 0` every 32; 8192 x 4096 x 4096 codes: 87 us, 115 behind `lane == 0`).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Not the .aligned forms: those take a warp to be converged, and lanes that waited
// for an elected one's long loop need not be.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// The cluster address of a CTA's copy of a shared-memory object.
__device__ __forceinline__ uint32_t in_cta(const void* p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t first_cta(const void* p) { return in_cta(p, 0); }
__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// Tensor-map copies into this CTA's shared memory; `bar` is a cluster address, in
// a pair of the first CTA's barrier.  No multicast.
template <int CG>
__device__ __forceinline__ void copy_2d(uint32_t dst, const CUtensorMap* m, int c0, int c1, uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
            "[%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
            "{%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void copy_3d(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
            "[%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
            "{%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
            : "memory");
}

// 32 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_read32(uint32_t t, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Shared-memory descriptor of a K-major operand in 128-byte swizzled rows
// (1024-byte groups of eight rows, one after another).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3fff) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor without N: M = 128 channels a CTA, both operands K-major.
__host__ __device__ constexpr uint32_t mma_idesc(int kind, int cg) {
    return ((uint32_t)(cg * kTileCh >> 4) << 24) |
           (kind == KIND_I8 ? (2u << 4) | (1u << 7) | (1u << 10)
                            : (1u << 4) | (kind == KIND_BF16 ? (1u << 7) | (1u << 10) : 0u));
}

// Whether an mbarrier's phase is over, waiting for it up to hint_ns.  CLUSTER: what threads of the
// cluster's other CTAs did before they arrived is seen too.
template <bool CLUSTER>
__device__ __forceinline__ bool bar_try(uint64_t* bar, uint32_t parity, uint32_t hint_ns) {
    if constexpr (!CLUSTER) return mbar_try_wait_hint(bar, parity, hint_ns);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(hint_ns)
        : "memory");
    return ok != 0;
}

// Bounded wait for an mbarrier phase; gives up at once when another role has.  The
// clock is read only once a wait is long: reading it costs as much as a whole
// step of the pipeline.
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* abort_v, uint64_t limit_ns) {
    for (int i = 0; i < 32; ++i)
        if (CLUSTER ? bar_try<true>(bar, parity, 0) : mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 0; i < (1u << 26); ++i) {
        if (bar_try<CLUSTER>(bar, parity, 20000u)) return true;
        if (*abort_v) return false;
        if ((i & 15) == 15 && global_timer_ns() - t0 > limit_ns) break;
    }
    *abort_v = 1;
    atomicExch(&g_ops_err, 1);
    return false;
}

// The end of a cluster's work: no CTA leaves, and gives up its shared memory, while
// another may still reach it.  Every CTA tells all `n` of them, itself included
// (`bye` counts n), and waits, with a limit, for all to have told it: each of them may
// have begun its last wait when this one's ran out, and may drain its ring after it.
// By all threads.
__device__ __forceinline__ void cluster_leave(uint64_t* bye, int n, uint64_t limit_ns) {
    __syncthreads();
    if ((int)threadIdx.x < n) bar_arrive_cluster(in_cta(bye, threadIdx.x));
    if (threadIdx.x == 0) {
        const uint64_t t0 = global_timer_ns();
        while (!bar_try<true>(bye, 0, 20000u)) {
            if (global_timer_ns() - t0 > 2 * limit_ns + (kMmaStagesMax + 2) * kOpsDrainNs) {
                atomicExch(&g_ops_err, 2);
                break;
            }
        }
    }
    __syncthreads();
}

// Waits, with a limit, for what is in flight: for a barrier's phase, and for the last
// uses (up to `issued`) of a ring whose next use would be stage st in phase ph.
__device__ __forceinline__ void bar_land(uint64_t* bar, uint32_t parity) {
    for (int i = 0; i < 32; ++i)
        if (mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait_hint(bar, parity, 20000u) && global_timer_ns() - t0 < kOpsDrainNs) {
    }
}
__device__ __forceinline__ void ring_land(uint64_t* bars, int stages, long long issued, int st, uint32_t ph) {
    for (int i = 0; i < stages && i < issued; ++i) {
        if (--st < 0) {
            st = stages - 1;
            ph ^= 1;
        }
        bar_land(bars + st, ph);
    }
}

// ---- units -----------------------------------------------------------------------

struct Unit {
    int e, ch0, row0, rows, n;      // expert, first channel, first row, rows, the MMA's N
};

// s_off: the offsets, clamped and raised; s_tile[e]: row tiles of the experts before e; tiles
// have rows in steps of 16 (32 in a pair, where each CTA brings half of them).
template <int CG>
__device__ __forceinline__ Unit unit_of(int u, const int* s_off, const int* s_tile, int E, int ch_tiles) {
    constexpr int step = 16 * CG;
    const int b = u / ch_tiles;
    int lo = 0, hi = E;             // the last e with s_tile[e] <= b
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tile[mid] <= b) lo = mid;
        else hi = mid;
    }
    const int nt = s_tile[lo + 1] - s_tile[lo], r = u - s_tile[lo] * ch_tiles;
    const int ct = r / nt, t = r - ct * nt, cnt = s_off[lo + 1] - s_off[lo];
    const int bn = ((cnt + nt - 1) / nt + step - 1) & ~(step - 1);     // the group's rows in nt even tiles
    Unit x;
    x.e = lo;
    x.ch0 = ct * kTileCh * CG;
    x.row0 = s_off[lo] + t * bn;
    x.rows = min(bn, cnt - t * bn);
    x.n = (x.rows + step - 1) & ~(step - 1);
    return x;
}

// ---- epilogue ----------------------------------------------------------------------
//
// A lane has one channel and 32 rows.  Eight warps have the whole tile's outputs to
// rescale and write while the next tile's MMAs run, so an output's share of
// instructions decides whether they keep up: the output type is chosen once per 32,
// the rows' scales come four at a time, and a row costs one pointer step.

// The accumulators r of 32 rows as outputs: times the rows' scales, then the
// channel's (codes), plus the bias.
template <int KIND>
__device__ __forceinline__ void scale32(const uint32_t (&r)[32], const float* sx, float sw, float bias, bool add,
                                        float (&v)[32]) {
    if (KIND != KIND_I8) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        const float4 s = *reinterpret_cast<const float4*>(sx + j);
        v[j] = __fmul_rn(__fmul_rn((float)(int)r[j], s.x), sw);
        v[j + 1] = __fmul_rn(__fmul_rn((float)(int)r[j + 1], s.y), sw);
        v[j + 2] = __fmul_rn(__fmul_rn((float)(int)r[j + 2], s.z), sw);
        v[j + 3] = __fmul_rn(__fmul_rn((float)(int)r[j + 3], s.w), sw);
    }
    if (add) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __fadd_rn(v[j], bias);
    }
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

// v's first nr values to p, p + ld, ...
template <typename T>
__device__ __forceinline__ void write32(T* p, int64_t ld, int nr, const float (&v)[32]) {
    if (nr == 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j, p += ld) put(p, v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 31; ++j, p += ld)
            if (j < nr) put(p, v[j]);
    }
}

// CG = 2: a pair of CTAs (a cluster, on the two SMs that share a tensor-core pair)
// works on 256 channels by up to 256 rows as one MMA: each CTA brings its own 128
// channels and half of the rows, so that a row travels from L2 to shared memory
// half as often.  The first CTA issues the MMAs; its barriers count both CTAs'
// copies and both epilogues.
template <int KIND, int CG>
__global__ void __launch_bounds__(kMmaThreads, 1) k_mma(const __grid_constant__ MmaArgs a) {
    extern __shared__ uint8_t smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);
    uint64_t* empty = full + kMmaStagesMax;
    uint64_t* tfull = empty + kMmaStagesMax;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint64_t* bye = drain + 1;
    uint64_t* tdone = bye + 1;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(tdone + 2);
    volatile int* abort_v = reinterpret_cast<volatile int*>(s_tmem + 1);
    float* s_sx = reinterpret_cast<float*>(smem + 512);
    int* s_off = reinterpret_cast<int*>(smem + kMmaHdr);
    int* s_tile = s_off + a.E + 1;
    const uint32_t tiles0 = (smem_addr(s_tile + a.E + 1) + 1023u) & ~1023u;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMmaStagesMax; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + i, 1);
            mbar_init(tempty + i, CG == 1 ? kMmaEpiWarps : 2);
            mbar_init(tdone + i, kMmaEpiWarps);
        }
        mbar_init(drain, 1);
        mbar_init(bye, CG);
        *abort_v = 0;
        fence_barrier_init();
    }
    if (warp == 2) tmem_alloc<CG>(s_tmem, 512);
    if (warp == 3 && lane < 2) prefetch_map(lane ? &a.tx : &a.tw);
    pdl_wait();
    for (int i = threadIdx.x; i <= a.E; i += kMmaThreads) s_off[i] = a.offsets ? __ldg(a.offsets + i) : (i ? a.M : 0);
    __syncthreads();
    if (warp == 0) {
        int top = 0, before = 0;        // the largest offset so far; row tiles so far
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int raw = e < a.E ? s_off[e + 1] : 0;         // this batch reads it before the next writes over it
            const int lo = raise_offsets(e < a.E ? s_off[e] : 0, a.M, top);
            const int hi = e < a.E ? max(lo, clamp_offset(raw, a.M)) : lo;
            int t = (hi - lo + a.bn - 1) / a.bn, s = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += v;
            }
            if (e < a.E) {
                s_off[e] = lo;
                s_tile[e] = before + s - t;
                if (e == a.E - 1) s_off[a.E] = hi;
            }
            before += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) s_tile[a.E] = before;
    }
    __syncwarp();
    tc_before();
    if (CG == 1) __syncthreads();
    else cluster_sync();
    tc_after();
    const uint32_t tmem = *s_tmem;
    const int ch_tiles = (a.N + CG * kTileCh - 1) / (CG * kTileCh);
    const int units = s_tile[a.E] * ch_tiles;
    const int steps = (a.Kb + kStepBytes - 1) / kStepBytes;
    const int stage_bytes = kABytes + a.bn / CG * kStepBytes;
    const int rank = CG == 1 ? 0 : (int)cluster_rank(), u0 = blockIdx.x / CG, du = gridDim.x / CG;

    if (warp == 0) {
        if (elect_one()) {
            int st = 0;
            uint32_t ph = 0;
            long long issued = 0;
            bool ok = true;
            for (int u = u0; ok && u < units; u += du) {
                const Unit x = unit_of<CG>(u, s_off, s_tile, a.E, ch_tiles);
                const int boxes = (x.n / CG + kBoxRows - 1) / kBoxRows, row0 = x.row0 + rank * (x.n / CG);
                for (int k = 0; k < steps; ++k) {
                    if (a.stall == 1 && blockIdx.x < CG && k == steps - 1) {
                        ok = false;
                        break;
                    }
                    if (!(ok = bar_wait(empty + st, ph ^ 1, abort_v, a.wait_ns))) break;
                    const uint32_t p = tiles0 + st * stage_bytes, fb = CG == 1 ? smem_addr(full + st) : first_cta(full + st);
                    const int c = k * (KIND == KIND_I8 ? kStepBytes : kStepBytes / 2);
                    if (rank == 0) mbar_arrive_expect_tx(full + st, CG * (kABytes + boxes * kBoxBytes));
                    copy_3d<CG>(p, &a.tw, c, x.ch0 + rank * kTileCh, x.e, fb);
                    for (int b = 0; b < boxes; ++b)
                        copy_2d<CG>(p + kABytes + b * kBoxBytes, &a.tx, c, row0 + b * kBoxRows, fb);
                    ++issued;
                    if (++st == a.stages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            // No copy may be in flight when the CTA gives up its memory, whichever role's wait ran out: the
            // last use of every stage is waited for (a pair's second CTA sees only that the MMAs read it).
            ring_land(rank == 0 ? full : empty, a.stages, issued, st, ph);
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            int st = 0, it = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int u = u0; ok && u < units; u += du, ++it) {
                const Unit x = unit_of<CG>(u, s_off, s_tile, a.E, ch_tiles);
                const int acc = it & 1;
                if (!(ok = bar_wait<CG == 2>(tempty + acc, ((it >> 1) & 1) ^ 1, abort_v, a.wait_ns))) break;
                tc_after();
                const uint32_t idesc = a.idesc | ((uint32_t)(x.n >> 3) << 17), d = tmem + acc * 256;
                for (int k = 0; k < steps; ++k) {
                    if (!(ok = bar_wait(full + st, ph, abort_v, a.wait_ns))) break;
                    tc_after();
                    const uint32_t p = tiles0 + st * stage_bytes;
                    const uint64_t ad = sw128_desc(p), bd = sw128_desc(p + kABytes);
                    const int parts = min(4, (a.Kb - k * kStepBytes + 31) / 32);
                    if (parts == 4) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) umma<KIND, CG>(d, ad + 2 * i, bd + 2 * i, idesc, k > 0 || i > 0);
                    } else {
                        for (int i = 0; i < parts; ++i) umma<KIND, CG>(d, ad + 2 * i, bd + 2 * i, idesc, k > 0 || i > 0);
                    }
                    umma_commit<CG>(empty + st);
                    if (++st == a.stages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                if (ok) umma_commit<CG>(tfull + acc);
            }
            umma_commit_here<CG>(drain);    // nor an MMA
            bar_land(drain, 0);
        }
    } else if (CG == 2 && warp == 3) {
        // A pair's accumulators go back to the first CTA, which issues the MMAs, by a release at cluster
        // scope.  That waits for the outputs stored before it, so this warp, which has nothing else to
        // do, passes the epilogue's arrivals on (released by the epilogue's warps themselves, 2048 x 1792
        // x 4096 took 17.1 us, 16.2 so).
        if (elect_one()) {
            int it = 0;
            for (int u = u0; u < units; u += du, ++it) {
                if (!bar_wait(tdone + (it & 1), (it >> 1) & 1, abort_v, a.wait_ns)) break;
                bar_arrive_cluster(first_cta(tempty + (it & 1)));
            }
        }
    } else if (warp >= 4) {
        const int q = warp & 3, half = (warp - 4) >> 2;
        float* sx = s_sx + (warp - 4) * 32;
        int it = 0;
        for (int u = u0; u < units; u += du, ++it) {
            const Unit x = unit_of<CG>(u, s_off, s_tile, a.E, ch_tiles);
            const int acc = it & 1, n = x.ch0 + rank * kTileCh + q * 32 + lane;
            float sw = 1.0f, bias = 0.0f;
            if (KIND == KIND_I8 && n < a.N) {
                sw = __ldg(a.sw + (int64_t)x.e * a.N + n);
                if (a.bias) bias = __ldg(a.bias + n);
            }
            if (!__all_sync(0xffffffffu, bar_wait(tfull + acc, (it >> 1) & 1, abort_v, a.wait_ns))) break;
            tc_after();
            // The accumulator goes back as soon as this warp's last values of it are in registers.
            auto give_back = [&] {
                tc_before();
                __syncwarp();
                if (lane == 0 && a.stall != 2) bar_arrive((CG == 1 ? tempty : tdone) + acc);
            };
            if (half * 32 >= x.rows) give_back();
            for (int c = half * 32; c < x.rows; c += 64) {
                uint32_t r[32];
                __syncwarp();
                tmem_read32(tmem + acc * 256 + c + ((uint32_t)(q * 32) << 16), r);
                if (c + 64 >= x.rows) give_back();
                const int nr = min(32, x.rows - c);
                if (KIND == KIND_I8) {
                    __syncwarp();
                    sx[lane] = lane < nr ? __ldg(a.sx + x.row0 + c + lane) : 0.0f;
                    __syncwarp();
                }
                float v[32];
                scale32<KIND>(r, sx, sw, bias, a.bias != nullptr, v);
                if (n < a.N) {
                    const int64_t at = (int64_t)(x.row0 + c) * a.ldy + n;
                    if (a.y_type == ELQ_F32) write32(reinterpret_cast<float*>(a.y) + at, a.ldy, nr, v);
                    else if (a.y_type == ELQ_BF16) write32(reinterpret_cast<__nv_bfloat16*>(a.y) + at, a.ldy, nr, v);
                    else write32(reinterpret_cast<__half*>(a.y) + at, a.ldy, nr, v);
                }
                __syncwarp();
            }
        }
    }
    __syncwarp();
    tc_before();
    if (CG == 1) __syncthreads();
    else cluster_leave(bye, CG, a.wait_ns);
    tc_after();
    if (warp == 2) tmem_free<CG>(tmem, 512);
}

// ---- split over K ------------------------------------------------------------------
//
// A dense product (they are of codes) with few tiles would leave most SMs idle and run each tile's K
// steps one after another.  Here a cluster of up to eight CTAs works on one tile,
// each on its share of the K steps; the partial accumulators go to shared memory
// and every CTA adds up and writes its share of the rows, reading the others'
// partials through distributed shared memory in rank order (so the result does
// not depend on timing).  Bound by latency: launch, one memory round trip, the
// steps of a share, one exchange.
__global__ void __launch_bounds__(kMmaThreads, 1) k_split(const __grid_constant__ MmaArgs a) {
    extern __shared__ uint8_t smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);
    uint64_t* empty = full + kMmaStagesMax;
    uint64_t* tfull = empty + kMmaStagesMax;
    uint64_t* bye = tfull + 1;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bye + 1);
    volatile int* abort_v = reinterpret_cast<volatile int*>(s_tmem + 1);
    const uint32_t tiles0 = (smem_addr(smem) + 512 + 1023u) & ~1023u;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int S = a.split, rank = (int)cluster_rank(), tile = blockIdx.x / S;
    const int ch_tiles = (a.N + kTileCh - 1) / kTileCh;
    const int ch0 = tile % ch_tiles * kTileCh, row0 = tile / ch_tiles * a.bn, rows = min(a.bn, a.M - row0);
    const int n = (rows + 15) & ~15, boxes = (n + kBoxRows - 1) / kBoxRows;
    const int steps = (a.Kb + kStepBytes - 1) / kStepBytes;
    const int k0 = (int)((int64_t)steps * rank / S), k1 = (int)((int64_t)steps * (rank + 1) / S);
    const int stage_bytes = kABytes + a.bn * kStepBytes;

    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        mbar_init(tfull, 1);
        mbar_init(bye, S);
        *abort_v = 0;
        fence_barrier_init();
    }
    if (warp == 2) tmem_alloc<1>(s_tmem, 256);
    if (warp == 3 && lane < 2) prefetch_map(lane ? &a.tx : &a.tw);
    pdl_wait();
    __syncwarp();
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *s_tmem;

    if (warp == 0) {
        if (elect_one()) {
            int st = 0, issued = 0;
            uint32_t ph = 0;
            for (int k = k0; k < k1; ++k) {
                if (a.stall == 1 && blockIdx.x == 0 && k == k1 - 1) break;
                if (!bar_wait(empty + st, ph ^ 1, abort_v, a.wait_ns)) break;
                const uint32_t p = tiles0 + st * stage_bytes, fb = smem_addr(full + st);
                const int c = k * kStepBytes;
                mbar_arrive_expect_tx(full + st, kABytes + boxes * kBoxBytes);
                copy_3d<1>(p, &a.tw, c, ch0, 0, fb);
                for (int b = 0; b < boxes; ++b) copy_2d<1>(p + kABytes + b * kBoxBytes, &a.tx, c, row0 + b * kBoxRows, fb);
                ++issued;
                if (++st == a.stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            ring_land(full, a.stages, issued, st, ph);      // as in k_mma
        }
    } else if (warp == 1) {
        if (elect_one()) {
            int st = 0;
            uint32_t ph = 0;
            const uint32_t idesc = a.idesc | ((uint32_t)(n >> 3) << 17);
            for (int k = k0; k < k1; ++k) {
                if (!bar_wait(full + st, ph, abort_v, a.wait_ns)) break;
                tc_after();
                const uint32_t p = tiles0 + st * stage_bytes;
                const uint64_t ad = sw128_desc(p), bd = sw128_desc(p + kABytes);
                const int parts = min(4, (a.Kb - k * kStepBytes + 31) / 32);
                if (parts == 4) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) umma<KIND_I8, 1>(tmem, ad + 2 * i, bd + 2 * i, idesc, k > k0 || i > 0);
                } else {
                    for (int i = 0; i < parts; ++i) umma<KIND_I8, 1>(tmem, ad + 2 * i, bd + 2 * i, idesc, k > k0 || i > 0);
                }
                umma_commit<1>(empty + st);
                if (++st == a.stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            umma_commit<1>(tfull);      // also after a wait that ran out: nothing may be in flight at the end
            bar_land(tfull, 0);
        }
    }
    __syncwarp();
    // Every warp waits for the MMAs (the ring is free then), eight of them move
    // the accumulators: word (row, channel) at part[row * 128 + channel].
    const bool done = __all_sync(0xffffffffu, bar_wait(tfull, 0, abort_v, a.wait_ns));
    __syncthreads();                    // and no warp reads a barrier in the ring's way any more
    tc_after();
    uint32_t* part = reinterpret_cast<uint32_t*>(smem + (tiles0 - smem_addr(smem)));
    if (warp >= 4 && done) {
        const int q = warp & 3;
        for (int c = ((warp - 4) >> 2) * 32; c < n; c += 64) {
            uint32_t r[32];
            tmem_read32(tmem + c + ((uint32_t)(q * 32) << 16), r);
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c + j < rows) part[(c + j) * kTileCh + q * 32 + lane] = r[j];
        }
    }
    __syncwarp();
    tc_before();
    cluster_sync();         // all partials are there
    tc_after();
    if (warp == 2) tmem_free<1>(tmem, 256);
    // this CTA's rows: a warp one row, a lane four channels
    const int r0 = rows * rank / S, r1 = rows * (rank + 1) / S, ch = ch0 + 4 * lane;
    float sw[4] = {1.0f, 1.0f, 1.0f, 1.0f}, bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (ch + j < a.N) {
            sw[j] = __ldg(a.sw + ch + j);
            if (a.bias) bias[j] = __ldg(a.bias + ch + j);
        }
    const bool quad = a.ldy % 4 == 0 && ch + 4 <= a.N;
    for (int r = r0 + warp; r < r1; r += kMmaThreads / 32) {
        const uint32_t mine = smem_addr(part) + (r * kTileCh + 4 * lane) * 4;
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = make_uint4(0, 0, 0, 0);
            if (i < S) {
                uint32_t at;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(mine), "r"(i));
                asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                             : "r"(at)
                             : "memory");
            }
        }
        float v[4];
        int t[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t[0] += (int)w[i].x;
            t[1] += (int)w[i].y;
            t[2] += (int)w[i].z;
            t[3] += (int)w[i].w;
        }
        const float sx = __ldg(a.sx + row0 + r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = __fmul_rn(__fmul_rn((float)t[j], sx), sw[j]);
            if (a.bias) v[j] = __fadd_rn(v[j], bias[j]);
        }
        const int64_t at = (int64_t)(row0 + r) * a.ldy + ch;
        if (quad) {
            if (a.y_type == ELQ_F32)
                *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.y) + at) = make_float4(v[0], v[1], v[2], v[3]);
            else
                *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + at) =
                    a.y_type == ELQ_BF16 ? make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]))
                                         : make_uint2(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (ch + j < a.N) store1(a.y, a.y_type, at + j, v[j]);
        }
    }
    cluster_leave(bye, S, a.wait_ns);
}

}  // namespace elqops
