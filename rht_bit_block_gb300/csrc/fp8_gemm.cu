// Matrix product of two E4M3 operands with an fp32 scale for each block of 128
// along the summed index (fp8_quantize.cu), the FPROP, DGRAD and WGRAD of a
// linear layer that keeps 8 bits (UFP4 summary, section 方法: Y^ = Q(X) Q(W)^T):
//
//   D[m, n] = sum over blocks b of  sA[m, b] sB[n, b]  sum over k in b of A[m, k] B[n, k]
//
// An fp32 scale cannot ride in a block-scaled MMA, whose scales are powers of
// two (or E4M3).  So the tensor core sums one block of 128 at a time, in fp32,
// into one of two to four buffers in tensor memory, and while it sums the next
// ones, other warps read the finished block and add it, scaled, to fp32 sums in
// registers.
//
// One operand's rows (P) lie along the lanes of tensor memory, the other's (Q)
// along its columns; three shapes:
//
// Pairs and singles (WIDE): P is A, Q is B.  Pairs are persistent CTA pairs with
// 256 x 256 tiles, tcgen05.mma .cta_group::2, where a CTA holds 128 rows of either
// operand; singles are 128 x 128 tiles of one CTA, for products with too few of
// the large ones.  A block of a pair's tile is 512 cycles of the tensor core.
// With square blocks of B a lane that holds a row needs one scale for 128 columns,
// and the sums are read a row a lane, the layout that tensor memory reads fastest
// (128 x 256 sums of an SM in about 155 cycles; 16 lanes x 128 bits 260, x 256
// bits 510).  With scales for the rows of either operand (WGRAD) every column has
// its own: brought from shared memory to every lane that would be 1024 cycles, so the
// sums are read 16 lanes x 128 bits, which gives a thread four rows and a quarter of
// the columns.
//
// Few tokens (up to 64): P is B, Q is A, so that the tile is as wide as there
// are tokens and the weights are read once.  A lane holds a row of B, and 32
// neighbouring results of a token are one store of a warp.
//
// Singles and few tokens share the summed index out over a cluster of up to eight
// CTAs, which add their sums through distributed shared memory, in the order of
// their ranks: no workspace, no atomics, and the same bits every time.
//
// What bounds it.  Pairs: 16384 x 7168 x 7168 takes 570 us in a burst (2950 TFLOP/s
// of 3777, twice the measured bf16 rate) and 670 under the power cap, 8192 x 5632 x
// 2048 82 us.  A block takes 820 cycles of which its MMAs are 512: with two buffers
// of 256 columns, all of tensor memory, the next block but one cannot start before
// this one is read (155), released, and its commit seen.  Four buffers of half the
// columns cost more hand-offs than they hide (8 % slower), and reads issued ahead of
// the additions change nothing.  With scales for the rows of both operands a block
// takes 1300 cycles, of which the reads are 260 and the scaling's issue slots most of
// the rest: 4096 x 4096 x 8192 167 us (1650 TFLOP/s; 107 us and 2580 with square
// blocks).  Singles: 0.29 us a block, what an SM takes in from L2 (32 KB, about 600
// cycles), for about 4 us of start and join beside (256 x 7168 x 7168 20 us).  Few
// tokens: reading B, at 4.5 TB/s of 6.8 with 1 x 7168 x 7168 (11.5 us) and 5.1 with
// 1 x 32000 x 2048 (12.9 us), about 3 us of it the start, the first copies and the join.
#include <algorithm>
#include <atomic>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_figure.h"
#include "internal.h"
#include "train.h"
#include "ufp4_device.cuh"

namespace ufp4 {

__device__ int g_fp8_error;

namespace {

constexpr int kLanes = 128;                // rows of P that one CTA holds: the lanes of tensor memory
constexpr int kStep = 128;                 // summed elements (and bytes) of a block: one 128-byte swizzle row
constexpr int kAtom = kLanes * kStep;
constexpr int kSlab = 4;                   // blocks whose scales are laid out at a time
constexpr int kSlabs = 2;
constexpr int kPad = 8;                    // floats between a slab's blocks, off the same bank
constexpr int kOthers = 4;                 // warps that do not scale
constexpr int kLoaders = 64;               // threads that lay out scales (warps 2 and 3)
constexpr int kMaxShares = 8;
constexpr int kGroup = 8;                  // tiles of P that advance before the tile of Q does
constexpr uint32_t kWaitLimit = 1u << 22;  // bounded polling; each poll may sleep up to kSuspendNs
constexpr uint32_t kSuspendNs = 1000;
constexpr uint32_t kLook = 1024;           // polls between looks at the abort flag
constexpr uint32_t kDrainLimit = 1u << 16; // polls for copies in flight, after a wait has given up

// CW columns a warp, GROUPS warps of each lane quadrant.
template <bool WIDE, bool PAIR, int CW, int GROUPS>
struct Cfg {
    static constexpr int kCols = CW * GROUPS;                 // columns of a tile
    static constexpr int kRows = PAIR ? 2 * kLanes : kLanes;  // rows of a tile
    static constexpr int kThreads = 32 * kOthers + 128 * GROUPS;
    static constexpr bool kSplit = CW == 128;                 // registers go from the first four warps to the others
    static constexpr int kQRows = PAIR ? kCols / 2 : kCols;   // rows of Q that a CTA holds
    static constexpr int kQ = kQRows * kStep;
    static constexpr int kStage = kAtom + kQ;
    static constexpr int kStages = WIDE || kCols <= 32 ? 5 : 4;
    static constexpr int kColPitch = kCols + kPad, kRowPitch = kLanes + kPad;
    static constexpr int kSlabFloats = kSlab * (kColPitch + kRowPitch);
    static constexpr int kOffScales = kStages * kStage;
    static constexpr int kOffOut = kOffScales + (kSlabs * kSlabFloats * 4 + 15) / 16 * 16;  // 4 KB for each scaling warp
    static constexpr int kOffBars = kOffOut + (WIDE ? 4 * GROUPS * 4096 : 0);
    static constexpr int kBufs = PAIR ? 2 : 4;  // buffers of partial sums
    // full, done; partial sums read; slabs full, empty; drain
    static constexpr int kNumBars = 2 * kStages + kBufs + 2 * kSlabs + 1;
    static constexpr int kOffWords = kOffBars + 8 * kNumBars;  // tensor memory address, abort flag, stages filled and used
    static constexpr int kSmem = kOffWords + 16 + 1024;
    static constexpr int kTmem = kBufs * kCols;
    static_assert(kTmem >= 32 && (kTmem & (kTmem - 1)) == 0 && kTmem <= 512, "tensor memory columns");
    static_assert(kSmem <= 232448, "shared memory overflow");
    // CTAs of an SM take tensor memory while they wait for their cluster's others: all that shared memory lets in must fit.
    static_assert(233472 / (kSmem + 1024) * kTmem <= 512, "CTAs that could wait for each other's tensor memory");
    static_assert(kCols * kLanes * 4 <= kStages * kStage, "a share's sums take the stages' place");
    static_assert(kQRows % 8 == 0 && kQ % 1024 == 0, "swizzle atoms");
    static_assert(!WIDE || CW % 64 == 0, "a wide tile's columns are read 64 at a time");
};

// ------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cbar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cbar) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives once this thread's copies so far have landed.
__device__ __forceinline__ void mbar_arrive_copies(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ int ld_shared(uint32_t saddr) {
    int v;
    asm volatile("ld.volatile.shared.b32 %0, [%1];" : "=r"(v) : "r"(saddr) : "memory");
    return v;
}
__device__ __forceinline__ float ld_shared_f(uint32_t saddr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(saddr));
    return v;
}
// Two pairs of floats, 16-byte aligned.
__device__ __forceinline__ void ld_shared_pairs(uint32_t saddr, uint64_t& a, uint64_t& b) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(saddr));
}
// Bounded wait of a whole warp on an mbarrier phase, the same answer in every
// lane: false at the limit (with the error word set), or once the word at
// `abort` (0: none) is set, which is looked at every kLook polls.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint32_t abort, uint32_t limit = kWaitLimit) {
    uint32_t ok;
    if (limit) {  // most waits find what they wait for: a test is answered in 15 cycles, a wait in 50
        asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(ok)
                     : "r"(bar), "r"(parity)
                     : "memory");
        if (__all_sync(0xFFFFFFFFu, ok)) return true;
    }
#pragma unroll 1
    for (uint32_t i = 0; i < limit; ++i) {
        asm volatile(
            "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(kSuspendNs)
            : "memory");
        if (__all_sync(0xFFFFFFFFu, ok)) return true;
        if ((i + 1) % kLook == 0 && abort && __any_sync(0xFFFFFFFFu, ld_shared(abort))) return false;
    }
    atomicExch(&g_fp8_error, 1);
    return false;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t caddr, int v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(caddr), "r"(v) : "memory");
}
__device__ __forceinline__ int ld_cluster(uint32_t caddr) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(caddr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t caddr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(caddr)
                 : "memory");
    return v;
}
// TMA box into this CTA's shared memory, counted on a barrier of either CTA of a pair.
template <bool PAIR>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t cbar) {
    if (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%2, %3}], [%4];"
            ::"r"(dst), "l"((uint64_t)map), "r"(x), "r"(y), "r"(cbar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
            ::"r"(dst), "l"((uint64_t)map), "r"(x), "r"(y), "r"(cbar)
            : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// K-major, 128-byte swizzle: 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f8f6f4: fp32 accumulator (bits 4..5 = 1), E4M3 operands (formats 0), both K-major, N >> 3, M >> 4.
__host__ __device__ constexpr uint32_t make_idesc(int rows, int cols) {
    return (1u << 4) | ((uint32_t)(cols >> 3) << 17) | ((uint32_t)(rows >> 4) << 24);
}
template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if (PAIR)
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p; }"
            ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }"
            ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}
// Arrives on the barrier once this thread's MMAs so far are done: in both CTAs of a pair ...
template <bool PAIR>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// ... or in this CTA alone.
template <bool PAIR>
__device__ __forceinline__ void tc_commit_local(uint32_t bar) {
    if (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, int cols) {
    if (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t tmem, int cols) {
    if (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
}
// 16 or 32 columns of a warp's 32 lanes, a lane a row ...
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&u)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]),
          "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]),
          "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]),
          "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]),
          "=r"(u[15])
        : "r"(taddr));
}
// ... or 32 columns of 16 lanes: r[2 j] is row lane / 4, r[2 j + 1] row lane / 4 + 8, column 4 j + lane % 4.
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x128b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]),
          "=r"(u[15])
        : "r"(taddr));
}
// One lane of a whole warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(one));
    return one != 0;
}
// Waits for all of this warp's reads; `r` are what one of them brings (they are
// not to be used before).
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}

// ------------------------------------------------------------------- kernel
struct Fp8Params {
    int p_rows, q_rows;        // extents of the operands
    int blocks;                // of the summed index
    int p_tiles, q_tiles;
    int group;                 // tile order: tiles of P that advance first
    int shares, per;           // CTAs of a cluster and blocks of each (one for pairs)
    int q_box;                 // rows of Q that a copy brings: up to a CTA's
    uint32_t wait_limit;       // polls of a stage's arrival; all other waits keep kWaitLimit
    const float* sp;
    const float* sq;
    int64_t ld_sp, ld_sq;
    int p_shift, q_shift;      // log2 of the rows that share a scale: 0 or 7
    void* d;
    int64_t ldd;
    int d_f32, accumulate;
    int d_vec;                 // bytes that neighbouring results can be stored by: 16 or their own
};

__device__ __forceinline__ void tile_at(const Fp8Params& p, int tile, int& pt, int& qt) {
    const int group = min(p.group, p.p_tiles);
    const int span = group * p.q_tiles, g = tile / span, first = g * group;
    const int rows = min(group, p.p_tiles - first), l = tile - g * span;
    qt = l / rows;
    pt = first + (l - qt * rows);
}

__device__ __forceinline__ void put(const Fp8Params& p, int64_t at, float v) {
    if (p.d_f32) {
        float* d = (float*)p.d + at;
        *d = p.accumulate ? *d + v : v;
    } else {
        ((__nv_bfloat16*)p.d)[at] = __float2bfloat16_rn(v);
    }
}
// Four neighbouring results, of which `live` exist.
__device__ __forceinline__ void put4(const Fp8Params& p, int64_t at, float4 v, int live) {
    if (live >= 4 && p.d_vec == 16) {
        if (p.d_f32) {
            float4* d = reinterpret_cast<float4*>((float*)p.d + at);
            if (p.accumulate) {
                const float4 o = *d;
                v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
            }
            *d = v;
        } else {
            const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
            *reinterpret_cast<uint2*>((__nv_bfloat16*)p.d + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        }
        return;
    }
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < live) put(p, at + i, f[i]);
}
__device__ __forceinline__ float column(const uint64_t* acc, int c) {
    float x, y;
    up2(acc[c >> 1], x, y);
    return c & 1 ? y : x;
}
__device__ __forceinline__ uint32_t pack_bf16(uint64_t v) {
    float lo, hi;
    up2(v, lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The sums of a wide tile's warp: 32 rows by CW columns.  Where 128 rows of B share a scale a lane holds a row, acc[c / 2] two
// of its columns; with scales for either's rows (BOTH) acc[h * CW / 4 + j] holds rows 16 h + lane / 4 and that + 8 of column 4 j
// + lane % 4.
//
// Their stores from the registers would touch 32 rows, or 16 bytes, at a time; instead 128 bytes of every row are turned around in
// `stage` (16-byte units, unit u of row i at u ^ (i & 7)) and stored four whole rows of them an instruction, or, where D's rows
// are not aligned or the tile is cut short, 32 neighbouring elements (4096 x 4095 x 2048: 40 us, 35 where aligned; from the
// registers 165).
template <bool BOTH, int CW>
__device__ __forceinline__ void store_wide(const Fp8Params& p, const uint64_t (&acc)[CW / 2], int row0, int col0,
                                           uint8_t* stage) {
    const int lane = threadIdx.x & 31, q = lane & 3;
    const bool vec = col0 + CW <= p.q_rows && p.d_vec == 16;
    uint4* mine = reinterpret_cast<uint4*>(stage + lane * 128);
    auto flush = [&](int c, auto element) {  // the stage holds columns col0 + c on
        using T = decltype(element);
        constexpr int kBytes = sizeof(T);
        __syncwarp();
        if (vec) {
            char* base = (char*)p.d + ((int64_t)(row0 + (lane >> 3)) * p.ldd + col0 + c) * kBytes + (lane & 7) * 16;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = i * 4 + (lane >> 3);
                uint4 v = reinterpret_cast<const uint4*>(stage + row * 128)[(lane & 7) ^ (row & 7)];
                if (row0 + row < p.p_rows) {
                    uint4* d = reinterpret_cast<uint4*>(base + (int64_t)i * 4 * p.ldd * kBytes);
                    if (p.accumulate) {
                        const uint4 o = *d;
                        v = make_uint4(__float_as_uint(__uint_as_float(o.x) + __uint_as_float(v.x)),
                                       __float_as_uint(__uint_as_float(o.y) + __uint_as_float(v.y)),
                                       __float_as_uint(__uint_as_float(o.z) + __uint_as_float(v.z)),
                                       __float_as_uint(__uint_as_float(o.w) + __uint_as_float(v.w)));
                    }
                    *d = v;
                }
            }
        } else {
            const int rows = min(32, p.p_rows - row0);
#pragma unroll
            for (int e = lane; e < 128 / kBytes; e += 32) {
                if (col0 + c + e >= p.q_rows) break;
                T* d = (T*)p.d + (int64_t)row0 * p.ldd + col0 + c + e;
                const uint8_t* from = stage + e % (16 / kBytes) * kBytes;
                const int unit = e / (16 / kBytes);
#pragma unroll 4
                for (int row = 0; row < rows; ++row) {
                    T v = *reinterpret_cast<const T*>(from + row * 128 + ((unit ^ (row & 7)) << 4));
                    if constexpr (kBytes == 4)
                        if (p.accumulate) v += *d;
                    *d = v;
                    d += p.ldd;
                }
            }
        }
        __syncwarp();
    };
    // BOTH: the pair of rows of column 4 j + q, the j-th four of the 128 bytes (all rows are lane / 4 modulo 8)
    auto put_pair = [&](int h, int j, int bytes, uint64_t v) {
        float x, y;
        up2(v, x, y);
        uint8_t* at = stage + (16 * h + (lane >> 2)) * 128 + (((j * bytes) >> 2) ^ (lane >> 2)) * 16;
        if (bytes == 4) {
            reinterpret_cast<float*>(at)[q] = x;
            reinterpret_cast<float*>(at + 8 * 128)[q] = y;
        } else {
            reinterpret_cast<__nv_bfloat16*>(at)[4 * (j & 1) + q] = __float2bfloat16_rn(x);
            reinterpret_cast<__nv_bfloat16*>(at + 8 * 128)[4 * (j & 1) + q] = __float2bfloat16_rn(y);
        }
    };
    if (p.d_f32) {
#pragma unroll
        for (int c = 0; c < CW; c += 32) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (BOTH) {
                    put_pair(0, u, 4, acc[c / 4 + u]);
                    put_pair(1, u, 4, acc[CW / 4 + c / 4 + u]);
                } else {
                    const uint64_t x = acc[c / 2 + 2 * u], y = acc[c / 2 + 2 * u + 1];
                    mine[u ^ (lane & 7)] = make_uint4((uint32_t)x, (uint32_t)(x >> 32), (uint32_t)y, (uint32_t)(y >> 32));
                }
            }
            flush(c, 0.0f);
        }
    } else {
#pragma unroll
        for (int c = 0; c < CW; c += 64) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (BOTH) {
#pragma unroll
                    for (int j = 2 * u; j < 2 * u + 2; ++j) {
                        put_pair(0, j, 2, acc[c / 4 + j]);
                        put_pair(1, j, 2, acc[CW / 4 + c / 4 + j]);
                    }
                } else {
                    const uint64_t* a = acc + c / 2 + 4 * u;
                    mine[u ^ (lane & 7)] = make_uint4(pack_bf16(a[0]), pack_bf16(a[1]), pack_bf16(a[2]), pack_bf16(a[3]));
                }
            }
            flush(c, __nv_bfloat16());
        }
    }
}

// Warp 0 copies the operands, warp 1 of the leader issues the MMAs, warps 2
// and 3 lay out the scales, the rest scale and add.  BOTH: the rows of either
// operand have scales of their own; otherwise 128 rows of B share one.
template <bool WIDE, bool PAIR, bool BOTH, int CW, int GROUPS>
__global__ void __launch_bounds__((Cfg<WIDE, PAIR, CW, GROUPS>::kThreads), WIDE ? 1 : 2)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                const __grid_constant__ Fp8Params p) {
    using C = Cfg<WIDE, PAIR, CW, GROUPS>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t bars = base + C::kOffBars;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto done_bar = [&](int s) { return bars + 8u * (S + s); };
    auto read_bar = [&](int b) { return bars + 8u * (2 * S + b); };
    auto slabf_bar = [&](int i) { return bars + 8u * (2 * S + C::kBufs + i); };
    auto slabe_bar = [&](int i) { return slabf_bar(kSlabs + i); };
    const uint32_t drain_bar = slabf_bar(2 * kSlabs);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffWords);
    const uint32_t abort_flag = base + C::kOffWords + 4;
    volatile int* stages_of = reinterpret_cast<volatile int*>(gbase + C::kOffWords + 8);  // filled, used

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int peer = PAIR ? (int)rank : 0;  // 0: the CTA that issues the MMAs
    const int cluster_id = PAIR ? blockIdx.x >> 1 : blockIdx.x / p.shares;
    const int num_clusters = PAIR ? gridDim.x >> 1 : gridDim.x / p.shares;
    const int num_tiles = p.p_tiles * p.q_tiles;
    // this CTA's share of the summed index
    const int k0 = PAIR ? 0 : (int)rank * p.per;
    const int k_blocks = PAIR ? p.blocks : max(0, min(p.per, p.blocks - k0));
    // Where each cluster has one tile they all walk the blocks at the same pace, and the tiles of a few tokens are what many
    // of them read: each starts at a block of its own and comes round, or the few lines of the block they share keep them
    // waiting (256 x 7168 x 7168 on single tiles: 46 us).
    const int turn = num_tiles <= num_clusters ? (int)((int64_t)cluster_id * k_blocks / num_tiles) : 0;
    auto block_at = [&](int i) { return k0 + i + turn - (i + turn >= k_blocks ? k_blocks : 0); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);  // the leader's expect_tx arrival (both CTAs' bytes)
            mbar_init(done_bar(s), 1);  // the leader's commit: the stage may be filled, its sums be read
        }
        for (int b = 0; b < C::kBufs; ++b) mbar_init(read_bar(b), (PAIR ? 2 : 1) * 4 * GROUPS);  // every scaling warp
        for (int i = 0; i < kSlabs; ++i) {
            mbar_init(slabf_bar(i), kLoaders);
            mbar_init(slabe_bar(i), 4 * GROUPS);
        }
        mbar_init(drain_bar, 1);
        *reinterpret_cast<volatile int*>(gbase + C::kOffWords + 4) = 0;
        stages_of[0] = stages_of[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<PAIR>(smem_u32(tmem_slot), C::kTmem);
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();  // both CTAs' barriers exist before any copy or commit targets them
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    griddep_launch();

    // Sets the abort flag of this CTA, and of its pair.
    auto give_up = [&] {
        *reinterpret_cast<volatile int*>(gbase + C::kOffWords + 4) = 1;
        if (PAIR) st_cluster(map_to_rank(abort_flag, rank ^ 1u), 1);
    };

    // With kSplit, what the threads of the first four warps give up of the launch's 168 registers, twice as many others
    // take: 128 x 72 + 256 x 216 = 384 x 168.
    if (warp < kOthers) {
        if (C::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        // The copier and the issuer are whole warps, of which one lane acts: what a lane alone computes has to be moved to
        // the uniform registers of its copies and MMAs each time (a step of the issuer took 1000 cycles).
        if (warp == 0) {
            // ---------------------------------------------------- copies
            const bool acts = elect_one();
            const uint32_t tx = PAIR ? 2 * C::kStage : kAtom + (uint32_t)p.q_box * kStep;
            const uint32_t remote = PAIR ? map_to_rank(bars, 0) : bars;
            int s = 0, stages = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int tile = cluster_id; tile < num_tiles && ok; tile += num_clusters) {
                int pt, qt;
                tile_at(p, tile, pt, qt);
                const int prow = pt * C::kRows + peer * kLanes, qrow = qt * C::kCols + peer * C::kQRows;
                for (int kb = 0; kb < k_blocks; ++kb) {
                    ok = mbar_wait(done_bar(s), ph ^ 1u, abort_flag);
                    if (!ok) break;
                    ++stages;
                    if (acts) {
                        if (peer == 0) mbar_expect_tx(full_bar(s), tx);
                        const uint32_t dst = base + s * C::kStage;
                        tma_load<PAIR>(dst, &map_p, block_at(kb) * kStep, prow, remote + 8u * s);
                        tma_load<PAIR>(dst + kAtom, &map_q, block_at(kb) * kStep, qrow, remote + 8u * s);
                    }
                    __syncwarp();
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) give_up();
            if (lane == 0) stages_of[0] = stages;
        } else if (warp == 1 && peer == 0) {
            // ------------------------------------------------ MMA issuer (leader only)
            const bool acts = elect_one();
            constexpr uint32_t idesc = make_idesc(C::kRows, C::kCols);
            int s = 0, stages = 0;
            uint32_t ph = 0, t = 0;  // t: blocks so far, buffer t % kBufs
            bool ok = true;
            for (int tile = cluster_id; tile < num_tiles && ok; tile += num_clusters) {
                for (int kb = 0; kb < k_blocks; ++kb) {
                    ok = mbar_wait(full_bar(s), ph, 0, p.wait_limit) && mbar_wait(read_bar(t % C::kBufs), (t / C::kBufs & 1) ^ 1u, abort_flag);
                    if (!ok) break;
                    ++stages;
                    tc_fence_after();
                    if (acts) {
                        const uint64_t dp = sw128_desc(base + s * C::kStage), dq = sw128_desc(base + s * C::kStage + kAtom);
#pragma unroll
                        for (int i = 0; i < 4; ++i)  // 32 bytes of the summed index each
                            mma<PAIR>(tmem + t % C::kBufs * C::kCols, dp + 2 * i, dq + 2 * i, idesc, i > 0 ? 1u : 0u);
                        tc_commit<PAIR>(done_bar(s));
                    }
                    ++t;
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) give_up();
            if (lane == 0) stages_of[1] = stages;
            __syncwarp();
            if (acts) tc_commit_local<PAIR>(drain_bar);
            mbar_wait(drain_bar, 0, 0);
        } else if (warp >= 2) {
            // ---------------------------------------------------- scales
            // A slab is the scales of up to kSlab blocks: those of the tile's columns and of the CTA's rows, each block's apart.
            // A thread takes one block, and every 16th column or row.  What lies past the operands is read at their edge
            // instead; nothing looks at it.  Few of them are loaded before the slab is free; where every row and every column
            // has its own, which is more than a thread's registers hold, they are copied straight into it.
            const int tid = threadIdx.x - 64;
            const int kk = tid & (kSlab - 1), each = tid >> 2;
            constexpr bool kOfCols = !WIDE || BOTH;  // every column its scale; otherwise one for each 128
            constexpr bool kOfRows = WIDE || BOTH;   // every row its scale; otherwise one, which is multiplied into the columns'
            constexpr bool kCopied = WIDE && BOTH;
            constexpr int kC = kOfCols ? C::kCols / 16 : 1, kR = kOfRows ? kLanes / 16 : 1;
            uint32_t u = 0;
            bool ok = true;
            for (int tile = cluster_id; tile < num_tiles && ok; tile += num_clusters) {
                int pt, qt;
                tile_at(p, tile, pt, qt);
                const int p0 = pt * C::kRows + peer * kLanes, q0 = qt * C::kCols;
                for (int kb = 0; kb < k_blocks; kb += kSlab, ++u) {
                    const int64_t b = block_at(min(kb + kk, k_blocks - 1));
                    const float* sp = p.sp + b;
                    const float* sq = p.sq + b;
                    auto of_p = [&](int j) {
                        return sp + (int64_t)(min(p0 + (kOfRows ? each + 16 * j : 0), p.p_rows - 1) >> p.p_shift) * p.ld_sp;
                    };
                    auto of_q = [&](int j) {
                        const int r = kOfCols ? each + 16 * j : min(each * 128, C::kCols - 1);
                        return sq + (int64_t)(min(q0 + r, p.q_rows - 1) >> p.q_shift) * p.ld_sq;
                    };
                    float v[kC], w[kR];
                    if (!kCopied) {
#pragma unroll
                        for (int j = 0; j < kC; ++j) v[j] = *of_q(j);
#pragma unroll
                        for (int j = 0; j < kR; ++j) w[j] = *of_p(j);
                    }
                    ok = mbar_wait(slabe_bar(u % kSlabs), (u / kSlabs & 1) ^ 1u, abort_flag);
                    if (!ok) break;
                    float* cols = reinterpret_cast<float*>(gbase + C::kOffScales) + (u % kSlabs) * C::kSlabFloats +
                                  kk * C::kColPitch + each;
                    float* rows = cols + (kSlab - kk) * C::kColPitch + kk * C::kRowPitch;
                    if (kCopied) {
#pragma unroll 2
                        for (int j = 0; j < kC; ++j) copy4(smem_u32(cols) + 64 * j, of_q(j));
#pragma unroll 2
                        for (int j = 0; j < kR; ++j) copy4(smem_u32(rows) + 64 * j, of_p(j));
                        mbar_arrive_copies(slabf_bar(u % kSlabs));
                    } else {
#pragma unroll
                        for (int j = 0; j < kC; ++j) cols[16 * j] = kOfRows ? v[j] : v[j] * w[0];
                        if (kOfRows) {
#pragma unroll
                            for (int j = 0; j < kR; ++j) rows[16 * j] = w[j];
                        }
                        mbar_arrive(slabf_bar(u % kSlabs));
                    }
                }
            }
            if (!ok) give_up();
            if (kCopied) asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        // ------------------------------------------------- scaling and adding
        if (C::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int quad = warp & 3, first = ((warp - kOthers) >> 2) * CW;  // a warp reads the quarter of the lanes that is its own
        const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + first;
        const uint32_t slabs = base + C::kOffScales;
        const uint32_t read = PAIR ? map_to_rank(read_bar(0), 0) : read_bar(0);  // the issuer's
        const uint32_t own_row = (kSlab * C::kColPitch + quad * 32 + (WIDE && BOTH ? lane >> 2 : lane)) * 4;
        uint32_t t = 0, u = 0;  // blocks and slabs so far: buffer t % kBufs, slab u % kSlabs
        int s = 0;              // stage of block t
        uint32_t ph = 0;
        bool ok = true;
        uint64_t acc[CW / 2];     // pairs of columns; WIDE: see store_wide
        for (int tile = cluster_id; tile < num_tiles; tile += num_clusters) {
#pragma unroll
            for (int c = 0; c < CW / 2; ++c) acc[c] = 0;
#pragma unroll 1
            for (int kb = 0; kb < k_blocks; ++kb) {
                const int kk = kb & (kSlab - 1);
                if (kk == 0) ok = mbar_wait(slabf_bar(u % kSlabs), u / kSlabs & 1, abort_flag);
                ok = ok && mbar_wait(done_bar(s), ph, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint32_t slab = slabs + (u % kSlabs) * (C::kSlabFloats * 4);
                const uint32_t cols = slab + (kk * C::kColPitch + first) * 4;
                const uint32_t at = from + t % C::kBufs * C::kCols;
                auto release = [&] {  // the buffer has been read and may be filled again
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR) mbar_arrive_cluster(read + 8u * (t % C::kBufs));
                        else mbar_arrive(read + 8u * (t % C::kBufs));
                    }
                };
                const uint32_t rows = slab + own_row + kk * C::kRowPitch * 4;
                if constexpr (WIDE && !BOTH) {
                    const float v = ld_shared_f(rows) * ld_shared_f(slab + (kk * C::kColPitch + (first >> 7)) * 4);
                    const uint64_t s2 = pk2(v, v);
#pragma unroll
                    for (int c = 0; c < CW; c += 32) {
                        uint32_t r[32];
                        tmem_ld(at + c, r);
                        tmem_wait(r);
                        if (c + 32 == CW) release();
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[c / 2 + j] = fma2(pair(r[2 * j], r[2 * j + 1]), s2, acc[c / 2 + j]);
                    }
                } else if constexpr (WIDE) {
                    uint64_t rs[2];  // the scales of the lane's pairs of rows
#pragma unroll
                    for (int h = 0; h < 2; ++h) rs[h] = pk2(ld_shared_f(rows + 64 * h), ld_shared_f(rows + 64 * h + 32));
#pragma unroll
                    for (int c = 0; c < CW; c += 32) {
                        float wv[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) wv[j] = ld_shared_f(cols + (c + 4 * j + (lane & 3)) * 4);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t r[16];
                            tmem_ld_rows(at + c + ((uint32_t)h << 20), r);
                            tmem_wait(r);
                            if (c + 32 == CW && h == 1) release();
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                uint64_t& a = acc[h * (CW / 4) + c / 4 + j];
                                a = fma2(mul2(pair(r[2 * j], r[2 * j + 1]), pk2(wv[j], wv[j])), rs[h], a);
                            }
                        }
                    }
                } else {
                    const float v = BOTH ? ld_shared_f(rows) : 1.0f;
                    const uint64_t s2 = pk2(v, v);
                    constexpr int kChunk = CW < 32 ? CW : 32;
#pragma unroll
                    for (int c = 0; c < CW; c += kChunk) {
                        uint32_t r[kChunk];
                        tmem_ld(at + c, r);
                        tmem_wait(r);
                        if (c + kChunk == CW) release();
#pragma unroll
                        for (int j = 0; j < kChunk; j += 4) {
                            uint64_t wx, wy;
                            ld_shared_pairs(cols + (c + j) * 4, wx, wy);
                            const uint64_t x = pair(r[j], r[j + 1]), y = pair(r[j + 2], r[j + 3]);
                            uint64_t &ax = acc[(c + j) / 2], &ay = acc[(c + j) / 2 + 1];
                            ax = BOTH ? fma2(mul2(x, wx), s2, ax) : fma2(x, wx, ax);
                            ay = BOTH ? fma2(mul2(y, wy), s2, ay) : fma2(y, wy, ay);
                        }
                    }
                }
                ++t;
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
                if (kk == kSlab - 1 || kb + 1 == k_blocks) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(slabe_bar(u % kSlabs));
                    ++u;
                }
            }
            if (!ok) {
                give_up();
                break;
            }
            if (!PAIR && p.shares > 1) {
                // every copy and MMA of this CTA is done: the sums take the stages' place, neighbouring results side by side
                float* sums = reinterpret_cast<float*>(gbase);
                if constexpr (WIDE && !BOTH) {
                    // 16-byte units of a row, unit u of row i at u ^ (i & 7): a warp's stores meet no bank twice
#pragma unroll
                    for (int c = 0; c < CW; c += 4)
                        *reinterpret_cast<ulonglong2*>(sums + (quad * 32 + lane) * C::kCols + (((first + c) >> 2) ^ (lane & 7)) * 4) =
                            make_ulonglong2(acc[c / 2], acc[c / 2 + 1]);
                } else if constexpr (WIDE) {
#pragma unroll
                    for (int i = 0; i < CW; ++i) {
                        const int row = quad * 32 + 16 * (i / (CW / 2)) + 8 * (i & 1) + (lane >> 2);
                        const int col = first + 4 * (i % (CW / 2) / 2) + (lane & 3);
                        sums[row * C::kCols + (col ^ (row & 7) << 2)] = column(acc, i);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < CW; ++c) sums[(first + c) * kLanes + quad * 32 + lane] = column(acc, c);
                }
                break;  // one tile a cluster
            }
            int pt, qt;
            tile_at(p, tile, pt, qt);
            const int p0 = pt * C::kRows + peer * kLanes + quad * 32, q0 = qt * C::kCols + first;
            if constexpr (WIDE) {
                store_wide<BOTH, CW>(p, acc, p0, q0, gbase + C::kOffOut + (warp - kOthers) * 4096);
            } else {
                const int live = p0 + lane < p.p_rows ? p.q_rows - q0 : 0;
                const int64_t at = (int64_t)q0 * p.ldd + p0 + lane;
#pragma unroll
                for (int c = 0; c < CW; ++c)
                    if (c < live) put(p, at + c * p.ldd, column(acc, c));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();  // neither CTA leaves while the other may still use its memory or barriers
    if (!PAIR && p.shares > 1) {
        cluster_sync_all();  // all shares' sums are there
        int pt, qt;
        tile_at(p, cluster_id, pt, qt);
        // each CTA adds its share of D's rows over the ranks, in their order
        constexpr int kDRows = WIDE ? kLanes : C::kCols, kDCols = WIDE ? C::kCols : kLanes;
        const int m0 = WIDE ? pt * kLanes : qt * C::kCols, n0 = WIDE ? qt * C::kCols : pt * kLanes;
        const int M = WIDE ? p.p_rows : p.q_rows, N = WIDE ? p.q_rows : p.p_rows;
        const int rows = min(kDRows, M - m0), share = (rows + p.shares - 1) / p.shares;
        const int begin = (int)rank * share, end = min(rows, begin + share);
        constexpr int kUnits = kDCols / 4;  // of four neighbouring results
        for (int i = begin * kUnits + (int)threadIdx.x; i < end * kUnits; i += C::kThreads) {
            const int row = i / kUnits, unit = i % kUnits;
            const uint32_t at = base + 16u * (row * kUnits + (WIDE ? unit ^ (row & 7) : unit));
            float4 v[kMaxShares];
#pragma unroll
            for (int r = 0; r < kMaxShares; ++r)
                if (r < p.shares) v[r] = ld_cluster4(map_to_rank(at, r));
            float4 sum = v[0];
#pragma unroll
            for (int r = 1; r < kMaxShares; ++r)
                if (r < p.shares) sum = make_float4(sum.x + v[r].x, sum.y + v[r].y, sum.z + v[r].z, sum.w + v[r].w);
            put4(p, (int64_t)(m0 + row) * p.ldd + n0 + 4 * unit, sum, N - (n0 + 4 * unit));
        }
        cluster_sync_all();  // no CTA leaves while another reads its sums
    }
    if (__builtin_expect(ld_shared(abort_flag), 0)) {
        // A wait gave up (both CTAs of a pair know): stages that were filled but not used may still be on their way into
        // either CTA.  They are waited for before any CTA leaves, with a limit, since a stage that only one of the
        // copiers filled never completes.
        if (warp == 0 && peer == 0) {
            int most = stages_of[0];
            if (PAIR) most = max(most, ld_cluster(map_to_rank(base + C::kOffWords + 8, 1)));
            for (int i = stages_of[1]; i < most; ++i) mbar_wait(full_bar(i % S), (i / S) & 1, 0, kDrainLimit);
        }
        __syncthreads();
        if (PAIR) cluster_sync_all();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_free<PAIR>(tmem, C::kTmem);
    }
}

// --------------------------------------------------------------------- host
// By how much the polls of a stage's arrival are lowered, per device.
std::atomic<uint32_t> g_lowered[64];

// Clusters of `ctas` CTAs (up to kMaxShares) that fit the device at once.
template <bool WIDE, bool PAIR, bool BOTH, int CW, int GROUPS>
int max_clusters(int dev, int ctas) {
    using C = Cfg<WIDE, PAIR, CW, GROUPS>;
    static DeviceFigure clusters[kMaxShares];
    return clusters[ctas - 1].get(dev, [&] {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)ctas);
        cfg.blockDim = dim3(C::kThreads);
        cfg.dynamicSmemBytes = C::kSmem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)ctas;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        return cudaOccupancyMaxActiveClusters(&n, fp8_gemm_kernel<WIDE, PAIR, BOTH, CW, GROUPS>, &cfg) == cudaSuccess ? n : 0;
    });
}

// Shares of the summed index, for tiles of which each cluster computes one: the fewest blocks in a row, with kRound blocks' time
// for a round of tiles (its start, its first copies and its join).  (768 x 7168 x 7168 on singles: 73 us with 10, 58 with 20.)
// Two CTAs of the kernels for few tokens run on an SM, though the occupancy query counts one (K = 128: 304 tiles 3.4 us, 312
// tiles 5.2); where they do, a block of each takes half as long again.  (37 x 7168 x 7168: 2 shares 15.6 us, 4 or 5 shares
// 14.1; 1 x 7168 x 7168: 12.5 and 11.7; 37 x 16384 x 4096: 1 share 17.2, 2 shares 16.3; 37 x 2816 x 2048: 6 shares on 132 SMs
// 5.6, 8 shares on two CTAs an SM 6.3.)
constexpr int kRound = 20;
struct Shared {
    int shares;
    int64_t rounds, per;  // of tiles, and blocks of each
};
template <bool BOTH, bool WIDE, int CW, int GROUPS>
Shared best_shares(int dev, int64_t tiles, int64_t blocks) {
    Shared b = {1, tiles, blocks};
    int64_t least = 1ll << 60;
    for (int s = 1; s <= kMaxShares && s <= blocks; ++s) {
        const int64_t one = max_clusters<WIDE, false, BOTH, CW, GROUPS>(dev, s), room = WIDE ? one : 2 * one;
        if (room <= 0) continue;
        const int64_t rounds = (tiles + room - 1) / room, per = (blocks + s - 1) / s;
        const int64_t cost = rounds * (2 * (per + kRound) + (!WIDE && tiles > one ? per : 0));
        if (cost < least) {
            least = cost;
            b = {s, rounds, per};
        }
    }
    return b;
}

template <bool WIDE, bool PAIR, bool BOTH, int CW, int GROUPS>
cudaError_t run(const Fp8GemmArgs& a, int dev, cudaStream_t st) {
    using C = Cfg<WIDE, PAIR, CW, GROUPS>;
    const Fp8Operand &op = WIDE ? a.a : a.b, &oq = WIDE ? a.b : a.a;
    const int64_t p_rows = WIDE ? a.M : a.N, q_rows = WIDE ? a.N : a.M;
    Fp8Params p = {};
    p.p_rows = (int)p_rows;
    p.q_rows = (int)q_rows;
    p.blocks = (int)((a.K + kStep - 1) / kStep);
    p.p_tiles = (int)((p_rows + C::kRows - 1) / C::kRows);
    p.q_tiles = (int)((q_rows + C::kCols - 1) / C::kCols);
    p.group = kGroup;
    const int64_t tiles = (int64_t)p.p_tiles * p.q_tiles;
    int shares = 1;
    if constexpr (!PAIR) shares = best_shares<BOTH, WIDE, CW, GROUPS>(dev, tiles, p.blocks).shares;
    p.shares = shares;
    p.per = (p.blocks + p.shares - 1) / p.shares;
    p.q_box = WIDE ? C::kQRows : (int)std::min<int64_t>(C::kQRows, (q_rows + 7) / 8 * 8);
    p.wait_limit = kWaitLimit - g_lowered[dev].load(std::memory_order_relaxed);
    p.sp = op.scales;
    p.sq = oq.scales;
    p.ld_sp = op.scales_ld;
    p.ld_sq = oq.scales_ld;
    p.p_shift = (WIDE ? a.a_square : a.b_square) ? 7 : 0;
    p.q_shift = (WIDE ? a.b_square : a.a_square) ? 7 : 0;
    p.d = a.d;
    p.ldd = a.ldd;
    p.d_f32 = a.d_f32;
    p.accumulate = a.accumulate;
    p.d_vec = (uintptr_t)a.d % 16 == 0 && a.ldd % (a.d_f32 ? 4 : 8) == 0 ? 16 : 1;
    CUtensorMap mp, mq;
    if (!encode_map_2d(&mp, CU_TENSOR_MAP_DATA_TYPE_UINT8, op.codes, (uint64_t)a.K, (uint64_t)p_rows, (uint64_t)op.codes_ld,
                       kStep, kLanes, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_map_2d(&mq, CU_TENSOR_MAP_DATA_TYPE_UINT8, oq.codes, (uint64_t)a.K, (uint64_t)q_rows, (uint64_t)oq.codes_ld,
                       kStep, (uint32_t)p.q_box, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    auto k = fp8_gemm_kernel<WIDE, PAIR, BOTH, CW, GROUPS>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PAIR ? 2 : shares;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    if (PAIR) {
        const int most = max_clusters<WIDE, PAIR, BOTH, CW, GROUPS>(dev, 2);
        if (most <= 0) return cudaErrorLaunchOutOfResources;
        cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(tiles, most));
    } else {
        cfg.gridDim = dim3((unsigned)(tiles * shares));
    }
    cfg.numAttrs = st ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, mp, mq, p);
}

template <bool BOTH>
cudaError_t launch(const Fp8GemmArgs& a, cudaStream_t st) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (a.M <= 16) return run<false, false, BOTH, 16, 1>(a, dev, st);
    if (a.M <= 32) return run<false, false, BOTH, 32, 1>(a, dev, st);
    if (a.M <= 64) return run<false, false, BOTH, 64, 1>(a, dev, st);
    // Measured, us, singles and pairs: 256 x 7168 x 7168 20.3 and 25.8; 512 x 7168 x 7168 45.7 and 27.3; 768 x 2816 x 2048 8.8 and
    // 11.2; 1024 x 2816 x 2048 16.4 and 11.7; 2048 x 1024 x 2048 8.8 and 11.1; 640 x 5632 x 2048 16.6 and 12.2.  With scales for the
    // rows of both operands: 256 x 7168 x 7168 26.3 and 39.1; 512 54.0 and 40.0; 1408 x 1408 x 4096 16.8 and 24.3; 1000 x 7168 x
    // 512 16.1 and 12.1.  In units of a single tile's block: a block of a pair's tile is kPairBlock tenths (square blocks of B, scales
    // for the rows of both), and the pairs, which walk their tiles without a pause, start once, kPairStart of their blocks; singles
    // start with every round, kSingleStart.  All ten of these cases go to the faster side.  (With kRound in place of kSingleStart
    // 768 x 2816 x 2048 and 2048 x 1024 x 2048 would not: kRound is what a further round costs beside shares, their join included.)
    constexpr int kPairBlock = BOTH ? 17 : 14, kPairStart = 6, kSingleStart = 10;
    const int64_t blocks = (a.K + kStep - 1) / kStep;
    const int64_t pairs = std::max(1, max_clusters<true, true, BOTH, 128, 2>(dev, 2));
    const int64_t tiles = (a.M + 255) / 256 * ((a.N + 255) / 256), rounds = (tiles + pairs - 1) / pairs;
    const Shared s = best_shares<BOTH, true, 64, 2>(dev, (a.M + kLanes - 1) / kLanes * ((a.N + kLanes - 1) / kLanes), blocks);
    if ((rounds * blocks + kPairStart) * kPairBlock <= s.rounds * (s.per + kSingleStart) * 10) return run<true, true, BOTH, 128, 2>(a, dev, st);
    return run<true, false, BOTH, 64, 2>(a, dev, st);
}

template <bool WIDE, bool PAIR, bool BOTH, int CW, int GROUPS>
cudaError_t preload() {
    return cudaFuncSetAttribute(fp8_gemm_kernel<WIDE, PAIR, BOTH, CW, GROUPS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg<WIDE, PAIR, CW, GROUPS>::kSmem);
}
template <bool BOTH>
cudaError_t preload_all() {
    cudaError_t e = preload<true, true, BOTH, 128, 2>();
    if (e == cudaSuccess) e = preload<true, false, BOTH, 64, 2>();
    if (e == cudaSuccess) e = preload<false, false, BOTH, 16, 1>();
    if (e == cudaSuccess) e = preload<false, false, BOTH, 32, 1>();
    return e == cudaSuccess ? preload<false, false, BOTH, 64, 1>() : e;
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, cudaStream_t st) {
    return a.b_square ? launch<false>(a, st) : launch<true>(a, st);
}

cudaError_t fp8_error_read_clear(int* value) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_fp8_error, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && *value) e = cudaMemcpyToSymbol(g_fp8_error, &zero, sizeof(int));
    return e;
}

cudaError_t set_fp8_wait_limit(uint32_t polls) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    g_lowered[dev].store(kWaitLimit - std::min(polls, kWaitLimit), std::memory_order_relaxed);
    return cudaSuccess;
}

cudaError_t preload_fp8_gemm_kernels() {
    const cudaError_t e = preload_all<false>();
    return e == cudaSuccess ? preload_all<true>() : e;
}

}  // namespace ufp4
