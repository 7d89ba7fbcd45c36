// Matrix product of two E4M3 operands with an fp32 scale for each block of 128
// along the summed index (fp8_quantize.cu), the FPROP, DGRAD and WGRAD of a
// linear layer that keeps 8 bits (UFP4 summary, section 方法: Y^ = Q(X) Q(W)^T):
//
//   D[m, n] = sum over blocks b of  sA[m, b] sB[n, b]  sum over k in b of A[m, k] B[n, k]
//
// An fp32 scale cannot ride in a block-scaled MMA, whose scales are powers of
// two (or E4M3).  So the tensor core sums one block of 128 at a time, in fp32,
// into one of two buffers in tensor memory, and while it sums the next one into
// the other, sixteen warps read the finished block and add it, scaled, to fp32
// sums in registers.  That costs a multiply-add for each element and block, and
// a second multiplication where both operands have a scale a row (WGRAD): on a
// 256 x 256 tile of a CTA pair a block is 512 cycles of the tensor core and 256
// of an SM's fp32 lanes (512 with both).
//
// Orientation.  The rows of B (a layer's outputs) lie along the lanes of tensor
// memory, the rows of A (tokens) along its columns, so the tile is D^T: a warp
// that writes a token's results writes 32 neighbouring ones, and what a token
// count gives, from 1 to thousands, is the width of the tile.  A square block of
// B has one scale for all 128 lanes of a tile's row block: it is multiplied into the
// tokens' scales as they are laid out in shared memory, once a block and column.
//
// Two shapes.  Pairs: persistent CTA pairs, 256 x 256 tiles, tcgen05.mma
// .cta_group::2; a pair holds 128 rows of B and half the tokens per CTA.  Shares:
// a single CTA's tile is 128 rows of B by 16 to 128 tokens, and the summed index
// is shared out over a cluster of up to eight CTAs, which add their sums through
// distributed shared memory, in the order of their ranks: no workspace, no
// atomics, and the same bits every time.
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

constexpr int kLanes = 128;                // rows of B that one CTA holds: the lanes of tensor memory
constexpr int kStep = 128;                 // summed elements (and bytes) of a block: one 128-byte swizzle row
constexpr int kAtom = kLanes * kStep;
constexpr int kSlab = 4;                   // blocks whose scales are laid out at a time
constexpr int kSlabs = 3;
constexpr int kPad = 8;                    // floats between a slab's blocks, off the same bank
constexpr int kLoaders = 64;               // threads that lay out scales (warps 2 and 3)
constexpr int kOthers = 128;               // threads of warps 0 to 3
constexpr int kMaxShares = 8;
constexpr uint32_t kWaitLimit = 1u << 22;  // bounded polling; each poll may sleep up to kSuspendNs
constexpr uint32_t kSuspendNs = 1000;
constexpr uint32_t kLook = 1024;           // polls between looks at the abort flag
constexpr uint32_t kDrainLimit = 1u << 16; // polls for copies in flight, after a wait has given up

// CW columns a warp, GROUPS warps of each lane quadrant: tiles of CW * GROUPS tokens.
template <bool PAIR, int CW, int GROUPS>
struct Cfg {
    static constexpr int kCols = CW * GROUPS;
    static constexpr int kThreads = kOthers + 128 * GROUPS;
    static constexpr int kRows = PAIR ? 2 * kLanes : kLanes;         // rows of B of a tile
    static constexpr int kQRows = PAIR ? kCols / 2 : kCols;          // tokens that a CTA holds
    static constexpr int kQ = kQRows * kStep;
    static constexpr int kStage = kAtom + kQ;
    static constexpr int kStages = PAIR ? 6 : (kCols <= 32 ? 5 : (kCols <= 64 ? 4 : 6));
    static constexpr int kColPitch = kCols + kPad, kRowPitch = kLanes + kPad;
    static constexpr int kSlabFloats = kSlab * (kColPitch + kRowPitch);
    static constexpr int kOffScales = kStages * kStage;
    static constexpr int kOffBars = kOffScales + kSlabs * kSlabFloats * 4;
    // full, empty; partial sums full x2, empty x2; slabs full, empty; drain
    static constexpr int kNumBars = 2 * kStages + 4 + 2 * kSlabs + 1;
    static constexpr int kOffWords = kOffBars + 8 * kNumBars;  // tensor memory address, abort flag, stages filled and used
    static constexpr int kSmem = kOffWords + 16 + 1024;
    static constexpr int kTmem = 2 * kCols;
    static_assert(kTmem >= 32 && (kTmem & (kTmem - 1)) == 0 && kTmem <= 512, "tensor memory columns");
    static_assert(kSmem <= 232448, "shared memory overflow");
    static_assert(kCols * kLanes * 4 <= kStages * kStage, "a share's sums take the stages' place");
    static_assert(kQRows % 8 == 0 && kQ % 1024 == 0, "swizzle atoms");
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
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cbar) : "memory");
}
// Bounded wait on an mbarrier phase; false at the limit (with the error word
// set), or once `abort` is set, which is looked at every kLook polls.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, const volatile int* abort,
                                          uint32_t limit = kWaitLimit) {
    for (uint32_t left = limit; left;) {
        const uint32_t n = min(left, kLook);
        for (uint32_t i = 0; i < n; ++i) {
            uint32_t ok;
            asm volatile(
                "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;"
                " selp.u32 %0, 1, 0, p; }"
                : "=r"(ok)
                : "r"(bar), "r"(parity), "r"(kSuspendNs)
                : "memory");
            if (ok) return true;
        }
        left -= n;
        if (abort && *abort) return false;
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
// 16 or 32 columns of a warp's 32 lanes.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[32]) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]),
          "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]),
          "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]),
          "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&r)[16]) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]),
          "=r"(u[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ------------------------------------------------------------------- kernel
struct Fp8Params {
    int M, N;
    int blocks;             // of the summed index
    int m_tiles, n_tiles;   // of tokens, of rows of B
    int group;              // tile order: rows of B that advance first
    int shares, per;        // CTAs of a cluster and blocks of each (single CTAs)
    int a_rows;             // tokens that a copy brings: up to a tile's
    uint32_t wait_limit;    // polls of a stage's arrival; all other waits keep kWaitLimit
    const float* sa;
    const float* sb;
    int64_t ld_sa, ld_sb;
    int a_shift, b_shift;   // log2 of the rows that share a scale: 0 or 7
    void* d;
    int64_t ldd;
    int d_f32, accumulate;
};

__device__ __forceinline__ void tile_at(const Fp8Params& p, int tile, int& mt, int& nt) {
    const int group = min(p.group, p.n_tiles);
    const int span = group * p.m_tiles, g = tile / span, first = g * group;
    const int rows = min(group, p.n_tiles - first), l = tile - g * span;
    mt = l / rows;
    nt = first + (l - mt * rows);
}

__device__ __forceinline__ void put(const Fp8Params& p, int m, int n, float v) {
    const int64_t at = (int64_t)m * p.ldd + n;
    if (p.d_f32) {
        float* d = (float*)p.d + at;
        *d = p.accumulate ? *d + v : v;
    } else {
        ((__nv_bfloat16*)p.d)[at] = __float2bfloat16_rn(v);
    }
}

__device__ __forceinline__ float column(const uint64_t* acc, int c) {
    float x, y;
    up2(acc[c >> 1], x, y);
    return c & 1 ? y : x;
}

// Warp 0 copies the operands (one thread), warp 1 of the leader issues the
// MMAs, warps 2 and 3 lay out the scales, the rest scale and add.  BOTH: the
// rows of B have scales of their own; otherwise a tile's 128 share one.
template <bool PAIR, bool BOTH, int CW, int GROUPS>
__global__ void __launch_bounds__((Cfg<PAIR, CW, GROUPS>::kThreads), 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ Fp8Params p) {
    using C = Cfg<PAIR, CW, GROUPS>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t bars = base + C::kOffBars;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto sumf_bar = [&](int b) { return bars + 8u * (2 * S + b); };
    auto sume_bar = [&](int b) { return bars + 8u * (2 * S + 2 + b); };
    auto slabf_bar = [&](int i) { return bars + 8u * (2 * S + 4 + i); };
    auto slabe_bar = [&](int i) { return bars + 8u * (2 * S + 4 + kSlabs + i); };
    const uint32_t drain_bar = bars + 8u * (2 * S + 4 + 2 * kSlabs);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffWords);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::kOffWords + 4);
    volatile int* stages_of = reinterpret_cast<volatile int*>(gbase + C::kOffWords + 8);  // filled, used
    auto slab_cols = [&](int i) { return reinterpret_cast<float*>(gbase + C::kOffScales) + i * C::kSlabFloats; };
    auto slab_rows = [&](int i) { return slab_cols(i) + kSlab * C::kColPitch; };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int peer = PAIR ? (int)rank : 0;  // 0: the CTA that issues the MMAs
    const int cluster_id = PAIR ? blockIdx.x >> 1 : blockIdx.x / p.shares;
    const int num_clusters = PAIR ? gridDim.x >> 1 : gridDim.x / p.shares;
    const int num_tiles = p.m_tiles * p.n_tiles;
    // this CTA's share of the summed index
    const int k0 = PAIR ? 0 : (int)rank * p.per;
    const int k_blocks = PAIR ? p.blocks : max(0, min(p.per, p.blocks - k0));

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);   // the leader's expect_tx arrival (both CTAs' bytes)
            mbar_init(empty_bar(s), 1);  // the leader's commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(sumf_bar(b), 1);                              // the leader's commit
            mbar_init(sume_bar(b), (PAIR ? 2 : 1) * 4 * GROUPS);    // every scaling warp
        }
        for (int i = 0; i < kSlabs; ++i) {
            mbar_init(slabf_bar(i), kLoaders);
            mbar_init(slabe_bar(i), 4 * GROUPS);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
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
        *abort_flag = 1;
        if (PAIR) st_cluster(map_to_rank(base + C::kOffWords + 4, rank ^ 1u), 1);
    };

    if (warp == 0 && lane == 0) {
        // ---------------------------------------------------- TMA copies
        int s = 0, stages = 0;
        uint32_t ph = 0;
        const uint32_t tx = PAIR ? 2 * C::kStage : kAtom + (uint32_t)p.a_rows * kStep;
        for (int tile = cluster_id; tile < num_tiles && !*abort_flag; tile += num_clusters) {
            int mt, nt;
            tile_at(p, tile, mt, nt);
            const int brow = nt * C::kRows + peer * kLanes, arow = mt * C::kCols + peer * C::kQRows;
            for (int kb = 0; kb < k_blocks; ++kb) {
                if (!mbar_wait(empty_bar(s), ph ^ 1u, abort_flag)) {
                    give_up();
                    break;
                }
                ++stages;
                const uint32_t fb = PAIR ? map_to_rank(full_bar(s), 0) : full_bar(s);
                if (peer == 0) mbar_expect_tx(full_bar(s), tx);
                const uint32_t dst = base + s * C::kStage;
                tma_load<PAIR>(dst, &map_b, (k0 + kb) * kStep, brow, fb);
                tma_load<PAIR>(dst + kAtom, &map_a, (k0 + kb) * kStep, arow, fb);
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        stages_of[0] = stages;
    } else if (warp == 1 && lane == 0 && peer == 0) {
        // ------------------------------------------------ MMA issuer (leader only)
        constexpr uint32_t idesc = make_idesc(C::kRows, C::kCols);
        int s = 0, stages = 0, buf = 0;
        uint32_t ph = 0, bph = 0;
        bool ok = true;
        for (int tile = cluster_id; tile < num_tiles && ok; tile += num_clusters) {
            for (int kb = 0; kb < k_blocks; ++kb) {
                if (!mbar_wait(full_bar(s), ph, nullptr, p.wait_limit) || !mbar_wait(sume_bar(buf), bph ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                ++stages;
                tc_fence_after();
                const uint64_t db = sw128_desc(base + s * C::kStage), da = sw128_desc(base + s * C::kStage + kAtom);
#pragma unroll
                for (int i = 0; i < 4; ++i)  // 32 bytes of the summed index each
                    mma<PAIR>(tmem + buf * C::kCols, db + 2 * i, da + 2 * i, idesc, i > 0 ? 1u : 0u);
                tc_commit<PAIR>(empty_bar(s));
                tc_commit<PAIR>(sumf_bar(buf));
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
                if (++buf == 2) {
                    buf = 0;
                    bph ^= 1u;
                }
            }
        }
        if (!ok) give_up();
        stages_of[1] = stages;
        tc_commit_local<PAIR>(drain_bar);
        mbar_wait(drain_bar, 0, nullptr);
    } else if (warp == 2 || warp == 3) {
        // ------------------------------------------------ scales
        const int tid = threadIdx.x - 64;
        const int kk = tid & (kSlab - 1);
        int i = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int tile = cluster_id; tile < num_tiles && ok; tile += num_clusters) {
            int mt, nt;
            tile_at(p, tile, mt, nt);
            const int m0 = mt * C::kCols, n0 = nt * C::kRows + peer * kLanes;
            for (int kb = 0; kb < k_blocks; kb += kSlab) {
                if (!mbar_wait(slabe_bar(i), ph ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                // this thread's block of the slab, of every 16th column or row
                const bool live = kb + kk < k_blocks;
                const int64_t b = k0 + kb + kk;
                const float* sa = p.sa + b;
                float common = 1.0f;
                if (!BOTH) common = live && n0 < p.N ? p.sb[(int64_t)(n0 >> p.b_shift) * p.ld_sb + b] : 0.0f;
                float* cols = slab_cols(i) + kk * C::kColPitch;
                constexpr int kEach = C::kCols * kSlab / kLoaders, kTurn = kEach < 8 ? kEach : 8;  // loads in flight
#pragma unroll 1
                for (int j0 = 0; j0 < kEach; j0 += kTurn) {
                    float v[kTurn];
                    const int q = (tid >> 2) + 16 * j0;
#pragma unroll
                    for (int j = 0; j < kTurn; ++j) {
                        const int m = m0 + q + 16 * j;
                        v[j] = live && m < p.M ? sa[(int64_t)(m >> p.a_shift) * p.ld_sa] : 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < kTurn; ++j) cols[q + 16 * j] = BOTH ? v[j] : v[j] * common;
                }
                if (BOTH) {
                    float* rows = slab_rows(i) + kk * C::kRowPitch;
                    float w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int n = n0 + (tid >> 2) + 16 * j;
                        w[j] = live && n < p.N ? p.sb[(int64_t)(n >> p.b_shift) * p.ld_sb + b] : 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) rows[(tid >> 2) + 16 * j] = w[j];
                }
                mbar_arrive(slabf_bar(i));
                if (++i == kSlabs) {
                    i = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!ok) give_up();
    } else if (warp >= 4) {
        // ------------------------------------------------- scaling and adding
        constexpr int kChunk = PAIR || CW < 32 ? 16 : 32;
        const int quad = warp & 3, first = ((warp - 4) >> 2) * CW;
        const int row = quad * 32 + lane;  // of the CTA's 128
        int buf = 0, i = 0;
        uint32_t bph = 0, ph = 0;
        bool ok = true;
        uint64_t acc[CW / 2];
        for (int tile = cluster_id; tile < num_tiles; tile += num_clusters) {
#pragma unroll
            for (int c = 0; c < CW / 2; ++c) acc[c] = 0;
            for (int kb = 0; kb < k_blocks; ++kb) {
                const int kk = kb & (kSlab - 1);
                if (kk == 0) ok = mbar_wait(slabf_bar(i), ph, abort_flag);
                ok = ok && mbar_wait(sumf_bar(buf), bph, abort_flag);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float* cols = slab_cols(i) + kk * C::kColPitch + first;
                uint64_t rs2 = 0;
                if (BOTH) {
                    const float rs = slab_rows(i)[kk * C::kRowPitch + row];
                    rs2 = pk2(rs, rs);
                }
                const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16) + buf * C::kCols + first;
#pragma unroll
                for (int c = 0; c < CW; c += kChunk) {
                    float r[kChunk];
                    tmem_ld(at + c, r);
                    if (c + kChunk == CW) {  // read: the buffer may be filled again
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (PAIR) mbar_arrive_cluster(map_to_rank(sume_bar(buf), 0));
                            else mbar_arrive(sume_bar(buf));
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kChunk; j += 4) {
                        const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(cols + c + j);
                        uint64_t x = pk2(r[j], r[j + 1]), y = pk2(r[j + 2], r[j + 3]);
                        uint64_t &ax = acc[(c + j) / 2], &ay = acc[(c + j) / 2 + 1];
                        if (BOTH) {
                            ax = fma2(mul2(x, w.x), rs2, ax);
                            ay = fma2(mul2(y, w.y), rs2, ay);
                        } else {
                            ax = fma2(x, w.x, ax);
                            ay = fma2(y, w.y, ay);
                        }
                    }
                }
                if (++buf == 2) {
                    buf = 0;
                    bph ^= 1u;
                }
                if (kk == kSlab - 1 || kb + 1 == k_blocks) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(slabe_bar(i));
                    if (++i == kSlabs) {
                        i = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) {
                give_up();
                break;
            }
            if (!PAIR && p.shares > 1) {
                // every copy and MMA of this CTA is done: the sums take the stages' place, [column][row]
                float* sums = reinterpret_cast<float*>(gbase);
#pragma unroll
                for (int c = 0; c < CW; c += 2) {
                    float x, y;
                    up2(acc[c / 2], x, y);
                    sums[(first + c) * kLanes + row] = x;
                    sums[(first + c + 1) * kLanes + row] = y;
                }
                break;  // one tile a cluster
            }
            int mt, nt;
            tile_at(p, tile, mt, nt);
            const int n = nt * C::kRows + peer * kLanes + row, m0 = mt * C::kCols + first;
            const int live = n < p.N ? p.M - m0 : 0;
            const int64_t at = (int64_t)m0 * p.ldd + n;
            if (p.d_f32) {
                float* d = (float*)p.d + at;
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    if (c < live) *d = p.accumulate ? *d + column(acc, c) : column(acc, c);
                    d += p.ldd;
                }
            } else {
                __nv_bfloat16* d = (__nv_bfloat16*)p.d + at;
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    if (c < live) *d = __float2bfloat16_rn(column(acc, c));
                    d += p.ldd;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();  // neither CTA leaves while the other may still use its memory or barriers
    if (!PAIR && p.shares > 1) {
        cluster_sync_all();  // all shares' sums are there
        int mt, nt;
        tile_at(p, cluster_id, mt, nt);
        // each CTA adds its share of the columns over the ranks, in their order
        const int share = (C::kCols + p.shares - 1) / p.shares;
        const int begin = (int)rank * share, end = min(C::kCols, begin + share);
        const int live = min(end, p.M - mt * C::kCols);
        for (int i = begin * kLanes + (int)threadIdx.x; i < live * kLanes; i += C::kThreads) {
            const int n = nt * C::kRows + (i & (kLanes - 1));
            float v[kMaxShares];
#pragma unroll
            for (int r = 0; r < kMaxShares; ++r)
                v[r] = r < p.shares ? __int_as_float(ld_cluster(map_to_rank(base + 4u * i, r))) : 0.0f;
            float sum = v[0];
#pragma unroll
            for (int r = 1; r < kMaxShares; ++r)
                if (r < p.shares) sum += v[r];
            if (n < p.N) put(p, mt * C::kCols + (i >> 7), n, sum);
        }
        cluster_sync_all();  // no CTA leaves while another reads its sums
    }
    if (__builtin_expect(*abort_flag, 0)) {
        // A wait gave up (both CTAs of a pair know): stages that were filled but not used may still be on their way into
        // either CTA.  They are waited for before any CTA leaves, with a limit, since a stage that only one of the
        // copiers filled never completes.
        if (threadIdx.x == 0 && peer == 0) {
            int most = stages_of[0];
            if (PAIR) most = max(most, ld_cluster(map_to_rank(base + C::kOffWords + 8, 1)));
            for (int i = stages_of[1]; i < most; ++i) mbar_wait(full_bar(i % S), (i / S) & 1, nullptr, kDrainLimit);
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

// Clusters of the pairs' kernel that fit the device at once.
template <bool BOTH>
int max_pairs(int dev, const cudaLaunchConfig_t& cfg) {
    static DeviceFigure clusters;
    return clusters.get(dev, [&] {
        int n = 0;
        return cudaOccupancyMaxActiveClusters(&n, fp8_gemm_kernel<true, BOTH, 64, 4>, &cfg) == cudaSuccess ? n : 0;
    });
}

template <bool PAIR, bool BOTH, int CW, int GROUPS>
cudaError_t run(const Fp8GemmArgs& a, int shares, cudaStream_t st) {
    using C = Cfg<PAIR, CW, GROUPS>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    Fp8Params p = {};
    p.M = (int)a.M;
    p.N = (int)a.N;
    p.blocks = (int)((a.K + kStep - 1) / kStep);
    p.m_tiles = (int)((a.M + C::kCols - 1) / C::kCols);
    p.n_tiles = (int)((a.N + C::kRows - 1) / C::kRows);
    p.group = PAIR ? 8 : 1 << 30;
    p.shares = PAIR ? 1 : shares;
    p.per = (p.blocks + p.shares - 1) / p.shares;
    p.a_rows = (int)std::min<int64_t>(C::kQRows, (a.M + 7) / 8 * 8);
    if (PAIR) p.a_rows = C::kQRows;
    p.wait_limit = kWaitLimit - g_lowered[dev].load(std::memory_order_relaxed);
    p.sa = a.a.scales;
    p.sb = a.b.scales;
    p.ld_sa = a.a.scales_ld;
    p.ld_sb = a.b.scales_ld;
    p.a_shift = a.a_square ? 7 : 0;
    p.b_shift = a.b_square ? 7 : 0;
    p.d = a.d;
    p.ldd = a.ldd;
    p.d_f32 = a.d_f32;
    p.accumulate = a.accumulate;
    CUtensorMap ma, mb;
    if (!encode_map_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.a.codes, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.a.codes_ld,
                       kStep, (uint32_t)p.a_rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_map_2d(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.b.codes, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.b.codes_ld,
                       kStep, kLanes, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    auto k = fp8_gemm_kernel<PAIR, BOTH, CW, GROUPS>;
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
    cfg.numAttrs = 1;
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
    if (PAIR) {
        const int most = max_pairs<BOTH>(dev, cfg);
        if (most <= 0) return cudaErrorLaunchOutOfResources;
        cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(tiles, most));
    } else {
        cfg.gridDim = dim3((unsigned)(tiles * shares));
    }
    cfg.numAttrs = st ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, ma, mb, p);
}

template <bool BOTH>
cudaError_t launch(const Fp8GemmArgs& a, int num_sms, cudaStream_t st) {
    const int64_t blocks = (a.K + kStep - 1) / kStep;
    const int64_t pair_tiles = (a.M + 255) / 256 * ((a.N + 255) / 256);
    if (a.M > 128 && pair_tiles >= num_sms / 4) return run<true, BOTH, 64, 4>(a, 1, st);
    const int64_t width = a.M <= 16 ? 16 : (a.M <= 32 ? 32 : (a.M <= 64 ? 64 : 128));
    const int64_t tiles = (a.M + width - 1) / width * ((a.N + kLanes - 1) / kLanes);
    const int64_t room = (width <= 64 ? 2 : 1) * (int64_t)num_sms;
    // shares: the fewest blocks for the busiest SM
    int shares = 1;
    int64_t best = 1ll << 60;
    for (int s = 1; s <= kMaxShares && s <= blocks; ++s) {
        const int64_t rounds = (tiles * s + room - 1) / room;
        const int64_t cost = rounds * ((blocks + s - 1) / s + 2);
        if (cost < best) {
            best = cost;
            shares = s;
        }
    }
    if (width == 16) return run<false, BOTH, 16, 1>(a, shares, st);
    if (width == 32) return run<false, BOTH, 32, 1>(a, shares, st);
    if (width == 64) return run<false, BOTH, 64, 1>(a, shares, st);
    return run<false, BOTH, 64, 2>(a, shares, st);
}

template <bool PAIR, bool BOTH, int CW, int GROUPS>
cudaError_t preload() {
    return cudaFuncSetAttribute(fp8_gemm_kernel<PAIR, BOTH, CW, GROUPS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg<PAIR, CW, GROUPS>::kSmem);
}
template <bool BOTH>
cudaError_t preload_all() {
    cudaError_t e = preload<true, BOTH, 64, 4>();
    if (e == cudaSuccess) e = preload<false, BOTH, 16, 1>();
    if (e == cudaSuccess) e = preload<false, BOTH, 32, 1>();
    if (e == cudaSuccess) e = preload<false, BOTH, 64, 1>();
    return e == cudaSuccess ? preload<false, BOTH, 64, 2>() : e;
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, int num_sms, cudaStream_t st) {
    return a.b_square ? launch<false>(a, num_sms, st) : launch<true>(a, num_sms, st);
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
