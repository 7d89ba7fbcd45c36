// Softmax cross entropy of a vocabulary head, and its gradient, without the
// logits in memory (the linear layer behind the last block of a model; its
// three products are the FPROP, DGRAD and WGRAD of UFP4 summary, section 方法,
// kept in bf16).
//
//   l = H W^T                       H: tokens x K, W: vocabulary x K
//   lse_t = log sum_v exp l_tv      loss_t = lse_t - l_t,target + z lse_t^2
//   dl_tv = w_t ((1 + 2 z lse_t) exp(l_tv - lse_t) - [v = target_t])
//   dH = scale dl W                 dW = scale dl^T H
//
// Tokens without a target (ignored) take no part in any product: the first
// kernel of either pass packs the rows of H that have one, so work goes with
// the number of valid tokens, and whatever an ignored row holds stays out of
// dW.  (Up to 128 tokens, forward, are read where they lie: W is what that call
// reads, and a logit's row meets no other.)  Forward, each tile of logits
// leaves its rows' running maximum and sum of exponentials, joined in the
// tiles' order by a last kernel.
// Backward, the vocabulary is walked in pieces: a piece's logits are computed
// again, become dl (bf16) in a workspace of two pieces, and are multiplied
// into dH (fp32 until the last piece) and dW.  Recomputing costs 2 of the 8
// products-and-sums per logit; keeping the logits would cost 4 bytes each.
//
// The tensor cores bound it from about a thousand tokens on: 8192 tokens (a
// tenth ignored) x 50001 x 2048 forward 0.86 to 0.91 ms by box when run without
// a pause, 1660 to 1750 TFLOP/s, and 4096 x 65536 x 7168 with the gradients 9.0 to
// 9.3 ms, 1650 to 1710 TFLOP/s with the recomputed logits (the library's bf16
// product sustains 1714, and 1924 in a burst).  With few tokens it is W: 16
// tokens x 65536 x 7168 forward 149 us, 6.3 TB/s.
//
// dl is rounded to bf16 because the tensor cores multiply it with bf16 W and H:
// a relative error of at most 2^-8 per entry, as the outputs' own rounding,
// and unbiased; the common factor `scale` is applied to the fp32 results, so
// that a uniform weight does not round every entry the same way.  Of many
// tokens' gradients that leaves 0.0024 of the exact ones (2-norm, bf16 results;
// their own rounding alone 0.0017); of few, where nothing averages it away, dl
// is kept in two bf16 parts (fine_backward).
//
// All products run in one persistent kernel of CTA pairs (tcgen05.mma
// .cta_group::2, 256 x 256 output tiles, fp32 accumulators in tensor memory,
// two of them, so that a tile's epilogue overlaps the next tile's main loop).
// A launch walks the tiles of up to three products (dH and dW of a piece and
// the logits of the next), which fills the SMs where one product has few
// tiles.  Operands are read as they lie in memory: where the summed index is
// not the contiguous one (W in dH; dl and H in dW) the tiles are staged
// MN-major and the instruction descriptor says so; nothing is transposed.
#include <algorithm>
#include <atomic>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_figure.h"
#include "internal.h"
#include "train.h"

namespace ufp4 {

__device__ int g_head_error;

namespace {

constexpr int kTile = 256;                 // output columns of a tile, and rows of a CTA pair's tile
constexpr int kHalf = 128;                 // rows of A that one CTA holds
constexpr int kAlone = 224;                // most columns of a single CTA's tile
constexpr int kStep = 64;                  // summed elements per step (one 128-byte swizzle row)
constexpr int kBlockBytes = 64 * 64 * 2;   // 64 rows of 64 bf16: one column block of an MN-major operand
constexpr int kAtom = 2 * kBlockBytes;     // 128 rows of one step
constexpr int kThreads = 384;
constexpr int kFine = kHalf;               // most tokens whose dl is kept in two parts (fine_backward)
constexpr int kRing = 4;                   // tiles handed out ahead (even: a place serves one epilogue group)
constexpr uint32_t kWaitLimit = 1u << 22;  // bounded polling; each poll may sleep up to kSuspendNs
constexpr uint32_t kSuspendNs = 1000;
constexpr uint32_t kLook = 1024;  // polls between looks at the abort flag
constexpr uint32_t kDrainLimit = 1u << 16;  // polls for copies in flight, after a wait has given up
// The copiers' polls for a free stage, about 70 ms for what takes
// microseconds: they do not look at the abort flag meanwhile (the look
// takes 128 x 5000 x 2048 forward from 18.7 to 20.7 us).
constexpr uint32_t kFreeLimit = 1u << 16;
constexpr float kLog2e = 1.4426950408889634f;

// A CTA pair's 256 x 256 tile, or a single CTA's 128 x (up to 224) tile.  A
// pair holds 128 rows of A and half the rows of B per CTA, so it moves two
// thirds of the single CTA's bytes per product; its stages hold two steps,
// which halves the hand-offs between the copies and the tensor core (one-step
// stages: 4096 x 16384 x 2048 logits 193 us, two-step stages 174 us).  A
// single CTA's tile is for reading W once: 224 columns leave room for a fifth
// stage (16 tokens, 131072 x 2048, when first built: 256 columns and four
// stages 124 us, 224 and five 111 us, 96 and eight 173 us; now 93 us, 5.8 TB/s).
template <bool PAIR>
struct Cfg {
    static constexpr int kRows = PAIR ? kTile : kHalf;   // rows of a tile
    static constexpr int kKps = PAIR ? 2 : 1;            // steps per stage
    static constexpr int kStages = PAIR ? 3 : 5;
    static constexpr int kBRows = PAIR ? kHalf : kAlone;  // rows of B per CTA
    static constexpr int kAtomB = kBRows * 128;
    static constexpr int kA = kKps * kAtom, kB = kKps * kAtomB;
    static constexpr int kOffA = 0;
    static constexpr int kOffB = kStages * kA;
    static constexpr int kOffOut = kOffB + kStages * kB;  // 4 KB for each epilogue warp
    static constexpr int kOut = PAIR ? 8 * 4096 : 0;
    static constexpr int kOffBars = kOffOut + kOut;
    // full, empty; accumulators full x2, empty x2; ring full, empty; drain
    static constexpr int kNumBars = 2 * kStages + 4 + 2 * kRing + 1;
    // tensor memory address, abort flag, ring of tiles; stages that the CTA's copiers filled (x2), and that were used
    static constexpr int kOffWords = kOffBars + 8 * kNumBars;
    static constexpr int kOffStages = kOffWords + 4 * (2 + kRing);
    static constexpr int kSmem = kOffStages + 4 * 3 + 1024;
    static_assert(kSmem <= 232448, "shared memory overflow");
};

// ------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Bounded wait on an mbarrier phase; false at the limit (with the error word
// set), or once `abort` (where given) is set, which is looked at every kLook
// polls.  CLUSTER: for what a thread of either CTA of the pair wrote before it
// arrived.
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, const volatile int* abort,
                                          uint32_t limit = kWaitLimit) {
    for (uint32_t left = limit; left;) {
        const uint32_t n = min(left, kLook);
        for (uint32_t i = 0; i < n; ++i) {
            uint32_t ok;
            if (CLUSTER)
                asm volatile(
                    "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;"
                    " selp.u32 %0, 1, 0, p; }"
                    : "=r"(ok)
                    : "r"(bar), "r"(parity), "r"(kSuspendNs)
                    : "memory");
            else
                asm volatile(
                    "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                    : "=r"(ok)
                    : "r"(bar), "r"(parity), "r"(kSuspendNs)
                    : "memory");
            if (ok) return true;
        }
        left -= n;
        if (abort && *abort) return false;
    }
    atomicExch(&g_head_error, 1);
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
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cbar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cbar) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t caddr, int v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(caddr), "r"(v) : "memory");
}
__device__ __forceinline__ int ld_cluster(uint32_t caddr) {
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(caddr) : "memory");
    return v;
}
// TMA box into this CTA's shared memory, counted on a barrier of either CTA of the pair.
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

// 128-byte swizzle shared-memory descriptor: 8-row groups 1024 bytes apart
// (stride offset); MN-major operands also have their 64-element column blocks
// one box apart (leading offset; unused K-major, where a stage is one column).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(kBlockBytes >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f16: fp32 accumulator, bf16 operands, MN-major A (bit 15) and B (bit 16), N >> 3, M >> 4.
__host__ __device__ constexpr uint32_t make_idesc(int rows, int cols, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(cols >> 3) << 17) | ((uint32_t)(rows >> 4) << 24);
}
template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if (PAIR)
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }"
            ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
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
__device__ __forceinline__ void tmem_alloc(uint32_t slot) {
    if (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t tmem) {
    if (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float r[32]) {
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
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// ------------------------------------------------------- packing the tokens
// Per packed row, for the epilogues: its target, and backward its lse * log2(e),
// weight * (1 + 2 z lse) and weight.
struct RowInfo {
    float lse2, a, weight;
    int target;
};

struct PackParams {
    const __nv_bfloat16* h;
    int64_t ldh;
    const int64_t* targets;
    int64_t T, V, K, Kp;      // Kp: columns of the packed rows (K rounded up to 8)
    int rows_per_cta;
    __nv_bfloat16* packed;    // rounded-up rows x Kp
    int* index;               // packed row -> token
    RowInfo* info;
    int* count;
    int* next;                // tile counters of the launches that follow, zeroed
    int launches;
    int fine;                 // backward: every packed row a second time, behind them all
    float* loss;              // forward: 0 for ignored tokens
    float* lse_out;
    const float* lse;         // backward
    const float* weight;
    float z;
    void* dh;                 // backward: 0 for ignored tokens
    int64_t ld_dh;
    int dh_f32;
};

// CTA b packs the valid tokens among its rows: it counts those before them,
// then, kPackRows rows at a time, each warp copies a row.  Rows from the count
// up to the next multiple of kStep are zeroed: dW sums over them.  Every CTA
// reads all targets, so there are no more of them than are resident at once,
// whatever the tokens (with one for each 64 rows, a million tokens read 137 GB
// of targets, and a pass over 1048576 x 256 x 256 took 8.6 ms; now 1.1).
constexpr int kPackRows = 64;
constexpr int kPackCtas = 5;  // an SM, at 48 registers a thread
template <bool BACK>
__global__ void __launch_bounds__(256, kPackCtas) head_pack_kernel(const PackParams p) {
    __shared__ int before_s, all_s;
    __shared__ int place[kPackRows];  // packed row of each of the rows in hand, or -1
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = (int64_t)blockIdx.x * p.rows_per_cta;
    const int64_t end = min(r0 + p.rows_per_cta, p.T);  // no rows in CTAs past the tokens
    auto valid = [&](int64_t r) {
        const int64_t t = p.targets[r];
        return t >= 0 && t < p.V;
    };
    if (threadIdx.x == 0) before_s = all_s = 0;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll 8
    for (int64_t r = threadIdx.x; r < p.T; r += blockDim.x) {
        const int v = valid(r);
        all += v;
        before += v && r < r0;
    }
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    all = __reduce_add_sync(0xFFFFFFFFu, all);
    if (lane == 0) {
        atomicAdd(&before_s, before);
        atomicAdd(&all_s, all);
    }
    __syncthreads();
    const int count = all_s;
    int next = before_s;  // warp 0's: packed row of the next valid token
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) *p.count = count;
        for (int i = threadIdx.x; i < p.launches; i += blockDim.x) p.next[i] = 0;
    }
    auto clear_row = [&](char* row, int64_t bytes) {  // a warp's; 2-byte multiples, 2-byte aligned at least
        const int64_t wide = (uintptr_t)row % 16 == 0 ? bytes / 16 : 0;
        for (int64_t i = lane; i < wide; i += 32) reinterpret_cast<uint4*>(row)[i] = make_uint4(0, 0, 0, 0);
        for (int64_t i = wide * 8 + lane; i < bytes / 2; i += 32) reinterpret_cast<uint16_t*>(row)[i] = 0;
    };
    for (int64_t first = r0; first < end; first += kPackRows) {
        const int rows = (int)min((int64_t)kPackRows, end - first);
        if (first > r0) __syncthreads();  // the places of the rows before are read
        if (warp == 0) {
            for (int i = 0; i < rows; i += 32) {
                const bool v = i + lane < rows && valid(first + i + lane);
                const uint32_t which = __ballot_sync(0xFFFFFFFFu, v);
                if (i + lane < rows) place[i + lane] = v ? next + __popc(which & ((1u << lane) - 1)) : -1;
                next += __popc(which);
            }
        }
        __syncthreads();
        for (int i = warp; i < rows; i += 8) {
            const int64_t r = first + i;
            const int at = place[i];
            if (at < 0) {
                if (BACK) {
                    const int es = p.dh_f32 ? 4 : 2;
                    if (p.dh) clear_row((char*)p.dh + r * p.ld_dh * es, p.K * es);
                } else if (lane == 0) {
                    p.loss[r] = 0.0f;
                    p.lse_out[r] = 0.0f;
                }
                continue;
            }
            for (int copy = 0; copy <= (BACK ? p.fine : 0); ++copy) {
                const int64_t row = at + (copy ? count : 0);
                const uint4* src = reinterpret_cast<const uint4*>(p.h + r * p.ldh);
                uint4* dst = reinterpret_cast<uint4*>(p.packed + row * p.Kp);
#pragma unroll 8
                for (int64_t j = lane; j < p.K / 8; j += 32) dst[j] = src[j];
                if (lane < p.K % 8) {  // nothing past a row's K elements is read
                    const int64_t j = p.K / 8 * 8 + lane;
                    p.packed[row * p.Kp + j] = p.h[r * p.ldh + j];
                }
            }
            if (lane == 0) {
                p.index[at] = (int)r;
                RowInfo info = {0.0f, 0.0f, 0.0f, (int)p.targets[r]};
                if (BACK) {
                    const float l = p.lse[r], w = p.weight ? p.weight[r] : 1.0f;
                    info.lse2 = l * kLog2e;
                    info.weight = w;
                    info.a = w * fmaf(2.0f * p.z, l, 1.0f);
                }
                p.info[at] = info;
            }
        }
    }
    if (BACK) {
        const int used = count << p.fine, last = (used + kStep - 1) / kStep * kStep;
        for (int z = used + blockIdx.x * 8 + warp; z < last; z += gridDim.x * 8)
            clear_row((char*)(p.packed + (int64_t)z * p.Kp), p.Kp * 2);
    }
}

// ------------------------------------------------------------- the products
enum JobKind { kStats = 0, kGrad = 1, kDH = 2, kDW = 3 };

// One product of a launch.
//   kStats  logits of all of W: rows' (max, sum) per tile, target logits
//   kGrad   logits of a piece of W -> dl of the piece
//   kDH     dl (packed rows x piece) times the piece of W -> dH
//   kDW     dl^T times the packed rows of H -> rows of dW
struct Job {
    int kind;
    int a, b;               // operands (Operand)
    int a_mn, b_mn;         // the operand's contiguous index is not the summed one
    int group;              // tile rows that advance before the column does
    int a_rows;             // rows of A that a CTA copies: kHalf, or the tokens there are (a multiple of 8)
    int width;              // columns of a tile: kTile, or less for single CTAs (a multiple of 16, up to kAlone)
    int m, n, k;            // extents; kernel-side: m (or k for kDW) comes from the token count
    int v0;                 // first vocabulary row of the piece
    int add;                // kDH: add to what earlier pieces left
    int slices, per;        // kDH: shares of the sum that tiles of their own take, and steps in each
    int slice0;             // kDH: index of the piece's first share
    __nv_bfloat16* dl;      // kGrad: output
    int64_t ld_dl;
};
constexpr int kMaxJobs = 3;
enum Operand { kOpH = 0, kOpW = 1, kOpDl = 2, kOperands = 4 };  // packed H, W, two pieces of dl
// Each operand's tensor map with boxes of 128 rows (K-major: a CTA's half of
// a tile) and of 64 rows (MN-major: one column block).  For single CTAs W's
// K-major boxes have half a tile's columns.
struct HeadMaps {
    CUtensorMap m[kOperands][2];
};
struct HeadParams {
    Job job[kMaxJobs];
    int jobs;
    uint32_t wait_limit;    // polls of a stage's arrival; all other waits keep kWaitLimit
    const int* count;       // null: all `tokens`, in place
    int tokens;
    const int64_t* targets; // with tokens in place
    int vocab;
    int* next;              // tiles handed out beyond one per cluster (pairs)
    const int* index;
    const RowInfo* info;
    float2* part;           // kStats: [row][vocabulary tile]
    int64_t ld_part;
    float* target_logit;
    int fine;               // backward: dl in two parts (fine_backward)
    float* rest;            // with `fine`: what the first part leaves of each row's entry at its target
    const __nv_bfloat16* w;
    int64_t ldw;
    float* dh_acc;          // fp32 dH of the packed rows (x Kp), or each share of it; null: dH is written at once
    int64_t Kp, Tp;
    int shares;
    const float* scale;
    void* dh;
    int64_t ld_dh;
    int dh_f32;
    void* dw;
    int64_t ld_dw;
    int dw_f32, accumulate;
};

struct TileAt {
    int job, m, n, k0, k_steps;  // k0: first step
    int slice;
};

// Tile rows that advance before the column does.  Tiles in flight walk the
// summed index together, so eight by about nine of them share few panels of
// either operand; where all of A stays in L2, all its rows go first, and B is
// read once.
constexpr int kGroupM = 8;
constexpr int64_t kResidentA = 48ll << 20;

template <int ROWS>
struct Walk {
    int m_tiles[kMaxJobs], n_tiles[kMaxJobs], k_steps[kMaxJobs], total;
    __device__ __forceinline__ Walk(const HeadParams& p, int count) {
        total = 0;
        for (int j = 0; j < kMaxJobs; ++j) {
            m_tiles[j] = n_tiles[j] = k_steps[j] = 0;
            if (j >= p.jobs) continue;
            const Job& q = p.job[j];
            const int m = q.kind == kDW ? q.m : count, k = q.kind == kDW ? count << p.fine : q.k;
            m_tiles[j] = (m + ROWS - 1) / ROWS;
            n_tiles[j] = (q.n + q.width - 1) / q.width;
            k_steps[j] = (k + kStep - 1) / kStep;
            total += m_tiles[j] * n_tiles[j] * q.slices;
        }
    }
    __device__ __forceinline__ TileAt at(const HeadParams& p, int tile) const {
        TileAt t;
        t.job = 0;
#pragma unroll
        for (int j = 0; j + 1 < kMaxJobs; ++j) {
            const int here = m_tiles[j] * n_tiles[j] * p.job[j].slices;
            if (t.job == j && tile >= here) {
                tile -= here;
                t.job = j + 1;
            }
        }
        int mt = m_tiles[0], nt = n_tiles[0];
        t.k_steps = k_steps[0];
#pragma unroll
        for (int j = 1; j < kMaxJobs; ++j)
            if (t.job == j) {
                mt = m_tiles[j];
                nt = n_tiles[j];
                t.k_steps = k_steps[j];
            }
        const Job& q = p.job[t.job];
        t.slice = q.slices > 1 ? tile / (mt * nt) : 0;
        tile -= t.slice * mt * nt;
        t.k0 = t.slice * q.per;
        if (q.slices > 1) t.k_steps = max(0, min(q.per, t.k_steps - t.k0));
        const int group = min(q.group, mt);
        const int span = group * nt, g = tile / span, first = g * group;
        const int rows = min(group, mt - first), l = tile - g * span;
        t.n = l / rows;
        t.m = first + (l - t.n * rows);
        return t;
    }
};

// Where a tile's results go: rows of `ld` bytes (row i at index[i], where
// given) up to `limit`, columns up to `cols`, as bf16 or fp32, added to what is
// there with `add` (fp32).
struct Dest {
    char* base;
    int64_t ld;
    int limit, cols;
    bool f32, add, fast;  // fast: rows are 16-byte aligned
    const int* index;
    __device__ __forceinline__ char* row(int r) const { return base + (index ? index[r] : r) * ld; }
};
__device__ __forceinline__ Dest make_dest(void* base, int64_t ld, int limit, int cols, bool f32, bool add,
                                          const int* index) {
    const int64_t bytes = ld * (f32 ? 4 : 2);
    return {(char*)base, bytes, limit, cols, f32, add, (((uintptr_t)base | (uintptr_t)bytes) & 15) == 0, index};
}

// Writes a warp's 32 rows of a tile.  A lane holds a row, so its own stores
// would touch 32 rows at a time, half a sector each; instead 128 bytes of every
// row are turned around in `stage` (16-byte units, unit u of row i at
// u ^ (i & 7)) and stored four whole rows of them an instruction.  Ragged or
// unaligned columns go out of the lanes' registers.
struct Writer {
    Dest d;
    uint8_t* stage;
    char* rows[8];  // the rows that this lane stores, from its 16 bytes on; null past the limit
    char* mine;     // the lane's own row
    __device__ __forceinline__ Writer(const Dest& dest, uint8_t* stage_, int row0) : d(dest), stage(stage_) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = row0 + i * 4 + (lane >> 3);
            rows[i] = r < d.limit ? d.row(r) + (lane & 7) * 16 : nullptr;
        }
        mine = row0 + lane < d.limit ? d.row(row0 + lane) : nullptr;
    }
    // 128 bytes of each row from the stage, at byte `at` of the rows.
    __device__ __forceinline__ void flush(int64_t at) const {
        const int lane = threadIdx.x & 31;
        __syncwarp();
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = i * 4 + (lane >> 3);
            v[i] = reinterpret_cast<const uint4*>(stage + row * 128)[(lane & 7) ^ (row & 7)];
        }
        if (d.add) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (rows[i]) {
                    const uint4 o = *reinterpret_cast<const uint4*>(rows[i] + at);
                    v[i] = make_uint4(__float_as_uint(__uint_as_float(v[i].x) + __uint_as_float(o.x)),
                                      __float_as_uint(__uint_as_float(v[i].y) + __uint_as_float(o.y)),
                                      __float_as_uint(__uint_as_float(v[i].z) + __uint_as_float(o.z)),
                                      __float_as_uint(__uint_as_float(v[i].w) + __uint_as_float(o.w)));
                }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (rows[i]) *reinterpret_cast<uint4*>(rows[i] + at) = v[i];
        __syncwarp();
    }
    // Columns c .. c + 31 of the tile from column n0 on, in turn for c = 0, 32, ... (r: of the lane's row).
    __device__ __forceinline__ void columns(int n0, int c, const float r[32]) const {
        const int lane = threadIdx.x & 31;
        uint4* unit = reinterpret_cast<uint4*>(stage + lane * 128);
        if (d.f32) {
            if (d.fast && n0 + c + 32 <= d.cols) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    unit[u ^ (lane & 7)] = make_uint4(__float_as_uint(r[4 * u]), __float_as_uint(r[4 * u + 1]),
                                                      __float_as_uint(r[4 * u + 2]), __float_as_uint(r[4 * u + 3]));
                flush((int64_t)(n0 + c) * 4);
                return;
            }
        } else if (d.fast && n0 + (c & ~63) + 64 <= d.cols) {
            const int half = c & 32 ? 4 : 0;
#pragma unroll
            for (int u = 0; u < 4; ++u)
                unit[(half + u) ^ (lane & 7)] =
                    make_uint4(pack_bf16(r[8 * u], r[8 * u + 1]), pack_bf16(r[8 * u + 2], r[8 * u + 3]),
                               pack_bf16(r[8 * u + 4], r[8 * u + 5]), pack_bf16(r[8 * u + 6], r[8 * u + 7]));
            if (half) flush((int64_t)(n0 + c - 32) * 2);
            return;
        }
        if (!mine) return;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int col = n0 + c + i;
            if (col < d.cols) {
                if (d.f32)
                    ((float*)mine)[col] = d.add ? ((float*)mine)[col] + r[i] : r[i];
                else
                    ((__nv_bfloat16*)mine)[col] = __float2bfloat16_rn(r[i]);
            }
        }
    }
};

// The logits epilogue of one row of a tile: running maximum and sum.
__device__ __forceinline__ void stats_chunk(float r[32], int n, float& m, float& s) {
    float top = m;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        if (i >= n) r[i] = -INFINITY;
        top = fmaxf(top, r[i]);
    }
    const float shift = top == -INFINITY ? 0.0f : top * kLog2e;
    s *= ex2(fmaf(m, kLog2e, -shift));
#pragma unroll
    for (int i = 0; i < 32; ++i) s += ex2(fmaf(r[i], kLog2e, -shift));
    m = top;
}

// 32 logits of a row, from vocabulary entry `v` on (n of them exist), become dl.
__device__ __forceinline__ void grad_chunk(float r[32], const RowInfo& info, int v, int n) {
    const int at = info.target - v;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        float x = info.a * ex2(fmaf(r[i], kLog2e, -info.lse2));
        if (at == i) x -= info.weight;
        r[i] = i < n ? x : 0.0f;
    }
}

// Warps 0 and 2 copy A and B (one thread each: a single thread issuing both is
// 5 % slower), warp 1 of the leader issues the MMAs, warp 3 of the leader hands
// out tiles, warps 4 to 7 and 8 to 11 run the epilogues of even and odd tiles
// (each with its accumulator: where a tile has few steps, as dW of few tokens,
// its epilogue is what takes the time).  Tiles differ in length by an order
// of magnitude between products, so clusters take the next one from a counter
// in global memory when they have room for it; which cluster computes a tile
// changes nothing in its result.  Single CTAs, whose tiles are all alike, take
// a fixed share.
template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
head_gemm_kernel(const __grid_constant__ HeadMaps maps, const __grid_constant__ HeadParams p) {
    using C = Cfg<PAIR>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t bars = base + C::kOffBars;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto accf_bar = [&](int b) { return bars + 8u * (2 * S + b); };
    auto acce_bar = [&](int b) { return bars + 8u * (2 * S + 2 + b); };
    auto ringf_bar = [&](int i) { return bars + 8u * (2 * S + 4 + i); };
    auto ringe_bar = [&](int i) { return bars + 8u * (2 * S + 4 + kRing + i); };
    const uint32_t drain_bar = bars + 8u * (2 * S + 4 + 2 * kRing);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffWords);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::kOffWords + 4);
    volatile int* ring = reinterpret_cast<volatile int*>(gbase + C::kOffWords + 8);
    volatile int* stages_of = reinterpret_cast<volatile int*>(gbase + C::kOffStages);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_rank() : 0;
    const int peer = (int)(rank & 1u);      // 0: leader (even CTA)
    const uint32_t leader = rank & ~1u;
    const int cluster_id = PAIR ? blockIdx.x >> 1 : blockIdx.x;
    const int num_clusters = PAIR ? gridDim.x >> 1 : gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);   // the leader's expect_tx arrival (both CTAs' bytes)
            mbar_init(empty_bar(s), 1);  // the leader's commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf_bar(b), 1);             // the leader's commit
            mbar_init(acce_bar(b), PAIR ? 8 : 4);  // one group of epilogue warps
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(ringf_bar(i), 1);               // the leader's warp 3
            mbar_init(ringe_bar(i), 13);              // two copiers and a group of four epilogue warps a CTA, the issuer
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<PAIR>(smem_u32(tmem_slot));
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();  // both CTAs' barriers exist before any copy or commit targets them
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    griddep_launch();

    const int count = p.count ? *p.count : p.tokens;
    const Walk<C::kRows> walk(p, count);

    // Sets the abort flag of every CTA of the cluster.
    auto give_up = [&] {
        *abort_flag = 1;
        if (PAIR) st_cluster(map_to_rank(base + C::kOffWords + 4, rank ^ 1u), 1);
    };

    // The tile number i of this cluster, or -1 when there is none (or a wait gave up).  `arrive`: this
    // thread speaks for its reader (a copier, the issuer, an epilogue warp).
    auto take = [&](int i, bool arrive) {
        if (!PAIR) {  // a fixed share
            const int tile = cluster_id + i * num_clusters;
            return tile < walk.total && !*abort_flag ? tile : -1;
        }
        const int at = i % kRing;
        if (!mbar_wait<true>(ringf_bar(at), (i / kRing) & 1, abort_flag)) {
            give_up();
            return -1;
        }
        const int tile = ring[at];
        if (arrive) mbar_arrive_cluster(map_to_rank(ringe_bar(at), leader));
        return tile < walk.total ? tile : -1;
    };

    if (PAIR && warp == 3 && lane == 0 && peer == 0) {
        // ------------------------------------------------ hands out tiles (leader only)
        for (int i = 0, ends = 0; ends < 2; ++i) {  // an end for either epilogue group
            const int at = i % kRing;
            if (!mbar_wait<true>(ringe_bar(at), ((i / kRing) & 1) ^ 1, abort_flag)) {
                give_up();
                break;
            }
            const int tile = i == 0 ? cluster_id : num_clusters + atomicAdd(p.next, 1);
            const uint32_t slot = smem_u32(const_cast<int*>(ring + at));
            for (uint32_t r = leader; r <= leader + 1; ++r) {
                st_cluster(map_to_rank(slot, r), tile);
                mbar_arrive_cluster(map_to_rank(ringf_bar(at), r));
            }
            ends += tile >= walk.total;
            if (*abort_flag) break;
        }
    } else if ((warp == 0 || warp == 2) && lane == 0) {
        // ---------------------------------------------------- TMA copies (both CTAs)
        const bool is_a = warp == 0;
        int s = 0, stages = 0;
        uint32_t ph = 0;
        for (int i = 0;; ++i) {
            const int tile = take(i, true);
            if (tile < 0 || *abort_flag) break;
            const TileAt t = walk.at(p, tile);
            const Job& q = p.job[t.job];
            const bool mn = is_a ? q.a_mn : q.b_mn;
            const CUtensorMap* map = &maps.m[is_a ? q.a : q.b][mn];
            // W's rows are the whole vocabulary, a piece starts at v0; dl's columns are the piece's own
            const int r0 = is_a ? t.m * C::kRows + peer * kHalf
                                : t.n * q.width + peer * C::kBRows + (q.b_mn ? 0 : q.v0);
            const int tx = PAIR ? 4 * kAtom : (q.a_rows + q.width) * 128;  // bytes of one step, of both CTAs
            // first summed element; of W, counted from its first row
            const int kb = t.k0 * kStep + (!is_a && q.kind == kDH ? q.v0 : 0);
            for (int ks = 0; ks < t.k_steps; ks += C::kKps) {
                if (!mbar_wait(empty_bar(s), ph ^ 1u, nullptr, kFreeLimit)) {
                    give_up();
                    break;
                }
                ++stages;
                const int nk = min(C::kKps, t.k_steps - ks);
                const uint32_t fb = PAIR ? map_to_rank(full_bar(s), leader) : full_bar(s);
                if (is_a && peer == 0) mbar_expect_tx(full_bar(s), nk * tx);
                for (int j = 0; j < nk; ++j) {
                    const uint32_t dst =
                        is_a ? base + C::kOffA + s * C::kA + j * kAtom : base + C::kOffB + s * C::kB + j * C::kAtomB;
                    const int k = kb + (ks + j) * kStep;
                    if (mn) {
                        tma_load<PAIR>(dst, map, r0, k, fb);
                        tma_load<PAIR>(dst + kBlockBytes, map, r0 + 64, k, fb);
                    } else {
                        tma_load<PAIR>(dst, map, k, r0, fb);
                        if (!PAIR && !is_a) tma_load<PAIR>(dst + q.width * 64, map, k, r0 + q.width / 2, fb);
                    }
                }
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        stages_of[is_a ? 0 : 1] = stages;
    } else if (warp == 1 && lane == 0 && peer == 0) {
        // ------------------------------------------------ MMA issuer (leader only)
        int s = 0, stages = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int tc = 0; ok; ++tc) {
            const int tile = take(tc, true);
            if (tile < 0) break;
            const TileAt t = walk.at(p, tile);
            const Job& q = p.job[t.job];
            const int buf = tc & 1;
            if (!mbar_wait(acce_bar(buf), ((tc >> 1) & 1) ^ 1, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + buf * kTile;
            const uint32_t idesc = make_idesc(C::kRows, q.width, q.a_mn, q.b_mn);
            // 16 summed elements: 32 bytes along a swizzle row, or 16 rows of 128 bytes
            const int astep = q.a_mn ? 2048 >> 4 : 32 >> 4, bstep = q.b_mn ? 2048 >> 4 : 32 >> 4;
            for (int ks = 0; ks < t.k_steps; ks += C::kKps) {
                if (!mbar_wait(full_bar(s), ph, nullptr, p.wait_limit)) {
                    ok = false;
                    break;
                }
                ++stages;
                tc_fence_after();
                const int nk = min(C::kKps, t.k_steps - ks);
                for (int j = 0; j < nk; ++j) {
                    const uint64_t da = sw128_desc(base + C::kOffA + s * C::kA + j * kAtom);
                    const uint64_t db = sw128_desc(base + C::kOffB + s * C::kB + j * C::kAtomB);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma<PAIR>(acc, da + i * astep, db + i * bstep, idesc, (ks + j > 0 || i > 0) ? 1u : 0u);
                }
                tc_commit<PAIR>(empty_bar(s));  // frees stage s in both CTAs
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (ok) tc_commit<PAIR>(accf_bar(buf));
        }
        if (!ok) give_up();
        stages_of[2] = stages;
        tc_commit_local<PAIR>(drain_bar);
        mbar_wait(drain_bar, 0, nullptr);
    } else if (warp >= 4) {
        // ------------------------------------------------- epilogue (both CTAs)
        const int q4 = warp & 3;
        const float scale = p.scale ? *p.scale : 1.0f;
        for (int tc = (warp - 4) >> 2;; tc += 2) {
            const int tile = take(tc, false);  // every lane reads the tile, then one arrives
            __syncwarp();
            if (PAIR && lane == 0) mbar_arrive_cluster(map_to_rank(ringe_bar(tc % kRing), leader));
            const int buf = tc & 1;
            if (__any_sync(0xFFFFFFFFu, tile < 0)) break;
            const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(accf_bar(buf), (tc >> 1) & 1, abort_flag));
            if (!ok) give_up();
            if (!ok || *abort_flag) break;
            tc_fence_after();
            const TileAt t = walk.at(p, tile);
            const Job& q = p.job[t.job];
            const int row = t.m * C::kRows + peer * kHalf + q4 * 32 + lane;
            const int n0 = t.n * q.width;
            const uint32_t acc = tmem + ((uint32_t)(q4 * 32) << 16) + buf * kTile;
            float r[32];
            if (q.kind == kStats) {
                int target = -1;
                if (row < count) {
                    if (p.targets) {
                        const int64_t v = p.targets[row];
                        target = v >= 0 && v < p.vocab ? (int)v : -1;
                    } else {
                        target = p.info[row].target;
                    }
                }
                float m = -INFINITY, sum = 0.0f, hit = 0.0f;
                for (int c = 0; c < q.width; c += 32) {
                    tmem_ld32(acc + c, r);
                    const int at = target - (n0 + c);
                    if (__any_sync(0xFFFFFFFFu, at >= 0 && at < 32)) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (at == i) hit = r[i];
                    }
                    stats_chunk(r, min(q.n - n0, q.width) - c, m, sum);
                }
                if (row < count) {
                    p.part[row * p.ld_part + t.n] = make_float2(m, sum);
                    if (target >= n0 && target < n0 + q.width) p.target_logit[row] = hit;
                }
            } else if (!PAIR) {
                // dl of few tokens: whole rows of the tile (zeros as below), in the last one up to a whole step
                RowInfo info = {0.0f, 0.0f, 0.0f, -1};
                if (row < count) info = p.info[row];
                const int end = (q.n + kStep - 1) / kStep * kStep - n0;
                const int cols = min(q.width, end);
                // In two parts, the second ones' rows stand behind all of the first ones', and the zeros that dW's last
                // step reads behind them both: the rows past the tokens (of the one tile) write those.
                const bool live = row < count;
                uint4* dst = reinterpret_cast<uint4*>(q.dl + (p.fine && !live ? row + count : row) * q.ld_dl + n0);
                uint4* second = reinterpret_cast<uint4*>(q.dl + (live ? row + count : row + kHalf) * q.ld_dl + n0);
                for (int c = 0; c < cols; c += 32) {
                    tmem_ld32(acc + c, r);
                    grad_chunk(r, info, n0 + c, live ? q.n - (n0 + c) : 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c + 8 * i < cols) {
                            const uint4 v =
                                make_uint4(pack_bf16(r[8 * i], r[8 * i + 1]), pack_bf16(r[8 * i + 2], r[8 * i + 3]),
                                           pack_bf16(r[8 * i + 4], r[8 * i + 5]), pack_bf16(r[8 * i + 6], r[8 * i + 7]));
                            dst[c / 8 + i] = v;
                            if (!p.fine) continue;
                            const uint32_t first[4] = {v.x, v.y, v.z, v.w};
                            uint32_t lo[4];
                            const int at = info.target - (n0 + c + 8 * i);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float a = r[8 * i + 2 * j] - __uint_as_float(first[j] << 16);
                                const float b = r[8 * i + 2 * j + 1] - __uint_as_float(first[j] & 0xFFFF0000u);
                                if (at == 2 * j) p.rest[row] = a;
                                if (at == 2 * j + 1) p.rest[row] = b;
                                lo[j] = pack_bf16(a, b);
                            }
                            second[c / 8 + i] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        }
                }
                if (n0 + q.width >= q.n)
                    for (int c = cols; c < end; c += 8) {
                        dst[c / 8] = make_uint4(0, 0, 0, 0);
                        if (p.fine) second[c / 8] = make_uint4(0, 0, 0, 0);
                    }
            } else {
                // a piece's dl whole (zeros beside the valid rows and columns: dH and dW sum over them);
                // dH of the valid rows; rows of dW
                RowInfo info = {0.0f, 0.0f, 0.0f, -1};
                float factor = scale;
                Dest d;
                if (q.kind == kGrad) {
                    if (row < count) info = p.info[row];
                    d = make_dest(q.dl, q.ld_dl, 1 << 30, 1 << 30, false, false, nullptr);
                } else if (q.kind == kDW) {
                    d = make_dest((char*)p.dw + (int64_t)q.v0 * p.ld_dw * (p.dw_f32 ? 4 : 2), p.ld_dw, q.m, q.n, p.dw_f32,
                                  p.accumulate, nullptr);
                } else if (p.dh_acc) {
                    factor = 1.0f;
                    d = make_dest(p.dh_acc + (int64_t)(q.slice0 + t.slice) * p.Tp * p.Kp, p.Kp, count, q.n, true, q.add,
                                  nullptr);
                } else {
                    d = make_dest(p.dh, p.ld_dh, count, q.n, p.dh_f32, false, p.index);
                }
                const Writer out(d, gbase + C::kOffOut + (warp - 4) * 4096, row - lane);
                const bool empty = t.k_steps == 0;  // a sum of nothing: 0, whatever tensor memory holds
                for (int c = 0; c < kTile; c += 32) {
                    tmem_ld32(acc + c, r);
                    if (q.kind == kGrad) {
                        grad_chunk(r, info, q.v0 + n0 + c, row < count ? q.n - (n0 + c) : 0);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = empty ? 0.0f : r[i] * factor;
                    }
                    out.columns(n0, c, r);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(acce_bar(buf), leader));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();  // neither CTA leaves while the other may still use its memory or barriers
    if (__builtin_expect(*abort_flag, 0)) {
        // A wait gave up (both CTAs of a pair know): stages that were filled but not used may still be on their way into
        // either CTA.  They are waited for before any CTA leaves, with a limit, since a stage that only some of the
        // copiers filled never completes.
        if (threadIdx.x == 0 && peer == 0) {
            int most = max(stages_of[0], stages_of[1]);
            if (PAIR)
                for (int i = 0; i < 2; ++i) most = max(most, ld_cluster(map_to_rank(base + C::kOffStages + 4 * i, leader + 1)));
            for (int i = stages_of[2]; i < most; ++i) mbar_wait(full_bar(i % S), (i / S) & 1, nullptr, kDrainLimit);
        }
        __syncthreads();
        if (PAIR) cluster_sync_all();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_free<PAIR>(tmem);
    }
}

// ------------------------------------------------------------ joining tiles
// lse and loss of a row from its tiles, a warp a row: 32 slices of the tiles,
// each in order, then the slices pairwise.
__global__ void __launch_bounds__(256) head_join_kernel(const HeadParams p, int tiles, float z, float* loss, float* lse) {
    griddep_wait();
    griddep_launch();
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= (p.count ? *p.count : p.tokens)) return;
    auto join = [](float2& a, float2 b) {
        const float m = fmaxf(a.x, b.x);
        const float shift = m == -INFINITY ? 0.0f : m * kLog2e;
        a.y = a.y * ex2(fmaf(a.x, kLog2e, -shift)) + b.y * ex2(fmaf(b.x, kLog2e, -shift));
        a.x = m;
    };
    float2 a = make_float2(-INFINITY, 0.0f);
    const float2* part = p.part + row * p.ld_part;
#pragma unroll 4
    for (int t = lane; t < tiles; t += 32) join(a, part[t]);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        join(a, make_float2(__shfl_xor_sync(0xFFFFFFFFu, a.x, o), __shfl_xor_sync(0xFFFFFFFFu, a.y, o)));
    if (lane) return;
    const float l = a.x + logf(a.y);
    int token = row;
    bool valid = true;
    if (p.targets) {
        const int64_t v = p.targets[row];
        valid = v >= 0 && v < p.vocab;
    } else {
        token = p.index[row];
    }
    lse[token] = valid ? l : 0.0f;
    loss[token] = valid ? fmaf(z * l, l, l - p.target_logit[row]) : 0.0f;
}

// dH from the fp32 sums of the packed rows, or their shares in order, and with
// dl in two parts what the first left at the target: a row's columns 256 at a
// time over the grid's second dimension.
__global__ void __launch_bounds__(256) head_dh_kernel(const HeadParams p, int cols) {
    griddep_wait();
    griddep_launch();
    const int row = blockIdx.x;
    if (row >= *p.count) return;
    const float scale = p.scale ? *p.scale : 1.0f;
    const int64_t out = (int64_t)p.index[row] * p.ld_dh, step = p.Tp * p.Kp;
    const float rest = p.fine ? p.rest[row] : 0.0f;
    const __nv_bfloat16* w = p.w + (int64_t)p.info[row].target * p.ldw;
    for (int64_t c = blockIdx.y * 256 + threadIdx.x; c < cols; c += gridDim.y * 256) {
        const float* part = p.dh_acc + row * p.Kp + c;
        float s = 0.0f;
#pragma unroll 8
        for (int i = 0; i < p.shares; ++i) s += part[i * step];
        if (p.fine) s += rest * __bfloat162float(w[c]);
        s *= scale;
        if (p.dh_f32)
            ((float*)p.dh)[out + c] = s;
        else
            ((__nv_bfloat16*)p.dh)[out + c] = __float2bfloat16_rn(s);
    }
}

// ------------------------------------------------------------------- host
int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Regions of the workspace, 256-byte aligned.
struct Plan {
    int64_t Tp, Kp;          // packed rows and columns
    int64_t pieces, piece;   // backward: vocabulary pieces and their width (a multiple of kTile)
    int64_t launches;        // of the product kernel
    int64_t slices;          // backward: shares of a piece's dH
    bool direct;             // forward: tokens in place, none packed
    bool fine;               // backward: dl in two parts
    bool sums;               // backward: dH as fp32 sums first
    int64_t width, tiles;    // columns of a tile of logits; forward: tiles of the vocabulary
    size_t count, next, index, info, packed, part, target, dl[2], rest, acc, total;
};

// Few tokens' logits are computed by single CTAs: a pair's tile costs the same
// for 16 tokens as for 256, and what should bound the call is the reading of W.
// Forward up to half a tile of tokens, which are then read where they lie (16 x
// 32000 x 2048: 45 us in pairs, 31 so).  The tiles' widths decide where its sums
// are joined; with more tokens all widths are the same, so that a row's bits do not
// depend on how many ignored tokens stand among the others.
constexpr int64_t kDirect = kHalf;

// Backward (dl, with the same bits from either).  One or three tiles of 128
// tokens leave half of a pair's last one empty: single CTAs are 3 to 10 %
// faster (the whole pass, in pairs and so: 128 x 32000 x 2048 140 and 131 us,
// 128 x 131072 x 4096 758 and 730, 320 x 32000 x 2048 182 and 170, 384 x 131072 x
// 4096 1118 and 1069).  Two tiles fill a pair, and single CTAs copy W's rows
// twice; what they gain is a fuller last round, which counts less the more
// rounds there are: 256 x 5000 x 2048 62 and 58, x 32000 149 and 146, x 77824
// 285 and 281, x 100000 333 and 333, x 116736 373 and 380, x 131072 411 and 416
// (and 107 and 110 where pairs' tiles are just one round, x 19456).  Four: 512 x
// 65536 x 7168 1056 and 1091.
constexpr int64_t kAloneBack = 3 * kHalf, kAloneVocab = 100000;
bool alone_backward(int64_t T, int64_t V) {
    return T <= kAloneBack && (up(T, kHalf) != 2 * kHalf || V <= kAloneVocab);
}

// Columns of such a tile: all CTAs have as many of them.
int64_t alone_width(int64_t T, int64_t V, int num_sms) {
    const int64_t all = std::max<int64_t>(1, (T + kHalf - 1) / kHalf) * V;
    const int64_t rounds = (all + (int64_t)kAlone * num_sms - 1) / ((int64_t)kAlone * num_sms);
    return std::max<int64_t>(32, up((all + rounds * num_sms - 1) / (rounds * num_sms), 16));
}

// The entry of dl at a token's target, weight (p - 1), dominates the token's
// row, and its rounding to bf16 scales the token's whole gradient by up to
// 2^-8.  Over many tokens these errors average to 0.0017 of the result; of few
// they do not (10 x 12140 x 3200: dh and dw 0.0028 from the exact ones, 0.0017
// of which are the bf16 results' own rounding).  Up to kFine tokens dl is
// therefore kept in two bf16 parts, 16 bits of every entry: dW sums over both
// (twice the summed index, which is still few steps), and dH gets what the
// first part left at the target from head_dh_kernel.  One tile of 128 tokens,
// so that the second parts are rows of the same 256.  It costs 2 % of the pass
// for 16 tokens (16 x 32000 x 2048 124.6 -> 127.1 us), 3 to 10 % for 128 (x
// 32000 x 2048 129.7 -> 136.1, x 131072 x 4096 729 -> 799); second parts for
// tiles of dW with a target only: 130, 136 and 751 us.
bool fine_backward(int64_t T, int64_t pieces) { return T <= kFine && pieces == 1; }

// A piece's dl takes about kPieceBytes.  Wider pieces mean fewer launches,
// longer sums and fewer passes over the fp32 dH; narrower ones a smaller
// workspace, and below 129 MB a dl that L2 holds, which measures no faster: the
// gradients of 4096 x 65536 x 7168 take 7.33, 7.00 and 6.90 ms with 64, 128 and
// 256 MB, of 2047 x 50001 x 2048 (a third ignored) 671, 613 and 610 us.
constexpr int64_t kPieceBytes = 256ll << 20;

// dH has few tiles, each with a long sum, where there are few tokens (16
// tokens, K = 2048: 8 tiles of 500 steps for a vocabulary of 32000).  The sum
// is then shared out so that no tile takes more than half of what a cluster
// takes of the launch, up to kMostShares and 256 MB of fp32 shares.
constexpr int64_t kMostShares = 32;
int64_t dh_slices(int64_t T, int64_t K, int64_t piece, int64_t pieces, int num_sms) {
    const int64_t mt = std::max<int64_t>(1, up(T, kTile) / kTile), vt = piece / kTile, kt = up(K, kTile) / kTile;
    const int64_t ts = up(T, kStep) / kStep, vs = piece / kStep, ks = up(K, kStep) / kStep;
    const int64_t steps = mt * kt * vs + vt * kt * ts + (pieces > 1 ? mt * vt * ks : 0);
    const int64_t share = std::max<int64_t>(8, steps / std::max(1, num_sms / 2) / 2);  // of a cluster, halved
    const int64_t most = std::min<int64_t>(kMostShares, (256ll << 20) / (4 * pieces * mt * kTile * up(K, 8)));
    return std::max<int64_t>(1, std::min((vs + share - 1) / share, most));
}

Plan make_plan(int64_t T, int64_t V, int64_t K, bool back, int num_sms) {
    Plan p = {};
    p.Tp = std::max<int64_t>(up(T, kTile), kTile);
    p.Kp = up(K, 8);
    size_t off = 0;
    auto take = [&](int64_t bytes) {
        const size_t at = off;
        off += (size_t)up(bytes, 256);
        return at;
    };
    if (back) {
        const int64_t want = std::max<int64_t>(kTile, kPieceBytes / (2 * p.Tp) / kTile * kTile);
        p.pieces = (V + want - 1) / want;
        p.piece = up((V + p.pieces - 1) / p.pieces, kTile);
        p.pieces = (V + p.piece - 1) / p.piece;
    }
    p.launches = p.pieces + 1;  // forward: one
    p.count = take(4);
    p.next = take(4 * p.launches);
    p.index = take(4 * p.Tp);
    p.info = take((int64_t)sizeof(RowInfo) * p.Tp);
    p.packed = take(2 * p.Tp * p.Kp);
    if (back) {
        p.width = alone_backward(T, V) && p.pieces == 1 ? alone_width(T, V, num_sms) : kTile;
        p.dl[0] = take(2 * p.Tp * p.piece);
        p.dl[1] = p.pieces > 1 ? take(2 * p.Tp * p.piece) : p.dl[0];
        p.slices = dh_slices(T, K, p.piece, p.pieces, num_sms);
        p.fine = fine_backward(T, p.pieces);
        p.rest = take(4 * p.Tp);
        p.sums = p.pieces > 1 || p.slices > 1 || p.fine;
        p.acc = p.sums ? take(4 * p.Tp * p.Kp * (p.slices > 1 ? p.slices * p.pieces : 1)) : 0;
    } else {
        p.direct = T <= kDirect;
        p.width = p.direct ? alone_width(T, V, num_sms) : kTile;
        p.tiles = (V + p.width - 1) / p.width;
        p.part = take((int64_t)sizeof(float2) * p.Tp * p.tiles);
        p.target = take(4 * p.Tp);
    }
    p.total = off;
    return p;
}

bool bf16_maps(CUtensorMap map[2], const void* ptr, int64_t inner, int64_t outer, int64_t ld, int rows = kHalf) {
    return encode_map_2d(&map[0], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ptr, (uint64_t)inner, (uint64_t)outer,
                         (uint64_t)ld * 2, 64, rows, CU_TENSOR_MAP_SWIZZLE_128B) &&
           encode_map_2d(&map[1], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, ptr, (uint64_t)inner, (uint64_t)outer,
                         (uint64_t)ld * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Clusters that fit the device at once (per device, from the first launch on it).
template <bool PAIR>
int max_clusters(int dev, const cudaLaunchConfig_t& cfg) {
    static DeviceFigure clusters;
    return clusters.get(dev, [&] {
        int n = 0;
        return cudaOccupancyMaxActiveClusters(&n, head_gemm_kernel<PAIR>, &cfg) == cudaSuccess ? n : 0;
    });
}

// By how much the polls of a stage's arrival are lowered, per device.
std::atomic<uint32_t> g_lowered[64];

template <bool PAIR>
cudaError_t run_gemm(const HeadMaps& maps, HeadParams& p, int64_t T, cudaStream_t st) {
    using C = Cfg<PAIR>;
    cudaError_t e = cudaFuncSetAttribute(head_gemm_kernel<PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    constexpr unsigned ctas = PAIR ? 2 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const int most = max_clusters<PAIR>(dev, cfg);
    if (most <= 0) return cudaErrorLaunchOutOfResources;
    p.wait_limit = kWaitLimit - g_lowered[dev].load(std::memory_order_relaxed);
    for (int j = 0; j < p.jobs; ++j) {
        Job& q = p.job[j];
        const int64_t m = q.kind == kDW ? q.m : T, k = q.kind == kDW ? T : q.k;
        q.group = 2 * m * k <= kResidentA ? 1 << 30 : kGroupM;
    }
    int64_t tiles = 0;  // with every token valid; the entry points refuse what would not fit 30 bits
    for (int j = 0; j < p.jobs; ++j) {
        const Job& q = p.job[j];
        tiles += up(q.kind == kDW ? q.m : T, C::kRows) / C::kRows * (up(q.n, q.width) / q.width) * q.slices;
    }
    cfg.gridDim = dim3(ctas * (unsigned)std::max<int64_t>(1, std::min<int64_t>(tiles, most)));
    cfg.numAttrs = st ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, head_gemm_kernel<PAIR>, maps, p);
}

cudaError_t run_pack(const HeadArgs& a, const Plan& pl, bool back, int num_sms, cudaStream_t st) {
    uint8_t* ws = (uint8_t*)a.workspace;
    PackParams p = {};
    p.h = (const __nv_bfloat16*)a.h;
    p.ldh = a.ldh;
    p.targets = a.targets;
    p.T = a.T;
    p.V = a.V;
    p.K = a.K;
    p.Kp = pl.Kp;
    p.packed = (__nv_bfloat16*)(ws + pl.packed);
    p.index = (int*)(ws + pl.index);
    p.info = (RowInfo*)(ws + pl.info);
    p.count = (int*)(ws + pl.count);
    p.next = (int*)(ws + pl.next);
    p.launches = (int)pl.launches;
    p.fine = pl.fine;
    p.loss = a.loss;
    p.lse_out = a.lse;
    p.lse = a.lse;
    p.weight = a.weight;
    p.z = a.z;
    p.dh = a.dh;
    p.ld_dh = a.ld_dh;
    p.dh_f32 = a.dh_f32;
    const auto share = [&](int64_t ctas) { return (a.T + ctas * num_sms - 1) / (ctas * num_sms); };
    p.rows_per_cta = (int)std::max(std::min<int64_t>(kPackRows, std::max<int64_t>(2, share(2))), share(kPackCtas));
    const unsigned grid = (unsigned)std::max<int64_t>(8, (a.T + p.rows_per_cta - 1) / p.rows_per_cta);
    return back ? launch_pdl(head_pack_kernel<true>, dim3(grid), dim3(256), 0, st, p)
                : launch_pdl(head_pack_kernel<false>, dim3(grid), dim3(256), 0, st, p);
}

cudaError_t make_maps(const HeadArgs& a, const Plan& pl, bool back, HeadMaps& maps) {
    uint8_t* ws = (uint8_t*)a.workspace;
    // tokens in place: boxes of the rows there are.  The accumulator rows past them hold whatever shared memory
    // did, and are not looked at; rows that the copy fills with zeros cost time (one token, 32000 x 2048: 37 us with 128 rows, 31 with 8).
    bool ok = (pl.direct ? bf16_maps(maps.m[kOpH], a.h, a.K, a.T, a.ldh, (int)up(a.T, 8))
                         : bf16_maps(maps.m[kOpH], ws + pl.packed, a.K, pl.Tp, pl.Kp)) &&
              bf16_maps(maps.m[kOpW], a.w, a.K, a.V, a.ldw, (int)pl.width / 2);
    for (int i = 0; i < 2; ++i) {
        if (back)
            ok = ok && bf16_maps(maps.m[kOpDl + i], ws + pl.dl[i], pl.piece, pl.Tp, pl.piece);
        else
            maps.m[kOpDl + i][0] = maps.m[kOpDl + i][1] = maps.m[kOpH][0];  // not used
    }
    return ok ? cudaSuccess : cudaErrorInvalidValue;
}

HeadParams make_params(const HeadArgs& a, const Plan& pl) {
    uint8_t* ws = (uint8_t*)a.workspace;
    HeadParams p = {};
    p.count = (const int*)(ws + pl.count);
    p.next = (int*)(ws + pl.next);
    p.index = (const int*)(ws + pl.index);
    p.info = (const RowInfo*)(ws + pl.info);
    p.part = (float2*)(ws + pl.part);
    p.target_logit = (float*)(ws + pl.target);
    p.ld_part = pl.tiles;
    p.fine = pl.fine;
    p.rest = (float*)(ws + pl.rest);
    p.w = (const __nv_bfloat16*)a.w;
    p.ldw = a.ldw;
    p.dh_acc = pl.sums ? (float*)(ws + pl.acc) : nullptr;
    p.Kp = pl.Kp;
    p.scale = a.scale;
    p.dh = a.dh;
    p.ld_dh = a.ld_dh;
    p.dh_f32 = a.dh_f32;
    p.dw = a.dw;
    p.ld_dw = a.ld_dw;
    p.dw_f32 = a.dw_f32;
    p.accumulate = a.accumulate;
    p.Tp = pl.Tp;
    p.shares = pl.slices > 1 ? (int)(pl.slices * pl.pieces) : 1;
    for (Job& q : p.job) {
        q.a_rows = kHalf;
        q.width = kTile;
        q.slices = 1;
    }
    if (pl.direct) {
        p.count = nullptr;
        p.tokens = (int)a.T;
        p.targets = a.targets;
        p.vocab = (int)a.V;
        p.next = nullptr;
        p.job[0].a_rows = (int)up(a.T, 8);
        p.job[0].width = (int)pl.width;
    }
    return p;
}

}  // namespace

size_t head_loss_bytes(int64_t T, int64_t V, int64_t K, int num_sms) { return make_plan(T, V, K, false, num_sms).total; }
size_t head_loss_backward_bytes(int64_t T, int64_t V, int64_t K, int num_sms) {
    return make_plan(T, V, K, true, num_sms).total;
}

cudaError_t launch_head_loss(const HeadArgs& a, int num_sms, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const Plan pl = make_plan(a.T, a.V, a.K, false, num_sms);
    HeadMaps maps;
    cudaError_t e = make_maps(a, pl, false, maps);
    if (e == cudaSuccess && !pl.direct) e = run_pack(a, pl, false, num_sms, st);
    if (e != cudaSuccess) return e;
    HeadParams p = make_params(a, pl);
    p.jobs = 1;
    p.job[0].kind = kStats;
    p.job[0].a = kOpH;
    p.job[0].b = kOpW;
    p.job[0].n = (int)a.V;
    p.job[0].k = (int)a.K;
    e = pl.direct ? run_gemm<false>(maps, p, a.T, st) : run_gemm<true>(maps, p, a.T, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(head_join_kernel, dim3((unsigned)((a.T + 7) / 8)), dim3(256), 0, st, p, (int)pl.tiles, a.z, a.loss,
                      a.lse);
}

cudaError_t launch_head_loss_backward(const HeadArgs& a, int num_sms, cudaStream_t st) {
    const Plan pl = make_plan(a.T, a.V, a.K, true, num_sms);
    uint8_t* ws = (uint8_t*)a.workspace;
    HeadMaps maps;
    cudaError_t e = make_maps(a, pl, true, maps);
    if (e == cudaSuccess) e = run_pack(a, pl, true, num_sms, st);
    auto width = [&](int64_t i) { return (int)std::min(pl.piece, a.V - i * pl.piece); };
    for (int64_t i = -1; i < pl.pieces && e == cudaSuccess; ++i) {
        HeadParams p = make_params(a, pl);
        if (i >= 0 && a.dh) {  // dH and dW of piece i
            Job& h = p.job[p.jobs++];
            h.kind = kDH;
            h.a = kOpDl + (int)(i & 1);
            h.b = kOpW;
            h.b_mn = 1;
            h.n = (int)a.K;
            h.k = width(i);
            h.v0 = (int)(i * pl.piece);
            h.add = i > 0 && pl.slices == 1;
            h.slices = (int)pl.slices;
            h.per = (int)((up(width(i), kStep) / kStep + pl.slices - 1) / pl.slices);
            h.slice0 = pl.slices > 1 ? (int)(i * pl.slices) : 0;
        }
        if (i >= 0 && a.dw) {
            Job& w = p.job[p.jobs++];
            w.kind = kDW;
            w.a = kOpDl + (int)(i & 1);
            w.b = kOpH;
            w.a_mn = w.b_mn = 1;
            w.m = width(i);
            w.n = (int)a.K;
            w.v0 = (int)(i * pl.piece);
        }
        if (i + 1 < pl.pieces) {  // dl of the next piece
            Job& g = p.job[p.jobs++];
            g.kind = kGrad;
            g.a = kOpH;
            g.b = kOpW;
            g.n = width(i + 1);
            g.k = (int)a.K;
            g.v0 = (int)((i + 1) * pl.piece);
            g.dl = (__nv_bfloat16*)(ws + pl.dl[(i + 1) & 1]);
            g.ld_dl = pl.piece;
        }
        p.next += i + 1;
        // the longest tiles first, so that the launch ends on short ones
        std::sort(p.job, p.job + p.jobs, [&](const Job& x, const Job& y) {
            return (x.kind == kDW ? a.T : x.k / x.slices) > (y.kind == kDW ? a.T : y.k / y.slices);
        });
        const bool alone = i < 0 && pl.width < kTile;
        if (alone) p.job[0].width = (int)pl.width;
        if (p.jobs) e = alone ? run_gemm<false>(maps, p, a.T, st) : run_gemm<true>(maps, p, a.T, st);
    }
    if (e == cudaSuccess && a.dh && pl.sums)
        e = launch_pdl(head_dh_kernel, dim3((unsigned)a.T, (unsigned)std::min<int64_t>((a.K + 255) / 256, 65535)), dim3(256),
                       0, st, make_params(a, pl), (int)a.K);
    return e;
}

cudaError_t head_error_read_clear(int* value) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_head_error, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && *value) e = cudaMemcpyToSymbol(g_head_error, &zero, sizeof(int));
    return e;
}

cudaError_t set_head_wait_limit(uint32_t polls) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    g_lowered[dev].store(kWaitLimit - std::min(polls, kWaitLimit), std::memory_order_relaxed);
    return cudaSuccess;
}

cudaError_t preload_head_kernels() {
    cudaFuncAttributes at;
    cudaFuncGetAttributes(&at, head_pack_kernel<false>);
    cudaFuncGetAttributes(&at, head_pack_kernel<true>);
    cudaFuncGetAttributes(&at, head_gemm_kernel<true>);
    cudaFuncGetAttributes(&at, head_gemm_kernel<false>);
    cudaFuncGetAttributes(&at, head_dh_kernel);
    return cudaFuncGetAttributes(&at, head_join_kernel);
}

}  // namespace ufp4
