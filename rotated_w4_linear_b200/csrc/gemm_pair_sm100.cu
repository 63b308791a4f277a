// Contraction on pairs of SMs (tcgen05, cta_group::2) above 16 tokens, for the
// layer with an activation and a residual and for the gated up-projection:
//   Y^T tile [256 rows][BN tokens] = w_hat * X'^T, then the epilogue.
//
// Two CTAs of a cluster share a tile: each keeps its own 128 rows of w_hat in
// its tensor memory and holds half of the tokens in shared memory, and one
// MMA (M = 256, N = BN, K = 16) reads both halves. Two forms:
//   BN = 256 (many tiles, of up to 256 tokens; bound by the tensor cores and
//     their power): persistent; a cluster of one pair walks the tiles cid, cid + clusters,
//     ... (row tiles first, so that the clusters at work share their tokens)
//     and its roles run ahead of each other across tiles;
//   BN = 64, 128 (17 to 128 tokens, and more where the tiles of 256 would be
//     few; bound by the weights' way to the tensor cores): one tile per cluster, whose one to four pairs split the channels,
//     since the row tiles alone would leave most SMs idle; the pairs' sums
//     meet through distributed shared memory in a fixed order.
// Per CTA, twenty warps (BN < 256: twenty-one):
//   warps 0, 19 (20)  TMA producers: per stage of 128 channels the CTA's half of
//               the tokens of X' (two 64-channel boxes, 128-byte swizzle), and
//               the int4 codes of its 8 row blocks with their scales and zeros,
//               whose ring is deeper; both CTAs' loads of X' complete on the
//               leader's barrier of the stage;
//   warps 3-10 (BN < 256: 3-14)  dequantise (w_hat = fp16((q - z) s), as the
//               other kernels do) into a ring of tensor-memory stages: two
//               (three) groups of four warps take turns, a warp takes one
//               quarter of the rows of its group's stage;
//   warp 2      gate: one lane reports to the pair's leader when its CTA's w_hat
//               of a stage, and in the leader X', is there;
//   warp 1      tensor memory; in the leader the warp issues the MMAs (A from
//               tensor memory, B from shared memory) of a stage that both
//               gates have reported, and commits it back to both CTAs;
//   warps 11-18 epilogue, BN = 256: a warp takes one quarter of the rows and
//               one half of the tokens, 64 tokens at a time from tensor memory
//               into registers (after the second 64 the accumulator is free
//               for the next tile), then through a 32-token buffer of its own
//               in shared memory, where the residual has arrived by TMA, to a
//               TMA store. BN < 256: warps 3-18 put the fp32 sums into shared
//               memory (the rings' space), and after a cluster barrier all
//               warps add the pairs' sums, apply the epilogue and store.
// All waits are bounded (sm100.cuh); a wait that runs out raises the CTA's
// abort flag, every role stops, what was issued is drained, and the cluster's
// CTAs meet at the last barrier.
//
// A stage (128 rows x 128 channels x 256 tokens per CTA) needs 1024 SM cycles
// of the tensor cores. On the way (4096 -> 28672): 1766 with a cluster-scope
// release by each dequantisation warp, 1290 with one reporter per CTA, 1191
// with the MMAs issued from a converged warp; loads issued the same way and
// the dequantisation in groups of four warps took another 12% off the time,
// which is then the power limit's: 1455 us for 4096 -> 2 x 14336 at 8192 tokens
// (1320 TFLOP/s at 1.2-1.35 GHz), 339 us and the tensor pipe 86% busy at 2048.
// BN = 64: 14336 -> 4096 at 64 tokens 19.8-20.2 us (one CTA per tile, unsplit: 94).
//
// A token's result does not depend on its place in the batch: the order of the
// channels goes by the row tile and the split alone.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "common.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "pair_plan.h"
#include "sm100.cuh"

namespace paro {

namespace {

constexpr uint32_t kWCodes = 8 * 1024;                  // 8 row blocks x 128 channels of codes
constexpr uint32_t kWScales = 8 * 64;                   // 8 row blocks x up to 2 groups x 8 words
constexpr uint32_t kWStage = kWCodes + kWScales + 128;  // zeros: 8 row blocks x 2 groups x 8 bytes
constexpr uint32_t kOutBuf = 32 * 64;                   // 32 tokens x 32 rows of fp16: two for each epilogue warp

// Rings and shared memory for a tile of BN tokens. Tensor memory: BN columns
// of fp32 sums, 64 columns per w_hat stage (as many stages as fit 512
// columns, and no more than the ring of X').
template <int BN>
struct PairCfg {
    static constexpr bool kSplit = BN < 256;
    // 20 warps, 21 in the split form (a second producer of the weights): one
    // warp more leaves 80 registers a thread, which the 256-token form's
    // epilogue does not fit
    static constexpr int kWProducers = kSplit ? 2 : 1, kThreads = 32 * (19 + kWProducers);
    static constexpr int kXStages = kSplit ? 6 : 4, kWStages = kSplit ? 12 : 6;
    // Dequantisation: groups of warps that take turns at the stages. A slot's
    // uses must all be one group's, for its waits by phase parity.
    static constexpr int kGroups = kSplit ? 3 : 2;
    static_assert(kXStages % kGroups == 0 && kWStages % kGroups == 0, "every slot belongs to one group");
    static constexpr uint32_t kHalfX = BN / 2 * 128;    // BN / 2 tokens x 64 channels
    static constexpr uint32_t kXStage = 2 * kHalfX;
    static constexpr uint32_t kOut = kSplit ? 0 : 16 * kOutBuf;
    static constexpr uint32_t kRings = kXStages * kXStage + kOut + kWStages * kWStage;
    static constexpr uint32_t kSums = kSplit ? BN * 128 * 4 : 0;       // in the rings' space
    static constexpr uint32_t kBody = kRings > kSums ? kRings : kSums;
    static constexpr int kBars = 4 * kXStages + 2 * kWStages + 3 + 16;
    // Never less than 200 KB: the kernel takes all of an SM's tensor memory, so
    // a second kernel that wants some must not share the SM with it (two that
    // each held one SM of a pair would wait for each other)
    static constexpr size_t kUsed = 1024 + (size_t)kBody + 8 * kBars + 16;
    static constexpr size_t kSmem = kUsed > 200 * 1024 ? kUsed : 200 * 1024;
    static_assert(kSmem + kLeastTmemSmem + 2 * kCtaReservedBytes > kSmSharedBytes,
                  "a second kernel with tensor memory would fit on the SM");
    static_assert(BN + 64 * kXStages <= 512, "tensor memory");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};
struct PairArgs {
    int T, out, nk;             // nk: 128-channel stages
    int mt, ntiles;             // 256-row tiles; tiles in all
    int bn;                     // tokens per tile: BN, or for BN = 256 a multiple of 32 up to it
    int pairs;                  // pairs per cluster (BN < 256: they split the channels)
    int width;                  // columns of Y (out, or out / 2 for the gated epilogue)
    int gs;                     // quantisation groups per 128 channels (1, or 2 for group 64)
    int act, has_res;
    const __half* bias;
    const __half* residual;     // BN < 256: read with plain loads
    __half* Y;                  // BN < 256: written with plain stores
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive_wait() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Without memory ordering (the readers' values are in use already): a release
// would also wait for this CTA's stores of Y.
__device__ __forceinline__ void cluster_arrive_wait_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrive at a barrier of the cluster's other CTA. Relaxed: what it orders is
// tensor memory alone (written with tcgen05.st, read by the MMA), which goes by
// the tcgen05 fences on both sides. A release at cluster scope costs about 900
// cycles.
__device__ __forceinline__ void mbar_arrive_other(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Wait for arrivals and loads of both CTAs: what either CTA's TMA wrote before
// it completed on this barrier is visible to what the warp does next.
__device__ __forceinline__ bool mbar_try_wait_pair(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_pair(uint32_t bar, uint32_t parity, unsigned int fault,
                                               volatile uint32_t* abort) {
    if (mbar_try_wait_pair(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_pair(bar, parity)) return true;
        if ((it & 255u) == 0) {
            if (*abort) return false;
            if (global_ns() - t0 > kWaitLimitNs) {
                atomicCAS(&g_paro_fault, 0u, fault);
                *abort = 1u;
                return false;
            }
        }
    }
}
// 2-D TMA tile load into this CTA's shared memory whose bytes complete on a
// barrier of either CTA of the pair (`bar` is a cluster address). No multicast.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {   // one warp of each CTA
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void umma_f16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// True in one lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// Arrive on `bar` of the CTAs in `mask` once every MMA issued so far by this thread has completed.
__device__ __forceinline__ void umma_commit_pair(uint32_t bar, uint16_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"(mask) : "memory");
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, float v) {
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(__half_as_ushort(__float2half_rn(v))) : "memory");
}
__device__ __forceinline__ float lds16(uint32_t addr) {
    uint16_t h;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(h) : "r"(addr) : "memory");
    return __half2float(__ushort_as_half(h));
}

// 32 tokens of one accumulator row per thread: the sums become fp16 in the
// warp's buffer [token][32 rows], over the residual where there is one.
struct PairAct {
    const uint32_t* r;
    float b;
    uint32_t at;                // this row in the buffer's first token (64 bytes per token)
    bool has_res;
    template <int ACT>
    __device__ __forceinline__ void run() const {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            float v = act_fn<ACT>(__uint_as_float(r[j]) + b);
            if (has_res) v += lds16(at + j * 64);
            sts16(at + j * 64, v);
        }
    }
};
// Gate rows (lanes with bit 3 clear) and up rows (8 lanes on) trade columns:
// of tokens t, t + 1 the gate lane finishes t, the up lane t + 1. Buffer
// [token][16 channels], 32 bytes per token.
struct PairGated {
    const uint32_t* r;
    float b;                    // this row's own bias
    uint32_t at;                // this lane's channel in the buffer's first token (up lanes: second token)
    bool up;
    template <int ACT>
    __device__ __forceinline__ void run() const {
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            const float v0 = __uint_as_float(r[j]) + b, v1 = __uint_as_float(r[j + 1]) + b;
            const float other = __shfl_xor_sync(0xffffffffu, up ? v0 : v1, 8);
            sts16(at + j * 32, act_fn<ACT>(up ? other : v0) * (up ? v1 : other));
        }
    }
};

// BN < 256: the pairs' sums of this CTA's rows, added in pair order, to the
// output: tokens [BN pair / pairs, BN (pair + 1) / pairs) of the tile, four
// rows (gated: four gate and four up rows) of one token per thread and step.
// A CTA whose rows or tokens lie outside takes no part.
template <int BN, int EPI>
__device__ __forceinline__ void split_epilogue(const PairArgs& a, uint32_t sums, int rb0, int n0, uint32_t rank,
                                               int pair, int pairs) {
    constexpr int kFours = EPI == kEpiGated ? 16 : 32;     // fours per token
    const int t0 = BN * pair / pairs, t1 = min(a.T - n0, BN * (pair + 1) / pairs);
    const int c0 = EPI == kEpiGated ? rb0 * 8 : rb0 * 16;
    for (int i = threadIdx.x; i < (t1 - t0) * kFours; i += PairCfg<BN>::kThreads) {
        const int t = t0 + i / kFours, k = i % kFours;
        // gated: the k-th four gate rows sit in row block k / 2, their up rows eight further on
        const int r = EPI == kEpiGated ? (k >> 1) * 16 + (k & 1) * 4 : 4 * k;
        const int c = c0 + 4 * k;
        if (c >= a.width) continue;
        const uint32_t at = sums + (uint32_t)(t * 128 + r) * 4;
        float4 v[kMaxPairs], u[kMaxPairs];
#pragma unroll
        for (int x = 0; x < kMaxPairs; ++x)
            if (x < pairs) {
                const uint32_t from = map_to_rank(at, 2 * x + rank);
                v[x] = ld_cluster_f4(from);
                if (EPI == kEpiGated) u[x] = ld_cluster_f4(from + 32);
            }
        auto sum = [&](const float4 (&w)[kMaxPairs], int bias_at) {
            float4 s = w[0];
#pragma unroll
            for (int x = 1; x < kMaxPairs; ++x)
                if (x < pairs) {
                    s.x += w[x].x;
                    s.y += w[x].y;
                    s.z += w[x].z;
                    s.w += w[x].w;
                }
            if (a.bias) {
                s.x += __half2float(a.bias[bias_at]);
                s.y += __half2float(a.bias[bias_at + 1]);
                s.z += __half2float(a.bias[bias_at + 2]);
                s.w += __half2float(a.bias[bias_at + 3]);
            }
            return s;
        };
        float4 y = sum(v, c);
        y = make_float4(act_any(y.x, a.act), act_any(y.y, a.act), act_any(y.z, a.act), act_any(y.w, a.act));
        const size_t to = (size_t)(n0 + t) * a.width + c;
        if (EPI == kEpiGated) {
            const float4 w = sum(u, a.width + c);
            y = make_float4(y.x * w.x, y.y * w.y, y.z * w.z, y.w * w.w);
        } else if (a.residual) {
            const uint2 h = *reinterpret_cast<const uint2*>(a.residual + to);
            const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&h.x));
            const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&h.y));
            y = make_float4(y.x + lo.x, y.y + lo.y, y.z + hi.x, y.w + hi.y);
        }
        *reinterpret_cast<uint2*>(a.Y + to) = make_uint2(pack_half2(y.x, y.y), pack_half2(y.z, y.w));
    }
}

// A ring position: slot and use count of the i-th item, advanced one by one.
template <int N>
struct RingPos {
    int slot = 0;
    uint32_t use = 0;           // uses of this slot before the current one
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            ++use;
        }
    }
};

}  // namespace

template <int BN, int EPI>
__global__ void __launch_bounds__(PairCfg<BN>::kThreads, 1)
gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                 const __grid_constant__ CUtensorMap tm_s, const __grid_constant__ CUtensorMap tm_z,
                 const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_r,
                 const PairArgs a) {
    using C = PairCfg<BN>;
    constexpr int kXStages = C::kXStages, kWStages = C::kWStages;
    constexpr uint32_t kHalfX = C::kHalfX, kXStage = C::kXStage;
    constexpr uint32_t kTokenBytes = EPI == kEpiGated ? 32 : 64;       // one token of an epilogue warp's buffer
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sX = smem_addr(smem), sOut = sX + kXStages * kXStage, sW = sOut + C::kOut;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBody);
    const uint32_t xfull0 = smem_addr(bars), free0 = xfull0 + 8 * kXStages, afull0 = free0 + 8 * kXStages;
    const uint32_t wfull0 = afull0 + 8 * kXStages, wfree0 = wfull0 + 8 * kWStages;
    const uint32_t accfull = wfree0 + 8 * kWStages, accfree = accfull + 8, fin = accfree + 8, rfull0 = fin + 8;
    const uint32_t go0 = rfull0 + 16 * 8;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + C::kBars);
    volatile uint32_t* abort = tslot + 1;

    const int bn = C::kSplit ? BN : a.bn;
    const uint32_t idesc = umma_idesc_f16(256, bn);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_rank(), rank = crank & 1;           // CTA of the cluster, of the pair
    const uint16_t both = (uint16_t)(3u << (crank & ~1u));             // the pair's CTAs
    // The channel stages of this pair, walked from a different one in every
    // row tile, so that concurrent requests spread over the memory channels.
    const int pair = C::kSplit ? (int)(crank >> 1) : 0, pairs = C::kSplit ? a.pairs : 1;
    const int k0 = a.nk * pair / pairs, nk = a.nk * (pair + 1) / pairs - k0;
    const int nclusters = gridDim.x / (2 * pairs);
    const int first_tile = blockIdx.x / (2 * pairs);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kXStages; ++s) {
            mbar_init(xfull0 + 8 * s, 1);                 // leader: both CTAs' halves of X' (the other CTA's is not used)
            mbar_init(free0 + 8 * s, 1);                  // the MMAs on X' stage and w_hat stage s are done
            mbar_init(afull0 + 8 * s, 4);                 // the dequantisation warps of one group
            mbar_init(go0 + 8 * s, 2);                    // leader: both CTAs' gates
        }
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(wfull0 + 8 * s, 1);
            mbar_init(wfree0 + 8 * s, 4);
        }
        mbar_init(accfull, 1);
        mbar_init(accfree, 8);                            // this CTA's epilogue warps have the sums
        mbar_init(fin, 1);
        for (int r = 0; r < 16; ++r) mbar_init(rfull0 + 8 * r, 1);
        *abort = 0u;
        mbar_fence_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_s);
        tma_prefetch_desc(&tm_z);
        tma_prefetch_desc(&tm_y);
        if (EPI == kEpiAct) tma_prefetch_desc(&tm_r);
    }
    if (warp == 1) tmem_alloc_pair(smem_addr(tslot), 512);
    tc_fence_before();
    __syncthreads();
    // The next kernel's CTAs may take SMs as this grid's leave them; it reads
    // nothing of ours before this grid is complete. Not before every CTA has its
    // tensor memory: a dependent that took some of an SM's first would wait for
    // this grid, and this grid for it.
    asm volatile("griddepcontrol.launch_dependents;");
    cluster_arrive_wait();                                // the other CTA's barriers exist too
    tc_fence_after();
    const uint32_t tbase = *tslot;
    const uint32_t tA = tbase + BN;                       // w_hat stages after the accumulator columns
    // X' is written by the rotation grid launched just before this one
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // tile -> row blocks of this CTA, first token, first channel stage (of k0 .. k0 + nk - 1)
    auto row_block0 = [&](int tile) { return ((tile % a.mt) * 2 + (int)rank) * 8; };
    auto token0 = [&](int tile) { return tile / a.mt * bn; };
    auto kstart = [&](int tile) { return k0 + (int)((((uint32_t)(tile % a.mt) * 0x9E3779B1u) >> 16) % (uint32_t)nk); };
    auto knext = [&](int kb) { return kb + 1 == k0 + nk ? k0 : kb + 1; };

    if (warp == 0 || warp >= 19) {
        // ---- TMA producers: X' (warp 0), weights (warp 19; BN < 256: warps 19
        // and 20 in turns, a stage's three loads and waits take one warp 650
        // cycles). As with the MMAs, the whole warp walks the stages and one
        // elected lane issues.
        const bool xs = warp == 0;
        const int w0 = xs ? 0 : warp - 19, step = xs ? 1 : C::kWProducers;
        static_assert(kWStages % C::kWProducers == 0, "every slot belongs to one warp");
        RingPos<kXStages> px;
        RingPos<kWStages> pw;
        if (w0) pw.next();
        uint32_t mine = 0;                                // loads issued by this warp
        const uint32_t xfull_leader0 = map_to_rank(xfull0, crank & ~1u);
        int ahead = w0;                                   // stages to the warp's next one, over tile borders
        bool ok = true;
        for (int tile = first_tile; ok && tile < a.ntiles; tile += nclusters) {
            const int rb0 = row_block0(tile), n0 = token0(tile) + bn / 2 * (int)rank;
            int i = ahead, kb = kstart(tile) + ahead;
            if (kb >= k0 + nk) kb -= nk;
            for (; i < nk; i += step) {
                const int slot = xs ? px.slot : pw.slot;
                const uint32_t use = xs ? px.use : pw.use;
                ok = use == 0 || mbar_wait((xs ? free0 : wfree0) + 8 * slot, (use - 1) & 1, kFaultGemmPair + kFaultTmaWait, abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (xs) {
                    // The leader expects the bytes of both CTAs. The other CTA's
                    // may come first: the phase stays open until the leader's
                    // arrival, and the slot's next loads wait for the MMAs of
                    // these (free), so no bytes count in a later phase.
                    const uint32_t bar = xfull_leader0 + 8 * slot, dst = sX + slot * kXStage;
                    if (elect_one()) {
                        if (rank == 0) mbar_arrive_expect_tx(xfull0 + 8 * slot, 2 * (uint32_t)bn * 128);
                        tma_load_2d_pair(dst, &tm_x, kb * 128, n0, bar);
                        tma_load_2d_pair(dst + kHalfX, &tm_x, kb * 128 + 64, n0, bar);
                    }
                    px.next();
                } else {
                    const uint32_t bar = wfull0 + 8 * slot, dst = sW + slot * kWStage;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(bar, kWCodes + 8 * 32 * a.gs + 128);
                        tma_load_2d(dst, &tm_w, kb * 256, rb0, bar);
                        tma_load_2d(dst + kWCodes, &tm_s, kb * 8 * a.gs, rb0, bar);
                        tma_load_2d(dst + kWCodes + kWScales, &tm_z, (a.gs == 2 ? kb : kb >> 1) * 16, rb0, bar);
                    }
#pragma unroll
                    for (int e = 0; e < C::kWProducers; ++e) pw.next();
                }
                __syncwarp();
                ++mine;
                kb += step;
                if (kb >= k0 + nk) kb -= nk;
            }
            ahead = i - nk;
        }
        if (*abort) {   // drain: every issued load must land before the CTA exits
            if (xs) {
                // the barrier that counts this CTA's X' also counts the other
                // CTA's, which may have stopped short: wait out the limit, far
                // longer than a load takes
                const uint64_t t0 = global_ns();
                while (mine > 0 && global_ns() - t0 <= kWaitLimitNs) __nanosleep(100000);
            } else {
                // the j-th load of this warp went to slot (w0 + step j) mod N
                const int per = kWStages / step;
                for (int t = 0; t < per; ++t) {
                    const uint32_t uses = (mine + (uint32_t)(per - 1 - t)) / (uint32_t)per;   // of its t-th slot
                    if (uses > 0)
                        mbar_wait(wfull0 + 8 * (w0 + step * t), (uses - 1) & 1, kFaultGemmPair + kFaultDrainWait, nullptr);
                }
            }
        }
    } else if (warp == 2) {
        if (lane == 0) {
            // ---- gate: one report per stage and CTA to the leader's MMA warp,
            // which then looks at one barrier instead of three (a look takes
            // about 100 cycles): the other CTA's that its w_hat is there, the
            // leader's that its own w_hat and both halves of X' are (4096 ->
            // 28672 at 64 tokens 36.7 us; with the MMA warp looking at X' too 38.3)
            const uint32_t go_leader0 = map_to_rank(go0, crank & ~1u);
            RingPos<kXStages> p;
            uint32_t tiles = 0;
            bool ok = true;
            for (int tile = first_tile; ok && tile < a.ntiles; tile += nclusters, ++tiles) {
                // the sums of the tile before are out of this CTA's tensor memory
                if (tiles > 0) ok = mbar_wait(accfree, (tiles - 1) & 1, kFaultGemmPair + kFaultMmaWait, abort);
                for (int i = 0; ok && i < nk; ++i, p.next()) {
                    ok = (rank != 0 || mbar_wait_pair(xfull0 + 8 * p.slot, p.use & 1, kFaultGemmPair + kFaultMmaWait, abort)) &&
                         mbar_wait(afull0 + 8 * p.slot, p.use & 1, kFaultGemmPair + kFaultMmaWait, abort);
                    if (!ok) break;
                    tc_fence_after();
                    tc_fence_before();
                    if (rank == 0) mbar_arrive(go0 + 8 * p.slot);      // release: X' goes with it
                    else mbar_arrive_other(go_leader0 + 8 * p.slot);
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            // ---- MMA issuer. The whole warp walks the stages, so that the
            // operands' addresses stay in uniform registers, and one elected
            // lane issues (with the loop inside a one-lane branch the eight
            // MMAs of a stage took 550 cycles to issue, and the tensor cores
            // idled a fifth of the time).
            RingPos<kXStages> p;
            bool ok = true;
            for (int tile = first_tile; ok && tile < a.ntiles; tile += nclusters) {
                for (int i = 0; i < nk; ++i, p.next()) {
                    const int s = p.slot;
                    ok = __all_sync(0xffffffffu, mbar_wait_pair(go0 + 8 * s, p.use & 1, kFaultGemmPair + kFaultMmaWait, abort));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t b = umma_desc_sw128_kmajor(sX + s * kXStage);
                    const uint32_t w = tA + s * 64;
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)     // two 64-channel boxes of four MMAs each
                            umma_f16_ts_pair(tbase, w + kk * 8, b + (uint64_t)((kk >> 2) * (int)(kHalfX >> 4) + (kk & 3) * 2), idesc,
                                             i + kk > 0 ? 1u : 0u);
                        umma_commit_pair(free0 + 8 * s, both);
                    }
                    __syncwarp();
                }
                if (ok && elect_one()) umma_commit_pair(accfull, both);
                __syncwarp();
            }
            if (elect_one()) umma_commit_pair(fin, both); // always: arrives once every MMA issued above has completed
            __syncwarp();
        }
    } else if (C::kSplit ? warp < 19 : warp < 11) {
        // ---- dequantisation: groups of four warps take turns at the stages,
        // each warp a quarter of the rows of its stage, so that a stage's waits
        // are paid once for its 16 KB of w_hat
        const int qw = warp & 3;                          // tensor-memory lanes 32 qw .. 32 qw + 31
        const int group = (warp - 3) >> 2;
        const int g = lane >> 2;
        RingPos<kXStages> p;
        RingPos<kWStages> pw;
        bool ok = true;
        for (int e = 0; e < group; ++e) p.next(), pw.next();
        int ahead = group;                                // stages to the group's next one, over tile borders
        for (int tile = first_tile; ok && group < C::kGroups && tile < a.ntiles; tile += nclusters) {
            int i = ahead, kb = kstart(tile) + ahead;
            if (kb >= k0 + nk) kb -= nk;
            for (; i < nk; i += C::kGroups) {
                const int s = p.slot;
                // the tensor-memory stores below are warp-collective: the whole
                // warp goes on only if every lane saw the stage arrive
                ok = mbar_wait(wfull0 + 8 * pw.slot, pw.use & 1, kFaultGemmPair + kFaultDequantWait, abort) && !*abort;
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                const uint32_t src = sW + pw.slot * kWStage;
                const bool two = a.gs == 2;               // a scale and a zero for each half of the channels
                uint4 wv[2][2];                           // [half][row block of the two]
                uint32_t sw[2][2], zb[2][2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int rbl = 2 * qw + r;
                    const uint32_t sc = src + kWCodes + (rbl * a.gs) * 32 + g * 4;
                    const uint32_t z = src + kWCodes + kWScales + rbl * 16 + g;
                    wv[0][r] = lds128(src + rbl * 1024 + lane * 16);
                    wv[1][r] = lds128(src + rbl * 1024 + 512 + lane * 16);
                    sw[0][r] = lds32(sc);
                    zb[0][r] = lds8(z + (two ? 0 : (kb & 1) * 8));
                    if (two) {
                        sw[1][r] = lds32(sc + 32);
                        zb[1][r] = lds8(z + 8);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(wfree0 + 8 * pw.slot);
                ok = p.use == 0 || mbar_wait(free0 + 8 * s, (p.use - 1) & 1, kFaultGemmPair + kFaultDequantWait, abort);
                if (!__all_sync(0xffffffffu, ok && !*abort)) { ok = false; break; }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t sc0, sc1, regs[16];
                    scale_pairs(sw[0][r], sc0, sc1);
                    Zero2 zc = zero_consts(zb[0][r]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h == 1 && two) {
                            scale_pairs(sw[1][r], sc0, sc1);
                            zc = zero_consts(zb[1][r]);
                        }
                        dequant_word(wv[h][r].x, zc, sc0, sc1, regs + 0);
                        dequant_word(wv[h][r].y, zc, sc0, sc1, regs + 4);
                        dequant_word(wv[h][r].z, zc, sc0, sc1, regs + 8);
                        dequant_word(wv[h][r].w, zc, sc0, sc1, regs + 12);
                        tmem_st_16x256b_x4(tA + s * 64 + h * 32 + ((uint32_t)(32 * qw + 16 * r) << 16), regs);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(afull0 + 8 * s);
#pragma unroll
                for (int e = 0; e < C::kGroups; ++e) {
                    kb = knext(kb);
                    p.next();
                    pw.next();
                }
            }
            ahead = i - nk;
        }
        if (C::kSplit) {
            // ---- the pair's sums into shared memory, fp32 [token][128 rows],
            // in the rings' space: every load and MMA of this CTA is done with
            // it. A warp takes its quarter of the rows of a quarter of the tokens.
            const int quarter = (warp - 3) >> 2;
            ok = mbar_wait(accfull, 0, kFaultGemmPair + kFaultEpilogueWait, abort) && !*abort;
            if (__all_sync(0xffffffffu, ok)) {
                tc_fence_after();
                const uint32_t at = sX + (uint32_t)(quarter * (BN / 4) * 128 + 32 * qw + lane) * 4;
#pragma unroll
                for (int c = 0; c < BN / 4; c += 16) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(tbase + ((uint32_t)(32 * qw) << 16) + quarter * (BN / 4) + c, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + (uint32_t)(c + j) * 512), "r"(r[j]) : "memory");
                }
            }
        }
    } else {
        // ---- epilogue: one accumulator row per thread, tokens 128 half .. + 127
        const int qw = warp & 3, half = (warp - 11) >> 2, ew = warp - 11;
        const bool up = EPI == kEpiGated && (lane & 8);
        const int ch = EPI == kEpiGated ? (lane >> 4) * 8 + (lane & 7) : lane;         // channel in the warp's buffer
        const uint32_t buf0 = sOut + (uint32_t)ew * 2 * kOutBuf, rbar0 = rfull0 + 16 * ew;
        const bool res = EPI == kEpiAct && a.has_res;
        uint32_t tiles = 0, loads[2] = {0, 0};            // residual loads issued into each buffer
        bool ok = true;
        for (int tile = first_tile; ok && tile < a.ntiles; tile += nclusters, ++tiles) {
            const int rb0 = row_block0(tile) + 2 * qw, t0 = token0(tile) + 128 * half;
            const int col0 = EPI == kEpiGated ? rb0 * 8 : rb0 * 16;
            const int row = rb0 * 16 + lane;
            const bool in_row = col0 < a.width;           // of the whole warp (a warp's rows are two row blocks)
            float b = 0.f;
            if (a.bias && row < a.out) b = __half2float(a.bias[EPI == kEpiGated ? col0 + ch + (up ? a.width : 0) : row]);
            // batch j: tokens t0 + 32 j .. + 31, buffer j & 1
            const int t_end = min(a.T, token0(tile) + bn);
            auto live = [&](int j) { return in_row && t0 + 32 * j < t_end; };
            auto load_residual = [&](int j) {             // lane 0, once the buffer's last store has been read
                mbar_arrive_expect_tx(rbar0 + 8 * (j & 1), kOutBuf);
                tma_load_2d(buf0 + (j & 1) * kOutBuf, &tm_r, col0, t0 + 32 * j, rbar0 + 8 * (j & 1));
            };
            if (lane == 0) bulk_wait_read<0>();           // the last tile's stores have read both buffers
            if (res) {                                    // the first two batches' residual, ahead of the sums
                if (lane == 0)
                    for (int j = 0; j < 2; ++j)
                        if (live(j)) load_residual(j);
                for (int j = 0; j < 2; ++j)
                    if (live(j)) ++loads[j];
            }
            ok = mbar_wait(accfull, tiles & 1, kFaultGemmPair + kFaultEpilogueWait, abort) && !*abort;
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {                 // 64 tokens
                uint32_t r[64];
                tmem_ld_32x32b_x32(tbase + ((uint32_t)(32 * qw) << 16) + half * 128 + q * 64, r);
                tmem_ld_32x32b_x32(tbase + ((uint32_t)(32 * qw) << 16) + half * 128 + q * 64 + 32, r + 32);
                tmem_wait_ld();
                if (q == 1) {                             // every sum is in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(accfree);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int j = 2 * q + h;
                    if (!live(j)) continue;
                    if (res) {
                        ok = mbar_wait(rbar0 + 8 * h, (loads[h] - 1) & 1, kFaultGemmPair + kFaultEpilogueWait, abort);
                        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    } else {
                        if (lane == 0) bulk_wait_read<1>();   // the buffer's last store has been read
                        __syncwarp();
                    }
                    const uint32_t at = buf0 + h * kOutBuf + (uint32_t)ch * 2 + (up ? kTokenBytes : 0);
                    if (EPI == kEpiGated) with_act(a.act, PairGated{r + 32 * h, b, at, up});
                    else with_act(a.act, PairAct{r + 32 * h, b, at, res});
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&tm_y, buf0 + h * kOutBuf, col0, t0 + 32 * j);
                        bulk_commit();
                    }
                    if (res && j + 2 < 4 && live(j + 2)) {
                        if (lane == 0) {
                            bulk_wait_read<0>();
                            load_residual(j + 2);
                        }
                        ++loads[h];
                    }
                }
                if (!ok) break;
            }
        }
        if (lane == 0) bulk_wait_read<0>();               // stores have read their buffers before the CTA exits
        if (*abort && lane == 0)
            for (int h = 0; h < 2; ++h)
                if (loads[h] > 0) mbar_wait(rbar0 + 8 * h, (loads[h] - 1) & 1, kFaultGemmPair + kFaultDrainWait, nullptr);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_arrive_wait();                                // no CTA leaves while another may still signal it
    if (C::kSplit) {
        // every CTA finishes its rows of its pair's share of the tokens
        if (*abort == 0) split_epilogue<BN, EPI>(a, sX, row_block0(first_tile), token0(first_tile), rank, pair, pairs);
        cluster_arrive_wait_relaxed();                    // the sums stay until every reader is done
    }
    if (warp == 1) {
        // no MMA may still write tensor memory when it is released
        mbar_wait(fin, 0, kFaultGemmPair + kFaultDrainWait, nullptr);
        tc_fence_after();
        tmem_dealloc_pair(tbase, 512);
    }
}

namespace {

// Clusters of `pairs` CTA pairs that can be resident at once (74 pairs on 148
// SMs), once per device; sets the kernel's attributes.
template <int BN, int EPI>
cudaError_t pair_clusters(int dev, int pairs, int* clusters) {
    static std::atomic<int> resident[64][kMaxPairs + 1] = {};
    static std::mutex mu;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int n = resident[dev][pairs].load(std::memory_order_acquire);
    if (n == 0) {
        std::lock_guard<std::mutex> lock(mu);
        auto k = gemm_pair_kernel<BN, EPI>;
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PairCfg<BN>::kSmem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2 * pairs, 1, 1);
        cfg.blockDim = dim3(PairCfg<BN>::kThreads, 1, 1);
        cfg.dynamicSmemBytes = PairCfg<BN>::kSmem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2 * pairs;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorLaunchOutOfResources;
        resident[dev][pairs].store(n, std::memory_order_release);
    }
    *clusters = n;
    return cudaSuccess;
}

template <int BN, int EPI>
cudaError_t launch_pair(int dev, const CUtensorMap* tm, PairArgs a, const PairPlan& plan, cudaStream_t s) {
    a.ntiles = a.mt * ((a.T + a.bn - 1) / a.bn);
    a.pairs = plan.pairs;
    int clusters = a.ntiles;                               // split form: one tile per cluster
    if (!PairCfg<BN>::kSplit) {
        const cudaError_t e = pair_clusters<BN, EPI>(dev, 1, &clusters);
        if (e != cudaSuccess) return e;
        clusters = std::min(clusters, a.ntiles);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * (unsigned)(a.pairs * clusters), 1, 1);
    cfg.blockDim = dim3(PairCfg<BN>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = PairCfg<BN>::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * a.pairs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, gemm_pair_kernel<BN, EPI>, tm[0], tm[1], tm[2], tm[3], tm[4], tm[5], a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// The operands' tensor maps: X' fp16 [T][in], box 64 channels x half a tile's tokens,
// 128-byte swizzle; codes as uint32 [out/16][in/128 * 256], box 128 channels x
// 8 row blocks; scales uint32 [out/16][G * 8], box the stage's groups x 8 row
// blocks; zeros uint8 [out/16][Gp * 8], box two groups x 8 row blocks; Y and
// the residual fp16 [T][width], box 32 (gated: 16) columns x 32 tokens (used by
// the 256-token form). Rows past T or out are read as zeros and not written.
template <int BN, int EPI>
cudaError_t encode_and_launch(int dev, const void* Xr, const void* qw, const void* scp, const void* zp, int64_t in,
                              int group, PairArgs a, const PairPlan& plan, cudaStream_t s) {
    a.bn = plan.bn;
    const uint64_t G = (uint64_t)(in / group), Gp = G + (G & 1), nrb = (uint64_t)(a.out / 16);
    const uint32_t cols = EPI == kEpiGated ? 16u : 32u;
    CUtensorMap tm[6];
    const bool ok =
        encode_tma_2d(&tm[0], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, Xr, (uint64_t)in, (uint64_t)a.T, (uint64_t)in * 2, 64u,
                      (uint32_t)a.bn / 2, CU_TENSOR_MAP_SWIZZLE_128B) &&
        encode_tma_2d(&tm[1], CU_TENSOR_MAP_DATA_TYPE_UINT32, qw, (uint64_t)a.nk * 256, nrb, (uint64_t)a.nk * 1024, 256u, 8u,
                      CU_TENSOR_MAP_SWIZZLE_NONE) &&
        encode_tma_2d(&tm[2], CU_TENSOR_MAP_DATA_TYPE_UINT32, scp, G * 8, nrb, G * 32, 8u * (uint32_t)a.gs, 8u,
                      CU_TENSOR_MAP_SWIZZLE_NONE) &&
        encode_tma_2d(&tm[3], CU_TENSOR_MAP_DATA_TYPE_UINT8, zp, Gp * 8, nrb, Gp * 8, 16u, 8u, CU_TENSOR_MAP_SWIZZLE_NONE) &&
        encode_tma_2d(&tm[4], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.Y, (uint64_t)a.width, (uint64_t)a.T, (uint64_t)a.width * 2,
                      cols, 32u, CU_TENSOR_MAP_SWIZZLE_NONE) &&
        encode_tma_2d(&tm[5], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.residual ? a.residual : a.Y, (uint64_t)a.width,
                      (uint64_t)a.T, (uint64_t)a.width * 2, cols, 32u, CU_TENSOR_MAP_SWIZZLE_NONE);
    return ok ? launch_pair<BN, EPI>(dev, tm, a, plan, s) : cudaErrorInvalidValue;
}

template <int EPI>
cudaError_t plan_and_launch(const void* Xr, const void* qw, const void* scp, const void* zp, int64_t in, int group,
                            const PairArgs& a, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const PairPlan plan = plan_pairs(a.mt, a.T, a.nk, [&](int form, int pairs) {
        int n = 0;
        const cudaError_t err = form == 64    ? pair_clusters<64, EPI>(dev, pairs, &n)
                                : form == 128 ? pair_clusters<128, EPI>(dev, pairs, &n)
                                              : pair_clusters<256, EPI>(dev, pairs, &n);
        if (err != cudaSuccess) e = err;
        return err == cudaSuccess ? n : 0;
    });
    if (e != cudaSuccess) return e;
    return plan.form == 64    ? encode_and_launch<64, EPI>(dev, Xr, qw, scp, zp, in, group, a, plan, s)
           : plan.form == 128 ? encode_and_launch<128, EPI>(dev, Xr, qw, scp, zp, in, group, a, plan, s)
                              : encode_and_launch<256, EPI>(dev, Xr, qw, scp, zp, in, group, a, plan, s);
}

}  // namespace

cudaError_t launch_gemm_pair(const void* Xr, const void* qw, const void* scp, const void* zp, const void* bias, void* Y,
                             int64_t T, int64_t in, int64_t out, int group, cudaStream_t s, const Epilogue& epi) {
    if (T <= 0) return cudaSuccess;
    if (group != 64 && group != 128) return cudaErrorInvalidValue;
    const bool gated = epi.kind == kEpiGated;
    PairArgs a{};
    a.T = (int)T;
    a.out = (int)out;
    a.nk = (int)(in / 128);
    a.mt = (int)((out / 16 + 15) / 16);
    a.width = (int)(gated ? out / 2 : out);
    a.gs = group == 64 ? 2 : 1;
    a.act = epi.act;
    a.has_res = epi.residual ? 1 : 0;
    a.bias = static_cast<const __half*>(bias);
    a.residual = static_cast<const __half*>(epi.residual);
    a.Y = static_cast<__half*>(Y);
    return gated ? plan_and_launch<kEpiGated>(Xr, qw, scp, zp, in, group, a, s)
                 : plan_and_launch<kEpiAct>(Xr, qw, scp, zp, in, group, a, s);
}

cudaError_t read_fault_gemm_pair(unsigned int* code, bool clear) { return read_fault_word(code, clear); }

}  // namespace paro
