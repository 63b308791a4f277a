// Prefill contraction on pairs of SMs (tcgen05, cta_group::2), for the layer
// with an activation and a residual and for the gated up-projection:
//   Y^T tile [256 rows][256 tokens] = w_hat * X'^T, then the epilogue.
//
// Two CTAs of a cluster share a tile: each keeps its own 128 rows of w_hat in
// its tensor memory and holds half of the tokens in shared memory, and one
// MMA (M = 256, N = 256, K = 16) reads both halves. The kernel is persistent:
// a cluster walks the tiles cid, cid + clusters, ... (row tiles first, so that
// the clusters at work share their tokens), and its roles run ahead of each
// other across tiles. Per CTA, nineteen warps:
//   warp 0      TMA producer: per stage of 128 channels the CTA's 128 tokens
//               of X' (two 64-channel boxes, 128-byte swizzle; ring of 4) and,
//               two stages ahead of it, the int4 codes of its 8 row blocks with
//               their scales and zeros (ring of 6);
//   warps 3-10  dequantise (w_hat = fp16((q - z) s), as the other kernels do)
//               into a ring of 4 tensor-memory stages: a warp takes one
//               quarter of the rows and one half of the stage's channels;
//   warp 2      gate: one lane reports to the leader CTA when its CTA's X' and
//               w_hat of a stage are there;
//   warp 1      tensor memory; in the leader CTA one lane issues the MMAs
//               (A from tensor memory, B from shared memory) of a stage that
//               both gates have reported, and commits it back to both CTAs;
//   warps 11-18 epilogue: a warp takes one quarter of the rows and one half of
//               the tokens, 64 tokens at a time from tensor memory into
//               registers (after the second 64 the accumulator is free for
//               the next tile), then through a 32-token buffer of its own in
//               shared memory, where the residual has arrived by TMA, to a TMA
//               store.
// Tensor memory: 256 columns of fp32 sums, 4 x 64 columns of w_hat (all 512),
// so there is one accumulator: the MMAs pause from a tile's last commit until
// its sums are in registers.
// All waits are bounded (sm100.cuh); a wait that runs out raises the CTA's
// abort flag, every role stops, what was issued is drained, and both CTAs meet
// at the last cluster barrier.
//
// A token's result does not depend on its place in the batch: the order of
// the channels goes by the row tile alone.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "common.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace paro {

namespace {

constexpr int kXStages = 4, kWStages = 6;
constexpr int kPairThreads = 608;
constexpr uint32_t kHalfX = 128 * 128;                  // 128 tokens x 64 channels
constexpr uint32_t kXStage = 2 * kHalfX;                // 32 KB: 128 tokens x 128 channels
constexpr uint32_t kWCodes = 8 * 1024;                  // 8 row blocks x 128 channels of codes
constexpr uint32_t kWScales = 8 * 64;                   // 8 row blocks x up to 2 groups x 8 words
constexpr uint32_t kWStage = kWCodes + kWScales + 128;  // zeros: 8 row blocks x 2 groups x 8 bytes
constexpr uint32_t kOutBuf = 32 * 64;                   // 32 tokens x 32 rows of fp16: two for each epilogue warp
constexpr uint32_t kPairBars = 8 * (4 * kXStages + 2 * kWStages + 8 + 16) + 16;
constexpr size_t kPairSmem = 1024 + (size_t)kXStages * kXStage + (size_t)kWStages * kWStage + 16 * kOutBuf + kPairBars;

struct PairArgs {
    int T, out, nk;             // nk: 128-channel stages
    int mt, ntiles;             // 256-row tiles; tiles in all
    int width;                  // columns of Y (out, or out / 2 for the gated epilogue)
    int gs;                     // quantisation groups per 128 channels (1, or 2 for group 64)
    int act, has_res;
    const __half* bias;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive_wait() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrive at a barrier of the cluster's other CTA, and wait for such arrivals.
// Relaxed: what they order is tensor memory (written with tcgen05.st, read by
// the MMA), which goes by the tcgen05 fences on both sides, and shared memory
// that TMA wrote and the MMA reads; no ordinary loads and stores meet here. A
// release at cluster scope costs about 900 cycles.
__device__ __forceinline__ void mbar_arrive_other(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_other(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_other(uint32_t bar, uint32_t parity, unsigned int fault,
                                                volatile uint32_t* abort) {
    if (mbar_try_wait_other(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_other(bar, parity)) return true;
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
// Arrive on `bar` of both CTAs once every MMA issued so far by this thread has completed.
__device__ __forceinline__ void umma_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"((uint16_t)3) : "memory");
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

template <int EPI>
__global__ void __launch_bounds__(kPairThreads, 1)
gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                 const __grid_constant__ CUtensorMap tm_s, const __grid_constant__ CUtensorMap tm_z,
                 const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_r,
                 const PairArgs a) {
    // the next kernel's CTAs may take SMs as this grid's leave them; it reads
    // nothing of ours before this grid is complete
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr uint32_t kIdesc = umma_idesc_f16(256, 256);
    constexpr uint32_t kTokenBytes = EPI == kEpiGated ? 32 : 64;       // one token of an epilogue warp's buffer
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sX = smem_addr(smem), sOut = sX + kXStages * kXStage, sW = sOut + 16 * kOutBuf;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (size_t)kXStages * kXStage + 16 * kOutBuf + (size_t)kWStages * kWStage);
    const uint32_t xfull0 = smem_addr(bars), free0 = xfull0 + 8 * kXStages, afull0 = free0 + 8 * kXStages;
    const uint32_t go0 = afull0 + 8 * kXStages, wfull0 = go0 + 8 * kXStages, wfree0 = wfull0 + 8 * kWStages;
    const uint32_t accfull = wfree0 + 8 * kWStages, accfree = accfull + 8, fin = accfree + 8, rfull0 = fin + 8;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 4 * kXStages + 2 * kWStages + 8 + 16);
    volatile uint32_t* abort = tslot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int nclusters = gridDim.x >> 1, nk = a.nk;
    const int first_tile = blockIdx.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kXStages; ++s) {
            mbar_init(xfull0 + 8 * s, 1);
            mbar_init(free0 + 8 * s, 1);                  // the MMAs on X' stage and w_hat stage s are done
            mbar_init(afull0 + 8 * s, 8);                 // this CTA's dequantisation warps
            mbar_init(go0 + 8 * s, 2);                    // leader: both CTAs' gates
        }
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(wfull0 + 8 * s, 1);
            mbar_init(wfree0 + 8 * s, 8);
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
    cluster_arrive_wait();                                // the other CTA's barriers exist too
    tc_fence_after();
    const uint32_t tbase = *tslot;
    const uint32_t tA = tbase + 256;                      // w_hat stages after the accumulator columns
    // X' is written by the rotation grid launched just before this one
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // tile -> row blocks of this CTA, first token, first channel stage.
    // Clusters walk the channels from different starting stages, so that
    // concurrent requests spread over the memory channels; the start goes by
    // the row tile alone.
    auto row_block0 = [&](int tile) { return ((tile % a.mt) * 2 + (int)rank) * 8; };
    auto token0 = [&](int tile) { return tile / a.mt * 256; };
    auto kstart = [&](int tile) { return (int)((((uint32_t)(tile % a.mt) * 0x9E3779B1u) >> 16) % (uint32_t)nk); };

    if (warp == 0) {
        if (lane == 0) {
            // ---- TMA producer: the weights of a stage go out two stages
            // before its X', so they never wait behind an X' slot
            constexpr int kAhead = kWStages - kXStages;
            RingPos<kXStages> px;
            RingPos<kWStages> pw;
            uint32_t xissued[kXStages], wissued[kWStages];    // loads issued so far per slot (for the drain)
#pragma unroll
            for (int s = 0; s < kXStages; ++s) xissued[s] = 0;
#pragma unroll
            for (int s = 0; s < kWStages; ++s) wissued[s] = 0;
            int wtile = first_tile, wi = 0, wkb = wtile < a.ntiles ? kstart(wtile) : 0;
            auto issue_w = [&]() {                        // the next stage's weights, if there is one
                if (wtile >= a.ntiles) return true;
                if (pw.use > 0 && !mbar_wait(wfree0 + 8 * pw.slot, (pw.use - 1) & 1, kFaultGemmPair + kFaultTmaWait, abort))
                    return false;
                const int rb0 = row_block0(wtile);
                const uint32_t bar = wfull0 + 8 * pw.slot, dst = sW + pw.slot * kWStage;
                mbar_arrive_expect_tx(bar, kWCodes + 8 * 32 * a.gs + 128);
                tma_load_2d(dst, &tm_w, wkb * 256, rb0, bar);
                tma_load_2d(dst + kWCodes, &tm_s, wkb * 8 * a.gs, rb0, bar);
                tma_load_2d(dst + kWCodes + kWScales, &tm_z, (a.gs == 2 ? wkb : wkb >> 1) * 16, rb0, bar);
#pragma unroll
                for (int t = 0; t < kWStages; ++t)
                    if (t == pw.slot) wissued[t] = pw.use + 1;
                pw.next();
                wkb = wkb + 1 == nk ? 0 : wkb + 1;
                if (++wi == nk) {
                    wi = 0;
                    wtile += nclusters;
                    if (wtile < a.ntiles) wkb = kstart(wtile);
                }
                return true;
            };
            bool ok = true;
            for (int i = 0; ok && i < kAhead; ++i) ok = issue_w();
            for (int tile = first_tile; ok && tile < a.ntiles; tile += nclusters) {
                const int n0 = token0(tile) + 128 * (int)rank;
                int kb = kstart(tile);
                for (int i = 0; i < nk; ++i) {
                    ok = issue_w() && (px.use == 0 || mbar_wait(free0 + 8 * px.slot, (px.use - 1) & 1,
                                                                kFaultGemmPair + kFaultTmaWait, abort)) && !*abort;
                    if (!ok) break;
                    const uint32_t bar = xfull0 + 8 * px.slot, dst = sX + px.slot * kXStage;
                    mbar_arrive_expect_tx(bar, kXStage);
                    tma_load_2d(dst, &tm_x, kb * 128, n0, bar);
                    tma_load_2d(dst + kHalfX, &tm_x, kb * 128 + 64, n0, bar);
#pragma unroll
                    for (int t = 0; t < kXStages; ++t)
                        if (t == px.slot) xissued[t] = px.use + 1;
                    px.next();
                    kb = kb + 1 == nk ? 0 : kb + 1;
                }
            }
            if (*abort) {   // drain: every issued load must land before the CTA exits
#pragma unroll
                for (int s = 0; s < kXStages; ++s)
                    if (xissued[s] > 0) mbar_wait(xfull0 + 8 * s, (xissued[s] - 1) & 1, kFaultGemmPair + kFaultDrainWait, nullptr);
#pragma unroll
                for (int s = 0; s < kWStages; ++s)
                    if (wissued[s] > 0) mbar_wait(wfull0 + 8 * s, (wissued[s] - 1) & 1, kFaultGemmPair + kFaultDrainWait, nullptr);
            }
        }
    } else if (warp == 2) {
        if (lane == 0) {
            // ---- gate: one report per stage to the leader's MMA thread, which
            // then looks at a single barrier (a look takes about 100 cycles,
            // and its MMA queue does not hold enough work for three)
            const uint32_t go_leader0 = map_to_rank(go0, 0);
            RingPos<kXStages> p;
            uint32_t tiles = 0;
            bool ok = true;
            for (int tile = first_tile; ok && tile < a.ntiles; tile += nclusters, ++tiles) {
                // the sums of the tile before are out of this CTA's tensor memory
                if (tiles > 0) ok = mbar_wait(accfree, (tiles - 1) & 1, kFaultGemmPair + kFaultMmaWait, abort);
                for (int i = 0; ok && i < nk; ++i, p.next()) {
                    ok = mbar_wait(xfull0 + 8 * p.slot, p.use & 1, kFaultGemmPair + kFaultMmaWait, abort) &&
                         mbar_wait(afull0 + 8 * p.slot, p.use & 1, kFaultGemmPair + kFaultMmaWait, abort);
                    if (!ok) break;
                    tc_fence_after();
                    tc_fence_before();
                    mbar_arrive_other(go_leader0 + 8 * p.slot);
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
                    ok = __all_sync(0xffffffffu, mbar_wait_other(go0 + 8 * s, p.use & 1, kFaultGemmPair + kFaultMmaWait, abort));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t b = umma_desc_sw128_kmajor(sX + s * kXStage);
                    const uint32_t w = tA + s * 64;
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)     // two 64-channel boxes of four MMAs each
                            umma_f16_ts_pair(tbase, w + kk * 8, b + (uint64_t)((kk >> 2) * (kHalfX >> 4) + (kk & 3) * 2), kIdesc,
                                             i + kk > 0 ? 1u : 0u);
                        umma_commit_pair(free0 + 8 * s);
                    }
                    __syncwarp();
                }
                if (ok && elect_one()) umma_commit_pair(accfull);
                __syncwarp();
            }
            if (elect_one()) umma_commit_pair(fin);       // always: arrives once every MMA issued above has completed
            __syncwarp();
        }
    } else if (warp < 11) {
        // ---- dequantisation
        const int qw = warp & 3;                          // tensor-memory lanes 32 qw .. 32 qw + 31
        const int half = (warp - 3) >> 2;                 // channels 64 half .. + 63 of a stage
        const int g = lane >> 2;
        RingPos<kXStages> p;
        RingPos<kWStages> pw;
        bool ok = true;
        for (int tile = first_tile; ok && tile < a.ntiles; tile += nclusters) {
            int kb = kstart(tile);
            for (int i = 0; i < nk; ++i, p.next(), pw.next()) {
                const int s = p.slot;
                // the tensor-memory stores below are warp-collective: the whole
                // warp goes on only if every lane saw the stage arrive
                ok = mbar_wait(wfull0 + 8 * pw.slot, pw.use & 1, kFaultGemmPair + kFaultDequantWait, abort) && !*abort;
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                const uint32_t src = sW + pw.slot * kWStage, zsel = a.gs == 2 ? half : kb & 1;
                uint4 wv[2];
                uint32_t sw[2], zb[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int rbl = 2 * qw + r;
                    wv[r] = lds128(src + rbl * 1024 + half * 512 + lane * 16);
                    sw[r] = lds32(src + kWCodes + (rbl * a.gs + (a.gs == 2 ? half : 0)) * 32 + g * 4);
                    zb[r] = lds8(src + kWCodes + kWScales + rbl * 16 + zsel * 8 + g);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(wfree0 + 8 * pw.slot);
                ok = p.use == 0 || mbar_wait(free0 + 8 * s, (p.use - 1) & 1, kFaultGemmPair + kFaultDequantWait, abort);
                if (!__all_sync(0xffffffffu, ok && !*abort)) { ok = false; break; }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t sc0, sc1, regs[16];
                    scale_pairs(sw[r], sc0, sc1);
                    const Zero2 zc = zero_consts(zb[r]);
                    dequant_word(wv[r].x, zc, sc0, sc1, regs + 0);
                    dequant_word(wv[r].y, zc, sc0, sc1, regs + 4);
                    dequant_word(wv[r].z, zc, sc0, sc1, regs + 8);
                    dequant_word(wv[r].w, zc, sc0, sc1, regs + 12);
                    tmem_st_16x256b_x4(tA + s * 64 + half * 32 + ((uint32_t)(32 * qw + 16 * r) << 16), regs);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(afull0 + 8 * s);
                kb = kb + 1 == nk ? 0 : kb + 1;
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
            auto live = [&](int j) { return in_row && t0 + 32 * j < a.T; };
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
    cluster_arrive_wait();                                // neither CTA leaves while the other may still signal it
    if (warp == 1) {
        // no MMA may still write tensor memory when it is released
        mbar_wait(fin, 0, kFaultGemmPair + kFaultDrainWait, nullptr);
        tc_fence_after();
        tmem_dealloc_pair(tbase, 512);
    }
}

namespace {

// Launch on as many clusters as can be resident (74 on 148 SMs), at most one per tile.
template <int EPI>
cudaError_t launch_pair(const CUtensorMap* tm, const PairArgs& a, cudaStream_t s) {
    // kernel attributes and residency, once per device (double-checked under a lock)
    static std::atomic<int> resident[64] = {};
    static std::mutex mu;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(kPairThreads, 1, 1);
    cfg.dynamicSmemBytes = kPairSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = resident[dev].load(std::memory_order_acquire);
    if (clusters == 0) {
        std::lock_guard<std::mutex> lock(mu);
        clusters = resident[dev].load(std::memory_order_relaxed);
        if (clusters == 0) {
            cudaError_t e = cudaFuncSetAttribute(gemm_pair_kernel<EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)kPairSmem);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, gemm_pair_kernel<EPI>, &cfg);
            if (e != cudaSuccess) return e;
            if (clusters < 1) return cudaErrorLaunchOutOfResources;
            resident[dev].store(clusters, std::memory_order_release);
        }
    }
    cfg.gridDim = dim3(2 * (unsigned)std::min(clusters, a.ntiles), 1, 1);
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, gemm_pair_kernel<EPI>, tm[0], tm[1], tm[2], tm[3], tm[4], tm[5], a);
}

}  // namespace

// Tensor maps: X' fp16 [T][in], box 64 channels x 128 tokens, 128-byte
// swizzle; codes as uint32 [out/16][in/128 * 256], box 128 channels x 8 row
// blocks; scales uint32 [out/16][G * 8], box the stage's groups x 8 row
// blocks; zeros uint8 [out/16][Gp * 8], box two groups x 8 row blocks; Y and
// the residual fp16 [T][width], box 32 (gated: 16) columns x 32 tokens. Rows past T or out are read as zeros and not
// written.
cudaError_t launch_gemm_pair(const void* Xr, const void* qw, const void* scp, const void* zp, const void* bias, void* Y,
                             int64_t T, int64_t in, int64_t out, int group, cudaStream_t s, const Epilogue& epi) {
    if (T <= 0) return cudaSuccess;
    if (group != 64 && group != 128) return cudaErrorInvalidValue;
    const bool gated = epi.kind == kEpiGated;
    PairArgs a{};
    a.T = (int)T;
    a.out = (int)out;
    a.nk = (int)(in / 128);
    a.width = (int)(gated ? out / 2 : out);
    a.gs = group == 64 ? 2 : 1;
    a.act = epi.act;
    a.has_res = epi.residual ? 1 : 0;
    a.bias = static_cast<const __half*>(bias);
    const uint64_t G = (uint64_t)(in / group), Gp = G + (G & 1), nrb = (uint64_t)(out / 16);
    CUtensorMap tm[6];
    const bool ok =
        encode_tma_2d(&tm[0], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, Xr, (uint64_t)in, (uint64_t)T, (uint64_t)in * 2, 64u, 128u,
                      CU_TENSOR_MAP_SWIZZLE_128B) &&
        encode_tma_2d(&tm[1], CU_TENSOR_MAP_DATA_TYPE_UINT32, qw, (uint64_t)a.nk * 256, nrb, (uint64_t)a.nk * 1024, 256u, 8u,
                      CU_TENSOR_MAP_SWIZZLE_NONE) &&
        encode_tma_2d(&tm[2], CU_TENSOR_MAP_DATA_TYPE_UINT32, scp, G * 8, nrb, G * 32, 8u * (uint32_t)a.gs, 8u,
                      CU_TENSOR_MAP_SWIZZLE_NONE) &&
        encode_tma_2d(&tm[3], CU_TENSOR_MAP_DATA_TYPE_UINT8, zp, Gp * 8, nrb, Gp * 8, 16u, 8u, CU_TENSOR_MAP_SWIZZLE_NONE) &&
        encode_tma_2d(&tm[4], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, Y, (uint64_t)a.width, (uint64_t)T, (uint64_t)a.width * 2,
                      gated ? 16u : 32u, 32u, CU_TENSOR_MAP_SWIZZLE_NONE) &&
        encode_tma_2d(&tm[5], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, epi.residual ? epi.residual : Y, (uint64_t)a.width,
                      (uint64_t)T, (uint64_t)a.width * 2, gated ? 16u : 32u, 32u, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (!ok) return cudaErrorInvalidValue;
    a.mt = (int)((nrb + 15) / 16);
    a.ntiles = a.mt * (int)((T + 255) / 256);
    const cudaError_t e = gated ? launch_pair<kEpiGated>(tm, a, s) : launch_pair<kEpiAct>(tm, a, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t read_fault_gemm_pair(unsigned int* code, bool clear) { return read_fault_word(code, clear); }

}  // namespace paro
