// Prefill contraction on pairs of SMs (tcgen05, cta_group::2), for the layer
// with an activation and a residual and for the gated up-projection:
//   Y^T tile [256 rows][256 tokens] = w_hat * X'^T, then the epilogue.
//
// The single-CTA kernel (gemm_sm100.cu) loads a 256-token X' tile for 128
// rows: 36 KB per 64 channels and SM, and its time is that traffic's, not the
// tensor pipe's. Here two CTAs of a cluster share the tile: each keeps its
// own 128 rows of w_hat in its tensor memory and holds half of the tokens in
// shared memory, and one MMA (M = 256, N = 256, K = 16) reads both halves, so
// an SM loads 20 KB per 64 channels for the same work.
//
// Per CTA, ten warps, a ring of four stages of 128 channels:
//   warp 0     TMA producer: per stage the CTA's 128 tokens of X' (two
//              64-channel boxes, 128-byte swizzle), the int4 codes of its 8
//              row blocks, their scales and zeros; then the residual's two
//              128-row x 128-token tiles into the next two stages of the ring
//              (they arrive while the last MMAs run); at the end it stores
//              the finished tile with TMA, 64 tokens at a time;
//   warp 1     tensor memory; in the leader CTA one lane issues the MMAs
//              (A from tensor memory, B from shared memory) once its eight
//              dequantisation warps and the other CTA have reported the
//              stage, and commits it back to both CTAs' producers; in the
//              other CTA one lane forwards its eight warps' reports;
//   warps 2-9  dequantise (w_hat = fp16((q - z) s), as the other kernels do):
//              a warp takes one quarter of the rows and one half of the
//              stage's channels; then the epilogue: the same quarter of the
//              rows and one half of the tokens, from tensor memory through
//              registers into shared memory as fp16 [token][row].
// Tensor memory: 256 columns of fp32 sums, 4 x 64 columns of w_hat (all 512).
// All waits are bounded (sm100.cuh); a wait that runs out raises the CTA's
// abort flag, what was issued is drained, both CTAs meet at the last cluster
// barrier and nothing is stored.
//
// A token's result does not depend on its place in the batch: the order of
// the channels goes by the row tile alone.
#include <cuda.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace paro {

namespace {

constexpr int kPairStages = 4;
constexpr int kPairThreads = 320;
constexpr uint32_t kHalfX = 128 * 128;                  // 128 tokens x 64 channels
constexpr uint32_t kPairX = 2 * kHalfX;                 // 32 KB: 128 tokens x 128 channels
constexpr uint32_t kPairW = 8 * 1024;                   // 8 row blocks x 128 channels of codes
constexpr uint32_t kPairS = 8 * 64;                     // scales: 8 row blocks x up to 2 groups x 8 words
constexpr uint32_t kPairZ = 8 * 16;                     // zeros: 8 row blocks x 2 groups x 8 bytes
constexpr uint32_t kPairStage = kPairX + kPairW + kPairS + kPairZ;
constexpr size_t kPairSmem = 1024 + (size_t)kPairStages * kPairStage + 256;

struct PairArgs {
    int T, out, nk;             // nk: 128-channel stages
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
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// mbar_wait for a barrier at which the other CTA's threads arrive too
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, unsigned int fault,
                                                  volatile uint32_t* abort) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
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
// tile [token][128 rows], over the residual where there is one.
struct PairAct {
    const uint32_t* r;
    float b;
    uint32_t at;                // this row in the first token's row of the tile (256 bytes per token)
    bool has_res;
    template <int ACT>
    __device__ __forceinline__ void run() const {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            float v = act_fn<ACT>(__uint_as_float(r[j]) + b);
            if (has_res) v += lds16(at + j * 256);
            sts16(at + j * 256, v);
        }
    }
};
// Gate rows (lanes with bit 3 clear) and up rows (8 lanes on) trade columns:
// of tokens t, t + 1 the gate lane finishes t, the up lane t + 1. Tile
// [token][64 channels], 128 bytes per token.
struct PairGated {
    const uint32_t* r;
    float b;                    // this row's own bias
    uint32_t at;                // this lane's channel in the first token's row of the tile
    bool up;
    template <int ACT>
    __device__ __forceinline__ void run() const {
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            const float v0 = __uint_as_float(r[j]) + b, v1 = __uint_as_float(r[j + 1]) + b;
            const float other = __shfl_xor_sync(0xffffffffu, up ? v0 : v1, 8);
            sts16(at + (j + (up ? 1 : 0)) * 128, act_fn<ACT>(up ? other : v0) * (up ? v1 : other));
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
    constexpr int S = kPairStages;
    constexpr uint32_t kIdesc = umma_idesc_f16(256, 256);
    constexpr uint32_t kTokenBytes = EPI == kEpiGated ? 128 : 256;     // one token of the finished tile
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const uint32_t sX = smem_addr(smem), sW = sX + S * kPairX, sS = sW + S * kPairW, sZ = sS + S * kPairS;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (size_t)S * kPairStage);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 3 * S + 7);
    volatile uint32_t* abort = tslot + 1;
    const uint32_t full0 = smem_addr(bars), afull0 = full0 + 8 * S, free0 = afull0 + 8 * S;
    const uint32_t done = free0 + 8 * S, rfull0 = done + 8, ready0 = rfull0 + 16;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int rb0 = blockIdx.x * 8, n0 = blockIdx.y * 256;
    const int nk = a.nk;
    // Pairs walk the channels from different starting stages, so that
    // concurrent requests spread over the memory channels; the start goes by
    // the row tile alone.
    const int kstart = (int)((((blockIdx.x >> 1) * 0x9E3779B1u) >> 16) % (uint32_t)nk);
    auto kstage = [&](int i) { const int j = i + kstart; return j >= nk ? j - nk : j; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(afull0 + 8 * s, rank == 0 ? 9 : 8); // this CTA's dequantisation warps (leader: and the other CTA)
            mbar_init(free0 + 8 * s, 1);
        }
        mbar_init(done, 1);
        for (int h = 0; h < 2; ++h) mbar_init(rfull0 + 8 * h, 1);
        for (int c = 0; c < 4; ++c) mbar_init(ready0 + 8 * c, 4);
        *abort = 0u;
        mbar_fence_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_s);
        tma_prefetch_desc(&tm_z);
        tma_prefetch_desc(&tm_y);
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

    // The ring's slots after the last stage hold the residual and then the
    // finished tile: half h (tokens 128 h .. + 127) is in slot (nk + h) mod S.
    auto tile_slot = [&](int h) { return sX + (uint32_t)((nk + h) % S) * kPairX; };

    if (warp == 0) {
        if (lane == 0) {
            int issued[S];                                // per stage: loads issued so far
#pragma unroll
            for (int s = 0; s < S; ++s) issued[s] = 0;
            for (int i = 0; i < nk; ++i) {
                const int s = i % S, u = i / S;
                if (u > 0 && !mbar_wait(free0 + 8 * s, (u - 1) & 1, kFaultGemmPair + kFaultTmaWait, abort)) break;
                if (*abort) break;
                const int kb = kstage(i), bar = full0 + 8 * s;
                mbar_arrive_expect_tx(bar, kPairX + kPairW + 8 * 32 * a.gs + kPairZ);
                tma_load_2d(sX + s * kPairX, &tm_x, kb * 128, n0 + 128 * rank, bar);
                tma_load_2d(sX + s * kPairX + kHalfX, &tm_x, kb * 128 + 64, n0 + 128 * rank, bar);
                tma_load_2d(sW + s * kPairW, &tm_w, kb * 256, rb0, bar);
                tma_load_2d(sS + s * kPairS, &tm_s, kb * 8 * a.gs, rb0, bar);
                tma_load_2d(sZ + s * kPairZ, &tm_z, (a.gs == 2 ? kb : kb >> 1) * 16, rb0, bar);
#pragma unroll
                for (int t = 0; t < S; ++t)
                    if (t == s) issued[t] = u + 1;
            }
            int res_issued = 0;
            if (EPI == kEpiAct && a.has_res)
                for (int h = 0; h < 2; ++h) {
                    const int i = nk + h, s = i % S, u = i / S;
                    if (*abort) break;
                    if (u > 0 && !mbar_wait(free0 + 8 * s, (u - 1) & 1, kFaultGemmPair + kFaultTmaWait, abort)) break;
                    mbar_arrive_expect_tx(rfull0 + 8 * h, kPairX);
                    tma_load_2d(tile_slot(h), &tm_r, rb0 * 16, n0 + 128 * h, rfull0 + 8 * h);
                    res_issued = h + 1;
                }
            // store the finished tile, 64 tokens at a time
            const int col0 = EPI == kEpiGated ? rb0 * 8 : rb0 * 16;
            for (int c = 0; c < 4; ++c) {
                if (!mbar_wait(ready0 + 8 * c, 0, kFaultGemmPair + kFaultEpilogueWait, abort) || *abort) break;
                if (col0 < a.width && n0 + 64 * c < a.T) {
                    tma_store_2d(&tm_y, tile_slot(c >> 1) + (uint32_t)(c & 1) * 64 * kTokenBytes, col0, n0 + 64 * c);
                    bulk_commit();
                }
            }
            bulk_wait_read<0>();
            if (*abort) {   // drain: every issued load must land before the CTA exits
#pragma unroll
                for (int s = 0; s < S; ++s)
                    if (issued[s] > 0) mbar_wait(full0 + 8 * s, (issued[s] - 1) & 1, kFaultGemmPair + kFaultDrainWait, nullptr);
                for (int h = 0; h < res_issued; ++h) mbar_wait(rfull0 + 8 * h, 0, kFaultGemmPair + kFaultDrainWait, nullptr);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            for (int i = 0; i < nk; ++i) {
                const int s = i % S, u = i / S;
                // every warp that reports a stage has seen that CTA's loads of it arrive
                if (!mbar_wait_cluster(afull0 + 8 * s, u & 1, kFaultGemmPair + kFaultMmaWait, abort)) break;
                if (!mbar_wait(full0 + 8 * s, u & 1, kFaultGemmPair + kFaultMmaWait, abort)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    umma_f16_ts_pair(tbase, tA + s * 64 + kk * 8,
                                     umma_desc_sw128_kmajor(sX + s * kPairX + (kk >> 2) * kHalfX) + (uint64_t)((kk & 3) * 2),
                                     kIdesc, i + kk > 0 ? 1u : 0u);
                umma_commit_pair(free0 + 8 * s);
            }
            umma_commit_pair(done);                       // always: arrives once every MMA issued above has completed
        } else if (lane == 0) {
            // the other CTA reports a stage once, for its eight warps: a
            // cluster-scope release by each of them cost 900 cycles a stage
            const uint32_t leader_afull0 = map_to_rank(afull0, 0);
            for (int i = 0; i < nk; ++i) {
                const int s = i % S, u = i / S;
                if (!mbar_wait(afull0 + 8 * s, u & 1, kFaultGemmPair + kFaultMmaWait, abort)) break;
                mbar_arrive_cluster(leader_afull0 + 8 * s);
            }
        }
    } else {
        const int qw = warp & 3;                          // tensor-memory lanes 32 qw .. 32 qw + 31
        const int half = (warp - 2) >> 2;                 // channels 64 half .. of a stage, then tokens 128 half ..
        const int g = lane >> 2;
        for (int i = 0; i < nk; ++i) {
            const int s = i % S, u = i / S;
            // the tensor-memory stores below are warp-collective: the whole
            // warp goes on only if every lane saw the stage arrive
            if (!__all_sync(0xffffffffu, mbar_wait(full0 + 8 * s, u & 1, kFaultGemmPair + kFaultDequantWait, abort) && !*abort))
                break;
            const uint32_t zsel = a.gs == 2 ? half : kstage(i) & 1;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int rbl = 2 * qw + r;
                const uint4 wv = lds128(sW + s * kPairW + rbl * 1024 + half * 512 + lane * 16);
                uint32_t sc0, sc1, regs[16];
                scale_pairs(lds32(sS + s * kPairS + (rbl * a.gs + (a.gs == 2 ? half : 0)) * 32 + g * 4), sc0, sc1);
                const Zero2 zc = zero_consts(lds8(sZ + s * kPairZ + rbl * 16 + zsel * 8 + g));
                dequant_word(wv.x, zc, sc0, sc1, regs + 0);
                dequant_word(wv.y, zc, sc0, sc1, regs + 4);
                dequant_word(wv.z, zc, sc0, sc1, regs + 8);
                dequant_word(wv.w, zc, sc0, sc1, regs + 12);
                tmem_st_16x256b_x4(tA + s * 64 + half * 32 + ((uint32_t)(32 * qw + 16 * r) << 16), regs);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(afull0 + 8 * s);
        }

        // ---- epilogue: one accumulator row per thread, tokens 128 half .. + 127
        // (skipped after an abort: the tile is not valid, and the fault word says so)
        bool ok = mbar_wait(done, 0, kFaultGemmPair + kFaultEpilogueWait, abort);
        if (ok && EPI == kEpiAct && a.has_res)
            ok = mbar_wait(rfull0 + 8 * half, 0, kFaultGemmPair + kFaultEpilogueWait, abort);
        if (__all_sync(0xffffffffu, ok && !*abort)) {
            tc_fence_after();
            const int rloc = 32 * qw + lane, row = rb0 * 16 + rloc;
            const bool up = EPI == kEpiGated && (lane & 8);
            const int ch = EPI == kEpiGated ? (rloc >> 4) * 8 + (lane & 7) : rloc;      // channel of the tile
            const int bias_at = EPI == kEpiGated ? rb0 * 8 + ch + (up ? a.width : 0) : row;
            const float b = a.bias && row < a.out ? __half2float(a.bias[bias_at]) : 0.f;
            const uint32_t at = tile_slot(half) + (uint32_t)ch * 2;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {                 // 32 tokens
                uint32_t r[32];
                tmem_ld_32x32b_x32(tbase + ((uint32_t)(32 * qw) << 16) + half * 128 + c * 32, r);
                tmem_wait_ld();
                const uint32_t to = at + (uint32_t)c * 32 * kTokenBytes;
                if (EPI == kEpiGated) with_act(a.act, PairGated{r, b, to, up});
                else with_act(a.act, PairAct{r, b, to, a.has_res != 0});
                if (c & 1) {                              // 64 tokens of this quarter of the rows are written
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ready0 + 8 * (2 * half + (c >> 1)));
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive_wait();                                // neither CTA leaves while the other may still signal it
    if (warp == 1) {
        // no MMA may still write tensor memory when it is released
        mbar_wait(done, 0, kFaultGemmPair + kFaultDrainWait, nullptr);
        tc_fence_after();
        tmem_dealloc_pair(tbase, 512);
    }
}

namespace {

template <int EPI>
cudaError_t launch_pair(const CUtensorMap* tm, const PairArgs& a, int mt, int nt, cudaStream_t s) {
    // kernel attributes, set once per device (double-checked under a lock)
    static std::atomic<bool> configured[64] = {};
    static std::mutex mu;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(mu);
        if (!configured[dev].load(std::memory_order_relaxed)) {
            const cudaError_t e = cudaFuncSetAttribute(gemm_pair_kernel<EPI>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPairSmem);
            if (e != cudaSuccess) return e;
            configured[dev].store(true, std::memory_order_release);
        }
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(mt, nt, 1);
    cfg.blockDim = dim3(kPairThreads, 1, 1);
    cfg.dynamicSmemBytes = kPairSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, gemm_pair_kernel<EPI>, tm[0], tm[1], tm[2], tm[3], tm[4], tm[5], a);
}

}  // namespace

// Tensor maps: X' fp16 [T][in], box 64 channels x 128 tokens, 128-byte
// swizzle; codes as uint32 [out/16][in/128 * 256], box 128 channels x 8 row
// blocks; scales uint32 [out/16][G * 8], box the stage's groups x 8 row
// blocks; zeros uint8 [out/16][Gp * 8], box two groups x 8 row blocks; Y fp16
// [T][width], box 128 (gated: 64) columns x 64 tokens; residual fp16 [T][out],
// box 128 columns x 128 tokens. Rows past T or out are read as zeros and not
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
                      gated ? 64u : 128u, 64u, CU_TENSOR_MAP_SWIZZLE_NONE) &&
        encode_tma_2d(&tm[5], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, epi.residual ? epi.residual : Y, (uint64_t)a.width,
                      (uint64_t)T, (uint64_t)a.width * 2, gated ? 64u : 128u, 128u, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (!ok) return cudaErrorInvalidValue;
    const int mt = 2 * (int)((nrb + 15) / 16), nt = (int)((T + 255) / 256);
    const cudaError_t e = gated ? launch_pair<kEpiGated>(tm, a, mt, nt, s) : launch_pair<kEpiAct>(tm, a, mt, nt, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t read_fault_gemm_pair(unsigned int* code, bool clear) { return read_fault_word(code, clear); }

}  // namespace paro
