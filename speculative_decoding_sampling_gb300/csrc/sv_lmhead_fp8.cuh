// sv_lmhead_fp8.cuh -- the target's LM head on e4m3 operands whose scales
// belong to blocks of 128.
//
//   z[m, v] = sum_b hs[m, b] ws[v / 128, b] sum_{k in block b} h[m, k] W[v, k]
//
// h e4m3 [M, d] with a scale per row and 128 hidden dims, W e4m3 [V, d] with
// a scale per 128 ids x 128 hidden dims; z is rounded once to bf16.  The
// inner sums (128 products, each exact in fp32) run on the tensor cores
// (tcgen05, kind f8f6f4) into tensor memory; the scales differ from block to
// block and are not powers of two, so each block's sums are read back and
// folded into fp32 accumulators in registers: one fp32 multiply-add per logit
// and block, while the tensor cores form the next block in the other half of
// tensor memory.
//
// Two shapes of one kernel.  PAIR false (M <= 128): a CTA per SM, tiles of
// 128 rows x NB ids; few rows leave the tensor cores idle most of the time
// and the kernel streams W.  PAIR true: a cluster of two CTAs on a pair of
// SMs, tiles of 256 rows x NB ids, each CTA loading its 128 rows of h and
// half of the tile of W (one tcgen05.mma of M 256 reads both), which halves
// what each SM takes from L2.  Tiles are walked rows fastest, so the CTAs
// running at one time share a few tiles of W.
//
// Warp 0 loads (2-D tensor-memory-accelerator boxes of 128 hidden dims, one
// 128-byte swizzle row each), warp 1 allocates tensor memory and issues the
// MMAs, warps 4..11 hold the accumulators: warp w owns the 32 rows of
// tensor-memory lane quarter w mod 4 and the first 128 columns of the tile
// (w < 8) or the others.  Every wait is bounded as in
// lm_head_kernel, with the same teardown.
#pragma once

#include "sv_lmhead.cuh"

namespace sv {

constexpr int kL8BK = 128;    // hidden dims per step: one scale block, one swizzle row
constexpr int kL8MaxNB = 256; // ids per tile
constexpr int kL8ABytes = kLmBM * kL8BK;
constexpr int kL8EpiWarps = 8;
constexpr int kL8Threads = 128 + 32 * kL8EpiWarps;
// Registers a thread: 168 at launch (64,512 in all); the accumulators' two
// warpgroups then take 224 and the first warpgroup keeps 40 (62,464).
constexpr int kL8AccRegs = 224, kL8OtherRegs = 40;
static_assert(32 * kL8EpiWarps * kL8AccRegs + 128 * kL8OtherRegs <= 168 * kL8Threads, "register split");
constexpr uint32_t kL8TmemCols = 2 * kL8MaxNB; // two fp32 sums of one step: all 512 columns

template <bool PAIR> struct L8Shape {
    static constexpr int kCtas = PAIR ? 2 : 1;
    static constexpr int kBBytes = kL8MaxNB / kCtas * kL8BK;
    static constexpr int kStageBytes = kL8ABytes + kBBytes;
    static constexpr int kStages = PAIR ? 6 : 4;
    static constexpr int kSmem = kStages * kStageBytes + 1024; // + alignment of the swizzled tiles
};

struct Lm8Params {
    int32_t M, N, KB;       // rows of h, vocabulary, scale blocks along the hidden dims
    int32_t MT, NT, NB;     // row tiles, id tiles, ids per tile (a multiple of 32)
    uint32_t idesc;         // tcgen05 instruction descriptor
    const float *hs;        // [M, KB]
    const float *ws;        // [ceil(N / 128), KB]
    uint16_t *logits;       // [M, N] bf16 out
    float2 *part;           // [M, NT * halves] (max, normaliser relative to fl(max c)), or nullptr
    int32_t halves;         // column halves of a tile: 1 (NB <= 128) or 2
    float c;                // log2(e) / T
    int32_t vec;            // N % 8 == 0 and 16-byte aligned logits: vector stores
    int32_t *status;
    uint64_t wait_ns;
};

// ------------------------------------------------------------- primitives

template <bool PAIR>
__device__ __forceinline__ void l8_tma_2d(uint32_t dst, const CUtensorMap *map, int32_t c0, int32_t c1, uint32_t bar)
{
    if constexpr (PAIR)
        lm_tma_2d(dst, map, c0, c1, bar);
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
                     : "memory");
}

template <bool PAIR> __device__ __forceinline__ void l8_tmem_alloc(uint32_t dst_smem, uint32_t ncols)
{
    if constexpr (PAIR) {
        lm_tmem_alloc(dst_smem, ncols);
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}

template <bool PAIR> __device__ __forceinline__ void l8_tmem_dealloc(uint32_t taddr, uint32_t ncols)
{
    if constexpr (PAIR)
        lm_tmem_dealloc(taddr, ncols);
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void l8_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc)
{
    if constexpr (PAIR)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                     "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                     "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
                     : "memory");
}

// one arrival, once the MMAs issued before are done, on this barrier of
// every CTA that takes part in them
template <bool PAIR> __device__ __forceinline__ void l8_commit(uint32_t bar)
{
    if constexpr (PAIR)
        lm_commit_both(bar);
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

template <bool PAIR> __device__ __forceinline__ void l8_cluster_sync()
{
    if constexpr (PAIR)
        lm_cluster_sync();
    else
        __syncthreads();
}

// One arrival on a barrier of the leader CTA, behind this warp's reads of
// tensor memory (tcgen05.wait::ld and the fence order those).  CTA scope: a
// cluster-scope release waits for every load and store of the warp that is
// still in flight, on each step.
__device__ __forceinline__ void l8_arrive(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// Instruction descriptor: D fp32, A and B e4m3 (format 0), both K-major.
inline uint32_t l8_idesc(int rows, int ids)
{
    return (1u << 4) | ((static_cast<uint32_t>(ids) >> 3) << 17) | ((static_cast<uint32_t>(rows) >> 4) << 24);
}

// ------------------------------------------------------------- the kernel

// A finished half tile: this lane's row, columns n .. n + 127 of the
// vocabulary (ncols of them inside it), from the fp32 accumulators.
__device__ __forceinline__ void l8_store(const Lm8Params &P, const float (&acc)[128], int row, int n, int ncols,
                                         int slot)
{
    uint16_t *lrow = P.logits + static_cast<int64_t>(row) * P.N + n;
    float mx = -INFINITY;
#pragma unroll
    for (int g = 0; g < 16; ++g) {
        uint32_t pk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = g * 8 + 2 * i;
            pk[i] = bf16_rn_pair(acc[col], acc[col + 1]);
            if (col < ncols)
                mx = fmaxf(mx, bf16_lo(pk[i]));
            if (col + 1 < ncols)
                mx = fmaxf(mx, bf16_hi(pk[i]));
        }
        if (P.vec && g * 8 + 8 <= ncols) {
            *reinterpret_cast<uint4 *>(lrow + g * 8) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (g * 8 + i < ncols)
                    lrow[g * 8 + i] = static_cast<uint16_t>(i & 1 ? pk[i >> 1] >> 16 : pk[i >> 1] & 0xFFFFu);
        }
    }
    if (!P.part)
        return;
    const float mc = mc_of(mx, P.c);
    float S = 0.0f;
#pragma unroll
    for (int col = 0; col < 128; col += 2) {
        const uint32_t pk = bf16_rn_pair(acc[col], acc[col + 1]);
        if (col < ncols)
            S += term(bf16_lo(pk), P.c, mc);
        if (col + 1 < ncols)
            S += term(bf16_hi(pk), P.c, mc);
    }
    P.part[static_cast<int64_t>(row) * (P.NT * P.halves) + slot] = make_float2(mx, S);
}

// Unit u (a pair of SMs, or one) takes tiles u, u + units, ...; tile t covers
// row tile t mod MT and ids NB (t div MT).
template <bool PAIR>
__global__ void __launch_bounds__(kL8Threads, 1)
    lm_head_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const Lm8Params P)
{
    using Sh = L8Shape<PAIR>;
    extern __shared__ uint8_t lm_smem_raw[];
    __shared__ __align__(8) unsigned long long full[Sh::kStages], empty[Sh::kStages], tfull[2], tempty[2], drain;
    __shared__ uint32_t tmem_base;
    __shared__ int stop;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(lm_smem_raw) + 1023) & ~uintptr_t{1023});
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? lm_cluster_rank() : 0u;
    const bool leader = rank == 0;
    const int64_t unit = blockIdx.x / Sh::kCtas, units = gridDim.x / Sh::kCtas;
    const int64_t ntiles = static_cast<int64_t>(P.MT) * P.NT;
    const volatile int *vstop = &stop;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Sh::kStages; ++s) {
            lm_mbar_init(smem_addr(&full[s]), 1);  // the leader's arrival with every CTA's bytes
            lm_mbar_init(smem_addr(&empty[s]), 1); // the MMAs of the stage
        }
        for (int a = 0; a < 2; ++a) {
            lm_mbar_init(smem_addr(&tfull[a]), 1);
            lm_mbar_init(smem_addr(&tempty[a]), Sh::kCtas * kL8EpiWarps);
        }
        lm_mbar_init(smem_addr(&drain), 1);
        stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1)
        l8_tmem_alloc<PAIR>(smem_addr(&tmem_base), kL8TmemCols);
    lm_tc_before();
    __syncthreads();
    l8_cluster_sync<PAIR>(); // every CTA's barriers exist before another CTA signals them
    lm_tc_after();
    const uint32_t tbase = tmem_base;
    auto fail = [&]() {
        if (!stop) {
            stop = 1;
            if (P.status)
                atomicOr(P.status, kTimeout);
        }
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kL8OtherRegs));
        if (warp == 0 && lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            int64_t it = 0;
            const uint32_t fb0 = PAIR ? lm_mapa(smem_addr(&full[0]), 0) : smem_addr(&full[0]);
            const uint32_t sbase = smem_addr(smem);
            const int brows = P.NB / Sh::kCtas; // ids of the tile this CTA loads
            const uint32_t bytes = static_cast<uint32_t>(Sh::kCtas * (kL8ABytes + brows * kL8BK));
            for (int64_t t = unit; t < ntiles && !*vstop; t += units) {
                const int m0 = (static_cast<int>(t % P.MT) * Sh::kCtas + static_cast<int>(rank)) * kLmBM;
                const int n0 = static_cast<int>(t / P.MT) * P.NB + static_cast<int>(rank) * brows;
                int kb = 0;
                for (; kb < P.KB; ++kb, ++it) {
                    if (it >= Sh::kStages && !lm_wait(smem_addr(&empty[s]), ph ^ 1u, vstop, P.wait_ns)) {
                        fail();
                        break;
                    }
                    const uint32_t sa = sbase + static_cast<uint32_t>(s * Sh::kStageBytes);
                    const uint32_t fb = fb0 + static_cast<uint32_t>(s * 8);
                    if (leader)
                        lm_mbar_expect(smem_addr(&full[s]), bytes);
                    l8_tma_2d<PAIR>(sa, &tmA, kb * kL8BK, m0, fb);
                    l8_tma_2d<PAIR>(sa + kL8ABytes, &tmB, kb * kL8BK, n0, fb);
                    if (++s == Sh::kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (kb < P.KB)
                    break;
            }
        } else if (warp == 1 && lane == 0 && leader) {
            const uint64_t ad0 = lm_desc(smem_addr(smem)), bd0 = lm_desc(smem_addr(smem + kL8ABytes));
            int s = 0;
            uint32_t ph = 0;
            int64_t it = 0; // steps so far: step `it` forms its sums in tensor-memory half it mod 2
            for (int64_t t = unit; t < ntiles && !*vstop; t += units) {
                int kb = 0;
                for (; kb < P.KB; ++kb, ++it) {
                    const int acc = static_cast<int>(it & 1);
                    if ((it >= 2 && !lm_wait(smem_addr(&tempty[acc]), static_cast<uint32_t>(((it >> 1) & 1) ^ 1), vstop,
                                             P.wait_ns)) ||
                        !lm_wait(smem_addr(&full[s]), ph, vstop, P.wait_ns)) {
                        fail();
                        break;
                    }
                    lm_tc_after();
                    const uint32_t tacc = tbase + static_cast<uint32_t>(acc * kL8MaxNB);
                    const uint64_t so = static_cast<uint64_t>((s * Sh::kStageBytes) >> 4);
#pragma unroll
                    for (int k = 0; k < kL8BK / 32; ++k)
                        l8_mma<PAIR>(tacc, ad0 + so + static_cast<uint64_t>(k * 2), bd0 + so + static_cast<uint64_t>(k * 2),
                                     P.idesc, k ? 1u : 0u);
                    l8_commit<PAIR>(smem_addr(&empty[s]));
                    l8_commit<PAIR>(smem_addr(&tfull[acc]));
                    if (++s == Sh::kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (kb < P.KB)
                    break;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kL8AccRegs));
        const int lq = warp & 3;
        const int half = warp >= 8 ? 1 : 0;
        const uint32_t tl0 = tbase + (static_cast<uint32_t>(lq * 32) << 16) + static_cast<uint32_t>(half * 128);
        const int mycols = P.NB - half * 128 < 128 ? P.NB - half * 128 : 128; // <= 0: nothing in this half
        const int wblocks = (P.N + 127) / 128;
        const uint32_t tempty0 = PAIR ? lm_mapa(smem_addr(&tempty[0]), 0) : smem_addr(&tempty[0]);
        int64_t it = 0;
        bool ok = true;
        for (int64_t t = unit; t < ntiles && ok; t += units) {
            const int row0 = (static_cast<int>(t % P.MT) * Sh::kCtas + static_cast<int>(rank)) * kLmBM + lq * 32;
            const int tn = static_cast<int>(t / P.MT);
            const int n = tn * P.NB + half * 128;
            const bool work = row0 < P.M && mycols > 0; // warp-uniform
            const int row = row0 + lane;
            const float *hs = P.hs + static_cast<int64_t>(row < P.M ? row : P.M - 1) * P.KB;
            const float *ws[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int wb = (n + g * 32) / 128;
                ws[g] = P.ws + static_cast<int64_t>(wb < wblocks ? wb : wblocks - 1) * P.KB;
            }
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; ++i)
                acc[i] = 0.0f;
            // a step's scales are loaded one step ahead
            float hn = 0.0f, wn[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (work) {
                hn = __ldg(hs);
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    wn[g] = __ldg(ws[g]);
            }
            for (int kb = 0; kb < P.KB; ++kb, ++it) {
                const int a = static_cast<int>(it & 1);
                float f[4];
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    f[g] = __fmul_rn(hn, wn[g]);
                if (work && kb + 1 < P.KB) {
                    hn = __ldg(hs + kb + 1);
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        wn[g] = __ldg(ws[g] + kb + 1);
                }
                ok = __all_sync(0xFFFFFFFFu, lm_wait(smem_addr(&tfull[a]), static_cast<uint32_t>((it >> 1) & 1), vstop,
                                                     P.wait_ns));
                if (!ok) {
                    if (lane == 0)
                        fail();
                    break;
                }
                lm_tc_after();
                if (work) {
                    const uint32_t tl = tl0 + static_cast<uint32_t>(a * kL8MaxNB);
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        if (g * 32 < mycols) {
                            uint32_t v[32];
                            lm_tmem_ld32(tl + g * 32, v);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                acc[g * 32 + i] = __fmaf_rn(__uint_as_float(v[i]), f[g], acc[g * 32 + i]);
                        }
                }
                lm_tc_before();
                __syncwarp();
                if (lane == 0) // this warp has read the step's sums
                    l8_arrive(tempty0 + static_cast<uint32_t>(a * 8));
            }
            if (ok && work && row < P.M) {
                int ncols = P.N - n;
                ncols = ncols < 0 ? 0 : (ncols < mycols ? ncols : mycols);
                l8_store(P, acc, row, n, ncols, tn * P.halves + half);
            }
        }
    }
    // ---- teardown: copies and MMAs in flight complete before the memory goes
    lm_tc_before();
    __syncthreads();
    if (stop) {
        if (threadIdx.x == 0) { // copies issued before the stop land within microseconds
            const uint64_t t0 = lm_ns();
            while (lm_ns() - t0 < 50000ull) {
            }
        }
        if (warp == 1 && lane == 0 && leader) { // every MMA issued is done
            if constexpr (PAIR)
                lm_commit_local(smem_addr(&drain));
            else
                l8_commit<PAIR>(smem_addr(&drain));
            (void)lm_wait(smem_addr(&drain), 0u, nullptr, P.wait_ns);
        }
    }
    __syncthreads();
    l8_cluster_sync<PAIR>(); // no CTA's memory goes while the MMAs or signals may still use it
    if (warp == 1) {
        lm_tc_after();
        l8_tmem_dealloc<PAIR>(tbase, kL8TmemCols);
    }
}

} // namespace sv
