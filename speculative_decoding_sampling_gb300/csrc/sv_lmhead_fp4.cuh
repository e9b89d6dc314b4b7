// sv_lmhead_fp4.cuh -- the LM head on microscaled 4-bit operands.
//
//   z[m, v] = gh[m] gw[v] sum_b sh[m, b] sw[v, b] sum_{k in block b} h[m, k] W[v, k]
//
// h [M, d] and W [V, d] as sv_fp4.cuh writes them: e2m1 values with a scale for
// each 16 of them (e4m3, and a factor gh, gw for each row) or each 32 (e8m0, no
// factors); z is rounded once to bf16.  The tensor cores multiply the blocks'
// scales in (tcgen05, kind mxf4nvf4, block_scale), so the whole sum over d stays
// in tensor memory in fp32 and only the rows' factors are left to the epilogue.
//
// Two shapes of one kernel, as for e4m3.  PAIR false (M <= 128, and where a pair's
// second CTA would have few rows): a CTA per SM, tiles of 128 rows x NB ids; W
// streams through.  PAIR true: a cluster of two CTAs on a pair of SMs, tiles of 256
// rows x NB ids, each CTA loading its 128 rows of h and half of the tile of W.  With
// many rows what bounds a stage is the round trip of its shared memory (MMA, commit,
// wait, load from L2, wait: about 2 us) over the stages that fit; a pair then forms
// two tiles of rows at a time from one tile of W, one in each accumulator (H 2),
// which halves what W takes of a stage.  Tiles are walked rows fastest.
//
// Warp 0 loads: a stage is 256 hidden dims, one 128-byte swizzle row of 4-bit
// values, with the 512-byte scale tiles that belong to it (both CTAs of a pair
// take the scales of all NB ids: each forms all columns of its rows).  Warp 1
// issues: the stage's scale tiles from shared into tensor memory (tcgen05.cp,
// the four lane quarters get copies), then an MMA for each 64 dims.  Copies and
// MMAs of one thread run in order, and two sets of scale columns alternate.
// Warps 2..9 are the epilogue, two for each 32 rows: two accumulators, so that a
// tile is read, scaled and stored (box by box through shared memory, as for e4m3)
// while the next is formed.
// Where a product of two factors may leave fp32's range a tile goes a way of its own
// (by way of fp64; inside the usual one it took M 131 from 16.3 to 17.3 us).
// 512 tensor-memory columns: 2 x 192 of sums, 2 x 64 of scales, hence NB <= 192.
// (A set: 16 columns for each row tile, 32 for the ids.)  Ids start at a multiple of
// 64 of their scale tile: two columns.
// Every wait is bounded (l8_wait), with lm_head_kernel's teardown.
//
// Measured (replayed; GB300): M 2304, V 151936, d 4096: 471 to 493 us = 5.8 to 6.1
// PFLOP/s; 532 with one row tile a pair and five stages.  In blocks of 32: 462 us.  M 64,
// V 128256, d 2048, blocks of 32: 27 us = 5.8 TB/s; M 1, V 32000, d 4096: 16 us = 4.5 TB/s,
// bound by the weights' bytes and some 5 us of launch, first loads and last tile.  M 131,
// V 32003, d 1056: 16 us, three tiles a pair and odd rows' plain stores.
// What bounds many rows is a stage's round trip, no single unit: at M 2304, V 32768 (117
// us) the tensor pipe is active 56 % of the time, which fits MMAs of 64 dims at 2 cycles an
// id (9.4 PFLOP/s if they never paused), L2 44 %, memory 20 %.  The first case took 380
// instead of 484 us with three quarters of the MMAs left out, 457 without the scales'
// copies, 472 with the first lines loaded again and again.
#pragma once

#include <type_traits>

#include "sv_lmhead_fp4_plan.h"
#include "sv_lmhead_fp8.cuh"

namespace sv {

constexpr int kL4BK = 256;                 // hidden dims of a stage
static_assert(kL4Rows == kLmBM, "rows of a tile");
constexpr int kL4EpiWarps = 8;             // two a lane quarter, each half of a tile's columns
constexpr int kL4Threads = 64 + 32 * kL4EpiWarps;
constexpr int kL4MaxStages = 8;
constexpr uint32_t kL4TmemCols = 512;
constexpr uint32_t kL4ScaleCol = 2 * kL4MaxNB; // first of 2 x 64 scale columns
// Shared memory: what the epilogue warps stage, 32 factors for each of them, then the
// ring, behind whose last stage lm4_launch leaves what the MMA reads of its 128 rows
// where a stage has fewer.  Tensor stores take a box of 32 rows x 32 logits at a time;
// rows that are no whole 16-byte units leave by plain stores (l8_store_rows), half a
// tile's 96 logits at a time, since each row's two ends go logit by logit (box by box
// 19.0 instead of 16.6 us at M 131, V 32003), and the ring has 32 KiB less.
constexpr int kL4Gws = kL4EpiWarps * 128;
constexpr int kL4StgTma = kL8BoxBytes, kL4StgPlain = kL4MaxNB / 64 * kL8BoxBytes; // of a warp
constexpr int kL4Bytes = 225 * 1024;                                              // staged, factors, ring
constexpr int kL4Smem = 1024 + kL4Bytes;
static_assert(kL4Smem <= 227 * 1024 - 512, "shared memory of a CTA, less the barriers");
// the ring's place: a multiple of 1024
inline int l4_front(bool tma) { return kL4EpiWarps * (tma ? kL4StgTma : kL4StgPlain) + kL4Gws; }
static_assert(kL4EpiWarps * kL4StgTma % 1024 == 0 && kL4EpiWarps * kL4StgPlain % 1024 == 0 && kL4Gws == 1024, "swizzled tiles");

struct Lm4Params {
    Lm8Params t;              // M, N, tiles (MT: groups of row tiles), logits, status (its own scales and sums unused)
    int32_t RT;               // row tiles
    int32_t front;            // bytes of shared memory before the ring
    int32_t d;                // hidden dims
    int32_t KT;               // scale tiles along d
    int32_t blocks;           // scale tiles across a tile's ids: 1 or 2
    uint32_t idesc;
    const float *gh, *gw;     // [M], [N] factors, or nullptr
};

// Tensor map coordinates and copies ---------------------------------------

// 16-byte rows without swizzle, 8-row groups 128 bytes apart: a 512-byte scale
// tile as tcgen05.cp reads it (32 rows x 128 bits).
__device__ __forceinline__ uint64_t l4_scale_desc(uint32_t saddr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(1u) << 16;          // leading byte offset (one column of 16 bytes: unused)
    d |= static_cast<uint64_t>(128u >> 4) << 32;   // stride byte offset
    d |= static_cast<uint64_t>(1u) << 46;          // descriptor version
    return d;                                      // no swizzle
}

template <bool PAIR> __device__ __forceinline__ void l4_copy_scales(uint32_t taddr, uint64_t desc)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <bool PAIR, int BLOCK>
__device__ __forceinline__ void l4_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sa,
                                       uint32_t sb, uint32_t acc)
{
#define SV_L4_MMA(GROUP, VEC)                                                                                          \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                                     \
                 "tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC                         \
                 " [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),                                               \
                 "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(sa), "r"(sb)                                        \
                 : "memory")
    if constexpr (PAIR && BLOCK == 16)
        SV_L4_MMA("2", "4X");
    else if constexpr (PAIR)
        SV_L4_MMA("2", "2X");
    else if constexpr (BLOCK == 16)
        SV_L4_MMA("1", "4X");
    else
        SV_L4_MMA("1", "2X");
#undef SV_L4_MMA
}

// Instruction descriptor: D fp32, A and B e2m1, both K-major, scales e4m3
// (block 16) or e8m0; the scale bytes used are the word's first.
inline uint32_t l4_idesc(int rows, int ids, int block)
{
    return (1u << 7) | (1u << 10) | ((static_cast<uint32_t>(ids) >> 3) << 17) | (block == 32 ? 1u << 23 : 0u) |
           ((static_cast<uint32_t>(rows) >> 4) << 24);
}

__device__ __forceinline__ float4 l4_lds4(uint32_t addr)
{
    float4 r;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(addr) : "memory");
    return r;
}

// Two logits, NaN where bf16 cannot hold them (-inf is a masked token to what reads
// them): an infinity, of the product or of its rounding, times 0 is NaN, and x * 0 + x
// is x for the others.
__device__ __forceinline__ uint32_t l4_round(float x0, float x1)
{
    const uint32_t p = bf16_rn_pair(x0, x1);
    uint32_t r;
    asm("{\n\t.reg .b32 z;\n\tmov.b32 z, 0;\n\tfma.rn.bf16x2 %0, %1, z, %1;\n\t}" : "=r"(r) : "r"(p));
    return r;
}

// Whether a factor is 0 or in [2^-63, 2^64): the product of two such is 0 by a factor or
// in fp32's normal range.
__device__ __forceinline__ bool l4_mild(float f)
{
    const uint32_t b = __float_as_uint(f) & 0x7FFFFFFFu;
    return b == 0 || b - 0x20000000u < 0x3F800000u;
}
// x gh gw.  WIDE: where gh gw leaves that range although the whole need not, by way of
// fp64, in which the product of the factors is exact; elsewhere what the short way gives.
template <bool WIDE> __device__ __forceinline__ float l4_scaled(float x, float gh, float gw)
{
    const float p = __fmul_rn(gh, gw);
    if (WIDE && (__float_as_uint(p) & 0x7FFFFFFFu) - 0x00800000u >= 0x7F000000u)
        return static_cast<float>(static_cast<double>(x) * (static_cast<double>(gh) * static_cast<double>(gw)));
    return __fmul_rn(x, p);
}

// The epilogue warps: warp w holds the tile's rows of tensor-memory lane quarter
// w mod 4, and the first or the second half of its ids.
template <bool PAIR, int H>
__device__ __forceinline__ void l4_epilogue(const Lm4Params &P, const CUtensorMap *map, uint32_t stg0, uint32_t tbase,
                                            uint32_t tfull, uint32_t tempty, int *stop, uint32_t rank, uint32_t unit,
                                            uint32_t units, uint32_t ntiles)
{
    const Lm8Params &T = P.t;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31u), lq = warp & 3;
    const int half = (warp - 2) >> 2, G = T.NB / 64; // groups of 32 ids: 1, 2 or 3
    const uint32_t stg = stg0 + static_cast<uint32_t>((warp - 2) * (T.tma ? kL4StgTma : kL4StgPlain));
    const uint32_t gws = stg0 + static_cast<uint32_t>(P.front - kL4Gws + (warp - 2) * 128);
    const uint32_t te = PAIR ? lm_mapa(tempty, 0) : tempty;
    bool alive = true, sent = false;
    uint32_t i = 0; // row tiles so far: accumulator i mod 2
    uint32_t t = unit, sub = 0;
    for (; t < ntiles; ++i) {
        const uint32_t a = i & 1u;
        const uint32_t m = l8_tile_m(T, t) * H + sub; // row tile
        const int row0 = static_cast<int>((m * (PAIR ? 2u : 1u) + rank) * kLmBM) + lq * 32;
        const int n0 = static_cast<int>(l8_tile_n(T, t)) * T.NB + half * G * 32;
        // the rows' and ids' factors, while the tile is formed
        float gh = 1.0f, gw[kL4MaxNB / 64];
        if (P.gh) {
            gh = row0 + lane < T.M ? __ldg(P.gh + row0 + lane) : 0.0f;
#pragma unroll
            for (int g = 0; g < kL4MaxNB / 64; ++g)
                gw[g] = g < G && n0 + 32 * g + lane < T.N ? __ldg(P.gw + n0 + 32 * g + lane) : 0.0f;
        }
        alive = __all_sync(0xFFFFFFFFu, l8_wait(tfull + a * 8u, (i >> 1) & 1u));
        if (!alive)
            break;
        lm_tc_after();
        const bool in = row0 < T.M && n0 < T.N;
        bool mild = true;
        if (P.gh) {
            mild = l4_mild(gh);
#pragma unroll
            for (int g = 0; g < kL4MaxNB / 64; ++g)
                mild = mild && l4_mild(gw[g]);
            mild = __all_sync(0xFFFFFFFFu, mild);
        }
        const uint32_t tl = tbase + (static_cast<uint32_t>(lq) << 21) + a * kL4MaxNB + static_cast<uint32_t>(half * G * 32);
        uint32_t v[2][32]; // the next group is on its way while one is scaled
        // the ids' factors of a group, read by every lane
        auto put_factors = [&](float f) {
            if (P.gh) {
                __syncwarp();
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(gws + static_cast<uint32_t>(lane) * 4u), "f"(f) : "memory");
                __syncwarp();
            }
        };
        auto release = [&] { // this warp has read the accumulator
            lm_tc_before();
            __syncwarp();
            if (lane == 0)
                l8_arrive(te + a * 8u);
        };
        // group g's sums times their factors (in WIDE form where the product of two may leave
        // fp32's range), rounded, staged and sent
        auto group = [&](int g, const uint32_t (&x)[32], auto wide) {
            constexpr bool WIDE = decltype(wide)::value;
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float4 w = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                if (P.gh)
                    w = l4_lds4(gws + static_cast<uint32_t>(4 * k) * 4u);
                pk[2 * k] = l4_round(l4_scaled<WIDE>(__uint_as_float(x[4 * k]), gh, w.x),
                                     l4_scaled<WIDE>(__uint_as_float(x[4 * k + 1]), gh, w.y));
                pk[2 * k + 1] = l4_round(l4_scaled<WIDE>(__uint_as_float(x[4 * k + 2]), gh, w.z),
                                         l4_scaled<WIDE>(__uint_as_float(x[4 * k + 3]), gh, w.w));
            }
            if (T.tma && sent) // the last store has read the box
                l8_stores_read();
            __syncwarp();
            l8_stage(T.tma ? stg : stg + g * kL8BoxBytes, pk, lane);
            const int n = n0 + 32 * g;
            if (T.tma) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (l8_elect() && n < T.N) {
                    l8_send(map, stg, n, row0);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
                sent = true;
            }
        };
        if (in && mild) {
            l8_ld_start(tl, v[0]);
#pragma unroll
            for (int g = 0; g < kL4MaxNB / 64; ++g) {
                if (g < G) {
                    put_factors(gw[g]);
                    l8_ld_wait(v[g & 1]);
                    if (g + 1 < G)
                        l8_ld_start(tl + 32 * (g + 1), v[(g + 1) & 1]);
                    else
                        release();
                    group(g, v[g & 1], std::false_type{});
                }
            }
        } else if (in) {
#pragma unroll 1
            for (int g = 0; g < G; ++g) {
                put_factors(g == 0 ? gw[0] : (g == 1 ? gw[1] : gw[2]));
                l8_ld_start(tl + 32 * g, v[0]);
                l8_ld_wait(v[0]);
                if (g + 1 == G)
                    release();
                group(g, v[0], std::true_type{});
            }
        } else {
            release();
        }
        if (in && !T.tma) {
            __syncwarp();
            uint32_t boxes = stg;
            l8_staged_now(boxes);
            l8_store_rows<kL4MaxNB / 64>(T, boxes, row0, n0, T.N - n0 < G * 32 ? T.N - n0 : G * 32, lane);
            __syncwarp();
        }
        if (++sub == H || m + 1 == static_cast<uint32_t>(P.RT)) {
            sub = 0;
            t += units;
        }
    }
    if (!alive && lane == 0)
        l8_fail(T, stop);
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); // this lane's stores are done
}

// Unit u (a pair of SMs, or one) takes tiles u, u + units, ...
template <bool PAIR, int H, int BLOCK>
__global__ void __launch_bounds__(kL4Threads, 1)
    lm_head_fp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                       const __grid_constant__ CUtensorMap tmC, const __grid_constant__ Lm4Params P)
{
    constexpr int kCtas = PAIR ? 2 : 1;
    constexpr int kDimsPerTile = 4 * BLOCK;            // hidden dims of a scale tile
    constexpr int kTiles = kL4BK / kDimsPerTile;       // scale tiles of a stage: 4 or 2
    extern __shared__ uint8_t lm_smem_raw[];
    __shared__ __align__(8) unsigned long long full[kL4MaxStages], empty[kL4MaxStages], tfull[2], tempty[2], drain;
    __shared__ uint32_t tmem_base;
    __shared__ int stop;
    const Lm8Params &T = P.t;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(lm_smem_raw) + 1023) & ~uintptr_t{1023});
    const uint32_t front = smem_addr(smem), sbase = front + static_cast<uint32_t>(P.front);
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? lm_cluster_rank() : 0u;
    const bool leader = rank == 0;
    const uint32_t unit = blockIdx.x / kCtas, units = gridDim.x / kCtas;
    const uint32_t ntiles = static_cast<uint32_t>(T.MT) * static_cast<uint32_t>(T.NT);
    const uint32_t abytes = static_cast<uint32_t>(T.a_rows) * 128u, bbytes = static_cast<uint32_t>(T.NB / kCtas) * 128u;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kL4MaxStages; ++s) {
            lm_mbar_init(smem_addr(&full[s]), 1);  // the leader's arrival with every CTA's bytes
            lm_mbar_init(smem_addr(&empty[s]), 1); // the MMAs of the stage
        }
        for (int a = 0; a < 2; ++a) {
            lm_mbar_init(smem_addr(&tfull[a]), 1);
            lm_mbar_init(smem_addr(&tempty[a]), kCtas * kL4EpiWarps);
        }
        lm_mbar_init(smem_addr(&drain), 1);
        stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1)
        l8_tmem_alloc<PAIR>(smem_addr(&tmem_base), kL4TmemCols);
    lm_tc_before();
    __syncthreads();
    l8_cluster_sync<PAIR>(); // every CTA's barriers exist before another CTA signals them
    lm_tc_after();
    const uint32_t tbase = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);
    pdl_wait_primary();
    pdl_launch_dependents();

    if (warp == 0) {
        int s = 0;
        uint32_t ph = 0;
        bool wrapped = false, ok = true;
        const uint32_t fb0 = PAIR ? lm_mapa(smem_addr(&full[0]), 0) : smem_addr(&full[0]);
        for (uint32_t t = unit; t < ntiles && ok; t += units) {
            const int m = static_cast<int>(l8_tile_m(T, t)) * H, n0 = static_cast<int>(l8_tile_n(T, t)) * T.NB;
            const int subs = P.RT - m < H ? P.RT - m : H; // row tiles of this group
            const int sb0 = (n0 >> 7) * P.KT;
            const uint32_t bytes = kCtas * (subs * (abytes + kTiles * 512) + bbytes + static_cast<uint32_t>(kTiles * 512 * P.blocks));
            for (int kb = 0; kb < T.KB; ++kb) {
                if (wrapped && !__all_sync(0xFFFFFFFFu, l8_wait(smem_addr(&empty[s]), ph ^ 1u))) {
                    ok = false;
                    break;
                }
                if (l8_elect()) {
                    uint32_t dst = sbase + static_cast<uint32_t>(s * T.stage_bytes);
                    const uint32_t fb = fb0 + static_cast<uint32_t>(s * 8);
                    if (leader)
                        lm_mbar_expect(smem_addr(&full[s]), bytes);
                    for (int h = 0; h < subs; ++h)
                        l8_tma_2d<PAIR>(dst + h * abytes, &tmA, kb * 128, ((m + h) * kCtas + static_cast<int>(rank)) * kLmBM, fb);
                    dst += H * abytes;
                    l8_tma_2d<PAIR>(dst, &tmB, kb * 128, n0 + static_cast<int>(rank) * (T.NB / kCtas), fb);
                    dst += bbytes;
                    for (int h = 0; h < subs; ++h)
                        l8_tma_2d<PAIR>(dst + h * kTiles * 512, &tmSA, 0,
                                        ((m + h) * kCtas + static_cast<int>(rank)) * P.KT + kb * kTiles, fb);
                    dst += H * kTiles * 512;
                    l8_tma_2d<PAIR>(dst, &tmSB, 0, sb0 + kb * kTiles, fb);
                    if (P.blocks == 2)
                        l8_tma_2d<PAIR>(dst + kTiles * 512, &tmSB, 0, sb0 + P.KT + kb * kTiles, fb);
                }
                __syncwarp();
                if (++s == T.stages) {
                    s = 0;
                    ph ^= 1u;
                    wrapped = true;
                }
            }
        }
        // every stage's last MMAs have signalled this CTA's barriers before
        // its shared memory goes
        int left = wrapped ? T.stages : s;
        if (!wrapped) {
            s = 0;
            ph = 1u;
        }
        for (; ok && left > 0; --left) {
            ok = __all_sync(0xFFFFFFFFu, l8_wait(smem_addr(&empty[s]), ph ^ 1u));
            if (++s == T.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
        if (!ok && lane == 0)
            l8_fail(T, &stop);
    } else if (warp == 1) {
        if (leader) {
            const uint64_t ad0 = lm_desc(sbase), bd0 = lm_desc(sbase + H * abytes);
            const uint64_t sd0 = l4_scale_desc(sbase + H * abytes + bbytes);
            int s = 0;
            uint32_t ph = 0, i = 0, set = 0; // i: row tiles so far, accumulator i mod 2
            bool ok = true;
            for (uint32_t t = unit; t < ntiles && ok; t += units) {
                const int m = static_cast<int>(l8_tile_m(T, t)) * H;
                const int subs = P.RT - m < H ? P.RT - m : H;
                const uint32_t shift = ((l8_tile_n(T, t) * static_cast<uint32_t>(T.NB)) & 127u) >> 5; // 0 or 2 columns
                for (int kb = 0; kb < T.KB && ok; ++kb) {
                    if (!__all_sync(0xFFFFFFFFu, l8_wait(smem_addr(&full[s]), ph))) {
                        ok = false;
                        break;
                    }
                    const uint64_t so = static_cast<uint64_t>((s * T.stage_bytes) >> 4);
                    const uint32_t sa0 = tbase + kL4ScaleCol + set * 64u, sb = sa0 + H * kTiles * 4u;
                    #pragma unroll
                    for (int h = 0; h < H; ++h) {
                        if (h >= subs)
                            break;
                        const uint32_t j = i + h, a = j & 1u;
                        if (kb == 0 && j >= 2 &&
                            !__all_sync(0xFFFFFFFFu, l8_wait(smem_addr(&tempty[a]), ((j >> 1) & 1u) ^ 1u))) {
                            ok = false;
                            break;
                        }
                        lm_tc_after();
                        if (l8_elect()) {
                            const uint32_t sa = sa0 + h * kTiles * 4u, tacc = tbase + a * kL4MaxNB;
                            const uint64_t ad = ad0 + so + static_cast<uint64_t>(h * static_cast<int>(abytes >> 4));
                            const uint64_t sd = sd0 + so;
                            const int left = P.d - kb * kL4BK; // hidden dims from here on
#pragma unroll
                            for (int k = 0; k < kTiles; ++k) {
                                l4_copy_scales<PAIR>(sa + 4 * k, sd + static_cast<uint64_t>((h * kTiles + k) * 32));
                                if (h == 0) {
                                    l4_copy_scales<PAIR>(sb + 4 * P.blocks * k, sd + static_cast<uint64_t>((H * kTiles + k) * 32));
                                    if (P.blocks == 2)
                                        l4_copy_scales<PAIR>(sb + 8 * k + 4, sd + static_cast<uint64_t>(((H + 1) * kTiles + k) * 32));
                                }
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (k * 64 >= left)
                                    break;
                                const int tile = k * 64 / kDimsPerTile; // of the stage's scale tiles
                                // two scales a row and MMA: the first or the second half of the word
                                const uint32_t half = BLOCK == 32 && (k & 1) ? (2u << 29) | (2u << 4) : 0u;
                                l4_mma<PAIR, BLOCK>(tacc, ad + static_cast<uint64_t>(k * 2),
                                                    bd0 + so + static_cast<uint64_t>(k * 2), P.idesc | half, sa + 4 * tile,
                                                    sb + 4 * P.blocks * tile + shift, (kb | k) ? 1u : 0u);
                            }
                            if (h == subs - 1)
                                l8_commit<PAIR>(smem_addr(&empty[s]));
                            if (kb == T.KB - 1)
                                l8_commit<PAIR>(smem_addr(&tfull[a]));
                        }
                        __syncwarp();
                    }
                    set ^= 1u;
                    if (++s == T.stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                i += subs;
            }
            if (!ok && lane == 0)
                l8_fail(T, &stop);
        }
    } else {
        l4_epilogue<PAIR, H>(P, &tmC, front, tbase, smem_addr(&tfull[0]), smem_addr(&tempty[0]), &stop, rank, unit, units,
                             ntiles);
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
        if (warp == 1 && leader && l8_elect()) { // every MMA issued is done
            if constexpr (PAIR)
                lm_commit_local(smem_addr(&drain));
            else
                l8_commit<PAIR>(smem_addr(&drain));
            (void)l8_wait(smem_addr(&drain), 0u);
        }
    }
    __syncthreads();
    l8_cluster_sync<PAIR>(); // no CTA's memory goes while the MMAs or signals may still use it
    if (warp == 1) {
        lm_tc_after();
        l8_tmem_dealloc<PAIR>(tbase, kL4TmemCols);
    }
}

} // namespace sv
