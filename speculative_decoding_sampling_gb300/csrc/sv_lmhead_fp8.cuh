// sv_lmhead_fp8.cuh -- the target's LM head on e4m3 operands whose scales
// belong to blocks of 128.
//
//   z[m, v] = sum_b hs[m, b] ws[v / 128, b] sum_{k in block b} h[m, k] W[v, k]
//
// h e4m3 [M, d] with a scale per row and 128 hidden dims, W e4m3 [V, d] with
// a scale per 128 ids x 128 hidden dims; z is rounded once to bf16.  The
// inner sums (fp32 sums of 128 products, each exact) run on the tensor cores
// (tcgen05, kind f8f6f4) into tensor memory; the scales differ from block to
// block and are not powers of two, so each block's sums are read back and
// folded into fp32 accumulators in registers: one fp32 multiply-add per logit
// and block, while the tensor cores form the next block's sums.
//
// Two shapes of one kernel.  PAIR false (M <= 128, and the row counts of
// several tiles that fill pairs badly: lm8_plan): a CTA per SM, tiles of 128
// rows x NB ids; few rows leave the tensor cores idle most of the time and the
// kernel streams W.  PAIR true: a cluster of two CTAs on a pair of SMs, tiles
// of 256 rows x NB ids, each CTA loading its 128 rows of h and half of the
// tile of W (one tcgen05.mma of M 256 reads both), which halves what each SM
// takes from L2.  Tiles are walked rows fastest, so the CTAs running at one
// time share a few tiles of W.
//
// Warp 0 loads (2-D tensor-memory-accelerator boxes of 128 hidden dims, one
// 128-byte swizzle row each); warps 1 and 2 issue the MMAs.  A step (128
// hidden dims) is two MMA groups, the first 128 columns of the tile (warp 1)
// and the rest (warp 2), each with its own half of one of two tensor-memory
// buffers and its own barriers: the sums of one half are read while the other
// half is formed, and neither warp's waits and commits (a few hundred cycles a
// step) hold up the other's MMAs.  Warp 3 brings the scales of 16 steps at a
// time into shared memory.  Warps 4..11 hold the accumulators (32 rows x 128 columns a
// warp, 128 registers a thread); they read the sums 64 columns ahead of the
// multiply-adds, and hand a buffer back before its last ones.  A finished tile
// goes through shared memory: tensor stores take it out behind the
// accumulator warps' backs, and warps 12..15 form each row's statistics from
// it (the fused verification), or store it where the logits' rows are not
// whole 16-byte units -- an SM gets rid of about 16 bytes a cycle while all of
// them write, so a warp that stores itself waits thousands of cycles a tile.
// Every wait is bounded (l8_wait), with lm_head_kernel's teardown.
//
// Measured (graph replay, weights larger than L2 or rotated): M 2304, V 151936,
// d 4096: 1.00 ms = 2870 TFLOP/s in a burst (1.14 ms under the power cap), the
// tensor pipe 61 % active; bound by the round trip of a buffer (MMA, commit,
// wait, read, hand back, wait: ~1400 cycles for two buffers' 2 x 512).  M 384,
// V 128256: 176 us (three row tiles on single CTAs).  M 8, V 151936:
// 98 us = 6.3 TB/s, and M 1, V 32000: 26 us = 5.0 TB/s, bound by the weights'
// bytes, the latter with ~6 us of launch, first loads and last tile.
// What the parts were worth on the large shape: hand-back without a
// cluster-scope release 3150 -> 1580 us with the register split; two issuing
// warps, scales through shared memory and waits without clock reads -> 1233;
// tensor stores -> 1124; reading ahead over a step's end -> 991.
#pragma once

#include "sv_lmhead.cuh"

namespace sv {

constexpr int kL8BK = 128;    // hidden dims per step: one scale block, one swizzle row
constexpr int kL8MaxNB = 256; // ids per tile
constexpr int kL8AccWarps = 8;
constexpr int kL8Threads = 256 + 32 * kL8AccWarps;
// Registers a thread: 128 at launch (65,536 in all); the accumulators' two
// warpgroups then take 216 and the others keep 40 (65,536).
constexpr int kL8AccRegs = 216, kL8OtherRegs = 40;
static_assert(32 * kL8AccWarps * kL8AccRegs + 256 * kL8OtherRegs <= 128 * kL8Threads, "register split");
constexpr uint32_t kL8TmemCols = 2 * kL8MaxNB; // two fp32 sums of one step: all 512 columns
constexpr int kL8MaxStages = 8;
// Several row tiles share each tile of W and ask for it at about the same time,
// so all of them wait for memory; the unit with the first row tile asks for it
// this many steps earlier (4 to 12 time the same, 24 worse): 282 -> 268 us at
// M 576, V 128256, d 4096.  With one row tile asking early is slower (98 us
// became 112 or more at M 8, V 151936).
constexpr int kL8Ahead = 8;
constexpr int kL8Chunk = 16;                                       // steps whose scales are brought in at a time
constexpr int kL8HsPitch = kLmBM + 1;
constexpr int kL8TabFloats = kL8Chunk * kL8HsPitch + kL8Chunk * 8; // [step][row], [step][32-column group]
constexpr int kL8TabBytes = 2 * kL8TabFloats * 4;                  // two chunks
constexpr int kL8BoxBytes = 32 * 64;                               // 32 rows x 32 logits of a warp
constexpr int kL8StgBytes = 4 * kL8BoxBytes;                       // a warp's half tile
constexpr int kL8RingBytes = 144 * 1024;
constexpr int kL8Smem = 1024 + kL8RingBytes + kL8AccWarps * kL8StgBytes + kL8TabBytes;
static_assert(kL8Smem <= 227 * 1024 - 512, "shared memory of a CTA, less the barriers");

struct Lm8Params {
    int32_t M, N, KB;       // rows of h, vocabulary, scale blocks along the hidden dims
    uint64_t mt_inv;        // ceil(2^64 / MT) (0 for MT 1): t / MT is the high word of its product with t
    int32_t MT, NT, NB;     // row tiles, id tiles, ids per tile (a multiple of 32; of 64 on pairs)
    int32_t a_rows;         // rows of h in a stage (128, or fewer when M is small)
    int32_t stages, stage_bytes;
    uint32_t idesc[2];      // tcgen05 instruction descriptors of the two column halves
    const float *hs;        // [M, KB]
    const float *ws;        // [ceil(N / 128), KB]
    uint16_t *logits;       // [M, N] bf16 out
    float2 *part;           // [M, NT] (max, normaliser relative to fl(max c)) per tile, or nullptr
    int32_t halves;         // column halves of a tile: 1 (NB <= 128) or 2
    float c;                // log2(e) / T
    int32_t tma;            // N % 8 == 0 and 16-byte aligned logits: tensor stores
    int32_t *status;
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

// The box into L2.
__device__ __forceinline__ void l8_prefetch_2d(const CUtensorMap *map, int32_t c0, int32_t c1)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1)
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

// Start loading 32 consecutive fp32 columns of this thread's lane; the values
// are there after l8_ld_wait on them.
__device__ __forceinline__ void l8_ld_start(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}

// Registers of a load that an earlier l8_ld_wait covered.
__device__ __forceinline__ void l8_ld_tie(uint32_t (&r)[32])
{
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                      "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                      "+r"(r[15]));
    asm volatile("" : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                      "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                      "+r"(r[30]), "+r"(r[31]));
}

// Every load started before is done; the registers pass through, so no use of
// them moves ahead of the wait.
__device__ __forceinline__ void l8_ld_wait(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}

// One lane of the warp, the same one each time.
__device__ __forceinline__ bool l8_elect()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Wait for phase `parity` of `bar`: true once it is complete, false after
// kL8Tries tries, each of which the hardware may suspend for about a
// microsecond (a second in all; tens of milliseconds if it never suspends,
// against microseconds that a step takes).  One loop without calls or clock
// reads: some warps wait several times a step.
constexpr uint32_t kL8Tries = 1u << 20;
__device__ __forceinline__ bool l8_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t.reg .u32 n;\n\t"
                 "mov.u32 n, %3;\n\t"
                 "L8_TRY:\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
                 "@p bra L8_DONE;\n\t"
                 "sub.u32 n, n, 1;\n\t"
                 "setp.ne.u32 p, n, 0;\n\t"
                 "@p bra L8_TRY;\n\t"
                 "L8_DONE:\n\t"
                 "setp.ne.u32 p, n, 0;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity), "n"(kL8Tries)
                 : "memory");
    return ok != 0;
}

// Whether phase `parity` of `bar` is complete, without waiting.
__device__ __forceinline__ uint32_t l8_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok;
}

// Instruction descriptor: D fp32, A and B e4m3 (format 0), both K-major.
inline uint32_t l8_idesc(int rows, int ids)
{
    return (1u << 4) | ((static_cast<uint32_t>(ids) >> 3) << 17) | ((static_cast<uint32_t>(rows) >> 4) << 24);
}

// ------------------------------------------------------------- the parts

__device__ __forceinline__ uint32_t l8_round(unsigned long long pair)
{
    float lo, hi;
    unpack2(pair, lo, hi);
    return bf16_rn_pair(lo, hi);
}

// ------------------------------------------------------------- the kernel

// Columns of column half h of a tile.
__device__ __forceinline__ int l8_half_cols(int NB, int h)
{
    return h == 0 ? (NB < 128 ? NB : 128) : (NB > 128 ? NB - 128 : 0);
}

// Shared memory by its 32-bit address (a generic pointer would order these
// accesses with those to global memory).
__device__ __forceinline__ float l8_lds(uint32_t addr)
{
    float r;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
    return r;
}

__device__ __forceinline__ float2 l8_lds2(uint32_t addr)
{
    float2 r;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(r.x), "=f"(r.y) : "r"(addr) : "memory");
    return r;
}

// Four bytes from global memory (zero where `in` is false), without registers
// in between.
__device__ __forceinline__ void l8_copy4(uint32_t dst, const float *src, bool in)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}

__device__ __forceinline__ void l8_sts4(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A finished tile leaves through shared memory: boxes of 32 rows x 32 logits,
// 2 KiB in the 64-byte swizzle layout (neither side conflicts), which tensor
// stores take out behind the warp's back -- plain stores held the accumulator
// warps up for ~900 cycles per box.  Rows and ids past the ends are clipped by
// the map.

// This lane's row of a box, from 16 packed pairs.
__device__ __forceinline__ void l8_stage(uint32_t box, const uint32_t (&pk)[16], int lane)
{
#pragma unroll
    for (int q = 0; q < 4; ++q)
        l8_sts4(box + lane * 64 + ((q ^ (lane >> 1)) & 3) * 16,
                make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]));
}

// The box of ids n.. and rows row0.., staged by the whole warp before a proxy
// fence and a warp barrier; one lane, which commits the group.
__device__ __forceinline__ void l8_send(const CUtensorMap *map, uint32_t box, int n, int row0)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(n), "r"(row0), "r"(box)
                 : "memory");
}

// The tensor stores this lane issued have read their shared memory.
__device__ __forceinline__ void l8_stores_read()
{
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// This thread's index, read anew each time: what only a tile's end needs is
// then not kept in registers through its steps.
__device__ __forceinline__ uint32_t l8_tid()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(r));
    return r;
}

// How many tiles a unit has.
__device__ __forceinline__ uint32_t l8_tiles(uint32_t unit, uint32_t units, uint32_t ntiles)
{
    return unit < ntiles ? (ntiles - unit - 1) / units + 1 : 0;
}

// Tile t covers ids NB (t div MT) and row tile t mod MT.
__device__ __forceinline__ uint32_t l8_tile_n(const Lm8Params &P, uint32_t t)
{
    return P.MT == 1 ? t : static_cast<uint32_t>(__umul64hi(P.mt_inv, t));
}

__device__ __forceinline__ uint32_t l8_tile_m(const Lm8Params &P, uint32_t t)
{
    return t - l8_tile_n(P, t) * static_cast<uint32_t>(P.MT);
}

// First row of lane quarter lq of tile t.
template <bool PAIR>
__device__ __forceinline__ int l8_row0(const Lm8Params &P, uint32_t t, uint32_t rank, int lq)
{
    return static_cast<int>((l8_tile_m(P, t) * (PAIR ? 2u : 1u) + rank) * kLmBM) + lq * 32;
}

__device__ __forceinline__ void l8_fail(const Lm8Params &P, int *stop)
{
    if (!*static_cast<volatile int *>(stop)) {
        *static_cast<volatile int *>(stop) = 1;
        if (P.status)
            atomicOr(P.status, kTimeout);
    }
}

// The scales: step kb's row scales and those of the tile's eight 32-column
// groups, 16 steps at a time, two chunks in flight, by asynchronous copies (a
// warp that waits for loads of 68 values a lane in turn is too slow).
template <bool PAIR>
__device__ __forceinline__ void l8_scales(const Lm8Params &P, uint32_t tabs, uint32_t sfull, uint32_t sempty, int *stop,
                                          uint32_t rank, uint32_t unit, uint32_t units, uint32_t ntiles, int lane)
{
    const int k = lane & (kL8Chunk - 1), sub = lane >> 4; // step, and which of 2 rows
    uint32_t chunk = 0;
    for (uint32_t t = unit; t < ntiles; t += units) {
        const int m0 = static_cast<int>((l8_tile_m(P, t) * (PAIR ? 2u : 1u) + rank) * kLmBM);
        const int n0 = static_cast<int>(l8_tile_n(P, t)) * P.NB;
        const int rows = P.M - m0 < kLmBM ? P.M - m0 : kLmBM;
        for (int kb0 = 0; kb0 < P.KB; kb0 += kL8Chunk, ++chunk) {
            const uint32_t b = chunk & 1u;
            if (chunk >= 2 && !__all_sync(0xFFFFFFFFu, l8_wait(sempty + b * 8, ((chunk >> 1) & 1u) ^ 1u))) {
                if (lane == 0)
                    l8_fail(P, stop);
                return;
            }
            if (kb0 + k < P.KB) {
                uint32_t dst = tabs + (b * kL8TabFloats + static_cast<uint32_t>(k * kL8HsPitch + sub)) * 4u;
                const float *src = P.hs + static_cast<int64_t>(m0 + sub) * P.KB + kb0 + k;
#pragma unroll 8
                for (int r = sub; r < rows; r += 2, dst += 8, src += 2 * static_cast<int64_t>(P.KB))
                    l8_copy4(dst, src, true);
                const uint32_t wd = tabs + (b * kL8TabFloats + kL8Chunk * kL8HsPitch + static_cast<uint32_t>(k) * 8u) * 4u;
#pragma unroll
                for (int g = sub; g < 8; g += 2) {
                    const int n = n0 + g * 32;
                    const bool in = g * 32 < P.NB && n < P.N;
                    l8_copy4(wd + g * 4, P.ws + static_cast<int64_t>(in ? n >> 7 : 0) * P.KB + kb0 + k, in);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                l8_arrive(sfull + b * 8);
        }
    }
}

// The scale of a block's sums.  One that is infinite becomes NaN (f + 0 f): a
// block's sum times an infinity would be an infinity of either sign, and -inf
// is a masked token to what reads the logits.
__device__ __forceinline__ float l8_scale(float hs, float ws)
{
    const float f = __fmul_rn(hs, ws);
    return __fmaf_rn(f, 0.0f, f);
}

// acc += f * the 32 columns in v
__device__ __forceinline__ void l8_fold(unsigned long long *acc, const uint32_t (&v)[32], float f)
{
    const unsigned long long ff = pack2(f, f);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        acc[i] = fma2(pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), ff, acc[i]);
}

// Whether warps 12..15 have work: logits that tensor stores can not write, or
// the rows' statistics.
__device__ __forceinline__ bool l8_helpers(const Lm8Params &P) { return !P.tma || P.part; }

// Loads of staged logits that the compiler may batch and move, but not above
// l8_staged_now, which a finished wait for them is followed by.
__device__ __forceinline__ void l8_staged_now(uint32_t &boxes) { asm volatile("" : "+r"(boxes)::"memory"); }

__device__ __forceinline__ uint4 l8_staged4(uint32_t addr)
{
    uint4 r;
    asm("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
    return r;
}

__device__ __forceinline__ uint16_t l8_staged1(uint32_t addr)
{
    uint16_t r;
    asm("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(addr));
    return r;
}

// Where column c of a staged row r is.
__device__ __forceinline__ uint32_t l8_staged_at(uint32_t boxes, int r, int c)
{
    return boxes + static_cast<uint32_t>((c >> 5) * kL8BoxBytes + r * 64 + (((c >> 3) ^ (r >> 1)) & 3) * 16 + (c & 7) * 2);
}

// 8 halfwords from halfword a (0..7) on of the 16 in u, v.
__device__ __forceinline__ uint4 l8_shift(uint4 u, uint4 v, int a)
{
    uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 6; ++i)
        w[i] = a & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i)
        w[i] = a & 2 ? w[i + 1] : w[i];
    const uint32_t sel = a & 1 ? 0x5432u : 0x3210u;
    return make_uint4(__byte_perm(w[0], w[1], sel), __byte_perm(w[1], w[2], sel), __byte_perm(w[2], w[3], sel),
                      __byte_perm(w[3], w[4], sel));
}

// A half tile's staged rows (ncols <= 128 ids from n on) by plain stores, at
// whatever alignment they have: first their whole 16-byte units, 16 lanes a
// row, each shifted out of two staged units; then the logits before the first
// and behind the last unit (8 a row, or up to 14 where the vocabulary ends),
// 8 lanes a row.
__device__ __forceinline__ void l8_store_rows(const Lm8Params &P, uint32_t boxes, int row0, int n, int ncols, int lane)
{
    const int rows = P.M - row0 < 32 ? P.M - row0 : 32;
    uint16_t *const dst0 = P.logits + static_cast<int64_t>(row0) * P.N + n;
    auto columns_before_unit = [&](const uint16_t *dst) {
        return (8 - static_cast<int>(reinterpret_cast<uintptr_t>(dst) >> 1)) & 7;
    };
    {
        const int u = (lane & 15) * 8;
#pragma unroll 1
        for (int r0 = lane >> 4; r0 < rows; r0 += 4) {
            uint4 lo[2], hi[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                lo[i] = l8_staged4(l8_staged_at(boxes, (r0 + 2 * i) & 31, u));
                hi[i] = l8_staged4(l8_staged_at(boxes, (r0 + 2 * i) & 31, u < 120 ? u + 8 : u));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint16_t *dst = dst0 + static_cast<int64_t>(r0 + 2 * i) * P.N;
                const int lead = columns_before_unit(dst);
                if (r0 + 2 * i < rows && u + lead + 8 <= ncols)
                    *reinterpret_cast<uint4 *>(dst + u + lead) = l8_shift(lo[i], hi[i], lead);
            }
        }
    }
    const int c = lane & 7;
#pragma unroll 1
    for (int r0 = lane >> 3; r0 < rows; r0 += 16) {
        uint16_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int lead = columns_before_unit(dst0 + static_cast<int64_t>(r0 + 4 * i) * P.N);
            const int units = ncols > lead ? (ncols - lead) >> 3 : 0; // whole units
            const int first = lead < ncols ? lead : ncols, p = c < first ? c : units * 8 + c;
            v[i] = l8_staged1(l8_staged_at(boxes, (r0 + 4 * i) & 31, p < 128 ? p : 0));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 4 * i;
            uint16_t *dst = dst0 + static_cast<int64_t>(r) * P.N;
            const int lead = columns_before_unit(dst);
            const int units = ncols > lead ? (ncols - lead) >> 3 : 0, edges = ncols - units * 8;
            const int first = lead < ncols ? lead : ncols;
            if (r < rows && c < edges)
                dst[c < first ? c : units * 8 + c] = v[i];
            if (r < rows && c + 8 < edges) {
                const int p = c + 8 < first ? c + 8 : units * 8 + c + 8;
                dst[p] = l8_staged1(l8_staged_at(boxes, r, p));
            }
        }
    }
}

// The maximum and normaliser of staged row r over the tile's first ncols ids:
// the maximum, then the softmax terms against it, four sums side by side.
__device__ __forceinline__ float2 l8_statistics(const Lm8Params &P, uint32_t half0, uint32_t half1, int r, int ncols)
{
    float mx = -INFINITY;
#pragma unroll 4
    for (int c = 0; c < ncols; c += 8) {
        const uint4 v = l8_staged4(l8_staged_at(c < 128 ? half0 : half1, r, c & 127));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mx = c + 2 * i < ncols ? fmaxf(mx, bf16_lo(w[i])) : mx;
            mx = c + 2 * i + 1 < ncols ? fmaxf(mx, bf16_hi(w[i])) : mx;
        }
    }
    const float mc = mc_of(mx, P.c);
    float S[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int c = 0; c < ncols; c += 8) {
        const uint4 v = l8_staged4(l8_staged_at(c < 128 ? half0 : half1, r, c & 127));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = term(bf16_lo(w[i]), P.c, mc), b = term(bf16_hi(w[i]), P.c, mc);
            S[i] += (c + 2 * i < ncols ? a : 0.0f) + (c + 2 * i + 1 < ncols ? b : 0.0f);
        }
    }
    return make_float2(mx, (S[0] + S[1]) + (S[2] + S[3]));
}

// Warps 12..15: warp 12 + lq works on the staged rows of lane quarter lq.
template <bool PAIR>
__device__ __forceinline__ void l8_finish(const Lm8Params &P, uint32_t tabs, uint32_t staged, uint32_t sfree, int *stop,
                                          uint32_t rank, uint32_t unit, uint32_t units, uint32_t ntiles, int lq, int lane)
{
    uint32_t odd = 0;
    uint32_t half0 = tabs - static_cast<uint32_t>(8 - lq) * kL8StgBytes;
    for (uint32_t t = unit; t < ntiles; t += units, odd ^= 1u) {
        if (!__all_sync(0xFFFFFFFFu, l8_wait(staged, odd))) {
            if (lane == 0)
                l8_fail(P, stop);
            return;
        }
        l8_staged_now(half0);
        const uint32_t half1 = half0 + 4 * kL8StgBytes;
        const int row0 = l8_row0<PAIR>(P, t, rank, lq), tn = static_cast<int>(l8_tile_n(P, t)), n0 = tn * P.NB;
        const int ncols = P.N - n0 < P.NB ? P.N - n0 : P.NB; // at least 1
        if (row0 < P.M) {
            if (!P.tma) {
                l8_store_rows(P, half0, row0, n0, ncols < 128 ? ncols : 128, lane);
                if (ncols > 128)
                    l8_store_rows(P, half1, row0, n0 + 128, ncols - 128, lane);
            }
            if (P.part) {
                const float2 ms = l8_statistics(P, half0, half1, lane, ncols);
                if (row0 + lane < P.M)
                    P.part[static_cast<int64_t>(row0 + lane) * P.NT + tn] = ms;
            }
        }
        __syncwarp();
        if (lane == 0)
            l8_arrive(sfree);
    }
}

// What a warp's steps go by.
struct L8Steps {
    uint32_t tl;                     // tensor-memory address of the warp's rows and column half
    uint32_t tfull, tempty;          // barriers of buffer 0 (buffer 1's are 16 bytes on)
    uint32_t hsp, wsp;               // this step's scales in shared memory
    uint32_t it;                     // steps so far
    bool ok;                         // no wait of this lane has run out
    __device__ __forceinline__ void wait()
    {
        if (ok)
            ok = l8_wait(tfull + (it & 1u) * 16u, (it >> 1) & 1u);
        __syncwarp();
        lm_tc_after();
    }
    // A wait costs ~180 cycles even where nothing is to be waited for, so the
    // next step's sums are asked for early, and waited for only if they were
    // not there.
    __device__ __forceinline__ uint32_t next_there() const
    {
        return l8_test(tfull + ((it + 1u) & 1u) * 16u, ((it + 1u) >> 1) & 1u);
    }
    __device__ __forceinline__ void wait_unless(uint32_t there)
    {
        if (!__all_sync(0xFFFFFFFFu, there != 0))
            wait();
        else
            lm_tc_after();
    }
    __device__ __forceinline__ uint32_t buffer() const { return tl + (it & 1u) * kL8MaxNB; }
    __device__ __forceinline__ void release() const // this warp has read the step's sums
    {
        lm_tc_before();
        __syncwarp();
        if ((l8_tid() & 31u) == 0)
            l8_arrive(tempty + (it & 1u) * 16u);
    }
    __device__ __forceinline__ void next()
    {
        ++it;
        hsp += kL8HsPitch * 4;
        wsp += 32;
    }
};

// Up to 16 steps of a warp whose half tile has all 128 columns.  The sums are
// read 64 columns at a time; the next ones are on their way while two 32s are
// folded in, over the end of a step too.
__device__ __forceinline__ void l8_steps_full(L8Steps &S, unsigned long long (&acc)[64], int steps)
{
    uint32_t v0[32], v1[32];
    S.wait();
    l8_ld_start(S.buffer(), v0);
    l8_ld_start(S.buffer() + 32, v1);
#pragma unroll 1
    for (; steps > 0; --steps) {
        const float hs = l8_lds(S.hsp);
        float2 ws = l8_lds2(S.wsp);
        l8_ld_wait(v0);
        l8_ld_tie(v1);
        l8_fold(acc, v0, l8_scale(hs, ws.x));
        l8_ld_start(S.buffer() + 64, v0);
        l8_fold(acc + 16, v1, l8_scale(hs, ws.y));
        l8_ld_start(S.buffer() + 96, v1);
        const uint32_t there = S.next_there();
        ws = l8_lds2(S.wsp + 8);
        l8_ld_wait(v0);
        l8_ld_tie(v1);
        S.release();
        S.next();
        l8_fold(acc + 32, v0, l8_scale(hs, ws.x));
        if (steps > 1) {
            S.wait_unless(there);
            l8_ld_start(S.buffer(), v0);
        }
        l8_fold(acc + 48, v1, l8_scale(hs, ws.y));
        if (steps > 1)
            l8_ld_start(S.buffer() + 32, v1);
    }
}

// The same for G < 4 32-column groups (none: rows past the end).
__device__ __forceinline__ void l8_steps_some(L8Steps &S, unsigned long long (&acc)[64], int steps, int G)
{
#pragma unroll 1
    for (; steps > 0; --steps) {
        S.wait();
        const float hs = l8_lds(S.hsp);
#pragma unroll
        for (int g = 0; g < 3; ++g)
            if (g < G) {
                uint32_t v[32];
                l8_ld_start(S.buffer() + 32 * g, v);
                const float2 ws = l8_lds2(S.wsp + (g >> 1) * 8);
                l8_ld_wait(v);
                l8_fold(acc + 16 * g, v, l8_scale(hs, g & 1 ? ws.y : ws.x));
            }
        S.release();
        S.next();
    }
}

// The accumulator warps: warp w (from 4 on) holds the tile's rows of
// tensor-memory lane quarter w mod 4 and column half (w - 4) / 4.
template <bool PAIR>
__device__ __forceinline__ void l8_accumulate(const Lm8Params &P, const CUtensorMap *map, uint32_t tabs, uint32_t tbase,
                                              uint32_t tfull, uint32_t tempty, uint32_t sfull, uint32_t sempty,
                                              uint32_t staged, uint32_t sfree, int *stop, uint32_t rank, uint32_t unit,
                                              uint32_t units, uint32_t ntiles)
{
    const int warp = static_cast<int>(l8_tid() >> 5), lane = static_cast<int>(l8_tid() & 31u);
    const int h = (warp - 4) >> 2, lq = warp & 3;
    const int groups = l8_half_cols(P.NB, h) / 32; // 32-column groups of this half: 0..4
    if (groups == 0)
        return;
    L8Steps S;
    S.tl = tbase + (static_cast<uint32_t>(lq) << 21) + static_cast<uint32_t>(h * 128);
    S.tfull = tfull + static_cast<uint32_t>(h) * 8u;
    S.tempty = (PAIR ? lm_mapa(tempty, 0) : tempty) + static_cast<uint32_t>(h) * 8u;
    S.it = 0;
    S.ok = true;
    uint32_t chunk = 0, odd = 0;
    bool alive = true;
    for (uint32_t t = unit; t < ntiles && alive; t += units) {
        const int G = l8_row0<PAIR>(P, t, rank, lq) < P.M ? groups : 0; // groups this warp folds
        unsigned long long acc[64];            // pairs of fp32 sums
#pragma unroll
        for (int i = 0; i < 64; ++i)
            acc[i] = 0;
        for (int kb0 = 0; kb0 < P.KB && alive; kb0 += kL8Chunk, ++chunk) {
            const uint32_t sb = chunk & 1u;
            S.ok = l8_wait(sfull + sb * 8, (chunk >> 1) & 1u);
            S.hsp = tabs + (sb * kL8TabFloats + static_cast<uint32_t>(lq * 32 + lane)) * 4u;
            S.wsp = tabs + (sb * kL8TabFloats + kL8Chunk * kL8HsPitch + static_cast<uint32_t>(h * 4)) * 4u;
            const int steps = P.KB - kb0 < kL8Chunk ? P.KB - kb0 : kL8Chunk;
            if (G == 4)
                l8_steps_full(S, acc, steps);
            else
                l8_steps_some(S, acc, steps, G);
            alive = __all_sync(0xFFFFFFFFu, S.ok);
            if (lane == 0) // this warp has read the chunk's scales
                l8_arrive(sempty + sb * 8);
        }
        if (!alive)
            break;
        // ---- the finished half tile
        const int warp = static_cast<int>(l8_tid() >> 5), lane = static_cast<int>(l8_tid() & 31u);
        const uint32_t stg = tabs - static_cast<uint32_t>(12 - warp) * kL8StgBytes;
        if (t != unit) { // the last tile's has left this warp's shared memory
            if (P.tma)
                l8_stores_read();
            if (l8_helpers(P))
                alive = l8_wait(sfree, odd ^ 1u);
        }
        if (!__all_sync(0xFFFFFFFFu, alive)) {
            alive = false;
            break;
        }
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (g < G) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    pk[i] = l8_round(acc[g * 16 + i]);
                l8_stage(stg + g * kL8BoxBytes, pk, lane);
            }
        if (P.tma)
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (l8_elect()) {
            if (P.tma) {
                const int n = static_cast<int>(l8_tile_n(P, t)) * P.NB + ((warp - 4) >> 2) * 128;
                const int row0 = l8_row0<PAIR>(P, t, rank, warp & 3);
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    if (g < G && n + 32 * g < P.N)
                        l8_send(map, stg + g * kL8BoxBytes, n + 32 * g, row0);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            if (l8_helpers(P))
                l8_arrive(staged);
        }
        odd ^= 1u;
    }
    if (!alive && lane == 0)
        l8_fail(P, stop);
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); // this lane's stores are done
}

// Unit u (a pair of SMs, or one) takes tiles u, u + units, ...; tile t covers
// row tile t mod MT and ids NB (t div MT).
template <bool PAIR>
__global__ void __launch_bounds__(kL8Threads, 1)
    lm_head_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmC, const __grid_constant__ Lm8Params P)
{
    constexpr int kCtas = PAIR ? 2 : 1;
    extern __shared__ uint8_t lm_smem_raw[];
    __shared__ __align__(8) unsigned long long full[kL8MaxStages], empty[kL8MaxStages], tfull[4], tempty[4],
        sfull[2], sempty[2], staged, sfree, drain;
    __shared__ uint32_t tmem_base;
    __shared__ int stop;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(lm_smem_raw) + 1023) & ~uintptr_t{1023});
    const uint32_t tabs = smem_addr(smem) + kL8RingBytes + kL8AccWarps * kL8StgBytes;
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? lm_cluster_rank() : 0u;
    const bool leader = rank == 0;
    const uint32_t unit = blockIdx.x / kCtas, units = gridDim.x / kCtas;
    const uint32_t ntiles = static_cast<uint32_t>(P.MT) * static_cast<uint32_t>(P.NT);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kL8MaxStages; ++s) {
            lm_mbar_init(smem_addr(&full[s]), 1);  // the leader's arrival with every CTA's bytes
            lm_mbar_init(smem_addr(&empty[s]), static_cast<uint32_t>(P.halves)); // the MMAs of the stage
        }
        for (int a = 0; a < 4; ++a) { // buffer a / 2, column half a mod 2
            lm_mbar_init(smem_addr(&tfull[a]), 1);
            lm_mbar_init(smem_addr(&tempty[a]), kCtas * kL8AccWarps / 2);
        }
        for (int a = 0; a < 2; ++a) {
            lm_mbar_init(smem_addr(&sfull[a]), 1);
            lm_mbar_init(smem_addr(&sempty[a]), static_cast<uint32_t>(P.halves) * kL8AccWarps / 2);
        }
        lm_mbar_init(smem_addr(&staged), static_cast<uint32_t>(P.halves) * kL8AccWarps / 2);
        lm_mbar_init(smem_addr(&sfree), 4);
        lm_mbar_init(smem_addr(&drain), 2);
        stop = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1)
        l8_tmem_alloc<PAIR>(smem_addr(&tmem_base), kL8TmemCols);
    lm_tc_before();
    __syncthreads();
    l8_cluster_sync<PAIR>(); // every CTA's barriers exist before another CTA signals them
    lm_tc_after();
    const uint32_t tbase = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);
    // Launched as a programmatic dependent: all of the above ran while the
    // kernel before drained.  Every thread waits for it here, so that no bounded
    // wait below counts the time that kernel still takes.
    pdl_wait_primary();
    pdl_launch_dependents();
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kL8OtherRegs));
        // Warps 0 and 1 run their loops as whole warps, so that addresses and
        // descriptors stay in uniform registers; one lane issues.
        if (warp == 0) {
            int s = 0;
            uint32_t ph = 0;
            bool wrapped = false;
            const uint32_t fb0 = PAIR ? lm_mapa(smem_addr(&full[0]), 0) : smem_addr(&full[0]);
            const uint32_t sbase = smem_addr(smem);
            const int brows = P.NB / kCtas; // ids of the tile this CTA loads: its share of each half
            const int box = l8_half_cols(P.NB, 0) / kCtas;
            const uint32_t bytes = static_cast<uint32_t>(kCtas * (P.a_rows + brows) * kL8BK);
            bool ok = true;
            uint32_t pt = unit; // kL8Ahead steps on: tile, step and first id (-1: not this unit's to ask for)
            int pkb = kL8Ahead, pn = -1;
            auto settle = [&]() {
                while (pkb >= P.KB && pt < ntiles) {
                    pkb -= P.KB;
                    pt += units;
                }
                pn = P.MT > 1 && pt < ntiles && l8_tile_m(P, pt) == 0
                         ? static_cast<int>(l8_tile_n(P, pt)) * P.NB + static_cast<int>(rank) * box
                         : -1;
            };
            settle();
            for (uint32_t t = unit; t < ntiles && ok; t += units) {
                const int m0 = static_cast<int>((l8_tile_m(P, t) * kCtas + rank) * kLmBM);
                const int n0 = static_cast<int>(l8_tile_n(P, t)) * P.NB + static_cast<int>(rank) * box;
                for (int kb = 0; kb < P.KB; ++kb) {
                    if (pn >= 0 && l8_elect()) {
                        l8_prefetch_2d(&tmB, pkb * kL8BK, pn);
                        if (PAIR && P.halves == 2)
                            l8_prefetch_2d(&tmB, pkb * kL8BK, pn + 128);
                    }
                    __syncwarp();
                    if (++pkb >= P.KB)
                        settle();
                    if (wrapped && !__all_sync(0xFFFFFFFFu, l8_wait(smem_addr(&empty[s]), ph ^ 1u))) {
                        ok = false;
                        break;
                    }
                    if (l8_elect()) {
                        const uint32_t sa = sbase + static_cast<uint32_t>(s * P.stage_bytes);
                        const uint32_t fb = fb0 + static_cast<uint32_t>(s * 8);
                        if (leader)
                            lm_mbar_expect(smem_addr(&full[s]), bytes);
                        l8_tma_2d<PAIR>(sa, &tmA, kb * kL8BK, m0, fb);
                        const uint32_t sb = sa + static_cast<uint32_t>(P.a_rows * kL8BK);
                        l8_tma_2d<PAIR>(sb, &tmB, kb * kL8BK, n0, fb);
                        if (PAIR && P.halves == 2)
                            l8_tma_2d<PAIR>(sb + static_cast<uint32_t>(box * kL8BK), &tmB, kb * kL8BK, n0 + 128, fb);
                    }
                    __syncwarp();
                    if (++s == P.stages) {
                        s = 0;
                        ph ^= 1u;
                        wrapped = true;
                    }
                }
            }
            // every stage's last MMAs have signalled this CTA's barriers before
            // its shared memory goes
            int left = wrapped ? P.stages : s;
            if (!wrapped) {
                s = 0;
                ph = 1u;
            }
            for (; ok && left > 0; --left) {
                ok = __all_sync(0xFFFFFFFFu, l8_wait(smem_addr(&empty[s]), ph ^ 1u));
                if (++s == P.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok && lane == 0)
                l8_fail(P, &stop);
        } else if (warp <= 2) {
            const int h = warp - 1; // the column half this warp issues
            const uint32_t idesc = h ? P.idesc[1] : P.idesc[0];
            const uint64_t ad0 = lm_desc(smem_addr(smem));
            const uint64_t bd0 = lm_desc(smem_addr(smem) + P.a_rows * kL8BK + h * (128 / kCtas * kL8BK));
            const uint32_t steps = leader && h < P.halves ? l8_tiles(unit, units, ntiles) * P.KB : 0u;
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            // step `it` forms its sums in tensor-memory buffer it mod 2
            for (uint32_t it = 0; it < steps; ++it) {
                const uint32_t b = it & 1u;
                ok = l8_wait(smem_addr(&full[s]), ph);
                if (it >= 2)
                    ok = l8_wait(smem_addr(&tempty[2 * b + h]), ((it >> 1) & 1u) ^ 1u) && ok;
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                lm_tc_after();
                const uint32_t tacc = tbase + b * kL8MaxNB + static_cast<uint32_t>(h * 128);
                const uint64_t so = static_cast<uint64_t>((s * P.stage_bytes) >> 4);
                if (l8_elect()) {
#pragma unroll
                    for (int k = 0; k < kL8BK / 32; ++k)
                        l8_mma<PAIR>(tacc, ad0 + so + static_cast<uint64_t>(k * 2),
                                     bd0 + so + static_cast<uint64_t>(k * 2), idesc, k ? 1u : 0u);
                    l8_commit<PAIR>(smem_addr(&tfull[2 * b + h]));
                    l8_commit<PAIR>(smem_addr(&empty[s]));
                }
                __syncwarp();
                if (++s == P.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok && lane == 0)
                l8_fail(P, &stop);
        } else {
            l8_scales<PAIR>(P, tabs, smem_addr(&sfull[0]), smem_addr(&sempty[0]), &stop, rank, unit, units, ntiles, lane);
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kL8AccRegs));
        l8_accumulate<PAIR>(P, &tmC, tabs, tbase, smem_addr(&tfull[0]), smem_addr(&tempty[0]), smem_addr(&sfull[0]),
                            smem_addr(&sempty[0]), smem_addr(&staged), smem_addr(&sfree), &stop, rank, unit, units,
                            ntiles);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kL8OtherRegs));
        if (l8_helpers(P))
            l8_finish<PAIR>(P, tabs, smem_addr(&staged), smem_addr(&sfree), &stop, rank, unit, units, ntiles, warp - 12,
                            lane);
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
        if ((warp == 1 || warp == 2) && leader && l8_elect()) { // every MMA issued is done
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
        l8_tmem_dealloc<PAIR>(tbase, kL8TmemCols);
    }
}

} // namespace sv
