// sv_block_norm.cuh -- the norms around the target's last block, fused with
// its gate and residual scale, and e4m3 block quantisation.
//
// Per row of d values, all in fp32:
//   a = x rsqrt(mean(x^2) + eps) (w_post + o)     (a = x without w_post)
//   r = rs residual + bs g a                      (g = 1 without a gate)
//   h = r rsqrt(mean(r^2) + eps) (w_pre + o)
// r is rounded once, to the residual's type, and h once, to its own; h is
// formed from r before that rounding.  An e4m3 h carries one fp32 scale per
// 128 values.
//
// A row is cut into segments of 256 values, one warp's 8 per lane; WPR warps
// hold a row in registers from the loads to the stores, so x, residual and
// gate are read once and r and h written once.  (Above 16384 values a lane has
// 64 of each, more than its registers hold, and some wait in local memory: 5
// rows of 32768 take 22.7 us, of 16384 9.2.)  The two row sums are warp sums
// joined through shared memory in a fixed order.  A few rows are bound by one
// launch's latency (5 rows of 4096: 4.0 us), so a row takes as many warps as it
// has segments; many rows take block_norm_rows_kernel, which adds a row's
// squares in another order, so h may differ from the same row's among few in
// its last bits.
#pragma once

#include "sv_device.cuh"

namespace sv {

constexpr int kSeg = 256;         // values of a segment: 8 per lane of a warp
constexpr int kNormMaxWarps = 16; // warps of a row
constexpr int kNormMaxSegs = 8;   // segments of a warp
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 0x1p-100f; // keeps the scale and its reciprocal normal numbers

enum ElemType { kElemBf16 = 0, kElemFp32 = 1, kElemE4m3 = 2 };

// Launched as a programmatic dependent: the CTAs are placed while the kernel
// before drains, and wait here for its memory; the next kernel may be placed in
// turn.
__device__ __forceinline__ void follow_primary()
{
    pdl_wait_primary();
    pdl_launch_dependents();
}

// The 8 values of a lane in a segment starting at `base`: consecutive ones
// (VEC: 16-byte accesses) or every 32nd (coalesced single accesses, for rows
// that are not whole 16-byte units).
template <bool VEC> __device__ __forceinline__ int seg_index(int base, int lane, int i)
{
    return VEC ? base + lane * 8 + i : base + i * 32 + lane;
}

__device__ __forceinline__ float elem_at(const void *p, int type, int64_t e)
{
    return type == kElemBf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[e]) << 16)
                             : static_cast<const float *>(p)[e];
}

// `row` points at the row's first element; values past d read as 0.  Plain
// loads, not the read-only path: the residual may be updated in place.
template <bool VEC>
__device__ __forceinline__ void seg_load(float (&v)[8], const void *row, int type, int base, int lane, int d)
{
    if constexpr (VEC) {
        const int e = base + lane * 8;
        if (e < d) { // d is a multiple of 8
            if (type == kElemBf16) {
                const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + e);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] = bf16_lo(w[i]);
                    v[2 * i + 1] = bf16_hi(w[i]);
                }
            } else {
                const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(row) + e);
                const float4 a = p[0], b = p[1];
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
                v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = seg_index<false>(base, lane, i);
            v[i] = e >= d ? 0.0f : elem_at(row, type, e);
        }
    }
}

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// two values as e4m3 bytes, nearest even, magnitudes above 448 to 448, NaN kept
__device__ __forceinline__ uint32_t e4m3x2_rn(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool VEC>
__device__ __forceinline__ void seg_store(const float (&v)[8], void *row, int type, int base, int lane, int d)
{
    if constexpr (VEC) {
        const int e = base + lane * 8;
        if (e >= d)
            return;
        if (type == kElemBf16) {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(row) + e) =
                make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
        } else if (type == kElemFp32) {
            float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(row) + e);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(row) + e) =
                make_uint2(e4m3x2_rn(v[0], v[1]) | e4m3x2_rn(v[2], v[3]) << 16,
                           e4m3x2_rn(v[4], v[5]) | e4m3x2_rn(v[6], v[7]) << 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = seg_index<false>(base, lane, i);
            if (e >= d)
                continue;
            if (type == kElemBf16)
                static_cast<uint16_t *>(row)[e] = static_cast<uint16_t>(bf16x2_rn(v[i], 0.0f));
            else if (type == kElemFp32)
                static_cast<float *>(row)[e] = v[i];
            else
                static_cast<uint8_t *>(row)[e] = static_cast<uint8_t>(e4m3x2_rn(v[i], 0.0f));
        }
    }
}

// the larger one; NaN if either is
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// amax / 448, correctly rounded: the product with the rounded reciprocal, then
// one correction by its exact remainder (Markstein's theorem: the quotient's
// estimate is within one unit of it, and no operand here is near the range's
// ends, thanks to the floor; infinite and NaN amax give themselves).
__device__ __forceinline__ float block_scale(float amax)
{
    const float a = max_nan(amax, kAmaxFloor), r = 1.0f / kE4m3Max;
    const float q = __fmul_rn(a, r);
    const float s = __fmaf_rn(__fmaf_rn(-kE4m3Max, q, a), r, q);
    return a < INFINITY ? s : a;
}

__device__ __forceinline__ uint32_t e4m3x4_scaled(float a, float b, float c, float d, float inv)
{
    return e4m3x2_rn(__fmul_rn(a, inv), __fmul_rn(b, inv)) | e4m3x2_rn(__fmul_rn(c, inv), __fmul_rn(d, inv)) << 16;
}

// A segment's two blocks of 128 as e4m3 with their scales.  VEC: lanes 0..15
// hold the first block, 16..31 the second; otherwise values 0..3 of every
// lane the first, 4..7 the second.
template <bool VEC>
__device__ __forceinline__ void seg_quantize(float (&v)[8], void *row, float *scale_row, int base, int lane, int d)
{
    float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a0 = max_nan(a0, fabsf(v[i]));
        a1 = max_nan(a1, fabsf(v[4 + i]));
    }
    if constexpr (VEC)
        a0 = max_nan(a0, a1);
#pragma unroll
    for (int o = VEC ? 8 : 16; o > 0; o >>= 1) {
        a0 = max_nan(a0, __shfl_xor_sync(0xFFFFFFFFu, a0, o));
        if constexpr (!VEC)
            a1 = max_nan(a1, __shfl_xor_sync(0xFFFFFFFFu, a1, o));
    }
    const float s0 = block_scale(a0), s1 = VEC ? s0 : block_scale(a1);
    const float i0 = __frcp_rn(s0), i1 = VEC ? i0 : __frcp_rn(s1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = __fmul_rn(v[i], i0);
        v[4 + i] = __fmul_rn(v[4 + i], i1);
    }
    seg_store<VEC>(v, row, kElemE4m3, base, lane, d);
    const int b = base / 128;
    if constexpr (VEC) {
        if ((lane & 15) == 0 && base + lane * 8 < d)
            scale_row[b + (lane >> 4)] = s0;
    } else {
        if (lane == 0 && base < d)
            scale_row[b] = s0;
        if (lane == 1 && base + 128 < d)
            scale_row[b + 1] = s1;
    }
}

// ------------------------------------------------------------- the norms

struct NormParams {
    const void *x, *residual, *post, *gate, *pre;
    int32_t x_type, r_type, w_type, h_type;
    int64_t M;
    uint32_t gate_div;   // row m is gated by row m / gate_div of the gate
    int32_t d, WPR, RPC; // warps per row (a power of two), rows per CTA
    float offset, rs, bs, eps;
    // Squares are added of values times sq_scale, a power of two at most
    // 1 / sqrt(d): a row's sum then stays at or below its mean square, and leaves
    // the fp32 range only where that does.  mean = sum * sq_inv_d (between 1 and
    // 4).  The same bits as without, at 1 % of the many-row norm's time.
    float sq_scale, sq_inv_d;
    void *r_out, *h;
    float *scales; // [M, ceil(d / 128)] (e4m3 h)
};

// Sum over the warps of a row; `red` has one float per warp of the CTA.  Every
// lane forms the same sum in the same order.
__device__ __forceinline__ float row_sum(float v, float *red, int warp, int first, int WPR)
{
    v = warp_sum_f(v);
    if (WPR == 1)
        return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0)
        red[warp] = v;
    __syncthreads();
    float s = red[first + (lane & (WPR - 1))];
#pragma unroll
    for (int o = kNormMaxWarps / 2; o > 0; o >>= 1)
        if (o < WPR)
            s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
    return s;
}

__device__ __forceinline__ const char *row_of(const void *base, int64_t row, int d, int type)
{
    return static_cast<const char *>(base) + row * d * (type == kElemBf16 ? 2 : 4);
}

template <int NSEG, bool VEC>
__global__ void __launch_bounds__(kNormMaxWarps * 32) block_norm_kernel(const NormParams P)
{
    __shared__ float red[2][kNormMaxWarps];
    follow_primary();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rl = warp / P.WPR, first = rl * P.WPR, wr = warp - first;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * P.RPC + rl;
    const bool ok = row < P.M; // warps of a missing row still meet the barriers
    const int d = ok ? P.d : 0;
    const int64_t rr = ok ? row : 0;
    float v[NSEG][8], r[NSEG][8];
#pragma unroll
    for (int s = 0; s < NSEG; ++s) {
        const int base = (s * P.WPR + wr) * kSeg;
        seg_load<VEC>(v[s], row_of(P.x, rr, P.d, P.x_type), P.x_type, base, lane, d);
        seg_load<VEC>(r[s], row_of(P.residual, rr, P.d, P.r_type), P.r_type, base, lane, d);
    }
    // g: the gate, times the post norm's weight where there is one; on its way
    // while the first sum is formed
    float g[NSEG][8];
    const bool post = P.post != nullptr, gated = P.gate != nullptr;
    if (post || gated) {
        const char *grow = gated ? row_of(P.gate, static_cast<uint32_t>(rr) / P.gate_div, P.d, P.x_type) : nullptr;
#pragma unroll
        for (int s = 0; s < NSEG; ++s) {
            const int base = (s * P.WPR + wr) * kSeg;
            if (post) {
                seg_load<VEC>(g[s], P.post, P.w_type, base, lane, d);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    g[s][i] += P.offset;
            }
            if (gated) {
                float w[8];
                seg_load<VEC>(w, grow, P.x_type, base, lane, d);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    g[s][i] = post ? g[s][i] * w[i] : w[i];
            }
        }
    }
    if (post) {
        float q = 0.0f;
#pragma unroll
        for (int s = 0; s < NSEG; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float t = v[s][i] * P.sq_scale;
                q = __fmaf_rn(t, t, q);
            }
        const float f = rsqrtf(__fmaf_rn(row_sum(q, red[0], warp, first, P.WPR), P.sq_inv_d, P.eps));
#pragma unroll
        for (int s = 0; s < NSEG; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[s][i] *= f;
    }
    float q = 0.0f;
#pragma unroll
    for (int s = 0; s < NSEG; ++s) {
        if (post || gated) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[s][i] *= g[s][i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[s][i] = __fmaf_rn(P.bs, v[s][i], __fmul_rn(P.rs, r[s][i]));
            const float t = r[s][i] * P.sq_scale;
            q = __fmaf_rn(t, t, q);
        }
        seg_store<VEC>(r[s], const_cast<char *>(row_of(P.r_out, rr, P.d, P.r_type)), P.r_type,
                       (s * P.WPR + wr) * kSeg, lane, d);
    }
#pragma unroll
    for (int s = 0; s < NSEG; ++s) // the norm's weight, before the second sum
        seg_load<VEC>(g[s], P.pre, P.w_type, (s * P.WPR + wr) * kSeg, lane, d);
    const float f = rsqrtf(__fmaf_rn(row_sum(q, red[1], warp, first, P.WPR), P.sq_inv_d, P.eps));
#pragma unroll
    for (int s = 0; s < NSEG; ++s) {
        const int base = (s * P.WPR + wr) * kSeg;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r[s][i] = r[s][i] * f * (g[s][i] + P.offset);
        if (P.h_type == kElemE4m3)
            seg_quantize<VEC>(r[s], static_cast<uint8_t *>(P.h) + rr * P.d,
                              P.scales + rr * ((P.d + 127) / 128), base, lane, d);
        else
            seg_store<VEC>(r[s], const_cast<char *>(row_of(P.h, rr, P.d, P.h_type)), P.h_type, base, lane, d);
    }
}

// Many rows: CTAs that stay, each with a run of consecutive rows.  A lane has
// the same 16 columns in every row, so the norm's weight is read and converted
// once and the branch's factors (gate, post norm's weight) once per gate row;
// its pieces of the next rows' x and residual are on their way into its own
// slots of shared memory (asynchronous copies that no other thread waits for)
// while this row's sums are formed.  A warp has 512 columns, lane l the four
// from 4 l on of each 128: every access covers whole sectors (a lane's 16
// consecutive columns would write fp32 rows in half sectors, twice as many
// transactions), and a block's largest magnitude is one warp-wide maximum of
// its bits, above which NaNs lie.  Pairs of values go through the packed fp32
// instructions.  2304 rows of 4096 (bf16 x, fp32 residual, gate, e4m3 out,
// 106 MB): 25.0 us = 4.25 TB/s, bound by the ~440 instructions a warp issues per
// row, each behind the last (33 us with one row per CTA and 8 values a lane,
// half of it half-sector stores; a third CTA per SM at 80 registers was slower,
// 28 us).  Rows of whole 16-byte units, up to 512 columns a warp (FULL:
// all of the CTA's warps have 512).  Warps and slots are rounded up to a power
// of two, so a width between two costs as much as the wider one (5120: 41 us,
// 8192: 44 us).
constexpr int kNormRing = 4; // rows in flight, this one included
constexpr int kNormCols = 512;
constexpr int kNormRowsMaxD = kNormMaxWarps * kNormCols;

template <bool FP32, bool FULL>
__device__ __forceinline__ void lane_fetch(uint8_t *slot, int pitch, const char *src, int left)
{
    constexpr int size = FP32 ? 4 : 2;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (FULL || i * 128 < left)
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(slot + i * pitch)),
                         "l"(src + i * 128 * size), "n"(4 * size)
                         : "memory");
}

template <bool FP32, bool FULL>
__device__ __forceinline__ void lane_take(unsigned long long (&v)[8], const uint8_t *slot, int pitch, int left)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = v[2 * i + 1] = 0;
        if (FULL || i * 128 < left) {
            if constexpr (FP32) {
                const uint4 a = lds_v4(slot + i * pitch);
                v[2 * i] = pack2(__uint_as_float(a.x), __uint_as_float(a.y));
                v[2 * i + 1] = pack2(__uint_as_float(a.z), __uint_as_float(a.w));
            } else {
                uint32_t x, y;
                asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x), "=r"(y) : "r"(smem_addr(slot + i * pitch)));
                v[2 * i] = pack2(bf16_lo(x), bf16_hi(x));
                v[2 * i + 1] = pack2(bf16_lo(y), bf16_hi(y));
            }
        }
    }
}

// A lane's values of a weight or gate row (`row` at the lane's first column),
// plus `offset`; 1 past the row's end.
__device__ __forceinline__ void lane_weights(unsigned long long (&w)[8], const char *row, int type, int left,
                                             float offset)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float t[4] = {1.0f, 1.0f, 1.0f, 1.0f};
        if (i * 128 < left) {
            if (type == kElemBf16) {
                const uint2 q = *reinterpret_cast<const uint2 *>(row + i * 256);
                t[0] = bf16_lo(q.x), t[1] = bf16_hi(q.x), t[2] = bf16_lo(q.y), t[3] = bf16_hi(q.y);
            } else {
                const float4 q = *reinterpret_cast<const float4 *>(row + i * 512);
                t[0] = q.x, t[1] = q.y, t[2] = q.z, t[3] = q.w;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                t[k] += offset;
        }
        w[2 * i] = pack2(t[0], t[1]);
        w[2 * i + 1] = pack2(t[2], t[3]);
    }
}

// A lane's values to a row of bf16 or fp32 (`row` at the lane's first column).
template <bool FULL>
__device__ __forceinline__ void lane_store(const unsigned long long (&v)[8], char *row, bool fp32, int left)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (FULL || i * 128 < left) {
            float a, b, c, d;
            unpack2(v[2 * i], a, b);
            unpack2(v[2 * i + 1], c, d);
            if (fp32)
                *reinterpret_cast<float4 *>(row + i * 512) = make_float4(a, b, c, d);
            else
                *reinterpret_cast<uint2 *>(row + i * 256) = make_uint2(bf16x2_rn(a, b), bf16x2_rn(c, d));
        }
}

__device__ __forceinline__ float sum_squares(const unsigned long long (&a)[8], unsigned long long k)
{
    unsigned long long v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = mul2(a[i], k);
    unsigned long long q = mul2(v[0], v[0]), p = mul2(v[1], v[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        q = fma2(v[i], v[i], q);
        p = fma2(v[i + 1], v[i + 1], p);
    }
    float lo, hi;
    unpack2(add2(q, p), lo, hi);
    return __fadd_rn(lo, hi);
}

template <bool XF32, bool RF32, bool FULL>
__global__ void __launch_bounds__(kNormMaxWarps * 32, 1) block_norm_rows_kernel(const NormParams P)
{
    constexpr int kXSize = XF32 ? 4 : 2, kRSize = RF32 ? 4 : 2;
    constexpr int kXType = XF32 ? kElemFp32 : kElemBf16;
    extern __shared__ __align__(16) uint8_t norm_smem[]; // [ring][x's 4 pieces, then the residual's][thread]
    __shared__ float red[2][2][kNormMaxWarps];
    follow_primary();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = P.d;
    const int e = warp * kNormCols + lane * 4, left = d - e; // first column; piece i is in the row where 128 i < left
    const int threads = static_cast<int>(blockDim.x), slot_bytes = threads * 16 * (kXSize + kRSize);
    uint8_t *own_x = norm_smem + threadIdx.x * 4 * kXSize;
    uint8_t *own_r = norm_smem + threads * 16 * kXSize + threadIdx.x * 4 * kRSize;
    const bool post = P.post != nullptr, gated = P.gate != nullptr;
    const int64_t begin = P.M * blockIdx.x / gridDim.x, end = P.M * (blockIdx.x + 1) / gridDim.x;
    const int wsize = P.w_type == kElemBf16 ? 2 : 4, hsize = P.h_type == kElemE4m3 ? 1 : P.h_type == kElemBf16 ? 2 : 4;
    const char *wpost = static_cast<const char *>(P.post) + e * wsize;
    const unsigned long long rs = pack2(P.rs, P.rs), bs = pack2(P.bs, P.bs), sq = pack2(P.sq_scale, P.sq_scale);
    unsigned long long wpre[8], branch[8];
    lane_weights(wpre, static_cast<const char *>(P.pre) + e * wsize, P.w_type, left, P.offset);
    lane_weights(branch, wpost, P.w_type, post ? left : 0, P.offset);
    // where this lane's columns of the next row to fetch, and of this row, are
    const char *x = static_cast<const char *>(P.x) + (begin * d + e) * kXSize;
    const char *res = static_cast<const char *>(P.residual) + (begin * d + e) * kRSize;
    char *r_out = static_cast<char *>(P.r_out) + (begin * d + e) * kRSize;
    char *h = static_cast<char *>(P.h) + (begin * d + e) * hsize;
    float *scales = P.scales + begin * ((d + 127) / 128) + warp * 4 + (lane & 3);
    int to_fetch = static_cast<int>(end - begin);
    auto fetch = [&](int slot) {
        if (to_fetch-- > 0) {
            lane_fetch<XF32, FULL>(own_x + slot * slot_bytes, threads * 4 * kXSize, x, left);
            lane_fetch<RF32, FULL>(own_r + slot * slot_bytes, threads * 4 * kRSize, res, left);
            x += static_cast<int64_t>(d) * kXSize;
            res += static_cast<int64_t>(d) * kRSize;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kNormRing - 1; ++i)
        fetch(i);
    uint32_t gate_left = 0; // rows that the factors in `branch` still serve
    int slot = 0, odd = 0;
#pragma unroll 1
    for (int64_t row = begin; row < end; ++row, odd ^= 1) {
        fetch(slot == 0 ? kNormRing - 1 : slot - 1); // the slot this lane has read last
        if (gated && gate_left == 0) {
            const uint32_t g = static_cast<uint32_t>(row) / P.gate_div;
            gate_left = (g + 1) * P.gate_div - static_cast<uint32_t>(row);
            lane_weights(branch, static_cast<const char *>(P.gate) + (static_cast<int64_t>(g) * d + e) * kXSize, kXType,
                         left, 0.0f);
            if (post) {
                unsigned long long w[8];
                lane_weights(w, wpost, P.w_type, left, P.offset);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    branch[i] = mul2(branch[i], w[i]);
            }
        }
        --gate_left;
        cp_async_wait<kNormRing - 1>();
        unsigned long long v[8], r[8];
        lane_take<XF32, FULL>(v, own_x + slot * slot_bytes, threads * 4 * kXSize, left);
        lane_take<RF32, FULL>(r, own_r + slot * slot_bytes, threads * 4 * kRSize, left);
        slot = slot == kNormRing - 1 ? 0 : slot + 1;
        if (post) { // before gate and weight, whose products with x may leave the fp32 range
            const float f =
                rsqrtf(__fmaf_rn(row_sum(sum_squares(v, sq), red[0][odd], warp, 0, P.WPR), P.sq_inv_d, P.eps));
            const unsigned long long ff = pack2(f, f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = mul2(v[i], ff);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r[i] = fma2(mul2(v[i], branch[i]), bs, mul2(r[i], rs));
        lane_store<FULL>(r, r_out, RF32, left);
        r_out += static_cast<int64_t>(d) * kRSize;
        const float fh =
            rsqrtf(__fmaf_rn(row_sum(sum_squares(r, sq), red[1][odd], warp, 0, P.WPR), P.sq_inv_d, P.eps));
        const unsigned long long hh = pack2(fh, fh);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r[i] = mul2(mul2(r[i], hh), wpre[i]);
        if (P.h_type == kElemE4m3) {
            uint32_t amax = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a, b, c, t;
                unpack2(r[2 * i], a, b);
                unpack2(r[2 * i + 1], c, t);
                const uint32_t m = max(max(__float_as_uint(a) & 0x7FFFFFFFu, __float_as_uint(b) & 0x7FFFFFFFu),
                                       max(__float_as_uint(c) & 0x7FFFFFFFu, __float_as_uint(t) & 0x7FFFFFFFu));
                const uint32_t block = __reduce_max_sync(0xFFFFFFFFu, m);
                amax = (lane & 3) == i ? block : amax;
            }
            // lane l has the scale of block l mod 4 of the warp's columns
            const float scale = block_scale(__uint_as_float(amax)), inv = __frcp_rn(scale);
            if (lane < 4 && (FULL || warp * kNormCols + lane * 128 < d))
                *scales = scale;
            scales += (d + 127) / 128;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float s = __shfl_sync(0xFFFFFFFFu, inv, i);
                float a, b, c, t;
                unpack2(mul2(r[2 * i], pack2(s, s)), a, b);
                unpack2(mul2(r[2 * i + 1], pack2(s, s)), c, t);
                if (FULL || i * 128 < left)
                    *reinterpret_cast<uint32_t *>(h + i * 128) = e4m3x2_rn(a, b) | e4m3x2_rn(c, t) << 16;
            }
        } else {
            lane_store<FULL>(r, h, P.h_type == kElemFp32, left);
        }
        h += static_cast<int64_t>(d) * hsize;
    }
}

// ------------------------------------------------------------- quantisation

struct QuantParams {
    const void *x;
    int32_t x_type;
    int64_t M;
    int32_t d;
    int64_t segs; // segments of a row (1 x 128 blocks) or blocks along a row (128 x 128)
    uint8_t *v;
    float *scales;
};

constexpr int kQuantWarps = 8;

// A scale per row and 128 values: a warp per segment of 256 values (384 rows of
// 4096: 3.7 us, one launch's latency).
template <bool VEC> __global__ void __launch_bounds__(kQuantWarps * 32) quantize_rows_kernel(const QuantParams P)
{
    follow_primary();
    const int lane = threadIdx.x & 31;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kQuantWarps + (threadIdx.x >> 5);
    const int64_t row = i / P.segs;
    if (row >= P.M) // warp-uniform
        return;
    const int base = static_cast<int>(i - row * P.segs) * kSeg;
    float v[8];
    seg_load<VEC>(v, row_of(P.x, row, P.d, P.x_type), P.x_type, base, lane, P.d);
    const int64_t blocks = (static_cast<int64_t>(P.d) + 127) / 128; // d may be the largest 32-bit number
    seg_quantize<VEC>(v, P.v + row * P.d, P.scales + row * blocks, base, lane, P.d);
}

// A scale per 128 x 128 block: a CTA per block, held in registers (64 values
// a thread; bf16 ones stay packed until they are scaled, so that more CTAs are
// resident: 88 -> 58 us for 32003 x 4112, 6.8 TB/s, bound by its bytes; fp32
// 97 us, 6.7 TB/s).  A half-warp per row, 8 consecutive values a lane; rows that
// are not whole 16-byte units take quantize_tiles_odd_kernel.
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The block's scale and its reciprocal, from every thread's largest magnitude.
__device__ __forceinline__ float tile_scale(float amax, float *red, float *scale_out)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        amax = max_nan(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantWarps; ++w)
        amax = max_nan(amax, red[w]);
    const float s = block_scale(amax);
    if (threadIdx.x == 0)
        *scale_out = s;
    return __frcp_rn(s);
}

template <bool FP32> __global__ void __launch_bounds__(kQuantWarps * 32) quantize_tiles_kernel(const QuantParams P)
{
    __shared__ float red[kQuantWarps];
    follow_primary();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t segs = static_cast<uint32_t>(P.segs), rb = blockIdx.x / segs, cb = blockIdx.x - rb * segs;
    const int64_t row0 = static_cast<int64_t>(rb) * 128 + warp * 2 + (lane >> 4); // rows row0, row0 + 16, ...
    const int e = static_cast<int>(cb) * 128 + (lane & 15) * 8;
    const int rows = P.M - row0 <= 0 || e >= P.d ? 0 : P.M - row0 < 128 ? static_cast<int>(P.M - row0 + 15) / 16 : 8;
    uint4 v[8][FP32 ? 2 : 1];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
        const int64_t at = (row0 + s * 16) * P.d + e;
#pragma unroll
        for (int i = 0; i < (FP32 ? 2 : 1); ++i)
            v[s][i] = s < rows ? *reinterpret_cast<const uint4 *>(static_cast<const char *>(P.x) +
                                                                  at * (FP32 ? 4 : 2) + i * 16)
                               : make_uint4(0, 0, 0, 0);
    }
    float amax = 0.0f;
    if constexpr (FP32) {
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                amax = max_nan(max_nan(max_nan(amax, fabsf(__uint_as_float(v[s][i].x))),
                                       fabsf(__uint_as_float(v[s][i].y))),
                               max_nan(fabsf(__uint_as_float(v[s][i].z)), fabsf(__uint_as_float(v[s][i].w))));
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            m = max_nan_bf16x2(m, v[s][0].x & 0x7FFF7FFFu);
            m = max_nan_bf16x2(m, v[s][0].y & 0x7FFF7FFFu);
            m = max_nan_bf16x2(m, v[s][0].z & 0x7FFF7FFFu);
            m = max_nan_bf16x2(m, v[s][0].w & 0x7FFF7FFFu);
        }
        amax = max_nan(bf16_lo(m), bf16_hi(m));
    }
    const float inv = tile_scale(amax, red, P.scales + blockIdx.x);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
        uint2 o;
        if constexpr (FP32) {
            const uint4 a = v[s][0], b = v[s][1];
            o.x = e4m3x4_scaled(__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w), inv);
            o.y = e4m3x4_scaled(__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w), inv);
        } else {
            const uint4 a = v[s][0];
            o.x = e4m3x4_scaled(bf16_lo(a.x), bf16_hi(a.x), bf16_lo(a.y), bf16_hi(a.y), inv);
            o.y = e4m3x4_scaled(bf16_lo(a.z), bf16_hi(a.z), bf16_lo(a.w), bf16_hi(a.w), inv);
        }
        if (s < rows)
            *reinterpret_cast<uint2 *>(P.v + (row0 + s * 16) * P.d + e) = o;
    }
}

// Rows that are not whole 16-byte units: 4 single values of a row per lane, 64
// in all (32003 x 4111: 234 us from bf16, bound by its 2-byte loads, 99 from
// fp32).
__global__ void __launch_bounds__(kQuantWarps * 32) quantize_tiles_odd_kernel(const QuantParams P)
{
    __shared__ float red[kQuantWarps];
    follow_primary();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t segs = static_cast<uint32_t>(P.segs), rb = blockIdx.x / segs, cb = blockIdx.x - rb * segs;
    const int64_t row0 = static_cast<int64_t>(rb) * 128 + warp; // rows row0, row0 + 8, ...
    const int e0 = static_cast<int>(cb) * 128 + lane;           // columns e0, e0 + 32, ...
    float v[16][4];
    float amax = 0.0f;
#pragma unroll
    for (int s = 0; s < 16; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = row0 + s * 8;
            const int e = e0 + i * 32;
            v[s][i] = row < P.M && e < P.d ? elem_at(P.x, P.x_type, row * P.d + e) : 0.0f;
            amax = max_nan(amax, fabsf(v[s][i]));
        }
    const float inv = tile_scale(amax, red, P.scales + blockIdx.x);
#pragma unroll
    for (int s = 0; s < 16; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = row0 + s * 8;
            const int e = e0 + i * 32;
            if (row < P.M && e < P.d)
                P.v[row * P.d + e] = static_cast<uint8_t>(e4m3x2_rn(__fmul_rn(v[s][i], inv), 0.0f));
        }
}

} // namespace sv
