// sv_fp4.cuh -- microscaled 4-bit floating point: quantisation and reading
// back.
//
//   block 16:  g = 2^k, the least with (largest finite |x| of the row) / g <= 6 * 448
//              s = e4m3(max|x| / (6 g)), at least 2^-9 for a block that is not zero
//              v = e2m1(x / (s g))                 x ~ v s g
//   block 32:  s = 2^(floor(log2 max|x|) - 2) (e8m0), v = e2m1(x / s), x ~ v s
//
// every rounding to nearest even, |v| <= 6.  g is a power of two so that s g
// and the decision between two values are exact: nothing is lost, e4m3's own
// exponent covers the blocks of a row.  A block with a NaN or an infinity
// gets a NaN scale and zeros, and does not count in its row's maximum.
//
// Two values a byte (the even column in the low half).  The scales lie as the
// tensor cores take them from shared memory: tiles of 128 rows x 4 blocks,
// 512 bytes, byte 16 (row mod 32) + 4 (row / 32 mod 4) + block mod 4; zeros
// behind the ends of the matrix.
//
// Work is cut in octets (8 values of a row, one lane): 16-byte loads of bf16,
// 4-byte stores, both whole lines a warp; a block is 2 or 4 neighbouring lanes.
// A row belongs to WPR warps, whose lanes keep its octets in registers between
// the row's maximum and the values (of longer rows the rest is read again), and
// have the next row's on their way meanwhile.
//
// Measured (replayed; GB300) at 128256 x 4096: quantising bf16 in blocks of 16 315 us =
// 4.3 TB/s, of 32 226 us = 5.9 TB/s, fp32 375 and 368 us = 6.4 TB/s; reading back to bf16
// 207 us = 6.5 TB/s and 241 us, to fp32 502 and 476 us = 4.8 and 5.0 TB/s.  Blocks of 16 are
// bound by instructions (136 an octet and lane, 70 % of the issue slots, the ALU pipe
// first); with divisions by the compiler and addresses by octet it was 500 us, 375 with
// corrected reciprocals, 319 with addresses by row.
#pragma once

#include "sv_device.cuh"

namespace sv {

constexpr int kF4Threads = 256;
constexpr int kF4Regs = 4; // octets a lane keeps between the two passes
// CTAs of an SM that stay and walk the rows, the next row's octets on their way
template <typename XT> constexpr int kF4Ctas = sizeof(XT) == 2 ? 3 : 2;

struct Fp4Params {
    const void *x;        // [M, d]
    int64_t M, Mpad;      // rows, rows of the scale tiles (a multiple of 128)
    int32_t d;
    int32_t octets;       // of a row, the padded blocks' included (4 blocks a tile)
    int32_t KT;           // scale tiles along d
    int32_t WPR;          // warps of a row: 1, 2, 4 or 8
    int32_t pairs;        // x is aligned to two of its elements (and so are all rows)
    uint8_t *v;           // [M, d / 2]
    uint8_t *s;           // [Mpad / 128, KT, 512]
    float *g;             // [M] (block 16)
};

struct Fp4BackParams {
    const uint8_t *v, *s;
    const float *g;       // [M] or nullptr
    int64_t M;
    int32_t d, octets, KT, WPR;
    int32_t pairs;        // out is aligned to two of its elements
    void *out;            // [M, d] bf16 or fp32
};

// Where the scale of block b of row r is.
__device__ __forceinline__ int64_t f4_scale_at(int64_t r, int32_t b, int32_t KT)
{
    return ((r >> 7) * KT + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

// Eight e2m1 values of a .. as 4 bytes, a[0] in the lowest half byte.
__device__ __forceinline__ uint32_t f4_pack(const float (&a)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(a[0]), "f"(a[1]), "f"(a[2]), "f"(a[3]), "f"(a[4]), "f"(a[5]), "f"(a[6]), "f"(a[7]));
    return r;
}

// The eight values of 4 bytes, exactly, as four pairs of fp16.
__device__ __forceinline__ void f4_unpack(uint32_t p, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(p));
}

__device__ __forceinline__ float2 f4_half2(uint32_t h)
{
    float2 f;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

// The value of an e4m3 byte.
__device__ __forceinline__ float f4_e4m3(uint32_t byte)
{
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(byte));
    return f4_half2(h).x;
}

// 2^(byte - 127); NaN for 255.
__device__ __forceinline__ float f4_e8m0(uint32_t byte)
{
    return __uint_as_float(byte == 0 ? 0x00400000u : (byte == 255 ? 0x7FFFFFFFu : byte << 23));
}

// A non-negative fp32 value as an e4m3 byte, nearest even, at most 448.
__device__ __forceinline__ uint32_t f4_to_e4m3(float s)
{
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.0f), "f"(s));
    return h & 0xFFu;
}

// One lane's octet of a row: raw bits as loaded.
template <typename XT> struct F4Octet;
template <> struct F4Octet<uint16_t> {
    uint4 w;
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const uint16_t *p) { w = ld_stream_v4(p); }
    // the first n (even), the others 0
    __device__ __forceinline__ void load_some(const uint16_t *p, int n, bool pairs)
    {
        uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (2 * i < n)
                u[i] = pairs ? __ldg(reinterpret_cast<const uint32_t *>(p) + i)
                             : __ldg(p + 2 * i) | static_cast<uint32_t>(__ldg(p + 2 * i + 1)) << 16;
        w = make_uint4(u[0], u[1], u[2], u[3]);
    }
    // the largest magnitude, as fp32 bits
    __device__ __forceinline__ uint32_t amax() const
    {
        const uint32_t k = 0x7FFF7FFFu;
        const uint32_t m = __vmaxu2(__vmaxu2(w.x & k, w.y & k), __vmaxu2(w.z & k, w.w & k));
        return max(m << 16, m & 0xFFFF0000u);
    }
    __device__ __forceinline__ void values(float (&f)[8]) const
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(u[i]);
            f[2 * i + 1] = bf16_hi(u[i]);
        }
    }
};
template <> struct F4Octet<float> {
    uint4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const float *p)
    {
        a = ld_stream_v4(p);
        b = ld_stream_v4(p + 4);
    }
    __device__ __forceinline__ void load_some(const float *p, int n, bool pairs)
    {
        float2 f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = make_float2(0.0f, 0.0f);
            if (2 * i < n)
                f[i] = pairs ? __ldg(reinterpret_cast<const float2 *>(p) + i) : make_float2(__ldg(p + 2 * i), __ldg(p + 2 * i + 1));
        }
        a = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
        b = make_uint4(__float_as_uint(f[2].x), __float_as_uint(f[2].y), __float_as_uint(f[3].x), __float_as_uint(f[3].y));
    }
    __device__ __forceinline__ uint32_t amax() const
    {
        const uint32_t k = 0x7FFFFFFFu;
        return max(max(max(a.x & k, a.y & k), max(a.z & k, a.w & k)), max(max(b.x & k, b.y & k), max(b.z & k, b.w & k)));
    }
    __device__ __forceinline__ void values(float (&f)[8]) const
    {
        const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = __uint_as_float(u[i]);
    }
};

// The first n (even) values of an octet's 4 bytes, in pieces as large as the address
// allows (the same for a whole row).
__device__ __forceinline__ void f4_store_some(uint8_t *v, uint32_t packed, int n)
{
    const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(v));
    if ((at & 3u) == 0 && n >= 8) {
        *reinterpret_cast<uint32_t *>(v) = packed;
    } else if ((at & 1u) == 0 && n >= 8) {
        reinterpret_cast<uint16_t *>(v)[0] = static_cast<uint16_t>(packed);
        reinterpret_cast<uint16_t *>(v)[1] = static_cast<uint16_t>(packed >> 16);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (2 * k < n)
                v[k] = static_cast<uint8_t>(packed >> (8 * k));
    }
}
__device__ __forceinline__ uint32_t f4_load_some(const uint8_t *v, int n)
{
    const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(v));
    uint32_t p = 0;
    if ((at & 3u) == 0 && n >= 8) {
        p = __ldg(reinterpret_cast<const uint32_t *>(v));
    } else if ((at & 1u) == 0 && n >= 8) {
        p = __ldg(reinterpret_cast<const uint16_t *>(v)) | static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(v) + 1)) << 16;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (2 * k < n)
                p |= static_cast<uint32_t>(__ldg(v + k)) << (8 * k);
    }
    return p;
}

// The row's power of two from its largest magnitude's bits: biased exponent
// of the least 2^k with amax <= 2688 * 2^k (2688 = 1.3125 * 2^11); 2^0 for a
// row of zeros, at least 2^-126.
__device__ __forceinline__ uint32_t f4_outer(uint32_t amax)
{
    if (amax == 0)
        return 127u;
    const int e = static_cast<int>(amax >> 23) - 11 + ((amax & 0x7FFFFFu) > 0x280000u ? 1 : 0);
    return static_cast<uint32_t>(e > 1 ? e : 1);
}

template <int BLOCK, typename XT, bool VEC>
__global__ void __launch_bounds__(kF4Threads, kF4Ctas<XT>) quantize_fp4_kernel(const Fp4Params P)
{
    constexpr int L = BLOCK / 8; // lanes of a block
    __shared__ uint32_t wmax[2][kF4Threads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = kF4Threads / 32 / P.WPR; // rows of a CTA at a time (128 is a multiple)
    const int first = (warp & (P.WPR - 1)) * 32 + lane, stride = P.WPR * 32;
    pdl_wait_primary();
    pdl_launch_dependents();
    // every warp's lanes take the same number of steps (the shuffles)
    const int steps = static_cast<int>((P.octets + stride - 1) / stride);
    const int64_t step_rows = static_cast<int64_t>(gridDim.x) * per;
    int64_t row = static_cast<int64_t>(blockIdx.x) * per + warp / P.WPR;
    const XT *x = static_cast<const XT *>(P.x) + row * P.d + first * 8; // this lane's first octet of the row
    const int64_t x_step = step_rows * P.d;
    auto fetch = [&](F4Octet<XT> &o, const XT *from, bool real, int t) {
        const int32_t left = real ? P.d - (first + t * stride) * 8 : 0;
        if (left <= 0)
            o.zero();
        else if (VEC)
            o.load(from + t * stride * 8);
        else
            o.load_some(from + t * stride * 8, left, P.pairs);
    };
    auto block_max = [&](const F4Octet<XT> &o) {
        uint32_t m = o.amax();
#pragma unroll
        for (int s = 1; s < L; s <<= 1)
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
        return m;
    };
    F4Octet<XT> keep[kF4Regs];
#pragma unroll
    for (int t = 0; t < kF4Regs; ++t)
        if (t < steps)
            fetch(keep[t], x, row < P.M, t);
    uint32_t parity = 0;
    for (; row < P.Mpad; row += step_rows, x += x_step, parity ^= 1u) { // (all warps of a CTA together)
        const bool real = row < P.M;
        uint32_t amax[kF4Regs];
        uint32_t top = 0;
#pragma unroll
        for (int t = 0; t < kF4Regs; ++t)
            if (t < steps) {
                amax[t] = block_max(keep[t]);
                top = max(top, amax[t] < 0x7F800000u ? amax[t] : 0u);
            }
        F4Octet<XT> next[kF4Regs];
#pragma unroll
        for (int t = 0; t < kF4Regs; ++t)
            if (t < steps)
                fetch(next[t], x + x_step, row + step_rows < P.M, t);
        uint32_t ge = 127u; // the row's biased exponent
        if (BLOCK == 16) {
            for (int t = kF4Regs; t < steps; ++t) {
                F4Octet<XT> o;
                fetch(o, x, real, t);
                const uint32_t m = block_max(o);
                top = max(top, m < 0x7F800000u ? m : 0u);
            }
            top = __reduce_max_sync(0xFFFFFFFFu, top);
            if (P.WPR > 1) {
                if (lane == 0)
                    wmax[parity][warp] = top;
                __syncthreads();
                for (int w = 0; w < P.WPR; ++w)
                    top = max(top, wmax[parity][(warp & ~(P.WPR - 1)) + w]);
            }
            ge = f4_outer(top);
            if (real && first == 0)
                P.g[row] = __uint_as_float(ge << 23);
        }
        // this lane's first scale and values; a step further lies a whole number of tiles
        uint8_t *const s0 = P.s + f4_scale_at(row, first / L, P.KT);
        uint8_t *const v0 = P.v + row * (P.d >> 1) + first * 4;
        const float ginv = __uint_as_float((254u - ge) << 23);
        auto finish = [&](const F4Octet<XT> &o, uint32_t m, int t) {
            float f[8];
            o.values(f);
            uint32_t byte;
            if (BLOCK == 16) {
                // x / g is exact.  Quotients by 6 and by s from a rounded reciprocal r and one
                // correction, which rounds correctly, and r itself from the unit's approximation
                // and one of its own (Markstein 1990): q = y r, q - (q s - y) r.  (That way round, and
                // y negative to begin with, a zero keeps its sign.)
                const float y = __fmul_rn(__uint_as_float(m), ginv), q6 = __fmul_rn(y, 1.0f / 6.0f);
                byte = f4_to_e4m3(__fmaf_rn(__fmaf_rn(q6, -6.0f, y), 1.0f / 6.0f, q6));
                byte = m ? max(byte, 1u) : 0u;
                const float s = m ? f4_e4m3(byte) : 1.0f;
                float r;
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
                r = __fmaf_rn(__fmaf_rn(-s, r, 1.0f), r, r);
                const unsigned long long gg = pack2(-ginv, -ginv), rr = pack2(-r, -r), ss = pack2(s, s);
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    const unsigned long long y2 = mul2(pack2(f[k], f[k + 1]), gg), q = mul2(y2, rr);
                    unpack2(fma2(fma2(q, ss, y2), rr, q), f[k], f[k + 1]);
                }
            } else {
                const int e = static_cast<int>(m >> 23) - 2;
                byte = static_cast<uint32_t>(e > 0 ? e : 0);
                const float sinv = __uint_as_float((254u - byte) << 23);
                const unsigned long long ss = pack2(sinv, sinv);
#pragma unroll
                for (int k = 0; k < 8; k += 2)
                    unpack2(mul2(pack2(f[k], f[k + 1]), ss), f[k], f[k + 1]);
            }
            uint32_t packed = f4_pack(f);
            if (m >= 0x7F800000u) { // a NaN or an infinity
                packed = 0;
                byte = BLOCK == 16 ? 0x7Fu : 0xFFu;
            }
            const int32_t i = first + t * stride;
            if (lane % L == 0 && i < P.octets)
                s0[static_cast<int64_t>(t) * ((stride / (4 * L)) * 512)] = static_cast<uint8_t>(byte);
            const int32_t left = real ? P.d - i * 8 : 0;
            uint8_t *v = v0 + t * stride * 4;
            if (VEC) {
                if (left > 0)
                    *reinterpret_cast<uint32_t *>(v) = packed;
            } else {
                f4_store_some(v, packed, left);
            }
        };
#pragma unroll
        for (int t = 0; t < kF4Regs; ++t)
            if (t < steps)
                finish(keep[t], amax[t], t);
        for (int t = kF4Regs; t < steps; ++t) {
            F4Octet<XT> o;
            fetch(o, x, real, t);
            finish(o, block_max(o), t);
        }
#pragma unroll
        for (int t = 0; t < kF4Regs; ++t)
            keep[t] = next[t];
    }
}

// v s g in fp32 (v s is exact there, its product with g rounded once), rounded
// once more to bf16.
template <int BLOCK, bool F32, bool VEC>
__global__ void __launch_bounds__(kF4Threads) dequantize_fp4_kernel(const Fp4BackParams P)
{
    constexpr int L = BLOCK / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = kF4Threads / 32 / P.WPR;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * per + warp / P.WPR;
    const int first = (warp & (P.WPR - 1)) * 32 + lane, stride = P.WPR * 32;
    pdl_wait_primary();
    pdl_launch_dependents();
    if (row >= P.M)
        return;
    const float g = P.g ? __ldg(P.g + row) : 1.0f;
    const uint8_t *v = P.v + row * (P.d >> 1);
#pragma unroll 4
    for (int32_t i = first; i < P.octets; i += stride) {
        const int32_t left = P.d - i * 8;
        uint32_t p = 0;
        if (VEC) {
            p = __ldg(reinterpret_cast<const uint32_t *>(v + i * 4));
        } else {
            p = f4_load_some(v + i * 4, left);
        }
        const uint32_t byte = __ldg(P.s + f4_scale_at(row, i / L, P.KT));
        const float s = BLOCK == 16 ? f4_e4m3(byte) : f4_e8m0(byte);
        uint32_t h[4];
        f4_unpack(p, h);
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 t = f4_half2(h[k]);
            f[2 * k] = __fmul_rn(__fmul_rn(t.x, s), g);
            f[2 * k + 1] = __fmul_rn(__fmul_rn(t.y, s), g);
        }
        if (F32) {
            float *o = static_cast<float *>(P.out) + row * P.d + i * 8;
            if (VEC) {
                reinterpret_cast<float4 *>(o)[0] = make_float4(f[0], f[1], f[2], f[3]);
                reinterpret_cast<float4 *>(o)[1] = make_float4(f[4], f[5], f[6], f[7]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; k += 2)
                    if (k < left) { // (left is even)
                        if (P.pairs) {
                            *reinterpret_cast<float2 *>(o + k) = make_float2(f[k], f[k + 1]);
                        } else {
                            o[k] = f[k];
                            o[k + 1] = f[k + 1];
                        }
                    }
            }
        } else {
            uint16_t *o = static_cast<uint16_t *>(P.out) + row * P.d + i * 8;
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[k]) : "f"(f[2 * k + 1]), "f"(f[2 * k]));
            if (VEC) {
                *reinterpret_cast<uint4 *>(o) = make_uint4(u[0], u[1], u[2], u[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (2 * k < left) {
                        if (P.pairs) {
                            reinterpret_cast<uint32_t *>(o)[k] = u[k];
                        } else {
                            o[2 * k] = static_cast<uint16_t>(u[k]);
                            o[2 * k + 1] = static_cast<uint16_t>(u[k] >> 16);
                        }
                    }
            }
        }
    }
}

} // namespace sv
