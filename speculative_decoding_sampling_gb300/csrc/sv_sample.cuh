// sv_sample.cuh -- one token a row from its logits: temperature, top-k, top-p,
// min-p and the draw by inverse CDF from a given uniform, with the processed
// distribution (the verification's q) where it is wanted.
//
// The ids of a row are ordered as sv_filter.cuh orders them (p descending, equal
// p by ascending id).  Every filter keeps a prefix of that order: top-k the
// first k finite ids, top-p the shortest prefix of those whose mass reaches
// top_p times theirs, min-p the ids with p >= min_p max p.  The token is the
// first id with u Z < C(id) over the kept masses in id order.
//
// Masses are integers, so sums are exact and free of order.  They carry 2^-28 of
// each value: with c = 32 log2(e) / T, k = round(z c) and r = z c - k,
//   e^(z / T) = 2^(k / 32) (1 + x + x^2/2 + x^3/6),  x = r ln(2) / 32,
// of which 2^(k / 32) counts from the whole number next above max c on.  z c - k is
// one multiply-add with c's high part and one with its low: z - max is not formed,
// which fp32 cannot hold where the two differ much in size.  Where max c is 2^21 or
// more the same is done with z - max, which is exact then wherever there is mass (z
// lies within a factor of 2 of the maximum).
// |x| <= 0.0122, the series' rest below 2^-30; 2^(j / 32) comes from a table of 32
// whose entries lie in different banks.  (exp2 in fp32 alone gives 2^-22: among
// 10^5 ids a draw then falls on a neighbour once in some hundred rows.)
//
// A cluster of C CTAs (1, 2, 4 or 8) takes a row, each a slice of its ids, read
// once from memory into shared memory (rows too long for eight stay in L2).  CTAs
// exchange through distributed shared memory; a step ends with a cluster barrier.
//  1. load, maximum;
//  2. top-k, top-p: the ids are counted in 512 bins from the maximum down (24
//     octaves of mass, and 16 of logits at least for top-k); where top-p refers to
//     the whole row its mass is formed in the same pass.  A scan finds top-k's bin;
//     for top-p the counts and the bins' edges bound the running mass to 3.3 % and
//     so the bins that its cut may lie in.  The ids down to the last of these bins
//     are listed (up to 1152 or 4096 a CTA; more are picked out of the slice each
//     time), and nothing below them is looked at again;
//  3. up to 256 listed ids are gathered by every CTA and ranked, which settles the
//     row.  Up to 1024 go, in a large batch, to the cluster's first CTA, which
//     settles the row alone as all would together: the ids of top-k's bin are ranked;
//     then masses are binned (four shared-memory additions an id) and the ids of
//     top-p's bin ranked; the draw finds its run of ids by such bins too.  (Of more
//     than 1024, and in small batches, the ranked ones are gathered by every CTA.)  A
//     bin of more than 256 is counted again digit by digit of the order key (512 bins
//     a digit) down to one value, as is all below the bins when a cut lies there;
//     among ids of one value the j-th in id order is found by an ordered count;
//  4. the kept masses by warp and CTA, the draw inside the warp that holds it;
//  5. q.
//
// Measured (calls replayed from a graph; GB300): 1 row of 32000 fp32, k 50, p 0.95:
// 11 us; 8 rows of 128256 bf16, p 0.9: 30 us; 133 rows of 32003 fp32, min-p: 11 us; 256
// rows of 128256 bf16, k 1000, p 0.9, min-p 0.01, with q: 135 us; 256 rows of 151936
// bf16 at temperature alone, with q: 80 us = 2.9 TB/s.  Without cuts a row's CTAs load,
// wait, form masses, wait and write (16 us: 3 load, 2 barrier, 4 masses, 3 exchange and
// draw, 2 q) and nothing of the next row is on its way: 59 % of the issue slots and 27 %
// of the memory's rate are used, neither is the bound.  With cuts it is the chain of a
// row's steps (about 26 us: 4 load and barrier, 5 counts, 2 scan, 4 list, 9 one CTA's
// settling, 2 q), four CTAs an SM, 33 % of the issue slots.
// What the parts were worth on 256 rows of 128256 with every filter: 614 us as first
// built (masses in bins, digit by digit over a list); 572 -> 369 bins of the value
// instead of digits of the key; 284 counts first, masses only where the cut may lie;
// 184 lists and ranked candidates; 151 one CTA settling; 137 asynchronous copies.
#pragma once

#include <type_traits>

#include "sv_filter.cuh"

namespace sv {

constexpr int kSmMaxWarps = 16; // CTAs of 256 or 512 threads (NT)
constexpr int kSmMaxCtas = 8;

struct SampleParams {
    const void *in;      // [rows, V]
    int64_t rows;
    int32_t V;
    const float *u;      // [rows]
    float c_hi, c_lo;    // 32 log2(e) / T
    float cq;            // log2(e) / T
    float dmin;          // differences below this have no mass: -(fix + 3) T ln 2
    float bins, width;   // bins of step 2 per unit of the logits, and a bin's width
    double min_off;      // T ln(min_p) (min_p > 0)
    int32_t top_k;       // <= 0: off
    float top_p;         // >= 1: off
    int32_t min_p;       // whether min_off counts
    int32_t C;           // CTAs of a cluster
    int32_t slice;       // ids of a CTA, a multiple of 16 bytes of them
    int32_t cap;         // ids a CTA lists (at least kSmOne)
    int32_t staged;      // the slices fit in shared memory
    int32_t fix;         // fractional bits of the masses (at most 45, sums of a row below 2^62)
    int32_t piece;       // bits of a mass that a bin adds up in one 32-bit word
    int32_t vec_q;       // q's vectors lie as the logits' do
    int32_t *tokens;     // [rows]
    float *prob;         // [rows] or nullptr
    int32_t *kept;       // [rows] or nullptr
    float *probs;        // [rows, V] or nullptr
    int32_t *status;     // or nullptr
};

constexpr int kSmFew = 256;    // ids gathered and ranked
constexpr int kSmBins = 512;   // bins of steps 2 and 3
constexpr int kSmOne = 1024;   // ids that one CTA settles

// A cut: ids with a larger key, and of those with this key the ones up to `id`.
struct SampleCutAt {
    uint32_t key;
    int32_t id;
};

struct SampleShared {
    float2 tab[32];                                  // 2^(j / 32) 2^27: as fp32, and as an integer less the shift's bits
    float cmax[kSmMaxCtas];
    unsigned long long cmass[4][kSmMaxCtas];         // exchanged sums, a row of slots for each use
    uint32_t ccnt[4][kSmMaxCtas];
    unsigned long long wmass[kSmMaxWarps];
    uint32_t wcnt[kSmMaxWarps];
    float wmax[kSmMaxWarps];
};

// What top-k and top-p need besides, behind the slice.
struct SampleBins {
    uint32_t first[4][kSmBins];                      // counts, masses in three pieces
    union {
        uint2 few[2][kSmFew];                        // this CTA's gathered (key, id): for top-k, for top-p
        uint2 ent[kSmOne];                           // every CTA's listed ones, in the first CTA
    };
    uint2 all[kSmFew];                               // every CTA's
    unsigned long long mass[kSmFew];                 // and their masses
    uint32_t nlist, nent, base;
    uint32_t nfew[2];
    // what the first CTA found: whether it did, the cut, the kept mass
    int settled;
    SampleCutAt rcut;
    unsigned long long rmass;
    unsigned long long smass[kSmMaxWarps];           // scan of the bins
    uint32_t scnt[kSmMaxWarps];
    // where a target was found: bin (or -1), and what lies before and in it
    int bin;
    unsigned long long bmass_before;
    uint32_t bcnt_before, bcnt_at;
    int32_t nth;
    SampleCutAt cut;
    unsigned long long upto;
    uint16_t list[1];                                // (P.cap) positions in the slice, in no order
};

__device__ __forceinline__ uint32_t sm_peer(const void *p, uint32_t rank)
{
    uint32_t d;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_addr(p)), "r"(rank));
    return d;
}
__device__ __forceinline__ void sm_put(const void *p, uint32_t rank, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(sm_peer(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void sm_put(const void *p, uint32_t rank, unsigned long long v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(sm_peer(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t sm_get(const void *p, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(sm_peer(p, rank)));
    return v;
}
__device__ __forceinline__ uint2 sm_get2(const void *p, uint32_t rank)
{
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(sm_peer(p, rank)));
    return v;
}
// A pair of words summed over the cluster's CTAs (every load is on its way before
// the first is used).
__device__ __forceinline__ uint2 sm_sum2(const void *p, uint32_t C)
{
    uint2 t[kSmMaxCtas], s = make_uint2(0u, 0u);
#pragma unroll
    for (uint32_t k = 0; k < kSmMaxCtas; ++k)
        t[k] = k < C ? sm_get2(p, k) : make_uint2(0u, 0u);
#pragma unroll
    for (uint32_t k = 0; k < kSmMaxCtas; ++k) {
        s.x += t[k].x;
        s.y += t[k].y;
    }
    return s;
}
// Two words of a mass in pieces, summed as 64-bit numbers.
__device__ __forceinline__ void sm_add2(unsigned long long (&m)[2], const void *p, uint32_t C, int shift)
{
    uint2 t[kSmMaxCtas];
#pragma unroll
    for (uint32_t k = 0; k < kSmMaxCtas; ++k)
        t[k] = k < C ? sm_get2(p, k) : make_uint2(0u, 0u);
#pragma unroll
    for (uint32_t k = 0; k < kSmMaxCtas; ++k) {
        m[0] += static_cast<unsigned long long>(t[k].x) << shift;
        m[1] += static_cast<unsigned long long>(t[k].y) << shift;
    }
}
// The last barrier of a CTA: it has no word left to read in another, or for another
// to write.  Nothing is handed over, so it does not wait for q's stores.
__device__ __forceinline__ void sm_cluster_leave()
{
    asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}
__device__ __forceinline__ void sm_cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

constexpr float kSmShift = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number
constexpr uint32_t kSmShiftBits = 0x4B400000u;
constexpr float kSmLn1 = 0.021660849392498290f, kSmLn2 = kSmLn1 * kSmLn1 / 2, kSmLn3 = kSmLn1 * kSmLn1 * kSmLn1 / 6; // ln(2) / 32

// What a row's masses are formed with.
struct SampleRow {
    float m;          // the maximum
    float off;        // what is taken off a logit first: 0 (or m, rows whose m c is 2^21 or more)
    float low;        // the least difference that is looked at: below it nothing has mass
    float shift;      // kSmShift less the whole number next above m c (0 with off m)
    float c_hi, c_lo;
    uint32_t tab;     // shared-memory address of the table
    int down;         // 59 - fix, and the shift's bits beside k's octaves
    // m and the constants of a call.  c = c_hi + c_lo to 2^-48 of itself.
    __device__ __forceinline__ void set(float mx, float hi, float lo, float dmin)
    {
        m = mx;
        c_hi = hi;
        c_lo = lo;
        const float mc = __fmaf_rn(mx, hi, __fmul_rn(mx, lo));
        const bool near = fabsf(mc) < 2097152.0f;
        off = near ? 0.0f : mx;
        low = near ? mx + dmin : dmin;
        shift = near ? kSmShift - ceilf(mc) : kSmShift;
    }
    // The masses of two logits z <= m, in units of 2^-fix, rounded; 0 for -inf.  The
    // maximum's is 1 (with off m), or less by at most the 32nd part of an octave.
    // (Pairs: the arithmetic is packed.)
    __device__ __forceinline__ void masses(float z0, float z1, unsigned long long &w0, unsigned long long &w1) const
    {
        float d0, d1;
        unpack2(add2(pack2(z0, z1), pack2(-off, -off)), d0, d1);
        const unsigned long long d = pack2(fmaxf(d0, low), fmaxf(d1, low)), S = pack2(shift, shift);
        const unsigned long long t = fma2(d, pack2(c_hi, c_hi), S);
        // d c less the whole number in t: the product's high part is not rounded before
        unsigned long long r = fma2(d, pack2(c_hi, c_hi), fma2(t, pack2(-1.0f, -1.0f), S));
        r = fma2(d, pack2(c_lo, c_lo), r);
        // e^x - 1, x = r ln(2) / 32: x + x^2 / 2 + x^3 / 6
        unsigned long long p = fma2(r, pack2(kSmLn3, kSmLn3), pack2(kSmLn2, kSmLn2));
        p = mul2(fma2(r, p, pack2(kSmLn1, kSmLn1)), r);
        float t0, t1, p0, p1;
        unpack2(t, t0, t1);
        unpack2(p, p0, p1);
        w0 = whole(t0, p0);
        w1 = whole(t1, p1);
    }
    __device__ __forceinline__ unsigned long long whole(float t, float p) const
    {
        const uint32_t bits = __float_as_uint(t); // k beside the shift's bits
        float2 e;
        asm("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(e.x), "=f"(e.y) : "r"(tab + ((bits & 31u) << 3)));
        const int s = down - static_cast<int>(bits >> 5); // 59 - fix + octaves below the maximum: 14 or more
        uint32_t half; // half a unit of the result, where bits are lost (a shift by a negative number gives 0)
        asm("shl.b32 %0, 1, %1;" : "=r"(half) : "r"(s - 33));
        const uint32_t E = __float_as_uint(e.y) + __float_as_uint(__fmaf_rn(e.x, p, kSmShift)) + half;
        return (static_cast<unsigned long long>(E) << 32) >> s;
    }
    __device__ __forceinline__ unsigned long long mass(float z) const
    {
        unsigned long long w0, w1;
        masses(z, z, w0, w1);
        return w0;
    }
};

__device__ __forceinline__ void sm_init_table(SampleShared &S)
{
    if (threadIdx.x < 32) {
        const double v = exp2(static_cast<double>(threadIdx.x) / 32.0) * 134217728.0;
        S.tab[threadIdx.x] =
            make_float2(static_cast<float>(v), __uint_as_float(static_cast<uint32_t>(v + 0.5) - kSmShiftBits));
    }
}

// This CTA's slice of a row.  Position p (16-byte vectors of PV positions) holds
// id first + p; positions outside the slice read as -inf.
template <typename LT> struct SampleSlice {
    using E = FilterElem<LT>;
    static constexpr int PV = E::kPerVec;
    const LT *row;     // the row's ids
    const uint4 *mem;  // staged vectors, or nullptr
    int32_t first;     // id of position 0 (may be below the slice's first)
    int32_t lo, hi;    // ids of the slice
    int32_t nv;        // vectors
    // vector v straight from memory
    __device__ __forceinline__ uint4 fetch(int32_t v) const
    {
        const int32_t i = first + v * PV;
        if (i >= lo && i + PV <= hi)
            return ld_stream_v4(row + i);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (PV == 8) {
                const int32_t a = i + 2 * k;
                const uint32_t l = a >= lo && a < hi ? filter_bits<LT>(row, a) : E::kNegInf;
                const uint32_t h = a + 1 >= lo && a + 1 < hi ? filter_bits<LT>(row, a + 1) : E::kNegInf;
                w[k] = l | (h << 16);
            } else {
                w[k] = i + k >= lo && i + k < hi ? filter_bits<LT>(row, i + k) : E::kNegInf;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ uint4 vec(int32_t v) const { return mem ? mem[v] : fetch(v); }
    __device__ __forceinline__ static uint32_t of(const uint4 &w, int j)
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        if constexpr (PV == 8)
            return j & 1 ? u[j >> 1] >> 16 : u[j >> 1] & 0xFFFFu;
        else
            return u[j];
    }
};

// Every CTA's sums (mass and cnt, the same in all threads of one) in every CTA:
// the row of slots that got them.  The rows are used in turn: between two uses of
// one lies a barrier that its readers had to reach.
__device__ __forceinline__ int sm_exchange(SampleShared &S, int &turn, uint32_t C, uint32_t rank, unsigned long long mass,
                                           uint32_t cnt)
{
    const int use = turn++ & 3;
    if (threadIdx.x < C) {
        sm_put(&S.cmass[use][rank], threadIdx.x, mass);
        sm_put(&S.ccnt[use][rank], threadIdx.x, cnt);
    }
    sm_cluster_sync();
    return use;
}

// Every thread gets the CTA's sums of (mass, cnt); each warp's own are left in
// S.wmass, S.wcnt.
template <int NT> __device__ __forceinline__ void sm_block_sum(SampleShared &S, unsigned long long &mass, uint32_t &cnt)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    mass = static_cast<unsigned long long>(warp_sum_ll(static_cast<long long>(mass)));
    cnt = __reduce_add_sync(0xFFFFFFFFu, cnt);
    __syncthreads();
    if (lane == 0) {
        S.wmass[warp] = mass;
        S.wcnt[warp] = cnt;
    }
    __syncthreads();
    mass = 0;
    cnt = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        mass += S.wmass[w];
        cnt += S.wcnt[w];
    }
}

// This thread's bins (the first is N threadIdx.x) in order: the bin where the
// running count (MASS false; masses are then not looked at) or mass reaches
// `target`, in S.bin, S.b*.  Also the sums of all bins.
template <bool MASS, int NT, int N>
__device__ __forceinline__ void sm_scan(SampleBins &S, const uint32_t (&cnt)[N], const unsigned long long (&mass)[N],
                                        unsigned long long target, uint32_t &cnt_all, unsigned long long &mass_all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t c = 0;
    unsigned long long m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        c += cnt[i];
        m += MASS ? mass[i] : 0ull;
    }
    unsigned long long mi = m;
    uint32_t ci = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, ci, o);
        ci += lane >= o ? n : 0u;
        if (MASS) {
            const unsigned long long k = __shfl_up_sync(0xFFFFFFFFu, mi, o);
            mi += lane >= o ? k : 0ull;
        }
    }
    __syncthreads(); // what was found before has been read
    if (lane == 31) {
        S.smass[warp] = mi;
        S.scnt[warp] = ci;
    }
    if (threadIdx.x == 0)
        S.bin = -1;
    __syncthreads();
    unsigned long long mb = mi - m;
    uint32_t cb = ci - c;
    mass_all = 0;
    cnt_all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const uint32_t sc = S.scnt[w];
        cb += w < warp ? sc : 0u;
        cnt_all += sc;
        if (MASS) {
            const unsigned long long sm = S.smass[w];
            mb += w < warp ? sm : 0ull;
            mass_all += sm;
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const unsigned long long before = MASS ? mb : cb, here = MASS ? mass[i] : cnt[i];
        if (before < target && target <= before + here) {
            S.bin = static_cast<int>(threadIdx.x) * N + i;
            S.bcnt_before = cb;
            S.bcnt_at = cnt[i];
            S.bmass_before = mb;
        }
        mb += MASS ? mass[i] : 0ull;
        cb += cnt[i];
    }
    __syncthreads();
}

// This thread's bins of S.first over the cluster.
template <int N> __device__ __forceinline__ void sm_counts(const SampleBins &S, uint32_t C, uint32_t (&cnt)[N])
{
    if constexpr (N == 2) {
        const uint2 c = sm_sum2(&S.first[0][2 * threadIdx.x], C);
        cnt[0] = c.x;
        cnt[1] = c.y;
    } else {
        uint32_t t[kSmMaxCtas];
#pragma unroll
        for (uint32_t k = 0; k < kSmMaxCtas; ++k)
            t[k] = k < C ? sm_get(&S.first[0][threadIdx.x], k) : 0u;
        cnt[0] = 0;
#pragma unroll
        for (uint32_t k = 0; k < kSmMaxCtas; ++k)
            cnt[0] += t[k];
    }
}
template <int N>
__device__ __forceinline__ void sm_masses(const SampleBins &S, uint32_t C, int piece, unsigned long long (&mass)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        mass[i] = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if constexpr (N == 2) {
            sm_add2(mass, &S.first[1 + i][2 * threadIdx.x], C, i * piece);
        } else {
            uint32_t t[kSmMaxCtas];
#pragma unroll
            for (uint32_t k = 0; k < kSmMaxCtas; ++k)
                t[k] = k < C ? sm_get(&S.first[1 + i][threadIdx.x], k) : 0u;
#pragma unroll
            for (uint32_t k = 0; k < kSmMaxCtas; ++k)
                mass[0] += static_cast<unsigned long long>(t[k]) << (i * piece);
        }
    }
}

// The same of this CTA alone.
template <int N> __device__ __forceinline__ void sm_counts_here(const SampleBins &S, uint32_t (&cnt)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        cnt[i] = S.first[0][N * threadIdx.x + i];
}
template <int N>
__device__ __forceinline__ void sm_masses_here(const SampleBins &S, int piece, unsigned long long (&mass)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        mass[i] = S.first[1][N * threadIdx.x + i] + (static_cast<unsigned long long>(S.first[2][N * threadIdx.x + i]) << piece) +
                  (static_cast<unsigned long long>(S.first[3][N * threadIdx.x + i]) << (2 * piece));
}

// An id's mass into bin b.
__device__ __forceinline__ void sm_add_mass(SampleBins &S, uint32_t b, unsigned long long e, int piece)
{
    const uint32_t low = (1u << piece) - 1u;
    atomicAdd(&S.first[0][b], 1u);
    atomicAdd(&S.first[1][b], static_cast<uint32_t>(e) & low);
    atomicAdd(&S.first[2][b], static_cast<uint32_t>(e >> piece) & low);
    atomicAdd(&S.first[3][b], static_cast<uint32_t>(e >> (2 * piece)));
}
template <int NT> __device__ __forceinline__ void sm_clear(SampleBins &S)
{
    for (int i = threadIdx.x; i < 4 * kSmBins; i += NT)
        S.first[0][i] = 0u;
    __syncthreads();
}

// A cut as it is found: all ids of larger keys, and the first j of the `ties` ids
// with this one (or, `known`, those up to an id).
struct SampleFound {
    bool any;                 // whether there is a cut: the target was reached
    bool known;
    uint32_t key;
    int32_t id;
    uint32_t j, ties;
    uint32_t below;           // of the ties, how many in the CTAs before this one
    uint32_t mine;            // and in this one
    unsigned long long upto;  // mass through the cut (through everything, without one)
};

// Step 2's bin of a logit, from 0 for the maximum up; kSmBins or more for what lies
// below the bins.  It never grows with the logit (a difference and a product, each
// rounded), so a bin is a range of keys.
__device__ __forceinline__ uint32_t sm_bin(const SampleRow &R, float z, float scale)
{
    return __float_as_uint(__fmaf_rn(R.m - z, scale, 8388608.0f)) - 0x4B000000u;
}
// The least key of bin b or one before, by bisection.
template <typename LT> __device__ __forceinline__ uint32_t sm_first_key(const SampleRow &R, float scale, uint32_t b, uint32_t ktop)
{
    using E = FilterElem<LT>;
    uint32_t lo = E::kKeyMin, hi = ktop; // (the maximum's bin is 0)
    while (lo < hi) {
        const uint32_t mid = lo + ((hi - lo) >> 1);
        if (sm_bin(R, E::value(E::bits_of_key(mid)), scale) <= b)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// The largest logit of a vector.
template <typename LT> __device__ __forceinline__ float sm_largest(const uint4 &w)
{
    if constexpr (sizeof(LT) == 2) {
        uint32_t a, b;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
        return fmaxf(bf16_lo(a), bf16_hi(a));
    } else {
        return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
}

// ... and its smallest.
template <typename LT> __device__ __forceinline__ float sm_smallest(const uint4 &w)
{
    if constexpr (sizeof(LT) == 2) {
        uint32_t a, b;
        asm("min.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
        asm("min.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
        asm("min.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
        return fminf(bf16_lo(a), bf16_hi(a));
    } else {
        return fminf(fminf(__uint_as_float(w.x), __uint_as_float(w.y)), fminf(__uint_as_float(w.z), __uint_as_float(w.w)));
    }
}

// The ids of bins 0 .. last of step 2 in this CTA: listed, or picked out of the slice.
template <typename LT, int NT> struct SampleSet {
    const SampleSlice<LT> &X;
    const SampleRow &R;
    float scale;
    uint32_t last;
    const uint16_t *list; // or nullptr
    uint32_t n;
    __device__ __forceinline__ uint32_t bits(uint32_t i) const
    {
        if constexpr (sizeof(LT) == 2)
            return reinterpret_cast<const unsigned short *>(X.mem)[list[i]];
        else
            return reinterpret_cast<const uint32_t *>(X.mem)[list[i]];
    }
    __device__ __forceinline__ int32_t id(uint32_t i) const { return X.first + list[i]; }
    // f(bits, id, bin) for each, in no order
    template <typename F> __device__ __forceinline__ void each(F &&f) const
    {
        using E = FilterElem<LT>;
        if (list) {
            for (uint32_t i = threadIdx.x; i < n; i += NT) {
                const uint32_t b = bits(i);
                f(b, id(i), sm_bin(R, E::value(b), scale));
            }
        } else {
            for (int32_t v = threadIdx.x; v < X.nv; v += NT) {
                const uint4 w = X.vec(v);
                if (sm_bin(R, sm_largest<LT>(w), scale) > last)
                    continue;
#pragma unroll 1
                for (int j = 0; j < E::kPerVec; ++j) {
                    const uint32_t b = SampleSlice<LT>::of(w, j), bin = sm_bin(R, E::value(b), scale);
                    if (bin <= last)
                        f(b, X.first + v * E::kPerVec + j, bin);
                }
            }
        }
    }
};

// Every CTA's gathered ids (`use`: 0 or 1), and their masses, in S.all, S.mass; how many.
template <typename LT>
__device__ __forceinline__ uint32_t sm_collect(const SampleRow &R, int use, uint32_t C, SampleBins &S)
{
    using E = FilterElem<LT>;
    sm_cluster_sync();
    // how many each CTA has, a lane each; then every thread its entry
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t c = lane < C ? min(sm_get(&S.nfew[use], lane), static_cast<uint32_t>(kSmFew)) : 0u;
    uint32_t i = threadIdx.x, from = C, n = 0;
#pragma unroll
    for (uint32_t r = 0; r < kSmMaxCtas; ++r) {
        const uint32_t cr = __shfl_sync(0xFFFFFFFFu, c, r);
        if (from == C && i < cr)
            from = r;
        if (from == C)
            i -= cr;
        n += cr;
    }
    n = min(n, static_cast<uint32_t>(kSmFew));
    if (threadIdx.x < n) {
        const uint2 e = sm_get2(&S.few[use][i], from);
        S.all[threadIdx.x] = e;
        S.mass[threadIdx.x] = R.mass(E::value(E::bits_of_key(e.x)));
    }
    __syncthreads();
    return n;
}

// How many of the n collected ids rank before `me`, and their mass.
__device__ __forceinline__ void sm_rank(const SampleBins &S, uint32_t n, uint2 me, uint32_t &before, unsigned long long &mass)
{
    before = 0;
    mass = 0;
#pragma unroll 4
    for (uint32_t i = 0; i < n; ++i) {
        const uint2 o = S.all[i];
        const bool b = o.x > me.x | (o.x == me.x & o.y < me.y);
        const unsigned long long w = S.mass[i];
        before += b ? 1u : 0u;
        mass += b ? w : 0ull;
    }
}

// The ids of bin `bin` that `bound` keeps, at most kSmFew in all: gathered by every
// CTA and ranked; the cut where the running count or mass reaches target.
template <typename LT, int NT, bool MASS>
__device__ SampleFound sm_gather(const SampleSet<LT, NT> &Set, uint32_t bin, unsigned long long above,
                                 unsigned long long target, SampleCutAt bound, int use, uint32_t C, SampleBins &S)
{
    Set.each([&](uint32_t bits, int32_t id, uint32_t b) {
        const uint32_t k = FilterElem<LT>::key(bits);
        if (b != bin || k < bound.key || (k == bound.key && id > bound.id))
            return;
        const uint32_t at = atomicAdd(&S.nfew[use], 1u);
        if (at < kSmFew) // (the bin's count bounds it)
            S.few[use][at] = make_uint2(k, static_cast<uint32_t>(id));
    });
    const uint32_t n = sm_collect<LT>(Set.R, use, C, S);
    if (threadIdx.x == 0)
        S.bin = -1;
    __syncthreads();
    if (threadIdx.x < n) {
        const uint2 me = S.all[threadIdx.x];
        uint32_t before;
        unsigned long long mass;
        sm_rank(S, n, me, before, mass);
        const unsigned long long w = S.mass[threadIdx.x];
        const unsigned long long b = MASS ? mass : before, here = MASS ? w : 1;
        if (b < target && target <= b + here) {
            S.bin = 0;
            S.cut = {me.x, static_cast<int32_t>(me.y)};
            S.upto = mass + w;
        }
    }
    __syncthreads();
    SampleFound f = {};
    f.any = S.bin == 0; // the target lies in the bin: found
    f.known = true;
    f.key = S.cut.key;
    f.id = S.cut.id;
    f.upto = above + S.upto;
    __syncthreads();
    return f;
}

// The cut among the ids with keys in [klo, khi], digit by digit.
template <typename LT, int NT, bool MASS>
__device__ SampleFound sm_narrow(const SampleSlice<LT> &X, const SampleRow &R, uint32_t klo, uint32_t khi,
                                 unsigned long long above, unsigned long long target, int piece, uint32_t C, uint32_t rank,
                                 SampleBins &S)
{
    using E = FilterElem<LT>;
    constexpr int N = kSmBins / NT;
    SampleFound f = {};
    for (;;) {
        const uint32_t span = khi - klo;
        const int sh = span < kSmBins ? 0 : 32 - __clz(span) - 9;
        sm_cluster_sync(); // every CTA has read the bins
        sm_clear<NT>(S);
        for (int32_t v = threadIdx.x; v < X.nv; v += NT) {
            const uint4 w = X.vec(v);
#pragma unroll 1
            for (int j = 0; j < E::kPerVec; ++j) {
                const uint32_t bits = SampleSlice<LT>::of(w, j), k = E::key(bits);
                if (k >= klo && k <= khi && E::finite(bits))
                    sm_add_mass(S, (khi - k) >> sh, R.mass(E::value(bits)), piece);
            }
        }
        sm_cluster_sync();
        uint32_t cnt[N], cnt_all;
        unsigned long long mass[N], mass_all;
        sm_counts(S, C, cnt);
        sm_masses(S, C, piece, mass);
        unsigned long long before = 0;
        if (MASS) {
            sm_scan<true, NT>(S, cnt, mass, target, cnt_all, mass_all);
        } else { // and the mass before the bin
            sm_scan<false, NT>(S, cnt, mass, target, cnt_all, mass_all);
            const int bin = S.bin;
            unsigned long long own = 0;
#pragma unroll
            for (int i = 0; i < N; ++i)
                own += static_cast<int>(threadIdx.x) * N + i < bin || bin < 0 ? mass[i] : 0ull;
            own = static_cast<unsigned long long>(warp_sum_ll(static_cast<long long>(own)));
            if ((threadIdx.x & 31) == 0)
                S.smass[threadIdx.x >> 5] = own;
            __syncthreads();
            for (int w = 0; w < NT / 32; ++w)
                before += S.smass[w];
            mass_all = before;
        }
        const int bin = S.bin;
        f.any = bin >= 0;
        if (!f.any) {
            f.upto = above + mass_all;
            return f;
        }
        above += MASS ? S.bmass_before : before;
        target -= MASS ? S.bmass_before : S.bcnt_before;
        khi -= static_cast<uint32_t>(bin) << sh;
        const uint32_t width = (1u << sh) - 1u;
        klo = khi - klo > width ? khi - width : klo;
        f.ties = S.bcnt_at;
        if (klo == khi) {
            for (uint32_t r = 0; r < rank; ++r)
                f.below += sm_get(&S.first[0][bin], r);
            f.mine = sm_get(&S.first[0][bin], rank);
            break;
        }
    }
    f.key = khi;
    const unsigned long long w = R.mass(E::value(E::bits_of_key(khi)));
    unsigned long long j = MASS ? (w ? (target + w - 1) / w : 1) : target;
    f.j = static_cast<uint32_t>(j < 1 ? 1 : (j > f.ties ? f.ties : j));
    f.upto = above + f.j * w;
    return f;
}

// An entry's place in S.all, with its mass.
__device__ __forceinline__ void sm_keep(SampleBins &S, uint2 e, unsigned long long w)
{
    const uint32_t at = atomicAdd(&S.nfew[0], 1u);
    if (at < kSmFew) { // (the bin's count bounds it)
        S.all[at] = e;
        S.mass[at] = w;
    }
}

// The first CTA settles a row from the n (key, id) in S.ent, the ids of bins 0 .. b1:
// the cuts (top-k's among the kties ids of bin b1, at the kleft-th; top-p's in bins
// b0 .. b1), the token, its probability, how many are kept.  False where a bin
// holds more ids than are ranked; nothing has been written then.
template <typename LT, int NT>
__device__ bool sm_settle_row(const SampleParams &P, const SampleRow &R, SampleShared &Sh, SampleBins &S, uint32_t n, uint32_t b0,
                              uint32_t b1, uint32_t kties, unsigned long long kleft, unsigned long long total, float zlo,
                              float u, int64_t r, SampleCutAt &cut, unsigned long long &Z)
{
    using E = FilterElem<LT>;
    constexpr int N = kSmBins / NT;
    const bool use_k = P.top_k > 0 && P.top_k < P.V, use_p = P.top_p < 1.0f;
    auto value = [&](uint2 e) { return E::value(E::bits_of_key(e.x)); };
    auto within = [](uint2 e, SampleCutAt c) { return e.x > c.key || (e.x == c.key && static_cast<int32_t>(e.y) <= c.id); };
    cut = {0u, 0x7FFFFFFF};
    auto rank_all = [&](auto by_mass, uint32_t m, unsigned long long target) { // the cut among S.all's m
        constexpr bool MASS = decltype(by_mass)::value;
        __syncthreads();
        if (threadIdx.x < m) {
            const uint2 me = S.all[threadIdx.x];
            uint32_t before;
            unsigned long long mass;
            sm_rank(S, m, me, before, mass);
            const unsigned long long w = S.mass[threadIdx.x], b = MASS ? mass : before, here = MASS ? w : 1;
            if (b < target && target <= b + here)
                S.cut = {me.x, static_cast<int32_t>(me.y)};
        }
        if (threadIdx.x == 0)
            S.nfew[0] = 0u;
        __syncthreads();
        cut = S.cut;
    };
    if (use_k) {
        if (kties > kSmFew)
            return false;
        for (uint32_t i = threadIdx.x; i < n; i += NT) {
            const uint2 e = S.ent[i];
            if (sm_bin(R, value(e), P.bins) == b1)
                sm_keep(S, e, 0ull);
        }
        rank_all(std::false_type{}, kties, kleft);
    }
    uint32_t cnt[N], cnt_all;
    unsigned long long mass[N], mass_all;
    if (use_p) {
        sm_clear<NT>(S);
        unsigned long long above = 0;
        uint32_t none = 0;
        for (uint32_t i = threadIdx.x; i < n; i += NT) {
            const uint2 e = S.ent[i];
            if (!within(e, cut))
                continue;
            const float z = value(e);
            const unsigned long long w = R.mass(z);
            const uint32_t b = sm_bin(R, z, P.bins);
            if (b < b0)
                above += w;
            else
                sm_add_mass(S, b, w, P.piece);
        }
        sm_block_sum<NT>(Sh, above, none);
        sm_counts_here(S, cnt);
        sm_masses_here(S, P.piece, mass);
        if (use_k) {
            sm_scan<true, NT>(S, cnt, mass, 1, cnt_all, mass_all);
            total = mass_all;
        }
        const double x = ceil(static_cast<double>(P.top_p) * static_cast<double>(total));
        const unsigned long long target = static_cast<unsigned long long>(x < 1.0 ? 1.0 : x);
        const unsigned long long left = target > above ? target - above : 1;
        sm_scan<true, NT>(S, cnt, mass, left, cnt_all, mass_all);
        const uint32_t bin = static_cast<uint32_t>(S.bin), ties = S.bcnt_at;
        const unsigned long long before = S.bmass_before;
        if (S.bin < 0 || ties > kSmFew)
            return false;
        for (uint32_t i = threadIdx.x; i < n; i += NT) {
            const uint2 e = S.ent[i];
            const float z = value(e);
            if (sm_bin(R, z, P.bins) == bin && within(e, cut))
                sm_keep(S, e, R.mass(z));
        }
        rank_all(std::true_type{}, ties, left - before);
    }
    // the kept masses by runs of ids
    const uint32_t run = (static_cast<uint32_t>(P.V) + kSmBins - 1) / kSmBins;
    sm_clear<NT>(S);
    Z = 0;
    uint32_t kept = 0;
    for (uint32_t i = threadIdx.x; i < n; i += NT) {
        const uint2 e = S.ent[i];
        const float z = value(e);
        if (!within(e, cut) || z < zlo)
            continue;
        const unsigned long long w = R.mass(z);
        Z += w;
        ++kept;
        sm_add_mass(S, e.y / run, w, P.piece);
    }
    sm_block_sum<NT>(Sh, Z, kept);
    sm_counts_here(S, cnt);
    sm_masses_here(S, P.piece, mass);
    const bool good = u >= 0.0f && u < 1.0f;
    const unsigned long long t = static_cast<unsigned long long>(mul_floor(good ? u : 0.0f, static_cast<long long>(Z)));
    sm_scan<true, NT>(S, cnt, mass, t + 1, cnt_all, mass_all);
    const uint32_t at = static_cast<uint32_t>(S.bin), m = S.bcnt_at;
    const unsigned long long before = S.bmass_before;
    if (m > kSmFew)
        return false;
    for (uint32_t i = threadIdx.x; i < n; i += NT) {
        const uint2 e = S.ent[i];
        const float z = value(e);
        if (e.y / run == at && within(e, cut) && z >= zlo)
            sm_keep(S, e, R.mass(z));
    }
    __syncthreads();
    if (threadIdx.x < m && good) {
        const uint2 me = S.all[threadIdx.x];
        unsigned long long upto = before;
        for (uint32_t i = 0; i < m; ++i)
            upto += S.all[i].y <= me.y ? S.mass[i] : 0ull;
        const unsigned long long w = S.mass[threadIdx.x];
        if (t < upto && t >= upto - w) {
            P.tokens[r] = static_cast<int32_t>(me.y);
            if (P.prob)
                P.prob[r] = static_cast<float>(static_cast<double>(w) / static_cast<double>(Z));
        }
    }
    if (threadIdx.x == 0 && P.kept)
        P.kept[r] = static_cast<int32_t>(kept);
    return true;
}

// A found cut as every CTA compares with it: (key, id).
template <typename LT>
__device__ SampleCutAt sm_settle(const SampleSlice<LT> &X, const SampleFound &f, int32_t v0, int32_t v1, SampleBins &S)
{
    using E = FilterElem<LT>;
    constexpr int PV = E::kPerVec;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!f.any)
        return {0u, 0x7FFFFFFF}; // everything finite
    if (f.known)
        return {f.key, f.id};
    if (f.j >= f.below + f.mine)
        return {f.key, 0x7FFFFFFF};
    if (f.j <= f.below)
        return {f.key, -1};
    // this CTA's want-th id of the value, in id order
    const uint32_t want = f.j - f.below;
    auto hits = [&](int32_t v) {
        uint32_t h = 0;
        if (v < v1) {
            const uint4 w = X.vec(v);
#pragma unroll
            for (int j = 0; j < PV; ++j) {
                const uint32_t bits = SampleSlice<LT>::of(w, j);
                h |= E::finite(bits) && E::key(bits) == f.key ? 1u << j : 0u;
            }
        }
        return h;
    };
    uint32_t n = 0;
    for (int32_t v = v0 + lane; v < v1; v += 32)
        n += __popc(hits(v));
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0)
        S.scnt[warp] = n;
    __syncthreads();
    uint32_t at = 0;
    for (int w = 0; w < warp; ++w)
        at += S.scnt[w];
    if (at < want && want <= at + n) {
        for (int32_t v = v0; v < v1; v += 32) {
            uint32_t h = hits(v + lane);
            const uint32_t c = __popc(h);
            uint32_t incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                incl += lane >= o ? up : 0u;
            }
            const uint32_t before = at + incl - c;
            if (before < want && want <= before + c) {
                for (uint32_t i = want - before; i > 1; --i)
                    h &= h - 1;
                S.nth = X.first + (v + lane) * PV + __ffs(h) - 1;
            }
            at += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
    }
    __syncthreads();
    const int32_t id = S.nth;
    __syncthreads();
    return {f.key, id};
}

// The processed distribution over this CTA's ids, Z its mass in units of 2^-fix.
template <typename LT, int NT, bool CUTS>
__device__ __forceinline__ void sm_write_q(const SampleSlice<LT> &X, const SampleRow &R, const SampleParams &P, float *qrow,
                                           float zlo, SampleCutAt cut, unsigned long long Z)
{
    using E = FilterElem<LT>;
    constexpr int PV = E::kPerVec;
    if (!qrow)
        return;
    float least = zlo;
    if (CUTS && cut.key)
        least = fmaxf(least, E::value(E::bits_of_key(cut.key)));
    const float cq = P.cq, scale = static_cast<float>(R.mass(R.m)) / static_cast<float>(Z);
    const bool filtered = CUTS || P.min_p;
    for (int32_t v = threadIdx.x; v < X.nv; v += NT) {
        const uint4 w = X.vec(v);
        const int32_t i = X.first + v * PV;
        float q[PV];
        if (!filtered) { // (exp2 of -inf is 0)
#pragma unroll
            for (int j = 0; j < PV; ++j)
                q[j] = ex2(__fmul_rn(E::value(SampleSlice<LT>::of(w, j)) - R.m, cq)) * scale;
        } else if (sm_largest<LT>(w) >= least) {
#pragma unroll
            for (int j = 0; j < PV; ++j) {
                const uint32_t b = SampleSlice<LT>::of(w, j);
                const bool in = E::finite(b) && E::value(b) >= least && (!CUTS || E::key(b) != cut.key || i + j <= cut.id);
                q[j] = in ? ex2(__fmul_rn(E::value(b) - R.m, cq)) * scale : 0.0f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < PV; ++j)
                q[j] = 0.0f;
        }
        if (P.vec_q && i >= X.lo && i + PV <= X.hi) {
#pragma unroll
            for (int j = 0; j < PV; j += 4)
                __stcs(reinterpret_cast<float4 *>(qrow + i + j), make_float4(q[j], q[j + 1], q[j + 2], q[j + 3]));
        } else {
#pragma unroll
            for (int j = 0; j < PV; ++j)
                if (i + j >= X.lo && i + j < X.hi)
                    qrow[i + j] = q[j];
        }
    }
}

// CUTS: whether there is a top-k or a top-p.
template <typename LT, int NT, bool CUTS>
__global__ void __launch_bounds__(NT, (CUTS ? 1024 : 1280) / NT) sample_kernel(const SampleParams P)
{
    using E = FilterElem<LT>;
    using Slice = SampleSlice<LT>;
    constexpr int PV = E::kPerVec;
    constexpr bool F32 = sizeof(LT) == 4;
    extern __shared__ __align__(16) uint8_t sm_raw[];
    __shared__ SampleShared S;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t C = static_cast<uint32_t>(P.C), rank = blockIdx.x % C;
    const int64_t r = blockIdx.x / C;
    const LT *row = static_cast<const LT *>(P.in) + r * P.V;
    // a CTA's shared memory may be written to once it has arrived here
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    sm_init_table(S);
    SampleBins &H = *reinterpret_cast<SampleBins *>(sm_raw + (P.staged ? static_cast<size_t>(P.slice) * sizeof(LT) : 0));
    if constexpr (CUTS) {
        for (int i = threadIdx.x; i < 4 * kSmBins; i += NT)
            H.first[0][i] = 0u;
        if (threadIdx.x < 2)
            H.nfew[threadIdx.x] = 0u;
        if (threadIdx.x == 0)
            H.nlist = H.nent = 0u;
    }
    pdl_wait_primary();
    pdl_launch_dependents();

    // this CTA's ids, in vectors from a 16-byte boundary on
    Slice X;
    X.row = row;
    const int32_t skew = static_cast<int32_t>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(LT));
    X.first = static_cast<int32_t>(rank) * P.slice - skew;
    X.lo = min(max(X.first, 0), P.V);
    X.hi = max(min(P.V, X.first + P.slice), X.lo);
    X.nv = X.hi > X.lo ? (X.hi - X.first + PV - 1) / PV : 0;
    X.mem = nullptr;
    uint4 *stage = reinterpret_cast<uint4 *>(sm_raw);
    // 1. load, maximum.  The maximum that passes NaN on is NaN or +inf for a row
    // that holds one.
    float mx = -INFINITY;
    {
        auto fold = [&](const uint4 &w) {
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            if constexpr (PV == 8) {
                uint32_t a, b;
                asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(u[0]), "r"(u[1]));
                asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(u[2]), "r"(u[3]));
                asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
                asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(bf16_lo(a)));
                asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(bf16_hi(a)));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(__uint_as_float(u[k])));
            }
        };
        if (P.staged) {
            // every vector on its way at once; a slice's ragged ends by way of registers
            for (int32_t v = threadIdx.x; v < X.nv; v += NT) {
                const int32_t i = X.first + v * PV;
                if (i >= X.lo && i + PV <= X.hi)
                    cp_async16(stage + v, row + i);
                else
                    stage[v] = X.fetch(v);
            }
            asm volatile("cp.async.wait_all;" ::: "memory"); // (a thread folds what it copied)
#pragma unroll 4
            for (int32_t v = threadIdx.x; v < X.nv; v += NT)
                fold(lds_v4(stage + v));
        } else {
#pragma unroll 4
            for (int32_t v = threadIdx.x; v < X.nv; v += NT)
                fold(X.fetch(v));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(__shfl_xor_sync(0xFFFFFFFFu, mx, o)));
        if (lane == 0)
            S.wmax[warp] = mx;
        __syncthreads();
        mx = S.wmax[0];
#pragma unroll
        for (int w = 1; w < NT / 32; ++w)
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(S.wmax[w]));
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        if (threadIdx.x < C)
            sm_put(&S.cmax[rank], threadIdx.x, __float_as_uint(mx));
        sm_cluster_sync();
        for (uint32_t k = 0; k < C; ++k)
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(S.cmax[k]));
    }
    if (P.staged)
        X.mem = stage;
    const float u = __ldg(P.u + r);
    const bool bad_row = !(fabsf(mx) < INFINITY), bad_u = !(u >= 0.0f && u < 1.0f);
    float *qrow = P.probs ? P.probs + r * P.V : nullptr;
    if ((bad_row || bad_u) && rank == 0 && threadIdx.x == 0) {
        if (P.status)
            atomicOr(P.status, (bad_row ? kBadRow : 0) | (bad_u ? kBadU : 0));
        P.tokens[r] = -1;
        if (P.prob)
            P.prob[r] = 0.0f;
        if (bad_row && P.kept)
            P.kept[r] = 0;
    }
    if (bad_row) { // the same in every CTA
        if (qrow)
            for (int32_t i = X.lo + threadIdx.x; i < X.hi; i += NT)
                qrow[i] = 0.0f;
        sm_cluster_leave();
        return;
    }
    SampleRow R;
    R.set(mx, P.c_hi, P.c_lo, P.dmin);
    R.tab = smem_addr(S.tab);
    R.down = 59 - P.fix + static_cast<int>(kSmShiftBits >> 5);
    // min-p: the least logit kept (p >= min_p max p, in logits)
    const float zlo = P.min_p ? __double2float_ru(static_cast<double>(mx) + P.min_off) : -INFINITY;
    const bool use_k = P.top_k > 0 && P.top_k < P.V, use_p = P.top_p < 1.0f;
    // a warp's part of the slice
    const int32_t part = (X.nv + NT / 32 - 1) / (NT / 32);
    const int32_t v0 = min(X.nv, warp * part), v1 = min(X.nv, v0 + part);

    SampleCutAt cut = {0u, 0x7FFFFFFF}; // everything finite
    int turn = 0;
    const uint16_t *list = nullptr; // of the ids that may be kept, with a cut
    uint32_t nlist = 0;
    if constexpr (CUTS) {
        // 2. counts in bins; the whole row's mass
        const uint32_t ktop = E::key(F32 ? __float_as_uint(mx) : __float_as_uint(mx) >> 16);
        const bool whole = !use_k; // what top-p refers to
        unsigned long long total = 0;
        auto pass = [&](auto with_mass) {
            constexpr bool kMass = decltype(with_mass)::value;
            for (int32_t v = v0 + lane; v < v1; v += 32) {
                const uint4 w = X.vec(v);
#pragma unroll
                for (int j = 0; j < PV; j += 2) {
                    const float z0 = E::value(Slice::of(w, j)), z1 = E::value(Slice::of(w, j + 1));
                    if (kMass) {
                        unsigned long long e0, e1;
                        R.masses(z0, z1, e0, e1);
                        total += e0 + e1;
                    }
                    const uint32_t b0 = sm_bin(R, z0, P.bins), b1 = sm_bin(R, z1, P.bins);
                    if (b0 < kSmBins)
                        atomicAdd(&H.first[0][b0], 1u);
                    if (b1 < kSmBins)
                        atomicAdd(&H.first[0][b1], 1u);
                }
            }
        };
        if (whole)
            pass(std::true_type{});
        else
            pass(std::false_type{});
        uint32_t none = 0;
        sm_block_sum<NT>(S, total, none);
        int use = sm_exchange(S, turn, C, rank, total, 0);
        total = 0;
        for (uint32_t k = 0; k < C; ++k)
            total += S.cmass[use][k];
        auto tau = [&](unsigned long long base) {
            const double x = ceil(static_cast<double>(P.top_p) * static_cast<double>(base));
            return static_cast<unsigned long long>(x < 1.0 ? 1.0 : x);
        };
        // this thread's bins over the cluster
        constexpr int N = kSmBins / NT;
        uint32_t cnt[N], cnt_all;
        unsigned long long mass[N], mass_all;
        sm_counts(H, C, cnt);
        // bins b0 .. b1 that the cut may lie in; `deep`: it lies below the bins
        const unsigned long long ktarget = static_cast<unsigned long long>(P.top_k);
        uint32_t b0 = 0, b1 = kSmBins - 1, down_to_b1;
        bool deep = false;
        unsigned long long kleft = 0; // of top-k, in its bin
        uint32_t kties = 0;
        if (use_k) {
            sm_scan<false, NT>(H, cnt, mass, ktarget, cnt_all, mass_all);
            deep = H.bin < 0;
            if (!deep) {
                b1 = static_cast<uint32_t>(H.bin);
                kleft = ktarget - H.bcnt_before;
                kties = H.bcnt_at;
            }
            down_to_b1 = deep ? cnt_all : H.bcnt_before + H.bcnt_at;
        } else {
            // the running mass through a bin lies between its count's at the bins' edges (a
            // fiftieth of a bin further, for the roundings of a bin's number)
            const unsigned long long target = tau(total);
#pragma unroll
            for (int i = 0; i < N; ++i)
                mass[i] = cnt[i] * R.mass(fminf(mx, mx - (N * threadIdx.x + i - 0.52f) * P.width));
            sm_scan<true, NT>(H, cnt, mass, target, cnt_all, mass_all);
            b0 = H.bin >= 0 ? static_cast<uint32_t>(H.bin) : kSmBins;
#pragma unroll
            for (int i = 0; i < N; ++i)
                mass[i] = cnt[i] * R.mass(mx - (N * threadIdx.x + i + 0.52f) * P.width);
            sm_scan<true, NT>(H, cnt, mass, target, cnt_all, mass_all);
            deep = H.bin < 0;
            if (!deep)
                b1 = static_cast<uint32_t>(H.bin);
            down_to_b1 = deep ? cnt_all : H.bcnt_before + H.bcnt_at;
        }
        SampleSet<LT, NT> Set = {X, R, P.bins, b1, nullptr, 0};
        if (!deep && down_to_b1 <= kSmFew) {
            // 3. few ids: the row is settled at once, by every CTA
            Set.each([&](uint32_t bits, int32_t id, uint32_t) {
                const uint32_t at = atomicAdd(&H.nfew[0], 1u);
                if (at < kSmFew) // (the count bounds it)
                    H.few[0][at] = make_uint2(E::key(bits), static_cast<uint32_t>(id));
            });
            const uint32_t m = sm_collect<LT>(R, 0, C, H);
            const uint2 me = threadIdx.x < m ? H.all[threadIdx.x] : make_uint2(0u, 0u);
            uint32_t before = 0;
            unsigned long long through = 0;
            if (threadIdx.x < m) {
                sm_rank(H, m, me, before, through);
                through += H.mass[threadIdx.x];
            }
            // the last of the top-k set, the last of top-p's, the last that min-p keeps
            const bool in_k = threadIdx.x < m && (!use_k || before < static_cast<uint32_t>(P.top_k));
            if (use_k && threadIdx.x < m && before + 1 == min(static_cast<uint32_t>(P.top_k), m))
                H.upto = through;
            __syncthreads();
            const unsigned long long target = use_p ? tau(use_k ? H.upto : total) : ~0ull;
            const unsigned long long own = threadIdx.x < m ? H.mass[threadIdx.x] : 0ull;
            const bool in = in_k && (!use_p || through - own < target) && E::value(E::bits_of_key(me.x)) >= zlo;
            if (threadIdx.x < m)
                H.mass[threadIdx.x] = in ? own : 0ull;
            if (threadIdx.x == 0) {
                H.cut = {ktop, -1};
                H.bin = -1;
            }
            const uint32_t kept = static_cast<uint32_t>(__syncthreads_count(in));
            if (in && before + 1 == kept) // (the kept are the first of the order)
                H.cut = {me.x, static_cast<int32_t>(me.y)};
            unsigned long long Z = 0, upto = 0;
            if (threadIdx.x < m)
#pragma unroll 4
                for (uint32_t i = 0; i < m; ++i) {
                    const unsigned long long w = H.mass[i];
                    Z += w;
                    upto += H.all[i].y <= me.y ? w : 0ull;
                }
            if (threadIdx.x == 0)
                H.upto = Z;
            __syncthreads();
            Z = H.upto;
            cut = H.cut;
            if (rank == 0) {
                const unsigned long long t = static_cast<unsigned long long>(mul_floor(u, static_cast<long long>(Z)));
                if (threadIdx.x == 0 && P.kept)
                    P.kept[r] = static_cast<int32_t>(kept);
                if (in && !bad_u && t < upto && t >= upto - own) {
                    P.tokens[r] = static_cast<int32_t>(me.y);
                    if (P.prob)
                        P.prob[r] = static_cast<float>(static_cast<double>(own) / static_cast<double>(Z));
                }
            }
            sm_write_q<LT, NT, true>(X, R, P, qrow, zlo, cut, Z);
            sm_cluster_leave();
            return;
        }
        // the list
        if (X.mem && P.slice <= 65536) {
            for (int32_t v = threadIdx.x; v < X.nv; v += NT) {
                const uint4 w = X.vec(v);
                if (sm_bin(R, sm_largest<LT>(w), P.bins) > b1)
                    continue;
                uint32_t h = 0;
#pragma unroll
                for (int j = 0; j < PV; ++j)
                    h |= sm_bin(R, E::value(Slice::of(w, j)), P.bins) <= b1 ? 1u << j : 0u;
                uint32_t at = atomicAdd(&H.nlist, static_cast<uint32_t>(__popc(h)));
                for (; h; h &= h - 1, ++at)
                    if (at < static_cast<uint32_t>(P.cap))
                        H.list[at] = static_cast<uint16_t>(v * PV + __ffs(h) - 1);
            }
            __syncthreads();
            if (H.nlist <= static_cast<uint32_t>(P.cap)) {
                Set.list = H.list;
                Set.n = H.nlist;
            }
        }
        // (clusters of a large batch work at the same time, and one CTA's work leaves the
        // SMs to them: 190 -> 154 us for 256 rows of 128256; 8 rows are settled sooner by all
        // CTAs together, 31 against 38 us)
        if (NT == 256 && Set.list && !deep && down_to_b1 <= kSmOne) {
            if (threadIdx.x == 0) {
                uint32_t base;
                asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
                             : "=r"(base)
                             : "r"(sm_peer(&H.nent, 0)), "r"(Set.n)
                             : "memory");
                H.base = base;
            }
            __syncthreads();
            const uint32_t base = H.base, to = sm_peer(&H.ent[0], 0);
            for (uint32_t i = threadIdx.x; i < Set.n; i += NT)
                asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(to + (base + i) * 8u), "r"(E::key(Set.bits(i))),
                             "r"(static_cast<uint32_t>(Set.id(i)))
                             : "memory");
            sm_cluster_sync();
            if (rank == 0) {
                unsigned long long Z = 0;
                SampleCutAt found;
                const bool done = sm_settle_row<LT, NT>(P, R, S, H, down_to_b1, b0, b1, kties, kleft, total, zlo, u, r, found, Z);
                __syncthreads();
                if (threadIdx.x < C) {
                    sm_put(&H.rcut.key, threadIdx.x, found.key);
                    sm_put(&H.rcut.id, threadIdx.x, static_cast<uint32_t>(found.id));
                    sm_put(&H.rmass, threadIdx.x, Z);
                    sm_put(&H.settled, threadIdx.x, done ? 1u : 0u);
                }
                if (threadIdx.x == 0)
                    H.nfew[0] = 0u;
            }
            sm_cluster_sync();
            if (H.settled) {
                sm_write_q<LT, NT, true>(X, R, P, qrow, zlo, H.rcut, H.rmass);
                sm_cluster_leave();
                return;
            }
        }
        // the cut of a target inside a bin of `ties` ids
        auto resolve = [&](auto by_mass, uint32_t bin, uint32_t ties, unsigned long long above, unsigned long long left, int few) {
            constexpr bool MASS = decltype(by_mass)::value;
            if (ties <= kSmFew)
                return sm_gather<LT, NT, MASS>(Set, bin, above, left, cut, few, C, H);
            const uint32_t klo = sm_first_key<LT>(R, P.bins, bin, ktop);
            const uint32_t khi = bin ? sm_first_key<LT>(R, P.bins, bin - 1, ktop) - 1 : ktop;
            return sm_narrow<LT, NT, MASS>(X, R, klo, khi, above, left, P.piece, C, rank, H);
        };
        // ... or below the bins
        auto resolve_below = [&](auto by_mass, unsigned long long above, unsigned long long left) {
            constexpr bool MASS = decltype(by_mass)::value;
            const uint32_t khi = sm_first_key<LT>(R, P.bins, kSmBins - 1, ktop) - 1;
            if (khi < E::kKeyMin) {
                SampleFound f = {};
                f.upto = above;
                return f;
            }
            return sm_narrow<LT, NT, MASS>(X, R, E::kKeyMin, khi, above, left, P.piece, C, rank, H);
        };
        SampleFound f = {};
        if (use_k) {
            f = deep ? resolve_below(std::false_type{}, 0, ktarget - cnt_all)
                     : resolve(std::false_type{}, b1, kties, 0, kleft, 0);
            cut = sm_settle<LT>(X, f, v0, v1, H);
        }
        if (use_p) {
            // masses: above those bins in one sum, in them by bin
            sm_cluster_sync(); // the bins have been read by every CTA
            sm_clear<NT>(H);
            unsigned long long above = 0;
            Set.each([&](uint32_t bits, int32_t id, uint32_t b) {
                const uint32_t key = E::key(bits);
                if (key < cut.key || (key == cut.key && id > cut.id))
                    return;
                const unsigned long long e = R.mass(E::value(bits));
                if (b < b0) {
                    above += e;
                } else {
                    sm_add_mass(H, b, e, P.piece);
                }
            });
            sm_block_sum<NT>(S, above, none);
            use = sm_exchange(S, turn, C, rank, above, 0);
            above = 0;
            for (uint32_t k = 0; k < C; ++k)
                above += S.cmass[use][k];
            sm_counts(H, C, cnt);
            sm_masses(H, C, P.piece, mass);
            if (use_k) { // the top-k set's
                sm_scan<true, NT>(H, cnt, mass, 1, cnt_all, mass_all);
                total = mass_all + (deep ? f.upto : 0);
            }
            const unsigned long long target = tau(total);
            const unsigned long long left = target > above ? target - above : 1;
            sm_scan<true, NT>(H, cnt, mass, left, cnt_all, mass_all);
            if (H.bin >= 0) {
                const unsigned long long before = H.bmass_before;
                const uint32_t bin = static_cast<uint32_t>(H.bin), ties = H.bcnt_at;
                f = resolve(std::true_type{}, bin, ties, above + before, left - before, 1);
            } else {
                f = resolve_below(std::true_type{}, above + mass_all, left - mass_all);
                deep = true;
            }
            cut = sm_settle<LT>(X, f, v0, v1, H);
        }
        list = Set.list;
        nlist = Set.n;
        if (deep) // (it may reach below what is listed)
            list = nullptr;
    }
    // 4. the kept masses.  An id is kept from `least` on (min-p, and below the cut's
    // value nothing is); of a vector that has none nothing else is looked at.
    const bool filtered = CUTS || P.min_p;
    float least = zlo;
    if (cut.key)
        least = fmaxf(least, E::value(E::bits_of_key(cut.key)));
    auto keeps = [&](uint32_t bits, int32_t id) {
        return E::finite(bits) && E::value(bits) >= least && (!CUTS || E::key(bits) != cut.key || id <= cut.id);
    };
    // the kept mass of vector v, and how many ids
    auto vec_mass = [&](int32_t v, uint32_t &n) {
        const uint4 w = X.vec(v);
        unsigned long long a = 0;
        if (!filtered) {
#pragma unroll
            for (int j = 0; j < PV; j += 2) {
                unsigned long long e0, e1;
                R.masses(E::value(Slice::of(w, j)), E::value(Slice::of(w, j + 1)), e0, e1);
                a += e0 + e1;
            }
            n += PV;
            if (sm_smallest<LT>(w) == -INFINITY)
#pragma unroll 1
                for (int j = 0; j < PV; ++j)
                    n -= E::finite(Slice::of(w, j)) ? 0u : 1u;
        } else if (sm_largest<LT>(w) >= least) {
#pragma unroll 1
            for (int j = 0; j < PV; ++j) {
                const uint32_t b = Slice::of(w, j);
                if (keeps(b, X.first + v * PV + j)) {
                    ++n;
                    a += R.mass(E::value(b));
                }
            }
        }
        return a;
    };
    const SampleSet<LT, NT> Kept = {X, R, 0.0f, 0u, list, nlist};
    auto entry_mass = [&](uint32_t i, uint32_t &n) {
        const uint32_t b = Kept.bits(i);
        if (!keeps(b, Kept.id(i)))
            return 0ull;
        ++n;
        return R.mass(E::value(b));
    };
    unsigned long long a = 0;
    uint32_t n = 0;
    if (list) {
        for (uint32_t i = threadIdx.x; i < nlist; i += NT)
            a += entry_mass(i, n);
    } else {
        for (int32_t v = v0 + lane; v < v1; v += 32)
            a += vec_mass(v, n);
    }
    sm_block_sum<NT>(S, a, n);
    const int use = sm_exchange(S, turn, C, rank, a, n);
    uint32_t kept = 0;
    unsigned long long Z = 0, below = 0;
    for (uint32_t k = 0; k < C; ++k) {
        if (k == rank)
            below = Z;
        Z += S.cmass[use][k];
        kept += S.ccnt[use][k];
    }
    if (rank == 0 && threadIdx.x == 0 && P.kept)
        P.kept[r] = static_cast<int32_t>(kept);
    const unsigned long long t = static_cast<unsigned long long>(mul_floor(u, static_cast<long long>(Z)));
    if (!bad_u && t >= below && t < below + a) { // this CTA's: the first id whose running mass exceeds t
        // vectors i0 .. i1 - 1 hold it, `at` the mass before them
        unsigned long long at = below;
        int32_t i0 = v0, i1 = v1;
        bool here;
        if (CUTS && list) { // the listed masses by runs of vectors, of which there are at most as many as bins
            if constexpr (CUTS) {
                constexpr int N = kSmBins / NT;
                const int32_t run = (X.nv + kSmBins - 1) / kSmBins;
                SampleBins &H = *reinterpret_cast<SampleBins *>(sm_raw + (P.staged ? static_cast<size_t>(P.slice) * sizeof(LT) : 0));
                // (no other CTA reads the bins any more: each has arrived at the barrier above)
                sm_clear<NT>(H);
                for (uint32_t i = threadIdx.x; i < nlist; i += NT) {
                    uint32_t no = 0;
                    const unsigned long long e = entry_mass(i, no);
                    if (e)
                        sm_add_mass(H, (list[i] / PV) / run, e, P.piece);
                }
                __syncthreads();
                uint32_t cnt[N], no;
                unsigned long long mass[N], none;
                sm_counts_here(H, cnt);
                sm_masses_here(H, P.piece, mass);
                sm_scan<true, NT>(H, cnt, mass, t - below + 1, no, none);
                i0 = H.bin * run;
                i1 = min(X.nv, i0 + run);
                at += H.bmass_before;
            }
            here = warp == 0;
        } else { // by warps' parts
            int w = 0;
            for (; w < NT / 32 - 1; ++w) {
                if (t < at + S.wmass[w])
                    break;
                at += S.wmass[w];
            }
            here = warp == w;
        }
        if (here) {
            for (int32_t i = i0; i < i1; i += 32) {
                uint32_t no = 0;
                const unsigned long long e = i + lane < i1 ? vec_mass(i + lane, no) : 0ull;
                const unsigned long long run =
                    at + static_cast<unsigned long long>(warp_incl_scan_ll(static_cast<long long>(e), lane));
                const uint32_t b = __ballot_sync(0xFFFFFFFFu, t < run);
                if (b) {
                    if (lane == __ffs(b) - 1) { // inside this lane's vector
                        unsigned long long to = run - e;
                        const uint4 x = X.vec(i + lane);
#pragma unroll 1
                        for (int j = 0; j < PV; ++j) {
                            const uint32_t bits = Slice::of(x, j);
                            const int32_t id = X.first + (i + lane) * PV + j;
                            const unsigned long long one = keeps(bits, id) ? R.mass(E::value(bits)) : 0ull;
                            to += one;
                            if (t < to) {
                                P.tokens[r] = id;
                                if (P.prob)
                                    P.prob[r] = static_cast<float>(static_cast<double>(one) / static_cast<double>(Z));
                                break;
                            }
                        }
                    }
                    break;
                }
                at = __shfl_sync(0xFFFFFFFFu, run, 31);
            }
        }
    }
    // 5. q
    sm_write_q<LT, NT, CUTS>(X, R, P, qrow, zlo, cut, Z);
    sm_cluster_leave();
}

} // namespace sv
