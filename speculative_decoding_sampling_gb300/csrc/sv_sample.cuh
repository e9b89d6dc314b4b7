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
// each value: with t = (z - max) 32 log2(e) / T and k = round(t), r = t - k (t from
// a factor in two parts; fp32 logits give their difference in two parts too),
//   e^((z - max) / T) = 2^(k / 32) (1 + x + x^2/2 + x^3/6),  x = r ln(2) / 32,
// |x| <= 0.0109, the series' rest below 2^-30; 2^(j / 32) comes from a table of 32
// whose entries lie in 32 different banks.  (exp2 in fp32 alone gives 2^-22: among
// 10^5 ids a draw then falls on a neighbour once in some hundred rows.)
//
// A cluster of C CTAs (1, 2, 4 or 8) takes a row, each a slice of its ids, read
// once from memory into shared memory (rows too long for eight stay in L2).
//  1. load, maximum;
//  2. the mass of the whole row, where it is asked for (top-p without top-k, or
//     no filter at all);
//  3. with a filter: the ids above a window below the maximum are listed (id order
//     within a warp's part); a window that does not hold the cut is widened, up to
//     the whole row, which needs no list;
//  4. the cut, digit by digit of the order key (512 bins a digit, counts and masses
//     of the listed ids; one digit for a bf16 window of up to 512 values), and
//     among equal keys the j-th id;
//  5. the kept masses by warp and CTA, the draw inside the warp that holds it;
//  6. q.
// CTAs exchange through distributed shared memory, one cluster barrier a step.
#pragma once

#include "sv_filter.cuh"

namespace sv {

constexpr int kSmThreads = 512;
constexpr int kSmWarps = kSmThreads / 32;
constexpr int kSmBins = 512;
constexpr int kSmMaxCtas = 8;

struct SampleParams {
    const void *in;      // [rows, V]
    int64_t rows;
    int32_t V;
    const float *u;      // [rows]
    float c_hi, c_lo;    // 32 log2(e) / T
    float cq;            // log2(e) / T
    float dmin;          // differences below this have no mass: -48 T ln 2
    float window;        // first window below the maximum, > 0: 10 T ln 2
    double min_off;      // T ln(min_p) (min_p > 0)
    int32_t top_k;       // <= 0: off
    float top_p;         // >= 1: off
    int32_t min_p;       // whether min_off counts
    int32_t C;           // CTAs of a cluster
    int32_t slice;       // ids of a CTA, a multiple of 16 bytes of them
    int32_t staged;      // the slices fit in shared memory
    int32_t cap;         // list entries of a warp (0: no lists)
    int32_t fix;         // fractional bits of the masses (at most 45, sums of a row below 2^62)
    int32_t piece;       // bits of a mass that a bin adds up in one 32-bit word
    int32_t vec_q;       // q's vectors lie as the logits' do
    int32_t *tokens;     // [rows]
    float *prob;         // [rows] or nullptr
    int32_t *kept;       // [rows] or nullptr
    float *probs;        // [rows, V] or nullptr
    int32_t *status;     // or nullptr
};

struct SampleShared {
    float2 tab[32];                                  // 2^(j / 32) 2^27: as fp32, and as an integer less the shift's bits
    float cmax[kSmMaxCtas];
    int cbad[kSmMaxCtas];
    unsigned long long cmass[4][kSmMaxCtas];         // exchanged sums, a row of slots for each use
    uint32_t ccnt[4][kSmMaxCtas];
    uint32_t hist[2][4][kSmBins];                    // counts, masses in three pieces; two, alternating
    unsigned long long wmass[kSmWarps];
    uint32_t wcnt[kSmWarps];
    unsigned long long smass[kSmWarps];              // scan of the bins
    uint32_t scnt[kSmWarps];
    uint32_t nlist[kSmWarps];
    float wmax[kSmWarps];
    int bad;
    uint32_t over;
    // the bin that holds the target
    int bin;
    unsigned long long bmass_before, bmass_at;
    uint32_t bcnt_before, bcnt_at;
    int32_t nth;
};

__device__ __forceinline__ uint32_t sm_peer(const void *p, uint32_t rank)
{
    uint32_t d;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_addr(p)), "r"(rank));
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
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(sm_peer(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void sm_cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

constexpr uint32_t kSmFull = 1u << 22; // a full list's count: above every row's

constexpr float kSmShift = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number
constexpr uint32_t kSmShiftBits = 0x4B400000u;

// What a row's masses are formed with.
struct SampleRow {
    float m, c_hi, c_lo, dmin;
    uint32_t tab; // shared-memory address of the table
    int up;       // fix - 27
    // the mass of logit z <= m, in 2^-fix of the maximum's, rounded; 0 for -inf
    template <bool F32> __device__ __forceinline__ unsigned long long mass(float z) const
    {
        float d = z - m, dl = 0.0f;
        if (F32) { // what the difference lost (Knuth's two-sum)
            const float bb = d - z;
            dl = (z - (d - bb)) + (-m - bb);
        }
        const bool in = d > dmin;
        d = in ? d : 0.0f;
        const float t = __fmaf_rn(d, c_hi, kSmShift);
        const float k = t - kSmShift;
        float r = __fmaf_rn(d, c_hi, -k);
        r = __fmaf_rn(d, c_lo, r);
        if (F32)
            r = __fmaf_rn(dl, c_hi, r);
        const float x = __fmul_rn(r, 0.021660849392498290f); // ln(2) / 32
        const float p = __fmaf_rn(__fmul_rn(x, x), __fmaf_rn(x, 0.16666667f, 0.5f), x);
        const int kb = static_cast<int>(__float_as_uint(t) - kSmShiftBits); // k, at most 0
        float2 e;
        asm("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(e.x), "=f"(e.y) : "r"(tab + ((static_cast<uint32_t>(kb) & 31u) << 3)));
        const int down = -(kb >> 5);
        uint32_t half; // half a unit of the result, where bits are lost (a shift by a negative number gives 0)
        asm("shl.b32 %0, 1, %1;" : "=r"(half) : "r"(down - up - 1));
        const uint32_t E = __float_as_uint(e.y) + __float_as_uint(__fmaf_rn(e.x, p, kSmShift)) + half;
        const unsigned long long w = (static_cast<unsigned long long>(E) << up) >> down;
        return in ? w : 0ull;
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

// A cut: ids with a larger key, and of those with this key the ones up to `id`.
struct SampleCut {
    uint32_t key;
    int32_t id;
    __device__ __forceinline__ bool keeps(uint32_t k, int32_t i) const { return k > key || (k == key && i <= id); }
};

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
    __device__ __forceinline__ uint32_t bits(int32_t p) const
    {
        if (!mem) {
            const int32_t i = first + p;
            return i >= lo && i < hi ? filter_bits<LT>(row, i) : E::kNegInf;
        }
        if constexpr (PV == 8)
            return reinterpret_cast<const unsigned short *>(mem)[p];
        else
            return reinterpret_cast<const uint32_t *>(mem)[p];
    }
    __device__ __forceinline__ static uint32_t of(const uint4 &w, int j)
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        if constexpr (PV == 8)
            return j & 1 ? u[j >> 1] >> 16 : u[j >> 1] & 0xFFFFu;
        else
            return u[j];
    }
};

// The listed ids of a warp's part, or (no list) all of it: f(in, id, bits) is
// called by whole warps, in ascending order of ids over the lanes of a call.
struct SampleList {
    const uint16_t *pos; // this warp's entries, or nullptr
    uint32_t n;
};

template <typename LT, typename F>
__device__ __forceinline__ void sm_each(const SampleSlice<LT> &X, const SampleList &L, int32_t v0, int32_t v1, F &&f)
{
    constexpr int PV = SampleSlice<LT>::PV;
    const int lane = threadIdx.x & 31;
    if (L.pos) {
        for (uint32_t i = 0; i < L.n; i += 32) {
            const bool in = i + lane < L.n;
            const int32_t p = in ? L.pos[i + lane] : 0;
            f(in, X.first + p, in ? X.bits(p) : FilterElem<LT>::kNegInf);
        }
    } else {
        for (int32_t p = v0 * PV; p < v1 * PV; p += 32) {
            const bool in = p + lane < v1 * PV;
            f(in, X.first + p + lane, in ? X.bits(p + lane) : FilterElem<LT>::kNegInf);
        }
    }
}

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
__device__ __forceinline__ void sm_block_sum(SampleShared &S, unsigned long long &mass, uint32_t &cnt)
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
    for (int w = 0; w < kSmWarps; ++w) {
        mass += S.wmass[w];
        cnt += S.wcnt[w];
    }
}

// The cut where the running count (MASS false) or mass of the members reaches
// `target`, from the largest key down; members: listed ids with keys in
// [klo, khi] that `bound` keeps.  upto gets the mass through the cut.
template <typename LT, bool MASS>
__device__ SampleCut sm_select(const SampleSlice<LT> &X, const SampleList &L, int32_t v0, int32_t v1, const SampleRow &R,
                               uint32_t klo, uint32_t khi, bool bounded, SampleCut bound, unsigned long long target,
                               unsigned long long &upto, int piece, int &buf, uint32_t C, uint32_t rank, SampleShared &S)
{
    using E = FilterElem<LT>;
    constexpr bool F32 = sizeof(LT) == 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    static_assert(kSmThreads == kSmBins, "a thread for each bin");
    const uint32_t low = (1u << piece) - 1u;
    unsigned long long above = 0;
    for (;;) {
        const uint32_t span = khi - klo;
        const int sh = span < kSmBins ? 0 : 32 - __clz(span) - 9;
        uint32_t(&H)[4][kSmBins] = S.hist[buf];
        buf ^= 1;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            H[k][threadIdx.x] = 0u;
        __syncthreads();
        sm_each<LT>(X, L, v0, v1, [&](bool in, int32_t id, uint32_t bits) {
            const uint32_t k = E::key(bits);
            if (!in || !E::finite(bits) || k < klo || k > khi || (bounded && !bound.keeps(k, id)))
                return;
            const uint32_t b = (khi - k) >> sh;
            const unsigned long long w = R.mass<F32>(E::value(bits));
            atomicAdd(&H[0][b], 1u);
            if (w) {
                atomicAdd(&H[1][b], static_cast<uint32_t>(w) & low);
                atomicAdd(&H[2][b], static_cast<uint32_t>(w >> piece) & low);
                atomicAdd(&H[3][b], static_cast<uint32_t>(w >> (2 * piece)));
            }
        });
        sm_cluster_sync();
        // bin threadIdx.x over the cluster
        uint32_t cnt = 0;
        unsigned long long mass = 0;
        for (uint32_t r = 0; r < C; ++r) {
            cnt += sm_get(&H[0][threadIdx.x], r);
            mass += sm_get(&H[1][threadIdx.x], r);
            mass += static_cast<unsigned long long>(sm_get(&H[2][threadIdx.x], r)) << piece;
            mass += static_cast<unsigned long long>(sm_get(&H[3][threadIdx.x], r)) << (2 * piece);
        }
        const unsigned long long mi = static_cast<unsigned long long>(warp_incl_scan_ll(static_cast<long long>(mass), lane));
        uint32_t ci = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, ci, o);
            ci += lane >= o ? n : 0u;
        }
        if (lane == 31) {
            S.smass[warp] = mi;
            S.scnt[warp] = ci;
        }
        if (threadIdx.x == 0)
            S.bin = -1;
        __syncthreads();
        unsigned long long mb = mi - mass;
        uint32_t cb = ci - cnt;
        for (int w = 0; w < warp; ++w) {
            mb += S.smass[w];
            cb += S.scnt[w];
        }
        const unsigned long long before = MASS ? mb : cb, here = MASS ? mass : cnt;
        if (before < target && target <= before + here) {
            S.bin = threadIdx.x;
            S.bcnt_before = cb;
            S.bcnt_at = cnt;
            S.bmass_before = mb;
            S.bmass_at = mass;
        }
        __syncthreads();
        const int bin = S.bin; // the target is at most the members' sum: found
        if (bin < 0)
            return {0u, 0x7FFFFFFF};
        above += S.bmass_before;
        target -= MASS ? S.bmass_before : S.bcnt_before;
        khi -= static_cast<uint32_t>(bin) << sh;
        const uint32_t width = (1u << sh) - 1u;
        klo = khi - klo > width ? khi - width : klo;
        const uint32_t ties = S.bcnt_at;
        if (sh > 0 && klo != khi) {
            __syncthreads();
            continue;
        }
        // one value: the j-th of its ids
        const unsigned long long w = R.mass<F32>(E::value(E::bits_of_key(khi)));
        unsigned long long j = target;
        if (MASS)
            j = w ? (target + w - 1) / w : 1;
        j = j < 1 ? 1 : (j > ties ? ties : j);
        upto = above + j * w;
        SampleCut cut = {khi, 0x7FFFFFFF};
        if (j < ties) { // the same in every CTA
            uint32_t below = 0; // ids of this value in the CTAs before
            for (uint32_t r = 0; r < rank; ++r)
                below += sm_get(&H[0][bin], r);
            const uint32_t mine = sm_get(&H[0][bin], rank);
            if (j <= below) {
                cut.id = -1;
            } else if (j - below < mine) {
                const uint32_t want = static_cast<uint32_t>(j) - below; // of this CTA's
                uint32_t n = 0;
                auto member = [&](bool in, int32_t id, uint32_t bits) {
                    const uint32_t k = E::key(bits);
                    return in && k == khi && E::finite(bits) && (!bounded || bound.keeps(k, id));
                };
                sm_each<LT>(X, L, v0, v1, [&](bool in, int32_t id, uint32_t bits) {
                    n += __popc(__ballot_sync(0xFFFFFFFFu, member(in, id, bits)));
                });
                if (lane == 0)
                    S.scnt[warp] = n;
                __syncthreads();
                uint32_t at = 0;
                for (int w2 = 0; w2 < warp; ++w2)
                    at += S.scnt[w2];
                if (at < want && want <= at + n) {
                    sm_each<LT>(X, L, v0, v1, [&](bool in, int32_t id, uint32_t bits) {
                        const uint32_t b = __ballot_sync(0xFFFFFFFFu, member(in, id, bits));
                        const uint32_t upto_lane = at + __popc(b & ((2u << lane) - 1u));
                        if ((b >> lane & 1u) && upto_lane == want)
                            S.nth = id;
                        at += __popc(b);
                    });
                }
                __syncthreads();
                cut.id = S.nth;
            }
        }
        __syncthreads();
        return cut;
    }
}

template <typename LT>
__global__ void __launch_bounds__(kSmThreads, 2) sample_kernel(const SampleParams P)
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
        constexpr int U = 8;
        for (int32_t v = threadIdx.x; v < X.nv; v += U * kSmThreads) {
            uint4 w[U];
#pragma unroll
            for (int t = 0; t < U; ++t)
                if (v + t * kSmThreads < X.nv)
                    w[t] = X.fetch(v + t * kSmThreads);
#pragma unroll
            for (int t = 0; t < U; ++t)
                if (v + t * kSmThreads < X.nv) {
                    fold(w[t]);
                    if (P.staged)
                        stage[v + t * kSmThreads] = w[t];
                }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(__shfl_xor_sync(0xFFFFFFFFu, mx, o)));
        if (lane == 0)
            S.wmax[warp] = mx;
        __syncthreads();
        mx = S.wmax[0];
#pragma unroll
        for (int w = 1; w < kSmWarps; ++w)
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
            for (int32_t i = X.lo + threadIdx.x; i < X.hi; i += kSmThreads)
                qrow[i] = 0.0f;
        sm_cluster_sync(); // no CTA leaves while another may write to it
        return;
    }
    SampleRow R = {mx, P.c_hi, P.c_lo, P.dmin, smem_addr(S.tab), P.fix - 27};
    // min-p: the least logit kept (p >= min_p max p, in logits)
    const float zlo = P.min_p ? __double2float_ru(static_cast<double>(mx) + P.min_off) : -INFINITY;
    const bool use_k = P.top_k > 0 && P.top_k < P.V, use_p = P.top_p < 1.0f;
    // a warp's part of the slice
    const int32_t part = (X.nv + kSmWarps - 1) / kSmWarps;
    const int32_t v0 = min(X.nv, warp * part), v1 = min(X.nv, v0 + part);

    SampleList list = {nullptr, 0};
    SampleCut cut = {0u, 0x7FFFFFFF}; // everything finite
    unsigned long long total = 0;
    int buf = 0, turn = 0;
    // 2. the whole row's mass
    auto row_sums = [&](unsigned long long &mass, uint32_t &cnt) {
        mass = 0;
        cnt = 0;
        for (int32_t v = v0 + lane; v < v1; v += 32) {
            const uint4 w = X.vec(v);
#pragma unroll
            for (int j = 0; j < PV; ++j) {
                const uint32_t b = Slice::of(w, j);
                cnt += E::finite(b) ? 1u : 0u;
                mass += R.mass<F32>(E::value(b));
            }
        }
        sm_block_sum(S, mass, cnt);
        const int use = sm_exchange(S, turn, C, rank, mass, cnt);
        mass = 0;
        cnt = 0;
        for (uint32_t k = 0; k < C; ++k) {
            mass += S.cmass[use][k];
            cnt += S.ccnt[use][k];
        }
    };
    uint32_t finite = 0;
    if (use_p && !use_k)
        row_sums(total, finite);
    auto mass_target = [&](unsigned long long base) {
        const double tau = ceil(static_cast<double>(P.top_p) * static_cast<double>(base));
        return static_cast<unsigned long long>(tau < 1.0 ? 1.0 : tau);
    };
    const bool filtered = use_k || use_p || P.min_p;
    if (filtered) {
        // 3. the ids of a window
        uint16_t *const mine = reinterpret_cast<uint16_t *>(sm_raw + (P.staged ? static_cast<size_t>(P.slice) * sizeof(LT) : 0)) +
                               static_cast<size_t>(warp) * P.cap;
        bool whole = P.cap == 0;
        float win = P.window, zc = -INFINITY;
        while (!whole) {
            zc = use_k || use_p ? mx - win : zlo;
            uint32_t n = 0;
            for (int32_t v = v0; v < v1; v += 32) {
                uint32_t hit = 0;
                if (v + lane < v1) {
                    const uint4 w = X.vec(v + lane);
#pragma unroll
                    for (int j = 0; j < PV; ++j)
                        hit |= E::value(Slice::of(w, j)) >= zc ? 1u << j : 0u;
                }
                if (__any_sync(0xFFFFFFFFu, hit)) {
                    const uint32_t own = __popc(hit);
                    uint32_t at = own;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, at, o);
                        at += lane >= o ? up : 0u;
                    }
                    const uint32_t sum = __shfl_sync(0xFFFFFFFFu, at, 31);
                    at += n - own;
                    for (uint32_t h = hit; h; h &= h - 1) {
                        if (at < static_cast<uint32_t>(P.cap))
                            mine[at] = static_cast<uint16_t>((v + lane) * PV + __ffs(h) - 1);
                        ++at;
                    }
                    n += sum;
                }
            }
            __syncwarp();
            const bool full = n > static_cast<uint32_t>(P.cap);
            list.pos = mine;
            list.n = n;
            unsigned long long have = 0;
            if (use_p && !use_k && !full)
                sm_each<LT>(X, list, v0, v1, [&](bool in, int32_t, uint32_t bits) {
                    have += in ? R.mass<F32>(E::value(bits)) : 0ull;
                });
            uint32_t count = lane == 0 ? (full ? kSmFull : n) : 0u; // (a cluster's 128 of them add up in 32 bits)
            sm_block_sum(S, have, count);
            const int use = sm_exchange(S, turn, C, rank, have, count);
            have = 0;
            count = 0;
            for (uint32_t k = 0; k < C; ++k) {
                have += S.cmass[use][k];
                count += S.ccnt[use][k];
            }
            whole = count >= kSmFull; // some list is full
            if (whole || (use_k ? count >= static_cast<uint32_t>(P.top_k) : !use_p || have >= mass_target(total)))
                break;
            win *= 2.0f;
            whole = !(win < -P.dmin); // (what has no mass may still count for top-k)
        }
        if (whole) {
            list.pos = nullptr;
            zc = -INFINITY;
        }
        // 4. the cuts
        if (use_k || use_p) {
            const uint32_t ktop = E::key(F32 ? __float_as_uint(mx) : __float_as_uint(mx) >> 16);
            uint32_t klow = E::kKeyMin;
            if (!whole) { // the key of zc, rounded down to the logits' type
                uint32_t b = __float_as_uint(zc);
                if (!F32)
                    b = (b >> 31 ? b + 0xFFFFu : b) >> 16;
                klow = max(E::key(b), E::kKeyMin);
            }
            bool have_cut = false;
            if (use_k) {
                bool cuts = true;
                if (whole) {
                    row_sums(total, finite);
                    cuts = finite > static_cast<uint32_t>(P.top_k);
                }
                if (cuts) {
                    cut = sm_select<LT, false>(X, list, v0, v1, R, klow, ktop, false, cut,
                                               static_cast<unsigned long long>(P.top_k), total, P.piece, buf,
                                               C, rank, S);
                    have_cut = true;
                }
            }
            if (use_p) { // of the top-k set's mass, or the row's
                unsigned long long upto = 0;
                cut = sm_select<LT, true>(X, list, v0, v1, R, klow, ktop, have_cut, cut, mass_target(total), upto,
                                          P.piece, buf, C, rank, S);
            }
        }
    }
    // 5. the kept masses
    auto keeps = [&](uint32_t bits, int32_t id) {
        return E::finite(bits) && E::value(bits) >= zlo && cut.keeps(E::key(bits), id);
    };
    unsigned long long a = 0;
    uint32_t n = 0;
    if (filtered) {
        sm_each<LT>(X, list, v0, v1, [&](bool in, int32_t id, uint32_t bits) {
            const bool k = in && keeps(bits, id);
            n += k ? 1u : 0u;
            a += k ? R.mass<F32>(E::value(bits)) : 0ull;
        });
    } else {
        for (int32_t v = v0 + lane; v < v1; v += 32) {
            const uint4 w = X.vec(v);
#pragma unroll
            for (int j = 0; j < PV; ++j) {
                const uint32_t b = Slice::of(w, j);
                n += E::finite(b) ? 1u : 0u;
                a += R.mass<F32>(E::value(b));
            }
        }
    }
    sm_block_sum(S, a, n);
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
        unsigned long long at = below;
        int w = 0;
        for (; w < kSmWarps - 1; ++w) {
            if (t < at + S.wmass[w])
                break;
            at += S.wmass[w];
        }
        if (warp == w) {
            bool done = false;
            sm_each<LT>(X, list, v0, v1, [&](bool in, int32_t id, uint32_t bits) {
                if (done)
                    return;
                const bool k = in && keeps(bits, id);
                const unsigned long long e = k ? R.mass<F32>(E::value(bits)) : 0ull;
                const unsigned long long run =
                    at + static_cast<unsigned long long>(warp_incl_scan_ll(static_cast<long long>(e), lane));
                const uint32_t b = __ballot_sync(0xFFFFFFFFu, t < run);
                if (b) {
                    if (lane == __ffs(b) - 1) {
                        P.tokens[r] = id;
                        if (P.prob)
                            P.prob[r] = static_cast<float>(static_cast<double>(e) / static_cast<double>(Z));
                    }
                    done = true;
                }
                at = __shfl_sync(0xFFFFFFFFu, run, 31);
            });
        }
    }
    // 6. q
    if (qrow) {
        const float scale = ldexpf(1.0f, P.fix) / static_cast<float>(Z);
        const float cq = P.cq;
        auto q_of = [&](uint32_t bits, int32_t id) {
            return keeps(bits, id) ? ex2(__fmul_rn(E::value(bits) - mx, cq)) * scale : 0.0f;
        };
        for (int32_t v = threadIdx.x; v < X.nv; v += kSmThreads) {
            const uint4 w = X.vec(v);
            const int32_t i = X.first + v * PV;
            float q[PV];
#pragma unroll
            for (int j = 0; j < PV; ++j)
                q[j] = q_of(Slice::of(w, j), i + j);
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
    sm_cluster_sync(); // no CTA leaves while another may read it
}

} // namespace sv
