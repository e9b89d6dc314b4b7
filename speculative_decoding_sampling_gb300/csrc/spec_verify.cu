// spec_verify.cu -- C ABI of the verification library: argument checks,
// workspace layout, and the launches on the caller's stream -- the row
// pass, the draw stream and, when the draw stream does not fill the GPU,
// the final draws -- each chained to the one before by programmatic
// dependent launch; the top-k / top-p filter; the target's last layer (norms,
// quantisation, LM head); and the draft's step (4-bit quantisation and LM head,
// the draw of tokens).  The operations themselves are documented in
// spec_verify.h.
#include "spec_verify.h"

#include <cmath>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <mutex>

#include "sv_block_norm.cuh"
#include "sv_filter.cuh"
#include "sv_final.cuh"
#include "sv_fp4.cuh"
#include "sv_lmhead.cuh"
#include "sv_lmhead_fp4.cuh"
#include "sv_lmhead_fp4_plan.h"
#include "sv_lmhead_fp8.cuh"
#include "sv_sample.cuh"
#include "sv_tree.cuh"
#include "sv_rows.cuh"

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

int ceil_log2_u64(uint64_t v)
{
    int n = 0;
    while ((uint64_t{1} << n) < v)
        ++n;
    return n;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How the work of one call is cut and where its scratch lives: a function of
// (B, K, V) only.
struct Plan {
    int64_t R;    // rows B*(K+1)
    int32_t PM;   // row_part slots per row
    int32_t CPS;  // final-draw chunks per sequence
    int32_t fix;  // fractional bits of the fixed-point masses
    size_t off_part, off_row_side, off_seq_info, off_seqE, off_cnt, off_rec_a, off_rec_q, bytes;
};

bool make_plan(int64_t B, int32_t K, int32_t V, Plan &p)
{
    if (B < 0 || K < 0 || V < 1 || V > SV_MAX_V)
        return false;
    if (B > 0 && static_cast<int64_t>(K) + 1 > INT64_MAX / B)
        return false;
    p.R = B * (static_cast<int64_t>(K) + 1);
    if (p.R > 0 && V > INT64_MAX / p.R)
        return false;
    // row_part slots per row: enough for any cut of the flat row array into
    // at most kRowMaxCtas spans (the launch widens spans to keep to it)
    p.PM = static_cast<int32_t>(p.R > 0 ? ceil_div(sv::kRowMaxCtas, p.R) + 3 : 4);
    p.CPS = static_cast<int32_t>(ceil_div(V, static_cast<int64_t>(sv::kChunkGroups) * sv::kGroup));
    const int fb = 62 - ceil_log2_u64(static_cast<uint64_t>(V) + 1);
    p.fix = fb < 40 ? fb : 40;
    const size_t Bz = static_cast<size_t>(B), R = static_cast<size_t>(p.R);
    size_t off = 0;
    p.off_part = off;     off = align_up(off + R * p.PM * sizeof(float2));
    p.off_row_side = off; off = align_up(off + R * sizeof(float4));
    p.off_seq_info = off; off = align_up(off + Bz * sizeof(int4));
    p.off_seqE = off;     off = align_up(off + Bz * sizeof(long long));
    p.off_cnt = off;      off = align_up(off + Bz * sizeof(uint32_t));
    p.off_rec_a = off;    off = align_up(off + Bz * p.CPS * sizeof(long long));
    p.off_rec_q = off;    off = align_up(off + Bz * p.CPS * sizeof(float));
    p.bytes = off;
    return true;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

enum Stage { kRows = 1, kSurvivors = 2, kBoth = 3 };

constexpr uint64_t kWaitLimitNs = 1000000000ull; // every bounded wait of a kernel gives up after 1 s

constexpr int kMaxDevices = 64;

// The current context's process-unique id, or 0 when none can be had (no
// context current yet, or a driver without the query).  The driver calls
// are reached through the runtime's entry-point lookup, so the library does
// not link the driver library itself.
unsigned long long current_context_id()
{
    using GetCurrent = CUresult (*)(CUcontext *);
    using GetId = CUresult (*)(CUcontext, unsigned long long *);
    static GetCurrent get_current = nullptr;
    static GetId get_id = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f, 4000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<GetCurrent>(f);
        f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<GetId>(f);
        (void)cudaGetLastError();
    });
    if (!get_current || !get_id)
        return 0;
    CUcontext ctx = nullptr;
    unsigned long long id = 0;
    if (get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr || get_id(ctx, &id) != CUDA_SUCCESS)
        return 0;
    return id;
}

// Per device and kernel instantiation: how many CTAs of each kernel fit on
// the device at once (the grids of the persistent kernels).  Cached per
// device for the context the figures were taken in: a context created anew
// (after cudaDeviceReset, or a caller's own context) has forgotten the draw
// kernel's shared-memory attribute, so the figures are taken again there.
struct Resident {
    int rows, draw;
    unsigned long long ctx; // context id the entry was made in (0: none)
};

template <typename LT, bool DENSE>
cudaError_t resident_ctas(Resident &out)
{
    static std::mutex mu;
    static Resident cache[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    const unsigned long long ctx = current_context_id();
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev].rows == 0 || cache[dev].ctx == 0 || cache[dev].ctx != ctx) {
        int sms = 0, rows = 0, draw = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess)
            return e;
        e = cudaFuncSetAttribute(sv::survivor_kernel<LT, DENSE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 sv::DrawShape<LT, DENSE>::kCtaBytes);
        if (e != cudaSuccess)
            return e;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&rows, sv::rows_kernel<LT, DENSE>, sv::kRowCtaThreads, 0);
        if (e != cudaSuccess)
            return e;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&draw, sv::survivor_kernel<LT, DENSE>,
                                                          sv::kDrawWarps * 32, sv::DrawShape<LT, DENSE>::kCtaBytes);
        if (e != cudaSuccess)
            return e;
        sms = sms > 0 ? sms : 1;
        cache[dev].rows = (rows > 0 ? rows : 1) * sms;
        cache[dev].draw = (draw > 0 ? draw : 1) * sms;
        cache[dev].ctx = current_context_id(); // taken after the calls above made the context current
    }
    out = cache[dev];
    return cudaSuccess;
}

int64_t clamp_grid(int64_t want, int64_t cap) { return want < 1 ? 1 : (want > cap ? cap : want); }

// CTAs of the draw stream: at least one chunk per warp, at most one wave
int64_t draw_grid(int64_t NC, const Resident &res) { return clamp_grid(ceil_div(NC, sv::kDrawWarps), res.draw); }

// A stream that fills every SM, with at least as many draw warps as
// sequences: each sequence has its own warps, and the last of them makes its
// final draw (no final kernel, whose CTAs would only be placed once the
// stream's CTAs leave).  A smaller stream leaves SMs free, where the final
// kernel's CTAs wait for it and draw with block-wide scans, sooner than one
// warp can.
bool inline_final(int64_t grid, int64_t B, const Resident &res)
{
    return grid == res.draw && grid * sv::kDrawWarps >= B;
}

// Kernels one whole call launches on the current device: the row pass, the
// draw stream and, unless the stream makes the final draws, the final kernel.
template <typename LT, bool DENSE>
cudaError_t launches_per_call(int64_t B, const Plan &plan, int32_t &n)
{
    Resident res;
    const cudaError_t e = resident_ctas<LT, DENSE>(res);
    if (e != cudaSuccess)
        return e;
    const int64_t grid = draw_grid(B * static_cast<int64_t>(plan.CPS), res);
    n = inline_final(grid, B, res) ? 2 : 3;
    return cudaSuccess;
}

template <typename LT, bool DENSE>
cudaError_t launch(sv::Params &P, const Plan &plan, int stages, cudaStream_t stream)
{
    if (stages == 0)
        return cudaSuccess;
    Resident res;
    cudaError_t e = resident_ctas<LT, DENSE>(res);
    if (e != cudaSuccess)
        return e;
    // the flat view of the logits and its cut into one span per CTA
    constexpr int64_t VW = 16 / sizeof(LT);
    P.total = plan.R * P.V;
    P.h = static_cast<int64_t>((16 - reinterpret_cast<uintptr_t>(P.logits) % 16) % 16) / static_cast<int64_t>(sizeof(LT));
    if (P.h > P.total)
        P.h = P.total;
    P.nvec = (P.total - P.h) / VW;
    P.NV = P.nvec + 2;
    {
        int64_t want = clamp_grid(ceil_div(P.NV, sv::kRowMinSpan), res.rows < sv::kRowMaxCtas ? res.rows : sv::kRowMaxCtas);
        if (want < ceil_div(P.NV, sv::kRowMaxSpan))
            want = ceil_div(P.NV, sv::kRowMaxSpan); // offsets inside a span stay in int
        int64_t span = ceil_div(P.NV, want);
        // a row touches at most `touch` vectors; spans of at least
        // touch / (PM - 2) vectors put it in at most PM - 1 CTAs
        const int64_t touch = ceil_div(P.V, VW) + 2;
        const int64_t span_min = ceil_div(touch, plan.PM - 2);
        P.span = span > span_min ? span : span_min;
    }
    if (stages & kRows) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(P.NV, P.span)));
        cfg.blockDim = dim3(sv::kRowCtaThreads);
        cfg.stream = stream;
        e = cudaLaunchKernelEx(&cfg, sv::rows_kernel<LT, DENSE>, P);
        if (e != cudaSuccess)
            return e;
    }
    if (stages & kSurvivors) {
        const int64_t grid = draw_grid(P.NC, res);
        P.inline_final = inline_final(grid, P.B, res) ? 1 : 0;
        // programmatic dependent launch: the draw's CTAs may be scheduled
        // while the row pass drains; they wait in griddepcontrol.wait for
        // its completion before reading anything it wrote
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.blockDim = dim3(sv::kDrawWarps * 32);
        cfg.dynamicSmemBytes = sv::DrawShape<LT, DENSE>::kCtaBytes;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, sv::survivor_kernel<LT, DENSE>, P);
        if (e != cudaSuccess)
            return e;
        if (P.inline_final)
            return cudaSuccess;
        // the final draws: one CTA per sequence, chained the same way
        cudaLaunchConfig_t fcfg = {};
        fcfg.gridDim = dim3(static_cast<unsigned>(P.B < 0x7FFFFFFF ? P.B : 0x7FFFFFFF));
        fcfg.blockDim = dim3(sv::kFinalThreads);
        fcfg.dynamicSmemBytes = static_cast<size_t>(plan.CPS) * (sizeof(long long) + sizeof(float));
        fcfg.stream = stream;
        fcfg.attrs = attr;
        fcfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&fcfg, sv::final_kernel<LT, DENSE>, P);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

sv_status_t run(int stages, const void *logits, sv_dtype_t dtype, const float *q, const int32_t *tokens,
                const float *u, float T, int64_t B, int32_t K, int32_t V, int32_t *out_tokens,
                int32_t *num_emitted, int8_t *accept_flags, float *accept_prob, float *residual_mass,
                int32_t *status_dev, void *workspace, size_t workspace_bytes, void *stream,
                unsigned long long *stats = nullptr, int one_part = 0)
{
    if (B < 0 || K < 0 || V < 1)
        return SV_EINVAL;
    if (V > SV_MAX_V)
        return SV_EUNSUPPORTED;
    if (dtype != SV_BF16 && dtype != SV_FP32)
        return SV_EINVAL;
    if (!std::isfinite(T) || !(T > 0.0f))
        return SV_EINVAL;
    const double c64 = 1.4426950408889634074 / static_cast<double>(T);
    const float c = static_cast<float>(c64);
    if (!std::isfinite(c) || !(c > 0.0f))
        return SV_EINVAL;
    if (!logits || !u || !out_tokens || !num_emitted || (K > 0 && !tokens) || !workspace)
        return SV_EINVAL;
    const size_t esize = dtype == SV_BF16 ? 2 : 4;
    if (!aligned(logits, esize) || (q && !aligned(q, 4)) || (tokens && !aligned(tokens, 4)) ||
        !aligned(u, 4) || !aligned(out_tokens, 4) || !aligned(num_emitted, 4) ||
        (accept_prob && !aligned(accept_prob, 4)) || (residual_mass && !aligned(residual_mass, 4)) ||
        (status_dev && !aligned(status_dev, 4)) || (stats && !aligned(stats, 8)) || !aligned(workspace, kAlign))
        return SV_EINVAL;
    Plan plan;
    if (!make_plan(B, K, V, plan))
        return SV_EUNSUPPORTED;
    if (workspace_bytes < plan.bytes)
        return SV_EINVAL;
    if (B == 0)
        return SV_OK;

    char *ws = static_cast<char *>(workspace);
    sv::Params P;
    P.logits = logits;
    P.q = K > 0 ? q : nullptr;
    P.tokens = tokens;
    P.u = u;
    P.c = c;
    P.B = B;
    P.K = K;
    P.V = V;
    P.out_tokens = out_tokens;
    P.num_emitted = num_emitted;
    P.accept_flags = accept_flags;
    P.accept_prob = accept_prob;
    P.residual_mass = residual_mass;
    P.status = status_dev;
    P.stats = stats;
    P.row_part = reinterpret_cast<float2 *>(ws + plan.off_part);
    P.row_side = reinterpret_cast<float4 *>(ws + plan.off_row_side);
    P.seq_info = reinterpret_cast<int4 *>(ws + plan.off_seq_info);
    P.seq_E = reinterpret_cast<long long *>(ws + plan.off_seqE);
    P.seq_cnt = reinterpret_cast<uint32_t *>(ws + plan.off_cnt);
    P.inline_final = 0;
    P.rec_a = reinterpret_cast<long long *>(ws + plan.off_rec_a);
    P.rec_q = reinterpret_cast<float *>(ws + plan.off_rec_q);
    P.PM = plan.PM;
    P.CPS = plan.CPS;
    P.NC = B * static_cast<int64_t>(plan.CPS);
    P.ring_ok = (V % sv::kGroup) == 0 && aligned(logits, 16) && (P.q == nullptr || aligned(P.q, 16)) ? 1 : 0;
    P.fix_bits = plan.fix;
    P.one_part = one_part;
    P.total = P.h = P.nvec = P.NV = P.span = 0;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    const bool dense = P.q != nullptr;
    if (dtype == SV_BF16)
        e = dense ? launch<uint16_t, true>(P, plan, stages, s) : launch<uint16_t, false>(P, plan, stages, s);
    else
        e = dense ? launch<float, true>(P, plan, stages, s) : launch<float, false>(P, plan, stages, s);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}

// ---------------------------------------------------------------- LM head

constexpr int64_t kLmMaxRows = int64_t{1} << 30;

int32_t lm_tiles(int32_t V) { return static_cast<int32_t>(ceil_div(V, sv::kLmBN)); }

size_t lm_part_bytes(int64_t M, int32_t V) { return align_up(static_cast<size_t>(M) * lm_tiles(V) * sizeof(float2)); }

// A 2-D tensor map of a row-major matrix [rows, cols] (bf16, or e4m3 bytes)
// with boxes of box_rows x 128 bytes in the 128-byte swizzle layout, or of
// box_rows x box_cols = 32 bf16 in the 64-byte one; out-of-range elements
// read as zero and are not written.  Reached through the runtime's
// entry-point lookup.
bool lm_tensor_map_of(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t rows, int64_t cols,
                      int64_t pitch, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle)
{
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static Encode encode = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            encode = reinterpret_cast<Encode>(f);
        (void)cudaGetLastError();
    });
    if (!encode)
        return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
    const cuuint32_t box[2] = {box_cols, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return encode(map, type, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool lm_tensor_map(CUtensorMap *map, const void *base, int64_t rows, int32_t cols, uint32_t box_rows,
                   bool fp8 = false, uint32_t box_cols = 0)
{
    return lm_tensor_map_of(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, rows, cols,
                            static_cast<int64_t>(cols) * (fp8 ? 1 : 2),
                            box_cols ? box_cols : static_cast<uint32_t>(fp8 ? sv::kL8BK : sv::kLmBK), box_rows,
                            box_cols ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

sv_status_t lm_check(const void *hidden, const void *lm_head, int64_t M, int32_t d, int32_t V, const void *logits)
{
    if (M < 0 || d < 8 || d % 8 != 0 || V < 1)
        return SV_EINVAL;
    if (V > SV_MAX_V || M > kLmMaxRows)
        return SV_EUNSUPPORTED;
    if (M > 0 && (!hidden || !lm_head || !logits || !aligned(hidden, 16) || !aligned(lm_head, 16) ||
                  !aligned(logits, 2)))
        return SV_EINVAL;
    return SV_OK;
}

// How many clusters of two LM-head CTAs fit on the current device at once
// (the persistent grid, in pairs); cached per device for the context it was
// taken in, like the verification kernels' figures.
cudaError_t lm_pairs(int &pairs)
{
    struct Entry {
        int pairs;
        unsigned long long ctx;
    };
    static std::mutex mu;
    static Entry cache[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    const unsigned long long ctx = current_context_id();
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev].pairs == 0 || cache[dev].ctx == 0 || cache[dev].ctx != ctx) {
        e = cudaFuncSetAttribute(sv::lm_head_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sv::kLmSmem);
        if (e != cudaSuccess)
            return e;
        int sms = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess)
            return e;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(sms > 1 ? sms & ~1 : 2));
        cfg.blockDim = dim3(sv::kLmThreads);
        cfg.dynamicSmemBytes = sv::kLmSmem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, sv::lm_head_kernel, &cfg);
        if (e != cudaSuccess)
            return e;
        if (n < 1)
            return cudaErrorInvalidConfiguration;
        cache[dev].pairs = n;
        cache[dev].ctx = current_context_id();
    }
    pairs = cache[dev].pairs;
    return cudaSuccess;
}

// logits = h W^T (bf16 out) and, with `part`, the per-tile row statistics.
cudaError_t lm_launch(const void *hidden, const void *lm_head, int64_t M, int32_t d, int32_t V, void *logits,
                      float2 *part, float c, int32_t *status, cudaStream_t stream)
{
    CUtensorMap ta, tb;
    if (!lm_tensor_map(&ta, hidden, M, d, sv::kLmBM) || !lm_tensor_map(&tb, lm_head, V, d, sv::kLmBN / 2))
        return cudaErrorInvalidValue;
    int pairs = 0;
    cudaError_t e = lm_pairs(pairs);
    if (e != cudaSuccess)
        return e;
    sv::LmParams L;
    L.M = static_cast<int32_t>(M);
    L.N = V;
    L.Kd = d;
    L.MT = static_cast<int32_t>(ceil_div(M, 2 * sv::kLmBM));
    L.logits = static_cast<uint16_t *>(logits);
    L.part = part;
    L.NT = lm_tiles(V);
    L.c = c;
    L.vec = (V % 8 == 0 && aligned(logits, 16)) ? 1 : 0;
    L.status = status;
    L.wait_ns = kWaitLimitNs;
    // persistent: as many pairs of SMs as hold a cluster at once (the ring
    // takes most of the shared memory: one CTA per SM)
    const int64_t tiles = static_cast<int64_t>(L.MT) * L.NT;
    const int64_t np = tiles < pairs ? tiles : pairs;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * np));
    cfg.blockDim = dim3(sv::kLmThreads);
    cfg.dynamicSmemBytes = sv::kLmSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sv::lm_head_kernel, ta, tb, L);
}

// ------------------------------------------------------- LM head on e4m3

constexpr int kNominalSms = 152; // GB300

// How the product is cut: a function of (M, V) only, so that the workspace is.
struct Lm8Plan {
    bool pair;
    int32_t MT, NT, NB, halves;
};

Lm8Plan lm8_plan(int64_t M, int32_t V)
{
    // Row tiles of 128 by CTAs alone or of 256 by pairs, and ids per tile: the
    // cut for which the waves of tiles cost least.  A step of a tile (128
    // hidden dims) costs at least the accumulator warps' chain of about 640
    // cycles, whatever its width, or the time its weights take from memory when
    // every step brings new ones (one row tile: 128 bytes an id at 23 bytes a
    // cycle and SM).  Lone CTAs over several row tiles load each weight tile
    // twice as often as pairs do; the rule takes a wave of theirs as 1.17 times a
    // pair's (measured 1.06 to 1.22 at d 2048 and 4096), so they are taken where a
    // pair would leave enough of its rows or of its last wave empty:
    //   M 384, V 128256, d 4096: 10 waves 179 us, pairs 14 waves 205 us;
    //   M 257, V 50000, d 2048: 4 waves 40 us, pairs 6 waves 52 us;
    //   M 2304, V 151936, d 4096: 71 waves 1072 us, pairs 71 waves 1010 us;
    //   M 896, V 151936, d 4096: 28 waves 439 us, pairs 32 waves 457 us (taken).
    // Narrower tiles on ties: they reach more SMs.  A pair's tiles are 64, 128
    // or 256 wide (two whole halves, each in boxes of one size).
    Lm8Plan p = {};
    int64_t best = INT64_MAX;
    for (int pair = M > sv::kLmBM ? 1 : 0; pair >= 0; --pair) {
        const int64_t rows = pair ? 2 * sv::kLmBM : sv::kLmBM, units = pair ? kNominalSms / 2 : kNominalSms;
        const int32_t mt = static_cast<int32_t>(ceil_div(M > 0 ? M : 1, rows));
        const int64_t chain = pair || mt == 1 ? 640 : 755;
        const int64_t per_id = pair ? 11 : 22; // quarter cycles an id
        int64_t low = INT64_MAX;
        int32_t NB = sv::kL8MaxNB;
        for (int32_t nb = sv::kL8MaxNB; nb >= (pair ? 64 : 32); nb = pair ? nb / 2 : nb - 32) {
            const int64_t bytes = mt == 1 ? per_id * nb / 4 : 0;
            const int64_t cost = ceil_div(mt * ceil_div(V, nb), units) * ((bytes > chain ? bytes : chain) + 40);
            if (cost <= low) {
                low = cost;
                NB = nb;
            }
        }
        if (low < best) { // a pair on ties
            best = low;
            p.pair = pair != 0;
            p.MT = mt;
            p.NB = NB;
        }
    }
    p.NT = static_cast<int32_t>(ceil_div(V, p.NB));
    p.halves = p.NB > 128 ? 2 : 1;
    return p;
}

size_t lm8_part_bytes(int64_t M, int32_t V)
{
    return align_up(static_cast<size_t>(M) * lm8_plan(M, V).NT * sizeof(float2));
}

sv_status_t lm8_check(const void *hidden, const float *hidden_scales, const void *lm_head, const float *lm_head_scales,
                      int64_t M, int32_t d, int32_t V, const void *logits)
{
    if (M < 0 || d < 16 || d % 16 != 0 || V < 1)
        return SV_EINVAL;
    if (V > SV_MAX_V || M > kLmMaxRows)
        return SV_EUNSUPPORTED;
    const Lm8Plan p = lm8_plan(M, V); // tiles, and steps of all tiles, are counted in 32 bits
    const int64_t tiles = static_cast<int64_t>(p.MT) * p.NT;
    if (tiles > INT32_MAX || tiles > INT32_MAX / ceil_div(d, sv::kL8BK) * (kNominalSms / 2))
        return SV_EUNSUPPORTED;
    if (M > 0 && (!hidden || !hidden_scales || !lm_head || !lm_head_scales || !logits || !aligned(hidden, 16) ||
                  !aligned(lm_head, 16) || !aligned(hidden_scales, 4) || !aligned(lm_head_scales, 4) ||
                  !aligned(logits, 2)))
        return SV_EINVAL;
    return SV_OK;
}

// How many CTAs (or clusters of two) of the e4m3 kernel fit on the current
// device at once; cached like the bf16 kernel's figure.
template <bool PAIR> cudaError_t lm8_units(int &units)
{
    struct Entry {
        int units;
        unsigned long long ctx;
    };
    static std::mutex mu;
    static Entry cache[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    const unsigned long long ctx = current_context_id();
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev].units == 0 || cache[dev].ctx == 0 || cache[dev].ctx != ctx) {
        constexpr int smem = sv::kL8Smem;
        e = cudaFuncSetAttribute(sv::lm_head_fp8_kernel<PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return e;
        int sms = 0, n = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess)
            return e;
        if (PAIR) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(sms > 1 ? sms & ~1 : 2));
            cfg.blockDim = dim3(sv::kL8Threads);
            cfg.dynamicSmemBytes = smem;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, sv::lm_head_fp8_kernel<PAIR>, &cfg);
        } else {
            n = sms;
        }
        if (e != cudaSuccess)
            return e;
        if (n < 1)
            return cudaErrorInvalidConfiguration;
        cache[dev].units = n;
        cache[dev].ctx = current_context_id();
    }
    units = cache[dev].units;
    return cudaSuccess;
}

template <bool PAIR>
cudaError_t lm8_launch_as(const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &tc, const sv::Lm8Params &L,
                          cudaStream_t stream)
{
    int units = 0;
    const cudaError_t e = lm8_units<PAIR>(units);
    if (e != cudaSuccess)
        return e;
    const int64_t tiles = static_cast<int64_t>(L.MT) * L.NT; // below 2^31 (lm8_check)
    const int64_t n = tiles < units ? tiles : units;
    cudaLaunchAttribute attr[2];
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (PAIR ? 2 : 1);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n * (PAIR ? 2 : 1)));
    cfg.blockDim = dim3(sv::kL8Threads);
    cfg.dynamicSmemBytes = sv::kL8Smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sv::lm_head_fp8_kernel<PAIR>, ta, tb, tc, L);
}

// logits (bf16 out) and, with `part`, the row statistics of each tile.
cudaError_t lm8_launch(const void *hidden, const float *hidden_scales, const void *lm_head, const float *lm_head_scales,
                       int64_t M, int32_t d, int32_t V, void *logits, float2 *part, float c, int32_t *status,
                       cudaStream_t stream)
{
    const Lm8Plan p = lm8_plan(M, V);
    const int32_t brows = p.pair ? p.NB / 2 : p.NB; // ids of a tile that one CTA loads
    sv::Lm8Params L;
    // A stage holds the rows of h that exist, in 32s: the MMA's 128 rows then
    // run on into the stage's ids, and the sums of those rows are not read.
    // (Only where that leaves 128 rows in the stage.)
    L.a_rows = static_cast<int32_t>(M < sv::kLmBM ? ceil_div(M, 32) * 32 : sv::kLmBM);
    if (L.a_rows + brows < sv::kLmBM)
        L.a_rows = sv::kLmBM;
    L.stage_bytes = (L.a_rows + brows) * sv::kL8BK;
    L.stages = sv::kL8RingBytes / L.stage_bytes;
    if (L.stages > sv::kL8MaxStages)
        L.stages = sv::kL8MaxStages;
    CUtensorMap ta, tb, tc = {};
    if (!lm_tensor_map(&ta, hidden, M, d, static_cast<uint32_t>(L.a_rows), true) ||
        !lm_tensor_map(&tb, lm_head, V, d, static_cast<uint32_t>(p.pair && p.halves == 2 ? brows / 2 : brows), true))
        return cudaErrorInvalidValue;
    L.M = static_cast<int32_t>(M);
    L.N = V;
    L.KB = static_cast<int32_t>(ceil_div(d, sv::kL8BK));
    L.mt_inv = p.MT > 1 ? UINT64_MAX / static_cast<uint64_t>(p.MT) + 1 : 0;
    L.MT = p.MT;
    L.NT = p.NT;
    L.NB = p.NB;
    const int mma_rows = p.pair ? 2 * sv::kLmBM : sv::kLmBM;
    L.idesc[0] = sv::l8_idesc(mma_rows, p.NB < 128 ? p.NB : 128);
    L.idesc[1] = sv::l8_idesc(mma_rows, p.NB - 128); // read only when NB > 128
    L.hs = hidden_scales;
    L.ws = lm_head_scales;
    L.logits = static_cast<uint16_t *>(logits);
    L.part = part;
    L.halves = p.halves;
    L.c = c;
    L.tma = (V % 8 == 0 && aligned(logits, 16)) ? 1 : 0;
    if (L.tma && !lm_tensor_map(&tc, logits, M, V, 32, false, 32))
        return cudaErrorInvalidValue;
    L.status = status;
    return p.pair ? lm8_launch_as<true>(ta, tb, tc, L, stream) : lm8_launch_as<false>(ta, tb, tc, L, stream);
}

// The statistics of the product's tiles merged per row with the draft data,
// then the draw stream and the final draws.
sv_status_t lm_finish(const Plan &plan, float2 *part, int32_t slots, const void *logits, const float *draft_probs,
                      const int32_t *draft_tokens, const float *uniforms, float temperature, int64_t B, int32_t K,
                      int32_t V, int32_t *out_tokens, int32_t *num_emitted, int8_t *accept_flags, float *accept_prob,
                      float *residual_mass, int32_t *status_dev, void *workspace, void *stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    sv::Params P = {};
    P.logits = logits;
    P.q = K > 0 ? draft_probs : nullptr;
    P.tokens = draft_tokens;
    P.u = uniforms;
    P.c = static_cast<float>(1.4426950408889634074 / static_cast<double>(temperature));
    P.B = B;
    P.K = K;
    P.V = V;
    P.row_part = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + plan.off_part);
    P.row_side = reinterpret_cast<float4 *>(static_cast<char *>(workspace) + plan.off_row_side);
    P.PM = plan.PM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(plan.R, 8)));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = P.q ? cudaLaunchKernelEx(&cfg, sv::lm_merge_kernel<true>, P, part, slots)
                              : cudaLaunchKernelEx(&cfg, sv::lm_merge_kernel<false>, P, part, slots);
    if (e != cudaSuccess)
        return SV_ECUDA;
    return run(kSurvivors, logits, SV_BF16, draft_probs, draft_tokens, uniforms, temperature, B, K, V, out_tokens,
               num_emitted, accept_flags, accept_prob, residual_mass, status_dev, workspace, plan.bytes, stream,
               nullptr, 1);
}

// ------------------------------------------------- norms and quantisation

constexpr int64_t kNormManyRows = 4 * kNominalSms;

// A launch as programmatic dependent of the kernel before on the stream.
template <typename Kernel, typename Args>
cudaError_t launch_behind(Kernel kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t s, const Args &args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

size_t elem_size(sv_dtype_t t) { return t == SV_BF16 ? 2 : (t == SV_FP32 ? 4 : 1); }

bool is_bf16_or_fp32(sv_dtype_t t) { return t == SV_BF16 || t == SV_FP32; }

// 16-byte accesses of 8 consecutive values, where the pointer may be NULL
bool vec_ok(const void *p, sv_dtype_t t) { return aligned(p, t == SV_E4M3 ? 8 : 16); }

// dynamic shared memory a CTA of sample_kernel may have, beside its own structures
constexpr size_t kSampleSmem = 227 * 1024 - sizeof(sv::SampleShared) - 1024;

// ------------------------------------------------------- 4-bit operands

// A row's steps and a matrix's rows of tiles are counted in 32 bits.
constexpr int64_t kFp4MaxRows = INT32_MAX - 127;
constexpr int32_t kFp4MaxD = INT32_MAX - 1024;

// Scale tiles (128 rows x 4 blocks) along d.
int32_t fp4_tiles(int32_t d, int32_t block) { return static_cast<int32_t>(ceil_div(d, 4 * static_cast<int64_t>(block))); }

// A matrix's scale tiles, 512 bytes each, `box` of them a copy.
bool lm4_scale_map(CUtensorMap *map, const void *base, int64_t tiles, uint32_t box)
{
    return lm_tensor_map_of(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, base, tiles, 128, 512, 128, box,
                            CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <bool PAIR, int H, int BLOCK> cudaError_t lm4_units(int &units)
{
    struct Entry {
        int units;
        unsigned long long ctx;
    };
    static std::mutex mu;
    static Entry cache[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    const unsigned long long ctx = current_context_id();
    std::lock_guard<std::mutex> lock(mu);
    if (cache[dev].units == 0 || cache[dev].ctx == 0 || cache[dev].ctx != ctx) {
        const auto kernel = sv::lm_head_fp4_kernel<PAIR, H, BLOCK>;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sv::kL4Smem);
        if (e != cudaSuccess)
            return e;
        int sms = 0, n = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess)
            return e;
        n = sms;
        if (PAIR) {
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(sms > 1 ? sms & ~1 : 2));
            cfg.blockDim = dim3(sv::kL4Threads);
            cfg.dynamicSmemBytes = sv::kL4Smem;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            if (e != cudaSuccess)
                return e;
        }
        if (n < 1)
            return cudaErrorInvalidConfiguration;
        cache[dev].units = n;
        cache[dev].ctx = current_context_id();
    }
    units = cache[dev].units;
    return cudaSuccess;
}

template <bool PAIR, int H, int BLOCK>
cudaError_t lm4_launch_as(const CUtensorMap (&m)[5], const sv::Lm4Params &L, cudaStream_t stream)
{
    int units = 0;
    const cudaError_t e = lm4_units<PAIR, H, BLOCK>(units);
    if (e != cudaSuccess)
        return e;
    const int64_t tiles = static_cast<int64_t>(L.t.MT) * L.t.NT; // below 2^31 (sv_lm_head_logits_fp4)
    const int64_t n = tiles < units ? tiles : units;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PAIR ? 2 : 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n * (PAIR ? 2 : 1)));
    cfg.blockDim = dim3(sv::kL4Threads);
    cfg.dynamicSmemBytes = sv::kL4Smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sv::lm_head_fp4_kernel<PAIR, H, BLOCK>, m[0], m[1], m[2], m[3], m[4], L);
}

template <int BLOCK>
cudaError_t lm4_launch_shape(const sv::Lm4Plan &p, const CUtensorMap (&m)[5], const sv::Lm4Params &L, cudaStream_t stream)
{
    if (!p.pair)
        return lm4_launch_as<false, 1, BLOCK>(m, L, stream);
    return p.H == 2 ? lm4_launch_as<true, 2, BLOCK>(m, L, stream) : lm4_launch_as<true, 1, BLOCK>(m, L, stream);
}

cudaError_t lm4_launch(const void *hidden, const void *hidden_scales, const float *gh, const void *lm_head,
                       const void *lm_head_scales, const float *gw, int32_t block, int64_t M, int32_t d, int32_t V,
                       void *logits, int32_t *status, cudaStream_t stream)
{
    const sv::Lm4Plan p = sv::lm4_plan(M, V, kNominalSms);
    sv::Lm4Params L = {};
    const int32_t brows = p.pair ? p.NB / 2 : p.NB; // ids of a tile that one CTA loads
    // A stage holds the rows of h that exist, in 8s (a swizzle group): the MMA's
    // 128 rows then run on into what lies behind, and those sums are not read.
    L.t.a_rows = static_cast<int32_t>(M < sv::kLmBM ? ceil_div(M, 8) * 8 : sv::kLmBM);
    L.KT = fp4_tiles(d, block);
    const int32_t per_stage = sv::kL4BK / (4 * block); // scale tiles
    L.blocks = p.NB > 128 ? 2 : 1;
    L.t.stage_bytes = static_cast<int32_t>((p.H * L.t.a_rows + brows) * 128 + per_stage * 512 * (p.H + L.blocks));
    L.t.stage_bytes = (L.t.stage_bytes + 1023) / 1024 * 1024;
    L.t.tma = (V % 8 == 0 && aligned(logits, 16)) ? 1 : 0;
    L.front = sv::l4_front(L.t.tma != 0);
    const int32_t ring = sv::kL4Bytes - L.front;
    L.t.stages = ring / L.t.stage_bytes;
    if (L.t.stages > sv::kL4MaxStages)
        L.t.stages = sv::kL4MaxStages;
    // (the last stage's first rows and what the MMA reads behind them lie in the ring)
    while ((L.t.stages - 1) * L.t.stage_bytes + (p.H - 1) * L.t.a_rows * 128 + sv::kLmBM * 128 > ring)
        --L.t.stages;
    CUtensorMap m[5] = {};
    if (!lm_tensor_map(&m[0], hidden, M, d / 2, static_cast<uint32_t>(L.t.a_rows), true) ||
        !lm_tensor_map(&m[1], lm_head, V, d / 2, static_cast<uint32_t>(brows), true) ||
        !lm4_scale_map(&m[2], hidden_scales, ceil_div(M, 128) * L.KT, static_cast<uint32_t>(per_stage)) ||
        !lm4_scale_map(&m[3], lm_head_scales, ceil_div(V, 128) * L.KT, static_cast<uint32_t>(per_stage)))
        return cudaErrorInvalidValue;
    L.t.M = static_cast<int32_t>(M);
    L.t.N = V;
    L.t.KB = static_cast<int32_t>(ceil_div(d, sv::kL4BK));
    L.t.mt_inv = p.MT > 1 ? UINT64_MAX / static_cast<uint64_t>(p.MT) + 1 : 0;
    L.t.MT = p.MT;
    L.RT = p.RT;
    L.t.NT = p.NT;
    L.t.NB = p.NB;
    L.t.logits = static_cast<uint16_t *>(logits);
    if (L.t.tma && !lm_tensor_map(&m[4], logits, M, V, 32, false, 32))
        return cudaErrorInvalidValue;
    L.t.status = status;
    L.d = d;
    L.idesc = sv::l4_idesc(p.pair ? 2 * sv::kLmBM : sv::kLmBM, p.NB, block);
    L.gh = gh;
    L.gw = gw;
    return block == 16 ? lm4_launch_shape<16>(p, m, L, stream) : lm4_launch_shape<32>(p, m, L, stream);
}

// Warps of a row of `octets` octets: as many as it takes for each lane to keep
// its share in registers, up to 8.
int32_t fp4_warps(int32_t octets)
{
    int32_t w = 1;
    while (w < 8 && octets > w * 32 * sv::kF4Regs)
        w *= 2;
    return w;
}

template <int BLOCK, typename XT>
cudaError_t quantize_fp4_launch(const sv::Fp4Params &P, bool vec, cudaStream_t s)
{
    const int64_t rows = ceil_div(P.Mpad, sv::kF4Threads / 32 / P.WPR);
    const int64_t stay = static_cast<int64_t>(kNominalSms) * sv::kF4Ctas<XT>;
    const unsigned grid = static_cast<unsigned>(rows < stay ? rows : stay);
    return launch_behind(vec ? sv::quantize_fp4_kernel<BLOCK, XT, true> : sv::quantize_fp4_kernel<BLOCK, XT, false>, grid,
                         sv::kF4Threads, 0, s, P);
}

template <int BLOCK, bool F32>
cudaError_t dequantize_fp4_launch(const sv::Fp4BackParams &P, bool vec, cudaStream_t s)
{
    const unsigned grid = static_cast<unsigned>(ceil_div(P.M, sv::kF4Threads / 32 / P.WPR));
    return launch_behind(vec ? sv::dequantize_fp4_kernel<BLOCK, F32, true> : sv::dequantize_fp4_kernel<BLOCK, F32, false>,
                         grid, sv::kF4Threads, 0, s, P);
}

// ------------------------------------------------------- the draw of tokens

template <typename LT, int NT, bool CUTS>
cudaError_t sample_launch_as(const sv::SampleParams &P, size_t smem, cudaStream_t stream)
{
    const auto kernel = sv::sample_kernel<LT, NT, CUTS>;
    if (smem > 40 * 1024) { // (48 KiB without it, the kernel's own structures among them)
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSampleSmem));
        if (e != cudaSuccess)
            return e;
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(P.C);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(P.rows * P.C));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, P);
}

template <typename LT>
cudaError_t sample_launch(const sv::SampleParams &P, int threads, bool cuts, size_t smem, cudaStream_t s)
{
    if (threads == 256)
        return cuts ? sample_launch_as<LT, 256, true>(P, smem, s) : sample_launch_as<LT, 256, false>(P, smem, s);
    return cuts ? sample_launch_as<LT, 512, true>(P, smem, s) : sample_launch_as<LT, 512, false>(P, smem, s);
}

template <bool VEC> cudaError_t norm_launch(const sv::NormParams &P, int nseg, unsigned grid, cudaStream_t s)
{
    const unsigned threads = static_cast<unsigned>(P.WPR * P.RPC * 32);
    switch (nseg) {
    case 1:
        return launch_behind(sv::block_norm_kernel<1, VEC>, grid, threads, 0, s, P);
    case 2:
        return launch_behind(sv::block_norm_kernel<2, VEC>, grid, threads, 0, s, P);
    case 4:
        return launch_behind(sv::block_norm_kernel<4, VEC>, grid, threads, 0, s, P);
    default:
        return launch_behind(sv::block_norm_kernel<8, VEC>, grid, threads, 0, s, P);
    }
}

// The staying CTAs: warps of a row, and the bytes of their rows in flight.
int norm_rows_warps(int32_t d)
{
    int w = 1;
    while (w * sv::kNormCols < d)
        w *= 2;
    return w;
}

size_t norm_rows_smem(int32_t d, size_t x_size, size_t r_size)
{
    return static_cast<size_t>(sv::kNormRing) * norm_rows_warps(d) * sv::kNormCols * (x_size + r_size);
}

// The most that a call may ask for; a multiprocessor has 227 KB, less the
// kernel's own.
constexpr size_t kNormRowsMaxSmem = 224 * 1024;

// How many staying CTAs of `warps` warps are resident at once on the current
// device; cached like lm8_units.  The kernel's limit on shared memory belongs
// to all of its callers, whatever their width and host thread, so it is raised
// once, to the most that any width may ask for, and never lowered: a limit
// fitted to each call's width would make a wider call that another thread is
// just launching fail.
template <bool XF32, bool RF32, bool FULL> cudaError_t norm_rows_resident(int warps, size_t smem, int64_t &ctas)
{
    struct Entry {
        int ctas[sv::kNormMaxWarps + 1]; // by warps of a row
        unsigned long long ctx;
    };
    static std::mutex mu;
    static Entry cache[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    const unsigned long long ctx = current_context_id();
    std::lock_guard<std::mutex> lock(mu);
    Entry &c = cache[dev];
    if (c.ctx == 0 || c.ctx != ctx)
        c = {};
    if (c.ctas[warps] == 0) {
        auto *kernel = sv::block_norm_rows_kernel<XF32, RF32, FULL>;
        int sms = 0, per_sm = 0;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kNormRowsMaxSmem));
        if (e == cudaSuccess)
            e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, warps * 32, smem);
        if (e != cudaSuccess)
            return e;
        if (per_sm < 1)
            return cudaErrorInvalidConfiguration;
        c.ctas[warps] = (sms > 0 ? sms : 1) * per_sm;
        c.ctx = current_context_id();
    }
    ctas = c.ctas[warps];
    return cudaSuccess;
}

template <bool XF32, bool RF32, bool FULL> cudaError_t norm_rows_launch_as(const sv::NormParams &P, cudaStream_t s)
{
    const size_t smem = norm_rows_smem(P.d, XF32 ? 4 : 2, RF32 ? 4 : 2);
    int64_t resident = 0;
    const cudaError_t e = norm_rows_resident<XF32, RF32, FULL>(P.WPR, smem, resident);
    if (e != cudaSuccess)
        return e;
    return launch_behind(sv::block_norm_rows_kernel<XF32, RF32, FULL>,
                         static_cast<unsigned>(P.M < resident ? P.M : resident), static_cast<unsigned>(P.WPR * 32), smem,
                         s, P);
}

template <bool XF32, bool RF32> cudaError_t norm_rows_launch(sv::NormParams P, cudaStream_t s)
{
    P.WPR = norm_rows_warps(P.d);
    return P.WPR * sv::kNormCols == P.d ? norm_rows_launch_as<XF32, RF32, true>(P, s)
                                        : norm_rows_launch_as<XF32, RF32, false>(P, s);
}

static_assert(int(sv::kElemBf16) == int(SV_BF16) && int(sv::kElemFp32) == int(SV_FP32) &&
                  int(sv::kElemE4m3) == int(SV_E4M3),
              "element types");
static_assert(sv::kNormMaxWarps * sv::kNormMaxSegs * sv::kSeg == SV_MAX_D, "widest row of the norms");

static_assert(sv::kTreeMaxNodes == SV_MAX_TREE_NODES, "tree size limit");
static_assert(sv::kBadTree == SV_BAD_TREE, "status bit");

} // namespace

extern "C" {

size_t sv_workspace_bytes(int64_t B, int32_t K, int32_t V)
{
    Plan p;
    if (!make_plan(B, K, V, p))
        return 0;
    return p.bytes;
}

sv_status_t spec_verify(const void *target_logits, sv_dtype_t logits_dtype, const float *draft_probs,
                        const int32_t *draft_tokens, const float *uniforms, float temperature, int64_t B,
                        int32_t K, int32_t V, int32_t *out_tokens, int32_t *num_emitted, int8_t *accept_flags,
                        float *accept_prob, float *residual_mass, int32_t *status_dev, void *workspace,
                        size_t workspace_bytes, void *stream)
{
    return run(kBoth, target_logits, logits_dtype, draft_probs, draft_tokens, uniforms, temperature, B, K, V,
               out_tokens, num_emitted, accept_flags, accept_prob, residual_mass, status_dev, workspace,
               workspace_bytes, stream);
}

sv_status_t spec_verify_stats(const void *target_logits, sv_dtype_t logits_dtype, const float *draft_probs,
                              const int32_t *draft_tokens, const float *uniforms, float temperature, int64_t B,
                              int32_t K, int32_t V, int32_t *out_tokens, int32_t *num_emitted, int8_t *accept_flags,
                              float *accept_prob, float *residual_mass, int32_t *status_dev, void *workspace,
                              size_t workspace_bytes, uint64_t *stats_dev, void *stream)
{
    if (!stats_dev)
        return SV_EINVAL;
    return run(kBoth, target_logits, logits_dtype, draft_probs, draft_tokens, uniforms, temperature, B, K, V,
               out_tokens, num_emitted, accept_flags, accept_prob, residual_mass, status_dev, workspace,
               workspace_bytes, stream, reinterpret_cast<unsigned long long *>(stats_dev));
}

sv_status_t sv_verify_rows(const void *target_logits, sv_dtype_t logits_dtype, const float *draft_probs,
                           const int32_t *draft_tokens, const float *uniforms, float temperature, int64_t B,
                           int32_t K, int32_t V, int32_t *out_tokens, int32_t *num_emitted, int8_t *accept_flags,
                           float *accept_prob, float *residual_mass, int32_t *status_dev, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    return run(kRows, target_logits, logits_dtype, draft_probs, draft_tokens, uniforms, temperature, B, K, V,
               out_tokens, num_emitted, accept_flags, accept_prob, residual_mass, status_dev, workspace,
               workspace_bytes, stream);
}

sv_status_t sv_sample_survivors(const void *target_logits, sv_dtype_t logits_dtype, const float *draft_probs,
                                const int32_t *draft_tokens, const float *uniforms, float temperature, int64_t B,
                                int32_t K, int32_t V, int32_t *out_tokens, int32_t *num_emitted,
                                int8_t *accept_flags, float *accept_prob, float *residual_mass,
                                int32_t *status_dev, void *workspace, size_t workspace_bytes, void *stream)
{
    return run(kSurvivors, target_logits, logits_dtype, draft_probs, draft_tokens, uniforms, temperature, B, K,
               V, out_tokens, num_emitted, accept_flags, accept_prob, residual_mass, status_dev, workspace,
               workspace_bytes, stream);
}

sv_status_t sv_kernel_launches(sv_dtype_t logits_dtype, int32_t dense, int64_t B, int32_t K, int32_t V,
                               int32_t *launches)
{
    if (!launches || B < 0 || K < 0 || V < 1 || (logits_dtype != SV_BF16 && logits_dtype != SV_FP32))
        return SV_EINVAL;
    if (V > SV_MAX_V)
        return SV_EUNSUPPORTED;
    Plan plan;
    if (!make_plan(B, K, V, plan))
        return SV_EUNSUPPORTED;
    if (B == 0) {
        *launches = 0;
        return SV_OK;
    }
    const bool d = dense != 0 && K > 0; // K = 0 has no draft probabilities to read
    int32_t n = 0;
    cudaError_t e;
    if (logits_dtype == SV_BF16)
        e = d ? launches_per_call<uint16_t, true>(B, plan, n) : launches_per_call<uint16_t, false>(B, plan, n);
    else
        e = d ? launches_per_call<float, true>(B, plan, n) : launches_per_call<float, false>(B, plan, n);
    if (e != cudaSuccess)
        return SV_ECUDA;
    *launches = n;
    return SV_OK;
}

sv_status_t sv_filter_logits(const void *logits, sv_dtype_t logits_dtype, int64_t rows, int32_t V,
                             float temperature, int32_t top_k, float top_p, void *out_logits, int32_t *kept,
                             int32_t *status_dev, void *stream)
{
    if (rows < 0 || V < 1 || (logits_dtype != SV_BF16 && logits_dtype != SV_FP32))
        return SV_EINVAL;
    if (V > SV_MAX_V)
        return SV_EUNSUPPORTED;
    if (!std::isfinite(temperature) || !(temperature > 0.0f) || !(top_p > 0.0f))
        return SV_EINVAL;
    const float c = static_cast<float>(1.4426950408889634074 / static_cast<double>(temperature));
    if (!std::isfinite(c) || !(c > 0.0f))
        return SV_EINVAL;
    const size_t esize = logits_dtype == SV_BF16 ? 2 : 4;
    if (rows > 0 && (!logits || !out_logits))
        return SV_EINVAL;
    if (!aligned(logits, esize) || !aligned(out_logits, esize) || (kept && !aligned(kept, 4)) ||
        (status_dev && !aligned(status_dev, 4)))
        return SV_EINVAL;
    if (rows > 0 && static_cast<int64_t>(V) > INT64_MAX / rows)
        return SV_EUNSUPPORTED;
    if (rows == 0)
        return SV_OK;
    sv::FilterParams F;
    F.in = logits;
    F.out = out_logits;
    F.rows = rows;
    F.V = V;
    F.c = c;
    F.top_k = top_k;
    F.top_p = top_p;
    const int fb = 62 - ceil_log2_u64(static_cast<uint64_t>(V) + 1);
    F.fb = fb < 40 ? fb : 40;
    F.yscale = static_cast<float>(sv::kYBins) / static_cast<float>(F.fb + 2);
    F.vec = aligned(logits, 16) && aligned(out_logits, 16) && (static_cast<size_t>(V) * esize) % 16 == 0 ? 1 : 0;
    F.kept = kept;
    F.status = status_dev;
    int dev = 0, sms = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = logits_dtype == SV_BF16
                ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, sv::filter_kernel<uint16_t>,
                                                                sv::kFilterThreads, 0)
                : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, sv::filter_kernel<float>,
                                                                sv::kFilterThreads, 0);
    if (e != cudaSuccess)
        return SV_ECUDA;
    const int64_t resident = static_cast<int64_t>(sms > 0 ? sms : 1) * (per_sm > 0 ? per_sm : 1);
    const int64_t grid = rows < resident ? rows : resident;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (logits_dtype == SV_BF16)
        sv::filter_kernel<uint16_t><<<static_cast<unsigned>(grid), sv::kFilterThreads, 0, s>>>(F);
    else
        sv::filter_kernel<float><<<static_cast<unsigned>(grid), sv::kFilterThreads, 0, s>>>(F);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ECUDA;
}

size_t sv_lm_head_workspace_bytes(int64_t B, int32_t K, int32_t V)
{
    Plan p;
    if (!make_plan(B, K, V, p))
        return 0;
    return p.bytes + lm_part_bytes(B * (static_cast<int64_t>(K) + 1), V);
}

sv_status_t sv_lm_head_logits(const void *hidden, const void *lm_head, int64_t M, int32_t d, int32_t V,
                              void *logits, int32_t *status_dev, void *stream)
{
    const sv_status_t st = lm_check(hidden, lm_head, M, d, V, logits);
    if (st != SV_OK || M == 0)
        return st;
    if (status_dev && !aligned(status_dev, 4))
        return SV_EINVAL;
    return lm_launch(hidden, lm_head, M, d, V, logits, nullptr, 1.0f, status_dev, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? SV_OK
               : SV_ECUDA;
}

sv_status_t spec_verify_lm_head(const void *hidden, const void *lm_head, int32_t d, const float *draft_probs,
                                const int32_t *draft_tokens, const float *uniforms, float temperature, int64_t B,
                                int32_t K, int32_t V, void *logits_out, int32_t *out_tokens, int32_t *num_emitted,
                                int8_t *accept_flags, float *accept_prob, float *residual_mass, int32_t *status_dev,
                                void *workspace, size_t workspace_bytes, void *stream)
{
    if (B < 0 || K < 0)
        return SV_EINVAL;
    if (B > 0 && static_cast<int64_t>(K) + 1 > kLmMaxRows / B)
        return SV_EUNSUPPORTED;
    const int64_t M = B * (static_cast<int64_t>(K) + 1);
    sv_status_t st = lm_check(hidden, lm_head, M, d, V, logits_out);
    if (st != SV_OK)
        return st;
    Plan plan;
    if (!make_plan(B, K, V, plan))
        return SV_EUNSUPPORTED;
    if (!workspace || workspace_bytes < plan.bytes + lm_part_bytes(M, V))
        return SV_EINVAL;
    // host checks of the verification (nothing launched yet)
    st = run(0, logits_out, SV_BF16, draft_probs, draft_tokens, uniforms, temperature, B, K, V, out_tokens,
             num_emitted, accept_flags, accept_prob, residual_mass, status_dev, workspace, plan.bytes, stream);
    if (st != SV_OK || B == 0)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    float2 *part = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + plan.bytes);
    const float c = static_cast<float>(1.4426950408889634074 / static_cast<double>(temperature));
    if (lm_launch(hidden, lm_head, M, d, V, logits_out, part, c, status_dev, s) != cudaSuccess)
        return SV_ECUDA;
    return lm_finish(plan, part, lm_tiles(V), logits_out, draft_probs, draft_tokens, uniforms, temperature, B, K, V,
                     out_tokens, num_emitted, accept_flags, accept_prob, residual_mass, status_dev, workspace, stream);
}

size_t sv_lm_head_fp8_workspace_bytes(int64_t B, int32_t K, int32_t V)
{
    Plan p;
    if (!make_plan(B, K, V, p) || p.R > kLmMaxRows)
        return 0;
    return p.bytes + lm8_part_bytes(p.R, V);
}

sv_status_t sv_lm_head_logits_fp8(const void *hidden, const float *hidden_scales, const void *lm_head,
                                  const float *lm_head_scales, int64_t M, int32_t d, int32_t V, void *logits,
                                  int32_t *status_dev, void *stream)
{
    const sv_status_t st = lm8_check(hidden, hidden_scales, lm_head, lm_head_scales, M, d, V, logits);
    if (st != SV_OK || M == 0)
        return st;
    if (status_dev && !aligned(status_dev, 4))
        return SV_EINVAL;
    return lm8_launch(hidden, hidden_scales, lm_head, lm_head_scales, M, d, V, logits, nullptr, 1.0f, status_dev,
                      static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SV_OK
               : SV_ECUDA;
}

sv_status_t spec_verify_lm_head_fp8(const void *hidden, const float *hidden_scales, const void *lm_head,
                                    const float *lm_head_scales, int32_t d, const float *draft_probs,
                                    const int32_t *draft_tokens, const float *uniforms, float temperature, int64_t B,
                                    int32_t K, int32_t V, void *logits_out, int32_t *out_tokens, int32_t *num_emitted,
                                    int8_t *accept_flags, float *accept_prob, float *residual_mass,
                                    int32_t *status_dev, void *workspace, size_t workspace_bytes, void *stream)
{
    if (B < 0 || K < 0)
        return SV_EINVAL;
    if (B > 0 && static_cast<int64_t>(K) + 1 > kLmMaxRows / B)
        return SV_EUNSUPPORTED;
    const int64_t M = B * (static_cast<int64_t>(K) + 1);
    sv_status_t st = lm8_check(hidden, hidden_scales, lm_head, lm_head_scales, M, d, V, logits_out);
    if (st != SV_OK)
        return st;
    Plan plan;
    if (!make_plan(B, K, V, plan))
        return SV_EUNSUPPORTED;
    if (!workspace || workspace_bytes < plan.bytes + lm8_part_bytes(M, V))
        return SV_EINVAL;
    // host checks of the verification (nothing launched yet)
    st = run(0, logits_out, SV_BF16, draft_probs, draft_tokens, uniforms, temperature, B, K, V, out_tokens,
             num_emitted, accept_flags, accept_prob, residual_mass, status_dev, workspace, plan.bytes, stream);
    if (st != SV_OK || B == 0)
        return st;
    float2 *part = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + plan.bytes);
    const float c = static_cast<float>(1.4426950408889634074 / static_cast<double>(temperature));
    if (lm8_launch(hidden, hidden_scales, lm_head, lm_head_scales, M, d, V, logits_out, part, c, status_dev,
                   static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return SV_ECUDA;
    return lm_finish(plan, part, lm8_plan(M, V).NT, logits_out, draft_probs, draft_tokens, uniforms, temperature, B, K,
                     V, out_tokens, num_emitted, accept_flags, accept_prob, residual_mass, status_dev, workspace, stream);
}

sv_status_t sv_block_norm(const void *x, sv_dtype_t x_dtype, const void *residual, sv_dtype_t residual_dtype,
                          const void *post_weight, const void *gate, int64_t gate_rows, const void *norm_weight,
                          sv_dtype_t weight_dtype, float weight_offset, float residual_scale, float branch_scale,
                          float eps, int64_t M, int32_t d, void *residual_out, void *hidden, sv_dtype_t hidden_dtype,
                          float *hidden_scales, void *stream)
{
    if (M < 0 || d < 1 || !is_bf16_or_fp32(x_dtype) || !is_bf16_or_fp32(residual_dtype) ||
        !is_bf16_or_fp32(weight_dtype) || (!is_bf16_or_fp32(hidden_dtype) && hidden_dtype != SV_E4M3))
        return SV_EINVAL;
    if (!std::isfinite(weight_offset) || !std::isfinite(residual_scale) || !std::isfinite(branch_scale) ||
        !std::isfinite(eps) || !(eps > 0.0f))
        return SV_EINVAL;
    if (d > SV_MAX_D || M > INT32_MAX)
        return SV_EUNSUPPORTED;
    if (gate && (gate_rows < 1 || M % gate_rows != 0))
        return SV_EINVAL;
    if (M == 0)
        return SV_OK;
    if (!x || !residual || !norm_weight || !residual_out || !hidden || (hidden_dtype == SV_E4M3) != (hidden_scales != nullptr))
        return SV_EINVAL;
    if (!aligned(x, elem_size(x_dtype)) || !aligned(residual, elem_size(residual_dtype)) ||
        !aligned(residual_out, elem_size(residual_dtype)) || !aligned(hidden, elem_size(hidden_dtype)) ||
        !aligned(post_weight, elem_size(weight_dtype)) || !aligned(norm_weight, elem_size(weight_dtype)) ||
        !aligned(gate, elem_size(x_dtype)) || !aligned(hidden_scales, 4))
        return SV_EINVAL;
    sv::NormParams P;
    P.x = x;
    P.residual = residual;
    P.post = post_weight;
    P.gate = gate;
    P.pre = norm_weight;
    P.x_type = x_dtype;
    P.r_type = residual_dtype;
    P.w_type = weight_dtype;
    P.h_type = hidden_dtype;
    P.M = M;
    P.gate_div = static_cast<uint32_t>(gate ? M / gate_rows : 1);
    P.d = d;
    const int segs = static_cast<int>(ceil_div(d, sv::kSeg));
    P.WPR = 1;
    while (P.WPR < segs && P.WPR < sv::kNormMaxWarps)
        P.WPR *= 2;
    P.RPC = P.WPR < 4 ? 4 / P.WPR : 1;
    int nseg = 1;
    while (nseg * P.WPR < segs)
        nseg *= 2;
    P.offset = weight_offset;
    P.rs = residual_scale;
    P.bs = branch_scale;
    P.eps = eps;
    // An eps this small does not cover what the smallest squares lose by the
    // scale (4 d 2^-150 of the mean): they are then added as they are.
    int half = 0;
    while (eps >= 0x1p-100f && (int64_t{1} << (2 * half)) < d)
        ++half;
    P.sq_scale = std::ldexp(1.0f, -half);
    P.sq_inv_d = std::ldexp(1.0f / static_cast<float>(d), 2 * half);
    P.r_out = residual_out;
    P.h = hidden;
    P.scales = hidden_scales;
    const bool vec = d % 8 == 0 && vec_ok(x, x_dtype) && vec_ok(residual, residual_dtype) &&
                     vec_ok(residual_out, residual_dtype) && vec_ok(hidden, hidden_dtype) &&
                     vec_ok(post_weight, weight_dtype) && vec_ok(norm_weight, weight_dtype) && vec_ok(gate, x_dtype);
    const unsigned grid = static_cast<unsigned>(ceil_div(M, P.RPC));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // rows enough for every SM to walk several (and not too wide for several to
    // be in flight in shared memory): CTAs that stay
    if (vec && d <= sv::kNormRowsMaxD && M >= kNormManyRows &&
        norm_rows_smem(d, elem_size(x_dtype), elem_size(residual_dtype)) <= kNormRowsMaxSmem) {
        const bool xf = x_dtype == SV_FP32, rf = residual_dtype == SV_FP32;
        const cudaError_t e = xf ? (rf ? norm_rows_launch<true, true>(P, s) : norm_rows_launch<true, false>(P, s))
                                 : (rf ? norm_rows_launch<false, true>(P, s) : norm_rows_launch<false, false>(P, s));
        return e == cudaSuccess ? SV_OK : SV_ECUDA;
    }
    return (vec ? norm_launch<true>(P, nseg, grid, s) : norm_launch<false>(P, nseg, grid, s)) == cudaSuccess ? SV_OK
                                                                                                        : SV_ECUDA;
}

sv_status_t sv_quantize_fp8(const void *x, sv_dtype_t x_dtype, int64_t rows, int32_t d, int32_t block_rows,
                            void *values, float *scales, void *stream)
{
    if (rows < 0 || d < 1 || !is_bf16_or_fp32(x_dtype) || (block_rows != 1 && block_rows != 128))
        return SV_EINVAL;
    if (rows > INT32_MAX)
        return SV_EUNSUPPORTED;
    if (rows == 0)
        return SV_OK;
    if (!x || !values || !scales || !aligned(x, elem_size(x_dtype)) || !aligned(scales, 4))
        return SV_EINVAL;
    sv::QuantParams P;
    P.x = x;
    P.x_type = x_dtype;
    P.M = rows;
    P.d = d;
    P.v = static_cast<uint8_t *>(values);
    P.scales = scales;
    const bool vec = d % 8 == 0 && vec_ok(x, x_dtype) && vec_ok(values, SV_E4M3);
    P.segs = ceil_div(d, block_rows == 1 ? sv::kSeg : 128);
    const int64_t grid = block_rows == 1 ? ceil_div(rows * P.segs, sv::kQuantWarps) : ceil_div(rows, 128) * P.segs;
    if (grid > INT32_MAX)
        return SV_EUNSUPPORTED;
    const unsigned g = static_cast<unsigned>(grid);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    constexpr unsigned threads = sv::kQuantWarps * 32;
    cudaError_t e;
    if (block_rows == 1)
        e = launch_behind(vec ? sv::quantize_rows_kernel<true> : sv::quantize_rows_kernel<false>, g, threads, 0, s, P);
    else if (!vec)
        e = launch_behind(sv::quantize_tiles_odd_kernel, g, threads, 0, s, P);
    else
        e = launch_behind(x_dtype == SV_FP32 ? sv::quantize_tiles_kernel<true> : sv::quantize_tiles_kernel<false>, g,
                          threads, 0, s, P);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}

size_t sv_fp4_scale_bytes(int64_t rows, int32_t d, int32_t block)
{
    if (rows < 0 || rows > kFp4MaxRows || d < 2 || d > kFp4MaxD || d % 2 != 0 || (block != 16 && block != 32))
        return 0;
    return static_cast<size_t>(ceil_div(rows, 128)) * static_cast<size_t>(fp4_tiles(d, block)) * 512;
}

sv_status_t sv_quantize_fp4(const void *x, sv_dtype_t x_dtype, int64_t rows, int32_t d, int32_t block, void *values,
                            void *scales, float *row_scales, void *stream)
{
    if (rows < 0 || d < 2 || d % 2 != 0 || !is_bf16_or_fp32(x_dtype) || (block != 16 && block != 32))
        return SV_EINVAL;
    if (rows > kFp4MaxRows || d > kFp4MaxD)
        return SV_EUNSUPPORTED;
    if (rows == 0)
        return SV_OK;
    if (!x || !values || !scales || (block == 16) != (row_scales != nullptr) || !aligned(x, elem_size(x_dtype)) ||
        !aligned(scales, 16) || !aligned(row_scales, 4))
        return SV_EINVAL;
    sv::Fp4Params P;
    P.x = x;
    P.M = rows;
    P.Mpad = ceil_div(rows, 128) * 128;
    P.d = d;
    P.KT = fp4_tiles(d, block);
    P.octets = static_cast<int32_t>(P.KT * (block / 2)); // 4 blocks a tile
    P.WPR = fp4_warps(P.octets);
    P.pairs = aligned(x, 2 * elem_size(x_dtype));
    P.v = static_cast<uint8_t *>(values);
    P.s = static_cast<uint8_t *>(scales);
    P.g = row_scales;
    const bool vec = d % 8 == 0 && aligned(x, 16) && aligned(values, 4);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (block == 16)
        e = x_dtype == SV_BF16 ? quantize_fp4_launch<16, uint16_t>(P, vec, s) : quantize_fp4_launch<16, float>(P, vec, s);
    else
        e = x_dtype == SV_BF16 ? quantize_fp4_launch<32, uint16_t>(P, vec, s) : quantize_fp4_launch<32, float>(P, vec, s);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}

sv_status_t sv_dequantize_fp4(const void *values, const void *scales, const float *row_scales, int64_t rows, int32_t d,
                              int32_t block, void *out, sv_dtype_t out_dtype, void *stream)
{
    if (rows < 0 || d < 2 || d % 2 != 0 || !is_bf16_or_fp32(out_dtype) || (block != 16 && block != 32))
        return SV_EINVAL;
    if (rows > kFp4MaxRows || d > kFp4MaxD)
        return SV_EUNSUPPORTED;
    if (rows == 0)
        return SV_OK;
    if (!values || !scales || !out || (block == 16) != (row_scales != nullptr) || !aligned(out, elem_size(out_dtype)) ||
        !aligned(row_scales, 4))
        return SV_EINVAL;
    sv::Fp4BackParams P;
    P.v = static_cast<const uint8_t *>(values);
    P.s = static_cast<const uint8_t *>(scales);
    P.g = row_scales;
    P.M = rows;
    P.d = d;
    P.octets = static_cast<int32_t>(ceil_div(d, 8));
    P.KT = fp4_tiles(d, block);
    P.WPR = fp4_warps(P.octets);
    P.pairs = aligned(out, 2 * elem_size(out_dtype));
    P.out = out;
    const bool vec = d % 8 == 0 && aligned(values, 4) && aligned(out, 16);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (block == 16)
        e = out_dtype == SV_BF16 ? dequantize_fp4_launch<16, false>(P, vec, s) : dequantize_fp4_launch<16, true>(P, vec, s);
    else
        e = out_dtype == SV_BF16 ? dequantize_fp4_launch<32, false>(P, vec, s) : dequantize_fp4_launch<32, true>(P, vec, s);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}

sv_status_t sv_lm_head_logits_fp4(const void *hidden, const void *hidden_scales, const float *hidden_row_scales,
                                  const void *lm_head, const void *lm_head_scales, const float *lm_head_row_scales,
                                  int32_t block, int64_t M, int32_t d, int32_t V, void *logits, int32_t *status_dev,
                                  void *stream)
{
    if (M < 0 || d < 32 || d % 32 != 0 || V < 1 || (block != 16 && block != 32) || !aligned(status_dev, 4))
        return SV_EINVAL;
    // (a tile's sum over d is one bounded wait)
    if (V > SV_MAX_V || M > kLmMaxRows || d > (1 << 20))
        return SV_EUNSUPPORTED;
    // tiles and scale tiles are counted in 32 bits
    const sv::Lm4Plan p = sv::lm4_plan(M, V, kNominalSms);
    const int64_t tiles = static_cast<int64_t>(p.MT) * p.NT, kt = fp4_tiles(d, block);
    if (tiles > INT32_MAX || ceil_div(M, 128) > INT32_MAX / kt - 4 || ceil_div(V, 128) > INT32_MAX / kt - 4)
        return SV_EUNSUPPORTED;
    if (M == 0)
        return SV_OK;
    if (!hidden || !hidden_scales || !lm_head || !lm_head_scales || !logits || !aligned(hidden, 16) ||
        !aligned(hidden_scales, 16) || !aligned(lm_head, 16) || !aligned(lm_head_scales, 16) || !aligned(logits, 2) ||
        (block == 16) != (hidden_row_scales != nullptr) || (block == 16) != (lm_head_row_scales != nullptr) ||
        !aligned(hidden_row_scales, 4) || !aligned(lm_head_row_scales, 4))
        return SV_EINVAL;
    return lm4_launch(hidden, hidden_scales, hidden_row_scales, lm_head, lm_head_scales, lm_head_row_scales, block, M, d, V,
                      logits, status_dev, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SV_OK
               : SV_ECUDA;
}

sv_status_t sv_sample_logits(const void *logits, sv_dtype_t logits_dtype, const float *uniforms, float temperature,
                             int32_t top_k, float top_p, float min_p, int64_t rows, int32_t V, int32_t *tokens,
                             float *prob, int32_t *kept, float *probs, int32_t *status_dev, void *stream)
{
    if (rows < 0 || V < 1 || !is_bf16_or_fp32(logits_dtype))
        return SV_EINVAL;
    if (V > SV_MAX_V)
        return SV_EUNSUPPORTED;
    if (!std::isfinite(temperature) || !(temperature > 0.0f) || !(top_p > 0.0f) || !(min_p >= 0.0f && min_p <= 1.0f))
        return SV_EINVAL;
    const double c = 32 * 1.4426950408889634074 / static_cast<double>(temperature);
    sv::SampleParams P = {};
    P.c_hi = static_cast<float>(c);
    P.c_lo = static_cast<float>(c - static_cast<double>(P.c_hi));
    P.cq = static_cast<float>(c / 32);
    const int fb = 62 - ceil_log2_u64(static_cast<uint64_t>(V) + 1);
    P.fix = fb < 45 ? fb : 45;
    P.dmin = static_cast<float>(-(P.fix + 3) * 32 / c); // (a shift by 62 bits: nothing is left)
    // 24 octaves of mass, and 16 of logits at least where top-k counts ids without mass
    const double low = top_k > 0 ? 16.0 : 0.0, octaves = 24 * 32 / c, range = octaves > low ? octaves : low;
    P.bins = static_cast<float>(sv::kSmBins / range);
    P.width = static_cast<float>(range / sv::kSmBins);
    // (a temperature so far from 1 that its factors leave the fp32 range)
    if (!std::isfinite(P.c_hi) || !std::isfinite(P.dmin) || !(P.cq > 0x1p-100f) || !(P.cq < 0x1p100f))
        return SV_EINVAL;
    if (rows > 0 && (!logits || !uniforms || !tokens))
        return SV_EINVAL;
    if (!aligned(logits, elem_size(logits_dtype)) || !aligned(uniforms, 4) || !aligned(tokens, 4) || !aligned(prob, 4) ||
        !aligned(kept, 4) || !aligned(probs, 4) || !aligned(status_dev, 4))
        return SV_EINVAL;
    if (rows > INT32_MAX / sv::kSmMaxCtas)
        return SV_EUNSUPPORTED;
    if (rows == 0)
        return SV_OK;
    P.in = logits;
    P.rows = rows;
    P.V = V;
    P.u = uniforms;
    P.min_p = min_p > 0.0f;
    P.min_off = min_p > 0.0f ? std::log(static_cast<double>(min_p)) * static_cast<double>(temperature) : 0.0;
    P.top_k = top_k;
    P.top_p = top_p;
    P.tokens = tokens;
    P.prob = prob;
    P.kept = kept;
    P.probs = probs;
    P.status = status_dev;
    P.vec_q = aligned(logits, 16) && aligned(probs, 16);
    // a CTA's ids of a bin add up in 32 bits: 15 bits of up to 2^16 ids each, or (rows
    // of more than 2^19, up to 2^18 a CTA, and then fix <= 42) 14
    P.piece = V <= (1 << 19) ? 15 : 14;
    // CTAs of a row: enough that two of them fit an SM with their slices (one loads
    // while the other works), and, for few rows, that the rows' clusters reach every
    // SM, down to 2048 ids a CTA.
    const int32_t es = static_cast<int32_t>(elem_size(logits_dtype)), pv = 16 / es;
    const bool cuts = (top_k > 0 && top_k < V) || top_p < 1.0f;
    // a large batch's CTAs have 256 threads, four of them (five without cuts) an SM
    const size_t bins = cuts ? sizeof(sv::SampleBins) : 0, slim = 1152 * sizeof(uint16_t), wide = 4096 * sizeof(uint16_t);
    constexpr size_t kQuarter = 227 * 1024 / 4 - sizeof(sv::SampleShared) - 1024 - 256;
    auto cut = [&](int32_t C) {
        P.C = C;
        P.slice = static_cast<int32_t>(ceil_div(ceil_div(static_cast<int64_t>(V) + pv, C), pv) * pv);
        return static_cast<size_t>(P.slice) * static_cast<size_t>(es) + bins + (cuts ? slim : 0);
    };
    int32_t C = 1;
    while (C < sv::kSmMaxCtas && (cut(C) > kQuarter || (rows * C * 2 <= 2 * kNominalSms && V / (2 * C) >= 2048)))
        C *= 2;
    size_t smem = cut(C);
    const int threads = rows * C > 2 * kNominalSms && smem <= kQuarter ? 256 : 512;
    P.cap = threads == 256 ? 1152 : 4096;
    const size_t more = bins + (cuts ? (threads == 256 ? slim : wide) : 0);
    smem = static_cast<size_t>(P.slice) * static_cast<size_t>(es) + more;
    P.staged = smem <= kSampleSmem;
    if (!P.staged)
        smem = more;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = logits_dtype == SV_BF16 ? sample_launch<uint16_t>(P, threads, cuts, smem, s)
                                                  : sample_launch<float>(P, threads, cuts, smem, s);
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}

size_t sv_tree_workspace_bytes(int64_t B, int32_t N, int32_t V)
{
    Plan p;
    if (N < 1 || N > SV_MAX_TREE_NODES || !make_plan(B, N - 1, V, p))
        return 0;
    return p.bytes;
}

sv_status_t spec_verify_tree(const void *logits, sv_dtype_t dtype, const float *draft_probs, const int32_t *parent,
                             const int32_t *tokens, const float *uniforms, float temperature, int64_t B, int32_t N,
                             int32_t V, int32_t *out_tokens, int32_t *out_nodes, int32_t *num_emitted,
                             float *accept_prob, int32_t *status_dev, void *workspace, size_t workspace_bytes,
                             void *stream)
{
    if (B < 0 || N < 1 || V < 1)
        return SV_EINVAL;
    if (N > SV_MAX_TREE_NODES || V > SV_MAX_V || B > 0x3FFFFFFFll)
        return SV_EUNSUPPORTED;
    if (dtype != SV_BF16 && dtype != SV_FP32)
        return SV_EINVAL;
    if (!std::isfinite(temperature) || !(temperature > 0.0f))
        return SV_EINVAL;
    const float c = static_cast<float>(1.4426950408889634074 / static_cast<double>(temperature));
    if (!std::isfinite(c) || !(c > 0.0f))
        return SV_EINVAL;
    if (!logits || !draft_probs || !parent || !tokens || !uniforms || !out_tokens || !num_emitted || !workspace)
        return SV_EINVAL;
    const size_t esize = dtype == SV_BF16 ? 2 : 4;
    if (!aligned(logits, esize) || !aligned(draft_probs, 4) || !aligned(parent, 4) || !aligned(tokens, 4) ||
        !aligned(uniforms, 4) || !aligned(out_tokens, 4) || !aligned(num_emitted, 4) ||
        (out_nodes && !aligned(out_nodes, 4)) || (accept_prob && !aligned(accept_prob, 4)) ||
        (status_dev && !aligned(status_dev, 4)) || !aligned(workspace, kAlign))
        return SV_EINVAL;
    Plan plan;
    if (!make_plan(B, N - 1, V, plan))
        return SV_EUNSUPPORTED;
    if (workspace_bytes < plan.bytes)
        return SV_EINVAL;
    if (B == 0)
        return SV_OK;
    char *ws = static_cast<char *>(workspace);
    sv::Params P = {};
    P.logits = logits;
    P.q = nullptr; // the row pass takes no draft data here; the tree kernel reads q
    P.tokens = tokens;
    P.u = uniforms;
    P.c = c;
    P.B = B;
    P.K = N - 1;
    P.V = V;
    P.row_part = reinterpret_cast<float2 *>(ws + plan.off_part);
    P.row_side = reinterpret_cast<float4 *>(ws + plan.off_row_side);
    P.PM = plan.PM;
    P.fix_bits = plan.fix;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // the row pass over all B*N rows: every row's (max, normaliser) partials
    cudaError_t e = dtype == SV_BF16 ? launch<uint16_t, false>(P, plan, kRows, s)
                                     : launch<float, false>(P, plan, kRows, s);
    if (e != cudaSuccess)
        return SV_ECUDA;
    sv::TreeArgs A;
    A.parent = parent;
    A.tokens = tokens;
    A.q = draft_probs;
    A.u = uniforms;
    A.N = N;
    A.out_tokens = out_tokens;
    A.out_nodes = out_nodes;
    A.num_emitted = num_emitted;
    A.accept_prob = accept_prob;
    A.status = status_dev;
    // one cluster of two CTAs per sequence
    const size_t smem = static_cast<size_t>(ceil_div(V, sv::kTreeChunk)) * sizeof(long long);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = sv::kTreeCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    // programmatic dependent launch: the walk checks its inputs while the row
    // pass drains and waits in griddepcontrol.wait before reading its partials
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(B * sv::kTreeCtas));
    cfg.blockDim = dim3(sv::kTreeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (dtype == SV_BF16) {
        if (smem > 48 * 1024 &&
            cudaFuncSetAttribute(sv::tree_kernel<uint16_t>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem)) != cudaSuccess)
            return SV_ECUDA;
        e = cudaLaunchKernelEx(&cfg, sv::tree_kernel<uint16_t>, P, A);
    } else {
        if (smem > 48 * 1024 &&
            cudaFuncSetAttribute(sv::tree_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem)) != cudaSuccess)
            return SV_ECUDA;
        e = cudaLaunchKernelEx(&cfg, sv::tree_kernel<float>, P, A);
    }
    return e == cudaSuccess ? SV_OK : SV_ECUDA;
}

const char *sv_status_string(sv_status_t status)
{
    switch (status) {
    case SV_OK:
        return "SV_OK: work enqueued";
    case SV_EINVAL:
        return "SV_EINVAL: invalid argument (null or misaligned pointer, bad size, temperature or workspace)";
    case SV_ECUDA:
        return "SV_ECUDA: a CUDA launch failed";
    case SV_EUNSUPPORTED:
        return "SV_EUNSUPPORTED: size beyond what one call supports";
    }
    return "unknown sv_status_t";
}

} // extern "C"

// ---------------------------------------------------------------------------
// Allocation-free entry point.  Some callers cannot hand the library a
// workspace: a server whose device memory is reserved up front by its own
// pool and that forbids cudaMalloc on the request path, or a plugin interface
// that passes a plugin its input and output buffers but no allocator.  For
// them, spec_verify_noalloc runs the same kernels with their scratch in a
// fixed-size array that lives in the library's device image.  The array is
// shared by every call on a device and keeps the last call's contents, so
// each call clears the bytes it needs before launching; calls that overlap on
// the GPU (two streams, two host threads) race on it.
#include <mutex>

namespace {
constexpr size_t kNoallocScratchBytes = SV_NOALLOC_SCRATCH_BYTES;
} // namespace

// Every GPU that loads this library holds this array until the process exits.
static __device__ __align__(256) unsigned char g_sv_noalloc_scratch[kNoallocScratchBytes];

namespace {
// The device address of the scratch array in the current context.  In host
// code the array's name is only a stand-in, so the address is looked up
// with the device current, on every call: the lookup is host-side and
// cheap, and a kept address would go stale when the context is destroyed
// and made again (cudaDeviceReset), which places the module anew.
sv_status_t noalloc_scratch(void **out)
{
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_sv_noalloc_scratch) != cudaSuccess || p == nullptr) {
        (void)cudaGetLastError();
        return SV_ECUDA;
    }
    *out = p;
    return SV_OK;
}
} // namespace

extern "C" sv_status_t spec_verify_noalloc(const void *target_logits, sv_dtype_t logits_dtype,
                                           const float *draft_probs, const int32_t *draft_tokens,
                                           const float *uniforms, float temperature, int64_t B, int32_t K,
                                           int32_t V, int32_t *out_tokens, int32_t *num_emitted,
                                           int8_t *accept_flags, float *accept_prob, float *residual_mass,
                                           int32_t *status_dev, void *stream)
{
    Plan plan;
    if (make_plan(B, K, V, plan) && plan.bytes > kNoallocScratchBytes)
        return SV_EUNSUPPORTED; // this batch needs more scratch than the array holds
    void *scratch = nullptr;
    sv_status_t st = noalloc_scratch(&scratch);
    if (st != SV_OK)
        return st;
    // host checks only (stage mask 0 launches nothing)
    st = run(0, target_logits, logits_dtype, draft_probs, draft_tokens, uniforms, temperature, B, K, V,
             out_tokens, num_emitted, accept_flags, accept_prob, residual_mass, status_dev, scratch,
             kNoallocScratchBytes, stream);
    if (st != SV_OK || B == 0)
        return st;
    // the kernels expect zeroed scratch; a previous call may not have finished cleanly
    if (cudaMemsetAsync(scratch, 0, plan.bytes, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return SV_ECUDA;
    return run(kBoth, target_logits, logits_dtype, draft_probs, draft_tokens, uniforms, temperature, B, K, V,
               out_tokens, num_emitted, accept_flags, accept_prob, residual_mass, status_dev, scratch,
               kNoallocScratchBytes, stream);
}
