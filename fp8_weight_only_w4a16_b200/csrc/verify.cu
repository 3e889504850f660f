// verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers (speculative sampling):
//
//   draft i is accepted while u_i * q_i(d_i) < p_i(d_i);
//   at the first one that is not, the next token is drawn from
//   max(p_i - q_i, 0) (normalised), or, if all are accepted, from the row of
//   the target that follows them, by inversion: the first token whose running
//   sum exceeds u_last times the total.
//
// A request is one cluster of CTAs.  Only the one row at stake is read (of
// target and draft): every CTA sums its slice of the vocabulary, the slices'
// totals are exchanged through distributed shared memory, and one warp of the
// CTA that holds the crossing walks the piece that holds it again (some hundred
// elements, still in L2).  Differences and sums are FP64: a product of two
// FP32 numbers is exact there, and running sums over a vocabulary stay far
// closer to exact than neighbouring tokens' probabilities are to each other.
// Bound by HBM for many requests, by latency for a few: on a B200, 64 requests
// of 151936 FP32 probabilities take 21.5 to 23.5 us (up to 78 MB, 3.6 TB/s), one
// 5.5 to 6.5 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <utility>

#include "../../include/skinny.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace skinny {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kStep = 128;            // elements a warp reads at once: 4 per lane

struct Params {
    const void* target;               // [B][S + 1][V], strides in elements
    const void* draft;                // [B][S][V] or null
    int64_t target_b, target_s, draft_b, draft_s;
    const int32_t* draft_tokens;      // [B][S]
    const float* uniform;             // [B][S + 1]
    const int32_t* num_drafts;        // [B] or null
    int32_t* tokens;                  // [B][S + 1]
    int32_t* accepted;                // [B]
    int S, V;
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// Four consecutive elements at an aligned address.
template <typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[4])
{
    if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4*>(p);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    } else {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        T h[4];
        memcpy(h, &a, 8);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = to_float(h[j]);
    }
}

// Four consecutive elements from v0 (a multiple of 4), 0 past the end.
template <typename T>
__device__ __forceinline__ void load4(const T* row, int v0, int V, bool vec, float (&f)[4])
{
    if (vec && v0 + 4 <= V) {
        load_vec(row + v0, f);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = v0 + j < V ? to_float(row[v0 + j]) : 0.f;
    }
}

// Whether p - q counts in the draw: positive, and within FP32's range (so
// neither an infinity nor a NaN counts).  The FP32 difference of two different
// numbers is never 0, so its sign is exact.
__device__ __forceinline__ bool counts(float p, float q)
{
    return __float_as_uint(p - q) - 1u < 0x7F7FFFFFu;
}

template <typename T>
struct Row {
    const T* p;
    const T* q;          // null: nothing is subtracted
    int without;         // a token that weighs nothing (-1: none)
    int V;
    bool vec;
    // The weights of tokens v0 .. v0 + 3 (v0 a multiple of 4).
    __device__ __forceinline__ void weights(int v0, double (&w)[4]) const
    {
        float a[4], b[4] = {0.f, 0.f, 0.f, 0.f};
        load4(p, v0, V, vec, a);
        if (q) load4(q, v0, V, vec, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = counts(a[j], b[j]) ? (double)a[j] - (double)b[j] : 0.0;
        const unsigned hole = (unsigned)without - (unsigned)v0;
        if (hole < 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (hole == j) w[j] = 0.0;
        }
    }
    // Sum of the weights from `begin` to `end` at one lane's places (4 in 128).
    template <bool Q>
    __device__ __forceinline__ double sum(int begin, int end, int lane) const
    {
        double sum = 0.0;
        int v = begin + lane * 4;
        if (vec) {
            // whole vectors, eight loads in flight
            const int whole = end & ~3;
            for (; v + 3 * kStep < whole; v += 4 * kStep) {
                float a[4][4], b[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    load_vec(p + v + i * kStep, a[i]);
                    if (Q) load_vec(q + v + i * kStep, b[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) sum += sum4<Q>(a[i], b[i], v + i * kStep);
            }
        }
        for (; v < end; v += kStep) {
            float a[4], b[4];
            load4(p, v, V, vec, a);
            if (Q) load4(q, v, V, vec, b);
            sum += sum4<Q>(a, b, v);
        }
        return sum;
    }
    template <bool Q>
    __device__ __forceinline__ double sum4(const float (&a)[4], const float (&b)[4], int v0) const
    {
        // With finite numbers, max(p - q, 0) = max(p, q) - q: one FP32 maximum, and
        // the conversions.  A sum of magnitudes that is not finite, or the token left
        // out, takes the way that looks at every element.  (No difference is larger
        // than that sum, so a finite sum leaves none outside FP32's range.)
        float all = (fabsf(a[0]) + fabsf(a[1])) + (fabsf(a[2]) + fabsf(a[3]));
        if (Q) all += (fabsf(b[0]) + fabsf(b[1])) + (fabsf(b[2]) + fabsf(b[3]));
        const unsigned hole = (unsigned)without - (unsigned)v0;      // (only a row without q has one)
        double w[4];
        if (all < INFINITY && (Q || hole >= 4)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = (double)fmaxf(a[j], Q ? b[j] : 0.f);
                if (Q) w[j] -= (double)b[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool ok = counts(a[j], Q ? b[j] : 0.f) && (Q || hole != j);
                w[j] = ok ? (double)a[j] - (Q ? (double)b[j] : 0.0) : 0.0;
            }
        }
        return (w[0] + w[1]) + (w[2] + w[3]);
    }
};

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(~0u, v, d);
    return v;
}

// Of up to 32 pieces (lane i holds the total of piece i, 0 past the last): the
// first with a positive total whose running sum, from `first` on, exceeds
// `limit`, or else the last with a positive total; -1 if none has.  *before
// receives the running sum in front of it.
__device__ __forceinline__ int crossing(double total, double first, double limit, double* before)
{
    const int lane = threadIdx.x & 31;
    double run = total;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const double o = __shfl_up_sync(~0u, run, d);
        if (lane >= d) run += o;
    }
    const unsigned some = __ballot_sync(~0u, total > 0.0);
    const unsigned over = __ballot_sync(~0u, total > 0.0 && first + run > limit);
    if (some == 0) return -1;
    const int at = over ? __ffs(over) - 1 : 31 - __clz(some);
    *before = first + __shfl_sync(~0u, run - total, at);
    return at;
}

// The token at which the running sum of weights from `begin` to `end`, with
// `before` in front, exceeds `limit`; or else the last with a weight.  One
// warp: a lane takes 16 neighbouring tokens at a time, so that the loads of
// 512 tokens are under way together.
template <typename T>
__device__ int find_token(const Row<T>& row, int begin, int end, double before, double limit)
{
    const int lane = threadIdx.x & 31;
    int last = -1;
    for (int v0 = begin; v0 < end; v0 += 512) {
        const int v = v0 + lane * 16;
        double x[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (v + 4 * i < end) row.weights(v + 4 * i, x[i]);
            else x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.0;
        }
        double own = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) own += (x[i][0] + x[i][1]) + (x[i][2] + x[i][3]);
        double run = own;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const double o = __shfl_up_sync(~0u, run, d);
            if (lane >= d) run += o;
        }
        const double whole = __shfl_sync(~0u, run, 31);
        double at = before + (run - own);
        int hit = -1, most = -1;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const double w = x[i / 4][i % 4];
            at += w;
            if (w > 0.0) {
                most = v + i;
                if (hit < 0 && at > limit) hit = v + i;
            }
        }
        const unsigned hits = __ballot_sync(~0u, hit >= 0), any = __ballot_sync(~0u, most >= 0);
        if (hits) return __shfl_sync(~0u, hit, __ffs(hits) - 1);
        if (any) last = __shfl_sync(~0u, most, 31 - __clz(any));
        before += whole;
    }
    return last;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) verify(const __grid_constant__ Params a)
{
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    const int64_t b = blockIdx.x / ctas;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    __shared__ int s_accepted, s_count;
    __shared__ double s_warp[kWarps];
    __shared__ double s_cta[2][kMaxCluster];

    // Before the first write to another CTA's shared memory, all have to run.
    auto started = cluster.barrier_arrive();
    // The next kernel may start once this one has seen the previous one's end:
    // what it reads early was then written two kernels ago at the latest.
    ptx::pdl_wait_prior_grid();
    ptx::pdl_launch_dependents();
    const T* target = static_cast<const T*>(a.target) + b * a.target_b;
    const T* draft = a.draft ? static_cast<const T*>(a.draft) + b * a.draft_b : nullptr;
    const int32_t* drafted = a.draft_tokens + b * a.S;
    const float* uniform = a.uniform + b * (a.S + 1);
    const double u = (double)uniform[a.S];

    if (warp == 0) {
        int count = a.num_drafts ? a.num_drafts[b] : a.S;
        int n = a.S;
        for (int i0 = 0; i0 < a.S; i0 += 32) {
            // all drafts are looked at, whatever the count: its load is not waited for first
            const int i = i0 + lane;
            bool ok = true;
            if (i < a.S) {
                const int d = drafted[i];
                const float x = uniform[i];
                ok = d >= 0 && d < a.V;
                if (ok) {
                    const float p = to_float(target[i * a.target_s + d]);
                    const float q = draft ? to_float(draft[i * a.draft_s + d]) : 1.f;
                    ok = (double)x * (double)q < (double)p;
                }
            }
            const unsigned bad = __ballot_sync(~0u, !ok);
            if (bad) {
                n = i0 + __ffs(bad) - 1;
                break;
            }
        }
        count = count < 0 ? 0 : count > a.S ? a.S : count;
        if (lane == 0) {
            s_accepted = n < count ? n : count;
            s_count = count;
        }
    }
    __syncthreads();
    const int n = s_accepted;
    const bool rejected = n < s_count;

    Row<T> row;
    row.p = target + n * a.target_s;
    row.q = rejected && draft ? draft + n * a.draft_s : nullptr;
    row.without = rejected && !draft ? drafted[n] : -1;
    row.V = a.V;
    constexpr int kAlign = 4 * sizeof(T);
    row.vec = (uintptr_t)row.p % kAlign == 0 && (!row.q || (uintptr_t)row.q % kAlign == 0);

    // Warp w of CTA c owns piece c * kWarps + w of the vocabulary.
    const int pieces = ctas * kWarps;
    const int piece = (a.V + pieces * kStep - 1) / (pieces * kStep) * kStep;
    auto bound = [&](int i) { return (int64_t)i * piece < a.V ? i * piece : a.V; };
    const int begin = bound(rank * kWarps + warp), end = bound(rank * kWarps + warp + 1);

    cluster.barrier_wait(std::move(started));
    // Second pass: the difference weighs nothing anywhere (the two rows are
    // equal, or rounded so): the target's own row is drawn from.
    for (int pass = 0; pass < 2; ++pass) {
        const double sum = warp_sum(row.q ? row.template sum<true>(begin, end, lane)
                                          : row.template sum<false>(begin, end, lane));
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            const double total = warp_sum(lane < kWarps ? s_warp[lane] : 0.0);
            if (lane < ctas) *cluster.map_shared_rank(&s_cta[pass][rank], lane) = total;
        }
        cluster.sync();
        const double total = lane < ctas ? s_cta[pass][lane] : 0.0;
        if (__any_sync(~0u, total > 0.0)) {
            if (warp == 0) {
                const double limit = u * warp_sum(total);
                double before;
                const int c = crossing(total, 0.0, limit, &before);
                if (c == rank) {
                    const int w = crossing(lane < kWarps ? s_warp[lane] : 0.0, before, limit, &before);
                    const int piece0 = rank * kWarps + w;
                    const int token = find_token(row, bound(piece0), bound(piece0 + 1), before, limit);
                    if (lane == 0) a.tokens[b * (a.S + 1) + n] = token;
                }
            }
            break;
        }
        if (pass == 1 || !rejected) {
            if (rank == 0 && threadIdx.x == 0) a.tokens[b * (a.S + 1) + n] = -1;      // nothing to draw from
            break;
        }
        row.q = nullptr;
        row.without = -1;
        row.vec = (uintptr_t)row.p % kAlign == 0;
        __syncthreads();      // s_warp is written again
    }
    if (rank == 0) {
        for (int i = threadIdx.x; i <= a.S; i += kThreads)
            if (i != n) a.tokens[b * (a.S + 1) + i] = i < n ? drafted[i] : -1;
        if (threadIdx.x == 0) a.accepted[b] = n;
    }
    // No CTA's shared memory goes away while another one may still write to it:
    // the writes precede the cluster barrier above, which all have passed.
}

template <typename T>
int launch(const Params& p, int64_t B, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
        return SKINNY_ERR_CUDA;
    // As many CTAs for each request as fit the GPU together (two to an SM), so
    // that few requests' rows are read in less time, between 4 and 16 (the
    // portable limit is 8).  Measured: one request 6.4 us with 16 CTAs and 12.2
    // with 4; 64 requests 20.2 us with 4 and 31.8 with 16.
    const int64_t fit = 2 * (int64_t)sms / B;
    const int ctas = fit >= 16 ? 16 : fit >= 8 ? 8 : 4;
    if (ctas > 8 && cudaFuncSetAttribute(verify<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return SKINNY_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify<T>, p) == cudaSuccess ? SKINNY_OK : SKINNY_ERR_CUDA;
}

}  // namespace
}  // namespace skinny

using namespace skinny;

extern "C" int skinny_verify_draft(const void* target, int64_t target_b, int64_t target_s, const void* draft,
                                   int64_t draft_b, int64_t draft_s, int prob_dtype, const int32_t* draft_tokens,
                                   const float* uniform, const int32_t* num_drafts, int64_t B, int64_t S, int64_t V,
                                   int32_t* tokens, int32_t* accepted, void* stream)
{
    if (prob_dtype < SKINNY_PROB_F16 || prob_dtype > SKINNY_PROB_BF16) return SKINNY_ERR_INVALID_ARG;
    if (B < 0 || S < 0 || V <= 0) return SKINNY_ERR_INVALID_ARG;
    if (B > (int64_t(1) << 20) || S > 1024 || V > (int64_t(1) << 28)) return SKINNY_ERR_UNSUPPORTED;
    if (B == 0) return SKINNY_OK;
    if (!target || !uniform || !tokens || !accepted || (S > 0 && !draft_tokens)) return SKINNY_ERR_INVALID_ARG;
    const uintptr_t size = prob_dtype == SKINNY_PROB_F32 ? 4 : 2;
    if ((uintptr_t)target % size || (uintptr_t)draft % size || (uintptr_t)draft_tokens % 4 || (uintptr_t)uniform % 4 ||
        (uintptr_t)num_drafts % 4 || (uintptr_t)tokens % 4 || (uintptr_t)accepted % 4)
        return SKINNY_ERR_ALIGNMENT;
    Params p{};
    p.target = target;
    p.draft = draft;
    p.target_b = target_b;
    p.target_s = target_s;
    p.draft_b = draft_b;
    p.draft_s = draft_s;
    p.draft_tokens = draft_tokens;
    p.uniform = uniform;
    p.num_drafts = num_drafts;
    p.tokens = tokens;
    p.accepted = accepted;
    p.S = (int)S;
    p.V = (int)V;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (prob_dtype == SKINNY_PROB_F32) return launch<float>(p, B, st);
    if (prob_dtype == SKINNY_PROB_F16) return launch<__half>(p, B, st);
    return launch<__nv_bfloat16>(p, B, st);
}
