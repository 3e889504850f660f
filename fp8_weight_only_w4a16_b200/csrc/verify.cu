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
// totals are exchanged through distributed shared memory, and the one warp
// whose piece holds the crossing walks its piece again (a few hundred
// elements, still in L2).  Differences and sums are FP64: a product of two
// FP32 numbers is exact there, and running sums over a vocabulary stay far
// closer to exact than neighbouring tokens' probabilities are to each other.
// Bound by HBM for many requests, by latency for a few.
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

// Four consecutive elements from v0 (a multiple of 4), 0 past the end.
template <typename T>
__device__ __forceinline__ void load4(const T* row, int v0, int V, bool vec, float (&f)[4])
{
    if (vec && v0 + 4 <= V) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = *reinterpret_cast<const float4*>(row + v0);
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        } else {
            const uint2 a = *reinterpret_cast<const uint2*>(row + v0);
            T h[4];
            memcpy(h, &a, 8);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = to_float(h[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = v0 + j < V ? to_float(row[v0 + j]) : 0.f;
    }
}

// What a token weighs in the draw.  Differences that are not positive finite
// numbers (NaN among them) weigh nothing.
__device__ __forceinline__ double weight(float p, float q)
{
    const double d = (double)p - (double)q;
    return d > 0.0 && d < INFINITY ? d : 0.0;
}

template <typename T>
struct Row {
    const T* p;
    const T* q;          // null: nothing is subtracted
    int without;         // a token that weighs nothing (-1: none)
    int V;
    bool vec;
    __device__ __forceinline__ void weights(int v0, double (&w)[4]) const
    {
        float a[4], b[4] = {0.f, 0.f, 0.f, 0.f};
        load4(p, v0, V, vec, a);
        if (q) load4(q, v0, V, vec, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = v0 + j == without ? 0.0 : weight(a[j], b[j]);
    }
};

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(~0u, v, d);
    return v;
}

// The piece that holds the crossing: the first with a positive total whose
// running sum exceeds `limit`, or else the last with a positive total (-1:
// none).  *before receives the sum of the pieces in front of it.
__device__ __forceinline__ int crossing(const double* totals, int n, double first, double limit, double* before)
{
    int at = -1;
    double sum = first, b = first;
    for (int i = 0; i < n; ++i) {
        if (totals[i] > 0.0) {
            at = i;
            b = sum;
            if (sum + totals[i] > limit) break;
        }
        sum += totals[i];
    }
    *before = b;
    return at;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify(const __grid_constant__ Params a)
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
    ptx::pdl_launch_dependents();
    ptx::pdl_wait_prior_grid();
    const T* target = static_cast<const T*>(a.target) + b * a.target_b;
    const T* draft = a.draft ? static_cast<const T*>(a.draft) + b * a.draft_b : nullptr;
    const int32_t* drafted = a.draft_tokens + b * a.S;
    const float* uniform = a.uniform + b * (a.S + 1);

    if (warp == 0) {
        int count = a.num_drafts ? a.num_drafts[b] : a.S;
        count = count < 0 ? 0 : count > a.S ? a.S : count;
        int n = count;
        for (int i0 = 0; i0 < count; i0 += 32) {
            const int i = i0 + lane;
            bool ok = true;
            if (i < count) {
                const int d = drafted[i];
                ok = d >= 0 && d < a.V;
                if (ok) {
                    const float p = to_float(target[i * a.target_s + d]);
                    const float q = draft ? to_float(draft[i * a.draft_s + d]) : 1.f;
                    ok = (double)uniform[i] * (double)q < (double)p;
                }
            }
            const unsigned bad = __ballot_sync(~0u, !ok);
            if (bad) {
                n = i0 + __ffs(bad) - 1;
                break;
            }
        }
        if (lane == 0) {
            s_accepted = n;
            s_count = count;
        }
    }
    __syncthreads();
    const int n = s_accepted;
    const bool rejected = n < s_count;
    const double u = (double)uniform[a.S];

    Row<T> row;
    row.p = target + n * a.target_s;
    row.q = rejected && draft ? draft + n * a.draft_s : nullptr;
    row.without = rejected && !draft ? drafted[n] : -1;
    row.V = a.V;
    constexpr int kAlign = 4 * sizeof(T);
    row.vec = (uintptr_t)row.p % kAlign == 0 && (!row.q || (uintptr_t)row.q % kAlign == 0);

    // Warp w of CTA c owns the w-th of ctas * kWarps equal pieces in turn.
    const int pieces = ctas * kWarps;
    const int piece = (a.V + pieces * kStep - 1) / (pieces * kStep) * kStep;
    const int64_t begin64 = (int64_t)(rank * kWarps + warp) * piece;
    const int begin = begin64 < a.V ? (int)begin64 : a.V;
    const int end = begin64 + piece < a.V ? (int)(begin64 + piece) : a.V;

    cluster.barrier_wait(std::move(started));
    int token = -1;
    bool mine = false;
    // Second pass: the difference weighs nothing anywhere (the two rows are
    // equal, or rounded so): the target's own row is drawn from.
    for (int pass = 0; pass < 2; ++pass) {
        double sum = 0.0;
#pragma unroll 4
        for (int v = begin + lane * 4; v < end; v += kStep) {
            double w[4];
            row.weights(v, w);
            sum += (w[0] + w[1]) + (w[2] + w[3]);
        }
        sum = warp_sum(sum);
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
        if (threadIdx.x < ctas) {
            double total = 0.0;
            for (int w = 0; w < kWarps; ++w) total += s_warp[w];
            *cluster.map_shared_rank(&s_cta[pass][rank], threadIdx.x) = total;
        }
        cluster.sync();
        double total = 0.0;
        for (int c = 0; c < ctas; ++c) total += s_cta[pass][c];
        const double limit = u * total;
        double before;
        const int c = crossing(s_cta[pass], ctas, 0.0, limit, &before);
        if (c < 0) {
            if (pass == 0 && rejected) {
                row.q = nullptr;
                row.without = -1;
                row.vec = (uintptr_t)row.p % kAlign == 0;
                __syncthreads();      // s_warp is written again
                continue;
            }
            mine = rank == 0 && threadIdx.x == 0;      // nothing to draw from: -1
            break;
        }
        if (c == rank) {
            const int w = crossing(s_warp, kWarps, before, limit, &before);
            if (w == warp) {
                // walk the piece again, with running sums
                int last = -1;
                for (int v0 = begin; v0 < end && token < 0; v0 += kStep) {
                    const int v = v0 + lane * 4;
                    double x[4] = {0.0, 0.0, 0.0, 0.0};
                    if (v < end) row.weights(v, x);
                    const double own = (x[0] + x[1]) + (x[2] + x[3]);
                    double run = own;
#pragma unroll
                    for (int d = 1; d < 32; d *= 2) {
                        const double o = __shfl_up_sync(~0u, run, d);
                        if (lane >= d) run += o;
                    }
                    const double step = __shfl_sync(~0u, run, 31);
                    double at = before + (run - own);
                    int hit = -1, most = -1;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        at += x[j];
                        if (x[j] > 0.0) {
                            most = v + j;
                            if (hit < 0 && at > limit) hit = v + j;
                        }
                    }
                    const unsigned hits = __ballot_sync(~0u, hit >= 0), any = __ballot_sync(~0u, most >= 0);
                    if (any) last = __shfl_sync(~0u, most, 31 - __clz(any));
                    if (hits) token = __shfl_sync(~0u, hit, __ffs(hits) - 1);
                    before += step;
                }
                if (token < 0) token = last;
                mine = lane == 0;
            }
        }
        break;
    }
    if (mine) a.tokens[b * (a.S + 1) + n] = token;
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
    // Few requests: sixteen CTAs each, to read their rows in less time (the
    // portable limit is eight).
    const int ctas = B <= 8 ? kMaxCluster : 8;
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
