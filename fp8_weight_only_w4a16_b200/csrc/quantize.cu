// quantize.cu -- activations to 8-bit integers, one FP32 scale per token:
//
//   scale[m] = max_k |x[m][k]| / 127,   q[m][k] = round_to_even(x[m][k] / scale[m])
//
// One group of warps per row holds the row in registers between the maximum
// and the rounding, so x is read once (2 or 4 bytes an element) and q written
// once (1 byte).  Bound by HBM, or by latency for a few rows.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/skinny.h"
#include "ptx.cuh"

namespace skinny {
namespace {

constexpr int kVec = 8;            // elements a thread reads at once
constexpr int kMaxVecs = 4;        // vectors a thread keeps in registers

template <bool F32>
__device__ __forceinline__ void load8(const void* x, int64_t i, float (&v)[kVec])
{
    if constexpr (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
        const float4 a = p[0], b = p[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const __half*>(x) + i);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
    }
}

// x / scale to the nearest whole number, ties to even, as if the quotient were
// exact.  x * (1 / scale) in FP32 is at most 127 * 2^-22 off (the reciprocal,
// the product and the scale's own range), so only quotients that close to the
// middle of two whole numbers need the division in 64 bits, whose own rounding
// cannot cross the middle: x has 24 bits and the middle times the scale 32.
// A scale whose reciprocal overflows comes this way too (t is inf or NaN).
__device__ __forceinline__ int round_quotient(float x, float scale, float inv)
{
    const float t = x * inv;
    float q = rintf(t);
    if (!(fabsf(fabsf(t - q) - 0.5f) > 127.f / (1 << 22))) q = (float)rint((double)x / (double)scale);
    return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// threads_per_row (a multiple of 32) threads work on a row; a block holds
// blockDim.x / threads_per_row rows.  KEEP: the row fits the registers;
// otherwise it is read a second time.
template <bool F32, bool KEEP>
__global__ void __launch_bounds__(1024)
    quantize(const void* __restrict__ x, int64_t M, int K, int threads_per_row, int8_t* __restrict__ q,
             float* __restrict__ row_scale)
{
    __shared__ uint32_t part[32];
    // The next kernel may start once this one has seen the previous one's end:
    // what it reads early was then written two kernels ago at the latest.
    ptx::pdl_wait_prior_grid();
    ptx::pdl_launch_dependents();
    const int r = threadIdx.x / threads_per_row, t = threadIdx.x % threads_per_row;
    const int64_t m = (int64_t)blockIdx.x * (blockDim.x / threads_per_row) + r;
    const bool live = m < M;
    const int64_t row = m * K;
    const int n = K / kVec;

    float v[KEEP ? kMaxVecs : 1][kVec];
    uint32_t top = 0;    // |x| as bits: ordered like the values, NaN above infinity
    if (live) {
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < kMaxVecs; ++i) {
                const int at = t + i * threads_per_row;
                if (at < n) {
                    load8<F32>(x, row + (int64_t)at * kVec, v[i]);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) top = max(top, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
                }
            }
        } else {
            for (int at = t; at < n; at += threads_per_row) {
                load8<F32>(x, row + (int64_t)at * kVec, v[0]);
#pragma unroll
                for (int j = 0; j < kVec; ++j) top = max(top, __float_as_uint(v[0][j]) & 0x7FFFFFFFu);
            }
        }
    }
    top = __reduce_max_sync(~0u, top);
    if (threads_per_row > 32) {
        const int warps = threads_per_row / 32, w0 = r * warps;
        if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = top;
        __syncthreads();
        for (int w = 0; w < warps; ++w) top = max(top, part[w0 + w]);
    }
    if (!live) return;
    const bool finite = top < 0x7F800000u;
    const float scale = finite ? __fdiv_rn(__uint_as_float(top), 127.f) : __uint_as_float(0x7FC00000u);
    const float inv = __fdiv_rn(1.f, scale);
    const bool zero = !(scale > 0.f);      // a row of zeros, or one that is not finite
    if (t == 0) row_scale[m] = scale;
    auto put = [&](int at, const float (&f)[kVec]) {
        uint32_t w[2] = {0, 0};
        if (!zero) {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                w[j / 4] |= (uint32_t)(uint8_t)(int8_t)round_quotient(f[j], scale, inv) << (8 * (j % 4));
        }
        *reinterpret_cast<uint2*>(q + row + (int64_t)at * kVec) = make_uint2(w[0], w[1]);
    };
    if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < kMaxVecs; ++i) {
            const int at = t + i * threads_per_row;
            if (at < n) put(at, v[i]);
        }
    } else {
        for (int at = t; at < n; at += threads_per_row) {
            load8<F32>(x, row + (int64_t)at * kVec, v[0]);
            put(at, v[0]);
        }
    }
}

}  // namespace
}  // namespace skinny

using namespace skinny;

extern "C" int skinny_quantize_int8(const void* x, int in_dtype, int64_t M, int64_t K, void* q, float* row_scale,
                                    void* stream)
{
    if (in_dtype != SKINNY_OUT_F16 && in_dtype != SKINNY_OUT_F32) return SKINNY_ERR_INVALID_ARG;
    if (M < 0 || K <= 0 || K % 16 != 0) return SKINNY_ERR_INVALID_ARG;
    if (M > (int64_t(1) << 24) || K > (int64_t(1) << 20)) return SKINNY_ERR_UNSUPPORTED;
    if (M == 0) return SKINNY_OK;
    if (!x || !q || !row_scale) return SKINNY_ERR_INVALID_ARG;
    if ((uintptr_t)x % 16 || (uintptr_t)q % 16 || (uintptr_t)row_scale % 4) return SKINNY_ERR_ALIGNMENT;
    // Few rows: one vector per thread, for the shortest chain of loads.  Many
    // rows: up to four per thread, so that more rows are in flight on an SM.
    const int n = (int)(K / kVec);
    const int want = M < 512 ? n : (n + kMaxVecs - 1) / kMaxVecs;
    int threads = (want + 31) / 32 * 32;
    threads = threads > 1024 ? 1024 : threads;
    const int rows = threads >= 256 ? 1 : 256 / threads;
    const bool keep = n <= threads * kMaxVecs, f32 = in_dtype == SKINNY_OUT_F32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((M + rows - 1) / rows));
    cfg.blockDim = dim3(threads * rows);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto* kernel = f32 ? (keep ? quantize<true, true> : quantize<true, false>)
                       : (keep ? quantize<false, true> : quantize<false, false>);
    return cudaLaunchKernelEx(&cfg, kernel, x, M, (int)K, threads, static_cast<int8_t*>(q), row_scale) == cudaSuccess
               ? SKINNY_OK
               : SKINNY_ERR_CUDA;
}
