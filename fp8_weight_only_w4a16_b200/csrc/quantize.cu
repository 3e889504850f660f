// quantize.cu -- activations to 8-bit integers, one FP32 scale per token:
//
//   scale[m] = max_k |x[m][k]| / 127,   q[m][k] = round_to_even(x[m][k] / scale[m])
//
// One group of warps per row holds the row in registers between the maximum
// and the rounding, so x is read once (2 or 4 bytes an element) and q written
// once (1 byte).  Bound by HBM for FP32 rows, by the arithmetic of eight
// elements a thread for FP16 ones, and by latency for a few rows.  On a B200:
// 8192 x 5120 in 33 us from FP32 (6.4 TB/s) and 32 us from FP16 (4.0 TB/s), one
// row in 2.4 us.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/skinny.h"
#include "ptx.cuh"

namespace skinny {
namespace {

constexpr int kVec = 8;            // elements a thread reads at once
constexpr int kMaxVecs = 4;        // vectors a thread keeps in registers

// Eight elements as they lie in memory.
template <bool F32>
struct Raw {
    uint4 w[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* x, int64_t i)
    {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + i * (F32 ? 4 : 2));
        w[0] = ptx::ld_global_v4(p);
        if (F32) w[F32 ? 1 : 0] = ptx::ld_global_v4(p + 1);
    }
    __device__ __forceinline__ void floats(float (&v)[kVec]) const
    {
        const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if (F32) {
                v[j] = __uint_as_float(u[j]);
            } else if (j % 2 == 0) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j / 2]));
                v[j] = f.x;
                v[j + 1] = f.y;
            }
        }
    }
    // The largest magnitude as FP32 bits: ordered like the values, NaN above infinity.
    __device__ __forceinline__ uint32_t top() const
    {
        const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
        if constexpr (F32) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < kVec; ++j) m = max(m, u[j] & 0x7FFFFFFFu);
            return m;
        } else {
            // two halves at a time, as 16-bit whole numbers
            uint32_t m = __vmaxu2(__vmaxu2(u[0] & 0x7FFF7FFFu, u[1] & 0x7FFF7FFFu),
                                  __vmaxu2(u[2] & 0x7FFF7FFFu, u[3] & 0x7FFF7FFFu));
            m = max(m & 0xFFFFu, m >> 16);
            return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
        }
    }
};

// x / scale to the nearest whole number, ties to even, of the exact quotient:
// the division in 64 bits, whose own rounding cannot cross the middle of two
// whole numbers (x has 24 bits, the middle times the scale 32).
__device__ __noinline__ int exact_quotient(float x, float scale)
{
    const double q = rint((double)x / (double)scale);
    return (int)fmin(fmax(q, -127.0), 127.0);
}

// Eight quotients as bytes.  fma(x, 1 / scale, 1.5 * 2^23) rounds the product to
// a whole number, which its low byte holds.  The reciprocal is at most 2^-24 of
// itself off, so the product is off by at most 127 * 2^-24, and only a quotient
// that close to the middle of two whole numbers can have gone wrong: twice that
// close (one in some 30,000), it is divided in 64 bits.  `normal`: the scale is
// a normal number, so that its reciprocal is one.
__device__ __forceinline__ uint2 quotients(const float (&x)[kVec], float scale, float inv, bool normal)
{
    constexpr float kMagic = 12582912.f, kNear = 0.5f - 127.f / (1 << 23);
    uint32_t b[kVec];
    float off = 0.f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const float r = __fmaf_rn(x[j], inv, kMagic);
        off = fmaxf(off, fabsf(__fmaf_rn(x[j], inv, kMagic - r)));
        b[j] = __float_as_uint(r);
    }
    if (!normal || off > kNear) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const float r = __fmaf_rn(x[j], inv, kMagic);
            if (!normal || fabsf(__fmaf_rn(x[j], inv, kMagic - r)) > kNear) b[j] = (uint32_t)exact_quotient(x[j], scale);
        }
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        w[h] = __byte_perm(__byte_perm(b[4 * h], b[4 * h + 1], 0x0040), __byte_perm(b[4 * h + 2], b[4 * h + 3], 0x0040),
                           0x5410);
    return make_uint2(w[0], w[1]);
}

// threads_per_row (a multiple of 32) threads work on a row; a block holds
// blockDim.x / threads_per_row rows.  KEEP: the row fits the registers;
// otherwise it is read a second time.
template <bool F32, bool KEEP>
__global__ void __launch_bounds__(1024)
    quantize(const void* x_in, int64_t M, int K, int threads_per_row, int8_t* q, float* row_scale)
{
    __shared__ uint32_t part[32];
    // The next kernel may start once this one has seen the previous one's end:
    // what it reads early was then written two kernels ago at the latest.
    ptx::pdl_wait_prior_grid();
    ptx::pdl_launch_dependents();
    // The previous kernel may be writing x until the wait is over: coherent loads, whose
    // address comes from behind it (x is no __restrict__ parameter, which would allow
    // read-only loads in front of it).
    const void* x = ptx::after_wait(static_cast<const uint8_t*>(x_in));
    const int r = threadIdx.x / threads_per_row, t = threadIdx.x % threads_per_row;
    const int64_t m = (int64_t)blockIdx.x * (blockDim.x / threads_per_row) + r;
    const bool live = m < M;
    const int64_t row = m * K;
    const int n = K / kVec;

    Raw<F32> v[KEEP ? kMaxVecs : 1];
    uint32_t top = 0;
    if (live) {
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < kMaxVecs; ++i)
                if (t + i * threads_per_row < n) v[i].load(x, row + (int64_t)(t + i * threads_per_row) * kVec);
#pragma unroll
            for (int i = 0; i < kMaxVecs; ++i)
                if (t + i * threads_per_row < n) top = max(top, v[i].top());
        } else {
#pragma unroll 4
            for (int at = t; at < n; at += threads_per_row) {
                v[0].load(x, row + (int64_t)at * kVec);
                top = max(top, v[0].top());
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
    const bool normal = scale >= 1.17549435e-38f;
    if (t == 0) row_scale[m] = scale;
    auto put = [&](int at, const Raw<F32>& raw) {
        float f[kVec];
        raw.floats(f);
        *reinterpret_cast<uint2*>(q + row + (int64_t)at * kVec) =
            zero ? make_uint2(0, 0) : quotients(f, scale, inv, normal);
    };
    if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < kMaxVecs; ++i) {
            const int at = t + i * threads_per_row;
            if (at < n) put(at, v[i]);
        }
    } else {
#pragma unroll 2
        for (int at = t; at < n; at += threads_per_row) {
            v[0].load(x, row + (int64_t)at * kVec);
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
