// tile_gemm.cu -- tcgen05 GEMMs for any number of tokens:
//
//   experts:  y[r] = x[r] . W_e^T for the rows r of expert e (rows sorted by
//             expert, ragged), W_e packed NVFP4 or FP8, x FP16;
//   int8:     y[m][n] = (sum_k q[m][k] c[n][k]) * row_scale[m] * channel_scale[n].
//
// One kernel serves both.  The weights are the rows of the matrix instruction
// (128, or 256 of a pair of CTAs) and the tokens its columns, so one token
// costs 16 columns and a long batch 192 (int8: 256), and the same kernel runs
// from one row to many thousands.  Per CTA (one per SM, persistent):
//
//   W producer   one thread, bulk copies of packed 128 x 128 blocks (experts)
//                or tiled TMA boxes of the plain [N][K] matrix (int8);
//   x producer   one thread, tiled TMA boxes of the activations;
//   decoders     two groups of four warps (experts only): a thread owns one
//                weight row of a block and writes its decoded FP16 values
//                straight into tensor memory, from where the matrix
//                instruction reads operand A.  The decoded weights never pass
//                through shared memory, whose bandwidth would not carry them
//                at the rate the codes arrive from HBM (2 bytes written and 2
//                read per weight against 0.56 bytes of HBM traffic);
//   MMA          one thread issues tcgen05.mma into FP32 (int8: S32) accumulators;
//   epilogue     four or eight warps: a thread owns one output channel.
//
// Every product is exact (e2m1 * ue4m3 and e4m3 fit FP16, s8 * s8 fits S32);
// the FP32 sums round as the tensor core's accumulator does, the S32 sums not
// at all.  The scales are applied to the finished sum in FP32, and the output
// is rounded once.
//
// What bounds it, and what it measured on a B200 (6.46 TB/s copy, 1708 TFLOP/s
// bf16 in a burst, 1437 sustained; back-to-back launches in a CUDA graph,
// weights from HBM):
//   few rows, FP8     HBM: 64 rows over 128 experts of 5120 x 1408, 46 to 54 us
//                     for the 36 to 49 experts that they hit (6.0 to 6.5 TB/s).
//   few rows, NVFP4   the decoders: 64 rows over 128 experts of 2816 x 5120,
//                     61 to 74 us (4.7 to 5.4 TB/s); a block takes its two
//                     groups ~430 clocks, HBM ~390.
//   many rows         the tensor cores, after some half second under the power
//                     limit: 16387 rows over 32 experts of 2816 x 5120, 357 us
//                     at first and 421 at 1.35 GHz (1.32 and 1.12 PFLOP/s); int8
//                     2048 x 34816 x 5120, 297 us and 357 at 0.96 GHz (2.5 and
//                     2.0 POP/s).
//   hundreds of rows  launch, first loads and an epilogue, 6 to 8 us together, and
//                     the last round's idle SMs: 1003 rows over 32 experts of
//                     2051 x 2048, 26 to 31 us; int8 200 x 6000 x 4096, 15 us.
//   one token         latency: eight experts of 2816 x 2048 (23 MB) 12 to 13 us.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "../../include/skinny.h"
#include "tcgen05.cuh"

namespace skinny {
namespace {

constexpr int kRows = 128;            // weight rows per tile: the lanes of tensor memory
constexpr int kBlockK = 128;          // columns per packed block
constexpr int kFmtInt8 = 2;           // next to SKINNY_FMT_NVFP4 and SKINNY_FMT_FP8
constexpr int kMaxExperts = SKINNY_MAX_EXPERTS;
constexpr int kMaxDevices = 64;
constexpr int kSlotWords = kRows * 256;   // one CTA's partial tile in the workspace
constexpr int kAheadBlocks = 4;           // int8 weight blocks prefetched before the previous kernel is done
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// Bits of g_tile_error: which bounded wait gave up.
constexpr unsigned kErrRing = 1u;         // a full or empty ring slot
constexpr unsigned kErrAccumulator = 2u;  // an accumulator to be filled or drained
constexpr unsigned kErrPartial = 4u;      // another CTA's partial sums

__device__ unsigned int g_tile_error;

// A slot's flags in the workspace: one for each epilogue warp, set when that
// warp has published its rows and columns, and cleared by the one warp that
// reads them (the same warp of another CTA).  Zero between calls.
constexpr int kFlags = 8;

// Bytes of one packed 128 x 128 block.  A decoder thread reads its row's 128
// columns as 16-byte words, 128 rows side by side (no bank conflicts):
//   NVFP4  [4 words][128 rows][32 codes], then [128 rows][8 block scales]
//   FP8    [8 words][128 rows][16 codes]
__host__ __device__ constexpr int block_bytes(int fmt) { return fmt == SKINNY_FMT_NVFP4 ? 9216 : 16384; }
constexpr int kNvfp4BlockScales = 8192;

struct Params {
    const uint8_t* w;            // packed blocks (experts)
    const float* scale;          // NVFP4 [E]; FP8 [E][N]; int8 [N]
    const float* row_scale;      // int8 [T]
    const int32_t* offsets;      // experts [E + 1]
    void* y;                     // [T][outputs]
    unsigned* partials;          // workspace: [P][kSlotWords], then [P][kFlags] flags (or null)
    unsigned* flags;
    int T, N, K, E;
    int G, C;                    // row tiles, K blocks
    float rcp_C, rcp_groups;     // 1 / C, 1 / (row tiles, or pairs of them)
    int outputs;                 // outputs per token: N, or N / 2 (SiLU*mul)
    int out_f32;
};

constexpr int at_most(int a, int b) { return a < b ? a : b; }

// Tiles of more than 64 columns are computed by pairs of CTAs.
__host__ __device__ constexpr bool is_pair(int TN) { return TN > 64; }

// Columns that the matrix instruction of a tile with n tokens has: it takes
// multiples of 16, a pair's of 32.  Columns past n hold other tokens' rows, or
// zeros, and are not stored.
__host__ __device__ constexpr int columns(int n, bool pair)
{
    const int step = pair ? 32 : 16;
    return (n + step - 1) / step * step;
}

// A step is what one turn of every role handles: two K blocks of a narrow
// tile, one of a wide one.  Every turn of a decoder or of the MMA thread costs
// it some hundred clocks of waits, arrivals and commits beside its work, and a
// narrow step has to fit in the ~780 clocks in which its weights arrive from
// HBM: steps of half the size measured 93 us for 71 (64 rows, 128 experts) and
// 484 us for 396 (16387 rows).
template <int FMT, int TN>
struct Cfg {
    static constexpr bool kInt8 = FMT == kFmtInt8;
    // Wide tiles are computed by pairs of CTAs (a cluster): 256 weight rows, 128
    // in each CTA, and half the tokens' rows loaded by each.  One CTA by itself
    // would read 96 bytes (experts: 80) from L2 per clock of matrix instructions,
    // where an SM gets about 64.
    static constexpr bool kPair = is_pair(TN);
    static constexpr int kStepBlocks = kPair ? 1 : 2;
    static constexpr int kTokens = kPair ? TN / 2 : TN;                         // tokens in this CTA's slots
    static constexpr int kChunksPerBlock = kInt8 ? 1 : 2;                       // 128-byte wide pieces of x per block
    static constexpr int kChunks = kStepBlocks * kChunksPerBlock;               // pieces per step
    static constexpr int kWBytes = block_bytes(FMT) * kStepBlocks;              // a weight slot
    static constexpr int kChunkBytes = kTokens * 128;
    static constexpr int kXBytes = kChunkBytes * kChunks;                       // a token slot
    // A narrow tile's tokens arrive in one box per step, a wide one's in one or
    // two boxes for each chunk, as many as it has tokens (a box costs the
    // producer ~90 clocks, a step of a wide tile takes 500 to 700).
    static constexpr bool kX3d = !kPair;
    static constexpr bool kW3d = kInt8 && kStepBlocks == 2;
    static constexpr int kBox = kX3d ? TN : kTokens / 2;
    // Tensor memory: two accumulators at columns 0 and TN, then a stage of
    // decoded blocks, 64 columns a block, for each group of decoder warps.
    static constexpr int kDStages = 2;
    static constexpr int kGroups = kInt8 ? 0 : 2;
    static constexpr int kACol = 512 - 64 * kStepBlocks * kGroups;
    static constexpr int kDecodeWarps = 4 * kGroups;
    // int8's wide tiles of few blocks are computed in less time than four warps
    // store them: 700 x 2048 with 12000 channels takes 24.1 us with eight, 25.5
    // with four; from 40 blocks on there is no difference.
    static constexpr int kEpilogueWarps = kInt8 && kPair ? 8 : 4;
    static constexpr int kWarps = 4 + kDecodeWarps + kEpilogueWarps;
    static constexpr int kThreads = kWarps * 32;
    // Ring slots.  Experts: weights first, up to what hides HBM's latency (150
    // KB; a wide tile asks for less), and the tokens' ring takes the rest.
    // int8 slots hold weights and tokens.
    static constexpr int kBudget = 218 * 1024;
    static constexpr int kWTarget = (kPair ? 96 : 150) * 1024;
    static constexpr int kWStages = kInt8 ? at_most(kBudget / (kWBytes + kXBytes), 12)
                                          : at_most((kBudget - 3 * kXBytes) / kWBytes, kWTarget / kWBytes);
    static constexpr int kXStages = kInt8 ? kWStages : at_most((kBudget - kWStages * kWBytes) / kXBytes, 12);
    // A group waits by parity for the copy of its step into a weight slot, which
    // is right only if the copy before it into that slot, kWStages steps ago, is
    // known to have landed: a wait that is a whole phase early passes.  A group
    // knows the copies of its own steps, and of every step up to kGroups before
    // its last one (it has waited for their matrix instructions), so the ring has
    // to hold 2 * kGroups steps, or a whole number of the groups' turns.  Where
    // shared memory has no room for it, a group first waits until its step's token
    // slot is free: the step kXStages ago is then done, and all before it.  (FP8's
    // 64 columns: 2000 rows over 64 experts of 4096 x 1408 take 74.0 us, with four
    // weight and two token slots instead 78.1; 1003 over 32 of 2051 x 2048 31.0, 33.3.)
    static constexpr bool kShortRing =
        !kInt8 && kWStages < 2 * kGroups && kWStages % (kGroups > 0 ? kGroups : 1) != 0;
    static_assert(!kShortRing || kXStages <= kWStages, "a free token slot says nothing of the weight slot's last copy");
    static constexpr int kXOff = 0;
    static constexpr int kWOff = kXStages * kXBytes;
    static constexpr int kBarOff = kWOff + kWStages * kWBytes;
    static constexpr int kBars = 2 * (kXStages + kWStages + kDStages) + kGroups + 1;
    static constexpr int kBytes = kBarOff + kBars * 8 + 1024;   // + alignment of the dynamic shared memory
    static_assert(kBytes + 8 * (kMaxExperts + 2) + 256 <= 232448, "shared memory per CTA");
    static_assert(kDStages * TN <= kACol, "accumulators and decoded blocks overlap");
    static_assert(kChunkBytes % 1024 == 0 && kWBytes % 1024 == 0 && kBox * 128 % 1024 == 0,
                  "swizzled tiles start on 1024 bytes");
    static_assert(kXStages >= 3 && kWStages >= 3, "rings");
    // A group that fills its stage again waits by parity for the token slot of its
    // last step, kGroups steps ago: the ring may not have come round in between.
    static_assert(kGroups <= kXStages, "a group's last token slot is in use again");
    // Two groups are what has been run and tested.  A version with three faulted on
    // FP8, whose ring of four slots holds less than two of their turns.
    static_assert(kInt8 || kGroups == 2, "groups of decoder warps");
    static_assert(columns(TN, kPair) == TN, "a full tile has no columns to spare");
};

// The tile sequence, from the experts' row counts: expert e has
// ceil(rows / TN) token tiles of q_e rows each (a whole number of the matrix
// instruction's steps, so the tiles of one expert are alike) times G row tiles.
struct Schedule {
    int tiles[kMaxExperts + 1];          // running number of tiles
    int rows[kMaxExperts + 1];           // running row offset (offsets made monotone and clamped to [0, T])
    int total;
    int splits, share, extra;            // see Walk
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ int token_tiles(int rows, int TN) { return (rows + TN - 1) / TN; }

// What a tile has of the weight's row tiles: one, or a pair's two.
template <bool PAIR>
__device__ __forceinline__ int row_groups(const Params& p)
{
    return PAIR ? (p.G + 1) / 2 : p.G;
}

// Largest e with a[e] <= v, 0 <= e < n (a[0] = 0, a ascending).
__device__ __forceinline__ int find(const int* a, int n, int v)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

// What a tile of TN columns takes, in ns: a block, the epilogue (what is left
// of a tile without blocks), and the exchange of partial sums where tiles are
// split.  Fitted to 27 shapes of both kinds, each run at every width.
struct TileCost {
    int block, epilogue, exchange;
};

__host__ __device__ constexpr TileCost tile_cost(int TN)
{
    return TN <= 16   ? TileCost{270, 1500, 1500}
           : TN <= 32 ? TileCost{270, 2000, 2000}
           : TN <= 64 ? TileCost{270, 3500, 3000}
           : TN <= 128 ? TileCost{320, 5000, 10000}
                       : TileCost{420, 6500, 20000};
}

// Which tiles are split, and how their blocks are shared out (see Walk).
template <int TN, bool PAIR>
__device__ __forceinline__ void finish_schedule(Schedule& s, const Params& p, int total)
{
    const int P = PAIR ? gridDim.x / 2 : gridDim.x;
    int splits = 0;
    if (p.partials != nullptr) {
        // The last round's `rest` tiles take C blocks' time if they are not
        // split, and rest * C / P and the exchange if they are.  A product of
        // 2048 x 5120 with 34816 channels takes 305 us with its rest whole and
        // 356 split, 2048 x 1024 with 1024 channels 16.6 and 27.4.
        const int rest = total % P;
        constexpr TileCost cost = tile_cost(TN);
        if (rest != 0 && (int64_t)p.C * (P - rest) * cost.block > (int64_t)cost.exchange * P)
            splits = 4 * rest >= P || total < P ? rest : rest + P;
    }
    s.total = total;
    s.splits = splits;
    s.share = splits * p.C / P;
    s.extra = splits * p.C % P;
}

// A piece of one CTA's work: K blocks [k0, k1) of a tile.
struct Segment {
    int e, row_tile, t0, n;   // expert, this CTA's row tile, first token row, token rows
    int tile, k0, k1;
};

// x / d for 0 <= x < 2^31 where the quotient is below 2^22; rcp = 1.f / d.
__device__ __forceinline__ int quotient(int x, int d, float rcp)
{
    int q = (int)((float)x * rcp);
    const int r = x - q * d;
    q += r >= d;
    q -= r < 0;
    return q;
}

// The CTA's pieces.  Whole tiles are dealt out one after another, so that the
// CTAs work on neighbouring tiles and share their operands in L2.  What would
// leave CTAs idle in the last round is split along K instead: the first
// `splits` tiles (the remainder, and one round more where the remainder is
// less than a quarter of a round, which would leave many CTAs on one tile) are
// cut into equal contiguous ranges of blocks, one per CTA, and the partial
// sums of a cut tile meet in the workspace.  They come first, so that the
// exchange is hidden behind the whole tiles, and a range is walked backwards,
// so that the sums another CTA waits for come first of all.
// A pair of CTAs counts as one here.
template <int TN, bool PAIR>
struct Walk {
    const Schedule& s;
    const Params& p;
    int P, self;        // CTAs (or pairs) of the grid, and which this is
    int u0, u;          // this CTA's first split block, and one past the next piece's last
    int tile;           // the next whole tile

    __device__ Walk(const Schedule& s_, const Params& p_) : s(s_), p(p_)
    {
        P = PAIR ? gridDim.x / 2 : gridDim.x;
        self = PAIR ? blockIdx.x / 2 : blockIdx.x;
        u0 = start(self);
        u = start(self + 1);
        tile = s.splits + self;
    }
    // split blocks: CTA b has share + (b < extra)
    __device__ int start(int b) const { return b * s.share + (b < s.extra ? b : s.extra); }
    // the workspace slot that this CTA reads of CTA (or pair) b
    __device__ int slot(int b) const { return PAIR ? 2 * b + (int)(blockIdx.x & 1) : b; }
    __device__ bool empty(int b) const { return s.share == 0 && b >= s.extra; }
    __device__ bool next(Segment& g)
    {
        if (u > u0) {
            g.tile = quotient(u - 1, p.C, p.rcp_C);
            g.k1 = u - g.tile * p.C;
            g.k0 = u0 > g.tile * p.C ? u0 - g.tile * p.C : 0;
            u = g.tile * p.C + g.k0;
        } else {
            if (tile >= s.total) return false;
            g.tile = tile;
            g.k0 = 0;
            g.k1 = p.C;
            tile += P;
        }
        g.e = find(s.tiles, p.E, g.tile);
        const int m = s.rows[g.e + 1] - s.rows[g.e];
        int q = m;
        if (m > TN) {
            const int nt = token_tiles(m, TN);
            q = columns((m + nt - 1) / nt, PAIR);
        }
        const int lt = g.tile - s.tiles[g.e];
        const int groups = row_groups<PAIR>(p), tt = quotient(lt, groups, p.rcp_groups), rt = lt - tt * groups;
        g.row_tile = PAIR ? rt * 2 + (int)(blockIdx.x & 1) : rt;
        const int t = tt * q;
        g.t0 = s.rows[g.e] + t;
        g.n = m - t < q ? m - t : q;
        return true;
    }
};

// A ring position.
struct Ring {
    int i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int n)
    {
        if (++i == n) {
            i = 0;
            phase ^= 1;
        }
    }
};

__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned code)
{
    // the clock only after some tries: reading it costs more than a short wait
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((i & 31u) == 0) {
            if (*abort) return false;
            const uint64_t now = ptx::globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitLimitNs) {
                *abort = 1;
                atomicOr(&g_tile_error, code);
                return false;
            }
        }
    }
}

// False once any wait of the CTA has given up: every role then stops.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* abort, unsigned code)
{
    if (ptx::mbar_try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, abort, code);
}

// Waits for a producer's copies in flight: the last `issued` slots before
// position r, at most one round.
__device__ __noinline__ void drain(Ring r, int issued, int stages, uint64_t* full)
{
    for (int k = issued < stages ? issued : stages; k > 0; --k) {
        if (r.i == 0) {
            r.i = stages;
            r.phase ^= 1;
        }
        --r.i;
        ptx::mbar_wait(full + r.i, r.phase, kWaitLimitNs);
    }
}

// The same for a whole warp, whose lanes leave the wait together: the loop's
// condition is a vote, so the warp cannot be apart when it comes to the
// tensor-memory loads and stores, which all lanes must execute as one.
__device__ __noinline__ bool wait_warp_slow(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned code)
{
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (__all_sync(~0u, ptx::mbar_try_wait(bar, parity))) return true;
        if ((i & 31u) == 0) {
            const uint64_t now = ptx::globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (__any_sync(~0u, now - t0 > kWaitLimitNs)) {
                *abort = 1;
                atomicOr(&g_tile_error, code);
            }
            if (__any_sync(~0u, *abort != 0)) return false;
        }
    }
}

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* abort, unsigned code)
{
    if (__all_sync(~0u, ptx::mbar_try_wait(bar, parity))) return true;
    return wait_warp_slow(bar, parity, abort, code);
}

template <int FMT, int TN>
struct Shared {
    using C = Cfg<FMT, TN>;
    uint8_t* base;
    __device__ uint8_t* x(int i) const { return base + C::kXOff + i * C::kXBytes; }
    __device__ uint8_t* w(int i) const { return base + C::kWOff + i * C::kWBytes; }
    __device__ uint64_t* bars() const { return reinterpret_cast<uint64_t*>(base + C::kBarOff); }
    // full: the copies have landed (a pair's tokens: those of both CTAs, in the
    // leader's x_full, as the instruction reads both).  x_empty: the step's matrix
    // instructions are done (which also frees the decoded stage that they read, and
    // int8's weights).
    __device__ uint64_t* x_full(int i) const { return bars() + i; }
    __device__ uint64_t* x_empty(int i) const { return bars() + C::kXStages + i; }
    __device__ uint64_t* w_full(int i) const { return bars() + 2 * C::kXStages + i; }
    __device__ uint64_t* w_empty(int i) const { return bars() + 2 * C::kXStages + C::kWStages + i; }
    __device__ uint64_t* d_full(int i) const { return bars() + 2 * (C::kXStages + C::kWStages) + i; }
    __device__ uint64_t* d_empty(int i) const { return d_full(i) + C::kDStages; }
    __device__ uint64_t* a_full(int i) const { return bars() + 2 * (C::kXStages + C::kWStages + C::kDStages) + i; }
    __device__ uint64_t* drained() const { return bars() + C::kBars - 1; }
};

// Inclusive running maximum / sum over the block's threads' values.
__device__ __forceinline__ int warp_scan_max(int v)
{
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(~0u, v, d);
        if ((threadIdx.x & 31) >= d) v = v > o ? v : o;
    }
    return v;
}
__device__ __forceinline__ uint32_t warp_scan_add(uint32_t v)
{
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t o = __shfl_up_sync(~0u, v, d);
        if ((threadIdx.x & 31) >= d) v += o;
    }
    return v;
}

// The experts' schedule, by one warp: a lane takes neighbouring experts.
// Offsets are device data that the host has not seen: they are clamped to
// [0, T] and made non-decreasing, so no row is outside x and y or has two experts.
template <int TN, bool PAIR>
__device__ void make_schedule(Schedule& s, const Params& p)
{
    const int lane = threadIdx.x & 31, per = (p.E + 31) / 32;
    const int e0 = lane * per < p.E ? lane * per : p.E, e1 = e0 + per < p.E ? e0 + per : p.E;
    auto clamp = [&](int v) { return v < 0 ? 0 : v > p.T ? p.T : v; };
    const int first = clamp(p.offsets[0]);
    int top = first;
    for (int e = e0; e < e1; ++e) {
        const int v = clamp(p.offsets[e + 1]);
        top = top > v ? top : v;
        s.rows[e + 1] = top;
    }
    int before = __shfl_up_sync(~0u, warp_scan_max(top), 1);
    before = lane == 0 ? first : before;
    const int groups = row_groups<PAIR>(p);
    int prev = before, n = 0;
    for (int e = e0; e < e1; ++e) {
        const int v = s.rows[e + 1] > before ? s.rows[e + 1] : before;
        s.rows[e + 1] = v;
        n += token_tiles(v - prev, TN) * groups;
        s.tiles[e + 1] = n;
        prev = v;
    }
    const int run = (int)warp_scan_add((uint32_t)n);
    for (int e = e0; e < e1; ++e) s.tiles[e + 1] += run - n;
    if (lane == 0) {
        s.rows[0] = first;
        s.tiles[0] = 0;
    }
    if (lane == 31) finish_schedule<TN, PAIR>(s, p, run);
    __syncwarp();
}

// Stores r[0..n) at y[at], y[at + step], ...  A branch around each store made
// a tile of 192 columns 10000 clocks, longer than 20 blocks of it: 8192 rows, 4
// experts of 2048 x 256 took 34.8 us for 20.1 with predicates.
template <int N>
__device__ __forceinline__ void put_column(void* y, int64_t at, int step, const float (&r)[N], int n, int f32)
{
    if (f32) {
        float* p = static_cast<float*>(y) + at;
#pragma unroll
        for (int j = 0; j < N; ++j, p += step) ptx::st_global_if(p, r[j], j < n);
    } else {
        __half* p = static_cast<__half*>(y) + at;
#pragma unroll
        for (int j = 0; j < N; ++j, p += step) ptx::st_global_if(p, __float2half_rn(r[j]), j < n);
    }
}

// One row's 128 columns of a packed block (shared-memory address `src`) to
// FP16, two to a word, in two halves.
template <int FMT>
__device__ __forceinline__ void decode(uint32_t src, int row, uint32_t (&v)[2][32])
{
    if constexpr (FMT == SKINNY_FMT_NVFP4) {
        uint32_t sc[2];
        ptx::lds64(src + kNvfp4BlockScales + row * 8, sc);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 c0 = ptx::lds128(src + (2 * h * kRows + row) * 16);
            const uint4 c1 = ptx::lds128(src + ((2 * h + 1) * kRows + row) * 16);
            uint32_t s01, s23;
            ptx::e4m3x4_to_f16x4(sc[h], s01, s23);
            const uint32_t sd[4] = {ptx::dup_lo(s01), ptx::dup_hi(s01), ptx::dup_lo(s23), ptx::dup_hi(s23)};
            const uint32_t words[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t f[4];
                ptx::e2m1x8_to_f16x8(words[i], f);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[h][4 * i + j] = ptx::hmul2(f[j], sd[i / 2]);
            }
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 w = ptx::lds128(src + ((4 * h + i) * kRows + row) * 16);
                ptx::e4m3x4_to_f16x4(w.x, v[h][8 * i], v[h][8 * i + 1]);
                ptx::e4m3x4_to_f16x4(w.y, v[h][8 * i + 2], v[h][8 * i + 3]);
                ptx::e4m3x4_to_f16x4(w.z, v[h][8 * i + 4], v[h][8 * i + 5]);
                ptx::e4m3x4_to_f16x4(w.w, v[h][8 * i + 6], v[h][8 * i + 7]);
            }
    }
}

// Adds the other CTAs' partial sums of a tile (slots of CTAs or pairs self - 1
// down to `lowest`) to this warp's rows of the accumulator, SLOTS slots and
// COLS columns at a time.
template <bool INT8, int SLOTS, int COLS, int TURNS, int TN, bool PAIR>
__device__ __forceinline__ void add_partials(const Params& p, const Walk<TN, PAIR>& walk, int lowest, int row,
                                             int turn, int n, uint32_t acc)
{
#pragma unroll 1
    for (int c0 = turn * COLS; c0 < n; c0 += TURNS * COLS) {
        uint32_t v[COLS];
        ptx::tmem_ld(acc + c0, v);
        const int left = n - c0;
#pragma unroll 1
        for (int c = walk.self - 1; c >= lowest; c -= SLOTS) {
            uint32_t part[SLOTS][COLS];
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                const bool there = c - i >= lowest && !walk.empty(c - i);
                const unsigned* slot = p.partials + (int64_t)walk.slot(c - i) * kSlotWords + row + c0 * kRows;
#pragma unroll
                for (int j = 0; j < COLS; ++j) part[i][j] = ptx::ld_global_cg_if(slot + j * kRows, there && j < left);
            }
#pragma unroll
            for (int i = 0; i < SLOTS; ++i)
#pragma unroll
                for (int j = 0; j < COLS; ++j)
                    v[j] = INT8 ? v[j] + part[i][j]
                                : __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(part[i][j]));
        }
        ptx::tmem_st(acc + c0, v);
    }
    ptx::tmem_wait_st();
}

// The W producer's thread: weight slots in the order of the walk.
template <int FMT, int TN>
struct Producer {
    using C = Cfg<FMT, TN>;
    int u0, u, tile;      // the walk's position
    int k, k1;            // blocks of the current piece
    int rt;               // its row tile
    uint32_t pair_bytes;  // int8 pairs: what both CTAs' copies of a step bring
    const uint8_t* src;
    bool ok;

    __device__ __forceinline__ void begin(const Schedule& s, const Params& p)
    {
        const Walk<TN, C::kPair> w(s, p);
        u0 = w.u0, u = w.u, tile = w.tile;
        k = k1 = 0;
        ok = true;
    }
    // Fills slots until `most` have been issued or the walk ends.
    __device__ __forceinline__ void produce(const Shared<FMT, TN>& sm, Ring& r, int& issued, int most, Schedule& s,
                                            const Params& p, const CUtensorMap* w_map, const CUtensorMap* w_map2,
                                            bool leader)
    {
        const uint64_t pol = TN <= 32 ? ptx::policy_evict_first() : ptx::policy_evict_normal();
        while (ok && issued < most) {
            if (k >= k1) {
                Walk<TN, C::kPair> w(s, p);
                w.u = u, w.tile = tile;
                Segment g;
                if (!w.next(g)) {
                    ok = false;
                    return;
                }
                u = w.u, tile = w.tile;
                k = g.k0, k1 = g.k1;
                // (an odd last row tile has no partner: its pair's second CTA computes it too, and stores nothing)
                rt = C::kPair && g.row_tile >= p.G ? p.G - 1 : g.row_tile;
                src = C::kInt8 ? nullptr : p.w + ((size_t)g.e * p.G + rt) * p.C * block_bytes(FMT);
                pair_bytes = 2 * (C::kWBytes + (columns(g.n, true) / 2 + C::kBox - 1) / C::kBox * C::kBox * 128);
            }
            ok = wait(C::kInt8 ? sm.x_empty(r.i) : sm.w_empty(r.i), r.phase ^ 1, &s.abort, kErrRing);
            if (!ok) return;
            if constexpr (C::kInt8 && C::kPair) {
                // the leader's barrier counts both CTAs' weights and tokens
                uint64_t* full = sm.x_full(r.i);
                if (leader) ptx::mbar_arrive_expect_tx(full, pair_bytes);
                ptx::tma_load_2d_pair(sm.w(r.i), w_map, k * kBlockK, rt * kRows, ptx::leader_addr(full), pol);
            } else if constexpr (C::kInt8) {
                uint64_t* full = sm.x_full(r.i);
                ptx::mbar_arrive_expect_tx(full, C::kWBytes);
                if (C::kW3d && (k + 2) * kBlockK <= p.K) {
                    ptx::tma_load_3d(sm.w(r.i), w_map, 0, rt * kRows, k, full, pol);
                } else {
                    // plain boxes: past K they fill in zeros
                    for (int b = 0; b < C::kStepBlocks; ++b)
                        ptx::tma_load_2d(sm.w(r.i) + b * block_bytes(FMT), C::kW3d ? w_map2 : w_map, (k + b) * kBlockK,
                                         rt * kRows, full, pol);
                }
            } else {
                const uint32_t bytes = (C::kStepBlocks == 2 && k + 1 < k1 ? 2 : 1) * block_bytes(FMT);
                ptx::mbar_arrive_expect_tx(sm.w_full(r.i), bytes);
                ptx::bulk_g2s(sm.w(r.i), src + (size_t)k * block_bytes(FMT), bytes, sm.w_full(r.i), pol);
            }
            r.step(C::kWStages);
            ++issued;
            k += C::kStepBlocks;
        }
    }
};

template <int FMT, int TN, bool SILU>
__global__ void __launch_bounds__(Cfg<FMT, TN>::kThreads, 1)
    tile_gemm(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap x_map,
              const __grid_constant__ CUtensorMap x_map2, const __grid_constant__ CUtensorMap w_map,
              const __grid_constant__ CUtensorMap w_map2)
{
    using C = Cfg<FMT, TN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Schedule s;
    const Shared<FMT, TN> sm{smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u)};
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kXStages; ++i) {
            ptx::mbar_init(sm.x_full(i), C::kInt8 && !C::kPair ? 2 : 1);      // int8: both producers' copies
            ptx::mbar_init(sm.x_empty(i), 1);
        }
        for (int i = 0; i < C::kWStages; ++i) {
            ptx::mbar_init(sm.w_full(i), 1);
            ptx::mbar_init(sm.w_empty(i), 4);
        }
        for (int i = 0; i < C::kGroups; ++i) ptx::mbar_init(sm.a_full(i), C::kPair ? 8 : 4);
        for (int i = 0; i < C::kDStages; ++i) {
            ptx::mbar_init(sm.d_full(i), 1);
            ptx::mbar_init(sm.d_empty(i), C::kEpilogueWarps * (C::kPair ? 2 : 1));
        }
        ptx::mbar_init(sm.drained(), 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&x_map);
        ptx::prefetch_tensormap(&x_map2);
        if (C::kInt8) ptx::prefetch_tensormap(&w_map);
        s.abort = 0;
    }
    if (warp == 2) ptx::tmem_alloc_all<C::kPair>(&s.tmem);
    __syncwarp();
    const int rank = C::kPair ? (int)ptx::cluster_rank() : 0;
    const bool leader = rank == 0;
    // The next kernel may start once this one has seen the previous one's end
    // (what it reads early was then written two kernels ago at the latest).
    if constexpr (C::kInt8) {
        // The schedule needs nothing of the previous kernel: only the roles
        // that touch its results wait for it.
        if (threadIdx.x == 0) {
            s.rows[0] = 0;
            s.rows[1] = p.T;
            s.tiles[0] = 0;
            s.tiles[1] = token_tiles(p.T, TN) * row_groups<C::kPair>(p);
            finish_schedule<TN, C::kPair>(s, p, s.tiles[1]);
        }
    } else {
        ptx::pdl_wait_prior_grid();
        ptx::pdl_launch_dependents();
        if (warp == 0) make_schedule<TN, C::kPair>(s, p);
    }
    Ring r;            // position of a single-thread role, and how much it has issued
    int issued = 0;
    // The single-thread roles run under elect.sync, which tells the compiler
    // that one thread is active: a matrix instruction of 16 columns then issues
    // every 9 clocks, under `lane == 0` every 68 (measured on B200).
    bool mine = false;
    Producer<FMT, TN> producer;
    if (!C::kInt8 && warp == 0 && ptx::elect_one()) {
        // the warp that made the schedule starts on its ring before the CTA is
        // ready: with two slots, as a copy takes ~160 ns to issue.  The other
        // CTA of a pair would wait for them: 62.5 us for 58.5 (8192 rows, 64
        // experts of 2048 x 1024).
        producer.begin(s, p);
        if (!C::kPair) producer.produce(sm, r, issued, 2, s, p, &w_map, &w_map2, leader);
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if constexpr (C::kPair) ptx::cluster_sync();      // the other CTA's barriers are ready, too
    ptx::tc_fence_after();
    const uint32_t tmem = s.tmem;
    Walk<TN, C::kPair> walk(s, p);
    Segment g;

    if (warp == 0) {
        // ---- W producer
        if (ptx::elect_one()) {
            mine = true;
            if constexpr (C::kInt8) {
                // Until the previous kernel is done, the weights are only brought into L2: they
                // are a plain tensor that it may have written.
                Walk<TN, C::kPair> ahead(s, p);
                if (ahead.next(g) && g.row_tile < p.G)
                    for (int k = g.k0; k < g.k1 && k < g.k0 + kAheadBlocks; ++k)
                        ptx::tma_prefetch_2d(C::kW3d ? &w_map2 : &w_map, k * kBlockK, g.row_tile * kRows);
                ptx::pdl_wait_prior_grid();
                producer.begin(s, p);
            }
            producer.produce(sm, r, issued, 0x7FFFFFFF, s, p, &w_map, &w_map2, leader);
        }
    } else if (warp == 1) {
        // ---- x producer
        if (ptx::elect_one()) {
            mine = true;
            bool ok = true;
            const uint64_t pol = TN <= 32 ? ptx::policy_evict_last() : ptx::policy_evict_normal();
            if (C::kInt8) {
                ptx::pdl_wait_prior_grid();
                ptx::pdl_launch_dependents();
            }
            constexpr int kChunkK = kBlockK / C::kChunksPerBlock;
            const int whole = p.K / kChunkK;      // pieces that lie within K entirely
            while (ok && walk.next(g)) {
                const int c1 = g.k1 * C::kChunksPerBlock;
                // a pair's CTA has half the tile's columns
                const int half = columns(g.n, C::kPair) / 2, first = g.t0 + rank * half;
                const int boxes = (half + C::kBox - 1) / C::kBox;
                for (int c = g.k0 * C::kChunksPerBlock; c < c1; c += C::kChunks) {
                    ok = wait(sm.x_empty(r.i), r.phase ^ 1, &s.abort, kErrRing);
                    if (!ok) break;
                    if constexpr (C::kX3d) {
                        // one box of kChunks pieces; where K ends inside one, a box for each
                        // piece, which fills in zeros past K
                        ptx::mbar_arrive_expect_tx(sm.x_full(r.i), C::kXBytes);
                        const int last = c + C::kChunks < c1 ? c + C::kChunks : c1;
                        if (last <= whole) {
                            ptx::tma_load_3d(sm.x(r.i), &x_map, 0, g.t0, c, sm.x_full(r.i), pol);
                        } else {
                            for (int b = 0; b < C::kChunks; ++b)
                                ptx::tma_load_2d(sm.x(r.i) + b * C::kChunkBytes, &x_map2, (c + b) * kChunkK, g.t0,
                                                 sm.x_full(r.i), pol);
                        }
                    } else {
                        // both CTAs' copies report to the leader's barrier (int8: the W producer announces them)
                        if (!C::kInt8 && leader)
                            ptx::mbar_arrive_expect_tx(sm.x_full(r.i), 2 * C::kChunks * boxes * C::kBox * 128);
                        for (int h = 0; h < C::kChunks; ++h)
                            for (int b = 0; b < boxes; ++b) {
                                uint8_t* dst = sm.x(r.i) + h * C::kChunkBytes + b * C::kBox * 128;
                                ptx::tma_load_2d_pair(dst, &x_map, (c + h) * kChunkK, first + b * C::kBox,
                                                      ptx::leader_addr(sm.x_full(r.i)), pol);
                            }
                    }
                    r.step(C::kXStages);
                    ++issued;
                }
            }
        }
    } else if (warp == 2) {
        // ---- MMA: one thread issues (a pair's: the leader's)
        if (leader && ptx::elect_one()) {
            mine = true;
            if (C::kInt8) ptx::pdl_wait_prior_grid();      // so that no bounded wait runs against another kernel
            Ring dr;
            constexpr uint32_t kXStep = C::kXBytes >> 4, kXChunkStep = C::kChunkBytes >> 4;
            constexpr uint32_t kAStep = C::kInt8 ? C::kWBytes >> 4 : 64 * C::kStepBlocks;
            constexpr uint32_t kAChunkStep = C::kInt8 ? block_bytes(FMT) >> 4 : 32;
            const uint32_t x0 = ptx::smem_desc_low(ptx::smem_addr(sm.x(0)));
            const uint32_t a0 = C::kInt8 ? ptx::smem_desc_low(ptx::smem_addr(sm.w(0))) : tmem + C::kACol;
            uint32_t xd = x0, ad = a0;
            int stage = 0;              // decoded stage (experts)
            uint32_t a_phase = 0;
            bool ok = true;
            while (ok && walk.next(g)) {
                ok = wait(sm.d_empty(dr.i), dr.phase ^ 1, &s.abort, kErrAccumulator);
                if (!ok) break;
                const int cols = columns(g.n, C::kPair);
                const uint32_t d = tmem + dr.i * TN;
                constexpr int kM = C::kPair ? 2 * kRows : kRows;
                const uint32_t idesc = C::kInt8 ? ptx::idesc_s8(kM, cols) : ptx::idesc_f16(kM, cols);
                uint32_t add = 0;
                for (int k = g.k0; k < g.k1; k += C::kStepBlocks) {
                    if constexpr (C::kInt8) ok = wait(sm.x_full(r.i), r.phase, &s.abort, kErrRing);
                    else ok = wait(sm.a_full(stage), a_phase, &s.abort, kErrRing);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const bool full = C::kStepBlocks == 1 || k + 1 < g.k1;
#pragma unroll
                    for (int c = 0; c < C::kChunks; ++c) {
                        if (c >= C::kChunksPerBlock && !full) break;
                        const uint32_t a = ad + c * kAChunkStep, b = xd + c * kXChunkStep;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if constexpr (C::kInt8) ptx::mma_s8_ss<C::kPair>(d, a + 2 * j, b + 2 * j, idesc, c + j ? 1u : add);
                            else ptx::mma_f16_ts<C::kPair>(d, a + 8 * j, b + 2 * j, idesc, c + j ? 1u : add);
                        }
                    }
                    add = 1;
                    ptx::tc_commit<C::kPair>(sm.x_empty(r.i));
                    r.step(C::kXStages);
                    xd = r.i == 0 ? x0 : xd + kXStep;
                    if constexpr (C::kInt8) {
                        ad = r.i == 0 ? a0 : ad + kAStep;
                    } else {
                        if (++stage == C::kGroups) {
                            stage = 0;
                            a_phase ^= 1;
                        }
                        ad = stage == 0 ? a0 : ad + kAStep;
                    }
                }
                if (!ok) break;
                ptx::tc_commit<C::kPair>(sm.d_full(dr.i));
                dr.step(C::kDStages);
            }
        }
    } else if (warp >= 4 && warp < 4 + C::kDecodeWarps) {
        // ---- decoders: thread = weight row (warp % 4, lane); the two groups take steps in turn
        if constexpr (!C::kInt8) {
            Ring wr, xr, done;      // done: the token slot of this group's last step
            const int row = (warp & 3) * 32 + lane;
            const int group = (warp - 4) >> 2;      // fills decoded stage `group`
            const uint32_t dst = tmem + ((uint32_t)(warp & 3) << 21) + C::kACol + group * 64 * C::kStepBlocks;
            int turn = group;                       // steps until this group's next
            bool first = true, ok = true;
            while (ok && walk.next(g)) {
                for (int k = g.k0; k < g.k1; k += C::kStepBlocks) {
                    if (turn == 0) {
                        turn = C::kGroups;
                        if constexpr (C::kShortRing) {
                            ok = wait_warp(sm.x_empty(xr.i), xr.phase ^ 1, &s.abort, kErrRing);
                            if (!ok) break;
                        }
                        ok = wait_warp(sm.w_full(wr.i), wr.phase, &s.abort, kErrRing);
                        if (!ok) break;
                        const uint32_t src = ptx::smem_addr(sm.w(wr.i));
                        const int blocks = C::kStepBlocks == 1 || k + 1 == g.k1 ? 1 : 2;
#pragma unroll
                        for (int b = 0; b < C::kStepBlocks; ++b) {
                            if (b >= blocks) break;
                            uint32_t v[2][32];
                            decode<FMT>(src + b * block_bytes(FMT), row, v);
                            if (b == 0 && !first) {
                                // the stage is free when the matrix instructions of the group's last step
                                // are done: the conversion does not wait for them
                                ok = wait_warp(sm.x_empty(done.i), done.phase, &s.abort, kErrRing);
                                if (!ok) break;
                            }
                            ptx::tc_fence_after();
                            ptx::tmem_st(dst + b * 64, v[0]);
                            ptx::tmem_st(dst + b * 64 + 32, v[1]);
                        }
                        if (!ok) break;
                        first = false;
                        done = xr;
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(sm.w_empty(wr.i));
                        ptx::tmem_wait_st();
                        ptx::tc_fence_before();
                        // one warp (a pair's: of the leader) waits for the tokens too, on the MMA thread's behalf
                        if ((warp & 3) == 0 && leader) ok = wait_warp(sm.x_full(xr.i), xr.phase, &s.abort, kErrRing);
                        if (!ok) break;
                        __syncwarp();
                        if (lane == 0) {
                            if constexpr (C::kPair) ptx::mbar_arrive_leader(sm.a_full(group));
                            else ptx::mbar_arrive(sm.a_full(group));
                        }
                    }
                    --turn;
                    wr.step(C::kWStages);
                    xr.step(C::kXStages);
                }
            }
        }
    } else if (warp >= 4 + C::kDecodeWarps) {
        // ---- epilogue: thread = output channel (warp % 4, lane)
        Ring dr;
        const int q = warp & 3, row = q * 32 + lane;
        // the chunks of columns that this warp stores: one in kTurns
        constexpr int kTurns = C::kEpilogueWarps / 4;
        const int turn = (warp - 4 - C::kDecodeWarps) >> 2;
        const uint32_t src = tmem + ((uint32_t)q << 21);
        bool ok = true;
        if (C::kInt8) ptx::pdl_wait_prior_grid();
        while (ok && walk.next(g)) {
            const bool publish = g.k1 < p.C;
            // This thread's channel and scale.  SiLU*mul tiles hold 16 gate
            // rows and their 16 up rows in the two halves of every warp.
            const int o = SILU ? g.row_tile * 64 + q * 16 + (lane & 15) : g.row_tile * kRows + row;
            const bool valid = o < p.outputs;
            float scale = 0.f;      // loaded while the tile is computed
            if (valid && !publish) {
                if (FMT == SKINNY_FMT_NVFP4) scale = p.scale[g.e];
                else if (FMT == SKINNY_FMT_FP8)
                    scale = p.scale[(size_t)g.e * p.N + o + (SILU && lane >= 16 ? p.outputs : 0)];
                else scale = p.scale[o];
            }
            // Narrow tiles go by few columns at a time: the loop's code is short (a first pass
            // through it comes from memory) and one token costs one turn.
            constexpr int kCols = TN <= 16 ? 8 : TN <= 64 ? 16 : 32;
            constexpr int kNext = kCols * kTurns;
            const int c_first = turn * kCols;
            // the row scales of all its chunks, of each chunk's column `lane`
            constexpr int kMine = TN / kNext;
            float rs[kMine] = {};
            if (C::kInt8 && !publish) {
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const int c = c_first + i * kNext + lane;
                    if (c < g.n) rs[i] = p.row_scale[g.t0 + c];
                }
            }
            ok = wait_warp(sm.d_full(dr.i), dr.phase, &s.abort, kErrAccumulator);
            if (!ok) break;
            ptx::tc_fence_after();
            int lowest = walk.self;     // first CTA (or pair) whose partial sums belong to this tile
            if (!publish && g.k0 > 0) {
                const int first = g.tile * p.C;
                while (lowest > 0 && walk.start(lowest) > first) --lowest;
                // lane i waits for the i-th CTA below, 32 at a time
                const uint64_t t0 = ptx::globaltimer_ns();
                for (int c = walk.self - 1; ok && c >= lowest; c -= 32) {
                    const int other = c - lane;
                    const bool there = other >= lowest && !walk.empty(other);
                    const unsigned* flag = p.flags + walk.slot(there ? other : c) * kFlags + turn * 4 + q;
                    while (!__all_sync(~0u, !there || ptx::ld_acquire_gpu(flag) != 0)) {
                        if (__any_sync(~0u, ptx::globaltimer_ns() - t0 > kWaitLimitNs)) {
                            s.abort = 1;
                            atomicOr(&g_tile_error, kErrPartial);
                        }
                        if (__any_sync(~0u, *(volatile int*)&s.abort != 0)) {
                            ok = false;
                            break;
                        }
                    }
                }
                __syncwarp();      // the other lanes' loads follow what each lane has acquired
                if (!ok) break;
            }
            const uint32_t acc = src + dr.i * TN;
            // Other CTAs' sums are added to the accumulator, from the nearest CTA down (a fixed
            // order), with 32 loads in flight per thread: four CTAs' for few tokens, else 32 tokens'.
            if (lowest < walk.self) {
                if (TN > 16 && g.n > 8) add_partials<C::kInt8, 1, 32, kTurns>(p, walk, lowest, row, turn, g.n, acc);
                else add_partials<C::kInt8, 4, 8, kTurns>(p, walk, lowest, row, turn, g.n, acc);
            }
#pragma unroll 1
            for (int c0 = c_first; c0 < g.n; c0 += kNext) {
                uint32_t v[kCols];
                ptx::tmem_ld(acc + c0, v);
                const int left = g.n - c0;
                if (publish) {
                    unsigned* slot = p.partials + (size_t)blockIdx.x * kSlotWords + row + c0 * kRows;
#pragma unroll
                    for (int j = 0; j < kCols; ++j) ptx::st_global_if(slot + j * kRows, v[j], j < left);
                    continue;
                }
                // y of this thread's channel at the chunk's first token
                const int64_t at = (int64_t)(g.t0 + c0) * p.outputs + o;
                if constexpr (SILU) {
                    float r[kCols / 2];
#pragma unroll
                    for (int j = 0; j < kCols; j += 2) {
                        // lanes 0..15 finish token j, lanes 16..31 token j + 1
                        const float a = __uint_as_float(v[j]) * scale, b = __uint_as_float(v[j + 1]) * scale;
                        const float other = __shfl_xor_sync(~0u, lane < 16 ? b : a, 16);
                        const float gate = lane < 16 ? a : other, up = lane < 16 ? other : b;
                        r[j / 2] = gate / (1.f + expf(-gate)) * up;
                    }
                    put_column<kCols / 2>(p.y, at + (lane >> 4) * p.outputs, 2 * p.outputs, r,
                                          valid ? (left + 1 - (lane >> 4)) / 2 : 0, p.out_f32);
                } else {
                    float r[kCols];
#pragma unroll
                    for (int j = 0; j < kCols; ++j) {
                        if constexpr (C::kInt8) r[j] = (float)(int)v[j] * __shfl_sync(~0u, rs[0], j) * scale;
                        else r[j] = __uint_as_float(v[j]) * scale;
                    }
                    put_column<kCols>(p.y, at, p.outputs, r, valid ? left : 0, p.out_f32);
                }
#pragma unroll
                for (int i = 1; i < kMine; ++i) rs[i - 1] = rs[i];
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (C::kPair) ptx::mbar_arrive_leader(sm.d_empty(dr.i));
                else ptx::mbar_arrive(sm.d_empty(dr.i));
            }
            dr.step(C::kDStages);
            if (publish) {
                if (lane == 0) ptx::st_release_gpu(p.flags + blockIdx.x * kFlags + turn * 4 + q, 1);
            } else {
                for (int c = walk.self - 1 - lane; c >= lowest; c -= 32) p.flags[walk.slot(c) * kFlags + turn * 4 + q] = 0;
            }
        }
    }

    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (s.abort && mine) {
        // A wait gave up: copies and matrix instructions may still be in
        // flight.  Let them end before the memory they use is given up.
        if (warp == 0 && !C::kInt8) drain(r, issued, C::kWStages, sm.w_full(0));
        if (warp == (C::kInt8 ? 0 : 1) && leader) drain(r, issued, C::kXStages, sm.x_full(0));
        if (warp == 2) {
            ptx::tc_commit<C::kPair>(sm.drained());
            ptx::mbar_wait(sm.drained(), 0, kWaitLimitNs);
        }
    }
    if (s.abort) __syncthreads();
    if constexpr (C::kPair) {
        // neither CTA's barriers go away while the other may still arrive on them
        __syncwarp();
        ptx::cluster_sync();
    }
    if (warp == 2) ptx::tmem_free_all<C::kPair>(tmem);
}

// Packs experts on the device: a CTA per block, a thread per 16 bytes of its codes.
__global__ void pack_experts(int fmt, const uint8_t* codes, const uint8_t* scales, int N, int K, int outputs, int G,
                             int Cb, int gate_up, uint8_t* packed)
{
    const int wb = block_bytes(fmt);
    const int64_t blk = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;   // (e * G + g) * Cb + c
    const int c = (int)(blk % Cb);
    const int64_t eg = blk / Cb;
    const int g = (int)(eg % G);
    const int64_t e = eg / G;
    uint8_t* out = packed + blk * wb;
    const int row_bytes = fmt == SKINNY_FMT_NVFP4 ? K / 2 : K;
    const int chunk_bytes = fmt == SKINNY_FMT_NVFP4 ? 64 : 128;
    const int words = chunk_bytes / 16;
    // the source row of packed row r, or -1 past the outputs
    auto source = [&](int r) -> int64_t {
        const int l = r & 31;
        const int o = gate_up ? g * 64 + (r / 32) * 16 + (l & 15) : g * kRows + r;
        return o < outputs ? e * N + o + (gate_up && l >= 16 ? outputs : 0) : -1;
    };
    // neighbouring threads read along a row; rows are multiples of 8 bytes
    for (int i = threadIdx.x; i < kRows * words; i += blockDim.x) {
        const int j = i % words, r = i / words, at = c * chunk_bytes + j * 16;
        const int64_t n = source(r);
        uint2 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            v[h] = n >= 0 && at + 8 * h < row_bytes
                       ? *reinterpret_cast<const uint2*>(codes + n * row_bytes + at + 8 * h)
                       : make_uint2(0, 0);
        *reinterpret_cast<uint4*>(out + (j * kRows + r) * 16) = make_uint4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
    if (fmt == SKINNY_FMT_NVFP4) {
        for (int i = threadIdx.x; i < kRows * 8; i += blockDim.x) {
            const int b = i % 8, r = i / 8, at = c * 8 + b;
            const int64_t n = source(r);
            out[kNvfp4BlockScales + i] = n >= 0 && at < K / 16 ? scales[n * (K / 16) + at] : 0;
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct DeviceState {
    bool ready = false;
    int sms = 0;
};
std::mutex g_mu;
DeviceState g_dev[kMaxDevices];
EncodeTiled g_encode = nullptr;

// Widest token tile: two accumulators, and (experts) two decoded blocks, fill
// the tensor memory.
template <int FMT>
constexpr int kWidest = FMT == kFmtInt8 ? 256 : 192;

template <int FMT, int TN, bool SILU>
bool allow_smem()
{
    return cudaFuncSetAttribute(tile_gemm<FMT, TN, SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg<FMT, TN>::kBytes) == cudaSuccess;
}

template <int FMT, bool SILU>
bool allow_smem_all()
{
    return allow_smem<FMT, 16, SILU>() && allow_smem<FMT, 32, SILU>() && allow_smem<FMT, 64, SILU>() &&
           allow_smem<FMT, 128, SILU>() && allow_smem<FMT, kWidest<FMT>, SILU>();
}

// SM count of the current device; on its first use, the kernels' shared
// memory limits and the tensor-map encoder.
int current_device(int* sms)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SKINNY_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState& d = g_dev[dev];
    if (!d.ready) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            return SKINNY_ERR_CUDA;
        if (!g_encode) {
            void* fn = nullptr;
            cudaDriverEntryPointQueryResult found;
            if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
                    cudaSuccess ||
                found != cudaDriverEntryPointSuccess || !fn)
                return SKINNY_ERR_CUDA;
            g_encode = reinterpret_cast<EncodeTiled>(fn);
        }
        if (!allow_smem_all<SKINNY_FMT_NVFP4, false>() || !allow_smem_all<SKINNY_FMT_NVFP4, true>() ||
            !allow_smem_all<SKINNY_FMT_FP8, false>() || !allow_smem_all<SKINNY_FMT_FP8, true>() ||
            !allow_smem_all<kFmtInt8, false>())
            return SKINNY_ERR_CUDA;
        d.sms = n;
        d.ready = true;
    }
    *sms = d.sms;
    return SKINNY_OK;
}

// A row-major [rows][cols] matrix read in boxes of 128 bytes x box_rows rows,
// or (pieces > 1) in boxes of `pieces` of these side by side in K, each a tile
// of its own in shared memory: the matrix is then seen as [cols / 128 bytes]
// pieces of rows, without the columns that fill no piece.
bool make_map(CUtensorMap* map, const void* base, bool f16, int64_t rows, int64_t cols, int box_rows, int pieces)
{
    const cuuint64_t pitch = (cuuint64_t)cols * (f16 ? 2 : 1);
    const cuuint32_t wide = f16 ? 64u : 128u;
    const cuuint64_t whole = (cuuint64_t)cols / wide;
    const bool split = pieces > 1;
    // Fewer columns than one piece: no box of this kind is read.
    if (split && whole == 0) return make_map(map, base, f16, rows, cols, box_rows, 1);
    const cuuint64_t dims[3] = {split ? wide : (cuuint64_t)cols, (cuuint64_t)rows, whole};
    const cuuint64_t strides[2] = {pitch, 128};
    const cuuint32_t box[3] = {wide, (cuuint32_t)box_rows, (cuuint32_t)pieces};
    const cuuint32_t unit[3] = {1, 1, 1};
    return g_encode(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, split ? 3 : 2,
                    const_cast<void*>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t workspace_size(int sms) { return (size_t)sms * (kSlotWords + kFlags) * 4; }

template <int FMT, int TN, bool SILU>
int launch(Params p, const void* x, const void* w, int grid, cudaStream_t stream)
{
    using C = Cfg<FMT, TN>;
    p.rcp_C = 1.f / p.C;
    p.rcp_groups = 1.f / (C::kPair ? (p.G + 1) / 2 : p.G);
    CUtensorMap xm, xm2, wm, wm2;
    if (!make_map(&xm, x, !C::kInt8, p.T, p.K, C::kBox, C::kX3d ? C::kChunks : 1)) return SKINNY_ERR_CUDA;
    wm = wm2 = xm2 = xm;
    // (read only where K ends inside a block)
    if (C::kX3d && p.K % kBlockK != 0 && !make_map(&xm2, x, !C::kInt8, p.T, p.K, C::kBox, 1)) return SKINNY_ERR_CUDA;
    if (C::kInt8) {
        if (!make_map(&wm, w, false, p.N, p.K, kRows, C::kW3d ? 2 : 1)) return SKINNY_ERR_CUDA;
        if (C::kW3d && !make_map(&wm2, w, false, p.N, p.K, kRows, 1)) return SKINNY_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    if (C::kPair && grid % 2 != 0) cfg.gridDim.x = --grid;
    if (grid == 0) return SKINNY_ERR_UNSUPPORTED;
    cfg.attrs = attr;
    cfg.numAttrs = C::kPair ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, tile_gemm<FMT, TN, SILU>, p, xm, xm2, wm, wm2) == cudaSuccess ? SKINNY_OK : SKINNY_ERR_CUDA;
}

// The time of a launch with tiles of TN tokens by tile_cost: in whole rounds
// or with its last round split, whichever the kernel will take.
int64_t launch_time(const Params& p, int TN, int grid)
{
    const TileCost cost = tile_cost(TN);
    const int64_t pair = is_pair(TN) ? 2 : 1, P = std::max<int64_t>(grid / pair, 1);
    // an expert's last tile is half full on average
    const int64_t columns = p.E == 1 ? ((int64_t)p.T + TN - 1) / TN
                                     : std::max<int64_t>(std::min(p.E, p.T), p.T / TN + p.E / 2);
    const int64_t tiles = columns * ((p.G + pair - 1) / pair);
    const int64_t tile = std::max<int64_t>((int64_t)p.C * cost.block, cost.epilogue);
    const int64_t whole = (tiles + P - 1) / P * tile + cost.epilogue;
    if (p.partials == nullptr) return whole;
    return std::min(whole, tiles * tile / P + cost.epilogue + cost.exchange);
}

// Token columns per tile.  Narrow tiles leave the shared memory to the weights'
// ring (the memory-bound range); wide ones reuse each decoded block more often.
template <int FMT>
int tile_width(const Params& p, int grid)
{
    constexpr int widest = kWidest<FMT>;
    // What a tile would like to hold.  Routers load experts unevenly: twice the mean.
    const int64_t rows = FMT == kFmtInt8 || p.T <= 32 ? p.T : 2 * (((int64_t)p.T + p.E - 1) / p.E);
    if (rows <= 16) return 16;
    if (rows <= 32) return 32;
    if (rows <= 64) return 64;
    // More tokens: a wide tile reads the weights fewer times, a narrower one
    // leaves fewer SMs idle where wide tiles are few.  Of those that do not
    // exceed the tokens, the one with the least time by tile_cost: 200 x 4096
    // with 6000 channels takes 15.8 us with 128 and 18.9 with 256, 2048 x 5120
    // with 34816 channels 460 with 128 and 305 with 256.
    const int64_t t64 = launch_time(p, 64, grid);
    const int64_t t128 = launch_time(p, 128, grid);
    const int64_t wide = rows <= 128 ? INT64_MAX : launch_time(p, widest, grid);
    if (wide <= t64 && wide <= t128) return widest;
    return t128 <= t64 ? 128 : 64;
}

template <int FMT, bool SILU>
int launch_any(const Params& p, const void* x, const void* w, int grid, cudaStream_t stream)
{
    switch (tile_width<FMT>(p, grid)) {
    case 16: return launch<FMT, 16, SILU>(p, x, w, grid, stream);
    case 32: return launch<FMT, 32, SILU>(p, x, w, grid, stream);
    case 64: return launch<FMT, 64, SILU>(p, x, w, grid, stream);
    case 128: return launch<FMT, 128, SILU>(p, x, w, grid, stream);
    default: return launch<FMT, kWidest<FMT>, SILU>(p, x, w, grid, stream);
    }
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxK = int64_t(1) << 20, kMaxN = int64_t(1) << 24, kMaxTokens = int64_t(1) << 24;

int check_sizes(int64_t T, int64_t K, int64_t N)
{
    if (T < 0 || K <= 0 || K % 16 != 0 || N <= 0) return SKINNY_ERR_INVALID_ARG;
    if (T > kMaxTokens || K > kMaxK || N > kMaxN) return SKINNY_ERR_UNSUPPORTED;
    return SKINNY_OK;
}

// Fills in the sizes; SILU*mul has half as many outputs as weight rows.
int set_sizes(Params* p, int64_t T, int64_t K, int64_t N, int64_t E, bool silu)
{
    p->T = (int)T;
    p->N = (int)N;
    p->K = (int)K;
    p->E = (int)E;
    p->outputs = (int)(silu ? N / 2 : N);
    p->G = (p->outputs + (silu ? 63 : kRows - 1)) / (silu ? 64 : kRows);
    p->C = (int)((K + kBlockK - 1) / kBlockK);
    // the running number of tiles is a 32-bit count
    return (T / 16 + E) * (int64_t)p->G < (int64_t(1) << 31) ? SKINNY_OK : SKINNY_ERR_UNSUPPORTED;
}

// Fills in the workspace.
int set_workspace(Params* p, void* workspace, size_t bytes, int sms)
{
    p->partials = nullptr;
    p->flags = nullptr;
    if (!workspace) return SKINNY_OK;
    if (bytes < workspace_size(sms)) return SKINNY_ERR_WORKSPACE;
    p->partials = static_cast<unsigned*>(workspace);
    p->flags = p->partials + (size_t)sms * kSlotWords;
    return SKINNY_OK;
}

int experts(int fmt, const void* x, int64_t T, int64_t K, const int32_t* offsets, int64_t E, const void* w_packed,
            const float* scale, int64_t N, bool silu, void* y, int out_dtype, void* workspace, size_t workspace_bytes,
            void* stream)
{
    if (fmt != SKINNY_FMT_NVFP4 && fmt != SKINNY_FMT_FP8) return SKINNY_ERR_INVALID_ARG;
    if (out_dtype != SKINNY_OUT_F16 && out_dtype != SKINNY_OUT_F32) return SKINNY_ERR_INVALID_ARG;
    if (E <= 0 || (silu && N % 2 != 0)) return SKINNY_ERR_INVALID_ARG;
    if (const int rc = check_sizes(T, K, N)) return rc;
    if (E > kMaxExperts) return SKINNY_ERR_UNSUPPORTED;
    if (T == 0) return SKINNY_OK;
    if (!x || !offsets || !w_packed || !scale || !y) return SKINNY_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w_packed, 16) || !aligned(offsets, 4) || !aligned(scale, 4) ||
        !aligned(y, out_dtype == SKINNY_OUT_F32 ? 4 : 2) || (workspace && !aligned(workspace, 16)))
        return SKINNY_ERR_ALIGNMENT;
    Params p{};
    p.w = static_cast<const uint8_t*>(w_packed);
    p.scale = scale;
    p.offsets = offsets;
    p.y = y;
    p.out_f32 = out_dtype == SKINNY_OUT_F32;
    if (const int rc = set_sizes(&p, T, K, N, E, silu)) return rc;
    int sms = 0;
    if (const int rc = current_device(&sms)) return rc;
    if (const int rc = set_workspace(&p, workspace, workspace_bytes, sms)) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (fmt == SKINNY_FMT_NVFP4)
        return silu ? launch_any<SKINNY_FMT_NVFP4, true>(p, x, nullptr, sms, st)
                    : launch_any<SKINNY_FMT_NVFP4, false>(p, x, nullptr, sms, st);
    return silu ? launch_any<SKINNY_FMT_FP8, true>(p, x, nullptr, sms, st)
                : launch_any<SKINNY_FMT_FP8, false>(p, x, nullptr, sms, st);
}

bool experts_shape(int fmt, int64_t E, int64_t N, int64_t K, int gate_up, int64_t* G, int64_t* C)
{
    if (fmt != SKINNY_FMT_NVFP4 && fmt != SKINNY_FMT_FP8) return false;
    if (E <= 0 || E > kMaxExperts || N <= 0 || N > kMaxN || K <= 0 || K > kMaxK || K % 16 != 0) return false;
    if (gate_up && N % 2 != 0) return false;
    *G = gate_up ? (N / 2 + 63) / 64 : (N + kRows - 1) / kRows;
    *C = (K + kBlockK - 1) / kBlockK;
    return true;
}

}  // namespace
}  // namespace skinny

using namespace skinny;

extern "C" size_t skinny_experts_packed_bytes(int fmt, int64_t E, int64_t N, int64_t K, int gate_up)
{
    int64_t G, C;
    return experts_shape(fmt, E, N, K, gate_up, &G, &C) ? (size_t)(E * G * C) * block_bytes(fmt) : 0;
}

extern "C" int skinny_pack_experts(int fmt, const void* codes, const void* scales, int64_t E, int64_t N, int64_t K,
                                   int gate_up, void* w_packed, void* stream)
{
    int64_t G, C;
    if (!experts_shape(fmt, E, N, K, gate_up, &G, &C)) return SKINNY_ERR_INVALID_ARG;
    if (!codes || !w_packed || (fmt == SKINNY_FMT_NVFP4 && !scales)) return SKINNY_ERR_INVALID_ARG;
    if (!aligned(w_packed, 16) || !aligned(codes, 8)) return SKINNY_ERR_ALIGNMENT;
    if (E * G >= 65536 * int64_t(1024)) return SKINNY_ERR_UNSUPPORTED;
    // block index = x + y * gridDim.x over exactly E * G * C blocks
    int64_t gx = E * G * C, gy = 1;
    if (gx >= (int64_t(1) << 31)) {
        gx = E * G;
        gy = C;
    }
    pack_experts<<<dim3((unsigned)gx, (unsigned)gy), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        fmt, static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), (int)N, (int)K,
        (int)(gate_up ? N / 2 : N), (int)G, (int)C, gate_up, static_cast<uint8_t*>(w_packed));
    return cudaGetLastError() == cudaSuccess ? SKINNY_OK : SKINNY_ERR_CUDA;
}

extern "C" int skinny_tile_workspace_bytes(size_t* bytes)
{
    if (!bytes) return SKINNY_ERR_INVALID_ARG;
    int sms = 0;
    if (const int rc = current_device(&sms)) return rc;
    *bytes = workspace_size(sms);
    return SKINNY_OK;
}

extern "C" int skinny_gemm_experts(int fmt, const void* x, int64_t T, int64_t K, const int32_t* offsets, int64_t E,
                                   const void* w_packed, const float* scale, int64_t N, void* y, int out_dtype,
                                   void* workspace, size_t workspace_bytes, void* stream)
{
    return experts(fmt, x, T, K, offsets, E, w_packed, scale, N, false, y, out_dtype, workspace, workspace_bytes,
                   stream);
}

extern "C" int skinny_gemm_experts_silu_mul(int fmt, const void* x, int64_t T, int64_t K, const int32_t* offsets,
                                            int64_t E, const void* w_packed, const float* scale, int64_t F, void* y,
                                            int out_dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    if (F <= 0 || F > kMaxN / 2) return SKINNY_ERR_INVALID_ARG;
    return experts(fmt, x, T, K, offsets, E, w_packed, scale, 2 * F, true, y, out_dtype, workspace, workspace_bytes,
                   stream);
}

extern "C" int skinny_int8_gemm(const void* q, const float* row_scale, int64_t M, int64_t K, const void* w,
                                const float* channel_scale, int64_t N, void* y, int out_dtype, void* workspace,
                                size_t workspace_bytes, void* stream)
{
    if (out_dtype != SKINNY_OUT_F16 && out_dtype != SKINNY_OUT_F32) return SKINNY_ERR_INVALID_ARG;
    if (const int rc = check_sizes(M, K, N)) return rc;
    if (K > SKINNY_MAX_INT8_K) return SKINNY_ERR_UNSUPPORTED;
    if (M == 0) return SKINNY_OK;
    if (!q || !row_scale || !w || !channel_scale || !y) return SKINNY_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(w, 16) || !aligned(row_scale, 4) || !aligned(channel_scale, 4) ||
        !aligned(y, out_dtype == SKINNY_OUT_F32 ? 4 : 2) || (workspace && !aligned(workspace, 16)))
        return SKINNY_ERR_ALIGNMENT;
    Params p{};
    p.scale = channel_scale;
    p.row_scale = row_scale;
    p.y = y;
    p.out_f32 = out_dtype == SKINNY_OUT_F32;
    if (const int rc = set_sizes(&p, M, K, N, 1, false)) return rc;
    int sms = 0;
    if (const int rc = current_device(&sms)) return rc;
    if (const int rc = set_workspace(&p, workspace, workspace_bytes, sms)) return rc;
    return launch_any<kFmtInt8, false>(p, q, w, sms, static_cast<cudaStream_t>(stream));
}

extern "C" int skinny_debug_tile_width(int fmt, int64_t T, int64_t K, int64_t N, int64_t E, int gate_up,
                                       int workspace, int sms, int* width)
{
    const bool int8 = fmt == -1, silu = gate_up != 0;
    if (!width || sms <= 0 || (!int8 && fmt != SKINNY_FMT_NVFP4 && fmt != SKINNY_FMT_FP8)) return SKINNY_ERR_INVALID_ARG;
    if (T == 0 || E <= 0 || (int8 && (E != 1 || silu)) || (silu && N % 2 != 0)) return SKINNY_ERR_INVALID_ARG;
    if (const int rc = check_sizes(T, K, N)) return rc;
    if (E > kMaxExperts || (int8 && K > SKINNY_MAX_INT8_K)) return SKINNY_ERR_UNSUPPORTED;
    Params p{};
    if (const int rc = set_sizes(&p, T, K, N, E, silu)) return rc;
    unsigned there;      // (only whether there is a workspace counts)
    p.partials = workspace ? &there : nullptr;
    *width = int8 ? tile_width<kFmtInt8>(p, sms)
             : fmt == SKINNY_FMT_NVFP4 ? tile_width<SKINNY_FMT_NVFP4>(p, sms) : tile_width<SKINNY_FMT_FP8>(p, sms);
    return SKINNY_OK;
}

namespace {
template <int FMT, int TN>
int rings(int* out)
{
    using C = Cfg<FMT, TN>;
    out[0] = C::kWStages;
    out[1] = C::kXStages;
    out[2] = C::kGroups;
    out[3] = C::kShortRing;
    return SKINNY_OK;
}

template <int FMT>
int rings_of(int width, int* out)
{
    return width == 16    ? rings<FMT, 16>(out)
           : width == 32  ? rings<FMT, 32>(out)
           : width == 64  ? rings<FMT, 64>(out)
           : width == 128 ? rings<FMT, 128>(out)
           : width == kWidest<FMT> ? rings<FMT, kWidest<FMT>>(out) : SKINNY_ERR_INVALID_ARG;
}
}  // namespace

extern "C" int skinny_debug_tile_rings(int fmt, int width, int* out)
{
    if (!out) return SKINNY_ERR_INVALID_ARG;
    return fmt == -1                  ? rings_of<kFmtInt8>(width, out)
           : fmt == SKINNY_FMT_NVFP4 ? rings_of<SKINNY_FMT_NVFP4>(width, out)
           : fmt == SKINNY_FMT_FP8   ? rings_of<SKINNY_FMT_FP8>(width, out) : SKINNY_ERR_INVALID_ARG;
}

extern "C" int skinny_debug_tile_columns(int width, int rows)
{
    if (width != 16 && width != 32 && width != 64 && width != 128 && width != 192 && width != 256) return -1;
    return rows >= 1 && rows <= width ? columns(rows, is_pair(width)) : -1;
}

extern "C" int skinny_tile_device_error(int clear, unsigned* flags)
{
    if (!flags) return SKINNY_ERR_INVALID_ARG;
    if (cudaDeviceSynchronize() != cudaSuccess) return SKINNY_ERR_CUDA;
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_tile_error, sizeof(v)) != cudaSuccess) return SKINNY_ERR_CUDA;
    *flags = v;
    if (clear) {
        const unsigned zero = 0;
        if (cudaMemcpyToSymbol(g_tile_error, &zero, sizeof(zero)) != cudaSuccess) return SKINNY_ERR_CUDA;
    }
    return SKINNY_OK;
}
