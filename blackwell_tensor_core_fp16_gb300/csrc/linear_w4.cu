// A linear layer of few tokens with 4-bit weights and group scales (C ABI in include/decode.h):
//
//     y[i][j] = act(bias[j] + sum_g s[j][g] sum_{c in g} x[i][c] (code[j][c] - z[j][g]))
//
// A weight is half a byte and takes part in 2 m operations, so for a few tokens HBM bounds the time,
// and what a weight costs in instructions on its way to the matrix units decides whether it does: the
// SMs have to take 47 of them a clock each.
//
// Work split.  A block takes 128 outputs (rows of the weights), 16 a warp, and 8 kTiles tokens, over a
// part of the columns; the blocks of a cluster share the columns out and add their sums through
// distributed shared memory, in a fixed order.  The rows' codes come through a ring of shared-memory
// stages of 256 columns (16-byte cp.async), and beside them the tokens' elements, which all warps read.
//
// The codes are the matrix instructions' first operand (m16n8k16, the rows its 16 rows, the tokens its
// 8 columns).  A lane's 32-bit word holds 8 neighbouring columns; a mask leaves two of them, 16 bits
// apart, as the last bits of two 16-bit numbers whose upper bits an `or` makes 2^7 (bfloat16) or 2^10
// (float16), from which the zero point, lifted the same way, is subtracted: exact, both being whole
// numbers of at most 5 bits.  So columns c and c + 4 are a step's neighbours, and the tokens' elements
// are put into that order once, in their stage, by the threads that loaded them.  The scale is left out of the product:
// each group's sums, of exact products in fp32, are multiplied by it and added to the running ones in
// fp32, so no weight is ever rounded.
#include "decode_mma.cuh"
#include "desc.h"
#include "ptx.cuh"

namespace {

using namespace decode;

constexpr int kRows = 128;                       // outputs of a block for more tokens
constexpr int kMostSplit = 8;
constexpr int kSumRow = kRows + 4;               // floats of a token's sums; the pad spreads the banks

struct LinearParams {
    const uint16_t* x;
    const uint8_t* codes;
    const uint16_t* scales;
    const uint8_t* zeros;
    const uint16_t* bias;
    uint16_t* y;
    int64_t x_stride, code_stride, scale_stride, zero_stride, y_stride;
    int32_t m, n, k, group, group_shift, split, activation;
    uint32_t* status;
    int32_t items_each, items_more, pieces_each, pieces_more, stages, waiting;    // for few tokens
};

// (x & mask) | magic in one instruction
__device__ __forceinline__ uint32_t pick(uint32_t x, uint32_t mask, uint32_t magic)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(mask), "r"(magic));
    return r;
}

// A row's zero point, as the differences need it, and the differences of a word's 8 columns: pairs
// (c, c + 4) for c = 0 .. 3.
template <typename T>
struct Differences;
template <>
struct Differences<__nv_bfloat16> {
    uint32_t zero;                               // twice 2^7 + z
    __device__ __forceinline__ void set(uint32_t z) { zero = (z & 15u) * 0x10001u | 0x43004300u; }
    __device__ __forceinline__ uint32_t less(uint32_t x) const
    {
        uint32_t r;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(zero));
        return r;
    }
    __device__ __forceinline__ void of(uint32_t word, uint32_t (&to)[4]) const
    {
#pragma unroll
        for (int c = 0; c < 4; ++c) to[c] = less(pick(word >> 4 * c, 0x000f000fu, 0x43004300u));
    }
};
template <>
struct Differences<__half> {
    uint32_t zero, above;                        // twice 2^10 + z; twice -(2^6 + z)
    __device__ __forceinline__ void set(uint32_t z)
    {
        zero = (z & 15u) * 0x10001u | 0x64006400u;
        above = (z & 15u) * 0x00100010u | 0xd400d400u;
    }
    __device__ __forceinline__ void of(uint32_t word, uint32_t (&to)[4]) const
    {
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
            const uint32_t x = word >> 4 * c;
            const uint32_t lo = pick(x, 0x000f000fu, 0x64006400u);
            // the next column's bits stand four higher: 2^10 + 16 code, a sixteenth of which is 2^6 + code
            const uint32_t hi = pick(x, 0x00f000f0u, 0x64006400u);
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(to[c]) : "r"(lo), "r"(zero));
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(to[c + 1]) : "r"(hi), "r"(0x2c002c00u), "r"(above));
        }
    }
};

// A token's 8 columns in the order of the differences: pairs (c, c + 4).
__device__ __forceinline__ uint4 sorted(const uint4& x)
{
    return make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                      __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
}

__device__ __forceinline__ float activated(float y, int activation)
{
    if (activation == DECODE_ACT_RELU) return y < 0.f ? 0.f : y;
    if (activation == DECODE_ACT_GELU) return y * normcdff(y);
    return y;
}

// ---- few tokens ------------------------------------------------------------------------------------
//
// Up to 8 tokens.  The tokens' elements fit shared memory, all of a block's columns, so nothing but the
// codes streams.  A block takes 16 outputs at a time (an item) and 2048 of their columns (a stage): their
// 16 rows come by bulk copies, a row each, into a ring of stages, with none of the SM's threads busy on the
// way.  Of a stage's 16 pieces of 128 columns each of eight warps takes two; its sums of an item go to
// shared memory, where the warps' are added after several items.  Two blocks an SM stay and take equal
// shares of the items; the blocks of a cluster share the columns out where there are few items, or where
// the tokens' elements would not fit.

constexpr int kFewWarps = 8, kFewThreads = kFewWarps * 32;
constexpr int kItem = 16;                        // outputs
constexpr int kPieces = 2 * kFewWarps;           // of a stage, of 128 columns
constexpr int kFewRow = kPieces * 64 + 64;       // bytes of a stage's row; two rows' 64 bytes lie in
                                                 // different banks
constexpr int kFewStage = kItem * kFewRow;
constexpr int kMostStages = 5;
constexpr int kFewMost = 233472 / 2 - 1024 - 2 * kMostStages * 8 - 16;   // bytes for elements, sums, stages
constexpr uint64_t kTimeout = 2000000000;        // ns that a copy may take

__device__ __forceinline__ void bulk_copy(uint32_t to, const void* from, uint32_t bytes, uint32_t barrier)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(to), "l"(from), "r"(bytes), "r"(barrier) : "memory");
}

// kWords: neighbouring 32-bit words of a row that a lane takes at once; four lanes' are columns of one
// scale, and as many of those as make up 128 columns are a piece.
template <typename T, int kWords>
__global__ void __launch_bounds__(kFewThreads, 2) linear_w4_few_kernel(const LinearParams p)
{
    constexpr int kParts = 4 / kWords;           // of a piece, each with a scale
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, q = lane & 3, r = lane >> 2;
    const int part = cluster_rank(), at = cluster_id();
    // the block's items and pieces, shares of all
    const int item0 = at * p.items_each + min(at, p.items_more);
    const int item1 = item0 + p.items_each + (at < p.items_more);
    const int piece0 = part * p.pieces_each + min(part, p.pieces_more);
    const int piece1 = piece0 + p.pieces_each + (part < p.pieces_more);
    // stages of an item (one, empty, without columns)
    const int rounds = max(1, (piece1 - piece0 + kPieces - 1) / kPieces);
    const int steps = (item1 - item0) * rounds;
    // (the same in all of a cluster's blocks; 64 bytes more than a multiple of 128 a token, as a row)
    const int pitch = (p.pieces_each + (p.pieces_more > 0)) * 256 + 64;
    // ring, sums, elements, barriers: a stage's copies have come; all warps have read it
    const uint32_t ring = smem_addr(smem);
    float* const sums = reinterpret_cast<float*>(smem + p.stages * kFewStage);
    const int item_sums = p.m * kItem;                              // a warp's
    uint8_t* const xs = reinterpret_cast<uint8_t*>(sums + p.waiting * kFewWarps * item_sums);
    uint64_t* const bars = reinterpret_cast<uint64_t*>(xs + p.m * pitch);
    const uint32_t full = smem_addr(bars), empty = full + kMostStages * 8;
    volatile uint32_t* const gave_up = reinterpret_cast<uint32_t*>(bars + 2 * kMostStages);
    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) {
            gf16::mbar_init(full + s * 8, 1);
            gf16::mbar_init(empty + s * 8, kFewWarps);
        }
        *gave_up = 0;
        gf16::fence_mbarrier_init();
    }
    __syncwarp();                                // (the other warps: before their first wait, below)
    dep_launch();
    dep_wait();

    auto wait = [&](uint32_t barrier, uint32_t parity) {
        if (gf16::mbar_wait(barrier, parity, gave_up, kTimeout)) return;
        *gave_up = 1;                            // nothing waits any more; the results are no results
        atomicOr(p.status, DECODE_TIMED_OUT);
    };
    // the copies of a step, by the first warp: rows past the last output are the last one's
    int next_item = item0, next_round = 0;
    auto fetch = [&](int stage, bool again, uint32_t parity) {
        if (next_item >= item1) return;
        const int first = piece0 + next_round * kPieces;
        const int columns = min(p.k, min(piece1, first + kPieces) * 128) - first * 128;
        if (again) wait(empty + stage * 8, parity);
        if (columns > 0) {
            if (lane == 0) gf16::mbar_arrive_expect_tx(full + stage * 8, kItem * (columns / 2));
            __syncwarp();
            if (lane < kItem)
                bulk_copy(ring + stage * kFewStage + lane * kFewRow,
                          p.codes + static_cast<int64_t>(min(next_item * kItem + lane, p.n - 1)) *
                                        p.code_stride + first * 64,
                          columns / 2, full + stage * 8);
        } else if (lane == 0) {
            gf16::mbar_arrive_local(full + stage * 8);
        }
        if (++next_round == rounds) {
            next_round = 0;
            ++next_item;
        }
    };
    if (w == 0)
        for (int s = 0; s < p.stages; ++s) fetch(s, false, 0);

    // Scales and zero points of a step: lane x has those of row x % 16 and the warp's piece x / 16; on
    // their way one step ahead, a scale's bits below its zero point.
    uint32_t scale[kParts], zero[kParts];
    int scale_item = item0, scale_round = 0;
    auto load_scales = [&]() {
        const int piece = piece0 + scale_round * kPieces + w + kFewWarps * (lane >> 4);
        const uint32_t row = min(scale_item * kItem + (lane & 15), p.n - 1);
#pragma unroll
        for (int x = 0; x < kParts; ++x) {
            const int column = piece * 128 + x * (32 * kWords);
            scale[x] = 0, zero[x] = 0;
            if (scale_item < item1 && piece < piece1 && column < p.k) {
                const uint32_t g = divide(column / 32, p.group, p.group_shift);
                scale[x] = p.scales[row * static_cast<uint32_t>(p.scale_stride) + g];
                zero[x] = p.zeros != nullptr ? p.zeros[row * static_cast<uint32_t>(p.zero_stride) + g] : 8u;
            }
        }
        if (++scale_round == rounds) {
            scale_round = 0;
            ++scale_item;
        }
    };
    load_scales();

    // ---- the tokens' elements, 8 columns at a time in the codes' order; of a scale's columns the lanes'
    // first 8, then their second ones and so on.  Zeros past the last column, whatever the codes there.
    const int units = (piece1 - piece0) * 16;
    constexpr int kBatch = 4;
    for (int i0 = tid; i0 < p.m * units; i0 += kFewThreads * kBatch) {
        uint4 x[kBatch];
        uint8_t* to[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = i0 + b * kFewThreads;
            to[b] = nullptr;
            if (i >= p.m * units) continue;
            const int token = i / units, u = i - token * units, in = u % (4 * kWords);
            const int column = (piece0 * 16 + u) * 8;
            x[b] = make_uint4(0u, 0u, 0u, 0u);
            if (column < p.k) x[b] = *reinterpret_cast<const uint4*>(p.x + token * p.x_stride + column);
            to[b] = xs + token * pitch + (u - in + in % kWords * 4 + in / kWords) * 16;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (to[b] != nullptr) *reinterpret_cast<uint4*>(to[b]) = sorted(x[b]);
    }
    __syncthreads();
    // (lanes without a token of their own read the last one's and have no result)
    const uint8_t* const mine = xs + min(r, p.m - 1) * pitch + w * 256 + q * 16;

    float sum[4] = {};
    int item = item0, round = 0, stage = 0, slot = 0;
    uint32_t parity = 0;
    for (int step = 0; step < steps; ++step) {
        uint32_t sz[kParts];
#pragma unroll
        for (int x = 0; x < kParts; ++x) sz[x] = scale[x] | zero[x] << 16;
        load_scales();
        wait(full + stage * 8, parity);
        const uint8_t* const from = smem + stage * kFewStage + r * kFewRow + w * 64;
        // the warp's pieces of the stage: kCount of them at once
        auto take = [&](auto count) {
            constexpr int kCount = decltype(count)::value;
            uint32_t word[kCount][2][4];         // piece, row
#pragma unroll
            for (int y = 0; y < kCount; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint8_t* const f = from + y * (kFewWarps * 64) + e * 8 * kFewRow;
                    if constexpr (kWords == 4) {
                        const uint4 b = *reinterpret_cast<const uint4*>(f + q * 16);
                        word[y][e][0] = b.x, word[y][e][1] = b.y, word[y][e][2] = b.z, word[y][e][3] = b.w;
                    } else if constexpr (kWords == 2) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint2 b = *reinterpret_cast<const uint2*>(f + x * 32 + q * 8);
                            word[y][e][2 * x] = b.x, word[y][e][2 * x + 1] = b.y;
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            word[y][e][x] = *reinterpret_cast<const uint32_t*>(f + x * 16 + q * 4);
                    }
                }
            __syncwarp();
            if (lane == 0) gf16::mbar_arrive_local(empty + stage * 8);
#pragma unroll
            for (int y = 0; y < kCount; ++y)
#pragma unroll
                for (int z = 0; z < kParts; ++z) {
                    Differences<T> diff[2];
                    float by[2], acc[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t got = __shfl_sync(0xffffffffu, sz[z], y * 16 + r + 8 * e);
                        by[e] = Half2<T>::unpack(got & 0xffffu).x;
                        diff[e].set(got >> 16);
                    }
#pragma unroll
                    for (int x = 0; x < kWords; ++x) {
                        uint32_t lower[4], upper[4];
                        diff[0].of(word[y][0][z * kWords + x], lower);
                        diff[1].of(word[y][1][z * kWords + x], upper);
                        const uint32_t a[2][4] = {{lower[0], upper[0], lower[1], upper[1]},
                                                  {lower[2], upper[2], lower[3], upper[3]}};
                        const uint4 b = *reinterpret_cast<const uint4*>(
                            mine + round * (kPieces * 256) + y * (kFewWarps * 256) + (z * kWords + x) * 64);
                        if (x == 0)
                            mma_first<T>(acc, a[0], b.x, b.y);
                        else
                            mma<T>(acc, a[0], b.x, b.y);
                        mma<T>(acc, a[1], b.z, b.w);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[e] = fmaf(acc[e], by[e >> 1], sum[e]);
                }
        };
        const int last = piece1 - (piece0 + round * kPieces + w);    // pieces from the warp's first one on
        if (last > kFewWarps)
            take(std::integral_constant<int, 2>());
        else if (last > 0)
            take(std::integral_constant<int, 1>());
        else if (lane == 0)
            gf16::mbar_arrive_local(empty + stage * 8);
        if (w == 0) fetch(stage, true, parity);
        if (++stage == p.stages) {
            stage = 0;
            parity ^= 1;
        }
        if (++round < rounds) continue;
        // ---- the item's end: [token][output] of the warp's sums
        round = 0;
        float* const to = sums + (slot * kFewWarps + w) * item_sums;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int token = q * 2 + (e & 1);
            if (token < p.m) to[token * kItem + r + 8 * (e >> 1)] = sum[e];
            sum[e] = 0.f;
        }
        ++item;
        if (++slot < p.waiting && item < item1) continue;
        // ---- enough of them: the warps' sums, and the cluster's blocks', in their order
        if (p.split > 1)
            cluster_barrier();
        else
            __syncthreads();
        const int first = item - slot;
        for (int i = part * kFewThreads + tid; i < slot * item_sums; i += p.split * kFewThreads) {
            const int in = i / item_sums, rest = i - in * item_sums, token = rest / kItem;
            const int output = (first + in) * kItem + rest % kItem;
            if (output >= p.n) continue;
            float y = 0.f;
            const float* const warps = sums + in * kFewWarps * item_sums + rest;
            for (int o = 0; o < p.split; ++o) {
                float parts[kFewWarps];
#pragma unroll
                for (int x = 0; x < kFewWarps; ++x)
                    parts[x] = p.split == 1
                                   ? warps[x * item_sums]
                                   : cluster_load(cluster_address(smem_addr(warps + x * item_sums), o));
#pragma unroll
                for (int x = 0; x < kFewWarps; ++x) y += parts[x];
            }
            if (p.bias != nullptr) y += Half2<T>::unpack(p.bias[output]).x;
            y = activated(y, p.activation);
            p.y[token * p.y_stride + output] = static_cast<uint16_t>(Half2<T>::pack(y, 0.f));
        }
        slot = 0;
        // (the others may still read this block's sums)
        if (p.split > 1)
            cluster_barrier();
        else if (item < item1)
            __syncthreads();
    }
    // after a wait that ran out: the copies in flight are waited for, once more
    if (*gave_up && w == 0)
        for (int step = max(0, steps - p.stages); step < steps; ++step)
            gf16::mbar_wait(full + step % p.stages * 8, step / p.stages & 1, nullptr, kTimeout);
}

// The kernel for few tokens; false if their elements do not fit it.
template <typename T, int kWords>
bool run_few(LinearParams p, int sms, cudaStream_t stream, int& rc)
{
    const int64_t items = (p.n + kItem - 1) / kItem, pieces = (p.k + 127) / 128;
    // The columns' parts: those with which the block with the most to do has the least, a block's beginning
    // and end counted as two stages, a cluster's as four.  What shared memory the elements and two stages
    // leave holds the sums of as many items as a block has, and more stages.
    int64_t best = -1, smem = 0, shares = 0;
    for (int split = 1; split <= kMostSplit && (split == 1 || split <= pieces); split *= 2) {
        const int64_t mine = (pieces + split - 1) / split;
        const int64_t most = 2 * sms / split < items ? 2 * sms / split : items, each = (items + most - 1) / most;
        const int64_t bytes = p.m * (mine * 256 + 64), sums = kFewWarps * p.m * kItem * 4;
        const int64_t stages = 2, room = kFewMost - bytes - stages * kFewStage;
        if (room < sums) continue;
        const int64_t cost = each * mine + (split > 1 ? 4 : 2) * kPieces;
        if (best >= 0 && cost >= best) continue;
        best = cost, p.split = split, shares = most;
        const int64_t waiting = room / sums < each ? room / sums : each;
        const int64_t more = (room - waiting * sums) / kFewStage;
        p.waiting = static_cast<int>(waiting);
        p.stages = static_cast<int>(stages + more < kMostStages ? stages + more : kMostStages);
        smem = bytes + waiting * sums + p.stages * kFewStage + 2 * kMostStages * 8 + 16;
    }
    if (best < 0) return false;
    p.items_each = static_cast<int>(items / shares), p.items_more = static_cast<int>(items % shares);
    p.pieces_each = static_cast<int>(pieces / p.split), p.pieces_more = static_cast<int>(pieces % p.split);
    static thread_local bool set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(dev < kMaxDevices && set[dev])) {
        e = cudaFuncSetAttribute(linear_w4_few_kernel<T, kWords>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, 233472 / 2 - 1024);
        if (e == cudaSuccess && dev < kMaxDevices) set[dev] = true;
    }
    if (e == cudaSuccess)
        e = launch_cluster(linear_w4_few_kernel<T, kWords>,
                           dim3(static_cast<uint32_t>(shares * p.split)), dim3(kFewThreads), smem, stream,
                           p.split, p);
    rc = e == cudaSuccess ? DECODE_OK
                          : fail(DECODE_ERR_CUDA, "linear_w4_few_kernel: %s", cudaGetErrorString(e));
    return true;
}

template <typename T>
bool few_with_words(const LinearParams& p, int sms, cudaStream_t stream, int& rc)
{
    if (p.group % 4 == 0) return run_few<T, 4>(p, sms, stream, rc);
    if (p.group % 2 == 0) return run_few<T, 2>(p, sms, stream, rc);
    return run_few<T, 1>(p, sms, stream, rc);
}

// ---- more tokens -------------------------------------------------------------------------------------
//
// A block takes 128 outputs and up to 64 tokens, over all columns or, in a cluster, a part of them, 128 at
// a time (a chunk).  Sixteen warps make the chunk's operands in shared memory, 128-byte swizzled: the
// codes' differences, a lane 32 columns of a row, and the tokens' elements, both of which each thread
// copies for itself several chunks ahead.  One thread issues the tcgen05.mma (128 x tokens x 16), a scale's
// columns into sums of their own in tensor memory, and four or eight warps read those, multiply them by
// the scales and add them to the running sums in registers, while the next chunks are on their way: two or
// three stages of operands, two of sums.

constexpr int kMakers = 16;                      // warps that make operands

template <int kTokens>
struct TileCfg {
    static constexpr int kReaders = kTokens > 32 ? 8 : 4;          // warps; four have 32 tokens
    static constexpr int kThreads = (kReaders + kMakers + 1) * 32;
    static constexpr int kABytes = kRows * 256, kBBytes = kTokens * 256;   // two swizzled 64-column halves
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kStages = kTokens > 32 ? 2 : 3;
    static constexpr int kAhead = kTokens > 32 ? 5 : 6;            // chunks on their way
    static constexpr int kUnits = (kTokens * 16 + kMakers * 32 - 1) / (kMakers * 32);   // of a maker's x
    static constexpr int kAhead0 = kStages * kStage;               // where they are, 16 bytes a thread
    static constexpr int kAheadBytes = kMakers * 512 * (1 + kUnits);
    static constexpr int kBarriers = kAhead0 + kAhead * kAheadBytes;
    static constexpr int kSmem = kBarriers + 128 + 1024;           // (the base is rounded up to 1024)
    static_assert(kSmem <= 232448, "more than an SM has");
    static_assert(kSmem > 233472 / 2, "one block an SM, so that a cluster's never wait for tensor memory");
    static_assert(kTokens * kSumRow * 4 <= kAhead0, "no room for the sums");
};

// kParts: sums of a chunk, each of the columns of one scale.
template <typename T, int kTokens, int kParts>
__global__ void __launch_bounds__(TileCfg<kTokens>::kThreads, 1) linear_w4_tile_kernel(const LinearParams p)
{
    using C = TileCfg<kTokens>;
    constexpr int kColumns = 2 * kParts * kTokens;                 // of tensor memory
    constexpr int kAlloc = kColumns <= 32 ? 32 : kColumns <= 64 ? 64 : kColumns <= 128 ? 128
                           : kColumns <= 256 ? 256 : 512;
    extern __shared__ uint8_t dynamic[];
    uint8_t* const smem = dynamic + (-smem_addr(dynamic) & 1023u);
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + C::kBarriers);
    // operands made; operands read; sums made; sums read
    const uint32_t full = smem_addr(bars), empty = full + C::kStages * 8, made = empty + C::kStages * 8,
                   taken = made + 16;
    uint32_t* const slot = reinterpret_cast<uint32_t*>(bars + 2 * C::kStages + 4);
    volatile uint32_t* const gave_up = slot + 1;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int part = cluster_rank(), j0 = cluster_id() * kRows, i0 = blockIdx.y * kTokens;
    const int c0 = part * p.pieces_each + min(part, p.pieces_more);
    const int chunks = p.pieces_each + (part < p.pieces_more);
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            gf16::mbar_init(full + s * 8, kMakers);
            gf16::mbar_init(empty + s * 8, 1);
        }
        for (int s = 0; s < 2; ++s) {
            gf16::mbar_init(made + s * 8, 1);
            gf16::mbar_init(taken + s * 8, C::kReaders);
        }
        *gave_up = 0;
        gf16::fence_mbarrier_init();
    }
    if (w == 0) {
        gf16::tmem_alloc<1>(smem_addr(slot), kAlloc);
        gf16::tmem_relinquish<1>();
    }
    gf16::tcgen05_fence_before();
    __syncthreads();
    gf16::tcgen05_fence_after();
    const uint32_t tmem = *slot;
    dep_launch();
    dep_wait();

    auto wait = [&](uint32_t barrier, uint32_t parity) {
        if (gf16::mbar_wait(barrier, parity, gave_up, kTimeout)) return;
        *gave_up = 1;                            // nothing waits any more; the results are no results
        atomicOr(p.status, DECODE_TIMED_OUT);
    };
    float* const sums = reinterpret_cast<float*>(smem);
    if (w < C::kReaders) {
        // ---- the sums: a thread has an output and up to 32 tokens
        constexpr int kMine = kTokens < 32 ? kTokens : 32, kAtOnce = kParts == 4 ? 16 : 8;
        const int t0 = w / 4 * 32;
        float sum[kMine] = {};
        const uint32_t row = min(j0 + tid % kRows, p.n - 1);
        const uint16_t* const scales = p.scales + row * static_cast<uint32_t>(p.scale_stride);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            // (on their way while the sums are made)
            uint32_t scale[kParts];
#pragma unroll
            for (int x = 0; x < kParts; ++x) {
                const int column = (c0 + c) * 128 + x * (128 / kParts);
                scale[x] = column < p.k ? scales[divide(column / 32, p.group, p.group_shift)] : 0;
            }
            wait(made + (c & 1) * 8, c >> 1 & 1);
            gf16::tcgen05_fence_after();
#pragma unroll
            for (int x = 0; x < kParts; ++x) {
                // (no part where there is no column: its scale stands for nothing)
                const bool there = x == 0 || (c0 + c) * 128 + x * (128 / kParts) < p.k;
                const float by = Half2<T>::unpack(scale[x]).x;
#pragma unroll
                for (int t = 0; t < kMine; t += kAtOnce) {
                    if (t0 + t >= kTokens) break;
                    uint32_t got[kAtOnce];
                    gf16::tmem_ld_32x32b(tmem + (static_cast<uint32_t>(w % 4 * 32) << 16) +
                                                 ((c & 1) * kParts + x) * kTokens + t0 + t, got);
                    gf16::tmem_ld_wait();
                    if (there)
#pragma unroll
                        for (int e = 0; e < kAtOnce; ++e)
                            sum[t + e] = fmaf(__uint_as_float(got[e]), by, sum[t + e]);
                }
            }
            gf16::tcgen05_fence_before();
            __syncwarp();
            if (lane == 0) gf16::mbar_arrive_local(taken + (c & 1) * 8);
        }
        // [token][output], where the operands were: all of them have been read
#pragma unroll
        for (int t = 0; t < kMine; ++t)
            if (t0 + t < kTokens) sums[(t0 + t) * kSumRow + tid % kRows] = sum[t];
    } else if (w < C::kReaders + kMakers) {
        // ---- the operands: a lane has 32 columns of a row, and 8 of some tokens
        const int m = tid - C::kReaders * 32, q = lane & 3, r = (w - C::kReaders) * 8 + (lane >> 2);
        const uint32_t row = min(j0 + r, p.n - 1);
        // what is left of the columns from the lane's first on
        const int mine = p.k - c0 * 128 - q * 32;
        const uint8_t* code = p.codes + (row * static_cast<uint32_t>(p.code_stride) + c0 * 64 + q * 16);
        const uint8_t* const zeros = p.zeros + row * static_cast<uint32_t>(p.zero_stride);
        // 16 bytes of codes and of each unit of elements.  Each thread reads what it has copied itself, so
        // nothing but its own copies is waited for.
        constexpr int kUnits = C::kUnits, kAhead = C::kAhead;
        const uint16_t* x_from[kUnits];
        int x_left[kUnits];                      // columns from the first on, 0 without a token
        uint32_t x_to[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = m + i * kMakers * 32, token = u / 16, piece = u % 16;
            const bool there = u < kTokens * 16 && i0 + token < p.m;
            x_from[i] = p.x + (there ? (i0 + token) * p.x_stride : 0) + c0 * 128 + piece * 8;
            x_left[i] = there ? p.k - c0 * 128 - piece * 8 : 0;
            x_to[i] = smem_addr(smem) + C::kABytes + piece / 8 * (kTokens * 128) + token * 128 +
                      ((piece % 8 ^ (token & 7)) << 4);
        }
        const uint32_t ahead = smem_addr(smem) + C::kAhead0 + m * 16;
        uint32_t copy_to = ahead, read_from = ahead;
        auto next = [&](uint32_t& at) {
            at += C::kAheadBytes;
            if (at == ahead + kAhead * C::kAheadBytes) at = ahead;
        };
        auto copy = [&](int c) {
            if (c < chunks) {
                if (c * 128 < mine) cp_async16(copy_to, code + c * 64);
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    const bool there = c * 128 < x_left[i];
                    cp_async16(copy_to + (1 + i) * (kMakers * 512), there ? x_from[i] + c * 128 : p.x,
                               there ? 16u : 0u);
                }
                next(copy_to);
            }
            cp_commit();
        };
        uint32_t zero[2];
        auto load_zero = [&](int c) {
            if (p.zeros == nullptr || c >= chunks || c * 128 >= mine) return 8u;
            return static_cast<uint32_t>(zeros[divide((c0 + c) * 4 + q, p.group, p.group_shift)]);
        };
#pragma unroll
        for (int a = 0; a < kAhead - 1; ++a) copy(a);
        zero[0] = load_zero(0), zero[1] = load_zero(1);
        // Where the lane's pieces go.  Lanes 2 and 3 of four write theirs in another order, so that no two of
        // eight lanes meet in a bank: their columns lie 16 KB behind the others'.
        const uint32_t back = q >> 1;
        uint32_t to[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
            to[y] = smem_addr(smem) + back * (kRows * 128) + r * 128 +
                    ((((q & 1) * 4 + (back * 2 ^ y)) ^ (r & 7)) << 4);
        uint32_t at = 0, parity = 1;             // the stage's place; the first pass waits for nothing
        uint32_t bar = 0;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            copy(c + kAhead - 1);
            cp_wait<kAhead - 1>();
            uint32_t words[4];
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                         : "=r"(words[0]), "=r"(words[1]) : "r"(read_from + back * 8) : "memory");
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                         : "=r"(words[2]), "=r"(words[3]) : "r"(read_from + 8 - back * 8) : "memory");
            uint4 x[kUnits];
#pragma unroll
            for (int i = 0; i < kUnits; ++i)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x[i].x), "=r"(x[i].y), "=r"(x[i].z), "=r"(x[i].w)
                             : "r"(read_from + (1 + i) * (kMakers * 512)) : "memory");
            next(read_from);
            Differences<T> diff;
            diff.set(zero[0]);
            zero[0] = zero[1];
            zero[1] = load_zero(c + 2);
            wait(empty + bar, parity);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                uint32_t d[4];
                diff.of(words[y], d);
                gf16::st_shared_v4(to[y] + at, d[0], d[1], d[2], d[3]);
            }
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const uint4 s = sorted(x[i]);
                if (kTokens * 16 % (kMakers * 32) == 0 || m < kTokens * 16)
                    gf16::st_shared_v4(x_to[i] + at, s.x, s.y, s.z, s.w);
            }
            gf16::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) gf16::mbar_arrive_local(full + bar);
            at += C::kStage, bar += 8;
            if (bar == C::kStages * 8) {
                at = bar = 0;
                parity ^= 1;
            }
        }
        cp_wait<0>();
    } else if (gf16::elect_one_sync()) {
        // ---- the products
        constexpr uint32_t idesc = gf16::make_idesc_f16(kRows, kTokens, std::is_same<T, __half>::value ? 0 : 1);
        int stage = 0;
        uint32_t parity = 0;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            wait(full + stage * 8, parity);
            if (c >= 2) wait(taken + (c & 1) * 8, (c >> 1) - 1 & 1);
            gf16::tcgen05_fence_after();
            const uint32_t base = smem_addr(smem) + stage * C::kStage;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint64_t a = gf16::make_smem_desc_sw128(base + k / 4 * (kRows * 128), 1024) + 2 * (k % 4);
                const uint64_t b = gf16::make_smem_desc_sw128(
                                       base + C::kABytes + k / 4 * (kTokens * 128), 1024) + 2 * (k % 4);
                gf16::mma_f16<1>(tmem + ((c & 1) * kParts + k * kParts / 8) * kTokens, a, b, idesc,
                                 k % (8 / kParts) != 0);
            }
            gf16::mma_commit(empty + stage * 8);
            gf16::mma_commit(made + (c & 1) * 8);
            if (++stage == C::kStages) {
                stage = 0;
                parity ^= 1;
            }
        }
        // (the last sums' reader waits for them; after a wait that ran out nothing else would)
        if (*gave_up && chunks > 0)
            gf16::mbar_wait(made + (chunks - 1 & 1) * 8, chunks - 1 >> 1 & 1, nullptr, kTimeout);
    }
    __syncwarp();

    // ---- the sums of the cluster's blocks, then the outputs
    gf16::tcgen05_fence_before();
    __syncthreads();
    gf16::tcgen05_fence_after();
    if (w == 0) gf16::tmem_dealloc<1>(tmem, kAlloc);
    if (p.split > 1) cluster_barrier();
    const int tokens = min(kTokens, p.m - i0);
    for (int at = part * C::kThreads + tid; at < tokens * kRows; at += p.split * C::kThreads) {
        const int token = at / kRows, row = at % kRows;
        if (j0 + row >= p.n) continue;
        float y = 0.f;
        if (p.split > 1) {
            const uint32_t here = smem_addr(sums + token * kSumRow + row);
            float parts[kMostSplit];
#pragma unroll
            for (int o = 0; o < kMostSplit; ++o)
                parts[o] = o < p.split ? cluster_load(cluster_address(here, o)) : 0.f;
#pragma unroll
            for (int o = 0; o < kMostSplit; ++o) y += parts[o];
        } else {
            y = sums[token * kSumRow + row];
        }
        if (p.bias != nullptr) y += Half2<T>::unpack(p.bias[j0 + row]).x;
        y = activated(y, p.activation);
        p.y[(i0 + token) * p.y_stride + j0 + row] = static_cast<uint16_t>(Half2<T>::pack(y, 0.f));
    }
    if (p.split > 1) cluster_barrier();          // the others may still read this block's sums
}

template <typename T, int kTokens, int kParts>
int run_tile(LinearParams p, int sms, cudaStream_t stream)
{
    using C = TileCfg<kTokens>;
    const int64_t blocks = (p.n + kRows - 1) / kRows, tokens = (p.m + kTokens - 1) / kTokens;
    const int64_t chunks = (p.k + 127) / 128;
    // the columns' parts: so many that the fullest SM has the least to do, a block's beginning and end
    // counted as six chunks
    int64_t best = -1;
    for (int split = 1; split <= kMostSplit && (split == 1 || split <= chunks); split *= 2) {
        const int64_t cost = (blocks * tokens * split + sms - 1) / sms * ((chunks + split - 1) / split + 6);
        if (best >= 0 && cost >= best) continue;
        best = cost, p.split = split;
    }
    p.pieces_each = static_cast<int>(chunks / p.split), p.pieces_more = static_cast<int>(chunks % p.split);
    if (blocks * p.split > (int64_t(1) << 31) - 1 || tokens > 65535)
        return fail(DECODE_ERR_UNSUPPORTED, "too many outputs or tokens for one call");
    static thread_local bool set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(dev < kMaxDevices && set[dev])) {
        e = cudaFuncSetAttribute(linear_w4_tile_kernel<T, kTokens, kParts>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e == cudaSuccess && dev < kMaxDevices) set[dev] = true;
    }
    if (e == cudaSuccess)
        e = launch_cluster(linear_w4_tile_kernel<T, kTokens, kParts>,
                           dim3(static_cast<uint32_t>(blocks * p.split), static_cast<uint32_t>(tokens)),
                           dim3(C::kThreads), C::kSmem, stream, p.split, p);
    if (e != cudaSuccess)
        return fail(DECODE_ERR_CUDA, "linear_w4_tile_kernel: %s", cudaGetErrorString(e));
    return DECODE_OK;
}

template <typename T, int kTokens>
int tile_with_parts(const LinearParams& p, int sms, cudaStream_t stream)
{
    if (p.group % 4 == 0) return run_tile<T, kTokens, 1>(p, sms, stream);
    if (p.group % 2 == 0) return run_tile<T, kTokens, 2>(p, sms, stream);
    return run_tile<T, kTokens, 4>(p, sms, stream);
}

template <typename T>
int dispatch(const LinearParams& p, int sms, cudaStream_t stream)
{
    int rc = DECODE_OK;
    if (p.m <= 8 && few_with_words<T>(p, sms, stream, rc)) return rc;
    if (p.m <= 16) return tile_with_parts<T, 16>(p, sms, stream);
    if (p.m <= 32) return tile_with_parts<T, 32>(p, sms, stream);
    return tile_with_parts<T, 64>(p, sms, stream);
}

}  // namespace

extern "C" {

int decode_linear_w4(const decode_linear_w4_args* a, cudaStream_t stream)
{
    clear_error();
    if (a == nullptr) return fail(DECODE_ERR_INVALID_ARG, "args is null");
    if (a->m < 0 || a->n < 0 || a->k < 0) return fail(DECODE_ERR_INVALID_ARG, "negative size");
    if (a->dtype != DECODE_F16 && a->dtype != DECODE_BF16)
        return fail(DECODE_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
    if (a->activation < DECODE_ACT_NONE || a->activation > DECODE_ACT_GELU)
        return fail(DECODE_ERR_INVALID_ARG, "unknown activation %d", a->activation);
    if (a->group <= 0) return fail(DECODE_ERR_INVALID_ARG, "groups of %lld", (long long)a->group);
    if (a->k % 32 != 0 || a->group % 32 != 0)
        return fail(DECODE_ERR_UNSUPPORTED, "%lld columns in groups of %lld: not multiples of 32",
                    (long long)a->k, (long long)a->group);
    if (a->m == 0 || a->n == 0) return DECODE_OK;
    if (!a->y || (a->k > 0 && (!a->x || !a->codes || !a->scales)))
        return fail(DECODE_ERR_INVALID_ARG, "null pointer");
    if (misaligned(a->x) || misaligned(a->codes))
        return fail(DECODE_ERR_UNSUPPORTED, "x and codes must be 16-byte aligned");
    constexpr int64_t kMost = (int64_t(1) << 31) - 1;
    if (a->m > kMost || a->n > kMost - kRows || a->k > kMost - 1024)
        return fail(DECODE_ERR_UNSUPPORTED, "problem too large for one call");
    // (32-bit offsets of the weights' rows)
    for (const int64_t stride : {a->code_stride, a->scale_stride, a->zeros ? a->zero_stride : 0})
        if (stride < 0 || stride > UINT32_MAX / a->n - 1)
            return fail(DECODE_ERR_UNSUPPORTED, "weights of more than 2^32 bytes for one call");
    const int64_t groups = (a->k + a->group - 1) / a->group;
    LinearParams p{};
    int64_t x_stride[1], code_stride[1], scale_stride[1], zero_stride[1], y_stride[1];
    // (rows without columns are not read, whatever their strides)
    const int64_t x_rows = a->k > 0 ? a->m : 0, rows = a->k > 0 ? a->n : 0;
    if (!take_strides(x_stride, {a->x_stride}, {x_rows}, 8))
        return fail(DECODE_ERR_UNSUPPORTED, "x's stride must be a multiple of 8");
    if (!take_strides(code_stride, {a->code_stride}, {rows}, 16))
        return fail(DECODE_ERR_UNSUPPORTED, "the codes' stride must be a multiple of 16");
    take_strides(scale_stride, {a->scale_stride}, {a->n}, 1);
    take_strides(zero_stride, {a->zero_stride}, {a->n}, 1);
    take_strides(y_stride, {a->y_stride}, {a->m}, 1);
    const int shared = refuse_shared({{"y", a->y, 2, a->n, {a->m}, y_stride}},
                                     {{"x", a->x, 2, a->k, {a->m}, x_stride},
                                      {"codes", a->codes, 1, a->k / 2, {a->n}, code_stride},
                                      {"scales", a->scales, 2, groups, {a->n}, scale_stride},
                                      {"zeros", a->zeros, 1, groups, {a->n}, zero_stride},
                                      {"bias", a->bias, 2, a->n}});
    if (shared != DECODE_OK) return shared;
    const int sms = sm_count();
    p.status = status_word();
    if (sms == 0 || p.status == nullptr) return DECODE_ERR_CUDA;
    p.x = static_cast<const uint16_t*>(a->x);
    p.codes = static_cast<const uint8_t*>(a->codes);
    p.scales = static_cast<const uint16_t*>(a->scales);
    p.zeros = static_cast<const uint8_t*>(a->zeros);
    p.bias = static_cast<const uint16_t*>(a->bias);
    p.y = static_cast<uint16_t*>(a->y);
    p.x_stride = x_stride[0], p.code_stride = code_stride[0], p.scale_stride = scale_stride[0];
    p.zero_stride = zero_stride[0], p.y_stride = y_stride[0];
    p.m = static_cast<int32_t>(a->m);
    p.n = static_cast<int32_t>(a->n);
    p.k = static_cast<int32_t>(a->k);
    // (in steps of 32 columns)
    p.group = static_cast<int32_t>((a->group < a->k ? a->group : a->k > 0 ? a->k : 32) / 32);
    p.group_shift = shift_of(p.group);
    p.activation = a->activation;
    return a->dtype == DECODE_BF16 ? dispatch<__nv_bfloat16>(p, sms, stream)
                                   : dispatch<__half>(p, sms, stream);
}

}  // extern "C"
