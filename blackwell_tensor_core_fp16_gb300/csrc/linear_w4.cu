// A linear layer of few tokens with 4-bit weights and group scales (C ABI in include/decode.h):
//
//     y[i][j] = act(bias[j] + sum_g s[j][g] sum_{c in g} x[i][c] (code[j][c] - z[j][g]))
//
// A weight is half a byte and takes part in 2 m operations, so for a few tokens HBM bounds the time, and what
// a weight costs in instructions on its way to the matrix units decides whether it does: to keep up with HBM,
// the SMs have to take 47 weights a clock each.
//
// From a code to an operand.  The difference of a code and its zero point is exact in 16 bits, being a whole
// number of at most 5 bits, and takes ten instructions for the 8 columns of a 32-bit word (below).  The scale
// is left out of the product: the sums of a scale's columns, of exact products in fp32, are multiplied by it
// and added to the running ones in fp32.  So no weight is ever rounded, and the only rounding to 16 bits is
// the output's.
//
// Two kernels.  One for up to 8 tokens with few elements streams the codes from global memory to the warps that
// use them; mma.sync is enough there, for the tensor cores have next to nothing to do.  The other, for more,
// spares the instructions: tcgen05.mma takes 128 outputs and up to 64 tokens at a time.
#include <atomic>

#include "decode_mma.cuh"
#include "desc.h"
#include "ptx.cuh"

namespace {

using namespace decode;

constexpr int kRows = 128;                       // outputs of a block for more tokens
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
    int32_t wide;                                // a chunk's scales, and its zero points, are one word
    uint32_t* status;
    int32_t items_each, items_more, pieces_each, pieces_more, stages, waiting;    // for few tokens
    int32_t fault;                               // for the tests: full[1] waits for one arrival too many
    uint32_t wait_ms;                            // that one wait may take
};

__device__ __forceinline__ uint64_t limit_ns(const LinearParams& p)
{
    return static_cast<uint64_t>(p.wait_ms) * 1000000;
}

std::atomic<uint32_t> g_wait_ms{2000};
std::atomic<int32_t> g_fault{0};

// How codes become 16-bit numbers.  Two masks split a word's bytes, a permutation deals a byte of each to the
// two halves of a register, and an fma makes them numbers.  (Masks that leave codes below the upper bits of
// 2^7 or 2^10, from which the lifted zero point is subtracted, take 13 for neighbours, and 11 for columns
// four apart, in whose order the tokens' elements have to be brought: 48 tokens, 14336 x 4096, 18.3 us for
// 17.3, one token 12.4 for 12.0; the pipe of the integer operations was 67% busy.)
//
// A half of 16 bits that holds a whole number v < 256 and no more is v times the type's least number (bfloat16
// has 7 bits behind the point and the exponents 0 and 1 the same unit, so this holds to 255): one fma brings it
// to its size and takes the zero point from it.  kUp: the factors of a code in the lower half and of 16 times a
// code in the upper one; kBack: what is left to be multiplied into the sums at the end, for the least number's
// inverse is no number of the type.  (Not into the scales, which may be the type's largest.)
template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
    static constexpr uint32_t kUp = 0x7d007f00u, kDown = 0xff00ff00u;      // 2^127, 2^123; twice -2^127
    static constexpr float kBack = 64.f;                                   // 2^133 / 2^127
    __device__ __forceinline__ static uint32_t fma(uint32_t x, uint32_t y, uint32_t z)
    {
        uint32_t r;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
        return r;
    }
};
template <>
struct Half<__half> {
    static constexpr uint32_t kUp = 0x68007800u, kDown = 0xf800f800u;      // 2^15, 2^11; twice -2^15
    static constexpr float kBack = 512.f;                                  // 2^24 / 2^15
    __device__ __forceinline__ static uint32_t fma(uint32_t x, uint32_t y, uint32_t z)
    {
        uint32_t r;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
        return r;
    }
};

// A row's zero point as the differences need it, and the differences of a word's 8 columns, neighbours in
// pairs, each over kBack.
template <typename T>
struct Differences {
    static constexpr float kBack = Half<T>::kBack;
    uint32_t zero;                               // twice -z / kBack
    __device__ __forceinline__ void set(uint32_t z)
    {
        zero = Half<T>::fma((z & 15u) * 0x10001u, Half<T>::kDown, 0u);
    }
    __device__ __forceinline__ void of(uint32_t word, uint32_t* to) const
    {
        const uint32_t even = word & 0x0f0f0f0fu, odd = word & 0xf0f0f0f0u;
#pragma unroll
        for (int c = 0; c < 4; ++c) {            // byte c of each, and as upper bytes an even one's sign: 0
            uint32_t two;
            asm("prmt.b32 %0, %1, %2, %3;"
                : "=r"(two) : "r"(even), "r"(odd), "r"(c | (4 + c) << 8 | (8 + c) * 0x1010));
            to[c] = Half<T>::fma(two, Half<T>::kUp, zero);
        }
    }
};

// kParts neighbouring scales or zero points, as one word.
template <int kParts>
__device__ __forceinline__ void load_together(const uint16_t* from, uint32_t (&to)[kParts])
{
    if constexpr (kParts == 4) {
        const uint2 b = *reinterpret_cast<const uint2*>(from);
        to[0] = b.x & 0xffffu, to[1] = b.x >> 16, to[2] = b.y & 0xffffu, to[3] = b.y >> 16;
    } else if constexpr (kParts == 2) {
        const uint32_t b = *reinterpret_cast<const uint32_t*>(from);
        to[0] = b & 0xffffu, to[1] = b >> 16;
    } else {
        to[0] = *from;
    }
}
template <int kParts>
__device__ __forceinline__ void load_together(const uint8_t* from, uint32_t (&to)[kParts])
{
    if constexpr (kParts == 4) {
        const uint32_t b = *reinterpret_cast<const uint32_t*>(from);
#pragma unroll
        for (int x = 0; x < 4; ++x) to[x] = b >> 8 * x & 0xffu;
    } else if constexpr (kParts == 2) {
        const uint32_t b = *reinterpret_cast<const uint16_t*>(from);
        to[0] = b & 0xffu, to[1] = b >> 8;
    } else {
        to[0] = *from;
    }
}

__device__ __forceinline__ float activated(float y, int activation)
{
    if (activation == DECODE_ACT_RELU) return y < 0.f ? 0.f : y;
    if (activation == DECODE_ACT_GELU) return y * normcdff(y);
    return y;
}

// How many clusters of 1, 2, 4 and 8 blocks the GPU runs at once, asked for once per thread and device, when
// the kernel is also allowed its shared memory.  Some SMs take part in no cluster of 4 or 8: of the 304
// blocks of the kernel for few tokens 296 and 288 run at once, of the other one's 152 144 and 120.  The
// clusters left over would begin when the others end: one token, 8192 x 28672, in 76 clusters of 4 took 72 us,
// not in parts 43.
constexpr int kMostSplit = 8, kSplits = 4;
struct Clusters {
    bool known;
    int at_once[kSplits];
};
template <auto kKernel>
cudaError_t clusters_of(int threads, int smem, const Clusters*& of)
{
    static thread_local Clusters held[kMaxDevices + 1] = {};       // (the last is asked for at every call)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    Clusters& c = held[dev < kMaxDevices ? dev : kMaxDevices];
    of = &c;
    if (c.known) return e;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    for (int s = 0; s < kSplits && e == cudaSuccess; ++s) {
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 1 << s;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(1 << s);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&c.at_once[s], kKernel, &cfg);
    }
    c.known = e == cudaSuccess && dev < kMaxDevices;
    return e;
}

// ---- few tokens ------------------------------------------------------------------------------------
//
// Up to 8 tokens (m16n8k16: the codes' differences are the first operand, the tokens its 8 columns).  The
// tokens' elements of all of a block's columns fit shared memory, so nothing but the codes streams.  A block
// takes 16 outputs at a time (an item) and 2048 of their columns (a stage): their 16 rows come by bulk
// copies, a row each, into a ring of stages, with none of the SM's threads busy on the way.  Of a stage's 16
// pieces of 128 columns each of eight warps takes two; its sums of an item go to shared memory, where the
// warps' are added after several items.  Two blocks an SM stay and take equal shares of the items; the
// blocks of a cluster share the columns out where there are few items, and add their sums through
// distributed shared memory, in a fixed order.
//
// One token, 14336 x 4096: 12.0 us (floor 4.5); 28672 x 8192: 40 (18), so large layers run at 3.1 TB/s, with
// 160 KB an SM on their way (why no faster is not shown: one warp computes and issues the copies of 16 rows, one
// after another); 4096 x 4096: 5.6 (1.3); 256 x 256: 2.8, a launch and the way there and back.
// 7 tokens, 5000 x 1024, groups of 32: 5.8 (0.5).

constexpr int kFewWarps = 8, kFewThreads = kFewWarps * 32;
constexpr int kItem = 16;                        // outputs
constexpr int kPieces = 2 * kFewWarps;           // of a stage, of 128 columns
constexpr int kFewRow = kPieces * 64 + 64;       // bytes of a stage's row; two rows' 64 bytes lie in
                                                 // different banks
constexpr int kFewStage = kItem * kFewRow;
constexpr int kMostStages = 5;
constexpr int kFewMost = 233472 / 2 - 1024 - 2 * kMostStages * 8 - 16;   // bytes for elements, sums, stages

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
            gf16::mbar_init(full + s * 8, p.fault == 1 && s == 1 ? 2 : 1);
            gf16::mbar_init(empty + s * 8, kFewWarps);
        }
        *gave_up = 0;
        gf16::fence_mbarrier_init();
    }
    __syncwarp();                                // (the other warps: before their first wait, below)
    dep_launch();
    dep_wait();

    auto wait = [&](uint32_t barrier, uint32_t parity) {
        if (gf16::mbar_wait(barrier, parity, gave_up, limit_ns(p))) return true;
        *gave_up = 1;                            // nothing waits any more; the results are no results
        atomicOr(p.status, DECODE_TIMED_OUT);
        return false;                            // (whoever gets this announces nothing)
    };
    // the copies of a step, by the first warp: rows past the last output are the last one's
    // (none any more once a stage is not given back: it may still be on its way)
    int next_item = item0, next_round = 0;
    auto fetch = [&](int stage, bool again, uint32_t parity) {
        if (next_item >= item1) return true;
        const int first = piece0 + next_round * kPieces;
        const int columns = min(p.k, min(piece1, first + kPieces) * 128) - first * 128;
        if (again && !__all_sync(0xffffffffu, wait(empty + stage * 8, parity))) {
            next_item = item1;
            return false;
        }
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
        return true;
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
        const uint16_t* const scales = p.scales + row * static_cast<uint32_t>(p.scale_stride);
        const uint8_t* const zeros = p.zeros + row * static_cast<uint32_t>(p.zero_stride);
        if (kParts > 1 && p.wide) {
#pragma unroll
            for (int x = 0; x < kParts; ++x) scale[x] = 0, zero[x] = p.zeros != nullptr ? 0u : 8u;
            if (scale_item < item1 && piece < piece1) {
                load_together(scales + piece * kParts, scale);
                if (p.zeros != nullptr) load_together(zeros + piece * kParts, zero);
            }
        } else {
#pragma unroll
            for (int x = 0; x < kParts; ++x) {
                const int column = piece * 128 + x * (32 * kWords);
                scale[x] = 0, zero[x] = 0;
                if (scale_item < item1 && piece < piece1 && column < p.k) {
                    const uint32_t g = divide(column / 32, p.group, p.group_shift);
                    scale[x] = scales[g];
                    zero[x] = p.zeros != nullptr ? zeros[g] : 8u;
                }
            }
        }
        if (++scale_round == rounds) {
            scale_round = 0;
            ++scale_item;
        }
    };
    load_scales();

    // ---- the tokens' elements, 8 columns at a time; of a scale's columns the lanes'
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
            if (to[b] != nullptr) *reinterpret_cast<uint4*>(to[b]) = x[b];
    }
    __syncthreads();
    // (lanes without a token of their own read the last one's and have no result)
    const uint8_t* const mine = xs + min(r, p.m - 1) * pitch + w * 256 + q * 16;

    float sum[4] = {};
    int item = item0, round = 0, stage = 0, slot = 0;
    int fetched = steps;                         // steps whose copies have begun, at the end
    uint32_t parity = 0;
    for (int step = 0; step < steps; ++step) {
        uint32_t sz[kParts];
#pragma unroll
        for (int x = 0; x < kParts; ++x) sz[x] = scale[x] | zero[x] << 16;
        load_scales();
        const bool come = wait(full + stage * 8, parity);
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
            if (lane == 0 && come) gf16::mbar_arrive_local(empty + stage * 8);
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
        else if (lane == 0 && come)
            gf16::mbar_arrive_local(empty + stage * 8);
        if (w == 0 && !fetch(stage, true, parity)) fetched = step + p.stages;
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
            if (token < p.m) to[token * kItem + r + 8 * (e >> 1)] = sum[e] * Differences<T>::kBack;
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
    // after a wait that ran out: the copies in flight are waited for, once more.  (A stage's former copies had
    // come before it was filled again, so a parity stands for the last ones.)
    if (*gave_up && w == 0)
        for (int step = max(0, fetched - p.stages); step < fetched; ++step)
            gf16::mbar_wait(full + step % p.stages * 8, step / p.stages & 1, nullptr, limit_ns(p));
}

// The kernel for few tokens; false if they have too many elements for it.  Each block brings its columns of
// all tokens into shared memory before it begins: its time grows with the tokens, the other kernel's does
// not.  Measured, us, this kernel and the other: 4096 x 4096, 1 token 5.6 and 7.0, 4 7.0 and 7.2, 8 9.3 and
// 7.4; 14336 x 4096, 1 12.0 and 13.6, 4 13.6 and 13.6, 8 16.7 and 13.8; 8192 x 8192, 1 15.0 and 14.7, 2 16.4
// and 14.8; 28672 x 8192, 1 40.3 and 46.1, 2 41.4 and 46.1; 1024 x 14336, split by 8, 4 7.5 and 8.7; 5000 x
// 1024, 8 5.7 and 5.8.  More parts than are best without regard to this lose more: 8192 x 8192, 8 tokens, 28.3.
// (The rule goes by elements alone, so 2 tokens of 8192 x 8192 stay with this kernel, which loses a tenth there.)
constexpr int kFewMostElements = 16384;
template <typename T, int kWords>
bool run_few(LinearParams p, cudaStream_t stream, int& rc)
{
    constexpr int kMost = 233472 / 2 - 1024;    // bytes of one of two blocks
    const Clusters* clusters = nullptr;
    cudaError_t e = clusters_of<linear_w4_few_kernel<T, kWords>>(kFewThreads, kMost, clusters);
    if (e != cudaSuccess) {
        rc = fail(DECODE_ERR_CUDA, "linear_w4_few_kernel: %s", cudaGetErrorString(e));
        return true;
    }
    const int64_t items = (p.n + kItem - 1) / kItem, pieces = (p.k + 127) / 128;
    // The columns' parts: those with which the block with the most to do has the least, a block's beginning
    // and end counted as two stages, a cluster's as four.  What shared memory the elements and two stages
    // leave holds the sums of as many items as a block has, and more stages.
    int64_t best = -1, smem = 0, shares = 0;
    bool fits = false;
    for (int s = 0; s < kSplits && (s == 0 || 1 << s <= pieces) && clusters->at_once[s] > 0; ++s) {
        const int split = 1 << s;
        const int64_t mine = (pieces + split - 1) / split;
        const int64_t most = clusters->at_once[s] < items ? clusters->at_once[s] : items,
                      each = (items + most - 1) / most;
        const int64_t bytes = p.m * (mine * 256 + 64), sums = kFewWarps * p.m * kItem * 4;
        const int64_t stages = 2, room = kFewMost - bytes - stages * kFewStage;
        const int64_t cost = each * mine + (split > 1 ? 4 : 2) * kPieces;
        if (best >= 0 && cost >= best) continue;
        best = cost, p.split = split, shares = most;
        fits = room >= sums && p.m * mine <= kFewMostElements / 128;
        if (!fits) continue;
        const int64_t waiting = room / sums < each ? room / sums : each;
        const int64_t more = (room - waiting * sums) / kFewStage;
        p.waiting = static_cast<int>(waiting);
        p.stages = static_cast<int>(stages + more < kMostStages ? stages + more : kMostStages);
        smem = bytes + waiting * sums + p.stages * kFewStage + 2 * kMostStages * 8 + 16;
    }
    if (!fits) return false;
    p.items_each = static_cast<int>(items / shares), p.items_more = static_cast<int>(items % shares);
    p.pieces_each = static_cast<int>(pieces / p.split), p.pieces_more = static_cast<int>(pieces % p.split);
    e = launch_cluster(linear_w4_few_kernel<T, kWords>, dim3(static_cast<uint32_t>(shares * p.split)),
                       dim3(kFewThreads), smem, stream, p.split, p);
    rc = e == cudaSuccess ? DECODE_OK
                          : fail(DECODE_ERR_CUDA, "linear_w4_few_kernel: %s", cudaGetErrorString(e));
    return true;
}

template <typename T>
bool few_with_words(const LinearParams& p, cudaStream_t stream, int& rc)
{
    if (p.group % 4 == 0) return run_few<T, 4>(p, stream, rc);
    if (p.group % 2 == 0) return run_few<T, 2>(p, stream, rc);
    return run_few<T, 1>(p, stream, rc);
}

// ---- more tokens -------------------------------------------------------------------------------------
//
// A block takes 128 outputs and up to 64 tokens, over all columns or, in a cluster, a part of them, 128 at
// a time (a chunk).  The matrix instruction (tcgen05.mma, 128 x tokens x 16) takes the codes' differences
// from tensor memory and the tokens' elements from shared memory.  Four groups of four warps take a chunk
// each in turn: a lane makes a row's differences of the codes that its warp has copied and stores them into
// tensor memory; the elements are copied to where the matrix instruction takes them, a chunk of the group
// ahead.  One thread issues the matrix instructions, a
// scale's columns into sums of their own, and four or eight warps read those, multiply them by the scales
// and add them to the running sums in registers.  So four chunks are made at once, while the sums of two
// are on their way.
//
// 48 tokens, 14336 x 4096: 17.3 us (floor 4.8), 0.4 us a chunk; 16 tokens 14.2; 200 tokens, 4096 x 4096: 17.3
// (3.5).  A block's 128 rows being indivisible, 112 of 152 SMs have one, and on those nothing is full: a
// scheduler issues for 600 of a chunk's 850 to 1000 cycles, the pipe of the integer operations, which make the
// operands, is 59% busy, and the warps wait for one another's chunks meanwhile.  Every 64 tokens convert the
// codes anew: 512 tokens, 14336 x 4096, take 115, 2048 take 419.  Differences through shared
// memory, all makers at one chunk: 27.9, of which shared memory alone, written and read twice a chunk, was more
// than half.  The elements by warps of their own, into one place a group: 20.5.  Scales loaded when their sums are
// awaited: 19.0.
constexpr int kGroups = 4, kMakers = 4 * kGroups;                  // warps
constexpr int kAhead = 3;                        // chunks of a warp whose codes are there or on their way

template <int kTokens, int kParts>
struct TileCfg {
    static constexpr int kReaders = kTokens > 32 ? 8 : 4;          // warps; four have 32 tokens
    static constexpr int kMma = kReaders + kMakers;                // the warp that issues
    static constexpr int kThreads = (kMma + 1) * 32;
    static constexpr int kSums = kParts * kTokens > 128 ? 1 : 2;   // chunks whose sums tensor memory holds
    static constexpr int kACols = 64, kSumCols = kSums * kParts * kTokens;
    static constexpr int kColumns = kSumCols + kGroups * kACols;
    static constexpr int kAlloc = 512;
    static_assert(kColumns > kAlloc / 2 && kColumns <= kAlloc, "allocations are powers of two");
    static constexpr int kBBytes = kTokens * 256;                  // two swizzled 64-column halves
    static constexpr int kCodes = 2 * kGroups * kBBytes;           // where the codes are: behind two chunks'
                                                                   // elements of each group
    static constexpr int kBarriers = kCodes + kMakers * kAhead * 2048;
    static constexpr int kSmem = kBarriers + 128 + 1024;           // (the base is rounded up to 1024)
    static_assert(kSmem <= 232448, "more than an SM has");
    static_assert(kSmem > 233472 / 2, "one block an SM, so that a cluster's never wait for tensor memory");
    static_assert(kTokens * kSumRow * 4 <= kCodes, "no room for the sums");
};

// kParts: sums of a chunk, each of the columns of one scale.
template <typename T, int kTokens, int kParts>
__global__ void __launch_bounds__(TileCfg<kTokens, kParts>::kThreads, 1)
linear_w4_tile_kernel(const LinearParams p)
{
    using C = TileCfg<kTokens, kParts>;
    constexpr int kSums = C::kSums;
    extern __shared__ uint8_t dynamic[];
    uint8_t* const smem = dynamic + (-smem_addr(dynamic) & 1023u);
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + C::kBarriers);
    // operands made; operands read; sums made; sums read; all products done
    const uint32_t full = smem_addr(bars), empty = full + kGroups * 8, made = empty + kGroups * 8,
                   taken = made + 16, done = taken + 16;
    uint32_t* const slot = reinterpret_cast<uint32_t*>(bars + 2 * kGroups + 5);
    volatile uint32_t* const gave_up = slot + 1;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int part = cluster_rank(), j0 = cluster_id() * kRows, i0 = blockIdx.y * kTokens;
    const int c0 = part * p.pieces_each + min(part, p.pieces_more);
    const int chunks = p.pieces_each + (part < p.pieces_more);
    // Every block begins elsewhere among its columns: were they all at the same ones, the few lines of L2
    // with those of the tokens would be asked for by all SMs at once.
    const int turn = chunks > 0 ? cluster_id() * 5 % chunks : 0;
    auto column_of = [&](int c) { return (c0 + (c + turn < chunks ? c + turn : c + turn - chunks)) * 128; };
    if (tid == 0) {
        for (int s = 0; s < kGroups; ++s) {
            gf16::mbar_init(full + s * 8, kMakers / kGroups + (p.fault == 1 && s == 1 ? 1 : 0));
            gf16::mbar_init(empty + s * 8, 1);
        }
        for (int s = 0; s < 2; ++s) {
            gf16::mbar_init(made + s * 8, 1);
            gf16::mbar_init(taken + s * 8, C::kReaders);
        }
        gf16::mbar_init(done, 1);
        *gave_up = 0;
        gf16::fence_mbarrier_init();
    }
    if (w == 0) {
        gf16::tmem_alloc<1>(smem_addr(slot), C::kAlloc);
        gf16::tmem_relinquish<1>();
    }
    gf16::tcgen05_fence_before();
    __syncthreads();
    gf16::tcgen05_fence_after();
    const uint32_t tmem = *slot, operands = tmem + C::kSumCols;
    dep_launch();
    dep_wait();

    auto wait = [&](uint32_t barrier, uint32_t parity) {
        if (gf16::mbar_wait(barrier, parity, gave_up, limit_ns(p))) return;
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
        // (with four scales and 64 tokens there are no registers for scales ahead)
        constexpr bool kPrefetch = kSums == 2;
        uint32_t next[kParts];                   // a chunk ahead
        auto load_scales = [&](int c) {
            const int begin = column_of(c);
            if (kParts > 1 && p.wide) {
                if (c < chunks) load_together(scales + begin / (128 / kParts), next);
                return;
            }
#pragma unroll
            for (int x = 0; x < kParts; ++x) {
                const int column = begin + x * (128 / kParts);
                next[x] = c < chunks && column < p.k ? scales[divide(column / 32, p.group, p.group_shift)] : 0;
            }
        };
        if constexpr (kPrefetch) load_scales(0);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            uint32_t scale[kParts];
            const int begin = column_of(c), at = c % kSums;
            if constexpr (!kPrefetch) load_scales(c);
#pragma unroll
            for (int x = 0; x < kParts; ++x) scale[x] = next[x];
            if constexpr (kPrefetch) load_scales(c + 1);
            wait(made + at * 8, c / kSums & 1);
            gf16::tcgen05_fence_after();
#pragma unroll
            for (int x = 0; x < kParts; ++x) {
                // (no part where there is no column: its scale stands for nothing)
                const bool there = x == 0 || begin + x * (128 / kParts) < p.k;
                const float by = Half2<T>::unpack(scale[x]).x;
#pragma unroll
                for (int t = 0; t < kMine; t += kAtOnce) {
                    if (t0 + t >= kTokens) break;
                    uint32_t got[kAtOnce];
                    gf16::tmem_ld_32x32b(tmem + (static_cast<uint32_t>(w % 4 * 32) << 16) +
                                                 (at * kParts + x) * kTokens + t0 + t, got);
                    gf16::tmem_ld_wait();
                    if (there)
#pragma unroll
                        for (int e = 0; e < kAtOnce; ++e)
                            sum[t + e] = fmaf(__uint_as_float(got[e]), by, sum[t + e]);
                }
            }
            gf16::tcgen05_fence_before();
            __syncwarp();
            if (lane == 0) gf16::mbar_arrive_local(taken + at * 8);
        }
        // [token][output], where the elements were: all of them have been read
#pragma unroll
        for (int t = 0; t < kMine; ++t)
            if (t0 + t < kTokens) sums[(t0 + t) * kSumRow + tid % kRows] = sum[t] * Differences<T>::kBack;
    } else if (w < C::kMma) {
        // ---- the operands.  The codes: a warp has 32 rows of every fourth chunk, those of its lanes of tensor
        // memory.  It copies them four lanes a row, and a lane reads its row back: nothing but the warp's
        // own copies is waited for.
        const int group = (w - C::kReaders) / 4, quarter = w % 4;
        const int piece = lane & 3;
        uint32_t from[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            from[i] = min(j0 + quarter * 32 + i * 8 + (lane >> 2), p.n - 1) *
                      static_cast<uint32_t>(p.code_stride);
        const uint8_t* const codes = p.codes + piece * 16;
        const uint8_t* const zeros =
            p.zeros + min(j0 + quarter * 32 + lane, p.n - 1) * static_cast<uint32_t>(p.zero_stride);
        // (a row's pieces are turned, so that lanes that read different rows' meet in no bank)
        const uint32_t ring = smem_addr(smem) + C::kCodes + (w - C::kReaders) * (kAhead * 2048);
        const uint32_t put = (lane >> 2) * 64 + ((piece ^ (lane >> 3)) << 4);
        uint32_t copy_to = 0, read_from = 0;
        auto copy_codes = [&](int c) {
            if (c >= chunks) return;
            const int begin = column_of(c);
            if (begin + piece * 32 < p.k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    cp_async16(ring + copy_to + put + i * 512, codes + from[i] + begin / 2);
            copy_to = copy_to == (kAhead - 1) * 2048 ? 0 : copy_to + 2048;
        };
        // The elements: a thread of a group's 128 has 8 columns of every eighth token.  What stands at tokens
        // that are not there is multiplied into sums of theirs, which nobody writes.
        const int first = quarter * 2 + lane / 16;
        const int there = (p.m - i0 - first + 7) >> 3;             // tokens
        const uint16_t* const x = p.x + (i0 + first) * p.x_stride + lane % 16 * 8;
        const int64_t step = 8 * p.x_stride;
        const uint32_t x_to = smem_addr(smem) + group * C::kBBytes + lane % 16 / 8 * (kTokens * 128) +
                              first * 128 + ((lane % 8 ^ first) << 4);
        auto copy_x = [&](int c, uint32_t half) {
            if (c >= chunks) return;
            const int begin = column_of(c);
            const bool column = begin + lane % 16 * 8 < p.k;       // (zeros behind the last)
            const uint16_t* at = column ? x + begin : p.x;
#pragma unroll
            for (int i = 0; i < kTokens / 8; ++i) {
                if (i < there)
                    cp_async16(x_to + half * (kGroups * C::kBBytes) + i * 1024, at, column ? 16u : 0u);
                if (column) at += step;
            }
        };
        uint32_t zero[kParts];
        auto load_zeros = [&](int c) {
            const int begin = column_of(c);
            if (kParts > 1 && p.wide && p.zeros != nullptr) {
                if (c < chunks) load_together(zeros + begin / (128 / kParts), zero);
                return;
            }
#pragma unroll
            for (int x = 0; x < kParts; ++x) {
                const int column = begin + x * (128 / kParts);
                zero[x] = p.zeros == nullptr || c >= chunks || column >= p.k
                              ? 8u : zeros[divide(column / 32, p.group, p.group_shift)];
            }
        };
        copy_codes(group);
        cp_commit();
        copy_codes(group + kGroups);
        copy_x(group, 0);
        cp_commit();
        load_zeros(group);
        cp_wait<1>();
        __syncwarp();
        const uint32_t to = operands + (static_cast<uint32_t>(quarter * 32) << 16) + group * C::kACols;
        uint32_t turn_of = 0;                    // the group's chunks so far, modulo 2
#pragma unroll 1
        for (int c = group; c < chunks; c += kGroups, turn_of ^= 1) {
            Differences<T> diff[kParts];
#pragma unroll
            for (int x = 0; x < kParts; ++x) diff[x].set(zero[x]);
            load_zeros(c + kGroups);
            wait(empty + group * 8, turn_of ^ 1);                  // (the first waits for nothing)
            gf16::tcgen05_fence_after();
            copy_codes(c + 2 * kGroups);
            copy_x(c + kGroups, turn_of ^ 1);
            cp_commit();
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                uint32_t words[4], d[16];
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(words[0]), "=r"(words[1]), "=r"(words[2]), "=r"(words[3])
                             : "r"(ring + read_from + lane * 64 + ((y ^ (lane >> 1 & 3)) << 4)) : "memory");
#pragma unroll
                for (int e = 0; e < 4; ++e) diff[y * kParts / 4].of(words[e], d + 4 * e);
                gf16::tmem_st_32x32b(to + y * 16, d);
            }
            read_from = read_from == (kAhead - 1) * 2048 ? 0 : read_from + 2048;
            // this chunk's elements and the codes of the group's next
            cp_wait<1>();
            gf16::fence_proxy_async_smem();
            gf16::tmem_st_wait();
            gf16::tcgen05_fence_before();
            __syncwarp();
            if (lane == 0) gf16::mbar_arrive_local(full + group * 8);
        }
        cp_wait<0>();
    } else if (gf16::elect_one_sync()) {
        // ---- the products
        constexpr uint32_t idesc = gf16::make_idesc_f16(kRows, kTokens, std::is_same<T, __half>::value ? 0 : 1);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int stage = c % kGroups, at = c % kSums;
            wait(full + stage * 8, c / kGroups & 1);
            if (c >= kSums) wait(taken + at * 8, (c / kSums & 1) ^ 1);
            gf16::tcgen05_fence_after();
            const uint32_t base = smem_addr(smem) + c % (2 * kGroups) * C::kBBytes;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint64_t b = gf16::make_smem_desc_sw128(base + k / 4 * (kTokens * 128), 1024) + 2 * (k % 4);
                gf16::mma_f16_tmem(tmem + (at * kParts + k * kParts / 8) * kTokens,
                                   operands + stage * C::kACols + k * 8, b, idesc, k % (8 / kParts) != 0);
            }
            gf16::mma_commit(empty + stage * 8);
            gf16::mma_commit(made + at * 8);
        }
        // All of them are waited for, on a barrier of their own, whoever has given up: tensor memory and the
        // elements go with the block.  (After a wait that ran out the others' parities stand for nothing.)
        gf16::mma_commit(done);
        if (!gf16::mbar_wait(done, 0, nullptr, limit_ns(p))) atomicOr(p.status, DECODE_TIMED_OUT);
    }
    __syncwarp();

    // ---- the sums of the cluster's blocks, then the outputs
    gf16::tcgen05_fence_before();
    __syncthreads();
    gf16::tcgen05_fence_after();
    if (w == 0) gf16::tmem_dealloc<1>(tmem, C::kAlloc);
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
int run_tile(LinearParams p, cudaStream_t stream)
{
    using C = TileCfg<kTokens, kParts>;
    const int64_t blocks = (p.n + kRows - 1) / kRows, tokens = (p.m + kTokens - 1) / kTokens;
    const int64_t chunks = (p.k + 127) / 128;
    const Clusters* clusters = nullptr;
    cudaError_t e = clusters_of<linear_w4_tile_kernel<T, kTokens, kParts>>(C::kThreads, C::kSmem, clusters);
    // the columns' parts: as many as leave all blocks running at once, with some chunks each
    p.split = 1;
    for (int s = 1; s < kSplits && e == cudaSuccess; ++s)
        if (blocks * tokens <= clusters->at_once[s] && chunks >= kGroups << s) p.split = 1 << s;
    p.pieces_each = static_cast<int>(chunks / p.split), p.pieces_more = static_cast<int>(chunks % p.split);
    if (blocks * p.split > (int64_t(1) << 31) - 1 || tokens > 65535)
        return fail(DECODE_ERR_UNSUPPORTED, "too many outputs or tokens for one call");
    if (e == cudaSuccess)
        e = launch_cluster(linear_w4_tile_kernel<T, kTokens, kParts>,
                           dim3(static_cast<uint32_t>(blocks * p.split), static_cast<uint32_t>(tokens)),
                           dim3(C::kThreads), C::kSmem, stream, p.split, p);
    if (e != cudaSuccess)
        return fail(DECODE_ERR_CUDA, "linear_w4_tile_kernel: %s", cudaGetErrorString(e));
    return DECODE_OK;
}

template <typename T, int kTokens>
int tile_with_parts(const LinearParams& p, cudaStream_t stream)
{
    if (p.group % 4 == 0) return run_tile<T, kTokens, 1>(p, stream);
    if (p.group % 2 == 0) return run_tile<T, kTokens, 2>(p, stream);
    return run_tile<T, kTokens, 4>(p, stream);
}

template <typename T>
int dispatch(const LinearParams& p, cudaStream_t stream)
{
    int rc = DECODE_OK;
    if (p.m <= 8 && few_with_words<T>(p, stream, rc)) return rc;
    if (p.m <= 16) return tile_with_parts<T, 16>(p, stream);
    if (p.m <= 32) return tile_with_parts<T, 32>(p, stream);
    return tile_with_parts<T, 64>(p, stream);
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
    p.status = status_word();
    if (p.status == nullptr) return DECODE_ERR_CUDA;
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
    p.fault = g_fault.load(), p.wait_ms = g_wait_ms.load();
    // Groups of 32 and 64: a lane's scales of 128 columns by one load, if a row's are aligned so.  Each lane has a
    // row, so a load costs as many cycles as it touches lines: 64 tokens, 14336 x 4096, groups of 32 42.0 us with
    // one for each, 16 tokens 27.9.
    const int parts = p.group <= 2 ? 4 / p.group : 1;
    p.wide = parts > 1 && a->k % 128 == 0 && scale_stride[0] % parts == 0 &&
             reinterpret_cast<uintptr_t>(a->scales) % (2 * parts) == 0 &&
             (!a->zeros || (zero_stride[0] % parts == 0 && reinterpret_cast<uintptr_t>(a->zeros) % parts == 0));
    return a->dtype == DECODE_BF16 ? dispatch<__nv_bfloat16>(p, stream)
                                   : dispatch<__half>(p, stream);
}

int decode_set_wait_timeout_ms(uint32_t ms)
{
    clear_error();
    if (ms == 0) return fail(DECODE_ERR_INVALID_ARG, "timeout must be at least 1 ms");
    g_wait_ms.store(ms);
    return DECODE_OK;
}

int decode_set_fault_injection(int mode)
{
    clear_error();
    if (mode < 0 || mode > 1) return fail(DECODE_ERR_INVALID_ARG, "unknown fault mode %d", mode);
    g_fault.store(mode);
    return DECODE_OK;
}

}  // extern "C"
