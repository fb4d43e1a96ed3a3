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
// stages of 256 columns (16-byte cp.async), the tokens' elements, which all warps read, through
// registers into two buffers, the next 256 columns' on their way while these are worked on.
//
// The codes are the matrix instructions' first operand (m16n8k16, the rows its 16 rows, the tokens its
// 8 columns).  A lane's 32-bit word holds 8 neighbouring columns; a mask leaves two of them, 16 bits
// apart, as the last bits of two 16-bit numbers whose upper bits an `or` makes 2^7 (bfloat16) or 2^10
// (float16), from which the zero point, lifted the same way, is subtracted: exact, both being whole
// numbers of at most 5 bits.  So columns c and c + 4 are a step's neighbours, and the tokens' elements
// are put into that order once, on their way to shared memory.  The scale is left out of the product:
// each group's sums, of exact products in fp32, are multiplied by it and added to the running ones in
// fp32, so no weight is ever rounded.
#include <cstdint>
#include <type_traits>

#include "decode_common.cuh"

namespace {

using namespace decode;

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kRows = kWarps * 16;               // outputs of a block
constexpr int kChunk = 256;                      // columns of a stage
constexpr int kRowBytes = kChunk / 2;
constexpr int kStageBytes = kRows * kRowBytes;
constexpr int kSteps = kChunk / 32;              // of 32 columns: 16 bytes of a row, a word a lane
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
    int32_t m, n, k, group, groups, split, activation;
};

template <int kTiles>
struct W4Cfg {
    static constexpr int kTokens = 8 * kTiles;
    static constexpr int kXBytes = kTokens * kChunk * 2;
    // (two blocks share an SM's 228 KB, of which the system takes 1 KB a block)
    static constexpr int kRoom = 233472 / 2 - 1024 - 2 * kXBytes;
    static constexpr int kStages = kRoom / kStageBytes < 6 ? kRoom / kStageBytes : 6;
    static constexpr int kSmem = kStages * kStageBytes + 2 * kXBytes;
    static_assert(kStages >= 2 && kTokens * kSumRow * 4 <= kSmem, "no room");
};

template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                     "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                     "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

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

__device__ __forceinline__ float activated(float y, int activation)
{
    if (activation == DECODE_ACT_RELU) return y < 0.f ? 0.f : y;
    if (activation == DECODE_ACT_GELU) return y * normcdff(y);
    return y;
}

__device__ __forceinline__ uint32_t rank_of_cluster()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

template <typename T, int kTiles>
__global__ void __launch_bounds__(kThreads, 2) linear_w4_kernel(const LinearParams p)
{
    using C = W4Cfg<kTiles>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* const xbuf = smem + C::kStages * kStageBytes;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int part = static_cast<int>(blockIdx.x) % p.split;
    const int j0 = static_cast<int>(blockIdx.x) / p.split * kRows;   // the block's first output
    const int i0 = blockIdx.y * C::kTokens;                         // and token
    const int chunks = (p.k + kChunk - 1) / kChunk;
    const int c0 = static_cast<int>(static_cast<int64_t>(chunks) * part / p.split);
    const int c1 = static_cast<int>(static_cast<int64_t>(chunks) * (part + 1) / p.split);
    dep_launch();
    dep_wait();

    // ---- loads of a chunk
    const uint32_t ring = smem_addr(smem);
    const int unit = tid & 7, row_of = tid >> 3;                    // of the codes: 16 bytes, 32 rows
    auto load_codes = [&](int c) {
        if (c < c1) {
            const uint32_t stage = ring + (c - c0) % C::kStages * kStageBytes;
            const int column = c * kChunk + unit * 32;
#pragma unroll
            for (int i = 0; i < kRows / 32; ++i) {
                const int row = row_of + 32 * i;
                const bool there = j0 + row < p.n && column < p.k;
                const uint8_t* from = p.codes + (j0 + row) * p.code_stride + column / 2;
                cp_async16(stage + row * kRowBytes + ((unit ^ (row & 7)) << 4),
                           there ? from : p.codes, there ? 16u : 0u);
            }
        }
        cp_commit();
    };
    uint4 xs[kTiles];                                               // 8 columns of a token each
    auto load_x = [&](int c) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            const int token = i0 + w + 8 * i, column = c * kChunk + lane * 8;
            xs[i] = make_uint4(0u, 0u, 0u, 0u);
            if (token < p.m && column < p.k && c < c1)
                xs[i] = *reinterpret_cast<const uint4*>(p.x + token * p.x_stride + column);
        }
    };
    auto put_x = [&](uint8_t* to) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            const int token = w + 8 * i;
            *reinterpret_cast<uint4*>(to + token * (kChunk * 2) + ((lane ^ (token & 1) << 2) << 4)) =
                make_uint4(__byte_perm(xs[i].x, xs[i].z, 0x5410), __byte_perm(xs[i].x, xs[i].z, 0x7632),
                           __byte_perm(xs[i].y, xs[i].w, 0x5410), __byte_perm(xs[i].y, xs[i].w, 0x7632));
        }
    };
    // scales and zero points of rows lane / 4 and 8 more: lane q of four has those of the chunk's groups
    // q and q + 4 (there are 8 at most), a scale's bits below its zero point
    const int q = lane & 3, r = w * 16 + (lane >> 2);
    uint32_t sz[2][2];
    auto load_scales = [&](int c) {
        const int g0 = c * kChunk / p.group;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = j0 + r + 8 * e, g = g0 + q + 4 * h;
                sz[h][e] = 0;
                if (row < p.n && g < p.groups && c < c1 && (h == 0 || p.group == 32)) {
                    sz[h][e] = p.scales[row * p.scale_stride + g];
                    sz[h][e] |= (p.zeros != nullptr ? p.zeros[row * p.zero_stride + g] : 8u) << 16;
                }
            }
    };

    float sum[kTiles][4] = {}, acc[kTiles][4] = {};
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) load_codes(c0 + s);
    load_x(c0);
    load_scales(c0);
    Differences<T> diff[2];
    float scale[2] = {0.f, 0.f};
    diff[0].set(0), diff[1].set(0);
    int group = -1;                                                 // the running sums'
    int until = 0;                                                  // steps left of it
    for (int c = c0; c < c1; ++c) {
        uint8_t* const x = xbuf + ((c - c0) & 1) * C::kXBytes;
        put_x(x);
        cp_wait<C::kStages - 2>();
        __syncthreads();
        uint32_t now[2][2] = {{sz[0][0], sz[0][1]}, {sz[1][0], sz[1][1]}};
        load_codes(c + C::kStages - 1);
        load_x(c + 1);
        load_scales(c + 1);
        const uint8_t* const stage = smem + (c - c0) % C::kStages * kStageBytes;
        const int g0 = c * kChunk / p.group;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            if (until == 0) {                                       // (for all lanes)
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum[t][e] = fmaf(acc[t][e], scale[e >> 1], sum[t][e]);
                        acc[t][e] = 0.f;
                    }
                const int column = c * kChunk + s * 32;
                group = column / p.group;
                until = p.group / 32 - (column - group * p.group) / 32;
                const int at = group - g0;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t got = __shfl_sync(0xffffffffu, at < 4 ? now[0][e] : now[1][e],
                                                     (lane & ~3) | (at & 3));
                    scale[e] = Half2<T>::unpack(got & 0xffffu).x;
                    diff[e].set(got >> 16);
                }
            }
            --until;
            uint32_t lower[4], upper[4];
            {
                const int at = ((s ^ (lane >> 2)) << 4) + q * 4;    // (rows of 8 more swizzle alike)
                diff[0].of(*reinterpret_cast<const uint32_t*>(stage + r * kRowBytes + at), lower);
                diff[1].of(*reinterpret_cast<const uint32_t*>(stage + (r + 8) * kRowBytes + at), upper);
            }
            const uint32_t a[2][4] = {{lower[0], upper[0], lower[1], upper[1]},
                                      {lower[2], upper[2], lower[3], upper[3]}};
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const int token = t * 8 + (lane >> 2);
                const uint4 b = *reinterpret_cast<const uint4*>(
                    x + token * (kChunk * 2) + (((s * 4 + q) ^ (token & 1) << 2) << 4));
                mma<T>(acc[t], a[0], b.x, b.y);
                mma<T>(acc[t], a[1], b.z, b.w);
            }
        }
    }

    // ---- the sums of the cluster's blocks, [token][output], then the outputs
    cp_wait<0>();
    __syncthreads();
    float* const sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sums[(t * 8 + q * 2 + (e & 1)) * kSumRow + r + (e >> 1) * 8] =
                fmaf(acc[t][e], scale[e >> 1], sum[t][e]);
    if (p.split > 1)
        asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
    else
        __syncthreads();
    const int tokens = min(C::kTokens, p.m - i0);
    const int rank = p.split > 1 ? static_cast<int>(rank_of_cluster()) : 0;
    for (int at = rank * kThreads + tid; at < tokens * kRows; at += p.split * kThreads) {
        const int token = at / kRows, row = at % kRows;
        if (j0 + row >= p.n) continue;
        float y = 0.f;
        if (p.split > 1) {
            const uint32_t here = smem_addr(sums + token * kSumRow + row);
            float parts[kMostSplit];
#pragma unroll
            for (int o = 0; o < kMostSplit; ++o) {
                parts[o] = 0.f;
                if (o < p.split) {
                    uint32_t there;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(o));
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(parts[o]) : "r"(there) : "memory");
                }
            }
#pragma unroll
            for (int o = 0; o < kMostSplit; ++o) y += parts[o];
        } else {
            y = sums[token * kSumRow + row];
        }
        if (p.bias != nullptr) y += Half2<T>::unpack(p.bias[j0 + row]).x;
        y = activated(y, p.activation);
        p.y[(i0 + token) * p.y_stride + j0 + row] = static_cast<uint16_t>(Half2<T>::pack(y, 0.f));
    }
    if (p.split > 1)                             // the others may still read this block's sums
        asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

template <typename T, int kTiles>
int run(LinearParams p, int sms, cudaStream_t stream)
{
    using C = W4Cfg<kTiles>;
    const int64_t blocks = (p.n + kRows - 1) / kRows, tokens = (p.m + C::kTokens - 1) / C::kTokens;
    const int chunks = (p.k + kChunk - 1) / kChunk;
    // as many parts as the GPU holds blocks for, two an SM
    int64_t split = 2 * sms / (blocks * tokens);
    split = split < 1 ? 1 : split > kMostSplit ? kMostSplit : split;
    if (split > chunks) split = chunks > 1 ? chunks : 1;
    p.split = static_cast<int>(split);
    if (blocks * split > (int64_t(1) << 31) - 1 || tokens > 65535)
        return fail(DECODE_ERR_UNSUPPORTED, "too many outputs or tokens for one call");
    static thread_local bool set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(dev < kMaxDevices && set[dev])) {
        e = cudaFuncSetAttribute(linear_w4_kernel<T, kTiles>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmem);
        if (e == cudaSuccess && dev < kMaxDevices) set[dev] = true;
    }
    if (e == cudaSuccess)
        e = launch_cluster(linear_w4_kernel<T, kTiles>,
                           dim3(static_cast<uint32_t>(blocks * split), static_cast<uint32_t>(tokens)),
                           dim3(kThreads), C::kSmem, stream, p.split, p);
    if (e != cudaSuccess)
        return fail(DECODE_ERR_CUDA, "linear_w4_kernel: %s", cudaGetErrorString(e));
    return DECODE_OK;
}

template <typename T>
int dispatch(const LinearParams& p, int sms, cudaStream_t stream)
{
    if (p.m <= 8) return run<T, 1>(p, sms, stream);
    if (p.m <= 16) return run<T, 2>(p, sms, stream);
    return run<T, 4>(p, sms, stream);
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
    if (a->m > kMost || a->n > kMost - kRows || a->k > kMost - 2 * kChunk)
        return fail(DECODE_ERR_UNSUPPORTED, "problem too large for one call");
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
    if (sms == 0) return DECODE_ERR_CUDA;
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
    p.group = static_cast<int32_t>(a->group < a->k ? a->group : a->k > 0 ? a->k : 32);
    p.groups = static_cast<int32_t>(groups);
    p.activation = a->activation;
    return a->dtype == DECODE_BF16 ? dispatch<__nv_bfloat16>(p, sms, stream)
                                   : dispatch<__half>(p, sms, stream);
}

}  // extern "C"
