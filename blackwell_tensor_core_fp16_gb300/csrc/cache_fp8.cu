// The write to a paged cache of E4M3 codes with an E8M0 scale for each block of tokens and head, and
// its reading back (C ABI and formulas in include/decode.h).
//
// Both move every element once, 3 bytes of it, and do a dozen operations on it: HBM bounds them.  32768 tokens
// of 8 heads of 128 are written in 39 us (5.2 TB/s; floor 29.7), 200001 of 2 heads of 256 read back in 101
// (6.1 TB/s, 90% of the copy rate; floor 90.6).
//
// Write.  A block's scale needs the largest of its new elements before the first code is known, and
// its other codes may have to follow, so one warp takes a block, of one head of the keys or of the
// values, as a whole: the block's first new token in the call (its leader, found from the slots
// beside it) stands for it.  The rows wait in registers while the maximum is taken (8 or 16 tokens;
// of larger blocks the rest is read again, from a cache), nothing else is shared between warps, and no
// order of blocks matters.  A scale being a power of two, x * 2^(127 - e) is exact and only the
// conversion rounds, and codes that follow keep their bits but for those that become subnormal.
#include <cstdint>
#include <type_traits>

#include "fp8.cuh"

namespace {

using namespace decode;

constexpr int kWarps = 8;
constexpr int kWindow = 16;           // most tokens of a block of threads; half the lanes that see slots
constexpr int kBack = 5;              // times 32 tokens before the window, looked through for its blocks

// A cache's two tensors (keys, values), and where its places are.
struct CacheParams {
    uint8_t* codes[2];
    uint8_t* scales[2];
    int64_t code_stride[2][3], scale_stride[2][3];
    const int32_t* slots;
    uint32_t* status;
    int32_t tokens, heads, page_size, page_shift, block, block_shift, places;
};
struct QuantizeParams : CacheParams {
    const uint16_t* x[2];
    int64_t x_stride[2][2];
    int32_t window, per;              // tokens of a block of threads; its warps that share a token
};
struct DequantizeParams : CacheParams {
    uint16_t* y[2];
    int64_t y_stride[2][2];
    int32_t units, at_once;           // 8-element units of a token; tokens of a block of threads
    uint32_t magic;                   // ceil(2^32 / units)
};

template <typename T>
constexpr uint32_t kInfinity = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;

template <typename T>
__device__ __forceinline__ float from_bits(uint32_t bits)
{
    return Half2<T>::unpack(bits).x;
}

// The larger magnitude of each half (with some sign); NaN counts for nothing.
template <typename T>
__device__ __forceinline__ uint32_t larger(uint32_t top, uint32_t x)
{
    uint32_t r;
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(top), "r"(x));
    else
        asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(top), "r"(x));
    return r;
}
// The larger of the halves' magnitudes, over the warp.
__device__ __forceinline__ uint32_t largest(uint32_t top)
{
    return __reduce_max_sync(0xffffffffu, max(top & 0x7fffu, top >> 16 & 0x7fffu));
}
// The least scale for a largest magnitude: 448 = 1.75 * 2^8.
template <typename T>
__device__ __forceinline__ int needed(uint32_t top)
{
    const uint32_t bits = __float_as_uint(from_bits<T>(top));
    return max(0, static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u));
}
// x with zeros for infinities and NaN.
template <typename T>
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t x)
{
    const uint32_t lo = x & 0x7fffu, hi = x >> 16 & 0x7fffu;
    return (lo < kInfinity<T> ? lo : 0u) | (hi < kInfinity<T> ? hi << 16 : 0u);
}

// (A warp that takes the keys' block and the values' has twice the rows on their way: 32768 tokens of 8
// heads of 128 40 us, 46 with a warp for each.  At 256 there are no registers for both.)
template <int D>
constexpr int kKinds = D == 256 ? 1 : 2;
// Blocks of an SM, by the loads that wait in registers, of keys and values.  (Calls of few tokens do not fill
// three.)
template <int D, int kHold, bool kSeveral>
constexpr int kResident = kHold * kKinds<D> > 8 || !kSeveral ? 2 : 3;

// kHold: loads of a warp (512 bytes) that wait in registers.  Rows that do not fit are read again from a cache,
// but with fewer of them in registers three blocks fit an SM instead of two.  us, blocks of 8, 16, 32 and 64
// tokens: 65536 tokens of 8 heads of 64, with 16 rows in registers 57, 42, 41, 44, with 32 80, 57, 45, 47; 32768
// of 128, with 8 rows 38.3, 38.6, 41.9, 53.8, with 16 49.6, 40.7, 41.7, 46.0; 16384 of 256, blocks of 8, 16 and 64,
// with 8 rows 44.5, 44.7, 62.9, with 16 46.3, 37.4, 44.8.
// kSeveral: windows of more than one token.
template <typename T, int D, int kHold, bool kSeveral>
__global__ void __launch_bounds__(kWarps * 32, (kResident<D, kHold, kSeveral>))
quantize_cache_kernel(const QuantizeParams p)
{
    constexpr int kBoth = kKinds<D>;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;     // a row's lanes; rows of one load
    constexpr uint32_t kAll = 0xffffffffu;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int combo = blockIdx.y * p.per + w % p.per, phase = w / p.per, phases = kWarps / p.per;
    if (combo >= 2 / kBoth * p.heads || phase >= phases) return;
    const int kv0 = combo >= p.heads, head = combo - kv0 * p.heads;
    dep_launch();
    dep_wait();

    // lane x sees the slot of token t0 + x, from the one before the window on
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.window - 1;
    const int64_t t = t0 + lane;
    const int slot = t >= 0 && t < p.tokens ? p.slots[t] : -1;
    const int before = __shfl_up_sync(kAll, slot, 1);
    const bool mine = lane > 0 && lane <= p.window;
    const bool valid = slot >= 0 && slot < p.places;
    const bool after_one = lane > 0 && before >= 0 && before < p.places;
    int earlier[kBack];
#pragma unroll
    for (int y = 0; y < kBack; ++y)
        earlier[y] = t0 - lane - y * 32 >= 0 ? p.slots[t0 - lane - y * 32] : -1;
    const int in_block = valid ? slot - divide(slot, p.block, p.block_shift) * p.block : 0;
    const bool goes_on = valid && after_one && slot == before + 1 && in_block > 0;
    auto within = [&](int s, int begin) {        // of the block that begins there
        return static_cast<uint32_t>(s - begin) < static_cast<uint32_t>(p.block);
    };
    const bool disordered = valid && after_one && !goes_on && within(before, slot - in_block);
    if (combo == 0 && phase == 0 && mine && (disordered || (!valid && slot != -1)))
        atomicOr(p.status, DECODE_BAD_CACHE_SLOT);
    uint32_t leaders = __ballot_sync(kAll, mine && valid && !goes_on && !disordered);
    // (one that begins another run of a block, a little behind the first, is refused)
    for (uint32_t left = leaders; left != 0; left &= left - 1) {
        const int lead = __ffs(left) - 1, begin = __shfl_sync(kAll, slot - in_block, lead);
        bool again = lane < lead && within(slot, begin);
#pragma unroll
        for (int y = 0; y < kBack; ++y) again = again || within(earlier[y], begin);
        if (!__any_sync(kAll, again)) continue;
        if (combo == 0 && phase == 0 && lane == 0) atomicOr(p.status, DECODE_BAD_CACHE_SLOT);
        leaders &= ~(1u << lead);
    }

    const int ch = lane % kLanes, sub = lane / kLanes;
    // a place, its scale and its codes (the lane's 8 of them)
    struct Place {
        int page, offset, block;
    };
    auto find = [&](int place) {
        const int page = divide(place, p.page_size, p.page_shift), offset = place - page * p.page_size;
        return Place{page, offset, divide(offset, p.block, p.block_shift)};
    };
    auto scale_at = [&](int kv, const Place& at) {
        return p.scales[kv] + at.page * p.scale_stride[kv][0] + at.block * p.scale_stride[kv][1] +
               head * p.scale_stride[kv][2];
    };
    auto codes_at = [&](int kv, const Place& at) {
        return p.codes[kv] + at.page * p.code_stride[kv][0] + at.offset * p.code_stride[kv][1] +
               head * p.code_stride[kv][2] + ch * 8;
    };
    // 8 elements' codes, and a block's other codes after its scale grew (from places `begin` on, all but the new
    // tokens; a factor below 2^-126 takes any to 0, as 0 does)
    auto convert = [&](const uint4& row, float by, bool odd) {
        uint32_t out[2];
        const uint32_t in[4] = {row.x, row.y, row.z, row.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float2 a = Half2<T>::unpack(in[2 * h]), b = Half2<T>::unpack(in[2 * h + 1]);
            if (odd) {                             // x * 0: NaN for an infinity
                a.x = fmaf(a.x, by, a.x * 0.f), a.y = fmaf(a.y, by, a.y * 0.f);
                b.x = fmaf(b.x, by, b.x * 0.f), b.y = fmaf(b.y, by, b.y * 0.f);
            } else {
                a = halves(mul2(pair(a.x, a.y), pair(by, by)));
                b = halves(mul2(pair(b.x, b.y), pair(by, by)));
            }
            out[h] = codes_of(a.x, a.y) | codes_of(b.x, b.y) << 16;
        }
        return make_uint2(out[0], out[1]);
    };
    auto follow = [&](int kv, uint8_t* codes, int from, int to, int run, int older, int e) {
        const float down = e - older < 127 ? power_of(127 + older - e) : 0.f;
        for (int r = from + sub; r < to; r += kRows) {
            if (r >= 0 && r < run) continue;
            uint2* const at = reinterpret_cast<uint2*>(codes + r * p.code_stride[kv][1]);
            const uint2 old = *at;
            uint32_t in[2] = {old.x, old.y};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 a = Half2<__half>::unpack(codes_to_half2(in[h]));
                const float2 b = Half2<__half>::unpack(codes_to_half2(in[h] >> 16));
                in[h] = codes_of(a.x * down, a.y * down) | codes_of(b.x * down, b.y * down) << 16;
            }
            *at = make_uint2(in[0], in[1]);
        }
    };

    // ---- blocks of which the call has one token, as a decode step's: where a window has several, as many at a
    // time as there are rows in registers, a row's lanes finding its maximum between them (one after the other
    // they take 1.3 us each: 8192 sequences' tokens 60 us, 26 so)
    const uint32_t single = kSeveral ? leaders & ~(__ballot_sync(kAll, goes_on) >> 1) : 0;
    if (kSeveral && (single & (single - 1)) != 0) {
        leaders &= ~single;
        for (int l0 = 1; l0 <= p.window; l0 += kHold * kRows) {
            uint4 row[kBoth][kHold];
            int e[kBoth][kHold];
#pragma unroll
            for (int i = 0; i < kHold; ++i) {
                const int l = l0 + i * kRows + sub;
                const int place = __shfl_sync(kAll, slot, l & 31), first = __shfl_sync(kAll, in_block, l & 31);
                const bool here = l < 32 && (single >> l & 1) != 0 && l % phases == phase;
                const Place at = find(place);
#pragma unroll
                for (int y = 0; y < kBoth; ++y) {
                    row[y][i] = make_uint4(0u, 0u, 0u, 0u);
                    e[y][i] = 0;
                    if (!here) continue;
                    row[y][i] = *reinterpret_cast<const uint4*>(p.x[kv0 + y] + (t0 + l) * p.x_stride[kv0 + y][0] +
                                                                head * p.x_stride[kv0 + y][1] + ch * 8);
                    if (first > 0) e[y][i] = *scale_at(kv0 + y, at);
                }
            }
#pragma unroll
            for (int i = 0; i < kHold; ++i) {
                const int l = l0 + i * kRows + sub;
                const int place = __shfl_sync(kAll, slot, l & 31), first = __shfl_sync(kAll, in_block, l & 31);
                const bool here = l < 32 && (single >> l & 1) != 0 && l % phases == phase;
                if (!__any_sync(kAll, here)) continue;
                const Place at = find(place);
#pragma unroll
                for (int y = 0; y < kBoth; ++y) {
                    const uint4& b = row[y][i];
                    auto top_of = [&](uint32_t x, uint32_t u, uint32_t v, uint32_t z) {
                        uint32_t top = larger<T>(larger<T>(x, u), larger<T>(v, z));
                        top = max(top & 0x7fffu, top >> 16 & 0x7fffu);
#pragma unroll
                        for (int d = 1; d < kLanes; d *= 2) top = max(top, __shfl_xor_sync(kAll, top, d));
                        return top;
                    };
                    uint32_t top = top_of(b.x, b.y, b.z, b.w);
                    const bool odd = __any_sync(kAll, top >= kInfinity<T>);
                    if (odd)
                        top = top_of(finite_or_zero<T>(b.x), finite_or_zero<T>(b.y), finite_or_zero<T>(b.z),
                                     finite_or_zero<T>(b.w));
                    const int older = e[y][i], now = max(needed<T>(top), older);
                    if (here) {
                        *reinterpret_cast<uint2*>(codes_at(kv0 + y, at)) = convert(b, power_of(254 - now), odd);
                        if (ch == 0) *scale_at(kv0 + y, at) = static_cast<uint8_t>(now);
                    }
                    // (all of the warp for each row whose scale grew)
                    uint32_t grown = __ballot_sync(kAll, here && first > 0 && now > older && ch == 0);
                    for (; grown != 0; grown &= grown - 1) {
                        const int of = __ffs(grown) - 1, its = __shfl_sync(kAll, first, of);
                        follow(kv0 + y, codes_at(kv0 + y, find(__shfl_sync(kAll, place, of))), -its, p.block - its, 1,
                               __shfl_sync(kAll, older, of), __shfl_sync(kAll, now, of));
                    }
                }
            }
        }
    }

    for (int nth = 0; leaders != 0; ++nth, leaders &= leaders - 1) {
        if (nth % phases != phase) continue;
        const int lead = __ffs(leaders) - 1;
        const int place = __shfl_sync(kAll, slot, lead), first = __shfl_sync(kAll, in_block, lead);
        const int most = p.block - first;
        const int64_t token = t0 + lead;
        // the run: how many tokens of the block follow
        uint32_t apart = __ballot_sync(kAll, lane > lead && (slot != place + lane - lead ||
                                                             lane - lead >= most));
        int run = apart != 0 ? __ffs(apart) - 1 - lead : 32 - lead;
        while (apart == 0 && run < most) {
            const int64_t next = token + run + lane;
            const int s = next < p.tokens ? p.slots[next] : -1;
            apart = __ballot_sync(kAll, s != place + run + lane || run + lane >= most);
            run += apart != 0 ? __ffs(apart) - 1 : 32;
        }

        const Place at = find(place);
        uint8_t* scale[kBoth];
        const uint16_t* x[kBoth];
        uint8_t* codes[kBoth];
        int older[kBoth];
#pragma unroll
        for (int y = 0; y < kBoth; ++y) {
            const int kv = kv0 + y;
            scale[y] = scale_at(kv, at);
            older[y] = first > 0 ? *scale[y] : 0;
            x[y] = p.x[kv] + token * p.x_stride[kv][0] + head * p.x_stride[kv][1] + ch * 8;
            codes[y] = codes_at(kv, at);
        }
        uint4 row[kBoth][kHold];
        auto load = [&](int from) {
#pragma unroll
            for (int y = 0; y < kBoth; ++y)
#pragma unroll
                for (int i = 0; i < kHold; ++i) {
                    const int r = from + i * kRows + sub;
                    row[y][i] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < run)
                        row[y][i] = *reinterpret_cast<const uint4*>(x[y] + r * p.x_stride[kv0 + y][0]);
                }
        };
        constexpr int kChunk = kHold * kRows;
        const int last = (run - 1) / kChunk * kChunk;
        uint32_t top[kBoth] = {};
        for (int from = 0; from <= last; from += kChunk) {
            load(from);
#pragma unroll
            for (int y = 0; y < kBoth; ++y)
#pragma unroll
                for (int i = 0; i < kHold; ++i)
                    top[y] = larger<T>(larger<T>(top[y], row[y][i].x), row[y][i].y),
                    top[y] = larger<T>(larger<T>(top[y], row[y][i].z), row[y][i].w);
        }
        bool odd = false;                                  // an infinity or NaN: rarely
#pragma unroll
        for (int y = 0; y < kBoth; ++y) {
            top[y] = largest(top[y]);
            odd = odd || top[y] >= kInfinity<T>;
        }
        if (odd) {
#pragma unroll
            for (int y = 0; y < kBoth; ++y) top[y] = 0;
            for (int from = 0; from <= last; from += kChunk) {
                load(from);
#pragma unroll
                for (int y = 0; y < kBoth; ++y)
#pragma unroll
                    for (int i = 0; i < kHold; ++i) {
                        const uint4& b = row[y][i];
                        top[y] = larger<T>(larger<T>(top[y], finite_or_zero<T>(b.x)), finite_or_zero<T>(b.y));
                        top[y] = larger<T>(larger<T>(top[y], finite_or_zero<T>(b.z)), finite_or_zero<T>(b.w));
                    }
            }
#pragma unroll
            for (int y = 0; y < kBoth; ++y)
                top[y] = largest(top[y]);
        }
        int e[kBoth];
#pragma unroll
        for (int y = 0; y < kBoth; ++y) {
            e[y] = max(needed<T>(top[y]), older[y]);
            if (lane == 0) *scale[y] = static_cast<uint8_t>(e[y]);
        }
        for (int from = last; from >= 0; from -= kChunk) {
            if (from != last) load(from);                  // (the last are still there)
#pragma unroll
            for (int y = 0; y < kBoth; ++y) {
                const float by = power_of(254 - e[y]);
#pragma unroll
                for (int i = 0; i < kHold; ++i) {
                    if (from + i * kRows >= run) break;    // (for all lanes)
                    const int r = from + i * kRows + sub;
                    if (r < run)
                        *reinterpret_cast<uint2*>(codes[y] + r * p.code_stride[kv0 + y][1]) =
                            convert(row[y][i], by, odd);
                }
            }
        }
        // the block's other codes follow a scale that grew
#pragma unroll
        for (int y = 0; y < kBoth; ++y)
            if (e[y] > older[y] && first > 0) follow(kv0 + y, codes[y], -first, most, run, older[y], e[y]);
    }
}

// A thread takes units of 8 neighbouring elements of a token's key and the same of its value, two at a
// time, so that their chains of slot, codes and stores run beside each other.  (With 16, whose results
// are two stores a thread, each fills half of every sector that a warp's store touches: 200001 tokens of 2
// heads of 256 took 107 us.)
template <typename T, int D>
__global__ void __launch_bounds__(256) dequantize_cache_kernel(const DequantizeParams p)
{
    constexpr int kUnits = 2;
    dep_launch();
    dep_wait();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.at_once;
    const int here = static_cast<int>(min(static_cast<int64_t>(p.at_once), p.tokens - t0)) * p.units;
    for (int u0 = threadIdx.x; u0 < here; u0 += 256 * kUnits) {
        uint2 codes[kUnits][2];
        int e[kUnits][2], token[kUnits], rest[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = u0 + i * 256;
            token[i] = -1;
            if (u >= here) continue;
            token[i] = p.at_once == 1 ? 0 : static_cast<int>(__umulhi(u, p.magic));
            rest[i] = u - token[i] * p.units;
            const int slot = p.slots[t0 + token[i]], head = rest[i] / (D / 8), ch = rest[i] % (D / 8);
            if (slot >= 0 && slot < p.places) {
                const int page = divide(slot, p.page_size, p.page_shift);
                const int offset = slot - page * p.page_size;
                const int block = divide(offset, p.block, p.block_shift);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    codes[i][kv] = *reinterpret_cast<const uint2*>(
                        p.codes[kv] + page * p.code_stride[kv][0] + offset * p.code_stride[kv][1] +
                        head * p.code_stride[kv][2] + ch * 8);
                    e[i][kv] = p.scales[kv][page * p.scale_stride[kv][0] + block * p.scale_stride[kv][1] +
                                            head * p.scale_stride[kv][2]];
                }
            } else {
                if (slot != -1 && rest[i] == 0) atomicOr(p.status, DECODE_BAD_CACHE_SLOT);
                codes[i][0] = codes[i][1] = make_uint2(0u, 0u);
                e[i][0] = e[i][1] = 127;
            }
        }
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            if (token[i] < 0) continue;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const float by = scale_of(e[i][kv]);
                const uint32_t in[2] = {codes[i][kv].x, codes[i][kv].y};
                uint32_t out[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 a = Half2<__half>::unpack(codes_to_half2(in[h]));
                    const float2 b = Half2<__half>::unpack(codes_to_half2(in[h] >> 16));
                    out[2 * h] = Half2<T>::pack(a.x * by, a.y * by);
                    out[2 * h + 1] = Half2<T>::pack(b.x * by, b.y * by);
                }
                *reinterpret_cast<uint4*>(p.y[kv] + (t0 + token[i]) * p.y_stride[kv][0] +
                                          rest[i] / (D / 8) * p.y_stride[kv][1] + rest[i] % (D / 8) * 8) =
                    make_uint4(out[0], out[1], out[2], out[3]);
            }
        }
    }
}

template <typename T, int D, int kHold>
int quantize(const QuantizeParams& p, cudaStream_t stream)
{
    const int64_t windows = (static_cast<int64_t>(p.tokens) + p.window - 1) / p.window;
    const int groups = (2 / kKinds<D> * p.heads + p.per - 1) / p.per;
    const cudaError_t e = launch(p.window > 1 ? quantize_cache_kernel<T, D, kHold, true>
                                              : quantize_cache_kernel<T, D, kHold, false>,
                                 dim3(static_cast<uint32_t>(windows), groups), dim3(kWarps * 32), 0, stream, p);
    if (e != cudaSuccess)
        return fail(DECODE_ERR_CUDA, "quantize_cache_kernel: %s", cudaGetErrorString(e));
    return DECODE_OK;
}

template <typename T, int D>
int dequantize(const DequantizeParams& p, cudaStream_t stream)
{
    const int64_t blocks = (static_cast<int64_t>(p.tokens) + p.at_once - 1) / p.at_once;
    const cudaError_t e = launch(dequantize_cache_kernel<T, D>, dim3(static_cast<uint32_t>(blocks)),
                                 dim3(256), 0, stream, p);
    if (e != cudaSuccess)
        return fail(DECODE_ERR_CUDA, "dequantize_cache_kernel: %s", cudaGetErrorString(e));
    return DECODE_OK;
}

// The checks of both calls; fills in what their parameters share.  Args: either argument struct.
template <typename Args>
int take_cache(CacheParams& p, int64_t (&half_stride)[2][2], const Args* a)
{
    if (a->dtype != DECODE_F16 && a->dtype != DECODE_BF16)
        return fail(DECODE_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
    if (a->tokens < 0) return fail(DECODE_ERR_INVALID_ARG, "negative size");
    const int rc = check_cache(a->pages, a->page_size, a->block_size, a->h_k, a->head_dim);
    if (rc != DECODE_OK || a->tokens == 0) return rc;
    if (!a->k || !a->v || !a->slots || (a->pages > 0 && (!a->k_cache || !a->v_cache || !a->k_scale ||
                                                         !a->v_scale)))
        return fail(DECODE_ERR_INVALID_ARG, "null pointer");
    if (misaligned(a->k) || misaligned(a->v) || misaligned(a->k_cache) || misaligned(a->v_cache))
        return fail(DECODE_ERR_UNSUPPORTED, "keys, values and codes must be 16-byte aligned");
    const int64_t rows[2] = {a->tokens, a->h_k};
    if (!take_strides(half_stride[0], a->k_stride, rows, 8) ||
        !take_strides(half_stride[1], a->v_stride, rows, 8))
        return fail(DECODE_ERR_UNSUPPORTED, "strides of k and v must be multiples of 8");
    const int64_t cs[3] = {a->pages, a->page_size, a->h_k};
    const int64_t ss[3] = {a->pages, a->page_size / a->block_size, a->h_k};
    if (!take_strides(p.code_stride[0], a->k_cache_stride, cs, 16) ||
        !take_strides(p.code_stride[1], a->v_cache_stride, cs, 16))
        return fail(DECODE_ERR_UNSUPPORTED, "cache strides must be multiples of 16");
    take_strides(p.scale_stride[0], a->k_scale_stride, ss, 1);
    take_strides(p.scale_stride[1], a->v_scale_stride, ss, 1);
    constexpr int64_t kMost = (int64_t(1) << 31) - 1;
    if (a->tokens > kMost - 64 || a->h_k > (1 << 15) || a->pages > kMost / a->page_size)
        return fail(DECODE_ERR_UNSUPPORTED, "too many tokens, heads or places for one call");
    p.codes[0] = static_cast<uint8_t*>(const_cast<void*>(static_cast<const void*>(a->k_cache)));
    p.codes[1] = static_cast<uint8_t*>(const_cast<void*>(static_cast<const void*>(a->v_cache)));
    p.scales[0] = static_cast<uint8_t*>(const_cast<void*>(static_cast<const void*>(a->k_scale)));
    p.scales[1] = static_cast<uint8_t*>(const_cast<void*>(static_cast<const void*>(a->v_scale)));
    p.slots = a->slots;
    p.tokens = static_cast<int32_t>(a->tokens);
    p.heads = static_cast<int32_t>(a->h_k);
    p.page_size = static_cast<int32_t>(a->page_size);
    p.page_shift = shift_of(a->page_size);
    p.block = a->block_size;
    p.block_shift = shift_of(a->block_size);
    p.places = static_cast<int32_t>(a->pages * a->page_size);
    return DECODE_OK;
}

}  // namespace

extern "C" {

int decode_quantize_cache(const decode_quantize_cache_args* a, cudaStream_t stream)
{
    clear_error();
    if (a == nullptr) return fail(DECODE_ERR_INVALID_ARG, "args is null");
    QuantizeParams p{};
    const int rc = take_cache(p, p.x_stride, a);
    if (rc != DECODE_OK || a->tokens == 0) return rc;
    const int64_t d = a->head_dim, rows[2] = {a->tokens, a->h_k};
    const int64_t cs[3] = {a->pages, a->page_size, a->h_k};
    const int64_t ss[3] = {a->pages, a->page_size / a->block_size, a->h_k};
    const int shared = refuse_shared({{"k_cache", a->k_cache, 1, d, cs, p.code_stride[0]},
                                      {"v_cache", a->v_cache, 1, d, cs, p.code_stride[1]},
                                      {"k_scale", a->k_scale, 1, 1, ss, p.scale_stride[0]},
                                      {"v_scale", a->v_scale, 1, 1, ss, p.scale_stride[1]}},
                                     {{"k", a->k, 2, d, rows, p.x_stride[0]},
                                      {"v", a->v, 2, d, rows, p.x_stride[1]},
                                      {"slots", a->slots, 4, a->tokens}});
    if (shared != DECODE_OK) return shared;
    const int sms = sm_count();
    p.status = status_word();
    if (sms == 0 || p.status == nullptr) return DECODE_ERR_CUDA;
    p.x[0] = static_cast<const uint16_t*>(a->k);
    p.x[1] = static_cast<const uint16_t*>(a->v);
    const int each = d == 256 ? 2 * p.heads : p.heads;      // warps' work of a token
    p.per = each < kWarps ? each : kWarps;
    // A warp takes the blocks that begin in its window of tokens: of few tokens, each of which may be a block's
    // only one, a window holds one; of more as many as leave the GPU 12 to 24 warps an SM, for windows in which
    // no block begins cost a warp all the same.  8 heads of 128, tokens of one sequence / of as many sequences, us:
    // 400 with windows of 1, 2, 4 4.8 / 4.8, 4.4 / 4.8, 4.2 / 6.0; 1200 of 4, 8 4.7 / 6.3, 4.6 / 8.4; 2400 of
    // 8, 16 4.8 / 8.7, 4.9 / 13.1.
    p.window = 1;
    while (p.window < kWindow && static_cast<int64_t>(p.tokens) * each > static_cast<int64_t>(sms) * 24 * p.window)
        p.window *= 2;
    const bool bf16 = a->dtype == DECODE_BF16;
    if (d == 64) return bf16 ? quantize<__nv_bfloat16, 64, 4>(p, stream) : quantize<__half, 64, 4>(p, stream);
    // (8 rows do for blocks of 8.  16 are two rounds of reads: worth it where the GPU is filled several times,
    // 20000 tokens of 8 heads 24.6 us for 25.7, not before, 4800 6.5 for 4.9, 400 4.9 for 4.6.)
    if (d == 128 && (p.block <= 8 ||
                     (p.block <= 16 && static_cast<int64_t>(p.tokens) * each >= static_cast<int64_t>(sms) * 1024)))
        return bf16 ? quantize<__nv_bfloat16, 128, 4>(p, stream) : quantize<__half, 128, 4>(p, stream);
    if (d == 128) return bf16 ? quantize<__nv_bfloat16, 128, 8>(p, stream) : quantize<__half, 128, 8>(p, stream);
    return bf16 ? quantize<__nv_bfloat16, 256, 16>(p, stream) : quantize<__half, 256, 16>(p, stream);
}

int decode_dequantize_cache(const decode_dequantize_cache_args* a, cudaStream_t stream)
{
    clear_error();
    if (a == nullptr) return fail(DECODE_ERR_INVALID_ARG, "args is null");
    DequantizeParams p{};
    const int rc = take_cache(p, p.y_stride, a);
    if (rc != DECODE_OK || a->tokens == 0) return rc;
    const int64_t d = a->head_dim, rows[2] = {a->tokens, a->h_k};
    const int64_t cs[3] = {a->pages, a->page_size, a->h_k};
    const int64_t ss[3] = {a->pages, a->page_size / a->block_size, a->h_k};
    const int shared = refuse_shared({{"k", a->k, 2, d, rows, p.y_stride[0]},
                                      {"v", a->v, 2, d, rows, p.y_stride[1]}},
                                     {{"k_cache", a->k_cache, 1, d, cs, p.code_stride[0]},
                                      {"v_cache", a->v_cache, 1, d, cs, p.code_stride[1]},
                                      {"k_scale", a->k_scale, 1, 1, ss, p.scale_stride[0]},
                                      {"v_scale", a->v_scale, 1, 1, ss, p.scale_stride[1]},
                                      {"slots", a->slots, 4, a->tokens}});
    if (shared != DECODE_OK) return shared;
    p.status = status_word();
    if (p.status == nullptr) return DECODE_ERR_CUDA;
    p.y[0] = static_cast<uint16_t*>(a->k);
    p.y[1] = static_cast<uint16_t*>(a->v);
    p.units = static_cast<int32_t>(a->h_k * d / 8);
    p.at_once = p.units < 512 ? 512 / p.units : 1;
    p.magic = static_cast<uint32_t>(((uint64_t(1) << 32) + p.units - 1) / p.units);
    const bool bf16 = a->dtype == DECODE_BF16;
    if (d == 64)
        return bf16 ? dequantize<__nv_bfloat16, 64>(p, stream) : dequantize<__half, 64>(p, stream);
    if (d == 128)
        return bf16 ? dequantize<__nv_bfloat16, 128>(p, stream) : dequantize<__half, 128>(p, stream);
    return bf16 ? dequantize<__nv_bfloat16, 256>(p, stream) : dequantize<__half, 256>(p, stream);
}

}  // extern "C"
