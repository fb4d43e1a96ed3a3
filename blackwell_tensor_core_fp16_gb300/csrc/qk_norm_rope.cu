// Norm of each query and key head, position rotation and write to the paged cache in one pass
// (C ABI in include/decode.h).
//
//     y = x * rsqrt(sum x^2 [/ d] + eps) * w;   (a, b) <- (a cos - b sin, b cos + a sin)
//
// Every element is read once and written once, with a handful of flops in between: the kernel is
// a copy bound by HBM, or by its launch when there are few tokens.
//
// Layout.  A lane holds 8 neighbouring elements (one 16-byte access), kLanes = 8, 16 or 32 lanes
// a head (head_dim up to 64, 128, 256), so a head's sum is a few shuffles and a warp takes 32 /
// kLanes heads at a time.  In the split pairing element e's partner lies rot / 2 elements, that is
// rot / 16 lanes, away and comes by shuffle, still as 16-bit pairs; in the interleaved pairing it
// is the lane's own neighbour.
//
// Norm and rotation are one linear map of a row up to its norm: with f the row's factor,
//     y_e = f (x_e (w_e cos) + x_partner (+-w_partner sin)),
// and the two factors in brackets are the same for all of a token's query (or key) heads.  So a
// warp's unit of work is one token and a run of its heads of one kind: it forms the factors once
// and spends two packed fp32 operations per pair of elements on each head.
#include <cstdint>

#include "decode_common.cuh"

namespace {

using namespace decode;

constexpr int kUnroll = 4;            // rows a lane has in flight
constexpr int kBlockWarps = 4;
enum Pairing { kNone, kSplit, kInterleaved };

struct NormParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* q_weight;
    const uint16_t* k_weight;
    const int32_t* positions;
    const float* table;
    uint16_t* q_out;
    uint16_t* k_out;
    uint16_t* k_cache;
    uint16_t* v_cache;
    const int32_t* slots;
    uint32_t* status;
    int64_t q_stride[2], k_stride[2], v_stride[2], q_out_stride[2], k_out_stride[2];
    int64_t k_cache_stride[3], v_cache_stride[3];
    int64_t position_stride, table_rows, cache_slots;
    uint32_t tokens, units;                 // units of a token: q_units, k_units, and as many of v
    int32_t q_units, k_units, steps;        // groups of heads of a unit
    int32_t h_q, h_k, head_dim, rot, axes, page_size, norm;
    int32_t section_end[DECODE_MAX_AXES];   // first pair of the next axis
    float eps;
};

__device__ __forceinline__ uint64_t pair_of(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 halves(uint64_t x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// The four 32-bit words of a lane's 8 elements, and their values as pairs.
template <typename T>
__device__ __forceinline__ uint64_t value2(uint32_t b)
{
    const float2 f = Half2<T>::unpack(b);
    return pair_of(f.x, f.y);
}
__device__ __forceinline__ uint32_t word(const uint4& b, int c)
{
    return c == 0 ? b.x : c == 1 ? b.y : c == 2 ? b.z : b.w;
}

// One unit: token t, `steps` groups of 32 / kLanes heads of its queries (kind 0), keys (1) or
// values (2), from the given group on.
template <typename T, int kLanes, Pairing kPairing>
__global__ void __launch_bounds__(kBlockWarps * 32, 6) qk_norm_rope_kernel(const NormParams p)
{
    constexpr int kHeads = 32 / kLanes;              // heads of a warp at a time
    const int lane = threadIdx.x & 31, l = lane % kLanes;
    const int e = 8 * l;                             // the lane's first element
    const bool in_head = e < p.head_dim, in_rot = e < p.rot;
    const int half = p.rot / 2;
    const uint32_t unit = blockIdx.x * kBlockWarps + (threadIdx.x >> 5);
    const uint32_t t = unit / p.units, part = unit - t * p.units;

    dep_launch();
    dep_wait();
    if (t >= p.tokens) return;
    const int kind = part < p.q_units ? 0 : part < p.q_units + p.k_units ? 1 : 2;
    const int heads = kind == 0 ? p.h_q : p.h_k;
    const int step0 = (part - (kind == 0 ? 0 : kind == 1 ? p.q_units : p.q_units + p.k_units)) * p.steps;
    int h = step0 * kHeads + lane / kLanes;          // the lane's head
    const int end = min(heads, (step0 + p.steps) * kHeads);

    // What the indices say is loaded first, the rows next, and the angles, which wait for the
    // positions, after them.
    int32_t pos[DECODE_MAX_AXES];
    if constexpr (kPairing != kNone) {
#pragma unroll
        for (int x = 0; x < DECODE_MAX_AXES; ++x)
            pos[x] = x < p.axes ? p.positions[x * p.position_stride + t] : 0;
    }
    int32_t slot = p.k_cache != nullptr && kind > 0 ? p.slots[t] : 0;

    const int64_t* from = kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride;
    const uint16_t* src = (kind == 0 ? p.q : kind == 1 ? p.k : p.v) + t * from[0] + h * from[1] + e;
    const int64_t src_step = kHeads * from[1];
    uint4 in[kUnroll];
    auto fetch = [&]() {
#pragma unroll
        for (int x = 0; x < kUnroll; ++x) {
            in[x] = make_uint4(0u, 0u, 0u, 0u);
            if (in_head && h + x * kHeads < end) in[x] = *reinterpret_cast<const uint4*>(src);
            src += src_step;
        }
    };
    fetch();

    const uint16_t* w = kind == 0 ? p.q_weight : p.k_weight;
    uint4 wb = make_uint4(0u, 0u, 0u, 0u);
    if (w != nullptr && in_head) wb = *reinterpret_cast<const uint4*>(w + e);

    // The factors of the lane's elements and of their partners.
    bool ok = true;
    uint64_t mine[4], other[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
        mine[c] = w != nullptr ? value2<T>(word(wb, c)) : pair_of(1.f, 1.f);
    const int partner = kPairing != kSplit || !in_rot ? lane
                        : lane + (e < half ? half / 8 : -(half / 8));
    if constexpr (kPairing != kNone) {
        if constexpr (kPairing == kSplit) {
#pragma unroll
            for (int c = 0; c < 4; ++c) other[c] = __shfl_sync(0xffffffffu, mine[c], partner);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 f = halves(mine[c]);
                other[c] = pair_of(f.y, f.x);
            }
        }
#pragma unroll
        for (int x = 0; x < DECODE_MAX_AXES; ++x)
            ok = ok && pos[x] >= 0 && (x >= p.axes || pos[x] < p.table_rows);
        if (ok && in_rot) {
            constexpr int kPairs = kPairing == kInterleaved ? 4 : 8;   // pairs that the lane meets
            const int pair0 = kPairing == kInterleaved ? e / 2 : (e < half ? e : e - half);
            auto axis_of = [&](int pair) {
                int axis = 0;
#pragma unroll
                for (int x = 1; x < DECODE_MAX_AXES; ++x)
                    axis += x < p.axes && pair >= p.section_end[x - 1];
                return axis;
            };
            auto table_row = [&](int axis) {
                int32_t at = pos[0];
#pragma unroll
                for (int x = 1; x < DECODE_MAX_AXES; ++x) at = axis == x ? pos[x] : at;
                return p.table + static_cast<int64_t>(at) * p.rot;
            };
            float cs[kPairs], sn[kPairs];
            const int axis = axis_of(pair0);
            if (axis == axis_of(pair0 + kPairs - 1)) {
                // one row of the table: its pairs lie side by side
                const float* row = table_row(axis) + pair0;
#pragma unroll
                for (int c = 0; c < kPairs; c += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(row + c);
                    const float4 y = *reinterpret_cast<const float4*>(row + half + c);
                    cs[c] = x.x, cs[c + 1] = x.y, cs[c + 2] = x.z, cs[c + 3] = x.w;
                    sn[c] = y.x, sn[c + 1] = y.y, sn[c + 2] = y.z, sn[c + 3] = y.w;
                }
            } else {
#pragma unroll
                for (int c = 0; c < kPairs; ++c) {
                    const float* row = table_row(axis_of(pair0 + c)) + pair0 + c;
                    cs[c] = row[0], sn[c] = row[half];
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if constexpr (kPairing == kInterleaved) {
                    mine[c] = mul2(mine[c], pair_of(cs[c], cs[c]));
                    other[c] = mul2(other[c], pair_of(-sn[c], sn[c]));
                } else {
                    const float sign = e < half ? -1.f : 1.f;
                    mine[c] = mul2(mine[c], pair_of(cs[2 * c], cs[2 * c + 1]));
                    other[c] = mul2(other[c], pair_of(sign * sn[2 * c], sign * sn[2 * c + 1]));
                }
            }
        }
        if (!ok && lane == 0 && part == 0) atomicOr(p.status, DECODE_BAD_POSITION);
    }

    // Where the rows go: to q_out or k_out, or to the token's place in a cache.
    uint16_t* dst;
    int64_t dst_step;
    if (kind == 0 || p.k_cache == nullptr) {
        const int64_t* to = kind == 0 ? p.q_out_stride : p.k_out_stride;
        dst = (kind == 0 ? p.q_out : p.k_out) + t * to[0] + h * to[1] + e;
        dst_step = kHeads * to[1];
    } else {
        if (slot < -1 || slot >= p.cache_slots) {
            if (lane == 0) atomicOr(p.status, DECODE_BAD_CACHE_SLOT);
            slot = -1;
        }
        if (slot < 0 || !ok) return;
        const int32_t page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page_size);
        const int32_t off = slot - page * p.page_size;
        const int64_t* to = kind == 1 ? p.k_cache_stride : p.v_cache_stride;
        dst = (kind == 1 ? p.k_cache : p.v_cache) + page * to[0] + off * to[1] + h * to[2] + e;
        dst_step = kHeads * to[2];
    }
    const float inv_d = p.norm == DECODE_NORM_RMS ? 1.f / p.head_dim : 1.f;

    for (int s = 0; s < p.steps; s += kUnroll) {     // trip counts do not depend on the lane
        if (s > 0) fetch();
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (s + u >= p.steps) break;
            uint4 b = in[u];
            if (kind < 2) {
                uint64_t x[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) x[c] = value2<T>(word(b, c));
                float f = 1.f;
                if (p.norm != DECODE_NORM_NONE) {
                    uint64_t s2 = mul2(x[0], x[0]);
#pragma unroll
                    for (int c = 1; c < 4; ++c) s2 = fma2(x[c], x[c], s2);
                    const float2 s1 = halves(s2);
                    float sum = s1.x + s1.y;
#pragma unroll
                    for (int m = 1; m < kLanes; m *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                    f = rsqrtf(fmaf(sum, inv_d, p.eps));
                }
                const uint64_t ff = pair_of(f, f);
                uint32_t out[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint64_t y = mul2(x[c], mine[c]);
                    if constexpr (kPairing == kSplit) {
                        const uint64_t z =
                            value2<T>(__shfl_sync(0xffffffffu, word(b, c), partner));
                        if (in_rot) y = fma2(z, other[c], y);
                    } else if constexpr (kPairing == kInterleaved) {
                        const float2 z = halves(x[c]);
                        if (in_rot) y = fma2(pair_of(z.y, z.x), other[c], y);
                    }
                    const float2 r = halves(mul2(y, ff));
                    out[c] = Half2<T>::pack(r.x, r.y);
                }
                b = ok ? make_uint4(out[0], out[1], out[2], out[3]) : make_uint4(0u, 0u, 0u, 0u);
            }
            if (in_head && h < end) *reinterpret_cast<uint4*>(dst) = b;
            h += kHeads;
            dst += dst_step;
        }
    }
}

template <typename T, int kLanes, Pairing kPairing>
cudaError_t run(NormParams p, int sms, cudaStream_t stream)
{
    constexpr int kHeads = 32 / kLanes;
    const int q_steps = (p.h_q + kHeads - 1) / kHeads, k_steps = (p.h_k + kHeads - 1) / kHeads;
    // Long units spend the least on their token's factors; shorter ones, when there would be less
    // than a wave of them, keep the GPU full and a single token's latency low.
    auto cut = [&](int steps) {
        p.steps = steps;
        p.q_units = (q_steps + steps - 1) / steps;
        p.k_units = (k_steps + steps - 1) / steps;
        p.units = p.q_units + p.k_units * (p.v != nullptr ? 2 : 1);
    };
    for (int steps = 2 * kUnroll; steps > 0; steps /= 2) {
        cut(steps);
        if (static_cast<int64_t>(p.tokens) * p.units >= static_cast<int64_t>(sms) * 24) break;
    }
    const int64_t blocks = (static_cast<int64_t>(p.tokens) * p.units + kBlockWarps - 1) / kBlockWarps;
    return launch(qk_norm_rope_kernel<T, kLanes, kPairing>, dim3(static_cast<uint32_t>(blocks)),
                  dim3(kBlockWarps * 32), 0, stream, p);
}

template <typename T, int kLanes>
cudaError_t run(const NormParams& p, bool interleaved, int sms, cudaStream_t stream)
{
    return p.rot == 0    ? run<T, kLanes, kNone>(p, sms, stream)
           : interleaved ? run<T, kLanes, kInterleaved>(p, sms, stream)
                         : run<T, kLanes, kSplit>(p, sms, stream);
}

template <typename T>
cudaError_t run(const NormParams& p, bool interleaved, int sms, cudaStream_t stream)
{
    return p.head_dim <= 64    ? run<T, 8>(p, interleaved, sms, stream)
           : p.head_dim <= 128 ? run<T, 16>(p, interleaved, sms, stream)
                               : run<T, 32>(p, interleaved, sms, stream);
}

}  // namespace

extern "C" int decode_qk_norm_rope(const decode_qk_norm_rope_args* a, cudaStream_t stream)
{
    clear_error();
    if (a == nullptr) return fail(DECODE_ERR_INVALID_ARG, "args is null");
    if (a->tokens < 0 || a->h_q < 0 || a->h_k < 0 || a->h_q + a->h_k == 0 || a->head_dim <= 0 ||
        a->rot < 0)
        return fail(DECODE_ERR_INVALID_ARG, "negative size or no heads");
    if (a->dtype != DECODE_F16 && a->dtype != DECODE_BF16)
        return fail(DECODE_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
    if (a->norm < DECODE_NORM_NONE || a->norm > DECODE_NORM_L2)
        return fail(DECODE_ERR_INVALID_ARG, "unknown norm %d", a->norm);
    if (a->head_dim % 8 || a->head_dim > 256)
        return fail(DECODE_ERR_UNSUPPORTED, "head_dim %lld (a multiple of 8 up to 256)",
                    (long long)a->head_dim);
    if (a->rot % 16 || a->rot > a->head_dim)
        return fail(DECODE_ERR_UNSUPPORTED, "rot %lld (a multiple of 16 up to head_dim)",
                    (long long)a->rot);
    if (a->rot > 0) {
        if (a->axes < 1 || a->axes > DECODE_MAX_AXES || a->table_rows < 0)
            return fail(DECODE_ERR_INVALID_ARG, "%lld axes, %lld table rows", (long long)a->axes,
                        (long long)a->table_rows);
        if (a->axes > 1) {
            int64_t sum = 0;
            for (int x = 0; x < a->axes; ++x) {
                if (a->sections[x] < 0) return fail(DECODE_ERR_INVALID_ARG, "negative section");
                sum += a->sections[x];
            }
            if (sum != a->rot / 2)
                return fail(DECODE_ERR_INVALID_ARG, "sections hold %lld pairs, rot / 2 is %lld",
                            (long long)sum, (long long)(a->rot / 2));
        }
    }
    if (a->tokens == 0) return DECODE_OK;
    const bool cache = a->k_cache != nullptr;
    if (cache != (a->v_cache != nullptr) || cache != (a->v != nullptr) ||
        cache != (a->slots != nullptr))
        return fail(DECODE_ERR_INVALID_ARG, "v, k_cache, v_cache and slots come together");
    if (cache && (a->pages < 0 || a->page_size <= 0 ||
                  a->pages >= (int64_t(1) << 31) / a->page_size))
        return fail(DECODE_ERR_INVALID_ARG, "%lld pages of %lld (fewer than 2^31 places)",
                    (long long)a->pages, (long long)a->page_size);
    if ((a->h_q > 0 && (!a->q || !a->q_out)) || (a->h_k > 0 && (!a->k || (!cache && !a->k_out))) ||
        (a->rot > 0 && (!a->positions || !a->table)))
        return fail(DECODE_ERR_INVALID_ARG, "null pointer");
    if (misaligned(a->q) || misaligned(a->k) || misaligned(a->v) || misaligned(a->q_out) ||
        misaligned(a->k_out) || misaligned(a->k_cache) || misaligned(a->v_cache) ||
        misaligned(a->q_weight) || misaligned(a->k_weight) || misaligned(a->table))
        return fail(DECODE_ERR_UNSUPPORTED, "16-bit tensors and the table must be 16-byte aligned");
    NormParams p{};
    if (!take_strides(p.q_stride, a->q_stride, {a->tokens, a->h_q}, 8) ||
        !take_strides(p.k_stride, a->k_stride, {a->tokens, a->h_k}, 8) ||
        !take_strides(p.q_out_stride, a->q_out_stride, {a->tokens, a->h_q}, 8) ||
        (!cache && !take_strides(p.k_out_stride, a->k_out_stride, {a->tokens, a->h_k}, 8)) ||
        (cache && !take_strides(p.v_stride, a->v_stride, {a->tokens, a->h_k}, 8)))
        return fail(DECODE_ERR_UNSUPPORTED, "strides must be multiples of 8");
    const int64_t cs[3] = {a->pages, a->page_size, a->h_k};
    if (cache && (!take_strides(p.k_cache_stride, a->k_cache_stride, cs, 8) ||
                  !take_strides(p.v_cache_stride, a->v_cache_stride, cs, 8)))
        return fail(DECODE_ERR_UNSUPPORTED, "cache strides must be multiples of 8");
    if (a->h_q >= (1 << 24) || a->h_k >= (1 << 24) ||
        a->tokens >= (int64_t(1) << 31) / (a->h_q + 2 * a->h_k))
        return fail(DECODE_ERR_UNSUPPORTED, "too many tokens or heads for one call");

    p.status = status_word();
    const int sms = sm_count();
    if (p.status == nullptr || sms == 0) return DECODE_ERR_CUDA;
    p.q = static_cast<const uint16_t*>(a->q);
    p.k = static_cast<const uint16_t*>(a->k);
    p.v = static_cast<const uint16_t*>(a->v);
    p.q_weight = static_cast<const uint16_t*>(a->q_weight);
    p.k_weight = static_cast<const uint16_t*>(a->k_weight);
    p.positions = a->positions;
    p.table = a->table;
    p.q_out = static_cast<uint16_t*>(a->q_out);
    p.k_out = static_cast<uint16_t*>(a->k_out);
    p.k_cache = static_cast<uint16_t*>(a->k_cache);
    p.v_cache = static_cast<uint16_t*>(a->v_cache);
    p.slots = a->slots;
    p.position_stride = a->position_stride;
    p.tokens = static_cast<uint32_t>(a->tokens);
    p.table_rows = a->table_rows;
    p.cache_slots = cache ? a->pages * a->page_size : 0;
    p.h_q = static_cast<int32_t>(a->h_q);
    p.h_k = static_cast<int32_t>(a->h_k);
    p.head_dim = static_cast<int32_t>(a->head_dim);
    p.rot = static_cast<int32_t>(a->rot);
    p.axes = a->rot > 0 ? static_cast<int32_t>(a->axes) : 0;
    p.page_size = cache ? static_cast<int32_t>(a->page_size) : 1;
    p.norm = a->norm;
    int32_t end = 0;
    for (int x = 0; x < DECODE_MAX_AXES; ++x) p.section_end[x] = end += a->sections[x];
    p.eps = a->eps;
    const bool inter = a->interleaved != 0;
    const cudaError_t e = a->dtype == DECODE_BF16
                              ? run<__nv_bfloat16>(p, inter, sms, stream)
                              : run<__half>(p, inter, sms, stream);
    if (e != cudaSuccess)
        return fail(DECODE_ERR_CUDA, "qk_norm_rope_kernel: %s", cudaGetErrorString(e));
    return DECODE_OK;
}
