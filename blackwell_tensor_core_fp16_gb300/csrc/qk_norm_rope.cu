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
// kLanes heads at a time.  A block takes one token: its angles are the same for every head, so each
// lane reads its cosines and sines once and keeps them in registers.  In the split pairing element
// e's partner lies rot / 2 elements, that is rot / 16 lanes, away and comes by shuffle; in the
// interleaved pairing it is the lane's own neighbour.
#include <cstdint>

#include "decode_common.cuh"

namespace {

using namespace decode;

constexpr int kUnroll = 4;       // heads a lane has in flight
constexpr int kMaxWarps = 8;
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
    int32_t h_q, h_k, head_dim, rot, axes, page_size, norm;
    int32_t section_end[DECODE_MAX_AXES];   // first pair of the next axis
    float eps;
};

template <typename T>
__device__ __forceinline__ void unpack8(float (&x)[8], uint4 b)
{
    const float2 a0 = Half2<T>::unpack(b.x), a1 = Half2<T>::unpack(b.y),
                 a2 = Half2<T>::unpack(b.z), a3 = Half2<T>::unpack(b.w);
    x[0] = a0.x, x[1] = a0.y, x[2] = a1.x, x[3] = a1.y;
    x[4] = a2.x, x[5] = a2.y, x[6] = a3.x, x[7] = a3.y;
}

template <typename T, int kLanes, Pairing kPairing>
__global__ void __launch_bounds__(kMaxWarps * 32) qk_norm_rope_kernel(const NormParams p)
{
    constexpr int kHeads = 32 / kLanes;              // heads of a warp at a time
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 31, l = lane % kLanes;
    const int warps = blockDim.x >> 5;
    const int first = (threadIdx.x >> 5) * kHeads + lane / kLanes;
    const int e = 8 * l;                             // the lane's first element
    const bool in_head = e < p.head_dim, in_rot = e < p.rot;
    const int half = p.rot / 2;
    const int total = p.h_q + p.h_k + (p.v != nullptr ? p.h_k : 0);

    dep_launch();
    dep_wait();

    // What the indices say is loaded first, the rows next, and the angles, which wait for the
    // positions, after them.
    int32_t pos[DECODE_MAX_AXES];
    if constexpr (kPairing != kNone) {
#pragma unroll
        for (int x = 0; x < DECODE_MAX_AXES; ++x)
            pos[x] = x < p.axes ? p.positions[x * p.position_stride + t] : 0;
    }
    int32_t slot = p.k_cache != nullptr ? p.slots[t] : -1;
    auto row_of = [&](int h) {
        return h < p.h_q           ? p.q + t * p.q_stride[0] + h * p.q_stride[1]
               : h < p.h_q + p.h_k ? p.k + t * p.k_stride[0] + (h - p.h_q) * p.k_stride[1]
                                   : p.v + t * p.v_stride[0] + (h - p.h_q - p.h_k) * p.v_stride[1];
    };
    uint4 in[kUnroll];
    auto fetch = [&](int h0) {
#pragma unroll
        for (int x = 0; x < kUnroll; ++x) {
            const int h = h0 + x * warps * kHeads + first;
            in[x] = make_uint4(0u, 0u, 0u, 0u);
            if (in_head && h < total) in[x] = *reinterpret_cast<const uint4*>(row_of(h) + e);
        }
    };
    fetch(0);
    const bool weights = p.q_weight != nullptr || p.k_weight != nullptr;
    uint4 wq = make_uint4(0u, 0u, 0u, 0u), wk = wq;
    if (in_head && p.q_weight) wq = *reinterpret_cast<const uint4*>(p.q_weight + e);
    if (in_head && p.k_weight) wk = *reinterpret_cast<const uint4*>(p.k_weight + e);

    // The token's angles at the lane's elements, and whether its positions lie in the table.
    bool ok = true;
    constexpr int kPairs = kPairing == kInterleaved ? 4 : 8;   // pairs that the lane meets
    float cs[kPairs], sn[kPairs];
    if constexpr (kPairing != kNone) {
#pragma unroll
        for (int x = 0; x < DECODE_MAX_AXES; ++x)
            ok = ok && pos[x] >= 0 && (x >= p.axes || pos[x] < p.table_rows);
#pragma unroll
        for (int c = 0; c < kPairs; ++c) cs[c] = 1.f, sn[c] = 0.f;
        if (ok && in_rot) {
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
            if (kPairing == kSplit && e < half) {
#pragma unroll
                for (int c = 0; c < kPairs; ++c) sn[c] = -sn[c];
            }
        }
        if (!ok && threadIdx.x == 0) atomicOr(p.status, DECODE_BAD_POSITION);
    }
    // The lane that holds the partners of this lane's elements (split pairing).
    const int partner = !in_rot ? lane : lane + (e < half ? half / 8 : -(half / 8));

    if (!ok) slot = -1;
    if (slot < -1 || slot >= p.cache_slots) {
        if (threadIdx.x == 0) atomicOr(p.status, DECODE_BAD_CACHE_SLOT);
        slot = -1;
    }
    const int32_t page = slot < 0 ? 0 : static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page_size);
    const int32_t off = slot < 0 ? 0 : slot - page * p.page_size;
    uint16_t* const k_row = p.k_cache == nullptr
                                ? p.k_out + t * p.k_out_stride[0]
                                : p.k_cache + page * p.k_cache_stride[0] + off * p.k_cache_stride[1];
    const int64_t k_head = p.k_cache == nullptr ? p.k_out_stride[1] : p.k_cache_stride[2];
    const float inv_d = p.norm == DECODE_NORM_RMS ? 1.f / p.head_dim : 1.f;

    // the trip counts are the same for all lanes: the shuffles need the whole warp
    for (int h0 = 0; h0 < total; h0 += warps * kHeads * kUnroll) {
        if (h0 > 0) fetch(h0);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (h0 + u * warps * kHeads >= total) break;
            const int h = h0 + u * warps * kHeads + first;
            const bool is_q = h < p.h_q, is_v = h >= p.h_q + p.h_k;
            float x[8];
            unpack8<T>(x, in[u]);
            float f = 1.f;
            if (p.norm != DECODE_NORM_NONE) {
                float s = 0.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) s = fmaf(x[c], x[c], s);
#pragma unroll
                for (int m = 1; m < kLanes; m *= 2) s += __shfl_xor_sync(0xffffffffu, s, m);
                f = rsqrtf(fmaf(s, inv_d, p.eps));
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) x[c] *= f;
            if (weights && (is_q ? p.q_weight : p.k_weight) != nullptr) {
                float w[8];
                unpack8<T>(w, is_q ? wq : wk);
#pragma unroll
                for (int c = 0; c < 8; ++c) x[c] *= w[c];
            }
            if constexpr (kPairing == kSplit) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float y = __shfl_sync(0xffffffffu, x[c], partner);
                    x[c] = in_rot ? fmaf(x[c], cs[c], y * sn[c]) : x[c];
                }
            } else if constexpr (kPairing == kInterleaved) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float a = x[2 * c], b = x[2 * c + 1];
                    x[2 * c] = in_rot ? fmaf(a, cs[c], -b * sn[c]) : a;
                    x[2 * c + 1] = in_rot ? fmaf(b, cs[c], a * sn[c]) : b;
                }
            }
            uint4 b = in[u];
            if (!is_v) {
                b = make_uint4(Half2<T>::pack(x[0], x[1]), Half2<T>::pack(x[2], x[3]),
                               Half2<T>::pack(x[4], x[5]), Half2<T>::pack(x[6], x[7]));
                if (!ok) b = make_uint4(0u, 0u, 0u, 0u);
            }
            if (!in_head || h >= total) continue;
            if (is_q)
                *reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride[0] +
                                          h * p.q_out_stride[1] + e) = b;
            else if (p.k_cache == nullptr || slot >= 0)
                *reinterpret_cast<uint4*>(
                    (is_v ? p.v_cache + page * p.v_cache_stride[0] + off * p.v_cache_stride[1] +
                                (h - p.h_q - p.h_k) * p.v_cache_stride[2]
                          : k_row + (h - p.h_q) * k_head) + e) = b;
        }
    }
}

template <typename T, int kLanes>
cudaError_t run(const NormParams& p, int64_t tokens, bool interleaved, cudaStream_t stream)
{
    auto* kernel = p.rot == 0    ? qk_norm_rope_kernel<T, kLanes, kNone>
                   : interleaved ? qk_norm_rope_kernel<T, kLanes, kInterleaved>
                                 : qk_norm_rope_kernel<T, kLanes, kSplit>;
    // as many warps as the token's heads keep busy with kUnroll heads a lane
    constexpr int kPass = 32 / kLanes * kUnroll;
    const int total = p.h_q + (p.v != nullptr ? 2 : 1) * p.h_k;
    const int warps = (total + kPass - 1) / kPass;
    return launch(kernel, dim3(static_cast<uint32_t>(tokens)),
                  dim3(32 * (warps < 1 ? 1 : warps > kMaxWarps ? kMaxWarps : warps)), 0, stream, p);
}

template <typename T>
cudaError_t run(const NormParams& p, int64_t tokens, bool interleaved, cudaStream_t stream)
{
    return p.head_dim <= 64    ? run<T, 8>(p, tokens, interleaved, stream)
           : p.head_dim <= 128 ? run<T, 16>(p, tokens, interleaved, stream)
                               : run<T, 32>(p, tokens, interleaved, stream);
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
    if (a->tokens >= (int64_t(1) << 31) || a->h_q + 2 * a->h_k >= (1 << 24))
        return fail(DECODE_ERR_UNSUPPORTED, "too many tokens or heads for one call");

    p.status = status_word();
    if (p.status == nullptr) return DECODE_ERR_CUDA;
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
                              ? run<__nv_bfloat16>(p, a->tokens, inter, stream)
                              : run<__half>(p, a->tokens, inter, stream);
    if (e != cudaSuccess)
        return fail(DECODE_ERR_CUDA, "qk_norm_rope_kernel: %s", cudaGetErrorString(e));
    return DECODE_OK;
}
