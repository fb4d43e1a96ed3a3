// The gated delta rule token by token on a pool of fp32 states (C ABI in include/decode.h).
//
//     S' = alpha S;  u = beta (v - S' k);  S = S' + u k^T;  o = scale S q
//
// Every value row of S evolves on its own: with s a row, both products that a token needs are
// taken of the row before its update,
//     p = s . k,   r = s . q,   u = beta (v - alpha p),   o = scale (alpha r + u (k . q)),
//     s <- alpha s + u k,
// so their two reductions overlap and the row is read once.  A state is 65,536 bytes and a token
// adds about 1 KB to it, so the bytes of the states, read once and written once, are the floor:
// the kernel is a copy with 6 flops per element on the way.
//
// Layout.  Eight lanes share a row of 128 floats, lane l of them holding the float4s l, l + 8,
// l + 16, l + 24 (each load of the eight lanes is one 128-byte line), and a lane group has four
// neighbouring rows, so a warp keeps 16 rows in 64 registers a thread for all of a call's tokens
// and has 8 KB of loads in flight.
#include <cstdint>

#include "decode_common.cuh"

namespace {

using namespace decode;

constexpr int kD = 128;
constexpr int kRows = 4;                 // rows of a lane group
constexpr int kWarpRows = 4 * kRows;     // rows of a warp

struct StepParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const float* alpha;
    const float* beta;
    float* state;
    const int32_t* slots;
    uint16_t* o;
    uint32_t* status;
    int64_t q_stride[3], k_stride[3], v_stride[3];
    int64_t alpha_stride[2], beta_stride[2];
    int64_t state_stride;
    int32_t tokens, h_v, h_o, kgroup, qgroup, queries, n_slots;
    float scale;
};

// Elements 4 (l + 8 j) .. + 3, j = 0 .. 3, of a row of 128.
template <typename T>
__device__ __forceinline__ void load_row(float (&x)[16], const uint16_t* row, int l)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint2 b = *reinterpret_cast<const uint2*>(row + 4 * (l + 8 * j));
        const float2 lo = Half2<T>::unpack(b.x), hi = Half2<T>::unpack(b.y);
        x[4 * j] = lo.x, x[4 * j + 1] = lo.y, x[4 * j + 2] = hi.x, x[4 * j + 3] = hi.y;
    }
}

__device__ __forceinline__ float sum8(float x)
{
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    return x + __shfl_xor_sync(0xffffffffu, x, 4);
}

// Block: kWarps warps, 16 value rows each, of one (sequence, value head).
template <typename T, int kWarps>
__global__ void __launch_bounds__(kWarps * 32) gdn_step_kernel(const StepParams p)
{
    constexpr int kParts = kD / (kWarpRows * kWarps);    // blocks of a state
    const int item = blockIdx.x / kParts, part = blockIdx.x % kParts;
    const int i = item / p.h_v, j = item % p.h_v;
    const int lane = threadIdx.x & 31, l = lane & 7;
    const int row0 = (part * kWarps + (threadIdx.x >> 5)) * kWarpRows + (lane >> 3) * kRows;

    dep_launch();
    dep_wait();
    const int slot = p.slots ? p.slots[i] : i;
    const bool active = slot >= 0 && slot < p.n_slots;
    const int64_t out0 = (static_cast<int64_t>(i) * p.tokens * p.h_o +
                          static_cast<int64_t>(j) * p.queries) * kD + row0;
    if (!active) {
        if (slot != -1 && threadIdx.x == 0) atomicOr(p.status, DECODE_BAD_STATE_SLOT);
        if (l == 0)
            for (int t = 0; t < p.tokens; ++t)
                for (int g = 0; g < p.queries; ++g)
                    *reinterpret_cast<uint2*>(
                        p.o + out0 + (static_cast<int64_t>(t) * p.h_o + g) * kD) =
                        make_uint2(0u, 0u);
        return;
    }

    float4* state = reinterpret_cast<float4*>(p.state + slot * p.state_stride +
                                              (static_cast<int64_t>(j) * kD + row0) * kD) + l;
    float s[kRows][16];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float4 x = state[r * (kD / 4) + 8 * c];
            s[r][4 * c] = x.x, s[r][4 * c + 1] = x.y, s[r][4 * c + 2] = x.z, s[r][4 * c + 3] = x.w;
        }

    const uint16_t* kp = p.k + i * p.k_stride[0] + (j / p.kgroup) * p.k_stride[2];
    const uint16_t* vp = p.v + i * p.v_stride[0] + j * p.v_stride[2] + row0;
    const uint16_t* qp = p.q + i * p.q_stride[0] +
                         static_cast<int64_t>(p.queries > 1 ? j * p.queries : j / p.qgroup) *
                             p.q_stride[2];
    const float* ap = p.alpha + i * p.alpha_stride[0] + j;
    const float* bp = p.beta + i * p.beta_stride[0] + j;

    for (int t = 0; t < p.tokens; ++t) {
        float k[16];
        load_row<T>(k, kp + t * p.k_stride[1], l);
        const float alpha = ap[t * p.alpha_stride[1]], beta = bp[t * p.beta_stride[1]];
        const uint2 vb = *reinterpret_cast<const uint2*>(vp + t * p.v_stride[1]);
        const float2 v01 = Half2<T>::unpack(vb.x), v23 = Half2<T>::unpack(vb.y);
        const float v[kRows] = {v01.x, v01.y, v23.x, v23.y};
        float u[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float d = 0.f;
#pragma unroll
            for (int c = 0; c < 16; ++c) d = fmaf(s[r][c], k[c], d);
            u[r] = beta * (v[r] - alpha * sum8(d));
        }
        for (int g = 0; g < p.queries; ++g) {
            float q[16];
            load_row<T>(q, qp + t * p.q_stride[1] + g * p.q_stride[2], l);
            float kq = 0.f;
#pragma unroll
            for (int c = 0; c < 16; ++c) kq = fmaf(k[c], q[c], kq);
            kq = sum8(kq);
            float o[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float d = 0.f;
#pragma unroll
                for (int c = 0; c < 16; ++c) d = fmaf(s[r][c], q[c], d);
                o[r] = p.scale * fmaf(alpha, sum8(d), u[r] * kq);
            }
            if (l == 0)
                *reinterpret_cast<uint2*>(p.o + out0 +
                                          (static_cast<int64_t>(t) * p.h_o + g) * kD) =
                    make_uint2(Half2<T>::pack(o[0], o[1]), Half2<T>::pack(o[2], o[3]));
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int c = 0; c < 16; ++c) s[r][c] = fmaf(u[r], k[c], alpha * s[r][c]);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            state[r * (kD / 4) + 8 * c] =
                make_float4(s[r][4 * c], s[r][4 * c + 1], s[r][4 * c + 2], s[r][4 * c + 3]);
}

}  // namespace

extern "C" int decode_gdn_step(const decode_gdn_step_args* a, cudaStream_t stream)
{
    clear_error();
    if (a == nullptr) return fail(DECODE_ERR_INVALID_ARG, "args is null");
    if (a->n < 0 || a->tokens < 0 || a->n_slots < 0 || a->h_q <= 0 || a->h_k <= 0 || a->h_v <= 0)
        return fail(DECODE_ERR_INVALID_ARG, "negative size or no heads");
    if (a->dtype != DECODE_F16 && a->dtype != DECODE_BF16)
        return fail(DECODE_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
    if (a->h_v % a->h_k != 0 || (a->h_q != a->h_k && a->h_q % a->h_v != 0))
        return fail(DECODE_ERR_INVALID_ARG, "heads q %lld, k %lld, v %lld form no supported layout",
                    (long long)a->h_q, (long long)a->h_k, (long long)a->h_v);
    if (a->head_dim != kD)
        return fail(DECODE_ERR_UNSUPPORTED, "head_dim %lld (128 only)", (long long)a->head_dim);
    const int64_t queries = a->h_q == a->h_k ? 1 : a->h_q / a->h_v;
    if (queries > 8) return fail(DECODE_ERR_UNSUPPORTED, "more than 8 query heads per state head");
    if (a->n == 0 || a->tokens == 0) return DECODE_OK;
    if (!a->q || !a->k || !a->v || !a->alpha || !a->beta || !a->state || !a->o)
        return fail(DECODE_ERR_INVALID_ARG, "null pointer");
    if (!a->slots && a->n > a->n_slots)
        return fail(DECODE_ERR_INVALID_ARG, "%lld sequences but %lld states", (long long)a->n,
                    (long long)a->n_slots);
    if (misaligned(a->q) || misaligned(a->k) || misaligned(a->v) || misaligned(a->state) ||
        misaligned(a->o))
        return fail(DECODE_ERR_UNSUPPORTED, "q, k, v, state and o must be 16-byte aligned");
    for (int d = 0; d < 3; ++d)
        if (a->q_stride[d] % 8 || a->k_stride[d] % 8 || a->v_stride[d] % 8)
            return fail(DECODE_ERR_UNSUPPORTED, "strides of q, k and v must be multiples of 8");
    if (a->state_stride % 4 || (a->n_slots > 1 && a->state_stride < a->h_v * kD * kD))
        return fail(DECODE_ERR_INVALID_ARG, "state_stride %lld", (long long)a->state_stride);
    constexpr int kWarps = 2;
    const int64_t blocks = a->n * a->h_v * (kD / (kWarpRows * kWarps));
    if (a->n >= (int64_t(1) << 31) / (a->h_v * 8) || a->tokens >= (1 << 24) ||
        a->n_slots >= (int64_t(1) << 31))
        return fail(DECODE_ERR_UNSUPPORTED, "too many states or tokens for one call");

    StepParams p{};
    p.status = status_word();
    if (p.status == nullptr) return DECODE_ERR_CUDA;
    p.q = static_cast<const uint16_t*>(a->q);
    p.k = static_cast<const uint16_t*>(a->k);
    p.v = static_cast<const uint16_t*>(a->v);
    p.alpha = a->alpha;
    p.beta = a->beta;
    p.state = a->state;
    p.slots = a->slots;
    p.o = static_cast<uint16_t*>(a->o);
    for (int d = 0; d < 3; ++d) {
        p.q_stride[d] = a->q_stride[d];
        p.k_stride[d] = a->k_stride[d];
        p.v_stride[d] = a->v_stride[d];
    }
    for (int d = 0; d < 2; ++d) {
        p.alpha_stride[d] = a->alpha_stride[d];
        p.beta_stride[d] = a->beta_stride[d];
    }
    p.state_stride = a->state_stride;
    p.tokens = static_cast<int32_t>(a->tokens);
    p.h_v = static_cast<int32_t>(a->h_v);
    p.h_o = static_cast<int32_t>(queries > 1 ? a->h_q : a->h_v);
    p.kgroup = static_cast<int32_t>(a->h_v / a->h_k);
    p.qgroup = a->h_q == a->h_k ? p.kgroup : 1;
    p.queries = static_cast<int32_t>(queries);
    p.n_slots = static_cast<int32_t>(a->n_slots);
    p.scale = a->scale;
    auto* kernel = a->dtype == DECODE_BF16 ? gdn_step_kernel<__nv_bfloat16, kWarps>
                                           : gdn_step_kernel<__half, kWarps>;
    const cudaError_t e = launch(kernel, dim3(static_cast<uint32_t>(blocks)), dim3(kWarps * 32), 0,
                                 stream, p);
    if (e != cudaSuccess)
        return fail(DECODE_ERR_CUDA, "gdn_step_kernel: %s", cudaGetErrorString(e));
    return DECODE_OK;
}
