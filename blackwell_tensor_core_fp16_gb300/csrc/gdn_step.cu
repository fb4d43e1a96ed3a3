// The gated delta rule token by token on a pool of fp32 states (C ABI in include/decode.h).
//
//     S' = alpha S;  u = beta (v - S' k);  S = S' + u k^T;  o = scale S q
//
// Every value row of S evolves on its own: with s a row, both products that a token needs are
// taken of the row before its update,
//     p = s . k,   r = s . q,   u = beta (v - alpha p),   o = scale (alpha r + u (k . q)),
//     s <- alpha s + u k,
// so their two reductions overlap (with several tokens o is taken of the row after it, below).
//
// What bounds it.  A state is 65,536 bytes and a token adds about 1 KB to it, so with one token
// the bytes of the states, read once and written once, are the floor: 256 sequences x 32 states
// (1.08 GB) take 156 us, 6.9 TB/s, which is what a plain copy reaches; one sequence of 16 states
// takes 2.7 us, its launch and two round trips to memory.  Each further token is a chain: a product
// of the rows with k, four shuffles, u, the rows' update, a product with q, four shuffles.  151
// sequences x 8 states with two queries each take 27.7 us with 2 tokens (86% of the copy rate),
// 34.2 us with 4 and 51.8 us with 8, issue slots 56% and FMA pipes 52% busy meanwhile at 14 warps
// an SM; 77 sequences x 4 tokens, two queries, take 19.4 us, issue slots 48% and FMA pipes 45%
// busy, the SMs 78% of the time.  (The chunked form on mma.m16n8k16 with operands in three bfloat16
// pieces was built and measured: 46 to 48 us for 2 to 8 tokens alike, bound by its chain of
// dependent products; it wins from 16 tokens on, where the prefill belongs.)
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

// Elements 4 (l + 8 j) .. + 3, j = 0 .. 3, of a row of 128, as eight pairs.
template <typename T>
__device__ __forceinline__ void load_row(uint64_t (&x)[8], const uint16_t* row, int l)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint2 b = *reinterpret_cast<const uint2*>(row + 4 * (l + 8 * j));
        const float2 lo = Half2<T>::unpack(b.x), hi = Half2<T>::unpack(b.y);
        x[2 * j] = pair(lo.x, lo.y), x[2 * j + 1] = pair(hi.x, hi.y);
    }
}
// Sums of d[0 .. 3] over a group of eight lanes, one row to a lane: lane l gets row l & 3, by
// halving the rows with the lanes (4 shuffles for the 12 of four butterflies).
__device__ __forceinline__ float sum_rows(const float (&d)[kRows], int l)
{
    const bool hi1 = l & 2, hi0 = l & 1;
    const float a = (hi1 ? d[2] : d[0]) + __shfl_xor_sync(0xffffffffu, hi1 ? d[0] : d[2], 2);
    const float b = (hi1 ? d[3] : d[1]) + __shfl_xor_sync(0xffffffffu, hi1 ? d[1] : d[3], 2);
    const float c = (hi0 ? b : a) + __shfl_xor_sync(0xffffffffu, hi0 ? a : b, 1);
    return c + __shfl_xor_sync(0xffffffffu, c, 4);
}

__device__ __forceinline__ float dot16(const uint64_t (&x)[8], const uint64_t (&y)[8])
{
    uint64_t a = mul2(x[0], y[0]), b = mul2(x[4], y[4]);
#pragma unroll
    for (int c = 1; c < 4; ++c) {
        a = fma2(x[c], y[c], a);
        b = fma2(x[4 + c], y[4 + c], b);
    }
    const float2 p = halves(a), q = halves(b);
    return (p.x + p.y) + (q.x + q.y);
}

__device__ __forceinline__ float sum8(float x)
{
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    return x + __shfl_xor_sync(0xffffffffu, x, 4);
}

template <typename T>
__device__ __forceinline__ float to_float(uint16_t x)
{
    return Half2<T>::unpack(x).x;
}
template <typename T>
__device__ __forceinline__ uint16_t from_float(float x)
{
    return static_cast<uint16_t>(Half2<T>::pack(x, 0.f));
}

// Block: kWarps warps, 16 value rows each, of one (sequence, value head).  kMany: several tokens
// a sequence.  Their keys, queries, values and gates are staged in shared memory kStage tokens at
// a time, on their way before the state's slot is even known, so that a token costs no round trip
// to L2; and a token's output is taken of the updated rows, which frees the key's registers for
// the queries (with fewer registers more blocks hide the states' latency).
constexpr int kStage = 8;

// Bytes of a staged token: its key, its queries, the block's values, (alpha, beta).
struct Staged {
    int q, v, gates, total;
    __host__ __device__ Staged(int queries, int rows)
        : q(2 * kD), v(2 * kD * (1 + queries)), gates(v + 2 * rows), total(gates + 16)
    {
    }
};

template <typename T, int kWarps, bool kMany>
__global__ void __launch_bounds__(kWarps * 32, 16 / kWarps)
    gdn_step_kernel(const StepParams p)
{
    constexpr int kBlockRows = kWarpRows * kWarps;
    constexpr int kParts = kD / kBlockRows;              // blocks of a state
    extern __shared__ __align__(16) uint8_t smem[];
    const int item = blockIdx.x / kParts, part = blockIdx.x % kParts;
    const int i = item / p.h_v, j = item % p.h_v;
    const int lane = threadIdx.x & 31, l = lane & 7;
    const int block_row = part * kBlockRows;
    const int row0 = block_row + (threadIdx.x >> 5) * kWarpRows + (lane >> 3) * kRows;

    const uint16_t* kp = p.k + i * p.k_stride[0] + (j / p.kgroup) * p.k_stride[2];
    const uint16_t* vp = p.v + i * p.v_stride[0] + j * p.v_stride[2] + block_row;
    const uint16_t* qp = p.q + i * p.q_stride[0] +
                         static_cast<int64_t>(p.queries > 1 ? j * p.queries : j / p.qgroup) *
                             p.q_stride[2];
    const float* ap = p.alpha + i * p.alpha_stride[0] + j;
    const float* bp = p.beta + i * p.beta_stride[0] + j;
    const int64_t out0 = (static_cast<int64_t>(i) * p.tokens * p.h_o +
                          static_cast<int64_t>(j) * p.queries) * kD + row0;
    const Staged at(p.queries, kBlockRows);
    auto stage = [&](int t0) {
        const int here = min(kStage, p.tokens - t0), pieces = at.gates / 16;
        const uint32_t dst = smem_addr(smem);
        for (int x = threadIdx.x; x < here * pieces; x += kWarps * 32) {
            const int t = x / pieces, b = (x - t * pieces) * 16;
            const uint16_t* src;
            if (b < at.q)
                src = kp + (t0 + t) * p.k_stride[1] + b / 2;
            else if (b < at.v)
                src = qp + (t0 + t) * p.q_stride[1] + (b / (2 * kD) - 1) * p.q_stride[2] +
                      b % (2 * kD) / 2;
            else
                src = vp + (t0 + t) * p.v_stride[1] + (b - at.v) / 2;
            cp_async16(dst + t * at.total + b, src);
        }
        for (int x = threadIdx.x; x < 2 * here; x += kWarps * 32)
            cp_async4(dst + x / 2 * at.total + at.gates + (x & 1) * 4,
                      x & 1 ? bp + (t0 + x / 2) * p.beta_stride[1]
                            : ap + (t0 + x / 2) * p.alpha_stride[1]);
        cp_commit();
    };

    dep_launch();
    dep_wait();
    const int slot = p.slots ? p.slots[i] : i;
    if constexpr (kMany) stage(0);
    const bool active = slot >= 0 && slot < p.n_slots;
    if (!active) {
        if (slot != -1 && threadIdx.x == 0) atomicOr(p.status, DECODE_BAD_STATE_SLOT);
        if (l == 0)
            for (int t = 0; t < p.tokens; ++t)
                for (int g = 0; g < p.queries; ++g)
                    *reinterpret_cast<uint2*>(
                        p.o + out0 + (static_cast<int64_t>(t) * p.h_o + g) * kD) =
                        make_uint2(0u, 0u);
        if constexpr (kMany) cp_wait<0>();
        return;
    }

    ulonglong2* state =
        reinterpret_cast<ulonglong2*>(p.state + slot * p.state_stride +
                                      (static_cast<int64_t>(j) * kD + row0) * kD) + l;
    uint64_t s[kRows][8];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const ulonglong2 x = state[r * (kD / 4) + 8 * c];
            s[r][2 * c] = x.x, s[r][2 * c + 1] = x.y;
        }
    const int row = row0 - block_row + (l & 3);          // the row whose sums this lane gets

    // s <- alpha s + u k, with u that of the lane's row
    auto update = [&](const uint64_t (&k)[8], float alpha, float u) {
        const uint64_t decay = pair(alpha, alpha);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float ur = __shfl_sync(0xffffffffu, u, (lane & 24) + r);
            const uint64_t uu = pair(ur, ur);
#pragma unroll
            for (int c = 0; c < 8; ++c) s[r][c] = fma2(uu, k[c], mul2(decay, s[r][c]));
        }
    };
    auto product = [&](const uint64_t (&x)[8]) {
        float d[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) d[r] = dot16(s[r], x);
        return sum_rows(d, l);
    };
    if constexpr (kMany) {
        for (int t0 = 0; t0 < p.tokens; t0 += kStage) {
            if (t0 > 0) {
                __syncthreads();
                stage(t0);
            }
            cp_wait<0>();
            __syncthreads();
            const int here = min(kStage, p.tokens - t0);
            for (int t = 0; t < here; ++t) {
                const uint8_t* tok = smem + t * at.total;
                const float2 gates = *reinterpret_cast<const float2*>(tok + at.gates);
                uint64_t x[8];
                load_row<T>(x, reinterpret_cast<const uint16_t*>(tok), l);
                const float v =
                    to_float<T>(reinterpret_cast<const uint16_t*>(tok + at.v)[row]);
                update(x, gates.x, gates.y * (v - gates.x * product(x)));
                for (int g = 0; g < p.queries; ++g) {
                    load_row<T>(x, reinterpret_cast<const uint16_t*>(tok + at.q) + kD * g, l);
                    const float o = p.scale * product(x);
                    if (l < kRows)
                        p.o[out0 + l + (static_cast<int64_t>(t0 + t) * p.h_o + g) * kD] =
                            from_float<T>(o);
                }
            }
        }
    } else {
        uint64_t k[8];
        load_row<T>(k, kp, l);
        const float alpha = ap[0], beta = bp[0], v = to_float<T>(vp[row]);
        const float u = beta * (v - alpha * product(k));
        for (int g = 0; g < p.queries; ++g) {
            uint64_t q[8];
            load_row<T>(q, qp + g * p.q_stride[2], l);
            const float kq = sum8(dot16(k, q));
            const float o = p.scale * fmaf(alpha, product(q), u * kq);
            if (l < kRows) p.o[out0 + l + static_cast<int64_t>(g) * kD] = from_float<T>(o);
        }
        update(k, alpha, u);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            state[r * (kD / 4) + 8 * c] = make_ulonglong2(s[r][2 * c], s[r][2 * c + 1]);
}

// Two warps a block for single tokens, so that few states spread over many SMs; four for several
// tokens, whose staging they share (77 sequences of 4 tokens: 19.4 us, 21.3 with two).
template <typename T, int kWarps, bool kMany>
cudaError_t run(const StepParams& p, int64_t items, int sms, size_t smem, cudaStream_t stream)
{
    constexpr auto kKernel = gdn_step_kernel<T, kWarps, kMany>;
    const int64_t blocks = items * (kD / (kWarpRows * kWarps));
    const cudaError_t e = allow_spread<kKernel>();
    if (e != cudaSuccess) return e;
    return launch(kKernel, dim3(static_cast<uint32_t>(blocks)), dim3(kWarps * 32),
                  spread(smem, blocks, sms, 16 / kWarps), stream, p);
}

template <typename T>
cudaError_t run(const StepParams& p, int64_t items, int sms, cudaStream_t stream)
{
    constexpr int kOne = 2, kSome = 4;
    if (p.tokens == 1) return run<T, kOne, false>(p, items, sms, 0, stream);
    const size_t smem = static_cast<size_t>(p.tokens < kStage ? p.tokens : kStage) *
                        Staged(p.queries, kWarpRows * kSome).total;
    return run<T, kSome, true>(p, items, sms, smem, stream);
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
    StepParams p{};
    if (!take_strides(p.q_stride, a->q_stride, {a->n, a->tokens, a->h_q}, 8) ||
        !take_strides(p.k_stride, a->k_stride, {a->n, a->tokens, a->h_k}, 8) ||
        !take_strides(p.v_stride, a->v_stride, {a->n, a->tokens, a->h_v}, 8))
        return fail(DECODE_ERR_UNSUPPORTED, "strides of q, k and v must be multiples of 8");
    take_strides(p.alpha_stride, a->alpha_stride, {a->n, a->tokens}, 1);
    take_strides(p.beta_stride, a->beta_stride, {a->n, a->tokens}, 1);
    if (a->n_slots > 1 && (a->state_stride % 4 || a->state_stride < a->h_v * kD * kD))
        return fail(DECODE_ERR_INVALID_ARG, "state_stride %lld", (long long)a->state_stride);
    if (a->n >= (int64_t(1) << 31) / (a->h_v * 8) || a->tokens >= (1 << 24) ||
        a->n_slots >= (int64_t(1) << 31))
        return fail(DECODE_ERR_UNSUPPORTED, "too many states or tokens for one call");

    // the blocks of a state read all of its q and k while others write their rows of o (of v each
    // reads just the rows that it writes)
    const int64_t h_o = queries > 1 ? a->h_q : a->h_v;
    const int64_t dense[3] = {a->tokens * h_o * kD, h_o * kD, kD};
    const int64_t gates[3] = {a->n, a->tokens, a->h_v};
    const int64_t alpha[3] = {p.alpha_stride[0], p.alpha_stride[1], 1};
    const int64_t beta[3] = {p.beta_stride[0], p.beta_stride[1], 1};
    const int shared = refuse_shared(
        {{"o", a->o, 2, kD, {a->n, a->tokens, h_o}, dense, "v"},
         {"state", a->state, 4, a->h_v * kD * kD, {a->n_slots}, {a->state_stride}}},
        {{"q", a->q, 2, kD, {a->n, a->tokens, a->h_q}, p.q_stride},
         {"k", a->k, 2, kD, {a->n, a->tokens, a->h_k}, p.k_stride},
         {"v", a->v, 2, kD, {a->n, a->tokens, a->h_v}, p.v_stride},
         {"alpha", a->alpha, 4, 1, gates, alpha},
         {"beta", a->beta, 4, 1, gates, beta},
         {"slots", a->slots, 4, a->n}});
    if (shared != DECODE_OK) return shared;

    p.status = status_word();
    const int sms = sm_count();
    if (p.status == nullptr || sms == 0) return DECODE_ERR_CUDA;
    p.q = static_cast<const uint16_t*>(a->q);
    p.k = static_cast<const uint16_t*>(a->k);
    p.v = static_cast<const uint16_t*>(a->v);
    p.alpha = a->alpha;
    p.beta = a->beta;
    p.state = a->state;
    p.slots = a->slots;
    p.o = static_cast<uint16_t*>(a->o);
    p.state_stride = a->n_slots > 1 ? a->state_stride : 0;
    p.tokens = static_cast<int32_t>(a->tokens);
    p.h_v = static_cast<int32_t>(a->h_v);
    p.h_o = static_cast<int32_t>(h_o);
    p.kgroup = static_cast<int32_t>(a->h_v / a->h_k);
    p.qgroup = a->h_q == a->h_k ? p.kgroup : 1;
    p.queries = static_cast<int32_t>(queries);
    p.n_slots = static_cast<int32_t>(a->n_slots);
    p.scale = a->scale;
    const int64_t items = a->n * a->h_v;
    const cudaError_t e = a->dtype == DECODE_BF16 ? run<__nv_bfloat16>(p, items, sms, stream)
                                                  : run<__half>(p, items, sms, stream);
    if (e != cudaSuccess)
        return fail(DECODE_ERR_CUDA, "gdn_step_kernel: %s", cudaGetErrorString(e));
    return DECODE_OK;
}
