// Norm of each query and key head, position rotation and write to the paged cache in one pass
// (C ABI in include/decode.h).
//
//     y = x * rsqrt(sum x^2 [/ d] + eps) * w;   (a, b) <- (a cos - b sin, b cos + a sin)
//
// Every element is read once and written once, with a handful of flops in between: the kernel is
// a copy bound by HBM, or by its launch when there are few tokens.
//
// Layout.  A lane holds 8 neighbouring elements (one 16-byte access), kLanes = 8, 16 or 32 lanes
// a head (head_dim up to 64, 128, 256), so a head's sum is a few shuffles.  In the split pairing
// element e's partner lies rot / 2 elements, that is rot / 16 lanes, away; in the interleaved
// pairing it is the lane's own neighbour.
//
// Norm and rotation are one linear map of a row up to its norm: with f the row's factor,
//     y_e = f (x_e (w_e cos) + x_partner (+-w_partner sin)),
// and the two factors in brackets are the same for all of a token's query (or key) heads.  So each
// group of kLanes lanes has a token of its own and takes its heads one after the other: it forms
// the factors once for the queries and once for the keys, and spends three packed fp32 operations
// per pair of elements on each head.  (With the factors formed anew for every eight heads the
// kernel issued twice the instructions, which bounded it; with a warp's groups on one token the
// keys' few heads left lanes idle.)
//
// A token is a chain of dependent loads (position, then its row of the table), so the warps stay
// for the whole call and load ahead: rows and angles go to shared memory by cp.async, a chunk of
// four heads ahead of the work, and the tokens' indices are read one set of tokens earlier.  Twenty
// warps an SM with two stages each keep as much in flight as sixteen with four and hide more of
// the instructions' latency, which bounds tokens of few heads: 38933 tokens of 6 + 2 heads take
// 44.8 us (46.9), 2844 of 16 + 2 heads of 256 13.4 us (18.8).
#include <cstdint>

#include "decode_common.cuh"

namespace {

using namespace decode;

constexpr int kSteps = 4;             // heads of a chunk
constexpr int kStages = 2;
constexpr int kBlockWarps = 2;
constexpr int kResident = 10;         // blocks of an SM
constexpr int kRowBytes = kSteps * 512;
constexpr int kAngleBytes = 1024 + 32;   // the angles of a warp's tokens, and (valid, slot) of each
constexpr int kWarpBytes = kStages * (kRowBytes + kAngleBytes);
enum Pairing { kSplit, kInterleaved };

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
    uint32_t tokens, sets, parts;           // sets of a warp's tokens; warps that share a set out
    int32_t q_chunks, k_chunks, all_chunks; // of q, of k, of a token (q, k and v)
    int32_t h_q, h_k, head_dim, rot, axes, page_size, norm;
    int32_t section_end[DECODE_MAX_AXES];   // first pair of the next axis
    float eps;
};

// The four 32-bit words of a lane's 8 elements, and their values as pairs.
template <typename T>
__device__ __forceinline__ uint64_t value2(uint32_t b)
{
    const float2 f = Half2<T>::unpack(b);
    return pair(f.x, f.y);
}
__device__ __forceinline__ uint32_t word(const uint4& b, int c)
{
    return c == 0 ? b.x : c == 1 ? b.y : c == 2 ? b.z : b.w;
}

// A token's chunks in order: its queries' (kind 0), its keys' (1), its values' (2).
template <typename T, int kLanes, Pairing kPairing>
__global__ void __launch_bounds__(kBlockWarps * 32, kResident) qk_norm_rope_kernel(const NormParams p)
{
    constexpr int kTokens = 32 / kLanes;             // tokens of a warp at a time: a set
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, l = lane % kLanes, mine_at = lane / kLanes;
    uint8_t* const ring = smem + (threadIdx.x >> 5) * kWarpBytes;      // [kStages][kRowBytes]
    uint8_t* const sets = ring + kStages * kRowBytes;                  // [kStages][kAngleBytes]
    const int e = 8 * l;                             // the lane's first element
    const bool in_head = e < p.head_dim, in_rot = e < p.rot;
    const int half = p.rot / 2;
    const int partner = kPairing != kSplit || !in_rot ? lane
                        : lane + (e < half ? half / 8 : -(half / 8));
    const float inv_d = p.norm == DECODE_NORM_RMS ? 1.f / p.head_dim : 1.f;

    // The warp's units: (set, part) number `first`, first + step, ...
    const uint32_t first = blockIdx.x * kBlockWarps + (threadIdx.x >> 5);
    const uint32_t step = gridDim.x * kBlockWarps, all = p.sets * p.parts;

    dep_launch();
    dep_wait();
    if (first >= all) return;

    // ---- loads: `at` is the unit and `chunk` its chunk whose loads come next, `token` the lane's
    uint32_t at = first, token = at / p.parts;
    int chunk = static_cast<int>(at - token * p.parts), set_ring = 0;
    token = token * kTokens + mine_at;
    int32_t pos[DECODE_MAX_AXES], slot = -1;         // of the token
    auto look = [&]() {
        slot = -1;
#pragma unroll
        for (int x = 0; x < DECODE_MAX_AXES; ++x)
            pos[x] = x < p.axes && token < p.tokens ? p.positions[x * p.position_stride + token] : 0;
        if (p.k_cache != nullptr && token < p.tokens) slot = p.slots[token];
    };
    look();
    bool begins = true;                              // the chunk is its unit's first
    auto load = [&](int stage) {
        if (at < all) {
            const int kind = chunk < p.q_chunks ? 0 : chunk < p.q_chunks + p.k_chunks ? 1 : 2;
            const int h = (kind == 0   ? chunk
                           : kind == 1 ? chunk - p.q_chunks
                                       : chunk - p.q_chunks - p.k_chunks) * kSteps;
            const int heads = kind == 0 ? p.h_q : p.h_k;
            const int64_t* by = kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride;
            const uint16_t* from =
                (kind == 0 ? p.q : kind == 1 ? p.k : p.v) + token * by[0] + h * by[1] + e;
            const uint32_t rows = smem_addr(ring) + stage * kRowBytes + lane * 16;
            const bool here = in_head && token < p.tokens;
#pragma unroll
            for (int x = 0; x < kSteps; ++x) {
                if (here && h + x < heads) cp_async16(rows + x * 512, from);
                from += by[1];
            }
            if (begins) {
                uint8_t* const to = sets + set_ring * kAngleBytes;
                bool ok = true;
#pragma unroll
                for (int x = 0; x < DECODE_MAX_AXES; ++x)
                    ok = ok && pos[x] >= 0 && (x >= p.axes || pos[x] < p.table_rows);
                if (!ok && l == 0) atomicOr(p.status, DECODE_BAD_POSITION);
                // the table's floats e .. e + 7: cosines or sines of the pairs pair0 ..
                // pair0 + 7
                if (ok && in_rot && here) {
                    const int pair0 = e < half ? e : e - half;
                    auto axis_of = [&](int pair) {
                        int axis = 0;
#pragma unroll
                        for (int x = 1; x < DECODE_MAX_AXES; ++x)
                            axis += x < p.axes && pair >= p.section_end[x - 1];
                        return axis;
                    };
                    auto table_row = [&](int axis) {
                        int32_t row = pos[0];
#pragma unroll
                        for (int x = 1; x < DECODE_MAX_AXES; ++x) row = axis == x ? pos[x] : row;
                        return p.table + static_cast<int64_t>(row) * p.rot;
                    };
                    const uint32_t angles = smem_addr(to) + lane * 32;
                    const int axis = axis_of(pair0);
                    if (axis == axis_of(pair0 + 7)) {
                        const float* row = table_row(axis) + e;
                        cp_async16(angles, row);
                        cp_async16(angles + 16, row + 4);
                    } else {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            cp_async4(angles + c * 4, table_row(axis_of(pair0 + c)) + e + c);
                    }
                }
                if (slot < -1 || slot >= p.cache_slots) {
                    if (l == 0) atomicOr(p.status, DECODE_BAD_CACHE_SLOT);
                    slot = -1;
                }
                if (l == 0)
                    *reinterpret_cast<int2*>(to + 1024 + mine_at * 8) =
                        make_int2(ok, ok ? slot : -1);
                set_ring = set_ring + 1 == kStages ? 0 : set_ring + 1;
            }
            chunk += p.parts;
            begins = chunk >= p.all_chunks;
            if (begins) {
                at += step;
                const uint32_t set = at / p.parts;
                chunk = static_cast<int>(at - set * p.parts);
                token = set * kTokens + mine_at;
                if (at < all) look();
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) load(s);

    // ---- the work
    uint4 wq = make_uint4(0u, 0u, 0u, 0u), wk = wq;
    if (in_head && p.q_weight) wq = *reinterpret_cast<const uint4*>(p.q_weight + e);
    if (in_head && p.k_weight) wk = *reinterpret_cast<const uint4*>(p.k_weight + e);
    int stage = 0, work_ring = 0;
    for (uint32_t unit = first; unit < all; unit += step) {
        const uint32_t set = unit / p.parts, t = set * kTokens + mine_at;
        const uint8_t* const head = sets + work_ring * kAngleBytes;
        const float* const angles = reinterpret_cast<const float*>(head) + mine_at * kLanes * 8;
        bool ok = true;
        int32_t place = -1, page = 0, off = 0;
        int have = -1;                               // the kind the factors are for
        uint64_t mine[4], other[4];
        for (int c0 = static_cast<int>(unit - set * p.parts); c0 < p.all_chunks; c0 += p.parts) {
            __syncwarp();
            load(stage == 0 ? kStages - 1 : stage - 1);
            cp_wait<kStages - 1>();
            __syncwarp();
            if (have < 0) {
                const int2 x = *reinterpret_cast<const int2*>(head + 1024 + mine_at * 8);
                ok = x.x;
                place = x.y;
                if (place >= 0) {
                    page = static_cast<uint32_t>(place) / static_cast<uint32_t>(p.page_size);
                    off = place - page * p.page_size;
                }
            }
            const int kind = c0 < p.q_chunks ? 0 : c0 < p.q_chunks + p.k_chunks ? 1 : 2;
            const int h = (kind == 0   ? c0
                           : kind == 1 ? c0 - p.q_chunks
                                       : c0 - p.q_chunks - p.k_chunks) * kSteps;
            if (kind != have && kind < 2) {
                const uint4 wb = kind == 0 ? wq : wk;
                const bool weights = (kind == 0 ? p.q_weight : p.k_weight) != nullptr;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mine[c] = weights ? value2<T>(word(wb, c)) : pair(1.f, 1.f);
                    if constexpr (kPairing == kSplit) {
                        const uint32_t x = __shfl_sync(0xffffffffu, word(wb, c), partner);
                        other[c] = weights ? value2<T>(x) : pair(1.f, 1.f);
                    } else if constexpr (kPairing == kInterleaved) {
                        const float2 f = halves(mine[c]);
                        other[c] = pair(f.y, f.x);
                    }
                }
                if constexpr (kPairing == kSplit) {
                    if (in_rot) {
                        const float* cs = angles + (e < half ? e : e - half);
                        const float sign = e < half ? -1.f : 1.f;
#pragma unroll
                        for (int c = 0; c < 4; c += 2) {
                            const float4 x = *reinterpret_cast<const float4*>(cs + 2 * c);
                            const float4 y = *reinterpret_cast<const float4*>(cs + half + 2 * c);
                            mine[c] = mul2(mine[c], pair(x.x, x.y));
                            mine[c + 1] = mul2(mine[c + 1], pair(x.z, x.w));
                            other[c] = mul2(other[c], pair(sign * y.x, sign * y.y));
                            other[c + 1] = mul2(other[c + 1], pair(sign * y.z, sign * y.w));
                        }
                    }
                } else if constexpr (kPairing == kInterleaved) {
                    if (in_rot) {
                        const float4 x = *reinterpret_cast<const float4*>(angles + e / 2);
                        const float4 y = *reinterpret_cast<const float4*>(angles + half + e / 2);
                        mine[0] = mul2(mine[0], pair(x.x, x.x));
                        mine[1] = mul2(mine[1], pair(x.y, x.y));
                        mine[2] = mul2(mine[2], pair(x.z, x.z));
                        mine[3] = mul2(mine[3], pair(x.w, x.w));
                        other[0] = mul2(other[0], pair(-y.x, y.x));
                        other[1] = mul2(other[1], pair(-y.y, y.y));
                        other[2] = mul2(other[2], pair(-y.z, y.z));
                        other[3] = mul2(other[3], pair(-y.w, y.w));
                    }
                }
            }
            have = kind;

            // where the rows go: to q_out or k_out, or to the token's place in a cache
            const int heads = kind == 0 ? p.h_q : p.h_k;
            uint16_t* dst;
            int64_t dst_step;
            bool write = in_head && t < p.tokens;
            if (kind == 0) {
                dst = p.q_out + t * p.q_out_stride[0] + h * p.q_out_stride[1] + e;
                dst_step = p.q_out_stride[1];
            } else if (p.k_cache == nullptr) {
                dst = p.k_out + t * p.k_out_stride[0] + h * p.k_out_stride[1] + e;
                dst_step = p.k_out_stride[1];
            } else {
                const int64_t* to = kind == 1 ? p.k_cache_stride : p.v_cache_stride;
                dst = (kind == 1 ? p.k_cache : p.v_cache) + page * to[0] + off * to[1] + h * to[2] + e;
                dst_step = to[2];
                write = write && place >= 0;
            }
            const uint4* const rows = reinterpret_cast<const uint4*>(ring + stage * kRowBytes);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                if (h + s >= heads) break;
                uint4 b = rows[s * 32 + lane];
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
                        float sum = in_head ? s1.x + s1.y : 0.f;
#pragma unroll
                        for (int m = 1; m < kLanes; m *= 2)
                            sum += __shfl_xor_sync(0xffffffffu, sum, m);
                        f = rsqrtf(fmaf(sum, inv_d, p.eps));
                    }
                    const uint64_t ff = pair(f, f);
                    [[maybe_unused]] uint4 z;
                    if constexpr (kPairing == kSplit) z = rows[s * 32 + partner];
                    uint32_t out[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint64_t y = mul2(x[c], mine[c]);
                        if constexpr (kPairing == kSplit) {
                            if (in_rot) y = fma2(value2<T>(word(z, c)), other[c], y);
                        } else if constexpr (kPairing == kInterleaved) {
                            const float2 v = halves(x[c]);
                            if (in_rot) y = fma2(pair(v.y, v.x), other[c], y);
                        }
                        const float2 r = halves(mul2(y, ff));
                        out[c] = Half2<T>::pack(r.x, r.y);
                    }
                    b = ok ? make_uint4(out[0], out[1], out[2], out[3]) : make_uint4(0u, 0u, 0u, 0u);
                }
                if (write) *reinterpret_cast<uint4*>(dst) = b;
                dst += dst_step;
            }
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
        work_ring = work_ring + 1 == kStages ? 0 : work_ring + 1;
    }
}

// Without a rotation nothing depends on an index but where keys and values go, so each lane group
// just loads a chunk of a token's heads into registers, norms and stores it, with as many warps as
// the registers allow: 8192 tokens of 8 + 8 heads take 12.0 us, against 14.5 us on the other kernel.
constexpr int kPlainWarps = 4;

template <typename T, int kLanes>
__global__ void __launch_bounds__(kPlainWarps * 32) qk_norm_kernel(const NormParams p)
{
    const int l = threadIdx.x % kLanes, e = 8 * l;
    const bool in_head = e < p.head_dim;
    const uint32_t unit = blockIdx.x * (kPlainWarps * 32 / kLanes) + threadIdx.x / kLanes;
    const uint32_t t = unit / p.all_chunks;
    const int c0 = static_cast<int>(unit - t * p.all_chunks);
    const int kind = c0 < p.q_chunks ? 0 : c0 < p.q_chunks + p.k_chunks ? 1 : 2;
    const int h = (kind == 0   ? c0
                   : kind == 1 ? c0 - p.q_chunks
                               : c0 - p.q_chunks - p.k_chunks) * kSteps;
    const int heads = t >= p.tokens || !in_head ? 0 : kind == 0 ? p.h_q : p.h_k;

    dep_launch();
    dep_wait();
    const int64_t* by = kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride;
    const uint16_t* from = (kind == 0 ? p.q : kind == 1 ? p.k : p.v) + t * by[0] + h * by[1] + e;
    uint4 in[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        in[s] = make_uint4(0u, 0u, 0u, 0u);
        if (h + s < heads) in[s] = *reinterpret_cast<const uint4*>(from + s * by[1]);
    }
    const uint16_t* w = kind == 0 ? p.q_weight : p.k_weight;
    uint4 wb = make_uint4(0u, 0u, 0u, 0u);
    if (w != nullptr && heads > 0) wb = *reinterpret_cast<const uint4*>(w + e);

    uint16_t* dst = nullptr;
    int64_t dst_step = 0;
    if (kind == 0) {
        dst = p.q_out + t * p.q_out_stride[0] + h * p.q_out_stride[1] + e;
        dst_step = p.q_out_stride[1];
    } else if (p.k_cache == nullptr) {
        dst = p.k_out + t * p.k_out_stride[0] + h * p.k_out_stride[1] + e;
        dst_step = p.k_out_stride[1];
    } else if (heads > 0) {
        const int32_t slot = p.slots[t];
        if (slot >= 0 && slot < p.cache_slots) {
            const int64_t page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page_size);
            const int64_t off = slot - page * p.page_size;
            const int64_t* to = kind == 1 ? p.k_cache_stride : p.v_cache_stride;
            dst = (kind == 1 ? p.k_cache : p.v_cache) + page * to[0] + off * to[1] + h * to[2] + e;
            dst_step = to[2];
        } else if (slot != -1 && l == 0) {
            atomicOr(p.status, DECODE_BAD_CACHE_SLOT);
        }
    }
    const float inv_d = p.norm == DECODE_NORM_RMS ? 1.f / p.head_dim : 1.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        uint64_t x[4];
        uint64_t s2 = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            x[c] = value2<T>(word(in[s], c));
            s2 = c == 0 ? mul2(x[c], x[c]) : fma2(x[c], x[c], s2);
        }
        float f = 1.f;
        if (p.norm != DECODE_NORM_NONE) {
            const float2 s1 = halves(s2);
            float sum = s1.x + s1.y;
#pragma unroll
            for (int m = 1; m < kLanes; m *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            f = rsqrtf(fmaf(sum, inv_d, p.eps));
        }
        uint4 b = in[s];
        if (kind < 2) {
            uint32_t out[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint64_t y = mul2(x[c], pair(f, f));
                if (w != nullptr) y = mul2(y, value2<T>(word(wb, c)));
                const float2 r = halves(y);
                out[c] = Half2<T>::pack(r.x, r.y);
            }
            b = make_uint4(out[0], out[1], out[2], out[3]);
        }
        if (h + s < heads && dst != nullptr) *reinterpret_cast<uint4*>(dst + s * dst_step) = b;
    }
}

template <typename T, int kLanes, Pairing kPairing>
cudaError_t run(NormParams p, int sms, cudaStream_t stream)
{
    constexpr int kTokens = 32 / kLanes;
    p.sets = (p.tokens + kTokens - 1) / kTokens;
    // A warp takes whole sets, or, where there are few, parts of them: the number of parts for which
    // the warp with the most work has the least, a unit costing as much as two chunks beside its own.
    // Neighbouring warps share a set of many chunks in any case, three from nine chunks on and two
    // for eight, since fewer tokens at a time suit the memory: 32768 tokens, keys and values to a
    // cache, with one, two and three warps a set take 151, 128 and 127 us (32 + 8 heads, 12 chunks),
    // 110, 105 and 100 us (28 + 4, nine), 101, 89 and 91 us (16 + 8, eight), 69, 75 and 76 us (16 +
    // 4, six, where the units' own cost shows).
    const int64_t most = static_cast<int64_t>(sms) * kResident, warps = most * kBlockWarps;
    int64_t least = INT64_MAX;
    for (int32_t parts = p.all_chunks >= 9 ? 3 : p.all_chunks >= 8 ? 2 : 1; parts <= p.all_chunks; ++parts) {
        const int64_t rounds = (static_cast<int64_t>(p.sets) * parts + warps - 1) / warps;
        const int64_t cost = rounds * ((p.all_chunks + parts - 1) / parts + 2);
        if (cost < least) {
            least = cost;
            p.parts = static_cast<uint32_t>(parts);
        }
        if (rounds > 8) break;       // rounding up no longer matters
    }
    const int64_t blocks = (static_cast<int64_t>(p.sets) * p.parts + kBlockWarps - 1) / kBlockWarps;
    constexpr auto kKernel = qk_norm_rope_kernel<T, kLanes, kPairing>;
    const cudaError_t e = allow_spread<kKernel>();
    if (e != cudaSuccess) return e;
    return launch(kKernel, dim3(static_cast<uint32_t>(blocks < most ? blocks : most)),
                  dim3(kBlockWarps * 32), spread(kBlockWarps * kWarpBytes, blocks, sms, kResident),
                  stream, p);
}

template <typename T, int kLanes>
cudaError_t run(NormParams p, bool interleaved, int sms, cudaStream_t stream)
{
    p.q_chunks = (p.h_q + kSteps - 1) / kSteps;
    p.k_chunks = (p.h_k + kSteps - 1) / kSteps;
    p.all_chunks = p.q_chunks + p.k_chunks * (p.v != nullptr ? 2 : 1);
    if (p.rot == 0) {
        constexpr int kUnitsPerBlock = kPlainWarps * 32 / kLanes;
        const int64_t units = static_cast<int64_t>(p.tokens) * p.all_chunks;
        return launch(qk_norm_kernel<T, kLanes>,
                      dim3(static_cast<uint32_t>((units + kUnitsPerBlock - 1) / kUnitsPerBlock)),
                      dim3(kPlainWarps * 32), 0, stream, p);
    }
    return interleaved ? run<T, kLanes, kInterleaved>(p, sms, stream)
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

    // (a head of q or k is read by the lanes that write it, before they do)
    const int64_t d = a->head_dim, q_sizes[2] = {a->tokens, a->h_q}, k_sizes[2] = {a->tokens, a->h_k};
    const int shared = refuse_shared(
        {{"q_out", a->q_out, 2, d, q_sizes, p.q_out_stride, "q"},
         {"k_out", cache ? nullptr : a->k_out, 2, d, k_sizes, p.k_out_stride, "k"},
         {"k_cache", a->k_cache, 2, d, cs, p.k_cache_stride},
         {"v_cache", a->v_cache, 2, d, cs, p.v_cache_stride}},
        {{"q", a->q, 2, d, q_sizes, p.q_stride},
         {"k", a->k, 2, d, k_sizes, p.k_stride},
         {"v", a->v, 2, d, k_sizes, p.v_stride},
         {"q_weight", a->q_weight, 2, d},
         {"k_weight", a->k_weight, 2, d},
         {"positions", a->rot > 0 ? a->positions : nullptr, 4, a->tokens, {a->axes},
          {a->position_stride}},
         {"table", a->table, 4, a->table_rows * a->rot},
         {"slots", a->slots, 4, a->tokens}});
    if (shared != DECODE_OK) return shared;

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
