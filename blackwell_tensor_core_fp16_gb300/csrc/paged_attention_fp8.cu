// Attention of one new token per sequence over a paged cache of E4M3 codes with an E8M0 scale for each
// block of tokens and head, with a sliding window and first tokens that stay visible (C ABI in
// include/decode.h):
//
//     s_t = scale q . K_t;   o = sum_t exp(s_t - m) V_t / sum_t exp(s_t - m)
//
// The split of the work over the blocks, the ring of stages and the joins are those of the 16-bit
// cache (paged_attention.cu).  A key and a value take 2 d bytes here, half of that, for the same
// products, and their codes have to become 16-bit numbers on the way: the cache is still read once and
// HBM bounds the time, but with less room for instructions.  What differs:
//
// Codes become float16, which holds every one exactly, after they have come to the registers.
// ldmatrix moves pairs of bytes: of keys a lane gets four neighbouring elements of a token's row, which
// are taken as two steps' operands (the queries' elements are dealt to steps in the same order), of
// values, transposed, two tokens' two neighbouring elements, whose bytes a permutation sorts by
// element; rows r and r + 8 of a tile stand for elements 2 r and 2 r + 1.
//
// Scales are read for each token of a slice (a byte each of keys and values) with its rows and wait
// beside its stage, so blocks may have any size.  A key's scale multiplies its scores.  A
// value's goes into its weight: times 2^15 over the slice's largest scale, so that a weight fits float16
// whatever the scales.  Weights are taken against the slice's own largest score, and where its scales are
// further apart than 2^8, against its largest product of weight and scale; what that leaves out multiplies the
// slice's sums when they are added to the running ones.  So the two float16 pieces of a weight leave out less
// than 2^-22 of it, or 2^-32 of the slice's largest product of weight and scale, however large the scale of a
// token that has no weight and however small all of a slice's weights.  (Against the running maximum and the
// largest scale alone, as they were, tokens whose scale is below 2^-40 of their slice's largest were lost.)
//
// bfloat16 queries become float16 too, each head's divided by a power of two that brings its largest
// element between 2^14 and 2^15: no bit is lost of elements above 2^-31 of the largest, and of smaller
// ones less than 2^-38 of it.
//
// Measured: 64 sequences of up to 8192 tokens, 32 heads over 8 of 128, 91 to 97 us by their lengths (5.7 TB/s,
// floor 79); 200001 tokens, 16 heads over 2 of 256, 47 (floor 30); 37 windows of 1000 and 4 first tokens, 12
// heads of 64, 19 (floor 7.4).  Twelve warps an SM, each a chain of
// dependent conversions, products and a softmax, keep half of the issue slots busy while the codes come, and no
// pipe above 44%: what bounds the time is how little of the chains' latency and the memory's overlap.  With 16
// query heads a key head there are eight warps an SM, for 256 four: 64 sequences of 4096 tokens, launch included,
// 8 key heads of 64 83 us with 8 query heads each and 123 with 16, of 128 130 and 172, 4 of 256 119 and 247.
//
// With a window the seen tokens are two ranges.  They are laid one after the other on one axis of rows,
// the first tokens' range rounded up and the window's start down to 16, so that 16 rows lie in one
// range, and the axis is cut into tiles as any other.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "fp8.cuh"
#include "paged_common.cuh"

namespace {

using namespace decode;

constexpr int kMostResident = 3;     // of Fp8Cfg::kResident
constexpr int kFar = 8;              // powers of two between scales, to which weights keep to the slice's largest
// The scales of a token that is not seen: a key's that no write leaves (a finite one: its codes are zeros), and
// a value's below all others.
constexpr uint32_t kUnseen = 250;

struct Fp8Params : SplitParams {
    const uint16_t* q;
    const uint8_t* k;
    const uint8_t* v;
    const uint8_t* scale[2];           // keys', values'
    const int32_t* table;
    int64_t q_stride[2], table_stride;
    int64_t head_stride[2], scale_head_stride[2];
    uint32_t stride[2][2], scale_stride[2][2];     // page, offset; page, block
    int32_t pages, page_size, page_shift, block, block_shift, window, sinks;
    int32_t same;                      // the strides of keys' and values' codes and scales are the same
    float scale_log2;
};

// A sequence's seen tokens: t < first and start <= t < len; len = 0 for a length the page table cannot
// hold.  Row r of the axis is token r below `edge` and token r + gap from there on.
struct Fp8Span {
    int start, len, first, edge, gap;
    __device__ __forceinline__ int rows() const { return len - gap; }
    __device__ __forceinline__ int token(int row) const { return row < edge ? row : row + gap; }
    __device__ __forceinline__ bool seen(int t) const { return t < len && (t >= start || t < first); }
    __device__ __forceinline__ static Fp8Span of(const Fp8Params& p, int i)
    {
        Fp8Span s;
        s.len = p.lens[i];
        if (s.len < 0 || s.len > p.max_len) s.len = 0;
        s.start = p.window > 0 && s.len > p.window ? s.len - p.window : 0;
        s.first = min(p.sinks, s.start);
        s.edge = (s.first + kSub - 1) & ~(kSub - 1);
        const int origin = s.start & ~(kSub - 1);
        s.gap = max(origin - s.edge, 0);           // none where the ranges' 16 rows meet
        return s;
    }
};

// What a warp needs of it for each tile: how many rows, and the first from which on all are seen.
struct Fp8Rows {
    int len, gap, clear;
    __device__ __forceinline__ int rows() const { return len - gap; }
    __device__ __forceinline__ bool all_seen(int row, int count) const
    {
        return row >= clear && row + count <= rows();
    }
    __device__ __forceinline__ static Fp8Rows of(const Fp8Params& p, int i)
    {
        const Fp8Span s = Fp8Span::of(p, i);
        return {s.len, s.gap, s.start - s.gap};
    }
};

template <int D, int kTiles>
struct Fp8Cfg {
    static constexpr int kD = D, kHeadTiles = kTiles;
    static constexpr int kWarps = D == 256 && kTiles == 2 ? 2 : 4;   // (the join needs room by them)
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kHeads = 8 * kHeadTiles;
    static constexpr int kSubs = 256 / D;                     // a slice is 8 KB
    template <typename T>
    static constexpr int kShift = 0;                          // (the sums carry no factor)
    static constexpr bool kRowPairs = true;
    // An item's end takes about as long as a tile; counted as nothing, blocks with many ends are the last:
    // 64 sequences of up to 2000 tokens, 32 heads over 8 of 128, 42.0 us and 35.7 so, of up to 8192 100.8 and 97.1.
    // A block an item spares the join's launch: 56 sequences of 1000 tokens 29.3 us and 26.3 so, 220 of 500 with
    // 2 heads of 256 31.8 and 26.3; where lengths differ it may lose, 37 of up to 1000 with 12 heads 21.2 and 22.9.
    static constexpr int kEndTiles = 1, kAloneTiles = 8;
    static constexpr int kResident = kTiles == 1 ? 3 : 2;   // blocks of an SM
    static constexpr int kSlice = kSubs * kSub;               // tokens of a warp's slice
    static constexpr int kTile = kWarps * kSlice;
    static constexpr int kPer = kSlice > 32 ? kSlice / 32 : 1;     // tokens of a slice by lane
    static constexpr int kScaleBytes = kPer * 64;             // 2 bytes a token: key's, value's
    static constexpr int kCodeBytes = 2 * kSlice * D;         // keys, then values
    static constexpr int kStageBytes = kCodeBytes + kScaleBytes;
    // Warps are joined through the stages whose slices they have just done, where there is room: each
    // head's elements, 16 at a time in an order of the head's own that spreads the banks (else a pad).
    static constexpr bool kMergeInRing = kHeads * D * 4 <= kCodeBytes;
    static constexpr int kSmallBytes = 2 * kWarps * kHeads * 4 + 256;
    // the queries stay in registers, but for the one shape whose sums leave no room for them
    static constexpr bool kQueriesShared = D == 256;
    static constexpr int kQueryRow = D + 16;                  // elements
    static constexpr int kQueryBytes = kQueriesShared ? kHeads * kQueryRow * 2 + kHeads * 4 : 0;
    static constexpr int kMergeBytes = kMergeInRing ? 0 : kWarps * kHeads * (D + 4) * 4;
    // (the blocks share an SM's 228 KB, of which the system takes 1 KB a block)
    static constexpr int kRoom =
        233472 / kResident - 1024 - kMergeBytes - kSmallBytes - kQueryBytes;
    static constexpr int kMostStages = kRoom / (kWarps * kStageBytes);
    static constexpr int kStages = kMostStages < 4 ? kMostStages : 4;
    static constexpr int kSmem = kWarps * kStages * kStageBytes + kMergeBytes + kSmallBytes +
                                 kQueryBytes;
    static_assert(kStages >= 2, "no room for two stages");
    static constexpr int kMergeWarp = kMergeInRing ? kStages * kCodeBytes / 4 : kHeads * (D + 4);   // floats
    __device__ static __forceinline__ int merge_at(int h, int d)
    {
        return kMergeInRing ? h * D + (d ^ (h >> 1 & 3) << 4) : h * (D + 4) + d;
    }
    // where a 16-byte piece of a row lies, so that 8 rows' pieces lie in 8 different bank groups
    __device__ static __forceinline__ int place(int row, int piece)
    {
        return row * D + ((piece ^ (D == 64 ? (row >> 1) & 3 : row & 7)) << 4);
    }
};

// kCluster: one cluster an item, for few items of few tiles.
template <typename T, int D, int kHeadTiles, bool kCluster>
__global__ void __launch_bounds__(Fp8Cfg<D, kHeadTiles>::kThreads, Fp8Cfg<D, kHeadTiles>::kResident)
    paged_attention_fp8_kernel(const Fp8Params p)
{
    using C = Fp8Cfg<D, kHeadTiles>;
    using H = __half;                              // what codes, queries and weights become
    constexpr int kHeads = C::kHeads, kWarps = C::kWarps, kTile = C::kTile;
    constexpr int kSlice = C::kSlice, kSubs = C::kSubs;
    constexpr int kChunks = D / 16;                // 16-byte pieces of a row
    constexpr int kRowsPerCopy = 32 / kChunks;     // rows that one cp.async of the warp covers
    constexpr uint32_t kAll = 0xffffffffu;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* ring = smem;
    float* merge = reinterpret_cast<float*>(
        smem + (C::kMergeInRing ? 0 : kWarps * C::kStages * C::kStageBytes));
    float* sm_m = reinterpret_cast<float*>(smem + kWarps * C::kStages * C::kStageBytes +
                                           C::kMergeBytes);       // [kWarps][kHeads]
    float* sm_l = sm_m + kWarps * kHeads;
    int* sm_i = reinterpret_cast<int*>(sm_l + kWarps * kHeads);   // 64 words
    uint16_t* sm_q = reinterpret_cast<uint16_t*>(sm_i + 64);      // [kHeads][kQueryRow]
    float* sm_q_scale = reinterpret_cast<float*>(sm_q + kHeads * C::kQueryRow);   // [kHeads]
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;

    dep_launch();
    dep_wait();

    Cursor<Fp8Rows> cur;
    Range r;
    if constexpr (kCluster) {
        if (!cluster_range<C>(p, cur, r, sm_i)) return;
    } else {
        if (!block_range<C>(p, cur, r, sm_i)) return;
    }
    const int t0 = r.t0, t1 = r.t1;
    Cursor<Fp8Span> pre = {cur.i, cur.item, cur.tile, cur.tiles, Fp8Span::of(p, cur.i)};   // of the loads
    int pre_t = t0;

    // ---- loads of a slice.  Lane x takes care of token x of it (and x + 32, if it has as many): it looks
    // its page up one slice ahead and its scales, and names its rows to the lanes that copy them.
    constexpr int kPer = C::kPer;
    const uint32_t ring0 = smem_addr(ring + w * C::kStages * C::kCodeBytes);
    uint16_t* const scales0 = reinterpret_cast<uint16_t*>(ring + kWarps * C::kStages * C::kCodeBytes +
                                                          w * C::kStages * C::kScaleBytes) + lane;
    const int ch = lane % kChunks, sub = lane / kChunks;
    int page[kPer], off[kPer];
    bool there[kPer];                              // the token is one that is seen
    auto look_up = [&]() {
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
            there[y] = false;
            if (pre_t >= t1) continue;
            const int row = pre.tile * kTile + w * kSlice + y * 32 + (lane & (kSlice - 1));
            const int pos = pre.span.token(row);
            if (row >= pre.span.rows() || !pre.span.seen(pos)) continue;
            there[y] = true;
            const int x = divide(pos, p.page_size, p.page_shift);
            off[y] = pos - x * p.page_size;
            page[y] = p.table[pre.i * p.table_stride + x];
        }
    };
    // (the scales are on their way while the warp goes on, and are put beside their stage at the next
    // load)
    uint32_t scale_byte[2][kPer];
    int scale_stage = -1;
    auto load = [&](int stage) {
        if (scale_stage >= 0) {
#pragma unroll
            for (int y = 0; y < kPer; ++y)
                scales0[scale_stage * (C::kScaleBytes / 2) + y * 32] =
                    static_cast<uint16_t>(scale_byte[0][y] | scale_byte[1][y] << 8);
        }
        scale_stage = -1;
        if (pre_t < t1) {
            const int kv = pre.item / p.head_items;
            scale_stage = stage;
            bool all = true;
#pragma unroll
            for (int y = 0; y < kPer; ++y) {
                scale_byte[0][y] = kUnseen, scale_byte[1][y] = 0;
                if (there[y] && static_cast<uint32_t>(page[y]) >= static_cast<uint32_t>(p.pages)) {
                    atomicOr(p.status, DECODE_BAD_PAGE);
                    there[y] = false;
                }
                all = all && there[y];
                if (!there[y]) continue;
                uint64_t from = 0;
#pragma unroll
                for (int of = 0; of < 2; ++of) {
                    if (of == 0 || !p.same)
                        from = kv * p.scale_head_stride[of] +
                               static_cast<uint64_t>(static_cast<uint32_t>(page[y])) * p.scale_stride[of][0] +
                               static_cast<uint64_t>(static_cast<uint32_t>(
                                   divide(off[y], p.block, p.block_shift))) * p.scale_stride[of][1];
                    scale_byte[of][y] = p.scale[of][from];
                }
            }
            all = __all_sync(kAll, all);
            // where the codes of the lane's own tokens lie
            uint64_t at[kPer];
            auto locate = [&](int of) {
#pragma unroll
                for (int y = 0; y < kPer; ++y)
                    at[y] = !there[y] ? 0
                                      : kv * p.head_stride[of] +
                                            static_cast<uint64_t>(static_cast<uint32_t>(page[y])) *
                                                p.stride[of][0] +
                                            static_cast<uint64_t>(static_cast<uint32_t>(off[y])) *
                                                p.stride[of][1];
            };
            const uint32_t dst0 = ring0 + stage * C::kCodeBytes;
            if (all && p.same) {
                locate(0);
#pragma unroll
                for (int x = 0; x < kSlice / kRowsPerCopy; ++x) {
                    const int row = x * kRowsPerCopy + sub;
                    const uint64_t from =
                        __shfl_sync(kAll, at[x * kRowsPerCopy / 32], row & 31) + ch * 16;
                    const uint32_t dst = dst0 + C::place(row, ch);
                    cp_async16(dst, p.k + from);
                    cp_async16(dst + kSlice * D, p.v + from);
                }
            } else {
                for (int of = 0; of < 2; ++of) {
                    locate(of);
                    const uint8_t* const base = of ? p.v : p.k;
#pragma unroll
                    for (int x = 0; x < kSlice / kRowsPerCopy; ++x) {
                        const int row = x * kRowsPerCopy + sub, y = x * kRowsPerCopy / 32;
                        const uint64_t from = __shfl_sync(kAll, at[y], row & 31) + ch * 16;
                        const uint32_t bytes = __shfl_sync(kAll, there[y], row & 31) ? 16u : 0u;
                        cp_async16(dst0 + of * kSlice * D + C::place(row, ch),
                                   bytes ? base + from : base, bytes);
                    }
                }
            }
            ++pre_t;
            if constexpr (kCluster) {
                ++pre.tile;
            } else {
                if (pre.tile + 1 == pre.tiles) pre_t += C::kEndTiles;
                if (pre_t < t1) advance<kTile>(pre, p);
            }
        }
        cp_commit();
        look_up();
    };
    look_up();
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) load(s);

    // ---- the tiles
    constexpr int kOwn = C::kQueriesShared ? 1 : kHeadTiles;      // head tiles of queries in registers
    uint32_t qf[kOwn][D / 16][2];
    float q_scale[kOwn][2];                        // what the lane's two heads' queries were divided by
    float acc[kHeadTiles][D / 16][4];
    float m[kHeadTiles][2], l[kHeadTiles][2];
    bool fresh = true;
    // the queries of an item's head tile x: of 16 elements a lane holds four neighbouring ones of head
    // lane / 4
    auto load_queries = [&](const Cursor<Fp8Rows>& of, int x, uint32_t (&f)[D / 16][2]) {
        const int kv = of.item / p.head_items;
        const int first = of.item % p.head_items * kHeads, heads = min(kHeads, p.group - first);
        const int h = x * 8 + (lane >> 2);
        const uint16_t* row = p.q + of.i * p.q_stride[0] +
                              (kv * p.group + first + h) * p.q_stride[1] + (lane & 3) * 4;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            const uint2 b = h < heads ? *reinterpret_cast<const uint2*>(row + d * 16)
                                      : make_uint2(0u, 0u);
            f[d][0] = b.x;
            f[d][1] = b.y;
        }
    };
    // makes them float16; what head lane / 4 was divided by
    auto convert_queries = [&](uint32_t (&f)[D / 16][2]) {
        if constexpr (std::is_same<T, __half>::value) return 1.f;
        uint32_t top = 0;                          // the largest exponent of a finite element
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t lo = f[d][e] >> 7 & 0xffu, hi = f[d][e] >> 23 & 0xffu;
                top = max(top, max(lo < 255u ? lo : 0u, hi < 255u ? hi : 0u));
            }
        top = max(top, __shfl_xor_sync(kAll, top, 1));
        top = max(top, __shfl_xor_sync(kAll, top, 2));
        const int up = min(268 - static_cast<int>(top), 253);
        const float by = power_of(up);
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 v = Half2<T>::unpack(f[d][e]);
                f[d][e] = Half2<H>::pack(v.x * by, v.y * by);
            }
        return power_of(254 - up);
    };
    auto begin_item = [&]() {
        if constexpr (C::kQueriesShared) {
            // (every warp has passed the barrier that ends the item before)
            for (int x = w; x < kHeadTiles; x += kWarps) {
                load_queries(cur, x, qf[0]);
                const float back = convert_queries(qf[0]);
                uint16_t* row = sm_q + (x * 8 + (lane >> 2)) * C::kQueryRow + (lane & 3) * 4;
#pragma unroll
                for (int d = 0; d < D / 16; ++d)
                    *reinterpret_cast<uint2*>(row + d * 16) = make_uint2(qf[0][d][0], qf[0][d][1]);
                if (lane % 4 == 0) sm_q_scale[x * 8 + (lane >> 2)] = back;
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int x = 0; x < kHeadTiles; ++x) {
                const float back = convert_queries(qf[x]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    q_scale[x][e] = std::is_same<T, H>::value
                                        ? 1.f
                                        : __shfl_sync(kAll, back, ((lane & 3) * 2 + e) * 4);
            }
        }
    };
    auto load_all_queries = [&](const Cursor<Fp8Rows>& of) {
        if constexpr (!C::kQueriesShared)
#pragma unroll
            for (int x = 0; x < kHeadTiles; ++x) load_queries(of, x, qf[x]);
    };
    load_all_queries(cur);
    for (int t = t0, stage = 0; t < t1;) {
        if (fresh) {
            fresh = false;
            begin_item();
#pragma unroll
            for (int x = 0; x < kHeadTiles; ++x) {
#pragma unroll
                for (int d = 0; d < D / 16; ++d)
                    acc[x][d][0] = acc[x][d][1] = acc[x][d][2] = acc[x][d][3] = 0.f;
                m[x][0] = m[x][1] = -INFINITY;
                l[x][0] = l[x][1] = 0.f;
            }
        }
        __syncwarp();
        load((stage + C::kStages - 1) % C::kStages);
        cp_wait<C::kStages - 1>();
        __syncwarp();

        const int row0 = cur.tile * kTile + w * kSlice;
        if (row0 < cur.span.rows()) {
            // the lane's piece of rows `lane & 15`, of which there are two a load: piece d lies at d ^ it
            const uint32_t ks = ring0 + stage * C::kCodeBytes, vs = ks + kSlice * D;
            const uint32_t at = C::place(lane & 15, lane >> 4);
            float s[kHeadTiles][kSubs][4];
#pragma unroll
            for (int d = 0; d < D / 16; d += 2) {
#pragma unroll
                for (int y = 0; y < kSubs; ++y) {
                    uint32_t two[4];               // rows 0 .. 7 and 8 .. 15 of elements d, of d + 1
                    ldsm4(two, ks + (at ^ d << 4) + y * kSub * D);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint32_t a[4] = {codes_to_half2(two[2 * z]), codes_to_half2(two[2 * z + 1]),
                                               codes_to_half2(two[2 * z] >> 16),
                                               codes_to_half2(two[2 * z + 1] >> 16)};
#pragma unroll
                        for (int x = 0; x < kHeadTiles; ++x) {
                            uint2 b;
                            if constexpr (C::kQueriesShared)
                                b = *reinterpret_cast<const uint2*>(
                                    sm_q + (x * 8 + (lane >> 2)) * C::kQueryRow + (d + z) * 16 +
                                    (lane & 3) * 4);
                            else
                                b = make_uint2(qf[x][d + z][0], qf[x][d + z][1]);
                            if (d + z == 0)
                                mma_first<H>(s[x][y], a, b.x, b.y);
                            else
                                mma<H>(s[x][y], a, b.x, b.y);
                        }
                    }
                }
            }
            // the scales of the lane's token, and of its rows, row0 + 8 j + lane / 4
            float k_scale[2 * kSubs], v_scale[2 * kSubs], slice_scale;
            bool far;                              // the values' scales are far apart (for the warp)
            {
                uint32_t two[kPer], largest = 0;
                float kf[kPer], vf[kPer];
#pragma unroll
                for (int y = 0; y < kPer; ++y) {
                    two[y] = scales0[stage * (C::kScaleBytes / 2) + y * 32];
                    largest = max(largest, two[y] >> 8);
                }
                largest = __reduce_max_sync(kAll, largest);
                slice_scale = power_of(static_cast<int>(largest) - 15);
                far = false;
#pragma unroll
                for (int y = 0; y < kPer; ++y) {
                    const int e = two[y] >> 8, below = static_cast<int>(largest) - e;
                    far = far || (below > kFar && two[y] != kUnseen);
                    kf[y] = scale_of(two[y] & 0xffu) * p.scale_log2;
                    vf[y] = e == 255 ? NAN : below < 142 ? power_of(142 - below) : 0.f;
                }
                far = __any_sync(kAll, far);
#pragma unroll
                for (int j = 0; j < 2 * kSubs; ++j) {
                    k_scale[j] = __shfl_sync(kAll, kf[j / 4 % kPer], (j * 8 + (lane >> 2)) & 31);
                    v_scale[j] = __shfl_sync(kAll, vf[j / 4 % kPer], (j * 8 + (lane >> 2)) & 31);
                }
            }
#pragma unroll
            for (int x = 0; x < kHeadTiles; ++x)
#pragma unroll
                for (int j = 0; j < 2 * kSubs; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) s[x][j / 2][j % 2 * 2 + e] *= k_scale[j];
            if (!cur.span.all_seen(row0, kSlice)) {
                const Fp8Span span = Fp8Span::of(p, cur.i);
#pragma unroll
                for (int j = 0; j < 2 * kSubs; ++j)
                    if (!span.seen(span.token(row0 + j * 8 + (lane >> 2)))) {
#pragma unroll
                        for (int x = 0; x < kHeadTiles; ++x)
                            s[x][j / 2][j % 2 * 2] = s[x][j / 2][j % 2 * 2 + 1] = -INFINITY;
                    }
            }
            uint32_t pb[kHeadTiles][kSubs][2][2];  // [piece][rows 0 .. 7, 8 .. 15]
            float corr[kHeadTiles][2], back[kHeadTiles][2];        // factors of the running sums, of the slice's
#pragma unroll
            for (int x = 0; x < kHeadTiles; ++x) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float by = !C::kQueriesShared               ? q_scale[C::kQueriesShared ? 0 : x][e]
                                     : std::is_same<T, H>::value      ? 1.f
                                                                      : sm_q_scale[x * 8 + (lane & 3) * 2 + e];
                    float own = -INFINITY;         // the slice's largest
#pragma unroll
                    for (int j = 0; j < 2 * kSubs; ++j) own = fmaxf(own, s[x][j / 2][j % 2 * 2 + e]);
                    own = fmaxf(own, __shfl_xor_sync(kAll, own, 4));
                    own = fmaxf(own, __shfl_xor_sync(kAll, own, 8));
                    own = fmaxf(own, __shfl_xor_sync(kAll, own, 16)) * by;
                    const float top = fmaxf(own, m[x][e]);
                    // scores of -infinity only: any finite reference leaves their weights 0
                    const float ref = fmaxf(top, -FLT_MAX), base = fmaxf(own, -FLT_MAX);
                    const float share = exp2_fast(own - ref);
                    corr[x][e] = exp2_fast(m[x][e] - ref);
                    m[x][e] = top;
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < 2 * kSubs; ++j) {
                        float& v = s[x][j / 2][j % 2 * 2 + e];
                        v = exp2_fast(fmaf(v, by, -base));
                        sum += v;
                        v *= v_scale[j];
                    }
                    l[x][e] = fmaf(l[x][e], corr[x][e], sum * share);
                    back[x][e] = slice_scale * share;
                }
            }
            if (far) {                             // each head's largest to 2^14 .. 2^15
#pragma unroll
                for (int x = 0; x < kHeadTiles; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float most = 0.f;
#pragma unroll
                        for (int j = 0; j < 2 * kSubs; ++j) most = fmaxf(most, s[x][j / 2][j % 2 * 2 + e]);
                        most = fmaxf(most, __shfl_xor_sync(kAll, most, 4));
                        most = fmaxf(most, __shfl_xor_sync(kAll, most, 8));
                        most = fmaxf(most, __shfl_xor_sync(kAll, most, 16));
                        const int up = min(max(141 - static_cast<int>(__float_as_uint(most) >> 23), 0), 127);
#pragma unroll
                        for (int j = 0; j < 2 * kSubs; ++j) s[x][j / 2][j % 2 * 2 + e] *= power_of(127 + up);
                        back[x][e] *= power_of(127 - up);
                    }
            }
#pragma unroll
            for (int x = 0; x < kHeadTiles; ++x) {
#pragma unroll
                for (int j = 0; j < 2 * kSubs; ++j) {
                    const float v0 = s[x][j / 2][j % 2 * 2], v1 = s[x][j / 2][j % 2 * 2 + 1];
                    const uint32_t piece = Half2<H>::pack(v0, v1);
                    const float2 f = Half2<H>::unpack(piece);
                    pb[x][j / 2][0][j % 2] = transpose8x8(piece);
                    pb[x][j / 2][1][j % 2] = transpose8x8(Half2<H>::pack(v0 - f.x, v1 - f.y));
                }
            }
            // a slice's products are summed on their own and added to the rescaled sums: a matrix
            // product cuts its sum's last bits off, which would add up over a long axis
#pragma unroll
            for (int d = 0; d < D / 16; d += 2) {
                // (two pieces of 16 elements beside each other, but for the shapes with the most sums)
                constexpr int kBeside = D == 256 ? 1 : 2;
                float o[kBeside][kHeadTiles][4];
                uint32_t two[4];                   // tokens 0 .. 7 and 8 .. 15 of elements d, of d + 1
#pragma unroll
                for (int z0 = 0; z0 < 2; z0 += kBeside) {
#pragma unroll
                    for (int y = 0; y < kSubs; ++y) {
                        static_assert(kBeside == 2 || kSubs == 1, "loaded once");
                        if (z0 == 0) ldsm4_trans(two, vs + (at ^ d << 4) + y * kSub * D);
                        uint32_t a[kBeside][4];
#pragma unroll
                        for (int z = 0; z < 2 * kBeside; ++z) {
                            const uint32_t sorted = __byte_perm(two[2 * z0 + z], 0u, 0x3120);
                            a[z / 2][z % 2 * 2] = codes_to_half2(sorted);
                            a[z / 2][z % 2 * 2 + 1] = codes_to_half2(sorted >> 16);
                        }
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int z = 0; z < kBeside; ++z)
#pragma unroll
                                for (int x = 0; x < kHeadTiles; ++x) {
                                    if (y + c == 0)
                                        mma_first<H>(o[z][x], a[z], pb[x][y][c][0], pb[x][y][c][1]);
                                    else
                                        mma<H>(o[z][x], a[z], pb[x][y][c][0], pb[x][y][c][1]);
                                }
                    }
#pragma unroll
                    for (int z = 0; z < kBeside; ++z)
#pragma unroll
                        for (int x = 0; x < kHeadTiles; ++x)
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                float* const sum = acc[x][d + z0 + z] + e;
                                const uint64_t old =
                                    mul2(pair(sum[0], sum[1]), pair(corr[x][0], corr[x][1]));
                                const float2 f = halves(fma2(pair(o[z][x][e], o[z][x][e + 1]),
                                                             pair(back[x][0], back[x][1]), old));
                                sum[0] = f.x, sum[1] = f.y;
                            }
                }
            }
        }

        // ---- the item's end, or the range's: join the warps (the next item's queries are on their way).
        // The stage just done is free until the next load; a cluster's blocks, which have nothing more
        // to load, use the first.
        const bool item_ends = cur.tile + 1 == cur.tiles;
        const int then = t + 1 + (!kCluster && item_ends ? C::kEndTiles : 0);      // the next tile
        [[maybe_unused]] Cursor<Fp8Rows> next = cur;
        if constexpr (!kCluster && !C::kQueriesShared) {
            if (then < t1) advance<kTile>(next, p);
            if (item_ends && then < t1) load_all_queries(next);
        }
        if (item_ends || then >= t1) {
            float* const to = merge + (C::kMergeInRing && !kCluster ? stage * (C::kCodeBytes / 4) : 0);
            join_warps<T, C, kCluster>(p, cur, r, t, acc, m, l, to, sm_m, sm_l, sm_i);
            fresh = true;
        }
        if constexpr (kCluster) {
            if (then < t1) ++cur.tile;
        } else if constexpr (C::kQueriesShared) {
            if (then < t1) advance<kTile>(cur, p);
        } else {
            cur = next;
        }
        t = then;
        stage = stage + 1 == C::kStages ? 0 : stage + 1;
    }
    if constexpr (kCluster) join_cluster<T, C>(p, cur, merge, sm_i);
}

template <typename T, int D, int kHeadTiles>
int run(const Fp8Params& p, int64_t most_tokens, int sms, cudaStream_t stream)
{
    return launch_attention<T, Fp8Cfg<D, kHeadTiles>,
                            paged_attention_fp8_kernel<T, D, kHeadTiles, false>,
                            paged_attention_fp8_kernel<T, D, kHeadTiles, true>>(p, most_tokens, sms,
                                                                               stream);
}

template <typename T>
int dispatch(const Fp8Params& p, int64_t d, int64_t most, int sms, cudaStream_t s)
{
    const bool two = p.group > 8;
    if (d == 64) return two ? run<T, 64, 2>(p, most, sms, s) : run<T, 64, 1>(p, most, sms, s);
    if (d == 128) return two ? run<T, 128, 2>(p, most, sms, s) : run<T, 128, 1>(p, most, sms, s);
    return two ? run<T, 256, 2>(p, most, sms, s) : run<T, 256, 1>(p, most, sms, s);
}

}  // namespace

extern "C" {

int decode_paged_attention_fp8_workspace_bytes(int64_t h_q, int64_t h_kv, int64_t head_dim,
                                               size_t* bytes)
{
    clear_error();
    if (bytes == nullptr) return fail(DECODE_ERR_INVALID_ARG, "bytes is null");
    const int rc = check_heads(h_q, h_kv, head_dim);
    if (rc != DECODE_OK) return rc;
    const int sms = sm_count();
    if (sms == 0) return DECODE_ERR_CUDA;
    *bytes = layout_for(sms, kMostResident, heads_of(h_q / h_kv), head_dim).total;
    return DECODE_OK;
}

int decode_paged_attention_fp8(const decode_paged_attention_fp8_args* a, cudaStream_t stream)
{
    clear_error();
    if (a == nullptr) return fail(DECODE_ERR_INVALID_ARG, "args is null");
    if (a->n < 0 || a->table_width < 0 || a->window < 0 || a->sinks < 0)
        return fail(DECODE_ERR_INVALID_ARG, "negative size");
    if (a->dtype != DECODE_F16 && a->dtype != DECODE_BF16)
        return fail(DECODE_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
    int rc = check_heads(a->h_q, a->h_kv, a->head_dim);
    if (rc == DECODE_OK) rc = check_cache(a->pages, a->page_size, a->block_size, a->h_kv, a->head_dim);
    if (rc != DECODE_OK || a->n == 0) return rc;
    if (!a->q || !a->o || !a->lens || !a->workspace ||
        (a->table_width > 0 && a->pages > 0 &&
         (!a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale || !a->page_table)))
        return fail(DECODE_ERR_INVALID_ARG, "null pointer");
    if (misaligned(a->q) || misaligned(a->k_cache) || misaligned(a->v_cache) || misaligned(a->o) ||
        misaligned(a->workspace))
        return fail(DECODE_ERR_UNSUPPORTED, "16-bit tensors, codes and workspace must be 16-byte aligned");
    Fp8Params p{};
    if (!take_strides(p.q_stride, a->q_stride, {a->n, a->h_q}, 8))
        return fail(DECODE_ERR_UNSUPPORTED, "strides must be multiples of 8");
    const int64_t cs[3] = {a->pages, a->page_size, a->h_kv};
    const int64_t ss[3] = {a->pages, a->page_size / a->block_size, a->h_kv};
    int64_t stride[2][3], scale_stride[2][3];
    if (!take_strides(stride[0], a->k_stride, cs, 16) || !take_strides(stride[1], a->v_stride, cs, 16))
        return fail(DECODE_ERR_UNSUPPORTED, "cache strides must be multiples of 16");
    take_strides(scale_stride[0], a->k_scale_stride, ss, 1);
    take_strides(scale_stride[1], a->v_scale_stride, ss, 1);
    for (int of = 0; of < 2; ++of) {
        for (int x = 0; x < 2; ++x) {
            if (stride[of][x] < 0 || stride[of][x] > UINT32_MAX || scale_stride[of][x] < 0 ||
                scale_stride[of][x] > UINT32_MAX)
                return fail(DECODE_ERR_UNSUPPORTED, "strides of pages, tokens and blocks must be below 2^32");
            p.stride[of][x] = static_cast<uint32_t>(stride[of][x]);
            p.scale_stride[of][x] = static_cast<uint32_t>(scale_stride[of][x]);
        }
        p.head_stride[of] = stride[of][2];
        p.scale_head_stride[of] = scale_stride[of][2];
    }
    p.same = std::equal(stride[0], stride[0] + 3, stride[1]) &&
             std::equal(scale_stride[0], scale_stride[0] + 3, scale_stride[1]);
    constexpr int64_t kMost = (int64_t(1) << 31) - 1;
    if (a->n > kMost || a->h_q >= (1 << 20) || a->table_width > kMost)
        return fail(DECODE_ERR_UNSUPPORTED, "problem too large for one call");
    const int sms = sm_count();
    if (sms == 0) return DECODE_ERR_CUDA;
    const int64_t group = a->h_q / a->h_kv;
    const int heads = heads_of(group);
    const Layout l = layout_for(sms, kMostResident, heads, a->head_dim);
    if (a->workspace_bytes < 0 || static_cast<size_t>(a->workspace_bytes) < l.total)
        return fail(DECODE_ERR_INVALID_ARG, "workspace of %zu bytes needed", l.total);
    // (an item's queries are in registers, in all of its blocks, before its results are written)
    const int64_t d = a->head_dim, sizes[2] = {a->n, a->h_q}, dense[2] = {a->h_q * d, d};
    const int shared = refuse_shared(
        {{"o", a->o, 2, d, sizes, dense, "q"},
         {"lse", a->lse, 4, a->n * a->h_q},
         {"workspace", a->workspace, 1, static_cast<int64_t>(l.total)}},
        {{"q", a->q, 2, d, sizes, p.q_stride},
         {"k_cache", a->k_cache, 1, d, cs, stride[0]},
         {"v_cache", a->v_cache, 1, d, cs, stride[1]},
         {"k_scale", a->k_scale, 1, 1, ss, scale_stride[0]},
         {"v_scale", a->v_scale, 1, 1, ss, scale_stride[1]},
         {"page_table", a->page_table, 4, a->table_width, {a->n}, {a->table_stride}},
         {"lens", a->lens, 4, a->n}});
    if (shared != DECODE_OK) return shared;
    // lengths are 32-bit: a table that could hold more holds no more than that (and the last
    // tile's positions stay below 2^31)
    int64_t max_len = a->pages == 0 ? 0 : a->page_size * a->table_width;
    if (max_len > kMost - 1024) max_len = kMost - 1024;

    p.status = status_word();
    if (p.status == nullptr) return DECODE_ERR_CUDA;
    auto* ws = static_cast<uint8_t*>(a->workspace);
    p.q = static_cast<const uint16_t*>(a->q);
    p.k = static_cast<const uint8_t*>(a->k_cache);
    p.v = static_cast<const uint8_t*>(a->v_cache);
    p.scale[0] = static_cast<const uint8_t*>(a->k_scale);
    p.scale[1] = static_cast<const uint8_t*>(a->v_scale);
    p.table = a->page_table;
    p.lens = a->lens;
    p.o = static_cast<uint16_t*>(a->o);
    p.lse = a->lse;
    p.split = reinterpret_cast<int4*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + l.ml);
    p.part_o = reinterpret_cast<float*>(ws + l.o);
    p.table_stride = a->n > 1 ? a->table_stride : 0;
    p.max_len = max_len;
    p.n = static_cast<int32_t>(a->n);
    p.h_q = static_cast<int32_t>(a->h_q);
    p.h_kv = static_cast<int32_t>(a->h_kv);
    p.group = static_cast<int32_t>(group);
    p.head_items = static_cast<int32_t>((group + heads - 1) / heads);
    p.pages = static_cast<int32_t>(a->pages);
    p.page_size = static_cast<int32_t>(a->page_size);
    p.page_shift = shift_of(a->page_size);
    p.block = static_cast<int32_t>(a->block_size);
    p.block_shift = shift_of(a->block_size);
    p.window = a->window > kMost ? 0 : static_cast<int32_t>(a->window);
    p.sinks = a->sinks > max_len ? static_cast<int32_t>(max_len) : static_cast<int32_t>(a->sinks);
    p.scale_log2 = a->scale * 1.4426950408889634f;
    // rows of a sequence's axis: window and first tokens, each rounded to 16 rows
    const int64_t seen = static_cast<int64_t>(p.window) + p.sinks + 2 * kSub;
    const int64_t most = p.window > 0 && seen < max_len ? seen : max_len;
    return a->dtype == DECODE_BF16 ? dispatch<__nv_bfloat16>(p, a->head_dim, most, sms, stream)
                                   : dispatch<__half>(p, a->head_dim, most, sms, stream);
}

}  // extern "C"
