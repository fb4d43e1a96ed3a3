// What the attention kernels over a paged cache share, whatever the cache holds (paged_attention.cu:
// 16-bit keys and values, paged_attention_fp8.cu: 8-bit codes with scales): matrix instructions, the
// split of all items' tiles into equal ranges, one a block, and the joins of warps, of a cluster's
// blocks and of an item's parts.  paged_attention.cu says why the work is split so.
#pragma once

#include <cstdint>
#include <type_traits>

#include "decode_mma.cuh"

namespace decode {

constexpr int kSub = 16;         // tokens of a matrix tile
constexpr int kClusterMost = 8;      // blocks of a cluster
constexpr int kClusterTiles = 3;     // tiles of each of them
constexpr int kSharedItems = 64;     // items up to which the join takes a block a head
constexpr int kListedItems = 1024;   // items up to which the join goes by item

// What splitting and joining go by; an attention kernel's parameters begin with it.
struct SplitParams {
    const int32_t* lens;
    uint16_t* o;
    float* lse;
    uint32_t* status;
    int4* split;       // by item or by its first block: (first block, -1 if in one block; last; i, item)
    float2* part_ml;   // [2 * blocks][kHeads]
    float* part_o;     // [2 * blocks][kHeads][D]
    int64_t max_len;
    int32_t n, h_q, h_kv, group, head_items, by_item, join_shared;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a row's sums are multiplied by, from the sum of its weights, which its products carry times
// 2^kShift: 0 where every score is -infinity; and two of its elements, which are then 0 whatever the
// values hold.
template <int kShift>
__device__ __forceinline__ float factor_of(float sum)
{
    return sum == 0.f ? 0.f : 1.f / (1 << kShift) / sum;
}
template <typename T>
__device__ __forceinline__ uint32_t result(float x, float y, float factor)
{
    return factor == 0.f ? 0u : Half2<T>::pack(x * factor, y * factor);
}

// Tiles [first, last) of block c when `total` tiles are dealt to `blocks` blocks; and the block
// that a tile is dealt to.
__device__ __forceinline__ int first_tile(int c, int total, int blocks)
{
    const int each = total / blocks, more = total % blocks;
    return c * each + min(c, more);
}
__device__ __forceinline__ int block_of(int tile, int total, int blocks)
{
    const int each = total / blocks, more = total % blocks;
    const int big = more * (each + 1);
    return tile < big ? tile / (each + 1) : more + (tile - big) / each;
}

// Where a warp is in the block's range of tiles.  Span, an attention's own, says which of a
// sequence's tokens are seen: rows() of them are dealt to tiles, none where len is 0, and
// Span::of(parameters, sequence) makes it.
template <typename Span>
struct Cursor {
    int i;              // sequence
    int item;           // of the sequence: key head * head_items + head tile group
    int tile;           // of the item
    int tiles;          // of each of the sequence's items
    Span span;
};

template <int kTileTokens, typename Span>
__device__ __forceinline__ int tiles_of(const Span& s)
{
    return (s.rows() + kTileTokens - 1) / kTileTokens;
}

template <int kTileTokens, typename Span, typename P>
__device__ __forceinline__ void advance(Cursor<Span>& c, const P& p)
{
    if (++c.tile < c.tiles) return;
    c.tile = 0;
    if (++c.item < p.h_kv * p.head_items) return;
    c.item = 0;
    do {
        if (++c.i >= p.n) return;     // past the last tile: the caller stops by its count
        c.span = Span::of(p, c.i);
        c.tiles = tiles_of<kTileTokens>(c.span);
    } while (c.tiles == 0);
}

// A block's share [t0, t1) of what is dealt, `total` of it in `blocks` blocks: an item's tiles in order and
// kEndTiles more for its end, at which the warps are joined and nothing is on its way.
struct Range {
    int t0, t1, total = 0, blocks = 0;
};

// The range of a block of a cluster: its share of its cluster's item, whose tiles are numbered from
// 0.  False, for all of the cluster's blocks, where the item has no tile: its result is written then.
template <typename C, typename Span, typename P>
__device__ __forceinline__ bool cluster_range(const P& p, Cursor<Span>& cur, Range& r, int* sm_i)
{
    constexpr int D = C::kD, kHeads = C::kHeads;
    const int tid = threadIdx.x, c = blockIdx.x;
    const int items_per_seq = p.h_kv * p.head_items;
    const int ranks = cluster_size(), item = c / ranks;
    cur.i = item / items_per_seq;
    cur.item = item % items_per_seq;
    cur.span = Span::of(p, cur.i);
    cur.tiles = tiles_of<C::kTile>(cur.span);
    if (cur.item == 0 && c % ranks == 0 && tid == 0 && p.lens[cur.i] != cur.span.len)
        atomicOr(p.status, DECODE_BAD_LENGTH);
    const int each = (cur.tiles + ranks - 1) / ranks;
    r.t0 = cur.tile = min(c % ranks * each, cur.tiles);
    r.t1 = min(r.t0 + each, cur.tiles);
    if (cur.tiles == 0) {                      // for all of the cluster's blocks
        if (c % ranks == 0) {
            const int h0 = cur.item / p.head_items * p.group + cur.item % p.head_items * kHeads;
            const int heads = min(kHeads, p.group - cur.item % p.head_items * kHeads);
            const int64_t row = static_cast<int64_t>(cur.i) * p.h_q + h0;
            for (int x = tid; x < heads * (D / 8); x += C::kThreads)
                reinterpret_cast<uint4*>(p.o + row * D)[x] = make_uint4(0, 0, 0, 0);
            if (p.lse != nullptr && tid < heads) p.lse[row + tid] = -INFINITY;
        }
        return false;
    }
    // the block's maxima and sums, for its cluster (a block may have no tile)
    if (tid < 2 * kHeads)
        reinterpret_cast<float*>(sm_i)[tid] = tid < kHeads ? -INFINITY : 0.f;
    __syncthreads();
    return true;
}

// The range of any other block: a scan of all sequences' tiles.  False where the block has no tile.
template <typename C, typename Span, typename P>
__device__ __forceinline__ bool block_range(const P& p, Cursor<Span>& cur, Range& r, int* sm_i)
{
    constexpr int D = C::kD, kTile = C::kTile, kWarps = C::kWarps;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, c = blockIdx.x;
    const int items_per_seq = p.h_kv * p.head_items;
    const int chunk = (p.n + C::kThreads - 1) / C::kThreads;
    const int i_lo = min(p.n, tid * chunk), i_hi = min(p.n, i_lo + chunk);
    // what a sequence's items are dealt as
    auto dealt = [&](int i) {
        const int tiles = tiles_of<kTile>(Span::of(p, i));
        return (tiles + (tiles > 0 ? C::kEndTiles : 0)) * items_per_seq;
    };
    int mine = 0;
    for (int i = i_lo; i < i_hi; ++i) mine += dealt(i);
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += x;
    }
    if (lane == 31) sm_i[w] = upto;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
        if (x == w) upto += r.total;
        r.total += sm_i[x];
    }
    r.blocks = min(static_cast<int>(gridDim.x), r.total);   // with a tile, or an item's end, each at least
    r.t0 = c < r.blocks ? first_tile(c, r.total, r.blocks) : r.total;
    r.t1 = c < r.blocks ? first_tile(c + 1, r.total, r.blocks) : r.total;
    if (r.t0 >= upto - mine && r.t0 < upto) {          // one thread: its sequences hold tile r.t0
        int at = upto - mine;
        for (int i = i_lo; i < i_hi; ++i) {
            const int tiles = dealt(i);
            if (r.t0 < at + tiles) {
                sm_i[32] = i;
                sm_i[33] = r.t0 - at;
                break;
            }
            at += tiles;
        }
    }
    // sequences without tokens have no tile: their results are written here
    for (int i = c; i < p.n; i += gridDim.x) {
        const int raw = p.lens[i];
        const Span s = Span::of(p, i);
        if (tid == 0 && raw != s.len) atomicOr(p.status, DECODE_BAD_LENGTH);
        if (s.len > 0) continue;
        uint4* row = reinterpret_cast<uint4*>(p.o + static_cast<int64_t>(i) * p.h_q * D);
        for (int x = tid; x < p.h_q * (D / 8); x += C::kThreads) row[x] = make_uint4(0, 0, 0, 0);
        if (p.lse != nullptr)
            for (int x = tid; x < p.h_q; x += C::kThreads)
                p.lse[static_cast<int64_t>(i) * p.h_q + x] = -INFINITY;
        if (p.by_item)
            for (int x = tid; x < items_per_seq; x += C::kThreads)
                p.split[i * items_per_seq + x] = make_int4(-1, 0, 0, 0);
    }
    if (tid == 0 && !p.by_item) p.split[c] = make_int4(-1, 0, 0, 0);
    if (r.t0 >= r.t1) return false;
    __syncthreads();
    cur.i = sm_i[32];
    cur.span = Span::of(p, cur.i);
    cur.tiles = tiles_of<kTile>(cur.span);
    cur.item = sm_i[33] / (cur.tiles + C::kEndTiles);
    cur.tile = sm_i[33] % (cur.tiles + C::kEndTiles);
    if (cur.tile >= cur.tiles) {                   // an end, which the block before has: the next item
        r.t0 += cur.tiles + C::kEndTiles - cur.tile;       // (of which there may be none in the share)
        cur.tile = cur.tiles - 1;
        if (r.t0 < r.t1) advance<kTile>(cur, p);
    }
    return r.t0 < r.t1;
}

// An item's end at tile t, or the range's: joins the warps' sums of their own tiles, through kMergeWarp
// floats of `merge` for each warp, where element d of head h lies at merge_at(h, d).  acc[x][d] are the
// products of 16 elements and a head tile as the matrix instruction leaves them, whose row r stands for
// element r, or (kRowPairs) rows r and r + 8 for elements 2 r and 2 r + 1.  Ends with a barrier.
template <typename T, typename C, bool kCluster, typename Span, typename P>
__device__ __forceinline__ void join_warps(const P& p, const Cursor<Span>& cur, const Range& r, int t,
                                           const float (&acc)[C::kHeadTiles][C::kD / 16][4],
                                           const float (&m)[C::kHeadTiles][2],
                                           const float (&l)[C::kHeadTiles][2], float* merge,
                                           float* sm_m, float* sm_l, int* sm_i)
{
    constexpr int D = C::kD, kHeadTiles = C::kHeadTiles, kHeads = C::kHeads, kWarps = C::kWarps;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, c = blockIdx.x;
    const int hq = (lane & 3) * 2, items_per_seq = p.h_kv * p.head_items;
    const int h0 = cur.item / p.head_items * p.group + cur.item % p.head_items * kHeads;
    const int heads = min(kHeads, p.group - cur.item % p.head_items * kHeads);
#pragma unroll
    for (int x = 0; x < kHeadTiles; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = l[x][e];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            if (lane < 4) {
                sm_m[w * kHeads + x * 8 + hq + e] = m[x][e];
                sm_l[w * kHeads + x * 8 + hq + e] = sum;
            }
        }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kHeadTiles; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = x * 8 + hq + e;
            float top = sm_m[h];
#pragma unroll
            for (int y = 1; y < kWarps; ++y) top = fmaxf(top, sm_m[y * kHeads + h]);
            const float f = exp2_fast(m[x][e] - (top == -INFINITY ? 0.f : top));
            float* to = merge + w * C::kMergeWarp;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                if constexpr (C::kRowPairs) {
                    *reinterpret_cast<float2*>(to + C::merge_at(h, d * 16 + (lane >> 2) * 2)) =
                        make_float2(acc[x][d][e] * f, acc[x][d][2 + e] * f);
                } else {
                    to[C::merge_at(h, d * 16 + (lane >> 2))] = acc[x][d][e] * f;
                    to[C::merge_at(h, d * 16 + (lane >> 2) + 8)] = acc[x][d][2 + e] * f;
                }
            }
        }
    __syncthreads();
    const int begin = t - cur.tile;                   // the item's tiles are dealt as [begin, end)
    const int end = begin + cur.tiles;
    const bool whole = begin >= r.t0 && end <= r.t1;
    const int slot = 2 * c + (begin >= r.t0 ? 1 : 0);
    for (int x = tid; x < heads * (D / 4); x += C::kThreads) {
        const int h = x / (D / 4), d = x % (D / 4) * 4;
        float top = sm_m[h];
#pragma unroll
        for (int y = 1; y < kWarps; ++y) top = fmaxf(top, sm_m[y * kHeads + h]);
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int y = 0; y < kWarps; ++y) {
            sum = fmaf(sm_l[y * kHeads + h], exp2_fast(sm_m[y * kHeads + h] - ref), sum);
            const float4 b = *reinterpret_cast<const float4*>(
                merge + y * C::kMergeWarp + C::merge_at(h, d));
            o.x += b.x, o.y += b.y, o.z += b.z, o.w += b.w;
        }
        if constexpr (kCluster) {
            // (each element of the first warp's rows is read by this thread alone)
            *reinterpret_cast<float4*>(merge + C::merge_at(h, d)) = o;
            if (d == 0) {
                reinterpret_cast<float*>(sm_i)[h] = top;
                reinterpret_cast<float*>(sm_i)[kHeads + h] = sum;
            }
        } else if (whole) {
            const int64_t row = static_cast<int64_t>(cur.i) * p.h_q + h0 + h;
            const float inv = factor_of<C::template kShift<T>>(sum);
            *reinterpret_cast<uint2*>(p.o + row * D + d) = make_uint2(
                result<T>(o.x, o.y, inv), result<T>(o.z, o.w, inv));
            if (d == 0 && p.lse != nullptr)
                p.lse[row] = (top + log2f(sum)) * 0.6931471805599453f;
        } else {
            const int64_t row = static_cast<int64_t>(slot) * kHeads + h;
            *reinterpret_cast<float4*>(p.part_o + row * D + d) = o;
            if (d == 0) p.part_ml[row] = make_float2(top, sum);
        }
    }
    if (!kCluster && tid == 0 && begin >= r.t0 && (p.by_item || !whole))
        p.split[p.by_item ? cur.i * items_per_seq + cur.item : c] = make_int4(
            whole ? -1 : c, whole ? 0 : block_of(end - 1, r.total, r.blocks), cur.i, cur.item);
    __syncthreads();
}

// The end of a cluster: joins its blocks, each an equal share of the elements.
template <typename T, typename C, typename Span, typename P>
__device__ __forceinline__ void join_cluster(const P& p, const Cursor<Span>& cur, const float* merge,
                                             const int* sm_i)
{
    constexpr int D = C::kD, kHeads = C::kHeads;
    const int tid = threadIdx.x;
    const uint32_t ranks = cluster_size(), rank = cluster_rank();
    const int h0 = cur.item / p.head_items * p.group + cur.item % p.head_items * kHeads;
    const int heads = min(kHeads, p.group - cur.item % p.head_items * kHeads);
    const int each = (cur.tiles + static_cast<int>(ranks) - 1) / static_cast<int>(ranks);
    const int used = (cur.tiles + each - 1) / each;      // blocks with a tile
    cluster_barrier();
    for (int x = rank * C::kThreads + tid; x < heads * (D / 4); x += ranks * C::kThreads) {
        const int h = x / (D / 4), d = x % (D / 4) * 4;
        float top = -INFINITY;
        for (int y = 0; y < used; ++y)
            top = fmaxf(top, cluster_load(cluster_address(smem_addr(sm_i + h), y)));
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int y = 0; y < used; ++y) {
            const float f =
                exp2_fast(cluster_load(cluster_address(smem_addr(sm_i + h), y)) - ref);
            const float4 b = cluster_load4(
                cluster_address(smem_addr(merge + C::merge_at(h, d)), y));
            sum = fmaf(cluster_load(cluster_address(smem_addr(sm_i + kHeads + h), y)), f, sum);
            o.x = fmaf(b.x, f, o.x), o.y = fmaf(b.y, f, o.y);
            o.z = fmaf(b.z, f, o.z), o.w = fmaf(b.w, f, o.w);
        }
        const int64_t row = static_cast<int64_t>(cur.i) * p.h_q + h0 + h;
        const float inv = factor_of<C::template kShift<T>>(sum);
        *reinterpret_cast<uint2*>(p.o + row * D + d) = make_uint2(
            result<T>(o.x, o.y, inv), result<T>(o.z, o.w, inv));
        if (d == 0 && p.lse != nullptr)
            p.lse[row] = (top + log2f(sum)) * 0.6931471805599453f;
    }
    cluster_barrier();                             // the others may still read this block's part
}

// Joins the parts of an item that went over several blocks' ranges: part 0 is its first block's slot
// 2 c + 1, the others are their blocks' slots 2 c'.  Block x has the item listed at x.  With one
// block an item each warp joins heads of its own; with a block (x, y) for each head, which is for
// few items of many parts, the block's warps share the head's parts out.  It is a chain of three
// dependent loads (the list, maxima and sums, outputs), so each is issued for all parts at once.
constexpr int kJoinWarps = 16;        // most warps of a block, else 8

// A warp's running join: its lanes hold D / 32 neighbouring outputs each.
template <int D>
struct Joined {
    static constexpr int kOut = D / 32;
    float top = -INFINITY, sum = 0.f, o[kOut] = {};

    // Takes in up to 32 parts; lane x has part x's maximum and sum (-infinity, 0: none), `row` is
    // the address of its output.
    __device__ __forceinline__ void take(float m, float l, const float* row, int count, int lane)
    {
        float next = fmaxf(m, top);
#pragma unroll
        for (int d = 16; d > 0; d /= 2) next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, d));
        const float ref = next == -INFINITY ? 0.f : next;
        const float old = exp2_fast(top - ref), f = exp2_fast(m - ref);
        top = next;
        sum *= old;
#pragma unroll
        for (int e = 0; e < kOut; ++e) o[e] *= old;
        constexpr int kBatch = 8;
        for (int x0 = 0; x0 < count; x0 += kBatch) {
            float b[kBatch][kOut];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                // lanes past the count name part 0 again, with weight 0
                const int at = x0 + x < count ? x0 + x : 0;
                const float* from = reinterpret_cast<const float*>(__shfl_sync(
                    0xffffffffu, reinterpret_cast<uint64_t>(row), at)) + lane * kOut;
                if constexpr (kOut == 2) {
                    const float2 v = *reinterpret_cast<const float2*>(from);
                    b[x][0] = v.x, b[x][1] = v.y;
                } else {
#pragma unroll
                    for (int e = 0; e < kOut; e += 4) {
                        const float4 v = *reinterpret_cast<const float4*>(from + e);
                        b[x][e] = v.x, b[x][e + 1] = v.y, b[x][e + 2] = v.z, b[x][e + 3] = v.w;
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                const float w = x0 + x < count ? __shfl_sync(0xffffffffu, f, (x0 + x) & 31) : 0.f;
                const float lx = x0 + x < count ? __shfl_sync(0xffffffffu, l, (x0 + x) & 31) : 0.f;
                if (x0 + x < count) {
                    sum = fmaf(lx, w, sum);
#pragma unroll
                    for (int e = 0; e < kOut; ++e) o[e] = fmaf(b[x][e], w, o[e]);
                }
            }
        }
    }
};

template <typename T, int D, int kHeadTiles, int kShift>
static __global__ void __launch_bounds__(kJoinWarps * 32, 1) paged_attention_join_kernel(const SplitParams p)
{
    constexpr int kHeads = 8 * kHeadTiles, kOut = Joined<D>::kOut;
    __shared__ __align__(16) float sm_o[kJoinWarps][D];
    __shared__ float2 sm_ml[kJoinWarps];
    dep_launch();
    dep_wait();
    const int4 item = p.split[blockIdx.x];
    if (item.x < 0) return;
    const int c = item.x, parts = item.y - c + 1;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h0 = item.w / p.head_items * p.group + item.w % p.head_items * kHeads;
    const int heads = min(kHeads, p.group - item.w % p.head_items * kHeads);
    const bool shared = p.join_shared;
    const int warps = blockDim.x >> 5;
    const int each = shared ? (parts + warps - 1) / warps : parts;
    const int first = shared ? min(w * each, parts) : 0, last = min(first + each, parts);

    for (int h = shared ? blockIdx.y : w; h < heads; h += shared ? gridDim.y : warps) {
        Joined<D> sums;
        for (int x0 = first; x0 < last; x0 += 32) {
            const int x = min(x0 + lane, last - 1);
            const int64_t slot = static_cast<int64_t>(x == 0 ? 2 * c + 1 : 2 * (c + x)) * kHeads + h;
            const float2 ml = p.part_ml[slot];
            const bool mine = x0 + lane < last;
            sums.take(mine ? ml.x : -INFINITY, mine ? ml.y : 0.f, p.part_o + slot * D,
                      min(32, last - x0), lane);
        }
        if (shared) {
#pragma unroll
            for (int e = 0; e < kOut; ++e) sm_o[w][lane * kOut + e] = sums.o[e];
            if (lane == 0) sm_ml[w] = make_float2(sums.top, sums.sum);
            __syncthreads();
            if (w == 0) {
                Joined<D> all;
                const float2 ml = sm_ml[min(lane, warps - 1)];
                all.take(lane < warps ? ml.x : -INFINITY, lane < warps ? ml.y : 0.f,
                         sm_o[min(lane, warps - 1)], warps, lane);
                sums = all;
            }
            __syncthreads();
            if (w != 0) continue;
        }
        const int64_t row = static_cast<int64_t>(item.z) * p.h_q + h0 + h;
        const float inv = factor_of<kShift>(sums.sum);
        uint32_t* out = reinterpret_cast<uint32_t*>(p.o + row * D + lane * kOut);
#pragma unroll
        for (int e = 0; e < kOut; e += 2)
            out[e / 2] = result<T>(sums.o[e], sums.o[e + 1], inv);
        if (lane == 0 && p.lse != nullptr)
            p.lse[row] = (sums.top + log2f(sums.sum)) * 0.6931471805599453f;
    }
}

struct Layout {
    size_t ml, o, total;
};
// (resident: the most blocks of an SM that any shape of the kernel has)
inline Layout layout_for(int sms, int resident, int heads, int64_t d)
{
    const size_t blocks = static_cast<size_t>(sms) * resident;
    Layout l{};
    size_t at = sizeof(int4) * (blocks > kListedItems ? blocks : kListedItems);
    l.ml = at = (at + 255) & ~size_t(255);
    at += sizeof(float2) * 2 * blocks * heads;
    l.o = at = (at + 255) & ~size_t(255);
    l.total = at + sizeof(float) * 2 * blocks * heads * static_cast<size_t>(d);
    return l;
}

inline int heads_of(int64_t group) { return group > 8 ? 16 : 8; }

// Launches an attention of at most `most_tokens` tokens a sequence: kFlat, then the join, or kClusters.
template <typename T, typename C, auto kFlat, auto kClusters, typename P>
int launch_attention(P p, int64_t most_tokens, int sms, cudaStream_t stream)
{
    const int64_t per_item = (most_tokens + C::kTile - 1) / C::kTile;
    const int64_t items = static_cast<int64_t>(p.n) * p.h_kv * p.head_items;
    if (per_item > 0 && items >= (int64_t(1) << 31) / (per_item + C::kEndTiles))
        return fail(DECODE_ERR_UNSUPPORTED, "too many tiles of the cache for one call");
    const int64_t tiles = (per_item + (per_item > 0 ? C::kEndTiles : 0)) * items;
    const int64_t most = static_cast<int64_t>(sms) * C::kResident;
    const int blocks = static_cast<int>(tiles < 1 ? 1 : tiles < most ? tiles : most);
    p.by_item = items <= kListedItems;
    p.join_shared = items <= kSharedItems;
    // Few items of few tiles: a cluster an item, which joins its blocks' parts itself, as large as
    // the GPU holds for all items, up to three tiles a block (8 key heads: one sequence of 500
    // tokens 5.7 us, 8.1 with the second kernel; 16 of up to 250 tokens 7.2 and 8.6; one of 1500
    // 7.5 and 8.8; with four tiles a block, one of 2000 took as long either way).  The lengths being
    // on the device, the page table's width stands for the longest (with a window, the window): short
    // sequences under a table made for long ones take the second kernel.
    int ranks = 1;
    while (ranks < kClusterMost && ranks < per_item && items * ranks * 2 <= most) ranks *= 2;
    // A block an item, as a cluster of one, where the items just fill the GPU and none has many tiles.
    const bool alone = ranks == 1 && per_item <= C::kAloneTiles && items <= most && 4 * items >= 3 * most;
    const bool cluster = alone || (ranks > 1 && per_item <= ranks * kClusterTiles);
    auto* kernel = cluster ? kClusters : kFlat;
    static thread_local bool set[2][kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(dev < kMaxDevices && set[cluster][dev])) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::kSmem > kSpreadMost ? C::kSmem : kSpreadMost);
        if (e == cudaSuccess && dev < kMaxDevices) set[cluster][dev] = true;
    }
    const int64_t grid = cluster ? items * ranks : blocks;
    if (e == cudaSuccess)
        e = launch_cluster(kernel, dim3(static_cast<uint32_t>(grid)), dim3(C::kThreads),
                           spread(C::kSmem, grid, sms, C::kResident), stream, cluster ? ranks : 1, p);
    if (e != cudaSuccess)
        return fail(DECODE_ERR_CUDA, "attention kernel: %s", cudaGetErrorString(e));
    if (cluster || per_item <= 1 || blocks == 1) return DECODE_OK;     // no item is cut
    const int64_t most_parts = per_item < blocks ? per_item : blocks;
    // (blocks of 16 warps need an SM each)
    const int64_t heads = !p.join_shared ? 1 : p.group < C::kHeads ? p.group : C::kHeads;
    const bool wide = p.join_shared && most_parts > 64 && items * heads <= sms;
    e = launch(paged_attention_join_kernel<T, C::kD, C::kHeadTiles, C::template kShift<T>>,
               dim3(p.by_item ? static_cast<uint32_t>(items) : blocks, static_cast<uint32_t>(heads)),
               dim3((wide ? kJoinWarps : 8) * 32), 0, stream, static_cast<SplitParams>(p));
    if (e != cudaSuccess)
        return fail(DECODE_ERR_CUDA, "attention join kernel: %s", cudaGetErrorString(e));
    return DECODE_OK;
}

inline int check_heads(int64_t h_q, int64_t h_kv, int64_t d)
{
    if (h_q <= 0 || h_kv <= 0 || h_q % h_kv != 0)
        return fail(DECODE_ERR_INVALID_ARG, "%lld query heads over %lld key heads", (long long)h_q,
                    (long long)h_kv);
    if (d != 64 && d != 128 && d != 256)
        return fail(DECODE_ERR_UNSUPPORTED, "head_dim %lld (64, 128 or 256)", (long long)d);
    return DECODE_OK;
}

}  // namespace decode
