// Attention of one new token per sequence over a paged key-value cache, split over the cache's
// length and joined (C ABI in include/decode.h).
//
//     s_t = scale q . K_t;   o = sum_t exp(s_t - m) V_t / sum_t exp(s_t - m)
//
// A key and a value of head_dim d are 4 d bytes and serve h_q / h_kv query heads with 4 d flops
// each: a few flops per byte, so the cache is read once and HBM bounds the time.  One pass: each
// warp keeps the running maximum and sum of its tokens' exponentials (log2 domain, fp32) and the
// unnormalised output, and results of warps and blocks are joined by their maxima.
//
// Work split.  An item is one (sequence, key head, up to 8 kHeadTiles of its query heads).  A tile is
// a slice (16 tokens, 32 at head_dim 64) of an item for each of a block's warps.  All items' tiles, in
// order, are cut into equal contiguous ranges, one a block, whatever the lengths: every block finds
// its range itself from a scan of the lengths.
// So a block has at most one item that began in an earlier block and one that goes on in a later
// one; those two go to the workspace as (maximum, sum, output) and a second kernel joins each
// item's parts in block order, the rest are written at once.  The order of every sum is fixed.
// Two blocks of four warps an SM, so that one streams while the other begins or joins an item: 64
// sequences of up to 8192 tokens, 8 key heads of 128, take 158 us (6.1 TB/s, 90% of what a copy
// reaches; the SMs are busy 91% of the time on average), against 175 us with one block of
// eight warps, whose SMs were busy 78% of the time; ranges four times finer than the
// GPU holds blocks, which even the SMs out, took 167 us, their blocks' beginnings cost more.
// Few items of few tiles, where the second kernel's launch would show, run as one thread-block
// cluster an item instead, whose blocks join their parts through distributed shared memory.
//
// Inside a block each warp streams its own slices through a ring of shared-memory stages
// (16-byte cp.async, rows looked up in the page table one slice ahead, so pages may have any size
// and the cache any strides) and needs no block barrier until an item ends; the ring runs on
// across items.  Tokens outside the sequence are filled with zeros and not read.
//
// Both products put the tokens or the head dimension on the 16 rows of mma.m16n8k16 and the
// query heads on its 8 columns, so up to 8 heads of a group cost no padding:
//     S^T[token][head] = K Q^T,     O^T[d][head] = V^T P^T.
// For the second product each weight is carried as 16-bit pieces, three of bfloat16 or two of
// float16 (each takes from p what the ones before left of it), which hold its 24 bits: with two pieces of
// bfloat16 a result that is a small difference of large terms was off by up to 2^-17 of them, and
// the third costs no time (64 sequences of up to 8192 tokens 161 us, one of 200001 tokens 74.6 us,
// with either), since the products are not what bounds it.  float16's weights are carried times
// 2^15 (and the results divided by it), which leaves them above 2^-40 of the warp's largest:
// unscaled, weights below 2^-25 vanished, and with them a long tail beside a token that takes
// nearly all the weight and has little to give.
#include <cstdint>
#include <type_traits>

#include "decode_common.cuh"

namespace {

using namespace decode;

constexpr int kSub = 16;         // tokens of a matrix tile
constexpr int kMostResident = 2;     // of Cfg::kResident
constexpr int kClusterMost = 8;      // blocks of a cluster
constexpr int kClusterTiles = 3;     // tiles of each of them
constexpr int kSharedItems = 64;     // items up to which the join takes a block a head
constexpr int kListedItems = 1024;   // items up to which the join goes by item

struct AttnParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const int32_t* table;
    const int32_t* lens;
    uint16_t* o;
    float* lse;
    uint32_t* status;
    int4* split;       // by item or by its first block: (first block, -1 if in one block; last; i, item)
    float2* part_ml;   // [2 * blocks][kHeads]
    float* part_o;     // [2 * blocks][kHeads][D]
    int64_t q_stride[2], k_stride[3], v_stride[3];
    int64_t table_stride, max_len;
    int32_t n, h_q, h_kv, group, head_items, pages, page_size, page_shift, window;
    int32_t by_item, join_shared;
    float scale_log2;
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
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16-bit pieces of a weight in the second product: what they leave out is less than the error of
// the exponential itself (2^-22), three of bfloat16's 8 bits nothing, two of float16's 11 2^-23.
template <typename T>
constexpr int kPieces = std::is_same<T, __half>::value ? 2 : 3;
// What the weights of the second product are multiplied by, a power of two.
template <typename T>
constexpr float kWeight = std::is_same<T, __half>::value ? 32768.f : 1.f;

// Takes piece c off a pair of weights.  An infinite value must come out infinite, so no piece of a
// weight above 0 may be 0 or below it where it meets one.  bfloat16: each piece but the last is cut
// off just below what is left of the weight (the product with 1 - 2^-23 takes a bit or two off), so
// that some of it always stays for the next; the three still hold all 24 bits.  float16, whose
// pieces run out of range first: the first piece is above 0, and the second's sums are cleared of
// infinities, below.
template <typename T>
__device__ __forceinline__ uint32_t take_piece(float& v0, float& v1, int c)
{
    if constexpr (std::is_same<T, __half>::value) {
        constexpr float kLeast = 5.9604645e-8f;          // 2^-24, the smallest number above 0
        const float f0 = c == 0 && v0 > 0.f && v0 < kLeast ? kLeast : v0;
        const float f1 = c == 0 && v1 > 0.f && v1 < kLeast ? kLeast : v1;
        const uint32_t piece = Half2<T>::pack(f0, f1);
        const float2 f = Half2<T>::unpack(piece);
        v0 -= f.x, v1 -= f.y;
        return piece;
    } else {
        if (c + 1 == kPieces<T>) return Half2<T>::pack(v0, v1);
        const uint32_t b0 = __float_as_uint(v0 * 0.99999988f), b1 = __float_as_uint(v1 * 0.99999988f);
        v0 -= __uint_as_float(b0 & 0xffff0000u), v1 -= __uint_as_float(b1 & 0xffff0000u);
        return __byte_perm(b0, b1, 0x7632);
    }
}

// What a row's sums are multiplied by, from the sum of its weights: 0 where every score is
// -infinity; and two of its elements, which are then 0 whatever the values hold.
template <typename T>
__device__ __forceinline__ float factor_of(float sum)
{
    return sum == 0.f ? 0.f : 1.f / kWeight<T> / sum;
}
template <typename T>
__device__ __forceinline__ uint32_t result(float x, float y, float factor)
{
    return factor == 0.f ? 0u : Half2<T>::pack(x * factor, y * factor);
}

// x, or a finite number for an infinity or NaN.
__device__ __forceinline__ float finite(float x)
{
    return fminf(fmaxf(x, -3.402823466e38f), 3.402823466e38f);
}

// ---- thread-block clusters: rank, barrier and reads of another block's shared memory
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" :::
                 "memory");
}
__device__ __forceinline__ uint32_t cluster_address(uint32_t smem, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem), "r"(rank));
    return r;
}
__device__ __forceinline__ float cluster_load(uint32_t address)
{
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(address) : "memory");
    return x;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t address)
{
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(address) : "memory");
    return x;
}

// A sequence's tokens [start, len); len = 0 for a length the page table cannot hold.  Its slices
// begin at `origin`, the start rounded down to a multiple of 16, so that where pages are multiples
// of 16 tokens, each 16 tokens of a slice lie in one page.
struct Span {
    int start, len;
    __device__ __forceinline__ int origin() const { return start & ~(kSub - 1); }
};
__device__ __forceinline__ Span span_of(const AttnParams& p, int i)
{
    int len = p.lens[i];
    if (len < 0 || len > p.max_len) len = 0;
    return {p.window > 0 && len > p.window ? len - p.window : 0, len};
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

// Where a warp is in the block's range of tiles.
struct Cursor {
    int i;              // sequence
    int item;           // of the sequence: key head * head_items + head tile group
    int tile;           // of the item
    int tiles;          // of each of the sequence's items
    Span span;
};

template <int kTileTokens>
__device__ __forceinline__ int tiles_of(const Span& s)
{
    return (s.len - s.origin() + kTileTokens - 1) / kTileTokens;
}

template <int kTileTokens>
__device__ __forceinline__ void advance(Cursor& c, const AttnParams& p)
{
    if (++c.tile < c.tiles) return;
    c.tile = 0;
    if (++c.item < p.h_kv * p.head_items) return;
    c.item = 0;
    do {
        if (++c.i >= p.n) return;     // past the last tile: the caller stops by its count
        c.span = span_of(p, c.i);
        c.tiles = tiles_of<kTileTokens>(c.span);
    } while (c.tiles == 0);
}

template <int D, int kHeadTiles>
struct Cfg {
    static constexpr int kWarps = D == 256 ? 2 : 4;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kHeads = 8 * kHeadTiles;
    // a slice is 8 KB at least: for short rows the look-up, the maxima and the loop cost as much as
    // the products (37 sequences with a window of 1000 tokens, 12 key heads of 64: 30.6 us, 39.3 us
    // with 16-token slices; more blocks an SM with fewer or smaller stages were no faster)
    static constexpr int kSubs = D == 64 ? 2 : 1;
    // the weights' lower pieces have sums of their own: with one head tile of 256, where they take
    // turns with the first piece's (bfloat16, 200001 tokens: 75.1 us, 77.9 in one sum; other shapes
    // no gain), and for float16, whose lower pieces' sums are cleared of infinities (37 windows of
    // 1000 tokens, 12 key heads of 64: 28.5 us, 27.9 without that)
    template <typename T>
    static constexpr int kSums =
        (D == 256 && kHeadTiles == 1) || std::is_same<T, __half>::value ? 2 : 1;
    static constexpr int kResident = 2;                       // blocks of an SM
    static constexpr int kSlice = kSubs * kSub;               // tokens of a warp's slice
    static constexpr int kTile = kWarps * kSlice;
    static constexpr int kStageBytes = 2 * kSlice * D * 2;    // keys, then values
    static constexpr int kMergeRow = D + 4;                   // floats; the pad spreads the banks
    static constexpr int kMergeBytes = kWarps * kHeads * kMergeRow * 4;
    static constexpr int kSmallBytes = 2 * kWarps * kHeads * 4 + 256;
    // the queries stay in registers, but for the one shape whose sums leave no room for them
    static constexpr bool kQueriesShared = D == 256 && kHeadTiles == 2;
    static constexpr int kQueryRow = D + 8;                   // elements
    static constexpr int kQueryBytes = kQueriesShared ? kHeads * kQueryRow * 2 : 0;
    // (the blocks share an SM's 228 KB, of which the system takes 1 KB a block)
    static constexpr int kRoom =
        233472 / kResident - 1024 - kMergeBytes - kSmallBytes - kQueryBytes;
    static constexpr int kStages = kRoom / (kWarps * kStageBytes);
    static constexpr int kSmem = kWarps * kStages * kStageBytes + kMergeBytes + kSmallBytes +
                                 kQueryBytes;
    static_assert(kStages >= 2, "no room for two stages");
};

// kCluster: one cluster an item, for few items of few tiles.
template <typename T, int D, int kHeadTiles, bool kCluster>
__global__ void __launch_bounds__(Cfg<D, kHeadTiles>::kThreads, Cfg<D, kHeadTiles>::kResident)
    paged_attention_kernel(const AttnParams p)
{
    using C = Cfg<D, kHeadTiles>;
    constexpr int kHeads = C::kHeads, kWarps = C::kWarps, kTile = C::kTile;
    constexpr int kSlice = C::kSlice, kSubs = C::kSubs;
    constexpr int kChunks = D / 8;                 // 16-byte pieces of a row
    constexpr int kRowsPerCopy = 32 / kChunks;     // rows that one cp.async of the warp covers
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* ring = smem;
    float* merge = reinterpret_cast<float*>(smem + kWarps * C::kStages * C::kStageBytes);
    float* sm_m = merge + C::kMergeBytes / 4;      // [kWarps][kHeads]
    float* sm_l = sm_m + kWarps * kHeads;
    int* sm_i = reinterpret_cast<int*>(sm_l + kWarps * kHeads);   // 64 words
    uint16_t* sm_q = reinterpret_cast<uint16_t*>(sm_i + 64);      // [kHeads][kQueryRow]

    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int c = blockIdx.x;
    const int items_per_seq = p.h_kv * p.head_items;

    dep_launch();
    dep_wait();

    Cursor cur;
    int t0, t1, total = 0, blocks = 0;             // the block's tiles, of how many in how many blocks
    if constexpr (kCluster) {
        // ---- the block's range: its share of its cluster's item, whose tiles are numbered from 0
        const int ranks = cluster_size(), item = c / ranks;
        cur.i = item / items_per_seq;
        cur.item = item % items_per_seq;
        cur.span = span_of(p, cur.i);
        cur.tiles = tiles_of<kTile>(cur.span);
        if (cur.item == 0 && c % ranks == 0 && tid == 0 && p.lens[cur.i] != cur.span.len)
            atomicOr(p.status, DECODE_BAD_LENGTH);
        const int each = (cur.tiles + ranks - 1) / ranks;
        t0 = cur.tile = min(c % ranks * each, cur.tiles);
        t1 = min(t0 + each, cur.tiles);
        if (cur.tiles == 0) {                      // for all of the cluster's blocks
            if (c % ranks == 0) {
                const int h0 = cur.item / p.head_items * p.group + cur.item % p.head_items * kHeads;
                const int heads = min(kHeads, p.group - cur.item % p.head_items * kHeads);
                const int64_t row = static_cast<int64_t>(cur.i) * p.h_q + h0;
                for (int x = tid; x < heads * (D / 8); x += C::kThreads)
                    reinterpret_cast<uint4*>(p.o + row * D)[x] = make_uint4(0, 0, 0, 0);
                if (p.lse != nullptr && tid < heads) p.lse[row + tid] = -INFINITY;
            }
            return;
        }
        // the block's maxima and sums, for its cluster (a block may have no tile)
        if (tid < 2 * kHeads)
            reinterpret_cast<float*>(sm_i)[tid] = tid < kHeads ? -INFINITY : 0.f;
        __syncthreads();
    } else {
        // ---- the block's range: a scan of all sequences' tiles
        const int chunk = (p.n + C::kThreads - 1) / C::kThreads;
        const int i_lo = min(p.n, tid * chunk), i_hi = min(p.n, i_lo + chunk);
        int mine = 0;
        for (int i = i_lo; i < i_hi; ++i) mine += tiles_of<kTile>(span_of(p, i)) * items_per_seq;
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
            if (x == w) upto += total;
            total += sm_i[x];
        }
        blocks = min(static_cast<int>(gridDim.x), total);   // with a tile each at least
        t0 = c < blocks ? first_tile(c, total, blocks) : total;
        t1 = c < blocks ? first_tile(c + 1, total, blocks) : total;
        if (t0 >= upto - mine && t0 < upto) {          // one thread: its sequences hold tile t0
            int at = upto - mine;
            for (int i = i_lo; i < i_hi; ++i) {
                const int tiles = tiles_of<kTile>(span_of(p, i)) * items_per_seq;
                if (t0 < at + tiles) {
                    sm_i[32] = i;
                    sm_i[33] = t0 - at;
                    break;
                }
                at += tiles;
            }
        }
        // sequences without tokens have no tile: their results are written here
        for (int i = c; i < p.n; i += gridDim.x) {
            const int raw = p.lens[i];
            const Span s = span_of(p, i);
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
        if (t0 >= t1) return;
        __syncthreads();
        cur.i = sm_i[32];
        cur.span = span_of(p, cur.i);
        cur.tiles = tiles_of<kTile>(cur.span);
        cur.item = sm_i[33] / cur.tiles;
        cur.tile = sm_i[33] % cur.tiles;
    }
    Cursor pre = cur;                              // where the loads are
    int pre_t = t0;

    // ---- loads of a slice.  The places in the cache of its 16-token pieces are looked up one slice
    // ahead: that of the first row where pages are multiples of 16 tokens, else that of row
    // `lane & 15`.
    const uint32_t ring0 = smem_addr(ring) + w * C::kStages * C::kStageBytes;
    const int ch = lane % kChunks, sub = lane / kChunks;
    const bool whole_pages = p.page_size % kSub == 0;
    const int ahead = whole_pages ? 0 : lane & 15;
    int page[kSubs], off[kSubs];
    bool there[kSubs];                             // the place is one of the sequence's
    auto look_up = [&]() {
#pragma unroll
        for (int y = 0; y < kSubs; ++y) {
            there[y] = false;
            if (pre_t >= t1) continue;
            const int pos = pre.span.origin() + pre.tile * kTile + w * kSlice + y * kSub + ahead;
            if (pos >= pre.span.len || (!whole_pages && pos < pre.span.start)) continue;
            there[y] = true;
            const int x = p.page_shift >= 0
                              ? pos >> p.page_shift
                              : static_cast<int>(static_cast<uint32_t>(pos) /
                                                 static_cast<uint32_t>(p.page_size));
            off[y] = pos - x * p.page_size;
            page[y] = p.table[pre.i * p.table_stride + x];
        }
    };
    auto load = [&](int stage) {
        if (pre_t < t1) {
            const int kv = pre.item / p.head_items;
            const uint16_t* k0 = p.k + kv * p.k_stride[2] + ch * 8;
            const uint16_t* v0 = p.v + kv * p.v_stride[2] + ch * 8;
#pragma unroll
            for (int y = 0; y < kSubs; ++y) {
                if (there[y] && (page[y] < 0 || page[y] >= p.pages)) {
                    atomicOr(p.status, DECODE_BAD_PAGE);
                    there[y] = false;
                }
                const int64_t ko = !there[y] ? 0 : page[y] * p.k_stride[0] + off[y] * p.k_stride[1];
                const int64_t vo = !there[y] ? 0 : page[y] * p.v_stride[0] + off[y] * p.v_stride[1];
                const uint32_t dst0 =
                    ring0 + stage * C::kStageBytes + (y * kSub + sub) * (D * 2);
                const int pos0 = pre.span.origin() + pre.tile * kTile + w * kSlice + y * kSub;
                // rows [lo, hi) of the 16 are read
                const int lo = pre.span.start - pos0;
                const int hi = whole_pages && !there[y] ? 0 : pre.span.len - pos0;
                if (whole_pages) {
                    const uint16_t* kb = k0 + ko + sub * p.k_stride[1];
                    const uint16_t* vb = v0 + vo + sub * p.v_stride[1];
                    const int64_t ks = kRowsPerCopy * p.k_stride[1], vs = kRowsPerCopy * p.v_stride[1];
#pragma unroll
                    for (int x = 0; x < kSub / kRowsPerCopy; ++x) {
                        const int row = x * kRowsPerCopy + sub;
                        const uint32_t bytes = row >= lo && row < hi ? 16u : 0u;
                        const uint32_t dst =
                            dst0 + x * kRowsPerCopy * (D * 2) + ((ch ^ (row & 7)) << 4);
                        cp_async16(dst, bytes ? kb : p.k, bytes);
                        cp_async16(dst + kSlice * D * 2, bytes ? vb : p.v, bytes);
                        kb += ks;
                        vb += vs;
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < kSub / kRowsPerCopy; ++x) {
                        const int row = x * kRowsPerCopy + sub;
                        const int64_t k1 = __shfl_sync(0xffffffffu, ko, row);
                        const int64_t v1 = __shfl_sync(0xffffffffu, vo, row);
                        const bool have = __shfl_sync(0xffffffffu, there[y], row);
                        const uint32_t bytes = have && row >= lo && row < hi ? 16u : 0u;
                        const uint32_t dst =
                            dst0 + x * kRowsPerCopy * (D * 2) + ((ch ^ (row & 7)) << 4);
                        cp_async16(dst, k0 + k1, bytes);
                        cp_async16(dst + kSlice * D * 2, v0 + v1, bytes);
                    }
                }
            }
            ++pre_t;
            if constexpr (kCluster)
                ++pre.tile;
            else
                advance<kTile>(pre, p);
        }
        cp_commit();
        look_up();
    };
    look_up();
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) load(s);

    // ---- the tiles
    const int hq = (lane & 3) * 2;                 // the lane's two heads (of each head tile)
    uint32_t qf[kHeadTiles][C::kQueriesShared ? 1 : D / 16][2];
    float acc[kHeadTiles][D / 16][4];
    float m[kHeadTiles][2], l[kHeadTiles][2];
    bool fresh = true;
    int stage = 0;
    // the queries of an item (their loads are on their way while the item before is joined)
    auto load_queries = [&](const Cursor& of) {
        const int kv = of.item / p.head_items;
        const int first = of.item % p.head_items * kHeads, heads = min(kHeads, p.group - first);
        const uint16_t* q0 = p.q + of.i * p.q_stride[0] + (kv * p.group + first) * p.q_stride[1] +
                             (lane & 3) * 2;
#pragma unroll
        for (int x = 0; x < kHeadTiles; ++x) {
            const int h = x * 8 + (lane >> 2);
            const uint16_t* row = q0 + h * p.q_stride[1];
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                qf[x][d][0] = h < heads ? *reinterpret_cast<const uint32_t*>(row + d * 16) : 0u;
                qf[x][d][1] = h < heads ? *reinterpret_cast<const uint32_t*>(row + d * 16 + 8) : 0u;
            }
        }
    };
    if constexpr (!C::kQueriesShared) load_queries(cur);
    for (int t = t0; t < t1; ++t) {
        const int kv = cur.item / p.head_items, h0 = kv * p.group + (cur.item % p.head_items) * kHeads;
        const int heads = min(kHeads, (kv + 1) * p.group - h0);
        if (fresh) {
            fresh = false;
            if constexpr (C::kQueriesShared) {
                // (every warp has passed the barrier that ends the item before)
                for (int x = tid; x < kHeads * kChunks; x += C::kThreads) {
                    const int h = x / kChunks, d = x % kChunks * 8;
                    uint4 b = make_uint4(0u, 0u, 0u, 0u);
                    if (h < heads)
                        b = *reinterpret_cast<const uint4*>(p.q + cur.i * p.q_stride[0] +
                                                            (h0 + h) * p.q_stride[1] + d);
                    *reinterpret_cast<uint4*>(sm_q + h * C::kQueryRow + d) = b;
                }
                __syncthreads();
            }
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

        const int pos0 = cur.span.origin() + cur.tile * kTile + w * kSlice;
        if (pos0 < cur.span.len) {
            const uint32_t ks = ring0 + stage * C::kStageBytes, vs = ks + kSlice * D * 2;
            float s[kHeadTiles][kSubs][4];
#pragma unroll
            for (int x = 0; x < kHeadTiles; ++x)
#pragma unroll
                for (int y = 0; y < kSubs; ++y)
                    s[x][y][0] = s[x][y][1] = s[x][y][2] = s[x][y][3] = 0.f;
            const int r = lane & 7, sel = lane >> 3;
            [[maybe_unused]] uint32_t qs[kHeadTiles][4];
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                if constexpr (C::kQueriesShared) {
                    if (d % 2 == 0) {
#pragma unroll
                        for (int x = 0; x < kHeadTiles; ++x)
                            ldsm4(qs[x], smem_addr(sm_q) + (x * 8 + r) * (C::kQueryRow * 2) +
                                             (2 * d + sel) * 16);
                    }
                }
#pragma unroll
                for (int y = 0; y < kSubs; ++y) {
                    uint32_t a[4];
                    ldsm4(a, ks + (y * kSub + (sel & 1) * 8 + r) * (D * 2) +
                                 (((2 * d + (sel >> 1)) ^ r) << 4));
#pragma unroll
                    for (int x = 0; x < kHeadTiles; ++x) {
                        if constexpr (C::kQueriesShared)
                            mma<T>(s[x][y], a, qs[x][d % 2 * 2], qs[x][d % 2 * 2 + 1]);
                        else
                            mma<T>(s[x][y], a, qf[x][d][0], qf[x][d][1]);
                    }
                }
            }
            // the lane's tokens are pos0 + 8 j + lane / 4
            bool in[2 * kSubs];
#pragma unroll
            for (int j = 0; j < 2 * kSubs; ++j) {
                const int pos = pos0 + j * 8 + (lane >> 2);
                in[j] = pos >= cur.span.start && pos < cur.span.len;
            }
            uint32_t pb[kHeadTiles][kSubs][kPieces<T>][2];   // [piece][tokens 0 .. 7, 8 .. 15]
            float corr[kHeadTiles][2];
#pragma unroll
            for (int x = 0; x < kHeadTiles; ++x) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 2 * kSubs; ++j) {
                        float& v = s[x][j / 2][j % 2 * 2 + e];
                        v = in[j] ? v * p.scale_log2 : -INFINITY;
                        top = fmaxf(top, v);
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    top = fmaxf(top, m[x][e]);
                    // scores of -infinity only: any finite reference leaves their weights 0
                    const float ref = top == -INFINITY ? 0.f : top;
                    corr[x][e] = exp2_fast(m[x][e] - ref);
                    m[x][e] = top;
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < 2 * kSubs; ++j) {
                        float& v = s[x][j / 2][j % 2 * 2 + e];
                        v = exp2_fast(v - ref);
                        sum += v;
                    }
                    l[x][e] = fmaf(l[x][e], corr[x][e], sum);
                }
#pragma unroll
                for (int j = 0; j < 2 * kSubs; ++j) {
                    float v0 = s[x][j / 2][j % 2 * 2] * kWeight<T>;
                    float v1 = s[x][j / 2][j % 2 * 2 + 1] * kWeight<T>;
#pragma unroll
                    for (int c = 0; c < kPieces<T>; ++c)
                        pb[x][j / 2][c][j % 2] = transpose8x8(take_piece<T>(v0, v1, c));
                }
            }
            // The slice's products are summed on their own and added to the rescaled sums: a matrix
            // product cuts its sum's last bits off, and over a long axis on one running sum the
            // losses add up (one sequence of 200001 tokens: 27 of 12288 results rounded otherwise
            // than the formula's in 64 bits, 16 since; 74.6 us then, 75.6 since)
            constexpr int kAtOnce = 2;             // blocks of 16 elements whose sums take turns
#pragma unroll
            for (int d0 = 0; d0 < D / 16; d0 += kAtOnce) {
                float o[kAtOnce][kHeadTiles][C::template kSums<T>][4] = {};
#pragma unroll
                for (int y = 0; y < kSubs; ++y) {
                    uint32_t a[kAtOnce][4];
#pragma unroll
                    for (int z = 0; z < kAtOnce; ++z)
                        ldsm4_trans(a[z], vs + (y * kSub + (sel >> 1) * 8 + r) * (D * 2) +
                                              (((2 * (d0 + z) + (sel & 1)) ^ r) << 4));
#pragma unroll
                    for (int c = 0; c < kPieces<T>; ++c)
#pragma unroll
                        for (int z = 0; z < kAtOnce; ++z)
#pragma unroll
                            for (int x = 0; x < kHeadTiles; ++x)
                                mma<T>(o[z][x][c > 0 ? C::template kSums<T> - 1 : 0], a[z], pb[x][y][c][0],
                                       pb[x][y][c][1]);
                }
#pragma unroll
                for (int z = 0; z < kAtOnce; ++z)
#pragma unroll
                    for (int x = 0; x < kHeadTiles; ++x)
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            float* const sum = acc[x][d0 + z] + e;
                            float2 add = make_float2(o[z][x][0][e], o[z][x][0][e + 1]);
                            if constexpr (std::is_same<T, __half>::value) {
                                add.x += finite(o[z][x][1][e]), add.y += finite(o[z][x][1][e + 1]);
                            } else if constexpr (C::template kSums<T> == 2) {
                                add.x += o[z][x][1][e], add.y += o[z][x][1][e + 1];
                            }
                            const float2 f = halves(fma2(pair(sum[0], sum[1]),
                                                         pair(corr[x][0], corr[x][1]),
                                                         pair(add.x, add.y)));
                            sum[0] = f.x, sum[1] = f.y;
                        }
            }
        }
        stage = stage + 1 == C::kStages ? 0 : stage + 1;

        // ---- the item's end, or the range's: join the warps
        const bool item_ends = cur.tile + 1 == cur.tiles;
        Cursor next = cur;
        if (!kCluster && t + 1 < t1) advance<kTile>(next, p);
        if constexpr (!kCluster && !C::kQueriesShared)
            if (item_ends && t + 1 < t1) load_queries(next);
        if (item_ends || t + 1 == t1) {
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
                    float* to = merge + (w * kHeads + h) * C::kMergeRow + (lane >> 2);
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        to[d * 16] = acc[x][d][e] * f;
                        to[d * 16 + 8] = acc[x][d][2 + e] * f;
                    }
                }
            __syncthreads();
            const int begin = t - cur.tile;                   // the item's tiles [begin, end)
            const int end = begin + cur.tiles;
            const bool whole = begin >= t0 && end <= t1;
            const int slot = 2 * c + (begin >= t0 ? 1 : 0);
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
                        merge + (y * kHeads + h) * C::kMergeRow + d);
                    o.x += b.x, o.y += b.y, o.z += b.z, o.w += b.w;
                }
                if constexpr (kCluster) {
                    // (each element of the first warp's rows is read by this thread alone)
                    *reinterpret_cast<float4*>(merge + h * C::kMergeRow + d) = o;
                    if (d == 0) {
                        reinterpret_cast<float*>(sm_i)[h] = top;
                        reinterpret_cast<float*>(sm_i)[kHeads + h] = sum;
                    }
                } else if (whole) {
                    const int64_t row = static_cast<int64_t>(cur.i) * p.h_q + h0 + h;
                    const float inv = factor_of<T>(sum);
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
            if (!kCluster && tid == 0 && begin >= t0 && (p.by_item || !whole))
                p.split[p.by_item ? cur.i * items_per_seq + cur.item : c] = make_int4(
                    whole ? -1 : c, whole ? 0 : block_of(end - 1, total, blocks), cur.i, cur.item);
            __syncthreads();
            fresh = true;
        }
        if (!kCluster)
            cur = next;
        else if (t + 1 < t1)
            ++cur.tile;
    }
    if constexpr (kCluster) {
        // ---- join the cluster's blocks, each an equal share of the elements
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
                    cluster_address(smem_addr(merge + h * C::kMergeRow + d), y));
                sum = fmaf(cluster_load(cluster_address(smem_addr(sm_i + kHeads + h), y)), f, sum);
                o.x = fmaf(b.x, f, o.x), o.y = fmaf(b.y, f, o.y);
                o.z = fmaf(b.z, f, o.z), o.w = fmaf(b.w, f, o.w);
            }
            const int64_t row = static_cast<int64_t>(cur.i) * p.h_q + h0 + h;
            const float inv = factor_of<T>(sum);
            *reinterpret_cast<uint2*>(p.o + row * D + d) = make_uint2(
                result<T>(o.x, o.y, inv), result<T>(o.z, o.w, inv));
            if (d == 0 && p.lse != nullptr)
                p.lse[row] = (top + log2f(sum)) * 0.6931471805599453f;
        }
        cluster_barrier();                         // the others may still read this block's part
    }
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

template <typename T, int D, int kHeadTiles>
__global__ void __launch_bounds__(kJoinWarps * 32, 1) paged_attention_join_kernel(const AttnParams p)
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
        const float inv = factor_of<T>(sums.sum);
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
Layout layout_for(int sms, int heads, int64_t d)
{
    const size_t blocks = static_cast<size_t>(sms) * kMostResident;
    Layout l{};
    size_t at = sizeof(int4) * (blocks > kListedItems ? blocks : kListedItems);
    l.ml = at = (at + 255) & ~size_t(255);
    at += sizeof(float2) * 2 * blocks * heads;
    l.o = at = (at + 255) & ~size_t(255);
    l.total = at + sizeof(float) * 2 * blocks * heads * static_cast<size_t>(d);
    return l;
}

int heads_of(int64_t group) { return group > 8 ? 16 : 8; }

template <typename T, int D, int kHeadTiles>
int run(AttnParams p, int64_t most_tokens, int sms, cudaStream_t stream)
{
    using C = Cfg<D, kHeadTiles>;
    const int64_t per_item = (most_tokens + C::kTile - 1) / C::kTile;
    const int64_t items = static_cast<int64_t>(p.n) * p.h_kv * p.head_items;
    if (per_item > 0 && items >= (int64_t(1) << 31) / per_item)
        return fail(DECODE_ERR_UNSUPPORTED, "too many tiles of the cache for one call");
    const int64_t tiles = per_item * items;
    const int64_t most = static_cast<int64_t>(sms) * C::kResident;
    const int blocks = static_cast<int>(tiles < 1 ? 1 : tiles < most ? tiles : most);
    p.by_item = items <= kListedItems;
    p.join_shared = items <= kSharedItems;
    // Few items of few tiles: a cluster an item, which joins its blocks' parts itself, as large as
    // the GPU holds for all items, up to three tiles a block (8 key heads: one sequence of 500
    // tokens 5.7 us, 8.1 with the second kernel; 16 of up to 250 tokens 7.2 and 8.6; one of 1500
    // 7.5 and 8.8; with four tiles a block, one of 2000 took as long either way).  The lengths being on the device, the page table's width
    // stands for the longest (with a window, the window): short sequences under a table made for
    // long ones take the second kernel.
    int ranks = 1;
    while (ranks < kClusterMost && ranks < per_item && items * ranks * 2 <= most) ranks *= 2;
    const bool cluster = ranks > 1 && per_item <= ranks * kClusterTiles;
    auto* kernel = cluster ? paged_attention_kernel<T, D, kHeadTiles, true>
                           : paged_attention_kernel<T, D, kHeadTiles, false>;
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
        return fail(DECODE_ERR_CUDA, "paged_attention_kernel: %s", cudaGetErrorString(e));
    if (cluster || per_item <= 1 || blocks == 1) return DECODE_OK;     // no item is cut
    const int64_t most_parts = per_item < blocks ? per_item : blocks;
    // (blocks of 16 warps need an SM each)
    const int64_t heads = !p.join_shared ? 1 : p.group < C::kHeads ? p.group : C::kHeads;
    const bool wide = p.join_shared && most_parts > 64 && items * heads <= sms;
    e = launch(paged_attention_join_kernel<T, D, kHeadTiles>,
               dim3(p.by_item ? static_cast<uint32_t>(items) : blocks, static_cast<uint32_t>(heads)),
               dim3((wide ? kJoinWarps : 8) * 32), 0, stream, p);
    if (e != cudaSuccess)
        return fail(DECODE_ERR_CUDA, "paged_attention_join_kernel: %s", cudaGetErrorString(e));
    return DECODE_OK;
}

template <typename T>
int dispatch(const AttnParams& p, int64_t d, int64_t most, int sms, cudaStream_t s)
{
    const bool two = p.group > 8;
    if (d == 64) return two ? run<T, 64, 2>(p, most, sms, s) : run<T, 64, 1>(p, most, sms, s);
    if (d == 128) return two ? run<T, 128, 2>(p, most, sms, s) : run<T, 128, 1>(p, most, sms, s);
    return two ? run<T, 256, 2>(p, most, sms, s) : run<T, 256, 1>(p, most, sms, s);
}

int check_heads(int64_t h_q, int64_t h_kv, int64_t d)
{
    if (h_q <= 0 || h_kv <= 0 || h_q % h_kv != 0)
        return fail(DECODE_ERR_INVALID_ARG, "%lld query heads over %lld key heads", (long long)h_q,
                    (long long)h_kv);
    if (d != 64 && d != 128 && d != 256)
        return fail(DECODE_ERR_UNSUPPORTED, "head_dim %lld (64, 128 or 256)", (long long)d);
    return DECODE_OK;
}

}  // namespace

extern "C" {

int decode_paged_attention_workspace_bytes(int64_t h_q, int64_t h_kv, int64_t head_dim,
                                           size_t* bytes)
{
    clear_error();
    if (bytes == nullptr) return fail(DECODE_ERR_INVALID_ARG, "bytes is null");
    const int rc = check_heads(h_q, h_kv, head_dim);
    if (rc != DECODE_OK) return rc;
    const int sms = sm_count();
    if (sms == 0) return DECODE_ERR_CUDA;
    *bytes = layout_for(sms, heads_of(h_q / h_kv), head_dim).total;
    return DECODE_OK;
}

int decode_paged_attention(const decode_paged_attention_args* a, cudaStream_t stream)
{
    clear_error();
    if (a == nullptr) return fail(DECODE_ERR_INVALID_ARG, "args is null");
    if (a->n < 0 || a->pages < 0 || a->page_size <= 0 || a->table_width < 0 || a->window < 0)
        return fail(DECODE_ERR_INVALID_ARG, "negative size or no page size");
    if (a->dtype != DECODE_F16 && a->dtype != DECODE_BF16)
        return fail(DECODE_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
    int rc = check_heads(a->h_q, a->h_kv, a->head_dim);
    if (rc != DECODE_OK) return rc;
    if (a->n == 0) return DECODE_OK;
    if (!a->q || !a->o || !a->lens || !a->workspace ||
        (a->table_width > 0 && a->pages > 0 && (!a->k_cache || !a->v_cache || !a->page_table)))
        return fail(DECODE_ERR_INVALID_ARG, "null pointer");
    if (misaligned(a->q) || misaligned(a->k_cache) || misaligned(a->v_cache) || misaligned(a->o) ||
        misaligned(a->workspace))
        return fail(DECODE_ERR_UNSUPPORTED, "16-bit tensors and workspace must be 16-byte aligned");
    AttnParams p{};
    if (!take_strides(p.q_stride, a->q_stride, {a->n, a->h_q}, 8))
        return fail(DECODE_ERR_UNSUPPORTED, "strides must be multiples of 8");
    const int64_t cs[3] = {a->pages, a->page_size, a->h_kv};
    if (!take_strides(p.k_stride, a->k_stride, cs, 8) ||
        !take_strides(p.v_stride, a->v_stride, cs, 8))
        return fail(DECODE_ERR_UNSUPPORTED, "cache strides must be multiples of 8");
    constexpr int64_t kMost = (int64_t(1) << 31) - 1;
    if (a->n > kMost || a->h_q >= (1 << 20) || a->pages > kMost || a->page_size > kMost ||
        a->table_width > kMost)
        return fail(DECODE_ERR_UNSUPPORTED, "problem too large for one call");
    const int sms = sm_count();
    if (sms == 0) return DECODE_ERR_CUDA;
    const int64_t group = a->h_q / a->h_kv;
    const int heads = heads_of(group);
    const Layout l = layout_for(sms, heads, a->head_dim);
    if (a->workspace_bytes < 0 || static_cast<size_t>(a->workspace_bytes) < l.total)
        return fail(DECODE_ERR_INVALID_ARG, "workspace of %zu bytes needed", l.total);
    // (an item's queries are in registers or shared memory, in all of its blocks, before its results
    // are written)
    const int64_t d = a->head_dim, sizes[2] = {a->n, a->h_q}, dense[2] = {a->h_q * d, d};
    const int shared = refuse_shared(
        {{"o", a->o, 2, d, sizes, dense, "q"},
         {"lse", a->lse, 4, a->n * a->h_q},
         {"workspace", a->workspace, 1, static_cast<int64_t>(l.total)}},
        {{"q", a->q, 2, d, sizes, p.q_stride},
         {"k_cache", a->k_cache, 2, d, cs, p.k_stride},
         {"v_cache", a->v_cache, 2, d, cs, p.v_stride},
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
    p.k = static_cast<const uint16_t*>(a->k_cache);
    p.v = static_cast<const uint16_t*>(a->v_cache);
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
    p.page_shift = -1;                // no power of two
    for (int x = 0; x < 31; ++x)
        if (p.page_size == 1 << x) p.page_shift = x;
    p.window = a->window > kMost ? 0 : static_cast<int32_t>(a->window);
    p.scale_log2 = a->scale * 1.4426950408889634f;
    // tokens of a sequence's slices, the rounding of its window's start included
    const int64_t most = p.window > 0 && p.window < max_len - kSub ? p.window + kSub : max_len;
    return a->dtype == DECODE_BF16 ? dispatch<__nv_bfloat16>(p, a->head_dim, most, sms, stream)
                                   : dispatch<__half>(p, a->head_dim, most, sms, stream);
}

}  // extern "C"
