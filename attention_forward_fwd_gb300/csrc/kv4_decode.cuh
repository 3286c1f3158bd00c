// kv4_decode.cuh -- attention of a few query rows over the quantised cache
// (fa_kv4_attention for at most 32 query rows a K/V head: single tokens,
// drafted tokens; grouped heads share the K/V row, so the rows of a K/V head
// are its group's heads times the call's tokens).
//
// Per sequence, K/V head and tile of 8 NT query rows, over blocks of 32 keys:
//   S^T = K Q^T    (keys x rows)   m16n8k16, A = codes of K, B = Q^T
//   z = S scale log2 e; p = 2^(z - m)  with a running reference m
//   O^T += V^T P^T (D x rows)      m16n8k16, A = codes of V, B = scaled P^T
//
// What bounds it is DRAM: 1.125 D bytes a key and head against 4 D flops a
// query row.  At the measured 6.69 TB/s an SM has to take in about 40 codes a
// clock, so the unpacking is what has to be cheap:
//  * Keys are the M side of both products: one m16n8k16 eats 256 codes for 8
//    query rows (with the queries on the M side it would eat 128).
//  * Codes go to the tensor cores as fp16 integers: (x & mask | 0x6400) minus
//    1032 or 1152 is n - 8 or 16 (n - 8), exactly, two codes at a time; V's are
//    paired over two keys by a byte permutation, K's over two runs of 4 elements.
//    (Subnormals, n 2^-24 or n 2^-20 by a mask alone, would save the
//    subtraction; but the tensor cores align them by their exponent field, with up
//    to 10 bits of nothing in front: results off by 2^-14 of a code.  Taking
//    the offset 8 off the end result loses bits too: V's accumulator runs over
//    the whole context and would carry an offset many times the result.)
//  * Each group's part of a score is scaled by the key's fp32 scale as it is
//    added up, so nothing of K is rounded.
//  * The scale of V belongs to (key, group): it multiplies P, one fp16 matrix
//    operand for each group, turned from the accumulator's layout to the
//    operand's by movmatrix.
// P s is rounded to fp16 (2^-12): s is bounded by 2^E with a running E, kept
// so that p s 2^(kHead - E) stays in fp16's range with 11 bits down to
// 2^-21 of the largest.
//
// Work: the (sequence, K/V head, row tile) items' key blocks are numbered in a
// row and cut into equal ranges, one for each CTA (the lengths are on the
// device only, so the cut is made there).  An item that a cut goes through
// leaves partial results, which combine_kernel joins in the order of the keys.
// Within a CTA four warps cut the range again and work alone, each with a ring
// of its own that its lanes fill with 16-byte asynchronous copies (they run ahead
// over the ends of items; no barrier but the warp's).  Bulk copies by a fifth
// warp took more instructions: their operands are uniform, so that the lanes' copies
// went out one by one.  Items that lie inside a warp's range are written by it; the parts of the others
// (at most two a warp) are joined once, at the end of the CTA.  Sharing each
// item's blocks out to the warps in turn, with a join for each item, left
// the warps waiting for one another: batch of 64 ragged contexts, 84 us.
// Short contexts are not cut like that: an item has a cluster of 1 to 8 CTAs
// (at most kWholeBlocks blocks each), which join through one another's shared
// memory: one launch, no workspace, and no search for the range.
#pragma once

#include "kv4_cache.cuh"

namespace kv4 {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kBlock = 32;              // keys a block
constexpr float kLazy = 8.f;            // p may reach 2^kLazy before m moves
constexpr int kHead = 7;                // p s 2^(kHead - E) < 2^(kLazy + kHead) < 65504
constexpr int kWholeBlocks = 16;        // most blocks a CTA of an item that has a cluster of its own
constexpr int kMaxCluster = 8;
constexpr float kNegInf = -INFINITY;
constexpr uint32_t kMid = 0x00f000f0u;  // bits 4..7 of both halves

struct Attend {
    const void* q;
    long long q_batch, q_row, q_head;    // strides in elements (q_batch 0 when packed)
    void* o;                             // contiguous [rows, H, D]
    float* lse;                          // [B, H, S] or [H, total]; may be null
    long long lse_batch, lse_head;
    float scale;
    int H, G;                            // query heads, of a K/V head
    int window;                          // key j is seen from pos iff pos - window <= j <= pos; -1: no bound
    float* part_o;                       // [2 grid][8 NT][D]
    float2* part_ml;                     // [2 grid][8 NT]: reference and sum
    int grid;                            // CTAs of decode_kernel
    int whole;                           // nonzero: a cluster an item, of this many items a sequence
    int cluster;                         // its CTAs
};

template <int NG>
struct Tile {
    static constexpr int D = NG * kGroup;
    static constexpr int kCodes = kBlock * 16 * NG;        // bytes of K's (V's) codes in a block
    static constexpr int kScales = kBlock * 2 * NG;
    static constexpr int kStage = 2 * (kCodes + kScales);
    // As many blocks in flight as leave room for three CTAs an SM (D <= 128; two
    // above).  A warp then waits some 20 cycles a block for its copies (131072 keys,
    // D = 128); more stages took as long.
    static constexpr int kStages = NG <= 2 ? 6 : NG == 3 ? 4 : NG <= 6 ? 3 : 2;
    static constexpr int kRing = kWarps * kStages * kStage;
};

// A warp's part of an item that it does not hold whole: [8 NT][D + 4] sums
// (the last 4 only pad the rows off one another's banks).
template <int NG, int NT>
constexpr int kPartFloats = 8 * NT * (Tile<NG>::D + 4);

// The ring, a part for each warp (the second one, of its last item, goes into
// its own ring, which is empty by then), the rest.
// A cluster's CTAs have room for their joined sums besides.
template <int NG, int NT>
constexpr int kClusterSmem = 8 * NT * (Tile<NG>::D * 4 + 8);

template <int NG, int NT>
constexpr int kDecodeSmem = Tile<NG>::kRing + kWarps * kPartFloats<NG, NT> * 4 + 2048;

// The first key that a row at `pos` sees.  (pos is negative for rows in front of
// a sequence, and the window may be any int: their difference need not fit one.)
__device__ __forceinline__ int first_key(int pos, int window) { return window < 0 ? 0 : max(0, max(0, pos) - window); }

// The rows of the call for a sequence as items: tiles x heads, each of `blocks` key blocks from key `first`.
struct Work {
    int n, len, row0, tiles, items, blocks, first;
};

__device__ __forceinline__ Work work_of(const Cache& c, const Attend& a, int b, int tile_rows, bool tell) {
    const Seq s = sequence(c, b);
    if (tell && s.status != 0) report(s.status);
    Work w;
    w.n = s.n;
    w.len = s.len;
    w.row0 = s.row0;
    w.tiles = (s.n * a.G + tile_rows - 1) / tile_rows;
    w.items = w.tiles * c.Hkv;
    w.first = 0;
    if (s.n > 0) w.first = first_key(s.len - s.n, a.window) / kBlock * kBlock;
    w.blocks = s.n > 0 ? max(1, (max(0, s.len - w.first) + kBlock - 1) / kBlock) : 0;
    return w;
}

// The blocks of a call in a row: their number, and the sequence that holds
// block quota * blockIdx.x with the number of its first block.  By the whole
// CTA; each round takes blockDim.x sequences, and a second pass is made only
// when there are more than that.
struct Range {
    long long all, quota, at;
    int b;
};

__device__ __forceinline__ long long quota_of(long long all, int grid) {
    return max((all + grid - 1) / grid, static_cast<long long>(kWarps));
}

__device__ __forceinline__ Range find_range(const Cache& c, const Attend& a, int tile_rows, long long* sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    Range r;
    r.all = 0;
    r.quota = 0;
    for (int pass = 0; pass < 2; ++pass) {
        long long base = 0;
        for (int b0 = 0; b0 < c.B; b0 += blockDim.x) {
            const int b = b0 + threadIdx.x;
            long long mine = 0;
            if (b < c.B) {
                const Work w = work_of(c, a, b, tile_rows, pass == 0 && blockIdx.x == 0);
                mine = static_cast<long long>(w.items) * w.blocks;
            }
            long long x = mine;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, m);
                if (lane >= m) x += y;
            }
            __syncthreads();
            if (lane == 31) sh[warp] = x;
            __syncthreads();
            long long before = base, here = 0;
            for (int i = 0; i < nw; ++i) {
                if (i < warp) before += sh[i];
                here += sh[i];
            }
            const long long start = before + x - mine;
            base += here;
            const bool one = c.B <= static_cast<int>(blockDim.x);
            if (one) {
                r.all = base;
                r.quota = quota_of(base, a.grid);
            }
            if (one || pass == 1) {
                const long long lo = r.quota * blockIdx.x;
                if (mine > 0 && start <= lo && lo < start + mine) {
                    sh[14] = b;
                    sh[15] = start;
                }
            }
        }
        if (c.B <= static_cast<int>(blockDim.x)) break;
        r.all = base;
        r.quota = quota_of(base, a.grid);
    }
    __syncthreads();
    r.b = static_cast<int>(sh[14]);
    r.at = sh[15];
    return r;
}

// A warp's place in the row of blocks.
struct Cursor {
    int b, item, blk;
    Work w;
    __device__ __forceinline__ void settle(const Cache& c, const Attend& a, int tile_rows) {
        // blk counts on from the item's first block; move to the item that holds it
        while (blk >= w.blocks) {
            blk -= w.blocks;
            if (++item >= w.items) {
                item = 0;
                do {
                    ++b;
                    if (b >= c.B) {
                        w.blocks = 0x7fffffff;
                        return;
                    }
                    w = work_of(c, a, b, tile_rows, false);
                } while (w.items == 0);
            }
        }
    }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {   // all but the last N groups of this thread have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared memory `at` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t at, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    return r;
}
__device__ __forceinline__ float2 cluster_load2(uint32_t at) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The key of a tile of 16 that matrix row `r` (K) or the contraction's index
// `r` (V) stands for.  Swapping odd pairs makes the rows that the lanes of a
// quarter warp read lie in different halves of the shared-memory banks, for
// both products.
__device__ __forceinline__ int key_of(int r) { return r ^ ((r >> 1) & 1); }

// n - 8 of the codes in bits 0..3, and 16 (n - 8) of those in bits 4..7, of
// each half of u, in fp16: 1024 + x is 0x6400 | x.
__device__ __forceinline__ uint32_t half_sub(uint32_t y, uint32_t c) {
    const __half2 z = __hsub2(*reinterpret_cast<const __half2*>(&y), *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&z);
}
__device__ __forceinline__ uint32_t low_codes(uint32_t u) {
    return half_sub((u & 0x000f000fu) | 0x64006400u, 0x64086408u);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t u) {
    return half_sub((u & kMid) | 0x64006400u, 0x64806480u);
}

// Where share `i` of n starts among some blocks.
__device__ __forceinline__ int share(int blocks, int i, int n) {
    return static_cast<int>(static_cast<long long>(blocks) * i / n);
}

// A warp's copies: the blocks of its range one after the other, each in runs of
// 32 or 16 keys that lie together in a page.  A whole run is copied as soon
// as one of its keys belongs to the sequence.
template <int NG>
struct Copier {
    Cursor cur;
    int left;              // blocks not copied yet
    int head, item;
    int pg, off;           // the block's first key: index into the page table, place in the page
    int page[2];           // numbers of its pages; they are asked for a block ahead of their use

    __device__ __forceinline__ void look_up(const Cache& c) {
        page[0] = page[1] = -1;
        if (left <= 0) return;
        if (item != cur.item) {   // `copy` sets it to -1 where the sequence may have changed
            item = cur.item;
            head = item / cur.w.tiles;
        }
        const int key0 = cur.w.first + cur.blk * kBlock;
        const int* row = c.table + static_cast<long long>(cur.b) * c.max_pages;
        if (key0 < cur.w.len) page[0] = __ldg(row + pg);
        // (looking at page[0] here would wait for it)
        if (key0 + 16 < cur.w.len && off + 16 >= c.P) page[1] = __ldg(row + pg + 1);
    }
    // The place of the block at `cur`, from scratch.
    __device__ __forceinline__ void locate(const Cache& c) {
        const int key0 = cur.w.first + cur.blk * kBlock;
        pg = key0 / c.P;
        off = key0 - pg * c.P;
    }

    // Copies the block at `cur` to `st` and moves on; bit i of the result: the
    // i-th 16 keys are there.
    __device__ __forceinline__ uint32_t copy(const Cache& c, const Attend& a, int tile_rows, uint8_t* st) {
        uint32_t in = 0;
        if (left > 0) {
            const int lane = threadIdx.x & 31;
            const int key0 = cur.w.first + cur.blk * kBlock;
            const bool ask0 = key0 < cur.w.len, ask1 = key0 + 16 < cur.w.len;
            const bool ok0 = ask0 && static_cast<unsigned>(page[0]) < static_cast<unsigned>(c.pages);
            const int page1 = off + 16 < c.P ? page[0] : page[1];
            const bool ok1 = ask1 && static_cast<unsigned>(page1) < static_cast<unsigned>(c.pages);
            if (ask0 != ok0 || ask1 != ok1) report(kStatusBadPages);
            in = (ok0 ? 1u : 0u) | (ok1 ? 2u : 0u);
            const uint32_t dst = fa::ptx::smem_addr(st) + lane * 16;
            const long long v_off = static_cast<long long>(c.Hkv) * c.P;   // rows from K to V
            const long long row0 = (static_cast<long long>(ok0 ? page[0] : 0) * 2 * c.Hkv + head) * c.P + off;
            if (in == 3u && off + 16 < c.P) {
                // 32 keys that lie together: 32 NG chunks of 16 bytes of codes, 4 NG of scales
                const uint8_t* k = c.codes + row0 * (16 * NG) + lane * 16;
                const uint8_t* v = k + v_off * (16 * NG);
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    copy16(dst + i * 512, k + i * 512);
                    copy16(dst + Tile<NG>::kCodes + i * 512, v + i * 512);
                }
                const uint8_t* ks = reinterpret_cast<const uint8_t*>(c.scales + row0 * NG);
#pragma unroll
                for (int i = 0; i < (8 * NG + 31) / 32; ++i) {
                    const int q = i * 32 + lane;   // K's, then V's
                    if (8 * NG % 32 == 0 || q < 8 * NG)
                        copy16(dst + 2 * Tile<NG>::kCodes + i * 512,
                               ks + q * 16 + (q >= 4 * NG ? v_off * (2 * NG) - 64 * NG : 0));
                }
            } else if (in != 0) {
                const int off1 = off + 16 < c.P ? off + 16 : 0;
                const long long row1 = (static_cast<long long>(ok1 ? page1 : 0) * 2 * c.Hkv + head) * c.P + off1;
#pragma unroll 1
                for (int i = 0; i < NG; ++i) {
                    const int q = i * 32 + lane;
                    const bool second = q >= 16 * NG;
                    if ((in >> (second ? 1 : 0)) & 1u) {
                        const uint8_t* src = c.codes + (second ? row1 : row0) * (16 * NG) + (second ? q - 16 * NG : q) * 16;
                        copy16(dst + i * 512, src);
                        copy16(dst + Tile<NG>::kCodes + i * 512, src + v_off * (16 * NG));
                    }
                }
#pragma unroll 1
                for (int i = 0; i < (8 * NG + 31) / 32; ++i) {
                    const int q = i * 32 + lane, which = q >= 4 * NG ? 1 : 0, qq = q - which * 4 * NG;
                    const bool second = qq >= 2 * NG;
                    if (q < 8 * NG && ((in >> (second ? 1 : 0)) & 1u))
                        copy16(dst + 2 * Tile<NG>::kCodes + i * 512,
                               c.scales + ((second ? row1 : row0) + which * v_off) * NG + (second ? qq - 2 * NG : qq) * 8);
                }
            }
            --left;
            ++cur.blk;
            off += kBlock;
            while (off >= c.P) {
                off -= c.P;
                ++pg;
            }
            if (left > 0 && cur.blk >= cur.w.blocks) {
                cur.settle(c, a, tile_rows);
                item = -1;
                locate(c);
            }
        }
        copies_commit();
        look_up(c);
        return in;
    }
};

// What the warps of a CTA left to be joined, in the order of the blocks: part 0
// carries an item on, part 1 starts one and does not end it.
struct Part {
    int b, item;      // b = -1: none
    int ends;         // the item ends with it
};

// O and LSE of one row's four elements from sums in units of 2^m.
template <bool BF16>
__device__ __forceinline__ void write_row(const Cache& c, const Attend& a, const Work& w, int b, int D, int rho, int head,
                                          int d, float4 o, float m, float l, bool lse) {
    const int qi = rho / a.G, h = head * a.G + (rho - qi * a.G);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* dst = static_cast<uint16_t*>(a.o) + (static_cast<long long>(w.row0 + qi) * a.H + h) * D + d;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack16<BF16>(o.x * inv, o.y * inv), pack16<BF16>(o.z * inv, o.w * inv));
    if (lse)
        a.lse[(c.cu != nullptr ? w.row0 : b * a.lse_batch) + h * a.lse_head + qi] =
            l == 0.f ? kNegInf : (m + log2f(l)) * 0.6931471805599453f;
}

template <int NG, int NT, bool BF16>
__global__ void __launch_bounds__(kThreads, NG <= 4 && NT == 1 ? 3 : 2) decode_kernel(Cache c, Attend a) {
    constexpr int D = NG * kGroup, R = 8 * NT, kStage = Tile<NG>::kStage, kStages = Tile<NG>::kStages;
    static_assert(kPartFloats<NG, NT> * 4 <= kStages * kStage, "a part fits the ring");
    constexpr int kPart = kPartFloats<NG, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* ring = smem;
    float* join = reinterpret_cast<float*>(smem + Tile<NG>::kRing);                       // [warp] part 0
    uint8_t* tail = reinterpret_cast<uint8_t*>(join + kWarps * kPart);
    float2* join_ml = reinterpret_cast<float2*>(tail);                                    // [warp][part][R], 1024 bytes
    long long* scan = reinterpret_cast<long long*>(tail + 1024);                          // 16
    Part* parts = reinterpret_cast<Part*>(tail + 1152);                                   // [warp][part]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, cc = lane & 3;

    // ---- this CTA's blocks: `blocks` from block seg.blk of item seg.item of sequence seg.b on
    Cursor seg;
    int blocks;
    if (a.whole) {
        const int x = blockIdx.x / a.cluster, rank = blockIdx.x - x * a.cluster;
        seg.b = x / a.whole;
        seg.item = x - seg.b * a.whole;
        seg.w = work_of(c, a, seg.b, R, tid == 0 && seg.item == 0 && rank == 0);
        if (seg.item >= seg.w.items) return;   // the whole cluster
        seg.blk = share(seg.w.blocks, rank, a.cluster);
        blocks = share(seg.w.blocks, rank + 1, a.cluster) - seg.blk;
    } else {
        const Range range = find_range(c, a, R, scan);
        fa::ptx::launch_dependents();
        const long long lo = range.quota * blockIdx.x;
        if (lo >= range.all) return;
        blocks = static_cast<int>(min(range.all - lo, range.quota));
        seg.b = range.b;
        seg.w = work_of(c, a, seg.b, R, false);
        const int off = static_cast<int>(lo - range.at);   // blocks of one sequence are numbered with an int
        seg.item = off / seg.w.blocks;
        seg.blk = off - seg.item * seg.w.blocks;
    }
    uint8_t* my_ring = ring + warp * kStages * kStage;
    int x = share(blocks, warp, kWarps);                    // this warp's next block
    const int x_end = share(blocks, warp + 1, kWarps);
    if (lane < 2) parts[warp * 2 + lane].b = -1;
    __syncwarp();
    seg.blk += x;
    if (x < x_end) seg.settle(c, a, R);
    Copier<NG> copier;
    copier.cur = seg;
    copier.left = x_end - x;
    copier.head = 0;
    copier.item = -1;
    copier.locate(c);
    copier.look_up(c);
    uint32_t there[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) there[i] = copier.copy(c, a, R, my_ring + i * kStage);
    int stage = 0;
    const uint16_t* q16 = static_cast<const uint16_t*>(a.q);

    while (x < x_end) {
        // ---- one item, or the part of it that is this warp's
        const Work w = seg.w;
        const int seg_blocks = min(x_end - x, w.blocks - seg.blk);
        const int head = seg.item / w.tiles, tile = seg.item - head * w.tiles;
        const int rows = min(R, w.n * a.G - tile * R);

        // ---- Q: fp16 with each row's largest magnitude in [2^11, 2^12), the
        // elements that meet codes in bits 4..7 divided by 16
        uint32_t qf[NT][NG][4];
        float fac[NT][2];
        int hi_key[NT][2], lo_key[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = t * 8 + r;   // this lane's query row (B operand: n = lane / 4)
            uint4 raw[NG];
            if (row < rows) {
                const int rho = tile * R + row, i = rho / a.G, h = head * a.G + rho % a.G;
                const uint16_t* src = q16 + (c.cu != nullptr ? static_cast<long long>(w.row0 + i) * a.q_row
                                                             : seg.b * a.q_batch + i * a.q_row) + h * a.q_head;
#pragma unroll
                for (int g = 0; g < NG; ++g) raw[g] = __ldg(reinterpret_cast<const uint4*>(src + g * kGroup + cc * 8));
            } else {
#pragma unroll
                for (int g = 0; g < NG; ++g) raw[g] = make_uint4(0, 0, 0, 0);
            }
            float most = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint32_t u[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = to_f32x2<BF16>(u[j]);
                    most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            // 2^up brings `most` to [2^11, 2^12)
            int up = most > 0.f ? 138 - static_cast<int>((__float_as_uint(most) >> 23) & 255u) : 0;
            up = max(-90, min(100, up));
            const float mul = __uint_as_float(static_cast<uint32_t>(127 + up) << 23), mul16 = mul * 0.0625f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                // elements 8 cc + e: e = j and 4 + j pair up; j odd sits in bits 4..7
                const float2 e01 = to_f32x2<BF16>(raw[g].x), e23 = to_f32x2<BF16>(raw[g].y);
                const float2 e45 = to_f32x2<BF16>(raw[g].z), e67 = to_f32x2<BF16>(raw[g].w);
                qf[t][g][0] = pack16<false>(e01.x * mul, e45.x * mul);       // j = 0
                qf[t][g][1] = pack16<false>(e23.x * mul, e67.x * mul);       // j = 2
                qf[t][g][2] = pack16<false>(e01.y * mul16, e45.y * mul16);   // j = 1
                qf[t][g][3] = pack16<false>(e23.y * mul16, e67.y * mul16);   // j = 3
            }
            // z = S 2^-up scale log2 e
            const float f = fmaxf(a.scale * 1.4426950408889634f *
                                      __uint_as_float(static_cast<uint32_t>(127 - up) << 23), 1.17549435e-38f);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int from = (2 * cc + e) * 4;   // a lane that holds row 2 cc + e
                fac[t][e] = __shfl_sync(0xffffffffu, f, from);
                // rows past the tile's last one see everything; nobody reads what comes of them
                const int rr = t * 8 + 2 * cc + e;
                const int pos = w.len - w.n + (tile * R + rr) / a.G;
                hi_key[t][e] = rr < rows ? pos : 0x7fffffff;
                lo_key[t][e] = rr < rows ? first_key(pos, a.window) : 0;
            }
        }
        // keys that every row of the tile sees
        const int all_hi = w.len - w.n + tile * R / a.G;
        const int all_lo = first_key(w.len - w.n + (tile * R + rows - 1) / a.G, a.window);

        float acc[NT][NG][2][4];
        float thr[NT][2], neg_ref[NT][2], l_sum[NT][2];   // raw score that moves the reference; -(m - kHead + E)
        float m_ref[NT][2];
        int e_ref = -90;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m_ref[t][e] = thr[t][e] = kNegInf;
                neg_ref[t][e] = static_cast<float>(kHead + 90);
                l_sum[t][e] = 0.f;
            }
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[t][g][i >> 2][i & 3] = 0.f;
        }

        for (int blk = 0; blk < seg_blocks; ++blk) {
            const int key0 = w.first + (seg.blk + blk) * kBlock;
            copies_wait<kStages - 1>();
            __syncwarp();
            uint8_t* st = my_ring + stage * kStage;
            const uint32_t in = there[0];
            const bool edge = key0 + (kBlock - 1) > all_hi || key0 < all_lo || in != 3u;

            // ---- S^T = K Q^T for 2 x 16 keys
            float s[2][NT][4];
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                const int k0 = kt * 16 + key_of(r), k1 = k0 + 8;
                Words<2 * NG> c0, c1;
                c0.load(st + k0 * 16 * NG + cc * 4 * NG);
                c1.load(st + k1 * 16 * NG + cc * 4 * NG);
                Words<NG> s0, s1;
                s0.load(st + 2 * Tile<NG>::kCodes + k0 * 2 * NG);
                s1.load(st + 2 * Tile<NG>::kCodes + k1 * 2 * NG);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    // r = 2 cc below r = 2 cc + 1
                    const uint32_t x0 = join_words(c0, g, c0, NG + g), x1 = join_words(c1, g, c1, NG + g);
                    const uint32_t y0 = x0 >> 8, y1 = x1 >> 8;
                    const uint32_t a_even[4] = {low_codes(x0), low_codes(x1), low_codes(y0), low_codes(y1)};
                    const uint32_t a_odd[4] = {high_codes(x0), high_codes(x1), high_codes(y0), high_codes(y1)};
                    const float f0 = s0.bf16(g), f1 = s1.bf16(g);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float d[4] = {0.f, 0.f, 0.f, 0.f};
                        mma16816(d, a_even, qf[t][g][0], qf[t][g][1]);
                        mma16816(d, a_odd, qf[t][g][2], qf[t][g][3]);
                        s[kt][t][0] = g == 0 ? f0 * d[0] : fmaf(f0, d[0], s[kt][t][0]);
                        s[kt][t][1] = g == 0 ? f0 * d[1] : fmaf(f0, d[1], s[kt][t][1]);
                        s[kt][t][2] = g == 0 ? f1 * d[2] : fmaf(f1, d[2], s[kt][t][2]);
                        s[kt][t][3] = g == 0 ? f1 * d[3] : fmaf(f1, d[3], s[kt][t][3]);
                    }
                }
            }
            // V's scales
            Words<NG> sv[2][2];
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sv[kt][h].load(st + 2 * Tile<NG>::kCodes + Tile<NG>::kScales + (kt * 16 + h * 8 + key_of(r)) * 2 * NG);

            if (edge) {
                // Masked scores are -inf.  V's scales are zero where the key was
                // not copied or lies past the sequence (there may be anything
                // there, NaN included).
#pragma unroll
                for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int key = key0 + kt * 16 + h * 8 + key_of(r);
                        const bool have = (in >> kt) & 1u;
                        if (!(have && key < w.len)) sv[kt][h].clear();
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (!(have && key <= min(hi_key[t][e], w.len - 1) && key >= lo_key[t][e]))
                                    s[kt][t][h * 2 + e] = kNegInf;
                    }
            }

            // ---- whether a reference has to move: a score past thr, or a
            // scale of 2^E or more (or a NaN, whose bits are larger still)
            uint32_t big = 0;
#pragma unroll
            for (int i = 0; i < Words<NG>::kRegs; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) big = __vmaxu2(big, sv[k >> 1][k & 1].u[i] & 0x7fff7fffu);
            big = max(big & 0xffffu, big >> 16);
            bool grow = static_cast<int>(big >> 7) - 126 > e_ref;
            float top[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[t][e] = fmaxf(fa::ptx::fmax3(s[0][t][e], s[0][t][2 + e], s[1][t][e]), s[1][t][2 + e]);
                    grow |= top[t][e] > thr[t][e];
                }
            if (__any_sync(0xffffffffu, grow)) {
                // A NaN scale of V makes its group NaN for the rows that see
                // the key (whatever p is) and must not reach the others, whose
                // p = 0 it would multiply: it is taken out of the product here.
                if (__any_sync(0xffffffffu, big >= 0x7f80u)) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t hit = 0;   // groups
#pragma unroll
                            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
#pragma unroll
                                    for (int g = 0; g < NG; ++g)
                                        if ((sv[kt][h].get(g) & 0x7fffu) >= 0x7f80u && !(s[kt][t][h * 2 + e] == kNegInf))
                                            hit |= 1u << g;
                            hit |= __shfl_xor_sync(0xffffffffu, hit, 4);
                            hit |= __shfl_xor_sync(0xffffffffu, hit, 8);
                            hit |= __shfl_xor_sync(0xffffffffu, hit, 16);
#pragma unroll
                            for (int g = 0; g < NG; ++g)
                                if ((hit >> g) & 1u) {
                                    const float nan = __uint_as_float(0x7fc00000u);
                                    acc[t][g][0][e] = acc[t][g][0][2 + e] = nan;
                                    acc[t][g][1][e] = acc[t][g][1][2 + e] = nan;
                                }
                        }
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int g = 0; g < NG; ++g)
                                if ((sv[kt][h].get(g) & 0x7fffu) >= 0x7f80u) sv[kt][h].set(g, 0);
                }
                uint32_t fin = 0;   // the largest scale
#pragma unroll
                for (int i = 0; i < Words<NG>::kRegs; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) fin = __vmaxu2(fin, sv[k >> 1][k & 1].u[i] & 0x7fff7fffu);
                fin = __reduce_max_sync(0xffffffffu, max(fin & 0xffffu, fin >> 16));
                // s < 2^(exponent + 1); the bound moves by one more than it has to
                const int need = static_cast<int>(fin >> 7) - 126;
                const int e_new = need > e_ref ? min(need + 1, 128) : e_ref;
                const float de = fa::ptx::ex2_approx(static_cast<float>(e_ref - e_new));
                e_ref = e_new;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = top[t][e];
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float mn = fmaxf(m_ref[t][e], mx * fac[t][e]);
                        const float al = (mn == kNegInf ? 1.f : fa::ptx::ex2_approx(m_ref[t][e] - mn)) * de;
                        m_ref[t][e] = mn;
                        thr[t][e] = (mn + kLazy) / fac[t][e];
                        neg_ref[t][e] = static_cast<float>(kHead - e_ref) - (mn == kNegInf ? 0.f : mn);
                        l_sum[t][e] *= al;
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            acc[t][g][0][e] *= al;
                            acc[t][g][0][2 + e] *= al;
                            acc[t][g][1][e] *= al;
                            acc[t][g][1][2 + e] *= al;
                        }
                    }
            }

            // ---- p 2^(kHead - E)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float& z = s[k >> 1][t][(k & 1) * 2 + e];
                        z = fa::ptx::ex2_approx(fmaf(z, fac[t][e], neg_ref[t][e]));
                        l_sum[t][e] += z;
                    }

            // ---- O^T += V^T P^T
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                // contraction index 2 cc + e (+ 8): keys of this lane
                Words<NG> v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int kk = kt * 16 + (i >> 1) * 8 + key_of(2 * cc + (i & 1));
                    v[i].load(st + Tile<NG>::kCodes + kk * 16 * NG + r * 2 * NG);
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint32_t xa = join_words(v[0], g, v[1], g), xb = join_words(v[2], g, v[3], g);
                    const uint32_t a01[4] = {low_codes(xa), high_codes(xa), low_codes(xb), high_codes(xb)};
                    const uint32_t a23[4] = {low_codes(xa >> 8), high_codes(xa >> 8), low_codes(xb >> 8),
                                             high_codes(xb >> 8)};
                    const float f0 = sv[kt][0].bf16(g), f1 = sv[kt][1].bf16(g);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const float p0 = s[kt][t][0] * f0, p1 = s[kt][t][1] * f0;
                        const float p2 = s[kt][t][2] * f1, p3 = s[kt][t][3] * f1;
                        const uint32_t h0 = pack16<false>(p0, p1), h1 = pack16<false>(p2, p3);
                        const uint32_t b0 = transpose8x8(h0), b1 = transpose8x8(h1);
                        mma16816(acc[t][g][0], a01, b0, b1);
                        mma16816(acc[t][g][1], a23, b0, b1);
                        if constexpr (!BF16) {
                            // fp16 results are held to 2^-12: what P's rounding leaves goes in as well
                            const float2 q0 = to_f32x2<false>(h0), q1 = to_f32x2<false>(h1);
                            const uint32_t r0 = transpose8x8(pack16<false>(p0 - q0.x, p1 - q0.y));
                            const uint32_t r1 = transpose8x8(pack16<false>(p2 - q1.x, p3 - q1.y));
                            mma16816(acc[t][g][0], a01, r0, r1);
                            mma16816(acc[t][g][1], a23, r0, r1);
                        }
                    }
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i + 1 < kStages; ++i) there[i] = there[i + 1];
            there[kStages - 1] = copier.copy(c, a, R, st);
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }

        // ---- the item's end: its result, or a part to be joined.  Sums are in
        // units of 2^(m - kHead + E).
        const bool whole = seg.blk == 0 && seg_blocks == w.blocks && a.cluster <= 1;
        const int part = seg.blk == 0 ? 1 : 0;
        float* dst = part == 0 ? join + warp * kPart : reinterpret_cast<float*>(ring + warp * kStages * kStage);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = t * 8 + 2 * cc + e;
                float l = l_sum[t][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const float m = m_ref[t][e] == kNegInf ? kNegInf : -neg_ref[t][e];
                if (whole) {
                    if (rr < rows) {
#pragma unroll
                        for (int g = 0; g < NG; ++g)
                            write_row<BF16>(c, a, w, seg.b, D, tile * R + rr, head, g * kGroup + 4 * r,
                                            make_float4(acc[t][g][0][e], acc[t][g][0][2 + e] * 0.0625f,
                                                        acc[t][g][1][e], acc[t][g][1][2 + e] * 0.0625f),
                                            m, l, g == 0 && r == 0 && a.lse != nullptr);
                    }
                } else {
                    if (r == 0) join_ml[(warp * 2 + part) * R + rr] = make_float2(m, l);
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        *reinterpret_cast<float4*>(dst + rr * (D + 4) + g * kGroup + 4 * r) =
                            make_float4(acc[t][g][0][e], acc[t][g][0][2 + e] * 0.0625f, acc[t][g][1][e],
                                        acc[t][g][1][2 + e] * 0.0625f);
                }
            }
        if (!whole && lane == 0) parts[warp * 2 + part] = {seg.b, seg.item, seg.blk + seg_blocks == w.blocks};
        x += seg_blocks;
        seg.blk += seg_blocks;
        if (x < x_end) seg.settle(c, a, R);
    }

    // ---- join the warps' parts.  Those of one item follow one another; a group
    // that starts and ends its item is the result, else it goes to the
    // CTA's slot 0 (carries an item on) or 1 (starts one).
    __syncthreads();
    if (a.whole && a.cluster > 1) {
        // all parts are of the cluster's item: join them here, then over the cluster
        float* sums = reinterpret_cast<float*>(smem + kDecodeSmem<NG, NT>);
        float2* mls = reinterpret_cast<float2*>(sums + R * D);
        const Work w = work_of(c, a, seg.b, R, false);
        const int item = (blockIdx.x / a.cluster) % a.whole;
        const int head = item / w.tiles, tile = item - head * w.tiles;
        const int rows = min(R, w.n * a.G - tile * R);
        for (int i = tid; i < rows * (D / 4); i += kThreads) {
            const int rr = i / (D / 4), d4 = i - rr * (D / 4);
            float m = kNegInf, l = 0.f;
#pragma unroll
            for (int k = 0; k < 2 * kWarps; ++k)
                if (parts[k].b >= 0) m = fmaxf(m, join_ml[k * R + rr].x);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 2 * kWarps; ++k) {
                if (parts[k].b < 0) continue;
                const float2 ml = join_ml[k * R + rr];
                const float f = ml.x == kNegInf ? 0.f : fa::ptx::ex2_approx(ml.x - m);
                const float* src = (k & 1) ? reinterpret_cast<const float*>(ring + (k >> 1) * kStages * kStage)
                                           : join + (k >> 1) * kPart;
                const float4 v = *reinterpret_cast<const float4*>(src + rr * (D + 4) + 4 * d4);
                l += f * ml.y;
                o.x += f * v.x;
                o.y += f * v.y;
                o.z += f * v.z;
                o.w += f * v.w;
            }
            *reinterpret_cast<float4*>(sums + rr * D + 4 * d4) = o;
            if (d4 == 0) mls[rr] = make_float2(m, l);
        }
        cluster_sync();
        const uint32_t sums_at = fa::ptx::smem_addr(sums), mls_at = fa::ptx::smem_addr(mls);
        for (int i = cluster_rank() * kThreads + tid; i < rows * (D / 4); i += a.cluster * kThreads) {
            const int rr = i / (D / 4), d4 = i - rr * (D / 4);
            float2 ml[kMaxCluster];
            float4 v[kMaxCluster];
            float m = kNegInf, l = 0.f;
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k) {
                if (k >= a.cluster) continue;
                ml[k] = cluster_load2(cluster_map(mls_at + rr * 8, k));
                v[k] = cluster_load4(cluster_map(sums_at + (rr * D + 4 * d4) * 4, k));
                m = fmaxf(m, ml[k].x);
            }
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k) {
                if (k >= a.cluster) continue;
                const float f = ml[k].x == kNegInf ? 0.f : fa::ptx::ex2_approx(ml[k].x - m);
                l += f * ml[k].y;
                o.x += f * v[k].x;
                o.y += f * v[k].y;
                o.z += f * v[k].z;
                o.w += f * v[k].w;
            }
            write_row<BF16>(c, a, w, seg.b, D, tile * R + rr, head, 4 * d4, o, m, l, d4 == 0 && a.lse != nullptr);
        }
        cluster_sync();   // no CTA's shared memory goes before the others have read it
        return;
    }
    for (int p = 0; p < 2 * kWarps;) {
        const Part first = parts[p];
        if (first.b < 0) {
            ++p;
            continue;
        }
        int end = p + 1, last = p;
        while (end < 2 * kWarps && (parts[end].b < 0 || (parts[end].b == first.b && parts[end].item == first.item))) {
            if (parts[end].b >= 0) last = end;
            ++end;
        }
        const Work w = work_of(c, a, first.b, R, false);
        const int head = first.item / w.tiles, tile = first.item - head * w.tiles;
        const int rows = min(R, w.n * a.G - tile * R);
        const bool starts = (p & 1) != 0, whole = starts && parts[last].ends;
        const int slot = blockIdx.x * 2 + (starts ? 1 : 0);
        for (int i = tid; i < rows * (D / 4); i += kWarps * 32) {
            const int rr = i / (D / 4), d4 = i - rr * (D / 4);
            float m = kNegInf;
            for (int k = p; k <= last; ++k)
                if (parts[k].b >= 0) m = fmaxf(m, join_ml[k * R + rr].x);
            float l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = p; k <= last; ++k) {
                if (parts[k].b < 0) continue;
                const float2 ml = join_ml[k * R + rr];
                const float f = ml.x == kNegInf ? 0.f : fa::ptx::ex2_approx(ml.x - m);
                const float* src = (k & 1) ? reinterpret_cast<const float*>(ring + (k >> 1) * kStages * kStage)
                                           : join + (k >> 1) * kPart;
                const float4 v = *reinterpret_cast<const float4*>(src + rr * (D + 4) + 4 * d4);
                l += f * ml.y;
                o.x += f * v.x;
                o.y += f * v.y;
                o.z += f * v.z;
                o.w += f * v.w;
            }
            if (whole) {
                write_row<BF16>(c, a, w, first.b, D, tile * R + rr, head, 4 * d4, o, m, l, d4 == 0 && a.lse != nullptr);
            } else {
                *reinterpret_cast<float4*>(a.part_o + (static_cast<long long>(slot) * R + rr) * D + 4 * d4) = o;
                if (d4 == 0) a.part_ml[slot * R + rr] = make_float2(m, l);
            }
        }
        p = end;
    }
}

// Joins the parts of the items that the ranges of decode_kernel cut: a CTA an
// item, a warp for each eighth row, lanes over the row's elements; in the
// order of the keys, so that the result does not depend on which CTA ended
// first.  All parts' references are read at once, then eight parts' elements at a
// time (one after the other, a context of 32768 keys took 25 us here).
constexpr int kJoinWarps = 8;

template <int NG, int NT, bool BF16>
__global__ void __launch_bounds__(kJoinWarps * 32) combine_kernel(Cache c, Attend a, int items_most) {
    constexpr int D = NG * kGroup, R = 8 * NT, E4 = (D / 4 + 31) / 32;   // float4s of a lane
    __shared__ long long two[2][kJoinWarps];
    const int b = blockIdx.x / items_most, item = blockIdx.x - b * items_most;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Work w = work_of(c, a, b, R, false);
    // blocks before sequence b, and of the whole call
    long long before = 0, all = 0;
    if (item < w.items) {
        for (int i = threadIdx.x; i < c.B; i += blockDim.x) {
            const Work v = work_of(c, a, i, R, false);
            const long long k = static_cast<long long>(v.items) * v.blocks;
            all += k;
            if (i < b) before += k;
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) {
            all += __shfl_xor_sync(0xffffffffu, all, m);
            before += __shfl_xor_sync(0xffffffffu, before, m);
        }
        if (lane == 0) {
            two[0][warp] = all;
            two[1][warp] = before;
        }
        __syncthreads();
        all = before = 0;
        for (int i = 0; i < kJoinWarps; ++i) {
            all += two[0][i];
            before += two[1][i];
        }
    }
    fa::ptx::grid_dependency_wait();   // every CTA waits: this launch ends after the one before it
    if (item >= w.items) return;
    const long long quota = quota_of(all, a.grid);
    const long long s = before + static_cast<long long>(item) * w.blocks, e = s + w.blocks;
    const int first = static_cast<int>(s / quota), parts = static_cast<int>((e - 1) / quota) - first + 1;
    if (parts == 1) return;   // decode_kernel wrote it
    const int head = item / w.tiles, tile = item - head * w.tiles;
    const int rows = min(R, w.n * a.G - tile * R);
    // part k lies in slot 2 (first + k), or behind it for the one that starts the item
    auto slot = [&](int k) { return 2 * (first + k) + (k == 0 ? 1 : 0); };
    for (int rr = warp; rr < rows; rr += kJoinWarps) {
        float m = kNegInf, l = 0.f;
        for (int k = lane; k < parts; k += 32) m = fmaxf(m, __ldcg(a.part_ml + slot(k) * R + rr).x);
#pragma unroll
        for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        float4 o[E4];
#pragma unroll
        for (int i = 0; i < E4; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < parts; k0 += 32) {
            // this lane's part of the next 32: its weight
            float f = 0.f, fl = 0.f;
            if (k0 + lane < parts) {
                const float2 ml = __ldcg(a.part_ml + slot(k0 + lane) * R + rr);
                f = ml.x == kNegInf ? 0.f : fa::ptx::ex2_approx(ml.x - m);
                fl = f * ml.y;
            }
#pragma unroll
            for (int x = 16; x; x >>= 1) fl += __shfl_xor_sync(0xffffffffu, fl, x);
            l += fl;
            const int n = min(32, parts - k0);
#pragma unroll 1
            for (int k = 0; k < n; k += 8) {
                float4 v[8][E4];
#pragma unroll
                for (int x = 0; x < 8; ++x)
#pragma unroll
                    for (int i = 0; i < E4; ++i)
                        v[x][i] = k + x < n && (D % 128 == 0 || i * 32 + lane < D / 4)
                                      ? __ldcg(reinterpret_cast<const float4*>(
                                                   a.part_o + (static_cast<long long>(slot(k0 + k + x)) * R + rr) * D) +
                                               i * 32 + lane)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float fx = __shfl_sync(0xffffffffu, f, k + x);
#pragma unroll
                    for (int i = 0; i < E4; ++i) {
                        o[i].x += fx * v[x][i].x;
                        o[i].y += fx * v[x][i].y;
                        o[i].z += fx * v[x][i].z;
                        o[i].w += fx * v[x][i].w;
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < E4; ++i)
            if (D % 128 == 0 || i * 32 + lane < D / 4)
                write_row<BF16>(c, a, w, b, D, tile * R + rr, head, 4 * (i * 32 + lane), o[i], m, l,
                                i == 0 && lane == 0 && a.lse != nullptr);
    }
}

}  // namespace kv4
