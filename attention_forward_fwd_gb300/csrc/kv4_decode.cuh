// kv4_decode.cuh -- attention of a few query rows over the quantised cache
// (fa_kv4_attention for at most 16 query rows a K/V head: single tokens,
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
//  * K's codes go to the tensor cores as fp16 subnormals: the nibble n in the
//    low bits of a half IS n 2^-24, in bits 4..7 it is n 2^-20, so a pair of
//    codes costs one AND.  Q's elements for the second kind carry a factor
//    1/16, and the accumulator of a group starts at -8 sum(q) 2^-24, which
//    turns n into n - 8.  Each group's product is scaled by the key's fp32
//    scale as it is added up, so nothing of K is rounded.
//  * V's codes are paired over two keys (one byte permutation), then
//    (x & mask | 0x6400) - 1032 gives n - 8 in fp16 exactly.  The offset is
//    taken off here and not at the end, because the accumulator runs over the
//    whole context and would carry an offset many times the result.
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
// Within a CTA the four warps take the blocks in turn, each with a ring of
// its own of asynchronous bulk copies (no barrier of the CTA in the loop; the
// copies run ahead over the ends of items), and join at the end of an item.
#pragma once

#include "kv4_cache.cuh"

namespace kv4 {

constexpr int kWarps = 4;
constexpr int kStages = 2;
constexpr int kBlock = 32;              // keys a block
constexpr float kLazy = 8.f;            // p may reach 2^kLazy before m moves
constexpr int kHead = 7;                // p s 2^(kHead - E) < 2^(kLazy + kHead) < 65504
constexpr float kNegInf = -INFINITY;

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
};

template <int NG>
struct Tile {
    static constexpr int D = NG * kGroup;
    static constexpr int kCodes = kBlock * 16 * NG;        // bytes of K's (V's) codes in a block
    static constexpr int kScales = kBlock * 2 * NG;
    static constexpr int kStage = 2 * (kCodes + kScales);
};

template <int NG, int NT>
constexpr int decode_smem() {
    return kWarps * kStages * Tile<NG>::kStage + kWarps * 8 * NT * (Tile<NG>::D + 4) * 4 + 1024;
}

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
    if (s.n > 0 && a.window >= 0) w.first = max(0, s.len - s.n - a.window) / kBlock * kBlock;
    w.blocks = s.n > 0 ? max(1, (max(0, s.len - w.first) + kBlock - 1) / kBlock) : 0;
    return w;
}

// All blocks of all sequences before b (b = B: of the call), by the whole CTA.
__device__ __forceinline__ long long scan_blocks(const Cache& c, const Attend& a, int tile_rows, bool tell,
                                                 long long target, int* found, long long* found_at,
                                                 long long* sh) {
    // Each round takes blockDim.x sequences; *found is the last b whose blocks
    // start at or before `target` and do not end there.
    long long base = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    for (int b0 = 0; b0 < c.B; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        long long mine = 0;
        if (b < c.B) {
            const Work w = work_of(c, a, b, tile_rows, tell);
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
        long long before = base, all = 0;
        for (int i = 0; i < nw; ++i) {
            if (i < warp) before += sh[i];
            all += sh[i];
        }
        const long long start = before + x - mine;
        if (mine > 0 && start <= target && target < start + mine) {
            *found = b;
            *found_at = start;
        }
        base += all;
    }
    __syncthreads();
    return base;
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

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity) {
    if (fa::ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = fa::ptx::globaltimer();
    for (uint32_t n = 1;; ++n) {
        if (fa::ptx::mbar_try_wait(bar, parity)) return true;
        if ((n & 31u) == 0 && fa::ptx::globaltimer() - t0 > 1000000000ull) {
            report(kStatusTimeout);
            return false;
        }
    }
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
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

// A lane's codes of a row of K: 2 r's, all groups, as pairs (r = 2 c, 2 c + 1).
template <int NG>
__device__ __forceinline__ uint32_t k_pair(const Words<2 * NG>& w, int g) {
    // halfwords g and NG + g; PRMT where they sit in registers
    return static_cast<uint32_t>(w.w[g]) | (static_cast<uint32_t>(w.w[NG + g]) << 16);
}

template <int NG, int NT, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(Cache c, Attend a) {
    constexpr int D = NG * kGroup, R = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* ring = smem;
    float* join = reinterpret_cast<float*>(smem + kWarps * kStages * Tile<NG>::kStage);   // [warp][R][D + 4]
    uint8_t* tail = reinterpret_cast<uint8_t*>(join + kWarps * R * (D + 4));
    float2* join_ml = reinterpret_cast<float2*>(tail);                                    // [warp][R], 512 bytes
    uint64_t* bars = reinterpret_cast<uint64_t*>(tail + 512);                             // [warp][stage], 64
    uint32_t* runs = reinterpret_cast<uint32_t*>(tail + 576);                             // [warp][stage]
    long long* scan = reinterpret_cast<long long*>(tail + 640);                           // [warps]
    int* sh_b = reinterpret_cast<int*>(tail + 704);
    long long* sh_at = reinterpret_cast<long long*>(tail + 712);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, cc = lane & 3;
    if (tid < kWarps * kStages) {
        fa::ptx::mbar_init(fa::ptx::smem_addr(bars + tid), 1);
        fa::ptx::fence_barrier_init();
    }

    // ---- this CTA's range of blocks
    const long long all = scan_blocks(c, a, R, blockIdx.x == 0, -1, sh_b, sh_at, scan);
    const long long quota = max((all + a.grid - 1) / a.grid, static_cast<long long>(kWarps));
    const long long lo = quota * blockIdx.x, hi = min(all, lo + quota);
    fa::ptx::launch_dependents();
    if (lo >= hi) return;
    scan_blocks(c, a, R, false, lo, sh_b, sh_at, scan);

    Cursor prod;   // the copies' place
    prod.b = *sh_b;
    prod.w = work_of(c, a, prod.b, R, false);
    const long long off = lo - *sh_at;
    prod.item = static_cast<int>(off / prod.w.blocks);
    prod.blk = static_cast<int>(off % prod.w.blocks);
    Cursor seg = prod;   // the CTA's place, the same in every warp
    prod.blk += warp;
    prod.settle(c, a, R);
    long long prod_x = lo + warp;

    uint8_t* my_ring = ring + warp * kStages * Tile<NG>::kStage;
    bool dead = false;
    const int run = (c.P % kBlock) == 0 ? kBlock : 16;   // tokens that lie together
    auto issue = [&](int stage) {
        if (prod_x >= hi) return;
        const uint32_t bar = fa::ptx::smem_addr(bars + warp * kStages + stage);
        const int head = prod.item / prod.w.tiles;
        const int key0 = prod.w.first + prod.blk * kBlock;
        const int left = prod.w.len - key0;              // may be <= 0: a sequence without keys
        // lane: (run of the block, K or V, codes or scales)
        const int sub = lane >> 2, which = (lane >> 1) & 1, scales = lane & 1;
        const int tok = key0 + sub * run;
        const int want = min(run, (left - sub * run + 15) & ~15);
        bool ok = sub * run < kBlock && want > 0;
        int page = 0;
        if (ok) {
            page = __ldg(c.table + static_cast<long long>(prod.b) * c.max_pages + tok / c.P);
            if (page < 0 || page >= c.pages) {
                report(kStatusBadPages);
                ok = false;
            }
        }
        const long long row = ((static_cast<long long>(page) * 2 + which) * c.Hkv + head) * c.P + tok % c.P;
        const uint32_t bytes = ok ? static_cast<uint32_t>(want) * (scales ? 2 * NG : 16 * NG) : 0;
        uint32_t sum = bytes;
#pragma unroll
        for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        const uint32_t mask = __ballot_sync(0xffffffffu, ok);
        if (lane == 0) {
            runs[warp * kStages + stage] = (mask & 1u) | ((mask >> 4) & 1u) << 1;
            fa::ptx::mbar_arrive_expect_tx(bar, sum);
        }
        __syncwarp();
        if (ok) {
            uint8_t* base = my_ring + stage * Tile<NG>::kStage;
            uint8_t* dst = scales ? base + 2 * Tile<NG>::kCodes + which * Tile<NG>::kScales + sub * run * 2 * NG
                                  : base + which * Tile<NG>::kCodes + sub * run * 16 * NG;
            const void* src = scales ? static_cast<const void*>(c.scales + row * NG)
                                     : static_cast<const void*>(c.codes + row * (16 * NG));
            bulk_load(fa::ptx::smem_addr(dst), src, bytes, bar);
        }
        prod_x += kWarps;
        prod.blk += kWarps;
        if (prod_x < hi) prod.settle(c, a, R);
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) issue(s);

    long long x = lo + warp;    // this warp's next block
    int stage = 0;
    uint32_t parity = 0;
    const uint16_t* q16 = static_cast<const uint16_t*>(a.q);

    for (long long seg_lo = lo; seg_lo < hi;) {
        // ---- one item, or the part of it that is this CTA's
        const Work w = seg.w;
        const long long seg_hi = min(hi, seg_lo + (w.blocks - seg.blk));
        const int head = seg.item / w.tiles, tile = seg.item - head * w.tiles;
        const int rows = min(R, w.n * a.G - tile * R);

        // ---- Q: fp16 with each row's largest magnitude in [2^11, 2^12), the
        // elements that meet codes in bits 4..7 divided by 16
        uint32_t qf[NT][NG][4];
        float cinit[NT][NG][2], fac[NT][2];
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
            float qsum[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                // elements 8 cc + e: e = j and 4 + j pair up; j odd sits in bits 4..7
                const float2 e01 = to_f32x2<BF16>(raw[g].x), e23 = to_f32x2<BF16>(raw[g].y);
                const float2 e45 = to_f32x2<BF16>(raw[g].z), e67 = to_f32x2<BF16>(raw[g].w);
                qf[t][g][0] = pack16<false>(e01.x * mul, e45.x * mul);       // j = 0
                qf[t][g][1] = pack16<false>(e23.x * mul, e67.x * mul);       // j = 2
                qf[t][g][2] = pack16<false>(e01.y * mul16, e45.y * mul16);   // j = 1
                qf[t][g][3] = pack16<false>(e23.y * mul16, e67.y * mul16);   // j = 3
                const float2 s0 = to_f32x2<false>(qf[t][g][0]), s1 = to_f32x2<false>(qf[t][g][1]);
                const float2 s2 = to_f32x2<false>(qf[t][g][2]), s3 = to_f32x2<false>(qf[t][g][3]);
                qsum[g] = ((s0.x + s0.y) + (s1.x + s1.y)) + 16.f * ((s2.x + s2.y) + (s3.x + s3.y));
                qsum[g] += __shfl_xor_sync(0xffffffffu, qsum[g], 1);
                qsum[g] += __shfl_xor_sync(0xffffffffu, qsum[g], 2);
                qsum[g] *= -8.f * 5.9604644775390625e-8f;                    // -8 2^-24
            }
            // z = S 2^24 2^-up scale log2 e
            const float f = a.scale * 1.4426950408889634f * 16777216.f *
                            __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int from = (2 * cc + e) * 4;   // a lane that holds row 2 cc + e
                fac[t][e] = __shfl_sync(0xffffffffu, f, from);
#pragma unroll
                for (int g = 0; g < NG; ++g) cinit[t][g][e] = __shfl_sync(0xffffffffu, qsum[g], from);
                const int rr = t * 8 + 2 * cc + e;
                const int pos = rr < rows ? w.len - w.n + (tile * R + rr) / a.G : -1;
                hi_key[t][e] = pos;
                lo_key[t][e] = a.window >= 0 ? max(0, pos - a.window) : 0;
            }
        }

        float acc[NT][NG][2][4];
        float m_ref[NT][2], l_sum[NT][2];
        int e_ref = -90;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m_ref[t][e] = kNegInf;
                l_sum[t][e] = 0.f;
            }
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[t][g][i >> 2][i & 3] = 0.f;
        }

        for (; x < seg_hi; x += kWarps) {
            const int key0 = w.first + (seg.blk + static_cast<int>(x - seg_lo)) * kBlock;
            if (!dead && !wait_bounded(fa::ptx::smem_addr(bars + warp * kStages + stage), parity)) dead = true;
            const uint8_t* st = my_ring + stage * Tile<NG>::kStage;
            const uint32_t good = runs[warp * kStages + stage];
            // bit r16 of `in`: sub-tile r16 (16 keys) has been copied
            const uint32_t in = run == kBlock ? ((good & 1u) ? 3u : 0u) : good;

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
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[kt][t][i] = 0.f;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint32_t x0 = k_pair<NG>(c0, g), x1 = k_pair<NG>(c1, g);
                    const uint32_t a_even[4] = {x0 & 0x000f000fu, x1 & 0x000f000fu, (x0 >> 8) & 0x000f000fu,
                                                (x1 >> 8) & 0x000f000fu};
                    const uint32_t a_odd[4] = {x0 & 0x00f000f0u, x1 & 0x00f000f0u, (x0 >> 8) & 0x00f000f0u,
                                               (x1 >> 8) & 0x00f000f0u};
                    const float f0 = bf16_bits(s0.w[g]), f1 = bf16_bits(s1.w[g]);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float d[4] = {cinit[t][g][0], cinit[t][g][1], cinit[t][g][0], cinit[t][g][1]};
                        mma16816(d, a_even, qf[t][g][0], qf[t][g][1]);
                        mma16816(d, a_odd, qf[t][g][2], qf[t][g][3]);
                        s[kt][t][0] = fmaf(f0, d[0], s[kt][t][0]);
                        s[kt][t][1] = fmaf(f0, d[1], s[kt][t][1]);
                        s[kt][t][2] = fmaf(f1, d[2], s[kt][t][2]);
                        s[kt][t][3] = fmaf(f1, d[3], s[kt][t][3]);
                    }
                }
            }

            // ---- z, masks, and whether a reference has to move
            bool grow = false;
            float top[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = kNegInf;
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int key = key0 + kt * 16 + h * 8 + key_of(r);
                            const bool seen = key <= hi_key[t][e] && key >= lo_key[t][e] && ((in >> kt) & 1u);
                            float& z = s[kt][t][h * 2 + e];
                            z = seen ? z * fac[t][e] : kNegInf;
                            mx = fmaxf(mx, z);
                        }
                    top[t][e] = mx;
                    grow |= mx > m_ref[t][e] + kLazy;
                }
            // V's scales, zero where the key was not copied or lies past the
            // sequence (there may be anything there, NaN included)
            Words<NG> sv[2][2];
            uint32_t big = 0;
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int kk = kt * 16 + h * 8 + key_of(r);
                    sv[kt][h].load(st + 2 * Tile<NG>::kCodes + Tile<NG>::kScales + kk * 2 * NG);
                    const bool there = key0 + kk < w.len && ((in >> kt) & 1u);
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        if (!there) sv[kt][h].w[g] = 0;
                        big = max(big, static_cast<uint32_t>(sv[kt][h].w[g]) & 0x7fffu);
                    }
                }
            // s < 2^(exponent + 1); the bound moves by one more than it has to
            grow |= static_cast<int>(big >> 7) - 126 > e_ref || big >= 0x7f80u;   // or a scale is a NaN
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
                                        if ((sv[kt][h].w[g] & 0x7fffu) >= 0x7f80u && !(s[kt][t][h * 2 + e] == kNegInf))
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
                                if ((sv[kt][h].w[g] & 0x7fffu) >= 0x7f80u) sv[kt][h].w[g] = 0;
                }
                uint32_t fin = 0;   // the largest scale
#pragma unroll
                for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            fin = max(fin, static_cast<uint32_t>(sv[kt][h].w[g]) & 0x7fffu);
                        }
                fin = __reduce_max_sync(0xffffffffu, fin);
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
                        const float mn = fmaxf(m_ref[t][e], mx);
                        const float al = (mn == kNegInf ? 1.f : fa::ptx::ex2_approx(m_ref[t][e] - mn)) * de;
                        m_ref[t][e] = mn;
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
            const float lift = static_cast<float>(kHead - e_ref);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ref = (m_ref[t][e] == kNegInf ? 0.f : m_ref[t][e]) - lift;
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float& z = s[kt][t][h * 2 + e];
                            z = fa::ptx::ex2_approx(z - ref);
                            l_sum[t][e] += z;
                        }
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
                    const uint32_t xa = static_cast<uint32_t>(v[0].w[g]) | (static_cast<uint32_t>(v[1].w[g]) << 16);
                    const uint32_t xb = static_cast<uint32_t>(v[2].w[g]) | (static_cast<uint32_t>(v[3].w[g]) << 16);
                    // n - 8 (bits 0..3) and 16 (n - 8) (bits 4..7) in fp16
                    auto low = [](uint32_t u) {
                        const uint32_t y = (u & 0x000f000fu) | 0x64006400u;
                        const __half2 z = __hsub2(*reinterpret_cast<const __half2*>(&y), __half2half2(__ushort_as_half(0x6408)));
                        return *reinterpret_cast<const uint32_t*>(&z);
                    };
                    auto high = [](uint32_t u) {
                        const uint32_t y = (u & 0x00f000f0u) | 0x64006400u;
                        const __half2 z = __hsub2(*reinterpret_cast<const __half2*>(&y), __half2half2(__ushort_as_half(0x6480)));
                        return *reinterpret_cast<const uint32_t*>(&z);
                    };
                    const uint32_t a01[4] = {low(xa), high(xa), low(xb), high(xb)};
                    const uint32_t a23[4] = {low(xa >> 8), high(xa >> 8), low(xb >> 8), high(xb >> 8)};
                    const float f0 = bf16_bits(sv[kt][0].w[g]), f1 = bf16_bits(sv[kt][1].w[g]);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint32_t b0 = transpose8x8(pack16<false>(s[kt][t][0] * f0, s[kt][t][1] * f0));
                        const uint32_t b1 = transpose8x8(pack16<false>(s[kt][t][2] * f1, s[kt][t][3] * f1));
                        mma16816(acc[t][g][0], a01, b0, b1);
                        mma16816(acc[t][g][1], a23, b0, b1);
                    }
                }
            }
            __syncwarp();
            issue(stage);
            if (++stage == kStages) {
                stage = 0;
                parity ^= 1u;
            }
        }

        // ---- join the warps
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = t * 8 + 2 * cc + e;
                float l = l_sum[t][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                // sums are in units of 2^(m - kHead + E)
                if (r == 0)
                    join_ml[warp * R + rr] = make_float2(
                        m_ref[t][e] == kNegInf ? kNegInf : m_ref[t][e] - static_cast<float>(kHead - e_ref), l);
                float* dst = join + (warp * R + rr) * (D + 4) + 4 * r;
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    *reinterpret_cast<float4*>(dst + g * kGroup) =
                        make_float4(acc[t][g][0][e], acc[t][g][0][2 + e] * 0.0625f, acc[t][g][1][e],
                                    acc[t][g][1][2 + e] * 0.0625f);
            }
        __syncthreads();
        const bool whole = seg.blk == 0 && seg_hi - seg_lo == w.blocks;
        const int slot = blockIdx.x * 2 + (seg.blk == 0 ? 1 : 0);
        for (int i = tid; i < rows * (D / 4); i += kWarps * 32) {
            const int rr = i / (D / 4), d4 = i - rr * (D / 4);
            float2 ml[kWarps];
            float m = kNegInf;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                ml[k] = join_ml[k * R + rr];
                m = fmaxf(m, ml[k].x);
            }
            float l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float f = ml[k].x == kNegInf ? 0.f : fa::ptx::ex2_approx(ml[k].x - m);
                l += f * ml[k].y;
                const float4 v = *reinterpret_cast<const float4*>(join + (k * R + rr) * (D + 4) + 4 * d4);
                o.x += f * v.x;
                o.y += f * v.y;
                o.z += f * v.z;
                o.w += f * v.w;
            }
            if (whole) {
                const int rho = tile * R + rr, qi = rho / a.G, h = head * a.G + rho % a.G;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                uint16_t* dst = static_cast<uint16_t*>(a.o) +
                                (static_cast<long long>(w.row0 + qi) * a.H + h) * D + 4 * d4;
                *reinterpret_cast<uint2*>(dst) =
                    make_uint2(pack16<BF16>(o.x * inv, o.y * inv), pack16<BF16>(o.z * inv, o.w * inv));
                if (a.lse != nullptr && d4 == 0)
                    a.lse[(c.cu != nullptr ? w.row0 : seg.b * a.lse_batch) + h * a.lse_head + qi] =
                        l == 0.f ? kNegInf : (m + log2f(l)) * 0.6931471805599453f;
            } else {
                *reinterpret_cast<float4*>(a.part_o + (static_cast<long long>(slot) * R + rr) * D + 4 * d4) = o;
                if (d4 == 0) a.part_ml[slot * R + rr] = make_float2(m, l);
            }
        }
        __syncthreads();
        seg.blk += static_cast<int>(seg_hi - seg_lo);
        seg_lo = seg_hi;
        if (seg_lo < hi) seg.settle(c, a, R);
    }
}

// Joins the parts of the items that the ranges of decode_kernel cut: one CTA
// an item, in the order of the keys (the result does not depend on which CTA
// ended first).
template <int NG, int NT, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) combine_kernel(Cache c, Attend a, int items_most) {
    constexpr int D = NG * kGroup, R = 8 * NT;
    __shared__ long long two[2][kWarps];
    const int b = blockIdx.x / items_most, item = blockIdx.x - b * items_most;
    const Work w = work_of(c, a, b, R, false);
    if (item >= w.items) {
        fa::ptx::grid_dependency_wait();   // every CTA waits: this launch ends after the one before it
        return;
    }
    // blocks before sequence b, and of the whole call
    long long before = 0, all = 0;
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        long long mine_all = 0, mine_before = 0;
        for (int i = threadIdx.x; i < c.B; i += blockDim.x) {
            const Work v = work_of(c, a, i, R, false);
            const long long k = static_cast<long long>(v.items) * v.blocks;
            mine_all += k;
            if (i < b) mine_before += k;
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) {
            mine_all += __shfl_xor_sync(0xffffffffu, mine_all, m);
            mine_before += __shfl_xor_sync(0xffffffffu, mine_before, m);
        }
        if (lane == 0) {
            two[0][warp] = mine_all;
            two[1][warp] = mine_before;
        }
        __syncthreads();
        for (int i = 0; i < kWarps; ++i) {
            all += two[0][i];
            before += two[1][i];
        }
    }
    const long long quota = max((all + a.grid - 1) / a.grid, static_cast<long long>(kWarps));
    const long long s = before + static_cast<long long>(item) * w.blocks, e = s + w.blocks;
    const int first = static_cast<int>(s / quota), last = static_cast<int>((e - 1) / quota);
    fa::ptx::grid_dependency_wait();
    if (first == last) return;   // decode_kernel wrote it
    const int head = item / w.tiles, tile = item - head * w.tiles;
    const int rows = min(R, w.n * a.G - tile * R);
    for (int i = threadIdx.x; i < rows * (D / 4); i += kWarps * 32) {
        const int rr = i / (D / 4), d4 = i - rr * (D / 4);
        // the first part starts the item (slot 1 of its CTA), the others carry it on (slot 0)
        float m = kNegInf, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = first; k <= last; ++k) {
            const int slot = 2 * k + (k == first ? 1 : 0);
            const float2 ml = __ldcg(a.part_ml + slot * R + rr);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(
                a.part_o + (static_cast<long long>(slot) * R + rr) * D + 4 * d4));
            const float mn = fmaxf(m, ml.x);
            if (mn == kNegInf) continue;
            const float f0 = fa::ptx::ex2_approx(m - mn), f1 = fa::ptx::ex2_approx(ml.x - mn);
            m = mn;
            l = l * f0 + ml.y * f1;
            o.x = o.x * f0 + v.x * f1;
            o.y = o.y * f0 + v.y * f1;
            o.z = o.z * f0 + v.z * f1;
            o.w = o.w * f0 + v.w * f1;
        }
        const int rho = tile * R + rr, qi = rho / a.G, h = head * a.G + rho % a.G;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* dst = static_cast<uint16_t*>(a.o) + (static_cast<long long>(w.row0 + qi) * a.H + h) * D + 4 * d4;
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(pack16<BF16>(o.x * inv, o.y * inv), pack16<BF16>(o.z * inv, o.w * inv));
        if (a.lse != nullptr && d4 == 0)
            a.lse[(c.cu != nullptr ? w.row0 : b * a.lse_batch) + h * a.lse_head + qi] =
                l == 0.f ? kNegInf : (m + log2f(l)) * 0.6931471805599453f;
    }
}

}  // namespace kv4
