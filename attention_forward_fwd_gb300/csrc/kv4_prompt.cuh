// kv4_prompt.cuh -- attention of many query rows over the quantised cache
// (fa_kv4_attention for more than kDecodeRows query rows a K/V head: parts of
// prompts), on the tcgen05 tensor cores.
//
// A CTA takes one sequence, one K/V head and TILES x 128 of its query rows (the
// group's heads times the call's tokens, so that the heads of a group share the
// unpacked K and V), and walks over tiles of BN keys:
//   unpack warps   codes and scales -> fp16 K and V tiles in shared memory
//   MMA warp       S_t = Q_t K^T, O_t += P_t V (fp32 in tensor memory)
//   softmax warps  thread = row = TMEM lane: S -> P (fp16, over S), the
//                  running maximum, O's rescaling, the row sum.  S is read in
//                  quarters, the next one while one is worked on.  The last
//                  two stay in registers from the maximum to the exponentials, and P
//                  goes over the second half of S, so that the first two can be read again.
// D <= 128: two row tiles that take turns on the tensor pipe (S_A, S_B, then
// P_A V, S_A of the next keys, P_B V, ...).  D > 128: one row tile, as two O
// tiles do not fit, with two S buffers (S of the next keys runs beside the softmax).
//
// Numbers.  A value is s (n - 8) with s of 8 bits and n - 8 of 3, so K and V
// are exact in fp16 once their scales are brought near one: each tile has
// exponents Ek and Ev from its largest scales, K' = K 2^-Ek and V' = V 2^-Ev.
// 2^Ek goes into the factor of the scores.  2^Ev goes into the exponent of P,
// p' = 2^(z + Ev - r), with one running reference r a row, and the tile's part of
// the row sum is multiplied by 2^-Ev.  Q is brought to [2^11, 2^12) row by row.  Then only
// P is rounded (fp16, 2^-12); for fp16 results what that leaves goes in as a
// second product.
//
// Elements 8 i .. 8 i + 7 of a row lie in the order 0 4 1 5 2 6 3 7 in all three
// tiles: codes come out of their words in pairs (j, 4 + j), and a contraction
// does not care; O's columns are put back in the epilogue.
//
// The code of the three roles has to stay small: with every loop unrolled and the
// masks inline the warps waited for instructions nearly twice as long as they
// ran them.  Tiles that need a mask have it written over S first, in a loop of its
// own, K and V share the unpacking code, both row tiles the issuing code.
//
// What bounds it: softmax and tensor pipe, as in the plain forward, and beside
// them the unpacking, 32,768 values a tile of 128 keys at D = 128 for about 2.2
// instructions each.  Two row tiles a CTA halve that.
#pragma once

#include "kv4_decode.cuh"

namespace kv4 {

constexpr int kRowTile = 128;
constexpr int kInfo = 4;               // tile descriptions in flight
constexpr float kPHead = 7.f;          // P is held as p 2^kPHead, p <= 2^kLazy

template <int NG>
struct Prompt {
    static constexpr int D = NG * kGroup;
    static constexpr bool kWide = NG > 4;
    static constexpr int TILES = kWide ? 1 : 2;
    static constexpr int BN = kWide ? 64 : 128;
    static constexpr int kBoxes = (NG + 1) / 2;            // 64 columns each
    static constexpr int N = kBoxes * 64;                  // columns of O (past D: zeros)
    static constexpr int kSoftWarps = 4 * TILES;
    static constexpr int kUnpackWarps = kWide ? 8 : 4;
    static constexpr int kMmaWarp = kSoftWarps + kUnpackWarps;
    static constexpr int kThreads = (kMmaWarp + 1) * 32;
    static constexpr int kQBox = kRowTile * 128, kBox = BN * 128;   // bytes
    static constexpr int kQTile = kBoxes * kQBox, kTile = kBoxes * kBox;
    static constexpr int kOffK = TILES * kQTile, kOffV = kOffK + 2 * kTile, kOffBar = kOffV + 2 * kTile;
    static constexpr int kSmem = kOffBar + 2048 + 1024;    // and room to align
    static constexpr uint32_t kO = 256;                    // TMEM: S at 0 and 128, O from here on
    static_assert(kO + TILES * N <= 512, "tensor memory");
    static_assert(kSmem <= 232448, "shared memory");
};

struct TileInfo {
    int ek, ev;
    uint32_t missing;      // bit i: the i-th 16 keys are not there (a bad page)
    uint32_t nan;          // nonzero: some V scale is a NaN
};

struct PromptBars {
    uint64_t q_full, full[2][2], empty[2][2];   // [K or V][slot]
    uint64_t s_full[2], p_full[2], o_done, o_last, info[kInfo], drain;
    TileInfo tile[kInfo];
    uint32_t top[2][8];                  // of each unpack warp: largest scales, K below V
    uint32_t gone[2][8];
    uint8_t nan_groups[kInfo][128];      // of each key of V
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(PromptBars) <= 2048, "barriers");

// The items (row tiles of R rows, K/V heads, sequences) in the order of the
// grid; those of whole waves have a CTA each, those behind them `splits`.
struct PromptPlan {
    int tiles_most;        // row tiles of a sequence and K/V head
    int whole;             // items that are not split
    int splits;            // CTAs that share the keys of one of the others
};

// Bounded wait; false (and the CTA's abort flag set) when it ran out, or when
// another role gave up.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort, bool heed = true) {
    if (fa::ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = fa::ptx::globaltimer();
    for (uint32_t n = 1;; ++n) {
        if (fa::ptx::mbar_try_wait(bar, parity)) return true;
        if ((n & 31u) == 0) {
            if (heed && *abort) return false;
            if (fa::ptx::globaltimer() - t0 > 1000000000ull) {
                *abort = 1;
                report(kStatusTimeout);
                return false;
            }
        }
    }
}

// 32 lanes x 8 columns of tensor memory
__device__ __forceinline__ void tmem_ld_x8(uint32_t at, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t at, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
}
template <int N>
__device__ __forceinline__ void store_p(uint32_t at, const uint32_t* p) {
    if constexpr (N == 16) fa::ptx::tmem_st_32x32b_x16(at, p);
    else fa::ptx::tmem_st_32x32b_x8(at, p);
}

__device__ __forceinline__ float pow2(int e) {   // -126 <= e <= 127
    return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&z);
}

// Eight values (groups' elements 8 c .. 8 c + 7) of each group of one key to
// their places in a tile: 16-byte chunk 4 (g mod 2) + c of box g / 2, 128-byte swizzle.
template <int NG, int BOX>
__device__ __forceinline__ void unpack_unit(const Words<2 * NG>& raw, const Words<NG>& scales, float down, int c, int key,
                                            uint8_t* tile) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const uint32_t x = join_words(raw, g, raw, NG + g), y = x >> 8;
        const float s = scales.bf16(g) * down;
        const uint32_t s1 = pack16<false>(s, s), s16 = pack16<false>(s * 0.0625f, s * 0.0625f);
        const uint4 v = make_uint4(hmul2(low_codes(x), s1), hmul2(high_codes(x), s16), hmul2(low_codes(y), s1),
                                   hmul2(high_codes(y), s16));
        const int chunk = 4 * (g & 1) + c;
        *reinterpret_cast<uint4*>(tile + (g >> 1) * BOX + key * 128 + ((chunk ^ (key & 7)) << 4)) = v;
    }
}

template <int NG, bool BF16>
__global__ void __launch_bounds__(Prompt<NG>::kThreads, 1) prompt_kernel(Cache c, Attend a, PromptPlan plan) {
    using L = Prompt<NG>;
    constexpr int D = L::D, TILES = L::TILES, BN = L::BN, NB = L::kBoxes, N = L::N;
    constexpr bool WIDE = L::kWide;
    constexpr int R = TILES * kRowTile, kUnpackWarps = L::kUnpackWarps;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = fa::ptx::smem_addr(smem);
    PromptBars* bars = reinterpret_cast<PromptBars*>(smem + L::kOffBar);
    volatile int* abort = &bars->abort;
    auto bar = [](const uint64_t* b) { return fa::ptx::smem_addr(b); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // ------------------------------------------------------------ the item
    const int behind = static_cast<int>(blockIdx.x) - plan.whole;
    const int splits = behind < 0 ? 1 : plan.splits;
    const int split = behind < 0 ? 0 : behind % plan.splits;
    const int y = behind < 0 ? static_cast<int>(blockIdx.x) : plan.whole + behind / plan.splits;
    const int bh = y % (c.B * c.Hkv), b = bh / c.Hkv, head = bh - b * c.Hkv;
    const int tile = plan.tiles_most - 1 - y / (c.B * c.Hkv);    // the longest first
    const Work w = work_of(c, a, b, R, tile == 0 && head == 0 && split == 0 && threadIdx.x == 0);
    if (tile >= w.tiles) return;
    const int rows = min(R, w.n * a.G - tile * R);
    // key tiles that some row sees, and this split's share of them
    const int pos0 = w.len - w.n + tile * R / a.G, pos1 = w.len - w.n + (tile * R + rows - 1) / a.G;
    const int t_lo = a.window >= 0 ? max(0, pos0 - a.window) / BN : 0;
    const int t_all = pos1 >= 0 ? pos1 / BN + 1 - t_lo : 0;
    const int jb = t_lo + static_cast<int>(static_cast<long long>(t_all) * split / splits);
    const int n_tiles = t_lo + static_cast<int>(static_cast<long long>(t_all) * (split + 1) / splits) - jb;

    if (threadIdx.x == 0) {
        fa::ptx::mbar_init(bar(&bars->q_full), R);
        for (int i = 0; i < 2; ++i) {
            for (int x = 0; x < 2; ++x) {
                fa::ptx::mbar_init(bar(&bars->full[x][i]), kUnpackWarps);
                fa::ptx::mbar_init(bar(&bars->empty[x][i]), 1);
            }
            fa::ptx::mbar_init(bar(&bars->s_full[i]), 1);
            fa::ptx::mbar_init(bar(&bars->p_full[i]), kRowTile);
        }
        for (int i = 0; i < kInfo; ++i) fa::ptx::mbar_init(bar(&bars->info[i]), 1);
        fa::ptx::mbar_init(bar(&bars->o_done), 1);
        fa::ptx::mbar_init(bar(&bars->o_last), 1);
        fa::ptx::mbar_init(bar(&bars->drain), 1);
        bars->abort = 0;
        fa::ptx::fence_barrier_init();
    }
    if (warp == L::kMmaWarp) {
        fa::ptx::tmem_alloc(fa::ptx::smem_addr(&bars->tmem), 512);
        fa::ptx::tmem_relinquish();
    }
    fa::ptx::tc_fence_before_sync();
    __syncthreads();
    fa::ptx::tc_fence_after_sync();
    const uint32_t tmem = bars->tmem;
    fa::ptx::launch_dependents();

    auto wait_warp = [&](uint32_t b_, uint32_t parity, bool heed = true) {
        return __all_sync(0xffffffffu, wait_bar(b_, parity, abort, heed));
    };

    if (warp == L::kMmaWarp) {
        // ------------------------------------------------------ MMA issue
        constexpr uint32_t kIdescS = fa::ptx::idesc_f16_f32(kRowTile, BN, false, false);
        constexpr uint32_t kIdescO = fa::ptx::idesc_f16_f32(kRowTile, N, false, true);
        const uint32_t hi = fa::ptx::sdesc_sw128_hi(1024);
        const uint32_t qlo = fa::ptx::sdesc_sw128_lo(sbase, 16);
        const uint32_t klo = fa::ptx::sdesc_sw128_lo(sbase + L::kOffK, 16);
        const uint32_t vlo = fa::ptx::sdesc_sw128_lo(sbase + L::kOffV, L::kBox);
        bool ok = n_tiles == 0 || wait_warp(bar(&bars->q_full), 0);
        // S of key tile j, row tile t, into buffer s: K steps of 16 elements, 4 to a box
        auto issue_s = [&](int j, int t, int s) {
            const uint32_t k = klo + (j & 1) * (L::kTile / 16), q = qlo + t * (L::kQTile / 16);
            fa::ptx::tc_fence_after_sync();
#pragma unroll
            for (int x = 0; x < 2 * NG; x += 4) {
                if (x + 4 <= 2 * NG) {
                    fa::ptx::mma_ss_x4_lo(tmem + s * 128, q + (x / 4) * (L::kQBox / 16), k + (x / 4) * (L::kBox / 16), hi,
                                          2u, kIdescS, x > 0 ? 1u : 0u);
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)   // half a box is left
                        fa::ptx::mma_ss_warp_lo(tmem + s * 128, q + (x / 4) * (L::kQBox / 16) + 2 * i,
                                                k + (x / 4) * (L::kBox / 16) + 2 * i, hi, kIdescS, x + i > 0 ? 1u : 0u);
                }
            }
            fa::ptx::tc_commit_warp(bar(&bars->s_full[s]));
        };
        // O of row tile t from P in buffer s (8 columns a K step of 16 keys)
        auto issue_o = [&](int j, int t, int s) {
            const uint32_t v = vlo + (j & 1) * (L::kTile / 16);
            fa::ptx::tc_fence_after_sync();
#pragma unroll
            for (int part = 0; part < (BF16 ? 1 : 2); ++part)     // and what P's rounding left
#pragma unroll
                for (int x = 0; x < BN / 16; x += 4)
                    fa::ptx::mma_ts_x4_lo(tmem + L::kO + t * N, tmem + s * 128 + (1 - part) * (BN / 2) + x * 8, v + x * 128, hi, 8u,
                                          128u, kIdescO, (j > 0 || x > 0 || part > 0) ? 1u : 0u);
        };
        if constexpr (!WIDE) {
            // j = -1: S of the first tile alone
            for (int j = -1; j < n_tiles && ok; ++j) {
#pragma unroll 1
                for (int t = 0; t < TILES; ++t) {
                  if (j >= 0) {
                    if (!(ok = wait_warp(bar(&bars->p_full[t]), static_cast<uint32_t>(j & 1)))) break;
                    if (t == 0 && !(ok = wait_warp(bar(&bars->full[1][j & 1]), static_cast<uint32_t>((j >> 1) & 1)))) break;
                    issue_o(j, t, t);
                    if (t == TILES - 1) {
                        fa::ptx::tc_commit_warp(bar(&bars->empty[1][j & 1]));
                        if (j + 1 == n_tiles) fa::ptx::tc_commit_warp(bar(&bars->o_last));
                    }
                  }
                    if (j + 1 < n_tiles) {
                        if (t == 0 &&
                            !(ok = wait_warp(bar(&bars->full[0][(j + 1) & 1]), static_cast<uint32_t>(((j + 1) >> 1) & 1))))
                            break;
                        issue_s(j + 1, t, t);
                        if (t == TILES - 1) fa::ptx::tc_commit_warp(bar(&bars->empty[0][(j + 1) & 1]));
                    }
                }
            }
        } else {
            for (int j = -1; j < n_tiles && ok; ++j) {
                if (j + 1 < n_tiles) {
                    const int i = j + 1;
                    if (!(ok = wait_warp(bar(&bars->full[0][i & 1]), static_cast<uint32_t>((i >> 1) & 1)))) break;
                    issue_s(i, 0, i & 1);
                    fa::ptx::tc_commit_warp(bar(&bars->empty[0][i & 1]));
                }
                if (j < 0) continue;
                if (!(ok = wait_warp(bar(&bars->p_full[j & 1]), static_cast<uint32_t>((j >> 1) & 1)))) break;
                if (!(ok = wait_warp(bar(&bars->full[1][j & 1]), static_cast<uint32_t>((j >> 1) & 1)))) break;
                issue_o(j, 0, j & 1);
                fa::ptx::tc_commit_warp(bar(&bars->empty[1][j & 1]));
                fa::ptx::tc_commit_warp(bar(&bars->o_done));
                if (j + 1 == n_tiles) fa::ptx::tc_commit_warp(bar(&bars->o_last));
            }
        }
        // every MMA must be complete before the tensor memory is freed
        fa::ptx::tc_commit_warp(bar(&bars->drain));
        wait_warp(bar(&bars->drain), 0, false);
    } else if (warp >= L::kSoftWarps) {
        // ---------------------------------------------------------- unpack
        constexpr int CU = BN * 4 / (kUnpackWarps * 32);   // of the 4 units (c = 0 .. 3) of a key
        const int u = static_cast<int>(threadIdx.x) - L::kSoftWarps * 32;
        const int key = u % BN, c0 = u / BN * CU;          // this thread's units: c0 .. c0 + CU - 1
        const int uw = u >> 5;
        const long long k_to_v = static_cast<long long>(c.Hkv) * c.P;   // rows
        if constexpr (NG % 2 == 1) {
            // the last box's right half is never written: columns of zeros
            for (int i = u; i < 2 * BN * 4; i += kUnpackWarps * 32) {
                const int st = i / (BN * 4), k = (i / 4) % BN, chunk = 4 + (i & 3);
                *reinterpret_cast<uint4*>(smem + L::kOffV + st * L::kTile + (NB - 1) * L::kBox + k * 128 +
                                          ((chunk ^ (k & 7)) << 4)) = make_uint4(0, 0, 0, 0);
            }
        }
        const int* table = c.table + static_cast<long long>(b) * c.max_pages;
        // K's rows of a tile, V's, K's of the next one, ...: each asked for as the
        // ones before them are unpacked; the scales a tile ahead, the page two.
        Words<2 * NG> raw[CU];
        Words<NG> ks, vs, ks2, vs2;
        long long row = -1, row2 = -1;   // of the key in the cache, this tile and the next; -1: none
        bool gone = false, gone2 = false;
        int next = jb * BN + key;   // position that `pg`, `off` and `page` stand for
        int pg = next / c.P, off = next - pg * c.P, page = -1, tile_at = 0;
        const int step_pg = BN / c.P, step_off = BN - step_pg * c.P;
        auto look_up = [&] { page = tile_at < n_tiles && next < w.len ? __ldg(table + pg) : -1; };
        // the page of tile `tile_at` is here: its row, its scales; ask for the next page
        auto advance = [&] {
            const bool mine = tile_at < n_tiles && next < w.len;
            const bool ok = mine && page >= 0 && page < c.pages;
            gone2 = mine && !ok;
            if (gone2) report(kStatusBadPages);
            row2 = ok ? (static_cast<long long>(page) * 2 * c.Hkv + head) * c.P + off : -1;
            ks2.clear();
            vs2.clear();
            if (ok) {
                ks2.load_global(c.scales + row2 * NG);
                vs2.load_global(c.scales + (row2 + k_to_v) * NG);
            }
            ++tile_at;
            next += BN;
            pg += step_pg;
            off += step_off;
            if (off >= c.P) {
                off -= c.P;
                ++pg;
            }
            look_up();
        };
        auto load_rows = [&](Words<2 * NG>* to, long long from) {
#pragma unroll
            for (int i = 0; i < CU; ++i) {
                to[i].clear();
                if (from >= 0) to[i].load_global(c.codes + from * (16 * NG) + (c0 + i) * (4 * NG));
            }
        };
        look_up();
        advance();
        load_rows(raw, row2);
        bool ok = true;
        for (int j = 0; j < n_tiles; ++j) {
            ks = ks2;
            vs = vs2;
            gone = gone2;
            row = row2;
            advance();
            // ---- the tile's largest finite scales, NaNs and holes
            uint32_t kt = 0, vt = 0, nan_groups = 0;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint32_t x = ks.get(g) & 0x7fffu, z = vs.get(g) & 0x7fffu;
                kt = max(kt, x < 0x7f80u ? x : 0u);
                if (z >= 0x7f80u) {
                    nan_groups |= 1u << g;
                    vs.set(g, 0);
                } else {
                    vt = max(vt, z);
                }
            }
            kt = __reduce_max_sync(0xffffffffu, kt);
            vt = __reduce_max_sync(0xffffffffu, vt);
            const uint32_t holes = __ballot_sync(0xffffffffu, gone);
            const bool any_nan = __any_sync(0xffffffffu, nan_groups != 0);
            // Slot j % kInfo is free: V of tile j - 1 waited for P V of j - 3, so the
            // softmax is done with tile j - 4.
            if (c0 == 0) bars->nan_groups[j % kInfo][key] = static_cast<uint8_t>(nan_groups);
            if (lane == 0) {
                bars->top[j & 1][uw] = kt | (vt << 16);
                bars->gone[j & 1][uw] = ((holes & 0xffffu) ? 1u : 0u) | ((holes >> 16) ? 2u : 0u) | (any_nan ? 4u : 0u);
            }
            fa::ptx::named_barrier_sync(2, kUnpackWarps * 32);
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < kUnpackWarps; ++i) top = __vmaxu2(top, bars->top[j & 1][i]);
            // largest scale 2^e (1 .. 2) -> 2^11 .. 2^12
            const int ek = max(static_cast<int>((top & 0xffffu) >> 7) - 127, -100) - 11;
            const int ev = max(static_cast<int>(top >> 23) - 127, -100) - 11;
            if (u == 0) {   // what the softmax has to know
                uint32_t missing = 0, flags = 0;
                for (int i = 0; i < kUnpackWarps; ++i) {
                    const uint32_t f = bars->gone[j & 1][i];
                    flags |= f & 4u;
                    missing |= (f & 3u) << (2 * (i % (BN / 32)));
                }
                bars->tile[j % kInfo] = {ek, ev, missing, flags};
                fa::ptx::mbar_arrive(bar(&bars->info[j % kInfo]));
            }
            // ---- K, then V, each once its slot is free
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
                if (j >= 2)
                    ok = ok && wait_warp(bar(&bars->empty[x][j & 1]), static_cast<uint32_t>(((j >> 1) - 1) & 1));
                Words<2 * NG> ahead[CU];
                load_rows(ahead, x == 0 ? (row < 0 ? -1 : row + k_to_v) : row2);
                if (ok) {
                    uint8_t* to = smem + (x == 0 ? L::kOffK : L::kOffV) + (j & 1) * L::kTile;
                    const float down = pow2(x == 0 ? -ek : -ev);
#pragma unroll
                    for (int i = 0; i < CU; ++i) unpack_unit<NG, L::kBox>(raw[i], ks, down, c0 + i, key, to);
                    fa::ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) fa::ptx::mbar_arrive(bar(&bars->full[x][j & 1]));
                }
                ks = vs;
#pragma unroll
                for (int i = 0; i < CU; ++i) raw[i] = ahead[i];
            }
        }
    } else {
        // --------------------------------------------------------- softmax
        const int t = warp >> 2;                                      // row tile
        const int r = static_cast<int>(threadIdx.x) & 127;            // row of the tile, TMEM lane
        const int row = t * kRowTile + r, rho = tile * R + row;
        const bool real = row < rows;
        const int qi = rho / a.G, h = head * a.G + rho - qi * a.G;
        const int pos = real ? w.len - w.n + qi : -1;
        const int first = a.window >= 0 ? max(0, pos - a.window) : 0;
        const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        float f;   // z = S 2^Ek f
        {
            const uint16_t* src = static_cast<const uint16_t*>(a.q) +
                                  (c.cu != nullptr ? static_cast<long long>(w.row0 + qi) * a.q_row
                                                   : b * a.q_batch + qi * a.q_row) + h * a.q_head;
            float most = 0.f;
            if (real) {
#pragma unroll 4
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 x = __ldg(reinterpret_cast<const uint4*>(src) + i);
                    const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 v = to_f32x2<BF16>(e[k]);
                        most = fmaxf(most, fmaxf(fabsf(v.x), fabsf(v.y)));
                    }
                }
            }
            int up = most > 0.f ? 138 - static_cast<int>((__float_as_uint(most) >> 23) & 255u) : 0;
            up = max(-90, min(100, up));
            const float mul = pow2(up);
            f = fmaxf(a.scale * 1.4426950408889634f * pow2(-up), 1.17549435e-38f);
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                const uint4 x = real ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
                const float2 e01 = to_f32x2<BF16>(x.x), e23 = to_f32x2<BF16>(x.y);
                const float2 e45 = to_f32x2<BF16>(x.z), e67 = to_f32x2<BF16>(x.w);
                const uint4 v = make_uint4(pack16<false>(e01.x * mul, e45.x * mul), pack16<false>(e01.y * mul, e45.y * mul),
                                           pack16<false>(e23.x * mul, e67.x * mul), pack16<false>(e23.y * mul, e67.y * mul));
                *reinterpret_cast<uint4*>(smem + t * L::kQTile + (i >> 3) * L::kQBox + r * 128 +
                                          (((i & 7) ^ (r & 7)) << 4)) = v;
            }
            fa::ptx::fence_proxy_async_smem();
            fa::ptx::mbar_arrive(bar(&bars->q_full));
        }
        const uint32_t tO = tmem + lane_off + L::kO + t * N;
        float ref = kNegInf, l = 0.f;
        uint32_t poison = 0;      // groups that met a NaN of V
        bool ok = true;
        for (int j = 0; j < n_tiles; ++j) {
            const int sb = WIDE ? (j & 1) : t;
            const uint32_t phase = WIDE ? static_cast<uint32_t>((j >> 1) & 1) : static_cast<uint32_t>(j & 1);
            ok = ok && wait_bar(bar(&bars->s_full[sb]), phase, abort) &&
                 wait_bar(bar(&bars->info[j % kInfo]), static_cast<uint32_t>((j / kInfo) & 1), abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            fa::ptx::tc_fence_after_sync();
            const TileInfo info = bars->tile[j % kInfo];
            const uint32_t tS = tmem + lane_off + sb * 128;
            const int kv0 = (jb + j) * BN;
            const uint32_t missing = info.missing;
            const bool edge = __any_sync(0xffffffffu, kv0 + BN - 1 > pos || kv0 < first || missing != 0);
            const float zf = f * pow2(info.ek), ev = static_cast<float>(info.ev);
            constexpr int QK = BN / 4;   // keys of a quarter
            auto read = [&](uint32_t* s, int q) {
                if constexpr (QK == 32) fa::ptx::tmem_ld_32x32b_x32(tS + q * QK, s);
                else tmem_ld_x16(tS + q * QK, s);
            };
            auto arrived = [&](uint32_t* s, int q) {
                fa::ptx::tmem_ld_wait();
                fa::ptx::reg_fence<QK>(s);
            };
            if (edge) {
                // masked scores become -inf where they are
#pragma unroll 1
                for (int q = 0; q < BN / 8; ++q) {
                    uint32_t s[8];
                    tmem_ld_x8(tS + q * 8, s);
                    fa::ptx::tmem_ld_wait();
                    fa::ptx::reg_fence<8>(s);
                    const bool hole = (missing >> (q / 2)) & 1u;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int key = kv0 + q * 8 + k;
                        if (hole || key > pos || key < first) s[k] = __float_as_uint(kNegInf);
                    }
                    fa::ptx::tmem_st_32x32b_x8(tS + q * 8, s);
                }
                fa::ptx::tmem_st_wait();
            }
            uint32_t buf[2][QK];
            float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
            read(buf[0], 0);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                arrived(buf[q & 1], q);
                if (q < 3) read(buf[(q + 1) & 1], q + 1);
                uint32_t* s = buf[q & 1];
#pragma unroll
                for (int k = 0; k < QK; k += 8)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mx[i] = fa::ptx::fmax3(mx[i], __uint_as_float(s[k + 2 * i]), __uint_as_float(s[k + 2 * i + 1]));
            }
            mx[0] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            // the reference moves lazily, when p' would pass 2^kLazy
            const float top = mx[0] == kNegInf ? kNegInf : fmaf(mx[0], zf, ev);
            float alpha = 1.f;
            const bool move = top > ref + kLazy;
            if (move) {
                alpha = fa::ptx::ex2_approx(ref - top);   // 0 on the first tile
                ref = top;
            }
            if (j > 0 && __any_sync(0xffffffffu, move)) {
                // S of this tile came after P V of the one before (D <= 128); else that has a barrier of its own
                if constexpr (WIDE) {
                    ok = wait_bar(bar(&bars->o_done), static_cast<uint32_t>((j - 1) & 1), abort);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    fa::ptx::tc_fence_after_sync();
                }
#pragma unroll 1
                for (int q = 0; q < N / 8; ++q) {   // few registers: the row of S is held
                    uint32_t o[8];
                    tmem_ld_x8(tO + q * 8, o);
                    fa::ptx::tmem_ld_wait();
                    fa::ptx::reg_fence<8>(o);
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                    fa::ptx::tmem_st_32x32b_x8(tO + q * 8, o);
                }
            }
            if (info.nan != 0) {
                for (int k = 0; k < BN; ++k) {
                    const int key = (jb + j) * BN + k;
                    if (key <= pos && key >= first) poison |= bars->nan_groups[j % kInfo][k];
                }
            }
            const float off = ev + kPHead - (ref == kNegInf ? 0.f : ref);
            const float2 zf2 = make_float2(zf, zf), off2 = make_float2(off, off);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            // the quarters 2, 3, 0, 1: P of q in columns BN / 2 + q QK / 2 on, what its
            // rounding left in q QK / 2 on, which has to wait until S has been read there
            uint32_t left[BF16 ? 1 : 2][QK / 2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int q = (i + 2) & 3;
                uint32_t* s = buf[i & 1];
                if (i >= 2) {
                    arrived(s, q);
                    if constexpr (!BF16)
                        if (i == 2) {   // the wait was for quarter 1 as well
#pragma unroll
                            for (int h = 0; h < 2; ++h) store_p<QK / 2>(tS + (2 + h) * (QK / 2), left[h]);
                        }
                }
                uint32_t pk[QK / 2];
#pragma unroll
                for (int k = 0; k < QK / 2; ++k) {
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])),
                                                zf2, off2);
                    const float2 p = make_float2(fa::ptx::ex2_approx(x.x), fa::ptx::ex2_approx(x.y));
                    sum[k & 1] = __fadd2_rn(sum[k & 1], p);
                    pk[k] = pack16<false>(p.x, p.y);
                    if constexpr (!BF16) {
                        const float2 got = to_f32x2<false>(pk[k]);
                        left[i & 1][k] = pack16<false>(p.x - got.x, p.y - got.y);
                    }
                }
                if (i < 2) read(s, i);   // quarter 0 or 1 again
                store_p<QK / 2>(tS + BN / 2 + q * (QK / 2), pk);
                if constexpr (!BF16)
                    if (i >= 2) store_p<QK / 2>(tS + q * (QK / 2), left[i & 1]);
            }
            l = l * alpha + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) * pow2(-info.ev);
            fa::ptx::tmem_st_wait();
            fa::ptx::tc_fence_before_sync();
            fa::ptx::mbar_arrive(bar(&bars->p_full[sb]));
        }
        // -------------------------------------------------------- epilogue
        ok = ok && (n_tiles == 0 || wait_bar(bar(&bars->o_last), 0, abort));
        ok = __all_sync(0xffffffffu, ok);
        fa::ptx::tc_fence_after_sync();
        const float m = ref == kNegInf ? kNegInf : ref - kPHead;
        const long long slot = (static_cast<long long>(y - plan.whole) * splits + split) * TILES + t;
        if (ok && splits > 1 && real) a.part_ml[slot * kRowTile + r] = make_float2(m, n_tiles > 0 ? l : 0.f);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (ok) {
#pragma unroll 1
            for (int q = 0; q < NG; ++q) {
                uint32_t o[32];
                if (n_tiles > 0) {
                    fa::ptx::tmem_ld_32x32b_x32(tO + q * 32, o);
                    fa::ptx::tmem_ld_wait();
                    fa::ptx::reg_fence<32>(o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0;
                }
                if ((poison >> q) & 1u) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0x7fc00000u;
                }
                if (!real) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) {   // columns 0 4 1 5 2 6 3 7 of eight
                    const float4 e = make_float4(__uint_as_float(o[8 * i]), __uint_as_float(o[8 * i + 2]),
                                                 __uint_as_float(o[8 * i + 4]), __uint_as_float(o[8 * i + 6]));
                    const float4 g = make_float4(__uint_as_float(o[8 * i + 1]), __uint_as_float(o[8 * i + 3]),
                                                 __uint_as_float(o[8 * i + 5]), __uint_as_float(o[8 * i + 7]));
                    if (splits > 1) {
                        float4* po = reinterpret_cast<float4*>(a.part_o) + (slot * (D / 4) + q * 8 + 2 * i) * kRowTile + r;
                        po[0] = e;
                        po[kRowTile] = g;
                    } else {
                        uint16_t* dst = static_cast<uint16_t*>(a.o) +
                                        (static_cast<long long>(w.row0 + qi) * a.H + h) * D + q * 32 + 8 * i;
                        *reinterpret_cast<uint4*>(dst) =
                            make_uint4(pack16<BF16>(e.x * inv, e.y * inv), pack16<BF16>(e.z * inv, e.w * inv),
                                       pack16<BF16>(g.x * inv, g.y * inv), pack16<BF16>(g.z * inv, g.w * inv));
                    }
                }
            }
            if (splits == 1 && real && a.lse != nullptr)
                a.lse[(c.cu != nullptr ? w.row0 : b * a.lse_batch) + h * a.lse_head + qi] =
                    l == 0.f ? kNegInf : (m + log2f(l)) * 0.6931471805599453f;
        }
    }

    fa::ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == L::kMmaWarp) {
        fa::ptx::tc_fence_after_sync();
        fa::ptx::tmem_dealloc(tmem, 512);
    }
}

// Joins the splits of prompt_kernel: thread = row, a CTA 32 columns of a row tile.
template <int NG, bool BF16>
__global__ void __launch_bounds__(kRowTile) prompt_combine_kernel(Cache c, Attend a, PromptPlan plan) {
    using L = Prompt<NG>;
    constexpr int D = L::D, TILES = L::TILES, R = TILES * kRowTile;
    fa::ptx::grid_dependency_wait();
    const int q = static_cast<int>(blockIdx.x) % NG, yt = static_cast<int>(blockIdx.x) / NG;
    const int t = yt % TILES, y = plan.whole + yt / TILES;
    const int bh = y % (c.B * c.Hkv), b = bh / c.Hkv, head = bh - b * c.Hkv;
    const int tile = plan.tiles_most - 1 - y / (c.B * c.Hkv);
    const Work w = work_of(c, a, b, R, false);
    const int r = threadIdx.x, rho = tile * R + t * kRowTile + r;
    if (tile >= w.tiles || rho >= w.n * a.G) return;
    float m = kNegInf, l = 0.f;
    for (int s = 0; s < plan.splits; ++s) {
        const long long slot = (static_cast<long long>(y - plan.whole) * plan.splits + s) * TILES + t;
        m = fmaxf(m, __ldcg(a.part_ml + slot * kRowTile + r).x);
    }
    float4 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < plan.splits; ++s) {
        const long long slot = (static_cast<long long>(y - plan.whole) * plan.splits + s) * TILES + t;
        const float2 ml = __ldcg(a.part_ml + slot * kRowTile + r);
        const float f = ml.x == kNegInf ? 0.f : fa::ptx::ex2_approx(ml.x - m);
        l += f * ml.y;
        const float4* po = reinterpret_cast<const float4*>(a.part_o) + (slot * (D / 4) + q * 8) * kRowTile + r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 v = __ldcg(po + i * kRowTile);
            o[i].x += f * v.x;
            o[i].y += f * v.y;
            o[i].z += f * v.z;
            o[i].w += f * v.w;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        write_row<BF16>(c, a, w, b, D, rho, head, q * 32 + 4 * i, o[i], m, l, q == 0 && i == 0 && a.lse != nullptr);
}

}  // namespace kv4
