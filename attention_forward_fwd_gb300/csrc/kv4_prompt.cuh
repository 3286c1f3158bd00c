// kv4_prompt.cuh -- attention of many query rows over the quantised cache
// (fa_kv4_attention for more than kDecodeRows query rows a K/V head: parts of
// prompts), on the tcgen05 tensor cores.
//
// A CTA takes one sequence, one K/V head and TILES x 128 of its query rows (the
// group's heads times the call's tokens, so that the heads of a group share the
// unpacked K and V), and walks over tiles of 64 keys:
//   unpack warps   codes and scales -> fp16 K and V tiles in shared memory
//   MMA warps      one a row tile: S = Q K^T, O += P V (fp32 in tensor memory);
//                  a single one spent half of its time between the products
//                  (waits, commits), with nothing queued
//   softmax warps  thread = row = TMEM lane: S -> P (fp16, over S), the
//                  running maximum, O's rescaling, the row sum
// Each row tile has two S buffers, and S runs two key tiles ahead: a softmax
// finds its next S ready, and the products are not on its way.  (With
// tiles of 128 keys and one buffer, S of a row tile had to wait for its P V and that
// for its P: softmax and products of a row tile took turns, 4500 cycles for
// 128 keys, although each of the two needs half of that.)  D <= 128: two row
// tiles; D > 128: one, as two O tiles do not fit the tensor memory.
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
constexpr int kKeys = 64;              // of a key tile, S's and P's
constexpr int kInfo = 4;               // descriptions of unpacked groups in flight
constexpr float kPHead = 7.f;          // P is held as p 2^kPHead, p <= 2^kLazy

template <int NG>
struct Prompt {
    static constexpr int D = NG * kGroup;
    static constexpr bool kWide = NG > 4;
    static constexpr int TILES = kWide ? 1 : 2;
    static constexpr int SUB = kWide ? 1 : 2;              // key tiles that are unpacked together, a group
    static constexpr int kSlots = 2;                       // groups of K, and of V, in shared memory
    static constexpr int kGroupKeys = SUB * kKeys;
    static constexpr int kBoxes = (NG + 1) / 2;            // 64 columns each
    static constexpr int N = kBoxes * 64;                  // columns of O (past D: zeros)
    static constexpr int kSoftWarps = 4 * TILES;
    static constexpr int kUnpackWarps = 8;
    static constexpr int kMmaWarp = kSoftWarps + kUnpackWarps;
    static constexpr int kThreads = (kMmaWarp + TILES) * 32;
    static constexpr int kQBox = kRowTile * 128, kBox = kKeys * 128;   // bytes
    static constexpr int kQTile = kBoxes * kQBox, kTile = kBoxes * kBox;
    static constexpr int kOffK = TILES * kQTile, kOffV = kOffK + kSlots * SUB * kTile,
                         kOffBar = kOffV + kSlots * SUB * kTile;
    static constexpr int kSmem = kOffBar + 2048 + 1024;    // and room to align
    // Registers a thread (D <= 128): 18 warps start with 96 each; 8 x 112 + 8 x 80
    // + 2 x 96 of the MMA warps is what they started with.
    static constexpr int kLaunchRegs = 96, kSoftRegs = 112, kUnpackRegs = 80;
    static_assert(kWide || kSoftWarps * kSoftRegs + kUnpackWarps * kUnpackRegs + TILES * kLaunchRegs <=
                               (kThreads / 32) * kLaunchRegs, "register split");
    static constexpr uint32_t kO = 256;                    // TMEM: S of row tile t at 128 t and 128 t + 64, O from here on
    static_assert(kO + TILES * N <= 512, "tensor memory");
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(kInfo > kSlots + 1, "descriptions outlive their groups");
};

struct TileInfo {
    int ek, ev;
    uint32_t missing;      // bit i: the i-th 16 keys are not there (a bad page)
    uint32_t nan;          // nonzero: some V scale is a NaN
};

struct PromptBars {
    uint64_t q_full, full[2][2], empty[2][2];   // [K or V][slot]
    uint64_t s_full[2][2], p_full[2][2];        // [row tile][buffer]
    uint64_t o_done[2], o_last[2], info[kInfo], drain[2];
    TileInfo tile[kInfo];
    uint32_t top[3][2], flags[3];        // of a group: largest scales of K and V; bit i: 16 keys
                                         // that are not there, bit 31: a NaN of V
    uint8_t nan_groups[kInfo][2 * kKeys];   // of each key of V
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
// another role gave up.  `nap`: nanoseconds to sleep between probes, for warps
// that have time, so that their asking takes no issue slots from the others.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort, bool heed = true,
                                         unsigned nap = 0) {
    if (fa::ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = fa::ptx::globaltimer();
    for (uint32_t n = 1;; ++n) {
        if (nap != 0) __nanosleep(nap);
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
    constexpr int D = L::D, TILES = L::TILES, BN = kKeys, NB = L::kBoxes, N = L::N, KS = L::kSlots, SUB = L::SUB, GK = L::kGroupKeys;
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
    // groups of keys that some row sees, and this split's share of them; the
    // last group's second tile is left out where no row sees it
    const int pos0 = w.len - w.n + tile * R / a.G, pos1 = w.len - w.n + (tile * R + rows - 1) / a.G;
    const int g_lo = first_key(pos0, a.window) / GK;
    const int g_all = pos1 >= 0 ? pos1 / GK + 1 - g_lo : 0;
    const int gb = g_lo + static_cast<int>(static_cast<long long>(g_all) * split / splits);        // first group
    const int n_groups = g_lo + static_cast<int>(static_cast<long long>(g_all) * (split + 1) / splits) - gb;
    const int jb = gb * SUB;                                                                       // first key tile
    const int n_tiles = max(0, min(n_groups * SUB, pos1 / kKeys + 1 - jb));

    if (threadIdx.x == 0) {
        fa::ptx::mbar_init(bar(&bars->q_full), R);
        for (int x = 0; x < 2; ++x) {
            for (int i = 0; i < KS; ++i) {
                fa::ptx::mbar_init(bar(&bars->full[x][i]), kUnpackWarps);
                fa::ptx::mbar_init(bar(&bars->empty[x][i]), TILES);
            }
            for (int i = 0; i < 2; ++i) {
                fa::ptx::mbar_init(bar(&bars->s_full[x][i]), 1);
                fa::ptx::mbar_init(bar(&bars->p_full[x][i]), kRowTile);
            }
            fa::ptx::mbar_init(bar(&bars->o_done[x]), 1);
            fa::ptx::mbar_init(bar(&bars->o_last[x]), 1);
            fa::ptx::mbar_init(bar(&bars->drain[x]), 1);
        }
        for (int i = 0; i < kInfo; ++i) fa::ptx::mbar_init(bar(&bars->info[i]), 1);
        for (int i = 0; i < 3; ++i) bars->top[i][0] = bars->top[i][1] = bars->flags[i] = 0;
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

    auto wait_warp = [&](uint32_t b_, uint32_t parity, bool heed = true, unsigned nap = 0) {
        return __all_sync(0xffffffffu, wait_bar(b_, parity, abort, heed, nap));
    };

    if (warp >= L::kMmaWarp) {
        // ------------------------------------------------------ MMA issue
        constexpr uint32_t kIdescS = fa::ptx::idesc_f16_f32(kRowTile, BN, false, false);
        constexpr uint32_t kIdescO = fa::ptx::idesc_f16_f32(kRowTile, N, false, true);
        const uint32_t hi = fa::ptx::sdesc_sw128_hi(1024);
        const uint32_t qlo = fa::ptx::sdesc_sw128_lo(sbase, 16);
        const uint32_t klo = fa::ptx::sdesc_sw128_lo(sbase + L::kOffK, 16);
        const uint32_t vlo = fa::ptx::sdesc_sw128_lo(sbase + L::kOffV, L::kBox);
        bool ok = n_tiles == 0 || wait_warp(bar(&bars->q_full), 0);
        const int t = warp - L::kMmaWarp;
        const uint32_t q = qlo + t * (L::kQTile / 16);
        // j = -2, -1: S of the first two key tiles alone
        for (int j = -2; j < n_tiles && ok; ++j) {
            if (j >= 0) {
                // O from P of key tile j (16 keys in 8 columns), and from what P's rounding left
                ok = wait_warp(bar(&bars->p_full[t][j & 1]), static_cast<uint32_t>((j >> 1) & 1));
                if (ok && j % SUB == 0)
                    ok = wait_warp(bar(&bars->full[1][j / SUB % KS]), static_cast<uint32_t>((j / (SUB * KS)) & 1));
                if (!ok) break;
                fa::ptx::tc_fence_after_sync();
                const uint32_t v = vlo + (j % (KS * SUB)) * (L::kTile / 16), p = tmem + t * 128 + (j & 1) * 64;
#pragma unroll
                for (int part = 0; part < (BF16 ? 1 : 2); ++part)
                    fa::ptx::mma_ts_x4_lo(tmem + L::kO + t * N, p + part * (BN / 2), v, hi, 8u, 128u, kIdescO,
                                          (j > 0 || part > 0) ? 1u : 0u);
            }
            const int i = j + 2;
            if (i < n_tiles) {
                // S of key tile i into buffer i % 2 (P of j lay there): K steps of 16 elements, 4 to a box
                if (i % SUB == 0) {
                    ok = wait_warp(bar(&bars->full[0][i / SUB % KS]), static_cast<uint32_t>((i / (SUB * KS)) & 1));
                    if (!ok) break;
                    fa::ptx::tc_fence_after_sync();
                }
                const uint32_t d = tmem + t * 128 + (i & 1) * 64, k = klo + (i % (KS * SUB)) * (L::kTile / 16);
#pragma unroll
                for (int x = 0; x < 2 * NG; x += 4) {
                    if (x + 4 <= 2 * NG) {
                        fa::ptx::mma_ss_x4_lo(d, q + (x / 4) * (L::kQBox / 16), k + (x / 4) * (L::kBox / 16), hi, 2u,
                                              kIdescS, x > 0 ? 1u : 0u);
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e)   // half a box is left
                            fa::ptx::mma_ss_warp_lo(d, q + (x / 4) * (L::kQBox / 16) + 2 * e,
                                                    k + (x / 4) * (L::kBox / 16) + 2 * e, hi, kIdescS, x + e > 0 ? 1u : 0u);
                    }
                }
                fa::ptx::tc_commit_warp(bar(&bars->s_full[t][i & 1]));
                if (i % SUB == SUB - 1) fa::ptx::tc_commit_warp(bar(&bars->empty[0][i / SUB % KS]));
            }
            if (j >= 0) {
                // (these report S of j + 2 along with P V of j)
                fa::ptx::tc_commit_warp(bar(&bars->o_done[t]));
                if (j % SUB == SUB - 1) fa::ptx::tc_commit_warp(bar(&bars->empty[1][j / SUB % KS]));
                if (j + 1 == n_tiles) fa::ptx::tc_commit_warp(bar(&bars->o_last[t]));
            }
        }
        // every MMA must be complete before the tensor memory is freed
        fa::ptx::tc_commit_warp(bar(&bars->drain[t]));
        wait_warp(bar(&bars->drain[t]), 0, false);
    } else if (warp >= L::kSoftWarps) {
        // ---------------------------------------------------------- unpack
        if constexpr (!WIDE) fa::ptx::setmaxnreg_dec<L::kUnpackRegs>();
        constexpr int CU = GK / 64;                        // units of this thread, of the 4 (c = 0 .. 3) of a key
        const int u = static_cast<int>(threadIdx.x) - L::kSoftWarps * 32;
        const int key = u % GK, c0 = u / GK * CU;          // its units: c0 .. c0 + CU - 1
        const int uw = u >> 5;
        const bool for_v = u / GK % 2 == 1;                // looks at V's scales (else at K's)
        const long long k_to_v = static_cast<long long>(c.Hkv) * c.P;   // rows
        if constexpr (NG % 2 == 1) {
            // the last box's right half is never written: columns of zeros
            for (int i = u; i < KS * SUB * BN * 4; i += kUnpackWarps * 32) {
                const int st = i / (BN * 4), k = (i / 4) % BN, chunk = 4 + (i & 3);
                *reinterpret_cast<uint4*>(smem + L::kOffV + st * L::kTile + (NB - 1) * L::kBox + k * 128 +
                                          ((chunk ^ (k & 7)) << 4)) = make_uint4(0, 0, 0, 0);
            }
        }
        const int* table = c.table + static_cast<long long>(b) * c.max_pages;
        // Rows and scales are asked for a tile ahead (a half tile's unpacking
        // is shorter than their latency), the page two.
        Words<2 * NG> raw[2][CU], ahead[2][CU];   // K's and V's
        Words<NG> ks, vs, ks2, vs2;
        bool gone = false, gone2 = false;
        int next = gb * GK + key;   // position that `pg`, `off` and `page` stand for
        int pg = next / c.P, off = next - pg * c.P, page = -1, at_group = 0;
        const int step_pg = GK / c.P, step_off = GK - step_pg * c.P;
        auto look_up = [&] { page = at_group < n_groups && next < w.len ? __ldg(table + pg) : -1; };
        // the page of group `at_group` is here: ask for its row and for the next page
        auto advance = [&] {
            const bool mine = at_group < n_groups && next < w.len;
            const bool ok = mine && page >= 0 && page < c.pages;
            gone2 = mine && !ok;
            if (gone2) report(kStatusBadPages);
            ks2.clear();
            vs2.clear();
#pragma unroll
            for (int i = 0; i < 2 * CU; ++i) ahead[i / CU][i % CU].clear();
            if (ok) {
                const long long row = (static_cast<long long>(page) * 2 * c.Hkv + head) * c.P + off;
                ks2.load_global(c.scales + row * NG);
                vs2.load_global(c.scales + (row + k_to_v) * NG);
                const uint8_t* codes = c.codes + row * (16 * NG) + c0 * (4 * NG);
#pragma unroll
                for (int i = 0; i < CU; ++i) {
                    ahead[0][i].load_global(codes + i * (4 * NG));
                    ahead[1][i].load_global(codes + k_to_v * (16 * NG) + i * (4 * NG));
                }
            }
            ++at_group;
            next += GK;
            pg += step_pg;
            off += step_off;
            if (off >= c.P) {
                off -= c.P;
                ++pg;
            }
            look_up();
        };
        look_up();
        advance();
        bool ok = true;
        int at3 = 0;   // g % 3
        for (int g = 0; g < n_groups; ++g) {
            ks = ks2;
            vs = vs2;
            gone = gone2;
#pragma unroll
            for (int i = 0; i < 2 * CU; ++i) raw[i / CU][i % CU] = ahead[i / CU][i % CU];
            advance();
            // ---- the group's largest finite scales (half of the warps look at K's,
            // half at V's), NaNs of V and holes
            uint32_t most = 0, nan_groups = 0;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const uint32_t x = (for_v ? vs.get(i) : ks.get(i)) & 0x7fffu;
                if (x >= 0x7f80u) nan_groups |= 1u << i;
                most = max(most, x < 0x7f80u ? x : 0u);
            }
            most = __reduce_max_sync(0xffffffffu, most);
            const uint32_t holes = __ballot_sync(0xffffffffu, gone);
            const bool any_nan = for_v && __any_sync(0xffffffffu, nan_groups != 0);
            // Slot g % kInfo is free: V of group g - 1 waited for P V of g - 1 - KS, so the
            // softmax is done with that group and those before it.
            if (u / GK == 1) bars->nan_groups[g % kInfo][key] = static_cast<uint8_t>(nan_groups);
            if (lane == 0) {
                atomicMax(&bars->top[at3][for_v ? 1 : 0], most);
                const uint32_t f = ((holes & 0xffffu) ? 1u : 0u) | ((holes >> 16) ? 2u : 0u);
                if (f != 0 || any_nan) atomicOr(&bars->flags[at3], f << (2 * (uw % (GK / 32))) | (any_nan ? 1u << 31 : 0u));
            }
            fa::ptx::named_barrier_sync(2, kUnpackWarps * 32);
            const uint32_t top_k = bars->top[at3][0], top_v = bars->top[at3][1], flags = bars->flags[at3];
            at3 = at3 == 2 ? 0 : at3 + 1;
            // (the slot of the group before is cleared below: everyone read it before this barrier)
            // largest scale 2^e (1 .. 2) -> 2^11 .. 2^12
            const int ek = max(static_cast<int>(top_k >> 7) - 127, -100) - 11;
            const int ev = max(static_cast<int>(top_v >> 7) - 127, -100) - 11;
            if (u == 0) {   // what the softmax has to know
                const int clear = at3 == 2 ? 0 : at3 + 1;
                bars->top[clear][0] = bars->top[clear][1] = bars->flags[clear] = 0;
                bars->tile[g % kInfo] = {ek, ev, flags & 0x7fffffffu, flags >> 31};
                fa::ptx::mbar_arrive(bar(&bars->info[g % kInfo]));
            }
            if (flags >> 31) {   // NaNs of V stay out of the products
#pragma unroll
                for (int i = 0; i < NG; ++i)
                    if ((vs.get(i) & 0x7fffu) >= 0x7f80u) vs.set(i, 0);
            }
            // ---- K, then V, each once its slot is free
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
                if (g >= KS)
                    ok = ok && wait_warp(bar(&bars->empty[x][g % KS]), static_cast<uint32_t>((g / KS - 1) & 1), true, 100);
                if (ok) {
                    uint8_t* to = smem + (x == 0 ? L::kOffK : L::kOffV) + (g % KS * SUB + key / kKeys) * L::kTile;
                    const float down = pow2(x == 0 ? -ek : -ev);
#pragma unroll
                    for (int i = 0; i < CU; ++i)
                        unpack_unit<NG, L::kBox>(raw[0][i], ks, down, c0 + i, key % kKeys, to);
                    fa::ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) fa::ptx::mbar_arrive(bar(&bars->full[x][g % KS]));
                }
                ks = vs;
#pragma unroll
                for (int i = 0; i < CU; ++i) raw[0][i] = raw[1][i];
            }
        }
    } else {
        // --------------------------------------------------------- softmax
        if constexpr (!WIDE) fa::ptx::setmaxnreg_inc<L::kSoftRegs>();
        const int t = warp >> 2;                                      // row tile
        const int r = static_cast<int>(threadIdx.x) & 127;            // row of the tile, TMEM lane
        const int row = t * kRowTile + r, rho = tile * R + row;
        const bool real = row < rows;
        const int qi = rho / a.G, h = head * a.G + rho - qi * a.G;
        // rows past the last one see everything (their Q is 0), so that they need no mask
        const int pos = real ? w.len - w.n + qi : 0x7fffffff;
        const int first = real ? first_key(pos, a.window) : 0;
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
            const int g = j / SUB;
            ok = ok && (j % SUB != 0 || wait_bar(bar(&bars->info[g % kInfo]), static_cast<uint32_t>((g / kInfo) & 1), abort)) &&
                 wait_bar(bar(&bars->s_full[t][j & 1]), static_cast<uint32_t>((j >> 1) & 1), abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            fa::ptx::tc_fence_after_sync();
            const TileInfo info = bars->tile[g % kInfo];
            const uint32_t tS = tmem + lane_off + t * 128 + (j & 1) * 64;
            const int kv0 = (jb + j) * BN;
            const uint32_t missing = info.missing >> (j % SUB * (kKeys / 16));
            const bool edge = __any_sync(0xffffffffu, kv0 + BN - 1 > pos || kv0 < first || (missing & 15u) != 0);
            const float zf = f * pow2(info.ek), ev = static_cast<float>(info.ev);
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
            uint32_t sv[BN];
            fa::ptx::tmem_ld_32x32b_x32(tS, sv);
            fa::ptx::tmem_ld_32x32b_x32(tS + 32, sv + 32);
            fa::ptx::tmem_ld_wait();
            fa::ptx::reg_fence<BN>(sv);
            float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
            for (int k = 0; k < BN; k += 8)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mx[i] = fa::ptx::fmax3(mx[i], __uint_as_float(sv[k + 2 * i]), __uint_as_float(sv[k + 2 * i + 1]));
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
                // S of this tile came after P V of the tile two before; the one before has to be waited for
                ok = wait_bar(bar(&bars->o_done[t]), static_cast<uint32_t>((j - 1) & 1), abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                fa::ptx::tc_fence_after_sync();
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
                    if (key <= pos && key >= first) poison |= bars->nan_groups[g % kInfo][j % SUB * kKeys + k];
                }
            }
            const float off = ev + kPHead - (ref == kNegInf ? 0.f : ref);
            const float2 zf2 = make_float2(zf, zf), off2 = make_float2(off, off);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            // P in the buffer's first half, what its rounding left in the second
#pragma unroll
            for (int q = 0; q < BN / 32; ++q) {
                uint32_t pk[16], left[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(sv[q * 32 + 2 * k]),
                                                            __uint_as_float(sv[q * 32 + 2 * k + 1])), zf2, off2);
                    const float2 p = make_float2(fa::ptx::ex2_approx(x.x), fa::ptx::ex2_approx(x.y));
                    sum[k & 1] = __fadd2_rn(sum[k & 1], p);
                    pk[k] = pack16<false>(p.x, p.y);
                    if constexpr (!BF16) {
                        const float2 got = to_f32x2<false>(pk[k]);
                        left[k] = pack16<false>(p.x - got.x, p.y - got.y);
                    }
                }
                fa::ptx::tmem_st_32x32b_x16(tS + q * 16, pk);
                if constexpr (!BF16) fa::ptx::tmem_st_32x32b_x16(tS + BN / 2 + q * 16, left);
            }
            l = l * alpha + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) * pow2(-info.ev);
            fa::ptx::tmem_st_wait();
            fa::ptx::tc_fence_before_sync();
            fa::ptx::mbar_arrive(bar(&bars->p_full[t][j & 1]));
        }
        // -------------------------------------------------------- epilogue
        ok = ok && (n_tiles == 0 || wait_bar(bar(&bars->o_last[t]), 0, abort));
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
