// kv4_cache.cuh -- the quantised K/V cache: its layout, and the kernels that
// write rows into it (fa_kv4_write) and read them back (fa_kv4_read).
//
// A row is the D values of one token and one K or V head.  It is cut in
// NG = D / 32 groups of 32 neighbours; a group has the scale s = -x_e / 8
// rounded to bf16 (x_e: its element of the largest magnitude, the first of
// equals) and each element the code n = clamp(rint(x / s), -8, 7) + 8, which
// stands for s (n - 8).  The signed scale puts x_e on the code 0, so that all
// sixteen codes are used (12 % less rms error on normal rows than s = |x_e| / 7).
// A group of zeros has s = 0 and the codes 8; one with an infinity or a NaN
// has s = NaN and the codes 8, and reads back as NaN.
//
// s has 8 significant bits and n - 8 three (or is a power of two), so
// s (n - 8) has at most 11: it is exact in fp16 wherever its exponent is in
// range.  The attention kernels rely on that.
//
// Row layout: the code of element 32 g + 4 r + j (r < 8, j < 4) is bits
// 4 j .. 4 j + 3 of the row's 16-bit word r * NG + g.  A thread that owns "r"
// therefore finds 4 elements of every group in 2 NG contiguous bytes, which
// is what the matrix fragments of the attention kernel want (all groups at
// once, each group's partial product apart from the others).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "sm103_ptx.cuh"

namespace kv4 {

constexpr int kGroup = 32;              // elements that share a scale
constexpr int kStatusTimeout = 4;       // the C-ABI's codes
constexpr int kStatusBadSeqlens = 5;
constexpr int kStatusBadPages = 7;

// Status word of these kernels; fa_device_status() reports it with the
// attention forward's own.
__device__ int g_kv4_status;

__device__ __forceinline__ void report(int code) { atomicCAS(&g_kv4_status, 0, code); }

// Which rows of which sequence a call concerns, and where the cache holds
// them.  Sequence b has lens[b] tokens in the cache and the call's n_b rows
// are its last n_b tokens: n_b = cu[b + 1] - cu[b] rows from row cu[b] of the
// packed tensors, or S rows from row b S when cu is null.
struct Cache {
    uint8_t* codes;         // [pages, 2, Hkv, P, 16 NG]
    uint16_t* scales;       // [pages, 2, Hkv, P, NG] bf16
    const int* table;       // [B, max_pages]
    const int* lens;        // [B]
    const int* cu;          // [B + 1] or null
    int B, S, total;        // S: rows a sequence (cu null), else the most; total: rows of the call
    int pages, max_pages, P, Hkv;
};

struct Seq {
    int n;        // rows of the call
    int len;      // tokens in the cache
    int row0;     // first row of the call's tensors
    int status;   // 0, or why the sequence is skipped
};

__device__ __forceinline__ Seq sequence(const Cache& c, int b) {
    Seq s;
    s.len = __ldg(c.lens + b);
    if (c.cu != nullptr) {
        const int r0 = __ldg(c.cu + b), r1 = __ldg(c.cu + b + 1);
        s.row0 = r0;
        s.n = r1 - r0;
        s.status = (r0 < 0 || r1 < r0 || r1 > c.total || s.n > c.S) ? kStatusBadSeqlens : 0;
    } else {
        s.row0 = b * c.S;
        s.n = c.S;
        s.status = 0;
    }
    if (s.status == 0 && (s.len < 0 || s.len > static_cast<long long>(c.max_pages) * c.P))
        s.status = kStatusBadPages;
    if (s.status != 0) s.n = 0;
    return s;
}

// The sequence that holds row t of the call, or -1 (rows behind the last one).
// With offsets that do not rise the search may end on a sequence that does
// not hold the row; the caller checks.
__device__ __forceinline__ int sequence_of(const Cache& c, int t) {
    if (c.cu == nullptr) return t / c.S;
    int lo = 0, hi = c.B;   // the last b in [0, B) with cu[b] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(c.cu + mid) <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// One block of a launch looks at every sequence, so that a bad one is reported
// whether or not some row's search ends on it.
__device__ __forceinline__ void check_sequences(const Cache& c) {
    for (int b = threadIdx.x; b < c.B; b += blockDim.x) {
        const int status = sequence(c, b).status;
        if (status != 0) report(status);
    }
}

enum RowPlace { kRowSkip = 0, kRowEmpty = 1, kRowOk = 2 };

// Where the cache holds row t's K (head 0): the token's index in units of
// (page, K or V, head, place).  kRowEmpty: the row lies before the sequence's
// first token (n_b > lens[b]); kRowSkip: there is nothing to do for it.
__device__ __forceinline__ RowPlace place_of(const Cache& c, int t, long long* page, int* at) {
    const int b = sequence_of(c, t);
    const Seq s = sequence(c, b);
    if (s.status != 0) return kRowSkip;   // reported by check_sequences
    const int i = t - s.row0;
    if (i < 0 || i >= s.n) return kRowSkip;
    const int pos = s.len - s.n + i;
    if (pos < 0) return kRowEmpty;
    const int pg = __ldg(c.table + static_cast<long long>(b) * c.max_pages + pos / c.P);
    if (pg < 0 || pg >= c.pages) {
        report(kStatusBadPages);
        return kRowSkip;
    }
    *page = pg;
    *at = pos % c.P;
    return kRowOk;
}

// ------------------------------------------------------------- 16-bit types
template <bool BF16>
__device__ __forceinline__ float2 to_f32x2(uint32_t u) {
    if constexpr (BF16) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    } else {
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
    }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t r;
    if constexpr (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float bf16_bits(uint32_t lo16) { return __uint_as_float(lo16 << 16); }

// N 16-bit words, two to a register, read and written in the widest accesses
// that their alignment (the largest power of two that divides 2 N, at most 16) allows.
template <int N>
struct Words {
    static constexpr int kRegs = (N + 1) / 2;
    uint32_t u[kRegs];
    using Unit = std::conditional_t<N % 8 == 0, uint4, std::conditional_t<N % 4 == 0, uint2, uint32_t>>;

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kRegs; ++i) u[i] = 0;
    }
    __device__ __forceinline__ void load(const void* p) {
        if constexpr (N % 2 == 0) {
#pragma unroll
            for (int i = 0; i < N * 2 / static_cast<int>(sizeof(Unit)); ++i) {
                const Unit v = static_cast<const Unit*>(p)[i];
                __builtin_memcpy(u + i * (sizeof(Unit) / 4), &v, sizeof(Unit));
            }
        } else {
            clear();
#pragma unroll
            for (int i = 0; i < N; ++i)
                u[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << (16 * (i & 1));
        }
    }
    // the same from memory that nothing writes during the launch
    __device__ __forceinline__ void load_global(const void* p) {
        if constexpr (N % 2 == 0) {
#pragma unroll
            for (int i = 0; i < N * 2 / static_cast<int>(sizeof(Unit)); ++i) {
                const Unit v = __ldg(static_cast<const Unit*>(p) + i);
                __builtin_memcpy(u + i * (sizeof(Unit) / 4), &v, sizeof(Unit));
            }
        } else {
            clear();
#pragma unroll
            for (int i = 0; i < N; ++i)
                u[i / 2] |= static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p) + i)) << (16 * (i & 1));
        }
    }
    __device__ __forceinline__ void store(void* p) const {
        if constexpr (N % 2 == 0) {
#pragma unroll
            for (int i = 0; i < N * 2 / static_cast<int>(sizeof(Unit)); ++i) {
                Unit v;
                __builtin_memcpy(&v, u + i * (sizeof(Unit) / 4), sizeof(Unit));
                static_cast<Unit*>(p)[i] = v;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(get(i));
        }
    }
    __device__ __forceinline__ uint32_t get(int i) const { return (i & 1) ? u[i / 2] >> 16 : u[i / 2] & 0xffffu; }
    __device__ __forceinline__ void set(int i, uint32_t w) {   // w < 2^16
        u[i / 2] = (i & 1) ? (u[i / 2] & 0xffffu) | (w << 16) : (u[i / 2] & 0xffff0000u) | w;
    }
    // word i from the low or the high half of w
    __device__ __forceinline__ void set_half(int i, uint32_t w, bool high) {
        u[i / 2] = __byte_perm(u[i / 2], w, (i & 1) ? (high ? 0x7610u : 0x5410u) : (high ? 0x3276u : 0x3254u));
    }
    // word i as a bfloat16
    __device__ __forceinline__ float bf16(int i) const {
        return __uint_as_float((i & 1) ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
    }
};

// Word i of a below word j of b.
template <int N, int M>
__device__ __forceinline__ uint32_t join_words(const Words<N>& a, int i, const Words<M>& b, int j) {
    return __byte_perm(a.u[i / 2], b.u[j / 2], ((i & 1) ? 0x0032u : 0x0010u) | ((j & 1) ? 0x7600u : 0x5400u));
}

// ------------------------------------------------------------------- write
struct RowIo {
    // 16-bit tensors of the call's rows; strides in elements
    const void* k;
    const void* v;
    long long k_batch, k_row, k_head, v_batch, v_row, v_head;
    void* k_out;     // contiguous [rows, Hkv, D]; may be null in a write
    void* v_out;
    int wide;        // a write's addresses allow 16-byte accesses (else 8)
    int per;         // rows a warp takes of each of its tokens, at most kRows
};

// Both kernels: a warp takes 32 / LANES tokens, LANES neighbouring threads
// each, and up to kRows<NG, LANES> of their rows (K or V of a head) one after the other: where
// a token lies is found once for all of them, while the first row's loads are
// under way.  The rows of an access are tokens of the same head, so that their
// scales fill whole sectors.
//  * read: 8 threads a row, thread r has elements 4 r .. 4 r + 3 of every group.
//  * write: 4 threads a row, thread c has elements 8 c .. 8 c + 7, because the search
//    for a group's extreme is paid once a thread and group, whatever they hold.
// CTAs of 128 threads, not 256: these have no more in common, and smaller ones follow one
// another more evenly (D = 128, prompts of 37000 tokens, 8 heads: write 69.7 -> 61.7 us,
// 84 % of the copy bandwidth; 65536 tokens of 8 rows of 64: 27.6 -> 24.2).
constexpr int kRowThreads = 128;
constexpr int kWriteLanes = 4, kReadLanes = 8;
// A write holds one row and the next; a read all of them, which pays for longer
// (D = 128: read of 80000 tokens 69.7 us with 4 rows, 67.5 with 8; the write above 61.7, 63.5).
template <int NG, int LANES>
constexpr int kRows = (NG <= 2 ? 8 : NG <= 4 ? 4 : 2) * (LANES == kReadLanes ? 2 : 1);

// Which rows a warp takes.
struct RowShare {
    int t, first, n;      // token, first row (K's heads, then V's), rows
};
template <int LANES>
__device__ __forceinline__ bool row_share(const Cache& c, int per, RowShare* s) {
    constexpr int TOK = 32 / LANES;
    const int rows = 2 * c.Hkv, chunks = (rows + per - 1) / per;
    const long long w = static_cast<long long>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
    const long long group = w / chunks;
    if (group >= (static_cast<long long>(c.total) + TOK - 1) / TOK) return false;
    s->first = static_cast<int>(w - group * chunks) * per;
    s->n = min(per, rows - s->first);
    const long long t = group * TOK + (threadIdx.x & 31) / LANES;
    s->t = static_cast<int>(t < c.total ? t : c.total);   // total: none
    return true;
}

template <bool BF16>
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {   // a NaN wins
    uint32_t r;
    if constexpr (BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <bool BF16>
__device__ __forceinline__ uint32_t min16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (BF16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A group's scale (its bits) from its elements x (this thread's eight, two a
// word), the same in the group's 4 threads.
template <bool BF16>
__device__ __forceinline__ uint32_t group_scale(const uint32_t* x, int sub) {
    // the largest x in the low half, the largest -x in the high half
    const uint32_t up = max16x2<BF16>(max16x2<BF16>(x[0], x[1]), max16x2<BF16>(x[2], x[3]));
    const uint32_t down = min16x2<BF16>(min16x2<BF16>(x[0], x[1]), min16x2<BF16>(x[2], x[3])) ^ 0x80008000u;
    uint32_t m = max16x2<BF16>(__byte_perm(up, down, 0x5410), __byte_perm(up, down, 0x7632));
#pragma unroll
    for (int i = 1; i < kWriteLanes; i <<= 1) m = max16x2<BF16>(m, __shfl_xor_sync(0xffffffffu, m, i));
    const float2 top = to_f32x2<BF16>(m);
    float xe = top.x > top.y ? top.x : -top.y;   // NaN if there is one
    const bool tie = top.x == top.y && top.x != 0.f;
    if (__any_sync(0xffffffffu, tie)) {
        // both signs at the largest magnitude: the first of them counts
        uint32_t key = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t v = (j & 1) ? x[j / 2] >> 16 : x[j / 2] & 0xffffu;
            key = max(key, ((v & 0x7fffu) << 16) | ((31u - (sub * 8 + j)) << 1) | (v >> 15));
        }
#pragma unroll
        for (int i = 1; i < kWriteLanes; i <<= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, i));
        if (tie && (key & 1u) == 0) xe = top.x;
    }
    const uint32_t sb = pack16<true>(xe * -0.125f, 0.f) & 0xffffu;
    return (sb & 0x7fffu) >= 0x7f80u ? 0x7fc0u : (sb & 0x7fffu) == 0 ? 0u : sb;
}

// ------------------------------------------------------------------- write
// Exactness: rint(x / s) is taken of x times an approximate 1 / s, which is off
// by less than 2^-20.  x has at most 11 significant bits and s at most 8, so x / s is
// either a tie k + 1/2 or at least 2^-13 away from one; rounding the product
// to multiples of 2^-14 first (768 is added to it, in the same instruction)
// restores the ties and moves nothing across one.  x / s is at least -8 (1 + 2^-8),
// which rounds to -8: only 7 needs a clamp, but for subnormal scales, whose own
// rounding is coarser.
//
// Bound by DRAM at D = 128 when the values come back, by instructions where rows are
// narrow and they do not (figures above).  The loop over the rows is not unrolled, for the
// instruction cache's sake; the next row is loaded ahead.
template <int NG, bool BF16, bool VALUES>
__global__ void __launch_bounds__(kRowThreads) write_kernel(Cache c, RowIo io) {
    constexpr int D = NG * kGroup;
    if (blockIdx.x == 0) check_sequences(c);
    RowShare own;
    if (!row_share<kWriteLanes>(c, io.per, &own)) return;
    const int sub = threadIdx.x & (kWriteLanes - 1);       // c
    const bool here = own.t < c.total;
    const uint16_t *k, *v;
    {
        const long long batch = c.cu != nullptr || !here ? 0 : own.t / c.S, row = here ? own.t - batch * c.S : 0;
        k = static_cast<const uint16_t*>(io.k) + batch * io.k_batch + row * io.k_row + sub * 8;
        v = static_cast<const uint16_t*>(io.v) + batch * io.v_batch + row * io.v_row + sub * 8;
    }
    uint4 next[NG];
    auto load = [&](int i) {
        const int y = own.first + i;
        const uint16_t* src = y < c.Hkv ? k + y * io.k_head : v + (y - c.Hkv) * io.v_head;
        const bool on = i < own.n && here;
        if (io.wide) {
#pragma unroll
            for (int g = 0; g < NG; ++g)
                next[g] = on ? *reinterpret_cast<const uint4*>(src + g * kGroup) : make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                next[g] = make_uint4(0, 0, 0, 0);
                if (on) {
                    const uint2 lo = *reinterpret_cast<const uint2*>(src + g * kGroup);
                    const uint2 hi = *reinterpret_cast<const uint2*>(src + g * kGroup + 4);
                    next[g] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
            }
        }
    };
    load(0);
    long long page = 0;
    int at = 0;
    const RowPlace place = here ? place_of(c, own.t, &page, &at) : kRowSkip;
#pragma unroll 1
    for (int i = 0; i < own.n; ++i) {
        const int y = own.first + i;
        uint4 x[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) x[g] = next[g];
        load(i + 1);
        Words<2 * NG> codes;
        Words<NG> scales;
        codes.clear();
        scales.clear();
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const uint32_t e[4] = {x[g].x, x[g].y, x[g].z, x[g].w};
            const uint32_t sb = group_scale<BF16>(e, sub);
            const float s = bf16_bits(sb);
            const bool tiny = (sb & 0x7fffu) < 0x80u;      // zero or subnormal
            float inv;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
            if (tiny) inv = 0.f;
            float2 t[4];   // 768 and x / s, to multiples of 2^-14
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = __ffma2_rn(to_f32x2<BF16>(e[j]), make_float2(inv, inv), make_float2(768.f, 768.f));
            if (__any_sync(0xffffffffu, tiny && sb != 0)) {
                const float lifted = __frcp_rn(s * 7.92281625e28f);   // 2^96
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = to_f32x2<BF16>(e[j]);
                    if (tiny && sb != 0)
                        t[j] = make_float2(__fadd_rn(fmaxf(f.x * 7.92281625e28f * lifted, -8.f), 768.f),
                                           __fadd_rn(fmaxf(f.y * 7.92281625e28f * lifted, -8.f), 768.f));
                }
            }
            uint32_t pair[4];   // codes 2 j and 2 j + 1, 16 bits each
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // 3 2^22 + 8 and the nearest integer, ties to even: the low bits are the code, or 16
                float2 r = __fadd2_rn(t[j], make_float2(12582152.f, 12582152.f));
                if constexpr (VALUES) {
                    r = make_float2(fminf(r.x, 12582927.f), fminf(r.y, 12582927.f));
                    const float2 n = __fadd2_rn(r, make_float2(-12582920.f, -12582920.f));
                    o[j] = pack16<BF16>(n.x * s, n.y * s);
                }
                pair[j] = __byte_perm(__float_as_uint(r.x), __float_as_uint(r.y), 0x5410);
                if constexpr (!VALUES) pair[j] = __vminu2(pair[j], 0x000f000fu);
            }
            // a code a byte; then two in bytes 0 and 2
            const uint32_t a0 = __byte_perm(pair[0], pair[1], 0x6420), a1 = __byte_perm(pair[2], pair[3], 0x6420);
            const uint32_t b0 = a0 + (a0 >> 4), b1 = a1 + (a1 >> 4);
            uint32_t both = __byte_perm(b0, b1, 0x6420);       // r = 2 c below r = 2 c + 1
            if (sb == 0x7fc0u) both = 0x88888888u;
            codes.set_half(g, both, false);
            codes.set_half(NG + g, both, true);
            scales.set(g, sb);
            if constexpr (VALUES) x[g] = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (place == kRowOk) {
            const long long row = (page * 2 * c.Hkv + y) * c.P + at;   // K's heads, then V's
            codes.store(c.codes + row * (16 * NG) + sub * (4 * NG));
            if (sub == 0) scales.store(c.scales + row * NG);
        }
        if constexpr (VALUES) {
            if (place != kRowSkip) {
                uint16_t* to = static_cast<uint16_t*>(y < c.Hkv ? io.k_out : io.v_out) +
                               (static_cast<long long>(own.t) * c.Hkv + (y < c.Hkv ? y : y - c.Hkv)) * D + sub * 8;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint4 o = place == kRowOk ? x[g] : make_uint4(0, 0, 0, 0);
                    if (io.wide) {
                        *reinterpret_cast<uint4*>(to + g * kGroup) = o;
                    } else {
                        *reinterpret_cast<uint2*>(to + g * kGroup) = make_uint2(o.x, o.y);
                        *reinterpret_cast<uint2*>(to + g * kGroup + 4) = make_uint2(o.z, o.w);
                    }
                }
            }
        }
    }
}

// -------------------------------------------------------------------- read
// The same shape backwards.  Two codes at a time become n - 8 in the result's
// own type, 2^k + n (k = 7 in bf16, 10 in fp16) less 2^k + 8, and are multiplied by
// the scale there: in bf16 that is the one rounding; in fp16 it is exact, or the
// one rounding to a subnormal, while the scale is a normal fp16 (others
// go through fp32).  A row before the sequence's first token is zeros; a row that is
// skipped stays as it was.
template <bool BF16>
__device__ __forceinline__ uint32_t code_values(uint32_t pair, uint32_t s2) {
    const uint32_t y = (pair & 0x000f000fu) | (BF16 ? 0x43004300u : 0x64006400u);
    uint32_t r;
    if constexpr (BF16) {
        asm("{\n\t.reg .b32 t;\n\tsub.rn.bf16x2 t, %1, %2;\n\tmul.rn.bf16x2 %0, t, %3;\n\t}"
            : "=r"(r) : "r"(y), "r"(0x43084308u), "r"(s2));
    } else {
        asm("{\n\t.reg .b32 t;\n\tsub.rn.f16x2 t, %1, %2;\n\tmul.rn.f16x2 %0, t, %3;\n\t}"
            : "=r"(r) : "r"(y), "r"(0x64086408u), "r"(s2));
    }
    return r;
}

template <int NG, bool BF16>
__global__ void __launch_bounds__(kRowThreads) read_kernel(Cache c, RowIo io) {
    constexpr int D = NG * kGroup, N = kRows<NG, kReadLanes>;
    if (blockIdx.x == 0) check_sequences(c);
    RowShare own;
    if (!row_share<kReadLanes>(c, io.per, &own) || own.t >= c.total) return;
    const int sub = threadIdx.x & 7;
    long long page = 0;
    int at = 0;
    const RowPlace place = place_of(c, own.t, &page, &at);
    if (place == kRowSkip) return;
    Words<NG> codes[N], scales[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        codes[i].clear();
        scales[i].clear();
        if (i < own.n && place == kRowOk) {
            const int y = own.first + i;   // K's heads, then V's: as they lie in the page
            const long long row = (page * 2 * c.Hkv + y) * c.P + at;
            codes[i].load_global(c.codes + row * (16 * NG) + sub * (2 * NG));
            scales[i].load_global(c.scales + row * NG);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (i >= own.n) break;
        const int y = own.first + i, which = y >= c.Hkv ? 1 : 0, head = y - which * c.Hkv;
        uint16_t* dst = static_cast<uint16_t*>(which == 0 ? io.k_out : io.v_out) +
                        (static_cast<long long>(own.t) * c.Hkv + head) * D + sub * 4;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const uint32_t w = codes[i].get(g), t = w | (w << 12);
            uint2 out;
            const uint32_t sb = scales[i].get(g);
            bool plain = true;
            uint32_t s2 = sb | (sb << 16);
            if constexpr (!BF16) {
                const float s = bf16_bits(sb);
                s2 = pack16<false>(s, s);
                const uint32_t mag = sb & 0x7fffu;
                plain = mag == 0 || (mag >= 0x3880u && mag < 0x4780u);     // 2^-14 <= |s| < 2^16
            }
            if (plain) {
                out = make_uint2(code_values<BF16>(t, s2), code_values<BF16>(t >> 8, s2));
            } else {
                const float s = bf16_bits(sb);
                float q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = static_cast<float>(static_cast<int>((w >> (4 * j)) & 15u) - 8) * s;
                out = make_uint2(pack16<BF16>(q[0], q[1]), pack16<BF16>(q[2], q[3]));
            }
            if (place != kRowOk) out = make_uint2(0, 0);
            *reinterpret_cast<uint2*>(dst + g * kGroup) = out;
        }
    }
}

}  // namespace kv4
