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
};

constexpr int kRowThreads = 256;   // 32 rows a block, 8 threads a row

// One row by 8 neighbouring threads: thread r holds elements 4 r .. 4 r + 3 of
// every group (8-byte loads, 64 contiguous bytes a group), the groups' extremes
// meet in three shuffles, and the thread's 2 NG bytes of codes leave in one
// store.  The four rows of a warp are four tokens of the same head, so that
// their scales fill whole sectors.
//
// Exactness: rint(x / s) is taken of x * (1 / s), which is off by less than
// 2^-21.  x has at most 11 significant bits and s at most 8, so x / s is
// either a tie k + 1/2 or at least 2^-13 away from one; rounding the product
// to multiples of 2^-14 first restores the ties and moves nothing across one.
template <int NG, bool BF16>
__global__ void __launch_bounds__(kRowThreads) write_kernel(Cache c, RowIo io) {
    constexpr int D = NG * kGroup;
    if (blockIdx.x == 0) check_sequences(c);
    const int sub = threadIdx.x & 7;                       // r
    const int tokens4 = (c.total + 3) >> 2;
    const long long warps = static_cast<long long>(tokens4) * 2 * c.Hkv;
    const long long w = static_cast<long long>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (w >= warps) return;
    const int head = static_cast<int>(w % c.Hkv);
    const long long w2 = w / c.Hkv;
    const int which = static_cast<int>(w2 & 1);
    const int t = static_cast<int>(w2 >> 1) * 4 + ((threadIdx.x >> 3) & 3);
    long long page = 0;
    int at = 0;
    RowPlace place = kRowSkip;
    uint2 x[NG];
    if (t < c.total) {
        const long long batch = c.cu != nullptr ? 0 : t / c.S, row = c.cu != nullptr ? t : t - batch * c.S;
        const uint16_t* src = which == 0
            ? static_cast<const uint16_t*>(io.k) + batch * io.k_batch + row * io.k_row + head * io.k_head
            : static_cast<const uint16_t*>(io.v) + batch * io.v_batch + row * io.v_row + head * io.v_head;
#pragma unroll
        for (int g = 0; g < NG; ++g) x[g] = *reinterpret_cast<const uint2*>(src + g * kGroup + sub * 4);
        place = place_of(c, t, &page, &at);
    } else {
#pragma unroll
        for (int g = 0; g < NG; ++g) x[g] = make_uint2(0, 0);
    }
    constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
    Words<NG> codes, scales;
    codes.clear();
    scales.clear();
    uint2 y[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        // (magnitude, first of equals, sign) in one word whose maximum is x_e
        const uint32_t e[4] = {x[g].x & 0xffffu, x[g].x >> 16, x[g].y & 0xffffu, x[g].y >> 16};
        uint32_t key = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t kj = ((e[j] & 0x7fffu) << 16) | ((31u - (sub * 4 + j)) << 1) | (e[j] >> 15);
            key = max(key, kj);
        }
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, m));
        const uint32_t mag = key >> 16;
        const float xe = to_f32x2<BF16>(mag | ((key & 1u) << 15)).x;
        uint32_t sb = pack16<true>(xe * -0.125f, 0.f) & 0xffffu;
        const bool finite = mag < kInf, some = finite && (sb & 0x7fffu) != 0;
        if (!some) sb = finite ? 0u : 0x7fc0u;
        const float s = bf16_bits(sb);
        // scales below 2^-64 are lifted by 2^96 (exactly) so that 1 / s is finite
        const float lift = fabsf(s) < 5.42101086e-20f ? 7.92281625e28f : 1.f;
        const float inv = some ? __frcp_rn(s * lift) : 0.f;
        const float2 a = to_f32x2<BF16>(x[g].x), b = to_f32x2<BF16>(x[g].y);
        const float v[4] = {a.x, a.y, b.x, b.y};
        uint32_t word = 0;
        float q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float u = some ? (v[j] * lift) * inv : 0.f;
            u = __fadd_rn(__fadd_rn(u, 768.f), -768.f);            // to multiples of 2^-14
            u = fminf(fmaxf(u, -8.f), 7.f);
            const float m = __fadd_rn(u, 12582912.f);              // to the nearest integer, ties to even
            word |= ((__float_as_uint(m) + 8u) & 15u) << (4 * j);
            q[j] = __fadd_rn(m, -12582912.f) * s;
        }
        codes.set(g, word);
        scales.set(g, sb);
        y[g] = make_uint2(pack16<BF16>(q[0], q[1]), pack16<BF16>(q[2], q[3]));
    }
    if (place == kRowOk) {
        const long long row = ((page * 2 + which) * c.Hkv + head) * c.P + at;
        codes.store(c.codes + row * (16 * NG) + sub * (2 * NG));
        if (sub == 0) scales.store(c.scales + row * NG);
    }
    void* out = which == 0 ? io.k_out : io.v_out;
    if (out != nullptr && place != kRowSkip) {
        uint16_t* dst = static_cast<uint16_t*>(out) + (static_cast<long long>(t) * c.Hkv + head) * D;
#pragma unroll
        for (int g = 0; g < NG; ++g)
            *reinterpret_cast<uint2*>(dst + g * kGroup + sub * 4) = place == kRowOk ? y[g] : make_uint2(0, 0);
    }
}

// -------------------------------------------------------------------- read
// The same shape backwards: 8 threads a row, 2 NG bytes of codes in and NG
// times 8 bytes out each.  A row before the sequence's first token is zeros;
// a row that is skipped stays as it was.
template <int NG, bool BF16>
__global__ void __launch_bounds__(kRowThreads) read_kernel(Cache c, RowIo io) {
    constexpr int D = NG * kGroup;
    if (blockIdx.x == 0) check_sequences(c);
    const int sub = threadIdx.x & 7;
    const int tokens4 = (c.total + 3) >> 2;
    const long long warps = static_cast<long long>(tokens4) * 2 * c.Hkv;
    const long long w = static_cast<long long>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (w >= warps) return;
    const int head = static_cast<int>(w % c.Hkv);
    const long long w2 = w / c.Hkv;
    const int which = static_cast<int>(w2 & 1);
    const int t = static_cast<int>(w2 >> 1) * 4 + ((threadIdx.x >> 3) & 3);
    if (t >= c.total) return;
    long long page = 0;
    int at = 0;
    const RowPlace place = place_of(c, t, &page, &at);
    if (place == kRowSkip) return;
    Words<NG> codes, scales;
    if (place == kRowOk) {
        const long long row = ((page * 2 + which) * c.Hkv + head) * c.P + at;
        codes.load(c.codes + row * (16 * NG) + sub * (2 * NG));
        scales.load(c.scales + row * NG);
    } else {
        codes.clear();
        scales.clear();
    }
    uint16_t* dst = static_cast<uint16_t*>(which == 0 ? io.k_out : io.v_out) +
                    (static_cast<long long>(t) * c.Hkv + head) * D;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const float s = scales.bf16(g);
        const uint32_t word = codes.get(g);
        float q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = static_cast<int>((word >> (4 * j)) & 15u) - 8;
            q[j] = place == kRowOk ? static_cast<float>(n) * s : 0.f;
        }
        *reinterpret_cast<uint2*>(dst + g * kGroup + sub * 4) =
            make_uint2(pack16<BF16>(q[0], q[1]), pack16<BF16>(q[2], q[3]));
    }
}

}  // namespace kv4
