// rotary.cuh -- rotary positions with several axes (fa_rotary).
//
// Frequency f of a token turns one pair of a head's elements by the angle
// position[axis[f]] * inv_freq[f]:  (x, y) -> (x cos - y sin, x sin + y cos);
// the pair is (f, f + F) of the first 2 F elements, or (2 f, 2 f + 1) when
// interleaved.  Elements past 2 F are copied.
//
// The angle: far positions need more than fp32's 24 bits (position 10^6 at
// frequency 1 is off by 0.03 rad in fp32), so it is taken in turns,
// t = p (inv_freq / 2 pi), with the factor as the sum of two floats and the
// product's rounding error recovered by an FMA; t's whole turns then drop out
// exactly.  Each angle is worked out once a token for all heads.
//
// Bound by DRAM (2 bytes in, 2 bytes out an element).  A CTA takes a few tokens
// of all heads; each thread loads its vectors before the angles are worked
// out, so that the two overlap.
#pragma once

#include "kv4_cache.cuh"

namespace rot {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;          // units a thread has in flight
constexpr int kMaxFreqs = 128;
constexpr int kMaxTokens = 16;      // of a CTA
constexpr int kStatusBadAxis = 8;

struct Rotary {
    const void* x[2];               // queries, keys (second may be absent)
    void* y[2];
    long long x_row[2], x_head[2], y_row[2], y_head[2];   // strides in elements
    int heads[2];
    const int* pos;                 // [T, A]
    const double* inv_freq;         // [F]
    const int* axes;                // [F]
    int T, A, F, D, inverse, tokens;   // tokens: of a CTA
};

__device__ __forceinline__ float2 cos_sin(int p, double inv_freq) {
    const double turns = inv_freq * 0.15915494309189533577;   // 1 / 2 pi
    const float fh = static_cast<float>(turns), fl = static_cast<float>(turns - static_cast<double>(fh));
    const int p_hi = p & ~0xffff, p_lo = p & 0xffff;          // both exact in fp32
    const float a = static_cast<float>(p_hi), b = static_cast<float>(p_lo);
    const float ta = a * fh, tb = b * fh;
    const float ea = fmaf(a, fh, -ta), eb = fmaf(b, fh, -tb);
    float u = (ta - rintf(ta)) + (tb - rintf(tb));
    u -= rintf(u);
    u += (ea + eb) + (a * fl + b * fl);
    float s, c;
    sincospif(2.f * u, &s, &c);
    return make_float2(c, s);
}

// A unit: VEC pairs of one head.  Interleaved pairs lie in 2 VEC contiguous
// elements, split ones in VEC and VEC.  VEC = 8 where F, D and the strides are
// multiples of 8 (16-byte accesses; 2 x 8 or 1 x 16 elements), else VEC = 1.
template <int VEC, bool INTER, bool BF16>
__global__ void __launch_bounds__(kThreads) rotary_kernel(Rotary p) {
    extern __shared__ float2 cs[];   // [tokens][F]
    const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0);
    const int heads = p.heads[0] + p.heads[1];
    const int per_head = p.F / VEC + (p.D - 2 * p.F + 2 * VEC - 1) / (2 * VEC);   // rotated, copied
    const int units = nt * heads * per_head;
    for (int u0 = threadIdx.x; u0 < units || u0 - static_cast<int>(threadIdx.x) == 0; u0 += kThreads * kUnroll) {
        kv4::Words<VEC> lo[kUnroll], hi[kUnroll];
        int at[kUnroll], tok[kUnroll], which[kUnroll], head[kUnroll];
        bool two[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int u = u0 + k * kThreads;
            if (u >= units) continue;
            const int th = u / per_head;
            at[k] = u - th * per_head;
            tok[k] = th / heads;
            head[k] = th - tok[k] * heads;
            which[k] = head[k] >= p.heads[0];
            if (which[k]) head[k] -= p.heads[0];
            const uint16_t* src = static_cast<const uint16_t*>(p.x[which[k]]) +
                                  (t0 + tok[k]) * p.x_row[which[k]] + head[k] * p.x_head[which[k]];
            const bool turn = at[k] < p.F / VEC;
            // first element of each half of the unit
            const int e0 = turn ? (INTER ? 2 * VEC * at[k] : VEC * at[k]) : 2 * p.F + 2 * VEC * (at[k] - p.F / VEC);
            const int e1 = turn && !INTER ? e0 + p.F : e0 + VEC;
            two[k] = e1 < p.D;
            lo[k].load(src + e0);
            if (two[k]) hi[k].load(src + e1);
        }
        if (u0 - static_cast<int>(threadIdx.x) == 0) {
            for (int i = threadIdx.x; i < nt * p.F; i += kThreads) {
                const int t = i / p.F, f = i - t * p.F;
                const int axis = __ldg(p.axes + f);
                float2 v = make_float2(1.f, 0.f);
                if (axis >= 0 && axis < p.A)
                    v = cos_sin(__ldg(p.pos + static_cast<long long>(t0 + t) * p.A + axis), p.inv_freq[f]);
                else
                    kv4::report(kStatusBadAxis);
                if (p.inverse) v.y = -v.y;
                cs[i] = v;
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int u = u0 + k * kThreads;
            if (u >= units) continue;
            const bool turn = at[k] < p.F / VEC;
            const int e0 = turn ? (INTER ? 2 * VEC * at[k] : VEC * at[k]) : 2 * p.F + 2 * VEC * (at[k] - p.F / VEC);
            const int e1 = turn && !INTER ? e0 + p.F : e0 + VEC;
            if (turn) {
                const float2* w = cs + tok[k] * p.F + at[k] * VEC;
                if constexpr (INTER) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        // pair j: elements 2 j, 2 j + 1 of the 2 VEC
                        const float2 r = w[j];
                        if constexpr (VEC == 1) {
                            const float2 f = kv4::to_f32x2<BF16>(kv4::join_words(lo[k], 0, hi[k], 0));
                            const uint32_t o = kv4::pack16<BF16>(f.x * r.x - f.y * r.y, f.y * r.x + f.x * r.y);
                            lo[k].u[0] = o & 0xffffu;
                            hi[k].u[0] = o >> 16;
                        } else {
                            uint32_t& u = j < VEC / 2 ? lo[k].u[j % (VEC / 2)] : hi[k].u[j % (VEC / 2)];
                            const float2 f = kv4::to_f32x2<BF16>(u);
                            u = kv4::pack16<BF16>(f.x * r.x - f.y * r.y, f.y * r.x + f.x * r.y);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < (VEC + 1) / 2; ++j) {   // pairs 2 j and 2 j + 1
                        const float2 x = kv4::to_f32x2<BF16>(lo[k].u[j]), y = kv4::to_f32x2<BF16>(hi[k].u[j]);
                        const float2 r0 = w[2 * j], r1 = VEC > 1 ? w[(2 * j + 1) % VEC] : make_float2(0.f, 0.f);
                        lo[k].u[j] = kv4::pack16<BF16>(x.x * r0.x - y.x * r0.y, x.y * r1.x - y.y * r1.y);
                        hi[k].u[j] = kv4::pack16<BF16>(y.x * r0.x + x.x * r0.y, y.y * r1.x + x.y * r1.y);
                    }
                }
            }
            uint16_t* dst = static_cast<uint16_t*>(p.y[which[k]]) + (t0 + tok[k]) * p.y_row[which[k]] +
                            head[k] * p.y_head[which[k]];
            lo[k].store(dst + e0);
            if (two[k]) hi[k].store(dst + e1);
        }
    }
}

}  // namespace rot
