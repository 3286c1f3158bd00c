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
// out, so that the two overlap.  What comes beside the copying has to stay small:
// with indexes and angles looked up for each head, and the factor of a
// frequency (64-bit arithmetic, which is slow here) worked out for each token,
// 32760 tokens of 32 heads of 128 took 109 us; they take 86 us (6.24 TB/s, 93 % of
// the copy bandwidth).  Two or eight heads a thread: 93 and 90 us.
#pragma once

#include "kv4_cache.cuh"

namespace rot {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;          // units a thread has in flight
constexpr int kMaxFreqs = 128;
// Angles of a CTA's tokens (32 KB).  With few heads a CTA needs many tokens to have
// work for its threads: 280582 tokens of 4 heads of 64 take 101 us, with 512 angles 134
// (there the angles, one for 4 pairs, are what it spends its time on).
constexpr int kMaxAngles = 4096;
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

// inv_freq / 2 pi as the sum of two floats
__device__ __forceinline__ float2 turns_of(double inv_freq) {
    const double turns = inv_freq * 0.15915494309189533577;
    const float hi = static_cast<float>(turns);
    return make_float2(hi, static_cast<float>(turns - static_cast<double>(hi)));
}

__device__ __forceinline__ float2 cos_sin(int p, float2 turns) {
    const float fh = turns.x, fl = turns.y;
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
// A thread has the same pairs of up to kUnroll heads of a token: where they lie and
// their angles are looked up once for all of them.
template <int VEC, bool INTER, bool BF16>
__global__ void __launch_bounds__(kThreads) rotary_kernel(Rotary p) {
    extern __shared__ __align__(16) float cs[];   // [tokens][cos, sin][F], then [F] turns
    const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0);
    const int heads = p.heads[0] + p.heads[1], step = (heads + kUnroll - 1) / kUnroll;
    const int per_head = p.F / VEC + (p.D - 2 * p.F + 2 * VEC - 1) / (2 * VEC);   // rotated, copied
    const int per_token = step * per_head, all = nt * per_token;
    for (int g0 = 0; g0 < all; g0 += kThreads) {
        const int g = g0 + static_cast<int>(threadIdx.x);
        const int tok = g / per_token, rest = g - tok * per_token, head0 = rest / per_head, at = rest - head0 * per_head;
        const bool turn = at < p.F / VEC;
        // first element of each half of the unit
        const int e0 = turn ? (INTER ? 2 * VEC * at : VEC * at) : 2 * p.F + 2 * VEC * (at - p.F / VEC);
        const int e1 = turn && !INTER ? e0 + p.F : e0 + VEC;
        const bool two = e1 < p.D;
        const int last = g < all ? heads : 0;   // heads head0, head0 + step, ... below it
        kv4::Words<VEC> lo[kUnroll], hi[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int head = head0 + k * step;
            if (head >= last) continue;
            const int which = head >= p.heads[0], h = which ? head - p.heads[0] : head;
            const uint16_t* src = static_cast<const uint16_t*>(p.x[which]) + (t0 + tok) * p.x_row[which] + h * p.x_head[which];
            lo[k].load(src + e0);
            if (two) hi[k].load(src + e1);
        }
        if (g0 == 0) {
            float2* turns = reinterpret_cast<float2*>(cs + p.tokens * 2 * p.F);
            for (int i = threadIdx.x; i < nt * p.F; i += kThreads) {
                const int t = i / p.F, f = i - t * p.F;
                const int axis = __ldg(p.axes + f);
                const bool known = axis >= 0 && axis < p.A;
                if (!known) kv4::report(kStatusBadAxis);
                const int at_pos = known ? __ldg(p.pos + static_cast<long long>(t0 + t) * p.A + axis) : 0;   // 0: no turn
                cs[t * 2 * p.F + f] = __int_as_float(at_pos);
            }
            for (int f = threadIdx.x; f < p.F; f += kThreads) turns[f] = turns_of(p.inv_freq[f]);
            __syncthreads();
            for (int i = threadIdx.x; i < nt * p.F; i += kThreads) {
                const int t = i / p.F, f = i - t * p.F;
                float* w = cs + t * 2 * p.F + f;
                const float2 v = cos_sin(__float_as_int(*w), turns[f]);
                w[0] = v.x;
                w[p.F] = p.inverse ? -v.y : v.y;
            }
            __syncthreads();
        }
        float co[VEC], si[VEC];
        if (turn && last > 0) {
            const float* w = cs + tok * 2 * p.F + at * VEC;
            if constexpr (VEC == 1) {
                co[0] = w[0];
                si[0] = w[p.F];
            } else {
#pragma unroll
                for (int i = 0; i < VEC; i += 4) {
                    *reinterpret_cast<float4*>(co + i) = *reinterpret_cast<const float4*>(w + i);
                    *reinterpret_cast<float4*>(si + i) = *reinterpret_cast<const float4*>(w + p.F + i);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int head = head0 + k * step;
            if (head >= last) continue;
            if (turn) {
                if constexpr (INTER) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        // pair j: elements 2 j, 2 j + 1 of the 2 VEC
                        if constexpr (VEC == 1) {
                            const float2 f = kv4::to_f32x2<BF16>(kv4::join_words(lo[k], 0, hi[k], 0));
                            const uint32_t o = kv4::pack16<BF16>(f.x * co[j] - f.y * si[j], f.y * co[j] + f.x * si[j]);
                            lo[k].u[0] = o & 0xffffu;
                            hi[k].u[0] = o >> 16;
                        } else {
                            uint32_t& u = j < VEC / 2 ? lo[k].u[j % (VEC / 2)] : hi[k].u[j % (VEC / 2)];
                            const float2 f = kv4::to_f32x2<BF16>(u);
                            u = kv4::pack16<BF16>(f.x * co[j] - f.y * si[j], f.y * co[j] + f.x * si[j]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < (VEC + 1) / 2; ++j) {   // pairs 2 j and 2 j + 1
                        const float2 x = kv4::to_f32x2<BF16>(lo[k].u[j]), y = kv4::to_f32x2<BF16>(hi[k].u[j]);
                        const int j0 = 2 * j, j1 = (2 * j + 1) % VEC;
                        lo[k].u[j] = kv4::pack16<BF16>(x.x * co[j0] - y.x * si[j0], x.y * co[j1] - y.y * si[j1]);
                        hi[k].u[j] = kv4::pack16<BF16>(y.x * co[j0] + x.x * si[j0], y.y * co[j1] + x.y * si[j1]);
                    }
                }
            }
            const int which = head >= p.heads[0], h = which ? head - p.heads[0] : head;
            uint16_t* dst = static_cast<uint16_t*>(p.y[which]) + (t0 + tok) * p.y_row[which] + h * p.y_head[which];
            lo[k].store(dst + e0);
            if (two) hi[k].store(dst + e1);
        }
    }
}

}  // namespace rot
