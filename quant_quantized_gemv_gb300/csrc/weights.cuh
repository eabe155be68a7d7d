// weights.cuh -- the weights of a row of logits as integers, and shares of their sums: what the draw of a
// token and the verification of drafted ones have in common (sample.cu states their accuracy).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "f32x2.cuh"

namespace mq {
namespace {

using u64 = unsigned long long;

constexpr int kBins = 4096;
constexpr float kBinsPerOctave = 64.0f;
constexpr int kFixBits = 42;  // a weight of 1 is 2^42
constexpr float kMagic = 12582912.0f;  // 1.5 x 2^23: a float + this has the rounded integer in its low bits

struct Weight {
    float top, c_hi, c_lo;  // the row's maximum; log2(e) / temperature in two parts

    // the quotient, and what its product leaves
    __device__ __forceinline__ explicit Weight(float temperature)
    {
        c_hi = fminf(1.44269502f / temperature, 5e36f);  // its product with the bins of an octave is finite
        c_lo = (fmaf(-c_hi, temperature, 1.44269502f) + 1.92596299e-8f) / temperature;
        if (!(fabsf(c_lo) < c_hi)) c_lo = 0.0f;  // clamped, or an infinite temperature
    }

    // The bin of a logit: t, in steps of 1 / kBinsPerOctave, rounded.
    __device__ __forceinline__ int bin(float x) const { return bin_of((top - x) * (c_hi * kBinsPerOctave)); }
    __device__ __forceinline__ static int bin_of(float steps)
    {
        return __float_as_int(fminf(steps, (float)(kBins - 1)) + kMagic) & 0xffff;
    }

    __device__ __forceinline__ void bins(float x0, float x1, int &b0, int &b1) const
    {
        const float c = c_hi * kBinsPerOctave;
        float s0, s1;
        split(mul2(fma2(two(x0, x1), two(-1.0f, -1.0f), two(top, top)), two(c, c)), s0, s1);
        b0 = bin_of(s0), b1 = bin_of(s1);
    }

    // The weights of two logits, each as a * m, two 32-bit factors (adding such a product to a sum is
    // one instruction), and their bins.
    __device__ __forceinline__ void pair(float x0, float x1, unsigned (&a)[2], unsigned (&m)[2], int (&bin)[2]) const
    {
        const Two x = two(x0, x1), tp = two(top, top), minus = two(-1.0f, -1.0f);
        const Two ch = two(c_hi, c_hi), cl = two(c_lo, c_lo);
        const Two d = fma2(x, minus, tp);
        const Two t = mul2(d, ch);
        // d + e = top - x exactly; t + r = (d + e) * (c_hi + c_lo) to f32's square
        const Two b = fma2(tp, minus, d);
        const Two e = fma2(add2(x, b), minus, fma2(fma2(b, minus, d), minus, tp));
        const Two nt = mul2(t, minus);
        const Two r = add2(fma2(d, ch, nt), fma2(d, cl, mul2(e, ch)));
        const Two nm = add2(t, two(kMagic, kMagic));
        const Two f = fma2(r, minus, add2(add2(nm, two(-kMagic, -kMagic)), nt));
        // 2^30 (2^f - 1) / f by its series in f ln2
        constexpr float k = 1073741824.0f;
        Two s = two(1.3215486790144307e-6f * k, 1.3215486790144307e-6f * k);
        s = fma2(s, f, two(1.5252733804059841e-5f * k, 1.5252733804059841e-5f * k));
        s = fma2(s, f, two(1.5403530393381609e-4f * k, 1.5403530393381609e-4f * k));
        s = fma2(s, f, two(1.3333558146428443e-3f * k, 1.3333558146428443e-3f * k));
        s = fma2(s, f, two(9.6181291076284772e-3f * k, 9.6181291076284772e-3f * k));
        s = fma2(s, f, two(5.5504108664821580e-2f * k, 5.5504108664821580e-2f * k));
        s = fma2(s, f, two(2.4022650695910071e-1f * k, 2.4022650695910071e-1f * k));
        s = fma2(s, f, two(6.9314718055994531e-1f * k, 6.9314718055994531e-1f * k));
        float p[2], tt[2], nn[2], steps[2];
        split(mul2(s, f), p[0], p[1]);
        split(t, tt[0], tt[1]);
        split(nm, nn[0], nn[1]);
        split(mul2(t, two(kBinsPerOctave, kBinsPerOctave)), steps[0], steps[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const unsigned one = (1u << 30) + (unsigned)__float2int_rn(p[i]);
            const int n = (int)(__float_as_uint(nn[i]) & 63u);  // the weight is one * 2^(42 - 30 - n)
            a[i] = tt[i] < (float)kFixBits + 0.5f ? one >> max(n - (kFixBits - 30), 0) : 0u;
            m[i] = 1u << max(kFixBits - 30 - n, 0);
            bin[i] = bin_of(steps[i]);
        }
    }

    // The weights of two logits as f32 (rounded once more, 2^-24), in units of the largest: for sums that take
    // something off them.
    __device__ __forceinline__ Two pair_f32(float x0, float x1) const
    {
        float w[2];
        unsigned a[2], m[2];
        int none[2];
        pair(x0, x1, a, m, none);
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = __uint2float_rn(a[i]) * (__uint2float_rn(m[i]) * 0x1p-42f);
        return two(w[0], w[1]);
    }

    // The same in units of the largest, each as two f32 whose sum it is (22 bits and the other 8).
    __device__ __forceinline__ void parts(float x0, float x1, Two &hi, Two &lo) const
    {
        unsigned a[2], m[2];
        int none[2];
        float h[2], l[2];
        pair(x0, x1, a, m, none);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float unit = __uint2float_rn(m[i]) * 0x1p-42f;
            h[i] = __uint2float_rn(a[i] & ~0xffu) * unit, l[i] = __uint2float_rn(a[i] & 0xffu) * unit;
        }
        hi = two(h[0], h[1]), lo = two(l[0], l[1]);
    }

    __device__ __forceinline__ u64 operator()(float x) const
    {
        unsigned a[2], m[2];
        int none[2];
        pair(x, x, a, m, none);
        return (u64)a[0] * m[0];
    }
};

// A share s < 1 of a sum: its floor, or that rounded up, by the 64 bits behind the point.
__device__ __forceinline__ u64 share_of(float s, u64 all, bool up)
{
    const u64 f = __float2ull_rz(s * 18446744073709551616.0f);
    return __umul64hi(f, all) + (up && f * all != 0 ? 1 : 0);
}

// r in [0, 1] in units of 2^-42, rounded: 21 bits and 22 more, by additions of 1.5 x 2^23.
__device__ __forceinline__ void fixed_of(float r, unsigned &hi, int &lo)
{
    constexpr float magic = 12582912.0f;
    const float v = r * 0x1p20f, h = v + magic;
    hi = __float_as_uint(h) - 0x4b400000u;
    lo = __float_as_int(fmaf(v - (h - magic), 0x1p22f, magic)) - 0x4b400000;
}
__device__ __forceinline__ u64 fixed_of(float r)
{
    unsigned hi;
    int lo;
    fixed_of(r, hi, lo);
    return ((u64)hi << 22) + (u64)(long long)lo;
}

}  // namespace
}  // namespace mq
