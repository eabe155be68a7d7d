// rope_append.cu -- what follows the q/k/v GEMVs of a decode step, in one
// launch: bias, per-head rms norm and position rotation of queries and keys,
// and the append of keys and values to the paged cache (f16, bf16 or q8).
//
// Per head x of head_dim values (one row of the batch):
//   x += bias;  x = (x * (1 / sqrt(mean(x^2) + eps))) * gain;
//   (a, b) -> (a cos phi - b sin phi, b cos phi + a sin phi),
//   phi_i = position * freq_i.
// The angle in turns is position * F_i mod 1, F_i = freq_i / 2 pi.  F_i is a
// 64-bit fraction of a turn, so the product modulo 2^64 is the angle exactly
// reduced, at any position, with one integer multiply; as a signed fraction
// in [-1/2, 1/2) it goes through sincospif (2 ulp, no range reduction).  An
// f32 product would be off by 2^-24 of the whole angle: 0.06 radian at
// position 10^6.
//
// Layout: a lane holds EPL consecutive values of a head (4, or 8 above 128
// values a head), so 16 lanes (head_dim <= 64) or 32 hold a head, loads and
// f32 stores are float4, and the partner of a value under MQ_ROPE_HALF is
// rope_dims / 2 values away in another lane at the same place (rope_dims a
// multiple of 2 EPL): one shuffle per value, no shared memory.  A lane's
// cosines and sines depend on its place in the head and the row's position
// only: computed once, used for every head the warp takes.  A q8 block is
// 32 / EPL lanes: max and codes as in the q8 producers.
//
// Work: a row has n_heads + 2 n_kv_heads heads; a warp takes `units` groups
// of heads of one row (a group is what its 32 lanes hold).  Few rows: one
// group a warp, for latency.  Many rows: more groups a warp share the angles
// (launch_rope_append states the rule and what it measured).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace mq {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;

template <int EPL>
struct Vals {
    float v[EPL];
};

template <int EPL>
__device__ __forceinline__ Vals<EPL> load_cg(const float *p)
{
    Vals<EPL> r;
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4 *>(p + i));
        r.v[i] = f.x, r.v[i + 1] = f.y, r.v[i + 2] = f.z, r.v[i + 3] = f.w;
    }
    return r;
}

// One cache entry's EPL values: rounded once to 16 bits, to nearest even.
template <int EPL, class T>
__device__ __forceinline__ void store16(uint8_t *dst, const Vals<EPL> &x)
{
    alignas(16) T t[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) t[i] = __float2half_rn(x.v[i]);
        else t[i] = __float2bfloat16_rn(x.v[i]);
    }
    if constexpr (EPL == 4) *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<uint2 *>(t);
    else *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<uint4 *>(t);
}

template <int EPL>
__global__ void __launch_bounds__(kWarps * 32) rope_append_kernel(const RopeAppendLaunch a)
{
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x / a.ctas_per_row;
    const int first = ((blockIdx.x - t * a.ctas_per_row) * kWarps + (threadIdx.x >> 5)) * a.units;
    const int lph = a.lanes_per_head;               // 16 or 32
    const int sub = lane & ~(lph - 1);              // first lane of this lane's head
    const int e = (lane - sub) * EPL;               // first value of this lane
    const int D = a.head_dim;
    const bool in_head = e < D;
    const int half = a.rope_dims >> 1;
    const bool rotated = e < a.rope_dims;
    const bool upper = e >= half;                   // MQ_ROPE_HALF: the b of its pairs
    const int hpw = 32 / lph;
    griddep_wait();  // q, k, v (and the positions) may come from the preceding kernels

    const int pos = __ldcg(a.positions + t);
    if (pos < 0) return;  // padding

    // the row's page; a row that names none writes nothing but NaN queries
    const int seq = a.seq ? __ldcg(a.seq + t) : t;
    const int pi = pos / a.page_size, slot = pos - pi * a.page_size;
    bool ok = (unsigned)seq < (unsigned)a.n_seqs && pi < a.pages_stride;
    const int page = ok ? __ldcg(a.pages + (size_t)seq * a.pages_stride + pi) : -1;
    ok = (unsigned)page < (unsigned)a.n_pages;
    if (!ok && a.status && first == 0 && lane == 0) atomicOr(a.status, 1);

    float cs[EPL], sn[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        cs[i] = 1.0f, sn[i] = 0.0f;
        if (!rotated) continue;
        const int at = a.style == 0 ? e + i - (upper ? half : 0) : (e + i) >> 1;
        if (a.style != 0 && (i & 1)) {
            cs[i] = cs[i - 1], sn[i] = -sn[i - 1];  // the pair's b
            continue;
        }
        const unsigned long long turn = (unsigned long long)pos * __ldg(a.rope_table + at);
        // a signed fraction of a turn, rounded once: x 2^-64, then x 2 for sincospi's half turns
        const float h = __ll2float_rn((long long)turn) * 0x1p-63f;
        float s, c;
        sincospif(h, &s, &c);
        cs[i] = c;
        sn[i] = a.style == 0 && upper ? s : -s;
    }
    const int heads = a.n_heads + 2 * a.n_kv_heads;
    const int groups = (heads + hpw - 1) / hpw;
    const int last = min(first + a.units, groups);
    for (int gr = first; gr < last; ++gr) {  // uniform across the warp: the shuffles below see all lanes
        const int hd = gr * hpw + (sub ? 1 : 0);
        const bool valid = in_head && hd < heads;
        const int kind = hd < a.n_heads ? 0 : hd < a.n_heads + a.n_kv_heads ? 1 : 2;
        const int h = kind == 0 ? hd : kind == 1 ? hd - a.n_heads : hd - a.n_heads - a.n_kv_heads;
        const float *src = kind == 0 ? a.q + t * a.q_stride : kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride;
        const float *bias = kind == 0 ? a.q_bias : kind == 1 ? a.k_bias : a.v_bias;
        const float *gain = kind == 0 ? a.q_gain : kind == 1 ? a.k_gain : nullptr;
        Vals<EPL> x;
#pragma unroll
        for (int i = 0; i < EPL; ++i) x.v[i] = 0.0f;
        if (valid) {
            x = load_cg<EPL>(src + h * D + e);
            if (bias) {
                const Vals<EPL> b = load_cg<EPL>(bias + h * D + e);
#pragma unroll
                for (int i = 0; i < EPL; ++i) x.v[i] += b.v[i];
            }
        }
        if (a.q_gain || a.k_gain) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) ss = fmaf(x.v[i], x.v[i], ss);
            for (int o = lph >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
            if (valid && gain) {
                const float scale = 1.0f / sqrtf(ss / (float)D + a.eps);
                const Vals<EPL> g = load_cg<EPL>(gain + e);
#pragma unroll
                for (int i = 0; i < EPL; ++i) x.v[i] = (x.v[i] * scale) * g.v[i];
            }
        }
        if (half > 0) {
            Vals<EPL> p;
            if (a.style == 0) {
                const int from = (lane + (rotated ? (upper ? -half : half) / EPL : 0)) & 31;
#pragma unroll
                for (int i = 0; i < EPL; ++i) p.v[i] = __shfl_sync(kFull, x.v[i], from);
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i) p.v[i] = x.v[i ^ 1];
            }
            if (kind < 2 && rotated) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) x.v[i] = fmaf(x.v[i], cs[i], p.v[i] * sn[i]);
            }
        }
        if (kind == 0 && valid) {
            float *dst = a.q_out + t * a.q_out_stride + h * D + e;
            if (!ok) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) x.v[i] = __int_as_float(0x7fc00000);
            }
#pragma unroll
            for (int i = 0; i < EPL; i += 4)
                *reinterpret_cast<float4 *>(dst + i) = make_float4(x.v[i], x.v[i + 1], x.v[i + 2], x.v[i + 3]);
        }
        uint8_t *base = (kind == 1 ? a.k_pages : a.v_pages) + (size_t)(ok ? page : 0) * a.page_stride +
                        (size_t)h * a.head_bytes;
        const bool cached = kind != 0 && valid && ok;
        const size_t at = (size_t)slot * D + e;
        if (a.type == 1) {
            if (cached) store16<EPL, __half>(base + at * 2, x);
        } else if (a.type == 2) {
            if (cached) store16<EPL, __nv_bfloat16>(base + at * 2, x);
        } else {
            float am = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) am = fmaxf(am, fabsf(x.v[i]));
#pragma unroll
            for (int o = 1; o < 32 / EPL; o <<= 1) am = fmaxf(am, __shfl_xor_sync(kFull, am, o));
            const float d = am / 127.0f;
            const float di = (d != 0.0f) ? 1.0f / d : 0.0f;
            uint32_t w[EPL / 4];
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int q = max(-128, min(127, __float2int_rn(x.v[i] * di)));
                w[i / 4] = (i & 3) ? w[i / 4] | ((uint32_t)(q & 0xff) << (8 * (i & 3))) : (uint32_t)(q & 0xff);
            }
            if (cached) {
#pragma unroll
                for (int i = 0; i < EPL / 4; ++i) reinterpret_cast<uint32_t *>(base + at)[i] = w[i];
                if ((e & 31) == 0)
                    reinterpret_cast<__half *>(base + (size_t)a.page_size * D)[at >> 5] = __float2half_rn(d);
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(RopeAppendLaunch a, int sms, int pdl, cudaStream_t st)
{
    a.lanes_per_head = a.head_dim <= 64 ? 16 : 32;
    const int hpw = 32 / a.lanes_per_head;
    const int groups = (a.n_heads + 2 * a.n_kv_heads + hpw - 1) / hpw;
    // One group a warp while the grid is within two resident waves of 32 warps an SM; then as
    // many as keep it there, up to 8.
    const long long wave = (long long)sms * 64;
    long long units = ((long long)a.nt * groups + wave - 1) / wave;
    a.units = (int)(units < 1 ? 1 : units > 8 ? 8 : units);
    const int warps = (groups + a.units - 1) / a.units;
    a.ctas_per_row = (warps + kWarps - 1) / kWarps;
    const dim3 grid((unsigned)((long long)a.nt * a.ctas_per_row));
    const auto kernel = a.head_dim <= 128 ? rope_append_kernel<4> : rope_append_kernel<8>;
    return launch_maybe_pdl(kernel, grid, dim3(kWarps * 32), 0, pdl, st, a);
}

}  // namespace mq
