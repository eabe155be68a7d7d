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
// Layout: a lane holds EPL values of a head, 4 or 8, so 8, 16 or 32 lanes hold a
// head and a warp 1 to 4 heads; loads and f32 stores are float4.  Where
// MQ_ROPE_HALF turns whole heads the 8 are four and their four partners, half a
// head away: nothing is exchanged.  Else they are consecutive, and the partner of
// a value under MQ_ROPE_HALF is in another lane at the same place (rope_dims a
// multiple of 2 EPL): one shuffle per value.  A q8 block is the 8 lanes' fours, or
// 32 / EPL lanes: max and codes as in the q8 producers.
//
// Work: a row's heads, queries | keys | values, in groups of what a warp's lanes
// hold, are shared by the CTAs of the row.  A CTA first writes down where each
// of its groups is read and what becomes of it; then its first loads are under
// way while one thread per pair computes an angle and the row's page is found,
// which only the cache entries wait for.
//
// What bounds it: few rows, the launch and three dependent loads (2.6 us a call
// in a captured chain).  Many rows, HBM and the latency of a CTA's loads, one batch
// after another.  4096 rows of 40 + 8 + 8 heads of 128, 218 MB, which take 33 us:
// f16 37 us (5.9 TB/s), with biases 39.5, q8 with norms 42.  With four values a lane
// in the place of eight: 40, 47 and 56.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kernels.h"

namespace mq {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kUnits = 14;  // groups of heads (of 4 values a lane) a warp takes when there are many rows
constexpr int kResident = 9;  // CTAs an SM holds, by registers
constexpr int kLoads = 4;  // float4 loads of a lane in flight
constexpr int kMaxGroups = kWarps * kUnits;
constexpr int kGridRows = 32768;  // rows along the grid's y
static_assert(kWarps * 32 >= 128, "a thread for each of the up to 128 angles");

template <int EPL>
struct Vals {
    float v[EPL];
};

// Biases and gains: shared by many rows, so through L1, but coherent: a preceding kernel may have written them.
template <int EPL>
__device__ __forceinline__ Vals<EPL> load_weight(const float *p, int gap)
{
    Vals<EPL> r;
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
        const float4 f = __ldca(reinterpret_cast<const float4 *>(p + (i ? gap : 0)));
        r.v[i] = f.x, r.v[i + 1] = f.y, r.v[i + 2] = f.z, r.v[i + 3] = f.w;
    }
    return r;
}

template <int EPL>
__device__ __forceinline__ Vals<EPL> load_cg(const float *p, int gap)
{
    Vals<EPL> r;
#pragma unroll
    for (int i = 0; i < EPL; i += 4) {
        const float4 f = __ldcg(reinterpret_cast<const float4 *>(p + (i ? gap : 0)));
        r.v[i] = f.x, r.v[i + 1] = f.y, r.v[i + 2] = f.z, r.v[i + 3] = f.w;
    }
    return r;
}

// One cache entry's EPL values: rounded once to 16 bits, to nearest even.
template <int EPL, bool SPLIT, class T>
__device__ __forceinline__ void store16(uint8_t *dst, const Vals<EPL> &x, int gap)
{
    alignas(16) T t[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) t[i] = __float2half_rn(x.v[i]);
        else t[i] = __float2bfloat16_rn(x.v[i]);
    }
    if constexpr (EPL == 4 || SPLIT) *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<uint2 *>(t);
    else *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<uint4 *>(t);
    if constexpr (SPLIT) *reinterpret_cast<uint2 *>(dst + 2 * gap) = *reinterpret_cast<uint2 *>(t + 4);
}

// A group of heads: where it is read, its biases, and its first head.
struct alignas(16) Group {
    const float *src, *bias;
    float *dst;             // queries: their place in q_out
    int kind, head, heads;  // 0 queries, 1 keys, 2 values; heads that exist (1 to 4)
};

// SPLIT: a lane's 8 values are 4 and their 4 partners, half a head away (MQ_ROPE_HALF of whole heads).
template <int EPL, bool SPLIT>
__global__ void __launch_bounds__(kWarps * 32, kResident) rope_append_kernel(const RopeAppendLaunch a)
{
    constexpr int kBatch = kLoads * 4 / EPL;  // groups a warp loads at a time
    __shared__ Group groups[kMaxGroups];
    __shared__ float cosine[128], sine[128];
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, D = a.head_dim;
    const int lg = a.heads_log, lph = 32 >> lg;  // a group is 1 << lg heads, of lph lanes each
    const int half = a.rope_dims >> 1;
    const int sub = lane / lph, e = (lane & (lph - 1)) * (SPLIT ? 4 : EPL);  // this lane's head of a group, first value
    const int gap = SPLIT ? half : 4;                   // from its first four values to the others
    const bool in_head = e < (SPLIT ? half : D), rotated = e < a.rope_dims;
    const bool upper = e >= half;  // MQ_ROPE_HALF: the b of its pairs
    const int from = (lane + (rotated ? (upper ? -half : half) / EPL : 0)) & 31;

    // this CTA's row and groups
    const int t = blockIdx.y + blockIdx.z * kGridRows, c = blockIdx.x;
    if (t >= a.nt) return;
    const int more = (1 << lg) - 1, gq = (a.n_heads + more) >> lg, gk = (a.n_kv_heads + more) >> lg;
    const int first = c * a.groups_per_cta, n = min(a.groups_per_cta, gq + 2 * gk - first);
    for (int i = tid; i < n; i += kWarps * 32) {
        const int gr = first + i, kind = gr < gq ? 0 : gr < gq + gk ? 1 : 2;
        const int h = (kind == 0 ? gr : kind == 1 ? gr - gq : gr - gq - gk) << lg;
        const float *bias = kind == 0 ? a.q_bias : kind == 1 ? a.k_bias : a.v_bias;
        Group &g = groups[i];
        g.src = (kind == 0 ? a.q + t * a.q_stride : kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride) + h * D;
        g.bias = bias ? bias + h * D : nullptr;
        g.dst = a.q_out + t * a.q_out_stride + h * D;
        g.kind = kind, g.head = h;
        g.heads = min(1 + more, (kind == 0 ? a.n_heads : a.n_kv_heads) - h);
    }
    __syncthreads();
    griddep_wait();  // nothing is read before: any of the inputs may come from the preceding kernels

    const unsigned long long step = tid < half ? __ldca(a.rope_table + tid) : 0;
    const int pos = __ldcg(a.positions + t);
    Vals<EPL> x[kBatch];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + k * kWarps;
#pragma unroll
            for (int j = 0; j < EPL; ++j) x[k].v[j] = 0.0f;
            if (i < n && in_head && sub < groups[i].heads) x[k] = load_cg<EPL>(groups[i].src + sub * D + e, gap);
        }
    };
    load(warp);  // on their way while the page and the angles are found
    if (pos < 0) return;  // padding

    if (tid < half) {
        // a signed fraction of a turn, rounded once: x 2^-64, then x 2 for sincospi's half turns
        const float h = __ll2float_rn((long long)((unsigned long long)pos * step)) * 0x1p-63f;
        sincospif(h, &sine[tid], &cosine[tid]);
    }
    // the row's page; a row that names none writes nothing but NaN queries, at the end
    const int seq = a.seq ? __ldcg(a.seq + t) : t;
    const int pi = a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size, slot = pos - pi * a.page_size;
    const bool named = (unsigned)seq < (unsigned)a.n_seqs && pi < a.pages_stride;
    const int page = named ? __ldcg(a.pages + (size_t)seq * a.pages_stride + pi) : -1;
    const bool ok = (unsigned)page < (unsigned)a.n_pages;
    const size_t page_at = (size_t)(ok ? page : 0) * a.page_stride, slot_at = (size_t)slot * D + e;
    __syncthreads();
    constexpr int kAngles = SPLIT ? 4 : EPL;
    float cs[kAngles], sn[kAngles];
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
        cs[i] = 1.0f, sn[i] = 0.0f;
        if (SPLIT) {
            if (in_head) cs[i] = cosine[e + i], sn[i] = sine[e + i];
            continue;
        }
        if (!rotated) continue;
        const int at = a.style == 0 ? e + i - (upper ? half : 0) : (e + i) >> 1;
        cs[i] = cosine[at];
        sn[i] = (a.style == 0 ? upper : (i & 1) != 0) ? sine[at] : -sine[at];
    }

    for (int i0 = warp; i0 < n; i0 += kBatch * kWarps) {
        if (i0 != warp) load(i0);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + k * kWarps;  // uniform across the warp: the shuffles below see all lanes
            if (i >= n) break;
            const Group &g = groups[i];
            const int kind = g.kind;
            const bool valid = in_head && sub < g.heads;
            if (g.bias && valid) {
                const Vals<EPL> b = load_weight<EPL>(g.bias + sub * D + e, gap);
#pragma unroll
                for (int j = 0; j < EPL; ++j) x[k].v[j] += b.v[j];
            }
            if (kind < 2) {
                const float *gain = kind == 0 ? a.q_gain : a.k_gain;
                if (gain) {
                    float ss = 0.0f;
#pragma unroll
                    for (int j = 0; j < EPL; ++j) ss = fmaf(x[k].v[j], x[k].v[j], ss);
                    for (int o = lph >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
                    if (valid) {
                        const float scale = 1.0f / sqrtf(ss / (float)D + a.eps);
                        const Vals<EPL> w = load_weight<EPL>(gain + e, gap);
#pragma unroll
                        for (int j = 0; j < EPL; ++j) x[k].v[j] = (x[k].v[j] * scale) * w.v[j];
                    }
                }
                if constexpr (SPLIT) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float lo = x[k].v[j], hi = x[k].v[EPL - 4 + j];
                        x[k].v[j] = fmaf(lo, cs[j], hi * -sn[j]);
                        x[k].v[EPL - 4 + j] = fmaf(hi, cs[j], lo * sn[j]);
                    }
                } else if (half > 0) {
                    Vals<EPL> p;
                    if (a.style == 0) {
#pragma unroll
                        for (int j = 0; j < EPL; ++j) p.v[j] = __shfl_sync(kFull, x[k].v[j], from);
                    } else {
#pragma unroll
                        for (int j = 0; j < EPL; ++j) p.v[j] = x[k].v[j ^ 1];
                    }
                    if (rotated) {
#pragma unroll
                        for (int j = 0; j < EPL; ++j) x[k].v[j] = fmaf(x[k].v[j], cs[j], p.v[j] * sn[j]);
                    }
                }
                if (kind == 0) {
                    if (valid) {
                        float *dst = g.dst + sub * D + e;
#pragma unroll
                        for (int j = 0; j < EPL; j += 4)
                            *reinterpret_cast<float4 *>(dst + (j ? gap : 0)) =
                                make_float4(x[k].v[j], x[k].v[j + 1], x[k].v[j + 2], x[k].v[j + 3]);
                    }
                    continue;
                }
            }
            uint8_t *base = (kind == 1 ? a.k_pages : a.v_pages) + page_at + (size_t)(g.head + sub) * a.head_bytes;
            const bool cached = valid && ok;  // the first use of the page: the queries do not wait for it
            if (a.type == 1) {
                if (cached) store16<EPL, SPLIT, __half>(base + slot_at * 2, x[k], gap);
            } else if (a.type == 2) {
                if (cached) store16<EPL, SPLIT, __nv_bfloat16>(base + slot_at * 2, x[k], gap);
            } else {
                // blocks of 32 values: 32 / EPL lanes, or 8 lanes' fours
                constexpr int kPer = SPLIT ? 4 : EPL;
#pragma unroll
                for (int i = 0; i < EPL; i += kPer) {
                    float am = 0.0f;
#pragma unroll
                    for (int j = 0; j < kPer; ++j) am = fmaxf(am, fabsf(x[k].v[i + j]));
#pragma unroll
                    for (int o = 1; o < 32 / kPer; o <<= 1) am = fmaxf(am, __shfl_xor_sync(kFull, am, o));
                    const float d = am / 127.0f;
                    const float di = (d != 0.0f) ? 1.0f / d : 0.0f;
                    uint32_t w[kPer / 4];
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        const int q = max(-128, min(127, __float2int_rn(x[k].v[i + j] * di)));
                        w[j / 4] = (j & 3) ? w[j / 4] | ((uint32_t)(q & 0xff) << (8 * (j & 3))) : (uint32_t)(q & 0xff);
                    }
                    if (cached) {
                        const size_t at = slot_at + (i ? gap : 0);
#pragma unroll
                        for (int j = 0; j < kPer / 4; ++j) reinterpret_cast<uint32_t *>(base + at)[j] = w[j];
                        if ((e & 31) == 0)
                            reinterpret_cast<__half *>(base + (size_t)a.page_size * D)[at >> 5] = __float2half_rn(d);
                    }
                }
            }
        }
    }
    if (!ok) {  // the row names no page: its queries become NaN
        for (int i = warp; i < n; i += kWarps) {
            const Group &g = groups[i];
            if (g.kind != 0 || !in_head || sub >= g.heads) continue;
            const float nan = __int_as_float(0x7fc00000);
#pragma unroll
            for (int j = 0; j < EPL; j += 4)
                *reinterpret_cast<float4 *>(g.dst + sub * D + e + (j ? gap : 0)) = make_float4(nan, nan, nan, nan);
        }
        if (a.status && c == 0 && tid == 0) atomicOr(a.status, 1);
    }
}

}  // namespace

cudaError_t launch_rope_append(RopeAppendLaunch a, int sms, int pdl, cudaStream_t st)
{
    a.page_shift = (a.page_size & (a.page_size - 1)) == 0 ? __builtin_ctz((unsigned)a.page_size) : -1;
    // 8 values a lane, partners in one lane, where pairs lie half a head apart and halves are whole blocks of q8.
    // Else 8 where rows are many. (Captured, us, 4 values / 8, 8 with partners: 40 + 8 + 8 heads of 128, biases: 1 row
    // 2.8 / 2.9, 2.7; 24 rows 3.3 / 3.5, 3.1; 64 rows 4.4 / 3.9, 3.2; 256 rows 5.1 / 5.9, 4.6; 1024 rows 18.3 / 16.9, 14.6;
    // 4096 rows 47 / 43, 39.5. q8, 28 + 4 + 4 heads: 1 row 3.1 / -, 3.3; 64 rows 4.1 / -, 3.9; 1024 rows 15.4 / -, 12.5.
    // Heads of 64: 64 rows 3.5 / 3.6, 3.1; 1024 rows 7.8 / 7.4, 6.)
    const long long heads = (long long)a.nt * (a.n_heads + 2 * a.n_kv_heads);
    const bool many = heads >= sms * (a.head_dim > 64 ? 8LL : 128LL);
    const bool q8 = a.type == 3, partners = a.style == 0 && a.rope_dims == a.head_dim && (!q8 || a.head_dim % 64 == 0);
    const bool wide = a.head_dim > 128 || (partners ? !q8 || heads >= sms * 8LL : many && a.rope_dims % 16 == 0);
    a.heads_log = wide ? (a.head_dim <= 64 ? 2 : a.head_dim <= 128 ? 1 : 0) : a.head_dim <= 64 ? 1 : 0;
    const int more = (1 << a.heads_log) - 1;
    const int groups = ((a.n_heads + more) >> a.heads_log) + 2 * ((a.n_kv_heads + more) >> a.heads_log);
    // Few rows: a group a warp, for latency.  More: up to kUnits groups a warp (as many values for 8 a lane),
    // which share the row's angles and its page.
    const int most = wide ? kUnits / 2 : kUnits;
    const long long wave = (long long)sms * 32;  // warps
    long long units = ((long long)a.nt * groups + wave - 1) / wave;
    units = units < 1 ? 1 : units > most ? most : units;
    const int ctas = (groups + (int)units * kWarps - 1) / ((int)units * kWarps);
    a.groups_per_cta = ((groups + ctas - 1) / ctas + kWarps - 1) / kWarps * kWarps;  // alike, whole warps' groups
    const dim3 grid((unsigned)ctas, (unsigned)std::min(a.nt, kGridRows), (unsigned)((a.nt + kGridRows - 1) / kGridRows));
    const auto kernel = wide && partners ? rope_append_kernel<8, true>
                        : wide           ? rope_append_kernel<8, false>
                                         : rope_append_kernel<4, false>;
    return launch_maybe_pdl(kernel, grid, dim3(kWarps * 32), 0, pdl, st, a);
}

}  // namespace mq
