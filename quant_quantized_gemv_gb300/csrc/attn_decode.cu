// attn_decode.cu -- attention of one new token per row over the paged cache.
//
//   s_j = scale q.k_j (capped: c tanh(s_j / c)),  out = sum p_j v_j / sum p_j,
//   p_j = exp(s_j - max s), in one pass over the tokens with the running
//   maximum m and sum l:  m' = max(m, s),  l = l e^(m - m') + e^(s - m'), and
//   the same for the sum of p v.
//
// Every cached byte is used by the 1..8 query heads of its kv head, a handful
// of operations a byte: the pass is bound by HBM when contexts are long and
// by latency when they are short, never by the tensor cores.  So each warp
// streams its tokens straight into registers, 16 at a time, with nothing
// shared between warps until the end: no barrier and no shared-memory copy
// of the cache.  tcgen05 products would need the tokens in shared memory and
// a hand-over per tile, to fill 8 of 128 rows.
//
// One warp's 16 tokens, with m16n8k16 products (lane = 4 g + t):
//   scores: rows 0..7 are the heads (one part of q), rows 8..15 the same heads
//     (the next part of q), columns 8 tokens.  A lane's 16-byte load is 8
//     consecutive values of token g; which values share a product's k slots is
//     free as long as q's fragments follow, so the load needs no exchange.
//   output: rows again heads and parts of p, k the 16 tokens, columns 8 values
//     of v: a lane holds 8 consecutive values of tokens 2t, 2t+1, 2t+8, 2t+9,
//     and one byte permute pairs two tokens of a value.  The scores' layout is
//     the one p needs, so p never leaves its lane.
// Parts: fp16 holds 11 bits, so q (scaled by a power of two a head) and p
// (times 2^14) go in as hi + lo = 22 bits in the two halves of the 16 rows;
// bf16 holds 8, so three parts in two products.  The cache's values are exact
// in both (int8 codes in fp16).  Results then are as an f32 computation's.
// q8: the scales of K (token, block of 32) multiply the block's partial
// scores; the scales of V multiply p, block by block, scaled by a power of two
// a tile (their maximum) to stay in fp16's range.
//
// Sums: every tile's products start from zero and are added to the f32
// accumulators by the same fused multiply-add that rescales them, so no
// accumulation inside the tensor core runs over more than a head's values.
//
// Work.  A unit is a row's group of up to 8 query heads of one kv head; its
// tokens come in rounds, a tile for every warp of a CTA.  The rounds of all
// units stand in one line, and each CTA of one resident wave takes an equal
// share of it (every CTA adds up the lengths, which only the device knows):
// ragged batches are as balanced as full ones.  A CTA's warps meet in shared
// memory at the end of a unit.  A unit that crosses from one share into the next
// is joined through the workspace: its CTAs leave their partial results, and the
// last to arrive (an atomic count; nobody waits) adds them in order.  Units of
// kWhole rounds or less are not cut: the join costs more than they do.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kernels.h"
#include "q8_block.cuh"

namespace mq {
namespace {

constexpr int kF16 = 1, kBF16 = 2, kQ8 = 3;  // MQ_KV_*
constexpr float kPScale = 16384.0f;          // p's factor in fp16 parts: 2^14
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// x, y as fp16 parts: hi rounds the value, lo the rest.
__device__ __forceinline__ void split_f16(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = bits(h);
    lo = bits(__floats2half2_rn(x - f.x, y - f.y));
}

// x, y as three bf16 parts.
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 m = __floats2bfloat162_rn(x - f.x, y - f.y);
    const float2 e = __bfloat1622float2(m);
    hi = bits(h);
    mid = bits(m);
    lo = bits(__floats2bfloat162_rn((x - f.x) - e.x, (y - f.y) - e.y));
}

// Two signed bytes (already xor 0x80) in the low or high half of w as fp16
// pairs: 0x6400 + u is 1024 + u, minus 1152 gives u - 128, exactly.
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, uint32_t sel)
{
    return bits(__hsub2(half2_of(__byte_perm(w, 0x64646464u, sel)), half2_of(0x64806480u)));
}

// Registers of one 16-token tile: K rows of tokens g and 8 + g, V rows of
// tokens 2t, 2t+1, 2t+8, 2t+9 (q8: and those tokens' scales).
template <int TYPE, int D>
struct Tile {
    static constexpr int KC = D / 32, VC = (D + 63) / 64;
    uint4 k[2][KC], v[4][VC];
};
template <int D>
struct Tile<kQ8, D> {
    static constexpr int KC = D / 32;
    uint2 k[2][KC];
    uint32_t v[4][KC];
    alignas(8) __half ks[4][KC];
    alignas(8) __half vs[4][KC];
};

template <int KC>
__device__ __forceinline__ void load_scales(__half (&s)[KC], const uint8_t *p)
{
    if constexpr (KC % 4 == 0) {
#pragma unroll
        for (int i = 0; i < KC; i += 4)
            *reinterpret_cast<uint2 *>(&s[i]) = __ldcg(reinterpret_cast<const uint2 *>(p) + i / 4);
    } else if constexpr (KC % 2 == 0) {
        *reinterpret_cast<unsigned *>(&s[0]) = __ldcg(reinterpret_cast<const unsigned *>(p));
    } else {
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            const unsigned short u = __ldcg(reinterpret_cast<const unsigned short *>(p) + i);
            s[i] = *reinterpret_cast<const __half *>(&u);
        }
    }
}

template <int TYPE, int D>
__device__ __forceinline__ void load_k(Tile<TYPE, D> &r, const uint8_t *head, int slot, int page_size, int g, int t)
{
    constexpr int KC = D / 32;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if constexpr (TYPE == kQ8) {
            const uint8_t *p = head + (size_t)(slot + 8 * j + g) * D + 8 * t;
#pragma unroll
            for (int c = 0; c < KC; ++c) r.k[j][c] = __ldcg(reinterpret_cast<const uint2 *>(p + 32 * c));
        } else {
            const uint8_t *p = head + ((size_t)(slot + 8 * j + g) * D + 8 * t) * 2;
#pragma unroll
            for (int c = 0; c < KC; ++c) r.k[j][c] = __ldcg(reinterpret_cast<const uint4 *>(p + 64 * c));
        }
    }
    if constexpr (TYPE == kQ8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int tok = slot + 8 * (i >> 1) + 2 * t + (i & 1);
            load_scales<KC>(r.ks[i], head + (size_t)page_size * D + (size_t)tok * (KC * 2));
        }
    }
}

// Tokens outside [lo, hi) (relative to the tile) are not read and count as 0.
template <int TYPE, int D>
__device__ __forceinline__ void load_v(Tile<TYPE, D> &r, const uint8_t *head, int slot, int page_size, int g, int t,
                                       int lo, int hi)
{
    constexpr int KC = D / 32, VC = (D + 63) / 64;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int tok = 8 * (i >> 1) + 2 * t + (i & 1);
        const bool seen = tok >= lo && tok < hi;
        if constexpr (TYPE == kQ8) {
            const uint8_t *p = head + (size_t)(slot + tok) * D + 4 * g;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                r.v[i][c] = 0;
                r.vs[i][c] = __ushort_as_half(0);
            }
            if (seen) {
#pragma unroll
                for (int c = 0; c < KC; ++c) r.v[i][c] = __ldcg(reinterpret_cast<const unsigned *>(p + 32 * c));
                load_scales<KC>(r.vs[i], head + (size_t)page_size * D + (size_t)(slot + tok) * (KC * 2));
            }
        } else {
            const uint8_t *p = head + ((size_t)(slot + tok) * D + 8 * g) * 2;
#pragma unroll
            for (int c = 0; c < VC; ++c) {
                r.v[i][c] = make_uint4(0, 0, 0, 0);
                if (seen && 64 * c + 8 * g < D) r.v[i][c] = __ldcg(reinterpret_cast<const uint4 *>(p + 128 * c));
            }
        }
    }
}

// Place of accumulator j (pair element e) of lane t within a head.
template <int TYPE>
__device__ __forceinline__ int value_of(int j, int e, int t)
{
    return TYPE == kQ8 ? 32 * (j >> 2) + 4 * (2 * t + e) + (j & 3) : 64 * (j >> 3) + 8 * (2 * t + e) + (j & 7);
}

template <int D>
struct Shape {
    static constexpr int warps = attn_warps(D), threads = warps * 32, round = warps * kAttnTile;
    static constexpr int ctas = attn_ctas(D);
};

// Shared memory: q's fragments, the warps' exchange (later the join's weights), the rows' rounds.
template <int TYPE, int D>
struct Smem {
    static constexpr int KC = D / 32, RS = D + 4;
    uint4 q_frag[2 * KC][32];                              // q's parts as the products take them
    uint2 q_low[TYPE == kBF16 ? 2 * KC : 1][32];           // bf16's third part
    union {
        float x_o[Shape<D>::warps][kAttnHeads][RS];        // padded rows
        float weight[kAttnMaxCtas][kAttnHeads];            // the join
    };
    float x_m[Shape<D>::warps][kAttnHeads], x_l[Shape<D>::warps][kAttnHeads];
    float total[kAttnHeads];
    int sums[Shape<D>::warps];
    int last;
    int rounds[kAttnMaxRows + 1];                          // of the rows before each row
};

template <int TYPE, int D>
__global__ void __launch_bounds__(Shape<D>::threads, Shape<D>::ctas) attn_decode_kernel(const AttnLaunch a)
{
    constexpr int KC = D / 32;
    constexpr int NJ = TYPE == kQ8 ? D / 8 : (D + 63) / 64 * 8;  // accumulator pairs a lane
    constexpr int kWarps = Shape<D>::warps, kThreads = Shape<D>::threads, kRound = Shape<D>::round;
    constexpr int kSlots = kAttnHeads * D / 4;                   // float4s of a unit's output
    constexpr int kPer = (kSlots + kThreads - 1) / kThreads;
    constexpr size_t part = kAttnHeads * (D + 2);                // attn_part_floats(D)
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<TYPE, D> &sh = *reinterpret_cast<Smem<TYPE, D> *>(raw);
    auto &q_frag = sh.q_frag;
    auto &q_low = sh.q_low;

    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    griddep_wait();  // queries, lengths, tables and the cache may come from the preceding kernels

    // first cached token and rounds of a row of n tokens (n < 0: padding, none; nothing to read: one)
    auto start_of = [&](int n) { return (a.window > 0 ? max(0, n - a.window) : 0) & ~(kAttnTile - 1); };
    auto too_long = [&](int n) { return n > a.max_len || (long long)n > (long long)a.pages_stride * a.page_size; };
    auto rounds_of = [&](int n) { return n < 0 ? 0 : n == 0 || too_long(n) ? 1 : (n - start_of(n) + kRound - 1) / kRound; };

    const int units = a.n_kv_heads * a.subgroups;  // of a row
    const bool shared_out = a.nt <= kAttnMaxRows;  // else a CTA per unit
    long long pos, end;
    long long share = 0;
    if (shared_out) {
        // rounds of the rows before each row
        int before = 0;
        for (int r0 = 0; r0 < a.nt; r0 += kThreads) {
            const int r = r0 + tid;
            const int mine = r < a.nt ? rounds_of(__ldcg(a.lens + r)) : 0;
            int s = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, s, o);
                if (lane >= o) s += v;
            }
            if (lane == 31) sh.sums[warp] = s;
            __syncthreads();
            int all = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) s += all;
                all += sh.sums[w];
            }
            if (r < a.nt) sh.rounds[r] = before + s - mine;
            before += all;
            __syncthreads();
        }
        if (tid == 0) sh.rounds[a.nt] = before;
        __syncthreads();
        const long long all = (long long)before * units;
        share = max((all + gridDim.x - 1) / gridDim.x, 1LL);
        pos = blockIdx.x * share;
        end = min(pos + share, all);
    } else {
        pos = 0, end = 1;
    }

    while (pos < end) {
        // the unit at pos, its rounds and the first of them for this CTA
        int row, unit, rounds, round;
        if (shared_out) {
            const int want = (int)(pos / units);
            int lo = 0, hi = a.nt - 1;  // the last row whose rounds begin at or before
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (sh.rounds[mid] <= want) lo = mid;
                else hi = mid - 1;
            }
            row = lo;
            rounds = sh.rounds[row + 1] - sh.rounds[row];
            const int in_row = (int)(pos - (long long)sh.rounds[row] * units);
            unit = in_row / rounds;
            round = in_row - unit * rounds;
        } else {
            row = blockIdx.x / units;
            unit = blockIdx.x - row * units;
            rounds = rounds_of(__ldcg(a.lens + row));
            if (rounds == 0) return;
            round = 0;
            end = rounds;
        }
        const long long unit_at = pos - round;
        int take = (int)min((long long)(rounds - round), end - pos);
        if (shared_out && rounds <= kAttnWhole) {
            // not cut: it belongs to the share in which it begins
            if (round > 0) {
                pos += rounds - round;
                continue;
            }
            take = rounds;
        }
        pos += take;
        const bool whole = take == rounds;
        const int sg = unit % a.subgroups, kvh = unit / a.subgroups;
        const int head0 = kvh * a.group + sg * kAttnHeads;
        const int heads = min(kAttnHeads, a.group - sg * kAttnHeads);

        const int n = __ldcg(a.lens + row);
        const int seq = a.seq ? __ldcg(a.seq + row) : row;
        bool bad = (unsigned)seq >= (unsigned)a.n_seqs || too_long(n);
        const int first = a.window > 0 ? max(0, n - a.window) : 0;  // tokens [first, n)
        const int from = start_of(n) + round * kRound;
        const int to = min(n, from + take * kRound);
        const int *table = a.pages + (bad ? 0 : (size_t)seq * a.pages_stride);

        // q's fragments: lane (g, t) holds values 32 c + 8 t .. + 7 of head g.  The
        // factor brings the head's largest magnitude to [2^13, 2^14): its parts then
        // hold 22 bits of it, and the scores take the factor back.
        float q_factor = 1.0f;
        {
            float x[KC][8];
            float am = 0.0f;
            const float *src = a.q + row * a.q_stride + (size_t)(head0 + g) * D + 8 * t;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                float4 u = make_float4(0.f, 0.f, 0.f, 0.f), w = u;
                if (g < heads) {
                    u = __ldcg(reinterpret_cast<const float4 *>(src + 32 * c));
                    w = __ldcg(reinterpret_cast<const float4 *>(src + 32 * c + 4));
                }
                x[c][0] = u.x, x[c][1] = u.y, x[c][2] = u.z, x[c][3] = u.w;
                x[c][4] = w.x, x[c][5] = w.y, x[c][6] = w.z, x[c][7] = w.w;
#pragma unroll
                for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(x[c][i]));
            }
            if constexpr (TYPE != kBF16) {
                am = fmaxf(am, __shfl_xor_sync(kFull, am, 1));
                am = fmaxf(am, __shfl_xor_sync(kFull, am, 2));
                // 2^(13 - exponent), within f32's normal range both ways
                const int e = min(max((int)(__float_as_uint(am) >> 23) - 127, -100), 100);
                const float up = __uint_as_float((unsigned)(127 + 13 - e) << 23);
                q_factor = __uint_as_float((unsigned)(127 - 13 + e) << 23);
#pragma unroll
                for (int c = 0; c < KC; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[c][i] *= up;
            }
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                if (c % kWarps != warp) continue;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint4 f;
                    const float *y = &x[c][4 * h];
                    if constexpr (TYPE == kBF16) {
                        uint2 low;
                        split_bf16(y[0], y[1], f.x, f.y, low.x);
                        split_bf16(y[2], y[3], f.z, f.w, low.y);
                        q_low[2 * c + h][lane] = low;
                    } else {
                        split_f16(y[0], y[1], f.x, f.y);
                        split_f16(y[2], y[3], f.z, f.w);
                    }
                    q_frag[2 * c + h][lane] = f;
                }
            }
        }
        __syncthreads();

        const bool capped = a.softcap > 0.0f;
        // score factor: to base 2 at once, or to the score itself when capped
        const float s_factor = q_factor * a.scale * (capped ? 1.0f : kLog2e);
        const float inv_cap = capped ? 1.0f / a.softcap : 0.0f;

        float o[NJ][2];
#pragma unroll
        for (int j = 0; j < NJ; ++j) o[j][0] = o[j][1] = 0.0f;
        float m = -INFINITY, l = 0.0f;  // head g: maximum (base 2) and this lane's part of the sum

        int tok = from + warp * kAttnTile;
        if (!bad && tok < to) {
            const size_t head_off = (size_t)kvh * a.head_bytes;
            auto page_at = [&](int token) {
                const int p = __ldcg(table + token / a.page_size);
                if ((unsigned)p < (unsigned)a.n_pages) return p;
                bad = true;
                return 0;
            };
            Tile<TYPE, D> r;
            int page = page_at(tok), slot = tok % a.page_size;
            load_k<TYPE, D>(r, a.k_pages + page * a.page_stride + head_off, slot, a.page_size, g, t);
            load_v<TYPE, D>(r, a.v_pages + page * a.page_stride + head_off, slot, a.page_size, g, t, first - tok, n - tok);
            int next = tok + kRound;
            int page_next = next < to ? page_at(next) : 0;
            for (;;) {
                // scores of 16 tokens: s[j][e] is token 8 j + 2 t + e, head g
                float s[2][2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if constexpr (TYPE == kQ8) {
                        s[j][0] = s[j][1] = 0.0f;
#pragma unroll
                        for (int c = 0; c < KC; ++c) {
                            const uint32_t w[2] = {r.k[j][c].x ^ 0x80808080u, r.k[j][c].y ^ 0x80808080u};
                            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint4 f = q_frag[2 * c + h][lane];
                                const uint32_t qa[4] = {f.x, f.y, f.z, f.w};
                                mma_f16(acc, qa, codes_f16(w[h], 0x4140), codes_f16(w[h], 0x4342));
                            }
                            s[j][0] = fmaf(acc[0] + acc[2], __half2float(r.ks[2 * j][c]), s[j][0]);
                            s[j][1] = fmaf(acc[1] + acc[3], __half2float(r.ks[2 * j + 1][c]), s[j][1]);
                        }
                    } else {
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int c = 0; c < KC; ++c) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint4 f = q_frag[2 * c + h][lane];
                                const uint32_t qa[4] = {f.x, f.y, f.z, f.w};
                                const uint32_t b0 = h ? r.k[j][c].z : r.k[j][c].x, b1 = h ? r.k[j][c].w : r.k[j][c].y;
                                if constexpr (TYPE == kBF16) {
                                    mma_bf16(acc, qa, b0, b1);
                                    const uint2 low = q_low[2 * c + h][lane];
                                    const uint32_t ql[4] = {low.x, 0u, low.y, 0u};
                                    mma_bf16(acc, ql, b0, b1);
                                } else {
                                    mma_f16(acc, qa, b0, b1);
                                }
                            }
                        }
                        s[j][0] = acc[0] + acc[2];
                        s[j][1] = acc[1] + acc[3];
                    }
                }
                const bool more = next < to;
                // the next tile's K is on its way while this one's probabilities are formed
                if (more) {
                    slot = next % a.page_size;
                    load_k<TYPE, D>(r, a.k_pages + page_next * a.page_stride + head_off, slot, a.page_size, g, t);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = s[j][e] * s_factor;
                        if (capped) x = a.softcap * tanhf(x * inv_cap) * kLog2e;
                        const int tk = tok + 8 * j + 2 * t + e;
                        s[j][e] = tk >= first && tk < n ? x : -INFINITY;
                    }
                float mx = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
                const float m_new = fmaxf(m, mx);
                const float m_use = m_new == -INFINITY ? 0.0f : m_new;  // nothing seen yet: every p is 0
                const float alpha = exp2f(m - m_use);
                m = m_new;
                float p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = exp2f(s[i >> 1][i & 1] - m_use);
                l = fmaf(l, alpha, (p[0] + p[1]) + (p[2] + p[3]));

                if constexpr (TYPE == kQ8) {
                    // the tile's largest V scale to [1/2, 1): 2^shift
                    __half2 big = __half2half2(__ushort_as_half(0));
#pragma unroll
                    for (int i = 0; i < 4; i += 2)
#pragma unroll
                        for (int c = 0; c < KC; ++c) big = __hmax2(big, __habs2(__halves2half2(r.vs[i][c], r.vs[i + 1][c])));
                    float bm = fmaxf(__low2float(big), __high2float(big));
                    bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 1));
                    bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 2));
                    const int e = (int)(__float_as_uint(bm) >> 23) - 126;  // bm < 2^e
                    const float up = __uint_as_float((unsigned)(127 + min(max(-e, -30), 30)) << 23);
                    const float down = __uint_as_float((unsigned)(127 - min(max(-e, -30), 30)) << 23);
                    float ps[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) ps[i] = p[i] * (kPScale * up);
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        uint32_t pa[4];
                        split_f16(ps[0] * __half2float(r.vs[0][c]), ps[1] * __half2float(r.vs[1][c]), pa[0], pa[1]);
                        split_f16(ps[2] * __half2float(r.vs[2][c]), ps[3] * __half2float(r.vs[3][c]), pa[2], pa[3]);
                        // bytes of two tokens side by side
                        const uint32_t x0 = r.v[0][c] ^ 0x80808080u, x1 = r.v[1][c] ^ 0x80808080u;
                        const uint32_t x2 = r.v[2][c] ^ 0x80808080u, x3 = r.v[3][c] ^ 0x80808080u;
                        const uint32_t lo[2] = {__byte_perm(x0, x1, 0x5140), __byte_perm(x0, x1, 0x7362)};
                        const uint32_t hi[2] = {__byte_perm(x2, x3, 0x5140), __byte_perm(x2, x3, 0x7362)};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t sel = (i & 1) ? 0x4342 : 0x4140;
                            float acc[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_f16(acc, pa, codes_f16(lo[i >> 1], sel), codes_f16(hi[i >> 1], sel));
                            const int j = 4 * c + i;
                            o[j][0] = fmaf(o[j][0], alpha, (acc[0] + acc[2]) * down);
                            o[j][1] = fmaf(o[j][1], alpha, (acc[1] + acc[3]) * down);
                        }
                    }
                } else {
                    uint32_t pa[4], pl[4] = {0, 0, 0, 0};
                    if constexpr (TYPE == kBF16) {
                        split_bf16(p[0], p[1], pa[0], pa[1], pl[0]);
                        split_bf16(p[2], p[3], pa[2], pa[3], pl[2]);
                    } else {
                        split_f16(p[0] * kPScale, p[1] * kPScale, pa[0], pa[1]);
                        split_f16(p[2] * kPScale, p[3] * kPScale, pa[2], pa[3]);
                    }
#pragma unroll
                    for (int c = 0; c < Tile<TYPE, D>::VC; ++c) {
                        const uint32_t *v0 = reinterpret_cast<const uint32_t *>(&r.v[0][c]);
                        const uint32_t *v1 = reinterpret_cast<const uint32_t *>(&r.v[1][c]);
                        const uint32_t *v2 = reinterpret_cast<const uint32_t *>(&r.v[2][c]);
                        const uint32_t *v3 = reinterpret_cast<const uint32_t *>(&r.v[3][c]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t sel = (i & 1) ? 0x7632 : 0x5410;
                            const uint32_t b0 = __byte_perm(v0[i >> 1], v1[i >> 1], sel);
                            const uint32_t b1 = __byte_perm(v2[i >> 1], v3[i >> 1], sel);
                            float acc[4] = {0.f, 0.f, 0.f, 0.f};
                            if constexpr (TYPE == kBF16) {
                                mma_bf16(acc, pl, b0, b1);
                                mma_bf16(acc, pa, b0, b1);
                            } else {
                                mma_f16(acc, pa, b0, b1);
                            }
                            const int j = 8 * c + i;
                            o[j][0] = fmaf(o[j][0], alpha, acc[0] + acc[2]);
                            o[j][1] = fmaf(o[j][1], alpha, acc[1] + acc[3]);
                        }
                    }
                }
                if (!more) break;
                load_v<TYPE, D>(r, a.v_pages + page_next * a.page_stride + head_off, slot, a.page_size, g, t, first - next,
                                n - next);
                tok = next;
                next += kRound;
                if (next < to) page_next = page_at(next);
            }
        }
        l += __shfl_xor_sync(kFull, l, 1);
        l += __shfl_xor_sync(kFull, l, 2);
        if (bad) {  // no row, or a page that is not there
            l = __int_as_float(0x7fc00000);
            if (a.status && lane == 0) atomicOr(a.status, 1);
        }

        // the warps meet
        if (t == 0) sh.x_m[warp][g] = m, sh.x_l[warp][g] = l;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int d = value_of<TYPE>(j, e, t);
                if (d < D) sh.x_o[warp][g][d] = o[j][e];
            }
        __syncthreads();
        const float o_scale = TYPE == kBF16 ? 1.0f : 1.0f / kPScale;
        // a cut unit: CTAs cta0 .. cta0 + pieces - 1 have a part of it; every CTA has room for the
        // part of a unit that began before its share (0) and of one that goes on behind it (1)
        const int cta0 = whole ? 0 : (int)(unit_at / share);
        const int pieces = whole ? 1 : (int)((unit_at + rounds - 1) / share) - cta0 + 1;
        auto part_of = [&](int p) { return a.ws_part + (size_t)(2 * (cta0 + p) + (p == 0 ? 1 : 0)) * part; };
        float *const mine = whole ? nullptr : part_of((int)blockIdx.x - cta0);

        float4 done[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int idx = tid + i * kThreads;
            if (idx >= kSlots) continue;
            const int h = idx / (D / 4), d = (idx - h * (D / 4)) * 4;
            float M = sh.x_m[0][h];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sh.x_m[w][h]);
            const float M_use = M == -INFINITY ? 0.0f : M;
            float L = 0.0f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2f(sh.x_m[w][h] - M_use);
                const float4 u = *reinterpret_cast<const float4 *>(&sh.x_o[w][h][d]);
                L = fmaf(sh.x_l[w][h], f, L);
                v.x = fmaf(u.x, f, v.x), v.y = fmaf(u.y, f, v.y);
                v.z = fmaf(u.z, f, v.z), v.w = fmaf(u.w, f, v.w);
            }
            if (!whole) {
                __stcg(reinterpret_cast<float4 *>(mine + 2 * kAttnHeads) + idx, v);
                if (d == 0) __stcg(mine + h, M), __stcg(mine + kAttnHeads + h, L);
            } else {
                const float inv = L == 0.0f ? 0.0f : o_scale / L;
                done[i] = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            }
        }
        __syncthreads();  // the exchange may be used again; the parts are written
        if (!whole) {
            if (tid == 0) {
                __threadfence();  // all of this CTA's part, before it is counted
                const unsigned arrived = atomicAdd(a.ws_cnt + cta0, 1u);
                sh.last = arrived + 1 == (unsigned)pieces;
                if (sh.last) a.ws_cnt[cta0] = 0;  // as the next call expects it
                __threadfence();  // and the others' parts after the count
            }
            __syncthreads();
            if (!sh.last) continue;
            // weights of the pieces: a warp a head
            for (int i = tid; i < pieces * kAttnHeads; i += kThreads)
                sh.weight[i / kAttnHeads][i % kAttnHeads] = __ldcg(part_of(i / kAttnHeads) + i % kAttnHeads);
            __syncthreads();
            for (int h = warp; h < kAttnHeads; h += kWarps) {
                float M = -INFINITY, L = 0.0f;
                for (int p = lane; p < pieces; p += 32) M = fmaxf(M, sh.weight[p][h]);
#pragma unroll
                for (int o2 = 16; o2 > 0; o2 >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o2));
                const float M_use = M == -INFINITY ? 0.0f : M;
                for (int p = lane; p < pieces; p += 32) {
                    const float f = exp2f(sh.weight[p][h] - M_use);
                    L = fmaf(__ldcg(part_of(p) + kAttnHeads + h), f, L);
                    sh.weight[p][h] = f;
                }
#pragma unroll
                for (int o2 = 16; o2 > 0; o2 >>= 1) L += __shfl_xor_sync(kFull, L, o2);
                if (lane == 0) sh.total[h] = L;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int idx = tid + i * kThreads;
                if (idx >= kSlots) continue;
                const int h = idx / (D / 4);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int p = 0; p < pieces; ++p) {
                    const float4 u = __ldcg(reinterpret_cast<const float4 *>(part_of(p) + 2 * kAttnHeads) + idx);
                    const float f = sh.weight[p][h];
                    v.x = fmaf(u.x, f, v.x), v.y = fmaf(u.y, f, v.y);
                    v.z = fmaf(u.z, f, v.z), v.w = fmaf(u.w, f, v.w);
                }
                const float L = sh.total[h];
                const float inv = L == 0.0f ? 0.0f : o_scale / L;
                done[i] = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            }
            __syncthreads();  // the weights have been read
        }
        // rows of out, and their q8 blocks (8 lanes each; every lane joins the shuffles)
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int idx = tid + i * kThreads;
            const int h = idx / (D / 4);
            const bool valid = idx < kSlots && h < heads;
            const float4 v = valid ? done[i] : make_float4(0.f, 0.f, 0.f, 0.f);
            if (valid)
                *reinterpret_cast<float4 *>(a.out + row * a.out_stride + (size_t)head0 * D + (size_t)idx * 4) = v;
            if (a.q8)
                quantize4(v, valid, (long long)head0 * (D / 4) + idx, a.q8 + (size_t)row * a.q8_stride, a.q8_d_off,
                          a.q8_sum_off);
        }
    }
}

constexpr int kMaxDevices = 64;

template <int TYPE, int D>
cudaError_t launch_dim(const AttnLaunch &a, int pdl, cudaStream_t st)
{
    static std::atomic<bool> opted[kMaxDevices];
    const auto kernel = attn_decode_kernel<TYPE, D>;
    constexpr size_t smem = sizeof(Smem<TYPE, D>);
    static_assert(smem * Shape<D>::ctas <= 220 * 1024, "the CTAs of an SM share 228 KB, 1 KB of each reserved");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices || !opted[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) opted[dev].store(true, std::memory_order_release);
    }
    return launch_maybe_pdl(kernel, dim3((unsigned)a.ctas), dim3(Shape<D>::threads), smem, pdl, st, a);
}

template <int TYPE>
cudaError_t launch_type(const AttnLaunch &a, int pdl, cudaStream_t st)
{
    return a.head_dim == 64    ? launch_dim<TYPE, 64>(a, pdl, st)
           : a.head_dim == 96  ? launch_dim<TYPE, 96>(a, pdl, st)
           : a.head_dim == 128 ? launch_dim<TYPE, 128>(a, pdl, st)
                               : launch_dim<TYPE, 256>(a, pdl, st);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnLaunch &a, int pdl, cudaStream_t st)
{
    return a.type == kF16 ? launch_type<kF16>(a, pdl, st)
           : a.type == kBF16 ? launch_type<kBF16>(a, pdl, st)
                             : launch_type<kQ8>(a, pdl, st);
}

}  // namespace mq
