// attn_decode.cu -- attention of one new token per row over the paged cache.
//
//   s_j = scale q.k_j (capped: c tanh(s_j / c)),  out = sum p_j v_j / sum p_j,
//   p_j = exp(s_j - max s), in one pass over the tokens with the running
//   maximum m and sum l:  m' = max(m, s),  l = l e^(m - m') + e^(s - m'), and
//   the same for the sum of p v.
//
// A unit of work reads its cached bytes for 1 to 8 query heads of a kv head, a
// handful of operations a byte: the pass is bound by HBM when contexts are long
// and by latency when they are short, never by the tensor cores.  tcgen05
// products would fill 8 of their 128 rows and hand every tile over twice.  Where
// a kv head has more query heads, or several rows name one sequence, each unit
// reads the cache for itself, partly from L2: 16 rows of 16384 tokens over one kv
// head, 8 query heads 28 us, 16 41 us (q8 25 and 37); one row of 32768, 40 and 8
// heads, 28 us, 4 such rows of one sequence 64 us.
//
// Each warp streams its tokens, 16 at a time (a tile), through stages of its
// own in shared memory, filled by 16-byte asynchronous copies: no warp waits for
// another between a unit's first token and its last, and a warp's next tiles are
// on their way, into the next unit too, while it works on one.  Rows are stored
// with their 16-byte chunks permuted (chunk xor a key of the row) so that the
// reads below touch every bank once.
//
// One tile, with m16n8k16 products (lane = 4 g + t):
//   scores: rows 0..7 are the heads (one part of q), rows 8..15 the same heads
//     (the next part of q), columns 8 tokens.  A lane reads 8 consecutive values
//     of token g; which values share a product's k slots is free as long as q's
//     fragments follow, so nothing is exchanged.
//   output: rows again heads and parts of p, k the 16 tokens, columns 8 values
//     of v: a lane reads consecutive values of tokens 2t, 2t+1, 2t+8, 2t+9, and
//     one byte permute pairs two tokens of a value.  The scores' layout is the
//     one p needs, so p never leaves its lane.
// Parts: fp16 holds 11 bits, so q (scaled by a power of two a head) and p
// (times 2^14) go in as hi + lo = 22 bits in the two halves of the 16 rows;
// bf16 holds 8, so three parts in two products.  The cache's values are exact
// in both (int8 codes in fp16).  Results then are as an f32 computation's.
// q8: the scales of K (token, block of 32) multiply the block's partial
// scores; the scales of V multiply p, block by block, in units of the largest
// power of two met so far, to stay in fp16's range.
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
// kAttnWhole rounds or less are not cut: the join costs more than they do.
//
// Measured (GB300, captured): 16 rows of 16384 tokens, 40 and 8 heads of 128:
// f16 and bf16 159 us, 6.68 TB/s of the cache, the rate of a plain copy; q8 117
// us, 4.9 TB/s, bound by 650 instructions a tile (f16: 360), a quarter of them
// to turn codes into fp16.  One row of 32768 tokens: 28.5 us, where the bytes
// take 20; of the rest 3 us pass before the first copy (length, page, launch)
// and 3 in the join.  One row of 117 tokens: 5.1 us, all of it latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "f32x2.cuh"
#include "kernels.h"
#include "q8_block.cuh"

namespace mq {
namespace {

constexpr int kF16 = 1, kBF16 = 2, kQ8 = 3;  // MQ_KV_*
constexpr float kPScale = 16384.0f;          // p's factor in fp16 parts: 2^14
constexpr float kLog2e = 1.4426950408889634f;

// c = a b, or c += a b; bf16 or fp16 operands.
template <bool BF16>
__device__ __forceinline__ void product(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
template <bool BF16>
__device__ __forceinline__ void add_product(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

// 2^x, to 2 ulp; below 2^-126 it is 0.
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// x, y as fp16 parts: hi rounds the value, lo the rest.
__device__ __forceinline__ void split_f16(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = bits(h);
    lo = bits(__floats2half2_rn(x - f.x, y - f.y));
}

__device__ __forceinline__ void split_f16(Two x, uint32_t &hi, uint32_t &lo)
{
    float a, b;
    split(x, a, b);
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    split(fma2(two(f.x, f.y), two(-1.0f, -1.0f), x), a, b);
    hi = bits(h);
    lo = bits(__floats2half2_rn(a, b));
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

// A token's scales, KC fp16 side by side.
template <int KC>
__device__ __forceinline__ void load_scales(__half (&s)[KC], const uint8_t *p)
{
    if constexpr (KC == 8) *reinterpret_cast<uint4 *>(&s[0]) = *reinterpret_cast<const uint4 *>(p);
    else if constexpr (KC == 4) *reinterpret_cast<uint2 *>(&s[0]) = *reinterpret_cast<const uint2 *>(p);
    else if constexpr (KC == 2) *reinterpret_cast<uint32_t *>(&s[0]) = *reinterpret_cast<const uint32_t *>(p);
    else {
#pragma unroll
        for (int i = 0; i < KC; ++i) s[i] = reinterpret_cast<const __half *>(p)[i];
    }
}

// 16 bytes to shared memory, asynchronously; `bytes` of them from src (0: all zero).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t shared_address(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Sizes of a kernel instance.
template <int TYPE, int D>
struct Shape {
    static constexpr int warps = attn_warps(TYPE, D), threads = warps * 32, round = warps * kAttnTile;
    static constexpr int stages = attn_stages(TYPE, D);
    static constexpr int meet = attn_meet_heads(TYPE, D);            // heads the warps exchange at a time
    static constexpr int KC = D / 32;
    static constexpr int row = TYPE == kQ8 ? D : 2 * D;              // bytes of a token's K or V
    static constexpr int pitch = row < 128 ? 128 : row == 192 ? 256 : row;  // the same in a stage: room for the permutation
    static constexpr int matrix = kAttnTile * pitch;
    static constexpr int scales = TYPE == kQ8 ? kAttnTile * KC * 2 : 0;  // bytes of a tile's K or V scales
    static constexpr int stage = 2 * matrix + 2 * scales;            // K, V, K's scales, V's scales
};

// Keys of a row's chunk permutation.  A quarter of a warp reads 16 bytes of K from rows 2k, 2k+1 at 4
// places each, and of V from rows of one parity at 2 places each; of q8's K it reads 32 bytes a row
// from 4 rows in turn, of its V from every other row.
template <int TYPE>
__device__ __forceinline__ int k_key(int row) { return TYPE == kQ8 ? (row & 3) << 1 : (row & 1) << 2 | ((row >> 1) & 3); }
template <int TYPE>
__device__ __forceinline__ int v_key(int row) { return TYPE == kQ8 ? ((row >> 1) & 3) << 1 : row & 7; }

// Place of accumulator j (pair element e) of lane t within a head.
template <int TYPE>
__device__ __forceinline__ int value_of(int j, int e, int t)
{
    return TYPE == kQ8 ? 32 * (j >> 2) + 4 * (2 * t + e) + (j & 3) : 64 * (j >> 3) + 8 * (2 * t + e) + (j & 7);
}

template <int TYPE, int D>
struct Smem {
    using S = Shape<TYPE, D>;
    alignas(128) uint8_t ring[S::warps][S::stages][S::stage];
    float q[S::stages + 1][kAttnHeads][D];                 // queries of the units on their way
    uint4 q_frag[2 * S::KC][32];                           // q's parts as the products take them
    uint2 q_low[TYPE == kBF16 ? 2 * S::KC : 1][32];        // bf16's third part
    union {
        float x_o[S::warps][S::meet][D + 4];               // the warps' exchange
        struct {
            float weight[kAttnMaxCtas][kAttnHeads], mass[kAttnMaxCtas][kAttnHeads];  // the join
        };
    };
    float x_m[S::warps][kAttnHeads], x_l[S::warps][kAttnHeads];
    float total[kAttnHeads];
    int sums[S::warps];
    int last;
    int rounds[kAttnMaxRows + 1], lens[kAttnMaxRows], seqs[kAttnMaxRows];  // rounds of the rows before each row; their tokens, sequences
};

// A place in the line of rounds: a unit, or the part of it that falls to this CTA.
struct Segment {
    int pos;                 // of its first round in the line
    int row, unit;           // unit of the row
    int rounds, round, take; // of the unit; the first one here; how many here
};

template <int TYPE, int D>
__global__ void __launch_bounds__(Shape<TYPE, D>::threads, 1) attn_decode_kernel(const AttnLaunch a)
{
    using S = Shape<TYPE, D>;
    constexpr int KC = S::KC, VC = (D + 63) / 64, NS = S::stages;
    constexpr int NJ = TYPE == kQ8 ? D / 8 : VC * 8;             // accumulator pairs a lane
    constexpr int kWarps = S::warps, kThreads = S::threads, kRound = S::round;
    constexpr int kSlots = kAttnHeads * D / 4;                   // float4s of a unit's output
    constexpr size_t part = kAttnHeads * (D + 2);                // attn_part_floats(D)
    extern __shared__ __align__(128) unsigned char raw[];
    Smem<TYPE, D> &sh = *reinterpret_cast<Smem<TYPE, D> *>(raw);

    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    griddep_wait();  // queries, lengths, tables and the cache may come from the preceding kernels

    // A small page table and the queries to L2 while the lengths are fetched: they lie on the way to the first
    // tile, one behind the other, and a long context's stream leaves nothing of them there. (One row of 32768: 28.6 us
    // without the table, 28.4 with it; by the rows' lengths, once they are there, it takes 28.5 and costs short rows
    // 0.2 us. A large table is mostly of places that no row of the call uses.)
    {
        const unsigned i = blockIdx.x * kThreads + tid;  // 128 bytes a thread
        const size_t entries = (size_t)a.n_seqs * a.pages_stride;
        if (entries <= kAttnTableAhead && (size_t)i * 32 < entries)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.pages + (size_t)i * 32));
        const unsigned lines = a.n_heads * (D / 32), r = i / lines;
        if (r < (unsigned)a.nt)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + r * a.q_stride + (size_t)(i - r * lines) * 32));
    }
    // first cached token and rounds of a row of n tokens (n < 0: padding, none; nothing to read: one).
    // In the line a unit has kAttnUnitCost rounds more, in front: what its beginning and end cost.
    auto first_of = [&](int n) { return a.window > 0 ? max(0, n - a.window) : 0; };
    auto start_of = [&](int n) { return first_of(n) & ~(kAttnTile - 1); };
    auto too_long = [&](int n) { return n > a.max_len || (long long)n > (long long)a.pages_stride * a.page_size; };
    auto rounds_of = [&](int n) { return n < 0 ? 0 : n == 0 || too_long(n) ? 1 : (n - start_of(n) + kRound - 1) / kRound; };

    auto line_of = [&](int n) { return n < 0 ? 0 : rounds_of(n) + kAttnUnitCost; };

    const int units = a.n_kv_heads * a.subgroups;  // of a row
    const bool shared_out = a.nt <= kAttnMaxRows;  // else a CTA per unit
    int end, share = 0, single_n = 0, single_seq = 0;
    Segment load_at;
    if (shared_out) {
        // rounds of the rows before each row: up to 32 rows by every warp for itself
        int before = 0;
        if (a.nt <= 32) {
            const int n = lane < a.nt ? __ldcg(a.lens + lane) : -1;
            const int seq = a.seq && lane < a.nt ? __ldcg(a.seq + lane) : lane;
            const int mine = line_of(n);
            int s = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, s, o);
                if (lane >= o) s += v;
            }
            before = __shfl_sync(kFull, s, 31);
            sh.rounds[lane] = s - mine;  // every warp writes the same
            if (lane < a.nt) sh.lens[lane] = n, sh.seqs[lane] = seq;
            __syncwarp();
        } else for (int r0 = 0; r0 < a.nt; r0 += kThreads) {
            const int r = r0 + tid;
            const int n = r < a.nt ? __ldcg(a.lens + r) : -1;
            const int seq = a.seq && r < a.nt ? __ldcg(a.seq + r) : r;
            const int mine = line_of(n);
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
            if (r < a.nt) sh.rounds[r] = before + s - mine, sh.lens[r] = n, sh.seqs[r] = seq;
            before += all;
            if (r0 + kThreads < a.nt) __syncthreads();
        }
        if (a.nt > 32) {
            if (tid == 0) sh.rounds[a.nt] = before;
            __syncthreads();
        } else if (lane == 0) {
            sh.rounds[a.nt] = before;
        }
        __syncwarp();
        const int all = before * units;
        share = max((int)((all + gridDim.x - 1) / gridDim.x), 1);
        load_at.pos = blockIdx.x * share;
        end = min(load_at.pos + share, all);
        if (load_at.pos >= end) return;
        const int want = load_at.pos / units;
        int lo = 0, hi = a.nt - 1;  // the last row whose rounds begin at or before
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (sh.rounds[mid] <= want) lo = mid;
            else hi = mid - 1;
        }
        load_at.row = lo;
        const int in_row = load_at.pos - sh.rounds[lo] * units, rounds = sh.rounds[lo + 1] - sh.rounds[lo];
        load_at.unit = in_row / rounds;
        load_at.round = in_row - load_at.unit * rounds;
    } else {
        load_at.row = blockIdx.x / units;
        load_at.unit = blockIdx.x - load_at.row * units;
        load_at.pos = load_at.round = 0;
        single_n = __ldcg(a.lens + load_at.row);
        single_seq = a.seq ? __ldcg(a.seq + load_at.row) : load_at.row;
        end = line_of(single_n);
    }
    auto kv_head = [&](int unit) { return a.subgroups == 1 ? unit : unit / a.subgroups; };
    auto n_of = [&](int row) { return shared_out ? sh.lens[row] : single_n; };
    auto seq_of = [&](int row) { return shared_out ? sh.seqs[row] : single_seq; };
    // completes a segment that begins where its fields say (its round counted with the unit's cost; from
    // then on without); false: none is left
    auto enter = [&](Segment &s) {
        for (;;) {
            if (s.pos >= end) return false;
            s.rounds = shared_out ? sh.rounds[s.row + 1] - sh.rounds[s.row] : end;
            s.take = min(s.rounds - s.round, end - s.pos);
            if (s.rounds > kAttnWhole + kAttnUnitCost) {
                if (s.round + s.take <= kAttnUnitCost) return false;  // nothing but the cost: the next CTA begins it
                // to the tokens' rounds
                const int cost = max(kAttnUnitCost - s.round, 0);
                s.pos += cost, s.round += cost, s.take -= cost;
                s.round -= kAttnUnitCost, s.rounds -= kAttnUnitCost;
                return true;
            }
            // not cut: it belongs to the share in which it begins
            if (s.round == 0) {
                s.pos += kAttnUnitCost;
                s.take = s.rounds -= kAttnUnitCost;
                return true;
            }
            s.take = s.rounds - s.round;
            s.pos += s.take, s.round = 0;
            if (++s.unit == units) {
                s.unit = 0;
                do ++s.row;
                while (s.row < a.nt && sh.rounds[s.row + 1] == sh.rounds[s.row]);
            }
        }
    };
    auto leave = [&](Segment &s) {  // to where the next one begins
        s.pos += s.take, s.round = 0;
        if (++s.unit == units) {
            s.unit = 0;
            if (shared_out)
                do ++s.row;
                while (s.row < a.nt && sh.rounds[s.row + 1] == sh.rounds[s.row]);
        }
    };

    // ---- the loading side: rounds ahead of the work
    bool load_live = enter(load_at);
    if (!load_live) return;
    Segment at = load_at;  // the working side
    int load_round = 0, load_count = 0;              // round of the segment; segments begun
    int l_first = 0, l_n = 0, l_from = 0, l_to = 0;
    int l_pages = -1, l_slots = 0;                   // pages and places in them: a lane a round, 32 at a time
    int asked_row = -1, asked_from = 0, asked_to = 0;  // of these tokens: the next unit of the row may need the same
    const int *l_table = nullptr;
    size_t l_head = 0;
    auto open_load = [&]() {
        l_n = n_of(load_at.row);
        const int seq = seq_of(load_at.row);
        const bool bad = (unsigned)seq >= (unsigned)a.n_seqs || too_long(l_n);
        l_first = first_of(l_n);
        l_from = start_of(l_n) + load_at.round * kRound + warp * kAttnTile;
        l_to = bad ? 0 : min(l_n, start_of(l_n) + (load_at.round + load_at.take) * kRound);
        l_table = a.pages + (bad ? 0 : (size_t)seq * a.pages_stride);
        l_head = (size_t)kv_head(load_at.unit) * a.head_bytes;
    };
    auto ask_pages = [&]() {
        if (asked_row == load_at.row && asked_from == l_from && asked_to == l_to) return;
        asked_row = load_at.row, asked_from = l_from, asked_to = l_to;
        const int tok = l_from + lane * kRound;
        if (tok < l_to) {
            const int i = tok / a.page_size;
            l_slots = tok - i * a.page_size;
            l_pages = __ldcg(l_table + i);
        }
    };
    open_load();
    ask_pages();
    unsigned missing = 0;  // stages whose page is not there
    auto issue = [&](int stage) {
        if (load_live) {
            if (load_round == 0) {  // the unit's queries
                const int kvh = kv_head(load_at.unit), sg = load_at.unit - kvh * a.subgroups;
                const int head0 = kvh * a.group + sg * kAttnHeads, heads = min(kAttnHeads, a.group - sg * kAttnHeads);
                const float *src = a.q + load_at.row * a.q_stride + (size_t)head0 * D;
                const uint32_t dst = shared_address(sh.q[load_count % (NS + 1)]);
                for (int i = tid; i < kSlots; i += kThreads)
                    copy16(dst + i * 16, i < heads * (D / 4) ? src + i * 4 : src, i < heads * (D / 4) ? 16 : 0);
            }
            const int l_page = __shfl_sync(kFull, l_pages, load_round & 31);
            const int slot = __shfl_sync(kFull, l_slots, load_round & 31);
            if (l_from < l_to) {
                const bool there = (unsigned)l_page < (unsigned)a.n_pages;
                missing = there ? missing & ~(1u << stage) : missing | 1u << stage;
                const size_t page = (size_t)(there ? l_page : 0) * a.page_stride + l_head;
                const uint8_t *k = a.k_pages + page + (size_t)slot * S::row, *v = a.v_pages + page + (size_t)slot * S::row;
                const uint32_t to = shared_address(sh.ring[warp][stage]);
                constexpr int kChunks = S::row / 16;
#pragma unroll
                for (int j = 0; j < kAttnTile * kChunks / 32; ++j) {
                    const int i = lane + 32 * j, r = i / kChunks, c = i % kChunks;
                    copy16(to + r * S::pitch + ((c ^ k_key<TYPE>(r)) << 4), k + i * 16, 16);
                }
                // V's rows outside [lo, hi) are zeros: p is 0 there, whatever the cache holds
                const int lo = l_first - l_from, hi = l_n - l_from;
                if (lo <= 0 && hi >= kAttnTile) {
#pragma unroll
                    for (int j = 0; j < kAttnTile * kChunks / 32; ++j) {
                        const int i = lane + 32 * j, r = i / kChunks, c = i % kChunks;
                        copy16(to + S::matrix + r * S::pitch + ((c ^ v_key<TYPE>(r)) << 4), v + i * 16, 16);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < kAttnTile * kChunks / 32; ++j) {
                        const int i = lane + 32 * j, r = i / kChunks, c = i % kChunks;
                        copy16(to + S::matrix + r * S::pitch + ((c ^ v_key<TYPE>(r)) << 4), v + i * 16,
                               r >= lo && r < hi ? 16 : 0);
                    }
                }
                if constexpr (TYPE == kQ8) {
                    const size_t scales = (size_t)a.page_size * D + (size_t)slot * (KC * 2);
                    const int i = lane & 15;
                    if (i < 2 * KC)
                        copy16(to + 2 * S::matrix + (lane >> 4) * S::scales + i * 16,
                               (lane < 16 ? a.k_pages : a.v_pages) + page + scales + i * 16, 16);
                }
            }
            ++load_round;
            l_from += kRound;
            if (load_round == load_at.take) {
                leave(load_at);
                load_live = enter(load_at);
                load_round = 0, ++load_count;
                if (load_live) {
                    open_load();
                    ask_pages();
                }
            } else if ((load_round & 31) == 0) {
                ask_pages();
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int s = 0; s < NS; ++s) issue(s);

    // ---- the working side
    const bool capped = a.softcap > 0.0f;
    const float inv_cap = capped ? fminf(1.0f / a.softcap, 3.4e38f) : 0.0f;  // finite: a score of 0 stays 0
    int stage = 0;
    for (int count = 0;; ++count) {
        const int kvh = kv_head(at.unit), sg = at.unit - kvh * a.subgroups;
        const int head0 = kvh * a.group + sg * kAttnHeads, heads = min(kAttnHeads, a.group - sg * kAttnHeads);
        const int n = n_of(at.row), first = first_of(n);
        const int from = start_of(n) + at.round * kRound + warp * kAttnTile;
        const int seq = seq_of(at.row);
        bool bad = (unsigned)seq >= (unsigned)a.n_seqs || too_long(n);
        const int to = bad ? 0 : min(n, start_of(n) + (at.round + at.take) * kRound);
        const bool whole = at.take == at.rounds;

        copies_wait<NS - 1>();
        __syncthreads();  // the queries are there, in every warp's copies
        // q's fragments: lane (g, t) holds values 32 c + 8 t .. + 7 of head g.  The
        // factor brings the head's largest magnitude to [2^13, 2^14): its parts then
        // hold 22 bits of it, and the scores take the factor back.
        float q_factor = 1.0f, up = 1.0f;
        const float *q = sh.q[count % (NS + 1)][g] + 8 * t;
        if constexpr (TYPE != kBF16) {
            float am = 0.0f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const float4 u = *reinterpret_cast<const float4 *>(q + 32 * c);
                const float4 w = *reinterpret_cast<const float4 *>(q + 32 * c + 4);
                am = fmaxf(am, fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(u.z), fabsf(u.w))));
                am = fmaxf(am, fmaxf(fmaxf(fabsf(w.x), fabsf(w.y)), fmaxf(fabsf(w.z), fabsf(w.w))));
            }
            am = fmaxf(am, __shfl_xor_sync(kFull, am, 1));
            am = fmaxf(am, __shfl_xor_sync(kFull, am, 2));
            // 2^(13 - exponent), a normal number as its inverse is: of every finite magnitude down to 2^-113, and what
            // is smaller still keeps its 22 bits
            const int e = min(max((int)(__float_as_uint(am) >> 23) - 127, -113), 127);
            up = __uint_as_float((unsigned)(127 + 13 - e) << 23);
            q_factor = __uint_as_float((unsigned)(127 - 13 + e) << 23);
        }
        for (int i = warp; i < 2 * KC; i += kWarps) {
            const float4 y = *reinterpret_cast<const float4 *>(q + 32 * (i >> 1) + 4 * (i & 1));
            uint4 f;
            if constexpr (TYPE == kBF16) {
                uint2 low;
                split_bf16(y.x, y.y, f.x, f.y, low.x);
                split_bf16(y.z, y.w, f.z, f.w, low.y);
                sh.q_low[i][lane] = low;
            } else {
                split_f16(y.x * up, y.y * up, f.x, f.y);
                split_f16(y.z * up, y.w * up, f.z, f.w);
            }
            sh.q_frag[i][lane] = f;
        }
        __syncthreads();
        // score factor: to base 2 at once, or to the score itself when capped
        const float s_factor = q_factor * a.scale * (capped ? 1.0f : kLog2e);

        Two o[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) o[j] = two(0.0f, 0.0f);
        float m = -INFINITY, l = 0.0f;  // head g: maximum (base 2) and this lane's part of the sum
        int unit_exp = -30;             // q8: the sums of p v are in units of 2^unit_exp

        for (int r = 0; r < at.take; ++r) {
            if (r > 0) copies_wait<NS - 1>();
            __syncwarp();
            const int tok = from + r * kRound;
            if (tok < to) {
                const uint8_t *kt = sh.ring[warp][stage], *vt = kt + S::matrix;
                bad = bad || (missing >> stage & 1);
                // scores of 16 tokens: s[j][e] is token 8 j + 2 t + e, head g
                float s[2][2];
                if constexpr (TYPE == kQ8) {
                    alignas(16) __half ks[4][KC];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        load_scales<KC>(ks[i], vt + S::matrix + (8 * (i >> 1) + 2 * t + (i & 1)) * (KC * 2));
                    Two sum[2] = {two(0.0f, 0.0f), two(0.0f, 0.0f)};
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        const uint4 f0 = sh.q_frag[2 * c][lane], f1 = sh.q_frag[2 * c + 1][lane];
                        const uint32_t q0[4] = {f0.x, f0.y, f0.z, f0.w}, q1[4] = {f1.x, f1.y, f1.z, f1.w};
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint2 w = *reinterpret_cast<const uint2 *>(kt + (8 * j + g) * S::pitch +
                                                                       (((2 * c + (t >> 1)) ^ k_key<TYPE>(g)) << 4) + (t & 1) * 8);
                            w.x ^= 0x80808080u, w.y ^= 0x80808080u;
                            float acc[4];
                            product<false>(acc, q0, codes_f16(w.x, 0x4140), codes_f16(w.x, 0x4342));
                            add_product<false>(acc, q1, codes_f16(w.y, 0x4140), codes_f16(w.y, 0x4342));
                            sum[j] = fma2(add2(two(acc[0], acc[1]), two(acc[2], acc[3])),
                                          two(__half2float(ks[2 * j][c]), __half2float(ks[2 * j + 1][c])), sum[j]);
                        }
                    }
                    split(sum[0], s[0][0], s[0][1]);
                    split(sum[1], s[1][0], s[1][1]);
                } else {
                    float acc[2][4], low_acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        uint4 k[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            k[j] = *reinterpret_cast<const uint4 *>(kt + (8 * j + g) * S::pitch +
                                                                    (((4 * c + t) ^ k_key<TYPE>(g)) << 4));
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 f = sh.q_frag[2 * c + h][lane];
                            const uint32_t qa[4] = {f.x, f.y, f.z, f.w};
                            uint32_t ql[4] = {0, 0, 0, 0};
                            if constexpr (TYPE == kBF16) {
                                const uint2 low = sh.q_low[2 * c + h][lane];
                                ql[0] = low.x, ql[2] = low.y;
                            }
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint32_t b0 = h ? k[j].z : k[j].x, b1 = h ? k[j].w : k[j].y;
                                if (c + h == 0) {
                                    product<TYPE == kBF16>(acc[j], qa, b0, b1);
                                    if constexpr (TYPE == kBF16) product<true>(low_acc[j], ql, b0, b1);
                                } else {
                                    add_product<TYPE == kBF16>(acc[j], qa, b0, b1);
                                    if constexpr (TYPE == kBF16) add_product<true>(low_acc[j], ql, b0, b1);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        s[j][0] = TYPE == kBF16 ? acc[j][0] + (acc[j][2] + low_acc[j][0]) : acc[j][0] + acc[j][2];
                        s[j][1] = TYPE == kBF16 ? acc[j][1] + (acc[j][3] + low_acc[j][1]) : acc[j][1] + acc[j][3];
                    }
                }
                const bool full = tok >= first && tok + kAttnTile <= n;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = s[j][e] * s_factor;
                        if (capped) x = a.softcap * tanhf(x * inv_cap) * kLog2e;
                        s[j][e] = x;
                    }
                if (!full) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int tk = tok + 8 * j + 2 * t + e;
                            if (tk < first || tk >= n) s[j][e] = -INFINITY;
                        }
                }
                float mx = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
                const float m_new = fmaxf(m, mx);
                const float m_use = m_new == -INFINITY ? 0.0f : m_new;  // nothing seen yet: every p is 0
                float alpha = ex2(m - m_use);
                m = m_new;
                float p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = ex2(s[i >> 1][i & 1] - m_use);
                l = fmaf(l, alpha, (p[0] + p[1]) + (p[2] + p[3]));

                if constexpr (TYPE == kQ8) {
                    alignas(16) __half vs[4][KC];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 8 * (i >> 1) + 2 * t + (i & 1);
                        load_scales<KC>(vs[i], vt + S::matrix + S::scales + row * (KC * 2));
                        if (!full && (tok + row < first || tok + row >= n)) {
#pragma unroll
                            for (int c = 0; c < KC; ++c) vs[i][c] = __ushort_as_half(0);
                        }
                    }
                    // the largest scale met: below 2^unit_exp
                    __half2 big = __half2half2(__ushort_as_half(0));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int c = 0; c < KC; c += 2)
                            big = __hmax2(big, __habs2(__halves2half2(vs[i][c], vs[i][c + 1 < KC ? c + 1 : c])));
                    float bm = fmaxf(__low2float(big), __high2float(big));
                    bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 1));
                    bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 2));
                    const int e = max(unit_exp, min((int)(__float_as_uint(bm) >> 23) - 126, 30));
                    alpha *= __uint_as_float((unsigned)(127 + unit_exp - e) << 23);
                    unit_exp = e;
                    const Two alpha2 = two(alpha, alpha);
                    const float up_p = kPScale * __uint_as_float((unsigned)(127 - e) << 23);
                    const Two ps[2] = {mul2(two(p[0], p[1]), two(up_p, up_p)), mul2(two(p[2], p[3]), two(up_p, up_p))};
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        uint32_t pa[4];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            split_f16(mul2(ps[i], two(__half2float(vs[2 * i][c]), __half2float(vs[2 * i + 1][c]))), pa[2 * i],
                                      pa[2 * i + 1]);
                        uint32_t x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i] = 0x80808080u ^ *reinterpret_cast<const uint32_t *>(
                                                     vt + (8 * (i >> 1) + 2 * t + (i & 1)) * S::pitch +
                                                     (((2 * c + (g >> 2)) ^ v_key<TYPE>(2 * t)) << 4) + (g & 3) * 4);
                        // bytes of two tokens side by side
                        const uint32_t lo[2] = {__byte_perm(x[0], x[1], 0x5140), __byte_perm(x[0], x[1], 0x7362)};
                        const uint32_t hi[2] = {__byte_perm(x[2], x[3], 0x5140), __byte_perm(x[2], x[3], 0x7362)};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t sel = (i & 1) ? 0x4342 : 0x4140;
                            float acc[4];
                            product<false>(acc, pa, codes_f16(lo[i >> 1], sel), codes_f16(hi[i >> 1], sel));
                            const int j = 4 * c + i;
                            o[j] = fma2(o[j], alpha2, add2(two(acc[0], acc[1]), two(acc[2], acc[3])));
                        }
                    }
                } else {
                    const Two alpha2 = two(alpha, alpha);
                    uint32_t pa[4], pl[4] = {0, 0, 0, 0};
                    if constexpr (TYPE == kBF16) {
                        split_bf16(p[0], p[1], pa[0], pa[1], pl[0]);
                        split_bf16(p[2], p[3], pa[2], pa[3], pl[2]);
                    } else {
                        split_f16(p[0] * kPScale, p[1] * kPScale, pa[0], pa[1]);
                        split_f16(p[2] * kPScale, p[3] * kPScale, pa[2], pa[3]);
                    }
#pragma unroll
                    for (int c = 0; c < VC; ++c) {
                        uint4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = *reinterpret_cast<const uint4 *>(vt + (8 * (i >> 1) + 2 * t + (i & 1)) * S::pitch +
                                                                    ((8 * c + (g ^ v_key<TYPE>(2 * t + (i & 1)))) << 4));
                        const uint32_t *v0 = reinterpret_cast<const uint32_t *>(&v[0]), *v1 = v0 + 4, *v2 = v0 + 8, *v3 = v0 + 12;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t sel = (i & 1) ? 0x7632 : 0x5410;
                            const uint32_t b0 = __byte_perm(v0[i >> 1], v1[i >> 1], sel);
                            const uint32_t b1 = __byte_perm(v2[i >> 1], v3[i >> 1], sel);
                            float acc[4];
                            if constexpr (TYPE == kBF16) {
                                product<true>(acc, pl, b0, b1);
                                add_product<true>(acc, pa, b0, b1);
                            } else {
                                product<false>(acc, pa, b0, b1);
                            }
                            const int j = 8 * c + i;
                            o[j] = fma2(o[j], alpha2, add2(two(acc[0], acc[1]), two(acc[2], acc[3])));
                        }
                    }
                }
            }
            __syncwarp();  // the stage has been read
            issue(stage);
            stage = stage + 1 == NS ? 0 : stage + 1;
        }
        l += __shfl_xor_sync(kFull, l, 1);
        l += __shfl_xor_sync(kFull, l, 2);
        if (bad) {  // no row, or a page that is not there
            l = __int_as_float(0x7fc00000);
            if (a.status && lane == 0) atomicOr(a.status, 1);
        }

        // the warps meet, S::meet heads at a time
        const float o_unit = TYPE == kBF16 ? 1.0f : (1.0f / kPScale) * (TYPE == kQ8 ? __uint_as_float((unsigned)(127 + unit_exp) << 23) : 1.0f);
        if (t == 0) sh.x_m[warp][g] = m, sh.x_l[warp][g] = l;
        // a cut unit: CTAs cta0 .. cta0 + pieces - 1 have a part of it; every CTA has room for the
        // part of a unit that began before its share (0) and of one that goes on behind it (1)
        const int unit_at = at.pos - at.round;  // of the unit's first tokens
        const int cta0 = whole ? 0 : unit_at / share;
        const int pieces = whole ? 1 : (unit_at + at.rounds - 1) / share - cta0 + 1;
        const int row = at.row;
        auto part_of = [&](int p) { return a.ws_part + (size_t)(2 * (cta0 + p) + (p == 0 ? 1 : 0)) * part; };
        float *const mine = whole ? nullptr : part_of((int)blockIdx.x - cta0);
        // four values of out, and their share of a q8 block (8 lanes; every lane joins the shuffles)
        auto emit = [&](int idx, bool in_range, float4 v) {
            const bool valid = in_range && idx / (D / 4) < heads;
            if (valid)
                *reinterpret_cast<float4 *>(a.out + row * a.out_stride + (size_t)head0 * D + (size_t)idx * 4) = v;
            if (a.q8)
                quantize4(valid ? v : make_float4(0.f, 0.f, 0.f, 0.f), valid, (long long)head0 * (D / 4) + idx,
                          a.q8 + (size_t)row * a.q8_stride, a.q8_d_off, a.q8_sum_off);
        };
#pragma unroll
        for (int h0 = 0; h0 < kAttnHeads; h0 += S::meet) {
            if (h0 > 0) __syncthreads();  // the heads before have been read
            if (g >= h0 && g < h0 + S::meet) {
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    float x[2];
                    split(mul2(o[j], two(o_unit, o_unit)), x[0], x[1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d = value_of<TYPE>(j, e, t);
                        if (d < D) sh.x_o[warp][g - h0][d] = x[e];
                    }
                }
            }
            __syncthreads();
            constexpr int kMeet = S::meet * D / 4;  // float4s of these heads
#pragma unroll 1
            for (int i0 = 0; i0 < kMeet; i0 += kThreads) {
                if (kMeet > kThreads && h0 + i0 / (D / 4) >= heads) break;  // heads that do not exist: a turn less
                const int i = i0 + tid, hh = i / (D / 4), d = (i - hh * (D / 4)) * 4, h = h0 + hh;
                const bool in_range = i < kMeet;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (in_range) {
                    float M = sh.x_m[0][h];
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sh.x_m[w][h]);
                    const float M_use = M == -INFINITY ? 0.0f : M;
                    float L = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float f = ex2(sh.x_m[w][h] - M_use);
                        const float4 u = *reinterpret_cast<const float4 *>(&sh.x_o[w][hh][d]);
                        L = fmaf(sh.x_l[w][h], f, L);
                        v.x = fmaf(u.x, f, v.x), v.y = fmaf(u.y, f, v.y);
                        v.z = fmaf(u.z, f, v.z), v.w = fmaf(u.w, f, v.w);
                    }
                    if (!whole) {
                        __stcg(reinterpret_cast<float4 *>(mine + 2 * kAttnHeads) + h0 * (D / 4) + i, v);
                        if (d == 0) __stcg(mine + h, M), __stcg(mine + kAttnHeads + h, L);
                    } else {
                        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
                        v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                    }
                }
                if (whole) emit(h0 * (D / 4) + i, in_range, v);
            }
        }
        if (!whole) {
            __syncthreads();  // the parts are written; the exchange has been read
            if (tid == 0) {
                // this CTA's part (all of it: the barrier) before the count, the others' after it
                unsigned arrived;
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(arrived) : "l"(a.ws_cnt + cta0) : "memory");
                sh.last = arrived + 1 == (unsigned)pieces;
                if (sh.last) a.ws_cnt[cta0] = 0;  // as the next call expects it
            }
            __syncthreads();
            if (sh.last) {
                // the pieces' values are asked for before their weights are known: kAhead at a time
                constexpr int kAhead = 16;
                float4 u[kAhead];
                auto ask = [&](int idx, int p0) {
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) {
                        u[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (idx < kSlots && p0 + k < pieces)
                            u[k] = __ldcg(reinterpret_cast<const float4 *>(part_of(p0 + k) + 2 * kAttnHeads) + idx);
                    }
                };
                ask(tid, 0);
                // weights of the pieces: a warp a head
                for (int h = warp; h < kAttnHeads; h += kWarps) {
                    float M = -INFINITY, L = 0.0f;
                    for (int p = lane; p < pieces; p += 32) {
                        sh.weight[p][h] = __ldcg(part_of(p) + h);
                        sh.mass[p][h] = __ldcg(part_of(p) + kAttnHeads + h);
                        M = fmaxf(M, sh.weight[p][h]);
                    }
#pragma unroll
                    for (int o2 = 16; o2 > 0; o2 >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o2));
                    const float M_use = M == -INFINITY ? 0.0f : M;
                    for (int p = lane; p < pieces; p += 32) {
                        const float f = ex2(sh.weight[p][h] - M_use);
                        L = fmaf(sh.mass[p][h], f, L);
                        sh.weight[p][h] = f;
                    }
#pragma unroll
                    for (int o2 = 16; o2 > 0; o2 >>= 1) L += __shfl_xor_sync(kFull, L, o2);
                    if (lane == 0) sh.total[h] = L;
                }
                __syncthreads();
#pragma unroll 1
                for (int i0 = 0; i0 < kSlots; i0 += kThreads) {
                    if (kSlots > kThreads && i0 / (D / 4) >= heads) break;
                    const int idx = i0 + tid, h = min(idx / (D / 4), kAttnHeads - 1);
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int p0 = 0; p0 < pieces; p0 += kAhead) {
                        if (i0 + p0 > 0) ask(idx, p0);
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            if (p0 + k >= pieces) break;
                            const float f = sh.weight[p0 + k][h];
                            v.x = fmaf(u[k].x, f, v.x), v.y = fmaf(u[k].y, f, v.y);
                            v.z = fmaf(u[k].z, f, v.z), v.w = fmaf(u[k].w, f, v.w);
                        }
                    }
                    const float L = sh.total[h];
                    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
                    emit(idx, idx < kSlots, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                }
            }
        }
        leave(at);
        if (!enter(at)) break;
        // the barrier at the next unit's start keeps the exchange until every thread has read it
    }
}

constexpr int kMaxDevices = 64;

template <int TYPE, int D>
cudaError_t launch_dim(const AttnLaunch &a, int pdl, cudaStream_t st)
{
    static std::atomic<bool> opted[kMaxDevices];
    const auto kernel = attn_decode_kernel<TYPE, D>;
    constexpr size_t smem = sizeof(Smem<TYPE, D>);
    static_assert(smem <= 227 * 1024, "what a CTA may have");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices || !opted[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) opted[dev].store(true, std::memory_order_release);
    }
    return launch_maybe_pdl(kernel, dim3((unsigned)a.ctas), dim3(Shape<TYPE, D>::threads), smem, pdl, st, a);
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
