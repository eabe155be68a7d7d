// verify_stream.cu -- the verification of many rows without a filter, in two passes over them.
//
// Without a filter a row's decision needs its largest logit and the sum of its weights alone, and a sequence draws
// in one row, so nothing has to stay on the SM between the steps, as it does where a cluster takes a row (sample.cu):
//   1. chunks of 8192 logits: a chunk's largest, and its weights' sum in units of that. The CTA that finishes a row's
//      last chunk (an atomic count; nobody waits) joins the chunks and decides on the drafted token; the sequence's last row
//      names the row that draws. CTAs of one resident wave share out the chunks, each with its next chunk on the way to
//      shared memory while it works on one.
//   2. a CTA takes a chunk of the row that a sequence draws in, from L2, and of its draft probabilities: the sum of
//      max(0, p - q). The last to finish finds the chunk and in it the token.
// A temperature of 0 takes no second pass: a chunk leaves the first place of its largest logit in place of a sum.
// Rows with a filter are left to the clusters.
//
// What bounds it: 112 rows of 152064, 69 MB of logits and 20 MB of probabilities, which take 13 us: 42.3 us captured. The
// sums 20 of them (3.5 TB/s): a CTA's row ends, each with barriers, an atomic and the next row's sequence, and what a
// launch begins and ends with (one warp left behind to finish a row: no faster); the rest 19 in one wave, its loads one
// behind the other (the sequence's first row, the row, the logits; the last CTA the sums, then the chunk again); 3 in the
// clusters that look for rows with filters. A CTA a chunk with an atomic for each took 26 and 24 us.
//
// Sums: a lane's 32 weights (of tokens 32 apart, wherever among 16 bytes the row begins) in f32, a weight of 2^-t of the
// largest being off by (t 2^-23.5 + 2^-22) of itself at the most (the difference of two logits, its factor, ex2.approx);
// everything above in integers of 2^-42 of the chunk's largest, times that one's weight in the row. In the second pass
// what is left of a token is rounded to units of 2^-42 of the row by itself, so that the pass that finds the chunk and the one
// that finds the token in it add up the same integers; of tokens that have more than 2^-10 of the row, whose errors would not
// vanish among the others', it goes by the draw's weight (for every token: 3 us more). Where nothing is left of p (which
// probabilities that are none leave), the draw goes by the first pass' sums, and in its chunk by the same part of the chunk's
// weights: 32 x 2 rows 48 us instead of 35.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <atomic>

#include "f32x2.cuh"
#include "kernels.h"
#include "verify.cuh"
#include "weights.cuh"

namespace mq {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxDevices = 64;
constexpr int kThreads = 256, kWarps = kThreads / 32, kPer = kVerifyChunk / kThreads;

// A row's logits in places counted from the last 16-byte border at or before it.
struct Row {
    const float *src;
    int shift, lo, hi;

    __device__ __forceinline__ Row(const float *row, int vocab)
    {
        shift = (int)(((uintptr_t)row >> 2) & 3);
        src = row - shift, lo = shift, hi = shift + vocab;
    }
    // Whether every place of a chunk is one of its values.
    __device__ __forceinline__ bool whole(int chunk) const { return chunk * kVerifyChunk >= lo && (chunk + 1) * kVerifyChunk <= hi; }
    // The four values from place p on (a multiple of 4); `none` where there is none.
    __device__ __forceinline__ float4 four(int p, float none) const
    {
        if (p >= lo && p + 4 <= hi) return __ldcg(reinterpret_cast<const float4 *>(src + p));
        float4 v = make_float4(none, none, none, none);
        if (p >= lo && p < hi) v.x = __ldcg(src + p);
        if (p + 1 >= lo && p + 1 < hi) v.y = __ldcg(src + p + 1);
        if (p + 2 >= lo && p + 2 < hi) v.z = __ldcg(src + p + 2);
        if (p + 3 >= lo && p + 3 < hi) v.w = __ldcg(src + p + 3);
        return v;
    }
};

// The weights of two logits, in units of `top`'s: 2^x to 2 ulp of the exponent that Weight forms. A NaN counts as -inf.
struct Fast {
    Two top, hi, lo;

    __device__ __forceinline__ Fast(const Weight &w, float zero)
        : top(two(-zero, -zero)), hi(two(w.c_hi, w.c_hi)), lo(two(w.c_lo, w.c_lo))
    {
    }
    __device__ __forceinline__ Two operator()(float x0, float x1) const
    {
        const Two d = add2(two(x0, x1), top);
        float t0, t1, w0, w1;
        split(fma2(d, hi, mul2(d, lo)), t0, t1);
        // (-inf may be a NaN by now, too: a weight of 0)
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w0) : "f"(fmaxf(t0, -1e30f)));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w1) : "f"(fmaxf(t1, -1e30f)));
        return two(w0, w1);
    }
};

// sum * unit / 2^42: a chunk's sum in its row's units.
__device__ __forceinline__ u64 in_units(u64 sum, u64 unit)
{
    return __umul64hi(sum, unit) << (64 - kFixBits) | (sum * unit) >> kFixBits;
}

__device__ __forceinline__ u64 warp_sum(u64 v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// A sum in units of its own largest weight's, as a part of one whose largest logit is top (which weight has, or 0).
__device__ __forceinline__ u64 joined(u64 sum, float sums_top, float top, const Weight &weight)
{
    if (top == INFINITY) return sums_top == INFINITY ? sum : 0;
    return sums_top == -INFINITY ? 0 : in_units(sum, weight(sums_top));
}

// Adds to a count, with what the CTA wrote before; what the others wrote before theirs can be read after.
__device__ __forceinline__ unsigned arrive(unsigned *count, unsigned by)
{
    unsigned before;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(before) : "l"(count), "r"(by) : "memory");
    return before;
}

// A row whose chunks are there, by one warp; and its sequence, where it is the last of it.
__device__ __forceinline__ void decide(Sequence &of, const VerifyLaunch &a, int row)
{
    const int lane = threadIdx.x & 31;
    if (lane == 0) read_row(of, a, row);
    VerifyRow &ws = a.ws[row];
    Weight weight(of.temperature);
    float tops_of[kVerifyLane];
    u64 sums_of[kVerifyLane];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kVerifyLane; ++j) {
        const int c = lane + 32 * j;
        tops_of[j] = c < a.chunks ? __ldcg(&ws.chunk[c].top) : -INFINITY;
        sums_of[j] = c < a.chunks ? __ldcg(&ws.chunk[c].sum) : 0;
        top = fmaxf(top, tops_of[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    weight.top = top == INFINITY ? 0.0f : top;
    u64 all = 0;
#pragma unroll
    for (int j = 0; j < kVerifyLane; ++j) all += joined(sums_of[j], tops_of[j], top, weight);
    all = warp_sum(all);
    const bool greedy = of.greedy();
    if (greedy) {  // the largest logit's place
        unsigned at = UINT_MAX;
#pragma unroll
        for (int j = kVerifyLane - 1; j >= 0; --j)
            if (lane + 32 * j < a.chunks && tops_of[j] == top) at = min(at, (unsigned)sums_of[j]);
        all = __reduce_min_sync(kAll, at);
    }
    const int n = of.to - of.from;
    VerifyRow &first_ws = a.ws[of.from];
    bool all_met = false;
    if (lane == 0) {
        bool stands = false;
        if (!of.final && top != -INFINITY && of.draft >= 0 && of.draft < a.vocab) {
            float x = fmaxf(__ldcg(a.logits + row * a.stride + of.draft) + 0.0f, -INFINITY);
            if (top == INFINITY) x = x == INFINITY ? 0.0f : -INFINITY;
            stands = greedy ? (u64)of.draft == all : draft_stands(of, weight(x), all);
        }
        ws.chunks_met = 0;  // as the next call expects it
        ws.all = all, ws.top = top, ws.temperature = of.temperature, ws.u_draw = of.u_draw, ws.draft = of.draft;
        ws.outcome = (stands ? 1u : 0u) | (top == -INFINITY ? 2u : 0u);
        all_met = n == 1 || arrive(&first_ws.rows_met, 1) + 1 == (unsigned)n;
        if (all_met) first_ws.rows_met = 0;
    }
    if (!__shfl_sync(kAll, all_met ? 1 : 0, 0)) return;
    __syncwarp();

    // ---- the sequence: its first row whose token does not stand draws (its last row's never does)
    int draws = -1;
    unsigned how = 0;
    for (int r0 = of.from; draws < 0; r0 += 32) {
        const unsigned o = r0 + lane < of.to ? __ldcg(&a.ws[r0 + lane].outcome) : 0;
        const unsigned not_standing = __ballot_sync(kAll, r0 + lane >= of.to || !(o & 1));
        if (not_standing) {
            const int at = __ffs(not_standing) - 1;
            draws = r0 + at, how = __shfl_sync(kAll, o, at);
        }
    }
    const int drawn = greedy && !(how & 2) ? (int)__ldcg(&a.ws[draws].all) : -1;
    for (int i = of.from + lane; i < of.to; i += 32) a.tokens[i] = i < draws ? __ldcg(a.drafts + i) : i == draws ? drawn : -1;
    if (lane == 0) {
        a.counts[of.seq] = draws - of.from + 1;
        if (!(how & 2) && !greedy) first_ws.draw = 2 * draws + (draws + 1 == of.to);  // (nothing to draw from: the token is -1)
    }
}

constexpr int kResident = 3;  // CTAs of the sums on an SM, each with two chunks in shared memory
// Tokens of a chunk that a warp sums, and fours that hold them wherever among 16 bytes the row begins: which weights
// a lane adds up goes by the tokens' numbers, not by their addresses.
constexpr int kSegment = kVerifyChunk / kWarps, kFours = kSegment / 4 + 1;
static_assert(kSegment == 32 * kPer, "a lane's tokens");

__global__ void __launch_bounds__(kThreads, kResident) verify_sums_kernel(const VerifyLaunch a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    float4(*const ring)[kFours] = reinterpret_cast<float4(*)[kFours]>(raw) + (threadIdx.x >> 5) * 2;  // the warp's
    __shared__ Sequence of;
    __shared__ float tops[kVerifyChunks][kWarps];  // of the row's chunks that are this CTA's, warp by warp
    __shared__ u64 sums[kVerifyChunks][kWarps];
    __shared__ bool last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long all_chunks = (long long)a.nt * a.chunks;
    const int begin = (int)(blockIdx.x * all_chunks / gridDim.x), end = (int)((blockIdx.x + 1) * all_chunks / gridDim.x);
    griddep_launch_dependents();
    griddep_wait();  // any of the inputs may come from the preceding kernels

    auto issue = [&](int i) {  // (-inf where the row has no value)
        const int row = i / a.chunks, chunk = i - row * a.chunks, from = chunk * kVerifyChunk + warp * kSegment;
        const Row r(a.logits + row * a.stride, a.vocab);
        const bool whole = from >= r.lo && from + kSegment <= r.hi;
        auto copy = [&](int f, bool inside) {
            const int p = from + 4 * f;
            if (inside || (p >= r.lo && p + 4 <= r.hi))
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(&ring[i & 1][f])), "l"(r.src + p) : "memory");
            else
                ring[i & 1][f] = r.four(p, -INFINITY);
        };
#pragma unroll
        for (int k = 0; k < kSegment / 128; ++k) copy(32 * k + lane, whole);
        if (lane == 0 && r.shift > 0) copy(kSegment / 4, false);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    issue(begin);
    for (int i = begin; i < end;) {
        // ---- the row's chunks that are this CTA's: no warp waits for another
        const int row = i / a.chunks, first = i - row * a.chunks, mine = min(a.chunks - first, end - i);
        __syncthreads();  // the row before has been dealt with
        if (tid == 0) of.seq = -1;
        __syncthreads();
        const bool bad = __syncthreads_or(find_sequence<false>(of, a, row, kThreads));
        if (i == 0) note_starts(a, bad, kThreads);
        const bool to_do = !bad && of.seq >= 0 && (of.greedy() || of.plain(a.vocab)), greedy = of.greedy();
        VerifyRow &ws = a.ws[row];
        if (first == 0 && tid == 0) ws.filtered = !bad && of.seq >= 0 && !to_do, ws.draw = -1;
        Weight weight(of.temperature);
        const int shift = Row(a.logits + row * a.stride, a.vocab).shift;
        for (int c = 0; c < mine; ++c, ++i) {
            if (i + 1 < end) issue(i + 1);
            else asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
            float v[kPer];  // of tokens 32 apart
            const float *const values = reinterpret_cast<const float *>(ring[i & 1]) + shift + lane;
            if (to_do) {
#pragma unroll
                for (int k = 0; k < kPer; ++k) v[k] = values[32 * k];
            }
            __syncwarp();  // the warp's next copies go where these lie
            if (!to_do) continue;
            float top = -INFINITY;
#pragma unroll
            for (float x : v) top = fmaxf(top, x);  // (no NaN)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
            if (greedy) {
                int at = INT_MAX;
#pragma unroll
                for (int k = kPer - 1; k >= 0; --k)
                    if (v[k] == top) at = (first + c) * kVerifyChunk + warp * kSegment + 32 * k + lane;
                at = __reduce_min_sync(kAll, at);
                if (lane == 0) tops[c][warp] = top, sums[c][warp] = (unsigned)at;
                continue;
            }
            const bool infinite = top == INFINITY;  // those logits share the draw: as equal ones
            if (infinite) {
#pragma unroll
                for (float &x : v) x = x == INFINITY ? 0.0f : -INFINITY;
            }
            float sum = 0.0f;
            if (top != -INFINITY) {
                const Fast fast(weight, infinite ? 0.0f : top);
                Two two_sums = two(0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < kPer; k += 2) two_sums = add2(two_sums, fast(v[k], v[k + 1]));
                float s0, s1;
                split(two_sums, s0, s1);
                sum = s0 + s1;
            }
            const u64 all = warp_sum(__float2ull_rn(sum * (float)(1ull << kFixBits)));
            if (lane == 0) tops[c][warp] = top, sums[c][warp] = all;
        }
        if (!to_do) continue;
        __syncthreads();
        if (tid < mine) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, tops[tid][w]);
            weight.top = top == INFINITY ? 0.0f : top;
            u64 s = greedy ? ~0ull : 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                if (!greedy) s += joined(sums[tid][w], tops[tid][w], top, weight);
                else if (tops[tid][w] == top && sums[tid][w] < s) s = sums[tid][w];
            ws.chunk[first + tid].sum = s, ws.chunk[first + tid].top = top;
        }
        __syncthreads();
        if (tid == 0) last = arrive(&ws.chunks_met, mine) + mine == (unsigned)a.chunks;
        __syncthreads();
        if (last && warp == 0) decide(of, a, row);
    }
}

// CTAs of the rest, two on an SM: a thread's 16 logits and 16 probabilities fit its 64 registers at a time.
constexpr int kRestThreads = 512, kRestWarps = kRestThreads / 32, kRestPer = kVerifyChunk / kRestThreads;

__global__ void __launch_bounds__(kRestThreads, 2) verify_rest_kernel(const VerifyLaunch a)
{
    __shared__ u64 sums[kRestWarps], target_at;
    __shared__ int chunk_at;
    __shared__ bool last, from_p;
    __shared__ double part_at;         // of a chunk's sum that lies before the draw
    __shared__ float found[kRestPer];  // of the thread that has the token
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int at = blockIdx.x / a.chunks, chunk = blockIdx.x - at * a.chunks;
    griddep_launch_dependents();
    griddep_wait();
    // a CTA for each chunk of each sequence, or of each row where those are fewer: a sequence's first row knows
    int first = at;
    if (a.n_seqs <= a.nt) {
        first = __ldcg(a.starts + at);
        if ((unsigned)first >= (unsigned)a.nt || first >= __ldcg(a.starts + at + 1)) return;
    }
    const int draw = __ldcg(&a.ws[first].draw);
    if (draw < 0) return;
    const int row = draw >> 1;
    VerifyRow &ws = a.ws[row];
    const float top = __ldcg(&ws.top), u_draw = __ldcg(&ws.u_draw);
    const u64 all = __ldcg(&ws.all);
    const int draft = __ldcg(&ws.draft);
    Weight weight(__ldcg(&ws.temperature));
    const bool final = draw & 1, infinite = top == INFINITY;
    weight.top = infinite ? 0.0f : top;
    Rest rest(all);
    const Row r(a.logits + row * a.stride, a.vocab);
    const float *q = a.draft_probs && !final ? a.draft_probs + row * a.q_stride - r.shift : nullptr;
    const bool fours = q && ((uintptr_t)q & 15) == 0;
    float v[kRestPer];
    Fast fast(weight, weight.top);
    float least = 0x1p-10f / rest.ih;
    // v: what is left of this thread's values of a chunk of places, fours kRestThreads apart or consecutive; or (of_p)
    // their weights alone, of a chunk of tokens, as the first pass has them. Everything is on its way before the first value is
    // used.
    auto place_in = [&](auto consecutive, int c, int k) {
        return c * kVerifyChunk + (decltype(consecutive)::value ? tid * kRestPer + k : (k & ~3) * kRestThreads + tid * 4 + (k & 3));
    };
    auto left = [&](auto consecutive, int c, bool of_p) {
        float t[kRestPer];  // what the draft takes off
        auto place = [&](int k) { return place_in(consecutive, c, k) + (of_p ? r.shift : 0); };
        const bool whole = r.whole(c);
        unsigned heavy = 0;
        if (of_p) {
#pragma unroll
            for (int k = 0; k < kRestPer; ++k) v[k] = place(k) < r.hi ? __ldcg(r.src + place(k)) : -INFINITY;
        } else {
#pragma unroll
            for (int k = 0; k < kRestPer; k += 4) {
                const float4 f = whole ? __ldcg(reinterpret_cast<const float4 *>(r.src + place(k))) : r.four(place(k), -INFINITY);
                v[k] = f.x, v[k + 1] = f.y, v[k + 2] = f.z, v[k + 3] = f.w;
            }
        }
#pragma unroll
        for (int k = 0; k < kRestPer; k += 4) {
            const int p = place(k);
            if (of_p || !q) {
#pragma unroll
                for (int i = 0; i < 4; ++i) t[k + i] = !of_p && !final && p + i - r.shift == draft ? 1.0f : 0.0f;
            } else if (fours && (whole || (p >= r.lo && p + 4 <= r.hi))) {
                const float4 f = __ldcg(reinterpret_cast<const float4 *>(q + p));
                t[k] = f.x, t[k + 1] = f.y, t[k + 2] = f.z, t[k + 3] = f.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) t[k + i] = p + i >= r.lo && p + i < r.hi ? __ldcg(q + p + i) : 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < kRestPer; k += 2) {
            float x0 = v[k], x1 = v[k + 1];
            if (infinite) x0 = x0 == INFINITY ? 0.0f : -INFINITY, x1 = x1 == INFINITY ? 0.0f : -INFINITY;
            // (a q that is NaN counts as 0)
            const Two w = fast(x0, x1);
            rest.quick(w, __saturatef(t[k]), __saturatef(t[k + 1]), v[k], v[k + 1]);
            split(w, x0, x1);
            if (x0 >= least) heavy |= 1u << k;
            if (x1 >= least) heavy |= 2u << k;
        }
        for (; heavy; heavy &= heavy - 1) {
            const int k = __ffs(heavy) - 1, p = place(k & ~3) + (k & 3);
            float x = __ldcg(r.src + p), none_left, exact;
            if (infinite) x = x == INFINITY ? 0.0f : -INFINITY;
            const float taken = of_p ? 0.0f : q ? __saturatef(__ldcg(q + p)) : !final && p - r.shift == draft ? 1.0f : 0.0f;
            rest(weight, x, x, taken, taken, exact, none_left);
#pragma unroll
            for (int i = 0; i < kRestPer; ++i)
                if (i == k) v[i] = exact;
        }
    };
    auto own_sum = [&]() {  // this thread's, in units of 2^-42
        unsigned sum_hi = 0;
        int sum_lo = 0;
#pragma unroll
        for (int k = 0; k < kRestPer; ++k) {
            unsigned h;
            int l;
            fixed_of(v[k], h, l);
            sum_hi += h, sum_lo += l;
        }
        return ((u64)sum_hi << 22) + (u64)(long long)sum_lo;
    };
    left(std::false_type(), chunk, false);
    const u64 mine = warp_sum(own_sum());
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    if (tid == 0) {
        u64 s = 0;
#pragma unroll
        for (int w = 0; w < kRestWarps; ++w) s += sums[w];
        ws.rest[chunk] = s;
        last = arrive(&ws.rest_met, 1) + 1 == (unsigned)a.chunks;
        if (last) ws.rest_met = 0;
    }
    __syncthreads();
    if (!last) return;

    // ---- the token: its chunk, by one warp
    if (warp == 0) {
        u64 s[kVerifyLane], total = 0;
#pragma unroll
        for (int j = 0; j < kVerifyLane; ++j) {
            const int c = lane + 32 * j;
            s[j] = c < a.chunks ? __ldcg(&ws.rest[c]) : 0;
            total += s[j];
        }
        total = warp_sum(total);
        const bool none = total == 0;  // nothing is left (probabilities that are none): from p itself, by the first pass' sums
        if (none) {
#pragma unroll
            for (int j = 0; j < kVerifyLane; ++j) {
                const int c = lane + 32 * j;
                const float t = c < a.chunks ? __ldcg(&ws.chunk[c].top) : -INFINITY;
                s[j] = t == -INFINITY ? 0 : joined(__ldcg(&ws.chunk[c].sum), t, top, weight);
                total += s[j];
            }
            total = warp_sum(total);
        }
        const u64 target = u_draw > 0.0f ? (u_draw < 1.0f ? share_of(u_draw, total, false) : total - 1) : 0;
        u64 before = 0;
#pragma unroll
        for (int j = 0; j < kVerifyLane; ++j) {
            u64 to = s[j];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 u = __shfl_up_sync(kAll, to, o);
                if (lane >= o) to += u;
            }
            if (before + to - s[j] <= target && target < before + to)
                chunk_at = lane + 32 * j, target_at = target - (before + to - s[j]), part_at = (double)target_at / (double)s[j], from_p = none;
            before += __shfl_sync(kAll, to, 31);
        }
    }
    __syncthreads();
    // and in it, in the order of the vocabulary
    if (from_p) {  // weights in units of the chunk's largest, which has one then: the chunk has a sum
        if (!infinite) weight.top = __ldcg(&ws.chunk[chunk_at].top);
        fast = Fast(weight, weight.top), rest.ih = 1.0f, rest.il = 0.0f, least = 0x1p-10f;
    }
    left(std::true_type(), chunk_at, from_p);
    const u64 own = own_sum();
    u64 to = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 u = __shfl_up_sync(kAll, to, o);
        if (lane >= o) to += u;
    }
    if (lane == 31) sums[warp] = to;
    __syncthreads();
    u64 before = to - own, total = 0;
#pragma unroll
    for (int w = 0; w < kRestWarps; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    // (what is left has the same integers in both passes: their sum ends behind the target; p's are the first pass' to some
    // 2^-22, and go by the part of the sum)
    const u64 target = from_p ? min((u64)(part_at * (double)total), total - 1) : target_at;
    if (before <= target && target < before + own) {
        int token = -1;
#pragma unroll
        for (int k = 0; k < kRestPer; ++k) found[k] = v[k];
#pragma unroll 1
        for (int k = 0; k < kRestPer; ++k) {
            const u64 w = fixed_of(found[k]);
            if (before <= target && target < before + w) token = place_in(std::true_type(), chunk_at, k) - (from_p ? 0 : r.shift);
            before += w;
        }
        a.tokens[row] = token;
    }
}

}  // namespace

cudaError_t launch_verify_stream(const VerifyLaunch &a, int sms, int pdl, cudaStream_t st)
{
    static_assert(kVerifyLane * 32 >= kVerifyChunks, "a warp's lanes hold a row's chunks");
    static_assert((long long)kVerifyMaxRows * kVerifyChunks < 1 << 30, "chunks, and rows with a bit, in an int");
    constexpr int room = 2 * kWarps * kFours * 16;
    static std::atomic<bool> opted[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices || !opted[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(verify_sums_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, room);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) opted[dev].store(true, std::memory_order_release);
    }
    const long long chunks = (long long)a.nt * a.chunks;
    const unsigned grid = (unsigned)(chunks < kResident * sms ? chunks : kResident * sms);
    e = launch_maybe_pdl(verify_sums_kernel, dim3(grid), dim3(kThreads), room, pdl, st, a);
    // (the second may start early whatever the caller's setting: it waits for the first before it reads)
    if (e == cudaSuccess)
        e = launch_maybe_pdl(verify_rest_kernel, dim3((unsigned)((a.n_seqs < a.nt ? a.n_seqs : a.nt) * a.chunks)), dim3(kRestThreads), 0, 1, st, a);
    return e;
}

}  // namespace mq
