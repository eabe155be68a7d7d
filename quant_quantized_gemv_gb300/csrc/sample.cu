// sample.cu -- the draw of a token from a row of logits: temperature, top-k,
// top-p, min-p and the inverse of the kept tokens' distribution at a given
// random number.
//
// One cluster of CTAs takes a row: each CTA reads its slice of the row once,
// into shared memory, and everything after that happens there and in the
// cluster's distributed shared memory: one launch, no workspace, no sort of
// the vocabulary.
//   0. a short top-k (up to 56 with 16 CTAs a row, 112 with 8, 224, then 256): every CTA
//      sends the first top_k tokens of its slice, by bins as in 2, to rank 0, which
//      narrows them to few more than top_k, applies every filter and draws: one
//      exchange instead of four (one row of 152064, top-k 40: 12.6 -> 10.5 us). What does
//      not fit its room (long ties) goes on with
//   1. the row's maximum;
//   2. if top-k or top-p is on: the tokens are counted in bins of
//      (max - logit) / temperature, 64 to a factor of two, and the bins summed
//      in 64 groups.  To find the bin where a sum ends, every CTA adds up the
//      groups over the cluster, then the bins of one group;
//   3. top-k ends in the bin where the counts reach k.  With few tokens down
//      to that bin (the usual chain of filters) they alone are gathered in
//      rank 0, which applies every filter and draws; up to 2047 of them too, in the
//      order of the vocabulary, where bins and bytes of the place find top-k's and
//      top-p's last (one row of 152064, top-k 1000: 27 -> 17 us, 64 rows 93 -> 42).
//      Else the bin's tokens are gathered and ranked, which gives the last token
//      kept, as a 64-bit place in the order (logit, then index): every CTA gets the
//      list and ranks its own tokens.  A bin of more tokens than the list holds
//      (ties) is first narrowed by 8 bits of that place at a time;
//   4. top-p: the counts times the bins' weights name a bin.  One pass then sums
//      the weights of all tokens, of those above a window of bins around it and
//      of the window's bins one by one, exactly, and sets the window's tokens
//      aside: that settles the bin (or moves the window), whose tokens are
//      ranked as in 3;
//   5. every CTA sums the weights of its kept tokens in the order of the
//      vocabulary (after 4: the sums above the window, and the window's tokens
//      that were set aside); the sums before it and the random number say which
//      CTA, which thread and which token is drawn.
//
// What bounds it: with many rows the load, the count and step 4's pass one after
// another (64 rows of 152064, flat, top-p 0.9: 63 us, of which loads 6, some 90
// instructions a token 30; each row is read once; greedy 25, temperature alone or
// min-p 33 to 34, top-k 40 38, top-k 1000 42); with few, the steps' barriers.
// Nothing uses 64-bit floating point (a division by every thread took 2.9 us), and
// conversions between float and integer, at an eighth of the rate of an addition,
// are kept to one a weight: the others add 1.5 x 2^23 and take the low bits.
//
// Weights.  w = 2^-t, t = (max - logit) log2(e) / temperature, as an integer in
// units of 2^-42: integer sums do not depend on their order, so neither
// atomics nor the split of the row over CTAs can change a draw.  t is formed
// with its rounding errors carried (max - logit and the product have two parts
// each): with t near 20 one f32 rounding would be 10^-6 of w, and a draw
// compares sums over the whole vocabulary with borders that close.  Then
// t = n - f, |f| <= 1/2, and 2^f - 1 = f ln2 + (f ln2)^2 / 2 + ... to degree 8
// (the rest is under 2^-32) is added to 1 as an integer: w is right to 5 x
// 2^-26 at worst, 2^-27 in the mean.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>
#include <utility>

#include "f32x2.cuh"
#include "kernels.h"

namespace mq {
namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kBins = 4096;
constexpr int kGroups = 64;      // groups of as many bins
constexpr float kBinsPerOctave = 64.0f;
constexpr int kList = 512;       // tokens that rank 0 ranks at once
constexpr int kMine = 1024;      // tokens that a CTA sets aside
constexpr int kSent = 1024;      // tokens that rank 0 chooses from, in equal rooms for the CTAs
constexpr int kLong = 2048;      // places for the tokens of a longer top-k, less one: sums in two halves fit 32 bits
constexpr int kRest = 64;        // of these, what is ranked at once
constexpr int kMostSmall = 256;  // the largest top-k that is chosen so
constexpr int kFew = 128;        // tokens that rank 0 ranks without narrowing them first
constexpr int kMaxCluster = 16;  // CTAs of a row (over 8: the non-portable size)
constexpr int kFixBits = 42;     // a weight of 1 is 2^42
constexpr int kWindow = 25;      // bins whose weights are summed one by one
constexpr int kDigits = 256;     // values of 8 bits of a place
// sums of the exact pass: all, above the window, its bins; the bins' counts; tokens that found no room
constexpr int kSums = 2 + 2 * kWindow + 1;

struct alignas(16) Shared {
    union {
        unsigned cnt[kBins];                     // this CTA's bins
        u64 longer[kLong];                       // rank 0: what a longer top-k may keep, in the order of the vocabulary
        struct {
            u64 mine[kMine];                     // afterwards: its tokens that may matter
            union {
                struct {
                    u64 list[kList], weight[kList];  // the gathered tokens
                };
                u64 extra[kThreads];             // at the end: what each thread's set-aside tokens weigh
            };
        };
    };
    union {
        u64 sums[kSums];                         // the exact pass
        struct {
            u64 digit_w[kDigits];                // narrowing a bin
            unsigned digit_n[kDigits];
        };
    };
    u64 all[kSums];                              // the sums over the cluster
    u64 part[2][kThreads / 32];                  // the exact pass: warps' sums, bins' sums and counts
    unsigned bin_lo[kWindow], bin_hi[kWindow], bin_n[kWindow];
    u64 group_w[kGroups], groups_w[kGroups];     // estimated weights of the groups: this CTA's, the row's
    unsigned group_n[kGroups], groups_n[kGroups];
    unsigned bins_n[kGroups];                    // the row's bins of one group
    u64 sent[kSent];                             // rank 0: every CTA's first tokens
    u64 octave[64];                              // 2^30 2^(-b / 64)
    u64 warp_sums[kThreads / 32];
    float maxes[kMaxCluster];
    int argmax[kMaxCluster], sent_n[kMaxCluster];
    u64 totals[kMaxCluster];
    u64 boundary, narrow_left;
    unsigned list_n, mine_n, at, at_n, narrow_n, narrow_digit;
};
static_assert(kBins / kGroups == 64 && kGroups == 64 && kThreads == 8 * kGroups,
              "8 threads a group, 8 bins a thread; 8 threads a bin of one group");

// Order of the logits as unsigned integers: larger logit, larger key.
__device__ __forceinline__ unsigned key_of(float x)
{
    const unsigned b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(unsigned key)
{
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
// Place in the row's order: larger is earlier (a larger logit, or an equal one of a lower index).
__device__ __forceinline__ u64 place_of(float x, int index)
{
    return (u64)key_of(x) << 32 | (0xffffffffu - (unsigned)index);
}

constexpr float kMagic = 12582912.0f;  // 1.5 x 2^23: a float + this has the rounded integer in its low bits

struct Weight {
    float top, c_hi, c_lo;  // the row's maximum; log2(e) / temperature in two parts

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

    __device__ __forceinline__ u64 operator()(float x) const
    {
        unsigned a[2], m[2];
        int none[2];
        pair(x, x, a, m, none);
        return (u64)a[0] * m[0];
    }
};

// Exclusive prefix sum over the CTA's threads, and the total (all threads call it).
__device__ __forceinline__ u64 block_scan(u64 v, u64 *warp_sums, u64 *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    __syncthreads();  // the last call's sums are read
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    u64 before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const u64 x = warp_sums[w];
        if (w < warp) before += x;
        all += x;
    }
    *total = all;
    return before + s - v;
}

// Where the sums of 64 values (this lane's are number 2 * lane and 2 * lane + 1), in order, reach
// the target: the value's number, and what is before it.  Every lane gets both, and the total.
__device__ __forceinline__ int reach(u64 v0, u64 v1, u64 target, u64 *before, u64 *total)
{
    const int lane = threadIdx.x & 31;
    u64 s = v0 + v1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    const unsigned reached = __ballot_sync(0xffffffffu, s >= target);
    const int at = reached ? __ffs(reached) - 1 : 31;
    u64 b = s - v0 - v1;
    const bool second = b + v0 < target;
    if (second) b += v0;
    *before = __shfl_sync(0xffffffffu, b, at);
    return __shfl_sync(0xffffffffu, 2 * lane + (second ? 1 : 0), at);
}

// A share s < 1 of a sum: its floor, or that rounded up, by the 64 bits behind the point.
__device__ __forceinline__ u64 share_of(float s, u64 all, bool up)
{
    const u64 f = __float2ull_rz(s * 18446744073709551616.0f);
    return __umul64hi(f, all) + (up && f * all != 0 ? 1 : 0);
}

// w / all: the quotient and one correction.
__device__ __forceinline__ float share_f32(u64 w, u64 all)
{
    const float wh = __ull2float_rn(w), ah = __ull2float_rn(all);
    const float wl = __ll2float_rn((long long)(w - __float2ull_rn(wh)));
    const float al = __ll2float_rn((long long)(all - __float2ull_rn(ah)));
    const float q = wh / ah;
    return q + ((fmaf(-q, ah, wh) + wl) - q * al) / ah;
}

// A row's filters and its random number.
struct Filters {
    float u, top_p;
    int top_k;
    u64 floor_w;     // min-p's least weight
    bool by_weight;  // top-p is on

    __device__ __forceinline__ u64 drawn_at(u64 all) const
    {
        return u > 0.0f ? (u < 1.0f ? share_of(u, all, false) : all - 1) : 0;
    }
    __device__ __forceinline__ u64 wanted(u64 all) const { return max(share_of(top_p, all, true), (u64)1); }  // top-p of a sum
};

// The draw from rank 0's longer list: n tokens in the order of the vocabulary, of which top-k keeps those
// before bin `bin` and the first `left` of that bin's `population`.
// A function of its own: its registers are not the kernel's.
__device__ __noinline__ void draw_from_longer(Shared &sh, const Weight weight, const Filters f, const SampleLaunch &a,
                                              int row, int n, int bin, unsigned left, unsigned population)
{
    const int tid = threadIdx.x, lane = tid & 31;
    constexpr int kOwn = kLong / kThreads;
    u64 p[kOwn], w[kOwn];
    unsigned in = 0, in_bin = 0;  // a bit a token
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        const int i = tid * kOwn + j;
        p[j] = i < n ? sh.longer[i] : 0;
        const float x = logit_of((unsigned)(p[j] >> 32));
        w[j] = p[j] ? weight(x) : 0;
        if (p[j] && weight.bin(x) == bin) in_bin |= 1u << j;
    }
    // Of the tokens in play, the place of the one at which their number, or their weights, reach `left`: by
    // coarse bins, bins, then bytes of the place (levels 0, 1, 2..9), until few are left, which are ranked.
    unsigned *const lo = reinterpret_cast<unsigned *>(sh.digit_w), *const hi = lo + kDigits;
    auto settle = [&](unsigned play, int level, u64 left, bool counts, unsigned population) {
        auto digit_of = [&](int j) {
            if (level >= 2) return kDigits - 1 - ((int)(p[j] >> (72 - 8 * level)) & (kDigits - 1));
            const int b = weight.bin(logit_of((unsigned)(p[j] >> 32)));
            return level == 0 ? b / (kBins / kDigits) : b % (kBins / kDigits);
        };
        for (; population > kRest && level < 10; ++level) {
            __syncthreads();
            if (tid < kDigits) sh.digit_n[tid] = lo[tid] = hi[tid] = 0;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
                if (play >> j & 1) {
                    const int d = digit_of(j);
                    atomicAdd(&sh.digit_n[d], 1u);
                    if (!counts) atomicAdd(&lo[d], (unsigned)w[j] & 0x1fffffu), atomicAdd(&hi[d], (unsigned)(w[j] >> 21));
                }
            __syncthreads();
            u64 v[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int d = 8 * lane + j;
                sum += v[j] = counts ? sh.digit_n[d] : ((u64)hi[d] << 21) + lo[d];
            }
            u64 to = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 t = __shfl_up_sync(0xffffffffu, to, o);
                if (lane >= o) to += t;
            }
            const int at = __ffs(__ballot_sync(0xffffffffu, to >= left)) - 1;  // left <= the sum of all
            u64 before = to - sum;
            int digit = 8 * lane;
            bool found = false;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (!found) {
                    found = before + v[j] >= left;
                    if (!found) before += v[j], ++digit;
                }
            digit = __shfl_sync(0xffffffffu, digit, at);
            left -= __shfl_sync(0xffffffffu, before, at);
            population = sh.digit_n[digit];
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
                if ((play >> j & 1) && digit_of(j) != digit) play &= ~(1u << j);
        }
        u64 *const rest = sh.sent, *const rest_w = sh.sent + kRest;
        if (tid == 0) sh.mine_n = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            if (play >> j & 1) {
                const unsigned at = atomicAdd(&sh.mine_n, 1u);
                rest[at] = p[j], rest_w[at] = w[j];
            }
        __syncthreads();
        const int m = (int)sh.mine_n, i = tid / (kThreads / kRest);
        u64 before = 0;
        if (i < m)
            for (int j = tid % (kThreads / kRest); j < m; j += kThreads / kRest)
                if (rest[j] > rest[i]) before += counts ? 1 : rest_w[j];
#pragma unroll
        for (int o = 1; o < kThreads / kRest; o <<= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
        if (i < m && tid % (kThreads / kRest) == 0 && before < left && left <= before + (counts ? 1 : rest_w[i]))
            sh.boundary = rest[i];
        __syncthreads();
        return sh.boundary;
    };
    const u64 last = settle(in_bin, 2, left, true, population);
    u64 sum = 0, all;
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
        if (p[j] >= last) in |= 1u << j, sum += w[j];
    if (f.by_weight) {
        block_scan(sum, sh.warp_sums, &all);
        const u64 end = settle(in, 0, f.wanted(all), false, (unsigned)f.top_k);
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            if (p[j] < end) in &= ~(1u << j);
    }
    sum = 0;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        if (!(in >> j & 1) || w[j] < f.floor_w) w[j] = 0;
        sum += w[j];
    }
    u64 before = block_scan(sum, sh.warp_sums, &all);
    const u64 target = f.drawn_at(all);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        if (before <= target && target < before + w[j]) {
            a.token[row] = (int)~(unsigned)p[j];
            if (a.prob) a.prob[row] = share_f32(w[j], all);
        }
        before += w[j];
    }
}

__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleLaunch a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    Shared &sh = *reinterpret_cast<Shared *>(raw);
    float *xs = reinterpret_cast<float *>(raw + sizeof(Shared));
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int row = blockIdx.x / ranks;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Shared &root = *cluster.map_shared_rank(&sh, 0);

    griddep_launch_dependents();
    for (int i = tid; i < kBins; i += kThreads) sh.cnt[i] = 0;
    if (tid < 64) sh.octave[tid] = __float2uint_rn(exp2f((float)tid * (-1.0f / kBinsPerOctave)) * 1073741824.0f);
    if (tid == 0) sh.list_n = sh.mine_n = 0;
    auto started = cluster.barrier_arrive();
    griddep_wait();  // the logits may come from the preceding kernel

    const float temperature = a.temperature ? __ldcg(a.temperature + row) : 1.0f;
    const float top_p = a.top_p ? __ldcg(a.top_p + row) : 1.0f;
    const float min_p = a.min_p ? __ldcg(a.min_p + row) : 0.0f;
    const int top_k = a.top_k ? __ldcg(a.top_k + row) : 0;
    const float u = __ldcg(a.u + row);

    // this CTA's slice: values [rank * slice, ..) counted from the last 16-byte border at or before the row
    const float *src = a.logits + row * a.stride;
    const int shift = (int)(((uintptr_t)src >> 2) & 3);
    src -= shift;
    const int base = rank * a.slice;  // in shifted places; index = place - shift
    const int lo = shift, hi = shift + a.vocab;
    float mx = -INFINITY;
    // NaN is never drawn (the maximum of NaN and a number is the number); -0 is 0
    auto clean = [&](float v) {
        v = fmaxf(v + 0.0f, -INFINITY);
        mx = fmaxf(mx, v);
        return v;
    };
    // whole groups of four inside the row; the row's first and last groups and the padding one by one
    const int whole = max(0, min(a.slice, (hi & ~3) - base));
#pragma unroll 4
    for (int i = tid * 4; i < whole; i += kThreads * 4) {
        if (base + i < lo) continue;
        const float4 f = __ldcg(reinterpret_cast<const float4 *>(src + base + i));
        *reinterpret_cast<float4 *>(xs + i) = make_float4(clean(f.x), clean(f.y), clean(f.z), clean(f.w));
    }
    for (int i = whole + tid; i < a.seg * kThreads; i += kThreads) {
        const int p = base + i;
        xs[i] = clean(i < a.slice && p >= lo && p < hi ? __ldcg(src + p) : -INFINITY);
    }
    if (base < lo && tid < 4 && whole > 0) {
        const int p = base + tid;
        xs[tid] = clean(p >= lo && p < hi ? __ldcg(src + p) : -INFINITY);
    }

    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) sh.warp_sums[warp] = __float_as_uint(mx);
    __syncthreads();
    float own = -INFINITY;  // this CTA's maximum
    for (int w = 0; w < kThreads / 32; ++w) own = fmaxf(own, __uint_as_float((unsigned)sh.warp_sums[w]));
    cluster.barrier_wait(std::move(started));  // every CTA of the row runs
    const bool single = !(temperature > 0.0f) || top_k == 1 || top_p <= 0.0f || min_p > 1.0f;  // one token is kept

    // log2(e) / temperature in two parts: the quotient, and what its product leaves
    Weight weight;
    weight.c_hi = fminf(1.44269502f / temperature, 5e36f);  // its product with the bins of an octave is finite
    weight.c_lo = (fmaf(-weight.c_hi, temperature, 1.44269502f) + 1.92596299e-8f) / temperature;
    if (!(fabsf(weight.c_lo) < weight.c_hi)) weight.c_lo = 0.0f;  // clamped, or an infinite temperature
    const u64 floor_w = min_p > 0.0f ? __float2ull_ru(min_p * (float)(1ull << kFixBits)) : 0;
    const bool by_count = top_k > 0 && top_k < a.vocab, by_weight = top_p < 1.0f;
    const Filters filters = {u, top_p, top_k, floor_w, by_weight};
    const int first = tid * a.seg;  // this thread's values, in the order of the vocabulary
    auto index_of = [&](int i) { return base + i - shift; };
    auto place = [&](int i) { return place_of(xs[i], index_of(i)); };
    auto drawn_at = [&](u64 all) { return filters.drawn_at(all); };
    auto wanted = [&](u64 all) { return filters.wanted(all); };

    // Ranks the tokens [from, to) of a list of n.  body(i, tokens before i, weights before i) runs in
    // one thread for each of them; several threads share the comparisons of one token.
    auto rank_list = [&](int n, int from, int to, auto &&body) {
        for (int i = tid; i < n; i += kThreads) sh.weight[i] = weight(logit_of((unsigned)(sh.list[i] >> 32)));
        __syncthreads();
        int by = 1;
        while (by < 32 && (to - from) * by * 2 <= kThreads) by *= 2;
        const int i = from + tid / by, sub = tid & (by - 1);
        int before = 0;
        u64 w_before = 0;
        if (i < to) {
            const u64 p = sh.list[i];
            for (int j = sub; j < n; j += by)
                if (sh.list[j] > p) ++before, w_before += sh.weight[j];
        }
        for (int o = 1; o < by; o <<= 1) {
            before += __shfl_xor_sync(0xffffffffu, before, o);
            w_before += __shfl_xor_sync(0xffffffffu, w_before, o);
        }
        if (i < to && sub == 0) body(i, before, w_before);
    };
    // The draw from a list in rank 0 that holds whatever top-k may keep.
    auto draw_from_list = [&](int n) {
        bool in = false;
        int my_i = 0;
        u64 my_w = 0, my_before = 0, all;
        rank_list(n, 0, n, [&](int i, int before_i, u64 w_before) {
            in = before_i < top_k;
            my_i = i, my_before = w_before;
            my_w = in ? sh.weight[i] : 0;
        });
        if (by_weight) {
            block_scan(my_w, sh.warp_sums, &all);
            in = in && my_before < wanted(all);
        }
        in = in && my_w >= floor_w && my_w > 0;
        const u64 kept_w = in ? my_w : 0;
        block_scan(kept_w, sh.warp_sums, &all);
        // in the order of the vocabulary: what is kept before each token
        if (tid < n) sh.weight[tid] = 0;
        __syncthreads();
        if (in) sh.weight[my_i] = kept_w;
        __syncthreads();
        const u64 target = drawn_at(all);
        if (in) {
            const unsigned mine_low = (unsigned)sh.list[my_i];
            u64 sum = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j)
                if ((unsigned)sh.list[j] > mine_low) sum += sh.weight[j];  // a lower index
            if (sum <= target && target < sum + kept_w) {
                a.token[row] = (int)~mine_low;
                if (a.prob) a.prob[row] = share_f32(kept_w, all);
            }
        }
    };

    // A short top-k: every CTA sends its own first top_k tokens, and all of their bin, to rank 0, which
    // chooses and draws. The others leave after one barrier. (Infinities and long ties: below.)
    const int room = kSent / ranks;  // a power of two
    if (!single && by_count && top_k <= min(room - room / 8, kMostSmall)) {
        int sent = 0;
        if (own == INFINITY) sent = kSent + 1;
        else if (own != -INFINITY) {
            weight.top = own;
#pragma unroll 2
            for (int i = tid * 2; i < a.seg * kThreads; i += 2 * kThreads) {
                const float2 x = *reinterpret_cast<const float2 *>(xs + i);
                int b0, b1;
                weight.bins(x.x, x.y, b0, b1);
                if (x.x != -INFINITY) atomicAdd(&sh.cnt[b0], 1u);
                if (x.y != -INFINITY) atomicAdd(&sh.cnt[b1], 1u);
            }
            __syncthreads();
            unsigned n = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) n += sh.cnt[(tid >> 3) * 64 + j * 8 + (tid & 7)];
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
            if ((tid & 7) == 0) sh.group_n[tid >> 3] = n;
            __syncthreads();
            u64 before, all, in_group;
            const int group = reach(sh.group_n[2 * lane], sh.group_n[2 * lane + 1], (u64)top_k, &before, &all);
            int last_bin = kBins - 1;
            sent = (int)all;
            if (all > (u64)top_k) {
                const unsigned *bins = sh.cnt + group * 64;
                const int at = reach(bins[2 * lane], bins[2 * lane + 1], (u64)top_k - before, &in_group, &all);
                last_bin = group * 64 + at;
                sent = (int)(before + in_group) + (int)bins[at];
            }
            if (sent <= room) {
                u64 *to = root.sent + rank * room;
                auto look = [&](float x, int b, int i) {
                    if (b <= last_bin && x != -INFINITY) to[atomicAdd(&sh.mine_n, 1u)] = place(i);
                };
#pragma unroll 2
                for (int i = tid * 2; i < a.seg * kThreads; i += 2 * kThreads) {
                    const float2 x = *reinterpret_cast<const float2 *>(xs + i);
                    int b0, b1;
                    weight.bins(x.x, x.y, b0, b1);
                    look(x.x, b0, i);
                    look(x.y, b1, i + 1);
                }
            }
        }
        if (tid < ranks) {
            Shared &o = *cluster.map_shared_rank(&sh, tid);
            o.sent_n[rank] = sent;
            o.maxes[rank] = own;
        }
        cluster.sync();
        int total = 0;
        bool fits = true;
        float top = -INFINITY;
        for (int r = 0; r < ranks; ++r) {
            fits = fits && sh.sent_n[r] <= room;
            total += sh.sent_n[r];
            top = fmaxf(top, sh.maxes[r]);
        }
        if (fits) {
            if (rank != 0) return;
            if (total == 0) {  // nothing to draw from
                if (tid == 0) {
                    a.token[row] = -1;
                    if (a.prob) a.prob[row] = 0.0f;
                }
                return;
            }
            weight.top = top;
            if (tid == 0) sh.mine_n = 0;
            static_assert(kSent == 2 * kThreads, "two tokens a thread");
            u64 p[2];
            int coarse[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int e = tid + j * kThreads;
                p[j] = (e & (room - 1)) < sh.sent_n[e / room] ? sh.sent[e] : 0;
                coarse[j] = weight.bin(logit_of((unsigned)(p[j] >> 32))) / (kBins / kDigits);
            }
            // To few: by the coarse bin of the last token kept, then by its place in it, 8 bits at a time.
            const int few = max(kFew, top_k);
            int last_coarse = kDigits - 1, bits = -8, kept = total, left = top_k;
            u64 prefix = 0;
            for (; kept > few && bits < 64; bits += 8) {
                __syncthreads();
                if (tid < kDigits) sh.digit_n[tid] = 0;
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (!p[j] || (bits >= 0 && (coarse[j] != last_coarse || (bits > 0 && p[j] >> (64 - bits) != prefix)))) continue;
                    const int digit = bits < 0 ? coarse[j] : kDigits - 1 - ((int)(p[j] >> (56 - bits)) & (kDigits - 1));
                    atomicAdd(&sh.digit_n[digit], 1u);
                }
                __syncthreads();
                unsigned n[8], sum = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += n[j] = sh.digit_n[8 * lane + j];
                unsigned to = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned t = __shfl_up_sync(0xffffffffu, to, o);
                    if (lane >= o) to += t;
                }
                const int at = __ffs(__ballot_sync(0xffffffffu, to >= (unsigned)left)) - 1;  // left <= the sum of all
                int digit = 8 * lane, before = (int)(to - sum), here = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (here == 0) {
                        if (before + (int)n[j] >= left) here = (int)n[j], digit += j;
                        else before += (int)n[j];
                    }
                digit = __shfl_sync(0xffffffffu, digit, at);
                before = __shfl_sync(0xffffffffu, before, at);
                here = __shfl_sync(0xffffffffu, here, at);
                left -= before;
                kept = top_k - left + here;
                if (bits < 0) last_coarse = digit;
                else prefix = prefix << 8 | (u64)(kDigits - 1 - digit);
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (p[j] && (coarse[j] < last_coarse || (coarse[j] == last_coarse && (bits <= 0 || p[j] >> (64 - bits) >= prefix))))
                    sh.list[atomicAdd(&sh.mine_n, 1u)] = p[j];
            __syncthreads();
            draw_from_list((int)sh.mine_n);
            return;
        }
        // the long way begins again
        for (int i = tid; i < kBins; i += kThreads) sh.cnt[i] = 0;
    }

    // the row's maximum
    if (tid < ranks) cluster.map_shared_rank(&sh, tid)->maxes[rank] = own;
    cluster.sync();
    mx = sh.maxes[0];
    for (int r = 1; r < ranks; ++r) mx = fmaxf(mx, sh.maxes[r]);

    if (mx == -INFINITY) {  // nothing to draw from
        if (rank == 0 && tid == 0) {
            a.token[row] = -1;
            if (a.prob) a.prob[row] = 0.0f;
        }
        return;
    }
    if (single) {  // the lowest index of the largest logit
        int best = 0x7fffffff;
        for (int i = tid; i < a.slice; i += kThreads)
            if (xs[i] == mx) {
                best = base + i - shift;
                break;
            }
        for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
        if (lane == 0) sh.warp_sums[warp] = (unsigned)best;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kThreads / 32; ++w) best = min(best, (int)sh.warp_sums[w]);
            root.argmax[rank] = best;
        }
        cluster.sync();
        if (rank == 0 && tid == 0) {
            for (int r = 0; r < ranks; ++r) best = min(best, sh.argmax[r]);
            a.token[row] = best;
            if (a.prob) a.prob[row] = 1.0f;
        }
        return;
    }

    if (mx == INFINITY) {  // those logits share the draw: as equal ones
        for (int i = tid; i < a.seg * kThreads; i += kThreads) xs[i] = xs[i] == mx ? 0.0f : -INFINITY;
        mx = 0.0f;
        __syncthreads();
    }

    weight.top = mx;

    // The filters' last token: logit and index (no filter: every finite logit passes).
    float last_x = -INFINITY;
    int last_i = -4;  // the padding before a row has indexes -3 to -1
    auto passes = [&](float x, int i) { return x > last_x || (x == last_x && index_of(i) <= last_i); };
    auto set_last = [&](u64 p) { last_x = logit_of((unsigned)(p >> 32)), last_i = (int)~(unsigned)p; };

    // This thread's tokens (0: none) into the list of every CTA, or of rank 0 alone; the CTA asks
    // rank 0 for room once.  They are known to fit.
    auto send = [&](u64 p0, u64 p1, bool everywhere) {
        if (tid == 0) sh.at_n = 0;
        __syncthreads();
        const unsigned n = (p0 ? 1 : 0) + (p1 ? 1 : 0);
        unsigned at = 0;
        if (n) at = atomicAdd(&sh.at_n, n);
        __syncthreads();
        if (tid == 0 && sh.at_n) sh.at = atomicAdd(&root.list_n, sh.at_n);
        __syncthreads();
        at += sh.at;
        if (n && at + n <= kList)
            for (int r = 0; r < (everywhere ? ranks : 1); ++r) {
                u64 *to = cluster.map_shared_rank(&sh, r)->list + at;
                to[0] = p0 ? p0 : p1;
                if (n == 2) to[1] = p1;
            }
    };
    // Sends this row's tokens of bins [bin_lo, bin_hi] that pass (and, with bits > 0, of places whose
    // top `bits` bits are prefix).
    auto gather = [&](int bin_lo, int bin_hi, int bits, u64 prefix, bool everywhere) {
        if (tid == 0) sh.mine_n = 0;
        __syncthreads();
        auto look = [&](float x, int b, int i) {
            if (b < bin_lo || b > bin_hi || !passes(x, i)) return;
            const u64 p = place(i);
            if (bits && p >> (64 - bits) != prefix) return;
            const unsigned at = atomicAdd(&sh.mine_n, 1u);
            if (at < kMine) sh.mine[at] = p;
        };
#pragma unroll 2
        for (int i = tid * 2; i < a.seg * kThreads; i += 2 * kThreads) {
            const float2 x = *reinterpret_cast<const float2 *>(xs + i);
            int b0, b1;
            weight.bins(x.x, x.y, b0, b1);
            look(x.x, b0, i);
            look(x.y, b1, i + 1);
        }
        __syncthreads();
        send(tid < (int)sh.mine_n ? sh.mine[tid] : 0, 0, everywhere);
        cluster.sync();
    };
    static_assert(kList <= kThreads, "one token a thread");
    // The last token of a list (in every CTA) whose order is followed until `left` counts or weights
    // are reached: the CTA that sent it finds it and tells the others.
    auto end_of_list = [&](int n, bool counts, u64 left) {
        const int from = sh.at_n ? (int)sh.at : 0, to = min(from + (int)sh.at_n, kList);
        rank_list(n, from, to, [&](int i, int before, u64 w_before) {
            const bool last = counts ? (u64)before + 1 == left : w_before < left && left <= w_before + sh.weight[i];
            if (last)
                for (int r = 0; r < ranks; ++r) cluster.map_shared_rank(&sh, r)->boundary = sh.list[i];
        });
        if (rank == 0 && tid == 0) sh.list_n = 0;
        cluster.sync();
        set_last(sh.boundary);
    };
    // The last token within a bin of `population` tokens that pass.
    auto end_of_bin = [&](int bin, unsigned population, bool counts, u64 left) {
        int bits = 0;
        u64 prefix = 0;
        while (population > kList && bits < 64) {  // a place is one token's: it ends there at the latest
            for (int i = tid; i < kDigits; i += kThreads) sh.digit_n[i] = 0, sh.digit_w[i] = 0;
            __syncthreads();
            for (int j = 0; j < a.seg; ++j) {
                const float x = xs[first + j];
                if (weight.bin(x) != bin || !passes(x, first + j)) continue;
                const u64 p = place(first + j);
                if (bits && p >> (64 - bits) != prefix) continue;
                const int digit = (int)(p >> (56 - bits)) & (kDigits - 1);
                atomicAdd(&sh.digit_n[kDigits - 1 - digit], 1u);
                if (!counts) atomicAdd(&sh.digit_w[kDigits - 1 - digit], weight(x));
            }
            cluster.sync();
            u64 n = 0, w = 0, total;
            if (tid < kDigits)
                for (int r = 0; r < ranks; ++r) {
                    const Shared &o = *cluster.map_shared_rank(&sh, r);
                    n += o.digit_n[tid];
                    w += o.digit_w[tid];
                }
            const u64 v = counts ? n : w;
            const u64 before = block_scan(v, sh.warp_sums, &total);
            if (before < left && left <= before + v)
                sh.narrow_left = left - before, sh.narrow_n = (unsigned)n, sh.narrow_digit = kDigits - 1 - tid;
            cluster.sync();  // and every CTA has read the others' digits
            left = sh.narrow_left;
            population = sh.narrow_n;
            prefix = prefix << 8 | sh.narrow_digit;
            bits += 8;
        }
        gather(bin, bin, bits, prefix, true);
        end_of_list(min((int)population, kList), counts, left);
    };

    bool summed = false;  // `mine` is what this thread's kept tokens weigh
    u64 mine = 0;
    if (by_count || by_weight) {
        // interleaved: the order does not matter here
#pragma unroll 2
        for (int i = tid * 2; i < a.seg * kThreads; i += 2 * kThreads) {
            const float2 x = *reinterpret_cast<const float2 *>(xs + i);
            int b0, b1;
            weight.bins(x.x, x.y, b0, b1);
            if (x.x != -INFINITY) atomicAdd(&sh.cnt[b0], 1u);
            if (x.y != -INFINITY) atomicAdd(&sh.cnt[b1], 1u);
        }
        __syncthreads();
        // a bin's weight in the estimate, 2^-30 of the largest
        auto middle = [&](int b) { return sh.octave[b & 63] >> (b >> 6); };
        {
            unsigned n = 0;
            u64 w = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int b = (tid >> 3) * 64 + j * 8 + (tid & 7);
                const unsigned here = sh.cnt[b];
                n += here;
                if (by_weight) w += here * middle(b);
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                n += __shfl_xor_sync(0xffffffffu, n, o);
                w += __shfl_xor_sync(0xffffffffu, w, o);
            }
            if ((tid & 7) == 0) sh.group_n[tid >> 3] = n, sh.group_w[tid >> 3] = w;
        }
        cluster.sync();
        {
            unsigned n = 0;
            u64 w = 0;
            for (int r = tid & 7; r < ranks; r += 8) {
                const Shared &o = *cluster.map_shared_rank(&sh, r);
                n += o.group_n[tid >> 3];
                w += o.group_w[tid >> 3];
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                n += __shfl_xor_sync(0xffffffffu, n, o);
                w += __shfl_xor_sync(0xffffffffu, w, o);
            }
            if ((tid & 7) == 0) sh.groups_n[tid >> 3] = n, sh.groups_w[tid >> 3] = w;
        }
        __syncthreads();
        // the row's bins of one group
        auto read_group = [&](int group) {
            unsigned n = 0;
            for (int r = tid & 7; r < ranks; r += 8) n += cluster.map_shared_rank(&sh, r)->cnt[group * 64 + (tid >> 3)];
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
            if ((tid & 7) == 0) sh.bins_n[tid >> 3] = n;
            __syncthreads();
        };
        bool cut = false;
        int cut_bin = kBins - 1;
        unsigned cut_left = 0;
        unsigned cut_n = 0;  // tokens of the cut's bin
        u64 cut_w = 0;       // estimated weights down to the cut
        if (by_count) {
            u64 before, n_all;
            const int group = reach(sh.groups_n[2 * lane], sh.groups_n[2 * lane + 1], (u64)top_k, &before, &n_all);
            // -inf is in no bin: with no more than top_k others, top-k leaves everything
            cut = n_all > (u64)top_k;
            if (cut) {
                read_group(group);
                u64 in_group, bins_all;
                const int at = reach(sh.bins_n[2 * lane], sh.bins_n[2 * lane + 1], (u64)top_k - before, &in_group, &bins_all);
                cut_bin = group * 64 + at;
                cut_left = (unsigned)((u64)top_k - before - in_group);
                cut_n = sh.bins_n[at];
                const unsigned cut_to = (unsigned)top_k - cut_left + cut_n;
                const bool longer = cut_to > kList && cut_to < kLong;
                if (longer) {  // how many of them are this CTA's
                    u64 n = 0, own_n;
#pragma unroll
                    for (int j = 0; j < kBins / kThreads; ++j) {
                        const int b = j * kThreads + tid;
                        if (b <= cut_bin) n += sh.cnt[b];
                    }
                    block_scan(n, sh.warp_sums, &own_n);
                    if (tid < ranks) cluster.map_shared_rank(&sh, tid)->sent_n[rank] = (int)own_n;
                }
                cluster.sync();  // nobody reads this CTA's bins for this any more
                if (longer) {
                    int to = 0;
                    for (int r = 0; r < rank; ++r) to += sh.sent_n[r];
                    auto hits_of = [&](int from) {  // of 64 of this thread's up to 128 values
                        u64 hits = 0;
                        for (int j = from; j < min(a.seg, from + 64); j += 2) {
                            const float x0 = xs[first + j], x1 = j + 1 < a.seg ? xs[first + j + 1] : -INFINITY;
                            int b0, b1;
                            weight.bins(x0, x1, b0, b1);
                            hits |= (u64)((b0 <= cut_bin && x0 != -INFINITY ? 1 : 0) |
                                          (b1 <= cut_bin && x1 != -INFINITY ? 2 : 0)) << (j - from);
                        }
                        return hits;
                    };
                    u64 hits0 = hits_of(0), hits1 = hits_of(64), all;
                    to += (int)block_scan((u64)(__popcll(hits0) + __popcll(hits1)), sh.warp_sums, &all);
                    for (; hits0; hits0 &= hits0 - 1) root.longer[to++] = place(first + __ffsll(hits0) - 1);
                    for (; hits1; hits1 &= hits1 - 1) root.longer[to++] = place(first + 63 + __ffsll(hits1));
                    cluster.sync();
                    if (rank == 0) draw_from_longer(sh, weight, filters, a, row, (int)cut_to, cut_bin, cut_left, cut_n);
                    return;
                }
                if (cut_to <= kList) {
                    // everything that can be kept, in one list; rank 0 alone goes on
                    gather(0, cut_bin, 0, 0, false);
                    if (rank == 0) draw_from_list(min((int)sh.list_n, kList));
                    return;
                }
                // the estimate of what top-k keeps, while the bins are at hand
                if (by_weight) {
                    u64 w0 = 0, w1 = 0, none, sum;
                    const int b = 2 * lane;
                    if (b < group) w0 = sh.groups_w[b];
                    if (b + 1 < group) w1 = sh.groups_w[b + 1];
                    if (b <= at) w0 += (b < at ? sh.bins_n[b] : cut_left) * middle(group * 64 + b);
                    if (b + 1 <= at) w1 += (b + 1 < at ? sh.bins_n[b + 1] : cut_left) * middle(group * 64 + b + 1);
                    reach(w0, w1, 1, &none, &sum);
                    cut_w = sum;
                }
            }
        }
        int guess_bin = 0;
        if (by_weight) {
            // where the estimate says that top-p ends
            u64 before, all, none;
            reach(sh.groups_w[2 * lane], sh.groups_w[2 * lane + 1], 1, &before, &all);
            const u64 guess = wanted(cut ? cut_w : all);
            const int group = reach(sh.groups_w[2 * lane], sh.groups_w[2 * lane + 1], guess, &before, &all);
            __syncthreads();  // every warp is done with the cut's bins
            read_group(group);
            const int b = 2 * lane;
            const int at = reach(sh.bins_n[b] * middle(group * 64 + b),
                                 sh.bins_n[b + 1] * middle(group * 64 + b + 1), guess - min(before, guess), &none, &all);
            guess_bin = min(group * 64 + at, cut_bin);
        }
        cluster.sync();  // every CTA has read the others' bins
        if (cut) end_of_bin(cut_bin, cut_n, true, cut_left);
        if (by_weight) {
            int from = max(0, min(guess_bin - kWindow / 2, kBins - kWindow));
            u64 left = 0;
            int bin = 0;
            unsigned population = 0;
            for (;;) {
                // exact sums: all that passes, above the window, the window's bins; its tokens are set aside
                for (int i = tid; i < kSums; i += kThreads) sh.sums[i] = 0;
                if (tid < kWindow) sh.bin_lo[tid] = sh.bin_hi[tid] = sh.bin_n[tid] = 0;
                if (tid == 0) sh.mine_n = 0;
                __syncthreads();
                u64 total = 0, above = 0;
                unsigned aside_bits = 0;  // of up to 32 values: those in the window
                // -inf (weight 0) is in the last bin, which nothing that matters is in
                const unsigned width = min(kWindow, kBins - 1 - from);
                auto pass = [&](auto limited) {
                    auto take = [&](float x, int i, unsigned wa, unsigned wm, int bin_x, int bit) {
                        const int b = bin_x - from;
                        bool in = true;
                        if constexpr (limited.value) in = passes(x, i);
                        if (in) total += (u64)wa * wm;
                        if (in && b < 0) above += (u64)wa * wm;
                        if (in && (unsigned)b < width) aside_bits |= 1u << bit;
                    };
                    unsigned wa[2], wm[2];
                    int bins[2];
                    for (int chunk = first; chunk < first + a.seg; chunk += 32) {
                        const int to = min(first + a.seg, chunk + 32);
                        int i = chunk;
#pragma unroll 2
                        for (; i + 1 < to; i += 2) {
                            const float x0 = xs[i], x1 = xs[i + 1];
                            weight.pair(x0, x1, wa, wm, bins);
                            take(x0, i, wa[0], wm[0], bins[0], i - chunk);
                            take(x1, i + 1, wa[1], wm[1], bins[1], i - chunk + 1);
                        }
                        if (i < to) {
                            weight.pair(xs[i], xs[i], wa, wm, bins);
                            take(xs[i], i, wa[0], wm[0], bins[0], i - chunk);
                        }
                        // room for the warp's at once
                        if (__any_sync(0xffffffffu, aside_bits != 0)) {
                            const unsigned n = __popc(aside_bits);
                            unsigned sum = n;
#pragma unroll
                            for (int o = 1; o < 32; o <<= 1) {
                                const unsigned t = __shfl_up_sync(0xffffffffu, sum, o);
                                if (lane >= o) sum += t;
                            }
                            unsigned room = 0;
                            if (lane == 31) room = atomicAdd(&sh.mine_n, sum);
                            room = __shfl_sync(0xffffffffu, room, 31) + sum - n;
                            for (; aside_bits; aside_bits &= aside_bits - 1, ++room)
                                if (room < kMine) sh.mine[room] = place(chunk + __ffs(aside_bits) - 1);
                        }
                    }
                };
                if (cut) pass(std::true_type());
                else pass(std::false_type());
                mine = above;
                for (int o = 16; o > 0; o >>= 1) {
                    total += __shfl_xor_sync(0xffffffffu, total, o);
                    above += __shfl_xor_sync(0xffffffffu, above, o);
                }
                if (lane == 0) sh.part[0][warp] = total, sh.part[1][warp] = above;
                __syncthreads();
                if (tid < 2) {
                    u64 sum = 0;
                    for (int w = 0; w < kThreads / 32; ++w) sum += sh.part[tid][w];
                    sh.sums[tid] = sum;
                }
                const int aside = (int)sh.mine_n;
                if (aside <= kMine) {
                    // a weight in 21 and 22 bits: 32-bit sums of up to kMine (shared memory adds 32-bit
                    // integers at once, 64-bit ones in a loop that 500 threads would queue for)
                    for (int i = tid; i < aside; i += kThreads) {
                        const float x = logit_of((unsigned)(sh.mine[i] >> 32));
                        const int b = weight.bin(x) - from;
                        const u64 w = weight(x);
                        atomicAdd(&sh.bin_lo[b], (unsigned)w & 0x1fffffu);
                        atomicAdd(&sh.bin_hi[b], (unsigned)(w >> 21));
                        atomicAdd(&sh.bin_n[b], 1u);
                    }
                    __syncthreads();
                    if (tid < kWindow) {
                        sh.sums[2 + tid] = ((u64)sh.bin_hi[tid] << 21) + sh.bin_lo[tid];
                        sh.sums[2 + kWindow + tid] = sh.bin_n[tid];
                    }
                } else {  // no room: from the values again
                    if (tid == 0) sh.sums[kSums - 1] = 1;
                    for (int j = 0; j < a.seg; ++j) {
                        const float x = xs[first + j];
                        const int b = weight.bin(x) - from;
                        if ((unsigned)b >= (unsigned)kWindow || !passes(x, first + j)) continue;
                        atomicAdd(&sh.sums[2 + b], weight(x));
                        atomicAdd(&sh.sums[2 + kWindow + b], 1ull);
                    }
                }
                cluster.sync();
                if (tid < kSums) {
                    u64 s = 0;
#pragma unroll 4
                    for (int r = 0; r < ranks; ++r) s += cluster.map_shared_rank(&sh, r)->sums[tid];
                    sh.all[tid] = s;
                }
                __syncthreads();
                const u64 target = wanted(sh.all[0]);
                u64 w = sh.all[1];
                bool in_window = false;
                if (target > w)
                    for (int b = 0; b < kWindow; ++b) {
                        const u64 here = sh.all[2 + b];
                        if (target <= w + here) {
                            in_window = true;
                            bin = from + b, left = target - w, population = (unsigned)sh.all[2 + kWindow + b];
                            break;
                        }
                        w += here;
                    }
                if (in_window) break;
                from = target <= sh.all[1] ? max(0, from - kWindow) : min(kBins - kWindow, from + kWindow);
                cluster.sync();  // every CTA has read the others' sums
            }
            summed = sh.all[kSums - 1] == 0 && population <= kList;
            if (summed) {
                // the bin's tokens are among those set aside
                const int n = (int)sh.mine_n;
                static_assert(kMine == 2 * kThreads, "two tokens a thread");
                auto of_bin = [&](int i) {
                    const u64 p = i < n ? sh.mine[i] : 0;
                    return p && weight.bin(logit_of((unsigned)(p >> 32))) == bin ? p : 0;
                };
                send(of_bin(tid), of_bin(tid + kThreads), true);
                cluster.sync();
                end_of_list((int)population, false, left);
                // what each thread keeps of them
                sh.extra[tid] = 0;
                __syncthreads();
                for (int i = tid; i < n; i += kThreads) {
                    const u64 p = sh.mine[i];
                    const int at = (int)~(unsigned)p + shift - base;
                    if (passes(xs[at], at)) atomicAdd(&sh.extra[at / a.seg], weight(xs[at]));
                }
                __syncthreads();
                mine += sh.extra[tid];
                summed = floor_w == 0;
            } else {
                cluster.sync();  // every CTA has read the others' sums
                end_of_bin(bin, population, false, left);
            }
        }
    }

    // the kept weights, in the order of the vocabulary
    auto kept = [&](int i) -> u64 {
        const float x = xs[i];
        if (!passes(x, i)) return 0;
        const u64 w = weight(x);
        return w >= floor_w ? w : 0;
    };
    if (!summed) {
        mine = 0;
        auto pass = [&](auto limited, auto floored) {
            auto take = [&](float x, int i, unsigned wa, unsigned wm) {
                bool in = true;
                if constexpr (limited.value) in = passes(x, i);
                if constexpr (floored.value) in = in && (u64)wa * wm >= floor_w;
                if (in) mine += (u64)wa * wm;
            };
            unsigned wa[2], wm[2];
            int bins[2];
            weight.pair(xs[first], xs[first], wa, wm, bins);
            take(xs[first], first, wa[0], wm[0]);
#pragma unroll 3
            for (int i = first + 1; i < first + a.seg; i += 2) {
                const float x0 = xs[i], x1 = xs[i + 1];
                weight.pair(x0, x1, wa, wm, bins);
                take(x0, i, wa[0], wm[0]);
                take(x1, i + 1, wa[1], wm[1]);
            }
        };
        if (last_x > -INFINITY) pass(std::true_type(), std::true_type());
        else if (floor_w > 0) pass(std::false_type(), std::true_type());
        else pass(std::false_type(), std::false_type());
    }
    u64 total;
    u64 before = block_scan(mine, sh.warp_sums, &total);
    if (tid < ranks) cluster.map_shared_rank(&sh, tid)->totals[rank] = total;
    cluster.sync();
    u64 all = 0;
    for (int r = 0; r < ranks; ++r) {
        if (r == rank) before += all;
        all += sh.totals[r];
    }
    // the first token whose sum exceeds u * all: its thread's warp looks for it together
    const u64 target = drawn_at(all);
    const unsigned owner = __ballot_sync(0xffffffffu, before <= target && target < before + mine);
    if (owner) {
        const int from = __ffs(owner) - 1;
        before = __shfl_sync(0xffffffffu, before, from);
        const int start = __shfl_sync(0xffffffffu, first, from);
        for (int j = 0; j < a.seg; j += 32) {
            const int i = start + j + lane;
            const u64 w = j + lane < a.seg ? kept(i) : 0;
            u64 to = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 t = __shfl_up_sync(0xffffffffu, to, o);
                if (lane >= o) to += t;
            }
            if (before + to - w <= target && target < before + to) {
                a.token[row] = index_of(i);
                if (a.prob) a.prob[row] = share_f32(w, all);
            }
            before += __shfl_sync(0xffffffffu, to, 31);
        }
    }
}

constexpr size_t kMaxSmem = 227 * 1024, kSmSmem = 228 * 1024;  // a CTA's most; an SM's (each CTA takes 1 KB more)

// Values of a CTA: whole groups of four; a row may start up to 3 values behind a 16-byte border.
int slice_of(int vocab, int c) { return ((vocab + 3 + c - 1) / c + 3) & ~3; }
// Values of a thread. Odd: the threads' segments lie in different banks.
int seg_of(int slice) { return (slice + kThreads - 1) / kThreads | 1; }
size_t smem_of(int slice) { return sizeof(Shared) + (size_t)seg_of(slice) * kThreads * sizeof(float); }

// CTAs per row: the ones that take the least, counted in values of a slice.  A wave of rows takes what its
// barriers and latencies are worth, kWaveCost, and its values on an SM: one slice, or two where a slice leaves
// room and the rows ask for it.  Clusters do not fill the GPU: `alone` of its SMs can hold one CTA each, `slots`
// is what it holds at once.  Equal costs: the fewer CTAs.  Captured, us, top-k 40 / top-p 0.9 of flat logits /
// min-p, C = 2, 4, 8, 16, the choice last (before the passes without limits took a tenth less):
//   152064 tokens,  1 row:   -, 16.3 / 32.6 / 17.5, 12.5 / 23.7 / 11.7, 10.4 / 20.4 /  8.4   (16)
//                  12 rows:  -, 16.8 / 32.9 / 17.3, 13.6 / 24.5 / 12.3, 14.8 / 28.4 / 12.4   (8)
//                  32 rows:  -, 17.6 / 33.9 / 18.1, 19.0 / 37.2 / 18.9, 27.4 / 67.1 / 26.7   (4)
//                  38 rows:  -, 28.6 / 63.5 / 32.6, 24.7 / 53.2 / 26.1, 30.5 / 77.3 / 31.1   (8)
//                  64 rows:  -, 33.6 / 66.0 / 34.9, 31.8 / 71.9 / 35.3, 44.6 / 118 / 48.7    (4)
//   50257 tokens,  16 rows: 13.9 / 25.6 / 13.3, 11.7 / 19.2 / 9.7, 13.7 / 22.0 / 10.5, 16.0 / 36.5 / 14.2   (4)
//                  64 rows: 14.9 / 26.5 / 14.2, 16.5 / 27.4 / 14.4, 24.0 / 45.0 / 20.7, 36.4 / 96.2 / 37.1  (2)
// CTAs of 1024 threads took longer in every one of these.
constexpr int kWaveCost = 30000;
constexpr int kLeast = 2048;  // values of a slice that are worth a CTA

int cluster_for(int nt, int vocab, int sms)
{
    int best = 16;
    long long least = -1;
    for (int c = 1; c <= 16 && (c == 1 || vocab / c >= kLeast); c <<= 1) {
        const long long slice = (vocab + 3) / c + 1, cost = kWaveCost + (c == 16 ? kWaveCost / 15 : 0);
        if (c < 16 && smem_of(slice_of(vocab, c)) > kMaxSmem) continue;
        const bool two = 2 * (smem_of(slice_of(vocab, c)) + 1024) <= kSmSmem;
        const int percent = c == 16 ? 74 : c == 8 ? 93 : 95;  // of the CTAs that its SMs could hold
        const long long alone = (long long)sms * (c == 16 ? 74 : c == 8 ? 67 : 85) / 100 / c;  // rows
        const long long slots = two ? (long long)sms * 2 * percent / 100 / c : alone;
        if (slots < 1) continue;
        const long long full = nt / slots, rest = nt % slots;
        const long long t = full * (cost + slice * (two ? 2 : 1)) + (rest == 0 ? 0 : cost + slice * (rest > alone ? 2 : 1));
        if (least < 0 || t < least) best = c, least = t;
    }
    return best;
}

constexpr int kMaxDevices = 64;
std::atomic<bool> g_opted[kMaxDevices];

}  // namespace

cudaError_t launch_sample(SampleLaunch a, int sms, int pdl, cudaStream_t st)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices || !g_opted[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) g_opted[dev].store(true, std::memory_order_release);
    }
    const int c = cluster_for(a.nt, a.vocab, sms);
    a.slice = slice_of(a.vocab, c);
    a.seg = seg_of(a.slice);  // what fits shared memory is under 128
    const size_t smem = smem_of(a.slice);
    if (smem > kMaxSmem || a.seg > 128) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.nt * c));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel, a);
}

}  // namespace mq
