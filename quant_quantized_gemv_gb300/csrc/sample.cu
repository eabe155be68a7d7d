// sample.cu -- the draw of a token from a row of logits: temperature, top-k,
// top-p, min-p and the inverse of the kept tokens' distribution at a given
// random number.
//
// One cluster of CTAs takes a row: each CTA reads its slice of the row once,
// into shared memory, and everything after that happens there and in the
// cluster's distributed shared memory: one launch, no workspace, no sort of
// the vocabulary.
//   1. the row's maximum;
//   2. if top-k or top-p is on: counts and weight sums of the tokens in bins
//      of (max - logit) / temperature, 32 to a factor of two; the CTAs add
//      theirs into rank 0's, which finds the bin where the filter ends;
//   3. the tokens of that bin alone are gathered in rank 0 and ranked, which
//      gives the last token kept, as a 64-bit place in the order (logit, then
//      index).  A bin of more tokens than the list holds (ties, flat logits)
//      is first narrowed by 11 bits of that place at a time;
//   4. every CTA sums the weights of its kept tokens in the order of the
//      vocabulary; the sums before it and the random number say which CTA,
//      which thread and which token the draw falls on.
//
// Weights.  w = 2^-t, t = (max - logit) log2(e) / temperature, as an integer in
// units of 2^-42: integer sums do not depend on their order, so neither the
// bins' atomics nor the split of the row over CTAs can change a draw.  t is
// formed with its rounding errors carried (max - logit and the product have
// two parts each): with t near 20 one f32 rounding would be 10^-6 of w, and a
// draw compares sums over the whole vocabulary with borders that close.  Then
// t = n - f, |f| <= 1/2, and 2^f - 1 = f ln2 + (f ln2)^2 / 2 + ... to degree 8
// (the rest is under 2^-32) is added to 1 as an integer: w is right to 5 x
// 2^-26 at worst, 2^-27 in the mean.  The bins hold weights in units of 2^-32, as two sums of 16 bits each
// (shared memory adds 32-bit integers at once, 64-bit ones in a loop).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kernels.h"

namespace mq {
namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kList = 1024;      // tokens that rank 0 ranks at once
constexpr int kMaxCluster = 16;  // CTAs of a row (over 8: the non-portable size)
constexpr int kFixBits = 42;     // a weight of 1 is 2^42

// What the CTAs of a row tell each other, and rank 0's findings (copied to all).
struct Control {
    float maxes[kMaxCluster];
    int argmax[kMaxCluster];
    u64 totals[kMaxCluster];
    u64 warp_sums[kThreads / 32];
    u64 target, above;       // what is still wanted of the current set; weights kept above it
    u64 prefix;              // set of a narrowed bin: places whose top `bits` bits are prefix
    u64 boundary;            // last place kept
    u64 total;               // weights that top-k left (2^-32)
    unsigned population, list_n;
    int bin, bits, found;
};

struct Shared {
    unsigned cnt[kBins], hi[kBins], lo[kBins];  // this CTA's bins; later rank 0's list
    u64 all_w[kBins];                            // rank 0: the row's
    unsigned all_cnt[kBins];
    Control c;
};
static_assert(sizeof(u64) * 2 * kList <= sizeof(unsigned) * 3 * kBins, "the list lies over the bins");

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

struct Weight {
    float top, c_hi, c_lo;  // the row's maximum; log2(e) / temperature in two parts

    __device__ __forceinline__ float exponent(float x) const { return (top - x) * c_hi; }

    __device__ __forceinline__ u64 operator()(float x) const
    {
        if (x == top) return 1ull << kFixBits;  // also +inf, whose difference is no number
        const float d = top - x;
        const float t = d * c_hi;
        if (!(t < (float)kFixBits + 0.5f)) return 0;  // also x = -inf, top = +inf
        // d + e = top - x exactly; t + r = (d + e) * (c_hi + c_lo) to f32's square
        const float b = d - top;
        const float e = (top - (d - b)) - (x + b);
        const float r = fmaf(d, c_hi, -t) + fmaf(d, c_lo, e * c_hi);
        const float n = rintf(t);
        const float f = (n - t) - r;
        // (2^f - 1) / f by its series in f ln2
        float s = 1.3215486790144307e-6f;
        s = fmaf(s, f, 1.5252733804059841e-5f);
        s = fmaf(s, f, 1.5403530393381609e-4f);
        s = fmaf(s, f, 1.3333558146428443e-3f);
        s = fmaf(s, f, 9.6181291076284772e-3f);
        s = fmaf(s, f, 5.5504108664821580e-2f);
        s = fmaf(s, f, 2.4022650695910071e-1f);
        s = fmaf(s, f, 6.9314718055994531e-1f);
        const u64 one = (1u << 30) + (unsigned)__float2int_rn(s * f * 1073741824.0f);
        return (one << (kFixBits - 30)) >> (int)n;
    }
};

// A weight in units of 2^-32 (the largest is one unit short: it has to fit 32 bits).
__device__ __forceinline__ unsigned coarse(u64 w)
{
    const u64 c = (w + (1u << 9)) >> 10;
    return c > 0xffffffffu ? 0xffffffffu : (unsigned)c;
}

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
    for (int i = tid; i < kBins; i += kThreads) {
        sh.cnt[i] = sh.hi[i] = sh.lo[i] = 0;
        sh.all_w[i] = 0;
        sh.all_cnt[i] = 0;
    }
    if (tid == 0) sh.c.list_n = 0;
    griddep_wait();  // the logits may come from the preceding kernel

    // this CTA's slice: values [rank * slice, ..) counted from the last 16-byte border at or before the row
    const float *src = a.logits + row * a.stride;
    const int shift = (int)(((uintptr_t)src >> 2) & 3);
    src -= shift;
    const int base = rank * a.slice;  // in shifted places; index = place - shift
    const int lo = shift, hi = shift + a.vocab;
    float mx = -INFINITY;
    for (int i = tid * 4; i < a.seg * kThreads; i += kThreads * 4) {
        const int p = base + i;
        float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (i < a.slice) {
            if (p >= lo && p + 4 <= hi) {
                const float4 f = __ldcg(reinterpret_cast<const float4 *>(src + p));
                v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (p + j >= lo && p + j < hi) v[j] = __ldcg(src + p + j);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = v[j] == v[j] ? v[j] + 0.0f : -INFINITY;  // NaN is never drawn; -0 is 0
            xs[i + j] = x;
            mx = fmaxf(mx, x);
        }
    }
    const float temperature = a.temperature ? __ldcg(a.temperature + row) : 1.0f;
    const float top_p = a.top_p ? __ldcg(a.top_p + row) : 1.0f;
    const float min_p = a.min_p ? __ldcg(a.min_p + row) : 0.0f;
    const int top_k = a.top_k ? __ldcg(a.top_k + row) : 0;
    const float u = __ldcg(a.u + row);

    // the row's maximum
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) sh.c.warp_sums[warp] = __float_as_uint(mx);
    cluster.sync();  // every CTA of the row runs, its bins are zero
    if (tid < ranks) {
        float m = -INFINITY;
        for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, __uint_as_float((unsigned)sh.c.warp_sums[w]));
        cluster.map_shared_rank(&sh, tid)->c.maxes[rank] = m;
    }
    cluster.sync();
    mx = sh.c.maxes[0];
    for (int r = 1; r < ranks; ++r) mx = fmaxf(mx, sh.c.maxes[r]);

    if (mx == -INFINITY) {  // nothing to draw from
        if (rank == 0 && tid == 0) {
            a.token[row] = -1;
            if (a.prob) a.prob[row] = 0.0f;
        }
        return;
    }
    if (!(temperature > 0.0f) || top_k == 1 || top_p <= 0.0f || min_p > 1.0f) {
        // one token is kept: the lowest index of the largest logit
        int best = 0x7fffffff;
        for (int i = tid; i < a.slice; i += kThreads)
            if (xs[i] == mx) {
                best = base + i - shift;
                break;
            }
        for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
        if (lane == 0) sh.c.warp_sums[warp] = (unsigned)best;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kThreads / 32; ++w) best = min(best, (int)sh.c.warp_sums[w]);
            root.c.argmax[rank] = best;
        }
        cluster.sync();
        if (rank == 0 && tid == 0) {
            for (int r = 0; r < ranks; ++r) best = min(best, sh.c.argmax[r]);
            a.token[row] = best;
            if (a.prob) a.prob[row] = 1.0f;
        }
        return;
    }

    const double c = 1.4426950408889634 / (double)temperature;
    Weight weight;
    weight.top = mx;
    weight.c_hi = (float)fmin(c, 1e30);
    weight.c_lo = c < 1e30 ? (float)(c - (double)weight.c_hi) : 0.0f;
    const u64 floor_w = min_p > 0.0f ? (u64)ceil((double)min_p * (double)(1ull << kFixBits)) : 0;
    const bool by_count = top_k > 0 && top_k < a.vocab, by_weight = top_p < 1.0f;
    auto bin_of = [&](float x) { return (int)fminf(weight.exponent(x) * 32.0f, (float)(kBins - 1)); };

    // Adds this CTA's tokens of the current set into its bins, then those into rank 0's.  Without
    // a set (c.bin < 0) the bins are bin_of's, else the next 11 bits of the place, largest first.
    auto histogram = [&](int bin, int bits, u64 prefix) {
        for (int j = 0; j < a.seg; ++j) {
            const float x = xs[tid * a.seg + j];
            if (x == -INFINITY) continue;
            int b = mx == INFINITY ? (x == mx ? 0 : kBins - 1) : bin_of(x);
            if (bin >= 0) {
                if (b != bin) continue;
                const u64 place = place_of(x, base + tid * a.seg + j - shift);
                if (bits && place >> (64 - bits) != prefix) continue;
                const int left = 64 - bits;
                b = kBins - 1 - (int)((left >= 11 ? place >> (left - 11) : place << (11 - left)) & (kBins - 1));
            }
            atomicAdd(&sh.cnt[b], 1u);
            if (by_weight) {
                const unsigned w = coarse(weight(x));
                if (w >> 16) atomicAdd(&sh.hi[b], w >> 16);
                if (w & 0xffffu) atomicAdd(&sh.lo[b], w & 0xffffu);
            }
        }
        __syncthreads();
        for (int b = tid; b < kBins; b += kThreads) {
            const unsigned n = sh.cnt[b];
            if (n) {
                atomicAdd(&root.all_cnt[b], n);
                const u64 w = ((u64)sh.hi[b] << 16) + sh.lo[b];
                if (w) atomicAdd(&root.all_w[b], w);
            }
        }
        cluster.sync();
    };
    // Rank 0: the bin where the target is reached; what is left of it, the weights above the bin
    // and the bin's tokens go to every CTA.
    auto find_bin = [&](bool counts) {
        if (rank == 0) {
            constexpr int kPer = kBins / kThreads;
            const u64 target = sh.c.target, kept_above = sh.c.above;  // read before the scans' barriers
            u64 mine = 0, weights = 0, total, all;
            for (int j = 0; j < kPer; ++j) {
                weights += sh.all_w[tid * kPer + j];
                mine += sh.all_cnt[tid * kPer + j];
            }
            u64 w_before = block_scan(weights, sh.c.warp_sums, &all);
            u64 before = counts ? block_scan(mine, sh.c.warp_sums, &total) : w_before;
            if (!counts) mine = weights;
            if (before < target && target <= before + mine) {
                for (int j = 0; j < kPer; ++j) {
                    const int b = tid * kPer + j;
                    const u64 here = counts ? sh.all_cnt[b] : sh.all_w[b];
                    if (target <= before + here) {
                        const u64 left = target - before, above = kept_above + w_before;
                        for (int r = 0; r < ranks; ++r) {
                            Control &o = cluster.map_shared_rank(&sh, r)->c;
                            o.bin = b, o.target = left, o.above = above, o.population = sh.all_cnt[b];
                        }
                        break;
                    }
                    before += here;
                    w_before += sh.all_w[b];
                }
            }
        }
        cluster.sync();
    };
    // The last place kept when the order's tokens are taken until `target` (of counts, or of
    // weights) is reached; rank 0 leaves it in every CTA's c.boundary, and the weights up to it in
    // its own c.total.
    auto select = [&](bool counts) {
        find_bin(counts);
        const int bin = sh.c.bin;
        int bits = 0;
        u64 prefix = 0;
        while (sh.c.population > kList) {
            for (int i = tid; i < kBins; i += kThreads) {
                sh.cnt[i] = sh.hi[i] = sh.lo[i] = 0;
                if (rank == 0) sh.all_w[i] = 0, sh.all_cnt[i] = 0;
            }
            cluster.sync();
            histogram(bin, bits, prefix);
            find_bin(counts);
            const int left = 64 - bits, step = left < 11 ? left : 11;
            const u64 digit = (u64)(kBins - 1 - sh.c.bin) >> (11 - step);
            prefix = prefix << step | digit;
            bits += step;
        }
        u64 *list = reinterpret_cast<u64 *>(root.cnt);  // rank 0's bins are used up
        for (int j = 0; j < a.seg; ++j) {
            const float x = xs[tid * a.seg + j];
            if (x == -INFINITY) continue;
            const int b = mx == INFINITY ? (x == mx ? 0 : kBins - 1) : bin_of(x);
            if (b != bin) continue;
            const u64 place = place_of(x, base + tid * a.seg + j - shift);
            if (bits && place >> (64 - bits) != prefix) continue;
            const unsigned at = atomicAdd(&root.c.list_n, 1u);
            if (at < kList) list[at] = place;
        }
        cluster.sync();
        if (rank == 0) {
            u64 *mine = reinterpret_cast<u64 *>(sh.cnt), *sorted = mine + kList;
            const int n = min((int)sh.c.list_n, kList);
            for (int i = tid; i < n; i += kThreads) {
                const u64 p = mine[i];
                int before = 0;
                for (int j = 0; j < n; ++j) before += mine[j] > p;
                sorted[before] = p;
            }
            __syncthreads();
            // two ranked tokens a thread: their weights and counts, added up in order
            constexpr int kPer = kList / kThreads;
            u64 w[kPer], mine_sum = 0, total;
            for (int j = 0; j < kPer; ++j) {
                const int i = tid * kPer + j;
                w[j] = i < n ? coarse(weight(logit_of((unsigned)(sorted[i] >> 32)))) : 0;
                mine_sum += w[j];
            }
            u64 sum = block_scan(mine_sum, sh.c.warp_sums, &total);
            const u64 target = sh.c.target, above = sh.c.above;
            for (int j = 0; j < kPer; ++j) {
                const int i = tid * kPer + j;
                const u64 before = sum;
                sum += w[j];
                const bool last = counts ? (u64)i + 1 == target : before < target && target <= sum;
                if (i < n && last) {
                    for (int r = 0; r < ranks; ++r) cluster.map_shared_rank(&sh, r)->c.boundary = sorted[i];
                    sh.c.total = above + sum;
                }
            }
            if (tid == 0) sh.c.list_n = 0;
        }
        cluster.sync();
        return bits > 0;  // the row's bins are gone
    };

    u64 boundary = 0;
    if (by_count || by_weight) {
        histogram(-1, 0, 0);
        bool stale = false, cut = false;
        if (by_count) {
            // tokens that are -inf are not in the bins: with fewer others than top_k nothing is cut
            u64 n = 0, total;
            if (rank == 0) {
                for (int b = tid; b < kBins; b += kThreads) n += sh.all_cnt[b];
                block_scan(n, sh.c.warp_sums, &total);
                if (tid == 0) {
                    for (int r = 0; r < ranks; ++r) {
                        Control &o = cluster.map_shared_rank(&sh, r)->c;
                        o.found = total > (u64)top_k;
                        o.target = (u64)top_k, o.above = 0;
                    }
                }
            }
            cluster.sync();
            cut = sh.c.found;
            cluster.sync();
            if (cut) {
                stale = select(true);
                boundary = sh.c.boundary;
            }
        }
        if (by_weight) {
            if (stale) {
                for (int i = tid; i < kBins; i += kThreads) {
                    sh.cnt[i] = sh.hi[i] = sh.lo[i] = 0;
                    if (rank == 0) sh.all_w[i] = 0, sh.all_cnt[i] = 0;
                }
                cluster.sync();
                histogram(-1, 0, 0);
            }
            if (rank == 0) {
                u64 w = 0, total;
                for (int b = tid; b < kBins; b += kThreads) w += sh.all_w[b];
                block_scan(w, sh.c.warp_sums, &total);
                if (tid == 0) {
                    if (cut) total = sh.c.total;
                    const u64 target = (u64)ceil((double)top_p * (double)total);
                    for (int r = 0; r < ranks; ++r) {
                        Control &o = cluster.map_shared_rank(&sh, r)->c;
                        o.target = target < 1 ? 1 : target, o.above = 0;
                    }
                }
            }
            cluster.sync();
            select(false);
            boundary = boundary > sh.c.boundary ? boundary : sh.c.boundary;
        }
    }

    // the kept weights, in the order of the vocabulary
    auto kept = [&](int j) -> u64 {
        const float x = xs[tid * a.seg + j];
        if (x == -INFINITY) return 0;
        if (boundary && place_of(x, base + tid * a.seg + j - shift) < boundary) return 0;
        const u64 w = weight(x);
        return w >= floor_w ? w : 0;
    };
    u64 mine = 0, total;
    for (int j = 0; j < a.seg; ++j) mine += kept(j);
    u64 before = block_scan(mine, sh.c.warp_sums, &total);
    if (tid < ranks) cluster.map_shared_rank(&sh, tid)->c.totals[rank] = total;
    cluster.sync();
    u64 all = 0;
    for (int r = 0; r < ranks; ++r) {
        if (r == rank) before += all;
        all += sh.c.totals[r];
    }
    // the first token whose sum exceeds u * all
    u64 target = u > 0.0f ? (u64)((double)u * (double)all) : 0;
    if (target >= all) target = all - 1;
    if (before <= target && target < before + mine) {
        for (int j = 0; j < a.seg; ++j) {
            const u64 w = kept(j);
            before += w;
            if (before > target) {
                a.token[row] = base + tid * a.seg + j - shift;
                if (a.prob) a.prob[row] = (float)((double)w / (double)all);
                break;
            }
        }
    }
}

// CTAs per row: all of them resident for few rows, for latency; fewer for many.
int cluster_for(int nt, int vocab, int sms)
{
    int c = 16;
    while (c > 1 && (long long)nt * c > sms) c >>= 1;
    if (c < 4) c = 4;
    while (c < 16 && (vocab + 3) / c > 20480) c <<= 1;
    while (c > 1 && (vocab + 3) / c < kThreads) c >>= 1;
    return c;
}

constexpr int kMaxDevices = 64;
std::atomic<bool> g_opted[kMaxDevices];
constexpr size_t kMaxSmem = 227 * 1024;

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
    // a row may start up to 3 values behind a 16-byte border
    a.slice = ((a.vocab + 3 + c - 1) / c + 3) & ~3;
    a.seg = (a.slice + kThreads - 1) / kThreads | 1;  // odd: the threads' segments lie in different banks
    const size_t smem = sizeof(Shared) + (size_t)a.seg * kThreads * sizeof(float);
    if (smem > kMaxSmem) return cudaErrorInvalidValue;
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
