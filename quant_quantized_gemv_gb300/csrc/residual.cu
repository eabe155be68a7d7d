// residual.cu -- the residual stream between two blocks of a layer, in one launch: the norm behind the
// block, its gate and scale, the addition, the norm before the next block, and that one's q8 plane.
//
//   y' = y / sqrt(mean(y^2) + eps) * post_gain       (where post_gain is given)
//   x' = x + (scale * gate) * y'
//   z  = x' / sqrt(mean(x'^2) + eps) * gain,  and its q8 plane.
//
// A CTA takes a row, and a lane K groups of four of its values, which stay in its registers from the load to the
// q8 codes: x and y are read once, and each of the two sums of squares is one exchange over the CTA (a lane's sum, a
// butterfly, the warps' sums in order: the same bits in every run).
//
// What bounds it (captured): one row of 5120, the launch, one load and two exchanges, 3.5 us (with a norm behind the block
// 4.6). 4096 rows of 5120, 360 MB: 55.5 us, 6.5 TB/s, the rate of a copy; with a norm behind the block and a gate for
// each row, 444 MB: 72.8 us, 6.1 TB/s. 8000 rows of 1024: 26 us, 5.4 TB/s: the CTAs' beginnings (a row a warp,
// without barriers, 34 us). 2000 rows of 13824: 104 us, 4.5 TB/s: one CTA of 864 threads an SM, whose loads wait for
// its sums. 1000 rows of 20480: 69.5 us, 5.1 TB/s, with gate and norm 101.5, 4.3 TB/s: x' once more from L2.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "q8_block.cuh"

namespace mq {
namespace {

constexpr int kMaxThreads = 1024;

__device__ __forceinline__ float dot(float4 v, float s)
{
    s = fmaf(v.x, v.x, s);
    s = fmaf(v.y, v.y, s);
    s = fmaf(v.z, v.z, s);
    return fmaf(v.w, v.w, s);
}

// The CTA's sum of a value of each thread (sums: 32 places of its own for each call).
__device__ __forceinline__ float cta_sum(float v, float *sums)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    const int warps = (blockDim.x + 31) >> 5;
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < warps; ++w) t += sums[w];
    return t;
}

__device__ __forceinline__ float4 times(float4 v, float s, float4 g)
{
    return make_float4((v.x * s) * g.x, (v.y * s) * g.y, (v.z * s) * g.z, (v.w * s) * g.w);
}

// A sum of squares of a long row: 16 groups of four at a time in f32, and what adding such a sum rounds off (which two f32
// additions find exactly) kept beside the others, so that the error does not grow with the row. (Rows of 2^26 equal values,
// 2^16 squares a thread, added one after the other were off by up to 8 x 10^-4.)
struct LongSum {
    float sum = 0.0f, rest = 0.0f, some = 0.0f;

    __device__ __forceinline__ void add(float4 v, int i)
    {
        some = dot(v, some);
        if ((i / kMaxThreads & 15) == 15) settle();
    }
    __device__ __forceinline__ void settle()
    {
        const float t = __fadd_rn(sum, some), b = __fsub_rn(t, sum);
        rest += __fadd_rn(__fsub_rn(sum, __fsub_rn(t, b)), __fsub_rn(some, b));
        sum = t, some = 0.0f;
    }
    __device__ __forceinline__ float total()
    {
        settle();
        return sum < INFINITY ? sum + rest : sum;  // (an infinite sum has no rest)
    }
};

// K groups of four a lane; K = 0: rows longer than a CTA holds, whose x' is read again from where it was written.
// GATE: a gate, which is loaded ahead of the first sum with x and y (4096 rows of 5120: 75.5 -> 72.8 us; its registers
// in a kernel without one cost a CTA an SM, 55.6 -> 59.7).
template <int K, bool GATE>
__global__ void __launch_bounds__(kMaxThreads) add_rmsnorm_kernel(const ResidualLaunch a)
{
    __shared__ float sums[2][32];
    griddep_launch_dependents();
    const int tid = threadIdx.x, n4 = a.n >> 2, T = blockDim.x;
    const size_t row = blockIdx.x;
    const float4 *x4 = reinterpret_cast<const float4 *>(a.x) + row * n4;
    const float4 *y4 = reinterpret_cast<const float4 *>(a.y) + row * n4;
    const float4 *gate4 = reinterpret_cast<const float4 *>(GATE ? a.gate + row * a.gate_stride : nullptr);
    const float4 *post4 = reinterpret_cast<const float4 *>(a.post_gain), *gain4 = reinterpret_cast<const float4 *>(a.gain);
    float4 *out4 = reinterpret_cast<float4 *>(a.x_out) + row * n4;
    float4 *z4 = a.z ? reinterpret_cast<float4 *>(a.z) + row * n4 : nullptr;
    uint8_t *q8 = a.q8 ? a.q8 + row * a.q8_stride : nullptr;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f), one = make_float4(1.f, 1.f, 1.f, 1.f);
    griddep_wait();  // any of the inputs may come from the preceding kernels

    auto factor = [&](float sum, int which) {  // 1 / sqrt(mean + eps) from this thread's squares
        return 1.0f / sqrtf(cta_sum(sum, sums[which]) / (float)a.n + a.eps);
    };
    auto added = [&](float4 x, float4 y, float4 g, float ys, int i) {
        if (post4) y = times(y, ys, __ldca(post4 + i));
        return make_float4(fmaf(a.scale * g.x, y.x, x.x), fmaf(a.scale * g.y, y.y, x.y), fmaf(a.scale * g.z, y.z, x.z),
                           fmaf(a.scale * g.w, y.w, x.w));
    };
    auto finish = [&](float4 v, float s, int i) {  // every lane of a warp calls it
        const bool valid = i < n4;
        const float4 z = valid ? times(v, s, __ldca(gain4 + i)) : zero;
        if (z4 && valid) z4[i] = z;
        if (q8) quantize4(z, valid, i, q8, a.q8_d_off, a.q8_sum_off);
    };
    if constexpr (K > 0) {
        float4 x[K], y[K], gate[GATE ? K : 1];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = tid + k * T;
            y[k] = i < n4 ? __ldcg(y4 + i) : zero;
            x[k] = i < n4 ? __ldcg(x4 + i) : zero;
            if constexpr (GATE) gate[k] = i < n4 ? __ldcg(gate4 + i) : one;
        }
        float ys = 1.0f;
        if (post4) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < K; ++k) s = dot(y[k], s);
            ys = factor(s, 0);
        }
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = tid + k * T;
            if (i < n4) {
                float4 g = one;
                if constexpr (GATE) g = gate[k];
                x[k] = added(x[k], y[k], g, ys, i);
                out4[i] = x[k];
            }
            s = dot(x[k], s);
        }
        const float xs = factor(s, 1);
#pragma unroll
        for (int k = 0; k < K; ++k) finish(x[k], xs, tid + k * T);
    } else {
        float ys = 1.0f;
        if (post4) {
            LongSum s;
            for (int i = tid; i < n4; i += T) s.add(__ldcg(y4 + i), i);
            ys = factor(s.total(), 0);
        }
        LongSum s;
        for (int i = tid; i < n4; i += T) {
            const float4 v = added(__ldcg(x4 + i), __ldcg(y4 + i), GATE ? __ldcg(gate4 + i) : one, ys, i);
            out4[i] = v;
            s.add(v, i);
        }
        const float xs = factor(s.total(), 1);
        for (int i0 = 0; i0 < n4; i0 += T) finish(i0 + tid < n4 ? out4[i0 + tid] : zero, xs, i0 + tid);
    }
}

template <int K>
cudaError_t launch_k(const ResidualLaunch &a, int threads, int pdl, cudaStream_t st)
{
    const auto kernel = a.gate ? add_rmsnorm_kernel<K, true> : add_rmsnorm_kernel<K, false>;
    return launch_maybe_pdl(kernel, dim3((unsigned)a.nt), dim3((unsigned)threads), 0, pdl, st, a);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const ResidualLaunch &a, int pdl, cudaStream_t st)
{
    const int n4 = a.n / 4;
    int k = 1;
    // as many threads as a CTA has: the fewest groups a lane (one row of 5120 in 640 threads 3.5 us, in 320 4.5; 4096 rows
    // 72.8 and 73.0). Four at the most: eight spill (1000 rows of 20480: 82 us where reading x' again takes 69, with a norm
    // behind the block and a gate 129 and 102; of 32768 123 and 107, 177 and 158).
    while (k < 4 && (n4 + k - 1) / k > kMaxThreads) k *= 2;
    const int threads = ((n4 + k - 1) / k + 31) / 32 * 32;
    if (threads > kMaxThreads) return launch_k<0>(a, kMaxThreads, pdl, st);
    return k == 1   ? launch_k<1>(a, threads, pdl, st)
           : k == 2 ? launch_k<2>(a, threads, pdl, st)
                    : launch_k<4>(a, threads, pdl, st);
}

}  // namespace mq
