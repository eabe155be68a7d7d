// verify.cuh -- what the kernels of the verification share: a row's sequence and the decision on its drafted token.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"
#include "weights.cuh"

namespace mq {
namespace {

// A row's sequence in a verification: its number (negative: none), its rows, its filters; the row's own.
struct Sequence {
    int seq, from, to, top_k, draft;
    bool final;                                  // its last row: nothing was drafted for it
    float temperature, top_p, min_p, u, u_draw, draft_q;

    __device__ __forceinline__ bool greedy() const { return !(temperature > 0.0f); }
    __device__ __forceinline__ bool plain(int vocab) const  // no filter
    {
        return !greedy() && !(top_k > 0 && top_k < vocab) && !(top_p < 1.0f) && !(min_p > 0.0f);
    }
};

// A row's numbers.
__device__ __forceinline__ void read_row(Sequence &of, const VerifyLaunch &a, int row)
{
    of.u = __ldcg(a.u + row), of.u_draw = __ldcg(a.u_draw + of.seq);
    of.draft = of.final ? -1 : __ldcg(a.drafts + row);
    of.draft_q = 1.0f;
    if (a.draft_probs && of.draft >= 0 && of.draft < a.vocab) {
        const float q = __ldcg(a.draft_probs + row * a.q_stride + of.draft);
        of.draft_q = q > 0.0f ? q : 0.0f;  // NaN counts as 0
    }
}

// The sequence that a row belongs to and its filters, by every CTA for itself (of.seq is -1 before, and stays it where
// there is none); whether the starts that this thread looked at do not ascend in [0, nt].
template <bool NUMBERS>  // the row's numbers too
__device__ __forceinline__ bool find_sequence(Sequence &of, const VerifyLaunch &a, int row, int threads)
{
    bool bad = false;
    for (int i = threadIdx.x; i < a.n_seqs; i += threads) {
        const int from = __ldcg(a.starts + i), to = __ldcg(a.starts + i + 1);
        bad = bad || from < 0 || to < from || to > a.nt;
        if (from <= row && row < to) {
            // formed in registers: where starts do not ascend several threads may find one, and none of them may take
            // another's numbers for an address
            Sequence mine = {};
            mine.seq = i, mine.from = from, mine.to = to;
            mine.final = row + 1 == to;
            mine.temperature = a.temperature ? __ldcg(a.temperature + i) : 1.0f;
            mine.top_p = a.top_p ? __ldcg(a.top_p + i) : 1.0f;
            mine.min_p = a.min_p ? __ldcg(a.min_p + i) : 0.0f;
            mine.top_k = a.top_k ? __ldcg(a.top_k + i) : 0;
            if (NUMBERS) read_row(mine, a, row);
            of = mine;
        }
    }
    return bad;
}

// By one CTA: starts that do not ascend, or the counts of sequences without rows, which nobody else writes.
__device__ __forceinline__ void note_starts(const VerifyLaunch &a, bool bad, int threads)
{
    if (bad && threadIdx.x == 0 && a.status) atomicOr(a.status, 1);
    if (!bad)
        for (int i = threadIdx.x; i < a.n_seqs; i += threads)
            if (__ldcg(a.starts + i) == __ldcg(a.starts + i + 1)) a.counts[i] = 0;
}

// Whether the drafted token stands, of whose row `all` is kept and w of that its own: u q < w / all in
// integers, u all and its share q rounded down.
__device__ __forceinline__ bool draft_stands(const Sequence &of, u64 w, u64 all)
{
    const u64 ua = share_of(fminf(fmaxf(of.u, 0.0f), 0x1.fffffep-1f), all, false);
    return (of.draft_q < 1.0f ? share_of(of.draft_q, ua, false) : ua) < w;
}

// What is left of a token's kept weight w where the draft is taken off: max(0, w - q all).
__device__ __forceinline__ u64 left_of(const VerifyLaunch &a, const Sequence &of, int row, int token, u64 w, u64 all)
{
    if (!a.draft_probs) return token == of.draft ? 0 : w;
    const float q = __ldcg(a.draft_probs + row * a.q_stride + token);
    const u64 taken = q >= 1.0f ? all : q > 0.0f ? share_of(q, all, false) : 0;
    return w > taken ? w - taken : 0;
}

// What is left of p, max(0, w / all - q): f32 of the exact difference. w is in two parts and 1 / all in two, and what the
// first product rounds off is added behind the subtraction: off by 2^-24 of itself and 2^-45 of p, however near q is.
// The sums are of these in units of 2^-42 (fixed_of), token by token, so that they are the same in whatever order and by
// whatever threads they are formed: a token found by a sum is found again.
struct Rest {
    float ih, il;

    __device__ __forceinline__ explicit Rest(u64 all)
    {
        const float ah = __ull2float_rn(all), al = __ll2float_rn((long long)(all - __float2ull_rn(ah)));
        ih = 1.0f / ah * 0x1p42f, il = ih * (fmaf(-ah, ih * 0x1p-42f, 1.0f) - al / ah);
    }
    __device__ __forceinline__ void operator()(const Weight &weight, float x0, float x1, float q0, float q1, float &r0, float &r1) const
    {
        Two hi, lo;
        weight.parts(x0, x1, hi, lo);
        const Two h = two(ih, ih), minus = two(-1.0f, -1.0f), p = mul2(hi, h);
        const Two low = fma2(hi, two(il, il), fma2(lo, h, fma2(hi, h, mul2(p, minus))));
        split(add2(add2(p, two(-q0, -q1)), low), r0, r1);
        r0 = __saturatef(r0), r1 = __saturatef(r1);
    }
    // The same from weights of f32, to 2^-23 of p beside what the weights are off by.
    __device__ __forceinline__ void quick(Two w, float q0, float q1, float &r0, float &r1) const
    {
        split(fma2(w, two(ih, ih), fma2(w, two(il, il), two(-q0, -q1))), r0, r1);
        r0 = __saturatef(r0), r1 = __saturatef(r1);
    }
};

}  // namespace
}  // namespace mq
