// decode.cpp -- the C ABI of the operators around the GEMVs of a decode step
// (include/mq.h: paged cache, rotation and append, attention, draw): argument
// checks, the attention's grid, then the launch.  Nothing here allocates.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kernels.h"
#include "layout.h"
#include "mq.h"

namespace {

using namespace mq;

bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

bool head_dim_ok(int d) { return d == 64 || d == 96 || d == 128 || d == 256; }

// Bytes of one head's part of a page; 0 on a bad type or shape.
size_t kv_head_bytes(int type, int page_size, int head_dim)
{
    if (!head_dim_ok(head_dim) || page_size < 16 || page_size % 16 != 0) return 0;
    const size_t n = (size_t)page_size * head_dim;
    return type == MQ_KV_F16 || type == MQ_KV_BF16 ? 2 * n : type == MQ_KV_Q8 ? n + n / 16 : 0;
}

// Checks a cache description; its page stride and head size in bytes.
int kv_check(const mq_kv_cache *kv, size_t *page_stride, size_t *head_bytes)
{
    if (!kv->k || !kv->v) return MQ_ERR_NULL;
    const size_t page = mq_kv_page_bytes(kv->type, kv->n_kv_heads, kv->page_size, kv->head_dim);
    if (page == 0 || kv->n_pages < 1 || kv->page_stride < 0) return MQ_ERR_SHAPE;
    if (kv->page_stride != 0 && (size_t)kv->page_stride < page) return MQ_ERR_SHAPE;
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || kv->page_stride % 16 != 0) return MQ_ERR_ALIGN;
    *page_stride = kv->page_stride ? (size_t)kv->page_stride : page;
    *head_bytes = kv_head_bytes(kv->type, kv->page_size, kv->head_dim);
    return MQ_OK;
}

// CTAs of an attention launch over `units` units (a row's group of up to 8
// heads of one kv head) of up to `span` tokens each: one resident wave, or fewer
// when there are fewer rounds of tokens than that.  Beyond kAttnMaxRows rows: a
// CTA per unit.
int attn_wave(int sms) { return sms < kAttnMaxCtas ? sms : kAttnMaxCtas; }

long long attn_rounds(long long span, int type, int head_dim)
{
    const int round = attn_warps(type, head_dim) * kAttnTile;
    return (span + round - 1) / round;
}

long long attn_grid(long long units, long long rounds, int nt, int sms)
{
    if (nt > kAttnMaxRows) return units;
    return units * rounds < attn_wave(sms) ? units * rounds : attn_wave(sms);
}

// Workspace of a call: a counter and two partial results for each CTA that
// shares out the work, in places that no call changes (a workspace may serve
// calls of different sizes, and every counter must be zero before each).  None
// for rows so short that no unit is cut.
size_t attn_count_bytes(int sms) { return ((size_t)attn_wave(sms) * 4 + 15) & ~(size_t)15; }

size_t attn_ws_bytes(const mq_kv_cache *kv, int max_len, int sms)
{
    if (attn_rounds((long long)max_len + kAttnTile - 1, kv->type, kv->head_dim) <= kAttnWhole) return 0;
    return attn_count_bytes(sms) + (size_t)attn_wave(sms) * 2 * attn_part_floats(kv->head_dim) * 4;
}

bool attn_shape_ok(const mq_kv_cache *kv, int n_heads, int nt, int max_len)
{
    if (mq_kv_page_bytes(kv->type, kv->n_kv_heads, kv->page_size, kv->head_dim) == 0) return false;
    if (nt < 1 || n_heads < 1 || n_heads % kv->n_kv_heads != 0 || max_len < 1) return false;
    if (max_len > MQ_ATTN_MAX_LEN) return false;  // places in 32 bits, of rounds asked for ahead too
    // the grid, a q8 plane's values and the rounds of all rows (a CTA's share ends up to its length behind them)
    const long long rounds = attn_rounds((long long)max_len + kAttnTile - 1, kv->type, kv->head_dim);
    return (long long)nt * n_heads < (1LL << 24) && (long long)n_heads * kv->head_dim < (1LL << 30) &&
           (long long)nt * n_heads * (rounds + kAttnUnitCost) < (1LL << 30);
}

long long attn_units(const mq_kv_cache *kv, int n_heads, int nt)
{
    const int group = n_heads / kv->n_kv_heads;
    return (long long)nt * kv->n_kv_heads * ((group + kAttnHeads - 1) / kAttnHeads);
}

}  // namespace

extern "C" {

size_t mq_kv_page_bytes(int type, int n_kv_heads, int page_size, int head_dim)
{
    if (n_kv_heads < 1) return 0;
    const size_t head = kv_head_bytes(type, page_size, head_dim);
    if (head == 0 || head > ((size_t)1 << 40) / (size_t)n_kv_heads) return 0;
    return head * (size_t)n_kv_heads;
}

int mq_rope_table(const double *freqs, int n, uint64_t *table)
{
    if (!freqs || !table) return MQ_ERR_NULL;
    if (n < 1) return MQ_ERR_SHAPE;
    for (int i = 0; i < n; ++i) {
        double t = freqs[i] / 6.283185307179586476925;  // turns per position
        if (!isfinite(t)) return MQ_ERR_SHAPE;
        t -= floor(t);                                   // modulo one turn, in [0, 1]
        table[i] = t >= 1.0 ? 0 : (uint64_t)(t * 0x1p64);
    }
    return MQ_OK;
}

int mq_rope_append(const mq_kv_cache *kv, const mq_rope_append_args *a, void *stream)
{
    if (!kv || !a) return MQ_ERR_NULL;
    size_t page_stride, head_bytes;
    const int st = kv_check(kv, &page_stride, &head_bytes);
    if (st != MQ_OK) return st;
    if (a->nt < 1) return MQ_ERR_SHAPE;  // empty tensors have no address
    if (!a->q || !a->k || !a->v || !a->q_out || !a->positions || !a->pages) return MQ_ERR_NULL;
    const int D = kv->head_dim;
    const long long nq = (long long)a->n_heads * D, nk = (long long)kv->n_kv_heads * D;
    if (a->n_heads < 1 || a->n_heads % kv->n_kv_heads != 0 || a->n_heads > (1 << 20) ||
        kv->n_kv_heads > (1 << 20) || a->n_seqs < 1 || a->pages_stride < 1)
        return MQ_ERR_SHAPE;
    if (a->rope_dims < 0 || a->rope_dims > D || a->rope_dims % (D > 128 ? 16 : 8) != 0 ||
        (a->rope_style != MQ_ROPE_HALF && a->rope_style != MQ_ROPE_PAIRS))
        return MQ_ERR_SHAPE;
    if (a->rope_dims > 0 && !a->rope_table) return MQ_ERR_NULL;
    if (a->q_stride < nq || a->q_out_stride < nq || a->k_stride < nk || a->v_stride < nk)
        return MQ_ERR_SHAPE;
    // rows lie along the grid's y (32768 of them) and z (65535 at most), a row's CTAs along x: well inside
    if ((long long)a->nt * (a->n_heads + 2 * kv->n_kv_heads) >= (1LL << 31)) return MQ_ERR_SHAPE;
    const void *p16[] = {a->q, a->k, a->v, a->q_out, a->q_bias, a->k_bias, a->v_bias, a->q_gain, a->k_gain};
    for (const void *p : p16)
        if (!aligned(p, 16)) return MQ_ERR_ALIGN;
    if ((a->q_stride | a->k_stride | a->v_stride | a->q_out_stride) % 4 != 0) return MQ_ERR_ALIGN;
    if (!aligned(a->rope_table, 8) || !aligned(a->positions, 4) || !aligned(a->seq, 4) ||
        !aligned(a->pages, 4) || !aligned(a->status, 4))
        return MQ_ERR_ALIGN;
    const int sms = mq_device_sms();
    if (sms <= 0) return MQ_ERR_CUDA;
    RopeAppendLaunch r = {};
    r.q = a->q, r.k = a->k, r.v = a->v, r.q_out = a->q_out;
    r.q_stride = a->q_stride, r.k_stride = a->k_stride, r.v_stride = a->v_stride;
    r.q_out_stride = a->q_out_stride;
    r.q_bias = a->q_bias, r.k_bias = a->k_bias, r.v_bias = a->v_bias;
    r.q_gain = a->q_gain, r.k_gain = a->k_gain;
    r.rope_table = reinterpret_cast<const unsigned long long *>(a->rope_table);
    r.positions = a->positions, r.seq = a->seq, r.pages = a->pages, r.status = a->status;
    r.k_pages = (uint8_t *)kv->k, r.v_pages = (uint8_t *)kv->v;
    r.page_stride = page_stride, r.head_bytes = head_bytes;
    r.type = kv->type, r.n_pages = kv->n_pages, r.page_size = kv->page_size;
    r.n_kv_heads = kv->n_kv_heads, r.head_dim = D;
    r.nt = a->nt, r.n_heads = a->n_heads, r.rope_dims = a->rope_dims, r.style = a->rope_style;
    r.n_seqs = a->n_seqs, r.pages_stride = a->pages_stride, r.eps = a->eps;
    const cudaError_t e = launch_rope_append(r, sms, pdl_setting(), (cudaStream_t)stream);
    return e == cudaSuccess ? MQ_OK : cuda_fail("rope_append launch", e);
}

size_t mq_attn_workspace_bytes(const mq_kv_cache *kv, int n_heads, int nt, int max_len)
{
    if (!kv || !attn_shape_ok(kv, n_heads, nt, max_len)) return 0;
    const int sms = mq_device_sms();
    if (sms <= 0) return 0;
    return attn_ws_bytes(kv, max_len, sms);
}

int mq_attn_decode(const mq_kv_cache *kv, const mq_attn_args *a, void *stream)
{
    if (!kv || !a) return MQ_ERR_NULL;
    size_t page_stride, head_bytes;
    const int st = kv_check(kv, &page_stride, &head_bytes);
    if (st != MQ_OK) return st;
    if (a->nt < 1) return MQ_ERR_SHAPE;  // empty tensors have no address
    if (!a->q || !a->out || !a->lens || !a->pages) return MQ_ERR_NULL;
    if (!attn_shape_ok(kv, a->n_heads, a->nt, a->max_len)) return MQ_ERR_SHAPE;
    const int D = kv->head_dim, n = a->n_heads * D;
    if (a->n_seqs < 1 || a->pages_stride < 1 || a->window < 0 || !isfinite(a->scale) ||
        !isfinite(a->softcap) || a->softcap < 0.0f || a->q_stride < n || a->out_stride < n)
        return MQ_ERR_SHAPE;
    if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->q8, 16) || !aligned(a->ws, 16) ||
        (a->q_stride | a->out_stride) % 4 != 0 || !aligned(a->lens, 4) || !aligned(a->seq, 4) ||
        !aligned(a->pages, 4) || !aligned(a->status, 4))
        return MQ_ERR_ALIGN;
    const int sms = mq_device_sms();
    if (sms <= 0) return MQ_ERR_CUDA;
    AttnLaunch r = {};
    r.group = a->n_heads / kv->n_kv_heads;
    r.subgroups = (r.group + kAttnHeads - 1) / kAttnHeads;
    const long long units = attn_units(kv, a->n_heads, a->nt);
    // a window starts inside a tile of its own
    long long span = a->max_len;
    if (a->window > 0 && (long long)a->window + kAttnTile - 1 < span) span = (long long)a->window + kAttnTile - 1;
    const long long rounds = attn_rounds(span, kv->type, D);
    r.ctas = (int)attn_grid(units, rounds, a->nt, sms);
    if (a->nt <= kAttnMaxRows && rounds > kAttnWhole) {
        if (!a->ws) return MQ_ERR_NULL;
        if (a->ws_bytes < attn_count_bytes(sms) + (size_t)r.ctas * 2 * attn_part_floats(D) * 4)
            return MQ_ERR_WORKSPACE;
        r.ws_cnt = (unsigned *)a->ws;
        r.ws_part = (float *)((uint8_t *)a->ws + attn_count_bytes(sms));
    }
    r.q = a->q, r.out = a->out, r.q_stride = a->q_stride, r.out_stride = a->out_stride;
    r.q8 = (uint8_t *)a->q8;
    r.q8_stride = (unsigned)q8_plane_bytes(n);
    r.q8_d_off = (unsigned)q8_d_offset(n), r.q8_sum_off = (unsigned)q8_sum_offset(n);
    r.lens = a->lens, r.seq = a->seq, r.pages = a->pages, r.status = a->status;
    r.k_pages = (const uint8_t *)kv->k, r.v_pages = (const uint8_t *)kv->v;
    r.page_stride = page_stride, r.head_bytes = head_bytes;
    r.type = kv->type, r.n_pages = kv->n_pages, r.page_size = kv->page_size;
    r.n_kv_heads = kv->n_kv_heads, r.head_dim = D;
    r.nt = a->nt, r.n_heads = a->n_heads, r.n_seqs = a->n_seqs, r.pages_stride = a->pages_stride;
    r.max_len = a->max_len, r.window = a->window, r.scale = a->scale, r.softcap = a->softcap;
    const cudaError_t e = launch_attn_decode(r, pdl_setting(), (cudaStream_t)stream);
    return e == cudaSuccess ? MQ_OK : cuda_fail("attn_decode launch", e);
}

int mq_sample(const mq_sample_args *a, void *stream)
{
    if (!a) return MQ_ERR_NULL;
    if (a->nt < 1 || a->vocab < 1) return MQ_ERR_SHAPE;  // empty tensors have no address
    if (!a->logits || !a->u || !a->token) return MQ_ERR_NULL;
    // the grid: up to 16 CTAs a row
    if (a->nt > (1 << 24) || a->vocab > MQ_SAMPLE_MAX_VOCAB || a->stride < a->vocab)
        return MQ_ERR_SHAPE;
    const void *p4[] = {a->logits, a->u, a->temperature, a->top_p, a->min_p, a->top_k, a->token, a->prob};
    for (const void *p : p4)
        if (!aligned(p, 4)) return MQ_ERR_ALIGN;
    const int sms = mq_device_sms();
    if (sms <= 0) return MQ_ERR_CUDA;
    SampleLaunch r = {};
    r.logits = a->logits, r.stride = a->stride, r.u = a->u;
    r.temperature = a->temperature, r.top_p = a->top_p, r.min_p = a->min_p, r.top_k = a->top_k;
    r.token = a->token, r.prob = a->prob;
    r.nt = a->nt, r.vocab = a->vocab;
    const cudaError_t e = launch_sample(r, sms, pdl_setting(), (cudaStream_t)stream);
    return e == cudaSuccess ? MQ_OK : cuda_fail("sample launch", e);
}

}  // extern "C"
