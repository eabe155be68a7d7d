// decode.cpp -- the C ABI of the operators around the GEMVs of a decode step
// (include/mq.h: paged cache, rotation and append): argument checks, then the
// launch.  Nothing here allocates.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kernels.h"
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
    if (!a->q || !a->k || !a->v || !a->q_out || !a->positions || !a->pages) return MQ_ERR_NULL;
    const int D = kv->head_dim;
    const long long nq = (long long)a->n_heads * D, nk = (long long)kv->n_kv_heads * D;
    if (a->nt < 1 || a->n_heads < 1 || a->n_heads % kv->n_kv_heads != 0 || a->n_heads > (1 << 20) ||
        kv->n_kv_heads > (1 << 20) || a->n_seqs < 1 || a->pages_stride < 1)
        return MQ_ERR_SHAPE;
    if (a->rope_dims < 0 || a->rope_dims > D || a->rope_dims % (D > 128 ? 16 : 8) != 0 ||
        (a->rope_style != MQ_ROPE_HALF && a->rope_style != MQ_ROPE_PAIRS))
        return MQ_ERR_SHAPE;
    if (a->rope_dims > 0 && !a->rope_table) return MQ_ERR_NULL;
    if (a->q_stride < nq || a->q_out_stride < nq || a->k_stride < nk || a->v_stride < nk)
        return MQ_ERR_SHAPE;
    // one CTA per row at the least: the grid's x dimension holds 2^31 - 1
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

}  // extern "C"
