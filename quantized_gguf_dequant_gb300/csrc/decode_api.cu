// decode_api.cu -- C entries of the decode-step operators next to the
// quantized products: the paged key-value cache, the attention that reads
// it, and the adjustment of logits.  As everywhere in the library, every
// check happens on the host before anything is launched, and a refused call
// launches nothing.
#include <algorithm>
#include <climits>
#include <cstring>
#include <new>

#include "qmm_internal.h"

using qmm::KvCache;
using qmm::record_error;

namespace {

qmm_status cuda_error(cudaError_t e, const char *fn)
{
    return record_error(QMM_ERR_CUDA, "%s: CUDA error %d (%s): %s", fn, int(e),
                        cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Bytes of an activation type, or 0.
int64_t type_bytes(int dtype)
{
    return dtype == QMM_F32 ? 4 : (dtype == QMM_F16 || dtype == QMM_BF16 ? 2 : 0);
}

// Row counts and bytes of one of a cache's two buffers; the sentence of a
// refusal through record_error.
qmm_status cache_shape(const char *fn, int type, int64_t n_pages, int32_t page_size,
                       int32_t n_kv_heads, int32_t head_dim, int64_t *rows, int64_t *codes,
                       int64_t *bytes)
{
    if (type != QMM_F16 && type != QMM_BF16 && type != QMM_Q8_0)
        return record_error(QMM_ERR_FORMAT, "%s: cache type %d is not supported (F16 = 1, "
                            "Q8_0 = 8 and BF16 = 30 are)", fn, type);
    if (n_pages < 1 || page_size < 1 || n_kv_heads < 1)
        return record_error(QMM_ERR_SHAPE, "%s: %lld pages of %d slots for %d heads; each must be "
                            "at least 1", fn, (long long)n_pages, page_size, n_kv_heads);
    if (!qmm::attn_takes_head_dim(head_dim))
        return record_error(QMM_ERR_UNSUPPORTED, "%s: head_dim = %d is not implemented (64, 96, "
                            "128, 192 and 256 are)", fn, head_dim);
    if (n_kv_heads > (1 << 20))
        return record_error(QMM_ERR_SHAPE, "%s: n_kv_heads = %d; 2^20 at most are supported", fn,
                            n_kv_heads);
    const int64_t per_page = int64_t(page_size) * n_kv_heads;
    if (per_page > INT_MAX || n_pages > int64_t(0xffffffffll) / per_page)
        return record_error(QMM_ERR_SHAPE, "%s: %lld pages x %d slots x %d heads exceed 2^32 - 1 "
                            "rows", fn, (long long)n_pages, page_size, n_kv_heads);
    *rows = n_pages * per_page;
    if (type == QMM_Q8_0) {
        *codes = *rows * head_dim;
        *bytes = *codes + *rows * ((head_dim / 32 + 1) / 2 * 2) * 2;
    } else {
        *codes = *rows * head_dim * 2;
        *bytes = *codes;
    }
    return QMM_OK;
}

KvCache *as_cache(qmm_kv_t h) { return reinterpret_cast<KvCache *>(h); }

qmm_status check_cache(qmm_kv_t h, const char *fn)
{
    if (!h)
        return record_error(QMM_ERR_NULL, "%s: the cache handle is NULL", fn);
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return cuda_error(e, fn);
    if (dev != as_cache(h)->device)
        return record_error(QMM_ERR_CUDA, "%s: the cache was created on device %d but device %d "
                            "is current", fn, as_cache(h)->device, dev);
    return QMM_OK;
}

qmm_status check_dtype(const char *fn, int dtype)
{
    if (!type_bytes(dtype))
        return record_error(QMM_ERR_FORMAT, "%s: type %d is not supported (F32 = 0, F16 = 1 and "
                            "BF16 = 30 are)", fn, dtype);
    return QMM_OK;
}

// A tensor of `rows` rows, ld elements apart, each `width` elements from a
// 16-byte boundary on.
qmm_status check_rows(const char *fn, const char *name, const void *p, int64_t ld, int64_t width,
                      int dtype)
{
    if (!p)
        return record_error(QMM_ERR_NULL, "%s: %s is NULL", fn, name);
    if (ld < width || ld > (int64_t(1) << 40))
        return record_error(QMM_ERR_SHAPE, "%s: rows of %s are %lld elements apart; a row holds "
                            "%lld", fn, name, (long long)ld, (long long)width);
    if (!aligned(p, 16) || ld * type_bytes(dtype) % 16)
        return record_error(QMM_ERR_ALIGN, "%s: %s must start its rows on 16-byte boundaries", fn,
                            name);
    return QMM_OK;
}

} // namespace

namespace qmm {

FastDiv make_fast_div(uint32_t d)
{
    FastDiv f;
    f.d = d;
    f.shift = 0;
    while ((uint64_t(1) << f.shift) < d)
        ++f.shift;
    f.mul = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - d)) / d + 1);
    return f;
}

} // namespace qmm

namespace {

// Nothing may leave a C entry as an exception.
template <typename Body>
qmm_status guarded(Body body)
{
    try {
        qmm::clear_error();
        return body();
    } catch (...) {
        return QMM_ERR_NOMEM;
    }
}

} // namespace

extern "C" {

int64_t qmm_kv_bytes(int32_t type, int64_t n_pages, int32_t page_size, int32_t n_kv_heads,
                     int32_t head_dim)
{
    try {
        qmm::clear_error();
        int64_t rows, codes, bytes;
        const qmm_status st = cache_shape("qmm_kv_bytes", type, n_pages, page_size, n_kv_heads,
                                          head_dim, &rows, &codes, &bytes);
        return st == QMM_OK ? bytes : st;
    } catch (...) {
        return QMM_ERR_NOMEM;
    }
}

qmm_status qmm_kv_create(int32_t type, int64_t n_pages, int32_t page_size, int32_t n_kv_heads,
                         int32_t head_dim, void *k_dev, void *v_dev, qmm_kv_t *out)
{
    return guarded([&]() -> qmm_status {
        const char *fn = "qmm_kv_create";
        if (!out)
            return record_error(QMM_ERR_NULL, "%s: the output handle pointer is NULL", fn);
        *out = nullptr;
        int64_t rows, codes, bytes;
        const qmm_status st = cache_shape(fn, type, n_pages, page_size, n_kv_heads, head_dim,
                                          &rows, &codes, &bytes);
        if (st != QMM_OK)
            return st;
        if (!k_dev || !v_dev)
            return record_error(QMM_ERR_NULL, "%s: the %s buffer is NULL", fn,
                                !k_dev ? "key" : "value");
        if (!aligned(k_dev, 16) || !aligned(v_dev, 16))
            return record_error(QMM_ERR_ALIGN, "%s: the %s buffer is not 16-byte aligned", fn,
                                !aligned(k_dev, 16) ? "key" : "value");
        KvCache *c = new (std::nothrow) KvCache;
        if (!c)
            return record_error(QMM_ERR_NOMEM, "%s: out of host memory", fn);
        c->type = type;
        c->view.k = static_cast<uint8_t *>(k_dev);
        c->view.v = static_cast<uint8_t *>(v_dev);
        c->view.ks = type == QMM_Q8_0 ? c->view.k + codes : nullptr;
        c->view.vs = type == QMM_Q8_0 ? c->view.v + codes : nullptr;
        c->view.page = qmm::make_fast_div(uint32_t(page_size));
        c->view.n_pages = uint32_t(n_pages);
        c->view.n_rows = uint32_t(rows);
        c->view.page_size = page_size;
        c->view.n_heads = n_kv_heads;
        c->view.D = head_dim;
        cudaError_t e = cudaGetDevice(&c->device);
        if (e == cudaSuccess)
            e = cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, c->device);
        if (e != cudaSuccess) {
            delete c;
            return cuda_error(e, fn);
        }
        const qmm::AttnSpace space = qmm::attn_space(type, head_dim);
        c->max_blocks = c->sm_count * space.blocks;
        const size_t words = size_t(c->max_blocks) * 3 + 64;  // tickets, status word
        c->ws_bytes = size_t(c->sm_count) * space.floats * 4;
        void *p = nullptr;
        e = cudaMalloc(&p, c->ws_bytes + words * 4);
        if (e != cudaSuccess) {
            const size_t need = c->ws_bytes + words * 4;
            delete c;
            return record_error(QMM_ERR_NOMEM, "%s: could not allocate the %zu-byte workspace (%s)",
                                fn, need, cudaGetErrorString(e));
        }
        c->ws = static_cast<float *>(p);
        c->tickets = reinterpret_cast<unsigned *>(static_cast<uint8_t *>(p) + c->ws_bytes);
        c->status = c->tickets + 3 * c->max_blocks;
        e = cudaMemset(c->tickets, 0, words * 4);
        if (e == cudaSuccess)
            e = cudaStreamSynchronize(nullptr);  // zeroed before a call on any stream
        if (e != cudaSuccess) {
            cudaFree(p);
            delete c;
            return cuda_error(e, fn);
        }
        *out = reinterpret_cast<qmm_kv_t>(c);
        return QMM_OK;
    });
}

qmm_status qmm_kv_destroy(qmm_kv_t h)
{
    return guarded([&]() -> qmm_status {
        if (!h)
            return record_error(QMM_ERR_NULL, "qmm_kv_destroy: the cache handle is NULL");
        KvCache *c = as_cache(h);
        int dev = -1;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess && dev != c->device)
            e = cudaSetDevice(c->device);
        if (e == cudaSuccess)
            e = cudaDeviceSynchronize();
        const cudaError_t e2 = cudaFree(c->ws);
        if (dev >= 0 && dev != c->device)
            cudaSetDevice(dev);
        delete c;
        if (e != cudaSuccess || e2 != cudaSuccess)
            return cuda_error(e != cudaSuccess ? e : e2, "qmm_kv_destroy");
        return QMM_OK;
    });
}

qmm_status qmm_kv_append(qmm_kv_t h, int32_t dtype, int64_t T, const void *k, int64_t ldk,
                         const void *v, int64_t ldv, const int64_t *slots, const void *q,
                         int64_t ldq, int32_t n_q_heads, void *q_out, int64_t ldqo,
                         const int32_t *pos, const qmm_rope *rope, qmm_stream stream)
{
    return guarded([&]() -> qmm_status {
        const char *fn = "qmm_kv_append";
        qmm_status st = check_cache(h, fn);
        if (st != QMM_OK)
            return st;
        const KvCache &c = *as_cache(h);
        const int D = c.view.D;
        if ((st = check_dtype(fn, dtype)) != QMM_OK)
            return st;
        if (T < 0 || T > INT_MAX)
            return record_error(QMM_ERR_SHAPE, "%s: T = %lld tokens; between 0 and 2^31 - 1 are "
                                "supported", fn, (long long)T);
        if (T == 0)
            return QMM_OK;
        const int64_t width = int64_t(c.view.n_heads) * D;
        if ((st = check_rows(fn, "k", k, ldk, width, dtype)) != QMM_OK ||
            (st = check_rows(fn, "v", v, ldv, width, dtype)) != QMM_OK)
            return st;
        if (!slots)
            return record_error(QMM_ERR_NULL, "%s: slots is NULL", fn);
        if (!aligned(slots, 8))
            return record_error(QMM_ERR_ALIGN, "%s: slots is not 8-byte aligned", fn);
        qmm::AppendArgs a;
        memset(&a, 0, sizeof(a));
        if (q) {
            if (n_q_heads < 1 || int64_t(n_q_heads) * D > (int64_t(1) << 30))
                return record_error(QMM_ERR_SHAPE, "%s: n_q_heads = %d", fn, n_q_heads);
            if ((st = check_rows(fn, "q", q, ldq, int64_t(n_q_heads) * D, dtype)) != QMM_OK ||
                (st = check_rows(fn, "q_out", q_out, ldqo, int64_t(n_q_heads) * D, dtype)) !=
                    QMM_OK)
                return st;
            if (q == q_out && ldq != ldqo)
                return record_error(QMM_ERR_SHAPE, "%s: q_out is q but its rows are %lld elements "
                                    "apart, those of q %lld", fn, (long long)ldqo, (long long)ldq);
            a.q = q;
            a.q_out = q_out;
            a.ldq = ldq;
            a.ldqo = ldqo;
            a.n_q = n_q_heads;
        }
        if (rope && rope->n_rot) {
            if (rope->n_rot < 0 || rope->n_rot > D || rope->n_rot % 2)
                return record_error(QMM_ERR_SHAPE, "%s: n_rot = %d; an even number up to head_dim "
                                    "= %d is required", fn, rope->n_rot, D);
            if (rope->pairing != QMM_ROPE_HALVES && rope->pairing != QMM_ROPE_ADJACENT)
                return record_error(QMM_ERR_UNSUPPORTED, "%s: pairing %d is not implemented "
                                    "(halves = 0 and adjacent = 1 are)", fn, rope->pairing);
            if (rope->n_axes < 1 || rope->n_axes > 4)
                return record_error(QMM_ERR_SHAPE, "%s: n_axes = %d; between 1 and 4 are supported",
                                    fn, rope->n_axes);
            int64_t sum = 0;
            for (int i = 0; i < 4; ++i) {
                if (i < rope->n_axes) {
                    if (rope->sections[i] < 0 || rope->sections[i] > D)
                        return record_error(QMM_ERR_SHAPE, "%s: section %d has %d pairs", fn, i,
                                            rope->sections[i]);
                    sum += rope->sections[i];
                }
                a.axis_end[i] = int(sum);
            }
            if (sum != rope->n_rot / 2)
                return record_error(QMM_ERR_SHAPE, "%s: the sections hold %lld pairs, n_rot = %d "
                                    "has %d", fn, (long long)sum, rope->n_rot, rope->n_rot / 2);
            if (!rope->inv_freq || !pos)
                return record_error(QMM_ERR_NULL, "%s: %s is NULL", fn,
                                    !pos ? "pos" : "rope->inv_freq");
            if (!aligned(rope->inv_freq, 4) || !aligned(pos, 4))
                return record_error(QMM_ERR_ALIGN, "%s: pos and inv_freq must be 4-byte aligned",
                                    fn);
            a.n_rot = rope->n_rot;
            a.adjacent = rope->pairing == QMM_ROPE_ADJACENT;
            a.n_axes = rope->n_axes;
            a.inv_freq = rope->inv_freq;
            a.pos = pos;
        }
        a.c = c.view;
        a.type = c.type;
        a.dtype = dtype;
        a.T = T;
        a.k = k;
        a.v = v;
        a.ldk = ldk;
        a.ldv = ldv;
        a.slots = slots;
        a.status = c.status;
        const cudaError_t e =
            qmm::launch_kv_append(a, c.sm_count, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? QMM_OK : cuda_error(e, fn);
    });
}

qmm_status qmm_kv_read(qmm_kv_t h, int32_t dtype, int64_t T, const int64_t *slots, void *k_out,
                       int64_t ldk, void *v_out, int64_t ldv, qmm_stream stream)
{
    return guarded([&]() -> qmm_status {
        const char *fn = "qmm_kv_read";
        qmm_status st = check_cache(h, fn);
        if (st != QMM_OK)
            return st;
        const KvCache &c = *as_cache(h);
        if ((st = check_dtype(fn, dtype)) != QMM_OK)
            return st;
        if (T < 0 || T > INT_MAX)
            return record_error(QMM_ERR_SHAPE, "%s: T = %lld tokens; between 0 and 2^31 - 1 are "
                                "supported", fn, (long long)T);
        if (T == 0)
            return QMM_OK;
        if (!slots || (!k_out && !v_out))
            return record_error(QMM_ERR_NULL, "%s: %s NULL", fn,
                                !slots ? "slots is" : "both outputs are");
        if (!aligned(slots, 8))
            return record_error(QMM_ERR_ALIGN, "%s: slots is not 8-byte aligned", fn);
        const int64_t width = int64_t(c.view.n_heads) * c.view.D;
        if ((k_out && (st = check_rows(fn, "k_out", k_out, ldk, width, dtype)) != QMM_OK) ||
            (v_out && (st = check_rows(fn, "v_out", v_out, ldv, width, dtype)) != QMM_OK))
            return st;
        qmm::KvReadArgs a;
        memset(&a, 0, sizeof(a));
        a.c = c.view;
        a.type = c.type;
        a.dtype = dtype;
        a.T = T;
        a.slots = slots;
        a.k = k_out;
        a.v = v_out;
        a.ldk = ldk;
        a.ldv = ldv;
        a.status = c.status;
        const cudaError_t e =
            qmm::launch_kv_read(a, c.sm_count, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? QMM_OK : cuda_error(e, fn);
    });
}

qmm_status qmm_attn_decode(qmm_kv_t h, int32_t dtype, int64_t n_seqs, int32_t n_q_heads,
                           const void *q, int64_t ldq, const int32_t *page_table,
                           int64_t ld_table, const int32_t *lens, const qmm_attn *attn, void *out,
                           int64_t ldo, float *lse, qmm_stream stream)
{
    return guarded([&]() -> qmm_status {
        const char *fn = "qmm_attn_decode";
        qmm_status st = check_cache(h, fn);
        if (st != QMM_OK)
            return st;
        const KvCache &c = *as_cache(h);
        if ((st = check_dtype(fn, dtype)) != QMM_OK)
            return st;
        if (n_seqs < 0 || n_seqs > (1 << 20))
            return record_error(QMM_ERR_SHAPE, "%s: n_seqs = %lld; between 0 and 2^20 are "
                                "supported", fn, (long long)n_seqs);
        if (n_q_heads < 1 || n_q_heads % c.view.n_heads || n_q_heads > (1 << 20))
            return record_error(QMM_ERR_SHAPE, "%s: n_q_heads = %d is not a positive multiple of "
                                "the cache's %d heads (2^20 at most)", fn, n_q_heads,
                                c.view.n_heads);
        if (!attn)
            return record_error(QMM_ERR_NULL, "%s: the attention options are NULL", fn);
        if (!(attn->scale - attn->scale == 0.f) || !(attn->softcap >= 0.f) ||
            !(attn->softcap - attn->softcap == 0.f))
            return record_error(QMM_ERR_SHAPE, "%s: scale = %g must be finite, softcap = %g finite "
                                "and not negative", fn, double(attn->scale),
                                double(attn->softcap));
        if (attn->window < 0)
            return record_error(QMM_ERR_SHAPE, "%s: window = %d; 0 (all keys) or more is required",
                                fn, attn->window);
        if (n_seqs == 0)
            return QMM_OK;
        const int64_t width = int64_t(n_q_heads) * c.view.D;
        if ((st = check_rows(fn, "q", q, ldq, width, dtype)) != QMM_OK ||
            (st = check_rows(fn, "out", out, ldo, width, dtype)) != QMM_OK)
            return st;
        if (!lens || !page_table)
            return record_error(QMM_ERR_NULL, "%s: %s is NULL", fn,
                                !lens ? "lens" : "the page table");
        if (ld_table < 1 || ld_table > INT_MAX)
            return record_error(QMM_ERR_SHAPE, "%s: ld_table = %lld pages a row; between 1 and "
                                "2^31 - 1 are supported", fn, (long long)ld_table);
        if (!aligned(lens, 4) || !aligned(page_table, 4) || !aligned(lse, 4) ||
            !aligned(attn->alibi, 4))
            return record_error(QMM_ERR_ALIGN, "%s: lens, the page table, alibi and lse must be "
                                "4-byte aligned", fn);
        qmm::AttnArgs a;
        memset(&a, 0, sizeof(a));
        a.c = c.view;
        a.type = c.type;
        a.dtype = dtype;
        a.n_seqs = int(n_seqs);
        a.n_q = n_q_heads;
        a.q = q;
        a.out = out;
        a.ldq = ldq;
        a.ldo = ldo;
        a.table = page_table;
        a.ld_table = ld_table;
        a.lens = lens;
        a.scale = attn->scale;
        a.softcap = attn->softcap;
        a.window = attn->window;
        a.alibi = attn->alibi;
        a.lse = lse;
        a.ws = c.ws;
        a.tickets = c.tickets;
        a.status = c.status;
        a.max_blocks = c.max_blocks;
        a.device = c.device;
        const cudaError_t e =
            qmm::launch_attn_decode(a, c.sm_count, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? QMM_OK : cuda_error(e, fn);
    });
}

qmm_status qmm_kv_get_status(qmm_kv_t h)
{
    return guarded([&]() -> qmm_status {
        const char *fn = "qmm_kv_get_status";
        const qmm_status st = check_cache(h, fn);
        if (st != QMM_OK)
            return st;
        KvCache *c = as_cache(h);
        unsigned word = 0;
        cudaError_t e = cudaDeviceSynchronize();
        if (e == cudaSuccess)
            e = cudaMemcpy(&word, c->status, 4, cudaMemcpyDeviceToHost);
        if (e == cudaSuccess && word) {
            e = cudaMemset(c->status, 0, 4);
            if (e == cudaSuccess)
                e = cudaStreamSynchronize(nullptr);
        }
        if (e != cudaSuccess)
            return cuda_error(e, fn);
        if (word & qmm::kStatusBadSlotBit)
            return record_error(QMM_ERR_PAGE, "%s: a slot was outside the cache's %u pages of %d; "
                                "it was not stored, or read as zeros", fn, c->view.n_pages,
                                c->view.page_size);
        if (word & qmm::kStatusBadPageBit)
            return record_error(QMM_ERR_PAGE, "%s: a page id was outside [0, %u); its keys were "
                                "left out", fn, c->view.n_pages);
        if (word & qmm::kStatusBadLengthBit)
            return record_error(QMM_ERR_PAGE, "%s: a length was negative or beyond its row of the "
                                "page table; it was cut to fit", fn);
        return QMM_OK;
    });
}

qmm_status qmm_logits_adjust(int32_t dtype, int64_t n_rows, int64_t n_vocab, const void *logits,
                             int64_t ld, const qmm_logit_rules *rules, void *out, int64_t ldo,
                             qmm_stream stream)
{
    return guarded([&]() -> qmm_status {
        const char *fn = "qmm_logits_adjust";
        qmm_status st = check_dtype(fn, dtype);
        if (st != QMM_OK)
            return st;
        if (n_rows < 0 || n_rows > INT_MAX)
            return record_error(QMM_ERR_SHAPE, "%s: n_rows = %lld; between 0 and 2^31 - 1 are "
                                "supported", fn, (long long)n_rows);
        if (n_vocab < 1 || n_vocab > (int64_t(1) << 26))
            return record_error(QMM_ERR_SHAPE, "%s: n_vocab = %lld; between 1 and 2^26 are "
                                "supported", fn, (long long)n_vocab);
        if (!rules)
            return record_error(QMM_ERR_NULL, "%s: the rules are NULL", fn);
        if (n_rows == 0)
            return QMM_OK;
        if (!logits || !out)
            return record_error(QMM_ERR_NULL, "%s: %s is NULL", fn, !logits ? "logits" : "out");
        if (ld < n_vocab || ldo < n_vocab || ld > (int64_t(1) << 40) || ldo > (int64_t(1) << 40))
            return record_error(QMM_ERR_SHAPE, "%s: rows are %lld and %lld elements apart; a row "
                                "holds %lld", fn, (long long)ld, (long long)ldo,
                                (long long)n_vocab);
        const size_t es = size_t(type_bytes(dtype));
        if (!aligned(logits, es) || !aligned(out, es))
            return record_error(QMM_ERR_ALIGN, "%s: logits and out must be %zu-byte aligned", fn,
                                es);
        if (logits == out && ld != ldo)
            return record_error(QMM_ERR_SHAPE, "%s: out is logits but its rows are %lld elements "
                                "apart, those of logits %lld", fn, (long long)ldo, (long long)ld);
        const qmm_logit_rules &r = *rules;
        if (r.n_history < 0 || r.n_biases < 0 || r.n_biases > INT_MAX)
            return record_error(QMM_ERR_SHAPE, "%s: %lld history tokens and %lld biases", fn,
                                (long long)r.n_history, (long long)r.n_biases);
        if (r.n_history > 0 && (!r.history || !r.history_offsets))
            return record_error(QMM_ERR_NULL, "%s: %s is NULL", fn,
                                !r.history ? "history" : "history_offsets");
        if (r.n_biases > 0 && (!r.bias_ids || !r.bias_values || !r.bias_offsets))
            return record_error(QMM_ERR_NULL, "%s: %s is NULL", fn,
                                !r.bias_ids ? "bias_ids"
                                            : (!r.bias_values ? "bias_values" : "bias_offsets"));
        if (r.mask && r.ld_mask != 0 && r.ld_mask < (n_vocab + 31) / 32)
            return record_error(QMM_ERR_SHAPE, "%s: mask rows of %lld words do not hold %lld bits "
                                "(0 shares one row)", fn, (long long)r.ld_mask,
                                (long long)n_vocab);
        if (!aligned(r.history, 4) || !aligned(r.bias_ids, 4) || !aligned(r.bias_values, 4) ||
            !aligned(r.repeat, 4) || !aligned(r.presence, 4) || !aligned(r.frequency, 4) ||
            !aligned(r.mask, 4) || !aligned(r.history_offsets, 8) || !aligned(r.bias_offsets, 8))
            return record_error(QMM_ERR_ALIGN, "%s: the rules' arrays must be aligned to their "
                                "elements", fn);
        int dev = 0, sms = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess)
            e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess)
            return cuda_error(e, fn);
        qmm::LogitsArgs a;
        memset(&a, 0, sizeof(a));
        a.dtype = dtype;
        a.B = n_rows;
        a.V = n_vocab;
        a.in = logits;
        a.out = out;
        a.ld_in = ld;
        a.ld_out = ldo;
        // without a penalty there is nothing to count for
        const bool penal = r.repeat || r.presence || r.frequency;
        a.history = r.history;
        a.history_offsets = r.history_offsets;
        a.n_history = penal ? r.n_history : 0;
        a.repeat = r.repeat;
        a.presence = r.presence;
        a.frequency = r.frequency;
        a.bias_ids = r.bias_ids;
        a.bias_values = r.bias_values;
        a.bias_offsets = r.bias_offsets;
        a.n_biases = r.n_biases;
        a.mask = r.mask;
        a.ld_mask = r.ld_mask;
        e = qmm::launch_logits_adjust(a, sms, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? QMM_OK : cuda_error(e, fn);
    });
}

} // extern "C"
