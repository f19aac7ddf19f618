// attn_api.cu -- the C ABI (include/sv_attention.h): argument checks and
// launches.
#include <cmath>

#include "attn_internal.h"
#include "sv_attention.h"

#define SV_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

constexpr int64_t kMax31 = int64_t(1) << 31;

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Host checks of a cache description, and the kernels' form of it.
int check_cache(const sv_paged_cache* d, sva::Cache* c)
{
    if (d == nullptr) return SV_ERR_ARG;
    if (d->dtype != SV_BF16 && d->dtype != SV_F16 && d->dtype != SV_E4M3) return SV_ERR_DTYPE;
    if (d->batch < 0 || d->kv_heads < 1 || d->num_pages < 0 || d->max_pages < 0 ||
        d->table_stride < d->max_pages)
        return SV_ERR_ARG;
    if (d->head_dim < 16 || d->head_dim > 256 || d->head_dim % 16 != 0) return SV_ERR_SIZE;
    if (d->page_size < 8 || d->page_size > 1024 || (d->page_size & (d->page_size - 1)) != 0)
        return SV_ERR_SIZE;
    if (d->batch >= kMax31 || d->num_pages >= kMax31 || d->max_pages >= kMax31 ||
        d->kv_heads > 65535 || d->table_stride >= (int64_t(1) << 40))
        return SV_ERR_SIZE;
    const int es = d->dtype == SV_E4M3 ? 1 : 2;
    *c = sva::Cache{};
    for (int i = 0; i < 2; ++i) {
        // Pages, slots, heads: elements, then bytes. Where there is one of a kind its
        // stride says nothing (torch leaves any number there).
        int64_t st[3] = {d->page_stride[i], d->slot_stride[i], d->head_stride[i]};
        int64_t ex[3] = {d->exp_page_stride[i], d->exp_slot_stride[i], d->exp_head_stride[i]};
        if (d->num_pages <= 1) st[0] = d->head_dim, ex[0] = 0;
        if (d->kv_heads == 1) st[2] = d->head_dim, ex[2] = 0;
        for (int64_t& s : st) {
            if (s < 0 || s >= (int64_t(1) << 40) / es) return SV_ERR_ARG;
            s *= es;
            if (s % 16 != 0) return SV_ERR_ALIGN;
        }
        if (d->batch > 0 && d->num_pages > 0) {
            if (d->pages[i] == nullptr) return SV_ERR_ARG;
            if (d->dtype == SV_E4M3 && d->exps[i] == nullptr) return SV_ERR_ARG;
        }
        if (d->dtype != SV_E4M3 && d->exps[i] != nullptr) return SV_ERR_ARG;
        if (!aligned(d->pages[i], 16)) return SV_ERR_ALIGN;
        if (d->dtype == SV_E4M3)
            for (int64_t s : ex)
                if (s < 0 || s >= (int64_t(1) << 40)) return SV_ERR_ARG;
        c->pages[i] = static_cast<uint8_t*>(d->pages[i]);
        c->exps[i] = d->exps[i];
        c->page_stride[i] = st[0];
        c->slot_stride[i] = st[1];
        c->head_stride[i] = st[2];
        c->exp_page_stride[i] = ex[0];
        c->exp_slot_stride[i] = ex[1];
        c->exp_head_stride[i] = ex[2];
    }
    if (d->batch > 0) {
        if ((d->max_pages > 0 && d->page_table == nullptr) || d->cached_lens == nullptr ||
            d->chunk_starts == nullptr)
            return SV_ERR_ARG;
        if (!aligned(d->page_table, 4) || !aligned(d->cached_lens, 4) ||
            !aligned(d->chunk_starts, 4))
            return SV_ERR_ALIGN;
    }
    c->table = d->page_table;
    c->cached = d->cached_lens;
    c->starts = d->chunk_starts;
    c->table_stride = d->table_stride;
    c->capacity = d->max_pages * d->page_size;
    c->num_pages = static_cast<int32_t>(d->num_pages);
    int shift = 0;
    while ((1 << shift) < d->page_size) ++shift;
    c->page_shift = shift;
    c->B = static_cast<int32_t>(d->batch);
    c->Hkv = d->kv_heads;
    c->D = d->head_dim;
    return SV_OK;
}

// dtype of the packed arrays against the cache's.
int check_dtype(int dtype, const sv_paged_cache* d)
{
    if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
    if (d->dtype != SV_E4M3 && d->dtype != dtype) return SV_ERR_DTYPE;
    return SV_OK;
}

// The strides of packed rows; those of one token or one head become 0.
int check_rows(const void* x, int64_t tokens, int64_t heads, int64_t& token_stride,
               int64_t& head_stride)
{
    if (tokens <= 1) token_stride = 0;
    if (heads == 1) head_stride = 0;
    if (token_stride < 0 || head_stride < 0 || token_stride >= (int64_t(1) << 40) ||
        head_stride >= (int64_t(1) << 40))
        return SV_ERR_ARG;
    if (tokens > 0 && x == nullptr) return SV_ERR_ARG;
    if (!aligned(x, 16) || token_stride % 8 != 0 || head_stride % 8 != 0) return SV_ERR_ALIGN;
    return SV_OK;
}

int clear_status(int32_t* status, int64_t batch, cudaStream_t s)
{
    if (status == nullptr || batch == 0) return SV_OK;
    return cudaMemsetAsync(status, 0, batch * sizeof(int32_t), s) == cudaSuccess ? SV_OK
                                                                                : SV_ERR_CUDA;
}

}  // namespace

SV_EXPORT int sv_kv_append(const sv_paged_cache* cache, const void* key, const void* value,
                           int dtype, int64_t tokens, int64_t key_token_stride,
                           int64_t key_head_stride, int64_t value_token_stride,
                           int64_t value_head_stride, int32_t* seq_status, void* stream)
{
    sva::Cache c;
    int rc = check_cache(cache, &c);
    if (rc == SV_OK) rc = check_dtype(dtype, cache);
    if (rc != SV_OK) return rc;
    if (tokens < 0) return SV_ERR_ARG;
    if (tokens >= kMax31) return SV_ERR_SIZE;
    rc = check_rows(key, tokens, c.Hkv, key_token_stride, key_head_stride);
    if (rc == SV_OK) rc = check_rows(value, tokens, c.Hkv, value_token_stride, value_head_stride);
    if (rc == SV_OK && !aligned(seq_status, 4)) rc = SV_ERR_ALIGN;
    if (rc != SV_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((rc = clear_status(seq_status, c.B, s)) != SV_OK) return rc;
    sva::Packed p{{static_cast<uint8_t*>(const_cast<void*>(key)),
                   static_cast<uint8_t*>(const_cast<void*>(value))},
                  {key_token_stride * 2, value_token_stride * 2},
                  {key_head_stride * 2, value_head_stride * 2},
                  tokens,
                  seq_status};
    return sva::launch_append(c, p, dtype == SV_F16, cache->dtype == SV_E4M3, s) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

SV_EXPORT int sv_kv_read(const sv_paged_cache* cache, void* key, void* value, int dtype,
                         int64_t tokens, int32_t* seq_status, void* stream)
{
    sva::Cache c;
    int rc = check_cache(cache, &c);
    if (rc == SV_OK) rc = check_dtype(dtype, cache);
    if (rc != SV_OK) return rc;
    if (tokens < 0) return SV_ERR_ARG;
    if (tokens >= kMax31) return SV_ERR_SIZE;
    int64_t hs = c.D, ts = static_cast<int64_t>(c.Hkv) * c.D;
    rc = check_rows(key, tokens, c.Hkv, ts, hs);
    if (rc == SV_OK) rc = check_rows(value, tokens, c.Hkv, ts, hs);
    if (rc == SV_OK && !aligned(seq_status, 4)) rc = SV_ERR_ALIGN;
    if (rc != SV_OK) return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((rc = clear_status(seq_status, c.B, s)) != SV_OK) return rc;
    sva::Packed p{{static_cast<uint8_t*>(key), static_cast<uint8_t*>(value)},
                  {ts * 2, ts * 2},
                  {hs * 2, hs * 2},
                  tokens,
                  seq_status};
    return sva::launch_read(c, p, dtype == SV_F16, cache->dtype == SV_E4M3, s) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

namespace {

int check_attention(int64_t batch, int64_t tokens, int64_t q_heads, int64_t kv_heads,
                    int64_t head_dim, int64_t* max_chunk)
{
    if (batch < 0 || tokens < 0 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 ||
        *max_chunk < 0)
        return SV_ERR_ARG;
    if (batch >= kMax31 || tokens >= kMax31 || q_heads > 65535 || head_dim < 16 ||
        head_dim > 256 || head_dim % 16 != 0 || tokens * q_heads >= (int64_t(1) << 40))
        return SV_ERR_SIZE;
    if (*max_chunk == 0 || *max_chunk > tokens) *max_chunk = tokens;
    // (a sequence's rows are counted in 32 bits)
    if (*max_chunk * (q_heads / kv_heads) >= kMax31 - 512) return SV_ERR_SIZE;
    return SV_OK;
}

}  // namespace

SV_EXPORT int sv_chunk_attention_workspace_bytes(int64_t batch, int64_t tokens, int64_t q_heads,
                                                 int64_t kv_heads, int64_t head_dim,
                                                 int64_t max_chunk, size_t* bytes)
{
    if (bytes == nullptr) return SV_ERR_ARG;
    const int rc = check_attention(batch, tokens, q_heads, kv_heads, head_dim, &max_chunk);
    if (rc != SV_OK) return rc;
    *bytes = sva::tiles_workspace(max_chunk, q_heads / kv_heads, head_dim);
    return SV_OK;
}

namespace {

int attention(const sv_paged_cache* cache, const void* query, int dtype, int64_t tokens,
              int64_t q_heads, int64_t query_token_stride, int64_t query_head_stride, float scale,
              int64_t window, int64_t max_chunk, void* out, float* lse, int32_t* seq_status,
              void* workspace, size_t workspace_bytes, void* stream, int32_t gate_block,
              const int32_t* gate)
{
    sva::Attn a{};
    int rc = check_cache(cache, &a.c);
    if (rc == SV_OK) rc = check_dtype(dtype, cache);
    if (rc == SV_OK)
        rc = check_attention(cache->batch, tokens, q_heads, cache->kv_heads, cache->head_dim,
                             &max_chunk);
    if (rc != SV_OK) return rc;
    if (!(scale > 0.f) || !std::isfinite(scale * 1.44269504f)) return SV_ERR_ARG;
    if (window < 0 || window >= kMax31) return SV_ERR_ARG;
    rc = check_rows(query, tokens, q_heads, query_token_stride, query_head_stride);
    if (rc != SV_OK) return rc;
    if (tokens > 0 && out == nullptr) return SV_ERR_ARG;
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(seq_status, 4)) return SV_ERR_ALIGN;
    size_t need = 0;
    rc = sv_chunk_attention_workspace_bytes(cache->batch, tokens, q_heads, cache->kv_heads,
                                            cache->head_dim, max_chunk, &need);
    if (rc != SV_OK) return rc;
    if (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 256))
        return SV_ERR_WORKSPACE;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((rc = clear_status(seq_status, cache->batch, s)) != SV_OK) return rc;
    if (cache->batch == 0 || (tokens == 0 && seq_status == nullptr)) return SV_OK;
    a.q = static_cast<const uint8_t*>(query);
    a.q_token = query_token_stride * 2;
    a.q_head = query_head_stride * 2;
    a.out = static_cast<uint8_t*>(out);
    a.lse = lse;
    a.status = seq_status;
    a.tokens = tokens;
    a.max_chunk = max_chunk;
    a.window = window;
    a.Hq = static_cast<int32_t>(q_heads);
    a.G = static_cast<int32_t>(q_heads / cache->kv_heads);
    a.scale = scale;
    a.scale_log2 = scale * 1.44269504088896341f;
    a.gate = gate;
    a.gate_block = gate_block;
    const bool f16 = dtype == SV_F16, e4m3 = cache->dtype == SV_E4M3;
    const bool few = max_chunk * a.G <= sva::kFewRows || a.c.D > sva::kMaxTileDim;
    const auto launch = few ? sva::launch_attention_few : sva::launch_attention_tiles;
    // (without rows there are only statuses to find)
    return (a.c.num_pages == 0 || tokens == 0 ? sva::launch_attention_no_pages(a, f16, s)
                                              : launch(a, f16, e4m3, workspace, s)) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

}  // namespace

SV_EXPORT int sv_chunk_attention(const sv_paged_cache* cache, const void* query, int dtype,
                                 int64_t tokens, int64_t q_heads, int64_t query_token_stride,
                                 int64_t query_head_stride, float scale, int64_t window,
                                 int64_t max_chunk, void* out, float* lse, int32_t* seq_status,
                                 void* workspace, size_t workspace_bytes, void* stream)
{
    return attention(cache, query, dtype, tokens, q_heads, query_token_stride, query_head_stride,
                     scale, window, max_chunk, out, lse, seq_status, workspace, workspace_bytes,
                     stream, -1, nullptr);
}

SV_EXPORT int sv_chunk_attention_gated(const sv_paged_cache* cache, const void* query, int dtype,
                                       int64_t tokens, int64_t q_heads,
                                       int64_t query_token_stride, int64_t query_head_stride,
                                       float scale, int64_t window, int64_t max_chunk, void* out,
                                       float* lse, int32_t* seq_status, void* workspace,
                                       size_t workspace_bytes, void* stream, int32_t block,
                                       const int32_t* gate)
{
    if (gate == nullptr) return SV_ERR_ARG;
    if (!aligned(gate, 4)) return SV_ERR_ALIGN;
    return attention(cache, query, dtype, tokens, q_heads, query_token_stride, query_head_stride,
                     scale, window, max_chunk, out, lse, seq_status, workspace, workspace_bytes,
                     stream, block, gate);
}
