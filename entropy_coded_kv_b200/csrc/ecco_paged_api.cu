// C ABI of the paged cache: argument checks and dispatch.  The device-side
// arrays (page table, lengths) are bounded by the kernels; everything the host
// can see is checked here, and nothing is enqueued on an error.
#include <algorithm>
#include <cmath>
#include <vector>

#include "ecco_paged.cuh"

using namespace ecco;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int status(cudaError_t e) { return e == cudaSuccess ? ECCO_OK : ECCO_ERR_CUDA; }

int check_tables(const ecco_tables* t)
{
    if (!t || !t->d) return ECCO_ERR_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return ECCO_ERR_CUDA;
    return dev == t->device ? ECCO_OK : ECCO_ERR_DEVICE;
}

constexpr int64_t kMaxElems = (int64_t)1 << 40;

int check_paged(const ecco_paged& p, bool queries)
{
    if (p.n_pages < 0 || p.n_pages > 0x7fffffff || p.page_size < 1 || p.page_size > 65536) return ECCO_ERR_ARG;
    if (p.kv_heads < 1 || p.kv_heads > 1024 || p.batch < 0 || p.batch > ECCO_MAX_BATCH) return ECCO_ERR_ARG;
    if (p.max_pages < 0 || (int64_t)p.max_pages * p.page_size > ((int64_t)1 << 30)) return ECCO_ERR_ARG;
    if (p.n_pages * p.kv_heads > kMaxElems / p.page_size) return ECCO_ERR_ARG;
    if (p.table_stride < 0 || p.table_stride > kMaxElems / ECCO_MAX_BATCH ||
        (p.batch > 1 && p.table_stride < p.max_pages))
        return ECCO_ERR_ARG;
    if (p.batch > 0 && ((p.max_pages > 0 && !p.page_table) || !p.kv_lens || (queries && !p.cu_q))) return ECCO_ERR_ARG;
    if (!aligned(p.page_table, 4) || !aligned(p.kv_lens, 4) || !aligned(p.cu_q, 4)) return ECCO_ERR_ALIGN;
    return ECCO_OK;
}

// Strides of a [tokens][heads][..] array whose rows hold 16-byte pieces of `per` elements.
int check_strides(int64_t tokens, int64_t heads, int64_t token, int64_t head, int per)
{
    if (token < 0 || head < 0 || token > kMaxElems || head > kMaxElems) return ECCO_ERR_ARG;
    if ((tokens > 0 && token > kMaxElems / tokens) || head > kMaxElems / heads) return ECCO_ERR_ARG;
    return (token % per || head % per) ? ECCO_ERR_ALIGN : ECCO_OK;
}

// Whether two rows of a written array share elements: it must be token-major
// or head-major, each level at least as wide as the one inside it.
bool rows_overlap(int64_t tokens, int64_t heads, int64_t token, int64_t head, int64_t width)
{
    if (heads > 1 && head < width) return true;
    if (tokens > 1 && token < width) return true;
    if (tokens <= 1 || heads <= 1) return false;
    return token < (heads - 1) * head + width && head < (tokens - 1) * token + width;
}

}  // namespace

extern "C" int ecco_rope_table(const double* inv_freq, int n_freq, double magnitude, int64_t n_positions, float* table,
                               void* stream)
{
    if (!inv_freq || !table || n_freq < 1 || n_freq > 512 || n_positions < 1 || n_positions > ((int64_t)1 << 30))
        return ECCO_ERR_ARG;
    if (!std::isfinite(magnitude)) return ECCO_ERR_ARG;
    for (int i = 0; i < n_freq; ++i)
        if (!std::isfinite(inv_freq[i])) return ECCO_ERR_ARG;
    if (!aligned(table, 8)) return ECCO_ERR_ALIGN;
    return status(launch_rope_table(inv_freq, n_freq, magnitude, n_positions, table, (cudaStream_t)stream));
}

extern "C" int ecco_rope(const void* x, int64_t x_token, int64_t x_head, void* y, int64_t y_token, int64_t y_head,
                         int dtype, int64_t tokens, int heads, int dim, const float* table, int64_t n_positions,
                         int rotary, const int32_t* positions, int flags, void* stream)
{
    if (dtype != ECCO_BF16 && dtype != ECCO_F16 && dtype != ECCO_F32) return ECCO_ERR_ARG;
    if (tokens < 0 || tokens > 0x7fffffff || heads < 1 || heads > 65535) return ECCO_ERR_ARG;
    if (dim < 8 || dim > 1024 || dim % 8 || rotary < 16 || rotary > dim || rotary % 16) return ECCO_ERR_ARG;
    if (n_positions < 1 || n_positions > ((int64_t)1 << 30)) return ECCO_ERR_ARG;
    if (flags & ~(ECCO_ROPE_INTERLEAVED | ECCO_ROPE_INVERSE)) return ECCO_ERR_ARG;
    if (tokens == 0) return ECCO_OK;
    if (!x || !y || !table || !positions) return ECCO_ERR_ARG;
    const int per = dtype == ECCO_F32 ? 4 : 8;
    int rc = check_strides(tokens, heads, x_token, x_head, per);
    if (rc || (rc = check_strides(tokens, heads, y_token, y_head, per))) return rc;
    if (rows_overlap(tokens, heads, y_token, y_head, dim)) return ECCO_ERR_ARG;
    const bool same = x == y;
    if (same && (x_token != y_token || x_head != y_head)) return ECCO_ERR_ARG;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(table, 16) || !aligned(positions, 4)) return ECCO_ERR_ALIGN;
    const RopeArgs a{x, y, x_token, x_head, y_token, y_head, tokens, n_positions, table, positions, heads, dim, rotary,
                     (flags & ECCO_ROPE_INTERLEAVED) != 0, (flags & ECCO_ROPE_INVERSE) != 0, !same};
    return status(launch_rope(a, dtype, (cudaStream_t)stream));
}

extern "C" int ecco_paged_append(const ecco_tables* kt, const ecco_tables* vt, ecco_paged p, const uint16_t* k,
                                 int64_t k_token, int64_t k_head, const uint16_t* v, int64_t v_token, int64_t v_head,
                                 int64_t tokens, uint8_t* k_pages, uint8_t* v_pages, const float* rope,
                                 int64_t n_positions, int rotary, const int32_t* positions, int flags,
                                 ecco_stats* stats, void* stream)
{
    int rc = check_tables(kt);
    if (rc || (rc = check_tables(vt)) || (rc = check_paged(p, true))) return rc;
    if (tokens < 0 || tokens > 0x7fffffff || tokens * p.kv_heads > ((int64_t)1 << 31)) return ECCO_ERR_ARG;
    if (flags & ~(ECCO_ROPE_INTERLEAVED | ECCO_ROPE_INVERSE)) return ECCO_ERR_ARG;
    if (rope && (rotary < 16 || rotary > kG || rotary % 16 || n_positions < 1 || n_positions > ((int64_t)1 << 30)))
        return ECCO_ERR_ARG;
    if ((rc = check_strides(tokens, p.kv_heads, k_token, k_head, 8)) ||
        (rc = check_strides(tokens, p.kv_heads, v_token, v_head, 8)))
        return rc;
    if (tokens == 0 || p.batch == 0 || p.n_pages == 0 || p.max_pages == 0) return ECCO_OK;
    if (!k || !v || !k_pages || !v_pages || k_pages == v_pages) return ECCO_ERR_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(rope, 16) ||
        !aligned(positions, 4) || !aligned(stats, 8))
        return ECCO_ERR_ALIGN;
    const AppendArgs a{p, {kt->d, vt->d}, {k, v}, {k_token, v_token}, {k_head, v_head}, {k_pages, v_pages}, tokens,
                       rope, n_positions, positions, rotary, (flags & ECCO_ROPE_INTERLEAVED) != 0,
                       (flags & ECCO_ROPE_INVERSE) != 0, stats};
    return status(launch_paged_append(a, (cudaStream_t)stream));
}

namespace {
bool attention_sizes(int batch, int kv_heads, int group, int max_q, int max_kv)
{
    if (batch < 0 || batch > ECCO_MAX_BATCH || kv_heads < 1 || kv_heads > 1024 || group < 1 || group > 16) return false;
    if (max_q < 0 || max_q > (1 << 26) || max_kv < 0 || max_kv > (1 << 30)) return false;
    // 2^24 tiles of a head (a scratch of 1 TiB): the kernels count them in 32 bits
    return (int64_t)batch * ((max_kv + 127) / 128) <= (1 << 24);
}
}  // namespace

extern "C" size_t ecco_paged_attention_workspace_bytes(int batch, int kv_heads, int group, int max_q, int max_kv)
{
    return attention_sizes(batch, kv_heads, group, max_q, max_kv)
               ? paged_attention_bytes(batch, kv_heads, group, max_q, max_kv) : 0;
}

extern "C" int ecco_paged_attention(const ecco_tables* kt, const ecco_tables* vt, ecco_paged p, const uint8_t* k_pages,
                                    const uint8_t* v_pages, const uint16_t* q, int64_t q_token, int64_t q_head,
                                    int group, int64_t tokens, int max_q, int max_kv, int window, float scale,
                                    uint16_t* out, int64_t out_token, int64_t out_head, float* lse, void* ws,
                                    size_t ws_bytes, void* stream)
{
    int rc = check_tables(kt);
    if (rc || (rc = check_tables(vt)) || (rc = check_paged(p, true))) return rc;
    if (!attention_sizes(p.batch, p.kv_heads, group, max_q, max_kv)) return ECCO_ERR_ARG;
    if (window < 0 || !std::isfinite(scale) || tokens < 0 || tokens > 0x7fffffff) return ECCO_ERR_ARG;
    const int64_t heads = (int64_t)p.kv_heads * group;
    if (tokens > kMaxElems / heads) return ECCO_ERR_ARG;
    if ((rc = check_strides(tokens, heads, q_token, q_head, 8)) ||
        (rc = check_strides(tokens, heads, out_token, out_head, 8)))
        return rc;
    if (rows_overlap(tokens, heads, out_token, out_head, kG)) return ECCO_ERR_ARG;
    if (q == out && (q_token != out_token || q_head != out_head)) return ECCO_ERR_ARG;
    if (tokens == 0 || p.batch == 0 || max_q == 0) return ECCO_OK;
    if (!q || !out || !ws || (p.n_pages > 0 && (!k_pages || !v_pages))) return ECCO_ERR_ARG;
    if (ws_bytes < ecco_paged_attention_workspace_bytes(p.batch, p.kv_heads, group, max_q, max_kv)) return ECCO_ERR_ARG;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(ws, 16))
        return ECCO_ERR_ALIGN;
    if (timeout_raised()) return ECCO_ERR_TIMEOUT;  // an earlier tensor-core launch gave up
    const PagedAttnArgs a{p, {kt->d, vt->d}, {k_pages, v_pages}, q, out, lse, q_token, q_head, out_token, out_head,
                          tokens, group, max_q, max_kv, std::min(window, 1 << 30), scale};
    return status(launch_paged_attention(a, ws, (cudaStream_t)stream));
}

extern "C" int ecco_selftest_paged_wait_timeout(void* stream)
{
    return status(launch_paged_wait_selftest((cudaStream_t)stream));
}

extern "C" int ecco_copy_pages(uint8_t* k, uint8_t* v, int64_t n_pages, int64_t page_bytes, const int32_t* src,
                               const int32_t* dst, int64_t n, void* stream)
{
    if (n < 0 || n_pages < 0 || n_pages > 0x7fffffff || page_bytes < 64 || page_bytes % 64) return ECCO_ERR_ARG;
    if (n > n_pages || (n > 0 && page_bytes > kMaxElems * 64 / n_pages)) return ECCO_ERR_ARG;
    if (n == 0) return ECCO_OK;
    if (!k || !v || !src || !dst) return ECCO_ERR_ARG;
    if (!aligned(k, 16) || !aligned(v, 16)) return ECCO_ERR_ALIGN;
    try {
        std::vector<bool> written((size_t)n_pages, false);
        for (int64_t i = 0; i < n; ++i) {
            if (src[i] < 0 || src[i] >= n_pages || dst[i] < 0 || dst[i] >= n_pages || written[dst[i]])
                return ECCO_ERR_ARG;
            written[dst[i]] = true;
        }
        for (int64_t i = 0; i < n; ++i)
            if (written[src[i]]) return ECCO_ERR_ARG;
    } catch (...) {  // no memory for the marks: nothing may leave a C entry
        return ECCO_ERR_ARG;
    }
    return status(launch_copy_pages(k, v, page_bytes, src, dst, n, (cudaStream_t)stream));
}

extern "C" int ecco_compact_pages(ecco_paged p, uint8_t* k_pages, uint8_t* v_pages, const uint8_t* keep,
                                  int64_t keep_stride, const int32_t* dst_table, int64_t dst_stride, int dst_max_pages,
                                  int32_t* new_lens, void* stream)
{
    const int rc = check_paged(p, false);
    if (rc) return rc;
    if (keep_stride < 0 || keep_stride > kMaxElems / ECCO_MAX_BATCH || dst_max_pages < 0 ||
        (int64_t)dst_max_pages * p.page_size > ((int64_t)1 << 30))
        return ECCO_ERR_ARG;
    if (dst_stride < 0 || dst_stride > kMaxElems / ECCO_MAX_BATCH || (p.batch > 1 && dst_stride < dst_max_pages))
        return ECCO_ERR_ARG;
    if (p.batch == 0) return ECCO_OK;
    if (!new_lens || (keep_stride > 0 && !keep) || (dst_max_pages > 0 && !dst_table)) return ECCO_ERR_ARG;
    if (p.n_pages > 0 && (!k_pages || !v_pages)) return ECCO_ERR_ARG;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(dst_table, 4) || !aligned(new_lens, 4))
        return ECCO_ERR_ALIGN;
    // the lengths are read by every CTA of a sequence and written by one of them
    const uintptr_t out = reinterpret_cast<uintptr_t>(new_lens), in = reinterpret_cast<uintptr_t>(p.kv_lens), n = 4u * (uintptr_t)p.batch;
    if (out < in + n && in < out + n) return ECCO_ERR_ARG;
    const CompactArgs a{p, {k_pages, v_pages}, keep, keep_stride, dst_table, dst_stride, dst_max_pages, new_lens};
    return status(launch_compact_pages(a, (cudaStream_t)stream));
}
