// libgdn C-ABI, serving side: argument validation, status codes and dispatch.
// Declarations and the contract of every entry point are in include/gdn_serve.h, and
// of the attention behind a common beginning in include/gdn_stack.h.
#include "gdn_serve.h"
#include "gdn_stack.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <new>
#include <vector>

#include "gdn_serve_kernels.h"

namespace {

bool aligned(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }
bool aligned_or_null(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool supported_d(int32_t d) { return d == 64 || d == 128; }
bool supported_page(int32_t p) { return p == 64 || p == 128 || p == 256; }
bool supported_dtype(int32_t t) { return t == GDN_F32 || t == GDN_BF16; }
bool validate_mode() {
    const char* e = std::getenv("GDN_VALIDATE");
    return e && e[0] == '1';
}
int32_t status_of(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_HIP; }

template <typename T>
bool to_host(std::vector<T>& to, const T* from, int64_t n, hipStream_t s) {
    to.resize((size_t)n);
    return n == 0 || (hipMemcpyAsync(to.data(), from, sizeof(T) * (size_t)n, hipMemcpyDeviceToHost, s) == hipSuccess &&
                      hipStreamSynchronize(s) == hipSuccess);
}
// Whether a value >= 0 repeats, or one is at or above `below`.
bool repeats(const std::vector<int32_t>& v, int64_t below, bool negative_is_fine) {
    std::vector<char> seen((size_t)below, 0);
    for (const int32_t x : v) {
        if (x < 0 && negative_is_fine) continue;
        if (x < 0 || x >= below) {
            if (negative_is_fine) continue;
            return true;
        }
        if (seen[(size_t)x]) return true;
        seen[(size_t)x] = 1;
    }
    return false;
}

int32_t validate_tables(const gdn::TablesLaunch& p, hipStream_t s) {
    std::vector<int32_t> ctx, added, rows, counts, state;
    if (!to_host(ctx, p.context_lens, p.num_seqs, s) || !to_host(added, p.new_lens, p.num_seqs, s) ||
        !to_host(state, p.free_state, 3, s) || !to_host(counts, p.page_counts, p.num_rows, s))
        return GDN_ERR_HIP;
    int64_t tokens = 0;
    for (const int32_t x : added) tokens += x > 0 ? x : 0;
    if (tokens > p.T_total) return GDN_ERR_DOMAIN;
    if (p.rows) {
        if (!to_host(rows, p.rows, p.num_seqs, s)) return GDN_ERR_HIP;
        if (repeats(rows, p.num_rows, false)) return GDN_ERR_DOMAIN;
    } else if (p.num_seqs > p.num_rows) {
        return GDN_ERR_DOMAIN;
    }
    for (const int32_t c : ctx)
        if (c < 0) return GDN_ERR_DOMAIN;
    for (const int32_t c : counts)
        if (c < 0 || c > p.max_blocks) return GDN_ERR_DOMAIN;
    if (state[0] < 0 || (state[0] >= p.num_pages && p.num_pages > 0) || state[1] < 0 || state[1] > p.num_pages)
        return GDN_ERR_DOMAIN;
    return GDN_OK;
}

int32_t validate_slots(const gdn::CacheWriteLaunch& p, hipStream_t s) {
    std::vector<int32_t> slots;
    if (!to_host(slots, p.slots, p.T_total, s)) return GDN_ERR_HIP;
    std::vector<char> seen((size_t)p.num_pages, 0);
    for (size_t t = 0; t < slots.size(); ++t) {
        const int64_t x = slots[t];
        if (x < 0 || x >= p.num_pages * p.page_size) continue;
        if (t > 0 && slots[t - 1] == x - 1 && x % p.page_size != 0) continue;
        if (seen[(size_t)(x / p.page_size)]) return GDN_ERR_DOMAIN;
        seen[(size_t)(x / p.page_size)] = 1;
    }
    return GDN_OK;
}

int32_t validate_attention(const gdn::CacheAttentionLaunch& p, hipStream_t s) {
    std::vector<int32_t> cu, kv, rows, table;
    if (!to_host(cu, p.cu_seqlens, (int64_t)p.num_seqs + 1, s) || !to_host(kv, p.kv_lens, p.num_seqs, s)) return GDN_ERR_HIP;
    if (cu.front() != 0 || cu.back() > p.T_total) return GDN_ERR_DOMAIN;
    for (size_t n = 1; n < cu.size(); ++n)
        if (cu[n] < cu[n - 1]) return GDN_ERR_DOMAIN;
    for (const int32_t x : kv)
        if (x < 0 || x > (int64_t)p.max_blocks * p.page_size) return GDN_ERR_DOMAIN;
    if (p.rows && !to_host(rows, p.rows, p.num_seqs, s)) return GDN_ERR_HIP;
    if (p.num_pages == 0) return GDN_OK;
    std::vector<float> scale[2];
    if (!to_host(table, p.block_table, (int64_t)p.num_rows * p.max_blocks, s) ||
        !to_host(scale[0], p.k_scale, p.num_pages * p.H_kv, s) || !to_host(scale[1], p.v_scale, p.num_pages * p.H_kv, s))
        return GDN_ERR_HIP;
    for (int32_t n = 0; n < p.num_seqs; ++n) {
        const int64_t row = p.rows ? rows[(size_t)n] : n;
        if (row < 0 || row >= p.num_rows) continue;
        for (int64_t b = 0; b * p.page_size < kv[(size_t)n]; ++b) {
            const int64_t page = table[(size_t)(row * p.max_blocks + b)];
            if (page < 0 || page >= p.num_pages) continue;
            int e;
            for (const auto& x : scale)
                for (int32_t h = 0; h < p.H_kv; ++h) {
                    const float f = x[(size_t)(page * p.H_kv + h)];
                    if (!(f > 0.f) || std::isinf(f) || std::frexp(f, &e) != 0.5f) return GDN_ERR_DOMAIN;
                }
        }
    }
    return GDN_OK;
}

int32_t validate_pool(const gdn::DecodePoolLaunch& p, hipStream_t s) {
    std::vector<int32_t> slots, cu;
    std::vector<float> g;
    if (!to_host(slots, p.slots, p.num_seqs, s)) return GDN_ERR_HIP;
    if (repeats(slots, p.num_slots, true)) return GDN_ERR_DOMAIN;
    if (p.cu_seqlens) {
        if (!to_host(cu, p.cu_seqlens, (int64_t)p.num_seqs + 1, s)) return GDN_ERR_HIP;
        if (cu.front() != 0 || cu.back() != p.T_total) return GDN_ERR_DOMAIN;
        for (size_t n = 1; n < cu.size(); ++n)
            if (cu[n] < cu[n - 1]) return GDN_ERR_DOMAIN;
    }
    if (!to_host(g, p.g, p.T_total * p.H * (p.head_gate ? 1 : p.dk), s)) return GDN_ERR_HIP;
    for (const float x : g)
        if (!(x <= 0.f)) return GDN_ERR_DOMAIN;
    return GDN_OK;
}

// The host checks allocate: no exception leaves a C entry point.
template <typename P>
int32_t validated(int32_t (*check)(const P&, hipStream_t), const P& p, hipStream_t s) {
    try {
        return check(p, s);
    } catch (const std::bad_alloc&) {
        return GDN_ERR_OOM;
    } catch (...) {
        return GDN_ERR_INVALID_ARG;
    }
}

int32_t attention_sizes(const gdn::CacheAttentionLaunch& p) {
    if (p.num_seqs < 0 || p.T_total < 0 || p.T_total > INT32_MAX || p.max_new < 0 || p.max_kv < 0 || p.max_blocks < 0)
        return GDN_ERR_INVALID_ARG;
    if (p.H < 1 || p.H_kv < 1 || p.H % p.H_kv != 0 || p.H_kv > 65535) return GDN_ERR_INVALID_ARG;
    if (!supported_d(p.dk) || !supported_d(p.dv) || !supported_page(p.page_size)) return GDN_ERR_UNSUPPORTED;
    if (p.T_total > 0 && p.num_seqs == 0) return GDN_ERR_INVALID_ARG;
    // grids of less than 2^24 workgroups
    if (p.T_total * p.H > ((int64_t)1 << 27) || (int64_t)p.num_seqs * p.H_kv > ((int64_t)1 << 18)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// Arguments of an attention call besides its workspace; GDN_OK and T_total 0: nothing to do.
int32_t attention_arguments(const gdn::CacheAttentionLaunch& p, int32_t dtype) {
    const int32_t st = attention_sizes(p);
    if (st != GDN_OK) return st;
    if (!supported_dtype(dtype)) return GDN_ERR_UNSUPPORTED;
    if (p.num_rows < 0 || p.num_pages < 0 || p.num_pages > INT32_MAX || !std::isfinite(p.scale)) return GDN_ERR_INVALID_ARG;
    if (p.T_total == 0) return GDN_OK;
    if (!aligned(p.q, 16) || !aligned(p.o, 16)) return GDN_ERR_INVALID_ARG;
    if (!aligned(p.kv_lens, 4) || !aligned(p.cu_seqlens, 4) || !aligned_or_null(p.rows, 4)) return GDN_ERR_INVALID_ARG;
    if (p.num_rows > 0 && p.max_blocks > 0 && !aligned(p.block_table, 4)) return GDN_ERR_INVALID_ARG;
    if (p.num_pages > 0 &&
        (!aligned(p.k_cache, 16) || !aligned(p.v_cache, 16) || !aligned(p.k_scale, 4) || !aligned(p.v_scale, 4)))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}
int32_t prefix_sizes(const gdn::CachePrefixLaunch& p) {
    const int32_t st = attention_sizes(p.all);
    return st != GDN_OK ? st : p.num_groups < 0 || p.max_prefix < 0 ? GDN_ERR_INVALID_ARG : GDN_OK;
}
int32_t validate_prefix(const gdn::CachePrefixLaunch& p, hipStream_t s) {
    const int32_t st = validate_attention(p.all, s);
    if (st != GDN_OK) return st;
    std::vector<int32_t> offsets, shared, rows, kv, cu, table;
    if (!to_host(offsets, p.group_offsets, (int64_t)p.num_groups + 1, s) || !to_host(shared, p.prefix_lens, p.num_groups, s) ||
        !to_host(kv, p.all.kv_lens, p.all.num_seqs, s) || !to_host(cu, p.all.cu_seqlens, (int64_t)p.all.num_seqs + 1, s) ||
        !to_host(table, p.all.block_table, (int64_t)p.all.num_rows * p.all.max_blocks, s) ||
        (p.all.rows && !to_host(rows, p.all.rows, p.all.num_seqs, s)))
        return GDN_ERR_HIP;
    if (offsets.front() != 0) return GDN_ERR_DOMAIN;
    for (int32_t g = 0; g < p.num_groups; ++g) {
        if (offsets[(size_t)g + 1] < offsets[(size_t)g] || offsets[(size_t)g + 1] > p.all.num_seqs || shared[(size_t)g] < 0)
            return GDN_ERR_DOMAIN;
        const int64_t blocks = std::min<int64_t>(shared[(size_t)g] / p.all.page_size, p.all.max_blocks);
        const int32_t* first = nullptr;
        for (int32_t n = offsets[(size_t)g]; n < offsets[(size_t)g + 1]; ++n) {
            const int64_t row = p.all.rows ? rows[(size_t)n] : n, len = cu[(size_t)n + 1] - cu[(size_t)n];
            if (row < 0 || row >= p.all.num_rows || len == 0 || kv[(size_t)n] - len < blocks * p.all.page_size) continue;
            const int32_t* const at = table.data() + row * p.all.max_blocks;
            if (first && !std::equal(first, first + blocks, at)) return GDN_ERR_DOMAIN;
            if (!first) first = at;
        }
    }
    return GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_batch_tables_workspace_bytes(int32_t num_seqs, int64_t T_total) {
    if (num_seqs < 0 || T_total < 0) return 0;
    return gdn::tables_workspace_bytes(num_seqs, T_total);
}

int32_t gdn_batch_tables(const int32_t* context_lens, const int32_t* new_lens, const int32_t* rows, int32_t num_seqs,
                         int64_t T_total, int32_t page_size, int32_t* block_table, int32_t num_rows,
                         int32_t max_blocks, int32_t* page_counts, int32_t* free_pages, int32_t num_pages,
                         int32_t* free_state, int32_t* cu_seqlens, int32_t* kv_lens, int32_t* slots,
                         int32_t* positions, void* workspace, size_t workspace_bytes, void* stream) {
    if (num_seqs < 0 || T_total < 0 || T_total > INT32_MAX || num_rows < 0 || max_blocks < 0 || num_pages < 0)
        return GDN_ERR_INVALID_ARG;
    if (!supported_page(page_size)) return GDN_ERR_UNSUPPORTED;
    if (!aligned(free_state, 4) || !aligned(cu_seqlens, 4)) return GDN_ERR_INVALID_ARG;
    if (T_total > 0 && (!aligned(slots, 4) || !aligned(positions, 4))) return GDN_ERR_INVALID_ARG;
    if (num_seqs > 0) {
        if (!aligned(context_lens, 4) || !aligned(new_lens, 4) || !aligned(kv_lens, 4) || !aligned_or_null(rows, 4))
            return GDN_ERR_INVALID_ARG;
        if (num_rows > 0 && !aligned(page_counts, 4)) return GDN_ERR_INVALID_ARG;
        if (num_rows > 0 && max_blocks > 0 && !aligned(block_table, 4)) return GDN_ERR_INVALID_ARG;
        if (num_pages > 0 && !aligned(free_pages, 4)) return GDN_ERR_INVALID_ARG;
        if (!aligned(workspace, 4) || workspace_bytes < gdn::tables_workspace_bytes(num_seqs, T_total))
            return GDN_ERR_INVALID_ARG;
    }
    const gdn::TablesLaunch p = {context_lens, new_lens, rows, num_seqs, T_total, page_size, block_table, num_rows,
                                 max_blocks, page_counts, free_pages, num_pages, free_state, cu_seqlens, kv_lens,
                                 slots, positions, workspace};
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (validate_mode() && num_seqs > 0) {
        const int32_t st = validated(validate_tables, p, s);
        if (st != GDN_OK) return st;
    }
    return status_of(gdn::launch_tables(p, s));
}

int32_t gdn_cache_write(const void* k, const void* v, const int32_t* slots, int64_t T_total, void* k_cache,
                        void* v_cache, float* k_scale, float* v_scale, int64_t num_pages, int32_t page_size,
                        int32_t H_kv, int32_t d_k, int32_t d_v, int32_t dtype, void* stream) {
    if (T_total < 0 || T_total > INT32_MAX || num_pages < 0 || H_kv < 1 || H_kv > 8191) return GDN_ERR_INVALID_ARG;
    if (!supported_dtype(dtype) || !supported_d(d_k) || !supported_d(d_v) || !supported_page(page_size))
        return GDN_ERR_UNSUPPORTED;
    if (num_pages > ((int64_t)INT32_MAX + 1) / page_size) return GDN_ERR_UNSUPPORTED;  // slots are int32
    if (T_total * H_kv > ((int64_t)1 << 28)) return GDN_ERR_UNSUPPORTED;  // a grid of less than 2^24 workgroups
    if (T_total == 0 || num_pages == 0) return GDN_OK;
    for (const void* x : {k, v, static_cast<const void*>(k_cache), static_cast<const void*>(v_cache)})
        if (!aligned(x, 16)) return GDN_ERR_INVALID_ARG;
    if (!aligned(slots, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4)) return GDN_ERR_INVALID_ARG;
    const gdn::CacheWriteLaunch p = {k, v, slots, T_total, static_cast<uint8_t*>(k_cache),
                                     static_cast<uint8_t*>(v_cache), k_scale, v_scale, num_pages, page_size,
                                     H_kv, d_k, d_v, dtype == GDN_BF16};
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (validate_mode()) {
        const int32_t st = validated(validate_slots, p, s);
        if (st != GDN_OK) return st;
    }
    return status_of(gdn::launch_cache_write(p, s));
}

size_t gdn_cache_attention_workspace_bytes(int32_t num_seqs, int64_t T_total, int64_t max_new, int64_t max_kv,
                                           int32_t page_size, int32_t max_blocks, int32_t H, int32_t H_kv,
                                           int32_t d_k, int32_t d_v) {
    gdn::CacheAttentionLaunch p = {};
    p.num_seqs = num_seqs; p.T_total = T_total; p.max_new = max_new; p.max_kv = max_kv;
    p.page_size = page_size; p.max_blocks = max_blocks; p.H = H; p.H_kv = H_kv; p.dk = d_k; p.dv = d_v;
    if (attention_sizes(p) != GDN_OK || T_total == 0) return 0;
    return gdn::cache_attention_workspace_bytes(p);
}

int32_t gdn_cache_attention(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                            const float* v_scale, const int32_t* block_table, const int32_t* rows,
                            const int32_t* kv_lens, const int32_t* cu_seqlens, int32_t num_seqs, int64_t T_total,
                            int64_t max_new, int64_t max_kv, int64_t num_pages, int32_t page_size, int32_t num_rows,
                            int32_t max_blocks, float scale, void* o, int32_t H, int32_t H_kv, int32_t d_k,
                            int32_t d_v, int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const gdn::CacheAttentionLaunch p = {q, static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache),
                                         k_scale, v_scale, block_table, rows, kv_lens, cu_seqlens, num_seqs, T_total,
                                         max_new, max_kv, num_pages, page_size, num_rows, max_blocks, scale, o, H,
                                         H_kv, d_k, d_v, dtype == GDN_BF16, workspace};
    const int32_t st = attention_arguments(p, dtype);
    if (st != GDN_OK || T_total == 0) return st;
    const size_t need = gdn::cache_attention_workspace_bytes(p);
    if (need > 0 && (!aligned(workspace, 16) || workspace_bytes < need)) return GDN_ERR_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (validate_mode()) {
        const int32_t v = validated(validate_attention, p, s);
        if (v != GDN_OK) return v;
    }
    return status_of(gdn::launch_cache_attention(p, s));
}

size_t gdn_cache_attention_prefix_workspace_bytes(int32_t num_seqs, int32_t num_groups, int64_t T_total,
                                                  int64_t max_new, int64_t max_kv, int64_t max_prefix,
                                                  int32_t page_size, int32_t max_blocks, int32_t H, int32_t H_kv,
                                                  int32_t d_k, int32_t d_v) {
    gdn::CachePrefixLaunch p = {};
    p.all.num_seqs = num_seqs; p.all.T_total = T_total; p.all.max_new = max_new; p.all.max_kv = max_kv;
    p.all.page_size = page_size; p.all.max_blocks = max_blocks; p.all.H = H; p.all.H_kv = H_kv; p.all.dk = d_k; p.all.dv = d_v;
    p.num_groups = num_groups; p.max_prefix = max_prefix;
    if (prefix_sizes(p) != GDN_OK || T_total == 0) return 0;
    return gdn::cache_prefix_workspace_bytes(p);
}

int32_t gdn_cache_attention_prefix(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                   const float* v_scale, const int32_t* block_table, const int32_t* rows,
                                   const int32_t* kv_lens, const int32_t* cu_seqlens, const int32_t* group_offsets,
                                   const int32_t* prefix_lens, int32_t num_seqs, int32_t num_groups, int64_t T_total,
                                   int64_t max_new, int64_t max_kv, int64_t max_prefix, int64_t num_pages,
                                   int32_t page_size, int32_t num_rows, int32_t max_blocks, float scale, void* o,
                                   int32_t H, int32_t H_kv, int32_t d_k, int32_t d_v, int32_t dtype, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    const gdn::CachePrefixLaunch p = {{q, static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache),
                                       k_scale, v_scale, block_table, rows, kv_lens, cu_seqlens, num_seqs, T_total,
                                       max_new, max_kv, num_pages, page_size, num_rows, max_blocks, scale, o, H, H_kv,
                                       d_k, d_v, dtype == GDN_BF16, workspace},
                                      group_offsets, prefix_lens, num_groups, max_prefix};
    int32_t st = prefix_sizes(p);
    if (st == GDN_OK) st = attention_arguments(p.all, dtype);
    if (st != GDN_OK || T_total == 0) return st;
    if (num_groups > 0 && (!aligned(group_offsets, 4) || !aligned(prefix_lens, 4))) return GDN_ERR_INVALID_ARG;
    const size_t need = gdn::cache_prefix_workspace_bytes(p);
    if (need > 0 && (!aligned(workspace, 16) || workspace_bytes < need)) return GDN_ERR_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (validate_mode()) {
        const int32_t v = num_groups > 0 ? validated(validate_prefix, p, s) : validated(validate_attention, p.all, s);
        if (v != GDN_OK) return v;
    }
    return status_of(gdn::launch_cache_prefix(p, s));
}

int32_t gdn_decode_pool(const void* q, const void* k, const void* v, const float* g, int32_t head_gate,
                        const float* beta, float* states, const int32_t* slots, const int32_t* cu_seqlens,
                        const int32_t* commit, int32_t num_seqs, int64_t T_total, int32_t num_slots, float q_scale,
                        float l2_eps, void* o, int32_t H, int32_t H_k, int32_t d_k, int32_t d_v, int32_t dtype,
                        void* stream) {
    if (num_seqs < 0 || T_total < 0 || T_total > INT32_MAX || num_slots < 0) return GDN_ERR_INVALID_ARG;
    if (H < 1 || H_k < 1 || H % H_k != 0) return GDN_ERR_INVALID_ARG;
    if (!supported_dtype(dtype) || !supported_d(d_k) || !supported_d(d_v)) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)num_seqs * H >= ((int64_t)1 << 24)) return GDN_ERR_UNSUPPORTED;  // one workgroup each
    if (!std::isfinite(q_scale) || !std::isfinite(l2_eps) || l2_eps < 0.f) return GDN_ERR_INVALID_ARG;
    if (!cu_seqlens && T_total != num_seqs) return GDN_ERR_INVALID_ARG;
    if (T_total > 0 && num_seqs == 0) return GDN_ERR_INVALID_ARG;
    if (T_total == 0 || num_slots == 0) return GDN_OK;
    for (const void* x : {q, k, v, static_cast<const void*>(states), static_cast<const void*>(o)})
        if (!aligned(x, 16)) return GDN_ERR_INVALID_ARG;
    if (!aligned(g, head_gate ? 4 : 16) || !aligned(beta, 4) || !aligned(slots, 4) || !aligned_or_null(cu_seqlens, 4) ||
        !aligned_or_null(commit, 4))
        return GDN_ERR_INVALID_ARG;
    const gdn::DecodePoolLaunch p = {q, k, v, g, head_gate != 0, beta, states, slots, cu_seqlens, commit, num_seqs,
                                     T_total, num_slots, q_scale, l2_eps, o, H, H_k, d_k, d_v, dtype == GDN_BF16};
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (validate_mode()) {
        const int32_t st = validated(validate_pool, p, s);
        if (st != GDN_OK) return st;
    }
    return status_of(gdn::launch_decode_pool(p, s));
}

}  // extern "C"
