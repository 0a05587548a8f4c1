// Host-side launchers of the serving kernels (include/gdn_serve.h).  Sizes and
// alignment are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

struct TablesLaunch {
    const int32_t *context_lens, *new_lens, *rows;
    int32_t num_seqs;
    int64_t T_total;
    int32_t page_size;
    int32_t* block_table;
    int32_t num_rows, max_blocks;
    int32_t *page_counts, *free_pages;
    int32_t num_pages;
    int32_t *free_state, *cu_seqlens, *kv_lens, *slots, *positions;
    void* workspace;
};
// One request as the fill step needs it.
struct TablesRequest {
    int32_t row;     // -1: refused, no slots
    int32_t ctx;     // tokens held
    int32_t base;    // first block that this call gives a page to
    int32_t ring;    // ring place of that page; for an ended request: of its first returned page
    int32_t given;   // pages of an ended request, 0 for the others
};
size_t tables_workspace_bytes(int32_t num_seqs, int64_t T_total);
hipError_t launch_tables(const TablesLaunch& p, hipStream_t stream);

struct CacheWriteLaunch {
    const void *k, *v;
    const int32_t* slots;
    int64_t T_total;
    uint8_t *k_cache, *v_cache;
    float *k_scale, *v_scale;
    int64_t num_pages;
    int32_t page_size, H_kv, dk, dv;
    bool bf16;
};
hipError_t launch_cache_write(const CacheWriteLaunch& p, hipStream_t stream);

struct CacheAttentionLaunch {
    const void* q;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t *block_table, *rows, *kv_lens, *cu_seqlens;
    int32_t num_seqs;
    int64_t T_total, max_new, max_kv, num_pages;
    int32_t page_size, num_rows, max_blocks;
    float scale;
    void* o;
    int32_t H, H_kv, dk, dv;
    bool bf16;
    void* workspace;
};
size_t cache_attention_workspace_bytes(const CacheAttentionLaunch& p);
hipError_t launch_cache_attention(const CacheAttentionLaunch& p, hipStream_t stream);

struct DecodePoolLaunch {
    const void *q, *k, *v;
    const float* g;
    bool head_gate;
    const float* beta;
    float* states;
    const int32_t *slots, *cu_seqlens, *commit;
    int32_t num_seqs;
    int64_t T_total;
    int32_t num_slots;
    float q_scale, l2_eps;
    void* o;
    int32_t H, H_k, dk, dv;
    bool bf16;
};
hipError_t launch_decode_pool(const DecodePoolLaunch& p, hipStream_t stream);

}  // namespace gdn
