// libgdn C-ABI, the calls around the layer: argument validation, status codes and
// dispatch.  Declarations and the contract of every entry point are in
// include/gdn_stack.h.
#include "gdn_stack.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdlib>
#include <new>
#include <vector>

#include "gdn_stack_kernels.h"

namespace {

bool aligned(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }
bool aligned_or_null(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool supported_dtype(int32_t t) { return t == GDN_F32 || t == GDN_BF16; }
int64_t size_of(int32_t dtype) { return dtype == GDN_BF16 ? 2 : 4; }
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
// Offsets that rise from 0 to T, or to at most T, and where they end; log-decays of at most 0.
int32_t check_offsets(const int32_t* cu_seqlens, int32_t num_seqs, int64_t T, bool whole, hipStream_t s, int64_t* end) {
    std::vector<int32_t> cu;
    if (!to_host(cu, cu_seqlens, (int64_t)num_seqs + 1, s)) return GDN_ERR_HIP;
    if (cu.front() != 0 || cu.back() > T || (whole && cu.back() != T)) return GDN_ERR_DOMAIN;
    for (size_t n = 1; n < cu.size(); ++n)
        if (cu[n] < cu[n - 1]) return GDN_ERR_DOMAIN;
    *end = cu.back();
    return GDN_OK;
}
int32_t check_gates(const float* gates, int64_t n, hipStream_t s) {
    std::vector<float> g;
    for (int64_t at = 0; at < n; at += 1 << 24) {
        if (!to_host(g, gates + at, n - at < 1 << 24 ? n - at : 1 << 24, s)) return GDN_ERR_HIP;
        for (const float x : g)
            if (!(x <= 0.f)) return GDN_ERR_DOMAIN;
    }
    return GDN_OK;
}
int32_t validate_scan(const gdn::ScanLaunch& p, hipStream_t s) {
    int64_t end = 0;
    const int32_t st = check_offsets(p.cu_seqlens, p.num_seqs, p.T, false, s, &end);
    return st != GDN_OK ? st : check_gates(p.g, end * p.C, s);  // (rows behind the sequences hold anything)
}
int32_t validate_pool(const gdn::ScanPoolLaunch& p, hipStream_t s) {
    std::vector<int32_t> slots;
    if (!to_host(slots, p.slots, p.num_seqs, s)) return GDN_ERR_HIP;
    std::vector<char> seen((size_t)p.num_slots, 0);
    for (const int32_t x : slots) {
        if (x < 0 || x >= p.num_slots) continue;
        if (seen[(size_t)x]) return GDN_ERR_DOMAIN;
        seen[(size_t)x] = 1;
    }
    int64_t end = p.T;
    const int32_t st = p.cu_seqlens ? check_offsets(p.cu_seqlens, p.num_seqs, p.T, true, s, &end) : GDN_OK;
    return st != GDN_OK ? st : check_gates(p.g, end * p.C, s);
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

int32_t norm_sizes(int64_t T, int32_t H, int32_t H_k, int32_t d) {
    if (T < 0 || T > INT32_MAX || H < 0 || H_k < 0) return GDN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)H + H_k > 1 << 20) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}
// What the forward and the backward call share.
int32_t norm_arguments(const gdn::QkNormLaunch& p, int32_t norm, int32_t dtype) {
    const int32_t st = norm_sizes(p.T, p.heads[0], p.heads[1], p.d);
    if (st != GDN_OK) return st;
    if (!supported_dtype(dtype) || norm < GDN_NORM_NONE || norm > GDN_NORM_RMS) return GDN_ERR_UNSUPPORTED;
    // (below its least normal number the hardware's reciprocal root takes an eps as 0)
    if (!std::isfinite(p.q_scale) || (norm != GDN_NORM_NONE && !(p.eps > 0.f && std::isnormal(p.eps)))) return GDN_ERR_INVALID_ARG;
    if (p.rotary < 0 || p.rotary > p.d || p.rotary % 8 != 0) return GDN_ERR_INVALID_ARG;
    if (p.T > 0 && p.rotary > 0 && (!aligned(p.positions, 4) || !aligned(p.inv_freq, 16))) return GDN_ERR_INVALID_ARG;
    for (int s = 0; s < 2; ++s) {
        if (!aligned_or_null(p.weight[s], 16) || !aligned_or_null(p.d_weight[s], 16)) return GDN_ERR_INVALID_ARG;
        if (p.T == 0 || p.heads[s] == 0) continue;
        if (!aligned(p.x[s], 16) || !aligned(p.out[s], 16)) return GDN_ERR_INVALID_ARG;
        for (const int64_t stride : {p.stride[s], p.out_stride[s]})
            if (stride < (int64_t)p.heads[s] * p.d || stride % (16 / size_of(dtype)) != 0 || stride > INT64_MAX / 16 / (p.T + 1))
                return GDN_ERR_INVALID_ARG;
    }
    return GDN_OK;
}

int32_t scan_sizes(int64_t T, int32_t C) {
    if (T < 0 || T > INT32_MAX || C < 1) return GDN_ERR_INVALID_ARG;
    if (C % 4 != 0) return GDN_ERR_UNSUPPORTED;
    const int64_t tiles = T > 0 ? (T + 63) / 64 : 1;  // (one without a token too: it writes the final states)
    if (tiles * (((int64_t)C + 255) / 256) >= 1 << 23) return GDN_ERR_UNSUPPORTED;  // grids of less than 2^32 threads
    return GDN_OK;
}
int32_t scan_arguments(const gdn::ScanLaunch& p, int32_t dtype) {
    const int32_t st = scan_sizes(p.T, p.C);
    if (st != GDN_OK) return st;
    if (p.num_seqs < 0) return GDN_ERR_INVALID_ARG;
    if (!supported_dtype(dtype)) return GDN_ERR_UNSUPPORTED;
    if (p.T > 0 && p.num_seqs == 0) return GDN_ERR_INVALID_ARG;
    if (p.num_seqs == 0) return GDN_OK;
    if (!aligned(p.cu_seqlens, 4)) return GDN_ERR_INVALID_ARG;
    if (p.T > 0 && (!aligned(p.x, 16) || !aligned(p.g, 16))) return GDN_ERR_INVALID_ARG;
    if (!aligned_or_null(p.initial_state, 16) || !aligned_or_null(p.final_state, 16) || !aligned_or_null(p.checkpoints, 16) ||
        !aligned_or_null(p.d_final_state, 16) || !aligned_or_null(p.d_initial_state, 16))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}
// Whether two arrays [num_seqs, C] share memory.
bool overlap(const float* a, const float* b, int32_t num_seqs, int32_t C) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b), n = (uintptr_t)num_seqs * C * sizeof(float);
    return a && b && x < y + n && y < x + n;
}

}  // namespace

extern "C" {

int32_t gdn_qk_norm(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t T_total, int32_t H,
                    int32_t H_k, int32_t d, int32_t norm, float eps, const float* q_weight, const float* k_weight,
                    const int32_t* positions, const float* inv_freq, int32_t rotary, int32_t interleaved, float q_scale,
                    void* q_out, void* k_out, int32_t dtype, void* stream) {
    gdn::QkNormLaunch p = {};
    p.x[0] = q; p.x[1] = k;
    p.stride[0] = q_stride; p.stride[1] = k_stride;
    p.out_stride[0] = (int64_t)H * d; p.out_stride[1] = (int64_t)H_k * d;
    p.out[0] = q_out; p.out[1] = k_out;
    p.weight[0] = q_weight; p.weight[1] = k_weight;
    p.heads[0] = H; p.heads[1] = H_k;
    p.T = T_total; p.d = d; p.norm = norm; p.eps = eps; p.positions = positions; p.inv_freq = inv_freq;
    p.rotary = rotary; p.interleaved = interleaved != 0; p.q_scale = q_scale; p.bf16 = dtype == GDN_BF16;
    const int32_t st = norm_arguments(p, norm, dtype);
    if (st != GDN_OK) return st;
    return status_of(gdn::launch_qk_norm(p, static_cast<hipStream_t>(stream)));
}

size_t gdn_qk_norm_backward_workspace_bytes(int64_t T_total, int32_t H, int32_t H_k, int32_t d) {
    if (norm_sizes(T_total, H, H_k, d) != GDN_OK) return 0;
    return gdn::qk_norm_backward_workspace_bytes(T_total, H, H_k, d);
}

int32_t gdn_qk_norm_backward(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* d_q_out,
                             const void* d_k_out, int64_t T_total, int32_t H, int32_t H_k, int32_t d, int32_t norm,
                             float eps, const float* q_weight, const float* k_weight, const int32_t* positions,
                             const float* inv_freq, int32_t rotary, int32_t interleaved, float q_scale, void* dq,
                             int64_t dq_stride, void* dk, int64_t dk_stride, float* d_q_weight, float* d_k_weight,
                             int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    gdn::QkNormLaunch p = {};
    p.x[0] = q; p.x[1] = k;
    p.dy[0] = d_q_out; p.dy[1] = d_k_out;
    p.stride[0] = q_stride; p.stride[1] = k_stride;
    p.out_stride[0] = dq_stride; p.out_stride[1] = dk_stride;
    p.out[0] = dq; p.out[1] = dk;
    p.weight[0] = q_weight; p.weight[1] = k_weight;
    p.d_weight[0] = d_q_weight; p.d_weight[1] = d_k_weight;
    p.heads[0] = H; p.heads[1] = H_k;
    p.T = T_total; p.d = d; p.norm = norm; p.eps = eps; p.positions = positions; p.inv_freq = inv_freq;
    p.rotary = rotary; p.interleaved = interleaved != 0; p.q_scale = q_scale; p.bf16 = dtype == GDN_BF16;
    p.workspace = workspace;
    const int32_t st = norm_arguments(p, norm, dtype);
    if (st != GDN_OK) return st;
    for (int s = 0; s < 2; ++s)
        if (T_total > 0 && p.heads[s] > 0 && !aligned(p.dy[s], 16)) return GDN_ERR_INVALID_ARG;
    const size_t need = d_q_weight || d_k_weight ? gdn::qk_norm_backward_workspace_bytes(T_total, H, H_k, d) : 0;
    if (need > 0 && (!aligned(workspace, 16) || workspace_bytes < need)) return GDN_ERR_INVALID_ARG;
    return status_of(gdn::launch_qk_norm_backward(p, static_cast<hipStream_t>(stream)));
}

size_t gdn_scan_checkpoint_bytes(int64_t T_total, int32_t C) {
    return scan_sizes(T_total, C) == GDN_OK ? gdn::scan_checkpoint_bytes(T_total, C) : 0;
}
size_t gdn_scan_workspace_bytes(int64_t T_total, int32_t C) {
    return scan_sizes(T_total, C) == GDN_OK ? gdn::scan_workspace_bytes(T_total, C) : 0;
}
size_t gdn_scan_backward_workspace_bytes(int64_t T_total, int32_t C) {
    return scan_sizes(T_total, C) == GDN_OK ? gdn::scan_backward_workspace_bytes(T_total, C) : 0;
}

int32_t gdn_scan(const void* x, const float* g, const int32_t* cu_seqlens, int32_t num_seqs, int64_t T_total, int32_t C,
                 int32_t mix, const float* initial_state, float* final_state, void* h, float* checkpoints,
                 int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    gdn::ScanLaunch p = {};
    p.x = x; p.g = g; p.cu_seqlens = cu_seqlens; p.num_seqs = num_seqs; p.T = T_total; p.C = C; p.mix = mix != 0;
    p.initial_state = initial_state; p.final_state = final_state; p.h = h; p.checkpoints = checkpoints;
    p.bf16 = dtype == GDN_BF16; p.workspace = workspace;
    const int32_t st = scan_arguments(p, dtype);
    if (st != GDN_OK || num_seqs == 0) return st;
    if (T_total > 0 && !aligned(h, 16)) return GDN_ERR_INVALID_ARG;
    if (overlap(initial_state, final_state, num_seqs, C)) return GDN_ERR_INVALID_ARG;
    const size_t need = gdn::scan_workspace_bytes(T_total, C);
    if (need > 0 && (!aligned(workspace, 16) || workspace_bytes < need)) return GDN_ERR_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (validate_mode()) {
        const int32_t v = validated(validate_scan, p, s);
        if (v != GDN_OK) return v;
    }
    return status_of(gdn::launch_scan(p, s));
}

int32_t gdn_scan_backward(const void* x, const float* g, const int32_t* cu_seqlens, int32_t num_seqs, int64_t T_total,
                          int32_t C, int32_t mix, const float* initial_state, const float* checkpoints,
                          const void* d_h, const float* d_final_state, void* dx, float* dg, float* d_initial_state,
                          int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    gdn::ScanLaunch p = {};
    p.x = x; p.g = g; p.cu_seqlens = cu_seqlens; p.num_seqs = num_seqs; p.T = T_total; p.C = C; p.mix = mix != 0;
    p.initial_state = initial_state; p.checkpoints = const_cast<float*>(checkpoints); p.d_h = d_h;
    p.d_final_state = d_final_state; p.dx = dx; p.dg = dg; p.d_initial_state = d_initial_state;
    p.bf16 = dtype == GDN_BF16; p.workspace = workspace;
    const int32_t st = scan_arguments(p, dtype);
    if (st != GDN_OK || num_seqs == 0) return st;
    if (T_total > 0 && (!aligned(d_h, 16) || !aligned(dx, 16) || !aligned(dg, 16))) return GDN_ERR_INVALID_ARG;
    if (overlap(d_final_state, d_initial_state, num_seqs, C)) return GDN_ERR_INVALID_ARG;
    const size_t need = gdn::scan_backward_workspace_bytes(T_total, C);
    if (need > 0 && (!aligned(workspace, 16) || workspace_bytes < need)) return GDN_ERR_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (validate_mode()) {
        const int32_t v = validated(validate_scan, p, s);
        if (v != GDN_OK) return v;
    }
    return status_of(gdn::launch_scan_backward(p, s));
}

int32_t gdn_scan_pool(const void* x, const float* g, float* states, const int32_t* slots, const int32_t* cu_seqlens,
                      const int32_t* commit, int32_t num_seqs, int64_t T_total, int32_t num_slots, int32_t C,
                      int32_t mix, void* h, int32_t dtype, void* stream) {
    const int32_t st = scan_sizes(T_total, C);
    if (st != GDN_OK) return st;
    if (num_seqs < 0 || num_slots < 0) return GDN_ERR_INVALID_ARG;
    if (!supported_dtype(dtype)) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)num_seqs * ((C + 255) / 256) >= ((int64_t)1 << 24)) return GDN_ERR_UNSUPPORTED;  // one workgroup each
    if (!cu_seqlens && T_total != num_seqs) return GDN_ERR_INVALID_ARG;
    if (T_total > 0 && num_seqs == 0) return GDN_ERR_INVALID_ARG;
    if (T_total == 0 || num_slots == 0) return GDN_OK;
    for (const void* v : {x, static_cast<const void*>(g), static_cast<const void*>(states), static_cast<const void*>(h)})
        if (!aligned(v, 16)) return GDN_ERR_INVALID_ARG;
    if (!aligned(slots, 4) || !aligned_or_null(cu_seqlens, 4) || !aligned_or_null(commit, 4)) return GDN_ERR_INVALID_ARG;
    const gdn::ScanPoolLaunch p = {x, g, states, slots, cu_seqlens, commit, num_seqs, T_total, num_slots, C, mix != 0,
                                   h, dtype == GDN_BF16};
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (validate_mode()) {
        const int32_t v = validated(validate_pool, p, s);
        if (v != GDN_OK) return v;
    }
    return status_of(gdn::launch_scan_pool(p, s));
}

}  // extern "C"
