// The delta rule's recurrent form on a pool of states (gdn_decode_pool): per
// (request, head), with S the request's state and for each of its tokens
//
//     S' = diag(e^g) S,   u = beta (v - S'^T k),   S = S' + k u^T,   o = S^T q
//
// and o formed as S'^T q + (k . q) u, so that one pass over S' gives both sums.
//
// One token does 7 flops for each element of S, which is read and written once
// per call (8 bytes): the call is bound by HBM up to about ten tokens.
// A wave owns all d_k rows of kCols value columns of one (request, head), since
// the columns of S evolve independently: a lane holds 4 neighbouring columns
// (16 bytes) of d_k / kRowGroups neighbouring rows in registers for all the
// tokens, and the sums over rows end in exchanges between the lanes of the wave.
// Tokens therefore need no barrier and no LDS.  The state is touched once: it
// is read and written with non-temporal hints.
//
// Measured: 512 requests of 32 heads of 128 x 128, one token, 2.17 GB, 380 to 396
// us, 5.5 to 5.7 TB/s (gdn_decode's kernel, which reads whole rows and takes no
// slots, 361 us for the same states, 6.0; a large in-place multiplication: 5.9);
// with 16 columns to a wave, half a line of each row, 628.  One request, 4.2 MB, 4.4 us, of which a
// launch is 3.5.  45 requests of 1 to 7 tokens, 12 heads of 64 x 128, fp32, 37.5
// MB, 13 us: two workgroups for each compute unit, and each token's sums wait for
// the token before.  A request of one token needs 128 registers, of more, with the
// next token's vectors on their way, more: a kernel for each.
#include "gdn_device.h"
#include "gdn_lanes.h"
#include "gdn_serve_kernels.h"

namespace gdn {
namespace {

constexpr int kCols = 32;                   // value columns of a wave
constexpr int kColLanes = kCols / 4;        // lanes side by side along a row
constexpr int kRowGroups = 64 / kColLanes;  // lanes along the rows

struct Pool {
    const void *q, *k, *v;
    const float *g, *beta;
    float* states;
    const int32_t *slots, *cu, *commit;
    int64_t T;
    int32_t num_slots, H, Hk;
    float q_scale, eps;
    void* o;
};

template <typename T, int N>
__device__ __forceinline__ void load_row(const T* p, T* x) {
    constexpr int V = (int)(16 / sizeof(T)) < N ? (int)(16 / sizeof(T)) : N;  // a load of 16 bytes, or all of N
    typedef T vec __attribute__((ext_vector_type(V)));
#pragma unroll
    for (int j = 0; j < N; j += V) {
        const vec y = *reinterpret_cast<const vec*>(p + j);
#pragma unroll
        for (int i = 0; i < V; ++i) x[j + i] = y[i];
    }
}

__device__ __forceinline__ float rows_sum(float x) { return across<Sum, kColLanes>(x); }
__device__ __forceinline__ floatx4 rows_sum(floatx4 x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = rows_sum(x[i]);
    return x;
}

// A token's vectors, as a lane needs them.
template <typename TI, int NR, bool HEAD>
struct Token {
    TI k[NR], q[NR], v[4];
    float g[HEAD ? 1 : NR], beta;
    __device__ __forceinline__ void load(const Pool& a, int64_t t, int32_t h, int32_t hk, int row, int dk, int col, int dv) {
        const int64_t th = t * a.H + h, tk = (t * a.Hk + hk) * dk + row;
        load_row<TI, NR>(static_cast<const TI*>(a.k) + tk, k);
        load_row<TI, NR>(static_cast<const TI*>(a.q) + tk, q);
        if constexpr (HEAD) g[0] = a.g[th];
        else load_row<float, NR>(a.g + th * dk + row, g);
        load_row<TI, 4>(static_cast<const TI*>(a.v) + th * dv + col, v);
        beta = a.beta[th];
    }
};

// MANY: a request may have more than one token.
template <typename TI, int DK, int DV, bool HEAD, bool MANY>
__global__ __launch_bounds__(DV / kCols * 64, MANY ? 2 : 4) void pool_kernel(Pool a) {
    constexpr int NR = DK / kRowGroups;  // rows of a lane
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = blockIdx.x / a.H;
    const int32_t h = (int32_t)(blockIdx.x - n * a.H), hk = h / (a.H / a.Hk);
    const int32_t slot = a.slots[n];
    if (slot < 0 || slot >= a.num_slots) return;
    int64_t t0 = n, t1 = n + 1;
    if (MANY) {
        t0 = a.cu[n]; t1 = a.cu[n + 1];
        if (t0 < 0) t0 = 0;
        if (t1 > a.T) t1 = a.T;
    }
    if (t1 <= t0) return;
    int64_t keep = t1 - t0;
    if (a.commit && a.commit[n] < keep) keep = a.commit[n];

    const int rg = lane / kColLanes, col = wave * kCols + 4 * (lane % kColLanes);
    const int row = rg * NR;
    float* S = a.states + (((int64_t)slot * a.H + h) * DK + row) * DV + col;
    Token<TI, NR, HEAD> next;
    next.load(a, t0, h, hk, row, DK, col, DV);
    floatx4 s[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j) s[j] = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(S + j * DV));
    for (int64_t t = t0; t < t1; ++t) {
        const Token<TI, NR, HEAD> x = next;
        // the next token's vectors are on their way while this one is worked on
        if (MANY && t + 1 < t1) next.load(a, t + 1, h, hk, row, DK, col, DV);
        float k[NR], q[NR];
        floatx4 v, r = {0.f, 0.f, 0.f, 0.f}, p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = to_f32(x.v[j]);
        const float head_decay = __expf(x.g[0]);  // with one gate per head
        float kq = 0.f, kk = 0.f, qq = 0.f;
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            k[j] = to_f32(x.k[j]);
            q[j] = to_f32(x.q[j]);
            s[j] *= HEAD ? head_decay : __expf(x.g[HEAD ? 0 : j]);
            r += s[j] * k[j];
            p += s[j] * q[j];
            kq += k[j] * q[j];
        }
        r = rows_sum(r);
        p = rows_sum(p);
        kq = rows_sum(kq);
        // With the norm, k and q stand for their unit vectors: every sum is
        // linear in them, so their factors are applied to the sums.
        float ck = 1.f, cq = a.q_scale;
        if (a.eps > 0.f) {
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                kk += k[j] * k[j];
                qq += q[j] * q[j];
            }
            ck = __builtin_amdgcn_rsqf(rows_sum(kk) + a.eps);  // good to one step of fp32
            cq *= __builtin_amdgcn_rsqf(rows_sum(qq) + a.eps);
        }
        const floatx4 u = x.beta * (v - ck * r);
        const floatx4 out = cq * (p + (ck * kq) * u);
        const floatx4 w = ck * u;
#pragma unroll
        for (int j = 0; j < NR; ++j) s[j] += w * k[j];
        if (rg == 0) {
            TI* o = static_cast<TI*>(a.o) + (t * a.H + h) * DV + col;
            if constexpr (sizeof(TI) == 4) *reinterpret_cast<floatx4*>(o) = out;
            else *reinterpret_cast<bf16x4*>(o) = bf16x4{(bf16)out[0], (bf16)out[1], (bf16)out[2], (bf16)out[3]};
        }
        if (t - t0 + 1 == keep)
#pragma unroll
            for (int j = 0; j < NR; ++j) __builtin_nontemporal_store(s[j], reinterpret_cast<floatx4*>(S + j * DV));
    }
}

template <typename TI, int DK, int DV>
hipError_t run(const Pool& a, bool head, unsigned units, hipStream_t s) {
    const dim3 grid(units), block(DV / kCols * 64);
    if (head && a.cu) hipLaunchKernelGGL((pool_kernel<TI, DK, DV, true, true>), grid, block, 0, s, a);
    else if (head) hipLaunchKernelGGL((pool_kernel<TI, DK, DV, true, false>), grid, block, 0, s, a);
    else if (a.cu) hipLaunchKernelGGL((pool_kernel<TI, DK, DV, false, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((pool_kernel<TI, DK, DV, false, false>), grid, block, 0, s, a);
    return hipGetLastError();
}
template <typename TI>
hipError_t run_t(const Pool& a, int32_t dk, int32_t dv, bool head, unsigned units, hipStream_t s) {
    if (dk == 128 && dv == 128) return run<TI, 128, 128>(a, head, units, s);
    if (dk == 128) return run<TI, 128, 64>(a, head, units, s);
    if (dv == 128) return run<TI, 64, 128>(a, head, units, s);
    return run<TI, 64, 64>(a, head, units, s);
}

}  // namespace

hipError_t launch_decode_pool(const DecodePoolLaunch& p, hipStream_t s) {
    const unsigned units = (unsigned)((int64_t)p.num_seqs * p.H);
    if (units == 0 || p.T_total == 0) return hipSuccess;
    const Pool a = {p.q, p.k, p.v, p.g, p.beta, p.states, p.slots, p.cu_seqlens, p.commit, p.T_total,
                    p.num_slots, p.H, p.H_k, p.q_scale, p.l2_eps, p.o};
    return p.bf16 ? run_t<bf16>(a, p.dk, p.dv, p.head_gate, units, s) : run_t<float>(a, p.dk, p.dv, p.head_gate, units, s);
}

}  // namespace gdn
