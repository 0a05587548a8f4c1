// New keys and values into the paged e4m3 cache (gdn_cache_write).
//
// The tokens of a call in one page share a scale, so the unit of work is a run:
// the call's tokens in one page, for one head, of the keys or of the values.  Its
// largest magnitude gives the scale, then its values are rounded; the values'
// 16-token groups are transposed on the way.  Each run belongs to one
// workgroup, so a page needs no atomics.  A workgroup looks at the runs that
// start in a tile of tokens: of few tokens where there are few (each token of a
// decode step is a run), of more where there are many (a prompt's runs are
// whole pages), which keeps the grid near the same size.
//
// Three operations per element: bound by the bytes read (2 or 4 for each) and
// written (1).
#include "gdn_e4m3.h"
#include "gdn_serve_kernels.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

struct Write {
    const void *k, *v;
    const int32_t* slots;
    int64_t T;
    uint8_t *kc, *vc;
    float *ks, *vs;
    int64_t places;  // num_pages * page_size
    int32_t page, H, dk, dv, tile;
};

struct Run {
    int64_t t;     // first token
    int64_t page;
    int a, b;      // places a .. b-1 of the page
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x) {
    if constexpr (sizeof(T) == 4) {
        const floatx4 a = *reinterpret_cast<const floatx4*>(p), b = *reinterpret_cast<const floatx4*>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) { x[i] = a[i]; x[i + 4] = b[i]; }
    } else {
        const bf16x8 a = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)a[i];
    }
}

// The scale of the run's page and, in *factor, what older codes are multiplied by.
template <typename T, int D>
__device__ float run_scale(const Write& w, const Run& r, const T* x, float* scale, float* lds, float* factor) {
    constexpr int L = D / 8;  // threads of a token
    float top = 0.f;
    for (int i = threadIdx.x / L; i < r.b - r.a; i += kThreads / L) {
        float e[8];
        load8(x + (r.t + i) * w.H * D + threadIdx.x % L * 8, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_abs(e[j]));
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    __syncthreads();  // the last run's use of lds
    if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = top;
    __syncthreads();
    top = fmaxf(fmaxf(lds[0], lds[1]), fmaxf(lds[2], lds[3]));
    const float need = e4m3_scale(top);
    float now = need;
    *factor = 0.f;
    if (r.a > 0) {
        const float was = *scale;
        now = fmaxf(was, need);
        *factor = was / now;
    }
    __syncthreads();  // every thread has read the scale
    if (threadIdx.x == 0) *scale = now;
    return now;
}

template <typename T, int D>
__device__ void write_keys(const Write& w, const Run& r, int h, float* lds) {
    constexpr int L = D / 8;
    const T* x = static_cast<const T*>(w.k) + (int64_t)h * D;
    float factor;
    const float now = run_scale<T, D>(w, r, x, w.ks + r.page * w.H + h, lds, &factor), inv = 1.f / now;
    uint8_t* to = w.kc + (r.page * w.H + h) * (int64_t)w.page * D + threadIdx.x % L * 8;
    const bool whole = r.a == 0 || factor != 1.f;  // the page begins anew, or all of it gets a larger scale
    const int first = whole ? 0 : r.a, last = whole ? w.page : r.b;
    for (int i = first + threadIdx.x / L; i < last; i += kThreads / L) {
        uintx2* at = reinterpret_cast<uintx2*>(to + (int64_t)i * D);
        uintx2 c = {0u, 0u};
        if (i >= r.a && i < r.b) {
            float e[8];
            load8(x + (r.t + i - r.a) * w.H * D + threadIdx.x % L * 8, e);
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = finite_or_nan(e[j]) * inv;
            c[0] = to_e4m3(e[0], e[1], e[2], e[3]);
            c[1] = to_e4m3(e[4], e[5], e[6], e[7]);
        } else if (r.a > 0) {
            c = *at;
            c[0] = e4m3_rescaled(c[0], factor);
            c[1] = e4m3_rescaled(c[1], factor);
        }
        *at = c;
    }
}

template <typename T, int D>
__device__ void write_values(const Write& w, const Run& r, int h, float* lds) {
    const T* x = static_cast<const T*>(w.v) + (int64_t)h * D;
    float factor;
    const float now = run_scale<T, D>(w, r, x, w.vs + r.page * w.H + h, lds, &factor), inv = 1.f / now;
    uint8_t* to = w.vc + (r.page * w.H + h) * (int64_t)w.page * D;
    const bool whole = r.a == 0 || factor != 1.f;
    const int first = whole ? 0 : r.a / 16, last = whole ? w.page / 16 : (r.b + 15) / 16;
    const int d = threadIdx.x % D;
    for (int grp = first + threadIdx.x / D; grp < last; grp += kThreads / D) {
        const int p0 = 16 * grp;
        uintx4* at = reinterpret_cast<uintx4*>(to + ((int64_t)grp * D + d) * 16);
        uintx4 old = {0u, 0u, 0u, 0u};
        if (r.a > 0 && (p0 < r.a || p0 + 16 > r.b)) old = *at;
        uintx4 c;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = p0 + 4 * q + j;
                e[j] = i >= r.a && i < r.b ? finite_or_nan(to_f32(x[(r.t + i - r.a) * w.H * D + d])) * inv : 0.f;
            }
            const uint32_t fresh = to_e4m3(e[0], e[1], e[2], e[3]);
            uint32_t run = 0;  // bytes of the run
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = p0 + 4 * q + j;
                if (i >= r.a && i < r.b) run |= 0xffu << (8 * j);
            }
            // the others: at the page's new scale, or 0 in a page that begins anew
            c[q] = (fresh & run) | (e4m3_rescaled(old[q], factor) & ~run);
        }
        *at = c;
    }
}

template <typename T, int DK, int DV>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(Write w) {
    __shared__ float lds[kThreads / 64];
    const int lane = threadIdx.x & 63;
    const int64_t t0 = (int64_t)blockIdx.x * w.tile;
    const bool values = (int)blockIdx.y >= w.H;
    const int h = values ? blockIdx.y - w.H : blockIdx.y;
    // Runs that start in this tile: every wave finds them, a lane for each token.
    bool leader = false;
    if (lane < w.tile && t0 + lane < w.T) {
        const int64_t t = t0 + lane, s = w.slots[t];
        if (s >= 0 && s < w.places) leader = t == 0 || s % w.page == 0 || w.slots[t - 1] != s - 1;
    }
    uint64_t todo = __ballot(leader);
    while (todo) {
        const int at = __ffsll((unsigned long long)todo) - 1;
        todo &= todo - 1;
        Run r;
        r.t = t0 + at;
        const int64_t s = w.slots[r.t];
        r.page = s / w.page;
        r.a = (int)(s - r.page * w.page);
        int len = 1;
        for (int i0 = 0; i0 < w.page - r.a; i0 += 64) {
            const int i = i0 + lane;
            const bool on = i < w.page - r.a && r.t + i < w.T && w.slots[r.t + i] == s + i;
            const uint64_t m = __ballot(on);
            if (~m) {
                len = i0 + __ffsll((unsigned long long)~m) - 1;
                break;
            }
            len = i0 + 64;
        }
        r.b = r.a + len;
        if (values) write_values<T, DV>(w, r, h, lds);
        else write_keys<T, DK>(w, r, h, lds);
    }
}

template <typename T>
void run(const Write& w, dim3 grid, hipStream_t s) {
    if (w.dk == 128 && w.dv == 128) hipLaunchKernelGGL((cache_write_kernel<T, 128, 128>), grid, dim3(kThreads), 0, s, w);
    else if (w.dk == 128) hipLaunchKernelGGL((cache_write_kernel<T, 128, 64>), grid, dim3(kThreads), 0, s, w);
    else if (w.dv == 128) hipLaunchKernelGGL((cache_write_kernel<T, 64, 128>), grid, dim3(kThreads), 0, s, w);
    else hipLaunchKernelGGL((cache_write_kernel<T, 64, 64>), grid, dim3(kThreads), 0, s, w);
}

}  // namespace

hipError_t launch_cache_write(const CacheWriteLaunch& p, hipStream_t s) {
    if (p.T_total == 0 || p.num_pages == 0) return hipSuccess;
    Write w = {p.k, p.v, p.slots, p.T_total, p.k_cache, p.v_cache, p.k_scale, p.v_scale,
               p.num_pages * p.page_size, p.page_size, p.H_kv, p.dk, p.dv, 1};
    // tokens of a tile: a power of two, at most a wave's lanes
    while (w.tile < 64 && (p.T_total + w.tile - 1) / w.tile * 2 * p.H_kv > 8192) w.tile *= 2;
    const dim3 grid((unsigned)((p.T_total + w.tile - 1) / w.tile), (unsigned)(2 * p.H_kv));
    if (p.bf16) run<bf16>(w, grid, s);
    else run<float>(w, grid, s);
    return hipGetLastError();
}

}  // namespace gdn
