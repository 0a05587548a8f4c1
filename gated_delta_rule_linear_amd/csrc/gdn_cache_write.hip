// New keys and values into the paged e4m3 cache (gdn_cache_write).
//
// The tokens of a call in one page share a scale, so the unit of work is a run:
// the call's tokens in one page, for one head, of the keys or of the values.  Its
// largest magnitude gives the scale, then its values are rounded; the values'
// 16-token groups are transposed on the way.  A run belongs to one workgroup (a
// long one) or one wave (a short one), so a page needs no atomics, and its
// values stay in registers between the two steps: they are read once.
//
// A workgroup looks at the runs that start in a tile of tokens: of few tokens
// where there are few (each token of a decode step is a run, and each wave takes
// its own, without a barrier), of more where there are many (a prompt's runs are
// whole pages, which the four waves share).
//
// Three operations per element: bound by the bytes read (2 or 4 for each) and
// written (1).
#include "gdn_e4m3.h"
#include "gdn_lanes.h"
#include "gdn_serve_kernels.h"

namespace gdn {
namespace {

#ifdef NTW
#define LDW(p) __builtin_nontemporal_load(p)
#else
#define LDW(p) (*(p))
#endif
constexpr int kWaves = 4;
constexpr int kShort = 4;  // a run of so many tokens is one wave's

struct Write {
    const void *k, *v;
    const int32_t* slots;
    int64_t T;
    uint8_t *kc, *vc;
    float *ks, *vs;
    int64_t places;  // num_pages * page_size
    int32_t page_log2, H, tile;
};

struct Run {
    int64_t t;     // first token
    int64_t page;
    int a, b;      // places a .. b-1 of the page
};

// Two neighbouring values of a token.
template <typename T>
struct Pair;
template <>
struct Pair<float> {
    floatx2 x;
    __device__ __forceinline__ float get(int i) const { return x[i]; }
};
template <>
struct Pair<bf16> {
    bf16x2 x;
    __device__ __forceinline__ float get(int i) const { return (float)x[i]; }
};
template <typename T>
__device__ __forceinline__ Pair<T> load_pair(const T* p) {
    return Pair<T>{LDW(reinterpret_cast<const decltype(Pair<T>::x)*>(p))};
}
// Eight of them.
template <typename T>
struct Eight {
    T x[8];
};
template <typename T>
__device__ __forceinline__ Eight<T> load_eight(const T* p) {
    Eight<T> e;
    if constexpr (sizeof(T) == 4) {
        const floatx4 a = LDW(reinterpret_cast<const floatx4*>(p)), b = LDW(reinterpret_cast<const floatx4*>(p + 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) { e.x[i] = a[i]; e.x[i + 4] = b[i]; }
    } else {
        const bf16x8 a = LDW(reinterpret_cast<const bf16x8*>(p));
#pragma unroll
        for (int i = 0; i < 8; ++i) e.x[i] = a[i];
    }
    return e;
}
template <typename T>
__device__ __forceinline__ uintx2 eight_codes(const Eight<T>& e, float inv) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = finite_or_nan(to_f32(e.x[i])) * inv;
    return uintx2{to_e4m3(f[0], f[1], f[2], f[3]), to_e4m3(f[4], f[5], f[6], f[7])};
}

// The page's scale behind the run and what its older codes are multiplied by (0:
// the page begins anew).
struct Scales {
    float now, factor;
};
__device__ __forceinline__ Scales new_scale(const Run& r, float was, float amax) {
    Scales s;
    s.now = e4m3_scale(amax);
    s.factor = 0.f;
    if (r.a > 0) {
        s.now = fmaxf(was, s.now);
        s.factor = was / s.now;
    }
    return s;
}

// Keys of a run, W waves.  A thread takes 8 neighbouring channels of a token;
// UNROLL tokens (one for each pass over the run) stay in registers.
template <typename T, int D, int W, int UNROLL>
__device__ void write_keys(const Write& w, const Run& r, int h, int thread, float* lds) {
    constexpr int L = D / 8, STEP = 64 * W / L;
    const int32_t page = 1 << w.page_log2;
    const int c = thread % L * 8, i0 = thread / L;
    const T* x = static_cast<const T*>(w.k) + (r.t * w.H + h) * D + c;
    const int len = r.b - r.a;
    Eight<T> e[UNROLL];
    float top = 0.f;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
        if (i0 + u * STEP < len) e[u] = load_eight(x + (int64_t)(i0 + u * STEP) * w.H * D);
    float* scale = w.ks + r.page * w.H + h;
    const float was = *scale;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
        if (i0 + u * STEP < len)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_abs(to_f32(e[u].x[j])));
    top = across<Max>(top);
    if constexpr (W > 1) {
        if (thread % 64 == 0) lds[thread / 64] = top;
        __syncthreads();  // every thread has read the scale, too
#pragma unroll
        for (int v = 0; v < W; ++v) top = fmaxf(top, lds[v]);
    }
    const Scales s = new_scale(r, was, top);
    const float inv = 1.f / s.now;
    if (thread == 0) *scale = s.now;
    uint8_t* to = w.kc + (r.page * w.H + h) * (int64_t)page * D + c;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
        if (i0 + u * STEP < len)
            *reinterpret_cast<uintx2*>(to + (int64_t)(r.a + i0 + u * STEP) * D) = eight_codes(e[u], inv);
    if (r.a > 0 && s.factor == 1.f) return;
    if (r.a == 0 && r.b == page) return;
    // the page's other places: cleared, or at the larger scale
#pragma unroll 8
    for (int i = i0; i < page; i += STEP) {
        if (i >= r.a && i < r.b) continue;
        uintx2* at = reinterpret_cast<uintx2*>(to + (int64_t)i * D);
        uintx2 old = {0u, 0u};
        if (r.a > 0) {
            old = *at;
            old[0] = e4m3_rescaled(old[0], s.factor);
            old[1] = e4m3_rescaled(old[1], s.factor);
        }
        *at = old;
    }
}

// Values of a run, W waves.  A thread takes 2 neighbouring channels of the 16
// places of a group, GROUPS groups of the page.
template <typename T, int D, int W, int GROUPS>
__device__ void write_values(const Write& w, const Run& r, int h, int thread, float* lds) {
    constexpr int L = D / 2, STEP = 64 * W / L;  // threads of a group; groups side by side
    const int32_t page = 1 << w.page_log2;
    const int d = thread % L * 2, g0 = thread / L;
    const T* x = static_cast<const T*>(w.v) + (r.t * w.H + h) * D + d;
    Pair<T> e[GROUPS][16];
#pragma unroll
    for (int u = 0; u < GROUPS; ++u)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int i = 16 * (g0 + u * STEP) + j - r.a;
            e[u][j] = Pair<T>{};
            if (i >= 0 && i < r.b - r.a) e[u][j] = load_pair(x + (int64_t)i * w.H * D);
        }
    float* scale = w.vs + r.page * w.H + h;
    const float was = *scale;
    float top = 0.f;
#pragma unroll
    for (int u = 0; u < GROUPS; ++u)
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, fmaxf(finite_abs(e[u][j].get(0)), finite_abs(e[u][j].get(1))));
    top = across<Max>(top);
    if constexpr (W > 1) {
        if (thread % 64 == 0) lds[thread / 64] = top;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < W; ++v) top = fmaxf(top, lds[v]);
    }
    const Scales s = new_scale(r, was, top);
    const float inv = 1.f / s.now;
    if (thread == 0) *scale = s.now;
    const bool whole = r.a == 0 || s.factor != 1.f;
    uint8_t* to = w.vc + (r.page * w.H + h) * (int64_t)page * D;
#pragma unroll
    for (int u = 0; u < GROUPS; ++u) {
        const int p0 = 16 * (g0 + u * STEP);
        if (p0 >= page || (!whole && (p0 >= r.b || p0 + 16 <= r.a))) continue;
        uintx4* at = reinterpret_cast<uintx4*>(to + (int64_t)p0 * D + d * 16);
        const bool full = p0 >= r.a && p0 + 16 <= r.b;
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
            uintx4 code = {0u, 0u, 0u, 0u};
            if (!full && r.a > 0) code = at[ch];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float f[4];
                uint32_t run = 0;  // bytes of the run
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[j] = finite_or_nan(e[u][4 * q + j].get(ch)) * inv;
                    const int i = p0 + 4 * q + j;
                    if (i >= r.a && i < r.b) run |= 0xffu << (8 * j);
                }
                const uint32_t fresh = to_e4m3(f[0], f[1], f[2], f[3]);
                // the others: at the page's new scale, or 0 in a page that begins anew
                if (full) code[q] = fresh;
                else code[q] = (fresh & run) | (e4m3_rescaled(code[q], s.factor) & ~run);
            }
            at[ch] = code;
        }
    }
}

// Values of a short run inside a page whose scale stays: single bytes; else the
// page's groups one after another.
template <typename T, int D>
__device__ void write_values_short(const Write& w, const Run& r, int h, int lane) {
    constexpr int C = D / 64;  // channels of a lane
    const int32_t page = 1 << w.page_log2;
    const T* x = static_cast<const T*>(w.v) + (r.t * w.H + h) * D + C * lane;
    const int len = r.b - r.a;
    float e[kShort][C], top = 0.f;
#pragma unroll
    for (int j = 0; j < kShort; ++j)
#pragma unroll
        for (int c = 0; c < C; ++c) e[j][c] = j < len ? to_f32(x[(int64_t)j * w.H * D + c]) : 0.f;
    float* scale = w.vs + r.page * w.H + h;
    const float was = *scale;
#pragma unroll
    for (int j = 0; j < kShort; ++j)
#pragma unroll
        for (int c = 0; c < C; ++c) top = fmaxf(top, finite_abs(e[j][c]));
    const Scales s = new_scale(r, was, across<Max>(top));
    const float inv = 1.f / s.now;
    if (lane == 0) *scale = s.now;
    uint8_t* to = w.vc + (r.page * w.H + h) * (int64_t)page * D + C * lane * 16;
    uint32_t code[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = finite_or_nan(e[j][c]) * inv;
        code[c] = to_e4m3(f[0], f[1], f[2], f[3]);
    }
    if (r.a > 0 && s.factor == 1.f) {
        for (int j = 0; j < len; ++j) {
            const int i = r.a + j;
#pragma unroll
            for (int c = 0; c < C; ++c) to[(int64_t)(i & ~15) * D + c * 16 + (i & 15)] = (uint8_t)(code[c] >> (8 * j));
        }
        return;
    }
#pragma unroll 4
    for (int p0 = 0; p0 < page; p0 += 16)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uintx4* at = reinterpret_cast<uintx4*>(to + (int64_t)p0 * D + c * 16);
            uintx4 old = {0u, 0u, 0u, 0u};
            if (r.a > 0) old = *at;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                old[q] = e4m3_rescaled(old[q], s.factor);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = p0 + 4 * q + j - r.a;  // the run's token here
                    if (i >= 0 && i < len)
                        old[q] = (old[q] & ~(0xffu << (8 * j))) | (((code[c] >> (8 * i)) & 0xffu) << (8 * j));
                }
            }
            *at = old;
        }
}
static_assert(kShort == 4, "a lane's new codes are one word");

// PG: page_size / 64.
template <typename T, int DK, int DV, int PG>
__global__ __launch_bounds__(64 * kWaves) void cache_write_kernel(Write w) {
    __shared__ float lds[2][kWaves];
    constexpr int page = 64 * PG;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The heads' keys and values of a tile of tokens are neighbours in memory and
    // in the grid.
    const int64_t t0 = (int64_t)(blockIdx.x / (2 * w.H)) * w.tile;
    const int y = blockIdx.x % (2 * w.H), h = y >= w.H ? y - w.H : y;
    const bool values = y >= w.H;
    // Runs that start in this tile: every wave finds them, a lane for each of the
    // 64 tokens from the tile's first.
    int64_t slot = -1, before = -1;
    if (t0 + lane < w.T) {
        slot = w.slots[t0 + lane];
        if (t0 + lane > 0) before = w.slots[t0 + lane - 1];
    }
    const bool on = slot >= 0 && slot < w.places, first = on && (slot % page == 0 || before != slot - 1);
    uint64_t todo = __ballot(first && lane < w.tile);
    const uint64_t joined = __ballot(on && !first);  // tokens in a run with the one before
    for (int shorts = 0, longs = 0; todo;) {
        const int at = __ffsll((unsigned long long)todo) - 1;
        todo &= todo - 1;
        Run r;
        r.t = t0 + at;
        const int64_t s = __builtin_amdgcn_readlane((int)slot, at);  // slots are int32
        r.page = s / page;
        r.a = (int)(s % page);
        const uint64_t stop = at == 63 ? 0 : ~joined >> (at + 1);
        int len = stop ? __ffsll((unsigned long long)stop) : 64 - at;
        if (at + len == 64)  // the run may go on behind these tokens
            for (int i0 = len; i0 < page - r.a; i0 += 64) {
                const int i = i0 + lane;
                const bool more = i < page - r.a && r.t + i < w.T && w.slots[r.t + i] == s + i;
                const uint64_t off = ~__ballot(more);
                len += off ? __ffsll((unsigned long long)off) - 1 : 64;
                if (off) break;
            }
        r.b = r.a + len;
        // All waves see the same runs in the same order, so they take the same
        // branches here and meet at the same barriers, one for each long run; two
        // sets of lds, taken in turn by long runs, keep a barrier between two uses
        // of one.
        if (len <= kShort) {
            if (shorts++ % kWaves != wave) continue;
            if (values) write_values_short<T, DV>(w, r, h, lane);
            else write_keys<T, DK, 1, (kShort * DK / 8 + 63) / 64>(w, r, h, lane, nullptr);
        } else {
            float* const l = lds[longs++ & 1];
            if (values) write_values<T, DV, kWaves, (PG * DV / 32 + kWaves - 1) / kWaves>(w, r, h, threadIdx.x, l);
            else write_keys<T, DK, kWaves, PG * DK / 8 / kWaves>(w, r, h, threadIdx.x, l);
        }
    }
}

template <typename T, int DK, int DV>
void run_d(const Write& w, dim3 grid, hipStream_t s) {
    const dim3 b(64 * kWaves);
    if (w.page_log2 == 6) hipLaunchKernelGGL((cache_write_kernel<T, DK, DV, 1>), grid, b, 0, s, w);
    else if (w.page_log2 == 7) hipLaunchKernelGGL((cache_write_kernel<T, DK, DV, 2>), grid, b, 0, s, w);
    else hipLaunchKernelGGL((cache_write_kernel<T, DK, DV, 4>), grid, b, 0, s, w);
}
template <typename T>
void run(const Write& w, int32_t dk, int32_t dv, dim3 grid, hipStream_t s) {
    if (dk == 128 && dv == 128) run_d<T, 128, 128>(w, grid, s);
    else if (dk == 128) run_d<T, 128, 64>(w, grid, s);
    else if (dv == 128) run_d<T, 64, 128>(w, grid, s);
    else run_d<T, 64, 64>(w, grid, s);
}

}  // namespace

hipError_t launch_cache_write(const CacheWriteLaunch& p, hipStream_t s) {
    if (p.T_total == 0 || p.num_pages == 0) return hipSuccess;
    Write w = {p.k, p.v, p.slots, p.T_total, p.k_cache, p.v_cache, p.k_scale, p.v_scale, p.num_pages * p.page_size,
               p.page_size == 64 ? 6 : p.page_size == 128 ? 7 : 8, p.H_kv, kWaves};
    // Tokens of a tile: one for each wave while the grid is small, at most a wave's lanes.
    while (w.tile < 64 && (p.T_total + w.tile - 1) / w.tile * 2 * p.H_kv > 16384) w.tile *= 2;
    const dim3 grid((unsigned)((p.T_total + w.tile - 1) / w.tile * 2 * p.H_kv));
    if (p.bf16) run<bf16>(w, p.dk, p.dv, grid, s);
    else run<float>(w, p.dk, p.dv, grid, s);
    return hipGetLastError();
}

}  // namespace gdn
