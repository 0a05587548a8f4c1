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
// whole pages, which all waves share).
//
// Three operations per element: bound by the bytes read (2 or 4 for each) and
// written (1).  Measured with 8 heads of 128 + 128 channels, bf16, pages of 64:
// 65,536 tokens of whole pages, 403 MB, in 83 us: 4.8 TB/s, what a large copy
// reaches (4.9).  512 single tokens move 3.2 MB and what growing scales make of
// their pages: 12 us, of which a launch is 3.5 and the rest a chain of slot,
// values, old scale, old codes, each behind the one before.
#include "gdn_e4m3.h"
#include "gdn_lanes.h"
#include "gdn_serve_kernels.h"

namespace gdn {
namespace {

// Waves of a workgroup for each 64 places of a page, so that a thread's part of a
// whole page is 16 words at every page size and four waves fit a SIMD.  (Four
// waves for pages of 256 need 64 words, one wave fits: 32,768 tokens with the
// grid below took 115 us and take 64 to 66, where a copy of as many bytes takes 41:
// a compute unit holds one such workgroup, whose loads, barrier and stores nothing
// overlaps.)
constexpr int kWaves = 4;
// Tiles grow, from a token for each wave up to a page, while the grid has more
// workgroups than this (of 4 waves): twice what the card holds at once
// shares out uneven runs, and more are mostly workgroups in which no run starts.
// 1024 / 2048 / 4096 / 16384: 2,048 tokens of a prompt 5.8 / 7.0 / 8.1 / 10.0 us,
// 8,192 tokens 13.6 / 13.6 / 20.4 / 27.5, 64 requests of 1 to 64 tokens
// 16.5 / 13.1 / 13.4 / 16.6, 4,096 single tokens 60 / 61 / 61 / 73.
constexpr int kGrid = 2048;
// A run of so many tokens is one wave's: these fit a lane's word of new codes, and
// a wave needs no barrier.
constexpr int kShort = 4;

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

// N neighbouring values of a token, as they are in memory, and the largest
// magnitude among such as bits: magnitudes order as the integers of their bits,
// Inf and NaN above all, and two bf16 are compared at once.
template <typename T, int N>
struct Values {
    static constexpr int WORDS = N * sizeof(T) / 4;
    typedef uint32_t words __attribute__((ext_vector_type(WORDS > 4 ? 4 : WORDS)));
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T* p) {
        constexpr int V = WORDS > 4 ? 4 : WORDS;
#pragma unroll
        for (int i = 0; i < WORDS; i += V) {
            const words x = __builtin_nontemporal_load(reinterpret_cast<const words*>(p) + i / V);
#pragma unroll
            for (int j = 0; j < V; ++j) w[i + j] = x[j];
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    // The largest magnitude so far, as `top_bits` undoes it.
    __device__ __forceinline__ uint32_t top(uint32_t t) const {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (sizeof(T) == 4) t = max(t, w[i] & 0x7fffffffu);
            else
                t = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, t),
                                                                           __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu)));
        }
        return t;
    }
    __device__ __forceinline__ float finite_top(float t) const {
#pragma unroll
        for (int i = 0; i < N; ++i) t = fmaxf(t, finite_abs(get(i)));
        return t;
    }
};
template <typename T>
__device__ __forceinline__ float top_bits(uint32_t t) {  // as the bits of an fp32
    if constexpr (sizeof(T) == 4) return __uint_as_float(t);
    else return __uint_as_float(max(t << 16, t & 0xffff0000u));
}
struct MaxBits {
    __device__ __forceinline__ static float of(float a, float b) { return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b))); }
};
__device__ __forceinline__ bool is_finite(float bits) { return __float_as_uint(bits) < 0x7f800000u; }

// Over W waves; one barrier, after which every thread has done what is before.
template <typename OP, int W>
__device__ __forceinline__ float over_waves(float x, float* lds) {
    x = across<OP>(x);
    if constexpr (W > 1) {
        if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = x;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < W; ++v) x = OP::of(x, lds[v]);
    }
    return x;
}
// The largest finite magnitude; *odd: there are others.
template <typename T, int W, typename F>
__device__ __forceinline__ float largest(uint32_t top, float* lds, bool* odd, F finite_top) {
    float amax = over_waves<MaxBits, W>(top_bits<T>(top), lds);
    *odd = !is_finite(amax);
    if (*odd) {  // the same for all threads
        if constexpr (W > 1) __syncthreads();
        amax = over_waves<Max, W>(finite_top(), lds);
    }
    return amax;
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
// UNROLL tokens (one for each pass over the run) stay in registers.  FULL: the
// run is a whole page.
template <typename T, int D, int W, int UNROLL, bool FULL>
__device__ void write_keys(const Write& w, const Run& r, int h, int thread, float* lds) {
    constexpr int L = D / 8, STEP = 64 * W / L;
    const int32_t page = 1 << w.page_log2;
    const int c = thread % L * 8, i0 = thread / L;
    // A run's first token is the wave's, a thread's part of an address is below
    // 2^31 bytes (256 tokens of at most 8191 heads).
    const T* x = static_cast<const T*>(w.k) + (r.t * w.H + h) * D;
    const uint32_t mine = (uint32_t)i0 * w.H * D + c;
    const int len = r.b - r.a;
    Values<T, 8> e[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
        if (!FULL) e[u].clear();
        if (FULL || i0 + u * STEP < len) e[u].load(x + (int64_t)(u * STEP) * w.H * D + mine);
    }
    float* scale = w.ks + r.page * w.H + h;
    const float was = *scale;
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) top = e[u].top(top);
    bool odd;
    const float amax = largest<T, W>(top, lds, &odd, [&]() {
        float t = 0.f;
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) t = e[u].finite_top(t);
        return t;
    });
    const Scales s = new_scale(r, was, amax);
    const float inv = 1.f / s.now;
    if (thread == 0) *scale = s.now;
    uint8_t* to = w.kc + (r.page * w.H + h) * (int64_t)page * D + c;
    auto write = [&](auto value) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            if (FULL || i0 + u * STEP < len) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = value(e[u].get(i)) * inv;
                *reinterpret_cast<uintx2*>(to + (int64_t)(r.a + i0 + u * STEP) * D) =
                    uintx2{to_e4m3(f[0], f[1], f[2], f[3]), to_e4m3(f[4], f[5], f[6], f[7])};
            }
    };
    if (odd) write([](float v) { return finite_or_nan(v); });
    else write([](float v) { return v; });
    if (FULL || (r.a > 0 && s.factor == 1.f)) return;
    // The page's other places: cleared, or at the larger scale.  Some are read
    // before the first of them is written: a load behind a store that might be to
    // the same place would wait for it.
    constexpr int MANY = W == 1 ? 16 : 4;
    for (int i1 = i0; i1 < page; i1 += MANY * STEP) {
        uintx2 old[MANY];
#pragma unroll
        for (int u = 0; u < MANY; ++u) {
            const int i = i1 + u * STEP;
            old[u] = uintx2{0u, 0u};
            if (r.a > 0 && i < page) old[u] = *reinterpret_cast<const uintx2*>(to + (int64_t)i * D);
        }
#pragma unroll
        for (int u = 0; u < MANY; ++u) {
            const int i = i1 + u * STEP;
            if (i < page && (i < r.a || i >= r.b))
                *reinterpret_cast<uintx2*>(to + (int64_t)i * D) =
                    uintx2{e4m3_rescaled(old[u][0], s.factor), e4m3_rescaled(old[u][1], s.factor)};
        }
    }
}

// Values of a run, W waves.  A thread takes 2 neighbouring channels of the 16
// places of a group, GROUPS groups of the page.
template <typename T, int D, int W, int GROUPS, bool FULL>
__device__ void write_values(const Write& w, const Run& r, int h, int thread, float* lds) {
    constexpr int L = D / 2, STEP = 64 * W / L;  // threads of a group; groups side by side
    const int32_t page = 1 << w.page_log2;
    const int d = thread % L * 2, g0 = thread / L;
    const T* x = static_cast<const T*>(w.v) + ((r.t - r.a) * w.H + h) * D;
    const uint32_t mine = (uint32_t)(16 * g0) * w.H * D + d;
    Values<T, 2> e[GROUPS][16];
#pragma unroll
    for (int u = 0; u < GROUPS; ++u) {
        const int p0 = 16 * (g0 + u * STEP);  // (with 64 channels, groups side by side may be more than a page's)
        const bool in = p0 < page;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int i = p0 + j - r.a;
            if (!FULL || D == 64) e[u][j].clear();
            if (FULL ? D == 128 || in : i >= 0 && i < r.b - r.a) e[u][j].load(x + (int64_t)(16 * u * STEP + j) * w.H * D + mine);
        }
    }
    float* scale = w.vs + r.page * w.H + h;
    const float was = *scale;
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < GROUPS; ++u)
#pragma unroll
        for (int j = 0; j < 16; ++j) top = e[u][j].top(top);
    bool odd;
    const float amax = largest<T, W>(top, lds, &odd, [&]() {
        float t = 0.f;
#pragma unroll
        for (int u = 0; u < GROUPS; ++u)
#pragma unroll
            for (int j = 0; j < 16; ++j) t = e[u][j].finite_top(t);
        return t;
    });
    const Scales s = new_scale(r, was, amax);
    const float inv = 1.f / s.now;
    if (thread == 0) *scale = s.now;
    const bool whole = r.a == 0 || s.factor != 1.f;
    uint8_t* to = w.vc + (r.page * w.H + h) * (int64_t)page * D;
    auto write = [&](auto value) {
#pragma unroll
        for (int u = 0; u < GROUPS; ++u) {
            const int p0 = 16 * (g0 + u * STEP);
            if (p0 >= page || (!whole && (p0 >= r.b || p0 + 16 <= r.a))) continue;
            uintx4* at = reinterpret_cast<uintx4*>(to + (int64_t)p0 * D + d * 16);
            const bool full = FULL || (p0 >= r.a && p0 + 16 <= r.b);
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
                uintx4 code = {0u, 0u, 0u, 0u};
                if (!full && r.a > 0) code = at[ch];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float f[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[j] = value(e[u][4 * q + j].get(ch)) * inv;
                    const uint32_t fresh = to_e4m3(f[0], f[1], f[2], f[3]);
                    if (full) {
                        code[q] = fresh;
                        continue;
                    }
                    uint32_t run = 0;  // bytes of the run
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int i = p0 + 4 * q + j;
                        if (i >= r.a && i < r.b) run |= 0xffu << (8 * j);
                    }
                    // the others: at the page's new scale, or 0 in a page that begins anew
                    code[q] = (fresh & run) | (e4m3_rescaled(code[q], s.factor) & ~run);
                }
                at[ch] = code;
            }
        }
    };
    if (odd) write([](float v) { return finite_or_nan(v); });
    else write([](float v) { return v; });
}

// A group's 16 codes with the run's, which begin `at` places in front of it, in
// their places: byte i of `code` is that of the run's token i.
__device__ __forceinline__ uintx4 with_new(uintx4 x, uint32_t code, int at, int len) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = at + 4 * q + j;
            if (i >= 0 && i < len) x[q] = (x[q] & ~(0xffu << (8 * j))) | (((code >> (8 * i)) & 0xffu) << (8 * j));
        }
    return x;
}

// Values of a short run inside a page whose scale stays: single bytes; else the
// page's groups one after another.
template <typename T, int D>
__device__ void write_values_short(const Write& w, const Run& r, int h, int lane) {
    constexpr int C = D / 64;  // channels of a lane
    const int32_t page = 1 << w.page_log2;
    const T* x = static_cast<const T*>(w.v) + (r.t * w.H + h) * D + C * lane;
    const int len = r.b - r.a;
    typedef T mine __attribute__((ext_vector_type(C)));
    float e[kShort][C], top = 0.f;
#pragma unroll
    for (int j = 0; j < kShort; ++j) {
        mine y = {};
        if (j < len) y = *reinterpret_cast<const mine*>(x + (int64_t)j * w.H * D);
#pragma unroll
        for (int c = 0; c < C; ++c) e[j][c] = to_f32(y[c]);
    }
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
    constexpr int MANY = 4;  // groups that are read before the first is written
    for (int p1 = 0; p1 < page; p1 += 16 * MANY) {
        uintx4 old[MANY][C];
#pragma unroll
        for (int u = 0; u < MANY; ++u)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                old[u][c] = uintx4{0u, 0u, 0u, 0u};
                if (r.a > 0) old[u][c] = *reinterpret_cast<const uintx4*>(to + (int64_t)(p1 + 16 * u) * D + c * 16);
            }
#pragma unroll
        for (int u = 0; u < MANY; ++u)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                uintx4 x16 = old[u][c];
#pragma unroll
                for (int q = 0; q < 4; ++q) x16[q] = e4m3_rescaled(x16[q], s.factor);
                *reinterpret_cast<uintx4*>(to + (int64_t)(p1 + 16 * u) * D + c * 16) = with_new(x16, code[c], p1 + 16 * u - r.a, len);
            }
    }
}
static_assert(kShort == 4, "a lane's new codes are one word");

// PG: page_size / 64.
template <typename T, int DK, int DV, int PG>
__global__ __launch_bounds__(64 * kWaves * PG) void cache_write_kernel(Write w) {
    constexpr int page = 64 * PG, W = kWaves * PG;
    __shared__ float lds[2][W];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The heads' keys and values of a tile of tokens are neighbours in memory and
    // in the grid.
    const int64_t begin = (int64_t)(blockIdx.x / (2 * w.H)) * w.tile, end = min(begin + w.tile, w.T);
    const int y = blockIdx.x % (2 * w.H), h = y >= w.H ? y - w.H : y;
    const bool values = y >= w.H;
    // Runs that start in this tile: every wave finds them, a lane for each of 64
    // tokens.
    int shorts = 0, longs = 0;
    int64_t t0 = begin, next;
    do {
        next = t0 + 64;  // or behind the last run
        int64_t slot = -1, before = -1;
        if (t0 + lane < w.T) {
            slot = w.slots[t0 + lane];
            if (t0 + lane > 0) before = w.slots[t0 + lane - 1];
        }
        const bool on = slot >= 0 && slot < w.places, first = on && (slot % page == 0 || before != slot - 1);
        uint64_t todo = __ballot(first && t0 + lane < end);
        const uint64_t joined = __ballot(on && !first);  // tokens in a run with the one before
        while (todo) {
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
            next = max(next, r.t + len);
            // All waves see the same runs in the same order, so they take the same
            // branches here and meet at the same barriers, one for each long run; two
            // sets of lds, taken in turn by long runs, keep a barrier between two uses
            // of one.
            if (len <= kShort) {
                if (shorts++ % W != wave) continue;
                if (values) write_values_short<T, DV>(w, r, h, lane);
                else write_keys<T, DK, 1, (kShort * DK / 8 + 63) / 64, false>(w, r, h, lane, nullptr);
            } else {
                float* const l = lds[longs++ & 1];
                constexpr int KU = DK / 8 / kWaves, VG = (DV / 32 + kWaves - 1) / kWaves;
                if (len == page) {
                    if (values) write_values<T, DV, W, VG, true>(w, r, h, threadIdx.x, l);
                    else write_keys<T, DK, W, KU, true>(w, r, h, threadIdx.x, l);
                } else if (values) {
                    write_values<T, DV, W, VG, false>(w, r, h, threadIdx.x, l);
                } else {
                    write_keys<T, DK, W, KU, false>(w, r, h, threadIdx.x, l);
                }
            }
        }
        t0 = next;
    } while (PG > 1 && t0 < end);  // (a tile is at most a page)
}

template <typename T, int DK, int DV>
void run_d(const Write& w, dim3 grid, hipStream_t s) {
    const dim3 b(kWaves << w.page_log2);
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
               p.page_size == 64 ? 6 : p.page_size == 128 ? 7 : 8, p.H_kv, 0};
    // Tokens of a tile: one for each wave while the grid is small, at most a page's.
    w.tile = kWaves * (int)(p.page_size / 64);
    while (w.tile < p.page_size && (p.T_total + w.tile - 1) / w.tile * 2 * p.H_kv > kGrid / (p.page_size / 64)) w.tile *= 2;
    const dim3 grid((unsigned)((p.T_total + w.tile - 1) / w.tile * 2 * p.H_kv));
    if (p.bf16) run<bf16>(w, p.dk, p.dv, grid, s);
    else run<float>(w, p.dk, p.dv, grid, s);
    return hipGetLastError();
}

}  // namespace gdn
