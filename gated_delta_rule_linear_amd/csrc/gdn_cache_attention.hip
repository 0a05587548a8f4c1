// Causal attention of a step's new tokens over the paged e4m3 cache
// (gdn_cache_attention).
//
// The query heads of one key/value head read the same keys, so the rows of a
// product are the (new token, query head of the group) pairs of one request and
// key/value head, flattened: row = token * G + head of the group.  A workgroup
// takes a tile of them and walks the cache in tiles of 64 tokens with the
// running maximum and sum of the softmax.  Requests with few rows (decode,
// verifying drafted tokens) go to attention_rows_kernel, which is bound by
// reading the cache; the others to attention_tile_kernel, which is bound by the
// matrix cores.  Where rows are few in all, and for the last of many, a request's
// cache is cut into parts that workgroups take side by side and
// attention_join_kernel joins.
//
// Scores are formed transposed, S^T = K Q^T, so that a lane holds scores of one
// row and the softmax statistics of a row are scalars of its lanes, and so that
// a lane's scores are those of 16 neighbouring tokens: K's rows are handed to the
// matrix core in the order that makes them so.  They are then, rounded to bf16,
// the operand that the second product O^T = V^T P^T takes from that lane.  Its
// other operand, V^T, is 16 tokens of one channel: one 16-byte load of the cache
// as it is stored.  Codes are converted to bf16 exactly, and a page's scale, a
// power of two, is applied exactly, to the scores and p or in the conversion.
#include <algorithm>
#include <cmath>
#include <limits>

#include "gdn_e4m3.h"
#include "gdn_lanes.h"
#include "gdn_mfma.h"
#include "gdn_serve_kernels.h"

namespace gdn {
namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));

constexpr int kTile = 64;      // tokens of a tile
constexpr int kFewRows = 32;   // a request with up to so many rows is one of few rows
constexpr int kMinPart = 512;  // tokens of a part of a request's cache, at least (measured for few rows)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInf = __builtin_inff();

struct Attention {
    const void* q;
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *rows, *kv_lens, *cu;
    int32_t num_seqs;
    int64_t T;
    int32_t num_pages, page_log2, num_rows, max_blocks;
    float scale2;   // |scale| * log2(e), above 0: scores in units of log 2
    bool negative;  // the scale is: q is negated
    void* o;
    int32_t H, Hkv, G;
    // Requests of few rows (at most few_rows) and the others: at most so many
    // parts of a request's cache.
    int32_t few_rows;
    int32_t splits[2];
    bool tiled;  // the others go to the tile kernel
    // The tile kernel's tiles of rows for each key/value head, and those of them,
    // the first, whose cache is cut into parts.
    int32_t tiles, tail;
    // Parts before they are joined, [part][row][d_v] and [part][row][2] (maximum
    // and sum).  Rows: for few, (n * Hkv + h) * few_rows + row; else the first of q.
    int64_t part_rows[2];
    float *ws_o[2], *ws_ml[2];
};

// Tiles of BR rows that the requests before n take at most: the tiles of
// request n start here.  (floor(x / BR) grows by at least ceil(rows / BR) - 1
// over a request's rows.)
__device__ __forceinline__ int64_t first_tile(const Attention& a, int64_t n, int br) {
    return (int64_t)a.cu[n] * a.G / br + n;
}
// The request whose tiles hold tile b: the last n with first_tile(n) <= b.
__device__ __forceinline__ int32_t request_of(const Attention& a, int64_t b, int br) {
    int32_t below = 0;
    for (int32_t n0 = 0; n0 < a.num_seqs; n0 += 64) {
        const int32_t n = n0 + (threadIdx.x & 63);
        below += __popcll(__ballot(n < a.num_seqs && first_tile(a, n, br) <= b));
    }
    return below - 1;
}

// A request, as every kernel sees it.
struct Request {
    int64_t t0;       // first new token
    int32_t len;      // new tokens
    int32_t rows;     // len * G
    int64_t kv;       // tokens held
    int64_t chunk;    // tokens of a part of its cache
    bool few;
    __device__ __forceinline__ Request(const Attention& a, int32_t n) {
        int64_t t1 = a.cu[n + 1];
        t0 = a.cu[n];
        const int64_t most = (int64_t)a.max_blocks << a.page_log2, held = a.kv_lens[n];
        t0 = t0 < 0 ? 0 : t0;
        t1 = t1 < a.T ? t1 : a.T;
        len = t1 > t0 ? (int32_t)(t1 - t0) : 0;
        rows = len * a.G;
        kv = held < 0 ? 0 : held < most ? held : most;
        few = rows <= a.few_rows;
        const int c = few ? 0 : 1;
        chunk = ((kv + a.splits[c] - 1) / a.splits[c] + kTile - 1) / kTile * kTile;
        if (chunk < kMinPart) chunk = kMinPart;
        if (!few && !a.tiled && chunk < kv) chunk = (kv + kTile - 1) / kTile * kTile;  // there is no room for its parts
    }
    __device__ __forceinline__ bool alone() const { return kv <= chunk; }
};

__device__ __forceinline__ const int32_t* table_of(const Attention& a, int32_t n) {
    const int32_t row = a.rows ? a.rows[n] : n;
    return row >= 0 && row < a.num_rows && a.num_pages > 0 ? a.table + (int64_t)row * a.max_blocks : nullptr;
}

// The lane's number where it is needed: what is made of threadIdx.x is kept in
// registers from the kernel's start, through loops that need them all.
__device__ __forceinline__ int late_lane() {
    uint32_t all = ~0u;
    asm volatile("" : "+s"(all));
    return (int)__builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0));
}

// Pages and scales of 64 tiles, `step` tokens apart, a lane for each: fetched
// ahead in one go, since a load in the tiles' loop whose result is needed at
// once would wait for every load before it, the keys and values among them.
struct Pages {
    int32_t page;  // -1: left out
    float ks, vs;
    __device__ __forceinline__ void fetch(const Attention& a, const int32_t* table, int32_t h, int64_t base, int64_t to, int step, int lane) {
        const int64_t at = base + (int64_t)lane * step;
        page = table && at < to ? table[at >> a.page_log2] : -1;
        if (page >= a.num_pages) page = -1;
        ks = vs = 0.f;
        if (page >= 0) {
            const int64_t ph = (int64_t)page * a.Hkv + h;
            ks = a.ks[ph];
            vs = a.vs[ph];
        }
    }
    __device__ __forceinline__ static float lane_of(float x, int i) {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), i));
    }
};

// Whether a row that sees the tokens up to `sees` sees one of the tiles at base,
// base + step, ... below `to`: some of them may have no page.  For rows whose
// maximum is -Inf: without a token their output is 0, with scores that are all
// -Inf it is NaN.
__device__ __forceinline__ bool sees_some(const Attention& a, const int32_t* table, int64_t base, int64_t to, int step,
                                          int64_t sees) {
    const int lane = late_lane();
    for (; base < to; base += 64 * (int64_t)step) {
        const int64_t at = base + (int64_t)lane * step;
        const int32_t page = table && at < to ? table[at >> a.page_log2] : -1;
        const uint64_t there = __ballot(page >= 0 && page < a.num_pages);
        if (there) return base + (__ffsll((unsigned long long)there) - 1) * (int64_t)step <= sees;
    }
    return false;
}
// Statistics of a part of a row are joined with those of the others by this
// factor, `all` the largest maximum.  Parts whose scores are all -Inf have a sum
// above 0, those without a token 0, and the factor keeps that apart: 1, where
// the exponential's argument is no number.
__device__ __forceinline__ float joined(float part, float all) {
    return part == all ? 1.f : __builtin_amdgcn_exp2f(part - all);
}
__device__ __forceinline__ float reciprocal_sum(float sum, float top) {
    return sum == 0.f ? 0.f : top == -kInf ? __builtin_nanf("") : 1.f / sum;
}

// A value split into NS bf16 parts: one rounds it, three hold all of an fp32.
template <int NS>
__device__ __forceinline__ void split_bf16(float x, bf16* part) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        part[s] = (bf16)x;
        x -= (float)part[s];
    }
}

// Eight neighbouring values, as they are in memory and as NS bf16 operands.
template <typename TI>
struct Eight;
template <>
struct Eight<float> {
    floatx4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const floatx4*>(p);
        b = *reinterpret_cast<const floatx4*>(p + 4);
    }
    __device__ __forceinline__ void split(bf16x8* part) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            bf16 x[3];
            split_bf16<3>(j < 4 ? a[j & 3] : b[j & 3], x);
#pragma unroll
            for (int s = 0; s < 3; ++s) part[s][j] = x[s];
        }
    }
};
template <>
struct Eight<bf16> {
    bf16x8 a;
    __device__ __forceinline__ void load(const bf16* p) { a = *reinterpret_cast<const bf16x8*>(p); }
    __device__ __forceinline__ void split(bf16x8* part) const { part[0] = a; }
};

template <typename TI>
__device__ __forceinline__ void store4(TI* p, floatx4 x) {
    if constexpr (sizeof(TI) == 4) *reinterpret_cast<floatx4*>(p) = x;
    else *reinterpret_cast<bf16x4*>(p) = bf16x4{(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]};
}

constexpr int kWaves = 4;

// ---------------------------------------------------------------- few rows
//
// One workgroup: 16 rows, one part of the cache; its waves take the part's tiles
// in turn, each with statistics of its own, and are joined at the end.  16x16x32
// products (lane l: r = l % 16, g = l / 16): row i of K's tile t (t = 0..3) is
// token 16 (i / 4) + 4 t + i % 4, so that a lane's scores of the four tiles are
// those of tokens 16 g .. 16 g + 15.  Nothing is shared between waves, so codes
// go from memory to registers and are converted there.  The loads of a tile's
// keys and values are in flight while the tile before is worked on: keys are
// asked for when the last keys have become scores, values when the last values
// have been used.
//
// Bound by reading the cache: 5.6 TB/s over 64 requests of 512 to 16384 tokens
// (8 heads of 128 channels, 8 KB of a page at a time in random order), which the
// same kernel with the loads alone does not exceed by more than 3%; 5.9 over one
// request of 65536 (22.6 us; with the join the call takes 28, 4.8 TB/s).  Keys'
// loads that take half a line of each row instead ran at 4.4, temporal loads at
// 4.7.  Requests of up to 32 rows take two workgroups side by side rather than a
// tile of the other kernel: 5 new tokens of 16 requests over 4000 take 43 us here
// and 47 there, in fp32 45 and 96, and 6 tokens over 300 7 and 14.
template <typename TI, int DK, int DV>
__global__ __launch_bounds__(64 * kWaves, 2) void attention_rows_kernel(Attention a) {
    constexpr int NS = sizeof(TI) == 4 ? 3 : 1;
    constexpr int BR = 16, KS = DK / 32, VT = DV / 16;
    // Of each wave: a tile's keys, and in the end its output.
    constexpr int PR = DK / 16, KEYS = kTile * PR, OUT = BR * (DV + 4) / 4;
    __shared__ uintx4 s_wave[kWaves][KEYS > OUT ? KEYS : OUT];
    __shared__ float s_m[kWaves][BR], s_l[kWaves][BR];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int h = blockIdx.y, per = (a.few_rows + BR - 1) / BR;  // workgroups side by side along a request's rows
    const int32_t n = blockIdx.x / per;
    const Request job(a, n);
    if (a.tiled && !job.few) return;
    const int64_t from = blockIdx.z * job.chunk;
    if (blockIdx.z > 0 && from >= job.kv) return;
    const int32_t* const table = table_of(a, n);
    const int page_mask = (1 << a.page_log2) - 1;
    // (With a request of more rows than it was planned for, more than one turn.)
    for (int32_t row0 = (blockIdx.x - n * per) * BR; row0 < job.rows; row0 += per * BR) {
    const int32_t last_row = (row0 + BR < job.rows ? row0 + BR : job.rows) - 1;
    int64_t to = job.kv - job.len + last_row / a.G + 1;  // no row of the tile sees more
    to = !table ? from : to < from + job.chunk ? to : from + job.chunk;
    const int64_t all_see = job.kv - job.len + row0 / a.G;  // every row of the tile sees up to here

    // this lane's row; lanes behind the last one work on the first, unseen
    const int32_t row = row0 + r;
    const bool live = row < job.rows;
    const int32_t i = live ? row / a.G : 0, head = h * a.G + (live ? row - i * a.G : 0);
    const int64_t sees = live ? job.kv - job.len + i : -1;  // the last token that the row sees
    Eight<TI> q8[KS];
#pragma unroll
    for (int m = 0; m < KS; ++m)
        q8[m].load(static_cast<const TI*>(a.q) + ((job.t0 + i) * a.H + head) * DK + 16 * g + 64 * (m >> 1) + 8 * (m & 1));

    uintx4 kr[PR], vr[VT];
    // Keys are read as they lie, whole lines at a time (a row of a product takes
    // half a line from each load otherwise, which halved the rate), and change
    // places through the wave's LDS: piece `c` of 16 channels of token `row` goes
    // to place c ^ turn(row), so that the 16 rows of a product's operand spread
    // over the banks.
    uintx4* const s_k = s_wave[wave];
    auto turn = [&](int row) { return ((row & 3) | (row >> 4 & 1) << 2) & (PR - 1); };
    // (The loads have no branch: one would make the wait for the loads before it
    // a wait for these too.  Where there is no tile they read page 0.)
    auto load_keys = [&](int64_t base, int32_t p) {
        const int64_t ph = (int64_t)(p < 0 ? 0 : p) * a.Hkv + h;
        const uintx4* at = reinterpret_cast<const uintx4*>(a.kc + ((ph << a.page_log2) + (base & page_mask)) * DK) + lane;
#pragma unroll
        for (int j = 0; j < PR; ++j) kr[j] = __builtin_nontemporal_load(at + 64 * j);
    };
    auto load_values = [&](int64_t base, int32_t p) {
        const int64_t ph = (int64_t)(p < 0 ? 0 : p) * a.Hkv + h;
        const uint8_t* at = a.vc + ((ph << a.page_log2) + (base & page_mask)) * DV + (g * DV + r) * 16;
#pragma unroll
        for (int d = 0; d < VT; ++d) vr[d] = __builtin_nontemporal_load(reinterpret_cast<const uintx4*>(at + d * 256));
    };
    constexpr int STEP = kWaves * kTile;
    const int64_t first = from + wave * kTile;
    Pages pages;
    pages.fetch(a, table, h, first, to, STEP, late_lane());
    int at = 0;  // the tile's lane of `pages`
    int32_t page = __builtin_amdgcn_readlane(pages.page, 0);
    float ks = Pages::lane_of(pages.ks, 0), vs = Pages::lane_of(pages.vs, 0);
    if (first < to) {
        load_keys(first, page);
        load_values(first, page);
    }

    bf16x8 qf[KS][NS];
#pragma unroll
    for (int m = 0; m < KS; ++m) q8[m].split(qf[m]);

    floatx4 O[VT];
#pragma unroll
    for (int d = 0; d < VT; ++d) O[d] = zero4();
    float mx = -kInf, sum = 0.f;
    for (int64_t base = first; base < to; base += STEP) {
        const bool there = page >= 0;
        float s[16];
        if (there) {
            const float c2 = a.negative ? -ks * a.scale2 : ks * a.scale2;
#pragma unroll
            for (int j = 0; j < PR; ++j) {
                const int row = (64 * j + lane) / PR, c = lane % PR;
                s_k[row * PR + (c ^ turn(row))] = kr[j];
            }
            asm volatile("" ::: "memory");  // the wave's writes and reads of s_k stay in this order
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                floatx4 x = zero4();
                const int row = 16 * (r >> 2) + 4 * c + (r & 3);
                uintx4 k16[DK / 64];
#pragma unroll
                for (int j = 0; j < DK / 64; ++j) k16[j] = s_k[row * PR + ((4 * j + g) ^ turn(row))];
#pragma unroll
                for (int m = 0; m < KS; ++m) {
                    const bf16x8 k8 = e4m3_to_bf16x8(k16[m >> 1][2 * (m & 1)], k16[m >> 1][2 * (m & 1) + 1]);
#pragma unroll
                    for (int p = NS - 1; p >= 0; --p) x = Mma<bf16>::mma(k8, qf[m][p], x);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) s[4 * c + j] = x[j] * c2;
            }
        }
        asm volatile("" ::: "memory");  // (and the next tile's writes behind them)
        if (++at == 64) {
            pages.fetch(a, table, h, base + STEP, to, STEP, late_lane());
            at = 0;
        }
        page = __builtin_amdgcn_readlane(pages.page, at);
        load_keys(base + STEP, page);
        if (there) {
            const bool edge = base + kTile - 1 > all_see;  // some row does not see all of the tile
            const int64_t see = sees - (base + 16 * g);
            if (edge) {
#pragma unroll
                for (int j = 0; j < 16; ++j) s[j] = j <= see ? s[j] : -kInf;
            }
            float top = s[0];
#pragma unroll
            for (int j = 1; j < 16; ++j) top = fmaxf(top, s[j]);
            top = across<Max, 16>(top);
            const float now = fmaxf(mx, top);
            const float ref = now == -kInf ? 0.f : now;
            const float fade = __builtin_amdgcn_exp2f(mx - ref);
            mx = now;
            sum *= fade;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                s[j] = __builtin_amdgcn_exp2f(s[j] - ref);
                sum += s[j];
            }
            bf16x8 pf[NS][2];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                bf16 part[NS];
                split_bf16<NS>(s[j] * vs, part);
#pragma unroll
                for (int p = 0; p < NS; ++p) pf[p][j >> 3][j & 7] = part[p];
            }
#pragma unroll
            for (int d = 0; d < VT; ++d) O[d] *= fade;
            if (edge) {
                // Codes behind the last held token may be anything, and a NaN of a
                // token that only some rows see must not reach the others as 0 * NaN.
                bool nan = false;
#pragma unroll
                for (int d = 0; d < VT; ++d) {
                    keep_codes(vr[d], job.kv - (base + 16 * g));
                    nan |= has_nan_code(vr[d]);
                }
                if (__ballot(nan)) {
                    bf16x8 see8[2];
#pragma unroll
                    for (int j = 0; j < 16; ++j) see8[j >> 3][j & 7] = (bf16)(j <= see ? 1.f : 0.f);
#pragma unroll
                    for (int d = 0; d < VT; ++d) {
                        uintx4 ones;
                        split_nan(vr[d], ones);
                        floatx4 hits = zero4();
                        hits = Mma<bf16>::mma(e4m3_to_bf16x8(ones[0], ones[1]), see8[0], hits);
                        hits = Mma<bf16>::mma(e4m3_to_bf16x8(ones[2], ones[3]), see8[1], hits);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (hits[j] > 0.f) O[d][j] = __builtin_nanf("");
                    }
                }
            }
#pragma unroll
            for (int d = 0; d < VT; ++d) {
                const bf16x8 v0 = e4m3_to_bf16x8(vr[d][0], vr[d][1]), v1 = e4m3_to_bf16x8(vr[d][2], vr[d][3]);
#pragma unroll
                for (int p = NS - 1; p >= 0; --p) {
                    O[d] = Mma<bf16>::mma(v0, pf[p][0], O[d]);
                    O[d] = Mma<bf16>::mma(v1, pf[p][1], O[d]);
                }
            }
        }
        load_values(base + STEP, page);
        ks = Pages::lane_of(pages.ks, at);
        vs = Pages::lane_of(pages.vs, at);
    }
    sum = across<Sum, 16>(sum);
    // The wave's output takes the place of its keys.
    float(*const s_o)[DV + 4] = reinterpret_cast<float(*)[DV + 4]>(s_k);
#pragma unroll
    for (int d = 0; d < VT; ++d) *reinterpret_cast<floatx4*>(&s_o[r][16 * d + 4 * g]) = O[d];
    if (g == 0) {
        s_m[wave][r] = mx;
        s_l[wave][r] = sum;
    }
    __syncthreads();
    // Join the waves: a thread takes DV / 16 channels of one row.
    constexpr int C = DV / 16;
    const int jr = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * C;
    const int32_t ji = (row0 + jr) / a.G;
    float m = s_m[0][jr], l = 0.f, f[kWaves];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, s_m[w][jr]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        f[w] = __builtin_amdgcn_exp2f(s_m[w][jr] - (m == -kInf ? 0.f : m));
        l += f[w] * s_l[w][jr];
    }
    if (__ballot(row0 + jr < job.rows && m == -kInf)) {
        const bool some = sees_some(a, table, from, to, kTile, job.kv - job.len + ji);
        if (m == -kInf && some) l += 1.f;
    }
    if (row0 + jr < job.rows) {
        float out[C];
#pragma unroll
        for (int k = 0; k < C; ++k) out[k] = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
#pragma unroll
            for (int k = 0; k < C; ++k) out[k] += f[w] * reinterpret_cast<const float(*)[DV + 4]>(s_wave[w])[jr][c0 + k];
        const int64_t orow = (job.t0 + ji) * a.H + h * a.G + (row0 + jr - ji * a.G);
        if (job.alone()) {
            const float inv = reciprocal_sum(l, m);
#pragma unroll
            for (int k = 0; k < C; k += 4)
                store4(static_cast<TI*>(a.o) + orow * DV + c0 + k,
                       floatx4{out[k] * inv, out[k + 1] * inv, out[k + 2] * inv, out[k + 3] * inv});
        } else {
            const int64_t prow = blockIdx.z * a.part_rows[0] + ((int64_t)n * a.Hkv + h) * a.few_rows + row0 + jr;
#pragma unroll
            for (int k = 0; k < C; k += 4)
                *reinterpret_cast<floatx4*>(a.ws_o[0] + prow * DV + c0 + k) = floatx4{out[k], out[k + 1], out[k + 2], out[k + 3]};
            if (c0 == 0) {
                a.ws_ml[0][2 * prow] = m;
                a.ws_ml[0][2 * prow + 1] = l;
            }
        }
    }
    __syncthreads();  // before the next turn's waves write s_o
    }
}

// ---------------------------------------------------------------- many rows
//
// One workgroup: 32 rows for each of its waves.  The waves read the same keys
// and values, so a tile's codes are converted once, by all of them, and staged
// in LDS as bf16 in the order in which the matrix core takes them: a fragment is
// 64 lanes x 16 bytes, read without conflicts.
//
// 32x32x16 products (lane l: c = l % 32, hf = l / 32; a result has rows
// 8 q + 4 hf + i, q and i 0..3): row 8 q + 4 hf + i of K's half-tile is token
// 16 hf + 4 q + i, so that a lane's 16 scores of a half-tile are those of tokens
// 16 hf .. 16 hf + 15.
//
// A tile costs a wave about as long on the matrix core as on the vector units,
// so both have to be busy at once, and a SIMD's two waves do not arrange that by
// themselves: they drift into waiting for the same unit.  So a wave's products
// run beside vector work that does not need them, in two blocks per tile: the
// next tile's scores beside this tile's exponentials, and this tile's output
// beside the next tile's maximum and the staging.  Of keys and of values two
// tiles are held; keys are one tile ahead.
//
// In full precision, rescaling the output for a new maximum is put off while the
// maximum has grown by at most 2^8 (p stays below 2^8, and all of it is kept).
// With p rounded to bf16 the largest p is kept at 1, which is exact: put off
// too, the rescaling would save 2%, but the largest terms would be rounded like
// the others and the output's error grow from 1.1 times that of its own rounding
// (1.15 over 16384 tokens) to 1.3.
//
// Bound by the matrix cores and the power they draw: 1.03 to 1.05 PFLOP/s over two
// prompts of 8192 tokens (32 heads, 8 for keys, 128 channels), 1.04 to 1.07 over
// chunks of 1021 to 2048 tokens behind 16384, on several devices of one model
// (0.91 and 0.92 on the slowest), where a plain product of 8192 x 8192 matrices
// reaches 1.18 to 1.24; with 64 channels, where a tile's
// products are half and its exponentials the same, 0.85.  In full precision
// (three products for one) 0.36.
template <typename TI, int DK, int DV>
__global__ __launch_bounds__(64 * kWaves, sizeof(TI) == 4 ? 1 : 2) void attention_tile_kernel(Attention a) {
    constexpr int NS = sizeof(TI) == 4 ? 3 : 1;
    constexpr int BR = 32 * kWaves, KS = DK / 16, DT = DV / 32;
    constexpr float kSlack = NS == 1 ? 0.f : 8.f;
    // A fragment's place is longer than the fragment: a wave writes pieces of the
    // same lanes of several fragments at once, which so fall into different banks.
    __shared__ uintx4 s_k[2][2 * KS][65];      // [tile % 2][half-tile * KS + step][lane]
    __shared__ uintx4 s_v[2][2 * 2 * DT][64];  // [tile % 2][(half-tile * 2 + step) * DT + channels][lane]
    __shared__ int32_t s_nan[2][kWaves];       // a wave's part of the tile's values had a NaN code
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 31, hf = lane >> 5;
    // Key/value heads are neighbours in the grid: workgroups go to the eight XCDs in
    // turn, so with eight heads the tiles of a head share one XCD's cache.  The
    // last rows, which see most, come first, and the parts of the first last.
    const int h = blockIdx.x % a.Hkv;
    const int32_t id = blockIdx.x / a.Hkv, over = id - a.tiles, part = over < 0 ? 0 : 1 + over / a.tail;
    const int32_t rtile = over < 0 ? a.tiles - 1 - id : a.tail - 1 - over % a.tail;
    const int32_t n = request_of(a, rtile, BR);
    if (n < 0) return;
    Request job(a, n);
    if (rtile >= a.tail) job.chunk = job.kv;
    const int64_t row0_ = (rtile - first_tile(a, n, BR)) * BR;
    if (job.few || row0_ < 0 || row0_ >= job.rows) return;
    const int32_t row0 = (int32_t)row0_, last_row = (row0 + BR < job.rows ? row0 + BR : job.rows) - 1;
    const int64_t from = part * job.chunk;
    if (part > 0 && from >= job.kv) return;
    const int32_t* const table = table_of(a, n);
    int64_t to = job.kv - job.len + last_row / a.G + 1;  // no row of the tile sees more
    to = !table ? from : to < from + job.chunk ? to : from + job.chunk;
    const int64_t all_see = job.kv - job.len + row0 / a.G;  // every row of the workgroup sees up to here
    const int32_t count = to > from ? (int32_t)((to - from + kTile - 1) / kTile) : 0;  // tiles
    const int page_mask = (1 << a.page_log2) - 1;

    // this lane's row; lanes behind the last one work on the first, unseen
    const int32_t row = row0 + 32 * wave + c;
    const bool live = row < job.rows;
    const int32_t i = live ? row / a.G : 0, head = h * a.G + (live ? row - i * a.G : 0);
    const int64_t orow = (job.t0 + i) * a.H + head;
    const int64_t sees = live ? job.kv - job.len + i - from : -1;  // the last token of the part that the row sees
    // Of this wave: no row sees tiles from wave_tiles on, every row sees the first wave_all.
    const int32_t wrow = row0 + 32 * wave, wlast = wrow + 31 < job.rows ? wrow + 31 : job.rows - 1;
    auto tiles_below = [&](int64_t tokens, int64_t up) {  // whole tiles, or tiles begun, of the part's first tokens
        const int64_t t = tokens <= 0 ? 0 : (tokens + up) / kTile;
        return (int32_t)(t < count ? t : count);
    };
    const int32_t wave_tiles = wrow < job.rows ? tiles_below(job.kv - job.len + wlast / a.G + 1 - from, kTile - 1) : 0;
    const int32_t wave_all = wrow < job.rows ? tiles_below(job.kv - job.len + wrow / a.G + 1 - from, 0) : 0;
    const int32_t group_all = tiles_below(all_see + 1 - from, 0);  // every row of the workgroup sees these tiles whole
    Eight<TI> q8[KS];
#pragma unroll
    for (int m = 0; m < KS; ++m) q8[m].load(static_cast<const TI*>(a.q) + orow * DK + 16 * m + 8 * hf);

    // Staging: a thread takes 16-byte pieces of keys (a token's 16 channels) and
    // of values (a channel's 16 tokens).
    constexpr int NT = 64 * kWaves, KP = kTile * DK / 16 / NT, VP = kTile * DV / 16 / NT;
    uintx4 kr[KP], vr[VP];
    Pages pages;
    int32_t window = 0;  // the tile of lane 0 of `pages`; tiles from `count` on have no page
    auto there = [&](int32_t tile) { return tile < count && __builtin_amdgcn_readlane(pages.page, tile - window) >= 0; };
    // The loads have no branch: one would make the wait for the loads before it a
    // wait for these too.  Where there is no tile they read page 0.
    auto place_of = [&](int32_t tile) {
        const int32_t p = __builtin_amdgcn_readlane(pages.page, tile - window);
        return ((((int64_t)(p < 0 ? 0 : p) * a.Hkv + h) << a.page_log2) + ((from + (int64_t)tile * kTile) & page_mask));
    };
    auto load_keys = [&](int32_t tile) {
        const uintx4* k = reinterpret_cast<const uintx4*>(a.kc + place_of(tile) * DK) + threadIdx.x;
#pragma unroll
        for (int j = 0; j < KP; ++j) kr[j] = k[j * NT];
    };
    auto load_values = [&](int32_t tile) {
        const uintx4* v = reinterpret_cast<const uintx4*>(a.vc + place_of(tile) * DV) + threadIdx.x;
#pragma unroll
        for (int j = 0; j < VP; ++j) vr[j] = v[j * NT];
    };
    // (Tiles without a page are staged all the same, from what the loads read.)
    // A thread's pieces: of one half-tile each, or of one tile.
    static_assert((KP == 2 && KS == 8) || (KP == 1 && KS == 4), "pieces of keys");
    static_assert((VP == 2 && DV == 128) || (VP == 1 && DV == 64), "pieces of values");
    const int ktoken = threadIdx.x / KS, kstep = threadIdx.x % KS;
    uintx4* const kto = &s_k[0][(KP == 1 ? ktoken >> 5 : 0) * KS + kstep][8 * ((ktoken >> 2) & 3) + 4 * ((ktoken >> 4) & 1) + (ktoken & 3)];
    const int vgroup = threadIdx.x / DV, vd = threadIdx.x % DV;
    uintx4* const vto = &s_v[0][(VP == 1 ? vgroup >> 1 : 0) * 2 * DT + vd / 32][32 * (vgroup & 1) + (vd & 31)];
    auto stage_keys = [&](int32_t tile, int buf) {
        const float ks = Pages::lane_of(pages.ks, tile - window);
#pragma unroll
        for (int j = 0; j < KP; ++j) {
            uintx4* const to_ = kto + (buf * 2 * KS + j * KS) * 65;
            to_[0] = __builtin_bit_cast(uintx4, e4m3_to_bf16x8(kr[j][0], kr[j][1], ks));
            to_[32] = __builtin_bit_cast(uintx4, e4m3_to_bf16x8(kr[j][2], kr[j][3], ks));
        }
    };
    // Codes behind the last token, and NaN codes, as in the rows kernel.
    auto clean_values = [&](int32_t tile, int buf) {
        const int64_t base = from + (int64_t)tile * kTile;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < VP; ++j) {
            uintx4 ones;
            keep_codes(vr[j], job.kv - (base + 16 * ((int)(threadIdx.x + j * NT) / DV)));
            nan |= has_nan_code(vr[j]);
            split_nan(vr[j], ones);
        }
        const bool any = __ballot(nan) != 0;
        if (lane == 0) s_nan[buf][wave] = any;
    };
    auto stage_values = [&](int32_t tile, int buf) {
        const float vs = Pages::lane_of(pages.vs, tile - window);
#pragma unroll
        for (int j = 0; j < VP; ++j) {
            uintx4* const to_ = vto + (buf * 4 * DT + j * 2 * DT) * 64;
            to_[0] = __builtin_bit_cast(uintx4, e4m3_to_bf16x8(vr[j][0], vr[j][1], vs));
            to_[DT * 64] = __builtin_bit_cast(uintx4, e4m3_to_bf16x8(vr[j][2], vr[j][3], vs));
        }
    };

    if (count > 0) {
        pages.fetch(a, table, h, from, to, kTile, lane);
        load_keys(0);
        load_values(0);
    }
    bf16x8 qf[KS][NS];
#pragma unroll
    for (int m = 0; m < KS; ++m) {
        q8[m].split(qf[m]);
        if (a.negative)
#pragma unroll
            for (int p = 0; p < NS; ++p) qf[m][p] = -qf[m][p];
    }
    if (count > 0) {
        stage_keys(0, 0);
        load_keys(1);
        if (0 >= group_all) clean_values(0, 0);
        stage_values(0, 0);
        load_values(1);
        stage_keys(1, 1);
        load_keys(2);
    }
    __syncthreads();

    floatx16 O[DT], x[2], y[2];  // x and y: scores of a tile, before the factor scale2 (the sign of the scale is in q)
#pragma unroll
    for (int d = 0; d < DT; ++d) O[d] = floatx16{};
    float mx = -kInf, ref = 0.f, sum = 0.f;  // ref: the maximum that O and sum are scaled by
    bf16x8 pf[NS][4];
    auto scores = [&](int buf, floatx16* z) {
        z[0] = z[1] = floatx16{};
#pragma unroll
        for (int m = 0; m < KS; ++m)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const bf16x8 k8 = __builtin_bit_cast(bf16x8, s_k[buf][half * KS + m][lane]);
#pragma unroll
                for (int p = NS - 1; p >= 0; --p)
                    z[half] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k8, qf[m][p], z[half], 0, 0, 0);
            }
    };
    // The lane's tokens that its row sees: those up to this of the first
    // half-tile's 16, up to this - 32 of the second's.
    auto see_of = [&](int32_t tile) {
        const int64_t see = sees - ((int64_t)tile * kTile + 16 * hf);
        return see < -1 ? -1 : see > 64 ? 64 : (int)see;
    };
    auto mask = [&](int32_t tile, floatx16* z) {
        const int see = see_of(tile);
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j >> 4][j & 15] = (j & 15) + 32 * (j >> 4) <= see ? z[j >> 4][j & 15] : -kInf;
    };
    auto maximum = [&](const floatx16* z) {
        float top = z[0][0];
#pragma unroll
        for (int j = 1; j < 32; ++j) top = fmaxf(top, z[j >> 4][j & 15]);
        mx = fmaxf(mx, across<Max, 32>(top) * a.scale2);
    };
    auto rescale = [&]() {
        if (__ballot(mx > ref + kSlack || (ref == 0.f && sum == 0.f))) {
            const float now = mx == -kInf ? 0.f : mx;
            // (At most 1: a row without a score yet has ref 0, whatever its maximum.
            // `sum` says nothing of that: it is of this lane's tokens, O of the row's.)
            const float fade = fminf(__builtin_amdgcn_exp2f(ref - now), 1.f);
            ref = now;
            sum *= fade;
#pragma unroll
            for (int d = 0; d < DT; ++d) O[d] *= fade;
        }
    };
    // p of the lane's scores j0 .. j1 - 1 (whole pairs)
    auto exponentials = [&](const floatx16* z, int j0, int j1) {
        const bf16x2 one = {(bf16)1.f, (bf16)1.f};
#pragma unroll
        for (int j = j0; j < j1; j += 2) {
            const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(z[j >> 4][j & 15], a.scale2, -ref)),
                        p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(z[j >> 4][(j & 15) + 1], a.scale2, -ref));
            bf16 part0[NS], part1[NS];
            split_bf16<NS>(p0, part0);
            split_bf16<NS>(p1, part1);
            // with one part, the sum is of p as it is rounded for the product
            if constexpr (NS == 1) sum = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{part0[0], part1[0]}, one, sum, false);
            else sum += p0 + p1;
#pragma unroll
            for (int q = 0; q < NS; ++q) {
                pf[q][j >> 3][j & 7] = part0[q];
                pf[q][j >> 3][(j & 7) + 1] = part1[q];
            }
        }
    };
    auto output = [&](int buf) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const bf16x8 v8 = __builtin_bit_cast(bf16x8, s_v[buf][k * DT + d][lane]);
#pragma unroll
                for (int p = NS - 1; p >= 0; --p) O[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v8, pf[p][k], O[d], 0, 0, 0);
            }
    };
    // Some value of a tile may be NaN (staged as 0): reads the codes again and
    // marks the outputs of the rows that see one.
    auto mark_nan = [&](int32_t tile, int buf) {
        int32_t nan = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) nan |= s_nan[buf][w];
        if (!__builtin_amdgcn_readfirstlane(nan)) return;
        const int64_t place = place_of(tile);
        const int see = see_of(tile);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            bf16x8 see8[2];
#pragma unroll
            for (int j = 0; j < 16; ++j) see8[j >> 3][j & 7] = (bf16)(j + 32 * half <= see ? 1.f : 0.f);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const int group = 2 * half + hf;
                uintx4 code = *reinterpret_cast<const uintx4*>(a.vc + place * DV + ((int64_t)group * DV + 32 * d + c) * 16), ones;
                keep_codes(code, job.kv - (from + (int64_t)tile * kTile + 16 * group));
                split_nan(code, ones);
                floatx16 hits = floatx16{};
                hits = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3_to_bf16x8(ones[0], ones[1]), see8[0], hits, 0, 0, 0);
                hits = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3_to_bf16x8(ones[2], ones[3]), see8[1], hits, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (hits[j] > 0.f) O[d][j] = __builtin_nanf("");
            }
        }
    };
    auto fetch_pages = [&](int32_t tile) {
        window = tile;
        pages.fetch(a, table, h, from + (int64_t)window * kTile, to, kTile, lane);
    };
    // One tile that every row sees whole, as it sees the one after it: `now` holds
    // its scores, in the maximum already; `next` receives those of the tile after
    // it.  buf: tile % 2.
    auto step = [&](int32_t tile, int buf, const floatx16* now, floatx16* next) {
        rescale();
        // The order is the one written, so that what is read ahead fits the
        // registers: a step's operands are read one step before their products.
        next[0] = next[1] = floatx16{};
        const auto key = [&](int m, int half) { return __builtin_bit_cast(bf16x8, s_k[buf ^ 1][half * KS + m][lane]); };
        bf16x8 k0 = key(0, 0), k1 = key(0, 1);
#pragma unroll
        for (int m = 0; m < KS; ++m) {
            const bf16x8 u0 = k0, u1 = k1;
            if (m + 1 < KS) {
                k0 = key(m + 1, 0);
                k1 = key(m + 1, 1);
            }
#pragma unroll
            for (int p = NS - 1; p >= 0; --p) {
                next[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(u0, qf[m][p], next[0], 0, 0, 0);
                next[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(u1, qf[m][p], next[1], 0, 0, 0);
            }
            exponentials(now, 32 / KS * m, 32 / KS * (m + 1));
            // (With 128 channels of keys the compiler's own order is 2% faster.)
            if (NS > 1 || KS < 8) __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_sched_barrier(0);
        const auto value = [&](int k, int d) { return __builtin_bit_cast(bf16x8, s_v[buf][k * DT + d][lane]); };
        bf16x8 v8[DT];
#pragma unroll
        for (int d = 0; d < DT; ++d) v8[d] = value(0, d);
        float top = -kInf;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            bf16x8 u[DT];
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                u[d] = v8[d];
                if (k < 3) v8[d] = value(k + 1, d);
            }
#pragma unroll
            for (int p = NS - 1; p >= 0; --p)
#pragma unroll
                for (int d = 0; d < DT; ++d) O[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(u[d], pf[p][k], O[d], 0, 0, 0);
#pragma unroll
            for (int j = 8 * k; j < 8 * (k + 1); ++j) top = fmaxf(top, next[j >> 4][j & 15]);
            if (k == 0) stage_values(tile + 1, buf ^ 1);
            if (k == 1) load_values(tile + 2);
            if (k == 2) stage_keys(tile + 2, buf);
            if (k == 3) load_keys(tile + 3);
            __builtin_amdgcn_sched_barrier(0);
        }
        mx = fmaxf(mx, across<Max, 32>(top) * a.scale2);
        __syncthreads();
    };
    // Any tile; the scores change in x.
    auto last_step = [&](int32_t tile, int buf) {
        if (tile + 3 >= window + 64) fetch_pages(tile);
        const bool mine = tile < wave_tiles && there(tile), more = tile + 1 < wave_tiles;
        if (mine) {
            rescale();
            exponentials(x, 0, 32);
        }
        if (more) {
            scores(buf ^ 1, x);
            if (tile + 1 >= wave_all) mask(tile + 1, x);
            if (there(tile + 1)) maximum(x);
        }
        if (mine) {
            if (tile >= group_all) mark_nan(tile, buf);
            output(buf);
        }
        if (tile + 1 < count) {
            if (tile + 1 >= group_all) clean_values(tile + 1, buf ^ 1);
            stage_values(tile + 1, buf ^ 1);
            load_values(tile + 2);
            stage_keys(tile + 2, buf);
            load_keys(tile + 3);
        }
        __syncthreads();
    };
    if (wave_tiles > 0) {
        scores(0, x);
        if (0 >= wave_all) mask(0, x);
        if (there(0)) maximum(x);
    }
    // The first scores' keys may be overwritten in the first step.
    __syncthreads();
    int32_t tile = 0;
    for (;;) {
        if (tile >= window + 60) fetch_pages(tile);
        // Pairs of steps, up to the first tile without a page or the window's end.  From
        // such a tile on the rest goes step by step, without the overlap: 2,048 tokens
        // over 16,384 (32 heads, 8 for keys, 128 channels) take 585 us, without the page
        // in the middle 622, without the first 679.
        const uint64_t gone = __ballot(pages.page < 0);
        const int32_t present = window + (gone ? __ffsll((unsigned long long)gone) - 1 : 64);
        int32_t stop = (present < group_all ? present : group_all) - 2;
        stop = stop < window + 60 ? stop : window + 60;
        if (tile >= stop) break;
        for (; tile < stop; tile += 2) {
            step(tile, 0, x, y);
            step(tile + 1, 1, y, x);
        }
    }
    for (; tile < count; ++tile) last_step(tile, tile & 1);
    sum = across<Sum, 32>(sum);
    if (__ballot(live && mx == -kInf)) {
        const bool some = sees_some(a, table, from, to, kTile, from + sees);
        if (mx == -kInf && some) sum += 1.f;
    }
    if (!live) return;
    const bool alone = job.alone();
    const float inv = alone ? reciprocal_sum(sum, mx) : 1.f;
    if (!alone && orow >= a.part_rows[1]) return;  // (with offsets that are no offsets)
    const int64_t prow = part * a.part_rows[1] + orow;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const floatx4 z = {O[d][4 * q] * inv, O[d][4 * q + 1] * inv, O[d][4 * q + 2] * inv, O[d][4 * q + 3] * inv};
            const int ch = 32 * d + 8 * q + 4 * hf;
            if (alone) store4(static_cast<TI*>(a.o) + orow * DV + ch, z);
            else *reinterpret_cast<floatx4*>(a.ws_o[1] + prow * DV + ch) = z;
        }
    if (!alone && hf == 0) {
        a.ws_ml[1][2 * prow] = mx == -kInf ? mx : ref;
        a.ws_ml[1][2 * prow + 1] = sum;
    }
}

// ---------------------------------------------------------------- joining parts
//
// W waves per row, one or four as there are few or many parts: DV / 4 lanes for
// the channels of a part, several parts side by side.
template <typename TI, int DV, bool FEW, int W>
__device__ void join_rows(const Attention& a, int32_t block) {
    constexpr int L = DV / 4, STEP = 64 * W / L, ROWS = kWaves / W;
    __shared__ floatx4 s_o[STEP * ROWS][L];
    __shared__ float s_l[STEP * ROWS], s_m[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, thread = threadIdx.x % (64 * W);
    const int64_t r = (int64_t)block * ROWS + wave / W;
    int32_t n = -1;
    int64_t orow = r;
    bool mine = r < a.part_rows[FEW ? 0 : 1];
    if (FEW) {
        n = (int32_t)(r / ((int64_t)a.Hkv * a.few_rows));
    } else if (mine) {
        const int64_t t = r / a.H;
        int32_t below = 0;
        for (int32_t n0 = 0; n0 <= a.num_seqs; n0 += 64) below += __popcll(__ballot(n0 + lane <= a.num_seqs && a.cu[n0 + lane] <= t));
        n = below - 1;
        if (n >= a.num_seqs) n = -1;  // behind the last request
    }
    int parts = 0;
    if (mine && n >= 0) {
        const Request q(a, n);
        parts = q.few == FEW && !q.alone() ? (int)((q.kv + q.chunk - 1) / q.chunk) : 0;
        if (FEW) {
            const int32_t row = (int32_t)(r % a.few_rows), h = (int32_t)(r / a.few_rows % a.Hkv), i = row / a.G;
            if (row >= q.rows) parts = 0;
            orow = (q.t0 + i) * a.H + h * a.G + (row - i * a.G);
        } else if (first_tile(a, n, 32 * kWaves) + ((r / a.H - q.t0) * a.G + r % a.H % a.G) / (32 * kWaves) >= a.tail) {
            parts = 0;
        }
    }
    if (W == kWaves && parts == 0) return;  // the whole workgroup
    const int64_t step = a.part_rows[FEW ? 0 : 1];
    const float *ml = a.ws_ml[FEW ? 0 : 1], *wo = a.ws_o[FEW ? 0 : 1];
    float m = -kInf;
    for (int s = thread; s < parts; s += 64 * W) m = fmaxf(m, ml[2 * (s * step + r)]);
    m = across<Max>(m);
    if (W > 1) {
        if (lane == 0) s_m[wave] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) m = fmaxf(m, s_m[w]);
    }
    const int c = thread % L, s0 = thread / L, at0 = wave / W * STEP;
    float l = 0.f;
    floatx4 out = zero4();
#pragma unroll 4
    for (int s = s0; s < parts; s += STEP) {
        const int64_t at = s * step + r;
        const float f = joined(ml[2 * at], m);
        l += f * ml[2 * at + 1];
        out += f * *reinterpret_cast<const floatx4*>(wo + at * DV + 4 * c);
    }
    s_o[at0 + s0][c] = out;
    if (c == 0) s_l[at0 + s0] = l;
    __syncthreads();
    if (s0 > 0 || parts == 0) return;
#pragma unroll
    for (int s = 1; s < STEP; ++s) {
        out += s_o[at0 + s][c];
        l += s_l[at0 + s];
    }
    const float inv = reciprocal_sum(l, m);
    store4(static_cast<TI*>(a.o) + orow * DV + 4 * c, out * inv);
}
// The requests of few rows, W waves to a row, and then the others: one launch,
// which is 4.5 us for either.
template <typename TI, int DV, int W>
__global__ __launch_bounds__(256) void attention_join_kernel(Attention a, int32_t few_blocks) {
    if ((int32_t)blockIdx.x < few_blocks) join_rows<TI, DV, true, W>(a, blockIdx.x);
    else join_rows<TI, DV, false, 1>(a, blockIdx.x - few_blocks);
}

// ---------------------------------------------------------------- planning

constexpr int64_t kAtOnce = 512;  // workgroups that the device holds: two on each compute unit
constexpr int64_t kTailCache = 2048;  // tokens in front of a call's last tiles, from which on they are cut

struct Plan {
    bool few, many;  // kernels that the call needs
    int32_t few_rows, splits[2], tiles, tail;
    int64_t part_rows[2];
    size_t off[4], bytes;  // ws_o and ws_ml of few, of the others
};

// The lengths are on the device, so the plan goes by sizes and bounds.  A
// request has at most max_new (or T_total) new tokens: whether that is few rows
// decides which kernels run.  A request's cache is cut into at most `splits`
// parts of at least kMinPart tokens, so that there are enough workgroups when
// every request is as long as the bound, and so that the lengths, which may
// differ much, do not leave the device waiting for a few long parts.
Plan plan(const CacheAttentionLaunch& p) {
    Plan r = {};
    auto up = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
    const int64_t room = (int64_t)p.max_blocks * p.page_size;
    const int64_t kv = p.max_kv > 0 && p.max_kv < room ? p.max_kv : room;
    const int64_t G = p.H / p.H_kv, all = p.T_total * G;
    const int64_t most = p.max_new > 0 && p.max_new < p.T_total ? p.max_new * G : all;
    r.many = most > kFewRows;
    r.few = !r.many || p.num_seqs > 1;
    r.few_rows = (int32_t)(most < kFewRows ? most : kFewRows);
    r.splits[0] = r.splits[1] = 1;
    if (r.few) {
        // From a workgroup for each compute unit on, a part for each request (32
        // requests over 4096, 256 workgroups: 44.6 us, in two parts 49.3); below,
        // enough parts to fill the device, since the lengths may differ much (23
        // over 1 to 4097, 92 units: 15.0 us with 512 at once, 18.2 with 256), none
        // below 512 tokens (with 256, 4 over 100 to 500 take 9.2 us instead of 7.0,
        // 1 over 1000 takes 9.0 instead of 9.8).  A very long request beside many
        // short ones is not waited for: at most 16384 tokens to a part (which is no cut
        // for 64 over 512 to 16384: 206 us; with 8192, 212; and one of 16384 beside 31
        // of 500 is waited for, 75 us).  For the
        // workspace's sake, not more parts than 16384 in all.
        const int64_t units = (int64_t)p.num_seqs * p.H_kv * up(r.few_rows, 16);
        int64_t splits = std::max(units >= kAtOnce / 2 ? 1 : up(kAtOnce, units), up(kv, 16384));
        splits = std::min(splits, std::min<int64_t>(up(kv, kMinPart), std::max<int64_t>(16384 / units, 1)));
        r.splits[0] = (int32_t)std::max<int64_t>(std::min<int64_t>(splits, 256), 1);
        r.part_rows[0] = (int64_t)p.num_seqs * p.H_kv * r.few_rows;
    }
    if (r.many) {
        // With fewer tiles than the device holds, all are cut (128 tokens over 32000,
        // 64 units: 83 us, with 256 at once 121 and with 1024 94.6).  Else the last
        // that start, where they would leave the device more than half empty and
        // each has a long cache before it.  2,100 tokens, 528 units, over 1024: 89.2 us
        // uncut, 92.6 cut; over 2048 134.8 and 125.1; over 8192, 176 units past 512
        // 442 and 432, 240 past it 458 and 471.  What is past a multiple of 512 goes by
        // the tiles that have rows: of one request they are known; of more they are
        // guessed, with the last tile of three requests out of four more than the full
        // ones, since too few cost more than too many (4 requests of 900 to 1,200
        // tokens over 8192, 24 units past 1024: 576 us with 24 or more cut, 653 with
        // 16).  The grid's other tiles end at once.  (The cut tiles are the batch's
        // first: behind requests of few rows, which have none, the tiles that end last
        // stay whole.)  Parts of the cut tiles come nearest to 512 (96 units: 373 us in
        // 5 parts, 381 in 6; 48: 337 in 10, 335 in 11).
        constexpr int32_t BR = 32 * kWaves;
        r.tiles = (int32_t)(all / BR + p.num_seqs);
        const int64_t full = up(all, BR), units = std::max<int64_t>(full, p.num_seqs) * p.H_kv;
        const int64_t rest = std::min<int64_t>(full + (int64_t)p.num_seqs * 3 / 4, r.tiles) * p.H_kv % kAtOnce;
        if (units < kAtOnce) r.tail = r.tiles;
        else if (rest <= kAtOnce * 3 / 8 && kv - most / G >= kTailCache) r.tail = (int32_t)up(rest, p.H_kv);
        const int64_t share = std::max<int64_t>((int64_t)r.tail * p.H_kv, 1);
        const int64_t cut = std::min(units < kAtOnce ? up(kAtOnce, units) : (kAtOnce + share / 2) / share, up(kv, kMinPart));
        if (r.tail > 0) r.splits[1] = (int32_t)std::max<int64_t>(cut, 1);
        if (r.splits[1] == 1) r.tail = 0;
        // Rows of the first `tail` tiles are among the first (tail + 1) * BR: see first_tile.
        r.part_rows[1] = std::min(p.T_total, up((int64_t)(r.tail + 1) * BR, G)) * p.H;
    }
    auto take = [&](size_t bytes) {
        const size_t at = r.bytes;
        r.bytes += (bytes + 255) & ~(size_t)255;
        return at;
    };
    for (int c = 0; c < 2; ++c)
        if (r.splits[c] > 1) {
            const size_t rows = (size_t)r.splits[c] * (size_t)r.part_rows[c];
            r.off[2 * c] = take(rows * p.dv * sizeof(float));
            r.off[2 * c + 1] = take(rows * 2 * sizeof(float));
        }
    return r;
}

template <typename TI, int DK, int DV>
hipError_t run(const Attention& a, const Plan& pl, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (pl.many) {
        const int64_t tiles = a.tiles + (int64_t)a.tail * (a.splits[1] - 1);
        hipLaunchKernelGGL((attention_tile_kernel<TI, DK, DV>), dim3((unsigned)(tiles * a.Hkv)), dim3(64 * kWaves), 0, s, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (pl.few) {
        const dim3 grid((unsigned)(a.num_seqs * ((a.few_rows + 15) / 16)), (unsigned)a.Hkv, (unsigned)a.splits[0]);
        hipLaunchKernelGGL((attention_rows_kernel<TI, DK, DV>), grid, dim3(64 * kWaves), 0, s, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const bool wide = a.splits[0] > 16;
    auto blocks = [&](int c, int at_once) { return a.splits[c] > 1 ? (a.part_rows[c] + at_once - 1) / at_once : 0; };
    const int64_t few = blocks(0, wide ? 1 : kWaves), all = few + blocks(1, kWaves);
    if (all > 0) {
        if (wide) hipLaunchKernelGGL((attention_join_kernel<TI, DV, kWaves>), dim3((unsigned)all), dim3(256), 0, s, a, (int32_t)few);
        else hipLaunchKernelGGL((attention_join_kernel<TI, DV, 1>), dim3((unsigned)all), dim3(256), 0, s, a, (int32_t)few);
        e = hipGetLastError();
    }
    return e;
}
template <typename TI>
hipError_t run_t(const Attention& a, const CacheAttentionLaunch& p, const Plan& pl, hipStream_t s) {
    if (p.dk == 128 && p.dv == 128) return run<TI, 128, 128>(a, pl, s);
    if (p.dk == 128) return run<TI, 128, 64>(a, pl, s);
    if (p.dv == 128) return run<TI, 64, 128>(a, pl, s);
    return run<TI, 64, 64>(a, pl, s);
}

}  // namespace

size_t cache_attention_workspace_bytes(const CacheAttentionLaunch& p) { return plan(p).bytes; }

hipError_t launch_cache_attention(const CacheAttentionLaunch& p, hipStream_t s) {
    if (p.T_total == 0 || p.num_seqs == 0) return hipSuccess;
    const Plan pl = plan(p);
    Attention a = {};
    a.q = p.q; a.kc = p.k_cache; a.vc = p.v_cache; a.ks = p.k_scale; a.vs = p.v_scale;
    a.table = p.block_table; a.rows = p.rows; a.kv_lens = p.kv_lens; a.cu = p.cu_seqlens;
    a.num_seqs = p.num_seqs; a.T = p.T_total; a.num_pages = (int32_t)p.num_pages;
    a.page_log2 = p.page_size == 64 ? 6 : p.page_size == 128 ? 7 : 8;
    a.num_rows = p.num_rows; a.max_blocks = p.max_blocks;
    // Scale 0 stands for the smallest factor: scores of masked tokens stay -Inf.
    a.scale2 = std::max(std::fabs(p.scale) * kLog2e, std::numeric_limits<float>::min());
    a.negative = p.scale < 0.f;
    a.o = p.o; a.H = p.H; a.Hkv = p.H_kv; a.G = p.H / p.H_kv;
    a.few_rows = pl.few_rows;
    a.tiled = pl.many;
    a.tiles = pl.tiles;
    a.tail = pl.tail;
    for (int c = 0; c < 2; ++c) {
        a.splits[c] = pl.splits[c];
        a.part_rows[c] = pl.part_rows[c];
        a.ws_o[c] = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + pl.off[2 * c]);
        a.ws_ml[c] = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + pl.off[2 * c + 1]);
    }
    if (!pl.few) a.few_rows = 0;  // every request goes to the tile kernel
    return p.bf16 ? run_t<bf16>(a, p, pl, s) : run_t<float>(a, p, pl, s);
}

}  // namespace gdn
