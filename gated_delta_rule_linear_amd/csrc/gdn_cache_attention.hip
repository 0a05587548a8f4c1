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
// matrix cores.  Where rows are few in all, a request's cache is cut into parts
// that workgroups take side by side and attention_join_kernel joins.
//
// Scores are formed transposed, S^T = K Q^T, so that a lane holds scores of one
// row and the softmax statistics of a row are scalars of its lanes, and so that
// a lane's scores are those of 16 neighbouring tokens: K's rows are handed to the
// matrix core in the order that makes them so.  They are then, rounded to bf16,
// the operand that the second product O^T = V^T P^T takes from that lane.  Its
// other operand, V^T, is 16 tokens of one channel: one 16-byte load of the cache
// as it is stored.  Codes are converted to bf16 exactly, and a page's scale, a
// power of two, is applied exactly, to the scores and p or in the conversion.
#include "gdn_e4m3.h"
#include "gdn_mfma.h"
#include "gdn_serve_kernels.h"

namespace gdn {
namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));

constexpr int kTile = 64;      // tokens of a tile
constexpr int kFewRows = 32;   // requests with up to so many rows go to the rows kernel
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
    float scale2;  // scale * log2(e): scores in units of log 2
    void* o;
    int32_t H, Hkv, G;
    int32_t splits, min_chunk;
    int64_t more_rows, most_rows;  // a kernel takes the requests with more_rows < rows <= most_rows
    float* ws_o;   // [splits][T * H][d_v]
    float* ws_ml;  // [splits][T * H][2]: maximum and sum
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
// A request's cache is cut into parts of `chunk` tokens (a multiple of kTile).
__device__ __forceinline__ int64_t chunk_of(const Attention& a, int64_t kv) {
    const int64_t c = ((kv + a.splits - 1) / a.splits + kTile - 1) / kTile * kTile;
    return c > a.min_chunk ? c : a.min_chunk;
}
__device__ __forceinline__ int64_t held_tokens(const Attention& a, int32_t n) {
    const int64_t most = (int64_t)a.max_blocks << a.page_log2, kv = a.kv_lens[n];
    return kv < 0 ? 0 : kv < most ? kv : most;
}

// What a workgroup works on: rows row0 .. of request n and key/value head h, in
// part z of its cache.
struct Job {
    int64_t t0, len, kv, row0, rows;  // first token, tokens, held tokens, first row, rows of the request
    int64_t from, to;                 // tokens of the part that some row of the tile sees
    int64_t all_see;                  // every row of the tile sees the tokens up to this one
    const int32_t* table;             // the request's row, null: it has none
    bool alone;                       // the request's cache is one part
};
template <int BR>
__device__ __forceinline__ bool find_job(const Attention& a, int64_t tile, int z, Job& j) {
    const int32_t n = request_of(a, tile, BR);
    if (n < 0) return false;
    int64_t t1 = a.cu[n + 1];
    j.t0 = a.cu[n];
    j.row0 = (tile - first_tile(a, n, BR)) * BR;
    j.t0 = j.t0 < 0 ? 0 : j.t0;
    t1 = t1 < a.T ? t1 : a.T;
    j.len = t1 - j.t0;
    j.rows = j.len * a.G;
    if (j.len <= 0 || j.row0 < 0 || j.row0 >= j.rows || j.rows <= a.more_rows || j.rows > a.most_rows) return false;
    j.kv = held_tokens(a, n);
    const int64_t chunk = chunk_of(a, j.kv);
    j.from = z * chunk;
    if (z > 0 && j.from >= j.kv) return false;
    j.alone = j.kv <= chunk;
    const int64_t last = j.row0 + BR < j.rows ? j.row0 + BR - 1 : j.rows - 1;
    j.to = j.kv - j.len + last / a.G + 1;
    j.to = j.to < j.from + chunk ? j.to : j.from + chunk;
    j.all_see = j.kv - j.len + j.row0 / a.G;
    const int32_t row = a.rows ? a.rows[n] : n;
    j.table = row >= 0 && row < a.num_rows ? a.table + (int64_t)row * a.max_blocks : nullptr;
    return true;
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

template <typename TI>
__device__ __forceinline__ void store4(TI* p, floatx4 x) {
    if constexpr (sizeof(TI) == 4) *reinterpret_cast<floatx4*>(p) = x;
    else *reinterpret_cast<bf16x4*>(p) = bf16x4{(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]};
}

constexpr int kWaves = 4;
#ifndef ROWS_OCC
#define ROWS_OCC 2
#endif

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
template <typename TI, int DK, int DV>
__global__ __launch_bounds__(64 * kWaves, ROWS_OCC) void attention_rows_kernel(Attention a) {
    constexpr int NS = sizeof(TI) == 4 ? 3 : 1;
    constexpr int BR = 16, KS = DK / 32, VT = DV / 16;
    __shared__ float s_o[kWaves][BR][DV + 4];
    __shared__ float s_m[kWaves][BR], s_l[kWaves][BR];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, g = lane >> 4;
    const int h = blockIdx.y;
    Job job;
    if (!find_job<BR>(a, blockIdx.x, blockIdx.z, job)) return;
    const int page_mask = (1 << a.page_log2) - 1;

    uintx4 kr[4][DK / 64], vr[VT];
    int32_t page = -1, next_page = -1;  // of the tile in kr and vr, and of the one after it
    float ks = 0.f, vs = 0.f;           // of the tile in kr and vr
    auto page_of = [&](int64_t base) -> int32_t {
        if (!job.table || base >= job.to) return -1;
        const int32_t p = __builtin_amdgcn_readfirstlane(job.table[base >> a.page_log2]);
        return p < a.num_pages ? p : -1;  // negative entries stay so: left out
    };
    auto load_keys = [&](int64_t base, int32_t p) {
        if (p < 0) return;
        const int64_t ph = (int64_t)p * a.Hkv + h;
        const uint8_t* at = a.kc + ((ph << a.page_log2) + (base & page_mask)) * DK + (16 * (r >> 2) + (r & 3)) * DK + 16 * g;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < DK / 64; ++j) kr[c][j] = *reinterpret_cast<const uintx4*>(at + 4 * c * DK + 64 * j);
        ks = a.ks[ph];
    };
    auto load_values = [&](int64_t base, int32_t p) {
        if (p < 0) return;
        const int64_t ph = (int64_t)p * a.Hkv + h;
        const uint8_t* at = a.vc + ((ph << a.page_log2) + (base & page_mask)) * DV + (g * DV + r) * 16;
#pragma unroll
        for (int d = 0; d < VT; ++d) vr[d] = *reinterpret_cast<const uintx4*>(at + d * 256);
        vs = a.vs[ph];
    };
    constexpr int STEP = kWaves * kTile;
    const int64_t first = job.from + wave * kTile;
    page = page_of(first);
    next_page = page_of(first + STEP);
    load_keys(first, page);
    load_values(first, page);

    // this lane's row
    const int64_t row = job.row0 + r;
    const bool live = row < job.rows;
    const int64_t i = live ? row / a.G : 0;
    const int32_t head = h * a.G + (int32_t)(live ? row - i * a.G : 0);
    const int64_t sees = live ? job.kv - job.len + i : -1;  // the last token that the row sees
    bf16x8 qf[NS][KS];
    {
        const TI* q = static_cast<const TI*>(a.q) + ((job.t0 + i) * a.H + head) * DK + 16 * g;
#pragma unroll
        for (int m = 0; m < KS; ++m)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                bf16 part[NS];
                split_bf16<NS>(live ? to_f32(q[64 * (m >> 1) + 8 * (m & 1) + j]) : 0.f, part);
#pragma unroll
                for (int s = 0; s < NS; ++s) qf[s][m][j] = part[s];
            }
    }

    floatx4 O[VT];
#pragma unroll
    for (int d = 0; d < VT; ++d) O[d] = zero4();
    float mx = -kInf, sum = 0.f;
    for (int64_t base = first; base < job.to; base += STEP) {
        const bool there = page >= 0;
        float s[16];
        if (there) {
            const float c2 = ks * a.scale2;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                floatx4 x = zero4();
#pragma unroll
                for (int m = 0; m < KS; ++m) {
                    const bf16x8 k8 = e4m3_to_bf16x8(kr[c][m >> 1][2 * (m & 1)], kr[c][m >> 1][2 * (m & 1) + 1]);
#pragma unroll
                    for (int p = NS - 1; p >= 0; --p) x = Mma<bf16>::mma(k8, qf[p][m], x);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) s[4 * c + j] = x[j] * c2;
            }
        }
        load_keys(base + STEP, next_page);
        if (there) {
            const bool edge = base + kTile - 1 > job.all_see;  // some row does not see all of the tile
            const int64_t see = sees - (base + 16 * g);
            if (edge) {
#pragma unroll
                for (int j = 0; j < 16; ++j) s[j] = j <= see ? s[j] : -kInf;
            }
            float top = s[0];
#pragma unroll
            for (int j = 1; j < 16; ++j) top = fmaxf(top, s[j]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
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
        load_values(base + STEP, next_page);
        page = next_page;
        next_page = page_of(base + 2 * STEP);
    }
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
#pragma unroll
    for (int d = 0; d < VT; ++d) *reinterpret_cast<floatx4*>(&s_o[wave][r][16 * d + 4 * g]) = O[d];
    if (g == 0) {
        s_m[wave][r] = mx;
        s_l[wave][r] = sum;
    }
    __syncthreads();
    // Join the waves: a thread takes DV / 16 channels of one row.
    constexpr int C = DV / 16;
    const int jr = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * C;
    if (job.row0 + jr >= job.rows) return;
    float m = s_m[0][jr];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, s_m[w][jr]);
    const float ref = m == -kInf ? 0.f : m;
    float l = 0.f, out[C];
#pragma unroll
    for (int c = 0; c < C; ++c) out[c] = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(s_m[w][jr] - ref);
        l += f * s_l[w][jr];
#pragma unroll
        for (int c = 0; c < C; ++c) out[c] += f * s_o[w][jr][c0 + c];
    }
    const int64_t ji = (job.row0 + jr) / a.G;
    const int64_t orow = (job.t0 + ji) * a.H + h * a.G + (job.row0 + jr - ji * a.G);
    if (job.alone) {
        const float inv = l == 0.f && m == -kInf ? 0.f : 1.f / l;
#pragma unroll
        for (int c = 0; c < C; c += 4)
            store4(static_cast<TI*>(a.o) + orow * DV + c0 + c,
                   floatx4{out[c] * inv, out[c + 1] * inv, out[c + 2] * inv, out[c + 3] * inv});
        return;
    }
    const int64_t at = blockIdx.z * (a.T * a.H) + orow;
#pragma unroll
    for (int c = 0; c < C; c += 4)
        *reinterpret_cast<floatx4*>(a.ws_o + at * DV + c0 + c) = floatx4{out[c], out[c + 1], out[c + 2], out[c + 3]};
    if (c0 == 0) {
        a.ws_ml[2 * at] = m;
        a.ws_ml[2 * at + 1] = l;
    }
}

// ---------------------------------------------------------------- many rows
//
// One workgroup: 32 rows for each of its waves.  The waves read the same keys
// and values, so a tile's codes are converted once, by all of them, and staged
// in LDS as bf16 in the order in which the matrix core takes them: a fragment is
// 64 lanes x 16 bytes, read without conflicts.  Two tiles are held: while one is
// worked on, the next is written and the one after it is on its way to
// registers, with one barrier per tile.
//
// 32x32x16 products (lane l: c = l % 32, hf = l / 32; a result has rows
// 8 q + 4 hf + i, q and i 0..3): row 8 q + 4 hf + i of K's half-tile is token
// 16 hf + 4 q + i, so that a lane's 16 scores of a half-tile are those of tokens
// 16 hf .. 16 hf + 15.
//
// Rescaling the output for a new maximum is put off while the maximum has grown
// by at most 2^8: p stays below 2^8, its sum is in fp32, and its rounding to
// bf16 is relative.
template <typename TI, int DK, int DV>
__global__ __launch_bounds__(64 * kWaves, sizeof(TI) == 4 ? 1 : 2) void attention_tile_kernel(Attention a) {
    constexpr int NS = sizeof(TI) == 4 ? 3 : 1;
    constexpr int BR = 32 * kWaves, KS = DK / 16, DT = DV / 32;
    constexpr float kSlack = 8.f;
    __shared__ uintx4 s_k[2][2 * KS][64];      // [buffer][half-tile * KS + step][lane ^ step % 8]
    __shared__ uintx4 s_v[2][2 * 2 * DT][64];  // [buffer][(half-tile * 2 + step) * DT + channels][lane]
    __shared__ int32_t s_nan[2], s_there[2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 31, hf = lane >> 5;
    // Key/value heads are neighbours in the grid: workgroups go to the eight XCDs in
    // turn, so with eight heads the tiles of a head share one XCD's cache.  The
    // last rows, which see most, come first.
    const int h = blockIdx.x % a.Hkv;
    const int64_t id = blockIdx.x / a.Hkv, tiles = gridDim.x / a.Hkv;
    Job job;
    if (!find_job<BR>(a, tiles - 1 - id, blockIdx.y, job)) return;
    const int page_mask = (1 << a.page_log2) - 1;

    // Staging: a thread takes 16-byte pieces of keys (a token's 16 channels) and
    // of values (a channel's 16 tokens).
    constexpr int NT = 64 * kWaves, KP = kTile * DK / 16 / NT, VP = kTile * DV / 16 / NT;
    uintx4 kr[KP], vr[VP];
    float ks = 0.f, vs = 0.f;
    int32_t page = -1;  // of the tile in kr and vr
    auto page_of = [&](int64_t base) -> int32_t {
        if (!job.table || base >= job.to) return -1;
        const int32_t p = __builtin_amdgcn_readfirstlane(job.table[base >> a.page_log2]);
        return p < a.num_pages ? p : -1;
    };
    auto load = [&](int64_t base, int32_t p) {
        page = p;
        if (p < 0) return;
        const int64_t ph = (int64_t)p * a.Hkv + h, place = (ph << a.page_log2) + (base & page_mask);
        const uintx4* k = reinterpret_cast<const uintx4*>(a.kc + place * DK) + threadIdx.x;
        const uintx4* v = reinterpret_cast<const uintx4*>(a.vc + place * DV) + threadIdx.x;
#pragma unroll
        for (int j = 0; j < KP; ++j) kr[j] = k[j * NT];
#pragma unroll
        for (int j = 0; j < VP; ++j) vr[j] = v[j * NT];
        ks = a.ks[ph];
        vs = a.vs[ph];
    };
    auto stage = [&](int64_t base, int buf) {
        if (threadIdx.x == 0) s_there[buf] = page >= 0;
        if (page < 0) return;
#pragma unroll
        for (int j = 0; j < KP; ++j) {
            const int piece = threadIdx.x + j * NT, token = piece / KS, step = piece % KS;
            const int t = token & 31, row = 8 * ((t >> 2) & 3) + 4 * (t >> 4) + (t & 3);
            uintx4* to = s_k[buf][(token >> 5) * KS + step];
            to[row ^ (step & 7)] = __builtin_bit_cast(uintx4, e4m3_to_bf16x8(kr[j][0], kr[j][1], ks));
            to[(row + 32) ^ (step & 7)] = __builtin_bit_cast(uintx4, e4m3_to_bf16x8(kr[j][2], kr[j][3], ks));
        }
        const bool edge = base + kTile - 1 > job.all_see;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < VP; ++j) {
            const int piece = threadIdx.x + j * NT, group = piece / DV, d = piece % DV;
            if (edge) {
                // as in the rows kernel: codes behind the last token, and NaN codes
                uintx4 ones;
                keep_codes(vr[j], job.kv - (base + 16 * group));
                nan |= has_nan_code(vr[j]);
                split_nan(vr[j], ones);
            }
            const int half = group >> 1, at = 32 * (group & 1) + (d & 31);
            s_v[buf][(half * 2 + 0) * DT + d / 32][at] = __builtin_bit_cast(uintx4, e4m3_to_bf16x8(vr[j][0], vr[j][1], vs));
            s_v[buf][(half * 2 + 1) * DT + d / 32][at] = __builtin_bit_cast(uintx4, e4m3_to_bf16x8(vr[j][2], vr[j][3], vs));
        }
        if (nan) s_nan[buf] = 1;
    };

    int32_t next_page = page_of(job.from + kTile);
    load(job.from, page_of(job.from));

    // this lane's row
    const int64_t row = job.row0 + 32 * wave + c;
    const bool live = row < job.rows;
    const int64_t i = live ? row / a.G : 0;
    const int32_t head = h * a.G + (int32_t)(live ? row - i * a.G : 0);
    const int64_t sees = live ? job.kv - job.len + i : -1;
    const int64_t orow = (job.t0 + i) * a.H + head;
    // Tokens that some row of this wave sees end here; before all_see every row does.
    const int64_t wrow = job.row0 + 32 * wave, wlast = wrow + 31 < job.rows ? wrow + 31 : job.rows - 1;
    const int64_t wave_to = wrow < job.rows ? job.kv - job.len + wlast / a.G + 1 : 0;
    const int64_t wave_all = job.kv - job.len + (wrow < job.rows ? wrow : 0) / a.G;
    bf16x8 qf[NS][KS];
    {
        const TI* q = static_cast<const TI*>(a.q) + orow * DK + 8 * hf;
#pragma unroll
        for (int m = 0; m < KS; ++m)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                bf16 part[NS];
                split_bf16<NS>(live ? to_f32(q[16 * m + j]) : 0.f, part);
#pragma unroll
                for (int s = 0; s < NS; ++s) qf[s][m][j] = part[s];
            }
    }

    floatx16 O[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) O[d] = floatx16{};
    float mx = -kInf, ref = 0.f, sum = 0.f;  // ref: the maximum that O and sum are scaled by
    if (threadIdx.x < 2) s_nan[threadIdx.x] = 0;
    __syncthreads();
    stage(job.from, 0);
    load(job.from + kTile, next_page);
    next_page = page_of(job.from + 2 * kTile);
    __syncthreads();
    int buf = 0;
    for (int64_t base = job.from; base < job.to; base += kTile, buf ^= 1) {
        if (s_there[buf] && base < wave_to) {
            float s[32];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                floatx16 x = floatx16{};
#pragma unroll
                for (int m = 0; m < KS; ++m) {
                    const bf16x8 k8 = __builtin_bit_cast(bf16x8, s_k[buf][half * KS + m][lane ^ (m & 7)]);
#pragma unroll
                    for (int p = NS - 1; p >= 0; --p) x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k8, qf[p][m], x, 0, 0, 0);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) s[16 * half + j] = x[j] * a.scale2;
            }
            const bool edge = base + kTile - 1 > wave_all;
            const int64_t see = sees - (base + 16 * hf);  // of the first half-tile's tokens; the second's are 32 further
            if (edge) {
#pragma unroll
                for (int j = 0; j < 32; ++j) s[j] = (j & 15) + 32 * (j >> 4) <= see ? s[j] : -kInf;
            }
            float top = s[0];
#pragma unroll
            for (int j = 1; j < 32; ++j) top = fmaxf(top, s[j]);
            top = fmaxf(top, __shfl_xor(top, 32));
            mx = fmaxf(mx, top);
            if (__ballot(mx > ref + kSlack || (ref == 0.f && sum == 0.f))) {
                const float now = mx == -kInf ? 0.f : mx;
                const float fade = sum == 0.f ? 1.f : __builtin_amdgcn_exp2f(ref - now);
                ref = now;
                sum *= fade;
#pragma unroll
                for (int d = 0; d < DT; ++d) O[d] *= fade;
            }
            bf16x8 pf[NS][4];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float p = __builtin_amdgcn_exp2f(s[j] - ref);
                sum += p;
                bf16 part[NS];
                split_bf16<NS>(p, part);
#pragma unroll
                for (int q = 0; q < NS; ++q) pf[q][j >> 3][j & 7] = part[q];
            }
            if (s_nan[buf]) {
                // Some value of the tile is NaN (staged as 0): read the codes again
                // and mark the outputs of the rows that see one.
                const int32_t pg = job.table[base >> a.page_log2];
                const int64_t place = (((int64_t)pg * a.Hkv + h) << a.page_log2) + (base & page_mask);
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    bf16x8 see8[2];
#pragma unroll
                    for (int j = 0; j < 16; ++j) see8[j >> 3][j & 7] = (bf16)(j + 32 * half <= see ? 1.f : 0.f);
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        const int group = 2 * half + hf;
                        uintx4 code = *reinterpret_cast<const uintx4*>(a.vc + place * DV + ((int64_t)group * DV + 32 * d + c) * 16), ones;
                        keep_codes(code, job.kv - (base + 16 * group));
                        split_nan(code, ones);
                        floatx16 hits = floatx16{};
                        hits = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3_to_bf16x8(ones[0], ones[1]), see8[0], hits, 0, 0, 0);
                        hits = __builtin_amdgcn_mfma_f32_32x32x16_bf16(e4m3_to_bf16x8(ones[2], ones[3]), see8[1], hits, 0, 0, 0);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (hits[j] > 0.f) O[d][j] = __builtin_nanf("");
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const bf16x8 v8 = __builtin_bit_cast(bf16x8, s_v[buf][k * DT + d][lane]);
#pragma unroll
                    for (int p = NS - 1; p >= 0; --p) O[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v8, pf[p][k], O[d], 0, 0, 0);
                }
        }
        if (base + kTile < job.to) {
            // The other buffer's readers have met at the last barrier.
            if (threadIdx.x == 0) s_nan[buf ^ 1] = 0;
            const bool may_be_nan = base + 2 * kTile - 1 > job.all_see;
            if (may_be_nan) __syncthreads();  // the flag is cleared before it is set
            stage(base + kTile, buf ^ 1);
            load(base + 2 * kTile, next_page);
            next_page = page_of(base + 3 * kTile);
            __syncthreads();
        }
    }
    sum += __shfl_xor(sum, 32);
    if (!live) return;
    const float inv = !job.alone ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
    const int64_t at = blockIdx.y * (a.T * a.H) + orow;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const floatx4 x = {O[d][4 * q] * inv, O[d][4 * q + 1] * inv, O[d][4 * q + 2] * inv, O[d][4 * q + 3] * inv};
            const int ch = 32 * d + 8 * q + 4 * hf;
            if (job.alone) store4(static_cast<TI*>(a.o) + orow * DV + ch, x);
            else *reinterpret_cast<floatx4*>(a.ws_o + at * DV + ch) = x;
        }
    if (!job.alone && hf == 0) {
        a.ws_ml[2 * at] = sum == 0.f ? -kInf : ref;
        a.ws_ml[2 * at + 1] = sum;
    }
}

// ---------------------------------------------------------------- joining parts
//
// A workgroup per row: DV / 4 threads for the channels of a part, several parts
// side by side.
template <typename TI, int DV>
__global__ __launch_bounds__(256) void attention_join_kernel(Attention a) {
    constexpr int L = DV / 4, STEP = 256 / L;
    __shared__ floatx4 s_o[STEP][L];
    __shared__ float s_l[STEP], s_m[4];
    const int lane = threadIdx.x & 63;
    const int64_t row = blockIdx.x, t = row / a.H;
    int32_t below = 0;
    bool in = false;
    for (int32_t n0 = 0; n0 <= a.num_seqs; n0 += 64) {
        const int32_t n = n0 + lane;
        const bool on = n <= a.num_seqs && a.cu[n] <= t;
        below += __popcll(__ballot(on && n < a.num_seqs));
        in |= __ballot(on && n == a.num_seqs) != 0;
    }
    const int32_t n = below - 1;
    if (in || n < 0) return;  // behind the last request
    const int64_t kv = held_tokens(a, n), chunk = chunk_of(a, kv);
    if (kv <= chunk) return;  // written by its one workgroup
    const int parts = (int)((kv + chunk - 1) / chunk);
    const int64_t step = a.T * a.H;
    float m = -kInf;
    for (int s = threadIdx.x; s < parts; s += 256) m = fmaxf(m, a.ws_ml[2 * (s * step + row)]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    if (lane == 0) s_m[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    const float ref = m == -kInf ? 0.f : m;
    const int c = threadIdx.x % L, s0 = threadIdx.x / L;
    float l = 0.f;
    floatx4 out = zero4();
#pragma unroll 4
    for (int s = s0; s < parts; s += STEP) {
        const int64_t at = s * step + row;
        const float f = __builtin_amdgcn_exp2f(a.ws_ml[2 * at] - ref);
        l += f * a.ws_ml[2 * at + 1];
        out += f * *reinterpret_cast<const floatx4*>(a.ws_o + at * DV + 4 * c);
    }
    s_o[s0][c] = out;
    if (c == 0) s_l[s0] = l;
    __syncthreads();
    if (s0 > 0) return;
#pragma unroll
    for (int s = 1; s < STEP; ++s) {
        out += s_o[s][c];
        l += s_l[s];
    }
    const float inv = l == 0.f && m == -kInf ? 0.f : 1.f / l;
    store4(static_cast<TI*>(a.o) + row * DV + 4 * c, out * inv);
}

// ---------------------------------------------------------------- planning

struct Plan {
    bool few, many;  // kernels that the call needs
    int32_t splits, min_chunk;
    size_t ml_off, bytes;
};

// The lengths are on the device, so the plan goes by sizes and bounds.  A
// request has at most max_new (or T_total) new tokens: whether that is few rows
// decides which kernels run.  Each request's cache is cut into at most `splits`
// parts of at least min_chunk tokens: enough of them to fill the device when
// every request is as long as the bound, and, for few rows, so that no part of
// the longest request is above 8192 tokens.
Plan plan(const CacheAttentionLaunch& p) {
    Plan r = {};
    const int64_t room = (int64_t)p.max_blocks * p.page_size;
    const int64_t kv = p.max_kv > 0 && p.max_kv < room ? p.max_kv : room;
    const int64_t G = p.H / p.H_kv, all = p.T_total * G;
    const int64_t most = p.max_new > 0 && p.max_new < p.T_total ? p.max_new * G : all;
    r.many = most > kFewRows;
    r.few = !r.many || p.num_seqs > 1;
    const int64_t per = r.many ? 32 * kWaves : 16, target = r.many ? 512 : 1024;
    const int64_t tiles = (all + per - 1) / per > p.num_seqs ? (all + per - 1) / per : p.num_seqs;
    const int64_t units = tiles * p.H_kv;
    int64_t splits = units >= target ? 1 : (target + units - 1) / units;
    r.min_chunk = units >= target ? 8192 : r.many ? 512 : 256;
    if (r.few && splits < (kv + 8191) / 8192) splits = (kv + 8191) / 8192;
    if (splits > (kv + r.min_chunk - 1) / r.min_chunk) splits = (kv + r.min_chunk - 1) / r.min_chunk;
    if (splits < 1) splits = 1;
    if (splits > 256) splits = 256;
    r.splits = (int32_t)splits;
    if (splits > 1) {
        const size_t rows = (size_t)splits * p.T_total * p.H;
        r.ml_off = (rows * p.dv * sizeof(float) + 255) & ~(size_t)255;
        r.bytes = r.ml_off + ((rows * 2 * sizeof(float) + 255) & ~(size_t)255);
    }
    return r;
}

template <typename TI, int DK, int DV>
hipError_t run(Attention a, const Plan& pl, hipStream_t s) {
    const int64_t all = a.T * a.G;
    if (pl.many) {
        a.more_rows = pl.few ? kFewRows : 0;
        a.most_rows = INT64_MAX;
        const int64_t tiles = all / (32 * kWaves) + a.num_seqs;
        hipLaunchKernelGGL((attention_tile_kernel<TI, DK, DV>), dim3((unsigned)(tiles * a.Hkv), (unsigned)a.splits),
                           dim3(64 * kWaves), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (pl.few) {
        a.more_rows = 0;
        a.most_rows = pl.many ? kFewRows : INT64_MAX;
        const int64_t tiles = all / 16 + a.num_seqs;
        hipLaunchKernelGGL((attention_rows_kernel<TI, DK, DV>), dim3((unsigned)tiles, (unsigned)a.Hkv, (unsigned)a.splits),
                           dim3(64 * kWaves), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.splits == 1) return hipSuccess;
    hipLaunchKernelGGL((attention_join_kernel<TI, DV>), dim3((unsigned)(a.T * a.H)), dim3(256), 0, s, a);
    return hipGetLastError();
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
    a.scale2 = p.scale * kLog2e; a.o = p.o; a.H = p.H; a.Hkv = p.H_kv; a.G = p.H / p.H_kv;
    a.splits = pl.splits; a.min_chunk = pl.min_chunk;
    a.ws_o = static_cast<float*>(p.workspace);
    a.ws_ml = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + pl.ml_off);
    return p.bf16 ? run_t<bf16>(a, p, pl, s) : run_t<float>(a, p, pl, s);
}

}  // namespace gdn
