// Causal attention of a step's new tokens over the paged e4m3 cache
// (gdn_cache_attention).
//
// The query heads of one key/value head read the same keys, so the rows of a
// product are the (new token, query head of the group) pairs of one request and
// key/value head, flattened: row = token * G + head of the group.  A workgroup
// takes a tile of them and walks the cache in tiles of 64 tokens with the
// running maximum and sum of the softmax.
//
// Matrix-core layout (16x16x32 bf16; lane l: r = l % 16, g = l / 16).  Scores
// are formed transposed, S^T = K Q^T, so that a lane holds scores of one row of
// the tile (its r) and the softmax statistics of a row are scalars of its lanes.
// Row a of K's tile t (t = 0..3) is token 16 (a / 4) + 4 t + a % 4, so that a
// lane's scores of the four tiles are those of 16 neighbouring tokens,
// 16 g .. 16 g + 15: the operand that the second product O^T = V^T P^T takes
// from the lane.  Its other operand, V^T, is 16 tokens of one channel: one
// 16-byte load of the cache as it is stored.  The codes are converted to bf16
// (exactly) between the load and the product; the page's scales are powers of
// two and multiply the scores and p.
#include "gdn_e4m3.h"
#include "gdn_mfma.h"
#include "gdn_serve_kernels.h"

namespace gdn {
namespace {

constexpr int kTile = 64;  // tokens of a tile
constexpr float kLog2e = 1.4426950408889634f;

struct Attention {
    const void* q;
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table, *rows, *kv_lens, *cu;
    int32_t num_seqs;
    int64_t T, num_pages;
    int32_t page, num_rows, max_blocks;
    float scale2;  // scale * log2(e): scores in units of log 2
    void* o;
    int32_t H, Hkv, G;
    int32_t splits, min_chunk;
    float* ws_o;   // [splits][T * H][d_v]
    float* ws_ml;  // [splits][T * H][2]: maximum and sum
};

// Tiles of BR rows that the requests before n take at most: the tiles of
// request n start here.  (With rows cu G: floor(x / BR) grows by at least
// ceil(len / BR) - 1 over len rows.)
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
    const int64_t most = (int64_t)a.max_blocks * a.page, kv = a.kv_lens[n];
    return kv < 0 ? 0 : kv < most ? kv : most;
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

__device__ __forceinline__ bool has_nan_code(uintx4 x) {
    uint32_t hit = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) hit |= (((x[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u);
    return hit != 0;
}
// 1 for a NaN code, 0 for the others, and the codes with 0 in the place of NaN.
__device__ __forceinline__ void split_nan(uint32_t& x, uint32_t& ones) {
    const uint32_t hit = (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
    x &= ~(hit * 0xffu);
    ones = hit * 0x38u;  // e4m3 code of 1
}

constexpr int kWaves = 4;

// One workgroup: 16 rows, one part of the cache; its waves take the part's
// tiles in turn, each with statistics of its own, and are joined at the end.
template <typename TI, int DK, int DV>
__global__ __launch_bounds__(64 * kWaves) void attention_rows_kernel(Attention a) {
    constexpr int NS = sizeof(TI) == 4 ? 3 : 1;
    constexpr int BR = 16, KS = DK / 32, VT = DV / 16;
    __shared__ float s_o[kWaves][BR][DV + 4];
    __shared__ float s_m[kWaves][BR], s_l[kWaves][BR];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int h = blockIdx.y;
    const int32_t n = request_of(a, blockIdx.x, BR);
    if (n < 0) return;
    int64_t t0 = a.cu[n], t1 = a.cu[n + 1];
    t0 = t0 < 0 ? 0 : t0;
    t1 = t1 < a.T ? t1 : a.T;
    const int64_t len = t1 - t0, row0 = (blockIdx.x - first_tile(a, n, BR)) * BR;
    if (len <= 0 || row0 < 0 || row0 >= len * a.G) return;
    const int64_t kv = held_tokens(a, n), chunk = chunk_of(a, kv);
    const int64_t from = blockIdx.z * chunk;
    if (blockIdx.z > 0 && from >= kv) return;
    const bool alone = kv <= chunk;
    // this lane's row
    const int64_t row = row0 + r;
    const bool live = row < len * a.G;
    const int64_t i = live ? row / a.G : 0;
    const int64_t t = t0 + i;
    const int32_t head = h * a.G + (int32_t)(live ? row - i * a.G : 0);
    const int64_t sees = live ? kv - len + i : -1;  // the last token that the row sees
    const int64_t last_row = row0 + BR < len * a.G ? row0 + BR - 1 : len * a.G - 1;
    int64_t to = kv - len + last_row / a.G + 1;  // no row of the tile sees more
    to = to < from + chunk ? to : from + chunk;
    const int64_t all_see = kv - len + row0 / a.G;  // every row sees up to here

    bf16x8 qf[NS][KS];
    {
        const TI* q = static_cast<const TI*>(a.q) + (t * a.H + head) * DK + 16 * g;
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
    const int32_t trow = a.rows ? a.rows[n] : n;
    const bool has_row = trow >= 0 && trow < a.num_rows;
    const int32_t* table = a.table + (int64_t)(has_row ? trow : 0) * a.max_blocks;

    floatx4 O[VT];
#pragma unroll
    for (int d = 0; d < VT; ++d) O[d] = zero4();
    float mx = -__builtin_inff(), sum = 0.f;
    for (int64_t base = from + wave * kTile; has_row && base < to; base += kWaves * kTile) {
        const int64_t block = base / a.page;
        const int32_t pg = table[block];
        if (pg < 0 || pg >= a.num_pages) continue;  // left out
        const int place = (int)(base - block * a.page);
        const int64_t ph = (int64_t)pg * a.Hkv + h;
        const uint8_t* kp = a.kc + (ph * a.page + place) * DK + (16 * (r >> 2) + (r & 3)) * DK + 16 * g;
        const uint8_t* vp = a.vc + (ph * a.page + place) * DV + (g * DV + r) * 16;
        uintx4 kr[4][DK / 64], vr[VT];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < DK / 64; ++j) kr[c][j] = *reinterpret_cast<const uintx4*>(kp + 4 * c * DK + 64 * j);
#pragma unroll
        for (int d = 0; d < VT; ++d) vr[d] = *reinterpret_cast<const uintx4*>(vp + d * 256);
        const float ks = a.ks[ph] * a.scale2, vs = a.vs[ph];

        float s[16];
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
            for (int j = 0; j < 4; ++j) s[4 * c + j] = x[j] * ks;
        }
        const bool edge = base + kTile - 1 > all_see;  // some row does not see all of the tile
        const int64_t see = sees - (base + 16 * g);
        if (edge) {
#pragma unroll
            for (int j = 0; j < 16; ++j) s[j] = j <= see ? s[j] : -__builtin_inff();
        }
        float top = s[0];
#pragma unroll
        for (int j = 1; j < 16; ++j) top = fmaxf(top, s[j]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float now = fmaxf(mx, top);
        const float ref = now == -__builtin_inff() ? 0.f : now;
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
        bool nan = false;
        if (edge) {
            // codes behind the last held token may be anything, and a NaN of a
            // token that only some rows see must not reach the others: 0 * NaN
            const int64_t held = kv - (base + 16 * g);
#pragma unroll
            for (int d = 0; d < VT; ++d) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int64_t left = held - 4 * w;
                    vr[d][w] &= left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * (int)left)) - 1u;
                }
                nan |= has_nan_code(vr[d]);
            }
            nan = __ballot(nan) != 0;
        }
        if (nan) {
            bf16x8 see8[2];
#pragma unroll
            for (int j = 0; j < 16; ++j) see8[j >> 3][j & 7] = (bf16)(j <= see ? 1.f : 0.f);
#pragma unroll
            for (int d = 0; d < VT; ++d) {
                floatx4 hits = zero4();
                uintx4 ones;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t x = vr[d][w], y;
                    split_nan(x, y);
                    vr[d][w] = x;
                    ones[w] = y;
                }
                hits = Mma<bf16>::mma(e4m3_to_bf16x8(ones[0], ones[1]), see8[0], hits);
                hits = Mma<bf16>::mma(e4m3_to_bf16x8(ones[2], ones[3]), see8[1], hits);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (hits[j] > 0.f) O[d][j] = __builtin_nanf("");
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
    if (row0 + jr >= len * a.G) return;
    float m = s_m[0][jr];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, s_m[w][jr]);
    const float ref = m == -__builtin_inff() ? 0.f : m;
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
    const int64_t ji = (row0 + jr) / a.G, jt = t0 + ji;
    const int64_t orow = jt * a.H + h * a.G + (row0 + jr - ji * a.G);
    if (alone) {
        const float inv = l == 0.f && m == -__builtin_inff() ? 0.f : 1.f / l;
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

// Joins the parts of each row: a wave per row.
template <typename TI, int DV>
__global__ __launch_bounds__(64 * kWaves) void attention_join_kernel(Attention a) {
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (row >= a.T * a.H) return;
    const int64_t t = row / a.H;
    if (t >= a.cu[a.num_seqs]) return;
    int32_t below = 0;
    for (int32_t n0 = 0; n0 < a.num_seqs; n0 += 64) {
        const int32_t n = n0 + lane;
        below += __popcll(__ballot(n < a.num_seqs && a.cu[n] <= t));
    }
    const int32_t n = below - 1;
    if (n < 0) return;
    const int64_t kv = held_tokens(a, n), chunk = chunk_of(a, kv);
    if (kv <= chunk) return;  // written by its one workgroup
    const int parts = (int)((kv + chunk - 1) / chunk);
    const int64_t step = a.T * a.H;
    float m = -__builtin_inff();
    for (int s = lane; s < parts; s += 64) m = fmaxf(m, a.ws_ml[2 * (s * step + row)]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    const float ref = m == -__builtin_inff() ? 0.f : m;
    float l = 0.f, out[DV / 64];
#pragma unroll
    for (int c = 0; c < DV / 64; ++c) out[c] = 0.f;
    for (int s = 0; s < parts; ++s) {
        const int64_t at = s * step + row;
        const float f = __builtin_amdgcn_exp2f(a.ws_ml[2 * at] - ref);
        l += f * a.ws_ml[2 * at + 1];
#pragma unroll
        for (int c = 0; c < DV / 64; ++c) out[c] += f * a.ws_o[at * DV + lane * (DV / 64) + c];
    }
    TI* o = static_cast<TI*>(a.o) + row * DV + lane * (DV / 64);
    const float inv = l == 0.f && m == -__builtin_inff() ? 0.f : 1.f / l;
#pragma unroll
    for (int c = 0; c < DV / 64; ++c) o[c] = from_f32<TI>(out[c] * inv);
}

struct Plan {
    int32_t splits, min_chunk;
    size_t ml_off, bytes;
};

// Parts of the cache.  The lengths are on the device, so the plan goes by
// bounds: each request's cache is cut into at most `splits` parts of at least
// min_chunk tokens, enough of them to fill the device when every request is as
// long as the bound, and no part of the longest request is above 8192 tokens.
Plan plan(const CacheAttentionLaunch& p) {
    Plan r = {1, kTile, 0, 0};
    const int64_t room = (int64_t)p.max_blocks * p.page_size;
    const int64_t kv = p.max_kv > 0 && p.max_kv < room ? p.max_kv : room;
    const int64_t G = p.H / p.H_kv;
    const int64_t units = ((p.T_total * G + 15) / 16 > p.num_seqs ? (p.T_total * G + 15) / 16 : p.num_seqs) * p.H_kv;
    const int64_t want = units >= 1024 ? 1 : (1024 + units - 1) / units;
    const int64_t chain = (kv + 8191) / 8192;
    int64_t splits = want > chain ? want : chain;
    const int64_t most = (kv + 255) / 256;
    if (splits > most) splits = most;
    if (p.T_total * G > 64 * (int64_t)p.num_seqs) splits = 1;  // many rows
    if (splits < 1) splits = 1;
    if (splits > 256) splits = 256;
    r.splits = (int32_t)splits;
    r.min_chunk = units >= 1024 ? 8192 : 256;
    if (splits > 1) {
        const size_t rows = (size_t)splits * p.T_total * p.H;
        r.ml_off = (rows * p.dv * sizeof(float) + 255) & ~(size_t)255;
        r.bytes = r.ml_off + ((rows * 2 * sizeof(float) + 255) & ~(size_t)255);
    }
    return r;
}

template <typename TI, int DK, int DV>
hipError_t run(const Attention& a, const CacheAttentionLaunch& p, hipStream_t s) {
    const int64_t tiles = p.T_total * a.G / 16 + p.num_seqs;
    hipLaunchKernelGGL((attention_rows_kernel<TI, DK, DV>), dim3((unsigned)tiles, (unsigned)a.Hkv, (unsigned)a.splits),
                       dim3(64 * kWaves), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t blocks = (p.T_total * a.H + kWaves - 1) / kWaves;
    hipLaunchKernelGGL((attention_join_kernel<TI, DV>), dim3((unsigned)blocks), dim3(64 * kWaves), 0, s, a);
    return hipGetLastError();
}
template <typename TI>
hipError_t run_t(const Attention& a, const CacheAttentionLaunch& p, hipStream_t s) {
    if (p.dk == 128 && p.dv == 128) return run<TI, 128, 128>(a, p, s);
    if (p.dk == 128) return run<TI, 128, 64>(a, p, s);
    if (p.dv == 128) return run<TI, 64, 128>(a, p, s);
    return run<TI, 64, 64>(a, p, s);
}

}  // namespace

size_t cache_attention_workspace_bytes(const CacheAttentionLaunch& p) { return plan(p).bytes; }

hipError_t launch_cache_attention(const CacheAttentionLaunch& p, hipStream_t s) {
    if (p.T_total == 0 || p.num_seqs == 0) return hipSuccess;
    const Plan pl = plan(p);
    Attention a;
    a.q = p.q; a.kc = p.k_cache; a.vc = p.v_cache; a.ks = p.k_scale; a.vs = p.v_scale;
    a.table = p.block_table; a.rows = p.rows; a.kv_lens = p.kv_lens; a.cu = p.cu_seqlens;
    a.num_seqs = p.num_seqs; a.T = p.T_total; a.num_pages = p.num_pages;
    a.page = p.page_size; a.num_rows = p.num_rows; a.max_blocks = p.max_blocks;
    a.scale2 = p.scale * kLog2e; a.o = p.o; a.H = p.H; a.Hkv = p.H_kv; a.G = p.H / p.H_kv;
    a.splits = pl.splits; a.min_chunk = pl.min_chunk;
    a.ws_o = static_cast<float*>(p.workspace);
    a.ws_ml = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + pl.ml_off);
    return p.bf16 ? run_t<bf16>(a, p, s) : run_t<float>(a, p, s);
}

}  // namespace gdn
