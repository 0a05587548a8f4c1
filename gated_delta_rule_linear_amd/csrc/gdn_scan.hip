// The gated linear recurrence with a vector state, over packed sequences
// (gdn_scan), and its gradients (gdn_scan_backward).  Per channel,
//
//     h_t = a_t h_{t-1} + b_t,     a_t = e^g_t,  b_t = x_t or (1 - a_t) x_t
//     l_t = dh_t + c_{t+1},        c_t = a_t l_t
//     dx_t = l_t or (1 - a_t) l_t, dg_t = c_t h_{t-1} or c_t (h_{t-1} - x_t)
//
// A token does some three operations for each 8 bytes: bound by HBM.  Channels alone
// are too few threads to keep HBM busy, so time is cut into tiles.  What a run of
// tokens does to a state is one map per channel, h -> A h + e, and maps of
// neighbouring runs join: (A2 A1, A2 e1 + e2).  A sequence's first token makes
// its run's map constant, so the packed tokens are one long recurrence whatever
// the sequences are.  A lane has 4 neighbouring channels, a wave L tokens of
// them in registers, a workgroup NW waves one after another in time.
#include <algorithm>

#include "gdn_device.h"
#include "gdn_scan.h"
#include "gdn_stack_kernels.h"

namespace gdn {
namespace {

constexpr int kChannels = 256;  // of a wave: 4 of each lane

struct Scan {
    const void* x;
    const float* g;
    const int32_t* cu;
    int32_t num_seqs;
    int64_t T;
    int32_t C;
    bool mix;
    const float* init;
    float* final;
    void* h;
    const void* dh;
    const float* d_final;
    void* dx;
    float *dg, *d_init;
    int64_t tiles;
    float* states;  // [tiles][C] state before each tile, or NULL
    floatx2* maps;  // [tiles][C] maps of the tiles
    float* carry;   // [tiles][C] c of the token after each tile (backward)
};

// A run's map per channel.  A constant map has A < 0: e alone counts, whatever
// the state before (Inf and NaN among it).
struct Map {
    floatx4 A, e;
    __device__ __forceinline__ static Map identity() { return {{1.f, 1.f, 1.f, 1.f}, {0.f, 0.f, 0.f, 0.f}}; }
    __device__ __forceinline__ floatx4 of(floatx4 s) const {
        floatx4 r;
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = A[k] < 0.f ? e[k] : __builtin_fmaf(A[k], s[k], e[k]);
        return r;
    }
    // This map after `first`.
    __device__ __forceinline__ Map after(const Map& first) const {
        Map r;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            r.A[k] = A[k] < 0.f || first.A[k] < 0.f ? -1.f : A[k] * first.A[k];
            r.e[k] = A[k] < 0.f ? e[k] : __builtin_fmaf(A[k], first.e[k], e[k]);
        }
        return r;
    }
};

// A wave's tokens: where sequences start and end among them.
template <int L>
struct Tokens {
    int64_t first;
    int32_t live;           // tokens that exist
    uint32_t starts, ends;  // bits of the tokens that begin or end a sequence
    const int32_t* cu;
    int32_t n;              // sequences
    int32_t base, bound;    // the last offset at or before the first token, and a lane's of the 64 from there on

    // The last offset's number at or before token t (offsets that decrease give some number).
    __device__ __forceinline__ int32_t last_at(int64_t t) const {
        int32_t lo = 0, hi = n + 1;
        const int lane = threadIdx.x & 63;
        while (hi - lo > 64) {
            const int32_t step = (hi - lo + 63) / 64, at = lo + lane * step;
            const int c = __popcll(__ballot(at < hi && cu[at < hi ? at : lo] <= t));
            if (c > 1) lo += (c - 1) * step;
            hi = hi < lo + step ? hi : lo + step;
        }
        const int32_t at = lo + lane;
        return lo + __popcll(__ballot(at < hi && cu[at < hi ? at : lo] <= t)) - 1;
    }
    __device__ __forceinline__ Tokens(const Scan& a, int64_t first_, int64_t end) : first(first_), cu(a.cu), n(a.num_seqs) {
        live = end - first < L ? (int32_t)(end - first) : L;
        starts = ends = 0;
        if (live <= 0) return;
        base = last_at(first);
        if (base < 0) base = 0;
        const int32_t at = base + (int32_t)(threadIdx.x & 63);
        bound = at <= n ? cu[at] : INT32_MAX;
        const int64_t off = bound - first;
#pragma unroll
        for (int i = 0; i <= L; ++i) {
            if (__ballot(off == i) == 0) continue;
            if (i < L) starts |= 1u << i;
            if (i > 0) ends |= 1u << (i - 1);
        }
        if (__builtin_amdgcn_readlane(bound, 63) <= first + L && base + 63 < n) {  // more empty sequences than lanes
            for (int i = 0; i <= live; ++i) {
                const int32_t m = last_at(first + i);
                if (m < 0 || cu[m] != first + i) continue;
                if (i < L) starts |= 1u << i;
                if (i > 0) ends |= 1u << (i - 1);
            }
        }
        if (first + live == end) ends |= 1u << (live - 1);
        starts &= live < 32 ? (1u << live) - 1 : ~0u;
        ends &= live < 32 ? (1u << live) - 1 : ~0u;
    }
    // The sequence of token i.
    __device__ __forceinline__ int32_t sequence(int i) const {
        const int32_t m = last_at(first + i);
        return m < 0 ? 0 : m < n ? m : n - 1;
    }
};

enum What { kSums, kBackSums, kForward, kBackward };

template <typename TI, int L, int NW, int WHAT>
__global__ __launch_bounds__(64 * NW) void scan_kernel(Scan a) {
    constexpr bool BACK = WHAT == kBackward, REVERSE = BACK || WHAT == kBackSums;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t blocks = (a.C + kChannels - 1) / kChannels;
    const int64_t tile = blockIdx.x / blocks;
    const int32_t c = (int32_t)(blockIdx.x - tile * blocks) * kChannels + 4 * lane, ch = c < a.C ? c : 0;
    const bool live = c < a.C;
    int64_t end = a.cu[a.num_seqs];
    end = end < a.T ? end : a.T;
    const int64_t first = tile * (L * NW) + wave * L;
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};

    if (tile * (L * NW) < end) {  // of the whole workgroup
        Four<TI> x[L], dh[REVERSE ? L : 1];
        floatx4 g[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int64_t at = (first + i < end ? first + i : end - 1) * a.C + ch;
            g[i] = *reinterpret_cast<const floatx4*>(a.g + at);
            if (WHAT != kBackSums) x[i].v = *reinterpret_cast<const typename Four<TI>::raw*>(static_cast<const TI*>(a.x) + at);
            if (REVERSE) dh[i].v = *reinterpret_cast<const typename Four<TI>::raw*>(static_cast<const TI*>(a.dh) + at);
        }
        const Tokens<L> tokens(a, first, end);
        auto vector = [&](const float* v, int i) {  // of token i's sequence
            return v ? *reinterpret_cast<const floatx4*>(v + (int64_t)tokens.sequence(i) * a.C + ch) : zero;
        };
        auto put = [&](float* v, int i, floatx4 y) {
            const int64_t m = tokens.sequence(i);  // (of all lanes)
            if (live) *reinterpret_cast<floatx4*>(v + m * a.C + c) = y;
        };
        auto gate = [&](int i, floatx4& al, floatx4& om) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                al[k] = decay(g[i][k]);
                om[k] = a.mix ? one_minus_decay(g[i][k], al[k]) : 1.f;
            }
        };
        auto next = [&](floatx4 s, int i) {  // the state after token i
            floatx4 al, om;
            gate(i, al, om);
            if (tokens.starts >> i & 1) s = vector(a.init, i);
            const floatx4 in = x[i].f();
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = __builtin_fmaf(al[k], s[k], om[k] * in[k]);
            return s;
        };
        auto before = [&](floatx4 s, int i, floatx4& l) {  // c of token i from the next token's
            floatx4 al, om;
            gate(i, al, om);
            if (tokens.ends >> i & 1) s = vector(a.d_final, i);
            l = dh[i].f() + s;
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = al[k] * l[k];
            return s;
        };
        // What the wave's tokens do to a state, or to the gradient that comes from behind.
        auto wave_map = [&](bool reverse) {
            Map m = Map::identity();
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (i < tokens.live)
#pragma unroll
                    for (int k = 0; k < 4; ++k) m.A[k] *= decay(g[i][k]);
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const int i = reverse ? L - 1 - j : j;
                floatx4 l;
                if (i < tokens.live) m.e = reverse ? before(m.e, i, l) : next(m.e, i);
            }
            const bool constant = (reverse ? tokens.ends : tokens.starts) != 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) m.A[k] = constant ? -1.f : m.A[k] < 0x1p-149f ? 0x1p-149f : m.A[k];
            return m;
        };
        __shared__ Map maps[2][NW][64];
        if (WHAT != kBackSums) maps[0][wave][lane] = wave_map(false);
        if (REVERSE) maps[1][wave][lane] = wave_map(true);
        __syncthreads();
        if (WHAT == kSums || WHAT == kBackSums) {
            if (wave > 0 || !live) return;
            Map m = Map::identity();
#pragma unroll
            for (int w = 0; w < NW; ++w) m = maps[REVERSE][REVERSE ? NW - 1 - w : w][lane].after(m);
#pragma unroll
            for (int k = 0; k < 4; ++k) a.maps[tile * a.C + c + k] = floatx2{m.A[k], m.e[k]};
            return;
        }
        floatx4 s = *reinterpret_cast<const floatx4*>(a.states + tile * a.C + ch);
        for (int w = 0; w < wave; ++w) s = maps[0][w][lane].of(s);
        if (!BACK) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (i >= tokens.live) continue;
                s = next(s, i);
                if (live) *reinterpret_cast<typename Four<TI>::raw*>(static_cast<TI*>(a.h) + (first + i) * a.C + c) = Four<TI>::of(s);
                if (a.final && (tokens.ends >> i & 1)) put(a.final, i, s);
            }
        } else {
            floatx4 past[L];
#pragma unroll
            for (int i = 0; i < L; ++i) {
                if (i >= tokens.live) continue;
                past[i] = tokens.starts >> i & 1 ? vector(a.init, i) : s;
                s = next(s, i);
                if (a.mix) past[i] -= x[i].f();
            }
            floatx4 r = *reinterpret_cast<const floatx4*>(a.carry + tile * a.C + ch);
            for (int w = NW - 1; w > wave; --w) r = maps[1][w][lane].of(r);
#pragma unroll
            for (int i = L - 1; i >= 0; --i) {
                if (i >= tokens.live) continue;
                floatx4 al, om, l;
                gate(i, al, om);
                r = before(r, i, l);
                if (live) {
                    *reinterpret_cast<typename Four<TI>::raw*>(static_cast<TI*>(a.dx) + (first + i) * a.C + c) = Four<TI>::of(om * l);
                    *reinterpret_cast<floatx4*>(a.dg + (first + i) * a.C + c) = r * past[i];
                }
                if (a.d_init && (tokens.starts >> i & 1)) put(a.d_init, i, r);
            }
        }
    }
    // Sequences without a token keep their state, or its gradient.
    float* const to = BACK ? a.d_init : a.final;
    const float* const from = BACK ? a.d_final : a.init;
    if (tile > 0 || !to || !live || WHAT == kSums || WHAT == kBackSums) return;
    for (int32_t m = wave; m < a.num_seqs; m += NW)
        if (a.cu[m + 1] <= a.cu[m])
            *reinterpret_cast<floatx4*>(to + (int64_t)m * a.C + c) = from ? *reinterpret_cast<const floatx4*>(from + (int64_t)m * a.C + c) : zero;
}

// The states before the tiles, or the gradients behind them, from the tiles' maps.
template <bool REVERSE>
__global__ __launch_bounds__(64) void fold_kernel(Scan a, int tokens) {
    const int32_t c = blockIdx.x * 64 + threadIdx.x;
    if (c >= a.C) return;
    int64_t end = a.cu[a.num_seqs];
    end = end < a.T ? end : a.T;
    const int64_t used = (end + tokens - 1) / tokens;
    float s = 0.f;
    float* const to = REVERSE ? a.carry : a.states;
    for (int64_t j = 0; j < used; ++j) {
        const int64_t tile = REVERSE ? used - 1 - j : j;
        const floatx2 m = a.maps[tile * a.C + c];
        to[tile * a.C + c] = s;
        s = m[0] < 0.f ? m[1] : __builtin_fmaf(m[0], s, m[1]);
    }
}

constexpr int kL = 8, kNW = 8, kTile = kL * kNW;

int64_t tiles_of(int64_t T) { return (T + kTile - 1) / kTile; }
size_t rounded(size_t bytes) { return (bytes + 255) & ~(size_t)255; }

Scan arguments(const ScanLaunch& p) {
    Scan a = {};
    a.x = p.x; a.g = p.g; a.cu = p.cu_seqlens; a.num_seqs = p.num_seqs; a.T = p.T; a.C = p.C; a.mix = p.mix;
    a.init = p.initial_state; a.final = p.final_state; a.h = p.h; a.dh = p.d_h; a.d_final = p.d_final_state;
    a.dx = p.dx; a.dg = p.dg; a.d_init = p.d_initial_state;
    a.tiles = std::max<int64_t>(tiles_of(p.T), 1);
    return a;
}
template <int WHAT>
hipError_t run(const Scan& a, bool half, hipStream_t s) {
    const unsigned blocks = (unsigned)(a.tiles * ((a.C + kChannels - 1) / kChannels));
    if (half) hipLaunchKernelGGL((scan_kernel<bf16, kL, kNW, WHAT>), dim3(blocks), dim3(64 * kNW), 0, s, a);
    else hipLaunchKernelGGL((scan_kernel<float, kL, kNW, WHAT>), dim3(blocks), dim3(64 * kNW), 0, s, a);
    return hipGetLastError();
}
template <bool REVERSE>
hipError_t fold(const Scan& a, hipStream_t s) {
    hipLaunchKernelGGL(fold_kernel<REVERSE>, dim3((a.C + 63) / 64), dim3(64), 0, s, a, kTile);
    return hipGetLastError();
}

}  // namespace

size_t scan_checkpoint_bytes(int64_t T, int32_t C) { return (size_t)tiles_of(T) * C * sizeof(float); }
size_t scan_workspace_bytes(int64_t T, int32_t C) {
    return rounded((size_t)tiles_of(T) * C * sizeof(floatx2)) + rounded(scan_checkpoint_bytes(T, C));
}
size_t scan_backward_workspace_bytes(int64_t T, int32_t C) { return scan_workspace_bytes(T, C) + rounded(scan_checkpoint_bytes(T, C)); }

hipError_t launch_scan(const ScanLaunch& p, hipStream_t s) {
    if (p.num_seqs == 0) return hipSuccess;
    Scan a = arguments(p);
    char* at = static_cast<char*>(p.workspace);
    a.maps = reinterpret_cast<floatx2*>(at);
    a.states = p.checkpoints ? p.checkpoints : reinterpret_cast<float*>(at + rounded((size_t)tiles_of(p.T) * p.C * sizeof(floatx2)));
    hipError_t e;
    if ((e = run<kSums>(a, p.bf16, s)) != hipSuccess || (e = fold<false>(a, s)) != hipSuccess) return e;
    return run<kForward>(a, p.bf16, s);
}

hipError_t launch_scan_backward(const ScanLaunch& p, hipStream_t s) {
    if (p.num_seqs == 0) return hipSuccess;
    Scan a = arguments(p);
    char* at = static_cast<char*>(p.workspace);
    a.maps = reinterpret_cast<floatx2*>(at);
    at += rounded((size_t)tiles_of(p.T) * p.C * sizeof(floatx2));
    a.carry = reinterpret_cast<float*>(at);
    hipError_t e;
    a.states = p.checkpoints;
    if (!p.checkpoints) {
        a.states = reinterpret_cast<float*>(at + rounded(scan_checkpoint_bytes(p.T, p.C)));
        if ((e = run<kSums>(a, p.bf16, s)) != hipSuccess || (e = fold<false>(a, s)) != hipSuccess) return e;
    }
    if ((e = run<kBackSums>(a, p.bf16, s)) != hipSuccess || (e = fold<true>(a, s)) != hipSuccess) return e;
    return run<kBackward>(a, p.bf16, s);
}

}  // namespace gdn
