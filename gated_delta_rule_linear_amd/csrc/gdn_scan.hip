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
    float* states;      // [T / kCheck][C] state before every kCheck tokens, or NULL
    uint64_t* maps;     // [tiles][C] maps of the tiles, and [groups][C] what comes into a group of them (NULL: one tile)
    uint32_t* tickets;  // workgroups that have begun
    int64_t tiles;
};

constexpr int kCheck = 64;
constexpr uint64_t kNotReady = ~0ull;       // of a tile's map
constexpr int32_t kMostPolls = 1 << 22;     // seconds: no wait is without end, whatever happened

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

// The map of a tile, as other workgroups read it: A and e in one word, so that it is
// there as a whole or not at all.
__device__ __forceinline__ void publish(uint64_t* at, const Map& m) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        // (No NaN of a caller's looks like a map that is not there yet.)
        const uint32_t A = m.A[k] != m.A[k] ? 0x7fc00000u : __float_as_uint(m.A[k]);
        __hip_atomic_store(at + k, (uint64_t)__float_as_uint(m.e[k]) << 32 | A, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}
__device__ __forceinline__ Map await(const uint64_t* at, bool live) {
    uint64_t w[4];
    for (int32_t n = 0;; ++n) {
        bool there = true;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[k] = __hip_atomic_load(at + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            there &= (uint32_t)w[k] != (uint32_t)kNotReady;
        }
        if (__ballot(live && !there) == 0 || n == kMostPolls) break;
        __builtin_amdgcn_s_sleep(1);
    }
    Map m;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        m.A[k] = __uint_as_float((uint32_t)w[k]);
        m.e[k] = __uint_as_float((uint32_t)(w[k] >> 32));  // (NaN where nothing came, as A)
    }
    return m;
}

template <typename TI, int L, int NW, bool BACK>
__global__ __launch_bounds__(64 * NW, 4) void scan_kernel(Scan a) {
    constexpr int TILE = L * NW;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t blocks = (a.C + kChannels - 1) / kChannels;
    __shared__ uint32_t s_ticket;
    // A workgroup waits for tiles before its own only (behind it, in the backward
    // pass): their workgroups have begun, since tiles are dealt out in that order.
    uint32_t ticket = blockIdx.x;
    if (a.maps) {
        if (threadIdx.x == 0) s_ticket = atomicAdd(a.tickets, 1u);
        __syncthreads();
        ticket = __builtin_amdgcn_readfirstlane(s_ticket);
    }
    const int64_t place = ticket / (uint32_t)blocks, tile = BACK ? a.tiles - 1 - place : place;
    const int32_t c = (int32_t)(ticket - (uint32_t)place * (uint32_t)blocks) * kChannels + 4 * lane, ch = c < a.C ? c : 0;
    const bool live = c < a.C;
    int64_t end = a.cu[a.num_seqs];
    end = end < a.T ? end : a.T;
    const int64_t first = tile * TILE + wave * L;
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};

    if (tile * TILE < end) {  // of the whole workgroup
        Four<TI> x[L], dh[BACK ? L : 1];
        floatx4 g[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int64_t at = (first + i < end ? first + i : end - 1) * a.C + ch;
            g[i] = *reinterpret_cast<const floatx4*>(a.g + at);
            x[i].v = *reinterpret_cast<const typename Four<TI>::raw*>(static_cast<const TI*>(a.x) + at);
            if (BACK) dh[i].v = *reinterpret_cast<const typename Four<TI>::raw*>(static_cast<const TI*>(a.dh) + at);
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
            if (tokens.ends >> i & 1) s = vector(a.d_final, i);
            l = dh[i].f() + s;
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = decay(g[i][k]) * l[k];
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
        __shared__ Map s_map[BACK ? 2 : 1][NW][64], s_before[NW][64];
        s_map[0][wave][lane] = wave_map(false);
        if (BACK) s_map[1][wave][lane] = wave_map(true);
        // What is computed again below is not kept until then: the registers are the tokens'.
#pragma unroll
        for (int i = 0; i < L; ++i) {
            asm volatile("" : "+v"(g[i]));
            asm volatile("" : "+v"(x[i].v));
            if (BACK) asm volatile("" : "+v"(dh[i].v));
        }
        __syncthreads();
        floatx4 s = zero;  // what comes into the tile
        if (a.maps) {
            // Tiles in the order in which this pass comes to them, in groups of NW.
            const int64_t last = (end + TILE - 1) / TILE - 1, nth = BACK ? last - tile : tile, group = nth / NW;
            const int in_group = (int)(nth - group * NW);
            auto word = [&](int64_t n) { return a.maps + (BACK ? last - n : n) * a.C + ch; };
            uint64_t* const entry = a.maps + (a.tiles + group) * a.C + ch;
            Map own = Map::identity();
            if (wave == 0) {
#pragma unroll
                for (int w = 0; w < NW; ++w) own = s_map[BACK][BACK ? NW - 1 - w : w][lane].after(own);
                if (live) publish(word(nth), own);
            }
            // A wave waits for one of the maps before it in the group, the last for the
            // group's entry: the order of the sums is always the same.
            if (wave < in_group) s_before[wave][lane] = await(word(group * NW + wave), live);
            if (wave == NW - 1 && group > 0) s_before[wave][lane] = await(entry, live);
            __syncthreads();
            if (group > 0) s = s_before[NW - 1][lane].e;
            for (int w = 0; w < in_group; ++w) s = s_before[w][lane].of(s);
            if (wave == 0 && in_group == NW - 1 && live) publish(entry + a.C, Map{floatx4{1.f, 1.f, 1.f, 1.f}, own.of(s)});
        }
        floatx4 r = s;  // the gradient, where s is the state
        if (BACK) s = *reinterpret_cast<const floatx4*>(a.states + tile * (TILE / kCheck) * a.C + ch);
        for (int w = 0; w < wave; ++w) s = s_map[0][w][lane].of(s);
        if (!BACK) {
            if (a.states && live && first % kCheck == 0 && first < end) *reinterpret_cast<floatx4*>(a.states + first / kCheck * a.C + c) = s;
            if (!a.h) return;
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
            for (int w = NW - 1; w > wave; --w) r = s_map[1][w][lane].of(r);
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
    if (tile > 0 || !to || !live) return;
    for (int32_t m = wave; m < a.num_seqs; m += NW)
        if (a.cu[m + 1] <= a.cu[m])
            *reinterpret_cast<floatx4*>(to + (int64_t)m * a.C + c) = from ? *reinterpret_cast<const floatx4*>(from + (int64_t)m * a.C + c) : zero;
}

// No map is there yet, and no workgroup has begun.
__global__ __launch_bounds__(256) void begin_kernel(uint64_t* maps, uint32_t* tickets, int64_t words) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *tickets = 0;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 2; i < words; i += (int64_t)gridDim.x * 512) {
        typedef uint64_t two __attribute__((ext_vector_type(2)));
        *reinterpret_cast<two*>(maps + i) = two{kNotReady, kNotReady};  // (an even number of words)
    }
}

constexpr int kWaves = 8;
template <typename TI, bool BACK>
constexpr int kTokens = BACK || sizeof(TI) == 4 ? 8 : 16;  // of a wave

int64_t up(int64_t x, int64_t y) { return (x + y - 1) / y; }
size_t rounded(size_t bytes) { return (bytes + 255) & ~(size_t)255; }
// Tiles of kCheck tokens at least, and their groups.
int64_t map_words(int64_t tiles, int32_t C) { return (tiles + tiles / kWaves + 1) * C; }
size_t maps_bytes(int64_t T, int32_t C) { return rounded((size_t)map_words(up(T, kCheck), C) * sizeof(uint64_t)) + 256; }

Scan arguments(const ScanLaunch& p) {
    Scan a = {};
    a.x = p.x; a.g = p.g; a.cu = p.cu_seqlens; a.num_seqs = p.num_seqs; a.T = p.T; a.C = p.C; a.mix = p.mix;
    a.init = p.initial_state; a.final = p.final_state; a.h = p.h; a.dh = p.d_h; a.d_final = p.d_final_state;
    a.dx = p.dx; a.dg = p.dg; a.d_init = p.d_initial_state;
    a.tickets = static_cast<uint32_t*>(p.workspace);
    a.maps = reinterpret_cast<uint64_t*>(static_cast<char*>(p.workspace) + 256);
    return a;
}
template <typename TI, bool BACK>
hipError_t run(Scan a, hipStream_t s) {
    constexpr int L = kTokens<TI, BACK>;
    a.tiles = std::max<int64_t>(up(a.T, L * kWaves), 1);
    if (a.tiles == 1) {
        a.maps = nullptr;
    } else {
        const int64_t words = map_words(a.tiles, a.C);
        hipLaunchKernelGGL(begin_kernel, dim3((unsigned)std::min<int64_t>(up(words, 512), 4096)), dim3(256), 0, s, a.maps, a.tickets, words);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)(a.tiles * up(a.C, kChannels)));
    hipLaunchKernelGGL((scan_kernel<TI, L, kWaves, BACK>), grid, dim3(64 * kWaves), 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t scan_checkpoint_bytes(int64_t T, int32_t C) { return (size_t)up(T, kCheck) * C * sizeof(float); }
size_t scan_workspace_bytes(int64_t T, int32_t C) { return maps_bytes(T, C); }
size_t scan_backward_workspace_bytes(int64_t T, int32_t C) { return maps_bytes(T, C) + rounded(scan_checkpoint_bytes(T, C)); }

hipError_t launch_scan(const ScanLaunch& p, hipStream_t s) {
    if (p.num_seqs == 0) return hipSuccess;
    Scan a = arguments(p);
    a.states = p.checkpoints;
    return p.bf16 ? run<bf16, false>(a, s) : run<float, false>(a, s);
}

hipError_t launch_scan_backward(const ScanLaunch& p, hipStream_t s) {
    if (p.num_seqs == 0) return hipSuccess;
    Scan a = arguments(p);
    a.states = p.checkpoints;
    if (!p.checkpoints) {
        a.states = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + maps_bytes(p.T, p.C));
        const hipError_t e = p.bf16 ? run<bf16, false>(a, s) : run<float, false>(a, s);
        if (e != hipSuccess) return e;
    }
    return p.bf16 ? run<bf16, true>(a, s) : run<float, true>(a, s);
}

}  // namespace gdn
