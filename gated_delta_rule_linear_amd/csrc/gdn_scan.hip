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
// them in registers, a workgroup kWaves waves one after another in time: 128
// tokens of bf16 forward, 64 else.
//
// One launch reads the inputs once.  A workgroup forms its tile's map, publishes it,
// waits for what comes into the tile and forms the outputs.  Tiles are in groups of
// kWaves * kEach: a wave waits for one of the group's maps before the tile's, and one
// for what comes into the group, which the last tile of the group before hands on.
// So the order of the sums is always the same, and bits do not depend on timing.  A
// group in which a sequence begins waits for nothing before it.  Tiles are dealt
// out by counters in the order of the pass, and a workgroup publishes its map
// before it waits: what is waited for has begun, and comes.  A map's A and e are one
// word, written and read as such, so nothing else orders them.
//
// Measured, bf16 (of what has to be read and written): 65,536 tokens of 4,096
// channels 372 us, 5.8 TB/s, where a copy reaches 5.1; four sequences of 8,192 191 us
// forward and 339 backward (5.6 and 5.6), with `mix` 209 (1 - e^g is formed for both
// passes over the registers) and 347; without the forward call's checkpoints, whose states
// are another pass, 494 and 505.  A forward pass for the maps, a fold and a
// pass for the outputs took 1,196 us for the first.  8,300 tokens of 1,028 channels in 8
// sequences, fp32, 37 us: 650 workgroups for 512 places, and a chain of ticket, inputs,
// maps and outputs.  What counts: nothing that the rare first and last tokens need may
// be waited for in the tokens' loop (the stores before it would be waited for too: 422
// against 492 us), maps that are read in whole lines (482 against 550 us with 64 tokens
// to a tile), and waiting on one word (461 against 493).
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
    const float* init;
    float* final;
    void* h;
    const void* dh;
    const float* d_final;
    void* dx;
    float *dg, *d_init;
    float* states;      // [T / kCheck][C] state before every kCheck tokens, or NULL
    uint64_t* maps;     // [tiles][blocks][4][64] maps of the tiles, and [groups][blocks][4][64] what comes into a group of
                        // them: a lane's four channels are 64 words apart (NULL: one tile)
    uint64_t* counters;  // of workgroups that have begun, a line each
    int64_t tiles;
    bool apart;  // the blocks of channels have counters of their own
};

constexpr int kCheck = 64;  // tokens
// Workgroups up to which blocks of channels have counters of their own.  Those that begin
// together, 512 of them, wait for each other at one counter (2,048 tokens of 4,096
// channels, fp32: 30.0 us, apart 24.1; 8,192, bf16: 67 and 60).  Where most begin one by
// one, one counter keeps the blocks of a tile together, which are neighbours in memory
// (32,768, bf16: 191 us, apart 199).
constexpr int64_t kApart = 2048;
constexpr int kLine = 16;   // words
constexpr int kEach = 1;    // maps that a wave waits for (2: 435 us where 1 takes 422; 4: 567)
constexpr uint64_t kNotReady = ~0ull;       // of a tile's map
// Some 0.8 s: no wait is without end, whatever happened to a workspace.  What is waited for
// comes within microseconds, since its workgroup has begun; the rest is for processes that
// share the device, whose time slices of some ten milliseconds may lie between the two.
// A call whose every entry is lost ends within a minute (16 turns of 512 workgroups, two
// waits each, for 8,192).
constexpr int32_t kMostPolls = 1 << 20;

// The decay of two runs: the product, and where it falls below fp32's numbers the least
// of them, so that an infinite state stays infinite behind runs as it does from token to
// token.  It is 0 where one of the two is, and 0 Inf is NaN from there on.
// (As integers, which numbers from 0 up are ordered as; NaN stays NaN.)
constexpr float kLeast = 0x1p-149f;
__device__ __forceinline__ float joined_decay(float a, float b) {
    return __uint_as_float(max(__float_as_uint(a * b), min(min(__float_as_uint(a), __float_as_uint(b)), 1u)));
}

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
    // This map after `first`.  (ROUGH: a decay of 0 may also be a product of others.)
    template <bool ROUGH = false>
    __device__ __forceinline__ Map after(const Map& first) const {
        Map r;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            r.A[k] = A[k] < 0.f || first.A[k] < 0.f ? -1.f : ROUGH ? A[k] * first.A[k] : joined_decay(A[k], first.A[k]);
            r.e[k] = A[k] < 0.f ? e[k] : __builtin_fmaf(A[k], first.e[k], e[k]);
        }
        return r;
    }
    // Whether a decay of some lane is 0.
    __device__ __forceinline__ bool some_zero() const {
        return __builtin_expect(__ballot(fminf(fminf(A[0], A[1]), fminf(A[2], A[3])) == 0.f) != 0, 0);
    }
};

// A wave's tokens: where sequences start and end among them.
template <int L>
struct Tokens {
    int32_t live;           // tokens that exist
    uint32_t starts, ends;  // bits of the tokens that begin or end a sequence
    int32_t number;         // lane i: the sequence of token i, if there is such a bit

    // The number of the last offset at or before token t (offsets that decrease give some number).
    __device__ __forceinline__ static int32_t last_at(const int32_t* cu, int32_t n, int64_t t) {
        int32_t lo = 0, hi = n + 1;
        const int lane = threadIdx.x & 63;
        for (;;) {
            const int32_t step = (hi - lo + 63) / 64, at = lo + lane * step;
            const int c = __popcll(__ballot(at < hi && cu[at < hi ? at : lo] <= t));
            if (step <= 1) return lo + c - 1;
            if (c > 1) lo += (c - 1) * step;
            hi = hi < lo + step ? hi : lo + step;
        }
    }
    __device__ __forceinline__ Tokens(const Scan& a, int64_t first, int64_t end) {
        const int32_t* const cu = a.cu;
        const int32_t n = a.num_seqs, lane = threadIdx.x & 63, some = end - first < L ? (int32_t)(end - first) : L;
        uint32_t begin = 0, stop = 0;
        number = 0;
        if (some > 0) {
            int32_t base = last_at(cu, n, first);
            if (base < 0) base = 0;
            const int32_t at = base + lane, bound = at <= n ? cu[at] : INT32_MAX;
            const int64_t off = bound - first;
#pragma unroll
            for (int i = 0; i <= L; ++i) {
                if (__ballot(off == i) == 0) continue;
                if (i < L) begin |= 1u << i;
                if (i > 0) stop |= 1u << (i - 1);
            }
            const bool crowded = __builtin_amdgcn_readlane(bound, 63) <= first + L && base + 63 < n;  // more empty sequences than lanes
            if (crowded) {
#pragma unroll 1
                for (int i = 0; i <= some; ++i) {
                    const int32_t m = last_at(cu, n, first + i);
                    if (lane == i) number = m;
                    if (m < 0 || cu[m] != first + i) continue;
                    if (i < L) begin |= 1u << i;
                    if (i > 0) stop |= 1u << (i - 1);
                }
            }
            if (first + some == end) stop |= 1u << (some - 1);
            begin &= (2u << (some - 1)) - 1;
            stop &= (2u << (some - 1)) - 1;
            if ((begin | stop) && !crowded) {
#pragma unroll 1
                for (int i = 0; i < some; ++i) {
                    const int32_t m = base + __popcll(__ballot(off <= i)) - 1;
                    if (lane == i) number = m;
                }
            }
            number = number < 0 ? 0 : number < n ? number : n - 1;
        }
        live = __builtin_amdgcn_readfirstlane(some);
        starts = __builtin_amdgcn_readfirstlane(begin);
        ends = __builtin_amdgcn_readfirstlane(stop);
    }
    // (Tested where it is asked: 2 L conditions known ahead would take up the scalar registers.)
    __device__ __forceinline__ static bool bit(uint32_t bits, int i) {
        asm volatile("" : "+s"(bits));
        return bits >> i & 1;
    }
    __device__ __forceinline__ bool starts_at(int i) const { return bit(starts, i); }
    __device__ __forceinline__ bool ends_at(int i) const { return bit(ends, i); }
    __device__ __forceinline__ bool there(int i) const {
        int32_t n = live;
        asm volatile("" : "+s"(n));
        return i < n;
    }
    __device__ __forceinline__ int32_t sequence(int i) const { return __builtin_amdgcn_readlane(number, i); }
};

// The map of a tile, as other workgroups read it: A and e in one word, so that it is
// there as a whole or not at all.
__device__ __forceinline__ void publish(uint64_t* at, const Map& m) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        // (No NaN of a caller's looks like a map that is not there yet.)
        const uint32_t A = m.A[k] != m.A[k] ? 0x7fc00000u : __float_as_uint(m.A[k]);
        __hip_atomic_store(at + 64 * k, (uint64_t)__float_as_uint(m.e[k]) << 32 | A, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}
// N maps joined, `step` words apart, as they come: the first `count` of them, the
// first of all at `one`.
template <int N>
__device__ __forceinline__ Map await(const uint64_t* one, int64_t step, int count, bool live) {
    const uint64_t* const at = one + (threadIdx.x & 63);
    uint64_t w[N][4];
    for (int32_t polls = 0;;) {
        int missing = N;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (j < count) {
#pragma unroll
                for (int k = 0; k < 4; ++k) w[j][k] = __hip_atomic_load(at + j * step + 64 * k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
#pragma unroll
        for (int j = N - 1; j >= 0; --j) {
            bool there = true;
            if (j < count) {
#pragma unroll
                for (int k = 0; k < 4; ++k) there &= (uint32_t)w[j][k] != (uint32_t)kNotReady;
            }
            if (__ballot(live && !there)) missing = j;
        }
        if (missing == N || polls >= kMostPolls) break;
        // All lanes wait for one word, one line instead of 32: the polls of whole waves
        // get in the way of those that write what they wait for.
        const uint64_t* const first = one + missing * step;
        do {
            __builtin_amdgcn_s_sleep(1);
        } while (++polls < kMostPolls && (uint32_t)__hip_atomic_load(first, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)kNotReady);
    }
    Map m = Map::identity();
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (j >= count) continue;
        Map next;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            next.A[k] = __uint_as_float((uint32_t)w[j][k]);
            next.e[k] = __uint_as_float((uint32_t)(w[j][k] >> 32));  // (NaN where nothing came, as A)
        }
        m = j == 0 ? next : next.after(m);
    }
    return m;
}

// What is far larger than the caches passes them by: 4 to 7% of time. (x and dh are
// read as usual: by the caches too it is the same or slower.)
template <typename T>
__device__ __forceinline__ T load(const T* p) {
    return __builtin_nontemporal_load(p);
}
template <typename T>
__device__ __forceinline__ void store(T* p, T x) {
    __builtin_nontemporal_store(x, p);
}

template <typename TI, int L, int NW, bool BACK, bool MIX>
__global__ __launch_bounds__(64 * NW, 4) void scan_kernel(Scan a) {
    constexpr int TILE = L * NW, GROUP = NW * kEach;
    static_assert(TILE % kCheck == 0, "tiles hold whole spans of checkpoints; the workspace is sized by them");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t blocks = (a.C + kChannels - 1) / kChannels, held = a.cu[a.num_seqs];
    __shared__ uint32_t s_ticket;
    // A workgroup waits for tiles of its channels before its own only (behind it, in the
    // backward pass): their workgroups have begun, since tiles are dealt out in that order,
    // by one counter or by one for each block of channels.
    uint32_t place = 0, block = blockIdx.x;
    if (a.maps) {
        const uint32_t counter = a.apart ? blockIdx.x % (uint32_t)blocks : 0;
        if (threadIdx.x == 0) s_ticket = atomicAdd(reinterpret_cast<uint32_t*>(a.counters + counter * kLine), 1u) + 1;
        __syncthreads();
        const uint32_t ticket = __builtin_amdgcn_readfirstlane(s_ticket);
        place = a.apart ? ticket : ticket / (uint32_t)blocks;
        block = a.apart ? counter : ticket - place * (uint32_t)blocks;
    }
    const int64_t tile = BACK ? a.tiles - 1 - place : place;
    const int32_t c = (int32_t)block * kChannels + 4 * lane;
    const uint32_t ch = c < a.C ? c : 0;
    const bool live = c < a.C;
    const int64_t end = __builtin_amdgcn_readfirstlane(held < a.T ? held : (int32_t)a.T), first = tile * TILE + wave * L;
    const floatx4 zero = {0.f, 0.f, 0.f, 0.f};

    if (tile * TILE < end) {  // of the whole workgroup
        Four<TI> x[L], dh[BACK ? L : 1];
        floatx4 g[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int64_t at = (first + i < end ? first + i : end - 1) * a.C;
            g[i] = load(reinterpret_cast<const floatx4*>(a.g + at + ch));
            x[i].v = *reinterpret_cast<const typename Four<TI>::raw*>(static_cast<const TI*>(a.x) + at + ch);
            if (BACK) dh[i].v = *reinterpret_cast<const typename Four<TI>::raw*>(static_cast<const TI*>(a.dh) + at + ch);
        }
        const Tokens<L> tokens(a, first, end);
        if (tokens.live < L) {  // tokens that are none change nothing
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (i >= tokens.live) {
                    g[i] = zero;
                    x[i] = {};
                    if (BACK) dh[i] = {};
                }
        }
        // (What is loaded where a sequence begins or ends is waited for there: behind it
        // the wait would be every token's, and for the stores before it too.)
        auto vector = [&](const float* v, int i) {  // of token i's sequence
            floatx4 y = zero;
            if (v) {
                y = *reinterpret_cast<const floatx4*>(v + (int64_t)tokens.sequence(i) * a.C + ch);
                asm volatile("" : "+v"(y));
            }
            return y;
        };
        auto put = [&](float* v, int i, floatx4 y) {
            if (live) *reinterpret_cast<floatx4*>(v + (int64_t)tokens.sequence(i) * a.C + ch) = y;
        };
        // The first pass leaves decays where the registers had g (346 to 339 us backward), and
        // with `mix` b where they had fp32's x (164 to 158 forward) or, for bf16's gradients,
        // 1 - e^g in LDS and in registers that are free (379 to 347).  Else there is no room for
        // 1 - e^g, and all is formed again in every pass (bf16 forward with 8 tokens to a wave,
        // where there is: 228 us for 209).
        constexpr bool KEPT = !MIX || (BACK ? sizeof(TI) == 2 : sizeof(TI) == 4);
        constexpr int IN_LDS = BACK && MIX && KEPT ? L / 2 : 0, OWN = IN_LDS > 0 ? L - IN_LDS : 0;
        __shared__ floatx4 s_rest[IN_LDS > 0 ? IN_LDS : 1][NW][64];
        floatx4 rest[OWN > 0 ? OWN : 1];
        auto rest_of = [&](int i) { return i < IN_LDS ? s_rest[i][wave][lane] : rest[OWN > 0 ? i - IN_LDS : 0]; };
        auto decay_of = [&](int i, int k) { return KEPT ? g[i][k] : decay(g[i][k]); };
        auto next = [&](floatx4 s, int i, bool first) {  // the state after token i
            if (tokens.starts_at(i)) s = vector(a.init, i);
            floatx4 in = x[i].f();
            if (KEPT && first) {
                floatx4 y;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float al = decay(g[i][k]);
                    if (MIX) y[k] = one_minus_decay(g[i][k], al);
                    g[i][k] = al;
                }
                if (MIX) {
                    in *= y;
                    if constexpr (!BACK && sizeof(TI) == 4) x[i].v = in;
                    if (i < IN_LDS) s_rest[i][wave][lane] = y;
                    else if (OWN > 0) rest[OWN > 0 ? i - IN_LDS : 0] = y;
                }
            } else if (IN_LDS > 0) {
                in *= rest_of(i);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float al = decay_of(i, k);
                s[k] = __builtin_fmaf(al, s[k], KEPT ? in[k] : one_minus_decay(g[i][k], al) * in[k]);
            }
            return s;
        };
        auto before = [&](floatx4 s, int i, floatx4& l) {  // c of token i from the next token's
            if (tokens.ends_at(i)) s = vector(a.d_final, i);
            l = dh[i].f() + s;
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = decay_of(i, k) * l[k];
            return s;
        };
        // What is computed again for another pass over the tokens is not kept until then,
        // nor is it computed ahead of its token: the registers are the inputs'.
        auto forget = [&](bool inputs, int from) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                asm volatile("" : "+v"(g[i]));
                if (OWN > 0 && i >= IN_LDS) asm volatile("" : "+v"(rest[OWN > 0 ? i - IN_LDS : 0]));
                if (inputs) asm volatile("" : "+v"(x[i].v));
                if (BACK && i >= from) asm volatile("" : "+v"(dh[i].v));
            }
        };
        // What the wave's tokens do to a state, or to the gradient that comes from behind.
        auto wave_map = [&](bool reverse) {
            Map m = Map::identity();
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const int i = reverse ? L - 1 - j : j;
                floatx4 l;
                m.e = reverse ? before(m.e, i, l) : next(m.e, i, true);
#pragma unroll
                for (int k = 0; k < 4; ++k) m.A[k] *= decay_of(i, k);
                asm volatile("" : "+v"(m.A));  // (here, not where a branch needs it)
                __builtin_amdgcn_sched_barrier(0);
            }
            // A product of 0 is put right by itself: it is rare, and joined_decay for each
            // token costs the bf16 kernels registers that they lack.
            if (m.some_zero()) {
                bool some[4] = {};  // of the decays is 0
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    asm volatile("" : "+v"(g[i]));
#pragma unroll
                    for (int k = 0; k < 4; ++k) some[k] |= decay_of(i, k) == 0.f;
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) m.A[k] = m.A[k] == 0.f && !some[k] ? kLeast : m.A[k];
            }
            const bool constant = (reverse ? tokens.ends : tokens.starts) != 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) m.A[k] = constant ? -1.f : m.A[k];
            return m;
        };
        __shared__ Map s_map[BACK ? 2 : 1][NW][64], s_before[(GROUP - 1 + kEach - 1) / kEach][64];  // (before the group's last tile)
        __shared__ floatx4 s_entry[64];
        // 128 registers are two workgroups to a compute unit.  What does not fit waits in LDS:
        // where the maps are joined, four gates of bf16's 16 tokens (spilled to memory, a ninth more
        // to read and write, 394 us for the 372 above); up to the outputs, gradients of the
        // first tokens in fp32 (with 142 registers and one workgroup 280 us for 238, with
        // `mix` 307 for 250, 4 sequences of 8,192 tokens of 2,048 channels).
        constexpr int PARKED = L > 8 ? 4 : 0, WAITING = BACK && sizeof(TI) == 4 ? 4 : 0;
        __shared__ floatx4 s_wait[PARKED + WAITING > 0 ? PARKED + WAITING : 1][NW][64];
        s_map[0][wave][lane] = wave_map(false);
        forget(true, 0);
        if (BACK) {
            s_map[1][wave][lane] = wave_map(true);
            forget(true, 0);
        }
#pragma unroll
        for (int i = 0; i < PARKED; ++i) s_wait[i][wave][lane] = g[L - 1 - i];
        if constexpr (WAITING > 0) {
#pragma unroll
            for (int i = 0; i < WAITING; ++i) s_wait[i][wave][lane] = dh[i].v;
        }
        __syncthreads();
        floatx4 s = zero;  // what comes into the tile
        if (a.maps) {
            // Tiles in the order in which this pass comes to them, in groups.
            const int64_t last = (end + TILE - 1) / TILE - 1, nth = BACK ? last - tile : tile, group = nth / GROUP, begin = group * GROUP;
            const int in_group = (int)(nth - begin);
            auto words = [&](int64_t n) { return a.maps + (n * blocks + block) * kChannels; };
            Map own = Map::identity();
            if (wave == 0) {
#pragma unroll 2
                for (int w = 0; w < NW; ++w) own = s_map[BACK][BACK ? NW - 1 - w : w][lane].template after<true>(own);
                // (Put right by itself too: with joined_decay in each join the chunks of 37 us above
                // take 1 us more, and 65,536 tokens 3.)
                if (own.some_zero()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float A = 1.f;  // (no map is constant where own's A is 0)
#pragma unroll 1
                        for (int w = 0; w < NW; ++w) A = joined_decay(A, s_map[BACK][w][lane].A[k]);
                        own.A[k] = own.A[k] == 0.f ? A : own.A[k];
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                if (live) publish(words(tile) + lane, own);
            }
            // A wave waits for kEach of the group's maps before the tile's: the order of
            // the sums is always the same.
            const int mine = wave * kEach;
            if (mine < in_group) {
                const int64_t step = (int64_t)blocks * kChannels;
                s_before[wave][lane] = await<kEach>(words(BACK ? last - begin - mine : begin + mine), BACK ? -step : step, in_group - mine, live);
            }
            __syncthreads();
            // What comes into the group matters where no sequence begins (ends) before the tile.
            bool open = true;
            for (int w = 0; w * kEach < in_group; ++w) open &= !(s_before[w][0].A[0] < 0.f);
            if (open && group > 0) {
                if (wave == 0) s_entry[lane] = await<1>(words(a.tiles + group), 0, 1, live).e;
                __syncthreads();
                s = s_entry[lane];
            }
#pragma unroll 2
            for (int w = 0; w * kEach < in_group; ++w) s = s_before[w][lane].of(s);
            if (wave == 0 && in_group == GROUP - 1 && live)
                publish(words(a.tiles + group + 1) + lane, Map{floatx4{1.f, 1.f, 1.f, 1.f}, own.of(s)});
        }
#pragma unroll
        for (int i = 0; i < PARKED; ++i) g[L - 1 - i] = s_wait[i][wave][lane];
        floatx4 r = s;  // the gradient, where s is the state
        if (BACK) s = *reinterpret_cast<const floatx4*>(a.states + tile * (TILE / kCheck) * a.C + ch);
#pragma unroll 2
        for (int w = 0; w < wave; ++w) s = s_map[0][w][lane].of(s);
        if (!BACK) {
            if (a.states && live && first % kCheck == 0 && first < end) *reinterpret_cast<floatx4*>(a.states + first / kCheck * a.C + c) = s;
            if (!a.h) return;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                s = next(s, i, false);
                if (live && tokens.there(i))
                    store(reinterpret_cast<typename Four<TI>::raw*>(static_cast<TI*>(a.h) + (first + i) * a.C + ch), Four<TI>::of(s));
                if (a.final && tokens.ends_at(i)) put(a.final, i, s);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            floatx4 past[L];  // h_{t-1} (- x_t)
#pragma unroll
            for (int i = 0; i < L; ++i) {
                past[i] = s;
                if (tokens.starts_at(i)) past[i] = vector(a.init, i);
                s = next(s, i, false);
                if (MIX) {
                    past[i] -= x[i].f();
                    asm volatile("" : "+v"(past[i]));  // (here: x is not needed any more)
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            forget(false, WAITING);
#pragma unroll 2
            for (int w = NW - 1; w > wave; --w) r = s_map[1][w][lane].of(r);
#pragma unroll
            for (int i = L - 1; i >= 0; --i) {
                floatx4 l;
                if constexpr (WAITING > 0)
                    if (i < WAITING) dh[i].v = s_wait[i][wave][lane];
                r = before(r, i, l);
                const floatx4 dg = r * past[i];
                if (MIX && KEPT) l *= rest_of(i);
                if (MIX && !KEPT)
#pragma unroll
                    for (int k = 0; k < 4; ++k) l[k] *= one_minus_decay(g[i][k], decay(g[i][k]));
                if (live && tokens.there(i)) {
                    store(reinterpret_cast<typename Four<TI>::raw*>(static_cast<TI*>(a.dx) + (first + i) * a.C + ch), Four<TI>::of(l));
                    store(reinterpret_cast<floatx4*>(a.dg + (first + i) * a.C + ch), dg);
                }
                if (a.d_init && tokens.starts_at(i)) put(a.d_init, i, r);
                __builtin_amdgcn_sched_barrier(0);
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

// No map is there yet, and no workgroup has begun (a counter's first value is all ones too).
__global__ __launch_bounds__(256) void begin_kernel(uint64_t* counters_and_maps, int64_t words) {
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 2; i < words; i += (int64_t)gridDim.x * 512) {
        typedef uint64_t two __attribute__((ext_vector_type(2)));
        *reinterpret_cast<two*>(counters_and_maps + i) = two{kNotReady, kNotReady};  // (an even number of words)
    }
}

constexpr int kWaves = 8;  // (16: 520 us where 8 take 460; 4: 528)
// Tokens of a wave, as many as the registers hold: bf16 forward 422 us with 16 and 446
// with 8, backward (two passes' inputs) 394 with 8 and 515 with 16.
template <typename TI, bool BACK>
constexpr int kTokens = BACK || sizeof(TI) == 4 ? 8 : 16;

int64_t up(int64_t x, int64_t y) { return (x + y - 1) / y; }
size_t rounded(size_t bytes) { return (bytes + 255) & ~(size_t)255; }
// Tiles of kCheck tokens at least, and their groups.
int64_t map_words(int64_t tiles, int32_t C) { return (tiles + tiles / (kWaves * kEach) + 1) * up(C, kChannels) * kChannels; }
int64_t counter_words(int32_t C) { return std::min(up(C, kChannels), kApart / 2) * kLine; }  // (of two tiles or more)
size_t maps_bytes(int64_t T, int32_t C) { return rounded((size_t)(counter_words(C) + map_words(up(T, kCheck), C)) * sizeof(uint64_t)); }

Scan arguments(const ScanLaunch& p) {
    Scan a = {};
    a.x = p.x; a.g = p.g; a.cu = p.cu_seqlens; a.num_seqs = p.num_seqs; a.T = p.T; a.C = p.C;
    a.init = p.initial_state; a.final = p.final_state; a.h = p.h; a.dh = p.d_h; a.d_final = p.d_final_state;
    a.dx = p.dx; a.dg = p.dg; a.d_init = p.d_initial_state;
    a.counters = static_cast<uint64_t*>(p.workspace);
    a.maps = a.counters + counter_words(p.C);
    return a;
}
template <typename TI, bool BACK, bool MIX>
hipError_t run(Scan a, hipStream_t s) {
    constexpr int L = kTokens<TI, BACK>;
    a.tiles = std::max<int64_t>(up(a.T, L * kWaves), 1);
    if (a.tiles == 1) {
        a.maps = nullptr;
    } else {
        const int64_t words = counter_words(a.C) + map_words(a.tiles, a.C);
        hipLaunchKernelGGL(begin_kernel, dim3((unsigned)std::min<int64_t>(up(words, 512), 4096)), dim3(256), 0, s, a.counters, words);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t all = a.tiles * up(a.C, kChannels);
    a.apart = all <= kApart;
    const dim3 grid((unsigned)all);
    hipLaunchKernelGGL((scan_kernel<TI, L, kWaves, BACK, MIX>), grid, dim3(64 * kWaves), 0, s, a);
    return hipGetLastError();
}

template <bool BACK>
hipError_t run(const Scan& a, const ScanLaunch& p, hipStream_t s) {
    if (p.bf16) return p.mix ? run<bf16, BACK, true>(a, s) : run<bf16, BACK, false>(a, s);
    return p.mix ? run<float, BACK, true>(a, s) : run<float, BACK, false>(a, s);
}

}  // namespace

size_t scan_checkpoint_bytes(int64_t T, int32_t C) { return (size_t)up(T, kCheck) * C * sizeof(float); }
size_t scan_workspace_bytes(int64_t T, int32_t C) { return maps_bytes(T, C); }
size_t scan_backward_workspace_bytes(int64_t T, int32_t C) { return maps_bytes(T, C) + rounded(scan_checkpoint_bytes(T, C)); }

hipError_t launch_scan(const ScanLaunch& p, hipStream_t s) {
    if (p.num_seqs == 0) return hipSuccess;
    Scan a = arguments(p);
    a.states = p.checkpoints;
    return run<false>(a, p, s);
}

hipError_t launch_scan_backward(const ScanLaunch& p, hipStream_t s) {
    if (p.num_seqs == 0) return hipSuccess;
    Scan a = arguments(p);
    a.states = p.checkpoints;
    if (!p.checkpoints) {
        a.states = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + maps_bytes(p.T, p.C));
        const hipError_t e = run<false>(a, p, s);
        if (e != hipSuccess) return e;
    }
    return run<true>(a, p, s);
}

}  // namespace gdn
