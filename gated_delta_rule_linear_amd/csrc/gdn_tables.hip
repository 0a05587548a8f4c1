// Block tables, slot map, positions and packed offsets of one step, from the
// requests' lengths (gdn_batch_tables).
//
// Two prefix sums decide everything: over the new tokens (the packed offsets)
// and over the pages that requests need (which free pages each one gets).  With
// n requests and T new tokens the step reads 7 n integers and writes 2 T, so
// even the largest is a few megabytes: it is bound by launches and by a chain
// of dependent loads, not by bandwidth.  One workgroup runs the sums (512
// requests per turn; a wave's sums by cross-lane adds in registers, the eight
// waves' through LDS).  The tokens, each of which only has to find its request,
// are filled by that workgroup in the same launch when there are few of them
// and of the requests, whose data then stays in LDS, and otherwise by a second
// launch over the whole device.  Measured in a graph, where a launch that does
// nothing is 3.5 us: 512 requests of one token 8.8 to 9.0 us, 64 prompts of 512 to 16,384
// tokens (4.3 MB written) 9.2 to 9.3 us.
#include "gdn_device.h"
#include "gdn_serve_kernels.h"

namespace gdn {
namespace {

constexpr int kScan = 512;       // threads of the summing workgroup
constexpr int kFill = 256;       // threads of a fill workgroup
constexpr int kPerThread = 4;    // tokens per thread of the fill step
constexpr int kCuLds = 4096;     // offsets held in LDS by the fill step
// Up to so many tokens (and kScan requests) one launch does all.  64 requests,
// one launch / two: 2,048 tokens 6.6 / 8.5 us, 4,096 tokens 9.0 / 8.4, 8,192 13.6 / 8.5.
constexpr int64_t kOneLaunch = 2048;

struct Tables {
    const int32_t *ctx, *nw, *rows;
    int32_t num_seqs;
    int32_t T, page_log2, max_blocks, num_rows, num_pages;
    int32_t *table, *counts, *free_pages, *state, *cu, *kv, *slots, *pos;
    TablesRequest* req;
};

// x + (x of the lane that the DPP control names, 0 where there is none).
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t add_dpp(int64_t x) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, CTRL, ROWS, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)((uint64_t)x >> 32), CTRL, ROWS, 0xf, false);
    return x + (int64_t)(((uint64_t)hi << 32) | lo);
}
// Inclusive sum over the 64 lanes: shifts by 1, 2, 4, 8 within rows of 16 lanes,
// then the rows' last lanes broadcast to the next row and to the upper half.
__device__ __forceinline__ int64_t wave_sum(int64_t x) {
    x = add_dpp<0x111, 0xf>(x);
    x = add_dpp<0x112, 0xf>(x);
    x = add_dpp<0x114, 0xf>(x);
    x = add_dpp<0x118, 0xf>(x);
    x = add_dpp<0x142, 0xa>(x);
    x = add_dpp<0x143, 0xc>(x);
    return x;
}

// Inclusive sums over the workgroup of kScan threads; all receives the totals.
// The two calls of a turn have LDS of their own: between two uses of either lies
// the barrier of the other.
__device__ __forceinline__ void block_sums(int64_t& x, int64_t& y, int64_t (*lds)[2], int64_t (&all)[2]) {
    const int wave = threadIdx.x >> 6;
    x = wave_sum(x);
    y = wave_sum(y);
    if ((threadIdx.x & 63) == 63) {
        lds[wave][0] = x;
        lds[wave][1] = y;
    }
    __syncthreads();
    int64_t bx = 0, by = 0;
    all[0] = all[1] = 0;
#pragma unroll
    for (int w = 0; w < kScan / 64; ++w) {
        const int64_t sx = lds[w][0], sy = lds[w][1];
        if (w < wave) {
            bx += sx;
            by += sy;
        }
        all[0] += sx;
        all[1] += sy;
    }
    x += bx;
    y += by;
}

__device__ __forceinline__ int32_t ring_place(int64_t at, int32_t cap) {  // at < 3 cap
    if (at >= cap) at -= cap;
    if (at >= cap) at -= cap;
    return (int32_t)at;
}

// Slot and position of token t.  `cu` and `req` are in LDS or global memory.
__device__ __forceinline__ void fill_token(const Tables& a, const int32_t* cu, const TablesRequest* req, int32_t t,
                                           int32_t& slot, int32_t& pos) {
    slot = -1;
    pos = 0;
    if (t >= cu[a.num_seqs]) return;
    int lo = 0, hi = a.num_seqs;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    const TablesRequest r = req[lo];
    const uint32_t p = (uint32_t)r.ctx + (uint32_t)(t - cu[lo]);
    pos = (int32_t)p;
    if (r.row < 0) return;
    const int32_t block = (int32_t)(p >> a.page_log2), place = (int32_t)(p & ((1u << a.page_log2) - 1));
    int32_t* entry = a.table + (int64_t)r.row * a.max_blocks + block;
    int64_t page;
    if (block >= r.base) {  // a page of this call; the token at its start enters it
        page = a.free_pages[ring_place((int64_t)r.ring + (block - r.base), a.num_pages)];
        if (place == 0) *entry = (int32_t)page;
    } else {
        page = *entry;
    }
    const int64_t s = page * (1 << a.page_log2) + place;
    if (page >= 0 && s <= INT32_MAX) slot = (int32_t)s;
}

// Pages of an ended request to the ring's end.
__device__ __forceinline__ void give_back(const Tables& a, const TablesRequest& r, int first, int step) {
    int32_t* row = a.table + (int64_t)r.row * a.max_blocks;
    for (int j = first; j < r.given; j += step) {
        a.free_pages[((int64_t)r.ring + j) % a.num_pages] = row[j];
        row[j] = -1;
    }
}

template <bool ALL>
__global__ __launch_bounds__(kScan) void tables_scan_kernel(Tables a) {
    __shared__ int64_t s_sum[2][kScan / 64][2];
    __shared__ int32_t s_taken, s_refused;
    __shared__ int32_t s_cu[ALL ? kScan + 1 : 1];
    __shared__ TablesRequest s_req[ALL ? kScan : 1];
    const int tid = threadIdx.x;
    const int64_t page = (int64_t)1 << a.page_log2;
    const int32_t cap = a.num_pages;
    // The state as it was: every thread reads it before the last barrier, thread
    // 0 changes it after that.
    int32_t head = a.state[0], left = a.state[1];
    if (tid == 0) {
        s_taken = s_refused = 0;
        s_cu[0] = 0;
    }
    if (cap == 0) head = left = 0;
    else if (head < 0 || head >= cap) head = (int32_t)(((int64_t)head % cap + cap) % cap);
    left = left < 0 ? 0 : left > cap ? cap : left;

    int64_t tokens = 0, pages = 0, back = 0;  // of the requests before this turn
    for (int64_t first = 0; first < a.num_seqs; first += kScan) {
        const int64_t n = first + tid;
        const bool live = n < a.num_seqs;
        int64_t ctx = 0, nw = 0, owned = 0;
        int32_t row = -1;
        if (live) {
            row = a.rows ? a.rows[n] : (int32_t)n;
            ctx = a.ctx[n];
            nw = a.nw[n];
            if (ctx < 0) ctx = 0;
            if (row < 0 || row >= a.num_rows) row = -1;
            if (row >= 0) {
                owned = a.counts[row];
                owned = owned < 0 ? 0 : owned > a.max_blocks ? a.max_blocks : owned;
            }
        }
        const bool ended = live && nw < 0;
        if (nw < 0) nw = 0;
        const int64_t given = ended && row >= 0 && cap > 0 ? owned : 0;
        int64_t all[2], end = nw, gave = given;
        block_sums(end, gave, s_sum[0], all);
        end += tokens;
        gave += back;
        tokens += all[0];
        back += all[1];
        const int64_t c1 = end < a.T ? end : a.T, c0 = end - nw < a.T ? end - nw : a.T;
        const int64_t held = (ctx + page - 1) >> a.page_log2, last = (ctx + (c1 - c0) + page - 1) >> a.page_log2;
        const bool room = live && !ended && row >= 0 && last <= a.max_blocks && held <= owned;
        const int64_t need = room && last > owned ? last - owned : 0;
        int64_t upto = need, none = 0;
        block_sums(upto, none, s_sum[1], all);
        upto += pages;
        pages += all[0];
        const bool fine = room && (need == 0 || upto <= left);
        if (need > 0 && fine) atomicAdd(&s_taken, (int32_t)need);  // sums of integers: any order
        if (live && !ended && !fine) atomicAdd(&s_refused, 1);
        if (live) {
            a.cu[n + 1] = (int32_t)c1;
            const int64_t kv = ended ? 0 : fine ? ctx + (c1 - c0) : ctx;
            a.kv[n] = (int32_t)(kv < INT32_MAX ? kv : INT32_MAX);
            if (row >= 0 && (fine || ended)) {
                const int32_t count = ended ? 0 : (int32_t)(owned + need);
                if (count != owned) a.counts[row] = count;
            }
            TablesRequest r;
            r.row = fine || ended ? row : -1;
            r.ctx = (int32_t)ctx;
            r.base = (int32_t)owned;
            r.given = (int32_t)given;
            r.ring = 0;
            if (ended && cap > 0) r.ring = (int32_t)((head + left + (gave - given)) % cap);
            else if (fine && need > 0) r.ring = ring_place(head + (upto - need), cap);
            if constexpr (ALL) {
                s_cu[n + 1] = (int32_t)c1;
                s_req[n] = r;
            } else {
                a.req[n] = r;
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        a.cu[0] = 0;
        a.state[0] = cap > 0 ? ring_place((int64_t)head + s_taken, cap) : 0;
        const int64_t now = left - s_taken + back;
        a.state[1] = (int32_t)(now < cap ? now : cap);
        a.state[2] = s_refused;
    }
    if constexpr (ALL) {
        for (int32_t t = tid; t < a.T; t += kScan) {
            int32_t slot, pos;
            fill_token(a, s_cu, s_req, t, slot, pos);
            a.slots[t] = slot;
            a.pos[t] = pos;
        }
        for (int n = tid >> 6; n < a.num_seqs; n += kScan / 64) {
            const TablesRequest r = s_req[n];
            if (r.given > 0) give_back(a, r, tid & 63, 64);
        }
    }
}

__global__ __launch_bounds__(kFill) void tables_fill_kernel(Tables a, int32_t token_blocks) {
    __shared__ int32_t s_cu[kCuLds];
    if ((int)blockIdx.x >= token_blocks) {  // the last blocks take the ended requests
        for (int n = blockIdx.x - token_blocks; n < a.num_seqs; n += gridDim.x - token_blocks) {
            const TablesRequest r = a.req[n];
            if (r.given > 0) give_back(a, r, threadIdx.x, kFill);
        }
        return;
    }
    const int32_t* cu = a.cu;
    if (a.num_seqs < kCuLds) {
        for (int i = threadIdx.x; i <= a.num_seqs; i += kFill) s_cu[i] = a.cu[i];
        __syncthreads();
        cu = s_cu;
    }
    const int64_t first = (int64_t)blockIdx.x * kFill * kPerThread + threadIdx.x;
    int32_t slot[kPerThread], pos[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int64_t t = first + i * kFill;
        if (t < a.T) fill_token(a, cu, a.req, (int32_t)t, slot[i], pos[i]);
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int64_t t = first + i * kFill;
        if (t < a.T) {
            a.slots[t] = slot[i];
            a.pos[t] = pos[i];
        }
    }
}

}  // namespace

size_t tables_workspace_bytes(int32_t num_seqs, int64_t) {
    return ((size_t)num_seqs * sizeof(TablesRequest) + 255) & ~(size_t)255;
}

hipError_t launch_tables(const TablesLaunch& p, hipStream_t s) {
    Tables a;
    a.ctx = p.context_lens; a.nw = p.new_lens; a.rows = p.rows;
    a.num_seqs = p.num_seqs; a.T = (int32_t)p.T_total;
    a.page_log2 = p.page_size == 64 ? 6 : p.page_size == 128 ? 7 : 8;
    a.max_blocks = p.max_blocks; a.num_rows = p.num_rows; a.num_pages = p.num_pages;
    a.table = p.block_table; a.counts = p.page_counts; a.free_pages = p.free_pages; a.state = p.free_state;
    a.cu = p.cu_seqlens; a.kv = p.kv_lens; a.slots = p.slots; a.pos = p.positions;
    a.req = static_cast<TablesRequest*>(p.workspace);
    if (p.T_total <= kOneLaunch && p.num_seqs <= kScan) {
        hipLaunchKernelGGL(tables_scan_kernel<true>, dim3(1), dim3(kScan), 0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(tables_scan_kernel<false>, dim3(1), dim3(kScan), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int32_t per = kFill * kPerThread, blocks = (int32_t)((p.T_total + per - 1) / per);
    const int32_t enders = p.num_seqs < 64 ? p.num_seqs : 64;
    if (blocks + enders == 0) return hipSuccess;
    hipLaunchKernelGGL(tables_fill_kernel, dim3((unsigned)(blocks + enders)), dim3(kFill), 0, s, a, blocks);
    return hipGetLastError();
}

}  // namespace gdn
