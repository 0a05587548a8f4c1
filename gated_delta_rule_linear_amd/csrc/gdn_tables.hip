// Block tables, slot map, positions and packed offsets of one step, from the
// requests' lengths (gdn_batch_tables).
//
// Two prefix sums decide everything: over the new tokens (the packed offsets)
// and over the pages that requests need (which free pages each one gets).  With
// n requests and T new tokens the step reads 7 n integers and writes 2 T, so
// even the largest is a few megabytes: it is bound by launches and by the
// latency of the sums, not by bandwidth.  One workgroup runs the sums (1024
// requests per turn, sums of a wave in registers, of the 16 waves through LDS);
// the tokens, each of which only has to find its request, are filled by that
// same workgroup in the same launch when there are few and by a second launch
// over the whole device when there are many.
#include "gdn_device.h"
#include "gdn_serve_kernels.h"

namespace gdn {
namespace {

constexpr int kScan = 1024;      // threads of the summing workgroup
constexpr int kFill = 256;       // threads of a fill workgroup
constexpr int kPerThread = 4;    // tokens per thread of the fill step
constexpr int kCuLds = 4096;     // offsets held in LDS by the fill step
constexpr int64_t kOneLaunch = 8192;  // up to so many tokens one launch does all

struct Tables {
    const int32_t *ctx, *nw, *rows;
    int32_t num_seqs;
    int32_t T, page, max_blocks, num_rows, num_pages;
    int32_t *table, *counts, *free_pages, *state, *cu, *kv, *slots, *pos;
    TablesRequest* req;
};

// Inclusive sum over the workgroup of kScan threads; *total receives the whole.
__device__ int64_t block_sum(int64_t x, int64_t* lds, int64_t* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t y = __shfl_up(x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();  // the last use of lds
    if (lane == 63) lds[wave] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kScan / 64; ++w) {
        const int64_t s = lds[w];
        if (w < wave) before += s;
        all += s;
    }
    *total = all;
    return x + before;
}

// Slot and position of token t.  `cu` is in LDS or global memory.
__device__ __forceinline__ void fill_token(const Tables& a, const int32_t* cu, int32_t t, int32_t& slot, int32_t& pos) {
    slot = -1;
    pos = 0;
    if (t >= cu[a.num_seqs]) return;
    int lo = 0, hi = a.num_seqs;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    const TablesRequest r = a.req[lo];
    const int64_t p = (int64_t)r.ctx + (t - cu[lo]);
    pos = (int32_t)p;
    if (r.row < 0) return;
    const int64_t block = p / a.page;
    const int32_t place = (int32_t)(p - block * a.page);
    int64_t page;
    int32_t* entry = a.table + (int64_t)r.row * a.max_blocks + block;
    if (block >= r.base) {  // a page of this call; the token at its start enters it
        page = a.free_pages[(r.ring + (block - r.base)) % a.num_pages];
        if (place == 0) *entry = (int32_t)page;
    } else {
        page = *entry;
    }
    const int64_t s = page * a.page + place;
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
    __shared__ int64_t lds[kScan / 64];
    const int tid = threadIdx.x;
    const int64_t cap = a.num_pages;
    // The state as it was: read by every thread before the last one changes it.
    int64_t head = cap > 0 ? a.state[0] % cap : 0;
    if (head < 0) head += cap;
    int64_t left = a.state[1];
    left = left < 0 ? 0 : left > cap ? cap : left;

    int64_t tokens = 0, pages = 0, taken = 0, back = 0, refused = 0;  // of the requests before this turn
    for (int64_t first = 0; first < a.num_seqs; first += kScan) {
        const int64_t n = first + tid;
        const bool live = n < a.num_seqs;
        int64_t ctx = 0, nw = 0, owned = 0;
        int32_t row = -1;
        if (live) {
            ctx = a.ctx[n];
            if (ctx < 0) ctx = 0;
            nw = a.nw[n];
            row = a.rows ? a.rows[n] : (int32_t)n;
            if (row < 0 || row >= a.num_rows) row = -1;
            if (row >= 0) {
                owned = a.counts[row];
                owned = owned < 0 ? 0 : owned > a.max_blocks ? a.max_blocks : owned;
            }
        }
        const bool ended = live && nw < 0;
        if (nw < 0) nw = 0;
        int64_t all;
        const int64_t end = tokens + block_sum(nw, lds, &all);
        const int64_t c1 = end < a.T ? end : a.T, c0 = end - nw < a.T ? end - nw : a.T;
        tokens += all;
        const int64_t held = (ctx + a.page - 1) / a.page;
        const int64_t last = (ctx + (c1 - c0) + a.page - 1) / a.page;
        const bool room = live && !ended && row >= 0 && last <= a.max_blocks && held <= owned;
        const int64_t need = room && last > owned ? last - owned : 0;
        const int64_t upto = pages + block_sum(need, lds, &all);
        pages += all;
        const bool fine = room && (need == 0 || upto <= left);
        const int64_t given = ended && row >= 0 && cap > 0 ? owned : 0;
        const int64_t gave = back + block_sum(given, lds, &all);
        back += all;
        (void)block_sum(fine ? need : 0, lds, &all);
        taken += all;
        (void)block_sum(live && !ended && !fine ? 1 : 0, lds, &all);
        refused += all;
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
            r.ring = cap > 0 ? (int32_t)((ended ? head + left + (gave - given) : head + (upto - need)) % cap) : 0;
            r.given = (int32_t)given;
            a.req[n] = r;
        }
    }
    if (tid == 0) {
        a.cu[0] = 0;
        a.state[0] = cap > 0 ? (int32_t)((head + taken) % cap) : 0;
        a.state[1] = (int32_t)(left - taken + back < cap ? left - taken + back : cap);
        a.state[2] = (int32_t)refused;
    }
    if (!ALL) return;
    __syncthreads();  // cu and req, written by this workgroup, are read by it
    for (int32_t t = tid; t < a.T; t += kScan) {
        int32_t slot, pos;
        fill_token(a, a.cu, t, slot, pos);
        a.slots[t] = slot;
        a.pos[t] = pos;
    }
    for (int n = tid >> 6; n < a.num_seqs; n += kScan / 64) {
        const TablesRequest r = a.req[n];
        if (r.given > 0) give_back(a, r, tid & 63, 64);
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
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int64_t t = first + i * kFill;
        if (t >= a.T) return;
        int32_t slot, pos;
        fill_token(a, cu, (int32_t)t, slot, pos);
        a.slots[t] = slot;
        a.pos[t] = pos;
    }
}

}  // namespace

size_t tables_workspace_bytes(int32_t num_seqs, int64_t) {
    return ((size_t)num_seqs * sizeof(TablesRequest) + 255) & ~(size_t)255;
}

hipError_t launch_tables(const TablesLaunch& p, hipStream_t s) {
    Tables a;
    a.ctx = p.context_lens; a.nw = p.new_lens; a.rows = p.rows;
    a.num_seqs = p.num_seqs; a.T = (int32_t)p.T_total; a.page = p.page_size;
    a.max_blocks = p.max_blocks; a.num_rows = p.num_rows; a.num_pages = p.num_pages;
    a.table = p.block_table; a.counts = p.page_counts; a.free_pages = p.free_pages; a.state = p.free_state;
    a.cu = p.cu_seqlens; a.kv = p.kv_lens; a.slots = p.slots; a.pos = p.positions;
    a.req = static_cast<TablesRequest*>(p.workspace);
    if (p.T_total <= kOneLaunch) {
        hipLaunchKernelGGL(tables_scan_kernel<true>, dim3(1), dim3(kScan), 0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(tables_scan_kernel<false>, dim3(1), dim3(kScan), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int32_t per = kFill * kPerThread, blocks = (int32_t)((p.T_total + per - 1) / per);
    const int32_t enders = p.num_seqs < 64 ? p.num_seqs : 64;
    hipLaunchKernelGGL(tables_fill_kernel, dim3((unsigned)(blocks + enders)), dim3(kFill), 0, s, a, blocks);
    return hipGetLastError();
}

}  // namespace gdn
