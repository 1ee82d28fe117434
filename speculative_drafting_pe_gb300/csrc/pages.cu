// Pages for a batch on the device: block tables and slot maps from request
// lengths (pe_assign_pages), and the pages of shortened or finished requests
// back to the free stack (pe_release_pages).
//
// With S_b committed entries, n_b new ones and c_b pages already in its row,
// request b needs ceil((S_b + n_b) / 16) pages and takes
//   grow_b = max(0, need_b - c_b)
// from the top of the stack, in request order: with E_b = sum_{b' < b} grow_b'
// and F free pages, table[b][c_b + i] = free[F - 1 - E_b - i]. A request is
// served while E_b + grow_b <= F.
//
// pe_assign_pages is one launch with no state that one block writes and
// another reads: every block sums E_b itself from the (small) length arrays,
// reads the table below c_b only and writes it from c_b on, and the new counts
// go to arrays of their own. It is bound by latency: three dependent loads
// (lengths, stack, slots) and a block sum. 64 requests with 8 new entries each
// take 2.9 us (in a captured run, where a launch alone is about 2), 256
// prompts of up to 2048 entries 4.1 us, 0.57 TB/s of slots and pages.
#include "common.cuh"
#include "internal.h"

namespace pe {
namespace {

constexpr int kPage = 16;
constexpr int kAssignThreads = 128;
constexpr int kSlotsPerBlock = 2048;   // new entries of one request that one block maps

struct Want {
    int st;      // PE_REQ_OK, _BAD_INPUT or _CAPACITY by the request alone
    int count;   // pages in its row
    int need;    // pages it needs in all
    int grow;    // pages it takes
};

__device__ __forceinline__ Want want_of(int S, int n, int c, int n_max, int max_pages) {
    Want w{PE_REQ_OK, c, 0, 0};
    if (S < 0 || n < 0 || n > n_max || c < 0 || c > max_pages || S > static_cast<long long>(c) * kPage) {
        w.st = PE_REQ_BAD_INPUT;
        return w;
    }
    const long long need = (static_cast<long long>(S) + n + kPage - 1) / kPage;
    if (need > max_pages) {
        w.st = PE_REQ_CAPACITY;
        return w;
    }
    w.need = static_cast<int>(need);
    w.grow = w.need > c ? w.need - c : 0;
    return w;
}

__global__ void __launch_bounds__(kAssignThreads)
    k_assign_pages(int B, const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ new_lens,
                   const int32_t* __restrict__ counts, int32_t* __restrict__ counts_out, int32_t* page_table,
                   int max_pages, const int32_t* __restrict__ free_pages, int free_cap,
                   const int32_t* __restrict__ free_count, int32_t* __restrict__ free_count_out, int num_pages,
                   int n_max, int32_t* __restrict__ slots, int32_t* __restrict__ status) {
    __shared__ long long s_sum[kAssignThreads / 32];
    __shared__ int s_lost;
    const int tid = threadIdx.x;
    const int F = min(max(free_count[0], 0), free_cap);
    long long before = 0;   // E_b: pages wanted by the requests below b
    int summed = 0;
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
        const int S = seq_lens[b], n = new_lens[b];
        const Want w = want_of(S, n, counts[b], n_max, max_pages);
        long long part = 0;
        for (int i = summed + tid; i < b; i += kAssignThreads)
            part += want_of(seq_lens[i], new_lens[i], counts[i], n_max, max_pages).grow;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        __syncthreads();
        if ((tid & 31) == 0) s_sum[tid >> 5] = part;
        if (tid == 0) s_lost = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kAssignThreads / 32; ++i) before += s_sum[i];
        summed = b;

        const bool short_ = w.grow > 0 && before + w.grow > F;
        const int take = short_ ? 0 : w.grow;
        int st = w.st != PE_REQ_OK ? w.st : (short_ ? PE_REQ_CAPACITY : PE_REQ_OK);
        int32_t* row = page_table + static_cast<size_t>(b) * max_pages;
        const int top = static_cast<int>(F - 1 - before);   // in range where take > 0
        auto page_of = [&](int i) { return i < w.count ? row[i] : free_pages[top - (i - w.count)]; };
        if (st == PE_REQ_OK) {
            int lost = 0;
            const int p_end = n > 0 ? w.need : 0;
            for (int i = S / kPage + tid; i < p_end; i += kAssignThreads) {
                const int pg = page_of(i);
                if (pg < 0 || pg >= num_pages) lost = 1;
            }
            if (lost) s_lost = 1;
        }
        __syncthreads();
        if (st == PE_REQ_OK && s_lost) st = PE_REQ_BAD_PAGE;
        for (int i = blockIdx.y * kAssignThreads + tid; i < take; i += gridDim.y * kAssignThreads)
            row[w.count + i] = free_pages[top - i];
        int32_t* out = slots + static_cast<size_t>(b) * n_max;
        const int i1 = min(n_max, static_cast<int>(blockIdx.y + 1) * kSlotsPerBlock);
        for (int i = blockIdx.y * kSlotsPerBlock + tid; i < i1; i += kAssignThreads) {
            int slot = -1;
            if (st == PE_REQ_OK && i < n) {
                const int e = S + i;
                slot = page_of(e / kPage) * kPage + e % kPage;
            }
            out[i] = slot;
        }
        if (blockIdx.y == 0 && tid == 0) {
            status[b] = st;
            counts_out[b] = w.count + take;
            // the first request that the stack cannot serve, or the last one
            // of a batch that it serves whole, knows what is left
            if (short_ && before <= F) free_count_out[0] = static_cast<int>(F - before);
            else if (b == B - 1 && before + w.grow <= F) free_count_out[0] = static_cast<int>(F - before - w.grow);
        }
        before += w.grow;
        summed = b + 1;
    }
}

// One block over the whole batch, 1024 requests at a time: a thread per
// request finds what it gives back; the warps check the given ids together
// (coalesced), the block sums the counts in request order, and the warps push
// the ids. Requests that give nothing back, nearly all of them in a step,
// cost two loads.
constexpr int kReleaseThreads = 1024;

__global__ void __launch_bounds__(kReleaseThreads)
    k_release_pages(int B, const int32_t* keep_lens, const int32_t* counts, int32_t* counts_out, int32_t* page_table,
                    int max_pages, int32_t* free_pages, int free_cap, const int32_t* free_count,
                    int32_t* free_count_out, int num_pages, int32_t* status) {   // counts and free_count in place as well
    __shared__ long long s_sum[kReleaseThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int F = min(max(free_count[0], 0), free_cap);
    long long before = 0;   // ids given back by the requests below this chunk
    int pushed = 0;         // of those, the ones that the stack had room for (the prefix that fits)
    for (int b0 = 0; b0 < B; b0 += kReleaseThreads) {
        const int b = b0 + tid;
        int st = PE_REQ_OK, keep = 0, give = 0, c = 0;
        if (b < B) {
            const int n = keep_lens[b];
            c = counts[b];
            if (n < 0 || c < 0 || c > max_pages || n > static_cast<long long>(c) * kPage) st = PE_REQ_BAD_INPUT;
            else {
                keep = (n + kPage - 1) / kPage;
                give = c - keep;
            }
        }
        // ids to be given back are pages of the pool, or the request keeps all
        for (unsigned todo = __ballot_sync(0xffffffffu, give > 0); todo; todo &= todo - 1) {
            const int src = __ffs(todo) - 1;
            const int k = __shfl_sync(0xffffffffu, keep, src), e = __shfl_sync(0xffffffffu, c, src);
            const int32_t* row = page_table + static_cast<size_t>(b0 + warp * 32 + src) * max_pages;
            int bad = 0;
            for (int i = k + lane; i < e; i += 32) bad |= row[i] < 0 || row[i] >= num_pages;
            if (__any_sync(0xffffffffu, bad) && lane == src) {
                st = PE_REQ_BAD_PAGE;
                give = 0;
            }
        }
        long long incl = give;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) s_sum[warp] = incl;
        __syncthreads();
        long long base = before, total = before;
        for (int i = 0; i < kReleaseThreads / 32; ++i) {
            if (i < warp) base += s_sum[i];
            total += s_sum[i];
        }
        incl += base;
        if (give > 0 && F + incl > free_cap) {
            st = PE_REQ_CAPACITY;
            give = 0;
        }
        const long long first = incl - give;   // meaningful where give > 0
        for (unsigned todo = __ballot_sync(0xffffffffu, give > 0); todo; todo &= todo - 1) {
            const int src = __ffs(todo) - 1;
            const int k = __shfl_sync(0xffffffffu, keep, src), e = __shfl_sync(0xffffffffu, c, src);
            const long long at = F + __shfl_sync(0xffffffffu, first, src);
            int32_t* row = page_table + static_cast<size_t>(b0 + warp * 32 + src) * max_pages;
            for (int i = k + lane; i < e; i += 32) {
                free_pages[at + (i - k)] = row[i];
                row[i] = -1;
            }
        }
        if (b < B) {
            status[b] = st;
            counts_out[b] = c - give;
        }
        __syncthreads();   // s_sum has been read
        // pages pushed by this chunk
        long long mine = give;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        if (lane == 0) s_sum[warp] = mine;
        __syncthreads();
        for (int i = 0; i < kReleaseThreads / 32; ++i) pushed += static_cast<int>(s_sum[i]);
        __syncthreads();
        before = total;
    }
    if (tid == 0) free_count_out[0] = F + pushed;
}

int check_pages(int B, int max_pages, int num_pages, int free_cap) {
    if (B < 1) { set_error("B must be >= 1"); return PE_ERR_ARG; }
    if (max_pages < 1 || num_pages < 1 || free_cap < 1) {
        set_error("max_pages, num_pages and free_cap must be >= 1");
        return PE_ERR_ARG;
    }
    if (num_pages > 0x7FFFFFFF / kPage || max_pages > 0x7FFFFFFF / kPage - 2) {
        set_error("num_pages * 16 and max_pages * 16 must fit a signed 32-bit entry index");
        return PE_ERR_ARG;
    }
    return PE_OK;
}

}  // namespace
}  // namespace pe

using namespace pe;

extern "C" int pe_assign_pages(int32_t B, const int32_t* seq_lens, const int32_t* new_lens,
                               const int32_t* page_counts, int32_t* page_counts_out, int32_t* page_table,
                               int32_t max_pages, int32_t num_pages, const int32_t* free_pages, int32_t free_cap,
                               const int32_t* free_count, int32_t* free_count_out, int32_t n_max,
                               int32_t* slot_mapping, int32_t* status, void* stream) {
    int rc = check_pages(B, max_pages, num_pages, free_cap);
    if (rc != PE_OK) return rc;
    if (n_max < 1) { set_error("n_max must be >= 1"); return PE_ERR_ARG; }
    if (!seq_lens || !new_lens || !page_counts || !page_counts_out || !page_table || !free_pages || !free_count ||
        !free_count_out || !slot_mapping || !status) {
        set_error("null tensor argument");
        return PE_ERR_ARG;
    }
    if (page_counts == page_counts_out || free_count == free_count_out) {
        set_error("page_counts_out and free_count_out must not alias their inputs");
        return PE_ERR_ARG;
    }
    const unsigned gy = static_cast<unsigned>((static_cast<long long>(n_max) + kSlotsPerBlock - 1) / kSlotsPerBlock);
    if (gy > 65535u) { set_error("n_max too large"); return PE_ERR_ARG; }
    const dim3 grid(B < 1024 ? B : 1024, gy);
    PE_CUDA_TRY(launch_ex(k_assign_pages, grid, dim3(kAssignThreads), 0, static_cast<cudaStream_t>(stream), false, B,
                          seq_lens, new_lens, page_counts, page_counts_out, page_table, max_pages, free_pages,
                          free_cap, free_count, free_count_out, num_pages, n_max, slot_mapping, status));
    return PE_OK;
}

extern "C" int pe_release_pages(int32_t B, const int32_t* keep_lens, const int32_t* page_counts,
                                int32_t* page_counts_out, int32_t* page_table, int32_t max_pages, int32_t num_pages,
                                int32_t* free_pages, int32_t free_cap, const int32_t* free_count,
                                int32_t* free_count_out, int32_t* status, void* stream) {
    int rc = check_pages(B, max_pages, num_pages, free_cap);
    if (rc != PE_OK) return rc;
    if (!keep_lens || !page_counts || !page_counts_out || !page_table || !free_pages || !free_count ||
        !free_count_out || !status) {
        set_error("null tensor argument");
        return PE_ERR_ARG;
    }
    PE_CUDA_TRY(launch_ex(k_release_pages, dim3(1), dim3(kReleaseThreads), 0, static_cast<cudaStream_t>(stream),
                          false, B, keep_lens, page_counts, page_counts_out, page_table, max_pages, free_pages,
                          free_cap, free_count, free_count_out, num_pages, status));
    return PE_OK;
}
