// Shared by the two kernels of the attention over the 8-bit KV cache: the
// parameters, the line of units that the CTAs divide, and the partial sums
// that k_kv8_merge joins.
//
// A unit is PPU pages of one kv head, with all the query rows over it. All
// units of the batch stand in one line (request, kv head, page) and every CTA
// takes an equal share of it, so ragged lengths, many requests and a single
// long one are split alike; the lengths stay on the device. A CTA has tables of
// so many units in shared memory and takes a longer share in windows of that
// length: the launch and its scratch follow the device, not the width of the
// page table. The first window is one kernel, without a loop around it; where
// the page table has room for more, a second one follows and takes the others,
// or returns at once (0.7 to 1.5 us; in one kernel a loop over the windows, in
// line or out of line, cost the many-rows kernel 2 to 8% in registers).
// A run of units of one head within a window is a segment. A CTA writes the heads that it covers whole; a head that several
// CTAs share leaves one partial tile per CTA in scratch, and k_kv8_merge joins
// them in order. A head that goes on in the CTA's next window leaves its sums
// at the same place, and the next segment's end adds them to its own.
#pragma once

#include <cuda_fp16.h>

#include "lowbit.cuh"

namespace pe {
namespace kv8 {

constexpr int kPage = 16;
constexpr float kRescale = 8.f;    // running maximum (log2) moves only by more than this
// Weights meet V as fp16. What a row sums up is w * scale of v, and the scales
// of V's pages may lie far apart, so next to the scores' running maximum m a
// row has one of its contributions, mo, the maximum of score + log2(scale) over
// the pages, and the fp16 weights are w * scale * 2^(m - mo + kLift): the
// largest one stands between 2^kLift and 2^(kLift + kRescale + 2), and what
// falls below fp16's normal range, 2^-14, is 2^-19 of it at most. (Taken
// relative to the largest scale alone, a page of values below 2^-14 of the
// largest lost its bits even where it had all the weight.)
constexpr float kLift = 5.f;
// mark in the place of a row's sum: the request's outputs are zero
constexpr float kMarkBadPage = -1.f;

struct Kv8Params {
    int B, K, nq, nkv, max_pages, num_pages;
    const __nv_bfloat16* q;
    long long ld_q;
    const int32_t* seq_lens;
    const int32_t* rows;
    const int32_t* page_table;
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const float* k_scale;
    const float* v_scale;
    float scale_log2;
    __nv_bfloat16* out;
    long long ld_out;
    int32_t* status;
    int4* cut;         // [grid] OUT: the run that CTA c's share begins inside of: {request, head, unit of the
                       // run (0: none, -1: this CTA gave up), units of the run}; [grid]: {positions of a share, shares}
    int stall;         // tests: the barrier (a kStall*) that waits for an arrival too many
    float* part;       // [2 * grid] partial tiles (part_floats each): of a CTA's run that began in an earlier share, and of the other one
};

// a partial tile: O [tr][hd], the running maxima (log2) [tr], the sums [tr]
__host__ __device__ constexpr int part_floats(int tr, int hd) { return tr * hd + 2 * tr; }

// What request b asks for: its live rows, or a status.
struct Req {
    int st, S, rows, pages, run, span;   // run: units of one head; span: positions of all heads
};
template <int PPU, int PAD>
__device__ __forceinline__ Req request_of(const Kv8Params& p, int b) {
    Req r{PE_REQ_OK, p.seq_lens[b], p.rows != nullptr ? p.rows[b] : p.K, 0, 0, 0};
    if (r.S < 0 || r.rows < 0 || r.rows > p.K) r.st = PE_REQ_BAD_INPUT;
    else if (static_cast<long long>(r.S) + r.rows > static_cast<long long>(p.max_pages) * kPage)
        r.st = PE_REQ_CAPACITY;
    if (r.st != PE_REQ_OK) r.rows = 0;
    if (r.rows > 0) {
        r.pages = (r.S + r.rows + kPage - 1) / kPage;
        r.run = (r.pages + PPU - 1) / PPU;
        r.span = (r.run + PAD) * p.nkv;
    }
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// v = part * 2^lg exactly, |part| in [1, 2) for scales of 2^-104 to 2^127 (a
// smaller one is a smaller part, so that 2^-lg and what is summed stay normal)
__device__ __forceinline__ void split_scale(float v, float& part, float& lg) {
    const uint32_t e = min(max((__float_as_uint(v) >> 23) & 0xFFu, 23u), 253u);
    part = v * __uint_as_float((254u - e) << 23);
    lg = static_cast<float>(static_cast<int>(e) - 127);
}
// what scales a weight 2^(score - m) by, next to `part`; from: m - mo + kLift.
// Never an infinity, which would meet weights of 0
__device__ __forceinline__ float lift(float from, float lg) { return ex2(fminf(from + lg, 127.f)); }
// a sum of such products back to the values that belong to M
__device__ __forceinline__ float unlift(float mo, float M) { return mo == -INFINITY ? 0.f : ex2(mo - kLift - M); }
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// asynchronous copies of this thread (4, 8 or 16 bytes), in groups
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t smem, const void* src, uint64_t policy) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(smem), "l"(src), "l"(policy) : "memory");
    else
        asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], %3, %2;" ::"r"(smem), "l"(src), "l"(policy), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// bytes of w that are E4M3's NaN become 0; `any` collects whether there were some
__device__ __forceinline__ uint32_t without_nan(uint32_t w, int& any) {
    const uint32_t other = ((w & 0x7F7F7F7Fu) ^ 0x7F7F7F7Fu) + 0x7F7F7F7Fu;   // bit 7 of a byte: not NaN
    const uint32_t nan = ~other & 0x80808080u;
    any |= nan != 0;
    return w & ~((nan >> 7) * 0xFFu);
}

// The rows that no unit covers: rows past a request's own, and requests that
// have none or are refused; the requests b = blockIdx.x (mod gridDim.x) are
// this CTA's to look after. gather_units says whether there are any, so that a
// batch without them pays nothing. By warp my_warp of the CTA's `warps` first.
template <int PPU, int PAD>
__device__ __forceinline__ void zero_idle_rows_by(const Kv8Params& p, int hd, int my_warp, int warps) {
    const int lane = threadIdx.x & 31;
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        const Req r = request_of<PPU, PAD>(p, b);
        if (my_warp == 0 && lane == 0 && r.span == 0) p.status[b] = r.st;
        for (int j = r.rows + my_warp; j < p.K; j += warps) {
            uint4* o = reinterpret_cast<uint4*>(p.out + (static_cast<long long>(b) * p.K + j) * p.ld_out);
            for (int c = lane; c < p.nq * hd / 8; c += 32) o[c] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

// What a CTA has in its tables, besides the units.
struct Window {
    int w;              // its number
    bool carry, early;  // of the first segment: its head's sums so far stand in scratch; its run began in an earlier share
    bool more;          // the share goes on
};

// Window w of this CTA's share of the line, and its units' pages in shared memory:
// info[i] of a unit that begins a segment = {request, head, unit within its
// run, units of the run}; of page q of unit i, entry i * PPU + q of tile
// (page * nkv + head, -1: outside the pool, -2: behind the request's last
// page). Returns the number of units. idle: whether zero_idle_rows_by has work.
// All NT threads of the CTA, after a barrier behind the last use of the tables.
// A share is at least `least` positions, a window at most MAX, which is what
// the tables hold.
// Behind each run of units lie PAD positions without work: what the end of a
// segment costs, so that the shares' times are even, not their units alone.
// The requests of the share are listed first, from one scan over the batch, and
// then all threads look their pages up: two dependent loads (lengths, pages)
// and three barriers (B=1 K=7 13.6 us; with a scan for the total, one for the
// list and the lengths read again 14.5).
template <int NT, int PPU, int PAD, int MAX>
__device__ int gather_units(const Kv8Params& p, int least, int w, int4* info, int* tile, Window* win, bool& idle) {
    constexpr int kWarps = NT / 32, kList = 128;
    static_assert(kWarps <= 32 && MAX / (1 + PAD) + 2 <= kList, "requests of a share");
    __shared__ int s_span[kWarps], s_some[kWarps];
    __shared__ int4 s_list[kList];   // of the window: request, its first position, units of a head, pages; at its rank among the requests with units
    __shared__ int s_edge[2];        // ranks of the window's first and last request
    constexpr unsigned kAll = 0xffffffffu;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Req mine0 = tid < p.B ? request_of<PPU, PAD>(p, tid) : Req{};   // most batches fit the CTA's threads
    int total = 0;
    if (p.B > NT) {
        for (int b = tid + NT; b < p.B; b += NT) total += request_of<PPU, PAD>(p, b).span;
        total = __reduce_add_sync(kAll, total);
        if (lane == 0) s_span[warp] = total;
        __syncthreads();
        total = __reduce_add_sync(kAll, lane < kWarps ? s_span[lane] : 0);
        __syncthreads();
    }
    const int grid = static_cast<int>(gridDim.x);
    int per = 0, share = 0, lo = 0, hi = 0, base = 0, ranks = 0, rest = 0;
    bool more = false;
    for (int b0 = 0; b0 < p.B; b0 += NT) {
        const int b = b0 + tid;
        const Req r = b0 == 0 ? mine0 : (b < p.B ? request_of<PPU, PAD>(p, b) : Req{});
        int incl = r.span;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned some = __ballot_sync(kAll, r.span > 0);
        if (b0 > 0) __syncthreads();   // the last round's sums have been read
        if (lane == 31) {
            s_span[warp] = incl;
            s_some[warp] = __popc(some);
        }
        __syncthreads();
        const int span = lane < kWarps ? s_span[lane] : 0, count = lane < kWarps ? s_some[lane] : 0;
        const int spans = __reduce_add_sync(kAll, span);
        if (b0 == 0) {
            total += spans;
            per = max(least, (total + grid - 1) / grid);
            const long long at = static_cast<long long>(blockIdx.x) * per;
            share = static_cast<int>(min(at, static_cast<long long>(total)));
            lo = share + w * MAX;
            hi = static_cast<int>(min(static_cast<long long>(total), at + per));
            more = hi - lo > MAX;
            hi = more ? lo + MAX : hi;
        }
        rest |= b < p.B && r.rows < p.K && b % grid == static_cast<int>(blockIdx.x);
        const int u0 = base + __reduce_add_sync(kAll, lane < warp ? span : 0) + incl - r.span;
        const int rank = ranks + __reduce_add_sync(kAll, lane < warp ? count : 0) + __popc(some & ((1u << lane) - 1u));
        if (r.span > 0 && u0 < hi && u0 + r.span > lo) {
            s_list[rank % kList] = make_int4(b, u0, r.run, r.pages);
            if (u0 <= lo) s_edge[0] = rank;
            if (u0 + r.span >= hi) s_edge[1] = rank;
        }
        base += spans;
        ranks += __reduce_add_sync(kAll, count);
    }
    idle = __syncthreads_or(rest) != 0;
    if (tid == 0 && blockIdx.x == 0 && w == 0) p.cut[grid] = make_int4(per, grid, 0, 0);
    if (lo >= hi) {
        if (tid == 0) {
            if (w == 0) p.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
            *win = Window{w, false, false, false};
        }
        __syncthreads();
        return 0;
    }
    const int rank0 = s_edge[0], listed = s_edge[1] - rank0 + 1;
    const int4 front = s_list[rank0 % kList], back = s_list[(rank0 + listed - 1) % kList];
    // Units of the listed requests ahead of position `in` of head `head` of
    // listed request j: the positions less the padding of the runs ahead.
    auto units_to = [&](int j, const int4& of, int head, int in) {
        return of.y - front.y - PAD * p.nkv * j + head * of.z + min(in, of.z);
    };
    const int head0 = (lo - front.y) / (front.z + PAD), in0 = lo - front.y - head0 * (front.z + PAD);
    const int head1 = (hi - back.y) / (back.z + PAD), in1 = hi - back.y - head1 * (back.z + PAD);
    const int skip = units_to(0, front, head0, in0), n = units_to(listed - 1, back, head1, in1) - skip;
    const bool inside = in0 > 0 && in0 < front.z;   // the window begins inside of a run
    if (tid == NT - 1 && w == 0)
        p.cut[blockIdx.x] = inside ? make_int4(front.x, head0, in0, front.z) : make_int4(0, 0, 0, 0);
    for (int x = tid; x < (hi - lo) * PPU; x += NT) {
        const int u = lo + x / PPU;
        int j = 0;   // the last listed request that begins at or before u
        for (int step = listed; step > 1;) {
            step = (step + 1) / 2;
            if (j + step < listed && s_list[(rank0 + j + step) % kList].y <= u) j += step;
        }
        while (j + 1 < listed && s_list[(rank0 + j + 1) % kList].y <= u) ++j;
        const int4 of = s_list[(rank0 + j) % kList];
        const int head = (u - of.y) / (of.z + PAD), in = u - of.y - head * (of.z + PAD);
        if (in >= of.z) continue;
        const int i = units_to(j, of, head, in) - skip, q = x % PPU, page = in * PPU + q;
        int id = -2;
        if (page < of.w) {
            id = p.page_table[static_cast<size_t>(of.x) * p.max_pages + page];
            id = id >= 0 && id < p.num_pages ? id * p.nkv + head : -1;
        }
        tile[i * PPU + q] = id;
        if (q == 0 && (i == 0 || in == 0)) info[i] = make_int4(of.x, head, in, of.z);
    }
    if (tid == 0) *win = Window{w, inside && w > 0, inside && lo - in0 < share, more};
    __syncthreads();
    return n;
}

__device__ __forceinline__ int status_of(float mark) {
    return mark == 0.f ? PE_REQ_OK : PE_REQ_BAD_PAGE;
}

constexpr int kStallK = 1, kStallV = 2, kStallP = 3;   // K codes, V tiles, weights

struct Plan {
    int tr;                  // rows of a tile
    int grid, sms, dev;      // a CTA per multiprocessor at most
    long long most;          // positions of the line at most
    size_t cut_floats, ws_floats;
};

int launch_merge(const Kv8Params& p, const Plan& a, int hd, cudaStream_t s);
// rows past which the tensor-memory kernel takes over, and its launch
int launch_umma(const Kv8Params& p, const Plan& a, int hd, cudaStream_t s);
constexpr int kUmmaPages = 4, kUmmaRows = 128, kUmmaUnits = 640;
// A share's positions at least (B=1 K=7, 2048 entries: 14.9 us, with 1 15.5, with 6 16.6), and the units' worth of a
// segment's end (B=128 K=11: 190 us, with 0 208; 64-wide heads 87 and 91; as all of these were then)
constexpr int kUmmaLeast = 3, kUmmaPad = 7;

}  // namespace kv8
}  // namespace pe
