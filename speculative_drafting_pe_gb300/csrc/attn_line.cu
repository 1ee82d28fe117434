// What the attention over any of the low-bit KV caches shares on the host's
// side of a launch, and the kernel that joins what several CTAs have of a head.
#include <algorithm>

#include "attn_line.cuh"

namespace pe {
namespace {

using namespace line;

// Joins the parts of every head that several CTAs share, in unit order. The
// part that a CTA left of such a run is its first one where the run began in
// an earlier share, its second one otherwise. Every block lists the cut runs
// and takes its blocks of rows from them (a block for every head and row, most
// of them with nothing to do, took 18.6 us at B=128 K=11). A
// thread per row and four dimensions; the parts are read eight at a time, all
// loads of a batch in flight, and folded with a running maximum. Where rows
// are few and parts many (one long request), SHARE teams of threads take a row
// together, each a run of its parts, and their sums meet in shared memory.
constexpr int kMergeThreads = 128;
constexpr int kMergeBatch = 8;
constexpr int kMergeBlocks = 16;   // blocks for an SM at most (6 to 40 measure alike)

struct Joined {
    float M = -INFINITY, bad = 0.f, total = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void raise(float top) {   // to a larger maximum
        if (top > M) {
            const float f = M == -INFINITY ? 0.f : ex2(M - top);
            total *= f;
            acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
            M = top;
        }
    }
    // nothing seen, or a mark, adds nothing; a NaN sum goes on
    __device__ __forceinline__ void add(float m, float l, const float4& o) {
        if (l <= 0.f) return;
        const float f = ex2(m - M);
        total = fmaf(l, f, total);
        acc.x = fmaf(o.x, f, acc.x);
        acc.y = fmaf(o.y, f, acc.y);
        acc.z = fmaf(o.z, f, acc.z);
        acc.w = fmaf(o.w, f, acc.w);
    }
};

template <int HD, int SHARE>
__global__ void __launch_bounds__(kMergeThreads) k_line_merge(const LineParams p, int tr, int grid) {
    constexpr int kPerRow = HD / 4, kTeam = kPerRow * SHARE, kBlockRows = kMergeThreads / kTeam, kWarps = kMergeThreads / 32;
    __shared__ float4 s_acc[SHARE > 1 ? kMergeThreads : 1];
    __shared__ float3 s_sum[SHARE > 1 ? kMergeThreads : 1];
    __shared__ int4 s_run[kMergeThreads];
    __shared__ int s_c[kMergeThreads], s_count[kWarps];
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // the table's entries are on their way before it is known how many count
    const int4 plan = p.cut[grid], near = p.cut[min(tid, grid)];
    const int after = p.cut[min(tid + kMergeThreads, grid)].z;
    const int per = plan.x, shares = plan.y;
    const int G = p.nq / p.nkv, blocks = (p.K * G + kBlockRows - 1) / kBlockRows;   // blocks of rows of a run
    int item = blockIdx.x, late = (tid < shares && near.z < 0) || (tid + kMergeThreads < shares && after < 0);
    for (int c = tid + 2 * kMergeThreads; c < shares; c += kMergeThreads) late |= p.cut[c].z < 0;
    if (__syncthreads_or(late)) {   // a CTA gave up waiting: no result of the call is kept
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            const Req q = request_of<1, 0>(p, b);
            if (q.rows > 0 && tid == 0) p.status[b] = PE_REQ_TIMEOUT;
            for (int j = warp; j < q.rows; j += kWarps) {
                uint4* o = reinterpret_cast<uint4*>(p.out + (static_cast<long long>(b) * p.K + j) * p.ld_out);
                for (int x = lane; x < p.nq * HD / 8; x += 32) o[x] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        return;
    }
    for (int c0 = 0; c0 < shares; c0 += kMergeThreads) {
        // the runs whose first cut is one of these
        const int c = c0 + tid;
        const int4 cut = c >= shares ? make_int4(0, 0, 0, 0) : c0 == 0 ? near : p.cut[c];
        const bool here = cut.z > 0 && cut.z <= per;
        const unsigned vote = __ballot_sync(0xffffffffu, here);
        __syncthreads();   // the last round's runs have been read
        if (lane == 0) s_count[warp] = __popc(vote);
        __syncthreads();
        int rank = __popc(vote & ((1u << lane) - 1u)), runs = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) rank += s_count[i];
            runs += s_count[i];
        }
        if (here) {
            s_run[rank] = cut;
            s_c[rank] = c;
        }
        __syncthreads();
        for (; item < runs * blocks; item += gridDim.x) {
            const int x0 = item / blocks, block = item - x0 * blocks;
            const int4 of = s_run[x0];
            const int b = of.x, head = of.y, first = s_c[x0] - 1;
            const int last = (s_c[x0] * per - of.z + of.w - 1) / per;   // the run's first and last share
            const int rows = p.rows != nullptr ? p.rows[b] : p.K;
            const int r = block * kBlockRows + tid / kTeam;
            const int piece = tid % kTeam / kPerRow, d = (tid % kPerRow) * 4;
            const bool mine = r < rows * G;
            Joined j;
            if (mine) {
                const int each = (last - first + SHARE) / SHARE;
                const int from = first + piece * each, to = min(last, from + each - 1);
                for (int q = from; q <= to; q += kMergeBatch) {
                    float mv[kMergeBatch], lv[kMergeBatch];
                    float4 ov[kMergeBatch];
#pragma unroll
                    for (int x = 0; x < kMergeBatch; ++x) {
                        mv[x] = lv[x] = 0.f;
                        if (q + x <= to) {
                            const int part = 2 * (q + x) + (q + x == first ? 1 : 0);
                            const float* src = p.part + static_cast<size_t>(part) * part_floats(tr, HD);
                            mv[x] = src[tr * HD + r];
                            lv[x] = src[tr * HD + tr + r];
                            ov[x] = *reinterpret_cast<const float4*>(src + r * HD + d);
                        }
                    }
                    float top = j.M;
#pragma unroll
                    for (int x = 0; x < kMergeBatch; ++x) {
                        if (lv[x] < 0.f) j.bad = fminf(j.bad, lv[x]);
                        else if (lv[x] != 0.f) top = fmaxf(top, mv[x]);
                    }
                    j.raise(top);
#pragma unroll
                    for (int x = 0; x < kMergeBatch; ++x)
                        if (q + x <= to) j.add(mv[x], lv[x], ov[x]);
                }
            }
            if constexpr (SHARE > 1) {
                s_acc[tid] = j.acc;
                s_sum[tid] = make_float3(j.M, j.total, j.bad);
                __syncthreads();
                if (piece == 0)
                    for (int x = 1; x < SHARE; ++x) {
                        const float3 o = s_sum[tid + x * kPerRow];
                        j.bad = fminf(j.bad, o.z);
                        j.raise(o.y != 0.f ? fmaxf(j.M, o.x) : j.M);
                        j.add(o.x, o.y, s_acc[tid + x * kPerRow]);
                    }
                __syncthreads();
            }
            if (!mine || piece != 0) continue;
            if (head == 0 && r == 0 && d == 0) p.status[b] = status_of(j.bad);
            const float inv = j.total == 0.f || j.bad < 0.f ? 0.f : 1.f / j.total;
            if (j.bad < 0.f) j.acc = make_float4(0.f, 0.f, 0.f, 0.f);
            const int row = r / G;
            __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(
                p.out + (static_cast<long long>(b) * p.K + row) * p.ld_out + static_cast<long long>(head * G + r - row * G) * HD + d);
            dst[0] = __floats2bfloat162_rn(j.acc.x * inv, j.acc.y * inv);
            dst[1] = __floats2bfloat162_rn(j.acc.z * inv, j.acc.w * inv);
        }
        item -= runs * blocks;
    }
}

}  // namespace

namespace line {
int check_shape(int B, int K, int nq, int nkv, int hd, int max_pages) {
    if (B < 1 || K < 1 || max_pages < 1) { set_error("B, K and max_pages must be >= 1"); return PE_ERR_ARG; }
    if (nkv < 1 || nq < 1 || nq % nkv != 0) { set_error("n_kv_heads must divide n_q_heads"); return PE_ERR_UNSUPPORTED; }
    if (hd != 64 && hd != 128) { set_error("head_dim must be 64 or 128"); return PE_ERR_UNSUPPORTED; }
    if (static_cast<long long>(K) * (nq / nkv) > 128) {
        set_error("K * (n_q_heads / n_kv_heads) must be <= 128");
        return PE_ERR_UNSUPPORTED;
    }
    if (max_pages > 0x7FFFFFFF / kPage - 2) {
        set_error("max_pages * 16 must fit a signed 32-bit entry index");
        return PE_ERR_ARG;
    }
    if (static_cast<long long>(B) * K > 0x7FFFFFFFll || static_cast<long long>(B) * nq > 0x7FFFFFFFll) {
        set_error("batch too large");
        return PE_ERR_ARG;
    }
    return PE_OK;
}

int plan_line(int B, int nkv, int hd, int max_pages, int unit, int pad, int least, int tr, Plan* out) {
    int dev = 0, sms = 0;
    const int rc = current_device(&dev, &sms);
    if (rc != PE_OK) return rc;
    Plan a{};
    a.dev = dev;
    a.tr = tr;
    a.sms = sms;
    const long long most = a.most = static_cast<long long>(B) * nkv * ((max_pages + unit - 1) / unit + pad);
    if (most > 0x3FFFFFFFll) {
        set_error("attention: batch * heads * pages is too large for one call");
        return PE_ERR_UNSUPPORTED;
    }
    const long long want = (most + least - 1) / least;
    a.grid = static_cast<int>(want < sms ? want : sms);
    a.cut_floats = (static_cast<size_t>(a.grid) + 2) / 2 * 8;
    a.ws_floats = a.cut_floats + 4 + 2 * static_cast<size_t>(a.grid) * part_floats(a.tr, hd);
    *out = a;
    return PE_OK;
}

int launch_merge(const LineParams& p, const Plan& a, int hd, cudaStream_t s) {
    const int rows = p.K * (p.nq / p.nkv);
    // four teams (a warp, of 64-wide heads half of one) to a row where rows are
    // few (B=1 K=1, 131072 entries: 36.6 us, one team 40.9; B=128 K=11: 195 us,
    // one team 177)
    const bool share = static_cast<long long>(p.B) * p.nkv * rows <= 1024;
    const int block_rows = std::max(1, kMergeThreads / (hd / 4) / (share ? 4 : 1));
    const long long runs = std::min<long long>(a.grid - 1, static_cast<long long>(p.B) * p.nkv);   // cut ones at most
    const long long blocks = runs * ((rows + block_rows - 1) / block_rows);
    const dim3 grid(static_cast<unsigned>(std::max(1ll, std::min<long long>(blocks, a.sms * kMergeBlocks))));
    auto kern = hd == 128 ? (share ? k_line_merge<128, 4> : k_line_merge<128, 1>) : (share ? k_line_merge<64, 4> : k_line_merge<64, 1>);
    PE_CUDA_TRY(launch_ex(kern, grid, dim3(kMergeThreads), 0, s, true, p, a.tr, a.grid));
    return PE_OK;
}
}  // namespace line
}  // namespace pe
