// Paged GQA attention over the 8-bit KV cache (pe_attention_kv8): E4M3 codes
// with one fp32 scale for each (page, kv head), bf16 queries and output.
//
//   o_r = sum_e w_re v_e / sum_e w_re,  w_re = exp(scale * q_r . k_e),
//   k_e = ks[page(e)] * kcode_e,  v_e = vs[page(e)] * vcode_e
//
// over the entries e <= S_b + j that row r (draft row j of request b) sees, in
// one pass with a running maximum (base 2). The page scales never touch the
// codes: ks multiplies the page's scores, vs its weights, both in fp32.
//
// Work. A unit is one page of one (kv head, tile of 16 query rows): 16 entries
// of K and of V. All units of the batch stand in one line (request, kv head,
// row tile, page) and every CTA takes the same number of them, so ragged
// lengths, many requests and a single long one are split alike; the lengths
// stay on the device. A CTA writes the heads that it covers whole; a head that
// several CTAs share leaves partial sums in scratch, at places that follow
// from the unit numbers, and k_kv8_merge joins them in order.
//
// A warp takes every eighth unit of its CTA through a ring of its own: lane 0
// fetches the page's K and V by TMA (swizzled, so that both read patterns
// below are free of bank conflicts) kStages units ahead. The codes are widened
// to fp16, which holds every E4M3 value, in registers, in the layout of
// mma.m16n8k16: the dimension order of a K word is permuted, and Q's with it,
// so a lane reads whole 16-byte chunks; pairs of V rows are interleaved by
// byte permutes. Queries enter as fp16 after an exact shift by a power of two
// per row, scores and sums are fp32, weights go to fp16 (2^-11) relative to
// the row's running maximum and the largest V scale seen.
#include <algorithm>

#include "attn_kv8.cuh"

namespace pe {
namespace {

using namespace kv8;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 4;         // units in flight per warp
constexpr int kTileRows = 16;      // query rows of a unit (the MMA's M)
constexpr int kMaxUnits = 1024;    // units of one CTA
constexpr int kMinUnits = kWarps;  // a CTA's share is at least one unit per warp
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ uint2 lds64(const uint8_t* p) { return *reinterpret_cast<const uint2*>(p); }
template <int HD>
struct Smem {
    static constexpr int kTile = kPage * HD;                 // a page's K or V of one head
    static constexpr int kRing = kWarps * kStages * 2 * kTile;
    static constexpr int kO = kRing;                         // [kWarps][16][HD] fp32
    static constexpr int kMl = kO + kWarps * kTileRows * HD * 4;
    static constexpr int kBar = kMl + kWarps * kTileRows * 8;
    static constexpr int kInfo = kBar + kWarps * kStages * 8;
    static constexpr int kUnit = kInfo + kMaxUnits * 16;     // tile, ks, vs
    static constexpr int kBytes = kUnit + kMaxUnits * 12 + 1024;
};

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_kv8(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Kv8Params p) {
    using L = Smem<HD>;
    constexpr int kSteps = HD / 16;       // MMA steps over the head dimension
    constexpr int kWords = HD / 16;       // 32-bit words of a lane's quarter of a K row
    constexpr int kCols = HD / 8;         // output column tiles = bytes of a lane's part of a V row
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    uint8_t* ring = sm + warp * kStages * 2 * L::kTile;
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBar) + warp * kStages;
    float* s_o = reinterpret_cast<float*>(sm + L::kO);
    float2* s_ml = reinterpret_cast<float2*>(sm + L::kMl);
    int4* s_info = reinterpret_cast<int4*>(sm + L::kInfo);
    int* s_tile = reinterpret_cast<int*>(sm + L::kUnit);
    float* s_ks = reinterpret_cast<float*>(s_tile + kMaxUnits);
    float* s_vs = s_ks + kMaxUnits;

    pdl_launch_dependents();
    if (lane == 0)
        for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
    int lo;
    const int n = gather_units<kThreads, 1, kTileRows>(p, kMinUnits, s_info, s_tile, s_ks, s_vs, lo);
    zero_idle_rows_by<1, kTileRows>(p, HD, warp, kWarps);

    const uint64_t policy = l2_policy_evict_first();
    auto fetch = [&](int i) {   // lane 0: unit i into its stage
        const int tile = i < n ? s_tile[i] : -1;
        if (tile < 0) return;
        const int st = (i / kWarps) % kStages;
        uint8_t* at = ring + st * 2 * L::kTile;
        mbar_arrive_expect_tx(&full[st], 2 * L::kTile);
        tma_load_2d(at, &tmK, &full[st], 0, tile * kPage, policy);
        tma_load_2d(at + L::kTile, &tmV, &full[st], 0, tile * kPage, policy);
    };
    if (lane == 0)
        for (int s = 0; s < kStages; ++s) fetch(warp + s * kWarps);
    uint32_t parity = 0;   // bit s: the phase that stage s completes next

    const int G = p.nq / p.nkv;
    int i = warp;          // this warp's next unit
    bool dead = false;
    for (int seg = 0; seg < n;) {
        const int4 info = s_info[seg];
        const int b = info.x, page0 = info.z;
        const int len = min(info.w - page0, n - seg);
        const int S = p.seq_lens[b];
        const int rows = p.rows != nullptr ? p.rows[b] : p.K;
        const int tiles = (rows * G + kTileRows - 1) / kTileRows;
        const int head = info.y / tiles, r0 = (info.y - head * tiles) * kTileRows;
        const int live = min(kTileRows, rows * G - r0);   // rows of this tile
        const int last = S + rows - 1;                    // last entry that any row sees
        float mark = 0.f;
        float o[kCols][4];
#pragma unroll
        for (int c = 0; c < kCols; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, vref = 0.f;

        if (i < seg + len && !dead) {
            // queries: rows g and g + 8, this lane's quarter of the dimensions
            uint32_t qa[kSteps][4];
            float cs[2];
            int lim[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = g + 8 * h;
                const int j = (r0 + r) / G;
                const __nv_bfloat16* src =
                    p.q + (static_cast<long long>(b) * p.K + j) * p.ld_q +
                    static_cast<long long>(head * G + (r0 + r) - j * G) * HD + t * (HD / 4);
                uint4 raw[HD / 32];
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    raw[c] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < live) raw[c] = *reinterpret_cast<const uint4*>(src + c * 8);
                }
                uint32_t top = 0;
                const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) top = max(top, max((w[c] << 16) & 0x7FFF0000u, w[c] & 0x7FFF0000u));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // the row times 2^(127 - E): its largest value lies in [1, 2)
                const int E = min(max(static_cast<int>(top >> 23), 1), 253);
                const float down = __uint_as_float(static_cast<uint32_t>(254 - E) << 23);
                cs[h] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(E) << 23);
                lim[h] = r < live ? S + j : -1;
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) {
                    const float x0 = __uint_as_float(w[c] << 16) * down, x1 = __uint_as_float(w[c] & 0xFFFF0000u) * down;
                    qa[c >> 1][(c & 1) * 2 + h] = pack_f16(x0, x1);
                }
            }
            for (; i < seg + len; i += kWarps) {
                const int st = (i / kWarps) % kStages;
                if (s_tile[i] < 0) {
                    mark = kMarkBadPage;
                    if (lane == 0) fetch(i + kStages * kWarps);
                    continue;
                }
                const bool ok = mbar_wait(&full[st], (parity >> st) & 1u, nullptr, 0u);
                if (!__all_sync(0xffffffffu, ok)) {
                    dead = true;
                    break;
                }
                parity ^= 1u << st;
                const uint8_t* kt = ring + st * 2 * L::kTile;
                const uint8_t* vt = kt + L::kTile;
                const float ks = s_ks[i], vs = s_vs[i];
                const int e0 = (page0 + i - seg) * kPage;   // the page's first entry
                const bool inner = e0 + kPage - 1 <= S;     // every row sees all of it

                // scores of entries g (columns 0-7) and g + 8 (columns 8-15)
                float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = g + 8 * h;
                    uint32_t w[kWords];
                    if constexpr (HD == 128) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint4 x = lds128(kt + r * 128 + (((2 * t + c) ^ (r & 7)) << 4));
                            w[4 * c] = x.x; w[4 * c + 1] = x.y; w[4 * c + 2] = x.z; w[4 * c + 3] = x.w;
                        }
                    } else {
                        const uint4 x = lds128(kt + r * 64 + ((t ^ ((r >> 1) & 3)) << 4));
                        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
                    }
#pragma unroll
                    for (int c = 0; c < kSteps; ++c) mma_f16(s[h], qa[c], widen_lo(w[c]), widen_hi(w[c]));
                }
                // V rows 2t, 2t+1, 2t+8, 2t+9: this lane's HD/8 columns
                uint32_t vw[4][kCols / 4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int r = 2 * t + (x & 1) + 8 * (x >> 1);
                    if constexpr (HD == 128) {
                        const uint4 y = lds128(vt + r * 128 + ((g ^ (r & 7)) << 4));
                        vw[x][0] = y.x; vw[x][1] = y.y; vw[x][2] = y.z; vw[x][3] = y.w;
                    } else {
                        const uint2 y = lds64(vt + r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
                        vw[x][0] = y.x; vw[x][1] = y.y;
                    }
                }
                __syncwarp();
                if (lane == 0) fetch(i + kStages * kWarps);

                const float f0 = cs[0] * ks, f1 = cs[1] * ks;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s[h][0] *= f0; s[h][1] *= f0; s[h][2] *= f1; s[h][3] *= f1;
                }
                if (!inner) {
                    // Entries that some row does not see. What stands behind
                    // the last one is no one's: its V is dropped. A NaN in a
                    // V that only some rows see would reach the others as
                    // 0 * NaN, so it enters through the score instead: the
                    // rows that see the entry are NaN as a whole.
                    int nan = 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int e = e0 + 2 * t + (x & 1) + 8 * (x >> 1);
                        int any = 0;
#pragma unroll
                        for (int c = 0; c < kCols / 4; ++c)
                            vw[x][c] = e > last ? 0u : without_nan(vw[x][c], any);
                        nan |= any << x;
                    }
                    nan |= __shfl_xor_sync(0xffffffffu, nan, 4);
                    nan |= __shfl_xor_sync(0xffffffffu, nan, 8);
                    nan |= __shfl_xor_sync(0xffffffffu, nan, 16);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int e = e0 + 2 * t + (x & 1) + 8 * (x >> 1);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float& v = s[x >> 1][2 * h + (x & 1)];
                            if ((nan >> x) & 1) v = NAN;
                            if (e > lim[h]) v = -INFINITY;
                        }
                    }
                }
                float top[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    top[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
                    top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
                    top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
                }
                const bool up = top[0] > m[0] + kRescale || top[1] > m[1] + kRescale;
                const float av = fabsf(vs);
                const bool grow = av > 16.f * vref;
                if (__any_sync(0xffffffffu, up) || grow) {
                    float f[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f[h] = 1.f;
                        if (top[h] > m[h] + kRescale) {
                            f[h] = m[h] == -INFINITY ? 0.f : ex2(m[h] - top[h]);
                            m[h] = top[h];
                        }
                        l[h] *= f[h];
                    }
                    if (grow) {
                        const float fv = vref / av;
                        vref = av;
                        f[0] *= fv;
                        f[1] *= fv;
                    }
#pragma unroll
                    for (int c = 0; c < kCols; ++c) {
                        o[c][0] *= f[0]; o[c][1] *= f[0]; o[c][2] *= f[1]; o[c][3] *= f[1];
                    }
                }
                const float vr = vref > 0.f ? vs / vref : 0.f;
                uint32_t pa[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float mm = m[h] == -INFINITY ? 0.f : m[h];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float w0 = ex2(s[x][2 * h] - mm), w1 = ex2(s[x][2 * h + 1] - mm);
                        l[h] += w0 + w1;
                        pa[2 * x + h] = pack_f16(w0 * vr, w1 * vr);
                    }
                }
#pragma unroll
                for (int c = 0; c < kCols / 4; ++c) {
                    const uint32_t a0 = __byte_perm(vw[0][c], vw[1][c], 0x5140), a1 = __byte_perm(vw[0][c], vw[1][c], 0x7362);
                    const uint32_t b0 = __byte_perm(vw[2][c], vw[3][c], 0x5140), b1 = __byte_perm(vw[2][c], vw[3][c], 0x7362);
                    mma_f16(o[4 * c], pa, widen_lo(a0), widen_lo(b0));
                    mma_f16(o[4 * c + 1], pa, widen_hi(a0), widen_hi(b0));
                    mma_f16(o[4 * c + 2], pa, widen_lo(a1), widen_lo(b1));
                    mma_f16(o[4 * c + 3], pa, widen_hi(a1), widen_hi(b1));
                }
            }
        }
        if (dead) mark = kMarkTimeout;

        // Join the warps. A lane holds, of rows g and g + 8, the 2 * kCols
        // columns from t * 2 * kCols on; row r's 16-byte chunk c of that
        // quarter goes to chunk c ^ (2t + (r & 1)) of it (banks).
        __syncthreads();   // the last segment's sums have been read
        constexpr int kChunks = kCols / 2;   // 16-byte chunks of a quarter row
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = g + 8 * h;
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (t == 0) s_ml[warp * kTileRows + r] = make_float2(m[h], mark != 0.f ? mark : l[h]);
            float* dst = s_o + (warp * kTileRows + r) * HD + t * (HD / 4);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                // column 2t of the tile stands for dimensions 2t * kCols + tile, column 2t + 1 for the next kCols
                const int x = c * 4 / kCols, y = c * 4 - x * kCols;
                const float4 v = make_float4(o[y][2 * h + x] * vref, o[y + 1][2 * h + x] * vref,
                                             o[y + 2][2 * h + x] * vref, o[y + 3][2 * h + x] * vref);
                *reinterpret_cast<float4*>(dst + ((c ^ ((2 * t + (r & 1)) & (kChunks - 1))) << 2)) = v;
            }
        }
        __syncthreads();
        {
            constexpr int kOut = HD / 16;    // columns of a thread
            const int r = tid >> 4, d0 = (tid & 15) * kOut;
            float M = -INFINITY, bad = 0.f;
            float2 ml[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                ml[w] = s_ml[w * kTileRows + r];
                if (ml[w].y < 0.f) bad = fminf(bad, ml[w].y);
                else M = fmaxf(M, ml[w].x);
            }
            float acc[kOut], sum = 0.f;
#pragma unroll
            for (int d = 0; d < kOut; ++d) acc[d] = 0.f;
            const int quarter = d0 / (HD / 4), c0 = (d0 - quarter * (HD / 4)) / 4;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (ml[w].y <= 0.f) continue;   // saw nothing (a NaN sum goes on)
                const float f = ex2(ml[w].x - M);
                sum += ml[w].y * f;
                const float* src = s_o + (w * kTileRows + r) * HD + quarter * (HD / 4);
#pragma unroll
                for (int c = 0; c < kOut / 4; ++c) {
                    const float4 v = *reinterpret_cast<const float4*>(
                        src + (((c0 + c) ^ ((2 * quarter + (r & 1)) & (kChunks - 1))) << 2));
                    acc[4 * c] += v.x * f;
                    acc[4 * c + 1] += v.y * f;
                    acc[4 * c + 2] += v.z * f;
                    acc[4 * c + 3] += v.w * f;
                }
            }
            if (len == info.w) {   // the whole head: write the output
                const float inv = bad < 0.f || sum == 0.f ? 0.f : 1.f / sum;
                if (r < live) {
                    const int j = (r0 + r) / G;
                    __nv_bfloat16* dst = p.out + (static_cast<long long>(b) * p.K + j) * p.ld_out +
                                         static_cast<long long>(head * G + (r0 + r) - j * G) * HD + d0;
#pragma unroll
                    for (int d = 0; d < kOut; d += 2)
                        *reinterpret_cast<__nv_bfloat162*>(dst + d) =
                            bad < 0.f ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(acc[d] * inv, acc[d + 1] * inv);
                }
                if (info.y == 0 && tid == 0)
                    p.status[b] = status_of(bad);
            } else {
                float* dst = p.part + static_cast<size_t>(2 * blockIdx.x + (seg == 0 ? 0 : 1)) * part_floats(kTileRows, HD);
#pragma unroll
                for (int d = 0; d < kOut; ++d) dst[r * HD + d0 + d] = acc[d];
                if ((tid & 15) == 0) {
                    dst[kTileRows * HD + r] = M;
                    dst[kTileRows * HD + kTileRows + r] = bad < 0.f ? bad : sum;
                }
            }
        }
        seg += len;
    }
    if (dead) __nanosleep(100000);   // a wait gave up: let copies still in flight land
}

// Joins the parts of every (head, row tile) that several CTAs share, in unit
// order. The part that CTA c left of a run of units [u0, u1) is its first one
// where the run begins at or before c's share, its second one otherwise. A
// thread per row and four dimensions; the parts are read eight at a time, all
// loads of a batch in flight, and folded with a running maximum: with one part
// at a time the loads' latency alone was 0.7 us a part.
constexpr int kMergeThreads = 128;
constexpr int kMergeBatch = 8;

template <int HD>
__global__ void __launch_bounds__(kMergeThreads) k_kv8_merge(const Kv8Params p, int tr, int ppu) {
    constexpr int kPerRow = HD / 4, kBlockRows = kMergeThreads / kPerRow;
    pdl_wait();
    const int b = blockIdx.z, head = blockIdx.y;
    const int u_b = p.first[b], units = p.first[b + 1] - u_b, per = p.first[p.B + 1];
    const int G = p.nq / p.nkv;
    const int S = p.seq_lens[b], rows = p.rows != nullptr ? p.rows[b] : p.K;
    if (units == 0) return;
    const int tiles = (rows * G + tr - 1) / tr;
    const int run = ((S + rows + kPage - 1) / kPage + ppu - 1) / ppu;
    const int d = (threadIdx.x % kPerRow) * 4;
    for (int rr = blockIdx.x * kBlockRows + threadIdx.x / kPerRow; rr < rows * G; rr += gridDim.x * kBlockRows) {
        const int tile = rr / tr, r = rr - tile * tr;
        const int u0 = u_b + (head * tiles + tile) * run, u1 = u0 + run;
        const int c0 = u0 / per, c1 = (u1 - 1) / per;
        if (c0 == c1) continue;   // written by its CTA
        float M = -INFINITY, bad = 0.f, total = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = c0; c <= c1; c += kMergeBatch) {
            float mv[kMergeBatch], lv[kMergeBatch];
            float4 ov[kMergeBatch];
#pragma unroll
            for (int x = 0; x < kMergeBatch; ++x) {
                lv[x] = 0.f;
                if (c + x <= c1) {
                    const int part = 2 * (c + x) + (u0 <= (c + x) * per ? 0 : 1);
                    const float* src = p.part + static_cast<size_t>(part) * part_floats(tr, HD);
                    mv[x] = src[tr * HD + r];
                    lv[x] = src[tr * HD + tr + r];
                    ov[x] = *reinterpret_cast<const float4*>(src + r * HD + d);
                }
            }
            float top = M;
#pragma unroll
            for (int x = 0; x < kMergeBatch; ++x) {
                if (lv[x] < 0.f) bad = fminf(bad, lv[x]);
                else if (lv[x] != 0.f) top = fmaxf(top, mv[x]);
            }
            if (top > M) {
                const float f = M == -INFINITY ? 0.f : ex2(M - top);
                total *= f;
                acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
                M = top;
            }
#pragma unroll
            for (int x = 0; x < kMergeBatch; ++x) {
                if (lv[x] <= 0.f) continue;   // nothing seen, or a mark; a NaN sum goes on
                if (c + x > c1) continue;
                const float f = ex2(mv[x] - M);
                total = fmaf(lv[x], f, total);
                acc.x = fmaf(ov[x].x, f, acc.x);
                acc.y = fmaf(ov[x].y, f, acc.y);
                acc.z = fmaf(ov[x].z, f, acc.z);
                acc.w = fmaf(ov[x].w, f, acc.w);
            }
        }
        if (head == 0 && rr == 0 && d == 0) p.status[b] = status_of(bad);
        const float inv = total == 0.f || bad < 0.f ? 0.f : 1.f / total;
        const int j = rr / G;
        __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(
            p.out + (static_cast<long long>(b) * p.K + j) * p.ld_out + static_cast<long long>(head * G + rr - j * G) * HD + d);
        if (bad < 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f);
        dst[0] = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        dst[1] = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    }
}

// Query rows of a head from which the tensor-memory kernel is taken: up to 16
// rows one tile of the register kernel covers them; above, it would read the
// cache once per 16 rows.
constexpr int kUmmaFrom = 17;

int plan_kv8(int B, int K, int nq, int nkv, int hd, int max_pages, Plan* out) {
    int dev = 0, sms = 0;
    PE_CUDA_TRY(cudaGetDevice(&dev));
    PE_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    Plan a{};
    const int rows = K * (nq / nkv);
    const bool umma = rows >= kUmmaFrom;
    a.ppu = umma ? kUmmaPages : 1;
    a.tr = umma ? kUmmaRows : kTileRows;
    const int max_units = umma ? kUmmaUnits : kMaxUnits, least = umma ? 1 : kMinUnits;
    a.tiles_max = (rows + a.tr - 1) / a.tr;
    const long long most = static_cast<long long>(B) * nkv * a.tiles_max * ((max_pages + a.ppu - 1) / a.ppu);
    if (most > 0x3FFFFFFFll || B > 65535 || nkv > 65535) {
        set_error("attention: batch * heads * pages is too large for one call");
        return PE_ERR_UNSUPPORTED;
    }
    // one CTA per SM, and as many rounds as keep a CTA's share in its tables
    const long long round = static_cast<long long>(sms) * max_units;
    const long long slots = static_cast<long long>(sms) * ((most + round - 1) / round);
    const long long want = (most + least - 1) / least;
    a.grid = static_cast<int>(want < slots ? want : slots);
    a.first_floats = (static_cast<size_t>(B) + 2 + 3) / 4 * 4;
    a.ws_floats = a.first_floats + 2 * static_cast<size_t>(a.grid) * part_floats(a.tr, hd);
    *out = a;
    return PE_OK;
}

template <int HD>
int launch_hd(const CUtensorMap& tk, const CUtensorMap& tv, const Kv8Params& p, const Plan& a, cudaStream_t s) {
    auto kern = k_attn_kv8<HD>;
    PE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<HD>::kBytes));
    PE_CUDA_TRY(launch_ex(kern, dim3(a.grid), dim3(kThreads), Smem<HD>::kBytes, s, false, tk, tv, p));
    return PE_OK;
}

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

}  // namespace

namespace kv8 {
int launch_merge(const Kv8Params& p, const Plan& a, int hd, cudaStream_t s) {
    // blocks for every row while the heads are few, a block for several rows
    // where there are enough of them
    const int block_rows = kMergeThreads / (hd / 4);
    const int all = (p.K * (p.nq / p.nkv) + block_rows - 1) / block_rows;
    const int some = std::max(1, 2048 / (p.B * p.nkv));
    const dim3 grid(all < some ? all : some, p.nkv, p.B);
    auto kern = hd == 128 ? k_kv8_merge<128> : k_kv8_merge<64>;
    PE_CUDA_TRY(launch_ex(kern, grid, dim3(kMergeThreads), 0, s, true, p, a.tr, a.ppu));
    return PE_OK;
}
}  // namespace kv8
}  // namespace pe

using namespace pe;

extern "C" int pe_attention_kv8_scratch(int32_t B, int32_t K, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                        int32_t max_pages, int64_t* ws_floats) {
    if (ws_floats == nullptr) { set_error("null argument"); return PE_ERR_ARG; }
    int rc = check_shape(B, K, n_q_heads, n_kv_heads, head_dim, max_pages);
    if (rc != PE_OK) return rc;
    Plan a;
    if ((rc = plan_kv8(B, K, n_q_heads, n_kv_heads, head_dim, max_pages, &a)) != PE_OK) return rc;
    *ws_floats = static_cast<int64_t>(a.ws_floats);
    return PE_OK;
}

extern "C" int pe_attention_kv8(int32_t B, int32_t K, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                const void* q, int64_t ld_q, const int32_t* seq_lens, const int32_t* rows,
                                const int32_t* page_table, int32_t max_pages, int32_t num_pages,
                                const uint8_t* k_codes, const uint8_t* v_codes, const float* k_scale,
                                const float* v_scale, float scale, void* out, int64_t ld_out, float* ws,
                                int64_t ws_floats, int32_t* status, void* stream) {
    int rc = check_shape(B, K, n_q_heads, n_kv_heads, head_dim, max_pages);
    if (rc != PE_OK) return rc;
    if (num_pages < 1 || static_cast<long long>(num_pages) * n_kv_heads * kPage > 0x7FFFFFFFll) {
        set_error("num_pages must be >= 1 and num_pages * n_kv_heads * 16 fit a signed 32-bit row index");
        return PE_ERR_ARG;
    }
    if (!q || !seq_lens || !page_table || !k_codes || !v_codes || !k_scale || !v_scale || !out || !ws || !status) {
        set_error("null tensor argument");
        return PE_ERR_ARG;
    }
    const int64_t width = static_cast<int64_t>(n_q_heads) * head_dim;
    if (ld_q < width || ld_out < width || ld_q % 8 != 0 || ld_out % 8 != 0) {
        set_error("row strides must be multiples of 8 and at least n_q_heads * head_dim");
        return PE_ERR_ARG;
    }
    const uintptr_t bits = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) |
                           reinterpret_cast<uintptr_t>(k_codes) | reinterpret_cast<uintptr_t>(v_codes) |
                           reinterpret_cast<uintptr_t>(ws);
    if ((bits & 15u) != 0) { set_error("q, out, ws and the code arrays must be 16-byte aligned"); return PE_ERR_ARG; }
    Plan a;
    if ((rc = plan_kv8(B, K, n_q_heads, n_kv_heads, head_dim, max_pages, &a)) != PE_OK) return rc;
    if (ws_floats < static_cast<int64_t>(a.ws_floats)) {
        set_error("attention scratch too small: " + std::to_string(a.ws_floats) + " floats needed");
        return PE_ERR_ARG;
    }
    CUtensorMap tk, tv;
    const uint64_t lines = static_cast<uint64_t>(num_pages) * n_kv_heads * kPage;
    if ((rc = encode_tmap_codes(&tk, k_codes, head_dim, lines)) != PE_OK) return rc;
    if ((rc = encode_tmap_codes(&tv, v_codes, head_dim, lines)) != PE_OK) return rc;
    Kv8Params p{};
    p.B = B;
    p.K = K;
    p.nq = n_q_heads;
    p.nkv = n_kv_heads;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.ld_q = ld_q;
    p.seq_lens = seq_lens;
    p.rows = rows;
    p.page_table = page_table;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.scale_log2 = scale * kLog2e;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.ld_out = ld_out;
    p.status = status;
    p.first = reinterpret_cast<int32_t*>(ws);
    p.part = ws + a.first_floats;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.tr == kUmmaRows) rc = launch_umma(tk, tv, p, a, head_dim, s);
    else rc = head_dim == 128 ? launch_hd<128>(tk, tv, p, a, s) : launch_hd<64>(tk, tv, p, a, s);
    // a grid of one covers every head whole
    return rc != PE_OK || a.grid == 1 ? rc : launch_merge(p, a, head_dim, s);
}
