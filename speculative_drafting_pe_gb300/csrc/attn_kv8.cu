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
// This file: the kernel for few query rows of a head (single tokens),
// whose unit is one page, the merge and the entry point; the line of units
// that both kernels divide is described in attn_kv8.cuh.
//
// A warp takes every twelfth unit of its CTA, kStages units ahead, through
// asynchronous copies of its own lanes: each lane fetches the very chunks that
// it will read, to a place of its own, so there is no barrier to wait at and
// no bank conflict. (TMA boxes of one page, 16 rows, took about 150 cycles
// each and held the kernel at 28 bytes/ns per SM.) Both products are
// transposed, S^T = K Q^T and O^T = V^T P^T, so that the entries and the
// dimensions fill the 16 rows of mma.m16n8k16 and 8 query rows its columns: a
// head with few rows leaves no part of the MMA idle. The codes are widened to
// fp16, which holds every E4M3 value, in registers and where they land: the
// dimension order of a K word is permuted, and Q's with it, so a lane takes
// whole 16-byte chunks; pairs of V rows are interleaved by byte permutes; P^T
// comes out of S^T's layout by two 8x8 transposes. Queries enter as fp16 after
// an exact shift by a power of two per row, scores and sums are fp32, weights
// times V's scale go to fp16 (2^-11) relative to the row's largest such product
// so far (kLift).
//
// Bound by the cache's bytes while it streams (a CTA's twelve warps take 1900
// cycles for twelve pages of K and V, 48 KB, the rate of the measured copy);
// around that stand the launch and the look-up of the share (about 4 us), a
// join of the warps per segment (1.7 us) and the merge. 64 requests of 512 to
// 8192 entries, one row of 8 heads to each of 4 of 128: 65 us, 4.4 TB/s, 66%
// of the measured copy; one of 131072 entries 36.7 us, 55%.
#include <algorithm>

#include "attn_kv8.cuh"

namespace pe {
namespace {

using namespace kv8;

constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;         // units in flight per warp: 96 KB per SM. More only lengthens the queue
                                   // in front of every other load
constexpr int kMaxUnits = 1024;    // units of a window
constexpr int kMinUnits = kWarps;  // a CTA's share is at least one unit per warp
constexpr int kPad = 32;           // a segment's end in units (B=64, 512..8192 entries: 66 us, with 0 73)
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// NT: tiles of 8 query rows
template <int HD, int NT>
struct Smem {
    static constexpr int kRows = 8 * NT;
    static constexpr int kTile = kPage * HD;                 // a page's K or V of one head
    // a stage of a warp: K chunks [HD / 32][lane] of 16 bytes, V chunks [4][lane] of HD / 8
    static constexpr int kRounds = NT;                       // warps that share a slot of sums
    static constexpr int kSlots = kWarps / kRounds;
    static constexpr int kRing = kWarps * kStages * 2 * kTile;
    static constexpr int kO = kRing;                         // [kSlots][kRows][HD] fp32
    static constexpr int kMl = kO + kSlots * kRows * HD * 4; // [2][kWarps][kRows] (max, sum)
    static constexpr int kScale = kMl + 2 * kWarps * kRows * 8;   // [kWarps][kStages] (ks, vs)
    static constexpr int kInfo = (kScale + kWarps * kStages * 8 + 15) / 16 * 16;
    static constexpr int kUnit = kInfo + kMaxUnits * 16;     // tile
    static constexpr int kBytes = kUnit + kMaxUnits * 4 + 1024;
    // 16-byte chunk c of row r of a slot stands at c ^ swizzle(r): the lanes
    // of a quarter warp (four row pairs, two runs of dimensions) meet no bank twice
    __device__ static __forceinline__ int swizzle(int r) {
        const int t = (r >> 1) & 3;
        return HD == 128 ? t : (t & 1) | ((t >> 1) << 2);
    }
};
static_assert(Smem<128, 1>::kBytes <= 232448 - 2048 && Smem<64, 2>::kBytes <= 232448 - 2048, "shared memory of a block");

// The n units of a window; FIRST: of the share's first one.
template <int HD, int NT, bool FIRST>
__device__ __forceinline__ void attend_window(const Kv8Params& p, uint8_t* sm, int n, const Window* win) {
    using L = Smem<HD, NT>;
    constexpr int kRows = L::kRows;
    constexpr int kSteps = HD / 16;       // MMA steps over the head dimension = words of a lane's quarter of a K row
    constexpr int kCols = HD / 8;         // dimensions of a lane's part of a V row
    constexpr int kMt = kCols / 2;        // 16-dimension tiles of the output
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    uint8_t* ring = sm + warp * kStages * 2 * L::kTile;
    float* s_o = reinterpret_cast<float*>(sm + L::kO);
    int4* s_info = reinterpret_cast<int4*>(sm + L::kInfo);
    int* s_tile = reinterpret_cast<int*>(sm + L::kUnit);

    const uint64_t policy = l2_policy_evict_first();
    const uint32_t ring_at = smem_u32(ring) + lane * 16, ring_v = smem_u32(ring) + L::kTile + lane * kCols;
    float2* scales = reinterpret_cast<float2*>(sm + L::kScale) + warp * kStages;
    const uint32_t scales_at = smem_u32(scales) + lane * 4;
    const float* scale_from = lane == 0 ? p.k_scale : p.v_scale;
    auto fetch = [&](int i, int st) {   // unit i into stage st; a group even where there is nothing to copy
        const int tile = i < n ? s_tile[i] : -1;
        if (tile >= 0) {
            if (lane < 2) copy_async<4>(scales_at + st * 8, scale_from + tile, policy);
            // K rows g and g + 8, chunks t and t + 4 (of 64-wide rows: t); V rows 2t, 2t+1, 2t+8, 2t+9, part g
            const uint8_t* k = p.k_codes + static_cast<size_t>(tile) * L::kTile + g * HD + t * 16;
            const uint8_t* v = p.v_codes + static_cast<size_t>(tile) * L::kTile + 2 * t * HD + g * kCols;
            const uint32_t at = ring_at + st * 2 * L::kTile, at_v = ring_v + st * 2 * L::kTile;
#pragma unroll
            for (int c = 0; c < HD / 32; ++c)
                copy_async<16>(at + c * 512, k + (HD == 128 ? (c >> 1) * 8 * HD + (c & 1) * 64 : c * 8 * HD), policy);
#pragma unroll
            for (int x = 0; x < 4; ++x) copy_async<kCols>(at_v + x * 32 * kCols, v + ((x & 1) + 8 * (x >> 1)) * HD, policy);
        }
        copies_commit();
    };
    for (int s = 0; s < kStages; ++s) fetch(warp + s * kWarps, s);
    int st = 0;            // the stage of this warp's next unit

    const int G = p.nq / p.nkv;
    int i = warp;          // this warp's next unit
    int turn = 0;
    for (int seg = 0; seg < n; turn ^= 1) {
        const int4 info = s_info[seg];
        const int b = info.x, page0 = info.z;
        const int len = min(info.w - page0, n - seg);
        const int S = p.seq_lens[b];
        const int rows = p.rows != nullptr ? p.rows[b] : p.K;
        const int head = info.y, live = rows * G;
        const int last = S + rows - 1;                    // last entry that any row sees
        float mark = 0.f;
        // of rows a * 8 + 2t + x: o[j][a][2y + x] is dimension g * kCols + 2j + y
        float o[kMt][NT][4];
#pragma unroll
        for (int j = 0; j < kMt; ++j)
#pragma unroll
            for (int a = 0; a < NT; ++a) o[j][a][0] = o[j][a][1] = o[j][a][2] = o[j][a][3] = 0.f;
        float m[NT][2], l[NT][2], mo[NT][2];
#pragma unroll
        for (int a = 0; a < NT; ++a) m[a][0] = m[a][1] = mo[a][0] = mo[a][1] = -INFINITY, l[a][0] = l[a][1] = 0.f;

        if (i < seg + len) {
            // queries: row a * 8 + g, this lane's quarter of the dimensions
            uint32_t qb[NT][kSteps][2];
            float cs[NT][2];   // of rows a * 8 + 2t + x
            int lim[NT][2];
#pragma unroll
            for (int a = 0; a < NT; ++a) {
                const int r = a * 8 + g, j = r / G;
                const __nv_bfloat16* src =
                    p.q + (static_cast<long long>(b) * p.K + j) * p.ld_q +
                    static_cast<long long>(head * G + r - j * G) * HD + t * 16;
                uint4 raw[HD / 32];
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    raw[c] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < live) raw[c] = *reinterpret_cast<const uint4*>(src + (c >> 1) * 64 + (c & 1) * 8);
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
                const float up = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(E) << 23);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    cs[a][x] = __shfl_sync(0xffffffffu, up, (2 * t + x) * 4);
                    const int rx = a * 8 + 2 * t + x;
                    lim[a][x] = rx < live ? S + rx / G : -1;
                }
#pragma unroll
                for (int c = 0; c < HD / 8; ++c)
                    qb[a][c >> 1][c & 1] = pack_f16(__uint_as_float(w[c] << 16) * down,
                                                    __uint_as_float(w[c] & 0xFFFF0000u) * down);
            }
            for (; i < seg + len; i += kWarps) {
                copies_wait<kStages - 1>();
                if (s_tile[i] < 0) {
                    mark = kMarkBadPage;
                    fetch(i + kStages * kWarps, st);
                    st = st + 1 == kStages ? 0 : st + 1;
                    continue;
                }
                const uint8_t* kt = ring + st * 2 * L::kTile + lane * 16;
                const uint8_t* vt = ring + st * 2 * L::kTile + L::kTile + lane * kCols;
                __syncwarp();   // the scales come by two lanes
                const float ks = scales[st].x, vs = scales[st].y;
                const int e0 = (page0 + i - seg) * kPage;   // the page's first entry
                const bool inner = e0 + kPage - 1 <= S;     // every row sees all of it

                // S^T: entries g and g + 8 of the page
                uint32_t kw[2][kSteps];
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    const uint4 x = *reinterpret_cast<const uint4*>(kt + c * 512);
                    uint32_t* w = HD == 128 ? &kw[c >> 1][(c & 1) * 4] : &kw[c][0];
                    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
                }
                // V rows 2t, 2t+1, 2t+8, 2t+9: this lane's kCols dimensions
                uint32_t vw[4][kCols / 4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if constexpr (HD == 128) {
                        const uint4 y = *reinterpret_cast<const uint4*>(vt + x * 512);
                        vw[x][0] = y.x; vw[x][1] = y.y; vw[x][2] = y.z; vw[x][3] = y.w;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2*>(vt + x * 256);
                        vw[x][0] = y.x; vw[x][1] = y.y;
                    }
                }
                __syncwarp();
                fetch(i + kStages * kWarps, st);
                st = st + 1 == kStages ? 0 : st + 1;

                float s[NT][4], s2[NT][4];   // two chains of MMAs
#pragma unroll
                for (int a = 0; a < NT; ++a)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[a][x] = s2[a][x] = 0.f;
#pragma unroll
                for (int c = 0; c < kSteps; ++c) {
                    const uint32_t ka[4] = {widen_lo(kw[0][c]), widen_lo(kw[1][c]), widen_hi(kw[0][c]), widen_hi(kw[1][c])};
#pragma unroll
                    for (int a = 0; a < NT; ++a) mma_f16((c & 1) ? s2[a] : s[a], ka, qb[a][c][0], qb[a][c][1]);
                }
#pragma unroll
                for (int a = 0; a < NT; ++a)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[a][x] = (s[a][x] + s2[a][x]) * (cs[a][x & 1] * ks);
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
                    nan = __shfl_sync(0xffffffffu, nan, g >> 1) >> (g & 1);   // bit 0: entry g, bit 2: entry g + 8
#pragma unroll
                    for (int a = 0; a < NT; ++a)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            if ((nan >> (x & 2)) & 1) s[a][x] = NAN;
                            if (e0 + g + 4 * (x & 2) > lim[a][x & 1]) s[a][x] = -INFINITY;
                        }
                }
                float top[NT][2], vpart, vlg;
                split_scale(vs, vpart, vlg);
                bool up = false;
#pragma unroll
                for (int a = 0; a < NT; ++a)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        top[a][x] = fmaxf(s[a][x], s[a][2 + x]);
                        top[a][x] = fmaxf(top[a][x], __shfl_xor_sync(0xffffffffu, top[a][x], 4));
                        top[a][x] = fmaxf(top[a][x], __shfl_xor_sync(0xffffffffu, top[a][x], 8));
                        top[a][x] = fmaxf(top[a][x], __shfl_xor_sync(0xffffffffu, top[a][x], 16));
                        up |= top[a][x] > m[a][x] + kRescale || top[a][x] + vlg > mo[a][x] + kRescale;
                    }
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int a = 0; a < NT; ++a)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            if (top[a][x] > m[a][x] + kRescale) {
                                l[a][x] *= m[a][x] == -INFINITY ? 0.f : ex2(m[a][x] - top[a][x]);
                                m[a][x] = top[a][x];
                            }
                            float f = 1.f;
                            if (top[a][x] + vlg > mo[a][x] + kRescale) {
                                f = mo[a][x] == -INFINITY ? 0.f : ex2(mo[a][x] - (top[a][x] + vlg));
                                mo[a][x] = top[a][x] + vlg;
                            }
#pragma unroll
                            for (int j = 0; j < kMt; ++j) {
                                o[j][a][x] *= f;
                                o[j][a][2 + x] *= f;
                            }
                        }
                    __syncwarp();
                }
                uint32_t pb[NT][2];
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    // 0 in the place of both maxima where a row has seen no entry
                    const float m0 = m[a][0] == -INFINITY ? 0.f : m[a][0], m1 = m[a][1] == -INFINITY ? 0.f : m[a][1];
                    const float o0 = mo[a][0] == -INFINITY ? 0.f : mo[a][0], o1 = mo[a][1] == -INFINITY ? 0.f : mo[a][1];
                    const float r0 = vpart * lift(m0 - o0 + kLift, vlg), r1 = vpart * lift(m1 - o1 + kLift, vlg);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float w0 = ex2(s[a][2 * h] - m0), w1 = ex2(s[a][2 * h + 1] - m1);
                        l[a][0] += w0;
                        l[a][1] += w1;
                        pb[a][h] = transpose8x8(pack_f16(w0 * r0, w1 * r1));
                    }
                }
#pragma unroll
                for (int c = 0; c < kCols / 4; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t lo2 = __byte_perm(vw[0][c], vw[1][c], h == 0 ? 0x5140 : 0x7362);
                        const uint32_t hi2 = __byte_perm(vw[2][c], vw[3][c], h == 0 ? 0x5140 : 0x7362);
                        const uint32_t va[4] = {widen_lo(lo2), widen_hi(lo2), widen_lo(hi2), widen_hi(hi2)};
#pragma unroll
                        for (int a = 0; a < NT; ++a) mma_f16(o[2 * c + h][a], va, pb[a][0], pb[a][1]);
                    }
            }
        }

        // what this head's earlier windows left: a thread per row and four dimensions
        const bool early = FIRST ? page0 > 0 : seg == 0 && win->early, carry = !FIRST && seg == 0 && win->carry;
        float* part = p.part + static_cast<size_t>(2 * blockIdx.x + (early ? 0 : 1)) * part_floats(kRows, HD);
        static_assert(kRows * (HD / 4) <= kThreads, "the end of a segment");
        const int r = tid / (HD / 4), q = tid - r * (HD / 4);
        float M0 = -INFINITY, sum0 = 0.f;
        float4 acc0 = make_float4(0.f, 0.f, 0.f, 0.f);
        if (carry && r < kRows) {
            acc0 = *reinterpret_cast<const float4*>(part + r * HD + q * 4);
            M0 = part[kRows * HD + r];
            sum0 = part[kRows * HD + kRows + r];
        }
        // Join the warps: maxima and sums through a table that two segments
        // take in turn, then every warp's output relative to the common
        // maximum, two warps to a slot.
        float2* s_ml = reinterpret_cast<float2*>(sm + L::kMl) + turn * kWarps * kRows;
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                l[a][x] += __shfl_xor_sync(0xffffffffu, l[a][x], 4);
                l[a][x] += __shfl_xor_sync(0xffffffffu, l[a][x], 8);
                l[a][x] += __shfl_xor_sync(0xffffffffu, l[a][x], 16);
                if (g == 0)
                    s_ml[warp * kRows + a * 8 + 2 * t + x] = make_float2(m[a][x], mark != 0.f ? mark : l[a][x]);
            }
        __syncthreads();
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = a * 8 + 2 * t + x;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w * kRows + r].x);
                const float f = unlift(mo[a][x], M);
#pragma unroll
                for (int j = 0; j < kMt; ++j) {
                    o[j][a][x] *= f;
                    o[j][a][2 + x] *= f;
                }
            }
#pragma unroll
        for (int round = 0; round < L::kRounds; ++round) {
            if (warp / L::kSlots == round) {
                float* slot = s_o + (warp - round * L::kSlots) * kRows * HD;
#pragma unroll
                for (int a = 0; a < NT; ++a)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int r = a * 8 + 2 * t + x;
#pragma unroll
                        for (int c = 0; c < kCols / 4; ++c) {
                            float4* at = reinterpret_cast<float4*>(slot + r * HD) + ((g * (kCols / 4) + c) ^ L::swizzle(r));
                            float4 v = make_float4(o[2 * c][a][x], o[2 * c][a][2 + x], o[2 * c + 1][a][x], o[2 * c + 1][a][2 + x]);
                            if (round > 0) {
                                const float4 u = *at;
                                v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
                            }
                            *at = v;
                        }
                    }
            }
            __syncthreads();
        }
        if (r < kRows) {
            float M = -INFINITY, bad = 0.f, sum = 0.f;
            float2 ml[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) ml[w] = s_ml[w * kRows + r];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                bad = fminf(bad, ml[w].y < 0.f ? ml[w].y : 0.f);
                // a warp that saw nothing adds 0, a NaN sum stays one
                sum += ml[w].y == 0.f ? 0.f : ml[w].y * (ml[w].x == -INFINITY ? 1.f : ex2(ml[w].x - M));
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < L::kSlots; ++w) {
                const float4 v = *(reinterpret_cast<const float4*>(s_o + (w * kRows + r) * HD) + (q ^ L::swizzle(r)));
                acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
            }
            if (carry) {
                const float top = fmaxf(M, M0), f = M == top ? 1.f : ex2(M - top), f0 = M0 == top ? 1.f : ex2(M0 - top);
                bad = fminf(bad, sum0 < 0.f ? sum0 : 0.f);
                sum = sum * f + (sum0 < 0.f ? 0.f : sum0 * f0);
                acc = make_float4(acc.x * f + acc0.x * f0, acc.y * f + acc0.y * f0, acc.z * f + acc0.z * f0, acc.w * f + acc0.w * f0);
                M = top;
            }
            if (!early && page0 + len == info.w) {   // the whole head: write the output
                if (r < live) {
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    if (bad < 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    else acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                    const int j = r / G;
                    __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(
                        p.out + (static_cast<long long>(b) * p.K + j) * p.ld_out +
                        static_cast<long long>(head * G + r - j * G) * HD + q * 4);
                    dst[0] = __floats2bfloat162_rn(acc.x, acc.y);
                    dst[1] = __floats2bfloat162_rn(acc.z, acc.w);
                }
                if (info.y == 0 && tid == 0) p.status[b] = status_of(bad);
            } else {
                *reinterpret_cast<float4*>(part + r * HD + q * 4) = acc;
                if (q == 0) {
                    part[kRows * HD + r] = M;
                    part[kRows * HD + kRows + r] = bad < 0.f ? bad : sum;
                }
            }
        }
        seg += len;
    }
    copies_wait<0>();
}

// FIRST: every share's first window. Otherwise the others.
template <int HD, int NT, bool FIRST>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_kv8(const Kv8Params p) {
    using L = Smem<HD, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int4* s_info = reinterpret_cast<int4*>(sm + L::kInfo);
    int* s_tile = reinterpret_cast<int*>(sm + L::kUnit);
    __shared__ Window s_win;
    bool idle;

    pdl_launch_dependents();
    if constexpr (FIRST) {
        const int n = gather_units<kThreads, 1, kPad, kMaxUnits>(p, kMinUnits, 0, s_info, s_tile, &s_win, idle);
        attend_window<HD, NT, true>(p, sm, n, &s_win);
        if (idle) zero_idle_rows_by<1, kPad>(p, HD, threadIdx.x >> 5, kWarps);
    } else {
        pdl_wait();
        if (p.cut[gridDim.x].x <= kMaxUnits) return;
        for (int w = 1;; ++w) {
            const int n = gather_units<kThreads, 1, kPad, kMaxUnits>(p, kMinUnits, w, s_info, s_tile, &s_win, idle);
            attend_window<HD, NT, false>(p, sm, n, &s_win);
            if (!s_win.more) break;
            __syncthreads();   // all warps are done with the tables
        }
    }
}

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
__global__ void __launch_bounds__(kMergeThreads) k_kv8_merge(const Kv8Params p, int tr, int grid) {
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

// Query rows of a head from which the tensor-memory kernel is taken; it reads
// the cache once for up to 128 rows, but its unit takes as long for few. 64
// requests: 16 rows of 128-wide heads 87 us, by the register kernel 90, 8 rows
// 86 and 65; 16 rows of 64-wide heads 82 and 60 (as both were then; 89, 65, 62 now).
constexpr int umma_from(int hd) { return hd == 64 ? 17 : 9; }

int plan_kv8(int B, int K, int nq, int nkv, int hd, int max_pages, Plan* out) {
    int dev = 0, sms = 0;
    const int rc = current_device(&dev, &sms);
    if (rc != PE_OK) return rc;
    Plan a{};
    a.dev = dev;
    const int rows = K * (nq / nkv);
    const bool umma = rows >= umma_from(hd);
    a.tr = umma ? kUmmaRows : (rows <= 8 ? 8 : 16);
    a.sms = sms;
    const int pages = umma ? kUmmaPages : 1, pad = umma ? kUmmaPad : kPad;
    const int least = umma ? kUmmaLeast : kMinUnits;
    const long long most = a.most = static_cast<long long>(B) * nkv * ((max_pages + pages - 1) / pages + pad);
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

template <int HD, int NT>
int launch_rows(const Kv8Params& p, const Plan& a, cudaStream_t s) {
    constexpr auto first = k_attn_kv8<HD, NT, true>, rest = k_attn_kv8<HD, NT, false>;
    constexpr int smem = Smem<HD, NT>::kBytes;
    int rc = allow_smem<first>(a.dev, smem);
    if (rc != PE_OK) return rc;
    PE_CUDA_TRY(launch_ex(first, dim3(a.grid), dim3(kThreads), smem, s, false, p));
    if (a.most <= static_cast<long long>(a.grid) * kMaxUnits) return PE_OK;
    if ((rc = allow_smem<rest>(a.dev, smem)) != PE_OK) return rc;
    PE_CUDA_TRY(launch_ex(rest, dim3(a.grid), dim3(kThreads), smem, s, true, p));
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
    const int rows = p.K * (p.nq / p.nkv);
    // four teams (a warp, of 64-wide heads half of one) to a row where rows are
    // few (B=1 K=1, 131072 entries: 36.6 us, one team 40.9; B=128 K=11: 195 us,
    // one team 177)
    const bool share = static_cast<long long>(p.B) * p.nkv * rows <= 1024;
    const int block_rows = std::max(1, kMergeThreads / (hd / 4) / (share ? 4 : 1));
    const long long runs = std::min<long long>(a.grid - 1, static_cast<long long>(p.B) * p.nkv);   // cut ones at most
    const long long blocks = runs * ((rows + block_rows - 1) / block_rows);
    const dim3 grid(static_cast<unsigned>(std::max(1ll, std::min<long long>(blocks, a.sms * kMergeBlocks))));
    auto kern = hd == 128 ? (share ? k_kv8_merge<128, 4> : k_kv8_merge<128, 1>) : (share ? k_kv8_merge<64, 4> : k_kv8_merge<64, 1>);
    PE_CUDA_TRY(launch_ex(kern, grid, dim3(kMergeThreads), 0, s, true, p, a.tr, a.grid));
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
    p.k_codes = k_codes;
    p.v_codes = v_codes;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.scale_log2 = scale * kLog2e;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.ld_out = ld_out;
    p.status = status;
    p.cut = reinterpret_cast<int4*>(ws);
    // whole sectors: a 16-byte aligned `ws` may be half of one off
    p.part = ws + a.cut_floats + (reinterpret_cast<uintptr_t>(ws) % 32 != 0 ? 4 : 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.tr == kUmmaRows) rc = launch_umma(p, a, head_dim, s);
    else if (a.tr == 16) rc = launch_rows<64, 2>(p, a, s);   // 128-wide heads: umma_from
    else rc = head_dim == 128 ? launch_rows<128, 1>(p, a, s) : launch_rows<64, 1>(p, a, s);
    return rc != PE_OK ? rc : launch_merge(p, a, head_dim, s);   // also where no head is shared: it reports a wait that gave up
}
