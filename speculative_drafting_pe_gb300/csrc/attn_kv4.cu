// Paged GQA attention over the 4-bit KV cache (pe_attention_kv4): codes 0..15
// with a scale and a base for each (entry, kv head), bf16 queries and output.
//
//   o_r = sum_e w_re v_e / sum_e w_re,  w_re = exp(scale * q_r . k_e),
//   k_e = ks_e (kcode_e - 8) + kc_e,  v_e = vs_e (vcode_e - 8) + vc_e,  c = base + 8 s
//
// over the entries e <= S_b + j that row r (draft row j of request b) sees, in
// one pass with a running maximum (base 2). Scales and bases never touch the
// codes: a score is ks_e (q_r . (kcode_e - 8)) + kc_e sum(q_r), and an output
// sum_e (w_re vs_e)(vcode_e - 8) + sum_e w_re vc_e, whose second term is one
// number a row. Everything but the two products is fp32.
//
// This file: the kernel for few query rows of a head (single tokens) and the
// entry point. The line of units that the CTAs divide is described in
// attn_line.cuh; a unit here is two pages.
//
// A warp takes every twelfth unit of its CTA, kStages units ahead, through
// asynchronous copies of its own lanes, so the warps never wait for each other
// while they stream. Both products are transposed, S^T = K Q^T and
// O^T = V^T P^T, so that the entries and the dimensions fill the 16 rows of
// mma.m16n8k16 and 8 query rows its columns. The codes are widened to fp16 in
// registers, 9 instructions for 8 of them: ldmatrix hands a lane a word of
// eight neighbouring dimensions of a K row, whose pairs (x, x + 4) are what the
// masks of `widen` leave (Q's fragments follow that order), and its transposed
// form four dimensions of two V rows in the two halves of a word, which is what
// a fragment of V^T wants. P^T comes out of S^T's layout by 8x8 transposes.
// What bounds it is instructions and their latency: some 900 for a unit's warp,
// 288 of them widening, of three warps a scheduler, which issue one in 54% of the
// cycles (ALU 49%). 64 single tokens over 512..8192 entries, 32/4 heads of 128:
// 50.4 us, 2.4 TB/s; one of 131072 entries 29; 64 single tokens over 1024..4096,
// 64/8 heads of 64: 47. 16 warps of 128 registers instead: 56 and 31 of the first
// two.
// Queries enter as fp16 after an exact shift by a power of two per row;
// weights times V's scale go to fp16 (2^-11) relative to the row's largest such
// product so far (kLift).
#include <algorithm>

#include "attn_kv4.cuh"

namespace pe {
namespace {

using namespace kv4;

constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;
constexpr int kPages = 2;          // pages of a unit
constexpr int kMaxUnits = 1024;    // units of a window
constexpr int kMinUnits = kWarps;  // a CTA's share is at least one unit per warp
constexpr int kPad = 16;           // a segment's end in units
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void load_transposed(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

// NT: tiles of 8 query rows
template <int HD, int NT>
struct Smem {
    static constexpr int kRows = 8 * NT;
    static constexpr int kRow = HD / 2;                      // bytes of an entry's codes
    static constexpr int kTile = kPage * kRow;               // a page's K or V codes of one head
    static constexpr int kPar = kPage * 4;                   // and their parameters
    static constexpr int kStages = HD == 128 ? 2 : 4;        // units in flight per warp: 104 (108) KB per SM
    static constexpr int kUnit = kPages * 2 * (kTile + kPar);   // codes (page, side), then parameters likewise
    static constexpr int kRounds = NT;                       // warps that share a slot of sums
    static constexpr int kSlots = kWarps / kRounds;
    static constexpr int kRing = kWarps * kStages * kUnit;
    static constexpr int kO = kRing;                         // [kSlots][kRows][HD] fp32
    static constexpr int kMl = kO + kSlots * kRows * HD * 4; // [2][kWarps][kRows] (max, sum, sum of w vc)
    static constexpr int kInfo = kMl + 2 * kWarps * kRows * 16;
    static constexpr int kTab = kInfo + kMaxUnits * 16;      // tile
    static constexpr int kBytes = kTab + kMaxUnits * kPages * 4 + 1024;
    // 16-byte chunk c of row r of a slot stands at c ^ swizzle(r): the lanes
    // of a quarter warp (four row pairs, two chunks) meet no bank twice
    __device__ static __forceinline__ int swizzle(int r) { return ((r >> 1) & 3) * 2; }
    // where chunk c of row r of a page's codes stands: eight rows of a chunk lie in different banks
    __device__ static __forceinline__ int place(int r, int c) {
        return HD == 128 ? (r * 4 + (c ^ ((r >> 1) & 3))) * 16 : (r * 2 + (c ^ ((r >> 2) & 1))) * 16;
    }
};
static_assert(Smem<128, 2>::kBytes <= 232448 - 2048 && Smem<64, 2>::kBytes <= 232448 - 2048, "shared memory of a block");

// exponent of a scale as 2^lg, kept within what stays normal in the products below
__device__ __forceinline__ float exponent_of(uint32_t par) {
    const uint32_t e = max((par >> 7) & 0xFFu, 23u);
    return __uint_as_float(0x4B000000u | e) - (8388608.f + 127.f);
}

// The n units of a window; FIRST: of the share's first one.
template <int HD, int NT, bool FIRST>
__device__ __forceinline__ void attend_window(const Kv4Params& p, uint8_t* sm, int n, const Window* win) {
    using L = Smem<HD, NT>;
    constexpr int kRows = L::kRows, kStages = L::kStages;
    constexpr int kChunks = HD / 32;      // 16-byte chunks of an entry's codes
    constexpr int kMt = HD / 16;          // 16-dimension tiles of the output
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    uint8_t* ring = sm + warp * kStages * L::kUnit;
    float* s_o = reinterpret_cast<float*>(sm + L::kO);
    int4* s_info = reinterpret_cast<int4*>(sm + L::kInfo);
    int* s_tile = reinterpret_cast<int*>(sm + L::kTab);

    const uint64_t policy = l2_policy_evict_first();
    const uint32_t ring_at = smem_u32(ring);
    auto fetch = [&](int i, int st) {   // unit i into stage st; a group even where there is nothing to copy
        if (i < n) {
            const uint32_t at = ring_at + st * L::kUnit;
#pragma unroll
            for (int q = 0; q < kPages; ++q) {
                const int tile = s_tile[i * kPages + q];
                if (tile < 0) continue;
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    const uint8_t* from = (side == 0 ? p.k_codes : p.v_codes) + static_cast<size_t>(tile) * L::kTile + lane * 16;
#pragma unroll
                    for (int x = 0; x < L::kTile / 512; ++x) {
                        const int c = lane + 32 * x;
                        copy_async<16>(at + (q * 2 + side) * L::kTile + L::place(c / kChunks, c % kChunks), from + x * 512, policy);
                    }
                }
            }
            // parameters: a lane has a quarter of a page's K or V ones
            const int q = lane >> 3, side = (lane >> 2) & 1, part = lane & 3;
            const int tile = lane < 8 * kPages ? s_tile[i * kPages + q] : -1;
            if (tile >= 0)
                copy_async<16>(at + kPages * 2 * L::kTile + (q * 2 + side) * L::kPar + part * 16,
                               (side == 0 ? p.k_params : p.v_params) + static_cast<size_t>(tile) * kPage + part * 4, policy);
        }
        copies_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) fetch(warp + s * kWarps, s);
    int st = 0;            // the stage of this warp's next unit
    // matrices of a page's codes: rows 0-7 and 8-15 of chunk 2j, then of chunk 2j + 1
    uint32_t mat[kChunks / 2];
#pragma unroll
    for (int j = 0; j < kChunks / 2; ++j) mat[j] = static_cast<uint32_t>(L::place(lane & 15, 2 * j + (lane >> 4)));

    const int G = p.nq / p.nkv;
    int i = warp;          // this warp's next unit
    int turn = 0;
    for (int seg = 0; seg < n; turn ^= 1) {
        const int4 info = s_info[seg];
        const int b = info.x, unit0 = info.z;
        const int len = min(info.w - unit0, n - seg);
        const int S = p.seq_lens[b];
        const int rows = p.rows != nullptr ? p.rows[b] : p.K;
        const int head = info.y, live = rows * G;
        const int last = S + rows - 1;                    // last entry that any row sees
        float mark = 0.f;
        // of rows a * 8 + 2t + x: o[2c + y][a][2z + x] is dimension 32c + 4g + 2y + z
        float o[kMt][NT][4];
#pragma unroll
        for (int j = 0; j < kMt; ++j)
#pragma unroll
            for (int a = 0; a < NT; ++a) o[j][a][0] = o[j][a][1] = o[j][a][2] = o[j][a][3] = 0.f;
        // maximum of the scores; of their products with V's scale, relative to it; sums of the weights and of weights
        // times vc
        float m[NT][2], md[NT][2], l[NT][2], u[NT][2];
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int x = 0; x < 2; ++x) m[a][x] = md[a][x] = -INFINITY, l[a][x] = u[a][x] = 0.f;

        if (i < seg + len) {
            // queries: row a * 8 + g, dimensions 32c + 8t .. + 7
            uint32_t qb[NT][kChunks][4];
            float cs[NT][2], cq[NT][2];   // of rows a * 8 + 2t + x: factor of a product, of kc
            int lim[NT][2];
#pragma unroll
            for (int a = 0; a < NT; ++a) {
                const int r = a * 8 + g, j = r / G;
                const __nv_bfloat16* src =
                    p.q + (static_cast<long long>(b) * p.K + j) * p.ld_q +
                    static_cast<long long>(head * G + r - j * G) * HD + t * 8;
                uint4 raw[kChunks];
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    raw[c] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < live) raw[c] = *reinterpret_cast<const uint4*>(src + c * 32);
                }
                uint32_t top = 0;
                const uint32_t* w = reinterpret_cast<const uint32_t*>(raw);
#pragma unroll
                for (int c = 0; c < kChunks * 4; ++c) top = max(top, max((w[c] << 16) & 0x7FFF0000u, w[c] & 0x7FFF0000u));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // the row times 2^(127 - E): its largest value lies in [1, 2)
                const int E = min(max(static_cast<int>(top >> 23), 1), 253);
                const float down = __uint_as_float(static_cast<uint32_t>(254 - E) << 23);
                // a row that holds an infinity (or a NaN) is NaN
                const float up = top >= 0x7F800000u ? NAN : p.scale_log2 * __uint_as_float(static_cast<uint32_t>(E) << 23);
                float total = 0.f;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    float f[8];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        f[2 * y] = __uint_as_float(w[c * 4 + y] << 16) * down;
                        f[2 * y + 1] = __uint_as_float(w[c * 4 + y] & 0xFFFF0000u) * down;
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        qb[a][c][y] = pack_f16(f[y], f[y + 4]);
                        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&qb[a][c][y]));
                        total += v.x + v.y;
                    }
                }
                total += __shfl_xor_sync(0xffffffffu, total, 1);
                total += __shfl_xor_sync(0xffffffffu, total, 2);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    cs[a][x] = __shfl_sync(0xffffffffu, up, (2 * t + x) * 4);
                    cq[a][x] = __shfl_sync(0xffffffffu, up * total, (2 * t + x) * 4);
                    const int rx = a * 8 + 2 * t + x;
                    lim[a][x] = rx < live ? S + rx / G : -1;
                }
            }
            for (; i < seg + len; i += kWarps) {
                copies_wait<kStages - 1>();
                __syncwarp();   // all lanes' copies
                if (s_tile[i * kPages] == -1 || s_tile[i * kPages + 1] == -1) {
                    mark = kMarkBadPage;
                    fetch(i + kStages * kWarps, st);
                    st = st + 1 == kStages ? 0 : st + 1;
                    continue;
                }
                const uint32_t at = ring_at + st * L::kUnit;
                const uint32_t* par = reinterpret_cast<const uint32_t*>(ring + st * L::kUnit + kPages * 2 * L::kTile);
                const int e0 = (unit0 + i - seg) * (kPages * kPage);   // the unit's first entry
                const bool inner = e0 + kPages * kPage - 1 <= S;       // every row sees all of it

                // S^T: entries g and g + 8 of both pages
                float s[kPages][NT][4];
                uint32_t vp[kPages][2];   // parameters of these entries' V
#pragma unroll
                for (int q = 0; q < kPages; ++q) {
                    uint32_t kw[kChunks][2];
#pragma unroll
                    for (int j = 0; j < kChunks / 2; ++j) {
                        uint32_t x[4];
                        load_matrices(x, at + q * 2 * L::kTile + mat[j]);
                        kw[2 * j][0] = x[0]; kw[2 * j][1] = x[1];
                        kw[2 * j + 1][0] = x[2]; kw[2 * j + 1][1] = x[3];
                    }
                    float s2[NT][4];   // two chains of MMAs
#pragma unroll
                    for (int a = 0; a < NT; ++a)
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[q][a][x] = s2[a][x] = 0.f;
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        uint32_t k0[4], k1[4];
                        widen(kw[c][0], k0);
                        widen(kw[c][1], k1);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t ka[4] = {k0[2 * h], k1[2 * h], k0[2 * h + 1], k1[2 * h + 1]};
#pragma unroll
                            for (int a = 0; a < NT; ++a)
                                mma_f16(h == 0 ? s[q][a] : s2[a], ka, qb[a][c][2 * h], qb[a][c][2 * h + 1]);
                        }
                    }
                    const uint32_t kp[2] = {par[q * 2 * kPage + g], par[q * 2 * kPage + g + 8]};
                    vp[q][0] = par[(q * 2 + 1) * kPage + g];
                    vp[q][1] = par[(q * 2 + 1) * kPage + g + 8];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float ks = scale_of(kp[h]), kc = mid_of(kp[h]);
#pragma unroll
                        for (int a = 0; a < NT; ++a)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const float acc = s[q][a][2 * h + x] + s2[a][2 * h + x];
                                s[q][a][2 * h + x] = fmaf(ks, acc * cs[a][x], kc * cq[a][x]);
                            }
                    }
                }
                // V: dimensions 32c + 4g .. + 3 of entries 2t, 2t + 1, and of 2t + 8, 2t + 9
                uint32_t vw[kPages][kChunks][2];
#pragma unroll
                for (int q = 0; q < kPages; ++q)
#pragma unroll
                    for (int j = 0; j < kChunks / 2; ++j) {
                        uint32_t x[4];
                        load_transposed(x, at + (q * 2 + 1) * L::kTile + mat[j]);
                        vw[q][2 * j][0] = x[0]; vw[q][2 * j][1] = x[1];
                        vw[q][2 * j + 1][0] = x[2]; vw[q][2 * j + 1][1] = x[3];
                    }
                __syncwarp();
                fetch(i + kStages * kWarps, st);
                st = st + 1 == kStages ? 0 : st + 1;

                if (!inner) {
                    // Entries that some row does not see. Parameters of V that
                    // are not finite would reach the other rows as 0 * NaN, so
                    // they enter through the score instead; what stands behind
                    // the last entry is no one's.
#pragma unroll
                    for (int q = 0; q < kPages; ++q)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int e = e0 + q * kPage + g + 8 * h;
                            const float mid = mid_of(vp[q][h]);
                            const bool odd = mid != mid;
                            if (odd || e > last) vp[q][h] = 0u;
#pragma unroll
                            for (int a = 0; a < NT; ++a)
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    if (odd) s[q][a][2 * h + x] = NAN;
                                    if (e > lim[a][x]) s[q][a][2 * h + x] = -INFINITY;
                                }
                        }
                }
                float vlg[kPages][2];
#pragma unroll
                for (int q = 0; q < kPages; ++q) vlg[q][0] = exponent_of(vp[q][0]), vlg[q][1] = exponent_of(vp[q][1]);
                // the running maximum, then scores relative to it
                float top[NT][2];
                bool up = false;
#pragma unroll
                for (int a = 0; a < NT; ++a)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        top[a][x] = fmaxf(fmaxf(s[0][a][x], s[0][a][2 + x]), fmaxf(s[1][a][x], s[1][a][2 + x]));
                        up |= top[a][x] > m[a][x] + kRescale;
                    }
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int a = 0; a < NT; ++a)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) top[a][x] = fmaxf(top[a][x], __shfl_xor_sync(0xffffffffu, top[a][x], d));
                            if (top[a][x] > m[a][x] + kRescale) {
                                if (m[a][x] != -INFINITY) {
                                    const float f = ex2(m[a][x] - top[a][x]);
                                    l[a][x] *= f;
                                    u[a][x] *= f;
                                    md[a][x] += m[a][x] - top[a][x];
                                }
                                m[a][x] = top[a][x];
                            }
                        }
                    __syncwarp();
                }
                up = false;
                float most[NT][2];
#pragma unroll
                for (int a = 0; a < NT; ++a)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float from = m[a][x] == -INFINITY ? 0.f : m[a][x];   // a row that has seen no entry
#pragma unroll
                        for (int q = 0; q < kPages; ++q) s[q][a][x] -= from, s[q][a][2 + x] -= from;
                        most[a][x] = fmaxf(fmaxf(s[0][a][x] + vlg[0][0], s[0][a][2 + x] + vlg[0][1]),
                                           fmaxf(s[1][a][x] + vlg[1][0], s[1][a][2 + x] + vlg[1][1]));
                        up |= most[a][x] > md[a][x] + kRescale;
                    }
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int a = 0; a < NT; ++a)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) most[a][x] = fmaxf(most[a][x], __shfl_xor_sync(0xffffffffu, most[a][x], d));
                            if (most[a][x] > md[a][x] + kRescale) {
                                const float f = md[a][x] == -INFINITY ? 0.f : ex2(md[a][x] - most[a][x]);
                                md[a][x] = most[a][x];
#pragma unroll
                                for (int j = 0; j < kMt; ++j) {
                                    o[j][a][x] *= f;
                                    o[j][a][2 + x] *= f;
                                }
                            }
                        }
                    __syncwarp();
                }
                uint32_t pb[kPages][NT][2];
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    // (nothing seen: weights of 0). A weight meets its scale first: 0 times any scale is 0, where scale
                    // times lift, of values far above all that has weight, would be an infinity and 0 times it NaN.
                    const float r0 = md[a][0] == -INFINITY ? 0.f : ex2(kLift - md[a][0]);
                    const float r1 = md[a][1] == -INFINITY ? 0.f : ex2(kLift - md[a][1]);
#pragma unroll
                    for (int q = 0; q < kPages; ++q)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float vs = scale_of(vp[q][h]), vc = mid_of(vp[q][h]);
                            const float w0 = ex2(s[q][a][2 * h]), w1 = ex2(s[q][a][2 * h + 1]);
                            l[a][0] += w0;
                            l[a][1] += w1;
                            u[a][0] = fmaf(w0, vc, u[a][0]);
                            u[a][1] = fmaf(w1, vc, u[a][1]);
                            pb[q][a][h] = transpose8x8(pack_f16(w0 * vs * r0, w1 * vs * r1));
                        }
                }
#pragma unroll
                for (int q = 0; q < kPages; ++q)
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        uint32_t v0[4], v1[4];   // words' four dimensions, of entries 2t, 2t + 1 and of 2t + 8, 2t + 9
                        widen(vw[q][c][0], v0);
                        widen(vw[q][c][1], v1);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t va[4] = {v0[2 * y], v0[2 * y + 1], v1[2 * y], v1[2 * y + 1]};
#pragma unroll
                            for (int a = 0; a < NT; ++a) mma_f16(o[2 * c + y][a], va, pb[q][a][0], pb[q][a][1]);
                        }
                    }
            }
        }

        // what this head's earlier windows left: a thread per row and four dimensions
        const bool early = FIRST ? unit0 > 0 : seg == 0 && win->early, carry = !FIRST && seg == 0 && win->carry;
        float* part = p.part + static_cast<size_t>(2 * blockIdx.x + (early ? 0 : 1)) * part_floats(kRows, HD);
        // Join the warps: maxima and sums through a table that two segments
        // take in turn, then every warp's output relative to the common
        // maximum, NT warps to a slot.
        float4* s_ml = reinterpret_cast<float4*>(sm + L::kMl) + turn * kWarps * kRows;
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l[a][x] += __shfl_xor_sync(0xffffffffu, l[a][x], d);
                    u[a][x] += __shfl_xor_sync(0xffffffffu, u[a][x], d);
                }
                if (g == 0)
                    s_ml[warp * kRows + a * 8 + 2 * t + x] = make_float4(m[a][x], mark != 0.f ? mark : l[a][x], u[a][x], 0.f);
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
                const float f = unlift(m[a][x], md[a][x], M);
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
                        for (int c = 0; c < kChunks; ++c) {
                            float4* to = reinterpret_cast<float4*>(slot + r * HD) + ((c * 8 + g) ^ L::swizzle(r));
                            float4 v = make_float4(o[2 * c][a][x], o[2 * c][a][2 + x], o[2 * c + 1][a][x], o[2 * c + 1][a][2 + x]);
                            if (round > 0) {
                                const float4 had = *to;
                                v.x += had.x; v.y += had.y; v.z += had.z; v.w += had.w;
                            }
                            *to = v;
                        }
                    }
            }
            __syncthreads();
        }
        constexpr int kQuads = HD / 4;
        for (int x = tid; x < kRows * kQuads; x += kThreads) {
            const int r = x / kQuads, q = x - r * kQuads;
            float M = -INFINITY, bad = 0.f, sum = 0.f, mid = 0.f;
            float4 ml[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) ml[w] = s_ml[w * kRows + r];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml[w].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                bad = fminf(bad, ml[w].y < 0.f ? ml[w].y : 0.f);
                // a warp that saw nothing adds 0, a NaN sum stays one
                const float f = ml[w].x == -INFINITY ? 1.f : ex2(ml[w].x - M);
                sum += ml[w].y == 0.f ? 0.f : ml[w].y * f;
                mid += ml[w].y == 0.f ? 0.f : ml[w].z * f;
            }
            float4 acc = make_float4(mid, mid, mid, mid);
#pragma unroll
            for (int w = 0; w < L::kSlots; ++w) {
                const float4 v = *(reinterpret_cast<const float4*>(s_o + (w * kRows + r) * HD) + (q ^ L::swizzle(r)));
                acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
            }
            if (carry) {
                const float4 acc0 = *reinterpret_cast<const float4*>(part + r * HD + q * 4);
                const float M0 = part[kRows * HD + r], sum0 = part[kRows * HD + kRows + r];
                const float top = fmaxf(M, M0), f = M == top ? 1.f : ex2(M - top), f0 = M0 == top ? 1.f : ex2(M0 - top);
                bad = fminf(bad, sum0 < 0.f ? sum0 : 0.f);
                sum = sum * f + (sum0 < 0.f ? 0.f : sum0 * f0);
                acc = make_float4(acc.x * f + acc0.x * f0, acc.y * f + acc0.y * f0, acc.z * f + acc0.z * f0, acc.w * f + acc0.w * f0);
                M = top;
            }
            if (!early && unit0 + len == info.w) {   // the whole head: write the output
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
                if (info.y == 0 && x == 0) p.status[b] = status_of(bad);
            } else {
                *reinterpret_cast<float4*>(part + r * HD + q * 4) = acc;
                __syncwarp();   // a carried row's maximum and sum have been read
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
    k_attn_kv4(const Kv4Params p) {
    using L = Smem<HD, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + (1024u - smem_u32(smem_raw) % 1024u) % 1024u;   // (an offset: still known to be shared memory)
    int4* s_info = reinterpret_cast<int4*>(sm + L::kInfo);
    int* s_tile = reinterpret_cast<int*>(sm + L::kTab);
    __shared__ Window s_win;
    bool idle;

    pdl_launch_dependents();
    if constexpr (FIRST) {
        const int n = gather_units<kThreads, kPages, kPad, kMaxUnits>(p, kMinUnits, 0, s_info, s_tile, &s_win, idle);
        attend_window<HD, NT, true>(p, sm, n, &s_win);
        if (idle) zero_idle_rows_by<kPages, kPad>(p, HD, threadIdx.x >> 5, kWarps);
    } else {
        pdl_wait();
        if (p.cut[gridDim.x].x <= kMaxUnits) return;
        for (int w = 1;; ++w) {
            const int n = gather_units<kThreads, kPages, kPad, kMaxUnits>(p, kMinUnits, w, s_info, s_tile, &s_win, idle);
            attend_window<HD, NT, false>(p, sm, n, &s_win);
            if (!s_win.more) break;
            __syncthreads();   // all warps are done with the tables
        }
    }
}

// Query rows of a head up to which the register kernel is taken. At 16 of them, 64 requests of 512..8192 entries: 83 us,
// by the tensor-memory kernel 107 (64-wide heads 102, 164); one request of 2048: 13.2, 13.6.
constexpr int kFewRows = 16;

int plan_kv4(int B, int K, int nq, int nkv, int hd, int max_pages, Plan* out) {
    const int rows = K * (nq / nkv);
    if (rows > kFewRows) return plan_umma(B, nkv, hd, max_pages, out);
    return plan_line(B, nkv, hd, max_pages, kPages, kPad, kMinUnits, rows <= 8 ? 8 : 16, out);
}

template <int HD, int NT>
int launch_rows(const Kv4Params& p, const Plan& a, cudaStream_t s) {
    constexpr auto first = k_attn_kv4<HD, NT, true>, rest = k_attn_kv4<HD, NT, false>;
    constexpr int smem = Smem<HD, NT>::kBytes;
    int rc = allow_smem<first>(a.dev, smem);
    if (rc != PE_OK) return rc;
    PE_CUDA_TRY(launch_ex(first, dim3(a.grid), dim3(kThreads), smem, s, false, p));
    if (a.most <= static_cast<long long>(a.grid) * kMaxUnits) return PE_OK;
    if ((rc = allow_smem<rest>(a.dev, smem)) != PE_OK) return rc;
    PE_CUDA_TRY(launch_ex(rest, dim3(a.grid), dim3(kThreads), smem, s, true, p));
    return PE_OK;
}

}  // namespace
}  // namespace pe

using namespace pe;

extern "C" int pe_attention_kv4_scratch(int32_t B, int32_t K, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                        int32_t max_pages, int64_t* ws_floats) {
    if (ws_floats == nullptr) { set_error("null argument"); return PE_ERR_ARG; }
    int rc = check_shape(B, K, n_q_heads, n_kv_heads, head_dim, max_pages);
    if (rc != PE_OK) return rc;
    Plan a;
    if ((rc = plan_kv4(B, K, n_q_heads, n_kv_heads, head_dim, max_pages, &a)) != PE_OK) return rc;
    *ws_floats = static_cast<int64_t>(a.ws_floats);
    return PE_OK;
}

extern "C" int pe_attention_kv4(int32_t B, int32_t K, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                const void* q, int64_t ld_q, const int32_t* seq_lens, const int32_t* rows,
                                const int32_t* page_table, int32_t max_pages, int32_t num_pages,
                                const uint8_t* k_codes, const uint8_t* v_codes, const void* k_params,
                                const void* v_params, float scale, void* out, int64_t ld_out, float* ws,
                                int64_t ws_floats, int32_t* status, void* stream) {
    int rc = check_shape(B, K, n_q_heads, n_kv_heads, head_dim, max_pages);
    if (rc != PE_OK) return rc;
    if (num_pages < 1 || static_cast<long long>(num_pages) * n_kv_heads * kPage > 0x7FFFFFFFll) {
        set_error("num_pages must be >= 1 and num_pages * n_kv_heads * 16 fit a signed 32-bit row index");
        return PE_ERR_ARG;
    }
    if (!q || !seq_lens || !page_table || !k_codes || !v_codes || !k_params || !v_params || !out || !ws || !status) {
        set_error("null tensor argument");
        return PE_ERR_ARG;
    }
    if (out == q || status == seq_lens || (rows != nullptr && status == rows)) {
        set_error("out must not be q, status neither seq_lens nor rows");
        return PE_ERR_ARG;
    }
    const int64_t width = static_cast<int64_t>(n_q_heads) * head_dim;
    if (ld_q < width || ld_out < width || ld_q % 8 != 0 || ld_out % 8 != 0) {
        set_error("row strides must be multiples of 8 and at least n_q_heads * head_dim");
        return PE_ERR_ARG;
    }
    const uintptr_t bits = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) |
                           reinterpret_cast<uintptr_t>(k_codes) | reinterpret_cast<uintptr_t>(v_codes) |
                           reinterpret_cast<uintptr_t>(k_params) | reinterpret_cast<uintptr_t>(v_params) |
                           reinterpret_cast<uintptr_t>(ws);
    if ((bits & 15u) != 0) { set_error("q, out, ws and the cache's arrays must be 16-byte aligned"); return PE_ERR_ARG; }
    Plan a;
    if ((rc = plan_kv4(B, K, n_q_heads, n_kv_heads, head_dim, max_pages, &a)) != PE_OK) return rc;
    if (ws_floats < static_cast<int64_t>(a.ws_floats)) {
        set_error("attention scratch too small: " + std::to_string(a.ws_floats) + " floats needed");
        return PE_ERR_ARG;
    }
    Kv4Params p{};
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
    p.k_params = static_cast<const uint32_t*>(k_params);
    p.v_params = static_cast<const uint32_t*>(v_params);
    p.scale_log2 = scale * kLog2e;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.ld_out = ld_out;
    p.status = status;
    p.cut = reinterpret_cast<int4*>(ws);
    // whole sectors: a 16-byte aligned `ws` may be half of one off
    p.part = ws + a.cut_floats + (reinterpret_cast<uintptr_t>(ws) % 32 != 0 ? 4 : 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.tr > kFewRows) rc = launch_umma(p, a, head_dim, s);
    else if (a.tr == 16) rc = head_dim == 128 ? launch_rows<128, 2>(p, a, s) : launch_rows<64, 2>(p, a, s);
    else rc = head_dim == 128 ? launch_rows<128, 1>(p, a, s) : launch_rows<64, 1>(p, a, s);
    return rc != PE_OK ? rc : launch_merge(p, a, head_dim, s);
}
