// Attention over the 8-bit KV cache for many query rows (a draft pass: K rows
// of every head of a group): the tensor-memory kernel behind pe_attention_kv8.
//
// A unit is 64 entries (4 pages) of one (request, kv head); all its query rows
// (at most 128, the MMA's M) share every entry, so the cache is read once. The
// codes are widened to fp16, which holds every E4M3 value, once per tile, in
// shared memory, by warps of their own; the products run as tcgen05.mma on
// fp16 with fp32 sums in tensor memory. Roles (448 threads):
//   warp 8      TMA: the tile's K and V pages into a ring of raw stages
//   warps 10-13 converters: raw codes to fp16 K and V tiles (128-byte swizzle;
//               V stays entry-major and is read as an MN-major operand), V of
//               entries that no row sees to zero, and at the start of a
//               segment the query rows, as fp16 after an exact shift by a
//               power of two per row, into one of two query tiles
//   warp 9      lane 0 issues S_t = Q K_t^T (M=128, N=64) and O += P_t V_t
//               (A = P_t from tensor memory)
//   warps 0-3, 4-7  two softmax groups, thread = query row = TMEM lane: group
//               x takes the tiles t = x (mod 2), with a running maximum, sum
//               and output accumulator of its own, so that neither waits for
//               the other; they meet at the end of a segment.
// One S_t buffer per group: P_t (fp16 pairs) overwrites the columns of S_t,
// and S_{t+2} is issued after P_t V_t. The MMAs of a CTA complete in order, so
// a complete S_{t+2} also says that the accumulator is at rest.
#include "attn_kv8.cuh"

namespace pe {
namespace {

using namespace kv8;

constexpr int kThreads = 448;
constexpr int kTile = kUmmaPages * kPage;   // entries of a unit
constexpr int kRows = kUmmaRows;
constexpr int kSoft = 256;                  // softmax threads
constexpr int kWarpTma = 8, kWarpMma = 9, kWarpConv = 10;

// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

template <int HD>
struct Layout {
    static constexpr int kSub = HD / 64;                     // 128-byte sub-tiles of an fp16 row
    static constexpr int kRaw = HD == 128 ? 3 : 6;           // raw stages
    static constexpr int kCv = HD == 128 ? 3 : 4;            // fp16 tiles
    static constexpr int kRawTile = kTile * HD;              // codes of K or V of a tile
    static constexpr int kCvTile = kTile * HD * 2;
    static constexpr int kQTile = kRows * HD * 2;
    static constexpr int kQ = 0;                             // [2]
    static constexpr int kConv = kQ + 2 * kQTile;            // [kCv][K, V]
    static constexpr int kRing = kConv + kCv * 2 * kCvTile;  // [kRaw][K, V]
    static constexpr int kInfo = kRing + kRaw * 2 * kRawTile;
    static constexpr int kUnit = kInfo + kUmmaUnits * 16;
    static constexpr int kCs = kUnit + kUmmaUnits * kUmmaPages * 12;   // [2][kRows]
    static constexpr int kEx = kCs + 2 * kRows * 4;          // [2][kRows] float4
    static constexpr int kNan = kEx + 2 * kRows * 16;        // [kCv][kTile] bytes
    static constexpr int kBar = kNan + kCv * kTile;
    // raw_full, raw_empty [kRaw], cv_full, cv_empty [kCv], s_full, p_full, o_done [2]
    static constexpr int kBars = 2 * kRaw + 2 * kCv + 6;
    static constexpr int kTmem = kBar + kBars * 8;
    static constexpr int kBytes = kTmem + 16 + 1024;
};
static_assert(Layout<128>::kBytes <= 232448 - 128 && Layout<64>::kBytes <= 232448 - 128, "shared memory of a block");

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_kv8_umma(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const Kv8Params p) {
    using L = Layout<HD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ int s_abort;
    const volatile int* abort = &s_abort;
    int4* s_info = reinterpret_cast<int4*>(sm + L::kInfo);
    int* s_tile = reinterpret_cast<int*>(sm + L::kUnit);
    float* s_ks = reinterpret_cast<float*>(s_tile + kUmmaUnits * kUmmaPages);
    float* s_vs = s_ks + kUmmaUnits * kUmmaPages;
    float* s_cs = reinterpret_cast<float*>(sm + L::kCs);
    float4* s_ex = reinterpret_cast<float4*>(sm + L::kEx);
    uint8_t* s_nan = sm + L::kNan;
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t* raw_empty = raw_full + L::kRaw;
    uint64_t* cv_full = raw_empty + L::kRaw;
    uint64_t* cv_empty = cv_full + L::kCv;
    uint64_t* s_full = cv_empty + L::kCv;
    uint64_t* p_full = s_full + 2;
    uint64_t* o_done = p_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::kTmem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.nq / p.nkv;

    pdl_launch_dependents();
    if (tid == 0) {
        s_abort = 0;
        for (int s = 0; s < L::kRaw; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], 4);
        }
        for (int s = 0; s < L::kCv; ++s) {
            mbar_init(&cv_full[s], 4);
            mbar_init(&cv_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 128);
            mbar_init(&o_done[s], 1);
        }
        fence_mbar_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    int lo;
    const int n = gather_units<kThreads, kUmmaPages, kRows>(p, 1, s_info, s_tile, s_ks, s_vs, lo);
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t t_o = tmem + 128;     // group x's output: columns 128 + x * HD ..
    bool ok = true;

    if (warp == kWarpTma) {
        if (lane == 0) {
            const uint64_t policy = l2_policy_evict_first();
            for (int i = 0; i < n; ++i) {
                const int st = i % L::kRaw;
                if (i >= L::kRaw && !mbar_wait_ab(&raw_empty[st], static_cast<uint32_t>((i / L::kRaw) & 1) ^ 1u, nullptr, 0u, abort)) {
                    ok = false;
                    break;
                }
                uint8_t* kt = sm + L::kRing + st * 2 * L::kRawTile;
                int pages = 0;
                for (int q = 0; q < kUmmaPages; ++q) pages += s_tile[i * kUmmaPages + q] >= 0;
                mbar_arrive_expect_tx(&raw_full[st], static_cast<uint32_t>(pages * 2 * kPage * HD));
                for (int q = 0; q < kUmmaPages; ++q) {
                    const int tile = s_tile[i * kUmmaPages + q];
                    if (tile < 0) continue;
                    tma_load_2d(kt + q * kPage * HD, &tmK, &raw_full[st], 0, tile * kPage, policy);
                    tma_load_2d(kt + L::kRawTile + q * kPage * HD, &tmV, &raw_full[st], 0, tile * kPage, policy);
                }
            }
        }
        __syncwarp();
    } else if (warp == kWarpMma) {
        // The whole warp walks the units and one elected lane issues: in
        // warp-uniform control flow the descriptors stay in uniform registers.
        // Issued by a branch on the lane number, each MMA took about 125
        // cycles to issue and the kernel 2000 cycles a unit.
        if (n > 0) {
            const uint32_t idesc_s = umma_idesc(0, kRows, kTile);
            const uint32_t idesc_o = umma_idesc(0, kRows, HD) | kIdescBMnMajor;
            const uint32_t q_base = smem_u32(sm + L::kQ), cv_base = smem_u32(sm + L::kConv);
            // S and P.V walk the segments each for itself
            int s_end = min(s_info[0].w - s_info[0].z, n), s_no = 0;
            auto issue_s = [&](int i) -> bool {
                if (i == s_end) {
                    s_end = i + min(s_info[i].w - s_info[i].z, n - i);
                    ++s_no;
                }
                const int c = i % L::kCv;
                if (!mbar_wait_ab(&cv_full[c], static_cast<uint32_t>((i / L::kCv) & 1), nullptr, 0u, abort)) return false;
                tc_fence_after_sync();
                const uint32_t q_addr = q_base + (s_no & 1) * L::kQTile, k_addr = cv_base + c * 2 * L::kCvTile;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) {
                        const uint32_t sub = static_cast<uint32_t>(kk >> 2), within = static_cast<uint32_t>((kk & 3) * 32);
                        UmmaKind<__nv_bfloat16>::mma(tmem + static_cast<uint32_t>((i & 1) * kTile),
                                                     umma_desc_sw128(q_addr + sub * kRows * 128 + within),
                                                     umma_desc_sw128(k_addr + sub * kTile * 128 + within), idesc_s,
                                                     kk > 0 ? 1u : 0u);
                    }
                    umma_commit(&s_full[i & 1]);
                }
                __syncwarp();
                return true;
            };
            ok = issue_s(0) && (n < 2 || issue_s(1));
            int o_seg = 0, o_end = min(s_info[0].w - s_info[0].z, n);
            for (int i = 0; i < n && ok; ++i) {
                if (i == o_end) {
                    o_seg = i;
                    o_end = i + min(s_info[i].w - s_info[i].z, n - i);
                }
                ok = mbar_wait_ab(&p_full[i & 1], static_cast<uint32_t>((i >> 1) & 1), nullptr, 0u, abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t p_tmem = tmem + static_cast<uint32_t>((i & 1) * kTile);
                const uint32_t v_addr = cv_base + (i % L::kCv) * 2 * L::kCvTile + L::kCvTile;
                const uint32_t more = i - o_seg > 1 ? 1u : 0u;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        umma_bf16_a_tmem(t_o + static_cast<uint32_t>((i & 1) * HD), p_tmem + static_cast<uint32_t>(kk * 8),
                                         umma_desc_sw128_mn(v_addr + kk * 16 * 128, kTile * 128), idesc_o,
                                         kk > 0 ? 1u : more);
                    umma_commit(&o_done[i & 1]);
                    umma_commit(&cv_empty[i % L::kCv]);
                }
                __syncwarp();
                if (i + 2 < n) {
                    ok = issue_s(i + 2);
                    ok = __all_sync(0xffffffffu, ok);
                }
            }
        }
        __syncwarp();
    } else if (warp >= kWarpConv) {
        const int ct = tid - kWarpConv * 32;
        const int row = ct >> 1, half = ct & 1;    // entry of the tile, half of its dimensions
        int seg = 0, end = 0, no = -1, S = 0, last = 0;
        for (int i = 0; i < n; ++i) {
            const int c = i % L::kCv, st = i % L::kRaw;
            const bool fresh = i == end;      // a segment begins: its query rows, all loads in flight at once
            uint4 q[HD / 8];
            if (fresh) {
                const int4 info = s_info[i];
                seg = i;
                end = i + min(info.w - info.z, n - i);
                ++no;
                const int b = info.x;
                S = p.seq_lens[b];
                const int rows = p.rows != nullptr ? p.rows[b] : p.K;
                last = S + rows - 1;
                const int j = ct / G;
                const __nv_bfloat16* src = p.q + (static_cast<long long>(b) * p.K + j) * p.ld_q +
                                           static_cast<long long>(info.y * G + ct - j * G) * HD;
#pragma unroll
                for (int x = 0; x < HD / 8; ++x) {
                    q[x] = make_uint4(0u, 0u, 0u, 0u);
                    if (ct < rows * G) q[x] = *reinterpret_cast<const uint4*>(src + x * 8);
                }
            }
            if (i >= L::kCv) ok = mbar_wait_ab(&cv_empty[c], static_cast<uint32_t>((i / L::kCv) & 1) ^ 1u, nullptr, 0u, abort);
            // The query tile was last read by the segment two back, which
            // ended at unit i - 2 at the latest: wait for that unit's products.
            if (ok && fresh && i >= 2) ok = mbar_wait_ab(&o_done[i & 1], static_cast<uint32_t>(((i - 2) >> 1) & 1), nullptr, 0u, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (fresh) {
                uint8_t* dst = sm + L::kQ + (no & 1) * L::kQTile + ct * 128;
                uint32_t top = 0;
#pragma unroll
                for (int x = 0; x < HD / 8; ++x) {
                    const uint32_t w[4] = {q[x].x, q[x].y, q[x].z, q[x].w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) top = max(top, max((w[y] << 16) & 0x7FFF0000u, w[y] & 0x7FFF0000u));
                }
                // the row times 2^(127 - E): its largest value lies in [1, 2)
                const int E = min(max(static_cast<int>(top >> 23), 1), 253);
                const float down = __uint_as_float(static_cast<uint32_t>(254 - E) << 23);
#pragma unroll
                for (int x = 0; x < HD / 8; ++x) {
                    const uint32_t w[4] = {q[x].x, q[x].y, q[x].z, q[x].w};
                    uint32_t o[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        o[y] = pack_f16(__uint_as_float(w[y] << 16) * down, __uint_as_float(w[y] & 0xFFFF0000u) * down);
                    *reinterpret_cast<uint4*>(dst + (x >> 3) * kRows * 128 + (((x & 7) ^ (ct & 7)) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
                s_cs[(no & 1) * kRows + ct] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(E) << 23);
            }
            ok = mbar_wait_ab(&raw_full[st], static_cast<uint32_t>((i / L::kRaw) & 1), nullptr, 0u, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int e0 = (s_info[seg].z + i - seg) * kTile;
            const int e = e0 + row;
            const bool inner = e0 + kTile - 1 <= S;
            int nan = 0;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint8_t* src = sm + L::kRing + (st * 2 + kv) * L::kRawTile + row * HD;
                uint8_t* dst = sm + L::kConv + (c * 2 + kv) * L::kCvTile + row * 128;
#pragma unroll
                for (int x = 0; x < HD / 32; ++x) {
                    const int ch = half * (HD / 32) + x;
                    const int at = HD == 128 ? ch ^ (row & 7) : ch ^ ((row >> 1) & 3);
                    const uint4 v = *reinterpret_cast<const uint4*>(src + (at << 4));
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    if (kv == 1 && !inner) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) w[y] = e > last ? 0u : without_nan(w[y], nan);
                    }
                    uint8_t* d = dst + (ch >> 2) * kTile * 128;
                    const int j0 = 2 * (ch & 3);
                    *reinterpret_cast<uint4*>(d + ((j0 ^ (row & 7)) << 4)) =
                        make_uint4(widen_lo(w[0]), widen_hi(w[0]), widen_lo(w[1]), widen_hi(w[1]));
                    *reinterpret_cast<uint4*>(d + (((j0 + 1) ^ (row & 7)) << 4)) =
                        make_uint4(widen_lo(w[2]), widen_hi(w[2]), widen_lo(w[3]), widen_hi(w[3]));
                }
            }
            if (!inner) {
                nan |= __shfl_xor_sync(0xffffffffu, nan, 1);
                if (half == 0) s_nan[c * kTile + row] = static_cast<uint8_t>(nan);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&cv_full[c]);
                mbar_arrive(&raw_empty[st]);
            }
        }
    } else {
        // ------------------------------------------------ softmax: thread = query row
        const int grp = warp >> 2, row = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lane_off + static_cast<uint32_t>(grp * kTile);
        const uint32_t t_mine = t_o + lane_off + static_cast<uint32_t>(grp * HD);
        int no = 0;
        for (int seg = 0; seg < n; ++no) {
            const int4 info = s_info[seg];
            const int b = info.x, head = info.y;
            const int len = min(info.w - info.z, n - seg);
            const int S = p.seq_lens[b];
            const int rows = p.rows != nullptr ? p.rows[b] : p.K;
            const int R = rows * G;
            const bool busy = (warp & 3) * 32 < R;      // some row of this warp is live
            const int j = row / G, lim = S + j;
            const int first = seg + ((seg ^ grp) & 1);  // this group's first tile of the segment
            const int count = first < seg + len ? (seg + len - first + 1) / 2 : 0;
            float m = -INFINITY, l = 0.f, vref = 0.f, vinv = 0.f, mark = 0.f, cs = 0.f;
            for (int i = first; i < seg + len; i += 2) {
                if (ok) ok = mbar_wait_ab(&s_full[grp], static_cast<uint32_t>((i >> 1) & 1), nullptr, 0u, abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) continue;
                tc_fence_after_sync();
                if (busy) {
                    if (i == first) cs = s_cs[(no & 1) * kRows + row];
                    float s[kTile];
                    tmem_ld64(t_s, s);
                    const float4 ks = *reinterpret_cast<const float4*>(s_ks + i * kUmmaPages);
                    const float4 vs = *reinterpret_cast<const float4*>(s_vs + i * kUmmaPages);
                    const int4 tl = *reinterpret_cast<const int4*>(s_tile + i * kUmmaPages);
                    if (tl.x == -1 || tl.y == -1 || tl.z == -1 || tl.w == -1) mark = kMarkBadPage;
                    const float kf[4] = {cs * ks.x, cs * ks.y, cs * ks.z, cs * ks.w};
#pragma unroll
                    for (int x = 0; x < kTile; ++x) s[x] *= kf[x >> 4];
                    const int e0 = (info.z + i - seg) * kTile;
                    if (e0 + kTile - 1 > S) {
                        // Some row does not see all of it. A NaN in a V that
                        // only some rows see enters through the score (the
                        // converters cleared it).
                        const uint8_t* nan = s_nan + (i % L::kCv) * kTile;
#pragma unroll
                        for (int x = 0; x < kTile; ++x) {
                            if (nan[x]) s[x] = NAN;
                            if (e0 + x > lim) s[x] = -INFINITY;
                        }
                    }
                    float top = s[0];
#pragma unroll
                    for (int x = 1; x < kTile; ++x) top = fmaxf(top, s[x]);
                    float f = 1.f;
                    if (top > m + kRescale) {
                        f = m == -INFINITY ? 0.f : ex2(m - top);
                        l *= f;
                        m = top;
                    }
                    const float av = fmaxf(fmaxf(fabsf(vs.x), fabsf(vs.y)), fmaxf(fabsf(vs.z), fabsf(vs.w)));
                    if (av > 16.f * vref) {
                        f *= vref / av;
                        vref = av;
                        vinv = 1.f / av;
                    }
                    if (i > first && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
                        for (int c = 0; c < HD / 16; ++c) {
                            float o[16];
                            tmem_ld16(t_mine + static_cast<uint32_t>(c * 16), o);
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[x] *= f;
                            tmem_st16(t_mine + static_cast<uint32_t>(c * 16), o);
                        }
                    }
                    const float mm = m == -INFINITY ? 0.f : m;
                    const float vr[4] = {vs.x * vinv, vs.y * vinv, vs.z * vinv, vs.w * vinv};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float pk[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const float w0 = ex2(s[h * 32 + 2 * x] - mm), w1 = ex2(s[h * 32 + 2 * x + 1] - mm);
                            l += w0 + w1;
                            const float r = vr[h * 2 + (x >> 3)];
                            pk[x] = __uint_as_float(pack_f16(w0 * r, w1 * r));
                        }
                        tmem_st16(t_s + static_cast<uint32_t>(h * 16), pk);
                    }
                }
                tc_fence_before_sync();
                mbar_arrive(&p_full[grp]);
            }
            if (ok && count > 0)
                ok = mbar_wait_ab(&o_done[grp], static_cast<uint32_t>(((first + 2 * (count - 1)) >> 1) & 1), nullptr, 0u, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) mark = kMarkTimeout;
            tc_fence_after_sync();
            // the two groups' sums of each row; each group writes half of the dimensions
            s_ex[grp * kRows + row] = make_float4(m, mark != 0.f ? mark : l, vref, 0.f);
            named_bar_sync(1, kSoft);
            const float4 xa = s_ex[row], xb = s_ex[kRows + row];
            const float bad = fminf(fminf(xa.y, xb.y), 0.f);   // a NaN sum is not less than 0
            const float M = fmaxf(xa.x, xb.x);
            const float fa = xa.y <= 0.f ? 0.f : ex2(xa.x - M), fb = xb.y <= 0.f ? 0.f : ex2(xb.x - M);
            const float sum = (xa.y <= 0.f ? 0.f : xa.y * fa) + (xb.y <= 0.f ? 0.f : xb.y * fb);
            const bool whole = len == info.w;
            const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
            const float ga = fa * xa.z * inv, gb = fb * xb.z * inv;
            __nv_bfloat16* out = p.out + (static_cast<long long>(b) * p.K + j) * p.ld_out +
                                 static_cast<long long>(head * G + row - j * G) * HD + grp * (HD / 2);
            float* part = p.part + static_cast<size_t>(2 * blockIdx.x + (seg == 0 ? 0 : 1)) * part_floats(kRows, HD);
            const bool all_ok = __all_sync(0xffffffffu, !(bad < 0.f));
            // which groups had a tile: the same for the whole segment
            const bool has_a = (seg & 1) == 0 || len > 1, has_b = (seg & 1) == 1 || len > 1;
            if (busy) {
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    float v[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) v[x] = 0.f;
                    const uint32_t col = t_o + lane_off + static_cast<uint32_t>(grp * (HD / 2) + c * 16);
                    if (has_a && all_ok) {
                        float o[16];
                        tmem_ld16(col, o);
                        if (xa.y > 0.f || xa.y != xa.y)
#pragma unroll
                            for (int x = 0; x < 16; ++x) v[x] = o[x] * ga;
                    }
                    if (has_b && all_ok) {
                        float o[16];
                        tmem_ld16(col + HD, o);
                        if (xb.y > 0.f || xb.y != xb.y)
#pragma unroll
                            for (int x = 0; x < 16; ++x) v[x] = fmaf(o[x], gb, v[x]);
                    }
                    if (row < R) {
                        if (whole) {
                            uint32_t w[8];
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * x], v[2 * x + 1]);
                                w[x] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                            *reinterpret_cast<uint4*>(out + c * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                            *reinterpret_cast<uint4*>(out + c * 16 + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                        } else {
#pragma unroll
                            for (int x = 0; x < 16; x += 4)
                                *reinterpret_cast<float4*>(part + row * HD + grp * (HD / 2) + c * 16 + x) =
                                    make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
                        }
                    }
                }
                if (!whole && grp == 0 && row < R) {
                    part[kRows * HD + row] = M;
                    part[kRows * HD + kRows + row] = bad < 0.f ? bad : sum;
                }
            }
            if (whole && head == 0 && tid == 0) p.status[b] = status_of(bad);
            tc_fence_before_sync();
            named_bar_sync(1, kSoft);     // both have read both accumulators and the sums
            tc_fence_after_sync();
            seg += len;
        }
        zero_idle_rows_by<kUmmaPages, kRows>(p, HD, warp, kSoft / 32);
    }
    if (!ok) {
        s_abort = 1;              // the other roles' waits end too
        __nanosleep(100000);      // copies still in flight land
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

template <int HD>
int launch_hd(const CUtensorMap& tk, const CUtensorMap& tv, const Kv8Params& p, const Plan& a, cudaStream_t s) {
    auto kern = k_attn_kv8_umma<HD>;
    PE_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<HD>::kBytes));
    PE_CUDA_TRY(launch_ex(kern, dim3(a.grid), dim3(kThreads), Layout<HD>::kBytes, s, false, tk, tv, p));
    return PE_OK;
}

}  // namespace

namespace kv8 {
int launch_umma(const CUtensorMap& tk, const CUtensorMap& tv, const Kv8Params& p, const Plan& a, int hd,
                cudaStream_t s) {
    return hd == 128 ? launch_hd<128>(tk, tv, p, a, s) : launch_hd<64>(tk, tv, p, a, s);
}
}  // namespace kv8
}  // namespace pe
