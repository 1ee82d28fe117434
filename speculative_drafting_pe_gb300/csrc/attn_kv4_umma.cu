// Attention over the 4-bit KV cache for many query rows (a draft pass: K rows
// of every head of a group): the tensor-memory kernel behind pe_attention_kv4.
//
// A unit is 64 entries (4 pages) of one (request, kv head); all its query rows
// (at most 128, the MMA's M) share every entry, so the cache is read once.
// Roles (448 threads):
//   warps 8-11  converters, kTeam warps to a unit. Each thread fetches 16-byte
//               chunks of codes, kDepth units ahead, by asynchronous copies to
//               a place of its own, and turns them into fp16 tiles of K and of
//               V (128-byte swizzle, entry-major: K a K-major operand, V an
//               MN-major one). A value is scale (n - 8) + mid, under a power of
//               two of its page that puts the page's largest one below 2^15:
//               n - 8 and the scale are exact, mid and the sum are rounded to
//               fp16 (2^-11 each). V of entries that no row sees is zero. At
//               the start of a segment the query rows, as fp16 after an exact
//               shift by a power of two per row, to tensor memory.
//   warp 12     one elected lane issues S_t = Q K_t^T (M=128, N=64, A = Q from
//               tensor memory: from shared memory its reads alone would take the
//               product's whole time)
//   warp 13     one elected lane issues O += P_t V_t (A = P_t from tensor
//               memory)
//   warps 0-3, 4-7  two softmax groups, thread = query row = TMEM lane: group
//               x takes the units t = x (mod 2), with a running maximum, sum
//               and output accumulator of its own; they meet at the end of a
//               segment.
// kTurns S_t buffers: P_t (fp16 pairs) overwrites the columns of S_t. Tiles of K
// and V and S_t have as many places; "S_t is complete" frees K_t's, "P_t V_t is
// complete" V_t's and S_t's: one commit for each product.
//
// `widen` leaves the dimensions of a word of eight in the order 0 4 1 5 2 6 3 7.
// The queries follow it, and the output's columns are put back where they are
// written.
#include "attn_kv4.cuh"
#include "attn_umma_line.cuh"

namespace pe {
namespace {

using namespace kv4;

constexpr int kThreads = 448;
constexpr int kUnitPages = 4;
constexpr int kTile = kUnitPages * kPage;   // entries of a unit
constexpr int kRows = 128;
constexpr int kUnits = 640;                 // units of a window
constexpr int kLeast = 3, kPad = 7;         // a share's positions at least, a segment's end in units
constexpr int kSoft = 256;                  // softmax threads
constexpr int kWarpConv = 8, kWarpS = 12, kWarpPv = 13;
constexpr int kScales = 16;                 // units whose page factors are kept: written kTurns ahead, read a few behind
constexpr int kScaleRec = 2 * kUnitPages;   // floats of a unit's
constexpr int kCsTurns = 8;                 // segments whose row factors are kept: the converters run fewer ahead

template <int HD>
struct Layout {
    static constexpr int kTeam = HD == 64 ? 1 : 4;           // converter warps to a unit
    static constexpr int kTurns = HD == 64 ? 5 : 3;          // places of K and V tiles and scores
    static constexpr int kQBufs = HD == 64 ? 2 : 1;          // places of the queries
    static constexpr int kDepth = HD == 64 ? 12 : 6;         // units whose codes are in flight
    static constexpr int kTileBytes = kTile * HD * 2;        // an fp16 tile
    static constexpr int kPageCodes = kPage * HD / 2;        // codes of K or V of a page
    static constexpr int kPagePar = kPage * 4;
    static constexpr int kPageBytes = 2 * (kPageCodes + kPagePar);   // codes of K, of V, parameters of K, of V
    static constexpr int kUnitBytes = kUnitPages * kPageBytes;
    static constexpr int kK = 0;
    static constexpr int kV = kK + kTurns * kTileBytes;
    static constexpr int kRing = kV + kTurns * kTileBytes;
    static constexpr int kInfo = kRing + kDepth * kUnitBytes;
    static constexpr int kUnit = kInfo + kUnits * 16;
    static constexpr int kCs = kUnit + kUnits * kUnitPages * 4;      // [kCsTurns][kRows]
    static constexpr int kEx = kCs + kCsTurns * kRows * 4;   // [2][kRows] float4
    static constexpr int kScale = kEx + 2 * kRows * 16;      // [kScales][factors of 4 pages' K, exponents of their V]
    static constexpr int kNan = kScale + kScales * kScaleRec * 4;    // [kTurns][kTile] bytes
    static constexpr int kBar = kNan + kTurns * kTile;
    static constexpr int kBars = 5 * kTurns + 2 * kQBufs;
    static constexpr int kTmem = kBar + kBars * 8;
    static constexpr int kBytes = kTmem + 16 + 1024;
    // tensor memory: S_t in columns 64 (t mod kTurns) .., group x's output x * HD behind them, then the queries
    static constexpr int kColO = kTurns * kTile, kColQ = kColO + 2 * HD;
    static_assert(kColQ + kQBufs * HD / 2 <= 512, "tensor memory");
    static_assert(kBytes <= 232448 - 2048, "shared memory of a block");
};
// the barriers of a window: k_full, v_full, s_full, p_full, pv_done [kTurns], q_full, q_empty [kQBufs]
template <int HD>
__device__ __forceinline__ void init_bars(uint64_t* bars, int stall) {
    using L = Layout<HD>;
    constexpr int kTurns = L::kTurns;
    for (int s = 0; s < kTurns; ++s) {
        mbar_init(&bars[s], L::kTeam + (stall == kStallK));
        mbar_init(&bars[kTurns + s], L::kTeam + (stall == kStallV));
        mbar_init(&bars[2 * kTurns + s], 1);
        mbar_init(&bars[3 * kTurns + s], 4 + (stall == kStallP));
        mbar_init(&bars[4 * kTurns + s], 1);
    }
    for (int s = 0; s < L::kQBufs; ++s) {
        mbar_init(&bars[5 * kTurns + s], 4);
        mbar_init(&bars[5 * kTurns + L::kQBufs + s], 1);
    }
    fence_mbar_init();
}

// What the CTA has set going in this window, units of each kind.
struct Issued {
    int s, pv;   // score products, P.V products
};

// Four words of codes of an entry as fp16, at the places of its chunk in a tile:
// chunk positions j0 .. j0 + 3 of row r. far: of a block's second 64 bytes' twin
// in the other block, written in another order so that no bank is met twice.
__device__ __forceinline__ void widen_chunk(const uint4& codes, uint32_t scale, uint32_t mid, uint8_t* row, int r, int j0, bool far) {
    const __half2 s2 = *reinterpret_cast<const __half2*>(&scale), c2 = *reinterpret_cast<const __half2*>(&mid);
    const uint32_t w[4] = {far ? codes.z : codes.x, far ? codes.w : codes.y, far ? codes.x : codes.z, far ? codes.y : codes.w};
    const int turn = (far ? 2 : 0) ^ j0 ^ (r & 7);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        uint32_t n[4], v[4];
        widen(w[x], n);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&n[y]), s2, c2);
            v[y] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(row + ((x ^ turn) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// The n units of a window by every role; FIRST: of the share's first one. false
// in the threads of a role that gave up waiting.
template <int HD, bool FIRST>
__device__ __forceinline__ bool attend_window(const Kv4Params& p, uint8_t* sm, int n, const Window* win, bool idle,
                                              const volatile int* abort, Issued* issued) {
    using L = Layout<HD>;
    constexpr int kTurns = L::kTurns, kQBufs = L::kQBufs;
    int4* s_info = reinterpret_cast<int4*>(sm + L::kInfo);
    int* s_tile = reinterpret_cast<int*>(sm + L::kUnit);
    float* s_cs = reinterpret_cast<float*>(sm + L::kCs);
    float4* s_ex = reinterpret_cast<float4*>(sm + L::kEx);
    float* s_scale = reinterpret_cast<float*>(sm + L::kScale);
    uint8_t* s_nan = sm + L::kNan;
    uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t* cv_full = k_full + kTurns;
    uint64_t* s_full = cv_full + kTurns;
    uint64_t* p_full = s_full + kTurns;
    uint64_t* pv_done = p_full + kTurns;
    uint64_t* q_full = pv_done + kTurns;
    uint64_t* q_empty = q_full + kQBufs;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.nq / p.nkv;

    const uint32_t tmem = *reinterpret_cast<const uint32_t*>(sm + L::kTmem);
    const uint32_t t_o = tmem + L::kColO, t_q = tmem + L::kColQ;
    bool ok = true;
    auto turn = [](int i) { return static_cast<uint32_t>((i / kTurns) & 1); };   // parity of unit i's use of its place
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_ab(bar, parity, nullptr, 0u, abort); };

    if (warp == kWarpS || warp == kWarpPv) {
        // The whole warp walks the units and one elected lane issues: in
        // warp-uniform control flow the descriptors stay in uniform registers.
        const bool scores = warp != kWarpPv;
        const uint32_t idesc_s = umma_idesc(0, kRows, kTile);   // format 0: fp16
        const uint32_t idesc_o = umma_idesc(0, kRows, HD) | kIdescBMnMajor;
        const uint32_t k_base = smem_u32(sm + L::kK), v_base = smem_u32(sm + L::kV);
        int seg = 0, end = 0, no = -1, i = 0;
        for (; i < n; ++i) {
            const int x = i % kTurns;
            if (i == end) {
                seg = i;
                end = i + min(s_info[i].w - s_info[i].z, n - i);
                ++no;
                if (scores) ok = wait(&q_full[no % kQBufs], static_cast<uint32_t>((no / kQBufs) & 1));
            }
            if (scores) ok = ok && wait(&k_full[x], turn(i)) && (i < kTurns || wait(&pv_done[x], turn(i) ^ 1u));
            else ok = ok && wait(&cv_full[x], turn(i)) && wait(&p_full[x], turn(i));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t t_s = tmem + static_cast<uint32_t>(x * kTile);
            if (scores) {
                const uint32_t q_addr = t_q + static_cast<uint32_t>(no % kQBufs * (HD / 2)), k_addr = k_base + x * L::kTileBytes;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk)
                        umma_bf16_a_tmem(t_s, q_addr + static_cast<uint32_t>(kk * 8),
                                         umma_desc_sw128(k_addr + (kk >> 2) * kTile * 128 + (kk & 3) * 32), idesc_s, kk > 0 ? 1u : 0u);
                    umma_commit(&s_full[x]);
                    if (i + 1 == end) umma_commit(&q_empty[no % kQBufs]);
                }
            } else {
                const uint32_t v_addr = v_base + x * L::kTileBytes;
                const uint32_t more = i - seg > 1 ? 1u : 0u;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        umma_bf16_a_tmem(t_o + static_cast<uint32_t>((i & 1) * HD), t_s + static_cast<uint32_t>(kk * 8),
                                         umma_desc_sw128_mn(v_addr + kk * 16 * 128, kTile * 128), idesc_o,
                                         kk > 0 ? 1u : more);
                    umma_commit(&pv_done[x]);
                }
            }
            __syncwarp();
        }
        if (lane == 0) (scores ? issued->s : issued->pv) = i;
        if (!FIRST && ok && win->more) {   // what this warp committed has arrived: the next window takes the barriers anew
            for (int i = max(0, n - kTurns); i < n; ++i) ok = ok && wait(scores ? &s_full[i % kTurns] : &pv_done[i % kTurns], turn(i));
            for (int x = max(0, no + 1 - kQBufs); scores && x <= no; ++x)
                ok = ok && wait(&q_empty[x % kQBufs], static_cast<uint32_t>((x / kQBufs) & 1));
            ok = __all_sync(0xffffffffu, ok);
        }
        __syncwarp();
    } else if (warp >= kWarpConv && warp < kWarpS) {
        constexpr int kTeam = L::kTeam, kTeams = 4 / kTeam, kAhead = L::kDepth / kTeams, kMine = kUnitPages / kTeam;
        static_assert(L::kDepth % kTeams == 0, "a warp's units");
        const int ct = tid & 127, team = (warp - kWarpConv) / kTeam, part = (warp - kWarpConv) % kTeam;
        constexpr int kChunks = HD / 32, kPasses = kPage * kChunks / 32, kPass = 32 / kChunks;   // chunks of an entry; passes over a page
        const int ch = lane % kChunks, row0 = lane / kChunks;
        const uint64_t policy = l2_policy_evict_first();
        const uint32_t ring_at = smem_u32(sm + L::kRing);
        // page q of this warp's of unit i: codes of K and V by all lanes, parameters of K by lanes 0-3, of V by 4-7
        auto fetch = [&](int i) {
            if (i < n) {
#pragma unroll
                for (int q = 0; q < kMine; ++q) {
                    const int page = part * kMine + q, tile = s_tile[i * kUnitPages + page];
                    if (tile < 0) continue;
                    const uint32_t at = ring_at + (i % L::kDepth) * L::kUnitBytes + page * L::kPageBytes;
#pragma unroll
                    for (int side = 0; side < 2; ++side) {
                        const uint8_t* from = (side == 0 ? p.k_codes : p.v_codes) + static_cast<long long>(tile) * L::kPageCodes + lane * 16;
#pragma unroll
                        for (int x = 0; x < kPasses; ++x)
                            copy_async<16>(at + side * L::kPageCodes + x * 512 + lane * 16, from + x * 512, policy);
                    }
                    if (lane < 8)
                        copy_async<16>(at + 2 * L::kPageCodes + lane * 16,
                                       (lane < 4 ? p.k_params : p.v_params) + static_cast<long long>(tile) * kPage + (lane & 3) * 4, policy);
                }
            }
            copies_commit();
        };
#pragma unroll
        for (int x = 0; x < kAhead; ++x) fetch(team + x * kTeams);
        int seg = 0, end = 0, no = -1, S = 0, last = 0;
        // the query rows of the segments up to the one of unit `upto`: every
        // warp has 32 of them
        auto queries = [&](int upto) {
            while (ok && end <= upto) {
                const int4 info = s_info[end];
                seg = end;
                end = seg + min(info.w - info.z, n - seg);
                ++no;
                const int b = info.x;
                S = p.seq_lens[b];
                const int rows = p.rows != nullptr ? p.rows[b] : p.K;
                last = S + rows - 1;
                const int j = ct / G;
                const __nv_bfloat16* src = p.q + (static_cast<long long>(b) * p.K + j) * p.ld_q +
                                           static_cast<long long>(info.y * G + ct - j * G) * HD;
                // twice over the row: its largest value, then fp16
                const bool live = ct < rows * G;
                auto load = [&](int x) {
                    return live ? *reinterpret_cast<const uint4*>(src + x * 8) : make_uint4(0u, 0u, 0u, 0u);
                };
                if (live) {
#pragma unroll
                    for (int x = 0; x < HD / 64; ++x) asm volatile("prefetch.global.L1 [%0];" ::"l"(src + x * 64));
                }
                uint32_t top = 0;
#pragma unroll
                for (int x = 0; x < HD / 8; ++x) {
                    const uint4 q = load(x);
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) top = max(top, max((w[y] << 16) & 0x7FFF0000u, w[y] & 0x7FFF0000u));
                }
                // the place's last reader: S of the segment kQBufs back
                if (no >= kQBufs) ok = wait(&q_empty[no % kQBufs], static_cast<uint32_t>((no / kQBufs) & 1) ^ 1u);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after_sync();
                // the row times 2^(127 - E): its largest value lies in [1, 2)
                const int E = min(max(static_cast<int>(top >> 23), 1), 253);
                const float down = __uint_as_float(static_cast<uint32_t>(254 - E) << 23);
                const uint32_t to = t_q + static_cast<uint32_t>(no % kQBufs * (HD / 2)) + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll 1
                for (int half = 0; half < HD / 64; ++half) {
                    uint32_t v[32];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const uint4 q = load(half * 8 + x);
                        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
                        float f[8];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            f[2 * y] = __uint_as_float(w[y] << 16) * down;
                            f[2 * y + 1] = __uint_as_float(w[y] & 0xFFFF0000u) * down;
                        }
#pragma unroll
                        for (int y = 0; y < 4; ++y) v[x * 4 + y] = pack_f16(f[y], f[y + 4]);
                    }
                    __syncwarp();
                    tmem_st32(to + static_cast<uint32_t>(half * 32), v);
                }
                // a row that holds an infinity (or a NaN) is NaN
                s_cs[(no & (kCsTurns - 1)) * kRows + ct] =
                    top >= 0x7F800000u ? NAN : p.scale_log2 * __uint_as_float(static_cast<uint32_t>(E) << 23);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[no % kQBufs]);
            }
        };
        for (int i = team; i < n; i += kTeams) {
            const int c = i % kTurns;
            queries(i);
            copies_wait<kAhead - 1>();
            __syncwarp();   // the parameters come by eight lanes
            const uint8_t* unit = sm + L::kRing + (i % L::kDepth) * L::kUnitBytes;
            const int e0 = (s_info[seg].z + i - seg) * kTile;
            const bool inner = e0 + kTile - 1 <= S;
            // Powers of two that put the pages' K and V below 2^15: of the
            // exponents of base and 15 scale, of entries that some row sees.
            float up[kMine][2];
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                const int page = part * kMine + q;
                const uint32_t par = reinterpret_cast<const uint32_t*>(unit + page * L::kPageBytes + 2 * L::kPageCodes)[lane];
                const uint32_t eb = (par >> 23) & 0xFFu, es = (par >> 7) & 0xFFu;
                uint32_t e = e0 + page * kPage + (lane & 15) > last || eb == 255u || es == 255u ? 0u : max(eb, es + 4u);
                const uint32_t ek = __reduce_max_sync(0xffffffffu, lane < 16 ? e : 0u), ev = __reduce_max_sync(0xffffffffu, lane < 16 ? 0u : e);
                // stored = value * 2^(14 - (e - 126)), |value| < 2^(e - 125)
                const uint32_t fk = min(max(ek, 24u), 254u), fv = min(max(ev, 24u), 254u);
                up[q][0] = __uint_as_float((267u - fk) << 23);
                up[q][1] = __uint_as_float((267u - fv) << 23);
                if (lane == 0) {
                    float* rec = s_scale + (i % kScales) * kScaleRec + page;
                    rec[0] = __uint_as_float((fk - 13u) << 23);
                    rec[kUnitPages] = static_cast<float>(static_cast<int>(fv) - 140);
                }
            }
            auto widen_page = [&](int q, int side, uint8_t* tile_at, bool keep_all) {
                const int page = part * kMine + q;
                const uint8_t* codes = unit + page * L::kPageBytes + side * L::kPageCodes;
                const uint32_t* par = reinterpret_cast<const uint32_t*>(unit + page * L::kPageBytes + 2 * L::kPageCodes) + side * kPage;
#pragma unroll
                for (int x = 0; x < kPasses; ++x) {
                    const uint4 w = *reinterpret_cast<const uint4*>(codes + x * 512 + lane * 16);
                    const int r = row0 + x * kPass, e = page * kPage + r;
                    const uint32_t pr = par[r];
                    float s = scale_of(pr) * up[q][side], m = mid_of(pr) * up[q][side];
                    if (!keep_all) {
                        // no one's, or not finite: it enters through the score
                        const bool odd = m != m, out = e0 + e > last;
                        if (odd || out) s = m = 0.f;
                        if (ch == 0) s_nan[c * kTile + e] = static_cast<uint8_t>(odd && !out);
                    }
                    const uint32_t s2 = pack_f16(s, s), c2 = pack_f16(m, m);
                    widen_chunk(w, s2, c2, tile_at + (ch >> 1) * kTile * 128 + e * 128, e, (ch & 1) * 4, (ch >> 1) != 0);
                }
            };
            if (i >= kTurns) ok = ok && wait(&s_full[c], turn(i) ^ 1u);   // S of the unit before it in this place
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
#pragma unroll
            for (int q = 0; q < kMine; ++q) widen_page(q, 0, sm + L::kK + c * L::kTileBytes, true);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_full[c]);
            if (i >= kTurns) ok = ok && wait(&pv_done[c], turn(i) ^ 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
#pragma unroll
            for (int q = 0; q < kMine; ++q) widen_page(q, 1, sm + L::kV + c * L::kTileBytes, inner);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&cv_full[c]);
            fetch(i + L::kDepth);   // (all lanes have read the unit's)
        }
        queries(n - 1);
        copies_wait<0>();
    } else if (warp < kWarpConv) {
        // ------------------------------------------------ softmax: thread = query row
        const int grp = warp >> 2, row = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_mine = t_o + lane_off + static_cast<uint32_t>(grp * HD);
        const bool flip = p.scale_log2 < 0.f;
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
            const int first = seg + ((seg ^ grp) & 1);  // this group's first unit of the segment
            const int count = first < seg + len ? (seg + len - first + 1) / 2 : 0;
            float m = -INFINITY, md = -INFINITY, l = 0.f, mark = 0.f, cs = 0.f;
            for (int i = first; i < seg + len; i += 2) {
                const uint32_t t_s = tmem + lane_off + static_cast<uint32_t>((i % kTurns) * kTile);
                if (ok) ok = wait(&s_full[i % kTurns], turn(i));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) continue;
                tc_fence_after_sync();
                if (busy) {
                    if (i == first) cs = s_cs[(no & (kCsTurns - 1)) * kRows + row];
                    const float4* sc = reinterpret_cast<const float4*>(s_scale + (i % kScales) * kScaleRec);
                    const float4 ks = sc[0], vlg = sc[1];   // factors of the pages' K, exponents of their V
                    const int4 tl = *reinterpret_cast<const int4*>(s_tile + i * kUnitPages);
                    float s[kTile];
                    tmem_ld64(t_s, s);
                    if (tl.x == -1 || tl.y == -1 || tl.z == -1 || tl.w == -1) mark = kMarkBadPage;
                    float kf[4] = {cs * ks.x, cs * ks.y, cs * ks.z, cs * ks.w};
                    const int e0 = (info.z + i - seg) * kTile;
                    const bool inner = e0 + kTile - 1 <= S;
                    if (!inner || flip) {
                        // the page factors first: a masked score must not meet
                        // a factor of 0, nor a maximum a negative one
#pragma unroll
                        for (int x = 0; x < kTile; ++x) s[x] *= kf[x >> 4];
                        kf[0] = kf[1] = kf[2] = kf[3] = 1.f;
                        if (!inner) {
                            // Some row does not see all of it. A NaN in a V
                            // that only some rows see enters through the score
                            // (the converters cleared it, before V.P needs it).
                            ok = wait(&cv_full[i % kTurns], turn(i));
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) continue;
                            const uint4* nan = reinterpret_cast<const uint4*>(s_nan + (i % kTurns) * kTile);
#pragma unroll 1
                            for (int q = 0; q < kTile / 16; ++q) {
                                const uint4 f = nan[q];
                                if ((f.x | f.y | f.z | f.w) == 0u) continue;   // as good as always
#pragma unroll
                                for (int x = 0; x < kTile; ++x) {
                                    const uint32_t w = (x & 12) == 0 ? f.x : (x & 12) == 4 ? f.y : (x & 12) == 8 ? f.z : f.w;
                                    if ((x >> 4) == q && ((w >> (8 * (x & 3))) & 0xFFu)) s[x] = NAN;
                                }
                            }
#pragma unroll
                            for (int x = 0; x < kTile; ++x)
                                if (e0 + x > lim) s[x] = -INFINITY;
                        }
                    }
                    const float vl[4] = {vlg.x, vlg.y, vlg.z, vlg.w};
                    float t[4], top = -INFINITY;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float* sq = s + q * 16;
                        float t4[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) t4[x] = fmaxf(fmaxf(sq[x], sq[x + 4]), fmaxf(sq[x + 8], sq[x + 12]));
                        t[q] = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * kf[q];
                        top = fmaxf(top, t[q]);
                    }
                    if (top > m + kRescale) {
                        l *= m == -INFINITY ? 0.f : ex2(m - top);
                        md += m - top;
                        m = top;
                    }
                    // 0 in the place of the maximum where a row has seen no entry
                    const float mm = m == -INFINITY ? 0.f : -m;
                    const float most = fmaxf(fmaxf(t[0] + mm + vl[0], t[1] + mm + vl[1]), fmaxf(t[2] + mm + vl[2], t[3] + mm + vl[3]));
                    float f = 1.f;
                    if (most > md + kRescale) {
                        f = md == -INFINITY ? 0.f : ex2(md - most);
                        md = most;
                    }
                    if (i > first && __any_sync(0xffffffffu, f != 1.f)) {
                        // this group's last P.V has to be done
                        ok = wait(&pv_done[(i - 2) % kTurns], turn(i - 2));
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) continue;
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < HD / 16; ++c) {
                            float o[16];
                            tmem_ld16(t_mine + static_cast<uint32_t>(c * 16), o);
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[x] *= f;
                            tmem_st16(t_mine + static_cast<uint32_t>(c * 16), o);
                        }
                    }
                    const uint64_t m2 = f2(mm, mm);
                    const float from = kLift - md;
                    const float vr[4] = {lift(from, vl[0]), lift(from, vl[1]), lift(from, vl[2]), lift(from, vl[3])};
                    uint64_t sum[2] = {0ull, 0ull};
                    uint32_t pk[32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint64_t k2 = f2(kf[q], kf[q]), r2 = f2(vr[q], vr[q]);
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            const float2 a = unf2(fma2(f2(s[q * 16 + 2 * x], s[q * 16 + 2 * x + 1]), k2, m2));
                            const uint64_t w = f2(ex2(a.x), ex2(a.y));
                            sum[x & 1] = add2(sum[x & 1], w);
                            const float2 r = unf2(mul2(w, r2));
                            pk[q * 8 + x] = pack_f16(r.x, r.y);
                        }
                    }
                    const float2 sa = unf2(add2(sum[0], sum[1]));
                    l += sa.x + sa.y;
                    __syncwarp();
                    tmem_st32(t_s, pk);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[i % kTurns]);
            }
            const int final = first + 2 * (count - 1);
            if (ok && count > 0) ok = wait(&pv_done[final % kTurns], turn(final));
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after_sync();
            // the two groups' sums of each row; each group writes half of the dimensions
            // and what the head's earlier windows left
            const bool early = FIRST ? info.z > 0 : seg == 0 && win->early, carry = !FIRST && seg == 0 && win->carry && row < R;
            float* part = p.part + static_cast<size_t>(2 * blockIdx.x + (early ? 0 : 1)) * part_floats(kRows, HD);
            const float M0 = carry ? part[kRows * HD + row] : -INFINITY, sum0 = carry ? part[kRows * HD + kRows + row] : 0.f;
            s_ex[grp * kRows + row] = make_float4(m, mark != 0.f ? mark : l, md, 0.f);
            named_bar_sync(1, kSoft);
            const float4 xa = s_ex[row], xb = s_ex[kRows + row];
            const float bad = fminf(fminf(fminf(xa.y, xb.y), sum0), 0.f);   // a NaN sum is not less than 0
            const float M = fmaxf(fmaxf(xa.x, xb.x), M0), f0 = M0 == M ? 1.f : ex2(M0 - M);
            const float fa = xa.y <= 0.f ? 0.f : ex2(xa.x - M), fb = xb.y <= 0.f ? 0.f : ex2(xb.x - M);
            const float sum = (xa.y <= 0.f ? 0.f : xa.y * fa) + (xb.y <= 0.f ? 0.f : xb.y * fb) + (sum0 <= 0.f ? 0.f : sum0 * f0);
            const bool whole = !early && info.z + len == info.w;
            const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
            const float ga = xa.z == -INFINITY ? 0.f : ex2(xa.x - M + xa.z - kLift) * inv;
            const float gb = xb.z == -INFINITY ? 0.f : ex2(xb.x - M + xb.z - kLift) * inv;
            __nv_bfloat16* out = p.out + (static_cast<long long>(b) * p.K + j) * p.ld_out +
                                 static_cast<long long>(head * G + row - j * G) * HD + grp * (HD / 2);
            const bool sectors = ((reinterpret_cast<uintptr_t>(p.out) | static_cast<uintptr_t>(p.ld_out) * 2) & 31u) == 0;
            const bool all_ok = __all_sync(0xffffffffu, !(bad < 0.f));
            // which groups had a tile: the same for the whole segment
            const bool has_a = (seg & 1) == 0 || len > 1, has_b = (seg & 1) == 1 || len > 1;
            if (busy) {
#pragma unroll
                for (int c = 0; c < HD / 2; c += 32) {
                    float v[32];
#pragma unroll
                    for (int x = 0; x < 32; ++x) v[x] = 0.f;
                    // (a warp's rows part ways below: whole again before it loads)
                    const uint32_t col = t_o + lane_off + static_cast<uint32_t>(grp * (HD / 2) + c);
                    __syncwarp();
                    if (has_a && all_ok) {
                        float o[32];
                        tmem_ld32(col, o);
                        if (xa.y > 0.f || xa.y != xa.y)
#pragma unroll
                            for (int x = 0; x < 32; ++x) v[x] = o[x] * ga;
                    }
                    __syncwarp();
                    if (has_b && all_ok) {
                        float o[32];
                        tmem_ld32(col + HD, o);
                        if (xb.y > 0.f || xb.y != xb.y)
#pragma unroll
                            for (int x = 0; x < 32; ++x) v[x] = fmaf(o[x], gb, v[x]);
                    }
                    if (row >= R) continue;
                    // columns back to dimensions (`widen`)
#pragma unroll
                    for (int x = 0; x < 32; x += 8) {
                        float w[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) w[y] = v[x + y];
#pragma unroll
                        for (int y = 0; y < 4; ++y) v[x + y] = w[2 * y], v[x + 4 + y] = w[2 * y + 1];
                    }
                    if (carry && all_ok) {
                        const float4* had = reinterpret_cast<const float4*>(part + row * HD + grp * (HD / 2) + c);
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            const float4 o = had[x];
                            v[4 * x] = fmaf(o.x, f0 * inv, v[4 * x]);
                            v[4 * x + 1] = fmaf(o.y, f0 * inv, v[4 * x + 1]);
                            v[4 * x + 2] = fmaf(o.z, f0 * inv, v[4 * x + 2]);
                            v[4 * x + 3] = fmaf(o.w, f0 * inv, v[4 * x + 3]);
                        }
                    }
                    if (whole) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t h[8];
#pragma unroll
                            for (int y = 0; y < 8; ++y) {
                                const __nv_bfloat162 two = __floats2bfloat162_rn(v[16 * x + 2 * y], v[16 * x + 2 * y + 1]);
                                h[y] = *reinterpret_cast<const uint32_t*>(&two);
                            }
                            if (sectors) {
                                store_sector(out + c + 16 * x, h);
                            } else {
                                reinterpret_cast<uint4*>(out + c + 16 * x)[0] = make_uint4(h[0], h[1], h[2], h[3]);
                                reinterpret_cast<uint4*>(out + c + 16 * x)[1] = make_uint4(h[4], h[5], h[6], h[7]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            uint32_t w[8];
#pragma unroll
                            for (int y = 0; y < 8; ++y) w[y] = __float_as_uint(v[8 * x + y]);
                            store_sector(part + row * HD + grp * (HD / 2) + c + 8 * x, w);
                        }
                    }
                }
                if (!whole && grp == 0 && row < R) {
                    part[kRows * HD + row] = M;
                    part[kRows * HD + kRows + row] = bad < 0.f ? bad : sum;
                }
            }
            if (whole && head == 0 && tid == 0) p.status[b] = status_of(bad);
            __syncwarp();
            tc_fence_before_sync();
            named_bar_sync(1, kSoft);     // both have read both accumulators and the sums
            tc_fence_after_sync();
            seg += len;
        }
        if (FIRST && idle) zero_idle_rows_by<kUnitPages, kPad>(p, HD, warp, kSoft / 32);
    }
    return ok;
}

// FIRST: every share's first window. Otherwise the others.
template <int HD, bool FIRST>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_kv4_umma(const Kv4Params p) {
    using L = Layout<HD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ int s_abort;
    __shared__ Window s_win;
    __shared__ Issued s_issued;
    int4* s_info = reinterpret_cast<int4*>(sm + L::kInfo);
    int* s_tile = reinterpret_cast<int*>(sm + L::kUnit);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::kTmem);
    const int tid = threadIdx.x, warp = tid >> 5;

    pdl_launch_dependents();
    if constexpr (!FIRST) {
        pdl_wait();
        // no share has another window, or this CTA gave up in the first
        if (p.cut[gridDim.x].x <= kUnits || p.cut[blockIdx.x].z < 0) return;
    }
    if (tid == 0) {
        s_abort = 0;
        s_issued = Issued{0, 0};
        init_bars<HD>(bars, p.stall);
    }
    if (warp == kWarpS) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    bool idle, ok = true;
    if constexpr (FIRST) {
        const int n = gather_units<kThreads, kUnitPages, kPad, kUnits>(p, kLeast, 0, s_info, s_tile, &s_win, idle);
        tc_fence_after_sync();
        ok = attend_window<HD, true>(p, sm, n, &s_win, idle, &s_abort, &s_issued);
    } else {
        for (int w = 1;; ++w) {
            const int n = gather_units<kThreads, kUnitPages, kPad, kUnits>(p, kLeast, w, s_info, s_tile, &s_win, idle);
            if (w == 1) tc_fence_after_sync();
            ok = attend_window<HD, false>(p, sm, n, &s_win, false, &s_abort, &s_issued);
            if (!s_win.more) break;
            if (!ok) s_abort = 1;
            __syncthreads();       // the tables and the barriers are not in use
            if (*static_cast<volatile int*>(&s_abort)) break;
            // units, segments and phases count from 0 again
            if (tid == 0) {
                for (int x = 0; x < L::kBars; ++x) mbar_inval(&bars[x]);
                init_bars<HD>(bars, p.stall);
            }
        }
    }
    if (!ok) s_abort = 1;         // the other roles' waits end too
    tc_fence_before_sync();
    __syncthreads();
    if (s_abort) {
        if (tid == 0) p.cut[blockIdx.x].z = -1;   // the merge refuses the call's results
        if (warp == kWarpS) {
            // what is in flight lands before the shared and tensor memory go
            // (the lanes' own copies have been waited for)
            constexpr int kTurns = L::kTurns;
            auto last = [&](uint64_t* of, int i) { settle(&of[i % kTurns], static_cast<uint32_t>((i / kTurns) & 1)); };
            if (s_issued.s > 0) last(bars + 2 * kTurns, s_issued.s - 1);
            if (s_issued.pv > 0) last(bars + 4 * kTurns, s_issued.pv - 1);
            __syncwarp();
        }
    }
    if (warp == kWarpS) {
        tc_fence_after_sync();
        tmem_dealloc(*tmem_slot, 512);
    }
}

template <int HD>
int launch_hd(const Kv4Params& p, const Plan& a, cudaStream_t s) {
    constexpr auto first = k_attn_kv4_umma<HD, true>, rest = k_attn_kv4_umma<HD, false>;
    constexpr int smem = Layout<HD>::kBytes;
    int rc = allow_smem<first>(a.dev, smem);
    if (rc != PE_OK) return rc;
    PE_CUDA_TRY(launch_ex(first, dim3(a.grid), dim3(kThreads), smem, s, false, p));
    if (a.most <= static_cast<long long>(a.grid) * kUnits) return PE_OK;
    if ((rc = allow_smem<rest>(a.dev, smem)) != PE_OK) return rc;
    PE_CUDA_TRY(launch_ex(rest, dim3(a.grid), dim3(kThreads), smem, s, true, p));
    return PE_OK;
}

}  // namespace

namespace kv4 {
static std::atomic<int> next_stall;   // of pe_test_stall_attention_kv4

int plan_umma(int B, int nkv, int hd, int max_pages, Plan* out) {
    return plan_line(B, nkv, hd, max_pages, kUnitPages, kPad, kLeast, kRows, out);
}

int launch_umma(const Kv4Params& params, const Plan& a, int hd, cudaStream_t s) {
    Kv4Params p = params;
    if (next_stall.load(std::memory_order_relaxed) != 0) p.stall = next_stall.exchange(0);
    return hd == 128 ? launch_hd<128>(p, a, s) : launch_hd<64>(p, a, s);
}
}  // namespace kv4
}  // namespace pe

extern "C" int pe_test_stall_attention_kv4(int32_t barrier) {
    if (barrier < pe::line::kStallK || barrier > pe::line::kStallP) {
        pe::set_error("barrier must be 1, 2 or 3");
        return PE_ERR_ARG;
    }
    pe::kv4::next_stall.store(barrier);
    return PE_OK;
}
