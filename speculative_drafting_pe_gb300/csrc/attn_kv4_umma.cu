// Attention over the 4-bit KV cache for many query rows (a draft pass: K rows
// of every head of a group): the tensor-memory kernel behind pe_attention_kv4.
//
// A unit is 64 entries (4 pages) of one (request, kv head); all its query rows
// (at most 128, the MMA's M) share every entry, so the cache is read once.
// Roles (640 threads):
//   warps 18, 19  fetch: the codes and parameters of a unit's pages, kDepth
//               units ahead, by asynchronous copies.
//   warps 8-15  converters, kTeam warps to a unit, two (64 wide: four) units at
//               a time. They turn codes into fp16 tiles of K and of V (128-byte
//               swizzle, entry-major: K a K-major operand, V an MN-major one)
//               under a power of two of the page: K as scale n + base, rounded
//               once, V as scale (n - 8) + mid, mid and the sum rounded (2^-11
//               each); fp16's smallest step is 2^-18 of the page's largest K
//               and 2^-36 of its largest V at most. Where some row does not
//               see all of the unit, an entry has a power of two to itself, so
//               that none moves a row that does not see it. At the start of a
//               segment the query rows, as fp16 after an exact shift by a power
//               of two per row, to tensor memory.
//   warp 16     one elected lane issues S_t = Q K_t^T (M=128, N=64, A = Q from
//               tensor memory: from shared memory its reads alone would take the
//               product's whole time)
//   warp 17     one elected lane issues O += P_t V_t (A = P_t from tensor
//               memory)
//   warps 0-3, 4-7  two softmax groups, thread = query row = TMEM lane: group
//               x takes the units t = x (mod 2), with a running maximum, sum
//               and output accumulator of its own; they meet at the end of a
//               segment.
// What bounds it is the instructions' supply more than any pipe: five roles'
// loops share the instruction cache and 51% of the issue slots go. So only the
// two innermost loops are unrolled (the whole kernel unrolled: 333 us for 244 at
// B=128 K=11, 512..8192 entries, 32/4 heads of 128; those two: 210 for 219), and
// shared memory is addressed as such, not by generic pointers (222 for 248).
// Eight converter warps for four: 244 for 270. Now 215 us; 64 requests of 10
// rows, 64/8 heads of 64, 1024..4096 entries: 99 (208 and 96 before large scores
// were rounded, contributions kept relative to them, and small products kept a bit
// more: about a third of it each). At 225 and 103 it took
// without the widening 187 and 93, without the softmax 183 and 70, without both
// 149 and 67: the hand-over of a unit between the roles. Scores of a unit in one
// pass with weights from the old maximum: 229 for 219 (a third of the units has a
// new one); parameters by warps of their own: 228 for 219, or a unit ahead 221 for
// 214; 136 registers for the softmax warps by setmaxnreg and scores kept in
// them: 273 for 244; query rows staged in shared memory 221 for 220.
// kTurns S_t buffers: P_t (fp16 pairs) overwrites the columns of S_t. Tiles of K
// and V and S_t have as many places; "S_t is complete" frees K_t's, "P_t V_t is
// complete" V_t's and S_t's: one commit for each product.
//
// `widen` leaves the dimensions of a word of eight in the order 0 4 1 5 2 6 3 7.
// The queries follow it, and the output's columns are put back where they are
// written.
#include "attn_kv4.cuh"
#include <type_traits>

#include "attn_umma_line.cuh"

namespace pe {
namespace {

using namespace kv4;

constexpr int kThreads = 640;
constexpr int kUnitPages = 4;
constexpr int kTile = kUnitPages * kPage;   // entries of a unit
constexpr int kRows = 128;
constexpr int kUnits = 640;                 // units of a window
// A share's positions at least (one request of 2048 entries, 4 heads of 56 rows: 1 14.8 us, 2 14.1, 3 15.1, 5 15.6; 5
// of some 500 with 32: 15.5, 15.5, 15.1, 16.3), a segment's end in units.
constexpr int kLeast = 2, kPad = 7;
constexpr int kSoft = 256;                  // softmax threads
constexpr int kWarpConv = 8, kWarpS = 16, kWarpPv = 17, kWarpFetch = 18;   // (and 19)
constexpr int kScales = 16;                 // units whose factors are kept: written with K kTurns ahead at most, read a few behind
constexpr int kScaleRec = 2 * kUnitPages;   // floats of a unit's
// A row's largest contribution stands at 2^(kLift - kHead) in fp16 when it is
// taken as the reference, which moves once one stands kRescale above it: by 2^12
// at least. (Moves by 2^15, from 10 above with a head of 5: 212 us for 215 at B=128
// K=11, 97.5 for 99 with 64-wide heads, and small products lose a bit.)
constexpr float kHead = 4.f;
constexpr int kCsTurns = 8;                 // segments whose row factors are kept: the converters run fewer ahead

template <int HD>
struct Layout {
    static constexpr int kTeam = HD == 64 ? 2 : 4;           // converter warps to a unit
    static constexpr int kTurns = HD == 64 ? 5 : 3;          // places of K and V tiles and scores
    static constexpr int kQBufs = HD == 64 ? 2 : 1;          // places of the queries
    static constexpr int kDepth = HD == 64 ? 12 : 6;         // units whose codes are in flight
    static constexpr int kTileBytes = kTile * HD * 2;        // an fp16 tile
    static constexpr int kPageCodes = kPage * HD / 2;        // codes of K or V of a page
    static constexpr int kPageBytes = 2 * kPageCodes;        // codes of K, of V
    static constexpr int kParams = kUnitPages * kPageBytes;  // behind the codes: [page][K, V][kPage]
    static constexpr int kUnitBytes = kParams + kUnitPages * 2 * kPage * 4;
    static constexpr int kK = 0;
    static constexpr int kV = kK + kTurns * kTileBytes;
    static constexpr int kRing = kV + kTurns * kTileBytes;
    static constexpr int kInfo = kRing + kDepth * kUnitBytes;
    static constexpr int kUnit = kInfo + kUnits * 16;
    static constexpr int kCs = kUnit + kUnits * kUnitPages * 4;      // [kCsTurns][kRows]
    static constexpr int kEx = kCs + kCsTurns * kRows * 4;   // [2][kRows] float4
    static constexpr int kScale = kEx + 2 * kRows * 16;      // [kScales][factors of 4 pages' K, exponents of their V]
    static constexpr int kEnt = kScale + kScales * kScaleRec * 4;    // [kScales][kTile] (factor of K, exponent of V)
    static constexpr int kPar = kEnt + kScales * kTile * 8;  // [kDepth][K, V][kTile] what widens an entry, as fp16
    static constexpr int kBar = kPar + kDepth * 2 * kTile * 8;
    static constexpr int kBars = 5 * kTurns + 2 * kQBufs + 2 * kDepth;
    static_assert(2 * kTurns + 4 <= kScales, "factors that are in use");
    static constexpr int kTmem = kBar + kBars * 8;
    static constexpr int kBytes = kTmem + 16 + 1024;
    // tensor memory: S_t in columns 64 (t mod kTurns) .., group x's output x * HD behind them, then the queries
    static constexpr int kColO = kTurns * kTile, kColQ = kColO + 2 * HD;
    static_assert(kColQ + kQBufs * HD / 2 <= 512, "tensor memory");
    static_assert(kBytes <= 232448 - 2048, "shared memory of a block");
};
// the barriers of a window: k_full, v_full, s_full, p_full, pv_done [kTurns], q_full, q_empty [kQBufs], full, empty [kDepth]
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
    for (int s = 0; s < L::kDepth; ++s) {
        uint64_t* ring = bars + 5 * kTurns + 2 * L::kQBufs + s;
        mbar_init(ring, 64);
        mbar_init(ring + L::kDepth, L::kTeam);
    }
    fence_mbar_init();
}

// A unit's place among N that are taken in turn, and the parity of its use.
template <int N>
struct Place {
    int at;
    uint32_t odd = 0;
    __device__ __forceinline__ void step(int by) {
        at += by;
        if (at >= N) at -= N, odd ^= 1u;
    }
};

// What the CTA has set going in this window, units of each kind.
struct Issued {
    int s, pv;   // score products, P.V products
};

// arrives once this thread's copies so far have landed
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The eight codes n of a word as scale * n + base, one rounding: a code under
// fp16's lowest exponent is n * 2^-24, one four bits further up n * 2^-20, and
// by: scale * 2^24 and scale * 2^20 in its halves.
__device__ __forceinline__ void widen_k(uint32_t w, uint32_t by, uint32_t base, uint32_t (&v)[4]) {
    const __half2 lo = __low2half2(*reinterpret_cast<const __half2*>(&by)), hi = __high2half2(*reinterpret_cast<const __half2*>(&by));
    const __half2 b2 = __low2half2(*reinterpret_cast<const __half2*>(&base));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t x = h == 0 ? w : w >> 8, n0 = x & 0x000F000Fu, n1 = x & 0x00F000F0u;
        const __half2 v0 = __hfma2(*reinterpret_cast<const __half2*>(&n0), lo, b2);
        const __half2 v1 = __hfma2(*reinterpret_cast<const __half2*>(&n1), hi, b2);
        v[2 * h] = *reinterpret_cast<const uint32_t*>(&v0);
        v[2 * h + 1] = *reinterpret_cast<const uint32_t*>(&v1);
    }
}
// As scale * (n - 8) + mid, two roundings (mid's, and the sum's).
__device__ __forceinline__ void widen_v(uint32_t w, uint32_t scale, uint32_t mid, uint32_t (&v)[4]) {
    uint32_t n[4];
    widen(w, n);
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&n[y]), *reinterpret_cast<const __half2*>(&scale),
                                  *reinterpret_cast<const __half2*>(&mid));
        v[y] = *reinterpret_cast<const uint32_t*>(&h);
    }
}
// Four words of codes of an entry to the places x ^ turn of its chunk of a tile's row.
template <int SIDE>
__device__ __forceinline__ void widen_chunk(const uint2& w0, const uint2& w1, const uint2& by, uint8_t* row, int turn) {
    const uint32_t w[4] = {w0.x, w0.y, w1.x, w1.y};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        uint32_t v[4];
        if constexpr (SIDE == 0) widen_k(w[x], by.x, by.y, v);
        else widen_v(w[x], by.x, by.y, v);
        *reinterpret_cast<uint4*>(row + (turn ^ (x << 4))) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
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
    float2* s_ent = reinterpret_cast<float2*>(sm + L::kEnt);
    uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t* cv_full = k_full + kTurns;
    uint64_t* s_full = cv_full + kTurns;
    uint64_t* p_full = s_full + kTurns;
    uint64_t* pv_done = p_full + kTurns;
    uint64_t* q_full = pv_done + kTurns;
    uint64_t* q_empty = q_full + kQBufs;
    uint64_t* full = q_empty + kQBufs;
    uint64_t* empty = full + L::kDepth;
    uint2* s_par = reinterpret_cast<uint2*>(sm + L::kPar);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.nq / p.nkv;

    const uint32_t tmem = *reinterpret_cast<const uint32_t*>(sm + L::kTmem);
    const uint32_t t_o = tmem + L::kColO, t_q = tmem + L::kColQ;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_ab(bar, parity, nullptr, 0u, abort); };

    if (warp == kWarpS || warp == kWarpPv) {
        // The whole warp walks the units and one elected lane issues: in
        // warp-uniform control flow the descriptors stay in uniform registers.
        const bool scores = warp != kWarpPv;
        const uint32_t idesc_s = umma_idesc(0, kRows, kTile);   // format 0: fp16
        const uint32_t idesc_o = umma_idesc(0, kRows, HD) | kIdescBMnMajor;
        const uint64_t k_desc = umma_desc_sw128(smem_u32(sm + L::kK)), v_desc = umma_desc_sw128_mn(smem_u32(sm + L::kV), kTile * 128);
        int seg = 0, end = 0, no = -1, i = 0;
        Place<kTurns> c{0};
        for (; i < n; ++i, c.step(1)) {
            const int x = c.at;
            if (i == end) {
                seg = i;
                end = i + min(s_info[i].w - s_info[i].z, n - i);
                ++no;
                if (scores) ok = wait(&q_full[no % kQBufs], static_cast<uint32_t>((no / kQBufs) & 1));
            }
            if (scores) ok = ok && wait(&k_full[x], c.odd) && (i < kTurns || wait(&pv_done[x], c.odd ^ 1u));
            else ok = ok && wait(&cv_full[x], c.odd) && wait(&p_full[x], c.odd);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t t_s = tmem + static_cast<uint32_t>(x * kTile);
            if (scores) {
                const uint32_t q_addr = t_q + static_cast<uint32_t>(no % kQBufs * (HD / 2));
                const uint64_t k_at = k_desc + static_cast<uint32_t>(x * L::kTileBytes / 16);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk)
                        umma_bf16_a_tmem(t_s, q_addr + static_cast<uint32_t>(kk * 8),
                                         k_at + static_cast<uint32_t>(((kk >> 2) * kTile * 128 + (kk & 3) * 32) / 16), idesc_s, kk > 0 ? 1u : 0u);
                    umma_commit(&s_full[x]);
                    if (i + 1 == end) umma_commit(&q_empty[no % kQBufs]);
                }
            } else {
                const uint64_t v_at = v_desc + static_cast<uint32_t>(x * L::kTileBytes / 16);
                const uint32_t more = i - seg > 1 ? 1u : 0u;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        umma_bf16_a_tmem(t_o + static_cast<uint32_t>((i & 1) * HD), t_s + static_cast<uint32_t>(kk * 8),
                                         v_at + static_cast<uint32_t>(kk * 16 * 128 / 16), idesc_o,
                                         kk > 0 ? 1u : more);
                    umma_commit(&pv_done[x]);
                }
            }
            __syncwarp();
        }
        if (lane == 0) (scores ? issued->s : issued->pv) = i;
        if (!FIRST && ok && win->more) {   // what this warp committed has arrived: the next window takes the barriers anew
            for (int i = max(0, n - kTurns); i < n; ++i)
                ok = ok && wait(&(scores ? s_full : pv_done)[i % kTurns], static_cast<uint32_t>((i / kTurns) & 1));
            for (int x = max(0, no + 1 - kQBufs); scores && x <= no; ++x)
                ok = ok && wait(&q_empty[x % kQBufs], static_cast<uint32_t>((x / kQBufs) & 1));
            ok = __all_sync(0xffffffffu, ok);
        }
        __syncwarp();
    } else if (warp >= kWarpConv && warp < kWarpS) {
        constexpr int kTeam = L::kTeam, kTeams = 8 / kTeam, kMine = kUnitPages / kTeam;
        static_assert(L::kDepth % kTeams == 0 && kTeams <= kTurns && (kQBufs == 1 || kQBufs == 2), "phases that a team does not see");
        const int ct = tid & 127, quad = (warp - kWarpConv) / 4, team = (warp - kWarpConv) / kTeam, part = (warp - kWarpConv) % kTeam;
        constexpr int kChunks = HD / 32, kPasses = kPage * kChunks / 32, kPass = 32 / kChunks;   // chunks of an entry; passes over a page
        const int ch = lane % kChunks, row0 = lane / kChunks;
        int seg = 0, end = 0, no = -1, S = 0, last = 0, unit0 = 0;
        // the query rows of the segments up to the one of unit `upto`: every
        // warp has 32 of them
        auto queries = [&](int upto) {
            while (ok && end <= upto) {
                const int4 info = s_info[end];
                seg = end;
                unit0 = info.z;
                end += min(info.w - info.z, n - end);
                const int b = info.x;
                const int rows = p.rows != nullptr ? p.rows[b] : p.K;
                S = p.seq_lens[b];
                last = S + rows - 1;
                // the place's last reader: S of the segment kQBufs back
                auto free_place = [&]() {
                    if (no >= kQBufs) ok = wait(&q_empty[no % kQBufs], static_cast<uint32_t>((no / kQBufs) & 1) ^ 1u);
                };
                if ((++no & 1) != quad) {   // the other four warps'
                    // (a single place's barrier is seen in every phase: a parity alone stands for two)
                    if (kQBufs == 1) free_place();
                    continue;
                }
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
#pragma unroll 4
                for (int x = 0; x < HD / 8; ++x) {
                    const uint4 q = load(x);
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) top = max(top, max((w[y] << 16) & 0x7FFF0000u, w[y] & 0x7FFF0000u));
                }
                free_place();
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after_sync();
                // the row times 2^(141 - E): its largest value lies in [2^14, 2^15)
                const int E = min(max(static_cast<int>(top >> 23), 14), 253);
                const float down = __uint_as_float(static_cast<uint32_t>(268 - E) << 23);
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
                // back from there (and K from 2^15 below its factor); a row
                // that holds an infinity (or a NaN) is NaN
                s_cs[(no & (kCsTurns - 1)) * kRows + ct] =
                    top >= 0x7F800000u ? NAN : p.scale_log2 * __uint_as_float(static_cast<uint32_t>(E + 1) << 23);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[no % kQBufs]);
            }
        };
        Place<kTurns> at{team};
        Place<L::kDepth> ring{team};
        for (int i = team;; i += kTeams, at.step(kTeams), ring.step(kTeams)) {
            queries(min(i, n - 1));
            if (i >= n) break;
            const int c = at.at, d = ring.at;
            ok = ok && wait(&full[d], ring.odd);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            // What widens the entries of this warp's pages: lanes 0-15 K's, 16-31 V's
            const int e0 = (unit0 + i - seg) * kTile;
            const bool alone = e0 + kTile - 1 > S || p.scale_log2 < 0.f;
            const bool v_side = lane >= kPage;
#pragma unroll
            for (int q = 0; q < kMine; ++q) {
                const int page = part * kMine + q, e = page * kPage + lane % kPage;
                const uint32_t pr = reinterpret_cast<const uint32_t*>(sm + L::kRing + d * L::kUnitBytes + L::kParams)[page * 32 + lane];
                // of base and of 15 scale
                const uint32_t eb = (pr >> 23) & 0xFFu, es = (pr >> 7) & 0xFFu;
                uint32_t f = e0 + e > last || eb == 255u || es == 255u ? 0u : max(eb, es + 4u);
                // Where some row does not see all of the unit an entry has a power of
                // two to itself: what a row does not see does not move its outputs.
                if (!alone) {
                    const uint32_t of_k = __reduce_max_sync(0xffffffffu, v_side ? 0u : f), of_v = __reduce_max_sync(0xffffffffu, v_side ? f : 0u);
                    f = v_side ? of_v : of_k;
                }
                // |base| and 16 scale are below 2^(f - 126). K is stored times
                // 2^(122 - f) (below 2^-3, its scale below 2^-8), V times
                // 2^(140 - f) (below 2^15).
                f = min(max(f, 24u), 254u);
                const float up = __uint_as_float((267u - f) << 23), mid = mid_of(pr), scale = scale_of(pr) * up;
                const float back = __uint_as_float((f - 10u) << 23), lg = static_cast<float>(static_cast<int>(f) - 140);
                const bool odd = mid != mid;
                uint2 by;
                if (!v_side) {
                    const float base = odd ? NAN : __uint_as_float(pr & 0xFFFF0000u) * up * 0x1p-18f;
                    by = make_uint2(pack_f16(scale * 64.f, scale * 4.f), pack_f16(base, base));
                } else {
                    by = make_uint2(pack_f16(scale, scale), pack_f16(mid * up, mid * up));
                    if (alone && (odd || e0 + e > last)) by = make_uint2(0u, 0u);
                }
                s_par[(d * 2 + v_side) * kTile + e] = by;
                if (alone) {
                    // A V that is not finite enters through the score, and only of the rows that see it.
                    const bool v_odd = __shfl_down_sync(0xffffffffu, static_cast<int>(odd), kPage) != 0;
                    float* ent = reinterpret_cast<float*>(s_ent + (i % kScales) * kTile + e);
                    ent[v_side] = v_side ? lg : v_odd ? NAN : back;
                } else if (lane % kPage == 0) {
                    s_scale[(i % kScales) * kScaleRec + v_side * kUnitPages + page] = v_side ? lg : back;
                }
            }
            __syncwarp();
            // far: words in another order, so that the lanes of a store meet no bank twice
            const bool far = (ch >> 1) != 0;
            const uint8_t* codes = sm + L::kRing + d * L::kUnitBytes + part * kMine * L::kPageBytes + lane * 16;
            const uint2* par = s_par + d * 2 * kTile + part * kMine * kPage + row0;
            uint8_t* tile = sm + c * L::kTileBytes + (ch >> 1) * kTile * 128 + (part * kMine * kPage + row0) * 128;
            const int place = ((far ? 2 : 0) ^ ((ch & 1) * 4) ^ (row0 & 7)) << 4;
            auto widen_side = [&](auto of) {
                constexpr int kSide = decltype(of)::value;
                // the last reader of the place: S, or P V, of the unit kTurns back
                if (i >= kTurns) ok = ok && wait(&(kSide == 0 ? s_full : pv_done)[c], at.odd ^ 1u);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
#pragma unroll 2
                for (int x = 0; x < kMine * kPasses; ++x) {
                    static_assert(kPass % 8 == 0, "the swizzle of a thread's rows");
                    const int r = x * kPass;
                    const uint8_t* from = codes + kSide * L::kPageCodes + (r / kPage) * L::kPageBytes + (r % kPage) * (HD / 2);
                    const uint2 w0 = *reinterpret_cast<const uint2*>(from + (far ? 8 : 0)), w1 = *reinterpret_cast<const uint2*>(from + (far ? 0 : 8));
                    widen_chunk<kSide>(w0, w1, par[kSide * kTile + r], tile + kSide * (L::kV - L::kK) + r * 128, place);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&(kSide == 0 ? k_full : cv_full)[c]);
            };
            widen_side(std::integral_constant<int, 0>{});
            if (ok) widen_side(std::integral_constant<int, 1>{});
            if (!ok) break;
            if (lane == 0) mbar_arrive(&empty[d]);
        }
    } else if (warp >= kWarpFetch) {
        // a warp for the codes of K, and one for V's and both sides' parameters
        const bool v_side = warp > kWarpFetch;
        const uint64_t policy = l2_policy_evict_first();
        const uint8_t* codes = (v_side ? p.v_codes : p.k_codes) + lane * 16;
        const uint32_t* params = ((lane >> 2) & 1 ? p.v_params : p.k_params) + (lane & 3) * 4;
        const uint32_t to = smem_u32(sm + L::kRing) + v_side * L::kPageCodes + lane * 16;
        const uint32_t to_params = smem_u32(sm + L::kRing) + L::kParams + lane * 16;
        Place<L::kDepth> at{0};
        for (int i = 0; i < n; ++i, at.step(1)) {
            const int d = at.at;
            if (i >= L::kDepth) ok = wait(&empty[d], at.odd ^ 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int4 tl = *reinterpret_cast<const int4*>(s_tile + i * kUnitPages);
            const int tile[kUnitPages] = {tl.x, tl.y, tl.z, tl.w};
#pragma unroll
            for (int q = 0; q < kUnitPages; ++q) {
                if (tile[q] < 0) continue;
                const uint8_t* from = codes + static_cast<size_t>(tile[q]) * L::kPageCodes;
#pragma unroll
                for (int x = 0; x < L::kPageCodes; x += 512)
                    copy_async<16>(to + d * L::kUnitBytes + q * L::kPageBytes + x, from + x, policy);
            }
            if (v_side) {
                const int mine = s_tile[i * kUnitPages + (lane >> 3)];
                if (mine >= 0) copy_async<16>(to_params + d * L::kUnitBytes, params + static_cast<size_t>(mine) * kPage, policy);
            }
            copies_arrive(&full[d]);
        }
        copies_commit();
        copies_wait<0>();
    } else if (warp < kWarpConv) {
        // ------------------------------------------------ softmax: thread = query row
        const int grp = warp >> 2, row = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_mine = t_o + lane_off + static_cast<uint32_t>(grp * HD);
        const bool flip = p.scale_log2 < 0.f;
        int no = 0;
        Place<kTurns> c{grp}, had{grp};   // of this group's next unit, and of its last one
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
            float m = -INFINITY, md = -INFINITY, l = 0.f, mark = 0.f, cs = 0.f;
            for (int i = first; i < seg + len; i += 2, had = c, c.step(2)) {
                const uint32_t t_s = tmem + lane_off + static_cast<uint32_t>(c.at * kTile);
                if (ok) ok = wait(&s_full[c.at], c.odd);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) continue;
                tc_fence_after_sync();
                if (busy) {
                    if (i == first) cs = s_cs[(no & (kCsTurns - 1)) * kRows + row];
                    const int4 tl = *reinterpret_cast<const int4*>(s_tile + i * kUnitPages);
                    if (tl.x == -1 || tl.y == -1 || tl.z == -1 || tl.w == -1) mark = kMarkBadPage;
                    const int e0 = (info.z + i - seg) * kTile;
                    const bool alone = e0 + kTile - 1 > S || flip;   // factors of entries, not of pages
                    const float* page = s_scale + (i % kScales) * kScaleRec;
                    const float* ent = reinterpret_cast<const float*>(s_ent + (i % kScales) * kTile);
                    // 16 of the unit's scores, rounded, with their entries' or their page's factors; -inf where the row
                    // does not see them. v: the exponents of their V, a step apart
                    const int step = alone ? 2 : 0;
                    auto scores = [&](int at, float (&s)[16], const float*& v) {
                        tmem_ld16(t_s + static_cast<uint32_t>(at), s);
                        const float* k = alone ? ent + 2 * at : page + at / kPage;
                        v = alone ? k + 1 : k + kUnitPages;
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            s[x] *= cs * k[x * step];
                            if (e0 + at + x > lim) s[x] = -INFINITY;
                        }
                        __syncwarp();
                    };
                    // largest score; largest score + exponent of its V, relative to the larger of m and the scores
                    float top = -INFINITY, most = -INFINITY, kf[4], vl[4];
                    if (!alone) {
                        const float4* sc = reinterpret_cast<const float4*>(page);
                        const float4 ks = sc[0], vlg = sc[1];   // of the pages
                        kf[0] = cs * ks.x; kf[1] = cs * ks.y; kf[2] = cs * ks.z; kf[3] = cs * ks.w;
                        vl[0] = vlg.x; vl[1] = vlg.y; vl[2] = vlg.z; vl[3] = vlg.w;
                        float s[kTile], t[4];
                        tmem_ld64(t_s, s);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float* sq = s + q * 16;
                            const float a = max3(max3(sq[0], sq[1], sq[2]), max3(sq[3], sq[4], sq[5]), max3(sq[6], sq[7], sq[8]));
                            const float b = max3(max3(sq[9], sq[10], sq[11]), max3(sq[12], sq[13], sq[14]), sq[15]);
                            t[q] = fmaxf(a, b) * kf[q];
                            top = fmaxf(top, t[q]);
                        }
                        const float high = fmaxf(top, m);
#pragma unroll
                        for (int q = 0; q < 4; ++q) most = fmaxf(most, t[q] - high + vl[q]);
                    } else {
                        float high = m;
#pragma unroll 1
                        for (int at = 0; at < kTile; at += 16) {
                            float s[16];
                            const float* v;
                            scores(at, s, v);
                            const float had = high;
#pragma unroll
                            for (int x = 0; x < 16; ++x) top = fmaxf(top, s[x]);
                            high = fmaxf(high, top);
                            most += had - high;   // (NaN while a row has seen no entry, and no maximum of what follows)
#pragma unroll
                            for (int x = 0; x < 16; ++x) most = fmaxf(most, s[x] - high + v[x * step]);
                        }
                    }
                    const float high = fmaxf(top, m);
                    if (top > m + kRescale) {
                        l *= m == -INFINITY ? 0.f : ex2(m - top);
                        md += m - top;
                        m = top;
                    }
                    // 0 in the place of the maximum where a row has seen no entry
                    const float mm = m == -INFINITY ? 0.f : -m;
                    most += high - m;   // (a row that has seen no entry: NaN, which moves nothing)
                    float f = 1.f;
                    if (most > md + kRescale) {
                        f = md == -INFINITY ? 0.f : ex2(md - most - kHead);
                        md = most + kHead;
                    }
                    if (i > first && __any_sync(0xffffffffu, f != 1.f)) {
                        // this group's last P.V has to be done
                        ok = wait(&pv_done[had.at], had.odd);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) continue;
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < HD / 32; ++c) {
                            float o[32];
                            uint32_t v[32];
                            tmem_ld32(t_mine + static_cast<uint32_t>(c * 32), o);
#pragma unroll
                            for (int x = 0; x < 32; x += 2) {
                                const float2 y = unf2(mul2(f2(o[x], o[x + 1]), f2(f, f)));
                                v[x] = __float_as_uint(y.x);
                                v[x + 1] = __float_as_uint(y.y);
                            }
                            tmem_st32(t_mine + static_cast<uint32_t>(c * 32), v);
                        }
                    }
                    const float from = kLift - md;
                    uint64_t sum[2] = {0ull, 0ull};
                    // P of a half goes where S of the first half stood
                    if (!alone && !__any_sync(0xffffffffu, fabsf(mm) > kFine)) {
                        const uint64_t m2 = f2(mm, mm);
                        const float vr[4] = {lift(from, vl[0]), lift(from, vl[1]), lift(from, vl[2]), lift(from, vl[3])};
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float s[32], pk[16];   // pk: pairs of fp16
                            tmem_ld32(t_s + static_cast<uint32_t>(half * 32), s);
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const float kq = half == 0 ? kf[q] : kf[2 + q], rq = half == 0 ? vr[q] : vr[2 + q];
                                const uint64_t k2 = f2(kq, kq), r2 = f2(rq, rq);
#pragma unroll
                                for (int x = 0; x < 8; ++x) {
                                    const float2 a = unf2(fma2(f2(s[q * 16 + 2 * x], s[q * 16 + 2 * x + 1]), k2, m2));
                                    const uint64_t w = f2(ex2(a.x), ex2(a.y));
                                    sum[x & 1] = add2(sum[x & 1], w);
                                    const float2 r = unf2(mul2(w, r2));
                                    pk[q * 8 + x] = __uint_as_float(pack_f16(r.x, r.y));
                                }
                            }
                            __syncwarp();
                            tmem_st16(t_s + static_cast<uint32_t>(half * 16), pk);
                        }
                    } else {
#pragma unroll 1
                        for (int at = 0; at < kTile; at += 16) {
                            float s[16];
                            const float* v;
                            uint32_t pk[8];
                            scores(at, s, v);
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                const float2 w = make_float2(ex2(s[2 * x] + mm), ex2(s[2 * x + 1] + mm));
                                sum[x & 1] = add2(sum[x & 1], f2(w.x, w.y));
                                pk[x] = pack_f16(w.x * lift(from, v[2 * x * step]), w.y * lift(from, v[(2 * x + 1) * step]));
                            }
                            __syncwarp();
                            tmem_st8(t_s + static_cast<uint32_t>(at / 2), pk);
                        }
                    }
                    const float2 sa = unf2(add2(sum[0], sum[1]));
                    l += sa.x + sa.y;
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[c.at]);
            }
            if (ok && first < seg + len) ok = wait(&pv_done[had.at], had.odd);
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
            const float ga = unlift(xa.x, xa.z, M) * inv, gb = unlift(xb.x, xb.z, M) * inv;
            __nv_bfloat16* out = p.out + (static_cast<long long>(b) * p.K + j) * p.ld_out +
                                 static_cast<long long>(head * G + row - j * G) * HD + grp * (HD / 2);
            const bool sectors = ((reinterpret_cast<uintptr_t>(p.out) | static_cast<uintptr_t>(p.ld_out) * 2) & 31u) == 0;
            const bool all_ok = __all_sync(0xffffffffu, !(bad < 0.f));
            // which groups had a tile: the same for the whole segment
            const bool has_a = (seg & 1) == 0 || len > 1, has_b = (seg & 1) == 1 || len > 1;
            if (busy) {
#pragma unroll 1
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
    uint8_t* sm = smem_raw + (1024u - smem_u32(smem_raw) % 1024u) % 1024u;   // (an offset: still known to be shared memory)
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
            // (the copies have been waited for)
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
