// Attention over the 8-bit KV cache for many query rows (a draft pass: K rows
// of every head of a group): the tensor-memory kernel behind pe_attention_kv8.
//
// A unit is 64 entries (4 pages) of one (request, kv head); all its query rows
// (at most 128, the MMA's M) share every entry, so the cache is read once.
// Roles (512 threads):
//   warps 14,15 the unit's K pages to where the MMA reads them (the swizzle of
//               a K-major operand), and the page scales. 128-wide heads: warp
//               14 the codes by TMA, a lane per page, warp 15 the scales;
//               64-wide ones: both warps in turn by asynchronous copies. A box of 16 rows takes about 150 cycles
//               whatever its rows hold, a copy instruction always 512 bytes
//               (128 wide: 181 us by boxes, 192 by copies; 64 wide: 85 and 80)
//   warps 8-11  converters, kTeam warps to a unit. Each thread fetches 16-byte
//               chunks of V, kDepth units ahead, by asynchronous copies to a
//               place of its own, and turns them into an fp16 tile (fp16 holds
//               every E4M3 value; 128-byte swizzle, entry-major, read as an
//               MN-major operand), V of entries that no row sees zero. A unit
//               of 64-wide heads to a warp each, in turn (80 us, all four warps
//               on every unit 85); four warps to each of 128-wide ones, whose V
//               tiles have fewer places (178 us, a warp each 261). At the start
//               of a segment the query rows: shifted by a power of two per row
//               so that the largest value lies in [128, 256) and split into two
//               E4M3 terms, q = hi + lo, which hold the 8 bits of a bf16 value
//               exactly from 1/4 on, 2^-9 of the row's largest, and to half of
//               E4M3's smallest step, 2^-17 of the largest, below.
//   warp 12     one elected lane issues S_t = Q_hi K_t^T + Q_lo K_t^T (M=128,
//               N=64, E4M3 operands: the codes themselves)
//   warp 13     one elected lane issues O += P_t V_t (fp16, A = P_t from
//               tensor memory)
//   warps 0-3, 4-7  two softmax groups, thread = query row = TMEM lane: group
//               x takes the units t = x (mod 2), with a running maximum, sum
//               and output accumulator of its own, so that neither waits for
//               the other; they meet at the end of a segment.
// kTurns S_t buffers: P_t (fp16 pairs) overwrites the columns of S_t, and S
// runs up to that many units ahead of P.V, so a group finds its next scores
// ready when it is done with the last. V tiles and S_t have as many places and
// "P_t V_t is complete" frees both, as "S_t is complete" frees K_t's place: one
// commit for each product. Waits, MMAs and commits cost their warp
// about 100, 40 and 100 cycles each; with both products and six commits in one
// warp that, 1550 cycles a unit, was what bounded the kernel.
//
// K codes as MMA operands leave only V to be widened: with K widened too the
// shared memory carried 128 KB a unit, a quarter more than now, at 128 bytes a
// cycle.
//
// A unit takes some 1150 cycles (64-wide heads: 1000), where its bytes would
// take 730 (370) and its products 640; no stage by itself holds it: without
// the softmax it is 8% faster (64-wide heads 15%), without the copies 3% (7%),
// without the widening 4% (2%), without the exponentials or either product no
// more than 4%. Units of 128 entries (64-wide heads 93 us where 87 were taken
// then, 128-wide ones 250 for 190), a third softmax group for 64-wide heads
// (100 for 87) and scores of two units in one product (242 for 235) did not
// help. 128 requests of 512 to 8192 entries, 11 rows of 8 heads to each of 4
// of 128: 181 us, 3.3 TB/s, 49% of the measured copy; 64 of 1024 to 4096, up
// to 10 rows of 8 heads to each of 8 of 64: 81 us, 29%.
#include "attn_kv8.cuh"

namespace pe {
namespace {

using namespace kv8;

constexpr int kThreads = 512;
constexpr int kTile = kUmmaPages * kPage;   // entries of a unit
constexpr int kRows = kUmmaRows;
constexpr int kSoft = 256;                  // softmax threads
constexpr int kWarpConv = 8, kWarpS = 12, kWarpPv = 13, kWarpK = 14;
constexpr int kDepth = 4;                   // units whose V copies are in flight
constexpr int kBehind = 1;                  // units whose K copies a warp has in flight while it waits for the one before
constexpr int kScales = 16;                 // units whose page scales are kept: fetched kDepth ahead, read a few behind
constexpr int kScaleRec = 3 * kUmmaPages;   // floats of a unit's scales
constexpr int kCsTurns = 8;                 // segments whose row factors are kept: the converters run fewer ahead

__device__ __forceinline__ void mbar_inval(uint64_t* bar) {
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// E4M3 x E4M3, K = 32
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// K-major operand of HD-byte rows under the swizzle of that width
template <int HD>
__device__ __forceinline__ uint64_t desc_codes(uint32_t smem_addr) {
    if constexpr (HD == 128) return umma_desc_sw128(smem_addr);
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(512 >> 4) << 32;   // 8 rows of 64 bytes
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(4) << 61;          // 64-byte swizzle
    return d;
}

// 32 consecutive columns of the lane's TMEM row. These are instructions of a
// whole warp: where its lanes can have taken different ways before, a
// __syncwarp stands in front.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

// 32 bytes in one store: a whole sector of L2
__device__ __forceinline__ void store_sector(void* to, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// two floats in one instruction
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unf2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <int HD>
struct Layout {
    static constexpr bool kTmaK = HD == 128;                 // K by TMA boxes, or by copies of two warps
    static constexpr int kTeam = HD == 64 ? 1 : 4;           // converter warps to a unit
    static constexpr int kTurns = HD == 64 ? 6 : 4;          // places of K codes, fp16 V tiles and scores
    static constexpr int kCodes = kTile * HD;                // codes of K or V of a unit
    static constexpr int kCvTile = kTile * HD * 2;
    static constexpr int kQTerm = kRows * HD;                // hi or lo
    static constexpr int kQ = 0;                             // [2][hi, lo]
    static constexpr int kConv = kQ + 4 * kQTerm;
    static constexpr int kKRing = kConv + kTurns * kCvTile;
    static constexpr int kVRing = kKRing + kTurns * kCodes;
    static constexpr int kInfo = kVRing + kDepth * kCodes;
    static constexpr int kUnit = kInfo + kUmmaUnits * 16;
    static constexpr int kCs = kUnit + kUmmaUnits * kUmmaPages * 4;   // [kCsTurns][kRows]
    static constexpr int kEx = kCs + kCsTurns * kRows * 4;   // [2][kRows] float4
    static constexpr int kScale = kEx + 2 * kRows * 16;      // [kScales][ks of 4 pages, vs of 4 pages as its part and its lg]
    static constexpr int kNan = kScale + kScales * kScaleRec * 4;        // [kTurns][kTile] bytes
    static constexpr int kBar = kNan + kTurns * kTile;
    static constexpr int kBars = 5 * kTurns + 4;
    static constexpr int kTmem = kBar + kBars * 8;
    static constexpr int kBytes = kTmem + 16 + 1024;
};
static_assert(Layout<128>::kBytes <= 232448 - 2048 && Layout<64>::kBytes <= 232448 - 2048, "shared memory of a block");
// the barriers of a window: k_full, cv_full, s_full, p_full, pv_done [kTurns], q_full, q_empty [2]
template <int HD>
__device__ __forceinline__ void init_bars(uint64_t* bars, int stall) {
    using L = Layout<HD>;
    constexpr int kTurns = L::kTurns;
    for (int s = 0; s < kTurns; ++s) {
        mbar_init(&bars[s], (L::kTmaK ? 2 : 1) + (stall == kStallK));
        mbar_init(&bars[kTurns + s], L::kTeam + (stall == kStallV));
        mbar_init(&bars[2 * kTurns + s], 1);
        mbar_init(&bars[3 * kTurns + s], 4 + (stall == kStallP));
        mbar_init(&bars[4 * kTurns + s], 1);
    }
    for (int s = 0; s < 2; ++s) {
        mbar_init(&bars[5 * kTurns + s], 4);
        mbar_init(&bars[5 * kTurns + 2 + s], 1);
    }
    fence_mbar_init();
}

// What the CTA has set going in this window, units of each kind.
struct Issued {
    int k, s, pv;   // TMA copies of K, score products, P.V products
};
// Waits for the phase a millisecond at most.
__device__ __forceinline__ void settle(uint64_t* bar, uint32_t parity) {
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < 1000000ull) {}
}

// The n units of a window by every role; FIRST: of the share's first one. false
// in the threads of a role that gave up waiting.
template <int HD, bool FIRST>
__device__ __forceinline__ bool attend_window(const CUtensorMap& tmK, const Kv8Params& p, uint8_t* sm, int n, const Window* win,
                                              bool idle, const volatile int* abort, Issued* issued) {
    using L = Layout<HD>;
    constexpr int kTurns = L::kTurns;
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
    uint64_t* q_empty = q_full + 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.nq / p.nkv;

    const uint32_t tmem = *reinterpret_cast<const uint32_t*>(sm + L::kTmem);
    const uint32_t t_o = tmem + kTurns * kTile;   // S_t in columns 64 (t mod kTurns) ..; group x's output x * HD behind them
    bool ok = true;
    auto turn = [](int i) { return static_cast<uint32_t>((i / kTurns) & 1); };   // parity of unit i's use of its place
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_ab(bar, parity, nullptr, 0u, abort); };
    // the K and V scales of unit i's pages, a lane each: fetched, and once they are there V's taken apart
    const uint64_t policy_s = l2_policy_evict_first();
    auto fetch_scales = [&](int i) {
        if (lane < 2 * kUmmaPages) {
            float* to = s_scale + (i % kScales) * kScaleRec + lane;
            const int tile = s_tile[i * kUmmaPages + lane % kUmmaPages];
            if (tile >= 0) copy_async<4>(smem_u32(to), (lane < kUmmaPages ? p.k_scale : p.v_scale) + tile, policy_s);
            else *to = 0.f;
        }
    };
    auto split_scales = [&](int i) {
        if (lane >= kUmmaPages && lane < 2 * kUmmaPages) {
            float* at = s_scale + (i % kScales) * kScaleRec + lane;
            split_scale(*at, at[0], at[kUmmaPages]);
        }
    };

    if (L::kTmaK && warp == kWarpK) {
        const uint64_t policy = l2_policy_evict_first();
        int i = 0;
        for (; i < n; ++i) {
            const int x = i % kTurns;
            const int tile = lane < kUmmaPages ? s_tile[i * kUmmaPages + lane] : -1;
            const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, tile >= 0)) * kPage * HD);
            if (i >= kTurns) ok = wait(&s_full[x], turn(i) ^ 1u);   // S of the unit before it in this place
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&k_full[x], bytes);
            __syncwarp();
            if (lane < kUmmaPages && tile >= 0)
                tma_load_2d(sm + L::kKRing + x * L::kCodes + lane * kPage * HD, &tmK, &k_full[x], 0, tile * kPage, policy);
        }
        if (lane == 0) issued->k = i;
        __syncwarp();
    } else if (L::kTmaK && warp == kWarpK + 1) {
        for (int i = 0; i < n + kDepth; ++i) {
            if (i < n) fetch_scales(i);
            copies_commit();
            const int u = i - kDepth, x = u % kTurns;
            if (u < 0) continue;
            if (u >= kTurns) ok = wait(&s_full[x], turn(u) ^ 1u);   // an arrival counts for this unit, not the one before it
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            copies_wait<kDepth>();
            split_scales(u);
            __syncwarp();
            if (lane == 0) mbar_arrive(&k_full[x]);
        }
        copies_wait<0>();
        __syncwarp();
    } else if (!L::kTmaK && warp >= kWarpK) {
        // two warps, a unit each in turn; chunk c of a row goes where the swizzle of a K-major operand has it
        constexpr int kChunks = HD / 16, kPass = 32 / kChunks, kPasses = kPage / kPass;
        const uint64_t policy = l2_policy_evict_first();
        const int row = lane / kChunks, c = lane % kChunks;
        const uint8_t* from = p.k_codes + lane * 16;
        uint32_t to[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = row + x * kPass;
            to[x] = smem_u32(sm + L::kKRing) + row * HD + ((c ^ ((r >> 1) & 3)) << 4);   // (64 wide)
        }
        const int first = warp - kWarpK;
        for (int i = first; i < n + 2 * kBehind; i += 2) {
            const int x = i % kTurns;
            if (i < n) {
                if (i >= kTurns) ok = wait(&s_full[x], turn(i) ^ 1u);   // S of the unit before it in this place
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
#pragma unroll
                for (int q = 0; q < kUmmaPages; ++q) {
                    const int tile = s_tile[i * kUmmaPages + q];
                    if (tile < 0) continue;
                    const uint8_t* src = from + static_cast<long long>(tile) * (kPage * HD);
#pragma unroll
                    for (int j = 0; j < kPasses; ++j)
                        copy_async<16>(to[j & 1] + x * L::kCodes + q * kPage * HD + j * 512, src + j * 512, policy);
                }
                fetch_scales(i);
            }
            copies_commit();
            if (i >= 2 * kBehind) {
                copies_wait<kBehind>();
                split_scales(i - 2 * kBehind);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&k_full[(i - 2 * kBehind) % kTurns]);
            }
        }
        copies_wait<0>();
        __syncwarp();
    } else if (warp == kWarpS || warp == kWarpPv) {
        // The whole warp walks the units and one elected lane issues: in
        // warp-uniform control flow the descriptors stay in uniform registers.
        const bool scores = warp != kWarpPv;
        const uint32_t idesc_s = umma_idesc(0, kRows, kTile);   // formats 0: E4M3 here, fp16 below
        const uint32_t idesc_o = umma_idesc(0, kRows, HD) | kIdescBMnMajor;
        const uint32_t q_base = smem_u32(sm + L::kQ), k_base = smem_u32(sm + L::kKRing);
        const uint32_t cv_base = smem_u32(sm + L::kConv);
        int seg = 0, end = 0, no = -1, i = 0;
        for (; i < n; ++i) {
            const int x = i % kTurns;
            if (i == end) {
                seg = i;
                end = i + min(s_info[i].w - s_info[i].z, n - i);
                ++no;
                if (scores) ok = wait(&q_full[no & 1], static_cast<uint32_t>((no >> 1) & 1));
            }
            if (scores) ok = ok && wait(&k_full[x], turn(i)) && (i < kTurns || wait(&pv_done[x], turn(i) ^ 1u));
            else ok = ok && wait(&cv_full[x], turn(i)) && wait(&p_full[x], turn(i));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t t_s = tmem + static_cast<uint32_t>(x * kTile);
            if (scores) {
                const uint32_t q_addr = q_base + (no & 1) * 2 * L::kQTerm, k_addr = k_base + x * L::kCodes;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < HD / 32; ++kk) {
                        const uint64_t kd = desc_codes<HD>(k_addr + kk * 32);
                        umma_e4m3(t_s, desc_codes<HD>(q_addr + kk * 32), kd, idesc_s, kk > 0 ? 1u : 0u);
                        umma_e4m3(t_s, desc_codes<HD>(q_addr + L::kQTerm + kk * 32), kd, idesc_s, 1u);
                    }
                    umma_commit(&s_full[x]);
                    if (i + 1 == end) umma_commit(&q_empty[no & 1]);
                }
            } else {
                const uint32_t v_addr = cv_base + x * L::kCvTile;
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
            for (int x = max(0, no - 1); scores && x <= no; ++x) ok = ok && wait(&q_empty[x & 1], static_cast<uint32_t>((x >> 1) & 1));
            ok = __all_sync(0xffffffffu, ok);
        }
        __syncwarp();
    } else if (warp >= kWarpConv && warp < kWarpS) {
        constexpr int kTeam = L::kTeam, kTeams = 4 / kTeam, kAhead = kDepth / kTeams;
        const int ct = tid & 127, team = (warp - kWarpConv) / kTeam, part = (warp - kWarpConv) % kTeam;
        // a pass of a warp covers kPass rows of its part of the unit; this lane's chunk of them
        constexpr int kChunks = HD / 16, kPass = 32 / kChunks, kPasses = kTile / kTeam / kPass, kMine = kUmmaPages / kTeam;
        const int ch = lane % kChunks, row0 = part * (kTile / kTeam) + lane / kChunks;
        const uint64_t policy = l2_policy_evict_first();
        const uint8_t* from = p.v_codes + lane * 16;
        uint8_t* ring = sm + L::kVRing + part * kMine * kPage * HD + lane * 16;
        const uint32_t v_at = smem_u32(ring);
        auto fetch = [&](int i) {
            if (i < n) {
#pragma unroll
                for (int q = 0; q < kMine; ++q) {
                    const int tile = s_tile[i * kUmmaPages + part * kMine + q];
                    if (tile < 0) continue;
                    const uint8_t* src = from + static_cast<long long>(tile) * (kPage * HD);
#pragma unroll
                    for (int x = 0; x < kPage / kPass; ++x)
                        copy_async<16>(v_at + (i % kDepth) * L::kCodes + q * kPage * HD + x * 512, src + x * 512, policy);
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
                // twice over the row, half of it at a time (registers): its
                // largest value, then its terms
                const bool live = ct < rows * G;
                constexpr int kHalf = HD / 16;
                if (live) {
#pragma unroll
                    for (int x = 0; x < HD / 64; ++x)
                        asm volatile("prefetch.global.L1 [%0];" ::"l"(src + x * 64));
                }
                auto load = [&](uint4 (&q)[kHalf], int half) {
#pragma unroll
                    for (int x = 0; x < kHalf; ++x) {
                        q[x] = make_uint4(0u, 0u, 0u, 0u);
                        if (live) q[x] = *reinterpret_cast<const uint4*>(src + (half * kHalf + x) * 8);
                    }
                };
                uint32_t top = 0;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint4 q[kHalf];
                    load(q, half);
#pragma unroll
                    for (int x = 0; x < kHalf; ++x) {
                        const uint32_t w[4] = {q[x].x, q[x].y, q[x].z, q[x].w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) top = max(top, max((w[y] << 16) & 0x7FFF0000u, w[y] & 0x7FFF0000u));
                    }
                }
                // the tile's last reader: S of the segment two back
                if (no >= 2) ok = wait(&q_empty[no & 1], static_cast<uint32_t>((no >> 1) & 1) ^ 1u);
                ok = __all_sync(0xffffffffu, ok);
                // the row times 2^(134 - E): its largest value lies in [128, 256)
                const int E = min(max(static_cast<int>(top >> 23), 8), 254);
                const float down = __uint_as_float(static_cast<uint32_t>(261 - E) << 23);
                uint8_t* dst = sm + L::kQ + (no & 1) * 2 * L::kQTerm + ct * HD;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint4 q[kHalf];
                    load(q, half);
#pragma unroll
                    for (int x = 0; x < kHalf / 2; ++x) {
                        const uint32_t w[8] = {q[2 * x].x, q[2 * x].y, q[2 * x].z, q[2 * x].w,
                                               q[2 * x + 1].x, q[2 * x + 1].y, q[2 * x + 1].z, q[2 * x + 1].w};
                        uint32_t hi[4], rest[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float v0 = __uint_as_float(w[2 * y] << 16) * down, v1 = __uint_as_float(w[2 * y] & 0xFFFF0000u) * down;
                            const float v2 = __uint_as_float(w[2 * y + 1] << 16) * down, v3 = __uint_as_float(w[2 * y + 1] & 0xFFFF0000u) * down;
                            hi[y] = e4m3x4(v0, v1, v2, v3);
                            const uint32_t a = widen_lo(hi[y]), d = widen_hi(hi[y]);
                            const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
                            const float2 fd = __half22float2(*reinterpret_cast<const __half2*>(&d));
                            rest[y] = e4m3x4(v0 - fa.x, v1 - fa.y, v2 - fd.x, v3 - fd.y);
                        }
                        const int part = half * (kHalf / 2) + x;   // 16 dimensions
                        const int to = (HD == 128 ? part ^ (ct & 7) : part ^ ((ct >> 1) & 3)) << 4;
                        *reinterpret_cast<uint4*>(dst + to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(dst + L::kQTerm + to) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
                    }
                }
                // E4M3 has no infinity: a row that holds one (or a NaN) is NaN
                s_cs[(no & (kCsTurns - 1)) * kRows + ct] =
                    top >= 0x7F800000u ? NAN : p.scale_log2 * __uint_as_float(static_cast<uint32_t>(E - 7) << 23);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[no & 1]);
            }
        };
        for (int i = team; i < n; i += kTeams) {
            const int c = i % kTurns;
            queries(i);
            copies_wait<kAhead - 1>();
            uint4 v[kPasses];
#pragma unroll
            for (int x = 0; x < kPasses; ++x)
                v[x] = *reinterpret_cast<const uint4*>(ring + (i % kDepth) * L::kCodes + x * 512);
            fetch(i + kDepth);
            if (i >= kTurns) ok = ok && wait(&pv_done[c], turn(i) ^ 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int e0 = (s_info[seg].z + i - seg) * kTile;
            const bool inner = e0 + kTile - 1 <= S;
            if (!inner) {
#pragma unroll
                for (int x = 0; x < kPasses; ++x) {
                    const int r = row0 + x * kPass;
                    const bool out = e0 + r > last;
                    int nan = 0;
                    v[x].x = out ? 0u : without_nan(v[x].x, nan);
                    v[x].y = out ? 0u : without_nan(v[x].y, nan);
                    v[x].z = out ? 0u : without_nan(v[x].z, nan);
                    v[x].w = out ? 0u : without_nan(v[x].w, nan);
#pragma unroll
                    for (int d = 1; d < kChunks; d <<= 1) nan |= __shfl_xor_sync(0xffffffffu, nan, d);
                    if (ch == 0) s_nan[c * kTile + r] = static_cast<uint8_t>(nan);
                }
            }
            // 32 bytes of fp16 a chunk; which half goes first keeps the banks apart
            uint8_t* dst = sm + L::kConv + c * L::kCvTile + (ch >> 2) * kTile * 128;
            const int j0 = 2 * (ch & 3), odd = (ch >> 2) & 1;
#pragma unroll
            for (int x = 0; x < kPasses; ++x) {
                const int r = row0 + x * kPass;
                const uint4 a = make_uint4(widen_lo(v[x].x), widen_hi(v[x].x), widen_lo(v[x].y), widen_hi(v[x].y));
                const uint4 b = make_uint4(widen_lo(v[x].z), widen_hi(v[x].z), widen_lo(v[x].w), widen_hi(v[x].w));
                *reinterpret_cast<uint4*>(dst + r * 128 + (((j0 + odd) ^ (r & 7)) << 4)) = odd ? b : a;
                *reinterpret_cast<uint4*>(dst + r * 128 + (((j0 + 1 - odd) ^ (r & 7)) << 4)) = odd ? a : b;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&cv_full[c]);
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
            float m = -INFINITY, mo = -INFINITY, l = 0.f, mark = 0.f, cs = 0.f;
            for (int i = first; i < seg + len; i += 2) {
                const uint32_t t_s = tmem + lane_off + static_cast<uint32_t>((i % kTurns) * kTile);
                if (ok) ok = wait(&s_full[i % kTurns], turn(i));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) continue;
                tc_fence_after_sync();
                if (busy) {
                    if (i == first) cs = s_cs[(no & (kCsTurns - 1)) * kRows + row];
                    const float4* sc = reinterpret_cast<const float4*>(s_scale + (i % kScales) * kScaleRec);
                    const float4 ks = sc[0], vpart = sc[1], vlg = sc[2];
                    const int4 tl = *reinterpret_cast<const int4*>(s_tile + i * kUmmaPages);
                    float s[kTile];
                    tmem_ld64(t_s, s);
                    if (tl.x == -1 || tl.y == -1 || tl.z == -1 || tl.w == -1) mark = kMarkBadPage;
                    float kf[4] = {cs * ks.x, cs * ks.y, cs * ks.z, cs * ks.w};
                    const int e0 = (info.z + i - seg) * kTile;
                    const bool inner = e0 + kTile - 1 <= S;
                    if (!inner || flip || ks.x < 0.f || ks.y < 0.f || ks.z < 0.f || ks.w < 0.f) {
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
                    float top = -INFINITY, most = -INFINITY;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float* sq = s + q * 16;
                        float t4[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) t4[x] = fmaxf(fmaxf(sq[x], sq[x + 4]), fmaxf(sq[x + 8], sq[x + 12]));
                        const float t = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * kf[q];
                        top = fmaxf(top, t);
                        most = fmaxf(most, t + vl[q]);
                    }
                    if (top > m + kRescale) {
                        l *= m == -INFINITY ? 0.f : ex2(m - top);
                        m = top;
                    }
                    float f = 1.f;
                    if (most > mo + kRescale) {
                        f = mo == -INFINITY ? 0.f : ex2(mo - most);
                        mo = most;
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
                    const float mm = m == -INFINITY ? 0.f : -m;
                    const uint64_t m2 = f2(mm, mm);
                    // 0 in the place of both maxima where a row has seen no entry
                    const float from = (mo == -INFINITY ? 0.f : -mo) - mm + kLift;
                    const float vr[4] = {vpart.x * lift(from, vl[0]), vpart.y * lift(from, vl[1]),
                                         vpart.z * lift(from, vl[2]), vpart.w * lift(from, vl[3])};
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
            s_ex[grp * kRows + row] = make_float4(m, mark != 0.f ? mark : l, mo, 0.f);
            named_bar_sync(1, kSoft);
            const float4 xa = s_ex[row], xb = s_ex[kRows + row];
            const float bad = fminf(fminf(fminf(xa.y, xb.y), sum0), 0.f);   // a NaN sum is not less than 0
            const float M = fmaxf(fmaxf(xa.x, xb.x), M0), f0 = M0 == M ? 1.f : ex2(M0 - M);
            const float fa = xa.y <= 0.f ? 0.f : ex2(xa.x - M), fb = xb.y <= 0.f ? 0.f : ex2(xb.x - M);
            const float sum = (xa.y <= 0.f ? 0.f : xa.y * fa) + (xb.y <= 0.f ? 0.f : xb.y * fb) + (sum0 <= 0.f ? 0.f : sum0 * f0);
            const bool whole = !early && info.z + len == info.w;
            const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
            const float ga = unlift(xa.z, M) * inv, gb = unlift(xb.z, M) * inv;
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
        if (FIRST && idle) zero_idle_rows_by<kUmmaPages, kUmmaPad>(p, HD, warp, kSoft / 32);
    }
    return ok;
}

// FIRST: every share's first window. Otherwise the others.
template <int HD, bool FIRST>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_kv8_umma(const __grid_constant__ CUtensorMap tmK, const Kv8Params p) {
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
        if (p.cut[gridDim.x].x <= kUmmaUnits || p.cut[blockIdx.x].z < 0) return;
    }
    if (tid == 0) {
        s_abort = 0;
        s_issued = Issued{0, 0, 0};
        init_bars<HD>(bars, p.stall);
    }
    if (warp == kWarpS) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    bool idle, ok = true;
    if constexpr (FIRST) {
        const int n = gather_units<kThreads, kUmmaPages, kUmmaPad, kUmmaUnits>(p, kUmmaLeast, 0, s_info, s_tile, &s_win, idle);
        tc_fence_after_sync();
        ok = attend_window<HD, true>(tmK, p, sm, n, &s_win, idle, &s_abort, &s_issued);
    } else {
        for (int w = 1;; ++w) {
            const int n = gather_units<kThreads, kUmmaPages, kUmmaPad, kUmmaUnits>(p, kUmmaLeast, w, s_info, s_tile, &s_win, idle);
            if (w == 1) tc_fence_after_sync();
            ok = attend_window<HD, false>(tmK, p, sm, n, &s_win, false, &s_abort, &s_issued);
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
            for (int i = max(0, s_issued.k - kTurns); i < s_issued.k; ++i) last(bars, i);
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
int launch_hd(const CUtensorMap& tk, const Kv8Params& p, const Plan& a, cudaStream_t s) {
    constexpr auto first = k_attn_kv8_umma<HD, true>, rest = k_attn_kv8_umma<HD, false>;
    constexpr int smem = Layout<HD>::kBytes;
    int rc = allow_smem<first>(a.dev, smem);
    if (rc != PE_OK) return rc;
    PE_CUDA_TRY(launch_ex(first, dim3(a.grid), dim3(kThreads), smem, s, false, tk, p));
    if (a.most <= static_cast<long long>(a.grid) * kUmmaUnits) return PE_OK;
    if ((rc = allow_smem<rest>(a.dev, smem)) != PE_OK) return rc;
    PE_CUDA_TRY(launch_ex(rest, dim3(a.grid), dim3(kThreads), smem, s, true, tk, p));
    return PE_OK;
}

}  // namespace

namespace kv8 {
static std::atomic<int> next_stall;   // of pe_test_stall_attention_kv8

int launch_umma(const Kv8Params& params, const Plan& a, int hd, cudaStream_t s) {
    CUtensorMap tk{};   // 64-wide heads: not read
    Kv8Params p = params;
    if (hd == 128) {
        const int rc = encode_tmap_codes(&tk, p.k_codes, static_cast<uint64_t>(p.num_pages) * p.nkv * kPage);
        if (rc != PE_OK) return rc;
    }
    if (next_stall.load(std::memory_order_relaxed) != 0) p.stall = next_stall.exchange(0);
    return hd == 128 ? launch_hd<128>(tk, p, a, s) : launch_hd<64>(tk, p, a, s);
}
}  // namespace kv8
}  // namespace pe

extern "C" int pe_test_stall_attention_kv8(int32_t barrier) {
    if (barrier < pe::kv8::kStallK || barrier > pe::kv8::kStallP) {
        pe::set_error("barrier must be 1, 2 or 3");
        return PE_ERR_ARG;
    }
    pe::kv8::next_stall.store(barrier);
    return PE_OK;
}
