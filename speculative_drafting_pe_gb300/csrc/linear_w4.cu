// y = x W^T for few token rows and 4-bit weights (pe_linear_w4): codes two to
// a byte, a scale and optionally a zero point for each group of 32, 64 or 128
// columns.
//
//   y[n, m] = sum_g s[m, g] * sum_{k in g} (c[m, k] - z[m, g]) x[n, k]
//
// The inner sum runs on the tensor cores over the whole numbers c - z, which
// fp16 holds exactly; the scale multiplies the group's fp32 sum, so no weight
// is ever rounded.
//
// Bound by the weight bytes, so a code has to cost few instructions. Under
// fp16's exponent of 1024 a nibble in the low four bits is 1024 + c, in the
// next four 1024 + 16 c: one AND-OR sets two of them apart, one subtraction or
// fused multiply-add makes them c - z, five or so instructions for four codes.
// (Bare nibbles as fp16 subnormals need no arithmetic at all, but the tensor
// cores align the products by the operands' exponents, so beside a large x
// the other products lost up to ten bits.) x is laid out once per CTA in
// shared memory in the order in which the nibbles come out, as fp16 shifted by
// a power of two per row and 256 columns so that the largest value lies in
// [2^14, 2^15): bf16 values down to 2^-28 of that stay exact.
//
// A warp owns 16 weight rows (the MMA's M; the token rows are N) and walks
// their columns 256 at a time, kStages blocks ahead, through asynchronous
// copies of its own lanes (128-byte rows, the 16-byte chunks swizzled: the word
// reads are free of bank conflicts), so the warps never wait for each other
// while they stream. (TMA boxes of these 16 rows took some 150 cycles each,
// 26 bytes/ns per SM: the LM head took 48 us.) Where there are few rows, `ks`
// warps of a CTA share one set of 16, block by block, and their sums are added
// in order at the end.
//
// 151936 x 2048 (an LM head) with 8 rows: 32.5 us, 5.2 TB/s, 78% of the
// measured copy, with 11 rows 41 us: the instructions per code, and the MMAs
// twice, are next. Small matrices are bound by laying out x and by one block's
// latency after a launch: 2048 x 4096 and one row 4.1 us, 6144 x 2048 and 11
// rows 7.8 us.
#include <cuda_fp16.h>

#include "lowbit.cuh"

namespace pe {
namespace {

constexpr int kWarps = 16;                  // one CTA to an SM: x is laid out once for all of them
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;                  // LM head 32.4 us; two CTAs of 8 warps with three stages 34.4
constexpr int kRows = 16;                    // weight rows of a warp
constexpr int kCols = 256;                   // columns of a stage
constexpr int kStageBytes = kRows * kCols / 2;

struct W4Params {
    int M, N, Kd, dev;
    int ng;            // groups of a weight row
    int ks;            // warps that share 16 rows (1, 2, 4, 8, 16)
    int nb;            // 256-column blocks
    int xr;            // token rows in shared memory at a time
    int cb;            // blocks of x in shared memory at a time: all, or a multiple of ks
    int whole;         // a block's scales and zero points are whole aligned words
    const uint8_t* w;
    const void* scale;
    const uint8_t* zero;
    const __nv_bfloat16* x;
    long long ld_x;
    float* y;
    long long ld_y;
};

// (a & mask) | magic in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t magic) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(mask), "r"(magic));
    return r;
}
// In the order of the program, as the MMAs are: left to the compiler, the loads
// of later steps moved up, and the LM head took 38 instead of 34 us.
template <int OFF>
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1+%2];" : "=r"(r) : "r"(at), "n"(OFF));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at));
    return r;
}
__device__ __forceinline__ __half2 h2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }
__device__ __forceinline__ uint32_t u32(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }

template <int GROUP, int NT>
struct W4Smem {
    static constexpr int kN = NT * 8;
    // x row pitch: consecutive rows half the banks apart
    __host__ __device__ static constexpr int pitch(int cb) { return cb * kCols * 2 + 64; }
    static constexpr int kX = kWarps * kStages * kStageBytes;
    __host__ __device__ static constexpr int up(int cb, int xr) { return kX + xr * pitch(cb); }   // xr: rows held
    __host__ __device__ static constexpr int red(int cb, int xr) { return up(cb, xr) + cb * kN * 4; }
    __host__ __device__ static constexpr int bytes(int cb, int xr) { return red(cb, xr) + kWarps * kRows * kN * 4 + 1024; }
};

// Blocks [b0, b0 + cb) of the token rows into shared memory: fp16 in code
// order, and for each row and block the factor that undoes its shift. A warp
// per (row, block), kBatch of them in flight.
template <int GROUP, int NT>
__device__ void load_x(const W4Params& p, uint8_t* sm, int b0, int n0) {
    using L = W4Smem<GROUP, NT>;
    constexpr int kBatch = 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* s_up = reinterpret_cast<float*>(sm + L::up(p.cb, p.xr));
    const int rows = min(L::kN, p.N - n0), items = min(p.cb, p.nb - b0) * rows;
    for (int i0 = warp; i0 < items; i0 += kWarps * kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * kWarps, n = n0 + i % rows, k = (b0 + i / rows) * kCols + lane * 8;
            v[j] = make_uint4(0u, 0u, 0u, 0u);
            if (i < items && k < p.Kd)
                v[j] = *reinterpret_cast<const uint4*>(p.x + static_cast<long long>(n) * p.ld_x + k);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * kWarps;
            if (i >= items) break;
            const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
            uint32_t top = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) top = max(top, max((w[q] << 16) & 0x7FFF0000u, w[q] & 0x7FFF0000u));
            top = __reduce_max_sync(0xffffffffu, top);
            const int E = min(max(static_cast<int>(top >> 23), 15), 254);
            const float down = __uint_as_float(static_cast<uint32_t>(268 - E) << 23);   // 2^(141 - E)
            const int r = i % rows, blk = i / rows;
            if (lane == 0) s_up[blk * L::kN + r] = __uint_as_float(static_cast<uint32_t>(E - 14) << 23);   // 2^(E - 141)
            float f[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f[2 * q] = __uint_as_float(w[q] << 16) * down;
                f[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u) * down;
            }
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = u32(__floats2half2_rn(f[q], f[q + 4]));
            *reinterpret_cast<uint4*>(sm + L::kX + r * L::pitch(p.cb) + (blk * kCols + lane * 8) * 2) =
                make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Scales and zero points of one block of a weight row.
template <int GROUP, typename S, bool ZERO>
struct Groups {
    static constexpr int kN = kCols / GROUP;
    static constexpr int kWords = kN * static_cast<int>(sizeof(S)) / 4;   // 1, 2, 4 or 8
    uint32_t scale[kWords];
    uint32_t zero[kN > 4 ? 2 : 1];

    __device__ __forceinline__ void load(const W4Params& p, int row, int kb) {
        const size_t at = static_cast<size_t>(row) * p.ng + kb * kN;
        const S* from = static_cast<const S*>(p.scale) + at;
        const uint8_t* z = p.zero + at;
        if (p.whole) {
            if constexpr (kWords == 1) {
                scale[0] = *reinterpret_cast<const uint32_t*>(from);
            } else if constexpr (kWords == 2) {
                const uint2 v = *reinterpret_cast<const uint2*>(from);
                scale[0] = v.x; scale[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < kWords / 4; ++i) {
                    const uint4 v = reinterpret_cast<const uint4*>(from)[i];
                    scale[4 * i] = v.x; scale[4 * i + 1] = v.y; scale[4 * i + 2] = v.z; scale[4 * i + 3] = v.w;
                }
            }
            if constexpr (ZERO) {
                if constexpr (kN == 2) zero[0] = *reinterpret_cast<const uint16_t*>(z);
                else if constexpr (kN == 4) zero[0] = *reinterpret_cast<const uint32_t*>(z);
                else {
                    const uint2 v = *reinterpret_cast<const uint2*>(z);
                    zero[0] = v.x; zero[kN > 4 ? 1 : 0] = v.y;
                }
            }
        } else {   // one by one; groups past the row's end count nothing
#pragma unroll
            for (int i = 0; i < kWords; ++i) scale[i] = 0u;
            zero[0] = zero[kN > 4 ? 1 : 0] = 0u;
#pragma unroll
            for (int q = 0; q < kN; ++q) {
                if (kb * kN + q >= p.ng) break;
                if constexpr (sizeof(S) == 4) scale[q] = *reinterpret_cast<const uint32_t*>(from + q);
                else scale[q / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(from + q)) << (16 * (q & 1));
                if constexpr (ZERO) zero[q / 4] |= static_cast<uint32_t>(z[q]) << (8 * (q & 3));
            }
        }
    }
    __device__ __forceinline__ float s(int q) const {
        if constexpr (sizeof(S) == 4) return __uint_as_float(scale[q]);
        else return __uint_as_float((q & 1) ? scale[q / 2] & 0xFFFF0000u : scale[q / 2] << 16);
    }
    __device__ __forceinline__ uint32_t z(int q) const { return ZERO ? (zero[q / 4] >> (8 * (q & 3))) & 0xFFu : 8u; }
};

// ZERO: zero points are given (8 otherwise)
template <int GROUP, int NT, typename S, bool ZERO>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_w4(const W4Params p) {
    using L = W4Smem<GROUP, NT>;
    using GR = Groups<GROUP, S, ZERO>;
    constexpr int kSub = GROUP / 32;         // 32-column steps of a group
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int ks = p.ks, wk = warp % ks, wt = warp / ks, per = kWarps / ks;
    const int n0 = blockIdx.y * L::kN;
    uint8_t* ring = sm + warp * kStages * kStageBytes;
    const float* s_up = reinterpret_cast<const float*>(sm + L::up(p.cb, p.xr));
    float* s_red = reinterpret_cast<float*>(sm + L::red(p.cb, p.xr));
    const int tiles = (p.M + kRows - 1) / kRows;
    const int iters = (tiles + per - 1) / per;

    // this warp's blocks in order: (row tile, wk), (row tile, wk + ks), ...,
    // then the next row tile; the copies run ahead of the sums. Rows past the
    // last one are copies of it that are never stored; what stands in columns
    // past the row's end meets an x of 0.
    const uint64_t policy = l2_policy_evict_first();
    const int half = p.Kd / 2, c8 = lane & 7, r4 = lane >> 3;   // row bytes; this lane's chunk, and its first row of four
    const uint32_t ring_at = smem_u32(ring) + r4 * 128;
    int f_it = blockIdx.x, f_kb = wk;
    const uint8_t* rows[4];   // of the tile being fetched
    auto turn_to = [&](int it) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            rows[j] = p.w + static_cast<size_t>(min((it * per + wt) * kRows + r4 + 4 * j, p.M - 1)) * half + c8 * 16;
    };
    turn_to(f_it);
    const uint32_t to0 = ring_at + ((c8 ^ r4) << 4), to1 = ring_at + ((c8 ^ (r4 + 4)) << 4);
    auto fetch = [&](int st) {   // the next block of the list; a group of copies even at its end
        if (f_kb >= p.nb) {
            f_it += gridDim.x;
            f_kb = wk;
            if (f_it < iters) turn_to(f_it);
        }
        const int col = f_kb * (kCols / 2);
        if (f_it < iters && col + c8 * 16 < half) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(((j & 1) ? to1 : to0) + st * kStageBytes + j * 512),
                             "l"(rows[j] + col), "l"(policy)
                             : "memory");
        }
        f_kb += ks;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) fetch(s);

    auto load_groups = [&](GR (&o)[2], int it, int kb) {
#pragma unroll
        for (int h = 0; h < 2; ++h) o[h].load(p, min((it * per + wt) * kRows + g + 8 * h, p.M - 1), kb);
    };

    const uint32_t wr0 = smem_u32(ring) + g * 128 + t * 4 + (g << 4);
    // columns of the MMA without a token row read the last one's again
    uint32_t xr0[NT];
#pragma unroll
    for (int a = 0; a < NT; ++a) xr0[a] = smem_u32(sm + L::kX) + min(a * 8 + g, p.xr - 1) * L::pitch(p.cb) + t * 16;
    const uint32_t low = 0x000F000Fu, high = 0x00F000F0u, magic = 0x64006400u;
    int st = 0;
    const int chunks = (p.nb + p.cb - 1) / p.cb;
    GR next[2];   // of rows g and g + 8
    if (wk < p.nb) load_groups(next, blockIdx.x, wk);
    for (int it = blockIdx.x; it < iters; it += gridDim.x) {
        const int tile = it * per + wt;
        const bool mine = tile < tiles;
        const int m[2] = {tile * kRows + g, tile * kRows + g + 8};
        float acc[NT][4];
#pragma unroll
        for (int a = 0; a < NT; ++a) acc[a][0] = acc[a][1] = acc[a][2] = acc[a][3] = 0.f;
        for (int c = 0; c < chunks; ++c) {
            if (chunks > 1 || it == static_cast<int>(blockIdx.x)) {
                __syncthreads();
                load_x<GROUP, NT>(p, sm, c * p.cb, n0);
                __syncthreads();
            }
            if (!mine) continue;
            const int end = min(p.nb, (c + 1) * p.cb);
            for (int kb = c * p.cb + wk; kb < end; kb += ks) {
                const GR now[2] = {next[0], next[1]};
                // the next block's scales are on their way during this one
                if (kb + ks < p.nb) load_groups(next, it, kb + ks);
                else if (it + static_cast<int>(gridDim.x) < iters) load_groups(next, it + gridDim.x, wk);
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
                __syncwarp();
                // word t of chunk i of row g stands at chunk i ^ g
                float sum[NT][4];   // the block's, relative to x's shift
#pragma unroll
                for (int a = 0; a < NT; ++a) sum[a][0] = sum[a][1] = sum[a][2] = sum[a][3] = 0.f;
                const uint32_t wr = wr0 + st * kStageBytes, xo = (kb - c * p.cb) * (kCols * 2);
#pragma unroll
                for (int q = 0; q < GR::kN; ++q) {
                    __half2 z1[2], z16[2];   // 1024 + z, and -(64 + z)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        z1[h] = h2(0x64006400u + now[h].z(q) * 0x00010001u);
                        z16[h] = __hsub2(h2(0x63806380u), z1[h]);   // 960 - (1024 + z)
                    }
                    float part[NT][4];
#pragma unroll
                    for (int a = 0; a < NT; ++a) part[a][0] = part[a][1] = part[a][2] = part[a][3] = 0.f;
#pragma unroll
                    for (int u = 0; u < kSub; ++u) {
                        const int i = q * kSub + u;
                        uint32_t lo[4], hi[4];
                        const uint32_t at = wr ^ (i << 4);
                        const uint32_t word[2] = {lds32<0>(at), lds32<8 * 128>(at)};
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t w = word[h], v = w >> 8;
                            lo[h] = u32(__hsub2(h2(and_or(w, low, magic)), z1[h]));
                            lo[2 + h] = u32(__hfma2(h2(and_or(w, high, magic)), h2(0x2C002C00u), z16[h]));
                            hi[h] = u32(__hsub2(h2(and_or(v, low, magic)), z1[h]));
                            hi[2 + h] = u32(__hfma2(h2(and_or(v, high, magic)), h2(0x2C002C00u), z16[h]));
                        }
#pragma unroll
                        for (int a = 0; a < NT; ++a) {
                            const uint4 xv = lds128(xr0[a] + xo + i * 64);
                            mma_f16(part[a], lo, xv.x, xv.y);
                            mma_f16(part[a], hi, xv.z, xv.w);
                        }
                    }
#pragma unroll
                    for (int a = 0; a < NT; ++a)
#pragma unroll
                        for (int j = 0; j < 4; ++j) sum[a][j] = fmaf(now[j >> 1].s(q), part[a][j], sum[a][j]);
                }
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    const float2 up = *reinterpret_cast<const float2*>(s_up + (kb - c * p.cb) * L::kN + a * 8 + 2 * t);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[a][j] = fmaf(sum[a][j], (j & 1) ? up.y : up.x, acc[a][j]);
                }
                __syncwarp();
                fetch(st);
                st = st + 1 == kStages ? 0 : st + 1;
            }
        }
        if (ks > 1) {
            __syncthreads();   // the last tile's sums have been read
#pragma unroll
            for (int a = 0; a < NT; ++a)
                *reinterpret_cast<float4*>(s_red + ((warp * NT + a) * 32 + lane) * 4) =
                    make_float4(acc[a][0], acc[a][1], acc[a][2], acc[a][3]);
            __syncthreads();
            if (wk == 0) {
                for (int w = 1; w < ks; ++w)
#pragma unroll
                    for (int a = 0; a < NT; ++a) {
                        const float4 v = *reinterpret_cast<const float4*>(s_red + (((warp + w) * NT + a) * 32 + lane) * 4);
                        acc[a][0] += v.x;
                        acc[a][1] += v.y;
                        acc[a][2] += v.z;
                        acc[a][3] += v.w;
                    }
            }
        }
        if (wk == 0 && mine) {
#pragma unroll
            for (int a = 0; a < NT; ++a)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = n0 + a * 8 + 2 * t + (j & 1), mm = m[j >> 1];
                    if (n < p.N && mm < p.M) p.y[static_cast<long long>(n) * p.ld_y + mm] = acc[a][j];
                }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Shared memory for x at most. Longer rows come in pieces, once for every tile
// of weight rows.
constexpr int kXBytes = 140 * 1024;
constexpr int kMaxSmem = 232448;             // of a block

template <int GROUP, int NT, typename S, bool ZERO>
int launch(W4Params p, int sms, cudaStream_t s) {
    using L = W4Smem<GROUP, NT>;
    const int tiles = (p.M + kRows - 1) / kRows;
    p.nb = (p.Kd + kCols - 1) / kCols;
    p.whole = p.ng % (kCols / GROUP) == 0 &&
              ((reinterpret_cast<uintptr_t>(p.scale) | reinterpret_cast<uintptr_t>(p.zero)) & 15u) == 0;
    p.xr = p.N < L::kN ? p.N : L::kN;
    const int fit = kXBytes / (p.xr * kCols * 2);
    p.cb = p.nb <= fit ? p.nb : fit / kWarps * kWarps;
    const int smem = L::bytes(p.cb, p.xr);
    // warps to a row tile: the rounds that the CTAs take, times a warp's blocks
    // in one and kRound blocks' worth of joining and starting anew (none: the LM
    // head with 8 rows took 45 us for 34, two: 40000 x 4096 with 16 rows 41 for 40)
    constexpr int kRound = 1;
    long long least = 0;
    int iters = 0;
    for (int ks = 1; ks <= kWarps && (ks == 1 || ks < 2 * p.nb); ks *= 2) {
        const int n = static_cast<int>((static_cast<long long>(tiles) * ks + kWarps - 1) / kWarps);
        const long long cost = static_cast<long long>((n + sms - 1) / sms) * ((p.nb + ks - 1) / ks + kRound);
        if (ks == 1 || cost <= least) {
            least = cost;
            p.ks = ks;
            iters = n;
        }
    }
    constexpr auto kern = k_linear_w4<GROUP, NT, S, ZERO>;
    const int rc = allow_smem<kern>(p.dev, kMaxSmem);
    if (rc != PE_OK) return rc;
    const dim3 grid(iters < sms ? iters : sms, (p.N + L::kN - 1) / L::kN);
    PE_CUDA_TRY(launch_ex(kern, grid, dim3(kThreads), smem, s, false, p));
    return PE_OK;
}

template <int GROUP, typename S>
int launch_nt(const W4Params& p, int sms, cudaStream_t s) {
    // eight rows at a time where sixteen, or as many as there are, do not fit
    // whole (2048 x 6144, 11 rows: 10.8 us, in two passes 13.7)
    const bool one = p.N <= 8 || static_cast<long long>(p.N < 16 ? p.N : 16) * ((p.Kd + kCols - 1) / kCols) > kXBytes / (kCols * 2);
    if (p.zero != nullptr) return one ? launch<GROUP, 1, S, true>(p, sms, s) : launch<GROUP, 2, S, true>(p, sms, s);
    return one ? launch<GROUP, 1, S, false>(p, sms, s) : launch<GROUP, 2, S, false>(p, sms, s);
}

template <typename S>
int launch_group(int group, const W4Params& p, int sms, cudaStream_t s) {
    if (group == 32) return launch_nt<32, S>(p, sms, s);
    if (group == 64) return launch_nt<64, S>(p, sms, s);
    return launch_nt<128, S>(p, sms, s);
}

}  // namespace
}  // namespace pe

using namespace pe;

extern "C" int pe_linear_w4(int32_t M, int32_t N, int32_t Kd, int32_t group, const uint8_t* w, int32_t scale_dtype,
                            const void* w_scale, const uint8_t* w_zero, const void* x, int64_t ld_x, float* y,
                            int64_t ld_y, void* stream) {
    if (!w || !w_scale || !x || !y) { set_error("null tensor argument"); return PE_ERR_ARG; }
    if (M < 1 || N < 1 || Kd < 32 || Kd % 32 != 0) {
        set_error("need M, N >= 1 and Kd a positive multiple of 32");
        return PE_ERR_ARG;
    }
    if (group != 32 && group != 64 && group != 128) { set_error("group must be 32, 64 or 128"); return PE_ERR_UNSUPPORTED; }
    if (scale_dtype != PE_DTYPE_BF16 && scale_dtype != PE_DTYPE_FP32) { set_error("scales are bf16 or fp32"); return PE_ERR_ARG; }
    if (ld_x < Kd || ld_x % 8 != 0 || ld_y < M) {
        set_error("ld_x must be a multiple of 8 and at least Kd, ld_y at least M");
        return PE_ERR_ARG;
    }
    if (((reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(x)) & 15u) != 0) {
        set_error("w and x must be 16-byte aligned");
        return PE_ERR_ARG;
    }
    const uintptr_t size = scale_dtype == PE_DTYPE_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(w_scale) % size != 0 || (reinterpret_cast<uintptr_t>(y) & 3u) != 0) {
        set_error("w_scale and y must be aligned to their elements");
        return PE_ERR_ARG;
    }
    if (M > 0x7FFFFFFF - 256 || N > 8 * 65535) { set_error("M or N too large"); return PE_ERR_ARG; }
    int dev = 0, sms = 0;
    const int rc = current_device(&dev, &sms);
    if (rc != PE_OK) return rc;
    W4Params p{};
    p.dev = dev;
    p.M = M;
    p.N = N;
    p.Kd = Kd;
    p.ng = (Kd + group - 1) / group;
    p.w = w;
    p.scale = w_scale;
    p.zero = w_zero;
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.ld_x = ld_x;
    p.y = y;
    p.ld_y = ld_y;
    return scale_dtype == PE_DTYPE_BF16 ? launch_group<__nv_bfloat16>(group, p, sms, static_cast<cudaStream_t>(stream))
                                        : launch_group<float>(group, p, sms, static_cast<cudaStream_t>(stream));
}
