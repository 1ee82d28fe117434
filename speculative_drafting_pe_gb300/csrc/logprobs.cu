// Log probabilities of given tokens, the entropy and the likeliest tokens of
// rows of logits (pe_token_logprobs). With y_i = (x_i - max x) / T and
// Z = sum_i e^{y_i}:
//
//   logprob(t) = y_t - ln Z,   H = ln Z - (1/Z) sum_i e^{y_i} y_i   (y_i <= 0: no cancellation)
//
// and the k largest x by (value, lower index first), their log probabilities
// from the same Z.
//
// One pass over a row: every thread keeps a running maximum of its own and its
// sums relative to it, rescaled once for a vector. A cluster of CTAs takes a
// row where rows are few; the first CTA joins their sums through distributed
// shared memory.
//
// The likeliest tokens cost the pass one store for kBatch vectors. Each thread's
// maximum is known behind it; of the warps' n-th largest ones (n times the warps
// make k) the k/n-th gives a bound that at least k values reach. Only cells (a
// thread's kBatch vectors, or a power of two as many) whose maximum reaches that
// bound can hold such values, a few dozen of thousands, and only theirs are read
// again, shared by all threads. (All vectors of the threads whose maximum
// reaches it, a sixth of a row's bytes at 20 alternatives, took 86 us where
// this takes 58.) Many values that equal the bound are looked for in index order
// until there are k.
//
// Memory bounds it in fp32 (1408 x 151936: 128 us, 98% of the copy rate; with 5
// alternatives 136, with 20 157), memory and the exponentials together in bf16
// (704 x 201088: 49 us, 85%; 54 and 58); a launch and the latency of a row's
// end where rows are few (one 5.2, 8 with 5 alternatives 8.5).
#include <cfloat>

#include "lowbit.cuh"

namespace pe {
namespace {

constexpr int kFew = 512, kMany = 256;      // threads of a CTA: rows that are split, rows with one each
constexpr int kMaxTop = 32;
constexpr float kMaxTemperature = 0x1p64f;
constexpr int kMaxCluster = 8;
constexpr int kMinSegment = 8 * kFew;   // values of a CTA at least, where a cluster shares a row
constexpr int kCand = 1024 + 64;            // values above the bound that are kept; see `collect`
constexpr int kTies = 512;                  // values equal to it that are
constexpr int kBatch = 4;                   // vectors of a thread whose loads are in flight together
constexpr int kCells = 8;                  // cells of a thread at most
constexpr unsigned kAll = 0xffffffffu;

struct LogprobParams {
    int R, V, k;
    const void* logits;
    long long ld;
    const int32_t* tokens;
    float c, inv_t;              // log2(e) / temperature, 1 / temperature
    float* logprobs;
    float* entropy;
    int32_t* top_tokens;
    float* top_logprobs;
};

// orders like the values (-0 = 0), NaN below everything
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t u) {
    return u == 0u ? NAN : __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// In base 2, t_i = c x_i with c = log2(e) / T: sums relative to a maximum m of
// the t, z = sum 2^(t - m) and s = sum 2^(t - m) (t - m). m is rounded, but every
// difference with it is one rounding (the product is exact in fma).
struct Sums {
    float m, z, s;
};
constexpr float kSafe = -1e15f;       // values from here on: times c (2^64 at most) they and their differences stay finite
constexpr float kFloor = -FLT_MAX;   // the maximum of no value
constexpr float kFar = -1e30f;       // a difference below it is this one: its weight is 0, and 0 times it is not NaN
__device__ __forceinline__ void rescale(Sums& a, float m) {   // to a maximum m >= a.m
    const float d = fmaxf(a.m - m, kFar), f = exp2_fast(d);
    a.s = f * fmaf(d, a.z, a.s);
    a.z *= f;
    a.m = m;
}
__device__ __forceinline__ Sums join(Sums a, Sums b) {
    const float m = fmaxf(a.m, b.m);
    if (a.z != 0.f) rescale(a, m);
    if (b.z != 0.f) rescale(b, m);
    return Sums{m, a.z + b.z, a.s + b.s};
}
// of the first N lanes of a warp, in each of them
template <int N>
__device__ __forceinline__ Sums join_lanes(Sums a) {
    float m = a.m;
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    if (a.z != 0.f) rescale(a, m);
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        a.z += __shfl_xor_sync(kAll, a.z, o);
        a.s += __shfl_xor_sync(kAll, a.s, o);
    }
    return Sums{m, a.z, a.s};
}

// 16 bytes of a row
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int kN = 4;
    __device__ static __forceinline__ void values(const uint4& x, float (&v)[4]) {
        v[0] = __uint_as_float(x.x);
        v[1] = __uint_as_float(x.y);
        v[2] = __uint_as_float(x.z);
        v[3] = __uint_as_float(x.w);
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int kN = 8;
    __device__ static __forceinline__ void values(const uint4& x, float (&v)[8]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};

// Values v of a row, the largest of which goes into `best`.
template <int N>
__device__ __forceinline__ void add(Sums& a, float& best, const float (&v)[N], float c) {
    float top = v[0], low = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, v[i]), low = fminf(low, v[i]);
    best = fmaxf(best, top);
    // (a maximum of -inf stays the floor; the lowest value may leave fp32's range here)
    rescale(a, fmaxf(a.m, top * c));
    if (N % 2 == 0 && low >= kSafe) {
        const uint64_t c2 = f2(c, c), m2 = f2(-a.m, -a.m);
        uint64_t z = f2(a.z, 0.f), s = f2(a.s, 0.f);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const uint64_t t = fma2(f2(v[2 * i], v[2 * i + 1]), c2, m2);
            const float2 y = unf2(t);
            const uint64_t e = f2(exp2_fast(y.x), exp2_fast(y.y));
            z = add2(z, e);
            s = fma2(e, t, s);
        }
        const float2 zz = unf2(z), ss = unf2(s);
        a.z = zz.x + zz.y;
        a.s = ss.x + ss.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // what lies far below adds nothing (-inf would be 0 * inf); a NaN goes on into both sums
            const float t = v[i] < kSafe ? (v[i] == -INFINITY ? kFar : fmaxf(fmaxf(v[i] * c, kFloor) - a.m, kFar)) : fmaf(v[i], c, -a.m);
            const float e = exp2_fast(t);
            a.z += e;
            a.s = fmaf(e, t, a.s);
        }
    }
}

// The segment [lo, hi) of a row as its threads share it: values up to the first
// 16-byte boundary and behind the last one singly, by threads 0 .. , and
// vectors in between, vector x by thread x mod kThreads.
template <typename T>
struct Segment {
    static constexpr int kN = Vec<T>::kN;
    const T* row;
    int lo, hi, body, vecs;   // body: first value of the vectors
    __device__ Segment(const T* r, int l, int h) : row(r), lo(l), hi(h) {
        const int off = static_cast<int>((reinterpret_cast<uintptr_t>(r + l) / sizeof(T)) % kN);
        body = min(h, l + (off == 0 ? 0 : kN - off));
        vecs = (h - body) / kN;
    }
    __device__ int tail() const { return body + vecs * kN; }
    // what of the values outside the vectors is thread t's (at most one at either end)
    __device__ int front(int t) const { return lo + t < body ? lo + t : -1; }
    __device__ int back(int t) const { return tail() + t < hi ? tail() + t : -1; }
};

// The cluster's barrier in two halves, for threads of a warp that may have parted.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1536 / kThreads) k_token_logprobs(const LogprobParams p) {
    constexpr int kN = Vec<T>::kN, kWarps = kThreads / 32;
    __shared__ Sums s_sums[kWarps];
    __shared__ uint32_t s_best[kWarps];
    __shared__ int s_count, s_equal, s_ties[kTies], s_scan[kWarps];
    __shared__ unsigned long long s_cand[kCand];
    __shared__ unsigned long long s_top[kMaxCluster * kMaxTop];   // this CTA's, in the first CTA everybody's
    __shared__ float4 s_all[kMaxCluster];                         // the parts' sums (m, z, s), in the first CTA
    __shared__ int s_work;
    extern __shared__ float s_cell[];                             // [kCells][kThreads] the cells' maxima
    uint16_t* s_list = reinterpret_cast<uint16_t*>(s_cell + kCells * kThreads);   // those that are read again
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int parts = static_cast<int>(gridDim.x), part = blockIdx.x, r = blockIdx.y + blockIdx.z * gridDim.y;
    if (r >= p.R) return;   // the whole cluster
    if (parts > 1) cluster_arrive();   // this CTA runs
    const float c = p.c;
    const T* row = static_cast<const T*>(p.logits) + static_cast<long long>(r) * p.ld;
    const int each = (p.V + parts - 1) / parts;
    const Segment<T> seg(row, min(p.V, part * each), min(p.V, part * each + each));

    const int token = tid == 0 && part == 0 ? p.tokens[r] : -1;   // (needed last, loaded first)

    Sums a{kFloor, 0.f, 0.f};
    float mine = -INFINITY;   // this thread's largest value
    const uint4* body = reinterpret_cast<const uint4*>(row + seg.body);
    int shift = 0;            // batches of a cell: 2^shift
    while ((seg.vecs / (kBatch * kThreads)) >> shift >= kCells) ++shift;
    const int last = (1 << shift) - 1;
    float cell = -INFINITY;
    int x = tid, batch = 0;
    for (; x + (kBatch - 1) * kThreads < seg.vecs; x += kBatch * kThreads, ++batch) {
        uint4 w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) w[i] = __ldg(body + x + i * kThreads);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float v[kN];
            Vec<T>::values(w[i], v);
            add(a, cell, v, c);
        }
        if ((batch & last) == last) {
            if (p.k > 0) s_cell[(batch >> shift) * kThreads + tid] = cell;
            mine = fmaxf(mine, cell);
            cell = -INFINITY;
        }
    }
    if (x < seg.vecs) {
        uint4 w[kBatch - 1];
#pragma unroll
        for (int i = 0; i < kBatch - 1; ++i)
            if (x + i * kThreads < seg.vecs) w[i] = __ldg(body + x + i * kThreads);
#pragma unroll
        for (int i = 0; i < kBatch - 1; ++i)
            if (x + i * kThreads < seg.vecs) {
                float v[kN];
                Vec<T>::values(w[i], v);
                add(a, cell, v, c);
            }
        ++batch;
    }
    // the last cell, where it is not a whole one (a row of few values: none at all)
    if (p.k > 0 && ((batch & last) != 0 || (batch > 0 && x < seg.vecs))) s_cell[((batch - 1) >> shift) * kThreads + tid] = cell;
    mine = fmaxf(mine, cell);
    const int cells = (batch + last) >> shift;   // of this thread
    {
        const int f = seg.front(tid), t = seg.back(tid);
        float v[1];
        if (f >= 0) { v[0] = static_cast<float>(row[f]); add(a, mine, v, c); }
        if (t >= 0) { v[0] = static_cast<float>(row[t]); add(a, mine, v, c); }
    }
    T asked = static_cast<T>(NAN);
    if (token >= 0 && token < p.V) asked = row[token];
    a = join_lanes<32>(a);
    if (lane == 0) s_sums[warp] = a;
    if (p.k > 0) {
        // the warp's largest maximum, or its n-th, where n of each warp make k
        uint32_t key = order_key(mine), best = __reduce_max_sync(kAll, key);
        for (int n = kWarps; n < p.k; n += kWarps) {
            if (lane == __ffs(__ballot_sync(kAll, key == best)) - 1) key = 0u;
            best = __reduce_max_sync(kAll, key);
        }
        if (lane == 0) s_best[warp] = best;
    }
    if (tid == 0) s_count = s_equal = s_work = 0;
    if (tid < kMaxTop) s_top[tid] = 0ull;   // (no key)
    __syncthreads();
    if (warp == kWarps - 1) {
        a = join_lanes<kWarps>(lane < kWarps ? s_sums[lane] : Sums{kFloor, 0.f, 0.f});
        __syncwarp();
        if (lane == 0) s_sums[0] = a;
    }

    const int want = min(p.k, seg.hi - seg.lo);
    if (want > 0) {
        // the bound: so many warps have n maxima that are as large
        const int n = (p.k + kWarps - 1) / kWarps, rank = (p.k + n - 1) / n;
        const uint32_t b = s_best[lane % kWarps];
        int ahead = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t o = s_best[w];
            ahead += o > b || (o == b && w < lane % kWarps);
        }
        const uint32_t bound = __shfl_sync(kAll, b, __ffs(__ballot_sync(kAll, ahead == rank - 1)) - 1);
        // values above the bound, and some that equal it, of the threads that have such
        const float level = key_value(bound);
        auto above = [&](float v, int i) {
            const int n = atomicAdd(&s_count, 1);
            if (n < kCand) s_cand[n] = (static_cast<unsigned long long>(order_key(v)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
        };
        auto equal_one = [&](int i) {
            if (*static_cast<volatile int*>(&s_equal) > kTies) return;
            const int n = atomicAdd(&s_equal, 1);
            if (n < kTies) s_ties[n] = i;
        };
        const bool has = mine >= level;
        if (has)
            for (int q = 0; q < cells; ++q)
                if (s_cell[q * kThreads + tid] >= level) s_list[atomicAdd(&s_work, 1)] = static_cast<uint16_t>(q * kThreads + tid);
        __syncthreads();
        const int each_vecs = kBatch << shift, work = s_work * each_vecs;
        for (int q = tid; q < work; q += kThreads) {
            const int of = q / each_vecs, id = s_list[of];
            const int y = id % kThreads + (id / kThreads * each_vecs + q - of * each_vecs) * kThreads;
            if (y >= seg.vecs) continue;
            float v[kN];
            Vec<T>::values(__ldg(body + y), v);
            unsigned more = 0, same = 0;
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                more |= v[e] > level ? 1u << e : 0u;
                same |= v[e] == level ? 1u << e : 0u;
            }
            const int at = seg.body + y * kN - 1;
            for (; more != 0; more &= more - 1) above(static_cast<float>(row[at + __ffs(more)]), at + __ffs(more));
            for (; same != 0; same &= same - 1) equal_one(at + __ffs(same));
        }
        if (has) {
            const int ends[2] = {seg.front(tid), seg.back(tid)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (ends[i] < 0) continue;
                const float v = static_cast<float>(row[ends[i]]);
                if (v > level) above(v, ends[i]);
                else if (v == level) equal_one(ends[i]);
            }
        }
        __syncthreads();
        const int equal = s_equal;
        int count = s_count;
        if (count > kCand) {
            // More than are kept (many of the row's largest values with one
            // thread): the largest keys one by one, each by a pass.
            unsigned long long below = ~0ull;
            for (int q = 0; q < want; ++q) {
                unsigned long long top = 0;
                for (int i = seg.lo + tid; i < seg.hi; i += kThreads) {
                    const unsigned long long key = (static_cast<unsigned long long>(order_key(static_cast<float>(row[i]))) << 32) |
                                                   (0xFFFFFFFFu - static_cast<uint32_t>(i));
                    if (key < below && key > top) top = key;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const unsigned long long other = __shfl_xor_sync(kAll, top, o);
                    top = other > top ? other : top;
                }
                __syncthreads();
                if (lane == 0) s_cand[warp] = top;
                __syncthreads();
                top = 0;
                for (int w = 0; w < kWarps; ++w) top = s_cand[w] > top ? s_cand[w] : top;
                if (tid == 0) s_top[q] = top;
                below = top;
            }
        } else {
            // All of the few that equal it stand with the others; many are looked
            // for in index order until there are enough. Where a row has fewer
            // numbers than alternatives are asked for, those that are NaN follow.
            const bool few = equal <= kTies && count + equal <= kCand;
            if (few && count < want) {
                for (int i = tid; i < equal; i += kThreads)
                    s_cand[count + i] = (static_cast<unsigned long long>(bound) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(s_ties[i]));
                count += equal;
                __syncthreads();
            }
            for (uint32_t at = few ? 0u : bound; count < want; at = 0u) {
                for (int i0 = seg.lo; i0 < seg.hi && count < want; i0 += kThreads) {
                    const int i = i0 + tid;
                    const bool tie = i < seg.hi && order_key(static_cast<float>(row[i])) == at;
                    const unsigned vote = __ballot_sync(kAll, tie);
                    if (lane == 0) s_scan[warp] = __popc(vote);
                    if (__syncthreads_or(tie)) {
                        int before = __popc(vote & ((1u << lane) - 1u)), all = 0;
                        for (int w = 0; w < kWarps; ++w) {
                            if (w < warp) before += s_scan[w];
                            all += s_scan[w];
                        }
                        if (tie && count + before < want)
                            s_cand[count + before] = (static_cast<unsigned long long>(at) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
                        count = min(want, count + all);
                    }
                    __syncthreads();
                }
                if (at == 0u) break;
            }
            // each key to its rank
            for (int i = tid; i < count; i += kThreads) {
                const unsigned long long key = s_cand[i];
                int ahead = 0;
#pragma unroll 8
                for (int q = 0; q < count; ++q) ahead += s_cand[q] > key;
                if (ahead < want) s_top[ahead] = key;
            }
        }
    }
    __syncthreads();

    // the first CTA of the cluster joins the parts
    if (parts > 1) {
        cluster_wait();
        if (part > 0) {
            const uint32_t sums = dsmem_addr(smem_u32(&s_all[part]), 0), top = dsmem_addr(smem_u32(s_top + part * kMaxTop), 0);
            if (tid == 0) {
                dsmem_st2(sums, s_sums[0].m, s_sums[0].z);
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(sums + 8), "f"(s_sums[0].s) : "memory");
            }
            if (p.k > 0 && tid < kMaxTop) {
                const unsigned long long key = s_top[tid];
                asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(top + tid * 8), "l"(key) : "memory");
            }
        }
        cluster_arrive();
        cluster_wait();
        if (part > 0) return;
    }
    Sums sum = s_sums[0];
    for (int q = 1; q < parts; ++q) sum = join(sum, Sums{s_all[q].x, s_all[q].y, s_all[q].z});
    // NaN where the row has no probability: none above -inf, an infinity, a NaN
    constexpr float kLn2 = 0.69314718055994531f;
    const float log_z = sum.z > 0.f ? log2f(sum.z) : NAN;
    auto logprob = [&](float x) {
        if (x < kSafe && sum.m >= kSafe) return x * p.inv_t - (sum.m + log_z) * kLn2;   // x c may leave fp32's range
        return ((x < kSafe ? fmaxf(x * c, kFloor) - sum.m : fmaf(x, c, -sum.m)) - log_z) * kLn2;
    };
    if (tid == 0) {
        p.logprobs[r] = logprob(static_cast<float>(asked));
        if (p.entropy != nullptr) p.entropy[r] = (log_z - sum.s / sum.z) * kLn2;
    }
    if (p.k == 0) return;
    // Every part's keys are in order: a key's rank is its place in its own part
    // and what is ahead of it in each other one, which a lane of `parts` looks up.
    for (int i0 = 0; i0 < parts * p.k; i0 += kThreads / parts) {
        const int i = i0 + tid / parts, q = tid % parts, from = i / p.k, at = i - from * p.k;
        const bool there = from < parts;
        const unsigned long long key = there ? s_top[from * kMaxTop + at] : 0ull;
        int ahead = at;
        if (q != from) {
            const unsigned long long* of = s_top + q * kMaxTop;
            ahead = 0;
#pragma unroll
            for (int step = kMaxTop / 2; step > 0; step /= 2)
                if (of[ahead + step - 1] > key) ahead += step;
            ahead += of[ahead] > key;
        }
        for (int o = 1; o < parts; o <<= 1) ahead += __shfl_xor_sync(kAll, ahead, o);
        if (!there || key == 0ull || ahead >= p.k || q != 0) continue;
        const long long to = static_cast<long long>(r) * p.k + ahead;
        p.top_tokens[to] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
        p.top_logprobs[to] = logprob(key_value(static_cast<uint32_t>(key >> 32)));
    }
}

template <typename T, int kThreads>
int launch(const LogprobParams& p, int parts, int dev, cudaStream_t s) {
    if (p.k > 0) {
        const int rc = allow_smem<k_token_logprobs<T, kThreads>>(dev, kCells * kThreads * 6);
        if (rc != PE_OK) return rc;
    }
    cudaLaunchConfig_t cfg = {};
    const unsigned rows_y = static_cast<unsigned>(p.R < 32768 ? p.R : 32768);
    cfg.gridDim = dim3(parts, rows_y, (p.R + rows_y - 1) / rows_y);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.dynamicSmemBytes = p.k > 0 ? kCells * kThreads * 6 : 0;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    PE_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_token_logprobs<T, kThreads>, p));
    return PE_OK;
}

}  // namespace
}  // namespace pe

using namespace pe;

extern "C" int pe_token_logprobs(int32_t R, int32_t V, int32_t dtype, const void* logits, int64_t ld,
                                 const int32_t* tokens, float temperature, float* logprobs, float* entropy,
                                 int32_t top, int32_t* top_tokens, float* top_logprobs, void* stream) {
    if (R < 1 || V < 1) { set_error("R and V must be >= 1"); return PE_ERR_ARG; }
    if (dtype != PE_DTYPE_BF16 && dtype != PE_DTYPE_FP32) { set_error("logits must be bf16 or fp32"); return PE_ERR_ARG; }
    if (top < 0 || top > kMaxTop || top > V) { set_error("top must lie in 0..32 and not exceed V"); return PE_ERR_ARG; }
    if (R > (1 << 30) || V > (1 << 30)) { set_error("R and V must be at most 2^30"); return PE_ERR_ARG; }
    const float c = 1.4426950408889634f / temperature;
    if (!(temperature > 0.f && temperature <= kMaxTemperature && c <= kMaxTemperature)) {
        set_error("temperature must lie in 2^-63 .. 2^64");
        return PE_ERR_ARG;
    }
    if (!logits || !tokens || !logprobs || (top > 0 && (!top_tokens || !top_logprobs))) {
        set_error("null tensor argument");
        return PE_ERR_ARG;
    }
    if (ld < V && ld != 0) { set_error("row stride must be at least V, or 0"); return PE_ERR_ARG; }
    if (reinterpret_cast<uintptr_t>(logits) % (dtype == PE_DTYPE_BF16 ? 2 : 4) != 0 ||
        ((reinterpret_cast<uintptr_t>(logprobs) | reinterpret_cast<uintptr_t>(entropy) | reinterpret_cast<uintptr_t>(tokens) |
          reinterpret_cast<uintptr_t>(top_tokens) | reinterpret_cast<uintptr_t>(top_logprobs)) & 3u) != 0) {
        set_error("tensors must be aligned to their elements");
        return PE_ERR_ARG;
    }
    int dev = 0, sms = 0;
    const int rc = current_device(&dev, &sms);
    if (rc != PE_OK) return rc;
    LogprobParams p{R, V, top, logits, ld, tokens, c, 1.f / temperature, logprobs, entropy, top_tokens, top_logprobs};
    // a cluster to a row while rows alone leave multiprocessors idle
    int parts = 1;
    while (parts < kMaxCluster && static_cast<long long>(R) * parts < 2ll * sms && V / (2 * parts) >= kMinSegment) parts *= 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Small CTAs once there are rows for most of them, so that what a row does behind its last value (a few
    // dependent reads) falls into others' streaming: 704 rows of 201088 bf16, 20 alternatives, 58 us for 66 with
    // large ones; 456 rows 43 for 38, and 36 for 31 without alternatives.
    if (parts == 1 && R >= 4 * sms && V >= kMinSegment)
        return dtype == PE_DTYPE_BF16 ? launch<__nv_bfloat16, kMany>(p, parts, dev, s) : launch<float, kMany>(p, parts, dev, s);
    return dtype == PE_DTYPE_BF16 ? launch<__nv_bfloat16, kFew>(p, parts, dev, s) : launch<float, kFew>(p, parts, dev, s);
}
