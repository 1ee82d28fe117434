// The write side of the 4-bit paged KV cache (pe_kv4_append): new query and key
// rows are turned to their positions, keys and values become 4-bit codes with
// a scale and a base for each (entry, kv head), queries go back in bf16.
//
//   (a_i, b_i) = (x_i, x_{i+hd/2}) -> (a cos - b sin, b cos + a sin), angle p * theta^(-2i/hd)
//   base = bf16(min x), scale = bf16(max(max x - base, 0) / 15), code = rn((x - base) / scale) in 0..15
//
// over the values x of one head of one row. An entry's codes depend on its row
// alone, so an append never touches an entry that is there, and what is
// written does not depend on how the rows came in calls.
//
// The angle is p times a frequency that is held as a fraction of a turn in 64
// bits (rotation.h): the product's lower half is the turn's remainder for every
// position, to 2^-34 of a turn, without a double on the device (FP64 runs at a
// few operations a cycle and SM). Its first 24 bits go through sincospif, the
// rest is a first-order term.
//
// A CTA takes `block` rows of one request, a warp two heads of a row at a time
// (four 64-wide ones). A lane has four dimensions of the lower half of a head
// and the four that they turn with, two 8-byte loads, and kBatch such pairs in
// flight. The rows' sines and cosines are computed once, for all heads.
//
// Few rows take a launch and three dependent loads, length, page and row (one
// row 3.2 us, 32 x 8 rows of 32 + 2 * 4 128-wide heads 3.6). Prompts are bound by
// memory and issue slots: 8 x 2048 rows of 64 + 2 * 8 64-wide heads 58 us, 78% of
// the copy rate (77 with queries, keys and values in one loop), one prompt of
// 32768 112 us, 82%; 2240 rows in room for 16384, most of whose bytes are zeros,
// 27 us. One to two rows a CTA: with four 31 for 29, with eight 34.
#include <cmath>
#include <cuda_fp16.h>

#include "lowbit.cuh"
#include "rotation.h"

namespace pe {
namespace {

constexpr int kPage = 16;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBatch = 4;        // heads of a warp whose loads are in flight together
constexpr int kMaxBlock = 2;     // rows of a CTA (its items are counted for one or two)

struct AppendParams {
    int B, n_max, nq, nkv, block, max_pages, num_pages;
    const __nv_bfloat16* x[3];   // q, k, v
    long long ld[3];
    const int32_t* seq_lens;
    const int32_t* rows;
    const int32_t* positions;
    const int32_t* page_table;
    uint8_t* codes[2];
    uint32_t* params[2];         // scale in the low half, base in the high one
    __nv_bfloat16* q_out;
    long long ld_q_out;
    int32_t* status;
    int turn;                    // whether there is a rotation
    unsigned long long freq[64]; // turns per position, in 2^-64
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// four bf16 values
__device__ __forceinline__ void unpack4(const uint2& w, float* x) {
    x[0] = __uint_as_float(w.x << 16);
    x[1] = __uint_as_float(w.x & 0xFFFF0000u);
    x[2] = __uint_as_float(w.y << 16);
    x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

template <int HD>
__global__ void __launch_bounds__(kThreads) k_kv4_append(const __grid_constant__ AppendParams p) {
    constexpr int kHalf = HD / 2;
    constexpr int kLanes = HD / 8;          // lanes of a head
    constexpr int kPer = 32 / kLanes;       // heads that a warp takes at a time
    __shared__ float4 s_cs[kMaxBlock * kHalf / 2];   // (cos, sin) of two pairs
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // (requests in turn: of ragged ones, blocks of rows run beside blocks that only zero)
    const int b = blockIdx.x % p.B, j0 = blockIdx.x / p.B * p.block;
    const int S = p.seq_lens[b];
    const int n = p.rows != nullptr ? p.rows[b] : p.n_max;
    const int first = p.positions != nullptr ? p.positions[b] : S;
    int st = PE_REQ_OK;
    if (S < 0 || n < 0 || n > p.n_max || (p.turn && (first < 0 || first > 0x7FFFFFFF - n))) st = PE_REQ_BAD_INPUT;
    else if (static_cast<long long>(S) + n > static_cast<long long>(p.max_pages) * kPage) st = PE_REQ_CAPACITY;
    const int live = st == PE_REQ_OK ? n : 0;
    if (j0 >= live) {
        // No row of the block is live: its queries' places are zeroed, 16 bytes
        // a store where they are aligned, as one run where they are one (8
        // prompts of 6 to 2048 rows in room for 2048, most of whose bytes
        // these are: 36 us by the loop below, 29 so).
        if (j0 == 0 && tid == 0) p.status[b] = st;
        if (p.q_out == nullptr) return;
        int count = min(p.n_max, j0 + p.block) - j0, bytes = p.nq * HD * 2;
        if (p.ld_q_out * 2 == bytes) bytes *= count, count = 1;
        for (int j = 0; j < count; ++j) {
            uint8_t* row = reinterpret_cast<uint8_t*>(p.q_out + (static_cast<long long>(b) * p.n_max + j0 + j) * p.ld_q_out);
            if (reinterpret_cast<uintptr_t>(row) % 16 == 0)
#pragma unroll 4
                for (int x = tid * 16; x < bytes; x += kThreads * 16) *reinterpret_cast<uint4*>(row + x) = make_uint4(0u, 0u, 0u, 0u);
            else
                for (int x = tid * 8; x < bytes; x += kThreads * 8) *reinterpret_cast<uint2*>(row + x) = make_uint2(0u, 0u);
        }
        return;
    }

    // Items: a row's heads of one kind, kPer at a time. Queries first, then keys
    // and values, so that neither pays for the other's steps; a warp's first ones
    // are on their way before anything else.
    const int sub = lane / kLanes, l = lane % kLanes;
    const int end = min(p.n_max, j0 + p.block), there = min(end, live) - j0;   // rows that may be read
    const int of_q = (p.nq + kPer - 1) / kPer, of_kv = (p.nkv + kPer - 1) / kPer;
    const int q_items = of_q * (end - j0), kv_items = 2 * of_kv * there;
    const long long row0 = static_cast<long long>(b) * p.n_max + j0;
    auto load = [&](const __nv_bfloat16* x, bool ok, uint2 (&v)[2]) {
        v[0] = v[1] = make_uint2(0u, 0u);
        if (ok) {
            v[0] = *reinterpret_cast<const uint2*>(x);
            v[1] = *reinterpret_cast<const uint2*>(x + kHalf);
        }
    };
    const __nv_bfloat16* xq = p.x[0] + row0 * p.ld[0] + l * 4;
    auto load_q = [&](int t, uint2 (&v)[2]) {
        const int row = t >= of_q, head = (t - (row ? of_q : 0)) * kPer + sub;
        load(xq + (row ? p.ld[0] : 0) + head * HD, t < q_items && row < there && head < p.nq, v);
    };
    struct Item {
        int row, side, head;
    };
    auto kv_item = [&](int t) {
        Item it{t >= 2 * of_kv, 0, 0};
        t -= it.row ? 2 * of_kv : 0;
        it.side = t >= of_kv;
        it.head = (t - (it.side ? of_kv : 0)) * kPer + sub;
        return it;
    };
    auto load_kv = [&](int t, uint2 (&v)[2]) {
        const Item it = kv_item(t);
        const long long ld = it.side ? p.ld[2] : p.ld[1];
        load((it.side ? p.x[2] : p.x[1]) + (row0 + it.row) * ld + it.head * HD + l * 4, t < kv_items && it.head < p.nkv, v);
    };
    uint2 v[kBatch][2], kv[2];
    load_kv(warp, kv);
    if (warp < q_items)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) load_q(warp + i * kWarps, v[i]);

    if (p.turn)
        for (int x = tid; x < (end - j0) * kHalf; x += kThreads) {
            const int row = x / kHalf, i = x - row * kHalf;
            const unsigned long long turns = static_cast<unsigned long long>(static_cast<uint32_t>(first + j0 + row)) * p.freq[i];
            // the remainder in half turns, -1 .. 1: 24 bits, which are a float, and the rest
            const int32_t top = static_cast<int32_t>(turns >> 32) & ~0xFF;
            const float rest = static_cast<float>(static_cast<uint32_t>(turns >> 8)) * 0x1p-55f * 3.14159265358979f;
            float sn, cs;
            sincospif(static_cast<float>(top) * 0x1p-31f, &sn, &cs);
            reinterpret_cast<float2*>(s_cs)[x] = make_float2(fmaf(-rest, sn, cs), fmaf(rest, cs, sn));
        }
    // every page that the request's new rows need, before any of them is written
    const int32_t* table = p.page_table + static_cast<size_t>(b) * p.max_pages;
    int bad = 0;
    if (live > 0)
        for (int i = S / kPage + tid; i < (S + live + kPage - 1) / kPage; i += kThreads)
            bad |= table[i] < 0 || table[i] >= p.num_pages;
    if (__syncthreads_or(bad)) st = PE_REQ_BAD_PAGE;
    if (j0 == 0 && tid == 0) p.status[b] = st;
    const int rows = st == PE_REQ_OK ? live : 0;

    auto turn = [&](int row, float (&x)[8]) {
        const float4* cs = s_cs + (row * kHalf + l * 4) / 2;
        const float4 c0 = cs[0], c1 = cs[1];
        const float co[4] = {c0.x, c0.z, c1.x, c1.z}, si[4] = {c0.y, c0.w, c1.y, c1.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float lo = x[c], hi = x[4 + c];
            x[c] = fmaf(lo, co[c], -(hi * si[c]));
            x[4 + c] = fmaf(hi, co[c], lo * si[c]);
        }
    };
    __nv_bfloat16* to_q = p.q_out + row0 * p.ld_q_out + l * 4;
    for (int t0 = warp; t0 < q_items; t0 += kBatch * kWarps) {
        if (t0 != warp)
#pragma unroll
            for (int i = 0; i < kBatch; ++i) load_q(t0 + i * kWarps, v[i]);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int t = t0 + i * kWarps, row = t >= of_q, head = (t - (row ? of_q : 0)) * kPer + sub;
            if (t >= q_items || head >= p.nq) continue;
            float x[8];   // dimensions 4l .., then hd/2 + 4l ..
            unpack4(v[i][0], x);
            unpack4(v[i][1], x + 4);
            if (p.turn) turn(row, x);
            uint2 lo = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
            uint2 hi = make_uint2(pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
            if (j0 + row >= rows) lo = hi = make_uint2(0u, 0u);   // no row here
            __nv_bfloat16* to = to_q + (row ? p.ld_q_out : 0) + head * HD;
            *reinterpret_cast<uint2*>(to) = lo;
            *reinterpret_cast<uint2*>(to + kHalf) = hi;
        }
    }
    if (rows == 0) return;   // refused
    for (int t = warp; t < kv_items; t += kWarps) {
        if (t != warp) load_kv(t, kv);
        const Item it = kv_item(t);
        float x[8];
        unpack4(kv[0], x);
        unpack4(kv[1], x + 4);
        if (p.turn && it.side == 0) turn(it.row, x);
        float lo = x[0], hi = x[0], odd = x[0] - x[0];   // odd: NaN where a value is not finite
#pragma unroll
        for (int c = 1; c < 8; ++c) {
            lo = fminf(lo, x[c]);
            hi = fmaxf(hi, x[c]);
            odd += x[c] - x[c];
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        const unsigned who = __ballot_sync(0xffffffffu, odd != 0.f);
        if (it.head >= p.nkv) continue;
        uint32_t par = pack_bf16(0.f, lo);
        const float base = __uint_as_float(par & 0xFFFF0000u);
        // (base may be rounded up past the largest value: the entry is one value throughout)
        const float range = hi - base;
        par |= pack_bf16(fmaxf(range, 0.f) / 15.f, 0.f);
        const float scale = __uint_as_float(par << 16);
        uint32_t code[2] = {0u, 0u};
        if (((who >> (sub * kLanes)) & ((1u << kLanes) - 1u)) != 0u || !(fabsf(range) < INFINITY)) {
            par = 0x7FC07FC0u;   // the entry is NaN
        } else if (scale >= 0x1p-100f) {
            // the quotient with its rounding error put right, as a division has it
            const float inv = 1.f / scale;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float d = x[c] - base, near = d * inv;
                code[c >> 2] |= min(__float2uint_rn(fmaf(fmaf(-scale, near, d), inv, near)), 15u) << (4 * (c & 3));
            }
        } else if (scale > 0.f) {
#pragma unroll
            for (int c = 0; c < 8; ++c) code[c >> 2] |= min(__float2uint_rn((x[c] - base) / scale), 15u) << (4 * (c & 3));
        }
        const int e = S + j0 + it.row;
        const size_t at = (static_cast<size_t>(table[e / kPage]) * p.nkv + it.head) * kPage + e % kPage;
        uint8_t* to = (it.side == 0 ? p.codes[0] : p.codes[1]) + at * kHalf + l * 2;
        *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(code[0]);
        *reinterpret_cast<uint16_t*>(to + kHalf / 2) = static_cast<uint16_t>(code[1]);
        if (l == 0) (it.side == 0 ? p.params[0] : p.params[1])[at] = par;
    }
}

// The frequencies of a base and width, kept for the calls that follow with the same.
const unsigned long long* frequencies(float theta, int hd) {
    static thread_local float had_theta = 0.f;
    static thread_local int had_hd = 0;
    static thread_local unsigned long long freq[64];
    if (had_theta != theta || had_hd != hd) {
        rotation_turns(theta, hd, freq);
        had_theta = theta;
        had_hd = hd;
    }
    return freq;
}

}  // namespace
}  // namespace pe

using namespace pe;

extern "C" int pe_kv4_append(int32_t B, int32_t n_max, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                             const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                             float rope_theta, const int32_t* positions, const int32_t* seq_lens, const int32_t* rows,
                             const int32_t* page_table, int32_t max_pages, int32_t num_pages, uint8_t* k_codes,
                             uint8_t* v_codes, void* k_params, void* v_params, void* q_out, int64_t ld_q_out,
                             int32_t* status, void* stream) {
    const int nq = n_q_heads, nkv = n_kv_heads, hd = head_dim;
    if (B < 1 || n_max < 1 || nkv < 1 || nq < 0) { set_error("B, n_max and nkv must be >= 1, nq >= 0"); return PE_ERR_ARG; }
    if (hd != 64 && hd != 128) { set_error("head_dim must be 64 or 128"); return PE_ERR_UNSUPPORTED; }
    if (max_pages < 1 || num_pages < 1) { set_error("max_pages and num_pages must be >= 1"); return PE_ERR_ARG; }
    if (max_pages > 0x7FFFFFFF / kPage - 2 || n_max > 0x7FFFFFFF / kPage || nq > (1 << 20) || nkv > (1 << 20)) {
        set_error("max_pages * 16 and n_max must fit a signed 32-bit entry index, head counts 2^20");
        return PE_ERR_ARG;
    }
    if (!(rope_theta == 0.f || (rope_theta >= 1.f && rope_theta < INFINITY))) {
        set_error("rope_theta must be 0 (no rotation) or at least 1");
        return PE_ERR_ARG;
    }
    if (!k || !v || !seq_lens || !page_table || !k_codes || !v_codes || !k_params || !v_params || !status ||
        (nq > 0 && (!q || !q_out))) {
        set_error("null tensor argument");
        return PE_ERR_ARG;
    }
    const int64_t wq = static_cast<int64_t>(nq) * hd, wkv = static_cast<int64_t>(nkv) * hd;
    if (ld_k < wkv || ld_v < wkv || ld_k % 4 != 0 || ld_v % 4 != 0 ||
        (nq > 0 && (ld_q < wq || ld_q_out < wq || ld_q % 4 != 0 || ld_q_out % 4 != 0))) {
        set_error("row strides must be multiples of 4 and at least heads * head_dim");
        return PE_ERR_ARG;
    }
    const uintptr_t in = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
                         (nq > 0 ? reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_out) : 0);
    if ((in & 7u) != 0 || ((reinterpret_cast<uintptr_t>(k_codes) | reinterpret_cast<uintptr_t>(v_codes)) & 15u) != 0 ||
        ((reinterpret_cast<uintptr_t>(k_params) | reinterpret_cast<uintptr_t>(v_params)) & 15u) != 0) {
        set_error("q, k, v and q_out must be 8-byte aligned, the code and parameter arrays 16-byte aligned");
        return PE_ERR_ARG;
    }
    if ((nq > 0 && q_out == q && ld_q_out != ld_q) || status == seq_lens || (rows != nullptr && status == rows) ||
        (positions != nullptr && status == positions)) {
        set_error("q_out over q must have its row stride, status must be none of the inputs");
        return PE_ERR_ARG;
    }
    int dev = 0, sms = 0;
    const int rc = current_device(&dev, &sms);
    if (rc != PE_OK) return rc;
    AppendParams p{};
    p.B = B;
    p.n_max = n_max;
    p.nq = nq;
    p.nkv = nkv;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.x[0] = static_cast<const __nv_bfloat16*>(q);
    p.x[1] = static_cast<const __nv_bfloat16*>(k);
    p.x[2] = static_cast<const __nv_bfloat16*>(v);
    p.ld[0] = ld_q;
    p.ld[1] = ld_k;
    p.ld[2] = ld_v;
    p.seq_lens = seq_lens;
    p.rows = rows;
    p.positions = positions;
    p.page_table = page_table;
    p.codes[0] = k_codes;
    p.codes[1] = v_codes;
    p.params[0] = static_cast<uint32_t*>(k_params);
    p.params[1] = static_cast<uint32_t*>(v_params);
    p.q_out = nq > 0 ? static_cast<__nv_bfloat16*>(q_out) : nullptr;
    p.ld_q_out = ld_q_out;
    p.status = status;
    p.turn = rope_theta != 0.f;
    if (p.turn) {
        const unsigned long long* f = frequencies(rope_theta, hd);
        for (int i = 0; i < hd / 2; ++i) p.freq[i] = f[i];
    }
    // a row to a CTA while that fills the device but once
    p.block = static_cast<long long>(B) * n_max <= 8ll * sms ? 1 : kMaxBlock;
    const long long blocks = static_cast<long long>(B) * ((n_max + p.block - 1) / p.block);
    if (blocks > 0x7FFFFFFFll) { set_error("pe_kv4_append: too many rows for one call"); return PE_ERR_ARG; }
    auto kern = hd == 128 ? k_kv4_append<128> : k_kv4_append<64>;
    PE_CUDA_TRY(launch_ex(kern, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), false, p));
    return PE_OK;
}
