// attention.cuh -- what the kernels of qift_paged_attention share: which rows a block owns, which
// keys they see, and how partial results are laid down and joined.
//
// A row is one (token, query head).  Rows that share a kv head are handled together: row r of a
// row set is token r / G, head r % G of the group (G = q_heads / kv_heads).  Two kinds of row set:
//   own     the tokens of one sequence, against that sequence's own pages
//   prefix  the tokens of the whole batch, against the pages every sequence starts with, so that
//           those keys are read once for all
// Key positions count from the start of the sequence; the own pages hold positions prefix_len, ...
//
// Partial results of a row over a set S of keys, with u_j = scale log2(e) q.k_j:
//   M, L = sum_S 2^(u_j - M), O = sum_S 2^(u_j - M) v_j
// and any number of them join by M* = max M, L* = sum L 2^(M - M*), O* likewise.  An empty set has
// M = kNone, L = 0, and no O; a row with a NaN or infinity in q has L = NaN over any other, which stays one.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace qift {
namespace attn {

constexpr int kMaxKeys = 1 << 30;  // of a sequence, so that positions plus a block stay in 32 bits
// The first byte of dynamic shared memory at a multiple of ALIGN (which the declaration's own alignment does
// not ensure in every build); the launch asks for ALIGN bytes more.
template <int ALIGN>
__device__ __forceinline__ uint8_t* aligned(uint8_t* raw) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(raw));
    return raw + ((ALIGN - (at & (ALIGN - 1))) & (ALIGN - 1));
}

constexpr float kNone = -1e30f;  // finite, so that the difference of two of them is a number
// A key whose values are all zero (value scale 0) adds nothing to O, so only the sum bounds its weight: a step's
// weights of a row may sum to this much before the row's reference is raised.  A value scale below 2^kLeastScale
// counts as that much where it is (the smallest a row of binary16 values can have is 2^-24 / 7).  So weights stay below
// 2^48 without another raise, and the sum of 2^30 of them below 2^78: no sum, nor the join of any, overflows.
constexpr float kMostSum = 281474976710656.0f;  // 2^48
constexpr float kLeastScale = -28.0f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One sequence as the device sees it; offsets and lengths that contradict the call's sizes are cut
// so that no index leaves the caller's arrays.
struct Sequence {
    int64_t first;  // first token
    int q_len, kv_len;
};
__device__ __forceinline__ Sequence sequence(const AttentionArgs& a, int b) {
    Sequence s = {0, 0, 0};
    if (!QIFT_CK_RANGE(b, 1, a.batch)) return s;
    if (a.cu_q) {
        int64_t lo = a.cu_q[b], hi = a.cu_q[b + 1];
        lo = lo < 0 ? 0 : lo;
        hi = hi > a.tokens ? a.tokens : hi;
        s.first = lo;
        s.q_len = hi > lo ? (int)(hi - lo) : 0;
        if (s.q_len > a.max_q) s.q_len = a.max_q;
    } else {
        s.first = (int64_t)b * a.max_q;
        s.q_len = a.max_q;
    }
    const int n = a.kv_lens[b];
    s.kv_len = n < 0 ? 0 : n > kMaxKeys ? kMaxKeys : n;
    return s;
}

// The sequence a token belongs to, -1 if none: the last b with cu_q[b] <= token < cu_q[b + 1].
__device__ __forceinline__ int sequence_of(const AttentionArgs& a, int64_t token) {
    if (!a.cu_q) return (int)((uint32_t)token / (uint32_t)a.max_q);
    int lo = 0, hi = a.batch;  // first b in [lo, hi] with cu_q[b] > token
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (QIFT_CK_RANGE(mid, 1, a.batch) && a.cu_q[mid] > token) hi = mid;
        else lo = mid + 1;
    }
    const int b = lo - 1;
    return b >= 0 && token < a.cu_q[b + 1] ? b : -1;
}

// Position of a token in its sequence, -1 (it sees nothing) or, if it belongs to no sequence, -2: such rows are
// left out, since one that sees nothing would have every step of its block masked.
__device__ __forceinline__ int position_of(const AttentionArgs& a, int64_t token) {
    const int b = sequence_of(a, token);
    if (b < 0) return -2;
    const Sequence s = sequence(a, b);
    const int64_t p = (int64_t)s.kv_len - s.q_len + (token - s.first);
    return p < 0 ? -1 : (int)p;
}

// The blocks of STEP keys that rows at positions [pmin, pmax] can see, of a table that holds
// positions [base, base + capacity): first those that hold sinks, then those of the window.
// Step s is key block s (s < head) or s - head + main; keys at table index >= limit do not exist.
struct Range {
    int head, main, steps, limit;
    __device__ __forceinline__ int block(int s) const { return s < head ? s : main + (s - head); }
};
template <int STEP>
__device__ __forceinline__ Range visible(const AttentionArgs& a, int pmin, int pmax, int base, int64_t capacity) {
    Range r;
    int64_t hi = (int64_t)pmax + 1 - base;
    if (hi > capacity) hi = capacity;
    if (hi < 0) hi = 0;
    int64_t lo = a.window ? (int64_t)pmin - a.window + 1 : 0;
    if (lo < 0) lo = 0;
    int64_t sinks = lo < a.sinks ? lo : a.sinks;  // sinks in front of the window
    sinks -= base;
    if (sinks < 0) sinks = 0;
    if (sinks > hi) sinks = hi;
    lo -= base;
    if (lo < 0) lo = 0;
    r.limit = (int)hi;
    r.head = (int)((sinks + STEP - 1) / STEP);
    int64_t m = lo / STEP;
    if (m < r.head) m = r.head;
    const int64_t end = (hi + STEP - 1) / STEP;
    r.main = (int)m;
    r.steps = r.head + (end > m ? (int)(end - m) : 0);
    return r;
}

// Row tile x of a batch whose sequences differ much: tile `tile` of PER rows of sequence b.  Sequence b's tiles
// begin at floor(its first row / PER) + b, which leaves room for ceil(its rows / PER) of them before the next
// one's whatever the lengths are, and for all of them in tokens * G / PER + batch.  (A tile for each PER of
// the longest sequence's rows, of every sequence, would be mostly empty.)  False: no rows.
template <int PER>
__device__ __forceinline__ bool ragged_tile(const AttentionArgs& a, int64_t x, uint32_t G, int& b, int& tile) {
    auto start = [&](int s) {
        int64_t first = QIFT_CK_RANGE(s, 1, a.batch) ? a.cu_q[s] : 0;
        first = first < 0 ? 0 : first > a.tokens ? a.tokens : first;
        return first * G / PER + s;
    };
    int lo = 0, hi = a.batch;  // the last sequence that begins at x or before is in [lo, hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start(mid) <= x) lo = mid;
        else hi = mid;
    }
    const int64_t t = x - start(lo);
    b = lo;
    tile = (int)t;
    return t >= 0 && t * PER < (int64_t)sequence(a, lo).q_len * G;
}

cudaError_t launch_wide(const AttentionArgs& a, const Deal& d, cudaStream_t s);
constexpr int kWideRows = 256;  // rows of a block of the kernel for many rows
constexpr int kWideStep = 128;  // keys it takes at a time

__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// Two query values with an infinity made NaN (x 0 + x; any other value stays what it is).  An infinity times the
// codes of the keys a row sees may be -infinity for all of them, and the row would look like one that sees nothing;
// its softmax is not defined, so its scores are NaN, whatever the codes (also 0) are.
__device__ __forceinline__ uint32_t no_infinity(uint32_t x) {
    const __half2 v = *reinterpret_cast<const __half2*>(&x);
    const __half2 r = __hfma2(v, __float2half2_rn(0.0f), v);
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint4 no_infinity(uint4 x) {
    return make_uint4(no_infinity(x.x), no_infinity(x.y), no_infinity(x.z), no_infinity(x.w));
}
// Two two's-complement nibbles, 16 bits apart, as binary16: from bits 0-3 exactly, from bits 4-7
// plus 72 (1 x 2^6 with the nibble, its sign bit flipped, above the last four bits), or exactly.
// Mask and flip are one three-input operation each; it takes one immediate at most, so the constants
// are kept in registers (given as immediates, the compiler makes two operations of it).
struct Nibbles {
    uint32_t mask_lo, mask_hi, one_lo, one_hi;
    __device__ __forceinline__ Nibbles() {
        asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(mask_lo));
        asm volatile("mov.b32 %0, 0x00F000F0;" : "=r"(mask_hi));
        asm volatile("mov.b32 %0, 0x64086408;" : "=r"(one_lo));
        asm volatile("mov.b32 %0, 0x54805480;" : "=r"(one_hi));
    }
    __device__ __forceinline__ static uint32_t and_xor(uint32_t w, uint32_t m, uint32_t c) {
        uint32_t r;
        asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(w), "r"(m), "r"(c));  // (w & m) ^ c
        return r;
    }
    __device__ __forceinline__ uint32_t lo(uint32_t w) const { return sub2(and_xor(w, mask_lo, one_lo), one_lo); }
    __device__ __forceinline__ uint32_t hi72(uint32_t w) const { return and_xor(w, mask_hi, one_hi); }
    __device__ __forceinline__ uint32_t hi(uint32_t w) const { return sub2(hi72(w), one_hi); }
};

// Partial results: slot p of row (token, head): D floats of O and (M, L).
struct Parts {
    float* o;
    float2* ml;
    int slots;
};
__host__ __device__ inline Parts parts(const AttentionArgs& a, int slots) {
    Parts p;
    p.o = a.workspace;
    p.ml = reinterpret_cast<float2*>(a.workspace + (int64_t)a.tokens * a.q_heads * slots * a.head_dim);
    p.slots = slots;
    return p;
}

// Bounds-checked build: query values, result rows and partial results lie inside the caller's arrays.
__device__ __forceinline__ bool in_queries(const AttentionArgs& a, int64_t at, int count) {
    return QIFT_CK_RANGE(at, count, (a.tokens - 1) * a.q_stride + (int64_t)a.q_heads * a.head_dim);
}
__device__ __forceinline__ bool in_result(const AttentionArgs& a, int64_t row) {
    return QIFT_CK_RANGE(row, 1, a.tokens * a.q_heads);
}
__device__ __forceinline__ bool in_parts(const AttentionArgs& a, int slots, int64_t at) {
    return QIFT_CK_RANGE(at, 1, a.tokens * a.q_heads * slots) &&
           QIFT_CK_RANGE((at + 1) * a.head_dim * 4, 0, a.workspace_bytes) &&
           QIFT_CK_RANGE((a.tokens * a.q_heads * slots * a.head_dim + 2 * at) * 4, 8, a.workspace_bytes);
}
// ... and a table's entry in the table.
__device__ __forceinline__ bool in_table(const AttentionArgs& a, bool prefix, int64_t entry) {
    return QIFT_CK_RANGE(entry, 1, prefix ? ((int64_t)a.prefix_len + (1 << a.log_page) - 1) >> a.log_page : (int64_t)a.max_pages);
}

// Rotates a row held by a warp, D / 32 contiguous values a lane, by blocks of `block` (0: not).
template <int D>
__device__ __forceinline__ void row_hadamard(float (&v)[D / 32], int lane, int block, float norm) {
    if (block == 0) return;
    constexpr int E = D / 32;
#pragma unroll
    for (int h = 1; h < E; h <<= 1) {
        if (block <= h) break;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (i & h) continue;
            const float x = v[i], y = v[i + h];
            v[i] = x + y;
            v[i + h] = x - y;
        }
    }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        if (block <= E * m) break;
        const float sgn = (lane & m) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = __fmaf_rn(sgn, v[i], __shfl_xor_sync(0xffffffffu, v[i], m));
    }
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= norm;
}

// Normalise, rotate back, round once and store a finished row (a warp's).  M, L as above.
template <int D>
__device__ __forceinline__ void finish_row(const AttentionArgs& a, float (&v)[D / 32], float M, float L, int64_t token,
                                           int head, int lane) {
    constexpr int E = D / 32;
    const float inv = L == 0.0f ? 0.0f : __fdiv_rn(1.0f, L);
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= inv;
    row_hadamard<D>(v, lane, a.block, a.norm);
    if (!in_result(a, token * a.q_heads + head)) return;
    const int64_t at = (token * a.q_heads + head) * D + lane * E;
    if (a.f16) {
        __half2 h[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        __half* o = static_cast<__half*>(a.out) + at;
        if constexpr (E == 2) *reinterpret_cast<__half2*>(o) = h[0];
        else if constexpr (E == 4) *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(h);
        else *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(h);
    } else {
        float* o = static_cast<float*>(a.out) + at;
        if constexpr (E == 2) *reinterpret_cast<float2*>(o) = make_float2(v[0], v[1]);
        else
#pragma unroll
            for (int i = 0; i < E; i += 4)
                *reinterpret_cast<float4*>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
    if (a.lse && lane == 0)
        a.lse[token * a.q_heads + head] = L == 0.0f ? -INFINITY : 0.69314718056f * (M + log2f(L));
}

}  // namespace attn
}  // namespace qift
