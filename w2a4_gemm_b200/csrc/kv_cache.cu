// kv_cache.cu -- qift_append_kv and qift_gather_kv: rows written to, and read back from, a paged
// KV4 cache.
//
// "Qift: Shift-Friendly No-Zero W2 Post-Training Quantization for Rotated W2A4/KV4 LLM
// Inference" names KV4; the cache holds the rows of qift_quantize_kv, one per token and kv head.
//
// One pass over the projection's output does what a decode step needs before attention:
//   y    = position rotation of the row (queries and keys),  (a c - b s, b c + a s)
//   x'   = fp16(H_b y / sqrt(b)),   the stages h = 1, 2, ... of qift_rotate in fp32, one rounding
//   codes = rint(x' * (7 / m)), s = m / 7, m = max |x'|      (keys and values, into their page)
// Layout: D / 16 lanes own a row of D values, eight from each half, so that loads and stores are whole
// lines, the half-split rotation's pairs lie in one lane, and the transform needs shuffles only between
// its three first and its last stage.  A lane's rows are heads of one token: the position's cosines and
// sines are read once for them.
// What bounds it: instruction issue (3.1 of 4 a cycle): 8192 tokens of 32 query and 32 + 32 key and value heads of
// 128 take 109 us, 2.8 TB/s, about 32 instructions a value, most of them the butterflies, their exchange and the
// roundings whose order and number the format fixes; reading the rows back 31 us, 5.5 TB/s.  Few tokens: the launch,
// 3.4 us for both.  Sums and products of two values at a time (fp32 pairs) gained nothing over the moves
// that form the pairs, and the compiler makes one rounding of a packed product and sum.  (16 contiguous values a lane, one row each, the partners by a second load:
// 150 us for 8192 tokens of 32 query and 32 + 32 key and value heads, on the L1 pipe.)
#include <math.h>

#include "act_quant.cuh"
#include "internal.h"

namespace qift {

constexpr int kKvThreads = 256;

// Stages h = 1 .. block/2 on a row: this lane (place ts of D / 16) holds values 8 ts .. 8 ts + 7 and D/2
// further.  block == 0: nothing.  The arithmetic and order of qift_rotate.
template <int D>
__device__ __forceinline__ void row_hadamard16(float (&v)[16], int ts, int block, float c) {
    if (block == 0) return;
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) {
        if (block <= h) break;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i & h) continue;
            const float a = v[i], b = v[i + h];
            v[i] = __fadd_rn(a, b);
            v[i + h] = __fsub_rn(a, b);
        }
    }
#pragma unroll
    for (int m = 1; m < D / 16; m <<= 1) {
        if (block <= 8 * m) break;
        const float sgn = (ts & m) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float p = __shfl_xor_sync(0xffffffffu, v[i], m);
            v[i] = __fmaf_rn(sgn, v[i], p);
        }
    }
    if (block > D / 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = v[i], b = v[i + 8];
            v[i] = __fadd_rn(a, b);
            v[i + 8] = __fsub_rn(a, b);
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(v[i], c);
}

__device__ __forceinline__ void load8(uint4 t, float* v) {
    const __half2* h = reinterpret_cast<const __half2*>(&t);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(h[j]);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
    }
}

// Position rotation of 8 values v = row[e .. e+7] (e and the rotated half multiples of 8, so the
// eight lie on one side of it).  tab: the position's cosines, then its sines.
__device__ __forceinline__ void rope8(float* v, const __half* row, int e, const float* __restrict__ tab, int dim,
                                      bool interleaved) {
    if (e >= dim) return;
    const int half = dim / 2;
    if (interleaved) {
        const float4 c4 = *reinterpret_cast<const float4*>(tab + e / 2);
        const float4 s4 = *reinterpret_cast<const float4*>(tab + half + e / 2);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = v[2 * i], b = v[2 * i + 1];
            v[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
            v[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
        }
    } else {
        const bool low = e < half;
        const int at = low ? e : e - half;
        float p[8];
        load8(QIFT_CK_RANGE(low ? e + half : e - half, 8, dim)
                  ? *reinterpret_cast<const uint4*>(row + (low ? e + half : e - half)) : make_uint4(0u, 0u, 0u, 0u), p);
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            const float4 c4 = *reinterpret_cast<const float4*>(tab + at + j);
            const float4 s4 = *reinterpret_cast<const float4*>(tab + half + at + j);
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float xc = __fmul_rn(v[j + i], c[i]), ps = __fmul_rn(p[j + i], s[i]);
                v[j + i] = low ? __fsub_rn(xc, ps) : __fadd_rn(xc, ps);
            }
        }
    }
}

// WHOLE: the usual call, known to the compiler: the whole row is rotated by its position, halves paired (the pairs
// and their cosines and sines are this lane's), and by a Hadamard block of its own length.
template <int D, bool WHOLE>
__global__ void __launch_bounds__(kKvThreads) append_kv_kernel(const AppendArgs a) {
    constexpr int LANES = D / 16;
    // Launched as a programmatic dependent: the inputs may come from the kernel before.
    griddep_wait();
    griddep_launch_dependents();
    const int ts = threadIdx.x % LANES, slot_of_block = threadIdx.x / LANES;
    const int64_t token = (int64_t)blockIdx.x * a.tokens_per_block + slot_of_block / a.slots_per_token;
    const int heads = a.q_heads + 2 * a.kv_heads;
    const int64_t position = a.rope && token < a.tokens ? a.positions[token] : 0;
    // A token whose position has no row in the table, or whose slot is not in the cache, is left out.
    const bool on = token < a.tokens && (!a.rope || ((uint64_t)position < (uint64_t)a.rope_len &&
                                                     QIFT_CK_RANGE(position * a.rope_dim, a.rope_dim, a.rope_len * a.rope_dim)));
    const int64_t slot = on ? a.slots[token] : -1;
    const bool kept = (uint64_t)slot < (uint64_t)(a.n_pages << a.log_page);
    const int64_t in_page = ((slot >> a.log_page) * a.kv_heads << a.log_page) + (slot & ((1 << a.log_page) - 1));
    const float* tab = a.rope + (on ? position : 0) * a.rope_dim;
    float cs[8], sn[8];
    if (WHOLE) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            *reinterpret_cast<float4*>(cs + i) = on ? *reinterpret_cast<const float4*>(tab + 8 * ts + i) : float4{};
            *reinterpret_cast<float4*>(sn + i) = on ? *reinterpret_cast<const float4*>(tab + D / 2 + 8 * ts + i) : float4{};
        }
    }
    // The row of a head, and whether there is anything to do for it.
    auto row_of = [&](int head) -> const __half* {
        if (!on || head >= heads || (head >= a.q_heads && !kept)) return nullptr;
        const int of = head < a.q_heads ? 0 : head < a.q_heads + a.kv_heads ? a.q_heads : a.q_heads + a.kv_heads;
        const int64_t stride = head < a.q_heads ? a.q_stride : head < a.q_heads + a.kv_heads ? a.k_stride : a.v_stride;
        if (!QIFT_CK_RANGE(token * stride + (int64_t)(head - of) * D, D,
                           (a.tokens - 1) * stride + (int64_t)(head < a.q_heads ? a.q_heads : a.kv_heads) * D))
            return nullptr;
        return head < a.q_heads                ? a.q + token * a.q_stride + (int64_t)head * D
               : head < a.q_heads + a.kv_heads ? a.k + token * a.k_stride + (int64_t)(head - a.q_heads) * D
                                               : a.v + token * a.v_stride + (int64_t)(head - a.q_heads - a.kv_heads) * D;
    };
    int head = blockIdx.y * a.slots_per_token * a.heads_per_slot + slot_of_block % a.slots_per_token;
    const __half* src = row_of(head);
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (src) lo = *reinterpret_cast<const uint4*>(src + 8 * ts), hi = *reinterpret_cast<const uint4*>(src + D / 2 + 8 * ts);
#pragma unroll 1
    for (int k = 0; k < a.heads_per_slot; ++k) {  // every lane of the block, for the shuffles
        const __half* row = src;
        float v[16];
        load8(lo, v);
        load8(hi, v + 8);
        const int this_head = head;
        head += a.slots_per_token;
        src = k + 1 < a.heads_per_slot ? row_of(head) : nullptr;  // the next row's loads run under this one's work
        if (src) lo = *reinterpret_cast<const uint4*>(src + 8 * ts), hi = *reinterpret_cast<const uint4*>(src + D / 2 + 8 * ts);
        if (this_head < a.q_heads + a.kv_heads) {
            if (WHOLE) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = v[i], y = v[i + 8];
                    v[i] = __fsub_rn(__fmul_rn(x, cs[i]), __fmul_rn(y, sn[i]));
                    v[i + 8] = __fadd_rn(__fmul_rn(y, cs[i]), __fmul_rn(x, sn[i]));
                }
            } else if (a.rope && row) {
                rope8(v, row, 8 * ts, tab, a.rope_dim, a.interleaved != 0);
                rope8(v + 8, row, D / 2 + 8 * ts, tab, a.rope_dim, a.interleaved != 0);
            }
        }
        row_hadamard16<D>(v, ts, WHOLE ? D : a.block, a.norm);
        uint4 packed[2];
        __half2* h2 = reinterpret_cast<__half2*>(packed);
        __half2 top = __float2half2_rn(0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h2[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            top = __hmax2(top, __habs2(h2[i]));
        }
        float m = fmaxf(__low2float(top), __high2float(top));
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (!row) continue;
        if (this_head < a.q_heads) {
            if (!QIFT_CK_RANGE((token * a.q_heads + this_head) * D, D, a.tokens * a.q_heads * D)) continue;
            __half* dst = a.q_out + (token * a.q_heads + this_head) * D + 8 * ts;
            *reinterpret_cast<uint4*>(dst) = packed[0];
            *reinterpret_cast<uint4*>(dst + D / 2) = packed[1];
            continue;
        }
        const bool is_k = this_head < a.q_heads + a.kv_heads;
        const int64_t at = in_page + ((int64_t)(this_head - a.q_heads - (is_k ? 0 : a.kv_heads)) << a.log_page);
        const uint2 w = m == 0.0f ? make_uint2(0u, 0u)
                                  : pack_int4_16(quant16(reinterpret_cast<const __half*>(packed), __fdiv_rn(7.0f, m)));
        if (!QIFT_CK_RANGE(at, 1, (a.n_pages * a.kv_heads) << a.log_page)) continue;
        uint8_t* codes = (is_k ? a.k_cache : a.v_cache) + at * (D / 2) + 4 * ts;
        *reinterpret_cast<uint32_t*>(codes) = w.x;
        *reinterpret_cast<uint32_t*>(codes + D / 4) = w.y;
        if (ts == 0) (is_k ? a.k_scales : a.v_scales)[at] = __fdiv_rn(m, 7.0f);
    }
}

// Rows of the cache as fp16 values, rotated back: the row-wise inverse of the above.  Rows of slots
// outside the cache are zeros.  A lane's key and value rows are loaded together (a row each: 37 us for 8192
// tokens of 32 heads, waiting for one load after the other).
template <int D>
__global__ void __launch_bounds__(kKvThreads) gather_kv_kernel(const GatherArgs a) {
    constexpr int LANES = D / 16;
    griddep_wait();
    griddep_launch_dependents();
    const int ts = threadIdx.x % LANES;
    const uint32_t row = blockIdx.x * (uint32_t)(kKvThreads / LANES) + threadIdx.x / LANES;
    const bool there = row < (uint32_t)a.rows;
    const uint32_t token = there ? row / (uint32_t)a.kv_heads : 0;
    const int h = there ? (int)(row - token * (uint32_t)a.kv_heads) : 0;
    const int64_t slot = there ? a.slots[token] : -1;
    const int64_t page = slot >> a.log_page;
    const int64_t at = ((page * a.kv_heads + h) << a.log_page) + (slot & ((1 << a.log_page) - 1));
    const bool on = (uint64_t)slot < (uint64_t)(a.n_pages << a.log_page) &&
                    QIFT_CK_RANGE(at, 1, (a.n_pages * a.kv_heads) << a.log_page);
    uint32_t w[2][2] = {{0u, 0u}, {0u, 0u}};
    float s[2] = {0.0f, 0.0f};
    if (on) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint8_t* codes = (kv ? a.v_cache : a.k_cache) + at * (D / 2) + 4 * ts;
            w[kv][0] = *reinterpret_cast<const uint32_t*>(codes);
            w[kv][1] = *reinterpret_cast<const uint32_t*>(codes + D / 4);
            s[kv] = (kv ? a.v_scales : a.k_scales)[at];
        }
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        // The nibble with its sign bit flipped, over 1.5 x 2^23: an fp32 whole number, and 1.5 x 2^23 + 8 off
        // it the code, exactly; the conversion instruction has an eighth of the rate.
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const uint32_t n = ((w[kv][j >> 3] >> (4 * (j & 7))) & 15u) ^ 0x4B400008u;
            v[j] = __fmul_rn(__fsub_rn(__uint_as_float(n), 12582920.0f), s[kv]);
        }
        row_hadamard16<D>(v, ts, a.block, a.norm);
        if (!there || !QIFT_CK_RANGE(row, 1, a.rows)) continue;
        uint4 packed[2];
        __half2* h2 = reinterpret_cast<__half2*>(packed);
#pragma unroll
        for (int i = 0; i < 8; ++i) h2[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        __half* dst = (kv ? a.v_out : a.k_out) + (int64_t)row * D + 8 * ts;
        *reinterpret_cast<uint4*>(dst) = packed[0];
        *reinterpret_cast<uint4*>(dst + D / 2) = packed[1];
    }
}

template <typename Kernel, typename Args>
static cudaError_t launch_rows(Kernel kernel, const Args& a, dim3 grid, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kKvThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

static float norm_of(int block) { return block ? (float)(1.0 / sqrt((double)block)) : 1.0f; }

template <int D>
static cudaError_t launch_append(AppendArgs a, cudaStream_t s) {
    constexpr int SLOTS = kKvThreads / (D / 16);  // rows a block has lanes for
    const int heads = a.q_heads + 2 * a.kv_heads;
    // Few tokens: a row a slot, the heads over blocks; many: a slot goes through several heads of its token, and the
    // slots of a token are as many as leave the fewest idle in the last turn.
    unsigned parts = 1;
    if (a.tokens * heads <= 148 * 8 * SLOTS) {
        a.slots_per_token = 1;
        while (a.slots_per_token < SLOTS && a.slots_per_token < heads) a.slots_per_token *= 2;
        a.heads_per_slot = 1;
        parts = (unsigned)((heads + a.slots_per_token - 1) / a.slots_per_token);
    } else {
        int best = 0;
        for (int n = SLOTS; n >= 1 && (heads + n - 1) / n <= 16; n /= 2) {
            const int waste = (heads + n - 1) / n * n - heads;
            if (best == 0 || waste < (heads + best - 1) / best * best - heads) best = n;
        }
        a.slots_per_token = best ? best : SLOTS;
        a.heads_per_slot = (heads + a.slots_per_token - 1) / a.slots_per_token;
    }
    a.tokens_per_block = SLOTS / a.slots_per_token;
    const dim3 grid((unsigned)((a.tokens + a.tokens_per_block - 1) / a.tokens_per_block), parts);
    return a.rope && a.rope_dim == D && !a.interleaved && a.block == D ? launch_rows(append_kv_kernel<D, true>, a, grid, s)
                                                                       : launch_rows(append_kv_kernel<D, false>, a, grid, s);
}

cudaError_t launch_append_kv(AppendArgs a, int head_dim, cudaStream_t s) {
    a.norm = norm_of(a.block);
    switch (head_dim) {
        case 64: return launch_append<64>(a, s);
        case 128: return launch_append<128>(a, s);
        case 256: return launch_append<256>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_gather_kv(GatherArgs a, int head_dim, cudaStream_t s) {
    a.norm = norm_of(a.block);
    const int64_t per = kKvThreads / (head_dim / 16);
    const dim3 grid((unsigned)((a.rows + per - 1) / per));
    switch (head_dim) {
        case 64: return launch_rows(gather_kv_kernel<64>, a, grid, s);
        case 128: return launch_rows(gather_kv_kernel<128>, a, grid, s);
        case 256: return launch_rows(gather_kv_kernel<256>, a, grid, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace qift
