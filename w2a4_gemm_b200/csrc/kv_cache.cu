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
// Layout: D / 16 lanes own a row of D values, 16 contiguous values each, so a lane reads 32 bytes,
// writes the 8 bytes of its codes, and the transform needs shuffles only for h >= 16.  Splitting a
// row over more lanes would trade register stages for shuffles.  The half-split rotation's partner
// values come from a second load of the same row (an L1 hit) instead of 16 shuffles.
#include <math.h>

#include "act_quant.cuh"
#include "internal.h"

namespace qift {

constexpr int kKvThreads = 256;

// Stages h = 1 .. block/2 on a row spread over lanes, 16 contiguous values a lane; ts is the lane's
// place in the row.  block == 0: nothing.  The arithmetic and order of qift_rotate.
template <int LANES>
__device__ __forceinline__ void row_hadamard16(float (&v)[16], int ts, int block, float c) {
    if (block == 0) return;
#pragma unroll
    for (int h = 1; h < 16; h <<= 1) {
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
    for (int m = 1; m < LANES; m <<= 1) {
        if (block <= 16 * m) break;
        const float sgn = (ts & m) ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float p = __shfl_xor_sync(0xffffffffu, v[i], m);
            v[i] = __fmaf_rn(sgn, v[i], p);
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(v[i], c);
}

__device__ __forceinline__ void load8(const __half* p, float* v) {
    const uint4 t = *reinterpret_cast<const uint4*>(p);
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
        load8(row + (low ? e + half : e - half), p);
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

template <int D>
__global__ void __launch_bounds__(kKvThreads) append_kv_kernel(const AppendArgs a) {
    constexpr int LANES = D / 16;
    // Launched as a programmatic dependent: the inputs may come from the kernel before.
    griddep_wait();
    griddep_launch_dependents();
    const int ts = threadIdx.x % LANES;
    const uint32_t row = blockIdx.x * (uint32_t)(kKvThreads / LANES) + threadIdx.x / LANES;
    const uint32_t heads = (uint32_t)(a.q_heads + 2 * a.kv_heads);
    const bool there = row < (uint32_t)a.rows;
    const uint32_t token = there ? row / heads : 0;
    const int head = there ? (int)(row - token * heads) : 0;
    const bool is_q = head < a.q_heads;
    const bool is_k = !is_q && head < a.q_heads + a.kv_heads;
    const int h = is_q ? head : is_k ? head - a.q_heads : head - a.q_heads - a.kv_heads;
    const __half* src = is_q   ? a.q + token * a.q_stride + (int64_t)h * D
                        : is_k ? a.k + token * a.k_stride + (int64_t)h * D
                               : a.v + token * a.v_stride + (int64_t)h * D;
    const int64_t position = a.rope && there ? a.positions[token] : 0;
    const int64_t slot = there && !is_q ? a.slots[token] : 0;
    // A token whose position has no row in the table, or whose slot is not in the cache, is left out.
    const bool on = there && (!a.rope || (uint64_t)position < (uint64_t)a.rope_len) &&
                    (is_q || (uint64_t)slot < (uint64_t)(a.n_pages << a.log_page));
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    if (on) {
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
            load8(src + ts * 16 + i, v + i);
            if (a.rope && (is_q || is_k))
                rope8(v + i, src, ts * 16 + i, a.rope + position * a.rope_dim, a.rope_dim, a.interleaved != 0);
        }
    }
    row_hadamard16<LANES>(v, ts, a.block, a.norm);
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
    if (!on) return;
    if (is_q) {
        __half* dst = a.q_out + ((int64_t)token * a.q_heads + h) * D + ts * 16;
        *reinterpret_cast<uint4*>(dst) = packed[0];
        *reinterpret_cast<uint4*>(dst + 8) = packed[1];
        return;
    }
    const int64_t page = slot >> a.log_page;
    const int64_t at = ((page * a.kv_heads + h) << a.log_page) + (slot & ((1 << a.log_page) - 1));
    uint8_t* codes = is_k ? a.k_cache : a.v_cache;
    float* scales = is_k ? a.k_scales : a.v_scales;
    const uint2 w = m == 0.0f ? make_uint2(0u, 0u)
                              : pack_int4_16(quant16(reinterpret_cast<const __half*>(packed), __fdiv_rn(7.0f, m)));
    if (!QIFT_CK_RANGE(at, 1, (a.n_pages * a.kv_heads) << a.log_page)) return;
    *reinterpret_cast<uint2*>(codes + at * (D / 2) + ts * 8) = w;
    if (ts == 0) scales[at] = __fdiv_rn(m, 7.0f);
}

// Rows of the cache as fp16 values, rotated back: the row-wise inverse of the above.  Rows of slots
// outside the cache are zeros.
template <int D>
__global__ void __launch_bounds__(kKvThreads) gather_kv_kernel(const GatherArgs a) {
    constexpr int LANES = D / 16;
    griddep_wait();
    griddep_launch_dependents();
    const int ts = threadIdx.x % LANES;
    const uint32_t row = blockIdx.x * (uint32_t)(kKvThreads / LANES) + threadIdx.x / LANES;
    const uint32_t heads = 2u * (uint32_t)a.kv_heads;
    const bool there = row < (uint32_t)a.rows;
    const uint32_t token = there ? row / heads : 0;
    const int head = there ? (int)(row - token * heads) : 0;
    const bool is_k = head < a.kv_heads;
    const int h = is_k ? head : head - a.kv_heads;
    const int64_t slot = there ? a.slots[token] : -1;
    const bool on = (uint64_t)slot < (uint64_t)(a.n_pages << a.log_page);
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    if (on) {
        const int64_t page = slot >> a.log_page;
        const int64_t at = ((page * a.kv_heads + h) << a.log_page) + (slot & ((1 << a.log_page) - 1));
        if (QIFT_CK_RANGE(at, 1, (a.n_pages * a.kv_heads) << a.log_page)) {
            const uint2 w = *reinterpret_cast<const uint2*>((is_k ? a.k_cache : a.v_cache) + at * (D / 2) + ts * 8);
            const float s = (is_k ? a.k_scales : a.v_scales)[at];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int q = (int)((j < 8 ? w.x : w.y) << (28 - 4 * (j & 7))) >> 28;  // sign-extended nibble
                v[j] = __fmul_rn((float)q, s);
            }
        }
    }
    row_hadamard16<LANES>(v, ts, a.block, a.norm);
    if (!there) return;
    uint4 packed[2];
    __half2* h2 = reinterpret_cast<__half2*>(packed);
#pragma unroll
    for (int i = 0; i < 8; ++i) h2[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    __half* dst = (is_k ? a.k_out : a.v_out) + ((int64_t)token * a.kv_heads + h) * D + ts * 16;
    *reinterpret_cast<uint4*>(dst) = packed[0];
    *reinterpret_cast<uint4*>(dst + 8) = packed[1];
}

template <typename Kernel, typename Args>
static cudaError_t launch_rows(Kernel kernel, const Args& a, int head_dim, cudaStream_t s) {
    const int64_t per_block = kKvThreads / (head_dim / 16);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.rows + per_block - 1) / per_block));
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

cudaError_t launch_append_kv(AppendArgs a, int head_dim, cudaStream_t s) {
    a.norm = norm_of(a.block);
    switch (head_dim) {
        case 64: return launch_rows(append_kv_kernel<64>, a, 64, s);
        case 128: return launch_rows(append_kv_kernel<128>, a, 128, s);
        case 256: return launch_rows(append_kv_kernel<256>, a, 256, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_gather_kv(GatherArgs a, int head_dim, cudaStream_t s) {
    a.norm = norm_of(a.block);
    switch (head_dim) {
        case 64: return launch_rows(gather_kv_kernel<64>, a, 64, s);
        case 128: return launch_rows(gather_kv_kernel<128>, a, 128, s);
        case 256: return launch_rows(gather_kv_kernel<256>, a, 256, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace qift
