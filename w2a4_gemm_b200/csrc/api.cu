// api.cu -- the extern "C" entry points of libqift.so: host-side validation and dispatch.
// Declarations, argument meaning, layouts and error behaviour are documented in qift.h.
#include <math.h>
#include <stdint.h>

#include <mutex>
#include <unordered_map>

#include "../../include/qift.h"
#include "../../include/qift_debug.h"
#include "internal.h"

namespace {

bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

constexpr int64_t kMaxInner = 32768;  // keeps |acc| < 2^24 and a token / row in shared memory

qift_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QIFT_OK : QIFT_ERR_CUDA; }

bool valid_block(int64_t b) { return is_pow2(b) && b >= 2 && b <= 4096; }

bool head_block(int32_t b, int32_t d) { return b == 0 || (valid_block(b) && d % b == 0); }

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

// Layouts of the paged cache: QIFT_OK if the library has kernels for them.
qift_status cache_shape(int64_t n_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim) {
    if (n_pages < 0 || page_size <= 0 || kv_heads <= 0 || head_dim <= 0) return QIFT_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return QIFT_ERR_UNSUPPORTED;
    if (!is_pow2(page_size) || page_size < 16 || page_size > 4096) return QIFT_ERR_UNSUPPORTED;
    if (kv_heads > 1 << 16 || n_pages > 0xfffffff0LL * 16 / kv_heads / page_size) return QIFT_ERR_UNSUPPORTED;  // a place is 16 rows, in 32 bits
    return QIFT_OK;
}
int log2_of(int32_t v) {
    int l = 0;
    while ((1 << l) < v) ++l;
    return l;
}

// Sizes of an attention call; `a` receives them, `deal` how its work is dealt out.
qift_status attention_sizes(qift::AttentionArgs* a, qift::attn::Deal* deal, int64_t tokens, int32_t q_heads,
                            int32_t kv_heads, int32_t head_dim, int32_t batch, int32_t max_q, int32_t page_size, int32_t max_pages, int32_t max_kv,
                            int32_t prefix_len, int32_t window, int32_t sinks) {
    const qift_status st = cache_shape(0, page_size, kv_heads, head_dim);
    if (st != QIFT_OK) return st;
    if (tokens < 0 || batch < 0 || max_q < 0 || max_pages < 0 || max_kv < 0 || prefix_len < 0 || window < 0 || sinks < 0)
        return QIFT_ERR_INVALID_ARG;
    if (q_heads <= 0 || q_heads % kv_heads != 0) return QIFT_ERR_INVALID_ARG;
    const int64_t keys = (int64_t)max_pages * page_size + prefix_len;
    if (keys > 1 << 30 || q_heads > 1 << 16 || tokens > (1LL << 40) / q_heads / head_dim) return QIFT_ERR_UNSUPPORTED;
    a->tokens = tokens;
    a->q_heads = q_heads;
    a->kv_heads = kv_heads;
    a->head_dim = head_dim;
    a->batch = batch;
    a->max_q = max_q;
    a->log_page = log2_of(page_size);
    a->max_pages = max_pages;
    a->max_kv = max_kv > 0 && max_kv < keys ? max_kv : (int)keys;
    a->prefix_len = prefix_len;
    a->window = window;
    a->sinks = sinks;
    if (tokens > 0 && batch > 0 && max_q > 0 && !qift::plan_attention(*a, deal)) return QIFT_ERR_UNSUPPORTED;
    return QIFT_OK;
}

}  // namespace

namespace qift {

// Debug pins (qift_debug.h), per host thread, so a pin set by one thread never changes the
// kernels another thread's calls launch.
static thread_local int g_linear_path = kPathAuto;
static thread_local bool g_pdl = true;
void debug_set_pdl(bool on) { g_pdl = on; }
bool pdl_enabled() { return g_pdl; }
void debug_set_linear_path(int path) { g_linear_path = path; }
int debug_linear_path() { return g_linear_path; }

cudaError_t ensure_smem_ptr(const void* kernel, size_t bytes) {
    static std::mutex mu;
    static std::unordered_map<uint64_t, size_t> granted;  // (kernel, device) -> bytes allowed
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t key = (reinterpret_cast<uintptr_t>(kernel) << 8) ^ (uint64_t)(dev & 0xff);
    std::lock_guard<std::mutex> lock(mu);
    auto it = granted.find(key);
    if (it != granted.end() && it->second >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) granted[key] = bytes;
    return e;
}

}  // namespace qift

extern "C" {

qift_status qift_rotate(const void* x, void* y, qift_dtype dt, int64_t rows, int64_t n, int32_t block,
                        void* stream) {
    if (dt != QIFT_F32 && dt != QIFT_F16) return QIFT_ERR_INVALID_ARG;
    if (rows < 0 || n < 0 || !valid_block(block) || n % block != 0) return QIFT_ERR_INVALID_ARG;
    if (rows == 0 || n == 0) return QIFT_OK;
    if (!x || !y || !aligned16(x) || !aligned16(y)) return QIFT_ERR_INVALID_ARG;
    const int64_t esz = dt == QIFT_F32 ? 4 : 2;
    if (rows > INT64_MAX / n / esz) return QIFT_ERR_INVALID_ARG;
    const uintptr_t bytes = (uintptr_t)(rows * n * esz);
    const uintptr_t xa = reinterpret_cast<uintptr_t>(x), ya = reinterpret_cast<uintptr_t>(y);
    if (xa != ya && xa < ya + bytes && ya < xa + bytes) return QIFT_ERR_INVALID_ARG;  // partial overlap
    return from_cuda(qift::launch_rotate(x, y, dt == QIFT_F16, rows, n, block, static_cast<cudaStream_t>(stream)));
}

qift_status qift_quantize_weights(const float* w_rot, int64_t n_out, int64_t n_in, qift_levelset set,
                                  int32_t grid_points, double lo, double hi, uint32_t* codes, float* scales,
                                  double* row_mse, void* stream) {
    if (set != QIFT_SET_QIFT && set != QIFT_SET_POT && set != QIFT_SET_STD && set != QIFT_SET_INT4)
        return QIFT_ERR_INVALID_ARG;
    if (n_out < 0 || n_in <= 0 || n_in % 16 != 0) return QIFT_ERR_INVALID_ARG;
    if (grid_points < 2 || grid_points > 256) return QIFT_ERR_INVALID_ARG;
    if (!(lo > 0.0) || !(hi >= lo) || !(hi <= 4.0)) return QIFT_ERR_INVALID_ARG;
    if (n_in > kMaxInner) return QIFT_ERR_UNSUPPORTED;
    if (n_out == 0) return QIFT_OK;
    if (!w_rot || !codes || !scales || !aligned16(w_rot) || !aligned16(codes) || !aligned4(scales))
        return QIFT_ERR_INVALID_ARG;
    if (row_mse && !aligned8(row_mse)) return QIFT_ERR_INVALID_ARG;
    if (n_out > 0x7fffffff) return QIFT_ERR_UNSUPPORTED;
    return from_cuda(qift::launch_quantize_weights(w_rot, n_out, n_in, (int)set, grid_points, lo, hi, codes, scales,
                                                   row_mse, static_cast<cudaStream_t>(stream)));
}

qift_status qift_quantize_weights_asym(const float* w_rot, int64_t n_out, int64_t n_in, int32_t grid_points,
                                       double lo, double hi, uint32_t* codes, float* scales, int32_t* zeros,
                                       double* row_mse, void* stream) {
    if (n_out < 0 || n_in <= 0 || n_in % 16 != 0) return QIFT_ERR_INVALID_ARG;
    if (grid_points < 2 || grid_points > 256) return QIFT_ERR_INVALID_ARG;
    if (!(lo > 0.0) || !(hi >= lo) || !(hi <= 4.0)) return QIFT_ERR_INVALID_ARG;
    if (n_in > kMaxInner) return QIFT_ERR_UNSUPPORTED;
    if (n_out == 0) return QIFT_OK;
    if (!w_rot || !codes || !scales || !zeros || !aligned16(w_rot) || !aligned16(codes) || !aligned4(scales) ||
        !aligned4(zeros))
        return QIFT_ERR_INVALID_ARG;
    if (row_mse && !aligned8(row_mse)) return QIFT_ERR_INVALID_ARG;
    if (n_out > 0x7fffffff) return QIFT_ERR_UNSUPPORTED;
    return from_cuda(qift::launch_quantize_weights_asym(w_rot, n_out, n_in, grid_points, lo, hi, codes, scales, zeros,
                                                        row_mse, static_cast<cudaStream_t>(stream)));
}

qift_status qift_rotate_quantize_weights(const float* w, int64_t n_out, int64_t n_in, int32_t block,
                                         qift_levelset set, int32_t grid_points, double lo, double hi,
                                         uint32_t* codes, float* scales, double* row_mse, void* stream) {
    if (set != QIFT_SET_QIFT && set != QIFT_SET_POT && set != QIFT_SET_STD && set != QIFT_SET_INT4)
        return QIFT_ERR_INVALID_ARG;
    if (n_out < 0 || n_in <= 0 || n_in % 16 != 0) return QIFT_ERR_INVALID_ARG;
    if (block != 0 && (!valid_block(block) || n_in % block != 0)) return QIFT_ERR_INVALID_ARG;
    if (grid_points < 2 || grid_points > 256) return QIFT_ERR_INVALID_ARG;
    if (!(lo > 0.0) || !(hi >= lo) || !(hi <= 4.0)) return QIFT_ERR_INVALID_ARG;
    if (n_in > kMaxInner) return QIFT_ERR_UNSUPPORTED;
    if (n_out == 0) return QIFT_OK;
    if (!w || !codes || !scales || !aligned16(w) || !aligned16(codes) || !aligned4(scales))
        return QIFT_ERR_INVALID_ARG;
    if (row_mse && !aligned8(row_mse)) return QIFT_ERR_INVALID_ARG;
    if (n_out > 0x7fffffff) return QIFT_ERR_UNSUPPORTED;
    return from_cuda(qift::launch_quantize_weights(w, n_out, n_in, (int)set, grid_points, lo, hi, codes, scales,
                                                   row_mse, static_cast<cudaStream_t>(stream), block));
}

qift_status qift_quantize_acts(const void* x, int64_t tokens, int64_t n_in, int32_t block, int8_t* q,
                               float* scales, void* stream) {
    if (tokens < 0 || n_in <= 0 || n_in % 16 != 0) return QIFT_ERR_INVALID_ARG;
    if (block != 0 && (!valid_block(block) || n_in % block != 0)) return QIFT_ERR_INVALID_ARG;
    if (n_in > kMaxInner) return QIFT_ERR_UNSUPPORTED;
    if (tokens == 0) return QIFT_OK;
    if (!x || !q || !scales || !aligned16(x) || !aligned16(q) || !aligned4(scales)) return QIFT_ERR_INVALID_ARG;
    if (tokens > 0x7fffffff) return QIFT_ERR_UNSUPPORTED;
    return from_cuda(
        qift::launch_quantize_acts(x, tokens, n_in, block, q, scales, static_cast<cudaStream_t>(stream)));
}

qift_status qift_quantize_kv(const void* x, int64_t tokens, int64_t n, int32_t block, uint8_t* packed,
                             float* scales, void* stream) {
    if (tokens < 0 || n <= 0 || n % 16 != 0) return QIFT_ERR_INVALID_ARG;
    if (block != 0 && (!valid_block(block) || n % block != 0)) return QIFT_ERR_INVALID_ARG;
    if (n > kMaxInner) return QIFT_ERR_UNSUPPORTED;
    if (tokens == 0) return QIFT_OK;
    if (!x || !packed || !scales || !aligned16(x) || !aligned16(packed) || !aligned4(scales))
        return QIFT_ERR_INVALID_ARG;
    if (tokens > 0x7fffffff) return QIFT_ERR_UNSUPPORTED;
    return from_cuda(qift::launch_quantize_kv(x, tokens, n, block, packed, scales, static_cast<cudaStream_t>(stream)));
}

qift_status qift_dequantize_kv(const uint8_t* packed, const float* scales, int64_t tokens, int64_t n, int32_t block,
                               void* out, void* stream) {
    if (tokens < 0 || n <= 0 || n % 16 != 0) return QIFT_ERR_INVALID_ARG;
    if (block != 0 && (!valid_block(block) || n % block != 0)) return QIFT_ERR_INVALID_ARG;
    if (n > 16384) return QIFT_ERR_UNSUPPORTED;
    if (tokens == 0) return QIFT_OK;
    if (!packed || !scales || !out || !aligned16(packed) || !aligned16(out) || !aligned4(scales))
        return QIFT_ERR_INVALID_ARG;
    if (tokens > 0x7fffffff) return QIFT_ERR_UNSUPPORTED;
    return from_cuda(
        qift::launch_dequantize_kv(packed, scales, tokens, n, block, out, static_cast<cudaStream_t>(stream)));
}

qift_status qift_linear(const int8_t* q_act, const float* act_scale, const uint32_t* codes, const float* w_scale,
                        qift_levelset set, int64_t tokens, int64_t n_out, int64_t n_in, void* y, qift_dtype out_dt,
                        void* stream) {
    if (set != QIFT_SET_QIFT && set != QIFT_SET_POT && set != QIFT_SET_STD && set != QIFT_SET_INT4)
        return QIFT_ERR_INVALID_ARG;
    if (out_dt != QIFT_F32 && out_dt != QIFT_F16) return QIFT_ERR_INVALID_ARG;
    if (tokens < 0 || n_out < 0 || n_in <= 0 || n_in % 16 != 0) return QIFT_ERR_INVALID_ARG;
    if (set == QIFT_SET_STD) return QIFT_ERR_UNSUPPORTED;
    if (n_in > kMaxInner) return QIFT_ERR_UNSUPPORTED;
    if (set == QIFT_SET_INT4 && !qift::linear_w4_supported(tokens == 0 ? 1 : tokens, n_in)) return QIFT_ERR_UNSUPPORTED;
    if (tokens == 0 || n_out == 0) return QIFT_OK;
    if (!q_act || !act_scale || !codes || !w_scale || !y) return QIFT_ERR_INVALID_ARG;
    if (!aligned16(q_act) || !aligned16(codes) || !aligned16(y) || !aligned4(act_scale) || !aligned4(w_scale))
        return QIFT_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f16 = out_dt == QIFT_F16;
    int path = qift::debug_linear_path();
    if (set == QIFT_SET_INT4) {
        // 4-bit weights: the tcgen05 pair GEMM from 17 tokens, the tensor-core skinny kernel for
        // 2..16, the CUDA-core GEMV for one; pinning "gemm_pair" or "skinny" forces that family,
        // any other pin the GEMV (which takes at most 16 tokens).
        if (path == qift::kPathAuto)
            path = tokens >= qift::kGemmMinTokens
                       ? qift::kPathGemmPair
                       : (tokens >= 2 && qift::linear_skinny_supported(tokens, n_out, n_in) ? qift::kPathSkinny
                                                                                            : qift::kPathGemv);
        if (path == qift::kPathGemmPair) {
            if (!qift::linear_gemm_supported(tokens, n_out, n_in)) return QIFT_ERR_UNSUPPORTED;
            return from_cuda(qift::launch_linear_gemm_pair(q_act, act_scale, codes, w_scale, (int)set, tokens, n_out,
                                                           n_in, y, f16, s));
        }
        if (path == qift::kPathSkinny) {
            if (!qift::linear_skinny_supported(tokens, n_out, n_in)) return QIFT_ERR_UNSUPPORTED;
            return from_cuda(qift::launch_linear_skinny(q_act, act_scale, codes, w_scale, (int)set, tokens, n_out,
                                                        n_in, y, f16, s));
        }
        if (tokens > 16) return QIFT_ERR_UNSUPPORTED;
        return from_cuda(qift::launch_linear_w4(q_act, act_scale, codes, w_scale, tokens, n_out, n_in, y, f16, s));
    }
    if (path == qift::kPathAuto) {
        if (tokens >= qift::kGemmMinTokens) {
            // Prefill sizes run on the tensor cores only.  The code matrix's rows must be 16-byte
            // multiples for the tensor-memory copies (n_in % 64 == 0); any other n_in is refused
            // rather than sent to the CUDA-core GEMV, whose cost grows with every token.
            if (!qift::linear_gemm_supported(tokens, n_out, n_in)) return QIFT_ERR_UNSUPPORTED;
            path = qift::kPathGemmPair;
        } else if (tokens >= 2 && qift::linear_skinny_supported(tokens, n_out, n_in))
            path = qift::kPathSkinny;
        else if (tokens == 1 && qift::linear_one_token_preferred(n_out, n_in))
            path = qift::kPathOneToken;
        else
            path = qift::kPathGemv;
    } else if ((path == qift::kPathGemmPair && !qift::linear_gemm_supported(tokens, n_out, n_in)) ||
               (path == qift::kPathGemv && !qift::linear_gemv_supported(tokens)) ||
               (path == qift::kPathSkinny && !qift::linear_skinny_supported(tokens, n_out, n_in)) ||
               (path == qift::kPathOneToken && (tokens != 1 || !qift::linear_one_token_supported(n_out, n_in)))) {
        return QIFT_ERR_UNSUPPORTED;
    }
    if (path == qift::kPathOneToken)
        return from_cuda(qift::launch_linear_one_token(q_act, act_scale, codes, w_scale, (int)set, n_out, n_in, y, f16,
                                                       s));
    if (path == qift::kPathGemmPair)
        return from_cuda(qift::launch_linear_gemm_pair(q_act, act_scale, codes, w_scale, (int)set, tokens, n_out,
                                                       n_in, y, f16, s));
    if (path == qift::kPathSkinny)
        return from_cuda(qift::launch_linear_skinny(q_act, act_scale, codes, w_scale, (int)set, tokens, n_out, n_in,
                                                    y, f16, s));
    return from_cuda(
        qift::launch_linear_gemv(q_act, act_scale, codes, w_scale, (int)set, tokens, n_out, n_in, y, f16, s));
}

qift_status qift_decode_linear(const void* x, int64_t tokens, int64_t n_in, int32_t block, const uint32_t* codes,
                               const float* w_scale, qift_levelset set, int64_t n_out, void* y, qift_dtype out_dt,
                               int8_t* q_out, float* act_scale_out, void* stream) {
    if (set != QIFT_SET_QIFT && set != QIFT_SET_POT && set != QIFT_SET_STD && set != QIFT_SET_INT4)
        return QIFT_ERR_INVALID_ARG;
    if (out_dt != QIFT_F32 && out_dt != QIFT_F16) return QIFT_ERR_INVALID_ARG;
    if (tokens < 0 || n_out < 0 || n_in <= 0 || n_in % 16 != 0) return QIFT_ERR_INVALID_ARG;
    if (block != 0 && (!valid_block(block) || n_in % block != 0)) return QIFT_ERR_INVALID_ARG;
    if (set == QIFT_SET_STD || tokens > 4 || n_in > 16384 || n_in % 64 != 0) return QIFT_ERR_UNSUPPORTED;
    if (tokens == 0 || n_out == 0) return QIFT_OK;
    if (!x || !codes || !w_scale || !y) return QIFT_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(codes) || !aligned16(y) || !aligned4(w_scale)) return QIFT_ERR_INVALID_ARG;
    if ((q_out && !aligned16(q_out)) || (act_scale_out && !aligned4(act_scale_out))) return QIFT_ERR_INVALID_ARG;
    if (n_out > 0x7fffffff / 2) return QIFT_ERR_UNSUPPORTED;
    const int path = qift::debug_linear_path();
    if (tokens == 1 && (path == qift::kPathAuto || path == qift::kPathOneToken) &&
        qift::decode_one_token_supported(n_out, n_in, block, (int)set))
        return from_cuda(qift::launch_decode_one_token(x, n_in, block, codes, w_scale, (int)set, n_out, y,
                                                       out_dt == QIFT_F16, q_out, act_scale_out,
                                                       static_cast<cudaStream_t>(stream)));
    return from_cuda(qift::launch_decode_linear(x, tokens, n_in, block, codes, w_scale, (int)set, n_out, y,
                                                out_dt == QIFT_F16, q_out, act_scale_out,
                                                static_cast<cudaStream_t>(stream)));
}

qift_status qift_append_kv(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                           const float* rope, int64_t rope_len, int32_t rope_dim, int32_t rope_interleaved,
                           const int64_t* positions, const int64_t* slots, int32_t block, void* q_out,
                           uint8_t* k_cache, float* k_scales, uint8_t* v_cache, float* v_scales, int64_t n_pages,
                           int32_t page_size, void* stream) {
    const qift_status st = cache_shape(n_pages, page_size, kv_heads, head_dim);
    if (st != QIFT_OK) return st;
    if (tokens < 0 || q_heads < 0 || (q == nullptr) != (q_heads == 0) || (q == nullptr) != (q_out == nullptr))
        return QIFT_ERR_INVALID_ARG;
    if (!head_block(block, head_dim)) return QIFT_ERR_INVALID_ARG;
    if (rope && (rope_len < 0 || rope_dim <= 0 || rope_dim > head_dim || rope_dim % 2 != 0 ||
                 (rope_interleaved != 0 && rope_interleaved != 1)))
        return QIFT_ERR_INVALID_ARG;
    if (rope && rope_dim % 16 != 0) return QIFT_ERR_UNSUPPORTED;
    if (q_heads > 1 << 16 || tokens > 0x7fffffff / ((int64_t)q_heads + 2 * kv_heads)) return QIFT_ERR_UNSUPPORTED;
    if (tokens == 0) return QIFT_OK;
    if (!k || !v || !slots || (rope && !positions)) return QIFT_ERR_INVALID_ARG;
    if (n_pages > 0 && (!k_cache || !k_scales || !v_cache || !v_scales)) return QIFT_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(rope) ||
        !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scales) || !aligned16(v_scales) ||
        !aligned8(slots) || !aligned8(positions))
        return QIFT_ERR_INVALID_ARG;
    const int64_t q_row = (int64_t)q_heads * head_dim, kv_row = (int64_t)kv_heads * head_dim;
    if ((q && (q_stride % 8 != 0 || q_stride < q_row)) || k_stride % 8 != 0 || k_stride < kv_row || v_stride % 8 != 0 ||
        v_stride < kv_row)
        return QIFT_ERR_INVALID_ARG;
    const int64_t most = INT64_MAX / 4 / tokens;
    if ((q && q_stride > most) || k_stride > most || v_stride > most) return QIFT_ERR_INVALID_ARG;
    if (q) {
        const int64_t out_bytes = tokens * q_row * 2;
        if (overlap(q_out, out_bytes, q, ((tokens - 1) * q_stride + q_row) * 2) ||
            overlap(q_out, out_bytes, k, ((tokens - 1) * k_stride + kv_row) * 2) ||
            overlap(q_out, out_bytes, v, ((tokens - 1) * v_stride + kv_row) * 2))
            return QIFT_ERR_INVALID_ARG;
    }
    qift::AppendArgs a = {};
    a.q = static_cast<const __half*>(q);
    a.k = static_cast<const __half*>(k);
    a.v = static_cast<const __half*>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.tokens = tokens;
    a.q_heads = q_heads;
    a.kv_heads = kv_heads;
    a.rope = rope;
    a.rope_len = rope_len;
    a.rope_dim = rope_dim;
    a.interleaved = rope_interleaved;
    a.positions = positions;
    a.slots = slots;
    a.block = block;
    a.q_out = static_cast<__half*>(q_out);
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.n_pages = n_pages;
    a.log_page = log2_of(page_size);
    return from_cuda(qift::launch_append_kv(a, head_dim, static_cast<cudaStream_t>(stream)));
}

qift_status qift_gather_kv(const uint8_t* k_cache, const float* k_scales, const uint8_t* v_cache,
                           const float* v_scales, int64_t n_pages, int32_t page_size, int32_t kv_heads,
                           int32_t head_dim, const int64_t* slots, int64_t tokens, int32_t block, void* k_out,
                           void* v_out, void* stream) {
    const qift_status st = cache_shape(n_pages, page_size, kv_heads, head_dim);
    if (st != QIFT_OK) return st;
    if (tokens < 0 || !head_block(block, head_dim)) return QIFT_ERR_INVALID_ARG;
    if (tokens > 0x7fffffff / (2 * (int64_t)kv_heads)) return QIFT_ERR_UNSUPPORTED;
    if (tokens == 0) return QIFT_OK;
    if (!slots || !k_out || !v_out) return QIFT_ERR_INVALID_ARG;
    if (n_pages > 0 && (!k_cache || !k_scales || !v_cache || !v_scales)) return QIFT_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scales) || !aligned16(v_scales) || !aligned8(slots) ||
        !aligned16(k_out) || !aligned16(v_out))
        return QIFT_ERR_INVALID_ARG;
    qift::GatherArgs a = {};
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.rows = tokens * kv_heads;
    a.n_pages = n_pages;
    a.log_page = log2_of(page_size);
    a.kv_heads = kv_heads;
    a.slots = slots;
    a.block = block;
    a.k_out = static_cast<__half*>(k_out);
    a.v_out = static_cast<__half*>(v_out);
    return from_cuda(qift::launch_gather_kv(a, head_dim, static_cast<cudaStream_t>(stream)));
}

int64_t qift_paged_attention_workspace(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                       int32_t batch, int32_t max_q, int32_t page_size, int32_t max_pages,
                                       int32_t max_kv, int32_t prefix_len, int32_t window, int32_t sinks) {
    qift::AttentionArgs a = {};
    qift::attn::Deal deal = {};
    if (attention_sizes(&a, &deal, tokens, q_heads, kv_heads, head_dim, batch, max_q, page_size, max_pages, max_kv, prefix_len,
                        window, sinks) != QIFT_OK)
        return -1;
    return tokens == 0 || batch == 0 || max_q == 0 ? 0 : qift::attention_workspace_bytes(a, deal);
}

qift_status qift_paged_attention(const void* q, int64_t q_stride, int64_t tokens, int32_t q_heads, int32_t kv_heads,
                                 int32_t head_dim, const int32_t* cu_q, int32_t batch, int32_t max_q,
                                 const uint8_t* k_cache, const float* k_scales, const uint8_t* v_cache,
                                 const float* v_scales, int64_t n_pages, int32_t page_size,
                                 const int32_t* page_table, int32_t max_pages, const int32_t* kv_lens,
                                 int32_t max_kv, const int32_t* prefix_table, int32_t prefix_len, int32_t window,
                                 int32_t sinks, float scale, int32_t block, void* out, qift_dtype out_dt, float* lse,
                                 void* workspace, int64_t workspace_bytes, void* stream) {
    if (out_dt != QIFT_F32 && out_dt != QIFT_F16) return QIFT_ERR_INVALID_ARG;
    qift_status st = cache_shape(n_pages, page_size, kv_heads, head_dim);
    if (st != QIFT_OK) return st;
    qift::AttentionArgs a = {};
    qift::attn::Deal deal = {};
    st = attention_sizes(&a, &deal, tokens, q_heads, kv_heads, head_dim, batch, max_q, page_size, max_pages, max_kv,
                         prefix_len, window, sinks);
    if (st != QIFT_OK) return st;
    if (!head_block(block, head_dim) || !isfinite(scale)) return QIFT_ERR_INVALID_ARG;
    if (!cu_q && tokens != (int64_t)batch * max_q) return QIFT_ERR_INVALID_ARG;
    if (tokens == 0 || batch == 0 || max_q == 0) return QIFT_OK;
    if (!q || !out || !kv_lens || (max_pages > 0 && !page_table) || (prefix_len > 0 && !prefix_table))
        return QIFT_ERR_INVALID_ARG;
    if (n_pages > 0 && (!k_cache || !k_scales || !v_cache || !v_scales)) return QIFT_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scales) ||
        !aligned16(v_scales) || !aligned4(cu_q) || !aligned4(kv_lens) || !aligned4(page_table) ||
        !aligned4(prefix_table) || !aligned4(lse) || !aligned16(workspace))
        return QIFT_ERR_INVALID_ARG;
    if (q_stride % 8 != 0 || q_stride < (int64_t)q_heads * head_dim || q_stride > INT64_MAX / 4 / tokens)
        return QIFT_ERR_INVALID_ARG;
    const int64_t row = (int64_t)q_heads * head_dim;  // a block reads its queries while another may have written its rows
    if (overlap(out, tokens * row * (out_dt == QIFT_F16 ? 2 : 4), q, ((tokens - 1) * q_stride + row) * 2))
        return QIFT_ERR_INVALID_ARG;
    const int64_t need = qift::attention_workspace_bytes(a, deal);
    if (need > 0 && (!workspace || workspace_bytes < need)) return QIFT_ERR_INVALID_ARG;
    a.q = static_cast<const __half*>(q);
    a.q_stride = q_stride;
    a.cu_q = cu_q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.n_pages = n_pages;
    a.page_table = page_table;
    a.kv_lens = kv_lens;
    a.prefix_table = prefix_table;
    a.scale_log2 = scale * 1.44269504089f;
    a.block = block;
    a.out = out;
    a.f16 = out_dt == QIFT_F16;
    a.lse = lse;
    a.workspace = static_cast<float*>(workspace);
    a.workspace_bytes = workspace_bytes;
    return from_cuda(qift::launch_attention(a, deal, static_cast<cudaStream_t>(stream)));
}

qift_status qift_device_error(void* stream, int32_t* detail) {
    if (detail) *detail = 0;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return QIFT_ERR_CUDA;
    int word = 0, word1 = 0;
    if (qift::read_and_clear_device_error(&word) != cudaSuccess) return QIFT_ERR_CUDA;
    if (qift::read_and_clear_one_token_error(&word1) != cudaSuccess) return QIFT_ERR_CUDA;
    int word2 = 0;
    if (qift::read_and_clear_attention_error(&word2) != cudaSuccess) return QIFT_ERR_CUDA;
    word |= word1 | word2;
    if (detail) *detail = word;
    if (word & 0x100) return QIFT_ERR_CUDA;  // a failed bounds check (checked build only)
    return word ? QIFT_ERR_TIMEOUT : QIFT_OK;
}

qift_status qift_debug_check_line(int32_t* line) {
    if (!line) return QIFT_ERR_INVALID_ARG;
    int v = 0;
    if (qift::read_and_clear_check_line(&v) != cudaSuccess) return QIFT_ERR_CUDA;
    *line = v;
    return QIFT_OK;
}

int32_t qift_debug_checked_build(void) {
#ifdef QIFT_CHECK
    return 1;
#else
    return 0;
#endif
}

qift_status qift_debug_set_wait_limit(int64_t cycles) {
    qift::debug_set_gemm_wait_limit((long long)cycles);
    qift::debug_set_one_token_wait_limit((long long)cycles);
    qift::debug_set_attention_wait_limit((long long)cycles);
    return QIFT_OK;
}

qift_status qift_debug_set_linear_path(int32_t path) {
    if (path != qift::kPathAuto && path != qift::kPathGemv && path != qift::kPathSkinny &&
        path != qift::kPathGemmPair && path != qift::kPathOneToken)
        return QIFT_ERR_INVALID_ARG;
    qift::debug_set_linear_path(path);
    return QIFT_OK;
}

qift_status qift_debug_set_pdl(int32_t enable) {
    qift::debug_set_pdl(enable != 0);
    return QIFT_OK;
}

qift_status qift_debug_stall_next_gemm(void) {
    qift::debug_stall_next_gemm();
    return QIFT_OK;
}

qift_status qift_debug_stall_next_one_token(void) {
    qift::debug_stall_next_one_token();
    return QIFT_OK;
}

qift_status qift_debug_set_attention_path(int32_t path) {
    if (path != qift::kAttentionAuto && path != qift::kAttentionStream && path != qift::kAttentionWide)
        return QIFT_ERR_INVALID_ARG;
    qift::debug_set_attention_path(path);
    return QIFT_OK;
}

qift_status qift_debug_stall_next_attention(void) {
    qift::debug_stall_next_attention();
    return QIFT_OK;
}

const char* qift_status_string(qift_status status) {
    switch (status) {
        case QIFT_OK: return "QIFT_OK";
        case QIFT_ERR_INVALID_ARG: return "QIFT_ERR_INVALID_ARG: an argument failed host-side validation";
        case QIFT_ERR_UNSUPPORTED: return "QIFT_ERR_UNSUPPORTED: valid request this build does not implement";
        case QIFT_ERR_CUDA: return "QIFT_ERR_CUDA: a CUDA launch or runtime call failed";
        case QIFT_ERR_TIMEOUT: return "QIFT_ERR_TIMEOUT: a bounded on-chip wait gave up";
        default: return "QIFT_UNKNOWN_STATUS";
    }
}

}  // extern "C"
