// attention_wide.cu -- qift_paged_attention for many rows a kv head (prompts, and the shared prefix
// of a whole batch), on the sm_100a tensor cores (tcgen05).
//
// "Qift: Shift-Friendly No-Zero W2 Post-Training Quantization for Rotated W2A4/KV4 LLM
// Inference" names KV4.  The formula is attention.cu's.  A block takes two tiles of 128 rows against
// the same keys, 128 at a time:
//   S = Q K^T   (binary16 x binary16 -> fp32 in tensor memory)
//   p_j = 2^(scale s_j S_j - ref) t_j, rounded to binary16 into tensor memory over S
//   O += P V    (P from tensor memory, O stays there)
// K and V come from the paged 4-bit cache: bulk copies bring the codes, and four warps write them as exact
// whole numbers in binary16 in the layout the tensor core reads: K rows of keys, V transposed (rows of
// values, so that both operands are contiguous along the sum), 128-byte swizzled.  The scales are applied
// in fp32 to S and to the weights, so the one rounding is that of p.  (Folded into the binary16 operands
// instead, scales cost nothing in the softmax and the prompt of 8192 tokens took 16 us less of 614, but the
// result's error was 5.5e-4 for 2.7e-4.)  The order of values inside each group of eight is that in which a
// word's nibbles come out; Q is laid out alike.
//
//   warps 0-3, 4-7   softmax of tile 0, 1: a thread has a row
//   warps 8-11       unpack K, V; copy the scales
//   warps 12, 13     issue the products of tile 0, 1 (12 owns tensor memory)
//   warp 14          copies codes and scales from the cache (15 fills the register group)
// One tile's products run under the other's softmax.
//
// A row's reference is raised (and O scaled down) only when the weights of a half step might not fit
// binary16: the test is the sum of 2^u of each 32 keys, which is needed anyway, times their largest t_j, or times
// kMostWeight / kMostSum where that is more, so that the sum itself stays below kMostSum.
//
// What bounds it, at the prompt of 8192 tokens (32 query and 8 key/value heads of 128; 614 us in a long run under
// the power limit, 55% of the measured bf16 matrix rate over the visible half; 581 us in a short one): a step of 256
// rows by 128 keys takes 4000 to 4400 cycles, and a block's start and end come to it.  At its full rate the tensor
// core would take 2050 of them, and its counter shows that much work (43% of the time); S against 64 keys at a time
// runs below that rate, since Q is read from shared memory for each half.  The exponentials of 256 x 128 weights
// take the special-function unit 2048.  Exponentials on the fp32 pipe (a polynomial for a quarter to a half of the
// weights) made it slower (690-740 us): the softmax waits for latency, not for that unit.  head_dim 64 does half the
// products a step for as many exponentials: a prompt of 8192 by 64 query heads of 64 takes 1139 us, 30%.
//
// Every wait is bounded: one that runs out sets a shared abort flag and the device error word, every
// role leaves its loop, the products in flight are waited for and tensor memory is freed.
#include <math.h>

#include <algorithm>

#include "attention.cuh"
#include "tc.cuh"

namespace qift {
namespace attn {
namespace wide {

__device__ int g_error = 0;  // bit 1: a wait ran out (read by qift_device_error)

constexpr int BM = 128, BN = kWideStep, BH = BN / 2, TILES = 2, STAGES = 2, RING = 4;
static_assert(BM * TILES == kWideRows, "rows of a block");
constexpr int kSoftWarps = 4 * TILES, kUnpackWarps = 4;
constexpr int kUnpackThreads = 32 * kUnpackWarps;
// Four groups of four warps, launched with 128 registers a thread and redistributed: a softmax thread holds a
// row's 128 weights in pairs.  The shares sum to the four groups' 4 x 128.
constexpr int kThreads = 32 * (kSoftWarps + kUnpackWarps + 4);
constexpr int kSoftRegs = 152, kUnpackRegs = 120, kIssueRegs = 88;
static_assert(TILES == 2 && 2 * kSoftRegs + kUnpackRegs + kIssueRegs == 4 * 128, "registers of the launch");
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
constexpr uint32_t kTmemCols = 512;
constexpr float kLift = 4.0f, kMostWeight = 32768.0f;
constexpr uint32_t kNowhere = 0xffffffffu;

constexpr long long kWaitCycles = 4000000000LL;  // ~2 s before a wait gives up
static thread_local long long g_wait_limit = kWaitCycles;
static thread_local bool g_stall_next = false;

template <int D>
struct Shape {
    static constexpr int CB = D / 64;                    // 128-byte columns of a row of Q or K
    static constexpr int ROW = D / 2;                    // bytes of a row of codes
    static constexpr int CH = D / 32;                    // 16-byte pieces of it
    static constexpr int VB = D == 64 ? 4 : 8;           // bytes of a value row that a thread transposes
    static constexpr int Q_BYTES = BM * D * 2, K_BYTES = BN * D * 2, V_BYTES = BN * D * 2;
    static constexpr int K_AT = TILES * Q_BYTES, V_AT = K_AT + STAGES * K_BYTES, SC_AT = V_AT + STAGES * V_BYTES;
    // Codes and scales as they come from the cache: keys one behind the other, values in eights of keys 16
    // bytes apart, so that the transposing reads meet no bank twice.
    static constexpr int V_STRIDE = 8 * ROW + 16;
    static constexpr int KC_AT = SC_AT + RING * (BN * 8 + 16 + 4), VC_AT = KC_AT + BN * ROW;
    static constexpr int KS_AT = VC_AT + (BN / 8) * V_STRIDE, VS_AT = KS_AT + BN * 4;
    static constexpr int BAR_AT = VS_AT + BN * 4;
    static constexpr int SMEM = BAR_AT + 320 + 1024;
    static_assert(KC_AT % 16 == 0 && VC_AT % 16 == 0 && KS_AT % 16 == 0 && BAR_AT % 16 == 0, "alignment");
    static constexpr int OPAD = D + 4;
    static_assert(TILES * BM * OPAD * 4 <= BAR_AT, "finished rows lie over the operands");
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(2 * BN + TILES * D <= (int)kTmemCols, "tensor memory");
};

struct Bars {
    uint64_t k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES];
    uint64_t scales[RING];
    uint64_t q_full[TILES];
    uint64_t kc_full, kc_empty, vc_full, vc_empty;  // codes and scales as they come from the cache
    uint64_t s_full[TILES][2], p_full[TILES][2], o_done[TILES][2];  // by halves of a step
    uint64_t done, never;
    uint32_t tmem;
    int abort;
    int pmin[TILES], pmax[TILES], least[TILES];
};
static_assert(sizeof(Bars) <= 320, "barrier area");

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* abort, long long limit) {
    if (tc::mbar_try_wait(bar, parity) || tc::mbar_wait_bounded(bar, parity, abort, limit)) return true;
    if (!*reinterpret_cast<volatile int*>(abort)) {
        atomicOr(&g_error, 1);
        *reinterpret_cast<volatile int*>(abort) = 1;
    }
    return false;
}

// kind::f16, A and B binary16, fp32 accumulate, both operands contiguous along the sum.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// An operand's descriptor is given as its lower word (the address part); the upper is the same for all.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // as tc::smem_desc_sw128
__device__ __forceinline__ uint32_t desc_low(uint32_t smem_addr) { return ((smem_addr >> 4) & 0x3FFFu) | (1u << 16); }
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
        : "memory");
}

// True in one lane of the warp.
__device__ __forceinline__ bool elect() {
    uint32_t yes;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

// Two fp32 at once.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
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
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void soft_bar() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftWarps) : "memory"); }

// Waits for this thread's loads from tensor memory; the values pass through, so that nothing that uses
// them can be moved before the wait.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&x)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                   "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15]),
                   "+r"(x[16]), "+r"(x[17]), "+r"(x[18]), "+r"(x[19]), "+r"(x[20]), "+r"(x[21]), "+r"(x[22]),
                   "+r"(x[23]), "+r"(x[24]), "+r"(x[25]), "+r"(x[26]), "+r"(x[27]), "+r"(x[28]), "+r"(x[29]),
                   "+r"(x[30]), "+r"(x[31])
                 :
                 : "memory");
}

// Whether s can be a scale of the cache.
__device__ __forceinline__ bool is_scale(float s) { return s >= 0.0f && s <= 9358.0f; }

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&x)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]),
        "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15])
        : "memory");
}

// What a softmax thread knows of its row's view of a step, where not every row sees every key.
struct View {
    int hi, lo, sinks;   // key j counts if j <= hi and (j > lo or j < sinks)
    int j0;              // position of the step's first key
    uint32_t gone;       // 16s of keys that are not there
    // The keys first .. first + 31 of the step that count, a bit each.
    __device__ __forceinline__ uint32_t bits(int first) const {
        const int j = j0 + first;
        const uint32_t g = (gone >> (first >> 4)) & 3u;
        return up_to(hi - j) & (~up_to(lo - j) | up_to(sinks - 1 - j)) & ~((g & 1u ? 0xFFFFu : 0u) | (g & 2u ? 0xFFFF0000u : 0u));
    }
    __device__ __forceinline__ static uint32_t up_to(int k) {  // bits 0 .. k
        return k < 0 ? 0u : k >= 31 ? 0xFFFFFFFFu : (2u << k) - 1u;
    }
};

// Weights of half a step: S of this thread's row from tensor memory, p = 2^(k_j S_j - ref) t_j in binary16
// pairs, k_j and t_j in shared memory; `first` is the half's first key in the view, `most` the largest t_j of
// each chunk of 32 keys.  total: at least the sum of p; the result: sum of 2^(k_j S_j - ref).
template <bool MASK>
__device__ __forceinline__ float weigh(uint32_t taddr, const ulonglong2* ks, const ulonglong2* ts, float most0,
                                       float most1, float ref, const View& view, int first, uint32_t (&p)[BH / 2],
                                       float& total) {
    uint32_t in[2][32];
    tc::tmem_ld_32x32b_x32(taddr, in[0]);
    const uint64_t off = pack2(-ref, -ref);
    float part = 0.0f;
    total = 0.0f;
#pragma unroll
    for (int c = 0; c < BH / 32; ++c) {
        uint32_t(&x)[32] = in[c & 1];
        tmem_ld_wait_for(x);
        if (c + 1 < BH / 32) tc::tmem_ld_32x32b_x32(taddr + 32 * (c + 1), in[(c + 1) & 1]);
        uint64_t sum = pack2(0.0f, 0.0f);
        const uint32_t seen = MASK ? view.bits(first + c * 32) : 0u;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const ulonglong2 k4 = ks[c * 8 + i / 2], t4 = ts[c * 8 + i / 2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int j = i + q;
                float u0, u1, p0, p1;
                unpack2(fma2(pack2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), q ? k4.y : k4.x, off), u0, u1);
                if (MASK) {
                    u0 = seen & (1u << (2 * j)) ? u0 : -INFINITY;
                    u1 = seen & (2u << (2 * j)) ? u1 : -INFINITY;
                }
                const uint64_t w = pack2(ex2(u0), ex2(u1));
                sum = add2(sum, w);
                unpack2(mul2(w, q ? t4.y : t4.x), p0, p1);
                const __half2 h = __floats2half2_rn(p0, p1);
                p[c * 16 + j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        float s0, s1;
        unpack2(sum, s0, s1);
        s0 += s1;
        total = __fmaf_rn(s0, c ? most1 : most0, total);
        part += s0;
    }
    return part;
}

// The largest k_j S_j + log2 t_j of half a step.
__device__ __forceinline__ float largest(uint32_t taddr, const float* ks, const float* ts, const View& view, int first,
                                         bool mask) {
    float top = -INFINITY;
#pragma unroll
    for (int c = 0; c < BH / 32; ++c) {
        uint32_t x[32];
        tc::tmem_ld_32x32b_x32(taddr + 32 * c, x);
        tmem_ld_wait_for(x);
        const uint32_t seen = mask ? view.bits(first + c * 32) : 0xFFFFFFFFu;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float u = __fmaf_rn(__uint_as_float(x[i]), ks[c * 32 + i], fmaxf(lg2(ts[c * 32 + i]), kLeastScale));
            if (seen & (1u << i)) top = fmaxf(top, u);
        }
    }
    return top;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    wide_kernel(const AttentionArgs a, const Deal deal, long long limit, int stall) {
    using S = Shape<D>;
    extern __shared__ __align__(16) uint8_t raw[];
    uint8_t* smem = aligned<1024>(raw);  // swizzled operands
    Bars& bar = *reinterpret_cast<Bars*>(smem + S::BAR_AT);
    const uint32_t base32 = tc::smem_u32(smem);
    float* key_scales = reinterpret_cast<float*>(smem + S::SC_AT);       // [RING][BN], times the softmax scale
    float* value_scales = key_scales + RING * BN;                        // [RING][BN]
    float4* most = reinterpret_cast<float4*>(value_scales + RING * BN);  // [RING] largest t of the step's four 32s of keys
    uint32_t* gone = reinterpret_cast<uint32_t*>(most + RING);           // [RING] 16s of keys that are not there
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int warp_u = __shfl_sync(0xffffffffu, warp, 0);  // known to be the same in all lanes
    const uint32_t G = (uint32_t)a.q_heads / (uint32_t)a.kv_heads;

    // ---- which rows and keys
    // Blocks and rows are numbered in 32 bits (the host refuses more): a division of 64 bits takes 100 instructions.
    uint32_t id = blockIdx.x;
    const uint32_t prefix_blocks = (uint32_t)a.kv_heads * deal.prefix_tiles * deal.prefix_splits;
    const bool prefix = id < prefix_blocks;
    if (!prefix) id -= prefix_blocks;
    const uint32_t splits = prefix ? deal.prefix_splits : deal.own_splits;
    const int split = (int)(id % splits);
    id /= splits;
    const int h = (int)(id % (uint32_t)a.kv_heads);
    id /= (uint32_t)a.kv_heads;
    int pair, b = 0;  // the last rows see the most keys: they start first; b: own only
    if (prefix) {
        pair = deal.prefix_tiles - 1 - (int)id;
    } else if (deal.own_ragged) {
        griddep_wait();  // before the offsets are read
        if (!ragged_tile<TILES * BM>(a, deal.own_sets - 1 - id, G, b, pair) ||
            deal.is_few((int64_t)sequence(a, b).q_len * G))
            return;
    } else {
        pair = deal.own_tiles - 1 - (int)(id % (uint32_t)deal.own_tiles);
        b = (int)(id / (uint32_t)deal.own_tiles);
    }
    const int32_t* table = prefix ? a.prefix_table : a.page_table + (int64_t)b * a.max_pages;
    const int base = prefix ? 0 : a.prefix_len;
    const int64_t capacity = prefix ? a.prefix_len : (int64_t)a.max_pages << a.log_page;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            tc::mbar_init(&bar.k_full[i], kUnpackThreads);
            tc::mbar_init(&bar.k_empty[i], TILES);
            tc::mbar_init(&bar.v_full[i], kUnpackThreads);
            tc::mbar_init(&bar.v_empty[i], TILES);
        }
        for (int i = 0; i < RING; ++i) tc::mbar_init(&bar.scales[i], kUnpackThreads);
        for (int i = 0; i < TILES; ++i) {
            for (int half = 0; half < 2; ++half) {
                tc::mbar_init(&bar.s_full[i][half], 1);
                tc::mbar_init(&bar.p_full[i][half], BM);
                tc::mbar_init(&bar.o_done[i][half], 1);
            }
            tc::mbar_init(&bar.q_full[i], BM);
            bar.pmin[i] = bar.least[i] = 0x7fffffff;
            bar.pmax[i] = -1;
        }
        tc::mbar_init(&bar.kc_full, 1);
        tc::mbar_init(&bar.vc_full, 1);
        tc::mbar_init(&bar.kc_empty, kUnpackThreads);
        tc::mbar_init(&bar.vc_empty, kUnpackThreads);
        tc::mbar_init(&bar.done, TILES);
        tc::mbar_init(&bar.never, 1);
        bar.abort = 0;
        tc::fence_mbar_init();
    }
    if (warp == kSoftWarps + kUnpackWarps) {
        tc::tmem_alloc(&bar.tmem, kTmemCols);
        tc::tmem_relinquish();
    }
    griddep_wait();
    griddep_launch_dependents();
    __syncthreads();

    // ---- rows and their positions
    const int tile = warp >> 2, r = (warp & 3) * 32 + lane;  // of a softmax thread
    int64_t token = -1;
    int pos = -1, head = 0;
    if (warp < kSoftWarps) {
        const uint32_t row = (uint32_t)(pair * TILES + tile) * BM + r;
        if (prefix) {
            if (row < a.tokens * G) token = row / G, pos = position_of(a, token);
            if (pos < -1) token = pos = -1;
        } else {
            const Sequence s = sequence(a, b);
            if (row < (int64_t)s.q_len * G) {
                token = s.first + row / G;
                const int p = s.kv_len - s.q_len + (int)(row / G);
                pos = p < 0 ? -1 : p;
            }
        }
        if (token >= a.tokens || token < 0) token = -1;
        head = (int)(h * G + row % G);
        const int least = __reduce_min_sync(0xffffffffu, token >= 0 ? pos : 0x7fffffff);
        const int pmin = __reduce_min_sync(0xffffffffu, token >= 0 && pos >= 0 ? pos : 0x7fffffff);
        const int pmax = __reduce_max_sync(0xffffffffu, token >= 0 ? pos : -1);
        if (lane == 0) atomicMin(&bar.least[tile], least), atomicMin(&bar.pmin[tile], pmin), atomicMax(&bar.pmax[tile], pmax);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = bar.tmem;
    const int pmax = max(bar.pmax[0], bar.pmax[1]);
    Range range = {0, 0, 0, 0};
    if (pmax >= 0) range = visible<BN>(a, min(bar.pmin[0], bar.pmin[1]), pmax, base, capacity);
    const int chunk = max(prefix ? deal.prefix_chunk : deal.own_chunk, (range.steps + (int)splits - 1) / (int)splits);
    const int s_begin = min(split * chunk, range.steps), n = min(chunk, range.steps - s_begin);
    const int shift = range.main - range.head;
    auto block_of = [&](int i) { return s_begin + i + (s_begin + i >= range.head ? shift : 0); };

    if (warp < kSoftWarps) {
        // ------------------------------------------------------------------------------ softmax
        more_registers<kSoftRegs>();
        {  // Q of this warp's 32 rows: whole lines, a row over D / 8 lanes
            constexpr int PIECES = D / 8, PER = 32 / PIECES;
            const int64_t from = token >= 0 ? token * a.q_stride + (int64_t)head * D : -1;
            const int c = lane % PIECES;
            const uint32_t dst = base32 + tile * S::Q_BYTES + (c >> 3) * (BM * 128) + (warp & 3) * 32 * 128;
            uint4 x[32 / PER];  // all loads in flight at once
#pragma unroll
            for (int q = 0; q < 32 / PER; ++q) {
                const int64_t at = __shfl_sync(0xffffffffu, from, q * PER + lane / PIECES);
                x[q] = make_uint4(0u, 0u, 0u, 0u);
                if (at >= 0 && in_queries(a, at + c * 8, 8)) x[q] = __ldg(reinterpret_cast<const uint4*>(a.q + at + c * 8));
            }
#pragma unroll
            for (int q = 0; q < 32 / PER; ++q) {
                const int k = q * PER + lane / PIECES;
                x[q] = no_infinity(x[q]);
                sts128(dst + k * 128 + (((c & 7) ^ (k & 7)) << 4), prmt(x[q].x, x[q].z, 0x5410u),
                       prmt(x[q].x, x[q].z, 0x7632u), prmt(x[q].y, x[q].w, 0x5410u), prmt(x[q].y, x[q].w, 0x7632u));
            }
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(&bar.q_full[tile]);
        }
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + quarter + tile * BN, t_o = tmem + quarter + 2 * BN + tile * D;
        const int t_least = bar.least[tile], t_pmax = bar.pmax[tile];
        float ref = kNone, sum = 0.0f;
        View view;
        view.hi = min(pos, base + range.limit - 1);
        view.lo = a.window ? max(pos - a.window, -1) : -1;
        view.sinks = a.sinks;
        bool ok = true;
        for (int i = 0; ok && i < n; ++i) {
            const int ring = i % RING;
            ok = __all_sync(0xffffffffu, wait(&bar.scales[ring], (i / RING) & 1, &bar.abort, limit));
            if (!ok) break;
            const float4 m4 = most[ring];
            const float *ks = key_scales + ring * BN, *ts = value_scales + ring * BN;
            view.j0 = base + block_of(i) * BN;
            view.gone = gone[ring];
            const bool mask = !(view.j0 + BN - 1 <= t_least && view.j0 + BN <= base + range.limit && view.gone == 0 &&
                                (!a.window || view.j0 > t_pmax - a.window || view.j0 + BN <= a.sinks));
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const ulonglong2* k2 = reinterpret_cast<const ulonglong2*>(ks + half * BH);
                const ulonglong2* t2 = reinterpret_cast<const ulonglong2*>(ts + half * BH);
                const float m0 = half ? m4.z : m4.x, m1 = half ? m4.w : m4.y;
                const uint32_t t_h = t_s + half * BH;
                ok = __all_sync(0xffffffffu, wait(&bar.s_full[tile][half], i & 1, &bar.abort, limit));
                if (!ok) break;
                tc::tc_fence_after();
                uint32_t p[BH / 2];
                float total;
                float part = mask ? weigh<true>(t_h, k2, t2, m0, m1, ref, view, half * BH, p, total)
                                  : weigh<false>(t_h, k2, t2, m0, m1, ref, view, half * BH, p, total);
                if (!__all_sync(0xffffffffu, total <= kMostWeight)) {
                    const float to = fmaxf(ref, largest(t_h, ks + half * BH, ts + half * BH, view, half * BH, mask) - kLift);
                    const float down = ex2(ref - to);
                    ref = to;
                    sum *= down;
                    if (i + half > 0) {  // the product of the half before
                        ok = __all_sync(0xffffffffu, wait(&bar.o_done[tile][half ^ 1], (i - 1 + half) & 1, &bar.abort, limit));
                        if (!ok) break;
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t x[16];
                            tc::tmem_ld_32x32b_x16(t_o + 16 * c, x);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int q = 0; q < 16; ++q) x[q] = __float_as_uint(__uint_as_float(x[q]) * down);
                            tmem_st_x16(t_o + 16 * c, x);
                        }
                        tc::tmem_st_wait();
                    }
                    part = mask ? weigh<true>(t_h, k2, t2, m0, m1, ref, view, half * BH, p, total)
                                : weigh<false>(t_h, k2, t2, m0, m1, ref, view, half * BH, p, total);
                }
                sum += part;
                tc::tmem_st_32x32b_x32(t_h, p);  // over the S that is read
                tc::tmem_st_wait();
                tc::tc_fence_before();
                tc::mbar_arrive(&bar.p_full[tile][half]);
            }
        }
        if (n > 0 && ok) ok = wait(&bar.o_done[tile][1], (n - 1) & 1, &bar.abort, limit);
        ok = __all_sync(0xffffffffu, ok);
        soft_bar();  // both tiles' products are done: the operands' memory is free
        ok = ok && !*reinterpret_cast<volatile int*>(&bar.abort);
        if (ok) {
            // A thread finishes its row (the rotation back needs no exchange), 32 values at a time and then
            // across those, and a warp's rows go out through shared memory as whole lines.  A warp a row, with
            // shuffles, took 19000 cycles a block, a quarter of the time of a block with a window of 1024 keys; a
            // row in registers, all of it unrolled, 9000, most of them for fetching the instructions.
            tc::tc_fence_after();
            const bool finish = deal.slots == 0;
            const int block = finish ? a.block : 0;
            const float by = (finish ? (sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum)) : 1.0f) *
                             (block ? a.norm : 1.0f);
            const uint64_t by2 = pack2(by, by), minus = pack2(-1.0f, -1.0f);
            int64_t at = token >= 0 && in_result(a, token * a.q_heads + head) ? token * a.q_heads + head : -1;
            if (finish) {
                if (a.lse && at >= 0) a.lse[at] = sum == 0.0f ? -INFINITY : 0.69314718056f * (ref + log2f(sum));
            } else if (at >= 0) {
                at = at * deal.slots + (prefix ? split : deal.prefix_splits + split);
                if (in_parts(a, deal.slots, at)) parts(a, deal.slots).ml[at] = make_float2(ref, sum);
                else at = -1;
            }
            float* rows = reinterpret_cast<float*>(smem) + (tile * BM + (warp & 3) * 32) * S::OPAD;
            float* mine = rows + lane * S::OPAD;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t x[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = 0u;
                if (n > 0) {
                    tc::tmem_ld_32x32b_x32(t_o + 32 * c, x);
                    tmem_ld_wait_for(x);
                }
                uint64_t v[16];  // two values at a time; x - y as x + (-1) y, exactly the same
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = mul2(pack2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), by2);
                if (block > 1) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float y, z;
                        unpack2(v[e], y, z);
                        v[e] = pack2(y + z, y - z);
                    }
                }
#pragma unroll
                for (int hd = 1; hd < 16; hd <<= 1) {
                    if (block > 2 * hd) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (e & hd) continue;
                            const uint64_t y = v[e], z = v[e + hd];
                            v[e] = add2(y, z);
                            v[e + hd] = fma2(z, minus, y);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; e += 2) *reinterpret_cast<ulonglong2*>(mine + 32 * c + 2 * e) = make_ulonglong2(v[e], v[e + 1]);
            }
            if (block > 32) {
#pragma unroll 2
                for (int e = 0; e < 32; e += 4) {
                    ulonglong2 v[D / 32];
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) v[c] = *reinterpret_cast<const ulonglong2*>(mine + 32 * c + e);
#pragma unroll
                    for (int hd = 1; hd < D / 32; hd <<= 1) {
                        if (block > 32 * hd) {
#pragma unroll
                            for (int c = 0; c < D / 32; ++c) {
                                if (c & hd) continue;
                                const ulonglong2 y = v[c], z = v[c + hd];
                                v[c] = make_ulonglong2(add2(y.x, z.x), add2(y.y, z.y));
                                v[c + hd] = make_ulonglong2(fma2(z.x, minus, y.x), fma2(z.y, minus, y.y));
                            }
                        }
                    }
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) *reinterpret_cast<ulonglong2*>(mine + 32 * c + e) = v[c];
                }
            }
            __syncwarp();
            if (finish && a.f16) {
                constexpr int PIECES = D / 8, PER = 32 / PIECES;  // of 16 bytes
                const int c = lane % PIECES;
#pragma unroll 4
                for (int k0 = 0; k0 < 32; k0 += PER) {
                    const int k = k0 + lane / PIECES;
                    const int64_t row = __shfl_sync(0xffffffffu, at, k);
                    const float4 x = *reinterpret_cast<const float4*>(rows + k * S::OPAD + c * 8);
                    const float4 y = *reinterpret_cast<const float4*>(rows + k * S::OPAD + c * 8 + 4);
                    const __half2 h[4] = {__floats2half2_rn(x.x, x.y), __floats2half2_rn(x.z, x.w), __floats2half2_rn(y.x, y.y),
                                          __floats2half2_rn(y.z, y.w)};
                    if (row >= 0)
                        *reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + row * D + c * 8) = *reinterpret_cast<const uint4*>(h);
                }
            } else {
                float* to = finish ? static_cast<float*>(a.out) : parts(a, deal.slots).o;
                constexpr int PIECES = D / 4, PER = 32 / PIECES;
                const int c = lane % PIECES;
#pragma unroll 4
                for (int k0 = 0; k0 < 32; k0 += PER) {
                    const int k = k0 + lane / PIECES;
                    const int64_t row = __shfl_sync(0xffffffffu, at, k);
                    if (row >= 0)
                        *reinterpret_cast<float4*>(to + row * D + c * 4) =
                            *reinterpret_cast<const float4*>(rows + k * S::OPAD + c * 4);
                }
            }
        }
    } else if (warp < kSoftWarps + kUnpackWarps) {
        // ------------------------------------------------------------------------------- unpack
        fewer_registers<kUnpackRegs>();
        const int w = warp - kSoftWarps, l8 = lane & 7, l4 = lane >> 3, u = w * 32 + lane;
        const Nibbles nib;
        const int v_kg = l8 + 8 * (w & 1), v_dc = l4 + 4 * (w >> 1);  // eight keys, VB bytes of each
        for (int i = 0; i < n; ++i) {
            const int st = i % STAGES, ring = i % RING;
            if (!__all_sync(0xffffffffu, wait(&bar.kc_full, i & 1, &bar.abort, limit) &&
                                             (i < STAGES || wait(&bar.k_empty[st], ((i - STAGES) / STAGES) & 1, &bar.abort, limit))))
                break;
            const bool is = block_of(i) * BN + u < range.limit && !((gone[ring] >> (u >> 4)) & 1u);
            const float ks = is ? reinterpret_cast<const float*>(smem + S::KS_AT)[u] : 0.0f;
            const float vs = is ? reinterpret_cast<const float*>(smem + S::VS_AT)[u] : 0.0f;
            // S of step i - 2 is done, so both tiles' softmax is past step i - 3: this place of the ring is free.
            // What is no scale becomes NaN in the scores of the rows that see the key; as a value scale it would
            // reach the others, by 0 times it.
            const bool good = is_scale(ks) && is_scale(vs);
            const float t = good ? vs : 0.0f;
            key_scales[ring * BN + u] = good ? ks * a.scale_log2 : __int_as_float(0x7fffffff);
            value_scales[ring * BN + u] = t;
            float top = fmaxf(t, kMostWeight / kMostSum);  // of this warp's 32 keys, for the test of their sum
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
            if (lane == 0) reinterpret_cast<float*>(most + ring)[w] = top;
            tc::mbar_arrive(&bar.scales[ring]);
            const uint32_t k_to = base32 + S::K_AT + st * S::K_BYTES;
            // 16-byte piece cc of key kk of this warp's 32 holds groups 4 cc .. 4 cc + 3 of eight values.  Lanes read
            // side by side; half of them write their groups in another order, so that no bank is met twice.
#pragma unroll
            for (int q = 0; q < S::CH; ++q) {
                const int piece = q * 32 + lane, kk = piece / S::CH, cc = piece % S::CH;
                const uint4 x4 = *reinterpret_cast<const uint4*>(smem + S::KC_AT + (w * 32 + kk) * S::ROW + cc * 16);
                const bool swap = (cc >> 1) & 1;
                const uint32_t words[4] = {swap ? x4.z : x4.x, swap ? x4.w : x4.y, swap ? x4.x : x4.z, swap ? x4.y : x4.w};
                const uint32_t to = k_to + (w * 32 + kk) * 128 + (cc >> 1) * (BN * 128);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = (cc & 1) * 4 + (swap ? e ^ 2 : e);
                    const uint32_t x = words[e], y = words[e] >> 8;
                    sts128(to + ((c ^ (kk & 7)) << 4), nib.lo(x), nib.hi(x), nib.lo(y), nib.hi(y));
                }
            }
            tc::mbar_arrive(&bar.kc_empty);
            tc::mbar_arrive(&bar.k_full[st]);
            if (!__all_sync(0xffffffffu, wait(&bar.vc_full, i & 1, &bar.abort, limit))) break;
            if (i >= STAGES &&
                !__all_sync(0xffffffffu, wait(&bar.v_empty[st], ((i - STAGES) / STAGES) & 1, &bar.abort, limit)))
                break;
            uint32_t vq[8][S::VB / 4];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint8_t* from = smem + S::VC_AT + v_kg * S::V_STRIDE + j * S::ROW + v_dc * S::VB;
                if constexpr (S::VB == 8) {
                    const uint2 x = *reinterpret_cast<const uint2*>(from);
                    vq[j][0] = x.x, vq[j][1] = x.y;
                } else {
                    vq[j][0] = *reinterpret_cast<const uint32_t*>(from);
                }
            }
            const uint32_t v_to = base32 + S::V_AT + st * S::V_BYTES + (v_kg >> 3) * (D * 128);
#pragma unroll
            for (int wd = 0; wd < S::VB / 4; ++wd)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[k] = prmt(vq[2 * k][wd], vq[2 * k + 1][wd], hf ? 0x7632u : 0x5410u);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d8 = 4 * hf + 2 * e;  // value's place among the word's eight
                        const uint32_t to = v_to + (v_dc * (2 * S::VB) + wd * 8 + d8) * 128;
                        sts128(to + (((v_kg & 7) ^ d8) << 4), nib.lo(x[0]), nib.lo(x[1]),
                               nib.lo(x[2]), nib.lo(x[3]));
                        sts128(to + 128 + (((v_kg & 7) ^ (d8 + 1)) << 4), nib.hi(x[0]),
                               nib.hi(x[1]), nib.hi(x[2]), nib.hi(x[3]));
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] >>= 8;
                    }
                }
            tc::mbar_arrive(&bar.vc_empty);
            tc::mbar_arrive(&bar.v_full[st]);
        }
    } else {
        fewer_registers<kIssueRegs>();
        // ----------------------------------------------------------------------------- products
        // By half steps of 64 keys: a tile has two places for S, P lies over the S that it comes from, and S
        // of half step j + 2 follows when P V of half step j is complete; so a half step's softmax has its S
        // while the products beside it run.  Each tile has a warp that issues its products (about 50 cycles
        // each, whatever their size): one warp for both, in a fixed order, made the tiles fall into step and
        // wait for each other (730 us for the prompt of 8192 tokens), and looking for the tile that can go
        // on took longer still (791 us).
        // The whole warp runs the loop and one lane, always the same, issues: what the issue needs is then
        // the same in all lanes; with the loop in one lane an issue took 72 cycles.
        constexpr uint32_t id_s = idesc_f16(BM, BH), id_o = idesc_f16(BM, D);
        const int t = warp_u - (kSoftWarps + kUnpackWarps);  // this warp's tile
        if (t < TILES) {
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), b32 = __shfl_sync(0xffffffffu, base32, 0);
            const int halves = 2 * __shfl_sync(0xffffffffu, n, 0);
            const uint32_t q0 = desc_low(b32 + t * S::Q_BYTES), k0 = desc_low(b32 + S::K_AT), v0 = desc_low(b32 + S::V_AT);
            const uint32_t t_s = tm + t * BN, t_o = tm + 2 * BN + t * D;
            const bool one = elect() && QIFT_CK((tm & 0xffffu) + 2 * BN + TILES * D <= kTmemCols);
            auto wait_all = [&](uint64_t* on, uint32_t parity) {
                return __all_sync(0xffffffffu, wait(on, parity, &bar.abort, limit));
            };
            auto product_s = [&](int j) {
                const int half = j & 1, st = (j >> 1) % STAGES;
                const uint32_t k1 = k0 + st * (S::K_BYTES >> 4) + half * ((BH * 128) >> 4);
                if (one) {
#pragma unroll
                    for (int c = 0; c < S::CB; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f16_ss(t_s + half * BH, q0 + ((c * BM * 128) >> 4) + 2 * k,
                                       k1 + ((c * BN * 128) >> 4) + 2 * k, id_s, c + k != 0);
                    tc::mma_commit(&bar.s_full[t][half]);
                    if (half == 1) tc::mma_commit(&bar.k_empty[st]);
                }
            };
            auto product_o = [&](int j) {
                const int half = j & 1, st = (j >> 1) % STAGES;
                const uint32_t v1 = v0 + st * (S::V_BYTES >> 4) + half * ((D * 128) >> 4);
                if (one) {
#pragma unroll
                    for (int k = 0; k < BH / 16; ++k)
                        mma_f16_ts(t_o, t_s + half * BH + k * 8, v1 + 2 * k, id_o, k != 0 ? 1u : (uint32_t)j);
                    tc::mma_commit(&bar.o_done[t][half]);
                    if (half == 1) tc::mma_commit(&bar.v_empty[st]);
                }
            };
            bool ok = true;
            if (stall) ok = wait_all(&bar.never, 0);  // test hook
            if (halves > 0) {
                ok = ok && wait_all(&bar.q_full[t], 0) && wait_all(&bar.k_full[0], 0);
                if (ok) {
                    tc::fence_proxy_async_smem();
                    tc::tc_fence_after();
                    product_s(0);
                    product_s(1);
                }
            }
            for (int j = 0; ok && j < halves; ++j) {
                const int i = j >> 1, half = j & 1;
                ok = (half == 1 || wait_all(&bar.v_full[i % STAGES], (i / STAGES) & 1)) &&
                     wait_all(&bar.p_full[t][half], i & 1);
                if (!ok) break;
                if (half == 0) tc::fence_proxy_async_smem();
                tc::tc_fence_after();
                product_o(j);
                if (j + 2 >= halves) continue;
                ok = (half == 1 || wait_all(&bar.k_full[(i + 1) % STAGES], ((i + 1) / STAGES) & 1)) &&
                     wait_all(&bar.o_done[t][half], i & 1);
                if (!ok) break;
                if (half == 0) tc::fence_proxy_async_smem();
                tc::tc_fence_after();
                product_s(j + 2);
            }
            // Nothing may still read this block's memory when it leaves, also after an abort.
            if (one) tc::mma_commit(&bar.done);
            int zero = 0;
            tc::mbar_wait_bounded(&bar.done, 0, &zero, limit);
        } else if (t == TILES) {
            // ---------------------------------------------------------------------------- loader
            // Lanes 0-7 have one 16 of keys each: it lies in one page, one head's rows one behind the other.
            // Copies instead of loads by the unpacking warps: those waited for their loads at every
            // fence, and for the page numbers, 2800 cycles of a step's 5000.
            auto find = [&](int i) -> uint32_t {
                uint32_t at = kNowhere;
                if (i < n && lane < 8) {
                    const int j = block_of(i) * BN + lane * 16;
                    if (j < range.limit && in_table(a, prefix, j >> a.log_page)) {
                        const int page = table[j >> a.log_page];
                        if ((uint32_t)page < (uint64_t)a.n_pages)
                            at = (uint32_t)(((((int64_t)page * a.kv_heads + h) << a.log_page) + (j & ((1 << a.log_page) - 1))) >> 4);
                    }
                    if (!QIFT_CK(at == kNowhere || (int64_t)at * 16 + 16 <= (a.n_pages * a.kv_heads) << a.log_page)) at = kNowhere;
                }
                return at;
            };
            bool ok = true;
            uint32_t at = find(0);
            int k_sent = 0, v_sent = 0;
            for (int i = 0; i < n; ++i) {
                const uint32_t away = __ballot_sync(0xffffffffu, lane < 8 && at == kNowhere);
                const uint32_t count = 8 - __popc(away);
                ok = __all_sync(0xffffffffu, i == 0 || wait(&bar.kc_empty, (i - 1) & 1, &bar.abort, limit));
                if (!ok) break;
                if (lane == 0) {
                    gone[i % RING] = away;
                    tc::mbar_arrive_expect_tx(&bar.kc_full, count * (16 * S::ROW + 128));
                }
                __syncwarp();
                if (at != kNowhere) {
                    bulk_copy(base32 + S::KC_AT + lane * 16 * S::ROW, a.k_cache + (uint64_t)at * (16 * S::ROW), 16 * S::ROW,
                              &bar.kc_full);
                    bulk_copy(base32 + S::KS_AT + lane * 64, a.k_scales + (uint64_t)at * 16, 64, &bar.kc_full);
                    bulk_copy(base32 + S::VS_AT + lane * 64, a.v_scales + (uint64_t)at * 16, 64, &bar.kc_full);
                }
                k_sent = i + 1;
                ok = __all_sync(0xffffffffu, i == 0 || wait(&bar.vc_empty, (i - 1) & 1, &bar.abort, limit));
                if (!ok) break;
                if (lane == 0) tc::mbar_arrive_expect_tx(&bar.vc_full, count * (16 * S::ROW));
                __syncwarp();
                if (at != kNowhere)
                    for (int e = 0; e < 2; ++e)
                        bulk_copy(base32 + S::VC_AT + (2 * lane + e) * S::V_STRIDE,
                                  a.v_cache + (uint64_t)at * (16 * S::ROW) + e * 8 * S::ROW, 8 * S::ROW, &bar.vc_full);
                v_sent = i + 1;
                at = find(i + 1);
            }
            // Copies in flight land before the block leaves, also after an abort.
            int zero = 0;
            if (k_sent > 0) tc::mbar_wait_bounded(&bar.kc_full, (k_sent - 1) & 1, &zero, limit);
            if (v_sent > 0) tc::mbar_wait_bounded(&bar.vc_full, (v_sent - 1) & 1, &zero, limit);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == kSoftWarps + kUnpackWarps) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
static cudaError_t launch_t(const AttentionArgs& a, const Deal& d, cudaStream_t s) {
    const cudaError_t e = ensure_smem(wide_kernel<D>, Shape<D>::SMEM);
    if (e != cudaSuccess) return e;
    const int stall = g_stall_next ? 1 : 0;
    g_stall_next = false;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)d.blocks(a.kv_heads));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<D>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, wide_kernel<D>, a, d, g_wait_limit, stall);
}

}  // namespace wide

cudaError_t launch_wide(const AttentionArgs& a, const Deal& d, cudaStream_t s) {
    if (a.head_dim == 64) return wide::launch_t<64>(a, d, s);
    return wide::launch_t<128>(a, d, s);
}

}  // namespace attn

void debug_set_attention_wait_limit(long long cycles) {
    attn::wide::g_wait_limit = cycles > 0 ? cycles : attn::wide::kWaitCycles;
}
void debug_stall_next_attention() { attn::wide::g_stall_next = true; }

cudaError_t read_and_clear_attention_error(int* word) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, attn::wide::g_error, sizeof(int));
    if (e != cudaSuccess) return e;
    if (v != 0) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(attn::wide::g_error, &zero, sizeof(int));
    }
    *word = v;
    return e;
}

}  // namespace qift
