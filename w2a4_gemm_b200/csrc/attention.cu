// attention.cu -- qift_paged_attention: attention over the paged KV4 cache, for few rows a
// sequence (decode), the join of partial results, and which kernel takes what.
//
// "Qift: Shift-Friendly No-Zero W2 Post-Training Quantization for Rotated W2A4/KV4 LLM
// Inference" names KV4.  For a row (token at position p, query head) with the cache's rotated
// codes k_j, v_j (whole numbers) and their scales s_j, t_j:
//   u_j = scale * s_j * (q . k_j),   out = sum_j softmax(u)_j t_j v_j,   rotated back by H_b
// over j <= p inside the window or among the sinks.  H_b is linear, so the rotation back is done
// once on the result instead of once a key.
//
// The scores are formed transposed, S^T = K Q^T, on mma.sync m16n8k16: 16 keys by 8 rows.  A decode
// step has few rows (the query heads of one kv head), so the keys take the wide side and half of
// the products that 16 padded rows would cost are not made.  Codes go from shared memory to
// fragments in registers: a lane takes a quarter of a key's row, and which product index a code
// meets is free as long as Q is permuted alike.  Half of the codes are made exact halves
// (1032 + c, minus 1032); the other half stay at c + 72 and the row's 72 * sum(q) is taken off
// beforehand as the accumulator's start value, which saves one operation in nine.  P^T needs
// tokens along its other axis: movmatrix transposes it 8 x 8.  V^T is the left operand of the
// second product: transposing loads pair its codes over two tokens, and they are made exact.
// Weights: t_j is multiplied into p_j before the rounding to binary16; the running reference is that
// of u_j + log2 t_j, so the rounded weights lie in [0, 2^15] whatever the size of the values, and
// keep 11 bits down to 2^-22 of the largest.  The sum of p_j, and O, stay in 32 bits.  Against 64 bits the result is
// off by 2.9e-4 of its norm, 2.1e-4 of it the rounding of a binary16 result.
//
// What bounds it: the bytes of the codes and scales at best (64 sequences of 8000-16384 keys, 32 query and 8
// key/value heads of 128: 190 us in a long run, 4.5 TB/s, 68% of a copy's rate); in fact the chain of a step, codes
// to scores to weights to products, of which four warps a scheduler run side by side: 470 instructions for 32 keys,
// 224 of them on the integer pipe at half rate and 160 to make binary16 of nibbles; issue is active 62%, the integer
// pipe 55%, the tensor pipe 28%.  So a run of it follows the clock: a short one, before the power limit, takes
// 166 us.  Tried and slower: shifts as high products on the multiply pipe (186 us for 177 then, in short runs), five
// blocks an SM with fewer registers (208), three stages of copies, eight warps a block.  One query head a kv head
// fills one of eight columns of the products at the same cost a key: 16 sequences of 300-4096 keys by 32 heads take
// 46 us, 3.3 TB/s.  head_dim 256: the same 64 sequences by 8 kv heads 294 us, 86%, by 2 of 8 query heads 99 us, 63%.
#include <math.h>

#include <algorithm>

#include "attention.cuh"

namespace qift {
namespace attn {

constexpr int kWarps = 4;
constexpr int kStep = 32;  // keys a warp takes at a time
// A row's reference `refl` is kLift below the largest u_j + log2 t_j when it was last raised; weights may grow
// to kMostWeight < 65504 before it is raised again.
constexpr float kLift = 8.0f, kMostWeight = 32768.0f;

template <int D>
struct Shape {
    static constexpr int ROW = D / 2;                      // bytes of a key's codes
    static constexpr int STAGE = 2 * kStep * ROW + 2 * kStep * 4;
    static constexpr int STAGES = 2;
    static constexpr int KW = D / 32;                      // 32-bit words of a key that a lane holds
    static constexpr int MT = D / 16;                      // 16-high tiles of O^T
    static constexpr int OPAD = D + 4;
    static constexpr int ring_bytes() { return kWarps * STAGES * STAGE; }
    static constexpr int join_bytes(int nr) { return kWarps * 8 * nr * (OPAD + 2) * 4; }
    static constexpr int smem(int nr) { return std::max(ring_bytes(), join_bytes(nr)) + 128; }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with the accumulator's start values (columns 2t, 2t + 1) in registers of their own.
__device__ __forceinline__ void mma16816_from(float (&d)[4], float s0, float s1, uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(s0), "f"(s1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void ldmatrix4t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}

template <int BYTES>
__device__ __forceinline__ void lds(uint32_t (&r)[BYTES / 4], const uint8_t* p) {
    if constexpr (BYTES == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    } else if constexpr (BYTES == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r[0] = v.x, r[1] = v.y;
    } else {
        r[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// Blocks an SM that the registers must leave room for.  Eight rows: four (three: 131071 keys 41 us for 36; five at
// head_dim 64: 33 windows of 4096 keys 32.5 us for 27.3).  Sixteen rows at head_dim 64: three (32 x 8192 keys by 4
// kv heads 42.3 us, two 49.4, four 42.0, but 16 x 3000 by 4 14.2, 18.1 and 16.2); at 128 three gain 5% on long
// batches and lose 13% on a short prefix (15.6 us for 13.8).
constexpr int blocks_per_sm(int D, int NR) { return D > 128 ? 1 : NR == 1 ? 4 : D == 64 ? 3 : 1; }
// Eight query rows are the columns of one product tile; NR of them a block.
template <int D, int NR>
__global__ void __launch_bounds__(32 * kWarps, blocks_per_sm(D, NR)) stream_kernel(const AttentionArgs a, const Deal deal) {
    using S = Shape<D>;
    constexpr int R = 8 * NR;
    extern __shared__ __align__(16) uint8_t raw[];
    uint8_t* smem = aligned<128>(raw);  // rows of codes are swizzled by address bits 5 and 6
    __shared__ int64_t row_token[R];
    __shared__ int row_pos[R];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t G = (uint32_t)a.q_heads / (uint32_t)a.kv_heads;
    griddep_wait();
    griddep_launch_dependents();

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
    int tile, b = 0;  // b: own only
    if (prefix) {
        tile = (int)id;
    } else if (deal.own_ragged) {
        if (!ragged_tile<R>(a, id, G, b, tile)) return;
    } else {
        tile = (int)(id % (uint32_t)deal.own_tiles);
        b = (int)(id / (uint32_t)deal.own_tiles);
        if (deal.few && !deal.is_few((int64_t)sequence(a, b).q_len * G)) return;
    }
    const int32_t* table = prefix ? a.prefix_table : a.page_table + (int64_t)b * a.max_pages;
    const int base = prefix ? 0 : a.prefix_len;
    const int64_t capacity = prefix ? a.prefix_len : (int64_t)a.max_pages << a.log_page;
    if (threadIdx.x < R) {
        const uint32_t r = (uint32_t)tile * R + threadIdx.x;
        int64_t token = -1;
        int pos = -1;
        if (prefix) {
            if (r < a.tokens * G) token = r / G, pos = position_of(a, token);
            if (pos < -1) token = pos = -1;
        } else {
            const Sequence s = sequence(a, b);
            if (r < (int64_t)s.q_len * G) {
                token = s.first + r / G;
                const int p = s.kv_len - s.q_len + (int)(r / G);
                pos = p < 0 ? -1 : p;
            }
        }
        if (token >= a.tokens || token < 0) token = -1;
        row_token[threadIdx.x] = token;
        row_pos[threadIdx.x] = pos;
    }
    __syncthreads();
    int pmin = 0x7fffffff, pmax = -1, least = 0x7fffffff;  // least: rows that see nothing (-1) included
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int p = row_pos[r];
        if (row_token[r] >= 0) least = min(least, p);
        if (p >= 0) pmin = min(pmin, p), pmax = max(pmax, p);
    }
    Range range = {0, 0, 0, 0};
    if (pmax >= 0) range = visible<kStep>(a, pmin, pmax, base, capacity);
    // The host's chunk covers lengths up to its bound; a longer sequence takes longer splits.
    const int chunk = max(prefix ? deal.prefix_chunk : deal.own_chunk, (range.steps + (int)splits - 1) / (int)splits);
    // The steps, from sure_from on, of which every row sees every key: inside all rows' windows.
    int sure_from = range.head;
    uint32_t sure_steps = 0;
    {
        const int end = min(least + 1 - base, range.limit) / kStep;  // blocks wholly before the first row's position
        const int from = a.window ? (max(pmax - a.window + 1 - base, 0) + kStep - 1) / kStep : 0;
        const int first = max(from, range.main);
        if (pmax >= 0 && end > first) sure_from = first - (range.main - range.head), sure_steps = end - first;
    }
    const int s_begin = min(split * chunk, range.steps), s_end = min(s_begin + chunk, range.steps);

    // ---- this lane's rows: column g of a tile as a right operand, columns 2t and 2t + 1 as a result
    uint32_t qf[NR][S::KW][4];
    float start[NR][2];
    int pos[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int64_t token = row_token[8 * n + g];
        const int head = (int)(h * G + ((uint32_t)tile * R + 8 * n + g) % G);
        float odd = 0.0f;
#pragma unroll
        for (int w = 0; w < S::KW; ++w) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            const int d = (w / 4) * 128 + (D >= 128 ? 32 : 16) * t + 8 * (w % 4);
            const int64_t at = token * a.q_stride + (int64_t)head * D + d;
            if (token >= 0 && in_queries(a, at, 8)) x = no_infinity(*reinterpret_cast<const uint4*>(a.q + at));
            qf[n][w][0] = prmt(x.x, x.z, 0x5410u);  // values 0, 4 of the eight that meet a word's nibbles
            qf[n][w][1] = prmt(x.x, x.z, 0x7632u);  // 1, 5
            qf[n][w][2] = prmt(x.y, x.w, 0x5410u);  // 2, 6
            qf[n][w][3] = prmt(x.y, x.w, 0x7632u);  // 3, 7
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&qf[n][w][1]));
            const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&qf[n][w][3]));
            odd += (f.x + f.y) + (e.x + e.y);
        }
        odd += __shfl_xor_sync(0xffffffffu, odd, 1);
        odd += __shfl_xor_sync(0xffffffffu, odd, 2);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            start[n][c] = -72.0f * __shfl_sync(0xffffffffu, odd, (2 * t + c) * 4);
            pos[n][c] = row_pos[8 * n + 2 * t + c];
        }
    }

    const Nibbles nib;
    float o[NR][S::MT][4];
    float refl[NR][2], sum[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
        for (int m = 0; m < S::MT; ++m)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[n][m][c] = 0.0f;
        refl[n][0] = refl[n][1] = kNone;
        sum[n][0] = sum[n][1] = 0.0f;
    }

    // ---- the ring of this warp: lanes 0-15 copy the first 16 keys of a step, lanes 16-31 the rest.
    // A lane's piece i (16 bytes) is piece c of key tok = l16 / CH + i * (16 / CH).  Pieces are swapped so that
    // the lanes' reads meet no bank twice; the swap is linear over the bits of the key's number, so a lane keeps
    // the part of its own bits and the part of i is a constant.
    uint8_t* ring = smem + warp * (S::STAGES * S::STAGE);
    const uint32_t ring32 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    const int half = lane >> 4, l16 = lane & 15;
    constexpr int CH = S::ROW / 16;
    auto k_swap = [](int tok) { return D == 256 ? (tok & 1) * 64 : 0; };
    auto v_swap = [](int tok) { return D == 256 ? (tok & 7) * 16 : D == 128 ? ((tok >> 1) & 3) * 16 : ((tok >> 2) & 1) * 16; };
    const int tok0 = l16 / CH, c0 = l16 % CH;
    const uint32_t k_dst = ring32 + (half * 16 + tok0) * S::ROW + ((c0 * 16) ^ k_swap(tok0));
    const uint32_t v_dst = ring32 + (kStep + half * 16 + tok0) * S::ROW + ((c0 * 16) ^ v_swap(tok0));
    // A lane reads the scales of keys k8, k8 + 8, + 16, + 24 at once: they lie side by side.
    const uint32_t s_dst = ring32 + 2 * kStep * S::ROW + ((l16 & 7) * 4 + half * 2 + (l16 >> 3)) * 4;
    const int shift = range.main - range.head;
    const int page_mask = (1 << a.log_page) - 1;
    // Where 16 keys lie in the pool, counted in 16s, for 16 turns of this warp at once: lane 2 i + half
    // holds turn i's.  kNowhere: the page is not there, or the sequence ends before.
    constexpr uint32_t kNowhere = 0xffffffffu;
    uint32_t places = kNowhere;
    bool lost = false;  // a page that should be there was not: every step is looked at key by key
    auto find = [&](int turn) {
        const int s = s_begin + warp + (turn + (lane >> 1)) * kWarps;
        const int j = (s + (s >= range.head ? shift : 0)) * kStep + (lane & 1) * 16;
        places = kNowhere;
        if (s < s_end && j < range.limit && in_table(a, prefix, j >> a.log_page)) {
            const int page = table[j >> a.log_page];
            if ((uint32_t)page < (uint64_t)a.n_pages)
                places = (uint32_t)(((((int64_t)page * a.kv_heads + h) << a.log_page) + (j & page_mask)) >> 4);
            else
                lost = true;
        }
        lost = __any_sync(0xffffffffu, lost);
    };
    const uint8_t* k_src = a.k_cache + l16 * 16;
    const uint8_t* v_src = a.v_cache + l16 * 16;
    const float* ks_src = a.k_scales + l16;
    const float* vs_src = a.v_scales + l16;
    auto issue = [&](int turn, int stage) {
        if ((turn & 15) == 0) find(turn);
        const uint32_t at = __shfl_sync(0xffffffffu, places, 2 * (turn & 15) + half);
        const uint32_t to = stage * S::STAGE;
        if (at != kNowhere && QIFT_CK((int64_t)at * 16 + 16 <= (a.n_pages * a.kv_heads) << a.log_page)) {
            const uint8_t* ks = k_src + (uint64_t)at * (16 * S::ROW);
            const uint8_t* vs = v_src + (uint64_t)at * (16 * S::ROW);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int tok = i * (16 / CH);
                cp16((k_dst + to + tok * S::ROW) ^ k_swap(tok), ks + i * 256);
                cp16((v_dst + to + tok * S::ROW) ^ v_swap(tok), vs + i * 256);
            }
            cp4(s_dst + to, ks_src + (uint64_t)at * 16);
            cp4(s_dst + to + kStep * 4, vs_src + (uint64_t)at * 16);
        } else {  // a scale below 0 marks keys that are not there
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(s_dst + to), "f"(-1.0f) : "memory");
        }
        cp_commit();
    };

#pragma unroll
    for (int i = 0; i < S::STAGES - 1; ++i) issue(i, i);
    int stage = 0, turn = S::STAGES - 1;
    for (int s = s_begin + warp; s < s_end; s += kWarps, ++turn) {
        __syncwarp();  // every lane is past its reads of the stage that is filled next
        issue(turn, stage == 0 ? S::STAGES - 1 : stage - 1);
        cp_wait<S::STAGES - 1>();
        __syncwarp();
        const uint8_t* st = ring + stage * S::STAGE;
        const float4 kf = reinterpret_cast<const float4*>(st + 2 * kStep * S::ROW)[g];
        const float4 vf = reinterpret_cast<const float4*>(st + 2 * kStep * S::ROW + kStep * 4)[g];
        const bool all = (uint32_t)(s - sure_from) < sure_steps && !lost;

        // ---- scores
        float x[2][NR][4];
        float ks[2][2] = {{kf.x * a.scale_log2, kf.y * a.scale_log2}, {kf.z * a.scale_log2, kf.w * a.scale_log2}};
        float vs[2][2] = {{vf.x, vf.y}, {vf.z, vf.w}};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            constexpr int KB = D >= 128 ? 16 : 8;  // bytes a read takes
#pragma unroll
            for (int i = 0; i < S::KW * 4 / KB; ++i) {
                uint32_t w0[KB / 4], w1[KB / 4];
                const int at = D == 256 ? ((4 * i + t) ^ ((g & 1) * 4)) * 16 : t * KB;
                lds<KB>(w0, st + (c * 16 + g) * S::ROW + at);
                lds<KB>(w1, st + (c * 16 + g + 8) * S::ROW + at);
#pragma unroll
                for (int w = 0; w < KB / 4; ++w) {
                    const int k = i * (KB / 4) + w;
                    uint32_t a0 = w0[w], a1 = w1[w];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t l0 = nib.lo(a0), l1 = nib.lo(a1), h0 = nib.hi72(a0), h1 = nib.hi72(a1);
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            if (k == 0 && e == 0)
                                mma16816_from(x[c][n], start[n][0], start[n][1], l0, l1, h0, h1, qf[n][k][0], qf[n][k][1]);
                            else
                                mma16816(x[c][n], l0, l1, h0, h1, qf[n][k][2 * e], qf[n][k][2 * e + 1]);
                        }
                        a0 >>= 8, a1 >>= 8;
                    }
                }
            }
        }
        // Masked scores become -infinity (their scale, which may hold anything, is multiplied in first), and
        // what no row sees gets the value scale 0.  A value scale that is no number would reach the rows that do
        // not see it by 0 times it: it goes into the score instead, of the rows that do.
        if (!all) {
            const int j0 = base + (s + (s >= range.head ? shift : 0)) * kStep;  // position of the step's first key
            const float there[2][2] = {{kf.x, kf.y}, {kf.z, kf.w}};
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = j0 + c * 16 + g + 8 * e;
                    const bool in = there[c][e] >= 0.0f && j - base < range.limit;
                    const bool odd = !(vs[c][e] <= 65504.0f);
                    const float k1 = odd ? __int_as_float(0x7fffffff) : ks[c][e];
                    bool any = false;
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int p = pos[n][q];
                            const bool see = in && j <= p && (!a.window || j > p - a.window || j < a.sinks);
                            x[c][n][2 * e + q] = see ? x[c][n][2 * e + q] * k1 : -INFINITY;
                            any |= see;
                        }
                    ks[c][e] = 1.0f;
                    if (!any || odd) vs[c][e] = 0.0f;
                }
        }

        // ---- weights, by the reference so far.  It is raised, and what is summed scaled down, only where a
        // weight would pass kMostWeight, or this lane's sum kMostSum (or one is no number: an overflow times a
        // scale of 0); a vote decides, so all lanes of a row agree.
        float part[NR][2];
        __half2 wv[2][NR][2];
        const __half2 most = __float2half2_rn(kMostWeight);
        auto weigh = [&]() {
            bool fits = true;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float w0 = ex2(__fmaf_rn(x[c][n][2 * e], ks[c][e], -refl[n][0]));
                        const float w1 = ex2(__fmaf_rn(x[c][n][2 * e + 1], ks[c][e], -refl[n][1]));
                        wv[c][n][e] = __floats2half2_rn(w0 * vs[c][e], w1 * vs[c][e]);
                        fits = fits && __hble2(wv[c][n][e], most);
                        part[n][0] = c + e ? part[n][0] + w0 : w0;
                        part[n][1] = c + e ? part[n][1] + w1 : w1;
                    }
                fits = fits && part[n][0] <= kMostSum && part[n][1] <= kMostSum;
            }
            return fits;
        };
        if (!__all_sync(0xffffffffu, weigh())) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float top = refl[n][q] + kLift;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            top = fmaxf(top, __fmaf_rn(x[c][n][2 * e + q], ks[c][e], fmaxf(lg2(vs[c][e]), kLeastScale)));
#pragma unroll
                    for (int m = 4; m < 32; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
                    const float down = ex2(refl[n][q] + kLift - top);
                    refl[n][q] = top - kLift;
                    sum[n][q] *= down;
#pragma unroll
                    for (int m = 0; m < S::MT; ++m) o[n][m][q] *= down, o[n][m][2 + q] *= down;
                }
            weigh();
        }

        // ---- the second product
#pragma unroll
        for (int n = 0; n < NR; ++n) sum[n][0] += part[n][0], sum[n][1] += part[n][1];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t p[NR][2];
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) p[n][e] = transpose8(*reinterpret_cast<const uint32_t*>(&wv[c][n][e]));
            // Four codes of a key are a 16-bit unit; the transposing load of 8 keys by 8 units leaves unit g of
            // keys 2t and 2t + 1 in a lane's register, as the left operand wants its pairs.  Four such loads an
            // instruction: units 8 u + g of keys 0-7 and 8-15, for two u.
#pragma unroll
            for (int u = 0; u < S::MT / 2; u += 2) {
                uint32_t v[4];
                const int tok = (lane & 7) + ((lane >> 3) & 1) * 8, piece = (u + (lane >> 4)) * 16;
                ldmatrix4t(v, ring32 + stage * S::STAGE + (kStep + c * 16 + tok) * S::ROW + (piece ^ v_swap(tok)));
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t lo = v[2 * w] >> (8 * e), hi = v[2 * w + 1] >> (8 * e);
                        const uint32_t a0 = nib.lo(lo), a1 = nib.hi(lo), a2 = nib.lo(hi), a3 = nib.hi(hi);
#pragma unroll
                        for (int n = 0; n < NR; ++n) mma16816(o[n][2 * (u + w) + e], a0, a1, a2, a3, p[n][0], p[n][1]);
                    }
            }
        }
        stage = stage + 1 == S::STAGES ? 0 : stage + 1;
    }
    cp_wait<0>();
    __syncthreads();

    // ---- join the warps.  Lane (g, t) holds values 32 u + 4 g + 0 .. 3 of rows 2t, 2t + 1.
    float* po = reinterpret_cast<float*>(smem);
    float* pm = po + kWarps * R * S::OPAD;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int m = 4; m < 32; m <<= 1) sum[n][q] += __shfl_xor_sync(0xffffffffu, sum[n][q], m);
            const int r = 8 * n + 2 * t + q;
            float* dst = po + (warp * R + r) * S::OPAD + g * 4;
#pragma unroll
            for (int u = 0; u < S::MT / 2; ++u)
                *reinterpret_cast<float4*>(dst + 32 * u) =
                    make_float4(o[n][2 * u][q], o[n][2 * u][2 + q], o[n][2 * u + 1][q], o[n][2 * u + 1][2 + q]);
            if (g == 0) {
                pm[(warp * R + r) * 2] = refl[n][q];
                pm[(warp * R + r) * 2 + 1] = sum[n][q];
            }
        }
    __syncthreads();
    constexpr int E = D / 32;
    for (int r = warp; r < R; r += kWarps) {
        const int64_t token = row_token[r];
        if (token < 0) continue;
        const int head = (int)(h * G + ((uint32_t)tile * R + r) % G);
        float M = kNone, L = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, pm[(w * R + r) * 2]);
        float acc[E];
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(pm[(w * R + r) * 2] - M);
            L += f * pm[(w * R + r) * 2 + 1];
            const float* src = po + (w * R + r) * S::OPAD + lane * E;
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] += f * src[i];
        }
        if (deal.slots == 0) {
            finish_row<D>(a, acc, M, L, token, head, lane);
        } else {
            const Parts p = parts(a, deal.slots);
            const int64_t at = (token * a.q_heads + head) * deal.slots + (prefix ? split : deal.prefix_splits + split);
            if (!in_parts(a, deal.slots, at)) continue;
            if (lane == 0) p.ml[at] = make_float2(M, L);
            if (!(L == 0.0f)) {
#pragma unroll
                for (int i = 0; i < E; ++i) p.o[at * D + lane * E + i] = acc[i];
            }
        }
    }
}

// The row-th row to be joined: its token (-1: none), head and number of partial results.  Rows are dealt out as
// (sequence, token, head), or as (token, head) where that is much less.
__device__ __forceinline__ int64_t joined_row(const AttentionArgs& a, const Deal& deal, bool by_token, uint32_t row, int& head,
                                              int& slots) {
    head = (int)(row % (uint32_t)a.q_heads);
    row /= (uint32_t)a.q_heads;
    const int b = by_token ? (row < a.tokens ? sequence_of(a, row) : -1) : (int)(row / (uint32_t)a.max_q);
    if (b < 0 || b >= a.batch) return -1;
    const Sequence s = sequence(a, b);
    const int64_t i = by_token ? row - s.first : row % (uint32_t)a.max_q;
    if (i < 0 || i >= s.q_len) return -1;
    slots = deal.prefix_splits +
            (deal.few && deal.is_few((int64_t)s.q_len * (a.q_heads / a.kv_heads)) ? deal.few_splits : deal.own_splits);
    return s.first + i;
}

// The same for rows of up to 32 slots, a warp a row: a lane holds a slot's weight.  (4096 rows of 10 slots, a
// block each: 17.8 us.)
template <int D>
__global__ void __launch_bounds__(256) join_few_kernel(const AttentionArgs a, const Deal deal, const bool by_token) {
    constexpr int E = D / 32;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    int head, slots;
    const int64_t token = joined_row(a, deal, by_token, blockIdx.x * 8 + (threadIdx.x >> 5), head, slots);
    if (token < 0) return;
    const Parts p = parts(a, deal.slots);
    const int64_t at = (token * a.q_heads + head) * deal.slots;
    const float2 ml = lane < slots && in_parts(a, deal.slots, at + lane) ? p.ml[at + lane] : make_float2(kNone, 0.0f);
    float M = ml.x;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
    const float f = ml.y == 0.0f ? 0.0f : ex2(ml.x - M);
    float L = f * ml.y, acc[E];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) L += __shfl_xor_sync(0xffffffffu, L, m);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    for (int k0 = 0; k0 < slots; k0 += 4) {
        float w[4], v[4][E];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            w[u] = __shfl_sync(0xffffffffu, f, (k0 + u) & 31);
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = 0.0f;
            if (k0 + u < slots && !(w[u] == 0.0f) && in_parts(a, deal.slots, at + k0 + u)) {  // an empty slot's O was never written
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    *reinterpret_cast<float2*>(&v[u][e]) =
                        *reinterpret_cast<const float2*>(p.o + (at + k0 + u) * D + lane * E + e);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = __fmaf_rn(k0 + u < slots ? w[u] : 0.0f, v[u][e], acc[e]);
    }
    finish_row<D>(a, acc, M, L, token, head, lane);
}

// Joins the partial results of a row, one block a row.
// All (M, L) are read at once and become weights in shared memory, then each warp sums every
// kJoinWarps-th slot with four loads in flight: what it costs is the chain of loads, so the chain is
// kept short (32 rows of 74 slots took 14.5 us with one load in flight and four warps).
constexpr int kJoinWarps = 8;
constexpr int kMostSlots = 4096;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const AttentionArgs a, const Deal deal, const bool by_token) {
    constexpr int E = D / 32;
    extern __shared__ float weight[];
    __shared__ float part[kJoinWarps][D], red[2][kJoinWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int head, slots;
    const int64_t token = joined_row(a, deal, by_token, blockIdx.x, head, slots);
    if (token < 0) return;
    const Parts p = parts(a, deal.slots);
    const int64_t at = (token * a.q_heads + head) * deal.slots;
    float M = kNone;
    for (int k = threadIdx.x; k < slots; k += 32 * kJoinWarps)
        if (in_parts(a, deal.slots, at + k)) M = fmaxf(M, p.ml[at + k].x);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
    if (lane == 0) red[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, red[0][w]);
    float L = 0.0f, acc[E];
    for (int k = threadIdx.x; k < slots; k += 32 * kJoinWarps) {
        const float2 ml = in_parts(a, deal.slots, at + k) ? p.ml[at + k] : make_float2(kNone, 0.0f);
        const float f = ml.y == 0.0f ? 0.0f : ex2(ml.x - M);
        weight[k] = f;
        L += f * ml.y;
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) L += __shfl_xor_sync(0xffffffffu, L, m);
    if (lane == 0) red[1][warp] = L;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
    __syncthreads();
    for (int k0 = warp; k0 < slots; k0 += 4 * kJoinWarps) {
        float w[4], v[4][E];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = k0 + u * kJoinWarps;
            w[u] = k < slots ? weight[k] : 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = 0.0f;
            if (!(w[u] == 0.0f) && in_parts(a, deal.slots, at + k)) {  // an empty slot's O was never written
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    *reinterpret_cast<float2*>(&v[u][e]) = *reinterpret_cast<const float2*>(p.o + (at + k) * D + lane * E + e);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = __fmaf_rn(w[u], v[u][e], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
    __syncthreads();
    if (warp != 0) return;
    L = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        L += red[1][w];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += part[w][lane * E + e];
    }
    finish_row<D>(a, acc, M, L, token, head, lane);
}

// How one kind of row sets (the prefix's, or the sequences' own) is cut into blocks.
struct Cut {
    int tiles, splits, chunk;
    int64_t sets;  // row tiles of all row sets
    bool ragged;
    double us;     // what it takes, roughly
};
// `batch` row sets of up to `rows` rows, `all_rows` in all, and at most `keys` keys, for each kv head, on the
// streaming kernel (`per` rows a block) or the one for many rows.
// Streaming: a split is at least 512 keys (four steps a warp) and, of a batch of unequal lengths, at most 4096.
// Rows of equal lengths are split into one turn of the GPU (four blocks an SM): 131071 keys by 8 kv heads
// take 37 us, with two turns 42; 33 windows of 4096 keys by 8 27.3 and 29.7.  Unequal ones into three turns, counted by
// the bound on their lengths, so that short ones leave no gap: 16 sequences of 300-4096 keys by 32 kv heads take
// 45.1 us with three turns, 46.7 with one or two, 46.6 with four and 50.6 with six; 64 of 8000-16384 by 8
// the same, 165 us, with any of them.
// Many rows: one block an SM, split only where there are fewer row sets than SMs.
static Cut cut(bool wide, int per, int64_t kv_heads, int64_t batch, int64_t rows, int64_t all_rows, int64_t keys, bool equal,
               int head_dim) {
    Cut c = {};
    const int64_t step = wide ? kWideStep : kStep;
    const int64_t least = 512 / step, most = wide || equal ? 1 << 20 : 4096 / step;
    const int64_t steps = (keys + step - 1) / step + 1;
    c.tiles = (int)((rows + per - 1) / per);
    c.sets = batch * c.tiles;
    const int64_t total = all_rows / per + batch;  // never less than the tiles of equal sets
    c.ragged = total < c.sets;  // an empty block of the kernel for many rows took 7 us, a search through the offsets 1
    if (c.ragged) c.sets = total;
    const int64_t blocks = kv_heads * c.sets;
    int64_t n = wide ? 148 / blocks : (equal ? 1 : 3) * 592 / blocks;
    n = std::max<int64_t>(std::max<int64_t>(1, (steps + most - 1) / most), std::min(n, steps / least));
    n = std::min<int64_t>(n, kMostSlots / 2);
    c.chunk = (int)((steps + n - 1) / n);
    c.splits = (int)((steps + c.chunk - 1) / c.chunk);
    // Measured with head_dim 128: a streamed key takes 0.038 ns for a block of 16 rows and 0.024 for one of 8
    // when the GPU is full, a block as much more as 300 keys, a launch 9 us; a step of 256 rows by 128 keys
    // takes an SM 2.3 us, a launch 17.  The same constants choose at head_dim 64 (64 and 32 query heads by 8 kv heads,
    // 16 by 4, 32 by 32; 1, 4 or 16 sequences of 4 to 256 tokens and 300 to 16000 keys, prefixes of 500 to 32000 keys by
    // up to 256 rows, each size on both kernels): the chosen one took at most 1.37 times the better's time (64
    // tokens each of 16 sequences of 300 keys, 22.3 us streamed for 16.4), 1% to 2% more on average; at 128 at most
    // 1.10 times with 8 kv heads, 1.23 with 32.
    const int64_t all = blocks * c.splits;
    c.us = wide ? 17.0 + (double)((all + 147) / 148) * c.chunk * 2.3
                : 9.0 + (double)all * ((double)c.chunk * kStep + 300.0) * (per == 8 ? 24e-6 : 38e-6) * head_dim / 128;
    return c;
}

// Rows of a block of the streaming kernel.
static int stream_rows(const AttentionArgs& a, const Deal& d) {
    const int64_t G = a.q_heads / a.kv_heads;
    return (d.few ? d.few <= 8 : d.own_wide || a.max_q * G <= 8) && (d.prefix_wide || !a.prefix_len || a.tokens * G <= 8) ? 8 : 16;
}

// Which kernel takes what: the one that takes less by the measure above.  A step of 256 rows costs the same
// for fewer, so few rows stream: 64 sequences' single tokens of four query heads a kv head against a
// prefix of 32000 keys took 52 us either way, 16 of them 27 us streamed and 53, 128 of them 85 and 57.
static Deal deal_out(const AttentionArgs& a) {
    const int64_t G = a.q_heads / a.kv_heads, own_rows = a.max_q * G, shared_rows = a.tokens * G;
    const bool equal = a.batch == 1 || a.window > 0;
    int64_t own = (int64_t)a.max_kv - a.prefix_len;
    if (a.window)  // rows of the whole batch stand far apart: no such bound on what they see of the prefix
        own = std::min(own, (int64_t)a.window + a.max_q + a.sinks + 2 * kStep);
    own = std::max<int64_t>(own, 1);
    auto own_cut = [&](bool wide, int per) {
        return cut(wide, wide ? kWideRows : per, a.kv_heads, a.batch, own_rows, shared_rows, own, equal, a.head_dim);
    };
    auto shared_cut = [&](bool wide, int per) {
        return cut(wide, wide ? kWideRows : per, a.kv_heads, 1, shared_rows, shared_rows, a.prefix_len, true, a.head_dim);
    };
    Cut own_is = {};
    Deal d = {};
    const int pin = debug_attention_path();
    if (pin == kAttentionWide) {
        d.own_wide = true;
        d.prefix_wide = a.prefix_len > 0;
    } else if (a.head_dim <= 128 && pin == kAttentionAuto) {
        const Cut many = own_cut(true, 0), few = own_cut(false, 16);
        d.own_wide = own_rows > 16 && many.us < few.us;
        if (own_rows > 16 && G <= 16 && 2 * many.sets <= (int64_t)a.batch * many.tiles) {
            // Long sequences among short ones (prompts among single tokens): each to its kernel, if one long
            // sequence with all the rows and single tokens of the others would be faster so.  Blocks of the
            // kernel for many rows that find a short sequence leave at once (about 1 us of an SM).
            const int most = G <= 8 ? 8 : 16;
            const Cut one = cut(true, kWideRows, a.kv_heads, 1, shared_rows, shared_rows, own, equal, a.head_dim);
            const Cut rest = cut(false, most, a.kv_heads, a.batch, most, most * (int64_t)a.batch, own, equal, a.head_dim);
            if (one.us + rest.us + (double)a.batch * a.kv_heads * one.splits / 148 < std::min(many.us, few.us)) {
                d.own_wide = true;
                d.few = most, d.few_splits = rest.splits, d.few_chunk = rest.chunk;
                own_is = one;
                own_is.sets = many.sets, own_is.ragged = true;
            }
        }
        d.prefix_wide = a.prefix_len && shared_rows > 16 && shared_cut(true, 0).us < shared_cut(false, 16).us;
    }
    const int per = stream_rows(a, d);
    const Cut c = d.few ? own_is : own_cut(d.own_wide, per);
    d.own_tiles = c.tiles, d.own_splits = c.splits, d.own_chunk = c.chunk, d.own_sets = c.sets, d.own_ragged = c.ragged;
    if (a.prefix_len) {
        const Cut p = shared_cut(d.prefix_wide, per);
        d.prefix_tiles = p.tiles, d.prefix_splits = p.splits, d.prefix_chunk = p.chunk;
    }
    const int splits = std::max(d.own_splits, d.few_splits);
    d.slots = a.prefix_len || splits > 1 ? d.prefix_splits + splits : 0;
    return d;
}

template <int D, int NR>
static cudaError_t launch_stream(const AttentionArgs& a, const Deal& d, cudaStream_t s) {
    const size_t smem = Shape<D>::smem(NR);
    if (smem > 48 * 1024) {  // what a kernel may have without asking
        const cudaError_t e = ensure_smem(stream_kernel<D, NR>, smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)d.blocks(a.kv_heads));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, stream_kernel<D, NR>, a, d);
}

template <int D>
static cudaError_t launch_join(const AttentionArgs& a, const Deal& d, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    const int slots = d.slots;
    const bool by_token = 2 * a.tokens <= (int64_t)a.batch * a.max_q;
    const int64_t rows = (by_token ? a.tokens : (int64_t)a.batch * a.max_q) * a.q_heads;
    const bool few = slots <= 32 && rows >= 148 * 2;  // a warp a row only where that fills the GPU
    cfg.gridDim = dim3((unsigned)(few ? (rows + 7) / 8 : rows));
    cfg.blockDim = dim3(few ? 256 : 32 * kJoinWarps);
    cfg.dynamicSmemBytes = few ? 0 : slots * sizeof(float);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, few ? join_few_kernel<D> : join_kernel<D>, a, d, by_token);
}

template <int D>
static cudaError_t launch_all(const AttentionArgs& a, const Deal& d, cudaStream_t s) {
    for (const bool wide : {true, false}) {  // one launch for each kernel that has rows to do
        const Deal part = d.of(wide, a.batch);
        if (part.blocks(a.kv_heads) == 0) continue;
        const cudaError_t e = wide                     ? launch_wide(a, part, s)
                              : stream_rows(a, d) == 8 ? launch_stream<D, 1>(a, part, s)
                                                    : launch_stream<D, 2>(a, part, s);
        if (e != cudaSuccess) return e;
    }
    return d.slots ? launch_join<D>(a, d, s) : cudaSuccess;
}

}  // namespace attn

static thread_local int g_attention_path = kAttentionAuto;
void debug_set_attention_path(int path) { g_attention_path = path; }
int debug_attention_path() { return g_attention_path; }

bool plan_attention(const AttentionArgs& a, attn::Deal* deal) {
    if (debug_attention_path() == kAttentionWide && a.head_dim > 128) return false;
    // Rows of the batch and of a launch in 32 bits, before anything is computed from their numbers.
    if ((int64_t)a.batch * a.max_q > 0x7fffffff / a.q_heads || a.tokens > 0x7fffffff / a.q_heads) return false;
    const attn::Deal d = *deal = attn::deal_out(a);
    return d.of(true, a.batch).blocks(a.kv_heads) <= 0x7fffffff && d.of(false, a.batch).blocks(a.kv_heads) <= 0x7fffffff;
}

int64_t attention_workspace_bytes(const AttentionArgs& a, const attn::Deal& deal) {
    return a.tokens * a.q_heads * deal.slots * (a.head_dim + 2) * 4;
}

cudaError_t launch_attention(AttentionArgs a, const attn::Deal& deal, cudaStream_t s) {
    a.norm = a.block ? (float)(1.0 / sqrt((double)a.block)) : 1.0f;
    switch (a.head_dim) {
        case 64: return attn::launch_all<64>(a, deal, s);
        case 128: return attn::launch_all<128>(a, deal, s);
        case 256: return attn::launch_all<256>(a, deal, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace qift
