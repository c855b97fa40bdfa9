// pa_decode_int4.cu -- paged decode attention over 4-bit caches (PA_INT4),
// every group size and head_dim.
//
// With codes u, row scales s, s' and lowest values l, l' (K and V),
//   x_t = c (s_t (q . u_t) + l_t sum(q)),   c = scale log2(e) k_scale
//   out = sum_t p_t (s'_t u'_t + l'_t) / sum_t p_t,   p_t = 2^(x_t - m)
// for any m; see below for the one taken.
// so the codes enter both products as integers 0..15 and the scales act on
// tokens: on a logit after the first product, on a weight before the second.
//
// One warp takes 32 tokens (two blocks) at a time with warp-level matrix
// instructions; for each block
//   S^T (16 tokens x rows) = U (16 x D) . Q^T       m16n8k32, u8 x s8 -> s32
//   O^T (D x rows)        += U'^T (D x 16) . W^T    m16n8k16, f16 -> f32
// with W = 2^-24 p s'.  Unpacking is what bounds such a kernel (logic runs at half
// the issue rate), so the nibbles are used where they stand:
//   - K: w & 0x0f0f0f0f are four codes as bytes, w & 0xf0f0f0f0 four codes
//     times 16 as unsigned bytes: one instruction for four.  The two halves
//     add up in accumulators of their own.  Q goes in as two s8 parts, q = (256
//     hi + lo) 2^-e rounded to integers of at most 32639, the largest |q| of a row
//     at 16320 or above (exact for fp16 elements down to a 15th of it, for bf16
//     ones down to a 127th); a row's two parts are two columns of the product, so
//     8 columns hold 4 rows and a lane gets both parts of one row and adds them as
//     integers.
//   - V pairs two tokens in a register: a transposing matrix load of 16-bit
//     elements brings four codes of one token and the same four dims' codes of
//     the next into one word, and w & 0x000f000f or w & 0x00f000f0 is then a
//     pair of fp16 subnormals u 2^-24 or 16 u 2^-24, exactly, which the matrix
//     units take as they are (with one shift by 8 five instructions for eight
//     codes).
// The contraction over dims may run in any order, so a lane's codes are the
// consecutive bytes that it loads, and Q is laid out to match.  S's
// accumulator layout (token, row) becomes W's operand layout by movmatrix.
// A warp needs no other warp: no shared-memory round trip, no barrier in the
// loop and no tensor memory:
// with 5th-generation MMAs the codes would be written back to shared memory,
// widened, before the MMA could read them, and each 128-token chunk would
// wait for S to come back from TMEM and for P to go in; the FP8 kernel that is
// built so takes 97 us for the 8B step, over about twice the bytes; this one 80
// (4.9 TB/s of 4-bit rows; 7B batch 62 us, 70B long context 64, four draft
// tokens 143).  What bounds it: with up to 8 rows the unpacking and the copies'
// issue beside DRAM (steady state 0.81 of the copy rate), with 16 the matrix
// instructions and two CTAs' worth of warps per SM (0.56); then what each
// context's start costs.
//
// Weights are f16, and so that they stay inside its range a row's m follows the
// running maximum of x_t + log2 |s'_t| of the tokens that the row attends to, not
// that of x_t: a V scale counts as far as the row's softmax lets it, and one that
// the row does not see not at all.  The largest weight stands between 2^6 and
// 2^15; below 2^-14 f16 loses bits and below 2^-25 everything, which is then
// under 2^-31 of that largest.  (s' counts at least as 2^-20 |l'|, so that the
// sum of p l' keeps inside fp32, and as 2^-70: fp32 holds p from 2^-126 to 2^127,
// the factor 2^-24 shares that range out between large and small scales.)
// A code is 0..15 and not -8..7, so a weight's rounding error would count 7.5
// codes where a centred code's would cancel.  With up to 4 rows the rounding's
// remainder, times 2^11, takes the second column of each row (hi + 2^-11 lo: 22
// bits, down to 2^-42 of the largest); with more, the weights' sum before and
// after the rounding (the latter by one more MMA against ones) says what it took,
// which is given back at the middle code 7.5.
//
// Two kernels share the warp's work.  decode_int4_kernel: CTA = (partition, KV
// head, sequence), the warps take every 4th pair of blocks and merge their
// states in shared memory; used for partitions that the caller sized and for
// short contexts.  decode_int4_balanced_kernel: one wave of resident warps,
// in teams on neighbouring KV heads, each team taking an equal share of all
// blocks in their flat order, whatever the lengths; a piece of a context that its warp does not
// hold whole goes to the workspace, and merge_int4_kernel joins the pieces.
#include <cfloat>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_int4.cuh"
#include "pa_simt.cuh"

namespace pa {

namespace {

constexpr int kWarps = kInt4Warps;
constexpr int kStages = 3;  // per warp, of two blocks each: up to 12 chunks in flight
constexpr float kTwo24 = 16777216.f;
constexpr float kScaleUnit = 1.f / kTwo24;  // of s' in W
constexpr float kLowUnit = 0x1p-44f;        // what |l'| counts as in W's range
constexpr float kLeastScale = 0x1p-94f;     // what any token counts as
constexpr float kNewWeight = 6.f;           // a new m puts the largest weight at 2^6,
constexpr float kMaxWeight = 15.f;          // and 2^15 calls for a new one: inside f16, as the remainder times 2^11 is
constexpr float kLowPart = 2048.f;

// D += A B, one m16n8k16 of f16.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D += A B, one m16n8k32 of u8 and s8.
__device__ __forceinline__ void mma_u8s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B: the first of a chain.
__device__ __forceinline__ void mma_u8s8_first(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// N 32-bit words from shared memory (N = 1, 2 or 4, aligned to N words).
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], uint32_t addr) {
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
}
__device__ __forceinline__ float2 load_ends(uint32_t addr) {
    uint32_t w[1];
    load_words<1>(w, addr);
    return int4_ends(w[0]);
}

// Four 8x8 matrices of 16-bit elements, each transposed: lane (r, q) gets
// elements (2q, r) and (2q + 1, r); lane 8 i + k gives the address of row k of
// matrix i.
__device__ __forceinline__ void load_matrix4_trans(uint32_t (&w)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
}

// Asynchronous copies of 16 bytes per lane from global to shared memory, in
// groups that complete in order.  A warp moves its chunks with these rather
// than with bulk copies: a bulk copy is issued by one thread with uniform
// operands, so four chunks at four addresses cost four issues of about ten
// instructions each, where nine copies per lane and their addresses cost
// thirty in all (measured at 592 contexts of 8192 tokens, 4 rows: 411 -> 337
// instructions for 32 tokens).
__device__ __forceinline__ void copy16(uint32_t dst, const unsigned char *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// max of three, NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The blocks of one (sequence, KV head) that a warp works on: pair j is table
// entries first + 2 stride j and the one after it, those below `end`.
struct Int4Span {
    int s, kvh, L, first, stride, end, pairs;
};

// A warp's state for RT tiles of 4 query rows (RT = 1, 2 or 4).  Lane (r, q) =
// (lane / 4, lane % 4) holds
//   of S: tokens r and 8 + r of each block, query row 4 n + q of each tile n;
//   of K: D / 4 dims from D / 4 q of those tokens;
//   of V: dims 32 g + 4 r .. + 3 of tokens 2q, 2q + 1, 8 + 2q and 9 + 2q;
//   of O: those dims, query rows 4 n + q.
template <typename T, int D, int RT, bool kMasked>
struct Int4Warp {
    using E = Elem<T>;
    static constexpr int KW = D / 32;                    // words of K per lane and token
    static constexpr int MT = D / 16;                    // tiles of 16 dims
    static constexpr int NP = RT == 1 ? 1 : RT / 2;      // column tiles of the second product
    static constexpr bool kSplit = RT == 1;              // weights as two f16 parts
    static constexpr bool kOneSum = RT > 1;              // odd dims' codes shifted, one accumulator
    static constexpr int kChunk = int4_chunk_bytes(D);

    uint32_t qb[RT][2 * KW];
    float fac[RT], off_q[RT];
    int lo[RT], hi[RT];   // attended positions
    int lo_any, lo_all, hi_all;  // seen by some row from lo_any; by all rows in [lo_all, hi_all]
    float m[RT], l[RT], z[RT], zw[RT], acc[NP][MT][4], accw[NP][4];

    // Query rows of (s, kvh): q = (256 hi + lo) 2^-e; this lane makes part r & 1 of
    // row 4 n + r / 2, the dims it holds of K, per word (8 dims) the even dims'
    // bytes and the odd dims'.  logit = s T fac + low off with T = 16 q . u (u
    // alone with kOneSum: q . u) as an integer.
    __device__ __forceinline__ void start(const DecodeParams &p, int s, int kvh, int L, int lane) {
        const int r = lane >> 2, q = lane & 3, rows = p.group * p.q_len;
#pragma unroll
        for (int n = 0; n < RT; ++n) {
            const int h = 4 * n + (r >> 1);
            const bool real = h < rows;
            const T *src = reinterpret_cast<const T *>(p.q) + query_row(p, s, kvh, real ? h : 0) * D + q * (D / 4);
            float y[D / 4];
#pragma unroll
            for (int i = 0; i < KW; ++i) {
                const uint4 w = real ? *reinterpret_cast<const uint4 *>(src + 8 * i) : make_uint4(0, 0, 0, 0);
                const float2 a = E::to_float2(w.x), b = E::to_float2(w.y), c = E::to_float2(w.z), d = E::to_float2(w.w);
                y[8 * i] = a.x, y[8 * i + 1] = a.y, y[8 * i + 2] = b.x, y[8 * i + 3] = b.y;
                y[8 * i + 4] = c.x, y[8 * i + 5] = c.y, y[8 * i + 6] = d.x, y[8 * i + 7] = d.y;
            }
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < D / 4; i += 2) mx = max3_nan(mx, fabsf(y[i]), fabsf(y[i + 1]));
            mx = max3_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 1), 0.f);
            mx = max3_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 2), 0.f);
            const bool fine = mx <= FLT_MAX;  // no NaN, no infinity
            int e = 0;
            if (mx > 0.f && fine) {
                const float half = frexpf(mx, &e);  // mx = half 2^e, half in [1/2, 1)
                e = min((half > 32639.f / 32768.f ? 14 : 15) - e, 120);
            }
            // 1.5 2^23 + v holds the integer v in its low bits.  |v| <= 32639, so
            // that v = 256 hi + lo with both parts in s8: lo the low byte, hi the
            // next one of v + 128.  (A row that is not fine may give anything: its
            // factor is NaN.)
            constexpr float kInt = 12582912.f;
            const float up = ldexpf(1.f, e);
            const uint32_t part_add = (r & 1) ? 0 : 128;
            const int part_shift = (r & 1) ? 0 : 8;
            uint32_t sum = 0;
#pragma unroll
            for (int w = 0; w < KW; ++w)
#pragma unroll
                for (int odd = 0; odd < 2; ++odd) {
                    uint32_t v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t k = __float_as_uint(fmaf(y[8 * w + 2 * i + odd], up, kInt));
                        sum += k;
                        v[i] = (k + part_add) >> part_shift;
                    }
                    qb[n][2 * w + odd] = __byte_perm(__byte_perm(v[0], v[1], 0x0040), __byte_perm(v[2], v[3], 0x0040), 0x5410);
                }
            sum -= (uint32_t)(D / 4) * 0x4b400000u;  // the constant's bits
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const float f = fine ? ldexpf(p.scale_log2, -e) : NAN;
            fac[n] = __shfl_sync(0xffffffffu, f, 8 * q) * (kOneSum ? 1.f : 0.0625f);
            off_q[n] = __shfl_sync(0xffffffffu, (float)(int)sum * f, 8 * q);
            m[n] = -INFINITY;
            l[n] = z[n] = zw[n] = 0.f;
            if constexpr (kMasked) row_range(p, L, 4 * n + q, &lo[n], &hi[n]);
        }
        if constexpr (kMasked) {
            lo_any = p.window > 0 ? L - p.q_len - p.window + 1 : 0;
            lo_all = p.window > 0 ? L - p.window : 0;
            hi_all = L - p.q_len;
        }
#pragma unroll
        for (int n = 0; n < NP; ++n) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][t][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) accw[n][i] = 0.f;
        }
    }

    // Folds the two blocks at shared address `stage` into the state.  kEdge: not
    // every row sees all 32 tokens; tok0 is the position of the first, tokens
    // from tend on are not there.  `release` is called once the stage is in
    // registers.
    template <bool kEdge, typename F>
    __device__ __forceinline__ void pair(uint32_t stage, int tok0, int tend, int lane, F release) {
        const int r = lane >> 2, q = lane & 3;
        float2 ke[4], ce[4];  // (scale, low) of the lane's tokens r, 8 + r, 16 + r, 24 + r in K and V
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t e = stage + 4 * r + 2 * (i >> 1) * kChunk + int4_ends_offset(D) + 32 * (i & 1);
            ke[i] = load_ends(e);
            ce[i] = load_ends(e + kChunk);
        }
        // S^T = U Q^T.  kOneSum: all dims' codes 0..15; otherwise the odd dims'
        // codes stay times 16, in accumulators of their own (one shift less per
        // word, two multiply-adds more per logit)
        float raw[RT][4], x[RT][4];  // T of the four tokens, the logits minus m
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t k0[KW], k1[KW];
            const uint32_t kp = stage + r * (D / 2) + q * (D / 8) + 2 * b * kChunk;
            load_words<KW>(k0, kp);
            load_words<KW>(k1, kp + 8 * (D / 2));
            int ev[RT][4], od[RT][4];
#pragma unroll
            for (int w = 0; w < KW; w += 2) {
                const uint32_t a0 = k0[w] & 0x0f0f0f0fu, a1 = k1[w] & 0x0f0f0f0fu, a2 = k0[w + 1] & 0x0f0f0f0fu,
                               a3 = k1[w + 1] & 0x0f0f0f0fu;
#pragma unroll
                for (int n = 0; n < RT; ++n) {
                    if (w == 0) mma_u8s8_first(ev[n], a0, a1, a2, a3, qb[n][2 * w], qb[n][2 * w + 2]);
                    else mma_u8s8(ev[n], a0, a1, a2, a3, qb[n][2 * w], qb[n][2 * w + 2]);
                }
                if constexpr (kOneSum) {
                    const uint32_t c0 = (k0[w] >> 4) & 0x0f0f0f0fu, c1 = (k1[w] >> 4) & 0x0f0f0f0fu,
                                   c2 = (k0[w + 1] >> 4) & 0x0f0f0f0fu, c3 = (k1[w + 1] >> 4) & 0x0f0f0f0fu;
#pragma unroll
                    for (int n = 0; n < RT; ++n) mma_u8s8(ev[n], c0, c1, c2, c3, qb[n][2 * w + 1], qb[n][2 * w + 3]);
                } else {
                    const uint32_t c0 = k0[w] & 0xf0f0f0f0u, c1 = k1[w] & 0xf0f0f0f0u, c2 = k0[w + 1] & 0xf0f0f0f0u,
                                   c3 = k1[w + 1] & 0xf0f0f0f0u;
#pragma unroll
                    for (int n = 0; n < RT; ++n) {
                        if (w == 0) mma_u8s8_first(od[n], c0, c1, c2, c3, qb[n][2 * w + 1], qb[n][2 * w + 3]);
                        else mma_u8s8(od[n], c0, c1, c2, c3, qb[n][2 * w + 1], qb[n][2 * w + 3]);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < RT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int e = ev[n][2 * i] * 256 + ev[n][2 * i + 1];
                    raw[n][2 * b + i] = (float)(kOneSum ? e : e * 16 + (od[n][2 * i] * 256 + od[n][2 * i + 1]));
                }
        }
        bool dead[RT][4];
        if constexpr (kEdge) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = tok0 + 8 * i + r;
                // rows that no query sees may hold anything
                if (tok >= tend || (kMasked && tok < lo_any)) ce[i] = make_float2(0.f, 0.f);
#pragma unroll
                for (int n = 0; n < RT; ++n) dead[n][i] = tok >= tend || (kMasked && (tok < lo[n] || tok > hi[n]));
            }
        }
        auto logits = [&](int n) {  // +inf before the first m
#pragma unroll
            for (int i = 0; i < 4; ++i) x[n][i] = fmaf(ke[i].x * fac[n], raw[n][i], fmaf(ke[i].y, off_q[n], -m[n]));
            if constexpr (kEdge) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (dead[n][i]) x[n][i] = -INFINITY;
            }
        };
        // m is raised only when a weight leaves its range: looked at is the lane's
        // largest p times its largest scale, by exponents (NaN takes this way too)
        float most = -INFINITY;
#pragma unroll
        for (int n = 0; n < RT; ++n) {
            logits(n);
            most = max3_nan(most, x[n][0], x[n][1]);
            most = max3_nan(most, x[n][2], x[n][3]);
        }
        const float big_s = max3_nan(max3_nan(fabsf(ce[0].x), fabsf(ce[1].x), fabsf(ce[2].x)), fabsf(ce[3].x), kLeastScale / kScaleUnit);
        const float big_l = max3_nan(max3_nan(fabsf(ce[0].y), fabsf(ce[1].y), fabsf(ce[2].y)), fabsf(ce[3].y), 0.f);
        const float big4 = max3_nan(big_s, big_l * (kLowUnit / kScaleUnit), 0.f);  // in [2^(e - 127), 2^(e - 126)), e its exponent bits
        const float e4 = __uint_as_float(0x4b000000u + (__float_as_uint(big4) >> 23));  // 2^23 + e
        if (__any_sync(0xffffffffu, !(most <= (8388608.f + kMaxWeight + 24.f + 126.f) - e4))) {
            float lg[4];  // what a token's scale adds to its logit
#pragma unroll
            for (int i = 0; i < 4; ++i)
                lg[i] = __log2f(max3_nan(fabsf(ce[i].x) * kScaleUnit, fabsf(ce[i].y) * kLowUnit, kLeastScale));
#pragma unroll
            for (int n = 0; n < RT; ++n) {
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = fmaf(ke[i].x * fac[n], raw[n][i], ke[i].y * off_q[n]) + lg[i];
                    if (kEdge && dead[n][i]) v = -INFINITY;
                    top = fmaxf(top, v != v ? 0.f : v);  // a NaN row gets a finite m and NaN sums
                }
#pragma unroll
                for (int o = 16; o > 2; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                float alpha = 1.f;
                if (top > m[n] + kMaxWeight) {  // a row's m does not depend on the other rows
                    alpha = ex2(m[n] - (top - kNewWeight));  // 0 on the first block
                    m[n] = top - kNewWeight;
                }
                l[n] *= alpha;
                z[n] *= alpha;
                zw[n] *= alpha;
                if constexpr (kSplit) {
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[0][t][i] *= alpha;
                } else {
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        acc[n / 2][t][n & 1] *= alpha;
                        acc[n / 2][t][2 + (n & 1)] *= alpha;
                    }
                    accw[n / 2][n & 1] *= alpha;
                }
                logits(n);
            }
        }
        // V's codes: pairs of tokens, four dims per word
        uint32_t vw[2][D / 32][2];  // [block][group of 32 dims][tokens 2q.., 8 + 2q..]
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint32_t vp = stage + (2 * b + 1) * kChunk;
            uint32_t w[4];
            if constexpr (D == 128) {
                uint32_t h[4];
                const uint32_t at = vp + (lane & 7) * 64 + (lane >> 3) * 16;
                load_matrix4_trans(w, at);
                load_matrix4_trans(h, at + 8 * 64);
#pragma unroll
                for (int g = 0; g < 4; ++g) vw[b][g][0] = w[g], vw[b][g][1] = h[g];
            } else {
                load_matrix4_trans(w, vp + ((lane & 7) + 8 * (lane >> 4)) * 32 + ((lane >> 3) & 1) * 16);
                vw[b][0][0] = w[0], vw[b][1][0] = w[1], vw[b][0][1] = w[2], vw[b][1][1] = w[3];
            }
        }
        __syncwarp();
        release();

        // weights, turned into the second product's operand
        uint32_t wb[NP][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float sv = ce[i].x * kScaleUnit;
            float w[RT];
#pragma unroll
            for (int n = 0; n < RT; ++n) {
                const float pr = ex2(x[n][i]);
                l[n] += pr;
                w[n] = pr * sv;
                float zz = ce[i].y;
                if (kEdge && kMasked && dead[n][i]) w[n] = zz = 0.f;  // a row that does not see a NaN stays clear of it
                z[n] = fmaf(pr, zz, z[n]);
                if constexpr (!kSplit) zw[n] += w[n];
            }
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                const __half2 h = kSplit ? __floats2half2_rn(w[0], (w[0] - __half2float(__float2half_rn(w[0]))) * kLowPart)
                                         : __floats2half2_rn(w[(2 * n) % RT], w[(2 * n + 1) % RT]);
                wb[n][i] = transpose8x8(*reinterpret_cast<const uint32_t *>(&h));
            }
        }
        // O^T += U'^T W^T: tile 2 g + u holds dims 32 g + 4 r + 2 u (and + 1, times 16)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int g = 0; g < D / 32; ++g) {
                const uint32_t a = vw[b][g][0], c = vw[b][g][1], a8 = a >> 8, c8 = c >> 8;
                const uint32_t a0 = a & 0x000f000fu, a1 = a & 0x00f000f0u, a2 = c & 0x000f000fu, a3 = c & 0x00f000f0u;
                const uint32_t c0 = a8 & 0x000f000fu, c1 = a8 & 0x00f000f0u, c2 = c8 & 0x000f000fu, c3 = c8 & 0x00f000f0u;
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    mma_f16(acc[n][2 * g], a0, a1, a2, a3, wb[n][2 * b], wb[n][2 * b + 1]);
                    mma_f16(acc[n][2 * g + 1], c0, c1, c2, c3, wb[n][2 * b], wb[n][2 * b + 1]);
                }
            }
            if constexpr (!kSplit) {
                constexpr uint32_t kOnes = 0x3c003c00u;
#pragma unroll
                for (int n = 0; n < NP; ++n) mma_f16(accw[n], kOnes, kOnes, kOnes, kOnes, wb[n][2 * b], wb[n][2 * b + 1]);
            }
        }
    }

    // The pairs of `span`, through the warp's kStages stages at shared address
    // `ring` (four chunks each: K and V of two blocks).
    __device__ __forceinline__ void run(const DecodeParams &p, uint32_t ring, const Int4Span &span, int lane) {
        const int32_t *row = p.block_tables + (int64_t)span.s * p.max_blocks_per_seq;
        // the blocks of pairs 16 w .. 16 w + 15, one per lane; a last pair of one
        // block brings that block twice (the second copy's tokens are past tend)
        auto window = [&](int w) -> int32_t {
            const int b = span.first + span.stride * (16 * w + (lane >> 1)) * 2 + (lane & 1);
            return 16 * w < span.pairs ? (int32_t)checked_block(p, row[min(b, span.end - 1)]) : 0;
        };
        int32_t cur = window(0), next = window(1);
        // lanes 0 .. 15 bring K's chunk of a block, lanes 16 .. 31 V's, 256 bytes
        // of each at a time: two addresses per pair, and a chunk's bytes together
        const uint32_t block_bytes = (uint32_t)(p.num_kv_heads * kChunk);
        const unsigned char *pool = reinterpret_cast<const unsigned char *>((lane & 16) ? p.v_cache : p.k_cache) +
                                    (int64_t)span.kvh * kChunk + 16 * (lane & 15);
        const uint32_t ring_lane = ring + (lane >> 4) * kChunk + 16 * (lane & 15);
        auto issue = [&](int j, int st) {  // pair j (ascending) into stage st
            if ((j & 15) == 0 && j > 0) {
                cur = next;
                next = window(j / 16 + 1);
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint32_t block = (uint32_t)__shfl_sync(0xffffffffu, cur, ((j & 15) << 1) + b);
                const unsigned char *src = pool + (uint64_t)block * block_bytes;
                const uint32_t dst = ring_lane + (st * 4 + 2 * b) * kChunk;
#pragma unroll
                for (int i = 0; i < 8 * D; i += 256) copy16(dst + i, src + i);
                if ((lane & 15) < 4) copy16(dst + 8 * D, src + 8 * D);
            }
        };
#pragma unroll
        for (int j = 0; j < kStages; ++j) {
            if (j < span.pairs) issue(j, j);
            copy_commit();
        }
        start(p, span.s, span.kvh, span.L, lane);
        const int tend = min(span.L, span.end * kBlock);
        int st = 0, tok0 = span.first * kBlock;
#pragma unroll 1
        for (int j = 0; j < span.pairs; ++j) {
            copy_wait<kStages - 1>();
            __syncwarp();
            auto release = [&] {  // the pair is in registers: its stage may be filled again
                if (j + kStages < span.pairs) issue(j + kStages, st);
                copy_commit();
            };
            const bool whole = tok0 + 2 * kBlock <= tend && (!kMasked || (tok0 >= lo_all && tok0 + 2 * kBlock - 1 <= hi_all));
            const uint32_t stage = ring + st * 4 * kChunk;
            if (whole) pair<false>(stage, tok0, tend, lane, release);
            else pair<true>(stage, tok0, tend, lane, release);
            tok0 += 2 * span.stride * kBlock;
            st = st == kStages - 1 ? 0 : st + 1;
        }
        __syncwarp();  // the stages may be filled again
    }

    // Sums over the warp's lanes; then row 4 n + q has weight l[n], and
    // output(n, g) its unnormalised dims 32 g + 4 r .. + 3.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int n = 0; n < RT; ++n) {
#pragma unroll
            for (int o = 16; o > 2; o >>= 1) {
                l[n] += __shfl_xor_sync(0xffffffffu, l[n], o);
                z[n] += __shfl_xor_sync(0xffffffffu, z[n], o);
                if constexpr (!kSplit) zw[n] += __shfl_xor_sync(0xffffffffu, zw[n], o);
            }
            if constexpr (!kSplit) z[n] = fmaf(zw[n] - accw[n / 2][n & 1], 7.5f / kScaleUnit, z[n]);
        }
    }
    __device__ __forceinline__ float4 output(int n, int g) const {
        constexpr float kUnit = kTwo24 / kScaleUnit;
        float o[4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float *a = acc[n / 2][2 * g + u];
            o[2 * u] = fmaf(kSplit ? fmaf(a[1], 1.f / kLowPart, a[0]) : a[n & 1], kUnit, z[n]);
            o[2 * u + 1] = fmaf(kSplit ? fmaf(a[3], 1.f / kLowPart, a[2]) : a[2 + (n & 1)], kUnit / 16.f, z[n]);
        }
        return make_float4(o[0], o[1], o[2], o[3]);
    }
};

// Tiles of 4 query rows a launch for `rows` rows takes: 1, 2 or 4.
constexpr int int4_row_tiles(int rows) { return rows <= 4 ? 1 : rows <= 8 ? 2 : 4; }

// CTAs per SM: 4 while the state fits 128 registers.
__host__ __device__ constexpr int int4_ctas_per_sm(int RT) { return RT == 1 ? 4 : RT == 2 ? 3 : 2; }

// Shared memory of a CTA: the warps' stages (reused for the warps' outputs by
// the partitioned kernel), then their m and l.
struct Int4Layout {
    int main, bytes;
    __host__ __device__ constexpr Int4Layout(int D, int rows)
        : main(kWarps * kStages * 4 * int4_chunk_bytes(D) > kWarps * rows * D * 4
                   ? kWarps * kStages * 4 * int4_chunk_bytes(D)
                   : kWarps * rows * D * 4),
          bytes(main + 2 * kWarps * rows * 4) {}
};

// CTA = (partition, KV head, sequence); warp w takes pairs w, w + 4, ...
template <typename T, int D, int RT, bool kMasked>
__global__ void __launch_bounds__(kWarps * 32, int4_ctas_per_sm(RT)) decode_int4_kernel(const DecodeParams p) {
    using E = Elem<T>;
    constexpr int RW = 4 * RT;
    constexpr Int4Layout Lay(D, RW);
    extern __shared__ __align__(128) unsigned char smem[];
    const int part = blockIdx.x, kvh = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, q = lane & 3;
    pdl_launch_dependents();
    pdl_wait();
    const int s = scheduled_seq(p, blockIdx.z, part == 0 && kvh == 0 && tid == 0);
    const SeqSplit sp = s < 0 ? SeqSplit{0, 0, 0, 0} : seq_split(p, s, part == 0 && kvh == 0 && tid == 0);
    if (part >= sp.nparts) return;  // s < 0 too
    const int rows = p.group * p.q_len;
    T *out = reinterpret_cast<T *>(p.out);
    if (sp.L == 0) {
        for (int i = tid; i < rows * D; i += blockDim.x) out[query_row(p, s, kvh, i / D) * D + i % D] = E::from_float(0.f);
        return;
    }
    const int b0 = sp.bfirst + part * p.part_blocks, b1 = min(b0 + p.part_blocks, sp.nblk);
    const int pairs = (b1 - b0 + 1) / 2;
    Int4Warp<T, D, RT, kMasked> w;
    const Int4Span span{s, kvh, sp.L, b0 + 2 * warp, kWarps, b1, max(0, (pairs - warp + kWarps - 1) / kWarps)};
    w.run(p, smem_addr(smem) + warp * kStages * 4 * int4_chunk_bytes(D), span, lane);
    __syncthreads();  // every warp is done with its stages
    w.finish();
    float *red_acc = reinterpret_cast<float *>(smem);
    float *red_m = reinterpret_cast<float *>(smem + Lay.main), *red_l = red_m + kWarps * RW;
#pragma unroll
    for (int n = 0; n < RT; ++n) {
        const int h = 4 * n + q;
        if (h >= rows) continue;
        // each warp's quotient and log-sum-exp: the m of two warps may be further apart than fp32's exponents
        const float inv = w.l[n] == 0.f ? 0.f : 1.f / w.l[n];
#pragma unroll
        for (int g = 0; g < D / 32; ++g) {
            const float4 v = w.output(n, g);
            *reinterpret_cast<float4 *>(red_acc + (warp * RW + h) * D + 32 * g + 4 * r) =
                w.l[n] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        }
        if (r == 0) {
            const float lse = w.l[n] == 0.f ? -INFINITY : w.m[n] + log2f(w.l[n]);
            red_m[warp * RW + h] = lse != lse ? 0.f : lse;  // the NaN is in the quotient
            red_l[warp * RW + h] = w.l[n] == 0.f ? 0.f : 1.f;
        }
    }
    __syncthreads();
    for (int i = tid; i < rows * D; i += blockDim.x) {
        const int h = i / D, d = i % D;
        float lse;
        const float o = combine_warps<D, RW, kWarps>(red_m, red_l, red_acc, h, d, &lse) * p.v_scale;
        const int64_t qr = query_row(p, s, kvh, h);
        if (sp.nparts == 1) {
            out[qr * D + d] = E::from_float(o);
        } else {
            const int64_t row = qr * p.max_parts + part;
            p.ws_o[row * D + d] = o;
            if (d == 0) p.ws_lse[row] = lse != lse ? 0.f : lse;  // the NaN is in o: the merge must not skip it
        }
    }
}

// ---------------------------------------------------------------------------
// equal shares
// ---------------------------------------------------------------------------
// A team of 2^team_bits warps (4, 2 or 1, whatever divides num_kv_heads) takes
// as many neighbouring KV heads of the same blocks, a warp each: the team's
// chunks of a block are one run of DRAM (measured, reads alone: 6.4 TB/s against
// 5.9-6.2 with every warp on a context of its own; the 4-token 8B step 210 ->
// 168 us).  The flat order: sequences, in each its head groups, in each
// start_cost places for what a context costs before its first block (its query
// rows, the first copies' latency) and then its blocks.  Team t owns places
// [t W, (t + 1) W).
// The start cost is 8 blocks' time, with 16 rows, whose queries and outputs are
// four times as many, 14 (the 8B batch with 16 rows per KV head: 160 us at 5, 150
// at 8, 143 at 14, 145 at 18; with 4 rows: 79 at 5, 80 at 8, 81 at 12, 92 at 18).
__host__ __device__ constexpr int int4_start_cost(int RT) { return RT == 4 ? 14 : 8; }

// Blocks that sequence s's queries attend to, from which entry, and its length.
struct Int4Seq {
    int L, first, n;
};
__device__ __forceinline__ Int4Seq int4_seq(const DecodeParams &p, int s, bool report) {
    const SeqSplit sp = seq_split(p, s, report);  // max_parts is 1: longer contexts are flagged and cut
    return {sp.L, sp.bfirst, min(sp.nblk - sp.bfirst, p.part_blocks)};
}

// A share is never less than a start and 8 blocks.
__device__ __forceinline__ int int4_share(int total, int teams, int start_cost) {
    return max(start_cost + 8, (total + teams - 1) / teams);
}

// places: int32 [num_seqs + 1] in the workspace, written for the merge: each
// sequence's first place and the total.  (The host keeps totals that pass 30
// bits off this kernel.)
template <typename T, int D, int RT, bool kMasked>
__global__ void __launch_bounds__(kWarps * 32, int4_ctas_per_sm(RT))
    decode_int4_balanced_kernel(const DecodeParams p, int32_t *places, const int team_bits) {
    using E = Elem<T>;
    constexpr int kThreads = kWarps * 32, kCost = int4_start_cost(RT);
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t chunk_end[kThreads];  // 64-bit: with half the static shared memory the compiler's code for the
    __shared__ int64_t warp_sum[kWarps];     // loop over blocks came out slower (7B batch 62 us against 69.5, 8B 80.5 against 90.5)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, q = lane & 3;
    pdl_launch_dependents();
    const uint32_t ring = smem_addr(smem) + warp * kStages * 4 * int4_chunk_bytes(D);
    const int groups = p.num_kv_heads >> team_bits, member = warp & ((1 << team_bits) - 1);
    pdl_wait();
    // places of all sequences: each thread sums a run of them, then a scan
    const int per = (p.num_seqs + kThreads - 1) / kThreads, s0 = min(tid * per, p.num_seqs), s1 = min(s0 + per, p.num_seqs);
    const bool report = blockIdx.x == 0;
    int sum = 0;
    for (int s = s0; s < s1; ++s) sum += groups * (kCost + int4_seq(p, s, report).n);
    int scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    for (int w = 0; w < warp; ++w) scan += (int)warp_sum[w];
    chunk_end[tid] = scan;
    __syncthreads();
    const int total = (int)chunk_end[kThreads - 1];
    const int teams = ((int)gridDim.x * kWarps) >> team_bits, share = int4_share(total, teams, kCost);
    if (blockIdx.x == 0) {
        int at = scan - sum;
        for (int s = s0; s < s1; ++s) {
            places[s] = at;
            at += groups * (kCost + int4_seq(p, s, false).n);
        }
        if (tid == 0) places[p.num_seqs] = total;
        if (p.seq_order)  // results and shares do not depend on it; it is checked all the same
            for (int i = tid; i < p.num_seqs; i += kThreads) (void)scheduled_seq(p, i, true);
    }
    const int me = (int)blockIdx.x * kWarps + warp;
    const int64_t begin = (int64_t)(me >> team_bits) * share;
    int x = (int)min((int64_t)total, begin);
    const int xend = (int)min((int64_t)total, begin + share);
    if (x >= xend) return;
    // the sequence of place x: the thread whose run holds it, then its run
    int c = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) c += __popc(__ballot_sync(0xffffffffu, chunk_end[32 * i + lane] <= x));
    int s = c * per;
    int at = c == 0 ? 0 : (int)chunk_end[c - 1];  // first place of sequence s
    Int4Seq seq = int4_seq(p, s, false);
    while (x >= at + groups * (kCost + seq.n)) {
        at += groups * (kCost + seq.n);
        seq = int4_seq(p, ++s, false);
    }
    int group = (x - at) / (kCost + seq.n);
    at += group * (kCost + seq.n);  // first place of (s, group)
    const int rows = p.group * p.q_len;
    T *out = reinterpret_cast<T *>(p.out);
    for (;;) {
        const int blocks_at = at + kCost;
        const int kvh = (group << team_bits) + member;
        const int from = max(0, x - blocks_at), to = min(seq.n, xend - blocks_at);
        if (seq.n == 0 && x <= at) {  // an empty context: zero rows
            for (int i = lane; i < rows * D; i += 32) out[query_row(p, s, kvh, i / D) * D + i % D] = E::from_float(0.f);
        } else if (to > from) {
            Int4Warp<T, D, RT, kMasked> w;
            const Int4Span span{s, kvh, seq.L, seq.first + from, 1, seq.first + to, (to - from + 1) / 2};
            w.run(p, ring, span, lane);
            w.finish();
            const bool all = from == 0 && to == seq.n;
            const int64_t slot = 2 * (int64_t)me + (from == 0 ? 1 : 0);  // the context's first piece, or a later one
#pragma unroll
            for (int n = 0; n < RT; ++n) {
                const int h = 4 * n + q;
                if (h >= rows) continue;
                const float inv = w.l[n] == 0.f ? 0.f : p.v_scale / w.l[n];
                const int64_t qr = query_row(p, s, kvh, h);
#pragma unroll
                for (int g = 0; g < D / 32; ++g) {
                    const float4 v = w.output(n, g);
                    const float4 o = w.l[n] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                   : make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                    if (all) {
                        const typename E::T2 a = {E::from_float(o.x), E::from_float(o.y)};
                        const typename E::T2 b = {E::from_float(o.z), E::from_float(o.w)};
                        *reinterpret_cast<uint2 *>(out + qr * D + 32 * g + 4 * r) =
                            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
                    } else {
                        *reinterpret_cast<float4 *>(p.ws_o + (slot * rows + h) * D + 32 * g + 4 * r) = o;
                    }
                }
                if (!all && r == 0) {
                    const float lse = w.l[n] == 0.f ? -INFINITY : w.m[n] + log2f(w.l[n]);
                    p.ws_lse[slot * rows + h] = lse != lse ? 0.f : lse;  // the NaN is in o: the merge must not skip it
                }
            }
        }
        at = blocks_at + seq.n;
        x = at;
        if (x >= xend) return;
        if (++group == groups) {
            group = 0;
            seq = int4_seq(p, ++s, false);
        }
    }
}

// Joins the pieces of contexts that no warp held whole: out = sum_i 2^(lse_i -
// M) o_i / sum_i 2^(lse_i - M), M = max lse.  CTA = (4 kRows / kRowWarps query
// rows of a sequence).  Where contexts have few pieces a warp takes kRows = 4
// neighbouring rows of one KV head, whose pieces and places are the same (1
// where the KV head's rows are no multiple of 4); where they have many, four
// warps share one row's pieces.
template <typename T, int D, int kRowWarps, int kRows>
__global__ void __launch_bounds__(128) merge_int4_kernel(const DecodeParams p, const int32_t *places, const int teams, const int team_bits,
                                                         const int start_cost) {
    using E = Elem<T>;
    constexpr int kV = D / 32;
    static_assert(kRowWarps == 1 || kRows == 1, "several warps share one row");
    __shared__ float red[kRowWarps == 4 ? 4 : 1][D + 1];
    const int s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    const Int4Seq seq = int4_seq(p, s, false);
    const int rows = p.group * p.q_len;
    const int row = (blockIdx.x * (4 / kRowWarps) + warp / kRowWarps) * kRows;  // query row of the sequence, KV head by KV head
    const bool real = row < p.num_kv_heads * rows;
    const int kvh = real ? row / rows : 0, h = real ? row % rows : 0;
    const int share = int4_share(places[p.num_seqs], teams, start_cost);
    const int at = places[s] + (kvh >> team_bits) * (start_cost + seq.n) + start_cost;
    const int ta = at / share;
    const int pieces = seq.n == 0 || !real ? 0 : (at + seq.n - 1) / share - ta + 1;
    if (pieces <= 1) return;  // written by its warp; with four warps to a row it is all four that leave
    // piece i: the first in the second slot of its warp, the others in the first
    const int member = kvh & ((1 << team_bits) - 1);
    auto slot = [&](int i) -> int64_t { return (2 * (((int64_t)(ta + i) << team_bits) + member) + (i == 0 ? 1 : 0)) * rows + h; };
    float M[kRows], acc[kRows][kV] = {}, wsum[kRows] = {};
#pragma unroll
    for (int n = 0; n < kRows; ++n) M[n] = -INFINITY;
    for (int i = lane; i < pieces; i += 32)
#pragma unroll
        for (int n = 0; n < kRows; ++n) M[n] = fmaxf(M[n], p.ws_lse[slot(i) + n]);
    constexpr int kInFlight = kRows == 4 ? 2 : 4;
    bool first = true;
    for (int i0 = warp % kRowWarps; i0 < pieces || first; i0 += kRowWarps * kInFlight) {
        float lse[kInFlight][kRows], v[kInFlight][kRows][kV];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {  // every piece was written: no need to look at its lse first
            const int i = i0 + k * kRowWarps;
            const int64_t at_row = slot(i);
#pragma unroll
            for (int n = 0; n < kRows; ++n) {
                lse[k][n] = i < pieces ? p.ws_lse[at_row + n] : -INFINITY;
                const float *src = p.ws_o + (at_row + n) * D + lane * kV;
                if constexpr (kV == 4) {
                    const float4 f = i < pieces ? *reinterpret_cast<const float4 *>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
                    v[k][n][0] = f.x, v[k][n][1] = f.y, v[k][n][2] = f.z, v[k][n][3] = f.w;
                } else {
                    const float2 f = i < pieces ? *reinterpret_cast<const float2 *>(src) : make_float2(0.f, 0.f);
                    v[k][n][0] = f.x, v[k][n][1] = f.y;
                }
            }
        }
        if (first) {
#pragma unroll
            for (int n = 0; n < kRows; ++n)
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) M[n] = fmaxf(M[n], __shfl_xor_sync(0xffffffffu, M[n], o));
            first = false;
        }
#pragma unroll
        for (int k = 0; k < kInFlight; ++k)
#pragma unroll
            for (int n = 0; n < kRows; ++n) {
                const float w = lse[k][n] == -INFINITY ? 0.f : ex2(lse[k][n] - M[n]);
                wsum[n] += w;
#pragma unroll
                for (int e = 0; e < kV; ++e) acc[n][e] = fmaf(w, v[k][n][e], acc[n][e]);
            }
    }
    if constexpr (kRowWarps == 4) {
#pragma unroll
        for (int e = 0; e < kV; ++e) red[warp][lane * kV + e] = acc[0][e];
        if (lane == 0) red[warp][D] = wsum[0];
        __syncthreads();
        if (warp != 0) return;
        wsum[0] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) wsum[0] += red[k][D];
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            acc[0][e] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[0][e] += red[k][lane * kV + e];
        }
    }
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
        const float inv = wsum[n] == 0.f ? 0.f : 1.f / wsum[n];
        T *dst = reinterpret_cast<T *>(p.out) + query_row(p, s, kvh, h + n) * D + lane * kV;
#pragma unroll
        for (int e = 0; e < kV; e += 2) {
            const typename E::T2 a = {E::from_float(acc[n][e] * inv), E::from_float(acc[n][e + 1] * inv)};
            *reinterpret_cast<typename E::T2 *>(dst + e) = a;
        }
    }
}

template <typename T, int D, int RT, bool kMasked>
cudaError_t launch_int4_t(const DecodeParams &p, int32_t *places, int ctas, cudaStream_t stream) {
    constexpr int kSmem = Int4Layout(D, 4 * RT).bytes;
    if (!places) {
        auto kern = decode_int4_kernel<T, D, RT, kMasked>;
        static FuncAttrCache attrs;
        cudaError_t e = ensure_smem(kern, kSmem, attrs, /*max_carveout=*/true);
        if (e != cudaSuccess) return e;
        e = launch_pdl(kern, dim3(p.max_parts, p.num_kv_heads, p.num_seqs), dim3(kWarps * 32), kSmem, stream, p);
        if (e != cudaSuccess || p.max_parts == 1) return e;
        return launch_merge_partitions(p, std::is_same<T, __nv_bfloat16>::value ? PA_BF16 : PA_F16, D, stream);
    }
    auto kern = decode_int4_balanced_kernel<T, D, RT, kMasked>;
    static FuncAttrCache attrs;
    cudaError_t e = ensure_smem(kern, kSmem, attrs, /*max_carveout=*/true);
    if (e != cudaSuccess) return e;
    const int team_bits = p.num_kv_heads % 4 == 0 ? 2 : p.num_kv_heads % 2 == 0 ? 1 : 0;
    const int teams = (ctas * kWarps) >> team_bits;
    e = launch_pdl(kern, dim3(ctas), dim3(kWarps * 32), kSmem, stream, p, places, team_bits);
    if (e != cudaSuccess) return e;
    // pieces a context may have: many on few sequences
    const int rows = p.num_heads * p.q_len, four = p.group * p.q_len % 4 == 0;
    const bool many = (int64_t)ctas * kWarps > 8 * (int64_t)p.num_seqs * p.num_kv_heads;
    const int32_t *at = places;
    const int cost = int4_start_cost(RT);
    if (many) return launch_pdl(merge_int4_kernel<T, D, 4, 1>, dim3(rows, p.num_seqs), dim3(128), 0, stream, p, at, teams, team_bits, cost);
    if (four) return launch_pdl(merge_int4_kernel<T, D, 1, 4>, dim3((rows + 15) / 16, p.num_seqs), dim3(128), 0, stream, p, at, teams, team_bits, cost);
    return launch_pdl(merge_int4_kernel<T, D, 1, 1>, dim3((rows + 3) / 4, p.num_seqs), dim3(128), 0, stream, p, at, teams, team_bits, cost);
}

template <typename T, int D>
cudaError_t launch_int4_d(const DecodeParams &p, int rows, int32_t *places, int ctas, cudaStream_t stream) {
    const bool masked = decode_masked(p);
    switch (int4_row_tiles(rows)) {
        case 1: return masked ? launch_int4_t<T, D, 1, true>(p, places, ctas, stream) : launch_int4_t<T, D, 1, false>(p, places, ctas, stream);
        case 2: return masked ? launch_int4_t<T, D, 2, true>(p, places, ctas, stream) : launch_int4_t<T, D, 2, false>(p, places, ctas, stream);
        default: return masked ? launch_int4_t<T, D, 4, true>(p, places, ctas, stream) : launch_int4_t<T, D, 4, false>(p, places, ctas, stream);
    }
}

}  // namespace

int decode_int4_ctas(int rows, int sms) { return sms * int4_ctas_per_sm(int4_row_tiles(rows)); }

cudaError_t launch_decode_int4(const DecodeParams &p, int dtype, int head_dim, int rows, int32_t *places, int ctas,
                               cudaStream_t stream) {
    if (dtype == PA_F16)
        return head_dim == 64 ? launch_int4_d<__half, 64>(p, rows, places, ctas, stream)
                              : launch_int4_d<__half, 128>(p, rows, places, ctas, stream);
    return head_dim == 64 ? launch_int4_d<__nv_bfloat16, 64>(p, rows, places, ctas, stream)
                          : launch_int4_d<__nv_bfloat16, 128>(p, rows, places, ctas, stream);
}

}  // namespace pa
