// pa_decode_int4.cu -- paged decode attention over 4-bit caches (PA_INT4),
// every group size and head_dim.
//
// With codes u, row scales s, s' and lowest values l, l' (K and V),
//   x_t = c (s_t (q . u_t) + l_t sum(q)),   c = scale log2(e) k_scale
//   out = sum_t p_t (s'_t u'_t + l'_t) / sum_t p_t,   p_t = 2^(x_t - m)
// so the codes enter both products as integers 0..15 and the scales act on
// tokens: on a logit after the first product, on a weight before the second.
//
// One warp takes 32 tokens (two blocks) at a time with warp-level matrix
// instructions; for each block
//   S^T (16 tokens x rows) = U (16 x D) . Q^T       m16n8k32, u8 x s8 -> s32
//   O^T (D x rows)        += U'^T (D x 16) . W^T    m16n8k16, f16 -> f32
// with W = p s'.  Unpacking is what bounds such a kernel (logic runs at half
// the issue rate), so the nibbles are used where they stand:
//   - K: w & 0x0f0f0f0f are four codes as bytes, w & 0xf0f0f0f0 four codes
//     times 16 as unsigned bytes: one instruction for four.  The two halves
//     add up in accumulators of their own.  Q goes in as two s8 parts, q =
//     (128 hi + lo) 2^-e rounded to 15 bits of the row's largest |q| (exact for
//     fp16 elements within 2^4 of it, for bf16 ones within 2^7); a row's two
//     parts are two columns of the product, so 8 columns hold 4 rows and a
//     lane gets both parts of one row and adds them as integers.
//   - V pairs two tokens in a register: a transposing matrix load of 16-bit
//     elements brings four codes of one token and the same four dims' codes of
//     the next into one word, and w & 0x000f000f or w & 0x00f000f0 is then a
//     pair of fp16 subnormals u 2^-24 or 16 u 2^-24, exactly, which the matrix
//     units take as they are (with one shift by 8 five instructions for eight
//     codes).
// The contraction over dims may run in any order, so a lane's codes are the
// consecutive bytes that it loads, and Q is laid out to match.  S's
// accumulator layout (token, row) becomes W's operand layout by movmatrix.
// No shared-memory round trip, no barrier in the loop and no tensor memory:
// with 5th-generation MMAs the codes would be written back to shared memory,
// widened, before the MMA could read them, and each 128-token chunk would
// wait for S to come back from TMEM and for P to go in; the FP8 kernel that is
// built so takes 97 us for the 8B step, over about twice the bytes.
//
// Weights are f16 under a power of two that follows the largest V scale seen.
// A code is 0..15 and not -8..7, so a weight's rounding error would count 7.5
// codes where a centred code's would cancel.  With up to 4 rows the rounding's
// remainder takes the second column of each row (hi + lo: 22 bits); with more,
// the remainders are summed and given back at the middle code 7.5.
#include <cfloat>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_int4.cuh"
#include "pa_simt.cuh"

namespace pa {

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 3;  // per warp, of two blocks each: up to 12 chunks in flight
constexpr float kTwo24 = 16777216.f;
constexpr float kMaxWeightScale = 64.f;  // times p <= 2^8 stays inside f16

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

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// N 32-bit words from shared memory (N = 1, 2 or 4, aligned to N words).
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const unsigned char *p) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
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

// Shared memory: per-warp stage rings (reused for the warps' outputs at the
// end), Q's operands (D / 16 words per lane and tile), the rows' factors, the
// warps' m and l, the mbarriers.
struct Int4Layout {
    int main, q_off, fac_off, ml_off, bar_off, bytes;
    __host__ __device__ constexpr Int4Layout(int D, int rows)
        : main(kWarps * kStages * 4 * int4_chunk_bytes(D) > kWarps * rows * D * 4
                   ? kWarps * kStages * 4 * int4_chunk_bytes(D)
                   : kWarps * rows * D * 4),
          q_off(main), fac_off(q_off + rows / 4 * (D / 16) * 128), ml_off(fac_off + rows * 8),
          bar_off(ml_off + 2 * kWarps * rows * 4), bytes(bar_off + kWarps * kStages * 8) {}
};

// Q's operands of row tile n (rows 4 n .. 4 n + 3), by one warp: lane (r, q)
// makes part r & 1 of row 4 n + r / 2, dims D / 4 q ..: per word w of K (8
// dims) the 4 even dims' parts, and the 4 odd dims'.
template <typename T, int D>
__device__ __forceinline__ void make_q_tile(uint32_t *dst, float2 *fac, const T *src, bool real, float scale_log2,
                                            int row, int lane) {
    using E = Elem<T>;
    constexpr int KW = D / 32;
    const int r = lane >> 2, q = lane & 3;
    float y[D / 4];
#pragma unroll
    for (int i = 0; i < KW; ++i) {
        const uint4 w = real ? *reinterpret_cast<const uint4 *>(src + q * (D / 4) + 8 * i) : make_uint4(0, 0, 0, 0);
        const float2 a = E::to_float2(w.x), b = E::to_float2(w.y), c = E::to_float2(w.z), d = E::to_float2(w.w);
        y[8 * i] = a.x, y[8 * i + 1] = a.y, y[8 * i + 2] = b.x, y[8 * i + 3] = b.y;
        y[8 * i + 4] = c.x, y[8 * i + 5] = c.y, y[8 * i + 6] = d.x, y[8 * i + 7] = d.y;
    }
    float mx = 0.f;
    int fine = 1;
#pragma unroll
    for (int i = 0; i < D / 4; ++i) {
        mx = fmaxf(mx, fabsf(y[i]));
        fine &= fabsf(y[i]) <= FLT_MAX;
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        fine &= __shfl_xor_sync(0xffffffffu, fine, o);
    }
    int e = 0;
    if (mx > 0.f && fine) {
        (void)frexpf(mx, &e);  // mx in [2^(e-1), 2^e)
        e = min(14 - e, 120);  // mx 2^e in [2^13, 2^14)
    }
    const float up = ldexpf(1.f, e);
    int sum = 0;
    uint32_t part[2 * KW];
#pragma unroll
    for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
            uint32_t bytes = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int v = fine ? min(__float2int_rn(y[8 * w + 2 * i + odd] * up), 16383) : 0;
                sum += v;
                bytes |= (uint32_t)(((r & 1) ? v & 127 : v >> 7) & 255) << (8 * i);
            }
            part[2 * w + odd] = bytes;
        }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
    for (int k = 0; k < 2 * KW; ++k) dst[k * 32 + lane] = part[k];
    // logit = s T f + l o with T = 16 q . u (as integers): f = c 2^-e / 16, o = c sum(q)
    if (q == 0 && (r & 1) == 0) {
        const float f = ldexpf(scale_log2, -e);
        fac[row] = fine ? make_float2(f * 0.0625f, (float)sum * f) : make_float2(NAN, NAN);
    }
}

// CTAs per SM: 4 while the state fits 128 registers.
__host__ __device__ constexpr int int4_ctas_per_sm(int RT) { return RT == 1 ? 4 : RT == 2 ? 3 : 2; }

// RT: tiles of 4 query rows (1, 2 or 4).  Lane (r, q) = (lane / 4, lane % 4)
// holds
//   of S: tokens r and 8 + r of each block, query row 4 n + q of each tile n;
//   of K: D / 4 dims from D / 4 q of those tokens;
//   of V: dims 32 g + 4 r .. + 3 of tokens 2q, 2q + 1, 8 + 2q and 9 + 2q;
//   of O: those dims, query rows 4 n + q.
template <typename T, int D, int RT, bool kMasked>
__global__ void __launch_bounds__(kWarps * 32, int4_ctas_per_sm(RT)) decode_int4_kernel(const DecodeParams p) {
    using E = Elem<T>;
    constexpr int KW = D / 32;   // words of K per lane and token
    constexpr int MT = D / 16;   // tiles of 16 dims
    constexpr int RW = 4 * RT;   // query rows
    constexpr int NP = RT == 1 ? 1 : RT / 2;  // column tiles of the second product
    constexpr bool kSplit = RT == 1;          // weights as two f16 parts
    constexpr int kChunk = int4_chunk_bytes(D);
    constexpr Int4Layout Lay(D, RW);
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int fail_s;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay.bar_off);
    const int part = blockIdx.x, kvh = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, q = lane & 3;
    pdl_launch_dependents();
    // Order, lengths and tables are read before the wait for the kernel in
    // front (no kernel of this library writes them), q and the caches after.
    const int s = scheduled_seq(p, blockIdx.z, part == 0 && kvh == 0 && tid == 0);
    const SeqSplit sp = s < 0 ? SeqSplit{0, 0, 0, 0} : seq_split(p, s, part == 0 && kvh == 0 && tid == 0);
    const int L = sp.L;
    // this warp's pairs of blocks: every kWarps-th of the partition
    const int b0 = sp.bfirst + part * p.part_blocks;
    const int b1 = min(b0 + p.part_blocks, sp.nblk);
    const int np = part < sp.nparts ? ((b1 - b0 + 1) / 2 - warp + kWarps - 1) / kWarps : 0;  // may be <= 0
    const int tend = min(L, b1 * kBlock);                                                    // this CTA's last token + 1
    auto block_of = [&](int e) -> int { return b0 + 2 * (warp + kWarps * (e >> 1)) + (e & 1); };
    auto window = [&](int w) -> int32_t {  // the blocks of pairs 16 w .. 16 w + 15, one per lane; -1 past the end
        const int b = block_of(32 * w + lane);
        return b < b1 && 16 * w < np ? (int32_t)checked_block(p, p.block_tables[(int64_t)s * p.max_blocks_per_seq + b]) : -1;
    };
    int32_t cur = window(0), next = window(1);
    uint64_t *wbar = bars + warp * kStages;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&wbar[i], 1);
        fence_mbar_init();
    }
    if (tid == 0) fail_s = 0;
    pdl_wait();
    if (part >= sp.nparts) return;  // s < 0 too
    const int rows = p.group * p.q_len;
    T *out = reinterpret_cast<T *>(p.out);
    auto row_of = [&](int h) -> int64_t {
        if constexpr (kMasked) return query_row(p, s, kvh, h);
        return (int64_t)s * p.num_heads + kvh * p.group + h;
    };
    if (L == 0) {
        for (int i = tid; i < rows * D; i += blockDim.x) out[row_of(i / D) * D + i % D] = E::from_float(0.f);
        return;
    }
    // the loads of pair j (all lanes, j in ascending order): lane i brings
    // chunk i of the stage (K and V of its first block, K and V of its second)
    unsigned char *ring = smem + warp * kStages * 4 * kChunk;
    const unsigned char *pool = reinterpret_cast<const unsigned char *>((lane & 1) ? p.v_cache : p.k_cache) + (int64_t)kvh * kChunk;
    const uint32_t block_bytes = (uint32_t)(p.num_kv_heads * kChunk);
    auto issue = [&](int j, int st) {
        if ((j & 15) == 0 && j > 0) {
            cur = next;
            next = window(j / 16 + 1);
        }
        const int32_t phys = __shfl_sync(0xffffffffu, cur, ((j & 15) << 1) + ((lane >> 1) & 1));
        const bool both = __shfl_sync(0xffffffffu, phys, 2) >= 0;
        if (lane < 4) {
            if (lane == 0) mbar_arrive_expect_tx(&wbar[st], both ? 4 * kChunk : 2 * kChunk);
            __syncwarp(15u);
            if (phys >= 0)
                bulk_g2s(ring + (st * 4 + lane) * kChunk, pool + (uint64_t)(uint32_t)phys * block_bytes, kChunk, &wbar[st]);
        }
    };
    __syncwarp();  // the barriers are initialised
    for (int j = 0; j < kStages && j < np; ++j) issue(j, j);

    // ---- query rows ---------------------------------------------------------
    uint32_t *q_s = reinterpret_cast<uint32_t *>(smem + Lay.q_off);
    float2 *fac_s = reinterpret_cast<float2 *>(smem + Lay.fac_off);
    if (warp < RT) {
        const int h = 4 * warp + (r >> 1);
        make_q_tile<T, D>(q_s + warp * (D / 16) * 32, fac_s, reinterpret_cast<const T *>(p.q) + row_of(h < rows ? h : 0) * D,
                          h < rows, p.scale_log2, h, lane);
    }
    __syncthreads();
    uint32_t qb[RT][2 * KW];
    float fac[RT], off_q[RT];
#pragma unroll
    for (int n = 0; n < RT; ++n) {
#pragma unroll
        for (int k = 0; k < 2 * KW; ++k) qb[n][k] = q_s[(n * 2 * KW + k) * 32 + lane];
        const float2 f = fac_s[4 * n + q];
        fac[n] = f.x;
        off_q[n] = f.y;
    }
    int lo[RT], hi[RT];  // attended positions
    int first = 0;       // first position any row attends to
    if constexpr (kMasked) {
        if (p.window > 0) first = L - p.q_len - p.window + 1;
#pragma unroll
        for (int n = 0; n < RT; ++n) row_range(p, L, 4 * n + q, &lo[n], &hi[n]);
    }

    // ---- state of rows 4 n + q ----------------------------------------------
    float m[RT], l[RT], z[RT], zc[RT], acc[NP][MT][4];
    float cv = 1.f;      // power of two the V scales are multiplied by (warp-uniform)
    float limit = 0.f;   // kMaxWeightScale / cv once it was chosen
#pragma unroll
    for (int n = 0; n < RT; ++n) {
        m[n] = -INFINITY;
        l[n] = z[n] = zc[n] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][t][i] = 0.f;
    const uint32_t ring_addr = smem_addr(ring);
    const int k_lane = r * (D / 2) + q * (D / 8);
    const int v_lane = D == 128 ? (lane & 7) * 64 + (lane >> 3) * 16 : ((lane & 7) + 8 * (lane >> 4)) * 32 + ((lane >> 3) & 1) * 16;
    bool ok = true;
    int j = 0, st = 0;
    uint32_t parity = 0;
#pragma unroll 1
    for (; j < np; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait(&wbar[st], parity))) {
            ok = false;
            break;
        }
        const unsigned char *stage = ring + st * 4 * kChunk;
        float2 ke[4], ce[4];  // (scale, low) of the lane's tokens r, 8 + r, 16 + r, 24 + r in K and V
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned char *e = stage + 2 * (i >> 1) * kChunk + int4_ends_offset(D) + 4 * (8 * (i & 1) + r);
            ke[i] = int4_ends(*reinterpret_cast<const uint32_t *>(e));
            ce[i] = int4_ends(*reinterpret_cast<const uint32_t *>(e + kChunk));
        }
        // S^T = U Q^T: even dims' codes, and odd dims' codes times 16
        float raw[RT][4], x[RT][4];  // T = 16 q . u of the four tokens, the logits minus m
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t k0[KW], k1[KW];
            load_words<KW>(k0, stage + 2 * b * kChunk + k_lane);
            load_words<KW>(k1, stage + 2 * b * kChunk + k_lane + 8 * (D / 2));
#pragma unroll
            for (int n = 0; n < RT; ++n) {
                int ev[4] = {0, 0, 0, 0}, od[4] = {0, 0, 0, 0};
#pragma unroll
                for (int w = 0; w < KW; w += 2) {
                    mma_u8s8(ev, k0[w] & 0x0f0f0f0fu, k1[w] & 0x0f0f0f0fu, k0[w + 1] & 0x0f0f0f0fu,
                             k1[w + 1] & 0x0f0f0f0fu, qb[n][2 * w], qb[n][2 * w + 2]);
                    mma_u8s8(od, k0[w] & 0xf0f0f0f0u, k1[w] & 0xf0f0f0f0u, k0[w + 1] & 0xf0f0f0f0u,
                             k1[w + 1] & 0xf0f0f0f0u, qb[n][2 * w + 1], qb[n][2 * w + 3]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    raw[n][2 * b + i] = (float)((ev[2 * i] * 128 + ev[2 * i + 1]) * 16 + (od[2 * i] * 128 + od[2 * i + 1]));
            }
        }
        // V's codes: pairs of tokens, four dims per word
        uint32_t vw[2][D / 32][2];  // [block][group of 32 dims][tokens 2q.., 8 + 2q..]
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint32_t at = ring_addr + (st * 4 + 2 * b + 1) * kChunk + v_lane;
            uint32_t w[4];
            load_matrix4_trans(w, at);
            if constexpr (D == 128) {
                uint32_t h[4];
                load_matrix4_trans(h, at + 8 * 64);
#pragma unroll
                for (int g = 0; g < 4; ++g) vw[b][g][0] = w[g], vw[b][g][1] = h[g];
            } else {
                vw[b][0][0] = w[0], vw[b][1][0] = w[1], vw[b][0][1] = w[2], vw[b][1][1] = w[3];
            }
        }
        __syncwarp();
        if (j + kStages < np) {  // the pair is in registers: its stage may be filled again
            fence_proxy_async_smem();
            issue(j + kStages, st);
        }
        if (++st == kStages) {
            st = 0;
            parity ^= 1;
        }

        const int base = (b0 + 2 * (warp + kWarps * j)) * kBlock + r;  // the lane's first token
        const bool whole = !kMasked && base - r + 2 * kBlock <= tend;
        bool dead[RT][4];
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = base + 8 * i;
                // rows that no query sees may hold anything
                if (tok >= tend || (kMasked && tok < first)) ce[i] = make_float2(0.f, 0.f);
#pragma unroll
                for (int n = 0; n < RT; ++n) dead[n][i] = tok >= tend || (kMasked && (tok < lo[n] || tok > hi[n]));
            }
        }
        auto logits = [&](int n) {  // +inf before the first maximum
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[n][i] = fmaf(ke[i].x * fac[n], raw[n][i], fmaf(ke[i].y, off_q[n], -m[n]));
                if (!whole && dead[n][i]) x[n][i] = -INFINITY;
            }
        };
        // running maxima, raised only when a logit beats one by 2^8 or a V
        // scale its power of two (NaN takes this way too)
        const float big4 = fmaxf(fmaxf(fabsf(ce[0].x), fabsf(ce[1].x)), fmaxf(fabsf(ce[2].x), fabsf(ce[3].x)));
        bool exceed = big4 > limit;
#pragma unroll
        for (int n = 0; n < RT; ++n) {
            logits(n);
#pragma unroll
            for (int i = 0; i < 4; ++i) exceed = exceed || !(x[n][i] <= kLazyMax);
        }
        if (__any_sync(0xffffffffu, exceed)) {
            float big = big4;
#pragma unroll
            for (int o = 16; o > 2; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            float turn = 1.f;  // new power of two over the old one
            if (big > limit) {
                const float was = cv;
                int e;
                (void)frexpf(fminf(big, FLT_MAX), &e);
                cv = ldexpf(1.f, -min(max(e, -120), 126));  // |scale| cv in [0.5, 1), or up to 4 at the range's end
                limit = kMaxWeightScale / cv;
                turn = cv / was;
            }
#pragma unroll
            for (int n = 0; n < RT; ++n) {
                float bm = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = fmaf(ke[i].x * fac[n], raw[n][i], ke[i].y * off_q[n]);
                    if (!whole && dead[n][i]) v = -INFINITY;
                    bm = fmaxf(bm, v != v ? 0.f : v);  // a NaN row gets a finite maximum and NaN sums
                }
#pragma unroll
                for (int o = 16; o > 2; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
                float alpha = 1.f;
                if (bm > m[n] + kLazyMax) {  // a row's maximum does not depend on the other rows
                    alpha = ex2(m[n] - bm);  // 0 on the first block
                    m[n] = bm;
                }
                l[n] *= alpha;
                z[n] *= alpha;
                alpha *= turn;
                zc[n] *= alpha;
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    if constexpr (kSplit) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[0][t][i] *= alpha;
                    } else {
                        acc[n / 2][t][n & 1] *= alpha;
                        acc[n / 2][t][2 + (n & 1)] *= alpha;
                    }
                }
                logits(n);
            }
        }
        // weights, turned into the second product's operand
        uint32_t wb[NP][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float sv = ce[i].x * cv;
            float w[RT];
#pragma unroll
            for (int n = 0; n < RT; ++n) {
                const float pr = ex2(x[n][i]);
                l[n] += pr;
                w[n] = pr * sv;
                float zz = pr * ce[i].y;
                if (kMasked && dead[n][i]) w[n] = zz = 0.f;  // a row that does not see a NaN stays clear of it
                z[n] += zz;
            }
            if constexpr (kSplit) {
                const __half2 h = __floats2half2_rn(w[0], w[0] - __half2float(__float2half_rn(w[0])));
                wb[0][i] = transpose8x8(*reinterpret_cast<const uint32_t *>(&h));
            } else {
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    const __half2 h = __floats2half2_rn(w[2 * n], w[2 * n + 1]);
                    const float2 back = __half22float2(h);
                    zc[2 * n] += w[2 * n] - back.x;
                    zc[2 * n + 1] += w[2 * n + 1] - back.y;
                    wb[n][i] = transpose8x8(*reinterpret_cast<const uint32_t *>(&h));
                }
            }
        }
        // O^T += U'^T W^T: tile 2 g + u holds dims 32 g + 4 r + 2 u (and + 1, times 16)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int g = 0; g < D / 32; ++g) {
                const uint32_t a = vw[b][g][0], c = vw[b][g][1], a8 = a >> 8, c8 = c >> 8;
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    mma_f16(acc[n][2 * g], a & 0x000f000fu, a & 0x00f000f0u, c & 0x000f000fu, c & 0x00f000f0u,
                            wb[n][2 * b], wb[n][2 * b + 1]);
                    mma_f16(acc[n][2 * g + 1], a8 & 0x000f000fu, a8 & 0x00f000f0u, c8 & 0x000f000fu, c8 & 0x00f000f0u,
                            wb[n][2 * b], wb[n][2 * b + 1]);
                }
            }
    }
    if (!ok) {
        // A copy never completed (the error word is set): every copy still out
        // gets one more bounded chance to land before the CTA exits.
        if (lane == 0)
            for (int jj = j; jj < j + kStages && jj < np; ++jj)
                mbar_wait(&wbar[jj % kStages], (jj / kStages) & 1, 200000000ll);
        atomicOr(&fail_s, 1);
    }

    // ---- merge the warps' states --------------------------------------------
    __syncthreads();  // every warp is done with its stages; reuse them
    if (fail_s) return;
    float *red_acc = reinterpret_cast<float *>(smem);
    float *red_m = reinterpret_cast<float *>(smem + Lay.ml_off), *red_l = red_m + kWarps * RW;
    const float back = 1.f / cv;  // a power of two
#pragma unroll
    for (int n = 0; n < RT; ++n) {
        const int h = 4 * n + q;
#pragma unroll
        for (int o = 16; o > 2; o >>= 1) {
            l[n] += __shfl_xor_sync(0xffffffffu, l[n], o);
            z[n] += __shfl_xor_sync(0xffffffffu, z[n], o);
            if constexpr (!kSplit) zc[n] += __shfl_xor_sync(0xffffffffu, zc[n], o);
        }
        if (h >= rows) continue;
        const float add = kSplit ? z[n] : fmaf(7.5f * zc[n], back, z[n]);
        float *dst = red_acc + (warp * RW + h) * D + 4 * r;
#pragma unroll
        for (int g = 0; g < D / 32; ++g) {
            float o[4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float *c = acc[n / 2][2 * g + u];
                o[2 * u] = fmaf((kSplit ? c[0] + c[1] : c[n & 1]) * kTwo24, back, add);
                o[2 * u + 1] = fmaf((kSplit ? c[2] + c[3] : c[2 + (n & 1)]) * (kTwo24 / 16.f), back, add);
            }
            *reinterpret_cast<float4 *>(dst + 32 * g) = make_float4(o[0], o[1], o[2], o[3]);
        }
        if (r == 0) {
            red_m[warp * RW + h] = m[n];
            red_l[warp * RW + h] = l[n];
        }
    }
    __syncthreads();
    for (int i = tid; i < rows * D; i += blockDim.x) {
        const int h = i / D, d = i % D;
        float lse;
        const float o = combine_warps<D, RW, kWarps>(red_m, red_l, red_acc, h, d, &lse) * p.v_scale;
        const int64_t qr = row_of(h);
        if (sp.nparts == 1) {
            out[qr * D + d] = E::from_float(o);
        } else {
            const int64_t row = qr * p.max_parts + part;
            p.ws_o[row * D + d] = o;
            if (d == 0) p.ws_lse[row] = lse != lse ? 0.f : lse;  // the NaN is in o: the merge must not skip it
        }
    }
}

template <typename T, int D, int RT, bool kMasked>
cudaError_t launch_int4_t(const DecodeParams &p, cudaStream_t stream) {
    auto kern = decode_int4_kernel<T, D, RT, kMasked>;
    static FuncAttrCache attrs;
    constexpr int kSmem = Int4Layout(D, 4 * RT).bytes;
    cudaError_t e = ensure_smem(kern, kSmem, attrs, /*max_carveout=*/true);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(p.max_parts, p.num_kv_heads, p.num_seqs), dim3(kWarps * 32), kSmem, stream, p);
    if (e != cudaSuccess || p.max_parts == 1) return e;
    return launch_merge_partitions(p, std::is_same<T, __nv_bfloat16>::value ? PA_BF16 : PA_F16, D, stream);
}

template <typename T, int D>
cudaError_t launch_int4_d(const DecodeParams &p, int rows, cudaStream_t stream) {
    const bool masked = decode_masked(p);
    if (rows <= 4) return masked ? launch_int4_t<T, D, 1, true>(p, stream) : launch_int4_t<T, D, 1, false>(p, stream);
    if (rows <= 8) return masked ? launch_int4_t<T, D, 2, true>(p, stream) : launch_int4_t<T, D, 2, false>(p, stream);
    return masked ? launch_int4_t<T, D, 4, true>(p, stream) : launch_int4_t<T, D, 4, false>(p, stream);
}

}  // namespace

cudaError_t launch_decode_int4(const DecodeParams &p, int dtype, int head_dim, int rows, cudaStream_t stream) {
    if (dtype == PA_F16)
        return head_dim == 64 ? launch_int4_d<__half, 64>(p, rows, stream) : launch_int4_d<__half, 128>(p, rows, stream);
    return head_dim == 64 ? launch_int4_d<__nv_bfloat16, 64>(p, rows, stream)
                          : launch_int4_d<__nv_bfloat16, 128>(p, rows, stream);
}

}  // namespace pa
