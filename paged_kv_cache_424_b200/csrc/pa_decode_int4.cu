// pa_decode_int4.cu -- paged decode attention over 4-bit caches (PA_INT4),
// every group size and head_dim.
//
// With codes u, row scales s, s' and lowest values l, l' (K and V),
//   x_t = c (s_t (q . u_t) + l_t sum(q)),   c = scale log2(e) k_scale
//   out = sum_t p_t (s'_t u'_t + l'_t) / sum_t p_t,   p_t = 2^(x_t - m)
// so the codes enter both products as integers 0..15 and the scales act on
// tokens: on a logit after the first product, on a weight before the second.
//
// One warp takes 16 tokens (a block) at a time with warp-level matrix
// instructions m16n8k16 (f16 in, f32 out):
//   S^T (16 tokens x 8 rows) = U (16 x D) . Q^T (D x 8)
//   O^T (D x 8 rows)        += U'^T (D x 16 tokens) . W^T (16 x 8),  W = p s'
// The unpacking is what bounds such a kernel, so it is one instruction per
// register: a nibble masked out of a word where it stands, w & 0x000f000f or
// w & 0x00f000f0, is the fp16 subnormal u 2^-24 or 16 u 2^-24, exactly, and
// the matrix units take subnormals as they are.  The factor 16 of every other
// dim goes into Q (an exact shift) and out of O; with one shift per word by 8
// eight codes cost five instructions.  The contraction over dims may run in
// any order, so a lane's codes are simply the 16 consecutive bytes that it
// loads and Q is laid out to match; for the second product, whose registers
// pair two tokens, two byte permutes bring the tokens' words together.
// S's accumulator layout (token, two rows) is turned into W's operand layout
// by movmatrix.  No shared-memory round trip, no barrier, and no tensor
// memory: with 5th-generation MMAs the codes would have to be written back to
// shared memory, widened, before the MMA could read them, and each 128-token
// chunk would wait for S to come back from TMEM and P to go in; the FP8 kernel
// that is built so takes 97 us for the 8B step, whatever the bytes.
//
// Q is rounded to f16 (11 bits) under a power of two per row; weights to
// f16, under a power of two that follows the largest V scale seen.  A code is
// 0..15 and not -8..7, so a weight's rounding error would count 7.5 codes
// where a centred code's would cancel: what the rounding took (w - f16(w)) is
// summed and given back at the middle code 7.5.
#include <cfloat>
#include <type_traits>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_int4.cuh"
#include "pa_simt.cuh"

namespace pa {

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 4;  // per warp: 4 x 2 chunks in flight
constexpr float kTwo24 = 16777216.f;
constexpr float kMaxWeightScale = 64.f;  // times p <= 2^8 stays inside f16

// D += A B, one m16n8k16.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
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

// Shared memory: per-warp stage rings (reused for the warps' outputs at the
// end), the warps' m and l, the mbarriers.
struct Int4Layout {
    int main, ml_off, bar_off, bytes;
    __host__ __device__ constexpr Int4Layout(int D, int rows)
        : main(kWarps * kStages * 2 * int4_chunk_bytes(D) > kWarps * rows * D * 4
                   ? kWarps * kStages * 2 * int4_chunk_bytes(D)
                   : kWarps * rows * D * 4),
          ml_off(main), bar_off(ml_off + 2 * kWarps * rows * 4), bytes(bar_off + kWarps * kStages * 8) {}
};

// NT: tiles of 8 query rows.  Lane (r, q) = (lane / 4, lane % 4) holds
//   of S: tokens tau(r) and 8 + tau(r), query rows 2q, 2q + 1 of each tile;
//   of K: D / 4 dims from D / 4 q of those two tokens; of Q the same dims of
//     row r of each tile;
//   of V: D / 8 dims from D / 8 r of tokens tau(2q), tau(2q + 1) and those + 8;
//   of O: those dims, query rows 2q and 2q + 1 of each tile.
// tau swaps the tokens of every other pair, so that the V rows of one load
// fall on both halves of the banks (2-way instead of 4-way conflicts).
template <typename T, int D, int NT, bool kMasked>
__global__ void __launch_bounds__(kWarps * 32) decode_int4_kernel(const DecodeParams p) {
    using E = Elem<T>;
    constexpr int KW = D / 32;   // words of K per lane and token
    constexpr int VW = D / 64;   // words of V per lane and token
    constexpr int MT = D / 16;   // tiles of 16 dims
    constexpr int RW = 8 * NT;
    constexpr int kChunk = int4_chunk_bytes(D);
    constexpr Int4Layout Lay(D, RW);
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int fail_s;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay.bar_off);
    const int part = blockIdx.x, kvh = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, q = lane & 3;
    pdl_launch_dependents();
    pdl_wait();
    const int s = scheduled_seq(p, blockIdx.z, part == 0 && kvh == 0 && tid == 0);
    if (s < 0) return;
    const int rows = p.group * p.q_len;
    const SeqSplit sp = seq_split(p, s, part == 0 && kvh == 0 && tid == 0);
    if (part >= sp.nparts) return;
    T *out = reinterpret_cast<T *>(p.out);
    auto row_of = [&](int h) -> int64_t {
        if constexpr (kMasked) return query_row(p, s, kvh, h);
        return (int64_t)s * p.num_heads + kvh * p.group + h;
    };
    const int L = sp.L;
    if (L == 0) {
        for (int i = tid; i < rows * D; i += blockDim.x) out[row_of(i / D) * D + i % D] = E::from_float(0.f);
        return;
    }
    uint64_t *wbar = bars + warp * kStages;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&wbar[i], 1);
        fence_mbar_init();
    }
    if (tid == 0) fail_s = 0;
    __syncthreads();

    // ---- this warp's blocks: every kWarps-th of the partition ---------------
    const int b0 = sp.bfirst + part * p.part_blocks;
    const int b1 = min(b0 + p.part_blocks, sp.nblk);
    const int nw = (b1 - b0 - warp + kWarps - 1) / kWarps;  // may be <= 0
    const int32_t *table = p.block_tables + (int64_t)s * p.max_blocks_per_seq + b0 + warp;
    auto window = [&](int w) -> int32_t {  // entries 32 w .. 32 w + 31, one per lane
        const int j = 32 * w + lane;
        return j < nw ? (int32_t)checked_block(p, table[kWarps * j]) : 0;
    };
    int32_t cur = window(0), next = nw > 32 ? window(1) : 0;
    unsigned char *ring = smem + warp * kStages * 2 * kChunk;
    const unsigned char *kc = reinterpret_cast<const unsigned char *>(p.k_cache);
    const unsigned char *vc = reinterpret_cast<const unsigned char *>(p.v_cache);
    // the loads of block j (all lanes, j in ascending order)
    auto issue = [&](int j) {
        if ((j & 31) == 0 && j > 0) {
            cur = next;
            next = 32 * (j / 32 + 1) < nw ? window(j / 32 + 1) : 0;
        }
        const int64_t phys = __shfl_sync(0xffffffffu, cur, j & 31);
        if (lane == 0) {
            const int64_t off = (phys * p.num_kv_heads + kvh) * kChunk;
            uint64_t *bar = &wbar[j % kStages];
            unsigned char *dst = ring + (j % kStages) * 2 * kChunk;
            mbar_arrive_expect_tx(bar, 2 * kChunk);
            bulk_g2s(dst, kc + off, kChunk, bar);
            bulk_g2s(dst + kChunk, vc + off, kChunk, bar);
        }
    };
    for (int j = 0; j < kStages && j < nw; ++j) issue(j);

    // ---- query rows: f16 under a power of two per row -----------------------
    uint32_t qb[NT][2 * KW][2];       // B operands: step 2 w + e of word w
    float fac[NT][2], off_q[NT][2];   // of rows 2q, 2q + 1: c 2^(24 - e), c sum(q)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int h = 8 * n + r;
        float y[D / 4];
        const T *src = reinterpret_cast<const T *>(p.q) + row_of(h < rows ? h : 0) * D + q * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 w = h < rows ? *reinterpret_cast<const uint4 *>(src + 8 * i) : make_uint4(0, 0, 0, 0);
            const float2 a = E::to_float2(w.x), b = E::to_float2(w.y), c = E::to_float2(w.z), d = E::to_float2(w.w);
            y[8 * i] = a.x, y[8 * i + 1] = a.y, y[8 * i + 2] = b.x, y[8 * i + 3] = b.y;
            y[8 * i + 4] = c.x, y[8 * i + 5] = c.y, y[8 * i + 6] = d.x, y[8 * i + 7] = d.y;
        }
        float mx = 0.f;
        bool finite = true;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) {
            mx = fmaxf(mx, fabsf(y[i]));
            finite = finite && fabsf(y[i]) <= FLT_MAX;
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        int e = 0;
        if (mx > 0.f && mx <= FLT_MAX) {
            (void)frexpf(mx, &e);  // mx in [2^(e-1), 2^e)
            e = 8 - e;
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) {
            y[i] = __half2float(__float2half_rn(ldexpf(y[i], e)));
            sum += y[i];
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // nibbles 2u, 2u + 4 and (times 1/16) 2u + 1, 2u + 5 of word w
                qb[n][2 * w + u][0] = half2_bits(y[8 * w + 2 * u], y[8 * w + 2 * u + 4]);
                qb[n][2 * w + u][1] = half2_bits(y[8 * w + 2 * u + 1] * 0.0625f, y[8 * w + 2 * u + 5] * 0.0625f);
            }
        const bool row_fine = __all_sync(0xfu << (lane & ~3), finite);
        const float f = row_fine ? ldexpf(p.scale_log2, 24 - e) : NAN, o = row_fine ? sum * ldexpf(p.scale_log2, -e) : NAN;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            fac[n][i] = __shfl_sync(0xffffffffu, f, (2 * q + i) * 4);
            off_q[n][i] = __shfl_sync(0xffffffffu, o, (2 * q + i) * 4);
        }
    }
    int lo[NT][2], hi[NT][2];  // attended positions of rows 2q, 2q + 1
    int first = 0;             // first position any row attends to
    if constexpr (kMasked) {
        if (p.window > 0) first = L - p.q_len - p.window + 1;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) row_range(p, L, 8 * n + 2 * q + i, &lo[n][i], &hi[n][i]);
    }

    // ---- state of rows 2q, 2q + 1 -------------------------------------------
    float m[NT][2], l[NT][2], z[NT][2], zc[NT][2], acc[NT][MT][4];
    float cv = 1.f;      // power of two the V scales are multiplied by (warp-uniform)
    float top = 0.f;     // largest |V scale| it was chosen for
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[n][i] = -INFINITY;
            l[n][i] = z[n][i] = zc[n][i] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][t][i] = 0.f;
    }
    const int tau = r ^ ((r >> 1) & 1), tv0 = (2 * q) ^ (q & 1), tv1 = tv0 ^ 1;
    bool ok = true;
    int j = 0;
#pragma unroll 1
    for (; j < nw; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait(&wbar[j % kStages], (j / kStages) & 1))) {
            ok = false;
            break;
        }
        const unsigned char *ks = ring + (j % kStages) * 2 * kChunk, *vs = ks + kChunk;
        uint32_t k0[KW], k1[KW], va[VW], vb[VW], vd[VW], ve[VW];
        load_words<KW>(k0, ks + tau * (D / 2) + q * (D / 8));
        load_words<KW>(k1, ks + (8 + tau) * (D / 2) + q * (D / 8));
        load_words<VW>(va, vs + tv0 * (D / 2) + r * (D / 16));
        load_words<VW>(vb, vs + tv1 * (D / 2) + r * (D / 16));
        load_words<VW>(vd, vs + (8 + tv0) * (D / 2) + r * (D / 16));
        load_words<VW>(ve, vs + (8 + tv1) * (D / 2) + r * (D / 16));
        float2 ke[2], ce[2];  // (scale, low) of the lane's two tokens in K and V
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ke[i] = int4_ends(*reinterpret_cast<const uint32_t *>(ks + int4_ends_offset(D) + 4 * (8 * i + tau)));
            ce[i] = int4_ends(*reinterpret_cast<const uint32_t *>(vs + int4_ends_offset(D) + 4 * (8 * i + tau)));
        }
        __syncwarp();
        if (j + kStages < nw) {  // the block is in registers: its stage may be filled again
            fence_proxy_async_smem();
            issue(j + kStages);
        }

        // S^T = U Q^T, two chains of accumulation
        float x[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const uint32_t a = k0[w], b = k1[w], a8 = a >> 8, b8 = b >> 8;
                mma16816(s0, a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u, qb[n][2 * w][0],
                         qb[n][2 * w][1]);
                mma16816(s1, a8 & 0x000f000fu, b8 & 0x000f000fu, a8 & 0x00f000f0u, b8 & 0x00f000f0u,
                         qb[n][2 * w + 1][0], qb[n][2 * w + 1][1]);
            }
            // x[n][2 t + i]: token t of the lane (tau, 8 + tau), row 2q + i
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[n][i] = fmaf(ke[i >> 1].x, (s0[i] + s1[i]) * fac[n][i & 1], ke[i >> 1].y * off_q[n][i & 1]);
        }
        const int base = (b0 + warp + kWarps * j) * kBlock;
        const bool whole = !kMasked && base + kBlock <= L;
        bool live[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = base + 8 * (i >> 1) + tau;
                live[n][i] = whole || tok < L;
                if constexpr (kMasked) live[n][i] = live[n][i] && tok >= lo[n][i & 1] && tok <= hi[n][i & 1];
                if (!live[n][i]) x[n][i] = -INFINITY;
            }
        if (!whole) {  // rows that no query sees may hold anything
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tok = base + 8 * i + tau;
                if (tok >= L || (kMasked && tok < first)) ce[i] = make_float2(0.f, 0.f);
            }
        }
        // running maxima, raised only when a logit beats one by 2^8 or a V
        // scale its power of two
        bool exceed = fabsf(ce[0].x) * cv > kMaxWeightScale || fabsf(ce[1].x) * cv > kMaxWeightScale || top == 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) exceed = exceed || x[n][i] > m[n][i & 1] + kLazyMax;
        if (__any_sync(0xffffffffu, exceed)) {
            float big = fmaxf(fabsf(ce[0].x), fabsf(ce[1].x));
#pragma unroll
            for (int o = 16; o > 2; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            float turn = 1.f;  // new power of two over the old one
            if (big > top) {
                top = big;
                const float was = cv;
                int e;
                (void)frexpf(fminf(big, FLT_MAX), &e);
                cv = ldexpf(1.f, -min(max(e, -120), 126));  // |scale| cv in [0.5, 1), or up to 4 at the range's end
                turn = cv / was;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float bm = fmaxf(x[n][i], x[n][2 + i]);
#pragma unroll
                    for (int o = 16; o > 2; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
                    float alpha = 1.f;
                    if (bm > m[n][i]) {
                        alpha = ex2(m[n][i] - bm);  // 0 on the first block
                        m[n][i] = bm;
                    }
                    l[n][i] *= alpha;
                    z[n][i] *= alpha;
                    alpha *= turn;
                    zc[n][i] *= alpha;
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        acc[n][t][i] *= alpha;
                        acc[n][t][2 + i] *= alpha;
                    }
                }
        }
        // weights, turned into the second product's operand
        uint32_t wb[NT][2];
        const float sv[2] = {ce[0].x * cv, ce[1].x * cv};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = 2 * t + i;
                    float pr = ex2(x[n][k] - m[n][i]);
                    if (!whole && !live[n][k]) pr = 0.f;  // m may still be -inf
                    l[n][i] += pr;
                    w[i] = pr * sv[t];
                    float zz = pr * ce[t].y;
                    if (kMasked && !live[n][k]) w[i] = zz = 0.f;  // a row that does not see a NaN stays clear of it
                    z[n][i] += zz;
                }
                const __half2 h = __floats2half2_rn(w[0], w[1]);
                const float2 back = __half22float2(h);
                zc[n][0] += w[0] - back.x;
                zc[n][1] += w[1] - back.y;
                wb[n][t] = transpose8x8(*reinterpret_cast<const uint32_t *>(&h));
            }
        // O^T += U'^T W^T: tile 4 w + 2 v + u holds dims 8 w + 4 v + 2 u (and + 1, times 16)
#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const uint32_t a = __byte_perm(va[w], vb[w], v ? 0x7632 : 0x5410);
                const uint32_t b = __byte_perm(vd[w], ve[w], v ? 0x7632 : 0x5410);
                const uint32_t a8 = a >> 8, b8 = b >> 8;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma16816(acc[n][4 * w + 2 * v], a & 0x000f000fu, a & 0x00f000f0u, b & 0x000f000fu, b & 0x00f000f0u,
                             wb[n][0], wb[n][1]);
                    mma16816(acc[n][4 * w + 2 * v + 1], a8 & 0x000f000fu, a8 & 0x00f000f0u, b8 & 0x000f000fu,
                             b8 & 0x00f000f0u, wb[n][0], wb[n][1]);
                }
            }
    }
    if (!ok) {
        // A copy never completed (the error word is set): every copy still out
        // gets one more bounded chance to land before the CTA exits.
        if (lane == 0)
            for (int jj = j; jj < j + kStages && jj < nw; ++jj)
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
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int h = 8 * n + 2 * q + i;
#pragma unroll
            for (int o = 16; o > 2; o >>= 1) {
                l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], o);
                z[n][i] += __shfl_xor_sync(0xffffffffu, z[n][i], o);
                zc[n][i] += __shfl_xor_sync(0xffffffffu, zc[n][i], o);
            }
            const float add = fmaf(7.5f * zc[n][i], back, z[n][i]);
            float *dst = red_acc + (warp * RW + h) * D + r * (D / 8);
#pragma unroll
            for (int t = 0; t < MT; ++t)
                *reinterpret_cast<float2 *>(dst + 2 * t) =
                    make_float2(fmaf(acc[n][t][i] * kTwo24, back, add), fmaf(acc[n][t][2 + i] * (kTwo24 / 16.f), back, add));
            if (r == 0) {
                red_m[warp * RW + h] = m[n][i];
                red_l[warp * RW + h] = l[n][i];
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
            if (d == 0) p.ws_lse[row] = lse;
        }
    }
}

template <typename T, int D, int NT, bool kMasked>
cudaError_t launch_int4_t(const DecodeParams &p, cudaStream_t stream) {
    auto kern = decode_int4_kernel<T, D, NT, kMasked>;
    static FuncAttrCache attrs;
    constexpr int kSmem = Int4Layout(D, 8 * NT).bytes;
    cudaError_t e = ensure_smem(kern, kSmem, attrs, /*max_carveout=*/true);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(p.max_parts, p.num_kv_heads, p.num_seqs), dim3(kWarps * 32), kSmem, stream, p);
    if (e != cudaSuccess || p.max_parts == 1) return e;
    return launch_merge_partitions(p, std::is_same<T, __nv_bfloat16>::value ? PA_BF16 : PA_F16, D, stream);
}

template <typename T, int D>
cudaError_t launch_int4_d(const DecodeParams &p, int rows, cudaStream_t stream) {
    if (rows <= 8) return decode_masked(p) ? launch_int4_t<T, D, 1, true>(p, stream) : launch_int4_t<T, D, 1, false>(p, stream);
    return decode_masked(p) ? launch_int4_t<T, D, 2, true>(p, stream) : launch_int4_t<T, D, 2, false>(p, stream);
}

}  // namespace

cudaError_t launch_decode_int4(const DecodeParams &p, int dtype, int head_dim, int rows, cudaStream_t stream) {
    if (dtype == PA_F16)
        return head_dim == 64 ? launch_int4_d<__half, 64>(p, rows, stream) : launch_int4_d<__half, 128>(p, rows, stream);
    return head_dim == 64 ? launch_int4_d<__nv_bfloat16, 64>(p, rows, stream)
                          : launch_int4_d<__nv_bfloat16, 128>(p, rows, stream);
}

}  // namespace pa
