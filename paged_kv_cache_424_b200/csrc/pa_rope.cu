// pa_rope.cu -- rotary positions, the cache write of rotated keys, the 4-bit
// cache write and the read-back of cached rows (pa_rope, pa_rope_and_cache,
// pa_reshape_and_cache_int4, pa_gather_cache).
//
// A pair (a, b) of a head at position p with frequency f turns by p f:
//   a' = m (a cos - b sin),  b' = m (b cos + a sin).
// All of it is data movement: each element is read once and written once.
//
// CTA = one token (or some of its rows, when there are few tokens).  Its first
// rotary_dim / 2 threads compute the token's (m cos, m sin) pairs in fp64 and
// share them through shared memory, so the sines are computed once per token
// and not once per head.  Then D / 16 lanes take a row (a head's D elements): a
// lane has two pieces of 8 elements that hold both ends of its pairs, so that
// nothing is exchanged and each sine serves both; the next pass's rows are in
// flight while one is worked on.
//
// 16-bit outputs are bounded by DRAM latency and bandwidth (8192 tokens of 40
// heads of 128: 31 us, 5.4 TB/s; one CTA per token 100 us, resident CTAs that
// walk over tokens with a pair's ends in two lanes 49), FP8 and 4-bit caches by
// instruction issue as well (4093 tokens of 32 + 32 + 32 heads into FP8: 36 us,
// 4.7 TB/s, in the first form 72; 8192 tokens of 64 + 8 + 8 heads into 4 bits 61
// us and 13 to read them back, in the first form 232 together).
#include <algorithm>

#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_int4.cuh"

namespace pa {

namespace {

constexpr int kBlock = 16;
constexpr int kThreads = 128;       // of the rotating kernel
constexpr int kGatherThreads = 256;
constexpr int kMaxHalf = 64;  // rotary_dim / 2 at most

// Cache kinds of the templates below.
enum { kCacheNone = 0, kCache16 = 1, kCacheE4m3 = 2, kCacheInt4 = 3 };

// sin and cos of 2 pi t: t reduced to the nearest quarter turn, then Taylor
// polynomials on |y| <= pi / 4 whose first dropped terms (y^17 / 17!, y^18 /
// 18!) are below 5e-17.
__device__ __forceinline__ void sincos_turns(double t, double *s, double *c) {
    t -= rint(t);
    const double quarter = rint(4.0 * t);
    const double y = (t - 0.25 * quarter) * 6.283185307179586476925;
    const double z = y * y;
    double ps = -1.0 / 1307674368000.0;
    ps = fma(ps, z, 1.0 / 6227020800.0);
    ps = fma(ps, z, -1.0 / 39916800.0);
    ps = fma(ps, z, 1.0 / 362880.0);
    ps = fma(ps, z, -1.0 / 5040.0);
    ps = fma(ps, z, 1.0 / 120.0);
    ps = fma(ps, z, -1.0 / 6.0);
    ps = fma(ps * z, y, y);
    double pc = 1.0 / 20922789888000.0;
    pc = fma(pc, z, -1.0 / 87178291200.0);
    pc = fma(pc, z, 1.0 / 479001600.0);
    pc = fma(pc, z, -1.0 / 3628800.0);
    pc = fma(pc, z, 1.0 / 40320.0);
    pc = fma(pc, z, -1.0 / 720.0);
    pc = fma(pc, z, 1.0 / 24.0);
    pc = fma(pc, z, -0.5);
    pc = fma(pc, z, 1.0);
    const int k = (int)quarter & 3;
    const double a = (k & 1) ? pc : ps, b = (k & 1) ? ps : pc;
    *s = (k & 2) ? -a : a;
    *c = (k == 1 || k == 2) ? -b : b;
}

template <typename T>
__device__ __forceinline__ void widen8(const uint4 &w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Elem<T>::to_float2(u[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <typename T>
__device__ __forceinline__ uint4 narrow8(const float (&x)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const typename Elem<T>::T2 h = {Elem<T>::from_float(x[2 * i]), Elem<T>::from_float(x[2 * i + 1])};
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ uint64_t pk2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 up2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
// Two single-precision operations in one instruction.
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// x / b for two x, correctly rounded, from y = RN(1 / b): q = RN(x y), r = x - b
// q (exact), RN(q + r y).  That is the quotient whenever b's significand is not
// all ones and nothing leaves the normal range (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990); the
// callers keep b between 2^-80 and 2^100 for quotients that matter.
__device__ __forceinline__ uint64_t divide2(uint64_t x, uint64_t y, uint64_t minus_b) {
    const uint64_t q = mul2(x, y);
    return fma2(fma2(minus_b, q, x), y, q);
}
__device__ __forceinline__ bool divide2_fits(float b) {
    return fabsf(b) > 0x1p-80f && fabsf(b) < 0x1p100f && (__float_as_uint(b) & 0x7fffffu) != 0x7fffffu;
}

// The 4-bit codes of 8 elements (element i in bits 4 i ..): round_half_even((x
// - low) / sc) clamped to 0..15, the quotient rounded to fp32 first.  sc is
// finite and not 0.
__device__ __forceinline__ uint32_t int4_codes(const float (&x)[8], float low, float sc) {
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, half to even
    uint32_t codes = 0;
    if (divide2_fits(sc)) {
        const float inv = __frcp_rn(sc);
        const uint64_t y = pk2(inv, inv), mb = pk2(-sc, -sc), ml = pk2(-low, -low), magic = pk2(kRound, kRound);
#pragma unroll
        for (int i = 6; i >= 0; i -= 2) {
            const float2 k = up2(add2(divide2(add2(pk2(x[i], x[i + 1]), ml), y, mb), magic));
            const float k0 = fminf(fmaxf(k.x, kRound), kRound + 15.f), k1 = fminf(fmaxf(k.y, kRound), kRound + 15.f);
            // the low bits of k are the integer: Horner in base 16, the constant part taken off at the end
            codes = (codes * 16u + __float_as_uint(k1)) * 16u + __float_as_uint(k0);
        }
        return codes - 0x4b400000u * 0x11111111u;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float u = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[i], low), sc)), 0.f), 15.f);
        codes |= (uint32_t)u << (4 * i);
    }
    return codes;
}

// E4M3 codes of x / scale (nearest, ties to even, clamped to 448, NaN kept).
__device__ __forceinline__ uint2 e4m3_codes(const float (&x)[8], float scale) {
    uint32_t u[2];
    if (divide2_fits(scale)) {
        // by -scale, with the codes' signs turned back at the end: so divided, a
        // zero keeps its sign (by a positive number the last sum makes it +0)
        const float inv = __frcp_rn(-scale), most = 512.f * scale;  // beyond it every quotient is clamped
        const uint64_t y = pk2(inv, inv), mb = pk2(scale, scale);
        uint16_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = min_nan(max_nan(x[2 * i], -most), most), b = min_nan(max_nan(x[2 * i + 1], -most), most);
            const float2 q = up2(divide2(pk2(a, b), y, mb));
            h[i] = float2_to_e4m3x2(q.x, q.y);
        }
        u[0] = ((uint32_t)h[0] | ((uint32_t)h[1] << 16)) ^ 0x80808080u;
        u[1] = ((uint32_t)h[2] | ((uint32_t)h[3] << 16)) ^ 0x80808080u;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t lo = float2_to_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
            const uint32_t hi = float2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
            u[i] = lo | (hi << 16);
        }
    }
    return make_uint2(u[0], u[1]);
}

// The row of `slot` and KV head h takes this lane's pieces xa (dims 8 ca ..) and
// xb (8 cb ..); all of the row's D / 16 lanes converged, `live`: the row is
// written.
template <typename T, int D, int kCache>
__device__ __forceinline__ void store_row(void *cache, const float (&xa)[8], const float (&xb)[8], int64_t slot, int h,
                                          int num_kv_heads, int ca, int cb, float scale, bool live) {
    constexpr int kPieces = D / 8;
    const int64_t blk = slot / kBlock;
    const int off = (int)(slot % kBlock);
    const int64_t chunk = blk * num_kv_heads + h;
    if constexpr (kCache == kCache16) {
        if (live) {
            uint4 *dst = reinterpret_cast<uint4 *>(cache) + (chunk * kBlock + off) * kPieces;
            dst[ca] = narrow8<T>(xa);
            dst[cb] = narrow8<T>(xb);
        }
    } else if constexpr (kCache == kCacheE4m3) {
        if (live) {
            uint2 *dst = reinterpret_cast<uint2 *>(cache) + (chunk * kBlock + off) * kPieces;
            dst[ca] = e4m3_codes(xa, scale);
            dst[cb] = e4m3_codes(xb, scale);
        }
    } else if constexpr (kCache == kCacheInt4) {
        // a NaN goes through both; an infinity makes the range infinite or NaN
        float lo = min_nan(xa[0], xb[0]), hi = max_nan(xa[0], xb[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            lo = min_nan(lo, min_nan(xa[i], xb[i]));
            hi = max_nan(hi, max_nan(xa[i], xb[i]));
        }
#pragma unroll
        for (int o = D / 32; o > 0; o >>= 1) {
            lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        if (!live) return;
        __nv_bfloat16 lb = __float2bfloat16_rn(lo);
        const float low = __bfloat162float(lb);
        __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, low), 15.f));
        const float sc = __bfloat162float(sb);
        uint32_t code_a = 0, code_b = 0;
        if (!(fabsf(sc) < INFINITY)) {  // a NaN or an infinity in the row, or a range past fp32's
            lb = sb = __float2bfloat16_rn(NAN);
        } else if (sc != 0.f) {
            code_a = int4_codes(xa, low, sc);
            code_b = int4_codes(xb, low, sc);
        }
        unsigned char *base = reinterpret_cast<unsigned char *>(cache) + chunk * int4_chunk_bytes(D);
        uint32_t *row = reinterpret_cast<uint32_t *>(base + off * (D / 2));
        if (cb == ca + 1) {
            *reinterpret_cast<uint2 *>(row + ca) = make_uint2(code_a, code_b);
        } else {
            row[ca] = code_a;
            row[cb] = code_b;
        }
        if (ca == 0) {
            const uint32_t ends = (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(lb) << 16);
            *reinterpret_cast<uint32_t *>(base + int4_ends_offset(D) + off * 4) = ends;
        }
    }
}

constexpr int kWave = 148 * 8;  // CTAs that a device holds at once

// How a row's pairs lie in its lanes' 8 dims.
enum { kPairsHalf = 0, kPairsInterleaved = 1, kPairsHalfOdd = 2 };  // kPairsHalf: rotary_dim / 2 a multiple of 8

// CTA = tokens blockIdx.x, blockIdx.x + gridDim.x, ...; of each the passes
// blockIdx.y, blockIdx.y + gridDim.y, ... over its rows, kRows rows each.
template <typename T, int D, int kCache, int kPairs>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const RopeParams p) {
    constexpr int LPR = D / 16;            // lanes per row
    constexpr int kRows = kThreads / LPR;  // rows of a pass
    __shared__ __align__(16) float cos_s[2][kMaxHalf], sin_s[2][kMaxHalf];
    const int tid = threadIdx.x, lane = tid & 31;
    // The next kernel may start early behind a cache write alone.  Behind rotated
    // queries or keys its CTAs would take the SMs' places while they wait (measured
    // with and without: 4093 tokens into FP8 40.9 us and 36.0; 64 sequences of 400
    // tokens, append and 4-bit decode 25.9 and 23.3, 16-bit 30.9 and 31.3).
    if (kCache != kCacheNone && p.num_heads == 0) pdl_launch_dependents();
    const int half = p.half;
    // this lane's pieces ca and cb of 8 dims: half: piece j and the one half / 8
    // behind it, which hold both ends of pairs 8 j .. 8 j + 7 (j < half / 8; the
    // dims past rotary_dim two by two); otherwise neighbours, which interleaved
    // hold the same pairs
    const int j = lane % LPR;
    const int q8 = kPairs == kPairsHalf ? half / 8 : 0;
    const int ca = kPairs != kPairsHalf ? 2 * j : j < q8 ? j : 2 * q8 + 2 * (j - q8);
    const int cb = kPairs != kPairsHalf ? 2 * j + 1 : j < q8 ? j + q8 : ca + 1;
    const int H = p.num_heads, Hk = p.num_kv_heads;
    const int total = H + (kCache == kCacheNone ? Hk : 2 * Hk);
    const int first = (int)blockIdx.y * kRows, step = kRows * (int)gridDim.y;  // of the CTA's passes
    const int mine = tid / LPR;                                                // this lane's row in a pass
    pdl_wait();  // the caller's last kernel may have written any input, positions and slots too
    // a token's sines are computed while the token before it is worked on
    const double freq = tid < half ? p.inv_freq[tid] * 0.15915494309189533576888 : 0.0;
    auto sines = [&](int t, int buf) {
        if (tid >= half) return;
        double s, co;
        sincos_turns((double)p.positions[t] * freq, &s, &co);
        if (p.inverse) s = -s;
        cos_s[buf][tid] = (float)(co * p.magnitude);
        sin_s[buf][tid] = (float)(s * p.magnitude);
    };
    auto slot_of = [&](int t) -> int64_t { return kCache == kCacheNone ? 0 : p.slots[t]; };
    auto load = [&](int t, int row, uint4 (&w)[2]) {  // queries, keys, values in this order
        w[0] = w[1] = make_uint4(0, 0, 0, 0);
        if (row >= total) return;
        const T *base = row < H ? reinterpret_cast<const T *>(p.q)
                        : row < H + Hk ? reinterpret_cast<const T *>(p.k) : reinterpret_cast<const T *>(p.v);
        const int64_t stride = row < H ? p.q_stride : row < H + Hk ? p.k_stride : p.v_stride;
        const int h = row < H ? row : row < H + Hk ? row - H : row - H - Hk;
        const uint4 *src = reinterpret_cast<const uint4 *>(base + t * stride) + h * (D / 8);
        w[0] = src[ca];
        w[1] = src[cb];
    };
    int t = blockIdx.x, buf = 0;
    int64_t slot = slot_of(t);
    uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (slot >= 0) {
        load(t, first + mine, w);
        sines(t, 0);
    }
    for (;;) {
        const int t2 = t + (int)gridDim.x;
        const bool more = t2 < p.num_tokens;
        const int64_t slot2 = more ? slot_of(t2) : -1;
        __syncthreads();  // this token's sines are there, those of the one before are done with
        if (more && slot2 >= 0) sines(t2, buf ^ 1);
        const bool slot_ok = kCache == kCacheNone || slot < p.num_slots;
        if (!slot_ok && tid == 0 && blockIdx.y == 0) flag_error(PA_DEVERR_SLOT);
        // a token with a negative slot is padding: nothing of it is read or written
        // (the loop's bounds are the CTA's: every lane of a warp stays in it)
        for (int pass = slot < 0 ? total : first; pass < total; pass += step) {
            const int row = pass + mine;
            uint4 w2[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};  // the next pass's row, or the next token's
            if (pass + step < total)
                load(t, row + step, w2);
            else if (slot2 >= 0)
                load(t2, first + mine, w2);
            const bool valid = row < total, is_q = row < H, is_v = row >= H + Hk;
            const int h = is_q ? row : is_v ? row - H - Hk : row - H;
            float xa[8], xb[8];
            widen8<T>(w[0], xa);
            widen8<T>(w[1], xb);
            if constexpr (kPairs == kPairsHalf) {
                if (!is_v && j < q8) {
                    // a' = a cos - b sin, b' = b cos + a sin
                    const float4 *co = reinterpret_cast<const float4 *>(cos_s[buf] + 8 * j);
                    const float4 *si = reinterpret_cast<const float4 *>(sin_s[buf] + 8 * j);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float4 f = co[k], g = si[k];
                        const uint64_t c2[2] = {pk2(f.x, f.y), pk2(f.z, f.w)}, s2[2] = {pk2(g.x, g.y), pk2(g.z, g.w)};
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int e = 4 * k + 2 * i;
                            const uint64_t a = pk2(xa[e], xa[e + 1]), b = pk2(xb[e], xb[e + 1]);
                            // sums of two single operations each: the compiler makes a packed
                            // multiply and the packed sum behind it one fused operation, which
                            // rounds once where the definition rounds twice
                            const float2 ac = up2(mul2(a, c2[i])), bs = up2(mul2(b, s2[i]));
                            const float2 bc = up2(mul2(b, c2[i])), as = up2(mul2(a, s2[i]));
                            xa[e] = __fsub_rn(ac.x, bs.x), xa[e + 1] = __fsub_rn(ac.y, bs.y);
                            xb[e] = __fadd_rn(bc.x, as.x), xb[e + 1] = __fadd_rn(bc.y, as.y);
                        }
                    }
                }
            } else if constexpr (kPairs == kPairsInterleaved) {
                if (!is_v) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float *x = i < 4 ? xa + 2 * i : xb + 2 * i - 8;
                        const int pair = 8 * j + i;
                        if (pair < half) {
                            const float co = cos_s[buf][pair], si = sin_s[buf][pair], a = x[0], b = x[1];
                            x[0] = __fsub_rn(__fmul_rn(a, co), __fmul_rn(b, si));
                            x[1] = __fadd_rn(__fmul_rn(b, co), __fmul_rn(a, si));
                        }
                    }
                }
            } else if constexpr (kPairs == kPairsHalfOdd) {
                // pairs that straddle the pieces: single elements, all read before
                // the row is written (it may be written in place)
                const T *src = is_q ? reinterpret_cast<const T *>(p.q) + t * p.q_stride + h * D
                                    : reinterpret_cast<const T *>(p.k) + t * p.k_stride + h * D;
                float o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int d = 16 * j + i;
                    o[i] = valid && !is_v && d < 2 * half ? Elem<T>::to_float(src[d < half ? d + half : d - half]) : 0.f;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int d = 16 * j + i;
                    float &x = i < 8 ? xa[i] : xb[i - 8];
                    if (!is_v && d < 2 * half) {
                        const int pair = d < half ? d : d - half;
                        const float a = __fmul_rn(x, cos_s[buf][pair]), b = __fmul_rn(o[i], sin_s[buf][pair]);
                        x = d < half ? __fsub_rn(a, b) : __fadd_rn(a, b);
                    }
                }
            }
            if (is_q || kCache == kCacheNone) {
                if (valid) {
                    uint4 *dst = is_q ? reinterpret_cast<uint4 *>(p.q_out) + ((int64_t)t * H + h) * (D / 8)
                                      : reinterpret_cast<uint4 *>(p.k_out) + ((int64_t)t * Hk + h) * (D / 8);
                    dst[ca] = narrow8<T>(xa);
                    dst[cb] = narrow8<T>(xb);
                }
            }
            if constexpr (kCache != kCacheNone) {
                if (__any_sync(0xffffffffu, valid && !is_q))  // a warp with queries alone has nothing to store
                    store_row<T, D, kCache>(is_v ? p.v_cache : p.k_cache, xa, xb, slot, h, Hk, ca, cb,
                                            is_v ? p.v_scale : p.k_scale, valid && !is_q && slot_ok);
            }
            w[0] = w2[0];
            w[1] = w2[1];
        }
        if (!more) return;
        if (slot < 0 && slot2 >= 0) load(t2, first + mine, w);  // nothing was in flight behind a padding token
        t = t2;
        slot = slot2;
        buf ^= 1;
    }
}

// The 4-bit cache write without a rotation: D / 16 lanes per (token, K or V,
// head) row, the rows of the whole call dealt out to the grid's lane groups, the
// next row in flight.  Issue-bound: 20001 tokens of 8 heads of 64 in 19 us.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) write_int4_kernel(const RopeParams p) {
    constexpr int LPR = D / 16;
    pdl_launch_dependents();
    const int j = threadIdx.x % LPR, Hk = p.num_kv_heads, rows = p.num_tokens * 2 * Hk;
    const int groups = (int)gridDim.x * (kThreads / LPR);
    // lanes of a warp stay together: its first row decides the loop
    int base = (int)blockIdx.x * (kThreads / LPR) + threadIdx.x / 32 * (32 / LPR);
    const int mine = threadIdx.x % 32 / LPR;
    auto slot_of = [&](int row) -> int64_t { return row < rows ? p.slots[row / (2 * Hk)] : -1; };
    auto load = [&](int row, int64_t slot, uint4 (&w)[2]) {
        w[0] = w[1] = make_uint4(0, 0, 0, 0);
        if (slot < 0 || slot >= p.num_slots) return;
        const int t = row / (2 * Hk), rr = row - t * 2 * Hk;
        const T *src = rr < Hk ? reinterpret_cast<const T *>(p.k) + t * p.k_stride + rr * D
                               : reinterpret_cast<const T *>(p.v) + t * p.v_stride + (rr - Hk) * D;
        w[0] = reinterpret_cast<const uint4 *>(src)[2 * j];
        w[1] = reinterpret_cast<const uint4 *>(src)[2 * j + 1];
    };
    pdl_wait();
    int64_t slot = slot_of(base + mine);
    uint4 w[2];
    load(base + mine, slot, w);
    for (; base < rows; base += groups) {
        const int row = base + mine, row2 = row + groups;
        const int64_t slot2 = row2 < rows ? slot_of(row2) : -1;
        uint4 w2[2];
        load(row2, slot2, w2);
        const int t = row / (2 * Hk), rr = row - t * 2 * Hk;
        if (slot >= p.num_slots && rr == 0 && j == 0) flag_error(PA_DEVERR_SLOT);
        float xa[8], xb[8];
        widen8<T>(w[0], xa);
        widen8<T>(w[1], xb);
        store_row<T, D, kCacheInt4>(rr < Hk ? p.k_cache : p.v_cache, xa, xb, slot, rr < Hk ? rr : rr - Hk, Hk, 2 * j, 2 * j + 1,
                                    1.f, slot >= 0 && slot < p.num_slots);
        slot = slot2;
        w[0] = w2[0];
        w[1] = w2[1];
    }
}

// Cached rows back as 16-bit rows: a lane takes 16 elements of a (token, K or
// V, head) row, up to four such in flight, a grid's width apart, to cover the
// latency of scattered slots (20001 tokens of 8 heads of 64: 14.5 us).
template <typename T, int D, int kCache>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const GatherParams p) {
    constexpr int LPR = D / 16;
    constexpr int kInFlight = 4;
    constexpr int kWords = kCache == kCache16 ? 8 : kCache == kCacheE4m3 ? 4 : 2;  // of a lane's 16 elements
    const int Hk = p.num_kv_heads, items = p.num_tokens * 2 * Hk * LPR, width = (int)gridDim.x * kGatherThreads;
    pdl_wait();
    {
        const int i0 = (int)blockIdx.x * kGatherThreads + threadIdx.x;
        uint32_t w[kInFlight][kWords], ends[kInFlight];
        int64_t dst[kInFlight];  // of the lane's 16 elements, in 16-byte words; -1: nothing
        bool value[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int64_t at = i0 + (int64_t)u * width;
            dst[u] = -1;
            if (at >= items) continue;
            const int i = (int)at;
            const int c = i % LPR, row = i / LPR, tok = row / (2 * Hk), rr = row - tok * 2 * Hk;
            const int64_t t = tok, slot = p.slots[t];
            if (slot < 0) continue;
            if (slot >= p.num_slots) {
                if (rr == 0 && c == 0) flag_error(PA_DEVERR_SLOT);
                continue;
            }
            value[u] = rr >= Hk;
            const int h = value[u] ? rr - Hk : rr;
            dst[u] = ((t * Hk + h) * LPR + c) * 2;
            const unsigned char *cache = reinterpret_cast<const unsigned char *>(value[u] ? p.v_cache : p.k_cache);
            const int64_t chunk = slot / kBlock * Hk + h;
            const int off = (int)(slot % kBlock);
            if constexpr (kCache == kCacheInt4) {
                const unsigned char *base = cache + chunk * int4_chunk_bytes(D);
                const uint2 v = *reinterpret_cast<const uint2 *>(base + off * (D / 2) + c * 8);
                w[u][0] = v.x, w[u][1] = v.y;
                ends[u] = *reinterpret_cast<const uint32_t *>(base + int4_ends_offset(D) + off * 4);
            } else {
                const uint4 *src = reinterpret_cast<const uint4 *>(cache) + ((chunk * kBlock + off) * LPR + c) * (kWords / 4);
#pragma unroll
                for (int k = 0; k < kWords / 4; ++k) {
                    const uint4 v = src[k];
                    w[u][4 * k] = v.x, w[u][4 * k + 1] = v.y, w[u][4 * k + 2] = v.z, w[u][4 * k + 3] = v.w;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            if (dst[u] < 0) continue;
            uint4 *out = reinterpret_cast<uint4 *>(value[u] ? p.value : p.key) + dst[u];
            if constexpr (kCache == kCache16) {
#pragma unroll
                for (int k = 0; k < 2; ++k) out[k] = make_uint4(w[u][4 * k], w[u][4 * k + 1], w[u][4 * k + 2], w[u][4 * k + 3]);
            } else {
                const float scale = value[u] ? p.v_scale : p.k_scale;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float x[8];
                    if constexpr (kCache == kCacheE4m3) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t v = w[u][2 * k + j];
                            const float2 a = e4m3x2_to_float2((uint16_t)(v & 0xffffu)), b = e4m3x2_to_float2((uint16_t)(v >> 16));
                            x[4 * j] = a.x, x[4 * j + 1] = a.y, x[4 * j + 2] = b.x, x[4 * j + 3] = b.y;
                        }
                    } else {
                        const float2 e = int4_ends(ends[u]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = fmaf((float)((w[u][k] >> (4 * j)) & 15u), e.x, e.y);  // the product is exact
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] *= scale;
                    out[k] = narrow8<T>(x);
                }
            }
        }
    }
}

template <typename T, int D, int kCache>
cudaError_t launch_rope_c(const RopeParams &p, cudaStream_t stream) {
    constexpr int kRows = kThreads / (D / 16);
    const int total = p.num_heads + (kCache == kCacheNone ? 1 : 2) * p.num_kv_heads;
    // many tokens: a resident wave that walks over them; fewer: as many CTAs to a
    // token's passes as still make one wave, each of which computes the sines again
    // (32 + 32 + 32 heads of 128 into FP8, a token's 6 passes in one CTA against the
    // rule's: 171 tokens 7.1 us and 4.3, 256 7.4 and 5.0, 512 8.4 and 7.0; 342
    // tokens of 32 + 8 heads 4.2 and 3.2)
    const int passes = (total + kRows - 1) / kRows;
    const int per_token = std::max(1, std::min(passes, kWave / p.num_tokens));
    const dim3 grid(std::min(p.num_tokens, kWave), per_token), block(kThreads);
    const int pairs = p.interleaved ? kPairsInterleaved : p.half % 8 == 0 ? kPairsHalf : kPairsHalfOdd;
    switch (pairs) {
        case kPairsHalf: return launch_pdl(rope_kernel<T, D, kCache, kPairsHalf>, grid, block, 0, stream, p);
        case kPairsInterleaved: return launch_pdl(rope_kernel<T, D, kCache, kPairsInterleaved>, grid, block, 0, stream, p);
        default: return launch_pdl(rope_kernel<T, D, kCache, kPairsHalfOdd>, grid, block, 0, stream, p);
    }
}

template <typename T, int D>
cudaError_t launch_rope_d(const RopeParams &p, int cache, cudaStream_t stream) {
    if (p.half == 0) {  // the 4-bit cache write
        constexpr int kRows = kThreads / (D / 16);
        const int64_t ctas = ((int64_t)p.num_tokens * 2 * p.num_kv_heads + kRows - 1) / kRows;
        return launch_pdl(write_int4_kernel<T, D>, dim3((unsigned)std::min<int64_t>(ctas, 148 * 12)), dim3(kThreads), 0, stream, p);
    }
    switch (cache) {
        case kCacheNone: return launch_rope_c<T, D, kCacheNone>(p, stream);
        case kCache16: return launch_rope_c<T, D, kCache16>(p, stream);
        case kCacheE4m3: return launch_rope_c<T, D, kCacheE4m3>(p, stream);
        default: return launch_rope_c<T, D, kCacheInt4>(p, stream);
    }
}

template <typename T, int D>
cudaError_t launch_gather_d(const GatherParams &p, int cache, cudaStream_t stream) {
    // one row per lane while that still fits the device's threads twice over, four
    // beyond (us with one always, four always and by this rule: 64 tokens of 32 heads
    // of 128 from 4 bits 1.7, 3.6, 1.7; 8192 of 8 13.6, 13.8, 12.2; 4096 of 32 25.1,
    // 22.3, 22.1)
    const int64_t items = (int64_t)p.num_tokens * 2 * p.num_kv_heads * (D / 16);
    const int64_t ctas = (items + kGatherThreads - 1) / kGatherThreads;
    const dim3 grid((unsigned)std::max(std::min<int64_t>(ctas, 2 * 148 * 8), (ctas + 3) / 4)), block(kGatherThreads);
    switch (cache) {
        case kCache16: return launch_pdl(gather_kernel<T, D, kCache16>, grid, block, 0, stream, p);
        case kCacheE4m3: return launch_pdl(gather_kernel<T, D, kCacheE4m3>, grid, block, 0, stream, p);
        default: return launch_pdl(gather_kernel<T, D, kCacheInt4>, grid, block, 0, stream, p);
    }
}

// The templates' cache kind of a pa_dims.kv_dtype (-1: no cache).
int cache_kind(int kv_dtype) {
    return kv_dtype < 0 ? kCacheNone : kv_dtype == PA_FP8_E4M3 ? kCacheE4m3 : kv_dtype == PA_INT4 ? kCacheInt4 : kCache16;
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, int dtype, int head_dim, int kv_dtype, cudaStream_t stream) {
    if (p.num_tokens == 0) return cudaSuccess;
    const int cache = cache_kind(kv_dtype);
    if (dtype == PA_F16)
        return head_dim == 64 ? launch_rope_d<__half, 64>(p, cache, stream) : launch_rope_d<__half, 128>(p, cache, stream);
    return head_dim == 64 ? launch_rope_d<__nv_bfloat16, 64>(p, cache, stream)
                          : launch_rope_d<__nv_bfloat16, 128>(p, cache, stream);
}

cudaError_t launch_gather_cache(const GatherParams &p, int dtype, int head_dim, int kv_dtype, cudaStream_t stream) {
    if (p.num_tokens == 0) return cudaSuccess;
    const int cache = cache_kind(kv_dtype);
    if (dtype == PA_F16)
        return head_dim == 64 ? launch_gather_d<__half, 64>(p, cache, stream)
                              : launch_gather_d<__half, 128>(p, cache, stream);
    return head_dim == 64 ? launch_gather_d<__nv_bfloat16, 64>(p, cache, stream)
                          : launch_gather_d<__nv_bfloat16, 128>(p, cache, stream);
}

}  // namespace pa
