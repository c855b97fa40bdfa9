// pa_rope.cu -- rotary positions, the cache write of rotated keys, the 4-bit
// cache write and the read-back of cached rows (pa_rope, pa_rope_and_cache,
// pa_reshape_and_cache_int4, pa_gather_cache).
//
// A pair (a, b) of a head at position p with frequency f turns by p f:
//   a' = m (a cos - b sin),  b' = m (b cos + a sin).
// All of it is data movement: each element is read once and written once.
//
// CTA = one token.  Its first rotary_dim / 2 threads compute the token's
// (m cos, m sin) pairs in fp64 and share them through shared memory, so the
// sines are computed once per token and not once per head.  Then D / 8 lanes
// take a row (a head's D elements): 16 bytes per lane, the partner elements
// of a pair by a shuffle.
#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_int4.cuh"

namespace pa {

namespace {

constexpr int kBlock = 16;
constexpr int kThreads = 256;
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

// The row of `slot` and KV head h takes the 8 elements x (dims 8 c ..) of
// each of the row's LPR lanes (all of them converged; `live`: this lane's
// row is written).
template <typename T, int D, int kCache>
__device__ __forceinline__ void store_row(void *cache, const float (&x)[8], int64_t slot, int h, int num_kv_heads,
                                          int c, float scale, bool live) {
    constexpr int LPR = D / 8;
    const int64_t blk = slot / kBlock;
    const int off = (int)(slot % kBlock);
    const int64_t chunk = blk * num_kv_heads + h;
    if constexpr (kCache == kCache16) {
        if (live) reinterpret_cast<uint4 *>(cache)[(chunk * kBlock + off) * LPR + c] = narrow8<T>(x);
    } else if constexpr (kCache == kCacheE4m3) {
        if (live) {
            uint32_t u[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t lo = float2_to_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
                const uint32_t hi = float2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
                u[i] = lo | (hi << 16);
            }
            reinterpret_cast<uint2 *>(cache)[(chunk * kBlock + off) * LPR + c] = make_uint2(u[0], u[1]);
        }
    } else if constexpr (kCache == kCacheInt4) {
        float lo = x[0], hi = x[0];
        bool fine = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, x[i]);
            hi = fmaxf(hi, x[i]);
            fine = fine && fabsf(x[i]) < INFINITY;  // false for NaN too
        }
        if (!fine) hi = INFINITY;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        if (!live) return;
        __nv_bfloat16 lb = __float2bfloat16_rn(lo);
        const float low = __bfloat162float(lb);
        __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, low), 15.f));
        const float sc = __bfloat162float(sb);
        uint32_t codes = 0;
        if (!(fabsf(sc) < INFINITY)) {  // a NaN or an infinity in the row, or a range past fp32's
            lb = sb = __float2bfloat16_rn(NAN);
        } else if (sc != 0.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[i], low), sc)), 0.f), 15.f);
                codes |= (uint32_t)u << (4 * i);
            }
        }
        unsigned char *base = reinterpret_cast<unsigned char *>(cache) + chunk * int4_chunk_bytes(D);
        *reinterpret_cast<uint32_t *>(base + off * (D / 2) + c * 4) = codes;
        if (c == 0) {
            const uint32_t ends = (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(lb) << 16);
            *reinterpret_cast<uint32_t *>(base + int4_ends_offset(D) + off * 4) = ends;
        }
    }
}

template <typename T, int D, int kCache>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
    constexpr int LPR = D / 8;        // lanes per row
    constexpr int RPW = 32 / LPR;     // rows per warp
    __shared__ __align__(16) float2 cs[kMaxHalf];
    const int t = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // The decode kernels read q before they wait for the kernel in front of
    // them, so a kernel that writes q or k does not let the next one start
    // early; a cache write alone does.
    if (!p.q_out && !p.k_out) pdl_launch_dependents();
    pdl_wait();
    int64_t slot = 0;
    if constexpr (kCache != kCacheNone) {
        slot = p.slots[t];
        if (slot < 0) return;  // padding token
    }
    const int half = p.half;
    if (tid < half) {
        double s, c;
        sincos_turns((double)p.positions[t] * p.inv_freq[tid] * 0.15915494309189533576888, &s, &c);
        if (p.inverse) s = -s;
        cs[tid] = make_float2((float)(c * p.magnitude), (float)(s * p.magnitude));
    }
    __syncthreads();
    bool slot_ok = true;
    if constexpr (kCache != kCacheNone) {
        slot_ok = slot < p.num_slots;
        if (!slot_ok && tid == 0) flag_error(PA_DEVERR_SLOT);
    }
    const int c = lane % LPR, d0 = 8 * c;  // this lane's dims d0 .. d0 + 7
    const int H = p.num_heads, Hk = p.num_kv_heads;
    const int total = H + (kCache == kCacheNone ? Hk : 2 * Hk);
    for (int base = warp * RPW; base < total; base += (kThreads / 32) * RPW) {
        const int row = base + lane / LPR;
        const bool valid = row < total;
        const bool is_q = row < H, is_v = row >= H + Hk;
        const int h = is_q ? row : is_v ? row - H - Hk : row - H;
        const T *src = is_q ? reinterpret_cast<const T *>(p.q) + t * p.q_stride
                       : is_v ? reinterpret_cast<const T *>(p.v) + t * p.v_stride
                              : reinterpret_cast<const T *>(p.k) + t * p.k_stride;
        src += (int64_t)h * D;
        float x[8];
        {
            const uint4 w = valid ? *reinterpret_cast<const uint4 *>(src + d0) : make_uint4(0, 0, 0, 0);
            widen8<T>(w, x);
        }
        const bool turn = valid && !is_v;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i];
        if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (turn && 4 * c + i < half) {
                    const float2 k = cs[4 * c + i];
                    y[2 * i] = __fsub_rn(__fmul_rn(x[2 * i], k.x), __fmul_rn(x[2 * i + 1], k.y));
                    y[2 * i + 1] = __fadd_rn(__fmul_rn(x[2 * i + 1], k.x), __fmul_rn(x[2 * i], k.y));
                }
            }
        } else {
            float o[8];  // the pair's other element
            if (half % 8 == 0) {
                const int step = half / 8;
                const int other = lane - c + (c < step ? c + step : c < 2 * step ? c - step : c);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, x[i], other);
            } else {
                // pairs that straddle the lanes' 8 dims: single elements, all
                // read before the row is written (it may be written in place)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int d = d0 + i;
                    o[i] = turn && d < 2 * half ? Elem<T>::to_float(src[d < half ? d + half : d - half]) : 0.f;
                }
                __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int d = d0 + i;
                if (turn && d < 2 * half) {
                    const float2 k = cs[d < half ? d : d - half];
                    const float a = __fmul_rn(x[i], k.x), b = __fmul_rn(o[i], k.y);
                    y[i] = d < half ? __fsub_rn(a, b) : __fadd_rn(a, b);
                }
            }
        }
        if (is_q) {
            if (valid) *reinterpret_cast<uint4 *>(reinterpret_cast<T *>(p.q_out) + ((int64_t)t * H + h) * D + d0) = narrow8<T>(y);
        } else if constexpr (kCache == kCacheNone) {
            if (valid) *reinterpret_cast<uint4 *>(reinterpret_cast<T *>(p.k_out) + ((int64_t)t * Hk + h) * D + d0) = narrow8<T>(y);
        }
        if constexpr (kCache != kCacheNone)
            store_row<T, D, kCache>(is_v ? p.v_cache : p.k_cache, y, slot, h, Hk, c, is_v ? p.v_scale : p.k_scale,
                                    valid && !is_q && slot_ok);
    }
}

// Cached rows back as 16-bit rows: D / 8 lanes per row, rows (token, K or V,
// head) in the order they are written.
template <typename T, int D, int kCache>
__global__ void __launch_bounds__(kThreads) gather_kernel(const GatherParams p) {
    constexpr int LPR = D / 8;
    pdl_wait();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int c = (int)(i % LPR);
    const int64_t row = i / LPR;
    const int Hk = p.num_kv_heads;
    const int64_t t = row / (2 * Hk);
    if (t >= p.num_tokens) return;
    const int rr = (int)(row % (2 * Hk)), h = rr % Hk;
    const bool is_v = rr >= Hk;
    const int64_t slot = p.slots[t];
    if (slot < 0) return;
    if (slot >= p.num_slots) {
        if (rr == 0 && c == 0) flag_error(PA_DEVERR_SLOT);
        return;
    }
    const void *cache = is_v ? p.v_cache : p.k_cache;
    const float scale = is_v ? p.v_scale : p.k_scale;
    const int64_t chunk = (slot / kBlock) * Hk + h;
    const int off = (int)(slot % kBlock);
    uint4 *dst = reinterpret_cast<uint4 *>(is_v ? p.value : p.key) + (t * Hk + h) * LPR + c;
    if constexpr (kCache == kCache16) {
        *dst = reinterpret_cast<const uint4 *>(cache)[(chunk * kBlock + off) * LPR + c];
    } else {
        float x[8];
        if constexpr (kCache == kCacheE4m3) {
            const uint2 w = reinterpret_cast<const uint2 *>(cache)[(chunk * kBlock + off) * LPR + c];
            const uint32_t u[2] = {w.x, w.y};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 a = e4m3x2_to_float2((uint16_t)(u[k] & 0xffffu)), b = e4m3x2_to_float2((uint16_t)(u[k] >> 16));
                x[4 * k] = a.x;
                x[4 * k + 1] = a.y;
                x[4 * k + 2] = b.x;
                x[4 * k + 3] = b.y;
            }
        } else {
            const unsigned char *base = reinterpret_cast<const unsigned char *>(cache) + chunk * int4_chunk_bytes(D);
            const uint32_t w = *reinterpret_cast<const uint32_t *>(base + off * (D / 2) + c * 4);
            const float2 e = int4_ends(*reinterpret_cast<const uint32_t *>(base + int4_ends_offset(D) + off * 4));
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = fmaf((float)((w >> (4 * k)) & 15u), e.x, e.y);  // the product is exact
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= scale;
        *dst = narrow8<T>(x);
    }
}

template <typename T, int D>
cudaError_t launch_rope_d(const RopeParams &p, int cache, cudaStream_t stream) {
    const dim3 grid(p.num_tokens), block(kThreads);
    switch (cache) {
        case kCacheNone: return launch_pdl(rope_kernel<T, D, kCacheNone>, grid, block, 0, stream, p);
        case kCache16: return launch_pdl(rope_kernel<T, D, kCache16>, grid, block, 0, stream, p);
        case kCacheE4m3: return launch_pdl(rope_kernel<T, D, kCacheE4m3>, grid, block, 0, stream, p);
        default: return launch_pdl(rope_kernel<T, D, kCacheInt4>, grid, block, 0, stream, p);
    }
}

template <typename T, int D>
cudaError_t launch_gather_d(const GatherParams &p, int cache, cudaStream_t stream) {
    const int64_t items = (int64_t)p.num_tokens * 2 * p.num_kv_heads * (D / 8);
    const dim3 grid((unsigned)((items + kThreads - 1) / kThreads)), block(kThreads);
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
