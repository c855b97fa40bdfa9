// pa_decode_int4.cu -- paged decode attention over 4-bit caches (PA_INT4).
//
// With codes u, row scales s and lowest values l,
//   logit of token t = c (s_t (q . u_t) + l_t sum(q)),   c = scale log2(e) k_scale
//   out = sum_t p_t (s'_t u'_t + l'_t) / sum_t p_t,      p_t = 2^(logit - m)
//
// CTA = (KV partition, KV head, sequence), 4 warps; warp w takes the
// partition's tokens w, w + 4, ...; a lane holds D / 32 dims of every query
// row of the KV head and its part of the running output.
#include "pa_common.cuh"
#include "pa_decode.h"
#include "pa_int4.cuh"
#include "pa_simt.cuh"

namespace pa {

namespace {

constexpr int kWarps = 4;

template <typename T, int D, int G>
__global__ void __launch_bounds__(kWarps * 32) decode_int4_kernel(const DecodeParams p) {
    using E = Elem<T>;
    constexpr int kV = D / 32;
    __shared__ float red_m[kWarps * G], red_l[kWarps * G], red_acc[kWarps * G * D];
    const int part = blockIdx.x, kvh = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int s = scheduled_seq(p, blockIdx.z, part == 0 && kvh == 0 && tid == 0);
    if (s < 0) return;
    const int rows = p.group * p.q_len;
    const SeqSplit sp = seq_split(p, s, part == 0 && kvh == 0 && tid == 0);
    if (part >= sp.nparts) return;
    T *out = reinterpret_cast<T *>(p.out);
    if (sp.L == 0) {
        for (int i = tid; i < rows * D; i += blockDim.x) out[query_row(p, s, kvh, i / D) * D + i % D] = E::from_float(0.f);
        return;
    }
    float q[G][kV], qsum[G], m[G], l[G], acc[G][kV];
    int lo[G], hi[G];
#pragma unroll
    for (int r = 0; r < G; ++r) {
        row_range(p, sp.L, r, &lo[r], &hi[r]);
        qsum[r] = 0.f;
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            q[r][e] = r < rows ? E::to_float(reinterpret_cast<const T *>(p.q)[query_row(p, s, kvh, r) * D + lane * kV + e]) : 0.f;
            qsum[r] += q[r][e];
            acc[r][e] = 0.f;
        }
    }
    const int b0 = sp.bfirst + part * p.part_blocks, b1 = min(b0 + p.part_blocks, sp.nblk);
    const int t1 = min(b1 * kBlock, sp.L);
    for (int t = b0 * kBlock + warp; t < t1; t += kWarps) {
        const int64_t phys = checked_block(p, p.block_tables[(int64_t)s * p.max_blocks_per_seq + t / kBlock]);
        const int64_t at = (phys * p.num_kv_heads + kvh) * int4_chunk_bytes(D);
        const unsigned char *kc = reinterpret_cast<const unsigned char *>(p.k_cache) + at;
        const unsigned char *vc = reinterpret_cast<const unsigned char *>(p.v_cache) + at;
        const int off = t % kBlock;
        const float2 ke = int4_ends(*reinterpret_cast<const uint32_t *>(kc + int4_ends_offset(D) + off * 4));
        const float2 ve = int4_ends(*reinterpret_cast<const uint32_t *>(vc + int4_ends_offset(D) + off * 4));
        float k[kV], v[kV];
#pragma unroll
        for (int e = 0; e < kV; ++e) {
            const int at_d = lane * kV + e;
            k[e] = (float)((kc[off * (D / 2) + at_d / 2] >> (4 * (at_d & 1))) & 15);
            v[e] = fmaf((float)((vc[off * (D / 2) + at_d / 2] >> (4 * (at_d & 1))) & 15), ve.x, ve.y);
        }
#pragma unroll
        for (int r = 0; r < G; ++r) {
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < kV; ++e) x = fmaf(q[r][e], k[e], x);
            x = fmaf(ke.x, x, ke.y * qsum[r]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (t < lo[r] || t > hi[r]) continue;
            x *= p.scale_log2;
            const float mn = fmaxf(m[r], x), alpha = exp2f(m[r] - mn), w = exp2f(x - mn);
            m[r] = mn;
            l[r] = fmaf(l[r], alpha, w);
#pragma unroll
            for (int e = 0; e < kV; ++e) acc[r][e] = fmaf(acc[r][e], alpha, w * v[e]);
        }
    }
#pragma unroll
    for (int r = 0; r < G; ++r) {
#pragma unroll
        for (int e = 0; e < kV; ++e) red_acc[(warp * G + r) * D + lane * kV + e] = acc[r][e];
        if (lane == 0) {
            red_m[warp * G + r] = m[r];
            red_l[warp * G + r] = l[r];
        }
    }
    __syncthreads();
    for (int i = tid; i < rows * D; i += blockDim.x) {
        const int h = i / D, d = i % D;
        float lse;
        const float o = combine_warps<D, G, kWarps>(red_m, red_l, red_acc, h, d, &lse) * p.v_scale;
        const int64_t qr = query_row(p, s, kvh, h);
        if (sp.nparts == 1) {
            out[qr * D + d] = E::from_float(o);
        } else {
            p.ws_o[(qr * p.max_parts + part) * D + d] = o;
            if (d == 0) p.ws_lse[qr * p.max_parts + part] = lse;
        }
    }
}

template <typename T, int D>
cudaError_t launch_int4_d(const DecodeParams &p, int rows, cudaStream_t stream) {
    const dim3 grid(p.max_parts, p.num_kv_heads, p.num_seqs), block(kWarps * 32);
    cudaError_t e = rows <= 8 ? launch_pdl(decode_int4_kernel<T, D, 8>, grid, block, 0, stream, p)
                              : launch_pdl(decode_int4_kernel<T, D, 16>, grid, block, 0, stream, p);
    if (e != cudaSuccess || p.max_parts == 1) return e;
    return launch_merge_partitions(p, std::is_same<T, __nv_bfloat16>::value ? PA_BF16 : PA_F16, D, stream);
}

}  // namespace

cudaError_t launch_decode_int4(const DecodeParams &p, int dtype, int head_dim, int rows, cudaStream_t stream) {
    if (dtype == PA_F16)
        return head_dim == 64 ? launch_int4_d<__half, 64>(p, rows, stream) : launch_int4_d<__half, 128>(p, rows, stream);
    return head_dim == 64 ? launch_int4_d<__nv_bfloat16, 64>(p, rows, stream)
                          : launch_int4_d<__nv_bfloat16, 128>(p, rows, stream);
}

}  // namespace pa
