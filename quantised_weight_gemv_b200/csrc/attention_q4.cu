// attention_q4.cu -- decode attention over a 4-bit KV cache, sm_100a.
//
//   s_t = scale * q . K[t]   p = softmax(s over t < lens[b] - (Tq - 1 - i))   o = sum_t p_t V[t]
//
// One CTA per (sequence, query token, query head); its warps take positions in
// turn, each with its own online softmax (running maximum m, sum l, output o;
// all fp32), and are merged in shared memory.
#include <cuda_fp16.h>

#include <cmath>
#include <cstring>

#include "bq_device.cuh"
#include "bq_internal.h"
#include "bq_kv.h"

namespace bq {
namespace aq {

constexpr int kWarpsCta = 4;
constexpr float kFloor = -1e30f;          // a running maximum that no score has reached

struct Args {
    const uint8_t *kc, *vc;
    const uint16_t *ks, *vs;
    const uint16_t *q;
    const int32_t *lens;
    void *o;
    int B, Tq, Hkv, G, Tmax;
    float scale2;                         // scale * log2(e)
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Lane l holds the elements of bytes l * D/64 .. of a row: low nibble element
// i, high nibble element i + 16 of the byte's block.
template <int D, typename O>
__global__ void __launch_bounds__(kWarpsCta * 32) attn_q4_kernel(const Args a)
{
    constexpr int NB = D / 64, NE = 2 * NB;           // bytes and elements per lane
    __shared__ float sm[kWarpsCta], sl[kWarpsCta], so[kWarpsCta][D];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int heads = a.Hkv * a.G;
    const int j = blockIdx.x % heads, i = blockIdx.x / heads % a.Tq;
    const int b = blockIdx.x / heads / a.Tq;
    const int h = j / a.G;
    const int n = min(max(a.lens[b], 0), a.Tmax) - (a.Tq - 1 - i);
    const size_t row0 = ((size_t)b * a.Hkv + h) * a.Tmax;
    const size_t qrow = (((size_t)b * a.Tq + i) * heads + j) * D;
    const int byte = lane * NB, blk = byte / 16;
    int el[NE];
    float qv[NE], o[NE];
#pragma unroll
    for (int e = 0; e < NE; e++) {
        el[e] = 32 * blk + (byte + (e >> 1)) % 16 + 16 * (e & 1);
        qv[e] = __half2float(__ushort_as_half(a.q[qrow + el[e]]));
        o[e] = 0.0f;
    }
    float m = kFloor, l = 0.0f;
    for (int t = warp; t < n; t += kWarpsCta) {
        const size_t r = row0 + t;
        float kk[NE], vv[NE];
        const float kd = __half2float(__ushort_as_half(a.ks[r * (D / 32) + blk]));
        const float vd = __half2float(__ushort_as_half(a.vs[r * (D / 32) + blk]));
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < NE; e++) {
            const int sh = 4 * (e & 1);
            kk[e] = (float)((int)(a.kc[r * (D / 2) + byte + (e >> 1)] >> sh & 15) - 8);
            vv[e] = (float)((int)(a.vc[r * (D / 2) + byte + (e >> 1)] >> sh & 15) - 8);
            s = fmaf(qv[e], kk[e], s);
        }
        s *= kd;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= a.scale2;
        const float mn = fmaxf(m, s);
        const float f = ex2(m - mn), p = ex2(s - mn);
        l = fmaf(l, f, p);
        m = mn;
#pragma unroll
        for (int e = 0; e < NE; e++)
            o[e] = fmaf(o[e], f, p * vd * vv[e]);
    }
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < NE; e++)
        so[warp][el[e]] = o[e];
    __syncthreads();
    if (threadIdx.x < D) {
        float M = kFloor, L = 0.0f, acc = 0.0f;
        for (int w = 0; w < kWarpsCta; w++)
            M = fmaxf(M, sm[w]);
        for (int w = 0; w < kWarpsCta; w++) {
            const float f = ex2(sm[w] - M);
            L = fmaf(f, sl[w], L);
            acc = fmaf(f, so[w][threadIdx.x], acc);
        }
        static_cast<O *>(a.o)[qrow + threadIdx.x] = (O)(n > 0 ? acc / L : 0.0f);
    }
}

}  // namespace aq
}  // namespace bq

using namespace bq;

extern "C" size_t bq_attn_q4_workspace_bytes(int32_t D, int32_t Tq, int32_t G)
{
    if ((D != 64 && D != 128) || Tq < 1 || Tq > 32 || G < 1 || G > 16)
        return 0;
    return 256;
}

extern "C" int32_t bq_attn_decode_q4(const bq_kv_cache_q4 *kv, const uint16_t *q, const int32_t *lens,
                                     int32_t B, int32_t Tq, int32_t Hkv, int32_t G, float scale, void *o,
                                     int32_t o_dtype, void *ws, size_t ws_bytes, int32_t *dev_status,
                                     void *stream)
{
    if (!kv || !kv->k_codes || !kv->k_scales || !kv->v_codes || !kv->v_scales || !q || !lens || !o || !ws)
        return BQ_ERR_NULL;
    const size_t need = bq_attn_q4_workspace_bytes(kv->D, Tq, G);
    if (need == 0 || kv->Tmax < 32 || kv->Tmax % 32 != 0 || Hkv < 1 || !std::isfinite(scale) ||
        (o_dtype != BQ_F32 && o_dtype != BQ_F16))
        return BQ_ERR_SHAPE;
    if (B < 1)
        return BQ_ERR_BATCH;
    if ((long long)B * Hkv >= (1LL << 31) || (long long)B * Hkv * kv->Tmax >= (1LL << 31) ||
        (long long)B * Hkv * Tq * G >= (1LL << 31))
        return BQ_ERR_SHAPE;
    if (!aligned16(kv->k_codes) || !aligned16(kv->k_scales) || !aligned16(kv->v_codes) ||
        !aligned16(kv->v_scales) || !aligned16(q) || !aligned16(o) || !aligned16(ws) ||
        (reinterpret_cast<uintptr_t>(lens) & 3u))
        return BQ_ERR_ALIGN;
    if (ws_bytes < need)
        return BQ_ERR_WORKSPACE;
    (void)dev_status;
    aq::Args a = {kv->k_codes, kv->v_codes, kv->k_scales, kv->v_scales, q, lens, o,
                  B, Tq, Hkv, G, kv->Tmax, scale * 1.4426950408889634f};
    const void *kernel = kv->D == 64 ? (o_dtype == BQ_F32 ? (const void *)aq::attn_q4_kernel<64, float>
                                                          : (const void *)aq::attn_q4_kernel<64, __half>)
                                     : (o_dtype == BQ_F32 ? (const void *)aq::attn_q4_kernel<128, float>
                                                          : (const void *)aq::attn_q4_kernel<128, __half>);
    void *args[] = {&a};
    return launch_pdl(kernel, dim3((unsigned)(B * Hkv * Tq * G)), dim3(aq::kWarpsCta * 32), 0,
                      static_cast<cudaStream_t>(stream), args) == cudaSuccess
               ? BQ_OK
               : BQ_ERR_CUDA;
}
