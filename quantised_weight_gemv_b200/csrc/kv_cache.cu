// kv_cache.cu -- writing new keys and values into a quantised KV cache and
// reading them back (Q4 and Q8), sm_100a.
//
// A row (one position of one KV head) is D elements in 32-element blocks:
//   a = max|x|,  d = fp16(a / L),  code = round-half-away(x / d) clamped,
// L = 7 (Q4) or 127 (Q8); value = d * code.  The bits are those of the host
// quantisers (bq_quantize_q4 / _q8), which the caches are defined by.
//
// Both directions are bound by memory: a thread moves 8 elements of a key row
// and the same 8 of the value row, four threads a block (its maximum takes two
// shuffles), so a row's threads read and write contiguous sectors.  A thread's
// elements are 4j .. 4j+3 and 16+4j .. 16+4j+3 of its block (j = 0..3): exactly
// the two nibbles of the Q4 bytes 4j .. 4j+3, one 32-bit store.
//
// The Q8 cache keeps values transposed ([D][Tmax]), so its value side goes
// through shared memory in tiles of 64 positions cut at multiples of 64: every
// tile inside a written range is whole sectors, and only the range's two ends
// use byte stores (bytes of one sector belong to different tokens, so wider
// read-modify-writes there would race with other calls' positions).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>
#include <type_traits>

#include "bq_device.cuh"
#include "bq_internal.h"
#include "bq_kv.h"

namespace bq {
namespace kvc {

constexpr int kStatusPosition = 1 << BQ_ERR_POSITION;
constexpr int kThreads = 256;
constexpr int kTile = 64;                 // positions per tile of the transposed Q8 values

struct Rows {
    const void *k, *v;                    // a read's destinations (cast at the store)
    int64_t k_batch, k_token, k_head, v_batch, v_token, v_head;
};
struct Args {
    uint8_t *kc, *vc;
    uint16_t *ks, *vs;
    Rows r;
    const int32_t *start, *count;
    int *status;
    int B, Hkv, T, Tmax;
};

// The rows of sequence b that exist, and the status of a count outside [0, T].
__device__ __forceinline__ int row_count(const Args &a, int b, bool *bad)
{
    const int n = a.count ? a.count[b] : a.T;
    *bad = n < 0 || n > a.T;
    return min(max(n, 0), a.T);
}

// ---------------------------------------------------------------- quantise ----
// 8 elements as fp32 from a row: 4 at p, 4 at p + 16.
template <typename E>
__device__ __forceinline__ void load8(const E *p, float (&x)[8])
{
    if constexpr (sizeof(E) == 4) {
        const float4 lo = __ldcs(reinterpret_cast<const float4 *>(p));
        const float4 hi = __ldcs(reinterpret_cast<const float4 *>(p + 16));
        x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w;
        x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
    } else {
        const uint2 w[2] = {__ldcs(reinterpret_cast<const uint2 *>(p)),
                            __ldcs(reinterpret_cast<const uint2 *>(p + 16))};
        E e[8];
        memcpy(e, w, sizeof(e));
#pragma unroll
        for (int i = 0; i < 8; i++)
            x[i] = (float)e[i];
    }
}

// Block scale and the thread's 8 integer codes (-8..7 or -127..127).  The 4
// threads of the block call it together (all 32 lanes of the warp execute it).
// Returns false if the block is not finite or its scale overflows fp16; its
// scale and codes are then 0.
//
// x / d is an IEEE quotient in the definition.  t = x * (1/d) differs from it
// by less than |x/d| 1.5 * 2^-23 (three fp32 roundings), and |x/d| <= 1.5 L at
// the worst subnormal scale: less than 2^-14 for Q8 and 2^-18 for Q4.  Where t
// is at least that far from a half both round to the same integer; otherwise
// (about 1 element in 10^4, 10^5) the thread divides.
template <int FMT>
__device__ __forceinline__ bool quantise8(float (&x)[8], int (&q)[8], uint16_t &scale)
{
    constexpr float kLevels = FMT == 4 ? 7.0f : 127.0f;
    constexpr float kLow = FMT == 4 ? -8.0f : -127.0f;
    uint32_t a = 0;                                   // |x| bits: NaN > inf > finite
#pragma unroll
    for (int i = 0; i < 8; i++)
        a = max(a, __float_as_uint(x[i]) & 0x7fffffffu);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    bool ok = a < 0x7f800000u;
    const __half dh = __float2half_rn(__fdiv_rn(__uint_as_float(a), kLevels));
    scale = __half_as_ushort(dh);
    ok = ok && (scale & 0x7c00u) != 0x7c00u;
    const float d = __half2float(dh);
    const bool live = ok && d != 0.0f;
    if (!ok)
        scale = 0;
    if (!live) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            q[i] = 0;
        return ok;
    }
    const float r = __frcp_rn(d);
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float t = x[i] * r;
        const float n = rintf(t);
        far = fmaxf(far, fabsf(t - n));
        q[i] = (int)fminf(fmaxf(n, kLow), kLevels);
    }
    if (far > (FMT == 4 ? 0.5f - 0x1p-18f : 0.5f - 0x1p-14f)) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            q[i] = (int)fminf(fmaxf(roundf(__fdiv_rn(x[i], d)), kLow), kLevels);
    }
    return ok;
}

__device__ __forceinline__ uint32_t bytes4(int a, int b, int c, int d)
{
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)(d & 255) << 24;
}
// Q4 code bytes 4j .. 4j+3 of the block: element 4j+c low, 16+4j+c high.
__device__ __forceinline__ uint32_t pack_q4(const int (&q)[8])
{
    return (bytes4(q[0], q[1], q[2], q[3]) & 0x0f0f0f0fu ^ 0x08080808u) |
           (bytes4(q[4], q[5], q[6], q[7]) & 0x0f0f0f0fu ^ 0x08080808u) << 4;
}

template <int D, typename E>
__global__ void __launch_bounds__(kThreads) append_q4_kernel(const Args a)
{
    constexpr int kLanes = D / 8;                     // threads per row
    pdl_launch_dependents();
    pdl_wait();
    const long long item = ((long long)blockIdx.x * kThreads + threadIdx.x) / kLanes;
    const int j = threadIdx.x % kLanes, blk = j >> 2, jj = j & 3;
    const bool in = item < (long long)a.T * a.Hkv;
    const int i = in ? (int)(item / a.Hkv) : 0, h = in ? (int)(item % a.Hkv) : 0;
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const E *kp = static_cast<const E *>(a.r.k) + b * a.r.k_batch + i * a.r.k_token + h * a.r.k_head + 32 * blk + 4 * jj;
        const E *vp = static_cast<const E *>(a.r.v) + b * a.r.v_batch + i * a.r.v_token + h * a.r.v_head + 32 * blk + 4 * jj;
        float x[2][8];
        load8(kp, x[0]);                              // (rows past the count exist and are dropped)
        load8(vp, x[1]);
        bool bad_count;
        const int n = row_count(a, b, &bad_count);
        const long long p = (long long)a.start[b] + i;
        const bool mine = in && i < n, there = p >= 0 && p < a.Tmax;
        const size_t row = ((size_t)b * a.Hkv + h) * a.Tmax + (size_t)(there ? p : 0);
        int bits = 0;
        if (in && (bad_count || (mine && !there)))
            bits = kStatusPosition;
#pragma unroll
        for (int s = 0; s < 2; s++) {
            int q[8];
            uint16_t sc;
            const bool ok = quantise8<4>(x[s], q, sc);
            if (!mine || !there)
                continue;
            if (!ok)
                bits |= kStatusRange;
            *reinterpret_cast<uint32_t *>((s ? a.vc : a.kc) + row * (D / 2) + 16 * blk + 4 * jj) = pack_q4(q);
            if (jj == 0)
                (s ? a.vs : a.ks)[row * (D / 32) + blk] = sc;
        }
        if (bits && a.status)
            atomicOr(a.status, bits);
    }
}

// One block: 64 positions (a tile cut at a multiple of 64) of one (sequence,
// head).  Keys go straight to their rows; value codes are laid down in shared
// memory as [D][64] and stored along positions.
template <typename E>
__global__ void __launch_bounds__(kThreads) append_q8_kernel(const Args a)
{
    constexpr int D = 128, kLanes = D / 8, kRowsPass = kThreads / kLanes, kLd = kTile + 4;
    __shared__ alignas(16) uint8_t vt[D * kLd];
    pdl_launch_dependents();
    pdl_wait();
    const int h = blockIdx.y;
    const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes, blk = lane >> 2, jj = lane & 3;
    for (int b = blockIdx.z; b < a.B; b += gridDim.z) {
        bool bad_count;
        const int n = row_count(a, b, &bad_count);
        const long long s0 = a.start[b];
        if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0 && a.status &&
            (bad_count || (n > 0 && (s0 < 0 || s0 + n > a.Tmax))))
            atomicOr(a.status, kStatusPosition);
        // positions lo .. hi-1 of this tile are written (row i = position - s0)
        const long long first = max(s0, 0LL), end = min(s0 + n, (long long)a.Tmax);
        const long long t0 = (first / kTile + blockIdx.x) * kTile;
        const int lo = (int)max(first - t0, 0LL), hi = (int)min(max(end - t0, 0LL), (long long)kTile);
        if (lo >= hi)
            continue;                                 // (the same for the whole block)
        const size_t bh = (size_t)b * a.Hkv + h;
        for (int p0 = lo; p0 < hi; p0 += kRowsPass) {
            const int p = p0 + sub;
            const bool live = p < hi;
            const long long i = t0 + (live ? p : lo) - s0;
            const E *kp = static_cast<const E *>(a.r.k) + b * a.r.k_batch + i * a.r.k_token + h * a.r.k_head + 32 * blk + 4 * jj;
            const E *vp = static_cast<const E *>(a.r.v) + b * a.r.v_batch + i * a.r.v_token + h * a.r.v_head + 32 * blk + 4 * jj;
            float x[2][8];
            load8(kp, x[0]);
            load8(vp, x[1]);
            const size_t row = bh * a.Tmax + (size_t)(t0 + p);
            bool fine = true;
#pragma unroll
            for (int s = 0; s < 2; s++) {
                int q[8];
                uint16_t sc;
                fine = quantise8<8>(x[s], q, sc) && fine;
                if (!live)
                    continue;
                if (s == 0) {
                    uint32_t *dst = reinterpret_cast<uint32_t *>(a.kc + row * D + 32 * blk + 4 * jj);
                    dst[0] = bytes4(q[0], q[1], q[2], q[3]);
                    dst[4] = bytes4(q[4], q[5], q[6], q[7]);
                } else {
#pragma unroll
                    for (int c = 0; c < 8; c++)
                        vt[(32 * blk + 4 * jj + (c & 3) + 16 * (c >> 2)) * kLd + p] = (uint8_t)q[c];
                }
                if (jj == 0)
                    (s ? a.vs : a.ks)[row * (D / 32) + blk] = sc;
            }
            if (live && !fine && a.status)
                atomicOr(a.status, kStatusRange);
        }
        __syncthreads();
        uint8_t *dst = a.vc + bh * D * a.Tmax + t0;
        for (int w = threadIdx.x; w < D * (kTile / 4); w += kThreads) {
            const int d = w / (kTile / 4), p = w % (kTile / 4) * 4;
            uint8_t *out = dst + (size_t)d * a.Tmax + p;
            const uint8_t *src = vt + d * kLd + p;
            if (p >= lo && p + 4 <= hi)
                *reinterpret_cast<uint32_t *>(out) = *reinterpret_cast<const uint32_t *>(src);
            else
                for (int c = 0; c < 4; c++)
                    if (p + c >= lo && p + c < hi)
                        out[c] = src[c];
        }
        __syncthreads();
    }
}

// -------------------------------------------------------------------- read ----
template <typename E>
__device__ __forceinline__ void store8(E *p, const float (&x)[8])
{
    if constexpr (sizeof(E) == 4) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
        __stcs(reinterpret_cast<float4 *>(p + 16), make_float4(x[4], x[5], x[6], x[7]));
    } else {
        E e[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if constexpr (sizeof(E) == 2 && std::is_same<E, __half>::value)
                e[i] = __float2half_rn(x[i]);
            else
                e[i] = __float2bfloat16_rn(x[i]);
        }
        uint2 w[2];
        memcpy(w, e, sizeof(e));
        __stcs(reinterpret_cast<uint2 *>(p), w[0]);
        __stcs(reinterpret_cast<uint2 *>(p + 16), w[1]);
    }
}

template <int D, typename E>
__global__ void __launch_bounds__(kThreads) read_q4_kernel(const Args a)
{
    constexpr int kLanes = D / 8;
    pdl_launch_dependents();
    pdl_wait();
    const long long item = ((long long)blockIdx.x * kThreads + threadIdx.x) / kLanes;
    if (item >= (long long)a.T * a.Hkv)
        return;
    const int j = threadIdx.x % kLanes, blk = j >> 2, jj = j & 3;
    const int i = (int)(item / a.Hkv), h = (int)(item % a.Hkv);
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        bool bad;
        const int n = row_count(a, b, &bad);
        const long long p = (long long)a.start[b] + i;
        const bool there = p >= 0 && p < a.Tmax;
        if ((bad || (i < n && !there)) && a.status)
            atomicOr(a.status, kStatusPosition);
        if (i >= n || !there)
            continue;
        const size_t row = ((size_t)b * a.Hkv + h) * a.Tmax + (size_t)p;
        uint32_t w[2] = {0, 0};
        uint16_t sc[2] = {0, 0};
        if (a.r.k) {
            w[0] = *reinterpret_cast<const uint32_t *>(a.kc + row * (D / 2) + 16 * blk + 4 * jj);
            sc[0] = a.ks[row * (D / 32) + blk];
        }
        if (a.r.v) {
            w[1] = *reinterpret_cast<const uint32_t *>(a.vc + row * (D / 2) + 16 * blk + 4 * jj);
            sc[1] = a.vs[row * (D / 32) + blk];
        }
#pragma unroll
        for (int s = 0; s < 2; s++) {
            const Rows &r = a.r;
            if (!(s ? r.v : r.k))
                continue;
            E *dst = s ? static_cast<E *>(const_cast<void *>(r.v)) + b * r.v_batch + i * r.v_token + h * r.v_head
                       : static_cast<E *>(const_cast<void *>(r.k)) + b * r.k_batch + i * r.k_token + h * r.k_head;
            const float d = __half2float(__ushort_as_half(sc[s]));
            float x[8];
#pragma unroll
            for (int c = 0; c < 8; c++)
                x[c] = d * (float)((int)(w[s] >> (8 * (c & 3) + 4 * (c >> 2)) & 15) - 8);
            store8(dst + 32 * blk + 4 * jj, x);
        }
    }
}

template <typename E>
__global__ void __launch_bounds__(kThreads) read_q8_kernel(const Args a)
{
    constexpr int D = 128, kLanes = D / 8, kRowsPass = kThreads / kLanes, kLd = kTile + 4;
    __shared__ alignas(16) uint8_t vt[D * kLd];
    pdl_launch_dependents();
    pdl_wait();
    const int h = blockIdx.y;
    const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes, blk = lane >> 2, jj = lane & 3;
    for (int b = blockIdx.z; b < a.B; b += gridDim.z) {
        bool bad_count;
        const int n = row_count(a, b, &bad_count);
        const long long s0 = a.start[b];
        if (threadIdx.x == 0 && blockIdx.x == 0 && h == 0 && a.status &&
            (bad_count || (n > 0 && (s0 < 0 || s0 + n > a.Tmax))))
            atomicOr(a.status, kStatusPosition);
        const long long first = max(s0, 0LL), end = min(s0 + n, (long long)a.Tmax);
        const long long t0 = (first / kTile + blockIdx.x) * kTile;
        const int lo = (int)max(first - t0, 0LL), hi = (int)min(max(end - t0, 0LL), (long long)kTile);
        if (lo >= hi)
            continue;
        const size_t bh = (size_t)b * a.Hkv + h;
        if (a.r.v) {
            const uint8_t *src = a.vc + bh * D * a.Tmax + t0;     // the whole tile lies inside the plane
            for (int w = threadIdx.x; w < D * (kTile / 4); w += kThreads) {
                const int d = w / (kTile / 4), p = w % (kTile / 4) * 4;
                *reinterpret_cast<uint32_t *>(vt + d * kLd + p) =
                    *reinterpret_cast<const uint32_t *>(src + (size_t)d * a.Tmax + p);
            }
        }
        __syncthreads();
        for (int p = lo + sub; p < hi; p += kRowsPass) {
            const long long i = t0 + p - s0;
            const size_t row = bh * a.Tmax + (size_t)(t0 + p);
            const Rows &r = a.r;
            float x[8];
            if (r.k) {
                const uint32_t *src = reinterpret_cast<const uint32_t *>(a.kc + row * D + 32 * blk + 4 * jj);
                const uint32_t w[2] = {src[0], src[4]};
                const float d = __half2float(__ushort_as_half(a.ks[row * (D / 32) + blk]));
#pragma unroll
                for (int c = 0; c < 8; c++)
                    x[c] = d * (float)(int8_t)(w[c >> 2] >> (8 * (c & 3)));
                store8(static_cast<E *>(const_cast<void *>(r.k)) + b * r.k_batch + i * r.k_token + h * r.k_head + 32 * blk + 4 * jj, x);
            }
            if (r.v) {
                const float d = __half2float(__ushort_as_half(a.vs[row * (D / 32) + blk]));
#pragma unroll
                for (int c = 0; c < 8; c++)
                    x[c] = d * (float)(int8_t)vt[(32 * blk + 4 * jj + (c & 3) + 16 * (c >> 2)) * kLd + p];
                store8(static_cast<E *>(const_cast<void *>(r.v)) + b * r.v_batch + i * r.v_token + h * r.v_head + 32 * blk + 4 * jj, x);
            }
        }
        __syncthreads();
    }
}

// -------------------------------------------------------------------- host ----
enum Op { kAppend, kRead };

// Checks common to the four calls; fills everything of Args but the planes.
int32_t check_rows(Op op, const bq_kv_rows *rows, int32_t B, int32_t Hkv, int32_t D, int32_t Tmax,
                   const int32_t *start, const int32_t *count, int32_t *dev_status, Args *a)
{
    if (!rows || !start || (op == kAppend ? !rows->k || !rows->v : !rows->k && !rows->v))
        return BQ_ERR_NULL;
    if (Hkv < 1 || Hkv > 65535 || rows->T < 1 || rows->T > Tmax || rows->dtype < BQ_F32 || rows->dtype > BQ_BF16)
        return BQ_ERR_SHAPE;
    if (B < 1)
        return BQ_ERR_BATCH;
    if ((long long)B * Hkv >= (1LL << 31) || (long long)B * Hkv * Tmax >= (1LL << 31))
        return BQ_ERR_SHAPE;
    const int64_t per16 = rows->dtype == BQ_F32 ? 4 : 8;      // elements in 16 bytes
    if (rows->k && (!aligned16(rows->k) || rows->k_batch % per16 || rows->k_token % per16 || rows->k_head % per16))
        return BQ_ERR_ALIGN;
    if (rows->v && (!aligned16(rows->v) || rows->v_batch % per16 || rows->v_token % per16 || rows->v_head % per16))
        return BQ_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(start) | reinterpret_cast<uintptr_t>(count)) & 3u)
        return BQ_ERR_ALIGN;
    a->r = {rows->k, rows->v, rows->k_batch, rows->k_token, rows->k_head, rows->v_batch, rows->v_token, rows->v_head};
    a->start = start;
    a->count = count;
    a->status = dev_status;
    a->B = B;
    a->Hkv = Hkv;
    a->T = rows->T;
    a->Tmax = Tmax;
    return BQ_OK;
}

int32_t launch(const void *kernel, dim3 grid, const Args &a, void *stream)
{
    void *args[] = {const_cast<Args *>(&a)};
    return launch_pdl(kernel, grid, dim3(kThreads), 0, static_cast<cudaStream_t>(stream), args) == cudaSuccess
               ? BQ_OK
               : BQ_ERR_CUDA;
}

template <int D>
const void *q4_kernel(Op op, int32_t dtype)
{
    if (op == kAppend)
        return dtype == BQ_F32   ? (const void *)append_q4_kernel<D, float>
               : dtype == BQ_F16 ? (const void *)append_q4_kernel<D, __half>
                                 : (const void *)append_q4_kernel<D, __nv_bfloat16>;
    return dtype == BQ_F32   ? (const void *)read_q4_kernel<D, float>
           : dtype == BQ_F16 ? (const void *)read_q4_kernel<D, __half>
                             : (const void *)read_q4_kernel<D, __nv_bfloat16>;
}

int32_t run_q4(Op op, const bq_kv_cache_q4 *kv, const bq_kv_rows *rows, int32_t B, int32_t Hkv,
               const int32_t *start, const int32_t *count, int32_t *dev_status, void *stream)
{
    if (!kv || !kv->k_codes || !kv->k_scales || !kv->v_codes || !kv->v_scales)
        return BQ_ERR_NULL;
    if ((kv->D != 64 && kv->D != 128) || kv->Tmax < 32 || kv->Tmax % 32 != 0)
        return BQ_ERR_SHAPE;
    Args a;
    memset(&a, 0, sizeof(a));
    const int32_t st = check_rows(op, rows, B, Hkv, kv->D, kv->Tmax, start, count, dev_status, &a);
    if (st != BQ_OK)
        return st;
    if (!aligned16(kv->k_codes) || !aligned16(kv->k_scales) || !aligned16(kv->v_codes) || !aligned16(kv->v_scales))
        return BQ_ERR_ALIGN;
    a.kc = kv->k_codes;
    a.vc = kv->v_codes;
    a.ks = kv->k_scales;
    a.vs = kv->v_scales;
    // T * Hkv * D / 8 threads: at most 2^31 * 16 / 256 = 2^27 blocks
    const long long threads = (long long)a.T * Hkv * (kv->D / 8);
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads), (unsigned)(B < 65535 ? B : 65535));
    return launch(kv->D == 64 ? q4_kernel<64>(op, rows->dtype) : q4_kernel<128>(op, rows->dtype), grid, a, stream);
}

int32_t run_q8(Op op, const bq_kv_cache *kv, const bq_kv_rows *rows, int32_t B, int32_t Hkv,
               const int32_t *start, const int32_t *count, int32_t *dev_status, void *stream)
{
    if (!kv || !kv->k_codes || !kv->k_scales || !kv->vt_codes || !kv->v_scales)
        return BQ_ERR_NULL;
    if (kv->D != 128 || kv->Tmax < 128 || kv->Tmax % 128 != 0)
        return BQ_ERR_SHAPE;
    Args a;
    memset(&a, 0, sizeof(a));
    const int32_t st = check_rows(op, rows, B, Hkv, kv->D, kv->Tmax, start, count, dev_status, &a);
    if (st != BQ_OK)
        return st;
    if (!aligned16(kv->k_codes) || !aligned16(kv->k_scales) || !aligned16(kv->vt_codes) || !aligned16(kv->v_scales))
        return BQ_ERR_ALIGN;
    a.kc = reinterpret_cast<uint8_t *>(const_cast<int8_t *>(kv->k_codes));
    a.vc = reinterpret_cast<uint8_t *>(const_cast<int8_t *>(kv->vt_codes));
    a.ks = const_cast<uint16_t *>(kv->k_scales);
    a.vs = const_cast<uint16_t *>(kv->v_scales);
    // tiles that T positions can touch, wherever they start
    const dim3 grid((unsigned)((a.T + kTile - 2) / kTile + 1), (unsigned)Hkv, (unsigned)(B < 65535 ? B : 65535));
    const int32_t t = rows->dtype;
    const void *kernel = op == kAppend ? (t == BQ_F32   ? (const void *)append_q8_kernel<float>
                                          : t == BQ_F16 ? (const void *)append_q8_kernel<__half>
                                                        : (const void *)append_q8_kernel<__nv_bfloat16>)
                                       : (t == BQ_F32   ? (const void *)read_q8_kernel<float>
                                          : t == BQ_F16 ? (const void *)read_q8_kernel<__half>
                                                        : (const void *)read_q8_kernel<__nv_bfloat16>);
    return launch(kernel, grid, a, stream);
}

}  // namespace kvc
}  // namespace bq

using namespace bq;

extern "C" int32_t bq_kv_append_q4(const bq_kv_cache_q4 *kv, const bq_kv_rows *rows, int32_t B, int32_t Hkv,
                                   const int32_t *start, const int32_t *count, int32_t *dev_status, void *stream)
{
    return kvc::run_q4(kvc::kAppend, kv, rows, B, Hkv, start, count, dev_status, stream);
}

extern "C" int32_t bq_kv_append_q8(const bq_kv_cache *kv, const bq_kv_rows *rows, int32_t B, int32_t Hkv,
                                   const int32_t *start, const int32_t *count, int32_t *dev_status, void *stream)
{
    return kvc::run_q8(kvc::kAppend, kv, rows, B, Hkv, start, count, dev_status, stream);
}

extern "C" int32_t bq_kv_read_q4(const bq_kv_cache_q4 *kv, const bq_kv_rows *rows, int32_t B, int32_t Hkv,
                                 const int32_t *start, const int32_t *count, int32_t *dev_status, void *stream)
{
    return kvc::run_q4(kvc::kRead, kv, rows, B, Hkv, start, count, dev_status, stream);
}

extern "C" int32_t bq_kv_read_q8(const bq_kv_cache *kv, const bq_kv_rows *rows, int32_t B, int32_t Hkv,
                                 const int32_t *start, const int32_t *count, int32_t *dev_status, void *stream)
{
    return kvc::run_q8(kvc::kRead, kv, rows, B, Hkv, start, count, dev_status, stream);
}
