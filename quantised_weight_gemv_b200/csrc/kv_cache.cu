// kv_cache.cu -- writing new keys and values into a quantised KV cache and
// reading them back (Q4 and Q8), sm_100a.
//
// A row (one position of one KV head) is D elements in 32-element blocks:
//   a = max|x|,  d = fp16(a / L),  code = round-half-away(x / d) clamped,
// L = 7 (Q4) or 127 (Q8); value = d * code.  The bits are those of the host
// quantisers (bq_quantize_q4 / _q8), which the caches are defined by.
//
// Both directions are bound by memory, as long as an element takes few
// instructions: at 16-bit rows the SMs have about 14 a lane and element.
// Measured at 16384 tokens of 8 heads of 128 (copy peak 6.45 TB/s; 2 to 4 us of
// each are the launch's ends):
//   from or to fp32:   Q4 append 28.2 us (5.4 TB/s), read 27.1 (5.6);
//                      Q8 append 33.9 (5.0), read 29.2 (5.8)
//   fp16 or bf16:      Q4 append 18.0 (4.8), read 17.8 (4.8);
//                      Q8 append 22.1 (4.6), read 19.7 (5.2)
// and 1.6 to 2.7 us for a token of 8 x 8 rows, the time of a launch.  A
// thread moves 8 elements of a key row and the same 8 of the value row, four
// threads a block (its maximum takes two shuffles), so a row's threads read and
// write contiguous sectors, and four rows of one head, whose addresses are one
// stride apart.  A thread's elements are 4j .. 4j+3 and 16+4j .. 16+4j+3 of its
// block (j = 0..3): exactly the two nibbles of the Q4 bytes 4j .. 4j+3, one
// 32-bit word.  (16-bit rows of the Q8 cache: 8 consecutive elements.)
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

// Row i of sequence b is position p0 + i; rows lo .. hi-1 exist and lie in the
// cache.  Thread 0 of the first block reports what does not.
struct Span {
    long long p0;
    int lo, hi;
    __device__ __forceinline__ bool has(int i) const { return i >= lo && i < hi; }
};
__device__ __forceinline__ Span span_of(const Args &a, int b)
{
    const int given = a.count ? a.count[b] : a.T, n = min(max(given, 0), a.T);
    Span s;
    s.p0 = a.start[b];
    s.lo = (int)min(max(-s.p0, 0LL), (long long)n);
    s.hi = (int)min(max((long long)a.Tmax - s.p0, 0LL), (long long)n);
    if (threadIdx.x == 0 && blockIdx.x == 0 && a.status && (given != n || s.lo > 0 || s.hi < n))
        atomicOr(a.status, kStatusPosition);
    return s;
}

// ---------------------------------------------------------------- quantise ----
// A thread's 8 elements of a row, as they are in memory: 4 at p, 4 at p + GAP
// (16, or 4: consecutive).
template <typename E, int GAP>
struct Raw {
    uint32_t w[2][sizeof(E)];             // 16-bit: 2 words each; fp32: 4
    __device__ __forceinline__ void load(const E *p)
    {
        if constexpr (sizeof(E) == 4) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p)), b = __ldcs(reinterpret_cast<const uint4 *>(p + GAP));
            w[0][0] = a.x, w[0][1] = a.y, w[0][2] = a.z, w[0][3] = a.w;
            w[1][0] = b.x, w[1][1] = b.y, w[1][2] = b.z, w[1][3] = b.w;
        } else if constexpr (GAP == 4) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p));
            w[0][0] = a.x, w[0][1] = a.y, w[1][0] = a.z, w[1][1] = a.w;
        } else {
            const uint2 a = __ldcs(reinterpret_cast<const uint2 *>(p)), b = __ldcs(reinterpret_cast<const uint2 *>(p + GAP));
            w[0][0] = a.x, w[0][1] = a.y, w[1][0] = b.x, w[1][1] = b.y;
        }
    }
    // fp32 bits of the largest magnitude: finite < inf < NaN in all three types
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t m = 0;
        if constexpr (sizeof(E) == 4) {
#pragma unroll
            for (int i = 0; i < 8; i += 2)
                m = __vimax3_u32(m, w[i >> 2][i & 3] & 0x7fffffffu, w[i >> 2][(i & 3) + 1] & 0x7fffffffu);
            return m;
        } else {
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                m = __vimax3_u16x2(m, w[i >> 1][0] & 0x7fff7fffu, w[i >> 1][1] & 0x7fff7fffu);
            m = max(m & 0xffffu, m >> 16);
            if constexpr (std::is_same<E, __half>::value)
                return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
            else
                return m << 16;
        }
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(E) == 4) {
            return __uint_as_float(w[i >> 2][i & 3]);
        } else {
            const uint32_t v = w[i >> 2][(i >> 1) & 1];
            if constexpr (std::is_same<E, __half>::value)
                return __half2float(__ushort_as_half((unsigned short)(i & 1 ? v >> 16 : v & 0xffffu)));
            else
                return __uint_as_float(i & 1 ? v & 0xffff0000u : v << 16);
        }
    }
};

// Block scale and the thread's 8 codes as bytes, c[0] for elements 0-3 and c[1]
// for 4-7: Q4 codes 0..15, Q8 codes in two's complement.  The 4 threads of the
// block call it together (all 32 lanes of the warp execute it).  Returns false
// if the block is not finite or its scale overflows fp16: it is then zeros.
//
// The code is round-half-away(x / d), the quotient rounded to fp32 first.  d
// has 11 significant bits and a half h = k + 1/2 at most 8, so d h is exact in
// 19 bits; x - d h is a multiple of x's last place or is 0, hence no quotient
// rounds onto a half that it is not, and the code is that of the exact x / d.
//   16-bit x: where it is not 0, |x - d h| is at least 2^-19 |d h|.  t = x r, with
//     r = 1 / d to 2^-23 and then 1.5 * 2^-21 larger, lies past every half that
//     x / d reaches and short of every other: t rounded to nearest is the code.
//   fp32 x: t = x r is within |x / d| 2^-22 of x / d.  Unless it is that close to
//     a half (1 block in 10^4 at continuous values, Q4), it rounds as x / d does;
//     otherwise the sign of x - d h decides (one fma: exact).
// The scale of a 16-bit block takes no division either: a / L is at least 2^-15
// (Q4; Q8: 2^-19) of itself away from every midpoint of normal fp16 numbers, since
// a has at most 11 significant bits and L times the midpoint's 12 has more; only
// subnormal scales, which go the careful way, can lie on one (bf16 has three such
// a; all 2^15 magnitudes of both types were compared).
// |x / d| < L + 0.1 at a normal scale, so codes need no clamp, and adding
// 1.5 * 2^23 (+ 8) to t leaves the code in the low bits.  Subnormal scales take
// the careful way, with the clamp.
template <int FMT, typename E, int GAP>
__device__ __forceinline__ bool quantise8(const Raw<E, GAP> &raw, uint32_t (&c)[2], uint16_t &scale)
{
    constexpr float kLevels = FMT == 4 ? 7.0f : 127.0f;
    constexpr float kMagic = FMT == 4 ? 12582920.0f : 12582912.0f;
    constexpr float kSafe = FMT == 4 ? 0.5f - 0x1p-19f : 0.5f - 0x1p-15f;   // 7.1, 127.1 times 2^-22 at most
    uint32_t a = raw.top();
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    float d, r;
    auto set_scale = [&](float q) {
        const __half dh = __float2half_rn(q);
        scale = __half_as_ushort(dh);
        d = __half2float(dh);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    };
    set_scale(sizeof(E) == 2 ? __uint_as_float(a) * (1.0f / kLevels) : __fdiv_rn(__uint_as_float(a), kLevels));
    const float rb = sizeof(E) == 2 ? fmaf(r, 0x1.8p-21f, r) : r;
    bool careful = (uint16_t)(scale - 0x0400u) >= 0x7c00u - 0x0400u;   // 0, subnormal, inf, NaN
    uint32_t n[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float x = raw.get(i), s = fmaf(x, rb, kMagic);
        n[i] = __float_as_uint(s);
        if constexpr (sizeof(E) == 4)
            careful = careful || !(fabsf(fmaf(x, rb, kMagic - s)) < kSafe);
    }
    bool ok = true;
    if (careful) {
        if constexpr (sizeof(E) == 2)
            set_scale(__fdiv_rn(__uint_as_float(a), kLevels));
        ok = (scale & 0x7c00u) != 0x7c00u;
        if (!ok)
            scale = 0;
        const bool live = ok && d != 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float x = raw.get(i), m = fabsf(x), t = m * r, k = rintf(t);
            const float h = t < k ? k - 0.5f : k + 0.5f;                // the nearest half
            float q = fmaf(-d, h, m) >= 0.0f ? h + 0.5f : h - 0.5f;
            q = fminf(q, x < 0.0f ? (FMT == 4 ? 8.0f : 127.0f) : kLevels);
            n[i] = __float_as_uint((live ? copysignf(q, x) : 0.0f) + kMagic);
        }
    }
#pragma unroll
    for (int h = 0; h < 2; h++)
        c[h] = prmt(prmt(n[4 * h], n[4 * h + 1], 0x0040), prmt(n[4 * h + 2], n[4 * h + 3], 0x0040), 0x5410);
    return ok;
}

// A thread's place in a Q4 row: block and quarter of the block.
struct Lane {
    int row, blk, jj;
    template <int D>
    static __device__ __forceinline__ Lane of(int thread)
    {
        const int j = thread % (D / 8);
        return {thread / (D / 8), j >> 2, j & 3};
    }
    __device__ __forceinline__ int element() const { return 32 * blk + 4 * jj; }
};

// Blocks an SM that the appends' registers leave room for, beside the 16-byte
// loads in flight a thread: fp32 rows, 2 loads of which are a row's 8 elements, run
// more threads (16384 tokens, Q4 and Q8: 28.2 and 33.9 us; 4 blocks 28.8 and 34.4;
// 8 x 1300 tokens 10.3 and 12.4, 4 blocks 12.4 and 14.9), 16-bit rows all loads of
// four rows (18.0 and 22.1 us; two rows 18.9 and 23.6).
template <typename E>
constexpr int kBlocks = sizeof(E) == 4 ? 5 : 4;

// One block: a tile of tokens of one head, for every sequence in turn of
// gridDim.y.  blockDim / (D / 8) rows at a time, ROWS times: 4 where that leaves
// every SM two full blocks, else 1 (a decode step's few rows finish sooner side
// by side).  Warps past a sequence's last row read nothing, and what remains is
// their launch (64 sequences of T = 4096 fp32 rows, one with all and 63 with 1:
// 42 us; 313 where every row is read).
template <int D, typename E, int ROWS>
__global__ void __launch_bounds__(kThreads, kBlocks<E>) append_q4_kernel(const Args a)
{
    pdl_launch_dependents();
    pdl_wait();
    const Lane t = Lane::of<D>(threadIdx.x);
    const int at_once = blockDim.x / (D / 8), h = blockIdx.x % a.Hkv;
    const int i0 = (int)(blockIdx.x / a.Hkv) * (at_once * ROWS) + t.row;
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const Span w = span_of(a, b);
        if (!__any_sync(0xffffffffu, i0 < w.hi))
            continue;
        const size_t row0 = ((size_t)b * a.Hkv + h) * a.Tmax + (size_t)(w.p0 + i0);   // (used where i0 is in the span)
        uint8_t *kc = a.kc + row0 * (D / 2) + 16 * t.blk + 4 * t.jj, *vc = a.vc + row0 * (D / 2) + 16 * t.blk + 4 * t.jj;
        uint16_t *ks = a.ks + row0 * (D / 32) + t.blk, *vs = a.vs + row0 * (D / 32) + t.blk;
        // (past the last row an earlier one is read again and dropped: rows from the count on are not read)
        const E *kp = static_cast<const E *>(a.r.k) + b * a.r.k_batch + h * a.r.k_head + t.element() + min(i0, w.hi - 1) * a.r.k_token;
        const E *vp = static_cast<const E *>(a.r.v) + b * a.r.v_batch + h * a.r.v_head + t.element() + min(i0, w.hi - 1) * a.r.v_token;
        const int64_t k_step = at_once * a.r.k_token, v_step = at_once * a.r.v_token;
        bool fine = true;
        constexpr int U = ROWS == 1 || sizeof(E) == 4 ? 1 : 4;      // rows whose loads are in flight together
#pragma unroll 1
        for (int i = i0; i < i0 + ROWS * at_once; i += U * at_once) {
            if (U < ROWS && !__any_sync(0xffffffffu, i < w.hi))
                break;
            Raw<E, 16> x[U][2];
#pragma unroll
            for (int s = 0; s < U; s++) {
                x[s][0].load(kp);
                x[s][1].load(vp);
                if (i + (s + 1) * at_once < w.hi) {
                    kp += k_step;
                    vp += v_step;
                }
            }
#pragma unroll
            for (int s = 0; s < U; s++) {
                uint32_t c[2][2];
                uint16_t sc[2];
                const bool ok = quantise8<4>(x[s][0], c[0], sc[0]) & quantise8<4>(x[s][1], c[1], sc[1]);
                if (w.has(i + s * at_once)) {
                    // byte: element j low, element j + 16 high
                    *reinterpret_cast<uint32_t *>(kc) = c[0][0] | c[0][1] << 4;
                    *reinterpret_cast<uint32_t *>(vc) = c[1][0] | c[1][1] << 4;
                    if (t.jj == 0) {
                        *ks = sc[0];
                        *vs = sc[1];
                    }
                    fine = fine && ok;
                }
                kc += at_once * (D / 2);
                vc += at_once * (D / 2);
                ks += at_once * (D / 32);
                vs += at_once * (D / 32);
            }
        }
        if (!fine && a.status)
            atomicOr(a.status, kStatusRange);
    }
}

// What a tile of the Q8 kernels covers: positions t0 + lo .. t0 + hi - 1 (row =
// position - s0); nothing where lo >= hi.
struct Tile {
    long long s0, t0;
    int lo, hi;
};
__device__ __forceinline__ Tile tile_of(const Args &a, int b)
{
    const Span w = span_of(a, b);
    const long long first = w.p0 + w.lo, end = w.p0 + w.hi;
    Tile t;
    t.s0 = w.p0;
    t.t0 = (first / kTile + blockIdx.x / a.Hkv) * kTile;
    t.lo = w.lo < w.hi ? (int)max(first - t.t0, 0LL) : 0;
    t.hi = w.lo < w.hi ? (int)min(max(end - t.t0, 0LL), (long long)kTile) : 0;
    return t;
}
// The Q8 kernels' places in a row, for 16 threads j: elements first(j) .. + 3
// and first(j) + kGap .. + 3.  16-bit rows move 16 bytes at once; fp32 rows keep
// 4 threads' 16 bytes together (24 against 27 us with 32 bytes a thread, 8 x 4
// heads x 2.6k positions read).
template <typename E>
struct Place {
    static constexpr int kGap = sizeof(E) == 4 ? 16 : 4;
    static __device__ __forceinline__ int first(int j) { return kGap == 16 ? 32 * (j >> 2) + 4 * (j & 3) : 8 * j; }
    // Word w (positions 4w .. 4w+3) of transposed value row d in a tile of shared
    // memory: the words a warp stores or loads together lie in different banks.
    static __device__ __forceinline__ int word(int d, int w)
    {
        return d * (kTile / 4) + (w ^ (kGap == 16 ? ((d >> 5) << 2) | ((d >> 2) & 3) : d >> 3));
    }
};

// Key codes of a thread: 4 bytes at p, 4 at p + GAP.
template <int GAP>
__device__ __forceinline__ void store_codes(uint8_t *p, uint32_t lo, uint32_t hi)
{
    if constexpr (GAP == 4) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
    } else {
        *reinterpret_cast<uint32_t *>(p) = lo;
        *reinterpret_cast<uint32_t *>(p + GAP) = hi;
    }
}
template <int GAP>
__device__ __forceinline__ uint2 load_codes(const uint8_t *p)
{
    if constexpr (GAP == 4)
        return __ldcs(reinterpret_cast<const uint2 *>(p));
    else
        return make_uint2(__ldcs(reinterpret_cast<const uint32_t *>(p)), __ldcs(reinterpret_cast<const uint32_t *>(p + GAP)));
}

// One block: 64 positions (a tile cut at a multiple of 64) of one (sequence,
// head).  Keys go straight to their rows; a thread takes 4 consecutive
// positions, whose codes of one element are one word of the value tile.  Up to
// 16 positions (a decode step) take one position a thread and store value bytes
// where they belong: 2.6 us for a token of 8 x 8 rows, where the tile took 1.7
// more.
template <typename E>
__global__ void __launch_bounds__(kThreads, kBlocks<E>) append_q8_kernel(const Args a)
{
    constexpr int D = 128, kLanes = D / 8, kGap = Place<E>::kGap;
    __shared__ alignas(16) uint32_t vt[D * kTile / 4];
    pdl_launch_dependents();
    pdl_wait();
    const int h = blockIdx.x % a.Hkv, row = threadIdx.x / kLanes, j = threadIdx.x % kLanes;
    const int e0 = Place<E>::first(j);
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const Tile t = tile_of(a, b);
        if (t.lo >= t.hi)
            continue;                                 // (the same for the whole block)
        const size_t bh = (size_t)b * a.Hkv + h;
        const bool few = t.hi - t.lo <= kThreads / kLanes;
        const int p0 = few ? t.lo + row : 4 * row;    // the thread's first position
        // (positions outside the span are read from its nearer end and dropped)
        const long long i = t.t0 + min(max(p0, t.lo), t.hi - 1) - t.s0;
        const E *kp = static_cast<const E *>(a.r.k) + b * a.r.k_batch + h * a.r.k_head + i * a.r.k_token + e0;
        const E *vp = static_cast<const E *>(a.r.v) + b * a.r.v_batch + h * a.r.v_head + i * a.r.v_token + e0;
        const size_t at = bh * a.Tmax + (size_t)(t.t0 + p0);
        uint8_t *kc = a.kc + at * D + e0;
        uint16_t *ks = a.ks + at * (D / 32) + j / 4, *vs = a.vs + at * (D / 32) + j / 4;
        int bits = 0;
        if (few) {
            Raw<E, kGap> x[2];
            x[0].load(kp);
            x[1].load(vp);
            uint32_t c[2][2];
            uint16_t sc[2];
            const bool ok = quantise8<8>(x[0], c[0], sc[0]) & quantise8<8>(x[1], c[1], sc[1]);
            if (p0 < t.hi) {
                store_codes<kGap>(kc, c[0][0], c[0][1]);
                uint8_t *out = a.vc + (bh * D + e0) * a.Tmax + (size_t)(t.t0 + p0);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    out[(size_t)(e + (e >> 2) * (kGap - 4)) * a.Tmax] = (uint8_t)(c[1][e >> 2] >> (8 * (e & 3)));
                if (j % 4 == 0) {
                    *ks = sc[0];
                    *vs = sc[1];
                }
                if (!ok && a.status)
                    atomicOr(a.status, kStatusRange);
            }
            continue;
        }
        uint32_t vc[4][2];
        if ((threadIdx.x / 32 + 1) * 8 > t.lo && threadIdx.x / 32 * 8 < t.hi) {   // the warp has a position
            constexpr int U = sizeof(E) == 4 ? 1 : 4;
#pragma unroll
            for (int s0 = 0; s0 < 4; s0 += U) {
                Raw<E, kGap> x[U][2];
#pragma unroll
                for (int s = s0; s < s0 + U; s++) {
                    x[s - s0][0].load(kp);
                    x[s - s0][1].load(vp);
                    if (p0 + s >= t.lo && p0 + s + 1 < t.hi) {
                        kp += a.r.k_token;
                        vp += a.r.v_token;
                    }
                }
#pragma unroll
                for (int s = s0; s < s0 + U; s++) {
                    uint32_t c[2];
                    uint16_t sc[2];
                    const bool ok = quantise8<8>(x[s - s0][0], c, sc[0]) & quantise8<8>(x[s - s0][1], vc[s], sc[1]);
                    if (p0 + s >= t.lo && p0 + s < t.hi) {
                        store_codes<kGap>(kc + s * D, c[0], c[1]);
                        if (j % 4 == 0) {
                            ks[s * (D / 32)] = sc[0];
                            vs[s * (D / 32)] = sc[1];
                        }
                        bits |= ok ? 0 : kStatusRange;
                    }
                }
            }
            // element e of the 4 positions: a 4 x 4 byte transpose of each half
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
                const uint32_t x01 = prmt(vc[0][hf], vc[1][hf], 0x5140), y01 = prmt(vc[2][hf], vc[3][hf], 0x5140);
                const uint32_t x23 = prmt(vc[0][hf], vc[1][hf], 0x7362), y23 = prmt(vc[2][hf], vc[3][hf], 0x7362);
                const int d = e0 + kGap * hf;
                vt[Place<E>::word(d, row)] = prmt(x01, y01, 0x5410);
                vt[Place<E>::word(d + 1, row)] = prmt(x01, y01, 0x7632);
                vt[Place<E>::word(d + 2, row)] = prmt(x23, y23, 0x5410);
                vt[Place<E>::word(d + 3, row)] = prmt(x23, y23, 0x7632);
            }
        }
        if (bits && a.status)
            atomicOr(a.status, bits);
        __syncthreads();
        uint8_t *dst = a.vc + bh * D * a.Tmax + t.t0;
#pragma unroll
        for (int k = 0; k < D * kTile / 4 / kThreads; k++) {
            const int w = threadIdx.x + k * kThreads, d = w / (kTile / 4), p = w % (kTile / 4) * 4;
            if (p + 4 <= t.lo || p >= t.hi)
                continue;
            uint8_t *out = dst + (size_t)d * a.Tmax + p;
            const uint32_t v = vt[Place<E>::word(d, p / 4)];
            if (p >= t.lo && p + 4 <= t.hi)
                *reinterpret_cast<uint32_t *>(out) = v;
            else
                for (int c = 0; c < 4; c++)
                    if (p + c >= t.lo && p + c < t.hi)
                        out[c] = (uint8_t)(v >> (8 * c));
        }
        __syncthreads();
    }
}

// -------------------------------------------------------------------- read ----
// 8 values d * code to a row: x[0..3] at p, x[4..7] at p + GAP; d * code is exact
// in fp32 and rounded once.
template <int GAP, typename E>
__device__ __forceinline__ void store8(E *p, float d, const float (&x)[8])
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float lo = d * x[i], hi = d * x[i + 1];
        if constexpr (sizeof(E) == 4) {
            w[i] = __float_as_uint(lo);
            w[i + 1] = __float_as_uint(hi);
        } else if constexpr (std::is_same<E, __half>::value) {
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i / 2]) : "f"(hi), "f"(lo));
        } else {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i / 2]) : "f"(hi), "f"(lo));
        }
    }
    if constexpr (sizeof(E) == 4) {
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
        __stcs(reinterpret_cast<uint4 *>(p + GAP), make_uint4(w[4], w[5], w[6], w[7]));
    } else if constexpr (GAP == 4) {
        __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
    } else {
        __stcs(reinterpret_cast<uint2 *>(p), make_uint2(w[0], w[1]));
        __stcs(reinterpret_cast<uint2 *>(p + GAP), make_uint2(w[2], w[3]));
    }
}
// Codes to fp32: 2^23 + u has u in its low bits.
__device__ __forceinline__ void codes_q4(uint32_t w, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        x[i] = __uint_as_float(0x4b000000u | ((w >> (8 * i)) & 15u)) - 8388616.0f;
        x[i + 4] = __uint_as_float(0x4b000000u | ((w >> (8 * i + 4)) & 15u)) - 8388616.0f;
    }
}
__device__ __forceinline__ void codes_q8(uint32_t lo, uint32_t hi, float (&x)[8])
{
    lo ^= 0x80808080u, hi ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        x[i] = __uint_as_float(prmt(lo, 0x4b000000u, 0x7440 + i)) - 8388736.0f;
        x[i + 4] = __uint_as_float(prmt(hi, 0x4b000000u, 0x7440 + i)) - 8388736.0f;
    }
}
__device__ __forceinline__ float f16(uint16_t s) { return __half2float(__ushort_as_half(s)); }

template <int D, typename E, int ROWS>
__global__ void __launch_bounds__(kThreads) read_q4_kernel(const Args a)
{
    pdl_launch_dependents();
    pdl_wait();
    const Lane t = Lane::of<D>(threadIdx.x);
    const int at_once = blockDim.x / (D / 8), h = blockIdx.x % a.Hkv;
    const int i0 = (int)(blockIdx.x / a.Hkv) * (at_once * ROWS) + t.row;
    const Rows &r = a.r;
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const Span w = span_of(a, b);
        const size_t row0 = ((size_t)b * a.Hkv + h) * a.Tmax + (size_t)(w.p0 + i0);   // (used where i0 is in the span)
        const uint8_t *kc = a.kc + row0 * (D / 2) + 16 * t.blk + 4 * t.jj, *vc = a.vc + row0 * (D / 2) + 16 * t.blk + 4 * t.jj;
        const uint16_t *ks = a.ks + row0 * (D / 32) + t.blk, *vs = a.vs + row0 * (D / 32) + t.blk;
        E *kp = static_cast<E *>(const_cast<void *>(r.k)) + b * r.k_batch + h * r.k_head + t.element() + i0 * r.k_token;
        E *vp = static_cast<E *>(const_cast<void *>(r.v)) + b * r.v_batch + h * r.v_head + t.element() + i0 * r.v_token;
        uint32_t c[ROWS][2];
        uint16_t sc[ROWS][2];
#pragma unroll
        for (int s = 0; s < ROWS; s++)
            if (w.has(i0 + s * at_once)) {
                if (r.k) {
                    c[s][0] = __ldcs(reinterpret_cast<const uint32_t *>(kc + s * at_once * (D / 2)));
                    sc[s][0] = __ldcs(ks + s * at_once * (D / 32));
                }
                if (r.v) {
                    c[s][1] = __ldcs(reinterpret_cast<const uint32_t *>(vc + s * at_once * (D / 2)));
                    sc[s][1] = __ldcs(vs + s * at_once * (D / 32));
                }
            }
#pragma unroll
        for (int s = 0; s < ROWS; s++) {
            float x[8];
            if (w.has(i0 + s * at_once)) {
                if (r.k) {
                    codes_q4(c[s][0], x);
                    store8<16>(kp + s * at_once * r.k_token, f16(sc[s][0]), x);
                }
                if (r.v) {
                    codes_q4(c[s][1], x);
                    store8<16>(vp + s * at_once * r.v_token, f16(sc[s][1]), x);
                }
            }
        }
    }
}

template <typename E>
__global__ void __launch_bounds__(kThreads, 4) read_q8_kernel(const Args a)
{
    constexpr int D = 128, kLanes = D / 8, kGap = Place<E>::kGap;
    __shared__ alignas(16) uint32_t vt[D * kTile / 4];
    pdl_launch_dependents();
    pdl_wait();
    const int h = blockIdx.x % a.Hkv, row = threadIdx.x / kLanes, j = threadIdx.x % kLanes;
    const int e0 = Place<E>::first(j);
    const Rows &r = a.r;
    for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
        const Tile t = tile_of(a, b);
        if (t.lo >= t.hi)
            continue;
        const size_t bh = (size_t)b * a.Hkv + h;
        const bool few = t.hi - t.lo <= kThreads / kLanes;   // a position a thread (see append)
        const int p0 = few ? t.lo + row : 4 * row;
        const size_t at = bh * a.Tmax + (size_t)(t.t0 + p0);
        const uint8_t *kc = a.kc + at * D + e0;
        const uint16_t *ks = a.ks + at * (D / 32) + j / 4, *vs = a.vs + at * (D / 32) + j / 4;
        const long long i = t.t0 + p0 - t.s0;         // (used where p0 .. are in the span)
        E *kp = static_cast<E *>(const_cast<void *>(r.k)) + b * r.k_batch + h * r.k_head + i * r.k_token + e0;
        E *vp = static_cast<E *>(const_cast<void *>(r.v)) + b * r.v_batch + h * r.v_head + i * r.v_token + e0;
        float x[8];
        if (few) {
            if (p0 >= t.hi)
                continue;
            if (r.k) {
                const uint2 w = load_codes<kGap>(kc);
                codes_q8(w.x, w.y, x);
                store8<kGap>(kp, f16(*ks), x);
            }
            if (r.v) {
                const int8_t *src = reinterpret_cast<const int8_t *>(a.vc) + (bh * D + e0) * a.Tmax + (size_t)(t.t0 + p0);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    x[e] = (float)src[(size_t)(e + (e >> 2) * (kGap - 4)) * a.Tmax];
                store8<kGap>(vp, f16(*vs), x);
            }
            continue;
        }
        uint2 kw[4];
        uint16_t sc[4][2];
#pragma unroll
        for (int s = 0; s < 4; s++)
            if (p0 + s >= t.lo && p0 + s < t.hi) {
                if (r.k) {
                    kw[s] = load_codes<kGap>(kc + s * D);
                    sc[s][0] = __ldcs(ks + s * (D / 32));
                }
                if (r.v)
                    sc[s][1] = __ldcs(vs + s * (D / 32));
            }
        if (r.v) {
            const uint8_t *src = a.vc + bh * D * a.Tmax + t.t0;   // the whole tile lies inside the plane
#pragma unroll
            for (int k = 0; k < D * kTile / 4 / kThreads; k++) {
                const int w = threadIdx.x + k * kThreads, d = w / (kTile / 4), q = w % (kTile / 4);
                if (4 * q + 4 > t.lo && 4 * q < t.hi)
                    vt[Place<E>::word(d, q)] = __ldcs(reinterpret_cast<const uint32_t *>(src + (size_t)d * a.Tmax + 4 * q));
            }
            __syncthreads();
        }
        if (r.k)
#pragma unroll
            for (int s = 0; s < 4; s++)
                if (p0 + s >= t.lo && p0 + s < t.hi) {
                    codes_q8(kw[s].x, kw[s].y, x);
                    store8<kGap>(kp + s * r.k_token, f16(sc[s][0]), x);
                }
        if (r.v) {
            uint32_t vc[4][2];
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
                const int d = e0 + kGap * hf;
                const uint32_t e0 = vt[Place<E>::word(d, row)], e1 = vt[Place<E>::word(d + 1, row)];
                const uint32_t e2 = vt[Place<E>::word(d + 2, row)], e3 = vt[Place<E>::word(d + 3, row)];
                const uint32_t x01 = prmt(e0, e1, 0x5140), y01 = prmt(e2, e3, 0x5140);
                const uint32_t x23 = prmt(e0, e1, 0x7362), y23 = prmt(e2, e3, 0x7362);
                vc[0][hf] = prmt(x01, y01, 0x5410);
                vc[1][hf] = prmt(x01, y01, 0x7632);
                vc[2][hf] = prmt(x23, y23, 0x5410);
                vc[3][hf] = prmt(x23, y23, 0x7632);
            }
#pragma unroll
            for (int s = 0; s < 4; s++)
                if (p0 + s >= t.lo && p0 + s < t.hi) {
                    codes_q8(vc[s][0], vc[s][1], x);
                    store8<kGap>(vp + s * r.v_token, f16(sc[s][1]), x);
                }
            __syncthreads();
        }
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
    // (row numbers of whole blocks stay below 2^31)
    if (Hkv < 1 || Hkv > 65535 || rows->T < 1 || rows->T > Tmax || rows->T > (1 << 30) || rows->dtype < BQ_F32 || rows->dtype > BQ_BF16)
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

int32_t launch(const void *kernel, dim3 grid, int threads, const Args &a, void *stream)
{
    void *args[] = {const_cast<Args *>(&a)};
    return launch_pdl(kernel, grid, dim3((unsigned)threads), 0, static_cast<cudaStream_t>(stream), args) == cudaSuccess
               ? BQ_OK
               : BQ_ERR_CUDA;
}

template <int D, int ROWS>
const void *q4_kernel(Op op, int32_t dtype)
{
    if (op == kAppend)
        return dtype == BQ_F32   ? (const void *)append_q4_kernel<D, float, ROWS>
               : dtype == BQ_F16 ? (const void *)append_q4_kernel<D, __half, ROWS>
                                 : (const void *)append_q4_kernel<D, __nv_bfloat16, ROWS>;
    return dtype == BQ_F32   ? (const void *)read_q4_kernel<D, float, ROWS>
           : dtype == BQ_F16 ? (const void *)read_q4_kernel<D, __half, ROWS>
                             : (const void *)read_q4_kernel<D, __nv_bfloat16, ROWS>;
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
    if (op == kRead && rows->k == rows->v)                // (two writers of the same rows)
        return BQ_ERR_SHAPE;
    a.kc = kv->k_codes;
    a.vc = kv->v_codes;
    a.ks = kv->k_scales;
    a.vs = kv->v_scales;
    const int sms = device_sm_count(), lanes = kv->D / 8;
    if (sms <= 0)
        return BQ_ERR_CUDA;
    const bool many = (long long)B * Hkv * a.T >= 2LL * sms * (kThreads / lanes * 4);
    const int rows_thread = many ? 4 : 1;
    // (a few tokens need no 256 threads)
    const long long want = ((long long)a.T * lanes / rows_thread + 31) / 32 * 32;
    const int threads = want < kThreads ? (want < 32 ? 32 : (int)want) : kThreads;
    const long long tile = (long long)(threads / lanes) * rows_thread;
    const long long blocks = (a.T + tile - 1) / tile * Hkv;         // < 2^31: T * Hkv is
    const dim3 grid((unsigned)blocks, (unsigned)(B < 65535 ? B : 65535));
    const void *kernel = kv->D == 64 ? (many ? q4_kernel<64, 4>(op, rows->dtype) : q4_kernel<64, 1>(op, rows->dtype))
                                     : (many ? q4_kernel<128, 4>(op, rows->dtype) : q4_kernel<128, 1>(op, rows->dtype));
    return launch(kernel, grid, threads, a, stream);
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
    if (op == kRead && rows->k == rows->v)
        return BQ_ERR_SHAPE;
    a.kc = reinterpret_cast<uint8_t *>(const_cast<int8_t *>(kv->k_codes));
    a.vc = reinterpret_cast<uint8_t *>(const_cast<int8_t *>(kv->vt_codes));
    a.ks = const_cast<uint16_t *>(kv->k_scales);
    a.vs = const_cast<uint16_t *>(kv->v_scales);
    // tiles that T positions can touch, wherever they start
    const long long tiles = ((long long)a.T + kTile - 2) / kTile + 1;
    if (tiles * Hkv >= (1LL << 31))
        return BQ_ERR_SHAPE;
    const dim3 grid((unsigned)(tiles * Hkv), (unsigned)(B < 65535 ? B : 65535));
    const int32_t t = rows->dtype;
    const void *kernel = op == kAppend ? (t == BQ_F32   ? (const void *)append_q8_kernel<float>
                                          : t == BQ_F16 ? (const void *)append_q8_kernel<__half>
                                                        : (const void *)append_q8_kernel<__nv_bfloat16>)
                                       : (t == BQ_F32   ? (const void *)read_q8_kernel<float>
                                          : t == BQ_F16 ? (const void *)read_q8_kernel<__half>
                                                        : (const void *)read_q8_kernel<__nv_bfloat16>);
    return launch(kernel, grid, kThreads, a, stream);
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
