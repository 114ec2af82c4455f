// attention_q4.cu -- decode attention over a 4-bit KV cache, sm_100a.
//
//   s_t = scale * q . K[t]   p = softmax(s over t < lens[b] - (Tq - 1 - i))   o = sum_t p_t V[t]
//
// Bound: a position of one KV head is 144 bytes (D = 128), read once for its
// R = Tq * G query rows: 4 D R / 144 flops a byte, so HBM up to about 16 rows;
// what stands against it is the number of instructions that unpack 256 codes.
// Measured in a chain of launches (D = 128, 8 KV heads, 5 query heads each): 8
// sequences of 32768 positions 75.5 us, 4.0 TB/s, bound by instructions (719 a
// unit of 32 positions; the copies alone 58 us); one of 32768 20 us; one of 4096
// 10 us, nearly all ends (plan, first loads, merges).  A launch by itself takes
// up to 6 us more, its start and end.  40 rows (8 query tokens) at 8 x 3k
// positions on average: 43 us.
//
// Work: a unit is 32 positions of one (sequence, KV head).  The valid units of
// all sequences form one line (lens are on the device: one warp of every CTA
// makes the plan, the others meanwhile clear the outputs of empty sequences).  A
// segment, one (sequence, KV head), gets CTAs of its own where that fits the
// grid; else CTAs take equal consecutive shares of the line (see make_plan).  A
// CTA's warps take equal consecutive shares of the CTA's.  Ragged lengths
// therefore cost no balance, and a sequence that ends inside a share just
// starts the next one: a warp never waits for another before its line ends.
// A warp streams its units through a ring of its own in shared memory with
// 16-byte cp.async, laid down in a swizzle that keeps ldmatrix free of bank
// conflicts; no barrier, and nothing that could wait for ever.  (Copies by TMA,
// a box of 32 rows of 64 bytes at a time, made 8 x 32768 81 us where these made
// it 69.)
//
// Softmax: one pass with a running maximum m a row; a warp's result of a
// segment (the part of a sequence's head in its share) is (m, l, O).  A whole
// segment is written out directly.  The two that may continue in a neighbour
// are merged at the end: warps through shared memory, CTAs through the
// workspace, where the last CTA to arrive merges in CTA order (deterministic).
//
// Tensor cores (mma.sync m16n8k16), fp32 accumulation, codes exact.  (Not
// tcgen05: positions, or head elements, would fill its 128 rows, but value scales
// differ by position and block, and 16 MMAs of 70 to 130 cycles each for 128
// positions are no less than the 1200 cycles that these take at up to 8 rows.)
//   scores  S^T[t][row]: A = key codes u - 8 (exact fp16: (0x6400 | u) - 1032),
//     B = q.  Positions fill the 16-row side, so no operand is padded.  Each
//     block's sum is scaled by dK in fp32.  q is multiplied by a power of two a
//     row first, so that subnormal queries are exact too.  (Signed codes: with
//     unsigned ones the zero point's cancellation would be the largest error.)
//   values  O^T[d][row]: A = value codes u - 8, signed so that sums over
//     thousands of positions do not cancel against a zero-point sum, B = p dV as
//     two fp16 terms, whatever the output's type: one term would round every
//     weight as coarsely as a 16-bit output is rounded, 1.4 times the error of
//     the output's own rounding (8 x 32768 positions: 2.9e-4 of the result instead
//     of 2.1e-4, in 61 us and not 75).  ldmatrix.trans on 16-bit units turns
//     position-major rows into pairs of positions per register.
//   p dV reaches B's layout by one movmatrix a tile and never leaves registers.
// Exponents: p = 2^((s - m) scale log2(e)) with s and m still unscaled sums, so
// that scores of any size keep their differences (a scaled maximum of 2^28 would
// be rounded by 32, and weights by 2^32).  m moves only when a score outgrows it
// by 2^4.  p dV must neither overflow fp16 nor go subnormal where it counts: the
// value scales are taken times 2^(25 - e), e the largest of their exponent bits so
// far, so that p dV < 2^15.  Both are exact: O and l scale by powers of two alone.
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <cstring>

#include "bq_device.cuh"
#include "bq_internal.h"
#include "bq_kv.h"

namespace bq {
namespace aq {

constexpr int kUnit = 32;                 // positions per unit
constexpr int kMaxGrid = 160;             // CTAs (one per SM)
constexpr int kMinUnits[2] = {4, 8};      // units per CTA of 16 or 8 warps, where there are few,
constexpr int kWhole = 12;                // and units up to which segments are whole then (see make_plan)
constexpr int kSnap = 32;                 // segments up to this length are never cut between CTAs (see below)
constexpr int kEdge = 1;                  // units that a segment's start counts for when the line is cut
constexpr float kFloor = -5.0e37f;        // a maximum no score has reached (times 4 finite; times any scale a long way down)
constexpr float kAllInf = -1.0e20f;       // in partials: every score seen is -inf (above each kFloor, below any score)
constexpr float kSlack = 4.0f;
constexpr int kBase = 25;                 // scales enter times 2^(25 - exponent bits): below 2^11
constexpr float kScaleMin = 1.0e-28f;     // softmax scales below leave every score below 2^-49

// D: head width; NT: 8-row tiles per warp (1 or 2: see tiles_of).
template <int D, int NT>
struct Cfg {
    static constexpr int kNB = D / 32;                        // blocks per row
    static constexpr int kWarps = NT == 1 ? 16 : 8;           // 128 / 255 registers a thread
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kSlots = NT == 1 ? 2 : 3;
    static constexpr int kRows = 8 * NT;                      // rows per warp
    static constexpr int kCodes = kUnit * D / 2, kScales = kUnit * kNB * 2;
    static constexpr int kSlotBytes = 2 * (kCodes + kScales);
    static constexpr int kRing = kSlots * kSlotBytes;         // per warp
    static constexpr int kLd = D;                             // floats per row of a partial in shared memory
    static constexpr int kConv = 2 * kUnit * kNB * 4;         // a unit's scales in fp32 (keys, values)
    static constexpr int kPart = kRows * kLd + 2 * kRows;     // floats: O, m, l
    static constexpr int kWarpBytes = kRing + kConv;          // (a multiple of 128); the warps' first partials follow
    static constexpr size_t kSmem = 128 + (size_t)kWarps * (kWarpBytes + kPart * 4);
    static_assert(kPart * 4 <= kRing, "a warp's last partial fits its drained ring");
    static_assert(kSlotBytes % 128 == 0 && kPart % 4 == 0, "slots and partials keep their alignment");
    static_assert(kSmem <= 227 * 1024 - 1024, "shared memory of an SM");
    static constexpr int kRoom = kWarps * (kWarpBytes + kPart * 4) / 4 / (D + 2);   // rows of CTA partials that fit there
    static_assert(kRoom >= 2 * kMaxGrid, "two rows of every CTA's partial");
};

struct Args {
    const uint8_t *kc, *vc;
    const uint16_t *ks, *vs, *q;
    const int32_t *lens;
    void *o;
    int B, Tq, Hkv, G, Tmax;
    int R;                                // Tq * G query rows per KV head
    int passes;                           // of 8 NT rows each
    float scale2;                         // scale * log2(e), kScaleMin at least
    int *counters;                        // [grid], by a shared segment's first CTA
    float *partials;                      // [grid][2]: O [rows][D], then (m, l) [rows]
};

struct Entry {                            // a shared segment's part, for the merges
    int b, hp, first, units;              // sequence (-1: none), head * passes + pass, first unit on the line, units
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 operations in one instruction: x = x a + c, a b, x a, x + y, x - y.
__device__ __forceinline__ void fma2(float (&x)[2], float a0, float a1, float c0, float c1)
{
    asm("{.reg .b64 u, v, w;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tmov.b64 w, {%4, %5};\n\t"
        "fma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;}"
        : "+f"(x[0]), "+f"(x[1]) : "f"(a0), "f"(a1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float (&x)[2], float a0, float a1, float b)
{
    asm("{.reg .b64 u, v;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %4};\n\tmul.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;}"
        : "=f"(x[0]), "=f"(x[1]) : "f"(a0), "f"(a1), "f"(b));
}
#define BQ_F32X2(name, op)                                                                                             \
    __device__ __forceinline__ void name(float (&x)[2], const float (&y)[2])                                           \
    {                                                                                                                  \
        asm("{.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t" op ".rn.f32x2 u, u, v;\n\t"         \
            "mov.b64 {%0, %1}, u;}" : "+f"(x[0]), "+f"(x[1]) : "f"(y[0]), "f"(y[1]));                                  \
    }
BQ_F32X2(mul2, "mul")
BQ_F32X2(add2, "add")
BQ_F32X2(sub2, "sub")
#undef BQ_F32X2
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float f16_lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))); }
__device__ __forceinline__ float f16_hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }   // -126 <= e <= 127
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// A position's fp32 scales.
template <int NB>
__device__ __forceinline__ void row_scales(float (&d)[NB], uint32_t addr)
{
    if constexpr (NB == 4)
        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(d[0]), "=f"(d[1]) : "r"(addr) : "memory");
}
// Scales of a position in fp16, or zeros (not live); the bits of the largest magnitude.
template <int NB>
__device__ __forceinline__ uint32_t load_scales(uint32_t (&w)[NB / 2], uint32_t src, bool live)
{
    if constexpr (NB == 4)
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(src) : "memory");
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(src) : "memory");
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < NB / 2; i++) {
        w[i] = live ? w[i] : 0u;
        mx = __vmaxu2(mx, w[i] & 0x7fff7fffu);
    }
    return max(mx & 0xffffu, mx >> 16);
}
// The same in fp32 times f.
template <int NB>
__device__ __forceinline__ void store_scales(uint32_t dst, const uint32_t (&w)[NB / 2], float f)
{
    if constexpr (NB == 4)
        asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "f"(f16_lo(w[0]) * f), "f"(f16_hi(w[0]) * f), "f"(f16_lo(w[1]) * f), "f"(f16_hi(w[1]) * f) : "memory");
    else
        asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(dst), "f"(f16_lo(w[0]) * f), "f"(f16_hi(w[0]) * f) : "memory");
}
// 16 bytes to shared memory, past L1.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x)      // an 8 x 8 tile of 16-bit elements over the warp
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// Byte offset of 16-byte chunk `chunk` (block) of position `row` in a unit: the
// chunks of 8 consecutive positions fall into all 32 banks.
template <int D>
__device__ __forceinline__ uint32_t swizzled(int row, int chunk)
{
    return D == 128 ? row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4) : row * 32 + ((chunk ^ ((row >> 2) & 1)) << 4);
}
// Four fp16 pairs u - 8 from a 16-bit unit of two positions: nibble k of each half.
__device__ __forceinline__ uint32_t nib_lo(uint32_t x)
{
    uint32_t h;
    asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(h) : "r"(x));        // (x & m) | 1024
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(h) : "r"(h), "r"(0xE408E408u));           // - 1032
    return h;
}
__device__ __forceinline__ uint32_t nib_hi(uint32_t x)
{
    uint32_t h;
    asm("lop3.b32 %0, %1, 0x00F000F0, 0x64006400, 0xEA;" : "=r"(h) : "r"(x));        // 1024 + 16 u
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h) : "r"(h), "r"(0x2C002C00u), "r"(0xD480D480u));   // / 16 - 72
    return h;
}

// Units shared by CTAs: q each, one more for the first r.
struct Shares {
    int q, r;
    __device__ __forceinline__ int start(int c) const { return c * q + min(c, r); }
    __device__ __forceinline__ int owner(int x) const
    {
        const int big = r * (q + 1);
        return x < big ? x / (q + 1) : r + (x - big) / q;
    }
};

template <typename O>
__device__ __forceinline__ void store2(O *p, float a, float b)
{
    if constexpr (sizeof(O) == 4)
        *reinterpret_cast<float2 *>(p) = make_float2(a, b);
    else
        *reinterpret_cast<uint32_t *>(p) = pack_f16x2(a, b);
}

template <typename O>
__device__ __forceinline__ void store4(O *p, const float4 &v, float f)
{
    if constexpr (sizeof(O) == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    else
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_f16x2(v.x * f, v.y * f), pack_f16x2(v.z * f, v.w * f));
}

// A place on the line of units: unit t of nu of (sequence b, head-pass hp).
struct Cursor {
    int b, hp, t, nu;
};

// A CTA's share of the line, made by its first warp.
struct Plan {
    int n_act;                            // CTAs with work
    int split;                            // 1: the CTA's segment has CTAs of its own, cf .. cl
    int edge;                             // units a segment's start counts for on the line (see make_plan)
    int r0, r1, cf, cl;                   // its units (split: counted from the segment's start)
    Shares line, warps;                   // even shares of the line and of r0 .. r1
};

__device__ __forceinline__ int length_of(const Args &a, int b) { return min(max(a.lens[b], 0), a.Tmax); }
__device__ __forceinline__ int units_in(const Args &a, int b) { return (length_of(a, b) + kUnit - 1) / kUnit; }

// f(units) for each of a lane's sequences b0 .. b1 - 1: in registers (PER), or read.
template <int PER, typename F>
__device__ __forceinline__ void each_own(const Args &a, const int (&own)[PER ? PER : 1], int b0, int b1, F f)
{
    if constexpr (PER > 0) {
#pragma unroll
        for (int i = 0; i < PER; i++)
            f(own[i]);
    } else {
        for (int b = b0; b < b1; b++)
            f(units_in(a, b));
    }
}

// ---------------------------------- how the CTAs share the units ----
// Split: every segment has CTAs of its own, about units / T of them, if that
// takes no more than the grid with T at most 24 units (3/16) above an even
// share.  Otherwise the line is cut evenly, and a CTA that shares two segments
// merges twice: 64 query rows over 2 segments of 64 units 22.5 us, split 15.6; 8
// segments of 256 units 13.5 and 13.1; but 76 us cut evenly and 83 split at 64
// segments of 1024 units, where T would be 69 more.  On the line a segment's start
// (queries read and scaled, outputs written) counts as kEdge units, laid before
// its first: without that a warp whose share was 14 segments of two units held up
// the others (256 sequences of 1 to 2048 positions, 8 KV heads: 97 us, so 83;
// 64 of 1 to 4096: 59 and 49).  A cut inside a segment of up to kSnap units moves
// to its nearer end.  A share has two cuts, so it may grow by kSnap units, against
// merges across CTAs: 152 segments of 32 units, whose largest share is then 66 and
// not 34, take 17.4 us, cut evenly 18.4; 64 x 8 of up to 32 units at D = 64 13.9 and
// 16.6; but 152 of 48 units, with shares of up to 98 and not 51, 22.9 and 21.8.
//
// Few units: where no segment has more than 12, each keeps one CTA (8 segments of
// 12 units 7.4 us; split 8.4); else a CTA of 16 warps takes 4 at least (8 segments
// of 16 units 8.4 us; with 8 at least 8.9), one of 8 warps 8 (64 query rows over 2
// segments of 64 units 15.6 us; with 4 at least 17.0).
//
// Up to 32 sequences a lane has one, up to 128 PER = 4, and the plan is
// straight-line code on registers; beyond (PER = 0), a lane has a chunk of them,
// and loops over it.  What this costs is fetching instructions that run once: one
// sequence of 32768 positions takes 21.6 us with loops and 21.1 so, one of 4096
// 10.7 and 10.2, 128 of 512 29.1 and 28.4 (the four-sequence code alone: 21.3, 10.5
// and 28.1); integer divisions throughout took 1 us more.  (Their units laid out in
// shared memory first: 1024 sequences of one unit 1.6 us less, but all small calls
// 0.1 to 0.2 us more for the code in between.)
template <int PER, int W>
__device__ __forceinline__ void make_plan(const Args &a, Plan *plan, Cursor *place)
{
    const int lane = threadIdx.x & 31, cta = blockIdx.x, HP = a.Hkv * a.passes, n_cta = gridDim.x;
    const int chunk = PER ? PER : (a.B + 31) / 32, b0 = lane * chunk, b1 = min(a.B, b0 + chunk);
    int own[PER ? PER : 1];                       // the lane's sequences' units
#pragma unroll
    for (int i = 0; i < PER; i++)
        own[i] = b0 + i < a.B ? units_in(a, b0 + i) : 0;
    int sum = 0, some = 0, longest = 0;           // (sum: units, later items, of one of the HP segments)
    each_own<PER>(a, own, b0, b1, [&](int n) {
        sum += n;
        some += n > 0;
        longest = max(longest, n);
    });
    constexpr int kMin = kMinUnits[W < 16];
    const int least = __reduce_max_sync(0xffffffffu, longest) <= kWhole ? kWhole : kMin;
    const int U = __reduce_add_sync(0xffffffffu, sum) * HP;
    const float N = (float)__reduce_add_sync(0xffffffffu, some) * (float)HP;
    // (T and the CTAs of a segment need not be exact, only the same in every CTA)
    const int T = max(least, (int)((float)U / (float)n_cta) + 1), more = min((T + 15) >> 4, 8);
    auto split_ctas = [](int nu, float inv) { return nu == 0 ? 0 : max(1, min(nu, (int)(nu * inv + 0.99f))); };
    float per_T = 0.0f;                           // 1 / T of a split, else 0
    if (N <= (float)n_cta) {
        float inv[4];
        int k[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; i++)
            inv[i] = __fdividef(1.0f, (float)(T + i * more));
        each_own<PER>(a, own, b0, b1, [&](int n) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                k[i] += split_ctas(n, inv[i]);
        });
#pragma unroll
        for (int i = 3; i >= 0; i--)
            if (__reduce_add_sync(0xffffffffu, k[i]) * HP <= n_cta) {
                per_T = inv[i];
                sum = k[i];                       // CTAs instead of units, from here on
            }
    }
    const bool split = per_T > 0.0f;
    auto items = [&](int nu) { return split ? split_ctas(nu, per_T) : nu + (nu > 0 ? kEdge : 0); };   // of a segment
    if (!split)
        sum += some * kEdge;
    int before = sum;                             // items of the sequences before the lane's
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, off);
        if (lane >= off)
            before += v;
    }
    const int all = __shfl_sync(0xffffffffu, before, 31) * HP;
    before -= sum;
    Plan pl;
    pl.n_act = split ? all : min(n_cta, (all + kMin - 1) / kMin);
    pl.split = split;
    pl.edge = split ? 0 : kEdge;
    // Item x (each lane its own): its sequence, head-pass, and number within
    // them; `per` items a segment.
    auto locate = [&](int x, int &per) {
        int ci = 0;                               // the lane holding it: the last that begins at or before it
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const int v = __shfl_sync(0xffffffffu, before, ci + off);
            if ((ci + off) * chunk < a.B && v * HP <= x)
                ci += off;
        }
        int left = x - __shfl_sync(0xffffffffu, before, ci) * HP;
        Cursor c = {ci * chunk, 0, 0, 0};
        if constexpr (PER > 0) {
            c.nu = __shfl_sync(0xffffffffu, own[0], ci);
            per = items(c.nu);
#pragma unroll
            for (int i = 1; i < PER; i++) {
                const int n = __shfl_sync(0xffffffffu, own[i], ci);
                if (c.b == ci * PER + i - 1 && left >= per * HP) {
                    left -= per * HP;
                    c.b++;
                    c.nu = n;
                    per = items(n);
                }
            }
        } else {
            for (; c.b < a.B; c.b++) {
                c.nu = units_in(a, c.b);
                per = items(c.nu);
                if (left < per * HP)
                    break;
                left -= per * HP;
            }
        }
        per = max(per, 1);
        if (HP > 1)
            c.hp = (unsigned)left / (unsigned)per;
        c.t = left - c.hp * per;
        return c;
    };
    if (cta < pl.n_act) {
        Cursor c;
        int k;
        if (split) {                              // units counted from the segment's start
            c = locate(cta, k);
            const int part = c.t;
            const Shares sp = {(int)((unsigned)c.nu / (unsigned)k), (int)((unsigned)c.nu % (unsigned)k)};
            pl.r0 = sp.start(part), pl.r1 = sp.start(part + 1);
            pl.cf = cta - part, pl.cl = pl.cf + k - 1;
        } else {
            pl.line = {(int)((unsigned)all / (unsigned)pl.n_act), (int)((unsigned)all % (unsigned)pl.n_act)};
            // (lane 0: the share's start, lane 1: its end)
            int x = pl.line.start(min(cta + lane, pl.n_act));
            c = locate(min(x, all - 1), k);
            if (x < all && c.nu <= kSnap)
                x += 2 * c.t < k ? -c.t : k - c.t;
            pl.r0 = __shfl_sync(0xffffffffu, x, 0), pl.r1 = __shfl_sync(0xffffffffu, x, 1);
            pl.cf = pl.cl = 0;
        }
        // (warps without units, if any, are the CTA's last: the merge counts on it)
        const unsigned len = pl.r1 - pl.r0;
        pl.warps = {(int)(len / W), (int)(len % W)};
        const int w0 = pl.r0 + pl.warps.start(min(lane, W));
        if (split)
            c.t = w0;
        else
            c = locate(min(w0, all - 1), k);
        if (lane < W)
            place[lane] = c;
    }
    if (lane == 0)
        *plan = pl;
}

template <int D, int NT, typename O>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1) attn_q4_kernel(const __grid_constant__ Args a)
{
    using C = Cfg<D, NT>;
    constexpr int NB = C::kNB, W = C::kWarps, S = C::kSlots;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Entry entry[2 * W];                    // warp w: 2w (began before its share), 2w + 1
    __shared__ int arrived[2];
    __shared__ Plan plan;
    __shared__ Cursor place[W], copy_at[W];           // warps' starts; what each copies next
    __shared__ int2 group[2 * W];                     // first entry, last warp of each merged segment

    uint8_t *sbase = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    uint8_t *const mine_raw = sbase + warp * C::kWarpBytes;
    const uint32_t ring = smem_u32(mine_raw), conv = ring + C::kRing;
    float *const last_part = reinterpret_cast<float *>(mine_raw);
    float *const first_part = reinterpret_cast<float *>(sbase + W * C::kWarpBytes) + warp * C::kPart;
    const int HP = a.Hkv * a.passes, cta = blockIdx.x;

    if (threadIdx.x < W * 2)
        entry[threadIdx.x].b = -1;
    pdl_launch_dependents();
    pdl_wait();

    auto length = [&](int b) { return length_of(a, b); };
    auto units_of = [&](int b) { return units_in(a, b); };

    if (warp == 0) {
        if (a.B <= 32)
            make_plan<1, W>(a, &plan, place);
        else if (a.B <= 128)
            make_plan<4, W>(a, &plan, place);
        else
            make_plan<0, W>(a, &plan, place);
    } else {
        // ------------------------------- sequences without positions ----
        for (int b = cta; b < a.B; b += gridDim.x)
            if (length(b) == 0) {
                const size_t n = (size_t)a.R * a.Hkv * D;
                O *o = static_cast<O *>(a.o) + b * n;
                for (size_t i = (threadIdx.x - 32) * 2; i < n; i += (C::kThreads - 32) * 2)
                    store2(o + i, 0.0f, 0.0f);
            }
    }
    __syncthreads();
    if (cta >= plan.n_act)
        return;
    auto next_seq = [&](Cursor &c) {                  // the next sequence with units
        c.hp = 0;
        do {
            c.b++;
            c.nu = c.b < a.B ? units_of(c.b) : 1;
        } while (c.nu == 0);
    };
    const int edge = plan.edge, w1 = plan.r0 + plan.warps.start(warp + 1);
    Cursor cur = place[warp];
    cur.t -= edge;                                    // (below 0: the segment's start)
    const int w0 = plan.r0 + plan.warps.start(warp) - min(cur.t, 0);
    cur.t = max(cur.t, 0);

    // ------------------------------------------------------- the ring ----
    // lane i copies chunk i % NB of positions i / NB, + 32 / NB, ... of keys and
    // values, then 16 bytes of the scales (one half-warp each)
    constexpr int kPer = 32 / NB;                     // positions per step: a multiple of the swizzle's period
    constexpr int kSc = C::kScales / 16;              // lanes per scale plane: 16 or 8
    const uint32_t lane_dst = swizzled<D>(lane / NB, lane % NB);
    // what is copied next: position row `is_row` of the planes, `is_left` units of its segment, `to_issue` in all
    if (lane == 0)
        copy_at[warp] = cur;
    __syncwarp();
    int is_left = cur.nu - cur.t, to_issue = w1 - w0;
    auto seg_row = [&](const Cursor &c) { return (c.b * a.Hkv + (a.passes == 1 ? c.hp : c.hp / a.passes)) * a.Tmax; };
    int is_row = seg_row(cur) + cur.t * kUnit;
    auto issue = [&](uint32_t base) {
        if (to_issue > 0) {
            const size_t off = (size_t)(unsigned)is_row * (D / 2) + lane * 16;
            const uint8_t *kp = a.kc + off, *vp = a.vc + off;
#pragma unroll
            for (int i = 0; i < kUnit / kPer; i++) {
                copy16(base + lane_dst + i * 512, kp + i * 512);
                copy16(base + lane_dst + C::kCodes + i * 512, vp + i * 512);
            }
            if (lane < 2 * kSc)
                copy16(base + 2 * C::kCodes + lane * 16,
                       (lane < kSc ? a.ks : a.vs) + (size_t)(unsigned)is_row * NB + (lane & (kSc - 1)) * 8);
            to_issue--;
            is_row += kUnit;
            // (only where there is more to copy: behind the last sequence lie idle slots, and each is a load to wait for)
            if (--is_left == 0 && (to_issue -= edge) > 0) {
                Cursor c = copy_at[warp];
                if (++c.hp == HP)
                    next_seq(c);
                is_left = c.nu;
                is_row = seg_row(c);
                __syncwarp();
                if (lane == 0)
                    copy_at[warp] = c;
                __syncwarp();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // ------------------------------------------------------ the stream ----
    uint32_t kb = ring;                               // slot of the unit at hand
    int u = w0;
    while (u < w1) {
        const int sb = cur.b, shp = cur.hp, st0 = cur.t, snu = cur.nu;
        const int ue = min(w1, u + snu - st0);
        const int pass = a.passes == 1 ? 0 : shp % a.passes, h = a.passes == 1 ? shp : shp / a.passes;
        const int row_base = pass * C::kRows;
        const int L = length(sb);

        // query fragments (B of the score product): block j, half hf (low / high
        // nibbles); the lane's row is g of each tile.  What follows a score is
        // held for the accumulator's rows, 2 t4 + e.
        uint32_t qf[NT][NB][2][2];
        float mul[NT][2];
        int lim[NT][2];                               // positions a row sees
        uint2 v[NT][NB][2];
        int tok[NT];
#pragma unroll
        for (int r = 0; r < NT; r++) {
            const int row = row_base + g + 8 * r;
            const bool live = row < a.R;
            tok[r] = live && a.Tq > 1 ? row / a.G : 0;
            const uint16_t *qp = a.q + (((size_t)sb * a.Tq + tok[r]) * a.Hkv * a.G + (size_t)h * a.G + (live ? row - tok[r] * a.G : 0)) * D;
#pragma unroll
            for (int j = 0; j < NB; j++)
#pragma unroll
                for (int hf = 0; hf < 2; hf++)
                    v[r][j][hf] = live ? *reinterpret_cast<const uint2 *>(qp + 32 * j + 16 * hf + 4 * t4) : make_uint2(0u, 0u);
        }
        if (u == w0) {                                // (the first copies queue behind the query, not before it)
#pragma unroll
            for (int k = 0; k < S; k++)
                issue(ring + k * C::kSlotBytes);
        }
#pragma unroll
        for (int r = 0; r < NT; r++) {
            uint32_t mx = 0;
#pragma unroll
            for (int j = 0; j < NB; j++)
#pragma unroll
                for (int hf = 0; hf < 2; hf++)
                    mx = __vmaxu2(mx, __vmaxu2(v[r][j][hf].x & 0x7fff7fffu, v[r][j][hf].y & 0x7fff7fffu));
            mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const int top = (int)max(mx & 0xffffu, mx >> 16);
            // max |q| 2^k in [2^13, 2^14) (exact for subnormal rows too); inf and NaN pass through
            const int k = top == 0 || top >= 0x7c00 ? 0 : 28 - max(top >> 10, 1);
            const float f = a.scale2 < 0.0f ? -pow2i(k) : pow2i(k);
            // positive and not 0, so that a masked score of -inf stays one
            const float back = fabsf(a.scale2) * pow2i(-k);
#pragma unroll
            for (int e = 0; e < 2; e++) {
                mul[r][e] = __shfl_sync(0xffffffffu, back, 8 * t4 + 4 * e);
                lim[r][e] = L - (a.Tq - 1 - __shfl_sync(0xffffffffu, tok[r], 8 * t4 + 4 * e));
            }
#pragma unroll
            for (int j = 0; j < NB; j++)
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    // register e holds elements 4 t4 + e and 4 t4 + 2 + e: the order of the masked key bytes
                    qf[r][j][hf][0] = pack_f16x2(f16_lo(v[r][j][hf].x) * f, f16_lo(v[r][j][hf].y) * f);
                    qf[r][j][hf][1] = pack_f16x2(f16_hi(v[r][j][hf].x) * f, f16_hi(v[r][j][hf].y) * f);
                }
        }
        float m[NT][2], l[NT][2], acc[NT][2 * NB][4];
        int ev = 0;                                   // exponent bits of the largest value scale so far
#pragma unroll
        for (int r = 0; r < NT; r++) {
            m[r][0] = m[r][1] = kFloor;
            l[r][0] = l[r][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2 * NB; i++)
                acc[r][i][0] = acc[r][i][1] = acc[r][i][2] = acc[r][i][3] = 0.0f;
        }

        int t0 = st0 * kUnit;
        for (; u < ue; u++, t0 += kUnit) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
            __syncwarp();                             // every lane's copies of this unit have landed
            const uint32_t vb = kb + C::kCodes;
            // ------------------------------------------ scales ----
            // lane i converts position i's; past the length the cache may
            // hold anything: scales of 0
            const bool valid = t0 + lane < L;
            uint32_t sc[NB / 2];
            (void)load_scales<NB>(sc, kb + 2 * C::kCodes + lane * NB * 2, valid);
            store_scales<NB>(conv + lane * NB * 4, sc, 1.0f);
            int top = (int)__reduce_max_sync(
                0xffffffffu, load_scales<NB>(sc, kb + 2 * C::kCodes + C::kScales + lane * NB * 2, valid)) >> 10;
            if (top == 31) {
                // Value scales that are not finite: they enter as 0, so that weights of 0
                // past a row's end stay 0, and the blocks of the rows that see one are NaN.
                uint32_t mx = 0;
#pragma unroll
                for (int j = 0; j < NB; j++) {
                    const uint32_t h = sc[j >> 1] >> 16 * (j & 1) & 0x7fffu;
                    const unsigned bad = __ballot_sync(0xffffffffu, h >= 0x7c00u);
                    if (h >= 0x7c00u)
                        sc[j >> 1] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
                    else
                        mx = max(mx, h);
#pragma unroll
                    for (int r = 0; r < NT; r++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const int n = lim[r][e] - t0;         // positions of the unit that the row sees
                            if (n > 0 && bad & (n < kUnit ? (1u << n) - 1u : ~0u))
                                acc[r][2 * j][e] = acc[r][2 * j][e + 2] = acc[r][2 * j + 1][e] = acc[r][2 * j + 1][e + 2] =
                                    __int_as_float(0x7fffffff);
                        }
                }
                top = (int)__reduce_max_sync(0xffffffffu, mx) >> 10;
            }
            const int en = max(ev, top);
            store_scales<NB>(conv + (kUnit + lane) * NB * 4, sc, pow2i(kBase - en));
            __syncwarp();
            // ------------------------------------------ scores ----
            // s[r][p][e]: row 2 t4 + e of tile r, position 8 p + g
            float s[NT][4][2];
#pragma unroll
            for (int mt = 0; mt < 2; mt++) {      // 16 positions
                uint32_t kx[2][NB];
                if constexpr (D == 128) {
#pragma unroll
                    for (int i = 0; i < 2; i++)
                        ldsm4(kx[i], kb + swizzled<D>(16 * mt + 8 * i + (lane & 7), lane >> 3));
                } else {
                    uint32_t t[4];                // positions 0-7: blocks 0, 1; positions 8-15: blocks 0, 1
                    ldsm4(t, kb + swizzled<D>(16 * mt + 8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1));
                    kx[0][0] = t[0], kx[0][1] = t[1], kx[1][0] = t[2], kx[1][1] = t[3];
                }
                float dk[2][NB];
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    row_scales<NB>(dk[i], conv + (16 * mt + 8 * i + g) * NB * 4);
                }
#pragma unroll
                for (int j = 0; j < NB; j++) {
                    const uint32_t x0 = kx[0][j], x1 = kx[1][j], y0 = x0 >> 8, y1 = x1 >> 8;
                    const uint32_t l0 = nib_lo(x0), l1 = nib_lo(x1), l2 = nib_lo(y0), l3 = nib_lo(y1);
                    const uint32_t h0 = nib_hi(x0), h1 = nib_hi(x1), h2 = nib_hi(y0), h3 = nib_hi(y1);
                    float c[NT][4];
#pragma unroll
                    for (int r = 0; r < NT; r++)
                        mma0(c[r], l0, l1, l2, l3, qf[r][j][0][0], qf[r][j][0][1]);
#pragma unroll
                    for (int r = 0; r < NT; r++)
                        mma(c[r], h0, h1, h2, h3, qf[r][j][1][0], qf[r][j][1][1]);
#pragma unroll
                    for (int r = 0; r < NT; r++)
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            float (&sp)[2] = s[r][2 * mt + i];
                            if (j == 0) {
                                mul2(sp, c[r][2 * i], c[r][2 * i + 1], dk[i][0]);
                            } else {
                                float cp[2] = {c[r][2 * i], c[r][2 * i + 1]};
                                fma2(cp, dk[i][j], dk[i][j], sp[0], sp[1]);
                                sp[0] = cp[0], sp[1] = cp[1];
                            }
                        }
                }
            }
            if (t0 + kUnit > L - (a.Tq - 1)) {    // some row's positions end in this unit
#pragma unroll
                for (int p = 0; p < 4; p++)
#pragma unroll
                    for (int r = 0; r < NT; r++)
#pragma unroll
                        for (int e = 0; e < 2; e++)
                            s[r][p][e] = t0 + 8 * p + g < lim[r][e] ? s[r][p][e] : -INFINITY;
            }
            // ----------------------------------- running maximum ----
            // (of the lane's positions: the whole row's is needed only where m moves)
            bool grow = en > ev;
            float mx[NT][2];
#pragma unroll
            for (int r = 0; r < NT; r++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    mx[r][e] = fmaxf(fmaxf(s[r][0][e], s[r][1][e]), fmaxf(s[r][2][e], s[r][3][e]));
                    grow = grow || (mx[r][e] - m[r][e]) * mul[r][e] > kSlack;
                }
            if (__any_sync(0xffffffffu, grow)) {
                const float fe = pow2i(ev - en);
                ev = en;
#pragma unroll
                for (int r = 0; r < NT; r++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1)
                            mx[r][e] = fmaxf(mx[r][e], __shfl_xor_sync(0xffffffffu, mx[r][e], off));
                        const float mn = fmaxf(m[r][e], mx[r][e]), f = ex2((m[r][e] - mn) * mul[r][e]);
                        m[r][e] = mn;
                        l[r][e] *= f;
#pragma unroll
                        for (int i = 0; i < 2 * NB; i++) {
                            acc[r][i][e] *= f * fe;
                            acc[r][i][e + 2] *= f * fe;
                        }
                    }
            }
#pragma unroll
            for (int r = 0; r < NT; r++)
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    sub2(s[r][p], m[r]);
                    mul2(s[r][p], mul[r]);
                    s[r][p][0] = ex2(s[r][p][0]);
                    s[r][p][1] = ex2(s[r][p][1]);
                    add2(l[r], s[r][p]);
                }
            // ------------------------------------------ values ----
#pragma unroll
            for (int k = 0; k < 2; k++) {         // 16 positions
                float dv[2][NB];
                row_scales<NB>(dv[0], conv + (kUnit + 16 * k + g) * NB * 4);
                row_scales<NB>(dv[1], conv + (kUnit + 16 * k + 8 + g) * NB * 4);
#pragma unroll
                for (int j2 = 0; j2 < NB / 2; j2++) {
                    uint32_t x[4];                // block 2 j2: positions 0-7, 8-15; block 2 j2 + 1
                    ldsm4t(x, vb + swizzled<D>(16 * k + (lane & 15), 2 * j2 + (lane >> 4)));
#pragma unroll
                    for (int jj = 0; jj < 2; jj++) {
                        const int j = 2 * j2 + jj;
                        uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
                        for (int r = 0; r < NT; r++)
#pragma unroll
                            for (int i = 0; i < 2; i++) {
                                float pv[2];
                                mul2(pv, s[r][2 * k + i][0], s[r][2 * k + i][1], dv[i][j]);
                                const uint32_t w = pack_f16x2(pv[0], pv[1]);
                                bh[r][i] = transposed(w);
                                bl[r][i] = transposed(pack_f16x2(pv[0] - f16_lo(w), pv[1] - f16_hi(w)));
                            }
                        const uint32_t x0 = x[2 * jj], x1 = x[2 * jj + 1], y0 = x0 >> 8, y1 = x1 >> 8;
                        const uint32_t e0 = nib_lo(x0), e1 = nib_hi(x0), e2 = nib_lo(x1), e3 = nib_hi(x1);
                        const uint32_t f0 = nib_lo(y0), f1 = nib_hi(y0), f2 = nib_lo(y1), f3 = nib_hi(y1);
#pragma unroll
                        for (int r = 0; r < NT; r++) {
                            mma(acc[r][2 * j], e0, e1, e2, e3, bh[r][0], bh[r][1]);
                            mma(acc[r][2 * j + 1], f0, f1, f2, f3, bh[r][0], bh[r][1]);
                            mma(acc[r][2 * j], e0, e1, e2, e3, bl[r][0], bl[r][1]);
                            mma(acc[r][2 * j + 1], f0, f1, f2, f3, bl[r][0], bl[r][1]);
                        }
                    }
                }
            }
            __syncwarp();
            issue(kb);                                // refill the slot just read
            kb += C::kSlotBytes;
            if (kb == ring + C::kRing)
                kb = ring;
        }
        // ---------------------------------------------- segment's end ----
#pragma unroll
        for (int r = 0; r < NT; r++)
#pragma unroll
            for (int e = 0; e < 2; e++)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l[r][e] += __shfl_xor_sync(0xffffffffu, l[r][e], off);
        const bool before = st0 > 0, after = t0 < snu * kUnit;
        const float unscale = pow2i(ev - kBase);
        if (!before && !after) {
#pragma unroll
            for (int r = 0; r < NT; r++) {
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    const float fi = lim[r][c] > 0 ? unscale / l[r][c] : 0.0f;   // (l = 0 where every score is -inf: 0 / 0)
                    const int row = row_base + 8 * r + 2 * t4 + c;
                    if (row < a.R) {
                        O *o = static_cast<O *>(a.o) +
                               (((size_t)sb * a.Tq + row / a.G) * a.Hkv * a.G + (size_t)h * a.G + row % a.G) * D;
#pragma unroll
                        for (int j = 0; j < NB; j++) {
                            store2(o + 32 * j + 2 * g, acc[r][2 * j][c] * fi, acc[r][2 * j + 1][c] * fi);
                            store2(o + 32 * j + 16 + 2 * g, acc[r][2 * j][c + 2] * fi, acc[r][2 * j + 1][c + 2] * fi);
                        }
                    }
                }
            }
        } else {
            // a segment that began before this share goes to the warp's first
            // slot; one that only continues after it is the share's last, and
            // the ring is drained
            float *pp = before ? first_part : last_part;
            if (lane == 0)
                entry[2 * warp + (before ? 0 : 1)] = {sb, shp, u - t0 / kUnit, snu};
#pragma unroll
            for (int r = 0; r < NT; r++) {
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    float *o = pp + (8 * r + 2 * t4 + c) * C::kLd;
#pragma unroll
                    for (int j = 0; j < NB; j++) {
                        *reinterpret_cast<float2 *>(o + 32 * j + 2 * g) = make_float2(acc[r][2 * j][c] * unscale, acc[r][2 * j + 1][c] * unscale);
                        *reinterpret_cast<float2 *>(o + 32 * j + 16 + 2 * g) = make_float2(acc[r][2 * j][c + 2] * unscale, acc[r][2 * j + 1][c + 2] * unscale);
                    }
                }
                if (g == 0) {                         // (m as q K[t]: mul is |scale2| times a power of two)
                    const float f0 = __int_as_float(__float_as_int(mul[r][0]) - __float_as_int(fabsf(a.scale2)) + __float_as_int(1.0f));
                    const float f1 = __int_as_float(__float_as_int(mul[r][1]) - __float_as_int(fabsf(a.scale2)) + __float_as_int(1.0f));
                    const float m0 = m[r][0] == kFloor && lim[r][0] > st0 * kUnit ? kAllInf : m[r][0] * f0;
                    const float m1 = m[r][1] == kFloor && lim[r][1] > st0 * kUnit ? kAllInf : m[r][1] * f1;
                    *reinterpret_cast<float4 *>(pp + C::kRows * C::kLd + 2 * (8 * r + 2 * t4)) = make_float4(m0, l[r][0], m1, l[r][1]);
                }
            }
        }
        // the next segment
        cur.t = 0;
        if (!after) {
            u += edge;
            if (u < w1 && ++cur.hp == HP)
                next_seq(cur);
        }
    }
    __syncthreads();

    // ------------------------------------------------ merge the warps ----
    constexpr size_t gp = (size_t)C::kRows * (D + 2); // floats of a CTA partial
    auto pass_of = [&](const Entry &e) { return a.passes == 1 ? 0 : e.hp % a.passes; };
    auto out_row = [&](const Entry &e, int row) {     // output of a pass's row (row < R checked by the caller)
        const int rr = pass_of(e) * C::kRows + row, tok = a.Tq == 1 ? 0 : rr / a.G;
        return static_cast<O *>(a.o) + (((size_t)e.b * a.Tq + tok) * a.Hkv * a.G +
                                        (size_t)(a.passes == 1 ? e.hp : e.hp / a.passes) * a.G + (rr - tok * a.G)) * D;
    };
    auto live_rows = [&](const Entry &e) { return min(C::kRows, a.R - pass_of(e) * C::kRows); };
    // Entries of one segment are consecutive (the invalid ones skipped): a group
    // is warp wa's entry and the first entry of each following warp.
    Entry mine = {-1, 0, 0, 0};
    if (lane < 2 * W)
        mine = entry[lane];
    const unsigned valid = __ballot_sync(0xffffffffu, mine.b >= 0);
    const unsigned earlier = valid & ((1u << lane) - 1u);
    const int prev_first = __shfl_sync(0xffffffffu, mine.first, earlier ? 31 - __clz(earlier) : 0);
    const unsigned heads = __ballot_sync(0xffffffffu, mine.b >= 0 && (!earlier || prev_first != mine.first));
    auto group_of = [&](int i) {                      // the entries of the group headed by entry i
        const unsigned after = heads & ~((2u << i) - 1u);
        return valid & ~((1u << i) - 1u) & (after ? (1u << (__ffs(after) - 1)) - 1u : ~0u);
    };
    auto entry_part = [&](int k) {
        const int w = k >> 1;
        return reinterpret_cast<const float *>(sbase + ((k & 1) ? w * C::kWarpBytes : W * C::kWarpBytes + w * C::kPart * 4));
    };
    if (warp == 0 && (heads >> lane & 1)) {
        const int k = __popc(heads & ((1u << lane) - 1u));
        group[k] = make_int2(lane, (31 - __clz(group_of(lane))) >> 1);
    }
    __syncthreads();
    const int n_groups = __popc(heads);
    constexpr int kItems = C::kRows * (D / 4);
#pragma unroll 1
    for (int it = threadIdx.x; it < n_groups * kItems; it += C::kThreads) {
        const int k = it / kItems, row = it % kItems / (D / 4), d = it % (D / 4) * 4;
        const int i = group[k].x, wb = group[k].y, wa = i >> 1;
        const Entry e = entry[i];
        if (row >= live_rows(e))
            continue;
        // warp wa's entry, then the first entries of wa + 1 .. wb
        const float *pa = entry_part(i), *pf = entry_part(0);
        constexpr int step = C::kPart;
        const int ml = C::kRows * C::kLd + 2 * row;
        float M = pa[ml];
#pragma unroll 8
        for (int w = wa + 1; w <= wb; w++)
            M = fmaxf(M, pf[w * step + ml]);
        float L = 0.0f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int w = wa; w <= wb; w++) {
            const float *pp = w == wa ? pa : pf + w * step;
            const float2 s2 = *reinterpret_cast<const float2 *>(pp + ml);
            const float4 v = *reinterpret_cast<const float4 *>(pp + row * C::kLd + d);
            const float f = ex2((s2.x - M) * fabsf(a.scale2));
            L = fmaf(f, s2.y, L);
            o.x = fmaf(f, v.x, o.x);
            o.y = fmaf(f, v.y, o.y);
            o.z = fmaf(f, v.z, o.z);
            o.w = fmaf(f, v.w, o.w);
        }
        if (e.first >= plan.r0 && e.first + e.units <= plan.r1) {
            store4(out_row(e, row) + d, o, M >= kAllInf ? 1.0f / L : 0.0f);
        } else {
            float *gpart = a.partials + ((size_t)cta * 2 + (e.first < plan.r0 ? 0 : 1)) * gp;
            __stcg(reinterpret_cast<float4 *>(gpart + (size_t)row * D + d), o);
            if (d == 0)
                __stcg(reinterpret_cast<float2 *>(gpart + (size_t)C::kRows * D) + row, make_float2(M, L));
        }
    }
    // segments other CTAs share: the first and the last group may be
    int shared_seg[2], n_shared = 0;
    for (int k = 0; k < n_groups; k += max(1, n_groups - 1)) {
        const Entry e = entry[group[k].x];
        if (e.first < plan.r0 || e.first + e.units > plan.r1)
            shared_seg[n_shared++] = group[k].x;
    }
    if (n_shared == 0)
        return;

    // --------------------------------------------------- merge the CTAs ----
    __syncthreads();
    if ((int)threadIdx.x < n_shared) {
        const Entry e = entry[shared_seg[threadIdx.x]];
        const int cf = plan.split ? plan.cf : plan.line.owner(e.first);
        const int cl = plan.split ? plan.cl : plan.line.owner(e.first + e.units - 1);
        // (release and acquire for the whole CTA: the barriers on both sides extend it to the other threads)
        arrived[threadIdx.x] = atom_add_acq_rel_gpu(a.counters + cf, 1) == cl - cf;
    }
    __syncthreads();
    for (int k = 0; k < n_shared; k++) {
        if (!arrived[k])
            continue;
        const Entry e = entry[shared_seg[k]];
        const int cf = plan.split ? plan.cf : plan.line.owner(e.first);
        const int cl = plan.split ? plan.cl : plan.line.owner(e.first + e.units - 1);
        const int rows = live_rows(e);
        // The segment starts inside cf (its second slot) and before every later
        // CTA (their first slots, 2 gp apart).  (Cuts inside segments that CTAs
        // share are where the even shares put them: owner() holds there.)
        float *base = a.partials + (size_t)cf * 2 * gp;
        // All partials of a few rows are copied to shared memory at once (the
        // rings and the warps' partials are done with) and summed there; warps
        // without a sum, or all after it, clear what was copied.  Loops, not
        // unrolled: this runs once, and fetching its code is what it would cost.
        const int P = cl - cf + 1;
        const int step = min(32, (C::kRoom / P) & ~1);   // (even, at least 2)
        float *so = reinterpret_cast<float *>(sbase);
        for (int row0 = 0; row0 < rows; row0 += step) {
            const int nr = min(step, rows - row0), n4 = nr * (D / 4), nr2 = (nr + 1) & ~1;
            float2 *sml = reinterpret_cast<float2 *>(so + P * nr * D);
#pragma unroll 1
            for (int p = warp; p < P; p += W) {
                const float *src = base + (size_t)p * 2 * gp + (p == 0 ? gp : 0);
#pragma unroll 1
                for (int i = lane; i < n4; i += 32)
                    copy16(smem_u32(so + (p * n4 + i) * 4), src + (size_t)row0 * D + i * 4);
                if (2 * lane < nr)
                    copy16(smem_u32(sml + p * nr2 + 2 * lane), src + (size_t)C::kRows * D + (row0 + 2 * lane) * 2);
            }
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
            __syncthreads();
#pragma unroll 1
            for (int it = threadIdx.x; it < nr * (D / 2); it += C::kThreads) {
                const int row = it / (D / 2), d = it % (D / 2) * 2;
                float M = sml[row].x, L = 0.0f;
                float2 o = make_float2(0.f, 0.f);
#pragma unroll 4
                for (int p = 1; p < P; p++)
                    M = fmaxf(M, sml[p * nr2 + row].x);
#pragma unroll 4
                for (int p = 0; p < P; p++) {
                    const float2 s2 = sml[p * nr2 + row];
                    const float2 v = *reinterpret_cast<const float2 *>(so + (p * nr + row) * D + d);
                    const float f = ex2((s2.x - M) * fabsf(a.scale2));
                    L = fmaf(f, s2.y, L);
                    o.x = fmaf(f, v.x, o.x);
                    o.y = fmaf(f, v.y, o.y);
                }
                const float inv = M >= kAllInf ? 1.0f / L : 0.0f;
                store2(out_row(e, row0 + row) + d, o.x * inv, o.y * inv);
            }
            const int busy = (nr * (D / 2) + 31) / 32, from = busy < W ? busy : 0;
#pragma unroll 1
            for (int p = warp - from; p >= 0 && p < P; p += W - from) {
                float *src = base + (size_t)p * 2 * gp + (p == 0 ? gp : 0);
#pragma unroll 1
                for (int i = lane; i < n4; i += 32)
                    __stcg(reinterpret_cast<float4 *>(src + (size_t)row0 * D) + i, make_float4(0.f, 0.f, 0.f, 0.f));
                if (2 * lane < nr)
                    __stcg(reinterpret_cast<float4 *>(src + (size_t)C::kRows * D + row0 * 2) + lane, make_float4(0.f, 0.f, 0.f, 0.f));
            }
            __syncthreads();                          // (the space is free again)
        }
        if (threadIdx.x == 0)
            a.counters[cf] = 0;
    }
}

template <int D, int NT, typename O>
int32_t launch(Args &a, int grid, void *stream)
{
    using C = Cfg<D, NT>;
    const void *kernel = (const void *)attn_q4_kernel<D, NT, O>;
    static std::atomic<bool> done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return BQ_ERR_CUDA;
    if (dev < 0 || dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem) != cudaSuccess)
            return BQ_ERR_CUDA;
        if (dev >= 0 && dev < 64)
            done[dev].store(true, std::memory_order_release);
    }
    void *args[] = {&a};
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(C::kThreads), C::kSmem, static_cast<cudaStream_t>(stream),
                      args) == cudaSuccess
               ? BQ_OK
               : BQ_ERR_CUDA;
}

template <int D, int NT>
int32_t launch(Args &a, int grid, bool f16, void *stream)
{
    return f16 ? launch<D, NT, __half>(a, grid, stream) : launch<D, NT, float>(a, grid, stream);
}

// 8-row tiles a warp takes of R query rows, in ceil(R / 8 tiles) passes over a
// segment.  At 64 segments of 8192 positions (D = 128) a further pass takes 15.7
// us with one tile; with two, which unpack codes once for both but run 2 warps a
// scheduler instead of 4, 26.5.  So 24 rows take 63 us in three passes and 70 in
// two, 40 rows 94 and 97, but 16 rows 47 and 43, 48 rows 109 and 98, and from 6
// tiles on two a pass are no slower (at D = 64: 24 rows 41 and 46, 48 rows 68 and
// 63, 56 rows 76 and 79).  (Tiles side by side in a CTA, over one copy
// of the cache in L2 or shared memory, were no faster in an earlier form, when these
// took 55, 63 and 79 us at 24, 32 and 40 rows: 60, 64 and 93; at 302 MB of cache,
// past L2, 180, 190 and 286 against 165, 185 and 263.)
int tiles_of(int R)
{
    const int t = (R + 7) / 8;
    return 169 * ((t + 1) / 2) < 100 * t ? 2 : 1;
}

}  // namespace aq
}  // namespace bq

using namespace bq;

extern "C" size_t bq_attn_q4_workspace_bytes(int32_t D, int32_t Tq, int32_t G)
{
    if ((D != 64 && D != 128) || Tq < 1 || Tq > 32 || G < 1 || G > 16)
        return 0;
    return aq::kMaxGrid * sizeof(int) + (size_t)aq::kMaxGrid * 2 * 8 * aq::tiles_of(Tq * G) * (D + 2) * sizeof(float);
}

extern "C" int32_t bq_attn_decode_q4(const bq_kv_cache_q4 *kv, const uint16_t *q, const int32_t *lens,
                                     int32_t B, int32_t Tq, int32_t Hkv, int32_t G, float scale, void *o,
                                     int32_t o_dtype, void *ws, size_t ws_bytes, int32_t *dev_status,
                                     void *stream)
{
    if (!kv || !kv->k_codes || !kv->k_scales || !kv->v_codes || !kv->v_scales || !q || !lens || !o || !ws)
        return BQ_ERR_NULL;
    const size_t need = bq_attn_q4_workspace_bytes(kv->D, Tq, G);
    // (|scale| <= 1e18 keeps scale log2(e) 2^2 finite)
    if (need == 0 || kv->Tmax < 32 || kv->Tmax % 32 != 0 || Hkv < 1 || !(std::fabs(scale) <= 1e18f) ||
        (o_dtype != BQ_F32 && o_dtype != BQ_F16))
        return BQ_ERR_SHAPE;
    if (B < 1)
        return BQ_ERR_BATCH;
    const long long rows = (long long)B * Hkv < (1LL << 31) ? (long long)B * Hkv * kv->Tmax : 1LL << 31;
    const int R = Tq * G;
    const int tiles = aq::tiles_of(R), passes = (R + 8 * tiles - 1) / (8 * tiles);
    // positions, and units of all passes, are 32-bit numbers
    if (rows >= (1LL << 31) || rows / 32 * passes >= (1LL << 31) / (1 + aq::kEdge))
        return BQ_ERR_SHAPE;
    if (!aligned16(kv->k_codes) || !aligned16(kv->k_scales) || !aligned16(kv->v_codes) ||
        !aligned16(kv->v_scales) || !aligned16(q) || !aligned16(o) || !aligned16(ws) ||
        (reinterpret_cast<uintptr_t>(lens) & 3u))
        return BQ_ERR_ALIGN;
    if (ws_bytes < need)
        return BQ_ERR_WORKSPACE;
    if (o == q)
        return BQ_ERR_SHAPE;
    (void)dev_status;                                 // nothing here can fail on the device
    const int sms = device_sm_count();
    if (sms <= 0)
        return BQ_ERR_CUDA;
    aq::Args a;
    memset(&a, 0, sizeof(a));
    a.kc = kv->k_codes;
    a.vc = kv->v_codes;
    a.ks = kv->k_scales;
    a.vs = kv->v_scales;
    a.q = q;
    a.lens = lens;
    a.o = o;
    a.B = B;
    a.Tq = Tq;
    a.Hkv = Hkv;
    a.G = G;
    a.Tmax = kv->Tmax;
    a.R = R;
    a.passes = passes;
    a.scale2 = std::copysign(std::fmax(std::fabs(scale) * 1.4426950408889634f, aq::kScaleMin), scale);
    a.counters = static_cast<int *>(ws);
    a.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + aq::kMaxGrid * sizeof(int));
    const int grid = sms < aq::kMaxGrid ? sms : aq::kMaxGrid;
    const bool f16 = o_dtype == BQ_F16;
    if (kv->D == 128)
        return tiles == 1 ? aq::launch<128, 1>(a, grid, f16, stream) : aq::launch<128, 2>(a, grid, f16, stream);
    return tiles == 1 ? aq::launch<64, 1>(a, grid, f16, stream) : aq::launch<64, 2>(a, grid, f16, stream);
}
