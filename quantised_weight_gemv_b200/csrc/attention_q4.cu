// attention_q4.cu -- decode attention over a 4-bit KV cache, sm_100a.
//
//   s_t = scale * q . K[t]   p = softmax(s over t < lens[b] - (Tq - 1 - i))   o = sum_t p_t V[t]
//
// Bound: a position of one KV head is 144 bytes (D = 128), read once for its
// R = Tq * G query rows: 4 D R / 144 flops a byte, so HBM up to about 16 rows;
// what stands against it is the number of instructions that unpack 256 codes.
//
// Work: a unit is 32 positions of one (sequence, KV head).  The valid units of
// all sequences form one line (lens are on the device, so every CTA builds the
// prefix sums itself); CTAs take equal consecutive shares of it, and a CTA's
// workers (warps) equal consecutive shares of the CTA's.  Ragged lengths
// therefore cost no balance, and a sequence that ends inside a share just
// starts the next one: a warp never waits for another before its line ends.
// A warp streams its units through a ring of its own in shared memory (TMA,
// refilled by the warp itself, so a slot needs no "empty" barrier).
//
// Softmax: one pass with a running reference m a row; a warp's result of a
// segment (the part of a sequence's head in its share) is (m, l, O).  A whole
// segment is written out directly.  The two that may continue in a neighbour
// are merged at the end: warps through shared memory, CTAs through the
// workspace, where the last CTA to arrive merges in CTA order (deterministic).
//
// Tensor cores (mma.sync m16n8k16; with 8 or 16 rows a tcgen05 tile of 128
// rows would be empty), fp32 accumulation, codes exact:
//   scores  S[row][t]: A = q, B = key codes u (0..15) as fp16 subnormals
//     u 2^-24 (the masked nibble is the whole conversion; the high nibble is
//     16 u, so q enters times 1/16 there).  The zero point is the accumulator's
//     start, -8 2^-24 sum(q) a block.  Each block is scaled by dK in fp32.  q is
//     multiplied by a power of two a row first so that both forms are exact.
//   values  O^T[d][row]: A = value codes u - 8 (exact fp16: (0x6400 | u) - 1032),
//     signed so that sums over thousands of positions do not cancel against a
//     zero-point sum, B = p dV rounded to fp16.  ldmatrix.trans on 16-bit units
//     turns position-major rows into pairs of positions per register.
//   The score accumulators have the layout B needs: p stays in registers.
// Scaling of p: fp16 must neither overflow nor go subnormal where it counts, so
// a row's reference bounds p dV instead of p: m = max(s + log2 dV) - 11, with
// log2 of a lane's largest value scale taken as bits / 1024 - 15 (at most 0.09
// low, up to 9 high for subnormals).  O and l carry the same 2^-m.  m moves
// only when the bound outgrows it by 2^4: p dV < 2^15.1.
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
constexpr int kMaxGrid = 256;             // CTAs (one per SM)
constexpr int kPassRows = 64;             // query rows per pass over a segment (NT = 2)
constexpr float kFloor = -3.0e38f;        // a reference no score has reached
constexpr float kBase = 11.0f, kSlack = 4.0f;
constexpr int kScan = 256;                // chunks of the prefix sums

// D: head width; NT: 8-row tiles per warp (1: R <= 8; 2: 16 rows).
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
    static constexpr int kLd = D + 8;                         // floats per row of a partial in shared memory
    static constexpr int kPart = kRows * kLd + 2 * kRows;     // floats: O, m, l
    static constexpr size_t kSmem = 1024 + (size_t)kWarps * (kRing + kPart * 4);
    static_assert(kPart * 4 <= kRing, "a warp's last partial fits its drained ring");
    static_assert(kSlotBytes % 512 == 0 || D == 64, "slots keep the swizzle's period");
    static_assert(kSlotBytes % 256 == 0, "slots keep the swizzle's period");
    static_assert(kSmem <= 227 * 1024, "shared memory of an SM");
};

struct Args {
    CUtensorMap tm_k, tm_v;               // (D/2 bytes, B*Hkv*Tmax rows), box 32 rows, swizzled
    const uint16_t *ks, *vs, *q;
    const int32_t *lens;
    void *o;
    int B, Tq, Hkv, G, Tmax;
    int R;                                // Tq * G query rows per KV head
    int rg, passes;                       // 16-row groups per CTA (1, 2, 4), passes of 16 rg rows
    float scale2;                         // scale * log2(e)
    int *counters;                        // [grid], by a shared segment's first CTA
    float *partials;                      // [grid][2][rows][D + 2]
    int *status;
};

struct Entry {                            // a shared segment's part, for the merges
    int b, hp, first, units;              // sequence, head * passes + pass, first unit on the line, units
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
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
// The scale words of two consecutive positions: w[position][block pair].
template <int NB>
__device__ __forceinline__ void scale_words(uint32_t (&w)[2][NB / 2], uint32_t addr)
{
    if constexpr (NB == 4)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0][0]), "=r"(w[0][1]), "=r"(w[1][0]), "=r"(w[1][1]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0][0]), "=r"(w[1][0]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar, uint64_t policy)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(policy) : "memory");
}
// Byte offset of 16-byte chunk `chunk` of a row as TMA's 64- or 32-byte swizzle lays it down.
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

// The CTA (or worker) owning unit x when n of them share U units.
__device__ __forceinline__ int owner_of(long long x, int U, int n) { return (int)(((x + 1) * n - 1) / U); }

template <typename O>
__device__ __forceinline__ void store2(O *p, float a, float b)
{
    if constexpr (sizeof(O) == 4)
        *reinterpret_cast<float2 *>(p) = make_float2(a, b);
    else
        *reinterpret_cast<uint32_t *>(p) = pack_f16x2(a, b);
}

// A place on the line of units: unit t of nu of (sequence b, head-pass hp).
struct Cursor {
    int b, hp, t, nu;
};

template <int D, int NT, typename O>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1) attn_q4_kernel(const __grid_constant__ Args a)
{
    using C = Cfg<D, NT>;
    constexpr int NB = C::kNB, W = C::kWarps, S = C::kSlots;
    constexpr bool kTwo = sizeof(O) == 4;             // p dV as two fp16 terms
    extern __shared__ uint8_t smem_raw[];
    __shared__ alignas(8) uint64_t bar_full[W][S];
    __shared__ int pre[kScan + 1];
    __shared__ Entry entry[W][2];
    __shared__ int scan_tmp[kScan / 32];
    __shared__ int arrived[2];

    uint8_t *sbase = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const uint32_t ring = smem_u32(sbase) + warp * C::kRing;
    float *first_part = reinterpret_cast<float *>(sbase + W * C::kRing) + warp * C::kPart;
    float *last_part = reinterpret_cast<float *>(sbase + warp * C::kRing);
    const int HP = a.Hkv * a.passes;

    if (lane == 0) {
        for (int i = 0; i < S; i++)
            mbar_init(smem_u32(&bar_full[warp][i]), 1);
        fence_barrier_init();
        prefetch_tensormap(&a.tm_k);
        prefetch_tensormap(&a.tm_v);
    }
    if (threadIdx.x < W * 2)
        entry[threadIdx.x >> 1][threadIdx.x & 1].b = -1;
    pdl_launch_dependents();
    pdl_wait();

    auto length = [&](int b) { return min(max(a.lens[b], 0), a.Tmax); };
    auto units_of = [&](int b) { return (length(b) + kUnit - 1) / kUnit; };

    // -------- prefix sums of the units per sequence (of one head and pass) ----
    const int chunk = (a.B + kScan - 1) / kScan;
    {
        int sum = 0;
        if (threadIdx.x < kScan)
            for (int b = threadIdx.x * chunk; b < min(a.B, ((int)threadIdx.x + 1) * chunk); b++)
                sum += units_of(b);
        int inc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off)
                inc += v;
        }
        if (threadIdx.x < kScan && lane == 31)
            scan_tmp[warp] = inc;
        __syncthreads();
        if (threadIdx.x < kScan) {
            int base = 0;
            for (int w = 0; w < warp; w++)
                base += scan_tmp[w];
            pre[threadIdx.x + 1] = base + inc;
            if (threadIdx.x == 0)
                pre[0] = 0;
        }
        __syncthreads();
    }
    const int U = pre[kScan] * HP;
    const int NW = W / a.rg;                          // workers; a worker is rg warps, one per row group
    const int n_act = min((int)gridDim.x, (U + NW - 1) / NW);
    const int cta = blockIdx.x;

    // -------- sequences without positions ----
    for (int b = cta; b < a.B; b += gridDim.x)
        if (length(b) == 0) {
            const size_t n = (size_t)a.R * a.Hkv * D;
            O *o = static_cast<O *>(a.o) + b * n;
            for (size_t i = threadIdx.x * 2; i < n; i += C::kThreads * 2)
                store2(o + i, 0.0f, 0.0f);
        }
    if (cta >= n_act)
        return;
    const int r0 = (int)((long long)cta * U / n_act), r1 = (int)((long long)(cta + 1) * U / n_act);
    const int wk = warp / a.rg, rgi = warp % a.rg;
    const int w0 = r0 + (int)((long long)wk * (r1 - r0) / NW), w1 = r0 + (int)((long long)(wk + 1) * (r1 - r0) / NW);

    auto next_seq = [&](Cursor &c) {                  // the next sequence with units
        c.hp = 0;
        do {
            c.b++;
            c.nu = c.b < a.B ? units_of(c.b) : 1;
        } while (c.nu == 0);
    };
    auto advance = [&](Cursor &c) {
        if (++c.t == c.nu) {
            c.t = 0;
            if (++c.hp == HP)
                next_seq(c);
        }
    };
    Cursor cur = {0, 0, 0, 1};
    if (w0 < w1) {
        // the chunk holding unit w0: the last with pre * HP <= w0
        const unsigned m1 = __ballot_sync(0xffffffffu, (long long)pre[8 * lane] * HP <= w0);
        const int c8 = (31 - __clz(m1)) * 8;
        const unsigned m2 = __ballot_sync(0xffffffffu, lane < 8 && (long long)pre[c8 + (lane & 7)] * HP <= w0);
        const int ci = c8 + 31 - __clz(m2);
        int left = w0 - pre[ci] * HP;
        cur.b = ci * chunk - 1;
        for (next_seq(cur); left >= cur.nu * HP; next_seq(cur))
            left -= cur.nu * HP;
        cur.hp = left / cur.nu;
        cur.t = left % cur.nu;
    }

    // ------------------------------------------------------- the ring ----
    const bool stream_once = a.passes == 1 && a.rg == 1;
    const uint64_t pol = stream_once ? policy_evict_first() : policy_evict_normal();
    Cursor is = cur;
    int issued = 0;
    // row groups past the last row have nothing to do
    auto idle_pass = [&](int hp) { return NT == 2 && (hp % a.passes) * kPassRows + rgi * 16 >= a.R; };
    auto issue = [&]() {                              // lane 0
        const int slot = issued % S;
        const uint32_t bar = smem_u32(&bar_full[warp][slot]), base = ring + slot * C::kSlotBytes;
        const size_t row = ((size_t)is.b * a.Hkv + is.hp / a.passes) * a.Tmax + is.t * kUnit;
        mbar_arrive_expect_tx(bar, C::kSlotBytes);
        tma_load_2d(base, &a.tm_k, bar, 0, (int)row, pol);
        tma_load_2d(base + C::kCodes, &a.tm_v, bar, 0, (int)row, pol);
        bulk_load(base + 2 * C::kCodes, a.ks + row * NB, C::kScales, bar, pol);
        bulk_load(base + 2 * C::kCodes + C::kScales, a.vs + row * NB, C::kScales, bar, pol);
    };
    const int total = w1 - w0;
    for (int k = 0; k < S && issued < total; k++) {
        if (lane == 0)
            issue();
        issued++;
        advance(is);
    }

    // ------------------------------------------------------ the stream ----
    bool ok = true;
    int n = 0;                                        // units consumed
    int u = w0;
    bool any_first = false, any_last = false;
    Entry ent_first, ent_last;
    while (u < w1 && ok) {
        const int sb = cur.b, shp = cur.hp, st0 = cur.t, snu = cur.nu;
        const int ue = min(w1, u + snu - st0);
        const int h = shp / a.passes, row_base = (shp % a.passes) * kPassRows + rgi * 16;
        const int L = length(sb);
        const bool idle = idle_pass(shp);

        // query fragments: block j, half hf (low / high nibbles); rows g (and g + 8)
        uint32_t qf[NT][NB][2][2];
        float mul[NT], koff[NT][NB];
        int lim[NT];                                  // positions row sees
#pragma unroll
        for (int r = 0; r < NT; r++) {
            const int row = row_base + g + 8 * r;
            const bool live = row < a.R;
            const int tok = live ? row / a.G : 0;
            lim[r] = L - (a.Tq - 1 - tok);
            const uint16_t *qp = a.q + (((size_t)sb * a.Tq + tok) * a.Hkv * a.G + (size_t)h * a.G + (live ? row % a.G : 0)) * D;
            uint2 v[NB][2];
            uint32_t mx = 0;
#pragma unroll
            for (int j = 0; j < NB; j++)
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    v[j][hf] = live ? *reinterpret_cast<const uint2 *>(qp + 32 * j + 16 * hf + 4 * t4) : make_uint2(0u, 0u);
                    mx = __vmaxu2(mx, __vmaxu2(v[j][hf].x & 0x7fff7fffu, v[j][hf].y & 0x7fff7fffu));
                }
            mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const int top = (int)max(mx & 0xffffu, mx >> 16);
            // max |q| 2^k in [2^13, 2^14) (exact for subnormal rows too); inf and NaN pass through
            const int k = top == 0 || top >= 0x7c00 ? 0 : 28 - max(top >> 10, 1);
            const float f = pow2i(k);
            mul[r] = a.scale2 * pow2i(24 - k);
#pragma unroll
            for (int j = 0; j < NB; j++) {
                float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    const float fh = hf ? f * 0.0625f : f;
                    // register e holds elements 4 t4 + e and 4 t4 + 2 + e: the order of the masked key bytes
                    qf[r][j][hf][0] = pack_f16x2(f16_lo(v[j][hf].x) * fh, f16_lo(v[j][hf].y) * fh);
                    qf[r][j][hf][1] = pack_f16x2(f16_hi(v[j][hf].x) * fh, f16_hi(v[j][hf].y) * fh);
                    // -8 2^-24 (-128 2^-24) as fp16 subnormals
                    const uint32_t zp = hf ? 0x80808080u : 0x80088008u;
                    mma(z, qf[r][j][hf][0], 0u, qf[r][j][hf][1], 0u, zp, zp);
                }
                koff[r][j] = z[0];
            }
        }
        float m[NT], l[NT], acc[NT][2 * NB][4];
#pragma unroll
        for (int r = 0; r < NT; r++) {
            m[r] = kFloor;
            l[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2 * NB; i++)
                acc[r][i][0] = acc[r][i][1] = acc[r][i][2] = acc[r][i][3] = 0.0f;
        }

        for (; u < ue; u++, n++) {
            const int slot = n % S;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_full[warp][slot]), (n / S) & 1));
            if (!ok)
                break;
            const uint32_t kb = ring + slot * C::kSlotBytes, vb = kb + C::kCodes;
            const uint32_t ksb = kb + 2 * C::kCodes, vsb = ksb + C::kScales;
            const int t0 = cur.t * kUnit;
            if (!idle) {
                // ------------------------------------------ scores ----
                float s[NT][4][2];
#pragma unroll
                for (int nt = 0; nt < 4; nt++) {
                    uint32_t kx[NB];
                    if constexpr (D == 128) {
                        ldsm4(kx, kb + swizzled<D>(8 * nt + (lane & 7), lane >> 3));
                    } else {
                        uint32_t two[4];              // n-tiles nt & ~1 and | 1, blocks 0 and 1
                        ldsm4(two, kb + swizzled<D>(8 * ((nt & ~1) + (lane >> 4)) + (lane & 7), (lane >> 3) & 1));
                        kx[0] = two[2 * (nt & 1)];
                        kx[1] = two[2 * (nt & 1) + 1];
                    }
                    uint32_t w[2][NB / 2];
                    scale_words<NB>(w, ksb + (8 * nt + 2 * t4) * NB * 2);
#pragma unroll
                    for (int r = 0; r < NT; r++)
                        s[r][nt][0] = s[r][nt][1] = 0.0f;
#pragma unroll
                    for (int j = 0; j < NB; j++) {
                        float c[4];
                        c[0] = c[1] = koff[0][j];
                        c[2] = c[3] = NT == 2 ? koff[NT - 1][j] : 0.0f;
                        const uint32_t x = kx[j], y = x >> 8;
                        mma(c, qf[0][j][0][0], NT == 2 ? qf[NT - 1][j][0][0] : 0u, qf[0][j][0][1],
                            NT == 2 ? qf[NT - 1][j][0][1] : 0u, x & 0x000F000Fu, y & 0x000F000Fu);
                        mma(c, qf[0][j][1][0], NT == 2 ? qf[NT - 1][j][1][0] : 0u, qf[0][j][1][1],
                            NT == 2 ? qf[NT - 1][j][1][1] : 0u, x & 0x00F000F0u, y & 0x00F000F0u);
                        const float d0 = j & 1 ? f16_hi(w[0][j >> 1]) : f16_lo(w[0][j >> 1]);
                        const float d1 = j & 1 ? f16_hi(w[1][j >> 1]) : f16_lo(w[1][j >> 1]);
#pragma unroll
                        for (int r = 0; r < NT; r++) {
                            s[r][nt][0] = fmaf(d0, c[2 * r], s[r][nt][0]);
                            s[r][nt][1] = fmaf(d1, c[2 * r + 1], s[r][nt][1]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < NT; r++) {
                        s[r][nt][0] *= mul[r];
                        s[r][nt][1] *= mul[r];
                    }
                }
                // ------------------------------------ value scales ----
                const bool edge = t0 + kUnit > L - (a.Tq - 1);    // some row's positions end in this unit
                uint32_t vw[4][2][NB / 2];
                uint32_t mxw = 0;
#pragma unroll
                for (int nt = 0; nt < 4; nt++) {
                    scale_words<NB>(vw[nt], vsb + (8 * nt + 2 * t4) * NB * 2);
                    if (edge) {
                        const int p = t0 + 8 * nt + 2 * t4;
#pragma unroll
                        for (int e = 0; e < 2; e++) {
#pragma unroll
                            for (int i = 0; i < NB / 2; i++)
                                vw[nt][e][i] = p + e < L ? vw[nt][e][i] : 0u;
#pragma unroll
                            for (int r = 0; r < NT; r++)
                                s[r][nt][e] = p + e < lim[r] ? s[r][nt][e] : -INFINITY;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; e++)
#pragma unroll
                        for (int i = 0; i < NB / 2; i++)
                            mxw = __vmaxu2(mxw, vw[nt][e][i]);
                }
                // --------------------------------- running reference ----
                // the lane's bound on log2(dV), and per row on s + log2(dV) - kBase
                const float eb = fmaf((float)max(mxw & 0x7fffu, (mxw >> 16) & 0x7fffu), 0x1p-10f, -15.0f - kBase);
                bool grow = false;
                float cand[NT];
#pragma unroll
                for (int r = 0; r < NT; r++) {
                    float mx = s[r][0][0];
#pragma unroll
                    for (int i = 1; i < 8; i++)
                        mx = fmaxf(mx, s[r][i >> 1][i & 1]);
                    mx = __fadd_ru(mx, eb);           // (rounded up: scores of any size keep p dV in range)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    cand[r] = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    grow = grow || cand[r] - m[r] > kSlack;
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int r = 0; r < NT; r++) {
                        const float mn = fmaxf(m[r], cand[r]);
                        const float f = ex2(m[r] - mn);
                        m[r] = mn;
                        l[r] *= f;
                        // accumulator columns are rows 2 t4 and 2 t4 + 1 of the tile
                        const float f0 = __shfl_sync(0xffffffffu, f, 8 * t4), f1 = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
#pragma unroll
                        for (int i = 0; i < 2 * NB; i++) {
                            acc[r][i][0] *= f0;
                            acc[r][i][1] *= f1;
                            acc[r][i][2] *= f0;
                            acc[r][i][3] *= f1;
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < NT; r++)
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        float &p = s[r][i >> 1][i & 1];
                        p = ex2(p - m[r]);
                        l[r] += p;
                    }
                // ------------------------------------------ values ----
#pragma unroll
                for (int k = 0; k < 2; k++) {         // 16 positions
#pragma unroll
                    for (int j2 = 0; j2 < NB / 2; j2++) {
                        uint32_t x[4];                // block 2 j2: positions 0-7, 8-15; block 2 j2 + 1
                        ldsm4t(x, vb + swizzled<D>(16 * k + (lane & 15), 2 * j2 + (lane >> 4)));
#pragma unroll
                        for (int jj = 0; jj < 2; jj++) {
                            const int j = 2 * j2 + jj;
                            uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
                            for (int hf = 0; hf < 2; hf++) {
                                const uint32_t w0 = vw[2 * k + hf][0][j2], w1 = vw[2 * k + hf][1][j2];
                                const float d0 = jj ? f16_hi(w0) : f16_lo(w0), d1 = jj ? f16_hi(w1) : f16_lo(w1);
#pragma unroll
                                for (int r = 0; r < NT; r++) {
                                    const float p0 = s[r][2 * k + hf][0] * d0, p1 = s[r][2 * k + hf][1] * d1;
                                    bh[r][hf] = pack_f16x2(p0, p1);
                                    if constexpr (kTwo)
                                        bl[r][hf] = pack_f16x2(p0 - f16_lo(bh[r][hf]), p1 - f16_hi(bh[r][hf]));
                                }
                            }
                            const uint32_t x0 = x[2 * jj], x1 = x[2 * jj + 1], y0 = x0 >> 8, y1 = x1 >> 8;
                            const uint32_t e0 = nib_lo(x0), e1 = nib_hi(x0), e2 = nib_lo(x1), e3 = nib_hi(x1);
                            const uint32_t f0 = nib_lo(y0), f1 = nib_hi(y0), f2 = nib_lo(y1), f3 = nib_hi(y1);
#pragma unroll
                            for (int r = 0; r < NT; r++) {
                                mma(acc[r][2 * j], e0, e1, e2, e3, bh[r][0], bh[r][1]);
                                mma(acc[r][2 * j + 1], f0, f1, f2, f3, bh[r][0], bh[r][1]);
                                if constexpr (kTwo) {
                                    mma(acc[r][2 * j], e0, e1, e2, e3, bl[r][0], bl[r][1]);
                                    mma(acc[r][2 * j + 1], f0, f1, f2, f3, bl[r][0], bl[r][1]);
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (issued < total) {                     // refill the slot just read
                if (lane == 0)
                    issue();
                issued++;
                advance(is);
            }
            cur.t++;
        }
        if (!ok)
            break;
        // ---------------------------------------------- segment's end ----
#pragma unroll
        for (int r = 0; r < NT; r++) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
        const bool before = st0 > 0, after = st0 + (ue - (u - (cur.t - st0))) < snu;
        if (!before && !after) {
            if (!idle) {
#pragma unroll
                for (int r = 0; r < NT; r++) {
                    const float inv = l[r] > 0.0f ? 1.0f / l[r] : 0.0f;
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        const float fi = __shfl_sync(0xffffffffu, inv, 8 * t4 + 4 * c);
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
            }
        } else {
            // a segment that began before this share goes to the warp's first
            // slot; one that only continues after it is the share's last, and
            // the ring is drained
            float *pp = before ? first_part : last_part;
            const Entry e = {sb, shp, u - (cur.t - st0) - st0, snu};
            if (before) {
                ent_first = e;
                any_first = true;
            } else {
                ent_last = e;
                any_last = true;
            }
#pragma unroll
            for (int r = 0; r < NT; r++) {
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    float *o = pp + (8 * r + 2 * t4 + c) * C::kLd;
#pragma unroll
                    for (int j = 0; j < NB; j++) {
                        *reinterpret_cast<float2 *>(o + 32 * j + 2 * g) = make_float2(acc[r][2 * j][c], acc[r][2 * j + 1][c]);
                        *reinterpret_cast<float2 *>(o + 32 * j + 16 + 2 * g) = make_float2(acc[r][2 * j][c + 2], acc[r][2 * j + 1][c + 2]);
                    }
                }
                if (t4 == 0) {
                    pp[C::kRows * C::kLd + 8 * r + g] = m[r];
                    pp[C::kRows * C::kLd + C::kRows + 8 * r + g] = l[r];
                }
            }
        }
        // the next segment
        cur.t = 0;
        if (!after && ++cur.hp == HP)
            next_seq(cur);
    }
    if (!ok) {                                        // copies in flight land before the CTA ends
        if (lane == 0 && a.status)
            atomicOr(a.status, kStatusTimeout);
        for (int i = n; i < issued; i++)
            (void)mbar_wait_bounded(smem_u32(&bar_full[warp][i % S]), (i / S) & 1);
    }
    if (lane == 0 && rgi == 0) {
        if (any_first)
            entry[wk][0] = ent_first;
        if (any_last)
            entry[wk][1] = ent_last;
    }
    __syncthreads();

    // ------------------------------------------------ merge the workers ----
    const int rows_cta = C::kRows * a.rg;             // rows of a pass
    const size_t gp = (size_t)rows_cta * (D + 2);     // floats of a CTA partial
    auto out_row = [&](const Entry &e, int row) {     // output of a pass's row (row < R checked by the caller)
        const int rr = (e.hp % a.passes) * kPassRows + row;
        return static_cast<O *>(a.o) +
               (((size_t)e.b * a.Tq + rr / a.G) * a.Hkv * a.G + (size_t)(e.hp / a.passes) * a.G + rr % a.G) * D;
    };
    auto live_rows = [&](const Entry &e) { return min(rows_cta, a.R - (e.hp % a.passes) * kPassRows); };
    Entry shared_seg[2];
    int n_shared = 0;
    for (int i = 0; i < 2 * NW;) {
        const Entry e = entry[i >> 1][i & 1];
        if (e.b < 0) {
            i++;
            continue;
        }
        int last = i;
        for (int k = i + 1; k < 2 * NW; k++) {
            const Entry f = entry[k >> 1][k & 1];
            if (f.b < 0)
                continue;
            if (f.b != e.b || f.hp != e.hp)
                break;
            last = k;
        }
        const bool whole = e.first >= r0 && e.first + e.units <= r1;
        const int gslot = e.first < r0 ? 0 : 1;
        float *gpart = a.partials + ((size_t)cta * 2 + gslot) * gp;
        const int rows = live_rows(e);
        for (int it = threadIdx.x; it < rows * (D / 2); it += C::kThreads) {
            const int row = it / (D / 2), d = it % (D / 2) * 2;
            const int rq = row / C::kRows, rr = row % C::kRows;
            float M = kFloor, Ls = 0.0f, o0 = 0.0f, o1 = 0.0f;
            for (int k = i; k <= last; k++) {
                if (entry[k >> 1][k & 1].b < 0)
                    continue;
                const int w = (k >> 1) * a.rg + rq;
                const float *pp = (k & 1) ? reinterpret_cast<const float *>(sbase + w * C::kRing)
                                          : reinterpret_cast<const float *>(sbase + W * C::kRing) + w * C::kPart;
                const float mk = pp[C::kRows * C::kLd + rr], lk = pp[C::kRows * C::kLd + C::kRows + rr];
                const float2 ok2 = *reinterpret_cast<const float2 *>(pp + rr * C::kLd + d);
                const float Mn = fmaxf(M, mk), fo = ex2(M - Mn), fk = ex2(mk - Mn);
                M = Mn;
                Ls = Ls * fo + lk * fk;
                o0 = o0 * fo + ok2.x * fk;
                o1 = o1 * fo + ok2.y * fk;
            }
            if (whole) {
                const float inv = Ls > 0.0f ? 1.0f / Ls : 0.0f;
                store2(out_row(e, row) + d, o0 * inv, o1 * inv);
            } else {
                __stcg(reinterpret_cast<float2 *>(gpart + (size_t)row * D + d), make_float2(o0, o1));
                if (d == 0) {
                    __stcg(gpart + (size_t)rows_cta * D + row, M);
                    __stcg(gpart + (size_t)rows_cta * (D + 1) + row, Ls);
                }
            }
        }
        if (!whole && n_shared < 2)
            shared_seg[n_shared++] = e;
        i = last + 1;
    }
    if (n_shared == 0)
        return;

    // --------------------------------------------------- merge the CTAs ----
    __threadfence();
    __syncthreads();
    if (threadIdx.x < n_shared) {
        const Entry e = threadIdx.x == 0 ? shared_seg[0] : shared_seg[1];
        const int cf = owner_of(e.first, U, n_act), cl = owner_of(e.first + e.units - 1, U, n_act);
        arrived[threadIdx.x] = atom_add_acq_rel_gpu(a.counters + cf, 1) == cl - cf;
    }
    __syncthreads();
    for (int k = 0; k < n_shared; k++) {
        if (!arrived[k])
            continue;
        __threadfence();
        const Entry e = k == 0 ? shared_seg[0] : shared_seg[1];
        const int cf = owner_of(e.first, U, n_act), cl = owner_of(e.first + e.units - 1, U, n_act);
        // the segment starts inside cf (its second slot) and before every later CTA (their first)
        auto part = [&](int c) { return a.partials + ((size_t)c * 2 + (c == cf ? 1 : 0)) * gp; };
        const int rows = live_rows(e);
        for (int it = threadIdx.x; it < rows * (D / 2); it += C::kThreads) {
            const int row = it / (D / 2), d = it % (D / 2) * 2;
            float M = kFloor, Ls = 0.0f, o0 = 0.0f, o1 = 0.0f;
            for (int c0 = cf; c0 <= cl; c0 += 8) {    // 8 partials' loads in flight
                float mc[8], lc[8];
                float2 oc[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const bool in = c0 + i <= cl;
                    const float *pc = part(in ? c0 + i : cf);
                    mc[i] = in ? __ldcg(pc + (size_t)rows_cta * D + row) : kFloor;
                    lc[i] = in ? __ldcg(pc + (size_t)rows_cta * (D + 1) + row) : 0.0f;
                    oc[i] = in ? __ldcg(reinterpret_cast<const float2 *>(pc + (size_t)row * D + d)) : make_float2(0.f, 0.f);
                }
                float Mn = M;
#pragma unroll
                for (int i = 0; i < 8; i++)
                    Mn = fmaxf(Mn, mc[i]);
                const float fo = ex2(M - Mn);
                M = Mn;
                Ls *= fo;
                o0 *= fo;
                o1 *= fo;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float f = ex2(mc[i] - Mn);
                    Ls = fmaf(f, lc[i], Ls);
                    o0 = fmaf(f, oc[i].x, o0);
                    o1 = fmaf(f, oc[i].y, o1);
                }
            }
            const float inv = Ls > 0.0f ? 1.0f / Ls : 0.0f;
            store2(out_row(e, row) + d, o0 * inv, o1 * inv);
        }
        __syncthreads();                              // every partial is read: leave the workspace zero
        for (int c = cf; c <= cl; c++) {
            float *pc = part(c);
            for (size_t i = threadIdx.x * 2; i < gp; i += C::kThreads * 2)
                __stcg(reinterpret_cast<float2 *>(pc + i), make_float2(0.f, 0.f));
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

// Rows of a CTA partial.
int part_rows(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : R <= 32 ? 32 : kPassRows; }

}  // namespace aq
}  // namespace bq

using namespace bq;

extern "C" size_t bq_attn_q4_workspace_bytes(int32_t D, int32_t Tq, int32_t G)
{
    if ((D != 64 && D != 128) || Tq < 1 || Tq > 32 || G < 1 || G > 16)
        return 0;
    return aq::kMaxGrid * sizeof(int) + (size_t)aq::kMaxGrid * 2 * aq::part_rows(Tq * G) * (D + 2) * sizeof(float);
}

extern "C" int32_t bq_attn_decode_q4(const bq_kv_cache_q4 *kv, const uint16_t *q, const int32_t *lens,
                                     int32_t B, int32_t Tq, int32_t Hkv, int32_t G, float scale, void *o,
                                     int32_t o_dtype, void *ws, size_t ws_bytes, int32_t *dev_status,
                                     void *stream)
{
    if (!kv || !kv->k_codes || !kv->k_scales || !kv->v_codes || !kv->v_scales || !q || !lens || !o || !ws)
        return BQ_ERR_NULL;
    const size_t need = bq_attn_q4_workspace_bytes(kv->D, Tq, G);
    // (|scale| <= 1e18 keeps scale log2(e) 2^26 and every score finite)
    if (need == 0 || kv->Tmax < 32 || kv->Tmax % 32 != 0 || Hkv < 1 || !(std::fabs(scale) <= 1e18f) ||
        (o_dtype != BQ_F32 && o_dtype != BQ_F16))
        return BQ_ERR_SHAPE;
    if (B < 1)
        return BQ_ERR_BATCH;
    const long long rows = (long long)B * Hkv < (1LL << 31) ? (long long)B * Hkv * kv->Tmax : 1LL << 31;
    const int R = Tq * G;
    const int passes = (R + aq::kPassRows - 1) / aq::kPassRows;
    // positions, and units of all passes, are 32-bit numbers
    if (rows >= (1LL << 31) || rows / 32 * passes >= (1LL << 31))
        return BQ_ERR_SHAPE;
    if (!aligned16(kv->k_codes) || !aligned16(kv->k_scales) || !aligned16(kv->v_codes) ||
        !aligned16(kv->v_scales) || !aligned16(q) || !aligned16(o) || !aligned16(ws) ||
        (reinterpret_cast<uintptr_t>(lens) & 3u))
        return BQ_ERR_ALIGN;
    if (ws_bytes < need)
        return BQ_ERR_WORKSPACE;
    const int sms = device_sm_count();
    if (sms <= 0)
        return BQ_ERR_CUDA;
    aq::Args a;
    memset(&a, 0, sizeof(a));
    const uint64_t dims[2] = {(uint64_t)kv->D / 2, (uint64_t)rows}, stride[1] = {(uint64_t)kv->D / 2};
    const uint32_t box[2] = {(uint32_t)kv->D / 2, (uint32_t)aq::kUnit};
    const CUtensorMapSwizzle sw = kv->D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
    if (!encode_tensor_map(&a.tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, kv->k_codes, dims, stride, box, sw,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
        !encode_tensor_map(&a.tm_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, kv->v_codes, dims, stride, box, sw,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
        return BQ_ERR_CUDA;
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
    a.rg = R <= 16 ? 1 : R <= 32 ? 2 : 4;
    a.passes = passes;
    a.scale2 = scale * 1.4426950408889634f;
    a.counters = static_cast<int *>(ws);
    a.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + aq::kMaxGrid * sizeof(int));
    a.status = dev_status;
    const int grid = sms < aq::kMaxGrid ? sms : aq::kMaxGrid;
    const bool f16 = o_dtype == BQ_F16;
    if (kv->D == 128) {
        if (R <= 8)
            return f16 ? aq::launch<128, 1, __half>(a, grid, stream) : aq::launch<128, 1, float>(a, grid, stream);
        return f16 ? aq::launch<128, 2, __half>(a, grid, stream) : aq::launch<128, 2, float>(a, grid, stream);
    }
    if (R <= 8)
        return f16 ? aq::launch<64, 1, __half>(a, grid, stream) : aq::launch<64, 1, float>(a, grid, stream);
    return f16 ? aq::launch<64, 2, __half>(a, grid, stream) : aq::launch<64, 2, float>(a, grid, stream);
}
