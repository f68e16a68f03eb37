// Rows in 8 bits: as they are, after a root-mean-square norm of x + residual, or
// after the norm of each head times silu(gate).
//
//   PLAIN  y = x
//   NORM   h = x + residual,  y = h rsqrt(mean h^2 + eps) w
//   GATED  y = x rsqrt(mean over the head of x^2 + eps) w gate / (1 + e^-gate)
//   scale = max|y| / 127,  q = rint(127 y / max|y|)
//
// Bound by memory: a row is read once, stays in registers (8 V numbers a thread)
// while its statistics go round the row's threads, and is written once.  The
// largest |h w| is found beside the sum of squares, since the norm's factor is
// positive and the same for the whole row, so NORM too has one exchange (a second one
// where the squares pass fp32).  Beside the bytes the instructions count (bf16 rows
// leave about 20 a number): everything is loaded before anything is waited for,
// products and sums go two in an instruction, and steps come from an fma instead of a
// conversion.
//
// Measured, of the copy rate: NORM of 8192 x 4096 bf16 with an fp32 residual 58 us
// (98%); PLAIN of 8224 x 2048 bf16 8.3 us (93%); GATED of 16384 rows of 16 heads of
// 128 32 us (79%: an exponential and a reciprocal a number, 3.0 instructions a cycle).
#include <cuda_bf16.h>

#include <type_traits>

#include "f32x2.cuh"
#include "gdn_serve.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

constexpr unsigned kInfBits = 0x7f800000u;

template <typename T>
struct Words {                           // 8 numbers as 32-bit words
    static constexpr int kCount = 2 * sizeof(T);
};

// 8 numbers from words, as pairs.
template <typename T>
__device__ __forceinline__ void widen(const uint32_t (&w)[Words<T>::kCount], F2 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) x[i] = pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else x[i] = pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
}
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// Numbers i .. i + 7 of a row of `width` (0 behind its end; i is below it).
// VEC: the row lies on 16 bytes and holds whole eights.  Else from the aligned 16-byte
// pieces that hold them, where those lie in the row: what a row is off by is the same
// for all its threads, so that the shift of the words is a few selects; the row's
// ends, one by one.
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T *row, int i, int width, uint32_t (&w)[Words<T>::kCount]) {
    constexpr int kW = Words<T>::kCount;
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + i);
    if constexpr (VEC) {
#pragma unroll
        for (int v = 0; v < kW / 4; ++v) {
            const uint4 y = __ldcs(reinterpret_cast<const uint4 *>(at) + v);
            w[4 * v] = y.x; w[4 * v + 1] = y.y; w[4 * v + 2] = y.z; w[4 * v + 3] = y.w;
        }
        return;
    }
    const uintptr_t from = at & ~(uintptr_t)15, off = at & 15;
    const uintptr_t need = from + (off ? 4 * kW + 16 : 4 * kW);
    if (from >= reinterpret_cast<uintptr_t>(row) && need <= reinterpret_cast<uintptr_t>(row + width)) {
        uint32_t y[kW + 4];
#pragma unroll
        for (int v = 0; v < kW / 4 + 1; ++v) {
            uint4 z = make_uint4(0, 0, 0, 0);
            if (v < kW / 4 || off) z = plain(reinterpret_cast<const uint4 *>(from) + v);
            y[4 * v] = z.x; y[4 * v + 1] = z.y; y[4 * v + 2] = z.z; y[4 * v + 3] = z.w;
        }
        if (off & 8) {
#pragma unroll
            for (int k = 0; k < kW + 2; ++k) y[k] = y[k + 2];
        }
        if (off & 4) {
#pragma unroll
            for (int k = 0; k < kW + 1; ++k) y[k] = y[k + 1];
        }
#pragma unroll
        for (int k = 0; k < kW; ++k) w[k] = sizeof(T) == 2 && (off & 2) ? __funnelshift_r(y[k], y[k + 1], 16) : y[k];
    } else {
#pragma unroll
        for (int k = 0; k < kW; ++k) w[k] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i + e < width) {
                if constexpr (sizeof(T) == 4) w[e] = reinterpret_cast<const uint32_t *>(row)[i + e];
                else w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(row)[i + e] << (16 * (e & 1));
            }
    }
}
template <int N>
__device__ __forceinline__ void zero(uint32_t (&w)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = 0;
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T *row, int i, int width, const F2 (&pairs)[4]) {
    uint32_t w[Words<T>::kCount];
    float x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) unpack(pairs[k], &x[2 * k], &x[2 * k + 1]);
#pragma unroll
    for (int k = 0; k < Words<T>::kCount; ++k) {
        if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(x[k]);
        else {
            const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t *>(&y);
        }
    }
    if constexpr (VEC) {
#pragma unroll
        for (int v = 0; v < Words<T>::kCount / 4; ++v)
            __stcs(reinterpret_cast<uint4 *>(row + i) + v, make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]));
        return;
    }
    // the widest stores that the row's address allows (the same for all its threads)
    constexpr int kW = Words<T>::kCount;
    T *to = row + i;
    const unsigned off = (unsigned)(reinterpret_cast<uintptr_t>(to) & 15);
    if (i + 8 > width) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i + e < width) put(to + e, x[e]);
    } else if (off == 0) {
#pragma unroll
        for (int k = 0; k < kW; k += 4) reinterpret_cast<uint4 *>(to)[k / 4] = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
    } else if (off == 8) {
#pragma unroll
        for (int k = 0; k < kW; k += 2) reinterpret_cast<uint2 *>(to)[k / 2] = make_uint2(w[k], w[k + 1]);
    } else if (off % 4 == 0) {
#pragma unroll
        for (int k = 0; k < kW; ++k) reinterpret_cast<uint32_t *>(to)[k] = w[k];
    } else {                             // bf16 on 2 bytes: words of an odd number and the one behind it
        put(to, x[0]);
#pragma unroll
        for (int k = 0; k + 1 < kW; ++k) reinterpret_cast<uint32_t *>(to + 1)[k] = __funnelshift_r(w[k], w[k + 1], 16);
        put(to + 7, x[7]);
    }
}

// Weights i .. i + 7 (0 behind the end).
template <bool VEC, typename T>
__device__ __forceinline__ void weight8(const T *weight, int i, int width, bool vec, uint32_t (&w)[Words<T>::kCount]) {
    if (VEC || (vec && i + 8 <= width)) {
#pragma unroll
        for (int v = 0; v < Words<T>::kCount / 4; ++v) {
            const uint4 y = plain(reinterpret_cast<const uint4 *>(weight + i) + v);
            w[4 * v] = y.x; w[4 * v + 1] = y.y; w[4 * v + 2] = y.z; w[4 * v + 3] = y.w;
        }
    } else {
        load8<false>(weight, i, width, w);
    }
}

// max(top, |x|) of 8 numbers, NaN if any is.
__device__ __forceinline__ float top_of(float top, const F2 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack(x[i], &lo, &hi);
        asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(lo), "f"(hi));
    }
    return top;
}

// 1 / x to an ulp or two, for normal x whose reciprocal is normal.
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLeast = 127 * 0x1p-126f;            // the largest of a row with the least scale
__device__ __forceinline__ bool fits(float x) { return x < __uint_as_float(kInfBits); }

// Quotients, by Markstein's correction q + (a - q b) r of an approximate one, with r about 1 / b
// ("Computation of elementary functions on the IBM RISC System/6000 processor", 1990): three
// instructions, where a division by its operator cost plain rows of 8192 x 8192 5 us of 32.
//
// The row's scale, top / 127: r is 1 / 127 rounded correctly, so the quotient is too.
__device__ __forceinline__ float scale_of(float top) {
    if (!fits(top)) return __uint_as_float(0x7fc00000u);
    const float r = 1.f / 127.f, q = top * r;
    return top < kLeast ? 0.f : fmaf(fmaf(-q, 127.f, top), r, q);
}
// The factor from numbers to steps, 127 / top rounded up (0 where the row has none), and what it
// is more than the quotient; with a sixteenth of both, which keeps the reciprocal normal for tops
// from kLeast to 3.4e38.
struct Factor { float f, over; };
__device__ __forceinline__ Factor steps_of(float top) {
    if (!(top >= kLeast) || !fits(top)) return {0.f, 0.f};
    const float t = top * 0.0625f, r = rcp(t), q = 7.9375f * r;
    float f = fmaf(fmaf(-q, t, 7.9375f), r, q);
    if (fmaf(-f, t, 7.9375f) > 0.f) f = __uint_as_float(__float_as_uint(f) + 1);
    return {f, fmaf(f, t, -7.9375f) * r};
}

// Steps of 8 numbers.  y f + 1.5 2^23 has rint(y f) in its low bits (|y f| <= 127 and little
// more): a sum in place of a conversion, which has a quarter of the rate, and one rounding for
// both.  In a row of bf16 the numbers of half the largest are ties, 63.5 steps, which go to 64:
// so they do with an f that is the quotient or above it, and no other number of such a row is
// so close to a tie that an f off by two units moves it (tried for every pair of significands;
// rounded to nearest, f took one tie in twelve to 63).
// EXACT, for rows of fp32, whose bytes leave the time for it: y (f - over), rounded, and then to a
// whole number.
template <bool VEC, bool EXACT>
__device__ __forceinline__ void store_steps8(int8_t *row, int i, int width, const F2 (&y)[4], Factor f, bool on8) {
    uint32_t b[8];
    const F2 ff = pack(f.f, f.f), over = pack(-f.over, -f.over), magic = pack(12582912.f, 12582912.f);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float lo, hi;
        if constexpr (EXACT) unpack(add2(fma2(y[e / 2], ff, mul2(y[e / 2], over)), magic), &lo, &hi);
        else unpack(fma2(y[e / 2], ff, magic), &lo, &hi);
        b[e] = __float_as_uint(lo);
        b[e + 1] = __float_as_uint(hi);
    }
    uint2 v;
    v.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    v.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    if (VEC || (on8 && i + 8 <= width)) {
        *reinterpret_cast<uint2 *>(row + i) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (i + e < width) row[i + e] = (int8_t)b[e];
    }
}
// A row without steps: zeros, also where it holds what is not finite.
template <int V>
__device__ __forceinline__ void clear(F2 (&y)[V][4]) {
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[j][e] = pack(0.f, 0.f);
}
__device__ __forceinline__ float squares(const F2 (&x)[4]) {
    F2 sum = mul2(x[0], x[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) sum = fma2(x[e], x[e], sum);
    return both(sum);
}
__device__ __forceinline__ void times(F2 (&x)[4], const F2 (&y)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = mul2(x[e], y[e]);
}
__device__ __forceinline__ void times(F2 (&x)[4], float y) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = mul2(x[e], pack(y, y));
}

// Squares of numbers from about 2^62 on leave fp32 in a row's sum.  Beside each sum of squares
// goes the sum of the squares of 2^-72 h, which holds any row (2^15 squares below 2^112) and is
// read only where the first is infinite: it is then at least 2^-16, and what the multiple below
// 2^-126 loses does not count.
constexpr float kSmall = 0x1p-72f, kSmall2 = 0x1p-144f;
__device__ __forceinline__ float small_squares(const F2 (&x)[4]) {
    F2 y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = mul2(x[e], pack(kSmall, kSmall));
    return squares(y);
}

// Sum and largest over the row's threads (blockDim.x of them, whole warps).  As whole
// numbers, values from 0 up order like themselves, with NaN above infinity.
struct Totals { float sum, top; };
template <bool SUM>
__device__ __forceinline__ Totals row_totals(float sum, float top_value) {
    __shared__ float sums[32];
    __shared__ unsigned tops[32];
    unsigned top = __reduce_max_sync(~0u, __float_as_uint(top_value));
    if (SUM)
#pragma unroll
        for (int m = 16; m; m /= 2) sum += __shfl_xor_sync(~0u, sum, m);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return {sum, __uint_as_float(top)};
    const int first = threadIdx.y * warps, lane = threadIdx.x & 31;
    if (lane == 0) {
        if (SUM) sums[first + (threadIdx.x >> 5)] = sum;
        tops[first + (threadIdx.x >> 5)] = top;
    }
    __syncthreads();
    top = __reduce_max_sync(~0u, lane < warps ? tops[first + lane] : 0u);
    if (SUM) {
        sum = lane < warps ? sums[first + lane] : 0.f;
#pragma unroll
        for (int m = 16; m; m /= 2) sum += __shfl_xor_sync(~0u, sum, m);
    }
    return {sum, __uint_as_float(top)};
}

// The sum alone, for a row whose sum of squares does not fit: its warps meet at a barrier of
// their own (the block's other rows may not come here).
__device__ __forceinline__ float row_sum(float sum) {
    __shared__ float sums[32];
#pragma unroll
    for (int m = 16; m; m /= 2) sum += __shfl_xor_sync(~0u, sum, m);
    const int warps = blockDim.x >> 5, first = threadIdx.y * warps, lane = threadIdx.x & 31;
    if (warps == 1) return sum;
    if (lane == 0) sums[first + (threadIdx.x >> 5)] = sum;
    sm100::named_bar(1 + threadIdx.y, blockDim.x);
    sum = lane < warps ? sums[first + lane] : 0.f;
#pragma unroll
    for (int m = 16; m; m /= 2) sum += __shfl_xor_sync(~0u, sum, m);
    return sum;
}

// PLAIN and NORM.  XT: type of x.  RT: type of the residual, or void for none.
// Thread i takes the eights i, i + blockDim.x, ... of its row.
template <bool NORM, typename XT, typename RT, typename WT, int V, int MOST, bool VEC>
__global__ void __launch_bounds__(MOST) rows_kernel(const RowsParams p) {
    if (p.early) { grid_next(); grid_wait(); }
    constexpr bool RES = !std::is_void<RT>::value;
    using R1 = typename std::conditional<RES, RT, float>::type;
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;      // (past 2^31 in the last block of as many)
    const int width = row < p.rows ? p.width : 0;
    const int64_t r = row < p.rows ? row : 0;
    const XT *x = reinterpret_cast<const XT *>(p.x) + r * p.x_row;
    const R1 *res = reinterpret_cast<const R1 *>(p.residual) + r * p.residual_row;
    auto at = [&](int j) { return (int)(threadIdx.x + j * blockDim.x) * 8; };
    // everything that is read, before anything waits for it
    uint32_t xw[V][Words<XT>::kCount], rw[V][Words<R1>::kCount], ww[V][Words<WT>::kCount];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        zero(xw[j]); zero(rw[j]); zero(ww[j]);
        if (at(j) < width) {
            load8<VEC>(x, at(j), width, xw[j]);
            if constexpr (RES) load8<VEC>(res, at(j), width, rw[j]);
            if (NORM && p.weight) weight8<VEC>(reinterpret_cast<const WT *>(p.weight), at(j), width, p.weight_vec, ww[j]);
        }
    }
    // in place and off 16 bytes a thread's pieces hold neighbours' numbers too, which it drops:
    // all of a row's loads come before its stores (4096 x 5001 in place 52.8 us, 48.0 without)
    if (RES && !VEC && p.in_place) __syncthreads();
    F2 h[V][4];
    float sum = 0.f, small = 0.f, top = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        widen<XT>(xw[j], h[j]);
        if constexpr (RES) {
            F2 b[4];
            widen<R1>(rw[j], b);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[j][e] = add2(h[j][e], b[e]);
            if (at(j) < width)
                store8<VEC>(reinterpret_cast<R1 *>(p.residual_out) + r * p.residual_out_row, at(j), width, h[j]);
        }
        if (NORM) sum += squares(h[j]);
    }
    if constexpr (NORM) {
        small = sum * kSmall2;
        if (!fits(sum)) {
            small = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) small += small_squares(h[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (NORM && p.weight) {
            F2 w[4];
            widen<WT>(ww[j], w);
            times(h[j], w);
        }
        top = top_of(top, h[j]);
    }
    const Totals t = row_totals<NORM>(sum, top);
    if (!width) return;
    // y f = (h w) 127 / max|h w|: the norm's factor is the whole row's.  It makes the largest y
    // of the largest h w.
    Factor f = steps_of(t.top);
    float most = t.top;
    if constexpr (NORM) {
        float norm = rsqrtf(fmaf(t.sum, p.inverse, p.eps));
        most *= norm;
        if (!fits(t.sum)) {              // (of a row that is not finite too: NaN, or infinity times 0)
            norm = rsqrtf(fmaf(row_sum(small), p.inverse, p.eps * kSmall2));
            most = t.top * 0x1p-36f * norm * 0x1p-36f;
        }
        if (t.top < kLeast) {            // h w far below the normal numbers: the norm may lift it back
            f = steps_of(most);
#pragma unroll
            for (int j = 0; j < V; ++j) times(h[j], norm);
        }
        if (!(most >= kLeast) || !fits(most)) f.f = 0.f;
    }
    if (threadIdx.x == 0) p.scale[r] = scale_of(most);
    if (f.f == 0.f) clear(h);
    int8_t *q = p.q + r * p.q_row;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (at(j) < width) store_steps8<VEC, !NORM && sizeof(XT) == 4>(q, at(j), width, h[j], f, p.q_vec);
}

// GATED.  `lanes` (a power of two, 8 channels each) threads take a head, idle
// where the head has fewer channels; a thread's V heads are blockDim.x / lanes
// apart.
template <typename XT, int V, int MOST, bool VEC>
__global__ void __launch_bounds__(MOST) gated_kernel(const RowsParams p, int lanes_log2, int heads) {
    if (p.early) { grid_next(); grid_wait(); }
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool on = row < p.rows;
    const int64_t r = on ? row : 0;
    const XT *x = reinterpret_cast<const XT *>(p.x) + r * p.x_row;
    const XT *g = reinterpret_cast<const XT *>(p.gate) + r * p.gate_row;
    const int lanes = 1 << lanes_log2, part = (threadIdx.x & (lanes - 1)) * 8;
    const int head0 = threadIdx.x >> lanes_log2, step = blockDim.x >> lanes_log2;
    const bool mine = on && part < p.head;
    auto at = [&](int j) { return (head0 + j * step) * p.head + part; };
    auto has = [&](int j) { return mine && head0 + j * step < heads; };
    uint32_t xw[V][Words<XT>::kCount], gw[V][Words<XT>::kCount];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        zero(xw[j]); zero(gw[j]);
        if (has(j)) {
            load8<VEC>(x, at(j), p.width, xw[j]);
            load8<VEC>(g, at(j), p.width, gw[j]);
        }
    }
    F2 w[4] = {pack(1.f, 1.f), pack(1.f, 1.f), pack(1.f, 1.f), pack(1.f, 1.f)};
    if (p.weight && part < p.head) {
        if (p.weight_bf16) {
            uint32_t ww[4];
            weight8<VEC>(reinterpret_cast<const __nv_bfloat16 *>(p.weight), part, p.head, p.weight_vec, ww);
            widen<__nv_bfloat16>(ww, w);
        } else {
            uint32_t ww[8];
            weight8<VEC>(reinterpret_cast<const float *>(p.weight), part, p.head, p.weight_vec, ww);
            widen<float>(ww, w);
        }
    }
    times(w, 0x1p-12f);
    F2 y[V][4];
    float norm[V], top = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        widen<XT>(xw[j], y[j]);
        norm[j] = squares(y[j]);
    }
#pragma unroll
    for (int m = 16; m; m /= 2)
        if (m < lanes)
#pragma unroll
            for (int j = 0; j < V; ++j) norm[j] += __shfl_xor_sync(~0u, norm[j], m);
    float all = norm[0];
#pragma unroll
    for (int j = 1; j < V; ++j) all += norm[j];
    if (__any_sync(~0u, !fits(all))) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float small = small_squares(y[j]);
#pragma unroll
            for (int m = 16; m; m /= 2)
                if (m < lanes) small += __shfl_xor_sync(~0u, small, m);
            const bool big = !fits(norm[j]);
            norm[j] = big ? rsqrtf(fmaf(small, p.inverse, p.eps * kSmall2)) : rsqrtf(fmaf(norm[j], p.inverse, p.eps));
            if (big) times(y[j], kSmall);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) norm[j] = rsqrtf(fmaf(norm[j], p.inverse, p.eps));
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        F2 gate[4], one[4];
        widen<XT>(gw[j], gate);
        // g / (1 + e^-g): an approximate exponential and reciprocal, off by some 2^-22 of the
        // result for |g| < 20 (an error of the exponent counts |g| times), against steps of 2^-7.
        // The sum is formed 2^-12 times, and w brings the rest back, so that its reciprocal is a
        // normal number down to g = -95 (-87 without); there silu is 1e-39, below any scale.
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float lo, hi;
            unpack(fma2(gate[e], pack(-1.44269504f, -1.44269504f), pack(-12.f, -12.f)), &lo, &hi);
            unpack(add2(pack(sm100::ex2_approx(lo), sm100::ex2_approx(hi)), pack(0x1p-12f, 0x1p-12f)), &lo, &hi);
            one[e] = pack(rcp(lo), rcp(hi));
        }
        times(y[j], norm[j]);
        times(y[j], w);
        times(y[j], gate);
        times(y[j], one);
        top = top_of(top, y[j]);
    }
    const Totals t = row_totals<false>(0.f, top);
    if (!on) return;
    if (threadIdx.x == 0) p.scale[r] = scale_of(t.top);
    const Factor f = steps_of(t.top);
    if (f.f == 0.f) clear(y);
    int8_t *q = p.q + r * p.q_row;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (has(j)) store_steps8<VEC, false>(q, at(j), p.width, y[j], f, p.q_vec);
}

struct Launch {
    dim3 grid, block;
    cudaStream_t stream;
    int lanes_log2;

    template <typename... A, typename... B>
    cudaError_t operator()(void (*kernel)(A...), B... args) const {
        return launch(is_early(grid.x), kernel, grid, block, 0, stream, 1, args...);
    }
};
template <bool NORM, typename XT, typename RT, typename WT, int V, int MOST>
cudaError_t launch_rows(const RowsParams &p, const Launch &l) {
    return p.vec ? l(rows_kernel<NORM, XT, RT, WT, V, MOST, true>, p) : l(rows_kernel<NORM, XT, RT, WT, V, MOST, false>, p);
}
template <typename XT, typename WT, int V, int MOST>
cudaError_t launch_norm(const RowsParams &p, const Launch &l) {
    if (!p.residual) return launch_rows<true, XT, void, WT, V, MOST>(p, l);
    if (p.residual_bf16) return launch_rows<true, XT, __nv_bfloat16, WT, V, MOST>(p, l);
    return launch_rows<true, XT, float, WT, V, MOST>(p, l);
}
template <typename XT, int V, int MOST>
cudaError_t launch_x(const RowsParams &p, const Launch &l) {
    if (p.op == GDN_ROWS_GATED)
        return p.vec ? l(gated_kernel<XT, V, MOST, true>, p, l.lanes_log2, p.width / p.head)
                     : l(gated_kernel<XT, V, MOST, false>, p, l.lanes_log2, p.width / p.head);
    if (p.op == GDN_ROWS_PLAIN) return launch_rows<false, XT, void, float, V, MOST>(p, l);
    if (p.weight_bf16) return launch_norm<XT, __nv_bfloat16, V, MOST>(p, l);
    return launch_norm<XT, float, V, MOST>(p, l);
}
template <int V, int MOST>
cudaError_t launch_v(const RowsParams &p, const Launch &l) {
    return p.x_bf16 ? launch_x<__nv_bfloat16, V, MOST>(p, l) : launch_x<float, V, MOST>(p, l);
}

}  // namespace

cudaError_t launch_rows_int8(const RowsParams &given, cudaStream_t stream) {
    RowsParams p = given;
    // threads that a row needs at 8 numbers each
    int lanes_log2 = 0, need = (p.width + 7) / 8;
    if (p.op == GDN_ROWS_GATED) {
        while ((8 << lanes_log2) < p.head) ++lanes_log2;
        need = p.width / p.head << lanes_log2;
    }
    // Two eights a thread halve what a row costs beside its numbers (8224 x 2048 plain: 10.5 us with
    // one, 8.0 with two, 8.2 with four), unless a warp would be left part empty (8192 x 128 after a
    // norm: 3.4 us with one, 4.1 with two); four only where 1024 threads do not reach.
    const int v = need <= 64 ? 1 : need <= 2048 ? 2 : 4;
    const int threads = ((need + v - 1) / v + 31) / 32 * 32;
    const int rows = threads >= 128 ? 1 : 128 / threads;
    if (threads > 1024) return cudaErrorInvalidValue;
    const Launch l = {dim3(((unsigned)p.rows + rows - 1) / rows), dim3(threads, rows), stream, lanes_log2};
    p.early = is_early(l.grid.x);
    if (v == 1) return launch_v<1, 128>(p, l);
    if (v == 2) return threads <= 512 ? launch_v<2, 512>(p, l) : launch_v<2, 1024>(p, l);
    return launch_v<4, 1024>(p, l);
}

}  // namespace gdn
