// Rows in 8 bits: as they are, after a root-mean-square norm of x + residual, or
// after the norm of each head times silu(gate).
//
//   PLAIN  y = x
//   NORM   h = x + residual,  y = h rsqrt(mean h^2 + eps) w
//   GATED  y = x rsqrt(mean over the head of x^2 + eps) w gate / (1 + e^-gate)
//   scale = max|y| / 127,  q = rint(y 127 / max|y|)
//
// Bound by memory: a row is read once, stays in registers (8 V numbers a thread)
// while its statistics go round the row's threads, and is written once.  The
// largest |h w| is found beside the sum of squares, since the norm's factor is
// positive and the same for the whole row, so NORM too has one exchange.
#include <cuda_bf16.h>

#include <type_traits>

#include "gdn_serve.cuh"

namespace gdn {
namespace {

constexpr unsigned kInfBits = 0x7f800000u;

__device__ __forceinline__ float cvt(const __nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float cvt(const float x) { return x; }

// 8 numbers from 16-byte aligned memory.
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store1(float *p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float weight1(const RowsParams &p, int i) {
    return p.weight_bf16 ? cvt(__ldg(reinterpret_cast<const __nv_bfloat16 *>(p.weight) + i))
                         : __ldg(reinterpret_cast<const float *>(p.weight) + i);
}
__device__ __forceinline__ void weight8(const RowsParams &p, int i, float (&w)[8]) {
    if (p.weight_bf16) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(p.weight) + i));
        const uint32_t b[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[2 * j] = __uint_as_float(b[j] << 16);
            w[2 * j + 1] = __uint_as_float(b[j] & 0xffff0000u);
        }
    } else {
        const float4 *s = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p.weight) + i);
        const float4 a = __ldg(s), b = __ldg(s + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
}

__device__ __forceinline__ unsigned abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The row's scale, and the factor from y to steps (0 where the row has none).
// `top` holds the bits of max|y|: as whole numbers they order like the values,
// with NaN above infinity, so that neither is lost in a maximum.
__device__ __forceinline__ float scale_of(unsigned top, float *factor) {
    *factor = 0.f;
    if (top >= kInfBits) return __uint_as_float(0x7fc00000u);
    const float s = __uint_as_float(top) / 127.f;
    if (s < 1.17549435e-38f) return 0.f;
    *factor = 127.f / __uint_as_float(top);
    return s;
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, float f) {
    return (__float2int_rn(a * f) & 255) | (__float2int_rn(b * f) & 255) << 8 | (__float2int_rn(c * f) & 255) << 16 |
           __float2int_rn(d * f) << 24;
}
__device__ __forceinline__ void store_steps8(int8_t *p, const float (&y)[8], float f) {
    if (f == 0.f) { *reinterpret_cast<uint2 *>(p) = make_uint2(0, 0); return; }
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack4(y[0], y[1], y[2], y[3], f), pack4(y[4], y[5], y[6], y[7], f));
}
__device__ __forceinline__ void store_step1(int8_t *p, float y, float f) {
    *p = f == 0.f ? (int8_t)0 : (int8_t)__float2int_rn(y * f);
}

// Sum and largest over the row's threads (blockDim.x of them, whole warps).
struct Totals { float sum; unsigned top; };
__device__ __forceinline__ Totals row_totals(float sum, unsigned top, bool want_sum) {
    __shared__ float sums[32];
    __shared__ unsigned tops[32];
    top = __reduce_max_sync(~0u, top);
    if (want_sum)
#pragma unroll
        for (int m = 16; m; m /= 2) sum += __shfl_xor_sync(~0u, sum, m);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return {sum, top};
    const int first = threadIdx.y * warps;
    if ((threadIdx.x & 31) == 0) {
        sums[first + (threadIdx.x >> 5)] = sum;
        tops[first + (threadIdx.x >> 5)] = top;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    sum = lane < warps ? sums[first + lane] : 0.f;
    top = lane < warps ? tops[first + lane] : 0u;
    top = __reduce_max_sync(~0u, top);
    if (want_sum)
#pragma unroll
        for (int m = 16; m; m /= 2) sum += __shfl_xor_sync(~0u, sum, m);
    return {sum, top};
}

// PLAIN and NORM.  XT: type of x.  RT: type of the residual, or void for none.
// VEC: 16-byte accesses, thread i takes vectors i, i + blockDim.x, ...; else
// single elements the same way.
template <bool NORM, typename XT, typename RT, int V, bool VEC>
__global__ void __launch_bounds__(1024) rows_kernel(const RowsParams p) {
    constexpr bool RES = !std::is_void<RT>::value;
    using R1 = typename std::conditional<RES, RT, float>::type;
    const int row = blockIdx.x * blockDim.y + threadIdx.y;
    const bool on = row < p.rows;
    const int64_t r = on ? row : 0;
    const XT *x = reinterpret_cast<const XT *>(p.x) + r * p.x_row;
    const R1 *res = RES ? reinterpret_cast<const R1 *>(p.residual) + r * p.residual_row : nullptr;
    float h[V][8];
    // what this thread holds at (j, e): element `at(j, e)` of the row, if it is below the width
    auto at = [&](int j, int e) { return VEC ? (int)((threadIdx.x + j * blockDim.x) * 8 + e) : (int)(threadIdx.x + (j * 8 + e) * blockDim.x); };
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if constexpr (VEC) {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[j][e] = 0.f;
            if (on && at(j, 0) < p.width) load8(x + at(j, 0), h[j]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[j][e] = on && at(j, e) < p.width ? cvt(x[at(j, e)]) : 0.f;
        }
    }
    if constexpr (RES) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (VEC) {
                float b[8];
                if (on && at(j, 0) < p.width) {
                    load8(res + at(j, 0), b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[j][e] += b[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (on && at(j, e) < p.width) h[j][e] += cvt(res[at(j, e)]);
            }
        }
        R1 *out = reinterpret_cast<R1 *>(p.residual_out) + r * p.residual_out_row;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (VEC) {
                if (on && at(j, 0) < p.width) store8(out + at(j, 0), h[j]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (on && at(j, e) < p.width) store1(out + at(j, e), h[j][e]);
            }
        }
    }
    float sum = 0.f;
    unsigned top = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if constexpr (NORM) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(h[j][e], h[j][e], sum);
            if (p.weight) {
                if constexpr (VEC) {
                    if (at(j, 0) < p.width) {
                        float w[8];
                        weight8(p, at(j, 0), w);
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[j][e] *= w[e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (at(j, e) < p.width) h[j][e] *= weight1(p, at(j, e));
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, abs_bits(h[j][e]));
    }
    const Totals t = row_totals(sum, top, NORM);
    if (!on) return;
    float norm = 1.f;
    top = t.top;
    if constexpr (NORM) {
        norm = 1.f / sqrtf(t.sum / (float)p.width + p.eps);
        top = abs_bits(__uint_as_float(top) * norm);
    }
    float f;
    const float scale = scale_of(top, &f);
    if (threadIdx.x == 0) p.scale[r] = scale;
    int8_t *q = p.q + r * p.q_row;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if constexpr (NORM)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[j][e] *= norm;
        if constexpr (VEC) {
            if (at(j, 0) < p.width) store_steps8(q + at(j, 0), h[j], f);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at(j, e) < p.width) store_step1(q + at(j, e), h[j][e], f);
        }
    }
}

// GATED.  `lanes` (a power of two, 8 channels each) threads take a head, idle
// where the head has fewer channels; a thread's V heads are blockDim.x / lanes
// apart.
template <typename XT, int V, bool VEC>
__global__ void __launch_bounds__(1024) gated_kernel(const RowsParams p, int lanes) {
    const int row = blockIdx.x * blockDim.y + threadIdx.y;
    const bool on = row < p.rows;
    const int64_t r = on ? row : 0;
    const XT *x = reinterpret_cast<const XT *>(p.x) + r * p.x_row;
    const XT *g = reinterpret_cast<const XT *>(p.gate) + r * p.gate_row;
    const int part = (threadIdx.x & (lanes - 1)) * 8, heads = p.width / p.head, step = blockDim.x / lanes;
    const int head0 = threadIdx.x / lanes;
    const bool mine = on && part < p.head;
    auto at = [&](int j) { return (head0 + j * step) * p.head + part; };
    auto has = [&](int j) { return mine && head0 + j * step < heads; };
    float y[V][8], gate[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[j][e] = gate[j][e] = 0.f;
        if (has(j)) {
            if constexpr (VEC) {
                load8(x + at(j), y[j]);
                load8(g + at(j), gate[j]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) { y[j][e] = cvt(x[at(j) + e]); gate[j][e] = cvt(g[at(j) + e]); }
            }
        }
    }
    float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (p.weight && part < p.head) {
        if constexpr (VEC) weight8(p, part, w);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = weight1(p, part + e);
    }
    unsigned top = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(y[j][e], y[j][e], sum);
        for (int m = lanes / 2; m; m /= 2) sum += __shfl_xor_sync(~0u, sum, m);
        const float norm = 1.f / sqrtf(sum / (float)p.head + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[j][e] = y[j][e] * norm * w[e] * (gate[j][e] / (1.f + expf(-gate[j][e])));
            if (has(j)) top = max(top, abs_bits(y[j][e]));
        }
    }
    const Totals t = row_totals(0.f, top, false);
    if (!on) return;
    float f;
    const float scale = scale_of(t.top, &f);
    if (threadIdx.x == 0) p.scale[r] = scale;
    int8_t *q = p.q + r * p.q_row;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (has(j)) {
            if constexpr (VEC) store_steps8(q + at(j), y[j], f);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e) store_step1(q + at(j) + e, y[j][e], f);
        }
}

template <bool NORM, typename XT, typename RT, int V>
void launch_vec(const RowsParams &p, dim3 grid, dim3 block, cudaStream_t s) {
    if (p.vec) rows_kernel<NORM, XT, RT, V, true><<<grid, block, 0, s>>>(p);
    else rows_kernel<NORM, XT, RT, V, false><<<grid, block, 0, s>>>(p);
}
template <typename XT, int V>
void launch_v(const RowsParams &p, dim3 grid, dim3 block, int lanes, cudaStream_t s) {
    if (p.op == GDN_ROWS_GATED) {
        if (p.vec) gated_kernel<XT, V, true><<<grid, block, 0, s>>>(p, lanes);
        else gated_kernel<XT, V, false><<<grid, block, 0, s>>>(p, lanes);
    } else if (p.op == GDN_ROWS_PLAIN) {
        launch_vec<false, XT, void, V>(p, grid, block, s);
    } else if (!p.residual) {
        launch_vec<true, XT, void, V>(p, grid, block, s);
    } else if (p.residual_bf16) {
        launch_vec<true, XT, __nv_bfloat16, V>(p, grid, block, s);
    } else {
        launch_vec<true, XT, float, V>(p, grid, block, s);
    }
}
template <typename XT>
void launch_x(const RowsParams &p, int v, dim3 grid, dim3 block, int lanes, cudaStream_t s) {
    if (v == 1) launch_v<XT, 1>(p, grid, block, lanes, s);
    else if (v == 2) launch_v<XT, 2>(p, grid, block, lanes, s);
    else launch_v<XT, 4>(p, grid, block, lanes, s);
}

}  // namespace

cudaError_t launch_rows_int8(const RowsParams &p, cudaStream_t stream) {
    // threads that a row needs at 8 numbers each
    int lanes = 1, need = (p.width + 7) / 8;
    if (p.op == GDN_ROWS_GATED) {
        while (lanes * 8 < p.head) lanes *= 2;
        need = p.width / p.head * lanes;
    }
    const int v = need <= 512 ? 1 : need <= 1024 ? 2 : 4;
    int threads = ((need + v - 1) / v + 31) / 32 * 32;
    if (p.op == GDN_ROWS_GATED && v * (threads / lanes) * lanes < need) return cudaErrorInvalidValue;
    if (threads > 1024) return cudaErrorInvalidValue;
    const int rows = threads >= 256 ? 1 : 256 / threads;
    const dim3 block(threads, rows), grid((p.rows + rows - 1) / rows);
    if (p.x_bf16) launch_x<__nv_bfloat16>(p, v, grid, block, lanes, stream);
    else launch_x<float>(p, v, grid, block, lanes, stream);
    return cudaGetLastError();
}

}  // namespace gdn
