// Gated delta rule, token by token, for a ragged batch on a pool of states
// (h = S^T, d_k x d_v, fp32):
//
//   p   = h^T k_t                          (= S_{t-1} k_t)
//   u   = beta_t (v_t - alpha_t p)
//   h  <- alpha_t h + k_t u^T
//   o_t = h^T q_t
//
// Columns of h never meet: a warp takes 16 of them through all tokens of one
// sequence and head, with its 16 columns of h in registers and no barrier.
// Lane = row group (8) x column quad (4): R = d_k / 8 rows by 4 columns a lane,
// so a row's 16 columns are 64 contiguous bytes of the state.  The two sums over
// d_k go by halving exchanges: 4 shuffles leave each lane one column's sum, in
// which it forms that column's u, and 3 more hand the 4 columns' u round.
//
// A step of one token is bound by reading and writing the states (8 d_k d_v
// bytes a head); a long sequence by the chain p -> u -> h of each token, beside
// which the next token's q, k, v and gates are already on their way.
#include <cuda_bf16.h>

#include "gdn_serve.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kCols = 16;       // value columns a warp
constexpr int kGroups = 8;      // row groups a warp

// Sequence whose cu_seqlens range or slot is out of bounds: 1 + its index.
__device__ unsigned int g_pool_error = 0;

__device__ __forceinline__ float load1(const void *p, int64_t i, bool bf16) {
    if (bf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
    return reinterpret_cast<const float *>(p)[i];
}

// R consecutive numbers as they lie in memory, so that a token's q and k wait
// in as few registers as they have bytes.
template <int R, bool BF16>
struct Raw {
    static constexpr int kWords = BF16 ? (R + 1) / 2 : R;
    uint32_t w[kWords];

    template <bool VEC>
    __device__ __forceinline__ void load(const void *base, int64_t i) {
        if constexpr (VEC && kWords % 4 == 0) {
            const uint4 *s = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(base) + i * (BF16 ? 2 : 4));
#pragma unroll
            for (int j = 0; j < kWords / 4; ++j) {
                const uint4 x = __ldg(s + j);
                w[4 * j] = x.x; w[4 * j + 1] = x.y; w[4 * j + 2] = x.z; w[4 * j + 3] = x.w;
            }
        } else if constexpr (BF16) {
            const uint16_t *s = reinterpret_cast<const uint16_t *>(base) + i;
#pragma unroll
            for (int j = 0; j < R / 2; ++j) w[j] = (uint32_t)__ldg(s + 2 * j) | ((uint32_t)__ldg(s + 2 * j + 1) << 16);
        } else {
            const uint32_t *s = reinterpret_cast<const uint32_t *>(base) + i;
#pragma unroll
            for (int j = 0; j < R; ++j) w[j] = __ldg(s + j);
        }
    }

    __device__ __forceinline__ float get(int r) const {
        if constexpr (BF16) return __uint_as_float(r & 1 ? w[r / 2] & 0xffff0000u : w[r / 2] << 16);
        else return __uint_as_float(w[r]);
    }
};

__device__ __forceinline__ float xor_add(float x, int mask) { return x + __shfl_xor_sync(~0u, x, mask); }

// Sums over the 8 row groups; lane gets the one of column `lane_col`.
__device__ __forceinline__ float reduce_columns(const float (&x)[4], int lane) {
    const bool hi = lane & 16, odd = lane & 8;
    const float a = hi ? x[2] : x[0], b = hi ? x[3] : x[1];
    const float c = a + __shfl_xor_sync(~0u, hi ? x[0] : x[2], 16);
    const float d = b + __shfl_xor_sync(~0u, hi ? x[1] : x[3], 16);
    const float e = (odd ? d : c) + __shfl_xor_sync(~0u, odd ? c : d, 8);
    return xor_add(e, 4);
}

template <int R, bool BF16, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) recurrent_pool_kernel(const PoolParams p) {
    const int lane = threadIdx.x & 31;
    const int slices = p.dv / kCols;
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (item >= (int64_t)p.seqs * p.H * slices) return;
    const int slice = (int)(item % slices);
    const int h = (int)(item / slices % p.H);
    const int s = (int)(item / slices / p.H);

    int begin = s, end = s + 1;
    if (p.cu_seqlens) {
        begin = p.cu_seqlens[s];
        end = p.cu_seqlens[s + 1];
        if (begin < 0 || end < begin || end > p.rows) {
            if (lane == 0) atomicCAS(&g_pool_error, 0u, (unsigned)s + 1u);
            return;
        }
    }
    int slot = p.slots ? p.slots[s] : s;
    if (slot < -1 || slot >= p.pool) {
        if (lane == 0) atomicCAS(&g_pool_error, 0u, (unsigned)s + 1u);
        slot = -1;
    }
    if (begin == end) return;
    if (slot < 0) {                      // no sequence: zero rows of o
        for (int64_t t = begin + (lane >> 4); t < end; t += 2) {
            const int64_t i = (t * p.H + h) * p.dv + slice * kCols + (lane & 15);
            if (p.o_bf16) reinterpret_cast<__nv_bfloat16 *>(p.o)[i] = __float2bfloat16_rn(0.f);
            else reinterpret_cast<float *>(p.o)[i] = 0.f;
        }
        return;
    }

    const int group = lane >> 2, quad = lane & 3;
    const int row0 = group * R, hk = h / (p.H / p.Hk);
    float4 *hp = reinterpret_cast<float4 *>(p.state + (((int64_t)slot * p.H + h) * p.dk + row0) * p.dv + slice * kCols) + quad;
    const int pitch = p.dv / 4;          // float4 a row
    float hr[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float4 x = __ldcg(hp + r * pitch);
        hr[r][0] = x.x; hr[r][1] = x.y; hr[r][2] = x.z; hr[r][3] = x.w;
    }

    // the column whose sums this lane holds after reduce_columns
    const int col = slice * kCols + quad * 4 + ((lane >> 4) & 1) * 2 + ((lane >> 3) & 1);
    const int64_t qo = (int64_t)hk * p.q_head + row0, ko = (int64_t)hk * p.k_head + row0;
    const int64_t vo = (int64_t)h * p.v_head + col;
    Raw<R, BF16> kn, qn;
    float vn, an, bn;
    auto fetch = [&](int64_t t) {
        kn.template load<VEC>(p.k, t * p.k_row + ko);
        qn.template load<VEC>(p.q, t * p.q_row + qo);
        vn = load1(p.v, t * p.v_row + vo, BF16);
        an = p.alpha ? __ldg(p.alpha + t * p.alpha_row + h) : 1.f;
        bn = p.beta ? __ldg(p.beta + t * p.beta_row + h) : 1.f;
    };
    fetch(begin);
    for (int64_t t = begin; t < end; ++t) {
        float ks[R], qs[R];
#pragma unroll
        for (int r = 0; r < R; ++r) { ks[r] = kn.get(r); qs[r] = qn.get(r); }
        const float v = vn, a = an, be = bn;
        if (t + 1 < end) fetch(t + 1);
        if (p.qk_norm) {
            float kk = 0.f, qq = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) { kk += ks[r] * ks[r]; qq += qs[r] * qs[r]; }
#pragma unroll
            for (int m = 4; m < 32; m *= 2) { kk = xor_add(kk, m); qq = xor_add(qq, m); }
            kk = 1.f / sqrtf(kk + p.qk_eps);
            qq = 1.f / sqrtf(qq + p.qk_eps);
#pragma unroll
            for (int r = 0; r < R; ++r) { ks[r] *= kk; qs[r] *= qq; }
        }
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) x[c] = fmaf(hr[r][c], ks[r], x[c]);
        const float uc = be * (v - a * reduce_columns(x, lane));
        // u of the quad's 4 columns: from the neighbours across bits 3 and 4
        const float un = __shfl_xor_sync(~0u, uc, 8);
        const bool hi = lane & 16, odd = lane & 8;
        const float u0 = odd ? un : uc, u1 = odd ? uc : un;
        const float w0 = __shfl_xor_sync(~0u, u0, 16), w1 = __shfl_xor_sync(~0u, u1, 16);
        const float u[4] = {hi ? w0 : u0, hi ? w1 : u1, hi ? u0 : w0, hi ? u1 : w1};
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                hr[r][c] = fmaf(ks[r], u[c], a * hr[r][c]);
                x[c] = fmaf(hr[r][c], qs[r], x[c]);
            }
        const float o = reduce_columns(x, lane);
        if (!(lane & 4)) {
            const int64_t i = (t * p.H + h) * p.dv + col;
            if (p.o_bf16) reinterpret_cast<__nv_bfloat16 *>(p.o)[i] = __float2bfloat16_rn(o);
            else reinterpret_cast<float *>(p.o)[i] = o;
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) __stcg(hp + r * pitch, make_float4(hr[r][0], hr[r][1], hr[r][2], hr[r][3]));
}

template <int R>
void launch_r(const PoolParams &p, unsigned blocks, cudaStream_t stream) {
    const int threads = kWarps * 32;
    if (p.io_bf16) {
        if (p.vec) recurrent_pool_kernel<R, true, true><<<blocks, threads, 0, stream>>>(p);
        else recurrent_pool_kernel<R, true, false><<<blocks, threads, 0, stream>>>(p);
    } else {
        if (p.vec) recurrent_pool_kernel<R, false, true><<<blocks, threads, 0, stream>>>(p);
        else recurrent_pool_kernel<R, false, false><<<blocks, threads, 0, stream>>>(p);
    }
}

}  // namespace

cudaError_t launch_recurrent_pool(const PoolParams &p, cudaStream_t stream) {
    const int64_t items = (int64_t)p.seqs * p.H * (p.dv / kCols);
    const unsigned blocks = (unsigned)((items + kWarps - 1) / kWarps);
    switch (p.dk / kGroups) {
        case 2: launch_r<2>(p, blocks, stream); break;
        case 4: launch_r<4>(p, blocks, stream); break;
        case 8: launch_r<8>(p, blocks, stream); break;
        case 16: launch_r<16>(p, blocks, stream); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

unsigned int pool_read_and_clear_error(cudaError_t *err) {
    unsigned int v = 0, zero = 0;
    *err = cudaMemcpyFromSymbol(&v, g_pool_error, sizeof(v));
    if (*err == cudaSuccess && v) *err = cudaMemcpyToSymbol(g_pool_error, &zero, sizeof(zero));
    return v;
}

}  // namespace gdn
