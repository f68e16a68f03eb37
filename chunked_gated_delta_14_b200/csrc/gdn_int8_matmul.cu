// Product of rows in 8 bits on the tensor cores:
//
//   out[m][n] = x_scale[m] w_scale[n] sum_k x[m][k] w[n][k] + bias[n]
//
// The weights' channels are the accumulator's rows (M = 128 of the instruction)
// and the tokens its columns (N = BN), so that a decode step of a few tokens
// still fills the instruction and reads every weight once.  A block is
// persistent: one warp brings 128-byte slices of both operands by TMA into a ring
// of stages, one issues tcgen05.mma kind::i8 (32-bit integer accumulators in
// TMEM, exact), four turn the other of two accumulators into output.
//
// Each thread of those four holds one channel: its weight scale and bias stay in
// registers, a token's scale is one broadcast load, and a warp's 32 channels of
// one token are contiguous in the output.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "gdn_serve.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kBM = 128;             // channels a tile
constexpr int kBK = 128;             // bytes of k a stage
constexpr int kThreads = 192;
constexpr uint64_t kLimit = 4000000000ull;   // cycles before a wait gives up (about two seconds)

__device__ unsigned int g_int8_error = 0;

template <int BN>
struct Cfg {
    static constexpr int kStageBytes = kBM * kBK + BN * kBK;
    static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : BN == 64 ? 8 : 10;
    static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
    static constexpr int kSmem = kStages * kStageBytes + 1024;
    // instruction descriptor: D s32, A and B s8, K-major
    static constexpr uint32_t kIdesc = (2u << 4) | (1u << 7) | (1u << 10) | ((BN / 8u) << 17) | ((kBM / 16u) << 24);
};

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void umma_i8_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 lanes x 32 bits, 16 consecutive columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

struct Tiles {
    int n_tiles, m_tiles, k_slices;
};

// Tiles of 16 token tiles by all channels at a time: the blocks that run at once
// share both operands' rows through L2.
__device__ __forceinline__ void tile_of(const Tiles &g, int t, int *n, int *m) {
    constexpr int kGroup = 16;
    const int per = kGroup * g.n_tiles, first = t / per * kGroup;
    const int high = min(kGroup, g.m_tiles - first), rest = t % per;
    *m = first + rest % high;
    *n = rest / high;
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
int8_matmul_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                   const Int8MatmulParams p, const Tiles g) {
    using C = Cfg<BN>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages], acc_full[2], acc_empty[2], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    volatile int *abort = &abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = g.n_tiles * g.m_tiles;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < C::kStages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], 4); }
        mbar_init(&drain, 1);
        fence_mbar_init();
        tma_prefetch_desc(&wmap);
        tma_prefetch_desc(&xmap);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    block_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == 0) {
        int it = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            int tn, tm;
            tile_of(g, t, &tn, &tm);
            for (int kb = 0; kb < g.k_slices; ++kb, ++it) {
                const int s = it % C::kStages;
                if (it >= C::kStages &&
                    !(ok = mbar_wait(&empty[s], (it / C::kStages - 1) & 1, abort, 1, kLimit))) break;
                if (lane == 0) {
                    unsigned char *a = smem + s * C::kStageBytes;
                    mbar_arrive_expect_tx(&full[s], C::kStageBytes);
                    tma_load_2d(a, &wmap, &full[s], kb * kBK, tn * kBM);
                    tma_load_2d(a + kBM * kBK, &xmap, &full[s], kb * kBK, tm * BN);
                }
                __syncwarp();
            }
        }
        // every copy and every instruction that reads the ring ends before the block does
        for (int j = max(0, it - C::kStages); j < it; ++j) {
            const int s = j % C::kStages, ph = (j / C::kStages) & 1;
            if (ok) ok = mbar_wait(&empty[s], ph, abort, 2, kLimit);
            if (!ok) mbar_wait_drain(&full[s], ph, kLimit / 4);
        }
    } else if (warp == 1) {
        int it = 0, i = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++i) {
            const int acc = i & 1;
            if (i >= 2 && !(ok = mbar_wait(&acc_empty[acc], (i / 2 - 1) & 1, abort, 3, kLimit))) break;
            tc_fence_after();
            for (int kb = 0; kb < g.k_slices; ++kb, ++it) {
                const int s = it % C::kStages;
                if (!(ok = mbar_wait_spin(&full[s], (it / C::kStages) & 1, abort, 4, kLimit))) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t a = smem_u32(smem + s * C::kStageBytes);
                    const uint64_t ad = sdesc_sw128(a, 0, 1024), bd = sdesc_sw128(a + kBM * kBK, 0, 1024);
#pragma unroll
                    for (int k = 0; k < kBK / 32; ++k)
                        umma_i8_ss(tmem + acc * BN, ad + 2 * k, bd + 2 * k, C::kIdesc, kb > 0 || k > 0);
                    umma_commit(&empty[s]);
                    if (kb == g.k_slices - 1) umma_commit(&acc_full[acc]);
                }
                __syncwarp();
            }
        }
        if (!ok) {
            if (lane == 0) umma_commit(&drain);
            __syncwarp();
            mbar_wait_drain(&drain, 0, kLimit / 4);
        }
    } else {
        const int quarter = warp & 3;
        int i = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++i) {
            int tn, tm;
            tile_of(g, t, &tn, &tm);
            const int acc = i & 1;
            const int n = tn * kBM + quarter * 32 + lane, m0 = tm * BN;
            const bool has = n < p.N;
            const float ws = has ? __ldg(p.w_scale + n) : 0.f;
            const float b = has && p.bias ? __ldg(p.bias + n) : 0.f;
            if (!mbar_wait(&acc_full[acc], (i / 2) & 1, abort, 5, kLimit)) break;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + acc * BN;
            constexpr int kCols = BN < 32 ? 16 : 32;
#pragma unroll 1
            for (int c = 0; c < BN; c += kCols) {
                if (m0 + c >= p.M) break;
                uint32_t r[kCols];
                if constexpr (kCols == 16) tmem_ld16(taddr + c, r);
                else tmem_ld32(taddr + c, r);
                tmem_wait_ld();
                const int left = min(kCols, p.M - m0 - c);
                const int64_t o = (int64_t)(m0 + c) * p.out_row + n;
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    if (j < left && has) {
                        const float y = fmaf((float)(int)r[j] * __ldg(p.x_scale + m0 + c + j), ws, b);
                        if (p.out_bf16) reinterpret_cast<__nv_bfloat16 *>(p.out)[o + j * p.out_row] = __float2bfloat16_rn(y);
                        else reinterpret_cast<float *>(p.out)[o + j * p.out_row] = y;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
        }
    }
    block_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
    if (threadIdx.x == 0 && abort_flag) atomicCAS(&g_int8_error, 0u, (unsigned)abort_flag);
}

// Rows of K bytes -> rows at a stride of 16 bytes' multiples.  Bytes behind a
// row's K are never read (the tensor map ends at K), so they stay as they are.
__global__ void __launch_bounds__(256) pad_rows_kernel(const int8_t *from, int64_t from_row, int8_t *to, int64_t to_row,
                                                       int rows, int K) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int k = threadIdx.x; k < K; k += blockDim.x) to[r * to_row + k] = from[r * from_row + k];
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }
    return fn;
}

bool make_map(CUtensorMap *map, const int8_t *base, int K, int rows, int64_t row, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)row};
    const cuuint32_t box[2] = {kBK, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(base), dims, strides, box, one,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN>
cudaError_t launch_bn(const Int8MatmulParams &p, int sms, cudaStream_t stream, const char **why) {
    using C = Cfg<BN>;
    CUtensorMap wmap, xmap;
    if (!make_map(&wmap, p.w, p.K, p.N, p.w_row, kBM) || !make_map(&xmap, p.x, p.K, p.M, p.x_row, BN)) {
        *why = "tensor map refused";
        return cudaErrorInvalidValue;
    }
    const Tiles g = {(p.N + kBM - 1) / kBM, (p.M + BN - 1) / BN, (p.K + kBK - 1) / kBK};
    cudaError_t e = cudaFuncSetAttribute(int8_matmul_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)g.n_tiles * g.m_tiles;
    int8_matmul_kernel<BN><<<(unsigned)(tiles < sms ? tiles : sms), kThreads, C::kSmem, stream>>>(wmap, xmap, p, g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_int8_matmul(const Int8MatmulParams &p, cudaStream_t stream, const char **why) {
    if (!encode_fn()) { *why = "cuTensorMapEncodeTiled not found"; return cudaErrorNotSupported; }
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (p.M <= 16) return launch_bn<16>(p, sms, stream, why);
    if (p.M <= 32) return launch_bn<32>(p, sms, stream, why);
    if (p.M <= 64) return launch_bn<64>(p, sms, stream, why);
    const int64_t wide = (int64_t)((p.N + kBM - 1) / kBM) * ((p.M + 255) / 256);
    if (wide >= sms) return launch_bn<256>(p, sms, stream, why);
    return launch_bn<128>(p, sms, stream, why);
}

cudaError_t launch_int8_pad_rows(const int8_t *from, int64_t from_row, int8_t *to, int64_t to_row, int rows, int K,
                                 cudaStream_t stream) {
    pad_rows_kernel<<<rows < 65536 ? rows : 65536, 256, 0, stream>>>(from, from_row, to, to_row, rows, K);
    return cudaGetLastError();
}

unsigned int int8_matmul_read_and_clear_error(cudaError_t *err) {
    unsigned int v = 0, zero = 0;
    *err = cudaMemcpyFromSymbol(&v, g_int8_error, sizeof(v));
    if (*err == cudaSuccess && v) *err = cudaMemcpyToSymbol(g_int8_error, &zero, sizeof(zero));
    return v;
}

}  // namespace gdn
