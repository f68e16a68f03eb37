// Product of rows in 8 bits on the tensor cores:
//
//   out[m][n] = x_scale[m] w_scale[n] sum_k x[m][k] w[n][k] + bias[n]
//
// The weights' channels are the accumulator's rows and the tokens its columns (BN),
// so that a decode step of a few tokens still fills the instruction and reads every
// weight once.  A block is persistent: one thread brings 128-byte slices of both
// operands by TMA into a ring of stages, one issues tcgen05.mma kind::i8 (32-bit
// integer accumulators in TMEM, exact), four warps turn the other of two
// accumulators into output.
//
// Each thread of those four holds one channel: its weight scale and bias stay in
// registers, a token's scale is one broadcast load, and a warp's 32 channels of
// one token are contiguous in the output.
//
// PAIR: two blocks of a cluster share a tile of 256 channels by 256 tokens
// (cta_group::2).  Each brings its own 128 channels and half of the tokens, and the
// instruction reads the other half from the other block's shared memory, which
// halves what a block has to bring for the tokens.
//
// Single blocks take `channels` (16 to 128) by BN: where tiles of 128 channels would
// leave SMs idle, a tile holds fewer.  The instruction still works on 128 rows; the
// sums of those that were not brought are not looked at.  What bounds such a block is
// its own port to L2, some 70 bytes a cycle, so more blocks are quicker although each
// has to bring the tokens.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <atomic>

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

template <int BN, bool PAIR>
struct Cfg {
    static constexpr int kTokens = PAIR ? BN / 2 : BN;           // rows of x a block brings
    static constexpr int kStageBytes = (kBM + kTokens) * kBK;
    static constexpr int kStages = kTokens >= 128 ? 6 : kTokens == 64 ? 8 : 10;
    static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
    static constexpr int kSmem = kStages * kStageBytes + 1024;
    // instruction descriptor: D s32, A and B s8, K-major
    static constexpr uint32_t kIdesc = (2u << 4) | (1u << 7) | (1u << 10) | ((BN / 8u) << 17) | (((PAIR ? 2 : 1) * kBM / 16u) << 24);
    static_assert(kTmemCols <= 512 && kSmem <= 227 * 1024 - 4096, "");
};

// One lane of a whole warp, the same each time.  Chosen this way the compiler knows that
// one thread runs what follows: under a test of the lane's number each tcgen05.mma takes
// 170 cycles to issue, whatever its size; under this one 40 for up to 64 columns, 65 for
// 128 and 129 for 256, which is the tensor core's rate.
__device__ __forceinline__ bool elect() {
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
    return is != 0;
}

// PAIR: `bar` may lie in the other block of the pair.
template <bool PAIR>
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4}], [%2];"
            ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
            ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void umma_i8_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Arrive on `bar`, PAIR: in both blocks, when every tcgen05.mma issued so far completes.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
            ::"r"(smem_u32(bar)), "h"((uint16_t)3)
            : "memory");
    else
        umma_commit(bar);
}

template <bool PAIR>
__device__ __forceinline__ void alloc(uint32_t *slot, uint32_t columns) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(slot, columns);
        tmem_relinquish();
    }
}
template <bool PAIR>
__device__ __forceinline__ void dealloc(uint32_t taddr, uint32_t columns) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(columns) : "memory");
    else
        tmem_dealloc(taddr, columns);
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
    int channels;           // of a tile (PAIR: of each block's half)
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

__device__ __forceinline__ void store_one(const Int8MatmulParams &p, int64_t i, int sum, float xs, float ws, float b) {
    const float y = fmaf((float)sum * xs, ws, b);
    if (p.out_bf16) reinterpret_cast<__nv_bfloat16 *>(p.out)[i] = __float2bfloat16_rn(y);
    else reinterpret_cast<float *>(p.out)[i] = y;
}

// N tokens of one channel.
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
template <int N, typename T>
__device__ __forceinline__ void store_column(T *to, int64_t row, const uint32_t (&r)[N], const float *xs, float ws, float b) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
        const float4 s = *reinterpret_cast<const float4 *>(xs + j);
        put(to, fmaf((float)(int)r[j] * s.x, ws, b)); to += row;
        put(to, fmaf((float)(int)r[j + 1] * s.y, ws, b)); to += row;
        put(to, fmaf((float)(int)r[j + 2] * s.z, ws, b)); to += row;
        put(to, fmaf((float)(int)r[j + 3] * s.w, ws, b)); to += row;
    }
}

template <int BN, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
int8_matmul_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                   const Int8MatmulParams p, const Tiles g) {
    using C = Cfg<BN, PAIR>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages], acc_full[2], acc_empty[2], drain;
    __shared__ __align__(16) float x_scales[4][BN];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    volatile int *abort = &abort_flag;
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_ctarank() : 0;
    const int tiles = g.n_tiles * g.m_tiles, group = PAIR ? 2 : 1;
    const int first = blockIdx.x / group, stride = gridDim.x / group;
    const uint32_t stage_tx = PAIR ? 2 * C::kStageBytes : (g.channels + C::kTokens) * kBK;

    grid_next();
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < C::kStages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], PAIR ? 8 : 4); }
        mbar_init(&drain, 1);
        fence_mbar_init();
        tma_prefetch_desc(&wmap);
        tma_prefetch_desc(&xmap);
    }
    if (warp == 1) alloc<PAIR>(&tmem_slot, C::kTmemCols);
    tc_fence_before();
    block_sync();
    if (PAIR) cluster_sync_all();        // the other block's barriers are there
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(~0u, tmem_slot, 0);
    grid_wait();

    if (warp == 0 && elect()) {          // the copies: one thread
        int it = 0;
        bool ok = true;
        for (int t = first; ok && t < tiles; t += stride) {
            int tn, tm;
            tile_of(g, t, &tn, &tm);
            const int n0 = (PAIR ? 2 * tn + rank : tn) * g.channels, m0 = tm * BN + (PAIR ? rank * C::kTokens : 0);
            for (int kb = 0; kb < g.k_slices; ++kb, ++it) {
                const int s = it % C::kStages;
                if (it >= C::kStages &&
                    !(ok = mbar_wait_cluster(&empty[s], (it / C::kStages - 1) & 1, abort, 1, kLimit))) break;
                unsigned char *a = smem + s * C::kStageBytes;
                // the pair's copies all count on the first block's barrier, where the instructions are issued
                const uint32_t bar = PAIR ? mapa_shared(smem_u32(&full[s]), 0) : smem_u32(&full[s]);
                if (rank == 0 || !PAIR) mbar_arrive_expect_tx(&full[s], stage_tx);
                tma_load_2d<PAIR>(a, &wmap, bar, kb * kBK, n0);
                tma_load_2d<PAIR>(a + kBM * kBK, &xmap, bar, kb * kBK, m0);
            }
        }
        // every copy and every instruction that reads the ring ends before the block does
        for (int j = max(0, it - C::kStages); j < it; ++j) {
            const int s = j % C::kStages, ph = (j / C::kStages) & 1;
            if (ok) ok = mbar_wait_cluster(&empty[s], ph, abort, 2, kLimit);
            if (!ok && (rank == 0 || !PAIR)) mbar_wait_drain(&full[s], ph, kLimit / 4);
        }
    } else if (warp == 1 && (rank == 0 || !PAIR) && elect()) {       // the instructions: one thread
        int it = 0, i = 0;
        bool ok = true;
        for (int t = first; ok && t < tiles; t += stride, ++i) {
            const int acc = i & 1;
            if (i >= 2 && !(ok = mbar_wait_cluster(&acc_empty[acc], (i / 2 - 1) & 1, abort, 3, kLimit))) break;
            tc_fence_after();
            for (int kb = 0; kb < g.k_slices; ++kb, ++it) {
                const int s = it % C::kStages;
                // (reading the clock, as the bounded wait does, takes 250 cycles)
                if (!(ok = mbar_try_wait(&full[s], (it / C::kStages) & 1) ||
                           mbar_wait_spin(&full[s], (it / C::kStages) & 1, abort, 4, kLimit))) break;
                tc_fence_after();
                const uint32_t a = smem_u32(smem + s * C::kStageBytes);
                const uint64_t ad = sdesc_sw128(a, 0, 1024), bd = sdesc_sw128(a + kBM * kBK, 0, 1024);
#pragma unroll
                for (int k = 0; k < kBK / 32; ++k)
                    umma_i8_ss<PAIR>(tmem + acc * BN, ad + 2 * k, bd + 2 * k, C::kIdesc, kb > 0 || k > 0);
                commit<PAIR>(&empty[s]);
                if (kb == g.k_slices - 1) commit<PAIR>(&acc_full[acc]);
            }
        }
        if (!ok) {
            // one block's barrier: the other's instructions are these
            if constexpr (PAIR)
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&drain)) : "memory");
            else
                umma_commit(&drain);
            mbar_wait_drain(&drain, 0, kLimit / 4);
        }
    } else if (warp >= 2) {
        const int quarter = warp & 3;
        int i = 0;
        for (int t = first; t < tiles; t += stride, ++i) {
            int tn, tm;
            tile_of(g, t, &tn, &tm);
            const int acc = i & 1;
            const int row = quarter * 32 + lane, n = (PAIR ? 2 * tn + rank : tn) * g.channels + row, m0 = tm * BN;
            const bool has = row < g.channels && n < p.N;
            const float ws = has ? plain(p.w_scale + n) : 0.f;
            const float b = has && p.bias ? plain(p.bias + n) : 0.f;
            // the tokens' scales, a copy for each warp, while the sums are formed: the four warps have
            // no barrier among them that one which gives up could leave the others in
            __syncwarp();
            for (int j = lane; j < BN; j += 32) x_scales[quarter][j] = m0 + j < p.M ? plain(p.x_scale + m0 + j) : 0.f;
            __syncwarp();
            if (!__all_sync(~0u, mbar_wait_cluster(&acc_full[acc], (i / 2) & 1, abort, 5, kLimit))) break;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + acc * BN;
            constexpr int kCols = BN < 32 ? 16 : 32;
#pragma unroll 1
            for (int c = 0; c < BN; c += kCols) {
                if (m0 + c >= p.M || quarter * 32 >= g.channels) break;
                __syncwarp();            // the loads below are the whole warp's, also behind a store of some lanes
                uint32_t r[kCols];
                if constexpr (kCols == 16) tmem_ld16(taddr + c, r);
                else tmem_ld32(taddr + c, r);
                tmem_wait_ld();
                const int left = min(kCols, p.M - m0 - c);
                const int64_t o = (int64_t)(m0 + c) * p.out_row + n;
                const float *xs = &x_scales[quarter][c];
                if (has) {
                    if (left == kCols) {
                        if (p.out_bf16) store_column<kCols>(reinterpret_cast<__nv_bfloat16 *>(p.out) + o, p.out_row, r, xs, ws, b);
                        else store_column<kCols>(reinterpret_cast<float *>(p.out) + o, p.out_row, r, xs, ws, b);
                    } else {
#pragma unroll
                        for (int j = 0; j < kCols; ++j)
                            if (j < left) store_one(p, o + j * p.out_row, (int)r[j], xs[j], ws, b);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR && rank == 1) mbar_arrive_remote(mapa_shared(smem_u32(&acc_empty[acc]), 0));
                else mbar_arrive(&acc_empty[acc]);
            }
        }
    }
    block_sync();
    if (PAIR) cluster_sync_all();        // no block leaves while another reads its shared memory
    tc_fence_after();
    if (warp == 1) dealloc<PAIR>(tmem, C::kTmemCols);
    if (threadIdx.x == 0 && abort_flag) atomicCAS(&g_int8_error, 0u, (unsigned)abort_flag);
}

// Rows of K bytes at any address and stride -> rows on 16 bytes, of one or both
// operands (first x's, then w's; a block a row).  Sixteen bytes a thread, from the five
// aligned words that hold them where those lie in the row, else byte by byte.  The
// bytes behind a row's K become 0 (they are not read: the tensor map ends at K).
__global__ void __launch_bounds__(256) pad_rows_kernel(const PadRows x, const PadRows w, int K) {
    grid_next();
    grid_wait();
    const unsigned job = blockIdx.x;
    const PadRows &p = job < (unsigned)x.rows ? x : w;
    const int64_t row = job < (unsigned)x.rows ? job : job - x.rows;
    const int8_t *from = p.from + row * p.from_row;
    int8_t *to = p.to + row * p.to_row;
    for (int k = threadIdx.x * 16; k < K; k += blockDim.x * 16) {
        uint32_t y[4] = {0, 0, 0, 0};
        const uintptr_t at = reinterpret_cast<uintptr_t>(from + k), word = at & ~(uintptr_t)3;
        if (word >= reinterpret_cast<uintptr_t>(from) && word + 20 <= reinterpret_cast<uintptr_t>(from + K)) {
            uint32_t z[5];
#pragma unroll
            for (int j = 0; j < 5; ++j) z[j] = plain(reinterpret_cast<const uint32_t *>(word) + j);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = __funnelshift_r(z[j], z[j + 1], (uint32_t)(at & 3) * 8);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (k + j < K) y[j / 4] |= (uint32_t)(uint8_t)from[k + j] << (8 * (j & 3));
        }
        *reinterpret_cast<uint4 *>(to + k) = make_uint4(y[0], y[1], y[2], y[3]);
    }
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

template <int BN, bool PAIR>
cudaError_t launch_bn(const Int8MatmulParams &p, int channels, int dev, int sms, cudaStream_t stream, const char **why) {
    using C = Cfg<BN, PAIR>;
    CUtensorMap wmap, xmap;
    if (!make_map(&wmap, p.w, p.K, p.N, p.w_row, channels) || !make_map(&xmap, p.x, p.K, p.M, p.x_row, C::kTokens)) {
        *why = "tensor map refused";
        return cudaErrorInvalidValue;
    }
    const int wide = (PAIR ? 2 : 1) * channels, group = PAIR ? 2 : 1;
    const Tiles g = {channels, (p.N + wide - 1) / wide, (p.M + BN - 1) / BN, (p.K + kBK - 1) / kBK};
    const int64_t tiles = (int64_t)g.n_tiles * g.m_tiles, most = sms / group;
    static std::atomic<uint64_t> ready{0};       // devices on which the kernel may have its shared memory
    cudaError_t e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(int8_matmul_kernel<BN, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    return launch(true, int8_matmul_kernel<BN, PAIR>, dim3((unsigned)((tiles < most ? tiles : most) * group)), dim3(kThreads), C::kSmem,
                        stream, (unsigned)group, wmap, xmap, p, g);
}

}  // namespace

cudaError_t launch_int8_matmul(const Int8MatmulParams &p, cudaStream_t stream, const char **why) {
    if (!encode_fn()) { *why = "cuTensorMapEncodeTiled not found"; return cudaErrorNotSupported; }
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    // The tile: the one whose blocks are done first, by cycles a slice of k.  A block brings 70
    // bytes a cycle and issues a slice's instructions in 230 cycles up to 64 tokens, 300 with
    // 128; a pair takes 540 for 256 by 256.  Of equal ones the one with more channels reads
    // the tokens less often.  Measured (us): 16 x 8224 x 2048: 64 channels by 16 tokens 6.9,
    // 128 by 16 6.9, 64 by 64 8.8; 333 x 1001 x 1537: 64 by 64 6.2, 128 by 128 9.9;
    // 256 x 8192 x 4096: 128 by 128 12.9, the pair 16.9; 1024 x 8224 x 2048: the pair 17.2,
    // 128 by 128 20.0.
    const int k_slices = (p.K + kBK - 1) / kBK;
    const auto waves = [&](int channels, int bn, int slots) {
        const int64_t tiles = (int64_t)((p.N + channels - 1) / channels) * ((p.M + bn - 1) / bn);
        return (tiles + slots - 1) / slots;
    };
    int channels = 256, bn = 256;
    int64_t best = waves(256, 256, sms / 2) * k_slices * 540 + 2500;
    for (int b = 16; b <= 128; b *= 2)
        for (int c = 16; c <= 128; c *= 2) {
            const int issue = b == 128 ? 300 : 230, bring = (c + b) * kBK / 70;
            const int64_t x = waves(c, b, sms) * (k_slices * (bring > issue ? bring : issue) + 300) + b * 8;
            if (x <= best) { best = x; channels = c; bn = b; }
        }
    switch (bn) {
        case 16: return launch_bn<16, false>(p, channels, dev, sms, stream, why);
        case 32: return launch_bn<32, false>(p, channels, dev, sms, stream, why);
        case 64: return launch_bn<64, false>(p, channels, dev, sms, stream, why);
        case 128: return launch_bn<128, false>(p, channels, dev, sms, stream, why);
        default: return launch_bn<256, true>(p, kBM, dev, sms, stream, why);
    }
}

cudaError_t launch_int8_pad_rows(const PadRows &x, const PadRows &w, int K, cudaStream_t stream) {
    const int threads = (K + 511) / 512 * 32;
    if ((int64_t)x.rows + w.rows > 0x7fffffff) return cudaErrorInvalidValue;
    return launch(true, pad_rows_kernel, dim3((unsigned)x.rows + (unsigned)w.rows), dim3(threads < 256 ? threads : 256), 0, stream, 1, x, w, K);
}

unsigned int int8_matmul_read_and_clear_error(cudaError_t *err) {
    unsigned int v = 0, zero = 0;
    *err = cudaMemcpyFromSymbol(&v, g_int8_error, sizeof(v));
    if (*err == cudaSuccess && v) *err = cudaMemcpyToSymbol(g_int8_error, &zero, sizeof(zero));
    return v;
}

}  // namespace gdn
