// Decode-layer operators: parameters resolved by the host layer (gdn_serve_api.cu)
// and the launchers it calls.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

struct PoolParams {
    int rows, seqs, H, Hk, dk, dv, pool;
    int io_bf16, o_bf16, qk_norm, vec;   // vec: every row of q, k, v starts on 16 bytes
    float qk_eps;
    const void *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;
    const float *alpha, *beta;
    int64_t alpha_row, beta_row;
    const int32_t *cu_seqlens, *slots;
    float *state;
    void *o;
    int early;          // set by the launcher: launched early
};
cudaError_t launch_recurrent_pool(const PoolParams &p, cudaStream_t stream);

struct RowsParams {
    int op, rows, width, head;
    int x_bf16, residual_bf16, weight_bf16;
    int vec;                             // every row starts on 16 bytes, width a multiple of 8
    int in_place;                        // residual_out is x or the residual
    int weight_vec, q_vec;               // the weight starts on 16 bytes, every row of q on 8
    float eps, inverse;                  // inverse: 1 / the numbers a norm is of
    const void *x, *residual, *gate, *weight;
    int64_t x_row, residual_row, gate_row, residual_out_row, q_row;
    void *residual_out;
    int8_t *q;
    float *scale;
    int early;                           // set by the launcher: launched early
};
cudaError_t launch_rows_int8(const RowsParams &p, cudaStream_t stream);

struct Int8MatmulParams {
    int M, N, K, out_bf16;
    const int8_t *x, *w;
    int64_t x_row, w_row, out_row;       // x_row, w_row multiples of 16, x and w on 16 bytes
    const float *x_scale, *w_scale, *bias;
    void *out;
};
cudaError_t launch_int8_matmul(const Int8MatmulParams &p, cudaStream_t stream, const char **why);
// Rows at any stride -> rows at stride `to_row` (a multiple of 16), of both operands at once.
struct PadRows {
    const int8_t *from;
    int64_t from_row;
    int8_t *to;
    int64_t to_row;
    int rows;           // 0: none
};
cudaError_t launch_int8_pad_rows(const PadRows &x, const PadRows &w, int K, cudaStream_t stream);

// A launch that may begin before the kernel ahead of it on the stream has ended (early): the
// kernel sets itself up, then waits (grid_wait) for that one's end before it reads or writes
// anything outside itself, in every thread, so that its own end comes after that one's.
// Back to back from the host a product of 16 rows takes 5.6 us so, 8.2 without, and a norm
// of 16 x 2048 on the device 0.25 us less.  So the product and its copies at every size (with
// copies of 1334 rows 8.8 us in a row of calls, 10.3 without; of 5001 rows 15.1, 18.6), the
// one-token recurrence (its blocks are equal), and others of few blocks.  Of others, grids of
// more blocks than run at once begin after that end as ever: taking the places of the last
// blocks one by one they were spread worse (long ragged sequences 588 us instead of 545), and
// the wait alone, in each of 8224 blocks, cost plain rows of 2048 1.4 of 8 us.
inline bool is_early(unsigned blocks) { return blocks <= 296; }      // two an SM
template <typename... A, typename... B>
cudaError_t launch(bool early, void (*kernel)(A...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, unsigned cluster,
                   B... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (early) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = cluster;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#ifdef __CUDACC__
// How these kernels read their operands: an ordinary load.  The read-only path (__ldg) is for
// data that nothing writes while the kernel lives, and one launched early lives while the
// kernel ahead still writes what it is going to read behind the wait.
template <typename T>
__device__ __forceinline__ T plain(const T *p) { return *p; }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The kernel behind this one, if launched early, may begin once every block has said this.
__device__ __forceinline__ void grid_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

// Return (and clear) the error word of these kernels; the caller has synchronised.
unsigned int pool_read_and_clear_error(cudaError_t *err);
unsigned int int8_matmul_read_and_clear_error(cudaError_t *err);

// A failed call's message, for gdn_last_error() (gdn_api.cu); returns s.
gdn_status api_fail(gdn_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// A call that succeeded: no message.
gdn_status api_ok();

}  // namespace gdn
