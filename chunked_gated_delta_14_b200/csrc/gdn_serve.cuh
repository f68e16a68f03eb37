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
};
cudaError_t launch_recurrent_pool(const PoolParams &p, cudaStream_t stream);

struct RowsParams {
    int op, rows, width, head;
    int x_bf16, residual_bf16, weight_bf16;
    int vec;                             // every row starts on 16 bytes, width a multiple of 8
    int weight_vec, q_vec;               // the weight starts on 16 bytes, every row of q on 8
    float eps, inverse;                  // inverse: 1 / the numbers a norm is of
    const void *x, *residual, *gate, *weight;
    int64_t x_row, residual_row, gate_row, residual_out_row, q_row;
    void *residual_out;
    int8_t *q;
    float *scale;
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

// Return (and clear) the error word of these kernels; the caller has synchronised.
unsigned int pool_read_and_clear_error(cudaError_t *err);
unsigned int int8_matmul_read_and_clear_error(cudaError_t *err);

// A failed call's message, for gdn_last_error() (gdn_api.cu); returns s.
gdn_status api_fail(gdn_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// A call that succeeded: no message.
gdn_status api_ok();

}  // namespace gdn
