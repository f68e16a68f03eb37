// Host side of the decode-layer operators: argument validation and launch.
#include <cstdlib>

#include "gdn_serve.cuh"

namespace {

using gdn::api_fail;
using gdn::api_ok;

struct Span {
    const char *begin, *end;
};

// The bytes from a strided array's first element to its last.
Span span(const void *p, int64_t rows, int64_t row, int64_t width, int64_t size) {
    const char *b = static_cast<const char *>(p);
    return {b, p && rows > 0 ? b + ((rows - 1) * row + width) * size : b};
}
Span span2(const void *p, int64_t rows, int64_t row, int64_t heads, int64_t head, int64_t width, int64_t size) {
    return span(p, rows, row, (heads - 1) * head + width, size);
}
bool overlap(const Span &a, const Span &b) { return a.begin < b.end && b.begin < a.end && a.begin < a.end && b.begin < b.end; }

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool on(const void *p, int64_t size) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(size - 1)) == 0; }
bool dtype_ok(int32_t t) { return t == GDN_F32 || t == GDN_BF16; }
int64_t size_of(int32_t t) { return t == GDN_BF16 ? 2 : 4; }

gdn_status resolve_pool(const gdn_recurrent_args *a, gdn::PoolParams *out) {
    if (!a) return api_fail(GDN_ERR_INVALID_ARG, "args is NULL");
    if (a->rows < 0 || a->seqs < 0) return api_fail(GDN_ERR_INVALID_ARG, "rows and seqs must be >= 0 (got %d, %d)", a->rows, a->seqs);
    if (a->H < 1 || a->Hk < 1 || a->H % a->Hk)
        return api_fail(GDN_ERR_INVALID_ARG, "H must be a multiple of Hk, both >= 1 (got %d, %d)", a->H, a->Hk);
    if (a->dk != 16 && a->dk != 32 && a->dk != 64 && a->dk != 128)
        return api_fail(GDN_ERR_INVALID_ARG, "dk must be 16, 32, 64 or 128 (got %d)", a->dk);
    if (a->dv != 32 && a->dv != 64 && a->dv != 96 && a->dv != 128)
        return api_fail(GDN_ERR_INVALID_ARG, "dv must be 32, 64, 96 or 128 (got %d)", a->dv);
    if (a->pool < 1) return api_fail(GDN_ERR_INVALID_ARG, "pool must be >= 1 (got %d)", a->pool);
    if (!dtype_ok(a->io_dtype) || !dtype_ok(a->o_dtype))
        return api_fail(GDN_ERR_INVALID_ARG, "dtype unknown (io %d, o %d)", a->io_dtype, a->o_dtype);
    if (a->qk_norm != 0 && a->qk_norm != 1) return api_fail(GDN_ERR_INVALID_ARG, "qk_norm must be 0 or 1");
    if (a->qk_norm && !(a->qk_eps > 0.f)) return api_fail(GDN_ERR_INVALID_ARG, "qk_norm needs qk_eps > 0");
    if (!a->cu_seqlens && a->rows != a->seqs)
        return api_fail(GDN_ERR_INVALID_ARG, "without cu_seqlens there is one token a sequence (got %d rows, %d sequences)", a->rows, a->seqs);
    if (!a->slots && a->pool < a->seqs)
        return api_fail(GDN_ERR_INVALID_ARG, "without slots the pool holds a state for every sequence (got %d, %d sequences)", a->pool, a->seqs);
    if (a->q_row < 0 || a->q_head < 0 || a->k_row < 0 || a->k_head < 0 || a->v_row < 0 || a->v_head < 0 ||
        a->alpha_row < 0 || a->beta_row < 0)
        return api_fail(GDN_ERR_INVALID_ARG, "strides must be >= 0");
    if ((int64_t)a->seqs * a->H > 0x7fffffff / 4) return api_fail(GDN_ERR_INVALID_ARG, "seqs * H too large");
    if (a->seqs > 0 && a->rows > 0) {
        if (!a->q || !a->k || !a->v || !a->o || !a->state)
            return api_fail(GDN_ERR_INVALID_ARG, "q, k, v, state and o are required");
        const int64_t io = size_of(a->io_dtype), od = size_of(a->o_dtype);
        if (!on16(a->state) || !on(a->q, io) || !on(a->k, io) || !on(a->v, io) || !on(a->o, od) || !on(a->alpha, 4) ||
            !on(a->beta, 4) || !on(a->cu_seqlens, 4) || !on(a->slots, 4))
            return api_fail(GDN_ERR_ALIGNMENT, "state must be 16-byte aligned, every other pointer aligned to its type");
        const Span ins[] = {span2(a->q, a->rows, a->q_row, a->Hk, a->q_head, a->dk, io),
                            span2(a->k, a->rows, a->k_row, a->Hk, a->k_head, a->dk, io),
                            span2(a->v, a->rows, a->v_row, a->H, a->v_head, a->dv, io),
                            span(a->alpha, a->rows, a->alpha_row, a->H, 4), span(a->beta, a->rows, a->beta_row, a->H, 4),
                            span(a->cu_seqlens, 1, 0, (int64_t)a->seqs + 1, 4), span(a->slots, 1, 0, a->seqs, 4)};
        const Span o = span(a->o, a->rows, (int64_t)a->H * a->dv, (int64_t)a->H * a->dv, od);
        const Span st = span(a->state, a->pool, (int64_t)a->H * a->dk * a->dv, (int64_t)a->H * a->dk * a->dv, 4);
        if (overlap(o, st)) return api_fail(GDN_ERR_INVALID_ARG, "o overlaps the states");
        for (const Span &x : ins)
            if (overlap(o, x) || overlap(st, x)) return api_fail(GDN_ERR_INVALID_ARG, "o or the states overlap an input");
    }
    gdn::PoolParams p{};
    p.rows = a->rows; p.seqs = a->seqs; p.H = a->H; p.Hk = a->Hk; p.dk = a->dk; p.dv = a->dv; p.pool = a->pool;
    p.io_bf16 = a->io_dtype == GDN_BF16; p.o_bf16 = a->o_dtype == GDN_BF16;
    p.qk_norm = a->qk_norm; p.qk_eps = a->qk_eps;
    p.q = a->q; p.k = a->k; p.v = a->v;
    p.q_row = a->q_row; p.q_head = a->q_head; p.k_row = a->k_row; p.k_head = a->k_head; p.v_row = a->v_row; p.v_head = a->v_head;
    p.alpha = a->alpha; p.beta = a->beta; p.alpha_row = a->alpha_row; p.beta_row = a->beta_row;
    p.cu_seqlens = a->cu_seqlens; p.slots = a->slots; p.state = a->state; p.o = a->o;
    const int64_t unit = 16 / size_of(a->io_dtype);
    p.vec = on16(a->q) && on16(a->k) && on16(a->v) && !(a->q_row % unit) && !(a->q_head % unit) && !(a->k_row % unit) &&
            !(a->k_head % unit) && !(a->v_row % unit) && !(a->v_head % unit);
    *out = p;
    return GDN_OK;
}

gdn_status resolve_rows(const gdn_rows_args *a, gdn::RowsParams *out) {
    if (!a) return api_fail(GDN_ERR_INVALID_ARG, "args is NULL");
    if (a->op < GDN_ROWS_PLAIN || a->op > GDN_ROWS_GATED) return api_fail(GDN_ERR_INVALID_ARG, "op %d unknown", a->op);
    if (a->rows < 0) return api_fail(GDN_ERR_INVALID_ARG, "rows must be >= 0 (got %d)", a->rows);
    if (a->width < 1) return api_fail(GDN_ERR_INVALID_ARG, "width must be >= 1 (got %d)", a->width);
    if (a->width > 32768) return api_fail(GDN_ERR_UNSUPPORTED, "rows of up to 32768 are held in registers (got %d)", a->width);
    if (!dtype_ok(a->x_dtype) || (a->residual && !dtype_ok(a->residual_dtype)) || (a->weight && !dtype_ok(a->weight_dtype)))
        return api_fail(GDN_ERR_INVALID_ARG, "dtype unknown (x %d, residual %d, weight %d)", a->x_dtype, a->residual_dtype, a->weight_dtype);
    const bool norm = a->op == GDN_ROWS_NORM, gated = a->op == GDN_ROWS_GATED;
    if ((norm || gated) && !(a->eps > 0.f)) return api_fail(GDN_ERR_INVALID_ARG, "eps must be > 0");
    if (!norm && (a->residual || a->residual_out)) return api_fail(GDN_ERR_INVALID_ARG, "a residual belongs to GDN_ROWS_NORM");
    if (!gated && a->gate) return api_fail(GDN_ERR_INVALID_ARG, "a gate belongs to GDN_ROWS_GATED");
    if (!norm && !gated && a->weight) return api_fail(GDN_ERR_INVALID_ARG, "GDN_ROWS_PLAIN takes no weight");
    if (gated) {
        if (a->head < 8 || a->head > 256 || a->head % 8 || a->width % a->head)
            return api_fail(GDN_ERR_INVALID_ARG, "head must be a multiple of 8 up to 256 that divides width (got %d, %d)", a->head, a->width);
        int lanes = 1;
        while (lanes * 8 < a->head) lanes *= 2;
        if (a->width / a->head * lanes > 4096)
            return api_fail(GDN_ERR_UNSUPPORTED, "%d heads of %d do not fit a block's registers", a->width / a->head, a->head);
    }
    if (a->x_row < 0 || a->residual_row < 0 || a->gate_row < 0 || a->residual_out_row < 0 || a->q_row < 0)
        return api_fail(GDN_ERR_INVALID_ARG, "strides must be >= 0");
    const int64_t xs = size_of(a->x_dtype), rs = size_of(a->residual_dtype), ws = size_of(a->weight_dtype);
    if (a->rows > 0) {
        if (!a->x || !a->q || !a->scale || (gated && !a->gate)) return api_fail(GDN_ERR_INVALID_ARG, "x, q, scale (and gate) are required");
        if (!a->residual != !a->residual_out) return api_fail(GDN_ERR_INVALID_ARG, "residual and residual_out come together");
        if (a->rows > 1 && (a->q_row < a->width || (a->residual_out && a->residual_out_row < a->width)))
            return api_fail(GDN_ERR_INVALID_ARG, "rows of an output overlap one another");
        if (!on(a->x, xs) || !on(a->gate, xs) || !on(a->residual, rs) || !on(a->residual_out, rs) || !on(a->weight, ws) || !on(a->scale, 4))
            return api_fail(GDN_ERR_ALIGNMENT, "pointers must be aligned to their types");
        const Span x = span(a->x, a->rows, a->x_row, a->width, xs), r = span(a->residual, a->rows, a->residual_row, a->width, rs);
        const Span g = span(a->gate, a->rows, a->gate_row, a->width, xs), w = span(a->weight, 1, 0, gated ? a->head : a->width, ws);
        const Span q = span(a->q, a->rows, a->q_row, a->width, 1), s = span(a->scale, 1, 0, a->rows, 4);
        const Span ro = span(a->residual_out, a->rows, a->residual_out_row, a->width, rs);
        const Span ins[] = {x, r, g, w};
        for (const Span &i : ins)
            if (overlap(q, i) || overlap(s, i)) return api_fail(GDN_ERR_INVALID_ARG, "q or scale overlaps an input");
        if (overlap(q, s) || overlap(q, ro) || overlap(s, ro)) return api_fail(GDN_ERR_INVALID_ARG, "outputs overlap one another");
        // in place: each element is read, by the thread that writes it, before it is written
        const bool is_r = a->residual_out == a->residual && a->residual_out_row == a->residual_row;
        const bool is_x = a->residual_out == a->x && a->residual_out_row == a->x_row && a->residual_dtype == a->x_dtype;
        if (overlap(ro, w) || (overlap(ro, r) && !is_r) || (overlap(ro, x) && !is_x))
            return api_fail(GDN_ERR_INVALID_ARG, "residual_out overlaps an input that it is not");
    }
    gdn::RowsParams p{};
    p.op = a->op; p.rows = a->rows; p.width = a->width; p.head = gated ? a->head : 1;
    p.x_bf16 = a->x_dtype == GDN_BF16; p.residual_bf16 = a->residual_dtype == GDN_BF16; p.weight_bf16 = a->weight_dtype == GDN_BF16;
    p.eps = a->eps; p.inverse = 1.f / (float)(gated ? a->head : a->width);
    p.x = a->x; p.residual = a->residual; p.gate = a->gate; p.weight = a->weight;
    p.x_row = a->x_row; p.residual_row = a->residual_row; p.gate_row = a->gate_row;
    p.residual_out_row = a->residual_out_row; p.q_row = a->q_row;
    p.residual_out = a->residual_out; p.q = a->q; p.scale = a->scale;
    const auto rows16 = [](const void *ptr, int64_t row, int64_t size) { return !ptr || (on16(ptr) && row * size % 16 == 0); };
    p.in_place = a->residual_out && (a->residual_out == a->residual || a->residual_out == a->x);
    p.weight_vec = on16(a->weight);
    p.q_vec = on(a->q, 8) && (a->q_row % 8 == 0 || a->rows == 1);
    p.vec = a->width % 8 == 0 && rows16(a->x, a->x_row, xs) && rows16(a->residual, a->residual_row, rs) &&
            rows16(a->gate, a->gate_row, xs) && rows16(a->residual_out, a->residual_out_row, rs) &&
            p.weight_vec && p.q_vec;
    *out = p;
    return GDN_OK;
}

// Rows that the tensor memory accelerator can read where they are.
bool tma_rows(const void *p, int64_t row, int rows) { return on16(p) && (rows == 1 || (row > 0 && row % 16 == 0)); }
int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }

struct MatmulPlan {
    gdn::Int8MatmulParams p;
    bool copy_x, copy_w;
    uint64_t workspace;
};

gdn_status resolve_matmul(const gdn_int8_matmul_args *a, MatmulPlan *out) {
    if (!a) return api_fail(GDN_ERR_INVALID_ARG, "args is NULL");
    if (a->M < 0 || a->N < 1 || a->K < 1) return api_fail(GDN_ERR_INVALID_ARG, "M must be >= 0, N and K >= 1 (got %d, %d, %d)", a->M, a->N, a->K);
    if (a->K > 131071) return api_fail(GDN_ERR_UNSUPPORTED, "K must be <= 131071 for the sum to fit 32 bits (got %d)", a->K);
    if ((int64_t)a->M * a->N > ((int64_t)1 << 40) || (int64_t)a->M + a->N > 0x7fffffff)
        return api_fail(GDN_ERR_INVALID_ARG, "M * N or M + N too large");
    if (!dtype_ok(a->out_dtype)) return api_fail(GDN_ERR_INVALID_ARG, "out_dtype %d unknown", a->out_dtype);
    if (a->x_row < 0 || a->w_row < 0 || a->out_row < 0) return api_fail(GDN_ERR_INVALID_ARG, "strides must be >= 0");
    MatmulPlan m{};
    const int64_t od = size_of(a->out_dtype), K16 = up16(a->K);
    if (a->M > 0) {
        if (!a->x || !a->w || !a->x_scale || !a->w_scale || !a->out)
            return api_fail(GDN_ERR_INVALID_ARG, "x, w, x_scale, w_scale and out are required");
        if (!on(a->x_scale, 4) || !on(a->w_scale, 4) || !on(a->bias, 4) || !on(a->out, od))
            return api_fail(GDN_ERR_ALIGNMENT, "scales, bias and out must be aligned to their types");
        if (a->M > 1 && a->out_row < a->N) return api_fail(GDN_ERR_INVALID_ARG, "rows of out overlap one another");
        m.copy_x = !tma_rows(a->x, a->x_row, a->M);
        m.copy_w = !tma_rows(a->w, a->w_row, a->N);
        const uint64_t xb = m.copy_x ? (uint64_t)a->M * K16 : 0, wb = m.copy_w ? (uint64_t)a->N * K16 : 0;
        m.workspace = xb + wb;
        const Span o = span(a->out, a->M, a->out_row, a->N, od), ws = span(a->workspace, 1, 0, (int64_t)m.workspace, 1);
        const Span ins[] = {span(a->x, a->M, a->x_row, a->K, 1), span(a->w, a->N, a->w_row, a->K, 1),
                            span(a->x_scale, 1, 0, a->M, 4), span(a->w_scale, 1, 0, a->N, 4), span(a->bias, 1, 0, a->N, 4)};
        if (overlap(o, ws)) return api_fail(GDN_ERR_INVALID_ARG, "out overlaps the workspace");
        for (const Span &i : ins)
            if (overlap(o, i) || overlap(ws, i)) return api_fail(GDN_ERR_INVALID_ARG, "out or the workspace overlaps an input");
    }
    m.p = {a->M, a->N, a->K, a->out_dtype == GDN_BF16, a->x, a->w, a->x_row, a->w_row, a->out_row, a->x_scale, a->w_scale, a->bias, a->out};
    if (a->M == 1) m.p.x_row = K16;      // a single row's stride is any number
    if (a->N == 1) m.p.w_row = K16;
    *out = m;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_recurrent_fwd(const gdn_recurrent_args *args, void *stream) {
    gdn::PoolParams p;
    const gdn_status s = resolve_pool(args, &p);
    if (s != GDN_OK) return s;
    if (p.seqs == 0 || p.rows == 0) return api_ok();
    const cudaError_t e = gdn::launch_recurrent_pool(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return api_fail(GDN_ERR_CUDA, "recurrent launch: %s", cudaGetErrorString(e));
    return api_ok();
}

gdn_status gdn_rows_int8(const gdn_rows_args *args, void *stream) {
    gdn::RowsParams p;
    const gdn_status s = resolve_rows(args, &p);
    if (s != GDN_OK) return s;
    if (p.rows == 0) return api_ok();
    const cudaError_t e = gdn::launch_rows_int8(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return api_fail(GDN_ERR_CUDA, "rows launch: %s", cudaGetErrorString(e));
    return api_ok();
}

uint64_t gdn_int8_matmul_workspace_bytes(const gdn_int8_matmul_args *args) {
    MatmulPlan m;
    if (resolve_matmul(args, &m) != GDN_OK) return 0;
    api_ok();
    return m.workspace;
}

gdn_status gdn_int8_matmul(const gdn_int8_matmul_args *args, void *stream) {
    MatmulPlan m;
    const gdn_status s = resolve_matmul(args, &m);
    if (s != GDN_OK) return s;
    if (m.p.M == 0) return api_ok();
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (m.workspace) {
        if (!args->workspace || args->workspace_bytes < m.workspace)
            return api_fail(GDN_ERR_INVALID_ARG, "the copies of unaligned rows need a workspace of %llu bytes (got %llu)",
                            (unsigned long long)m.workspace, (unsigned long long)args->workspace_bytes);
        if (!on16(args->workspace)) return api_fail(GDN_ERR_ALIGNMENT, "the workspace must be 16-byte aligned");
        int8_t *to = static_cast<int8_t *>(args->workspace);
        const int64_t row = up16(m.p.K);
        gdn::PadRows x{}, w{};
        if (m.copy_x) {
            x = {m.p.x, m.p.x_row, to, row, m.p.M};
            m.p.x = to; m.p.x_row = row;
            to += (int64_t)m.p.M * row;
        }
        if (m.copy_w) {
            w = {m.p.w, m.p.w_row, to, row, m.p.N};
            m.p.w = to; m.p.w_row = row;
        }
        e = gdn::launch_int8_pad_rows(x, w, m.p.K, st);
    }
    const char *why = "";
    if (e == cudaSuccess) e = gdn::launch_int8_matmul(m.p, st, &why);
    if (e != cudaSuccess) return api_fail(GDN_ERR_CUDA, "int8 product launch: %s %s", cudaGetErrorString(e), why);
    return api_ok();
}

}  // extern "C"
