// Gated delta rule, token by token, on a pool of states (h = S^T, d_k x d_v, fp32):
//
//   p   = h^T k_t                          (= S_{t-1} k_t)
//   u   = beta_t (v_t - alpha_t p)
//   h  <- alpha_t h + k_t u^T
//   o_t = h^T q_t
//
// Two kernels: one token a sequence (step), and ragged sequences.
#include <cuda_bf16.h>

#include <type_traits>

#include "f32x2.cuh"
#include "gdn_serve.cuh"

namespace gdn {
namespace {

constexpr int kGroups = 8;      // threads that share a column's d_k rows

// Sequence whose cu_seqlens range or slot is out of bounds: 1 + its index.
__device__ unsigned int g_pool_error = 0;

__device__ __forceinline__ float load1(const void *p, int64_t i, bool bf16) {
    if (bf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
    return reinterpret_cast<const float *>(p)[i];
}

// N consecutive numbers as they lie in memory, so that they wait in as few registers
// as they have bytes, and nothing waits for them before they are used.
template <int N, bool BF16>
struct Raw {
    static constexpr int kWords = BF16 ? (N + 1) / 2 : N;
    uint32_t w[kWords];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < kWords; ++j) w[j] = 0;
    }
    // VEC: base + i lies on N numbers' bytes, or on 16
    template <bool VEC>
    __device__ __forceinline__ void load(const void *base, int64_t i) {
        const char *from = reinterpret_cast<const char *>(base) + i * (BF16 ? 2 : 4);
        if constexpr (BF16 && N == 1) {
            w[0] = plain(reinterpret_cast<const uint16_t *>(from));
        } else if constexpr (VEC && kWords % 4 == 0) {
#pragma unroll
            for (int j = 0; j < kWords / 4; ++j) {
                const uint4 x = plain(reinterpret_cast<const uint4 *>(from) + j);
                w[4 * j] = x.x; w[4 * j + 1] = x.y; w[4 * j + 2] = x.z; w[4 * j + 3] = x.w;
            }
        } else if constexpr (VEC && kWords == 2) {
            const uint2 x = plain(reinterpret_cast<const uint2 *>(from));
            w[0] = x.x; w[1] = x.y;
        } else if constexpr (VEC || !BF16) {
#pragma unroll
            for (int j = 0; j < kWords; ++j) w[j] = plain(reinterpret_cast<const uint32_t *>(from) + j);
        } else {
            const uint16_t *x = reinterpret_cast<const uint16_t *>(from);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) w[j] = (uint32_t)plain(x + 2 * j) | ((uint32_t)plain(x + 2 * j + 1) << 16);
        }
    }
    __device__ __forceinline__ float get(int r) const {
        if constexpr (BF16) return __uint_as_float(r & 1 ? w[r / 2] & 0xffff0000u : w[r / 2] << 16);
        else return __uint_as_float(w[r]);
    }
};

__device__ __forceinline__ void store_o(const PoolParams &p, int64_t i, float x) {
    if (p.o_bf16) reinterpret_cast<__nv_bfloat16 *>(p.o)[i] = __float2bfloat16_rn(x);
    else reinterpret_cast<float *>(p.o)[i] = x;
}

// The state of sequence s (-1: none), and its rows.  False where nothing is to be done.
__device__ __forceinline__ bool sequence(const PoolParams &p, int s, int *slot, int *begin, int *end) {
    *begin = s;
    *end = s + 1;
    if (p.cu_seqlens) {
        *begin = p.cu_seqlens[s];
        *end = p.cu_seqlens[s + 1];
        if (*begin < 0 || *end < *begin || *end > p.rows) {
            if (threadIdx.x == 0) atomicCAS(&g_pool_error, 0u, (unsigned)s + 1u);
            return false;
        }
    }
    *slot = p.slots ? p.slots[s] : s;
    if (*slot < -1 || *slot >= p.pool) {
        if (threadIdx.x == 0) atomicCAS(&g_pool_error, 0u, (unsigned)s + 1u);
        *slot = -1;
    }
    return *begin < *end;
}

// One token a sequence.  Bound by reading and writing the states, 8 d_k d_v bytes
// a head (256 sequences x 16 heads of 128 x 128: 86 us, 96% of the copy rate).  A
// block takes one sequence, head and 1 / slices of its columns: thread = row group
// (8) x column quad, R = d_k / 8 rows by 4 columns in registers, so that a warp reads
// whole pieces of the state's rows.  With both sums over d_k taken from the old state,
//
//   o = h_new^T q = alpha (h^T q) + (k . q) u,
//
// they (and the squares of k and q, since both sums are linear in them) cross the
// block in one exchange through shared memory.
template <int QUADS>
struct StepShared {                      // of a block of up to QUADS column quads
    float4 sums[2][kGroups][QUADS];
    float dots[3][kGroups];
};
template <int R, bool BF16, bool VEC, int QUADS>
__device__ __forceinline__ void step(const PoolParams &p, int slot, int64_t t, int h, int slice, int slices, StepShared<QUADS> &shared) {
    auto &sums = shared.sums;
    auto &dots = shared.dots;
    const int pitch = p.dv / 4, quads = pitch / slices;      // float4 a row, and of this block
    const int group = threadIdx.x / quads, quad = threadIdx.x % quads;
    const int col = (slice * quads + quad) * 4;
    const int64_t oi = (t * p.H + h) * p.dv + col;
    const int row0 = group * R, hk = h / (p.H / p.Hk);
    float4 *hp = reinterpret_cast<float4 *>(p.state + (((int64_t)slot * p.H + h) * p.dk + row0) * p.dv + col);
    float4 x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = __ldcg(hp + r * pitch);
    Raw<R, BF16> k, q;
    k.template load<VEC>(p.k, t * p.k_row + (int64_t)hk * p.k_head + row0);
    q.template load<VEC>(p.q, t * p.q_row + (int64_t)hk * p.q_head + row0);
    float v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = load1(p.v, t * p.v_row + (int64_t)h * p.v_head + col + c, BF16);
    const float a = p.alpha ? plain(p.alpha + t * p.alpha_row + h) : 1.f;
    const float be = p.beta ? plain(p.beta + t * p.beta_row + h) : 1.f;

    float4 hk4 = make_float4(0.f, 0.f, 0.f, 0.f), hq4 = hk4;
    float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float kr = k.get(r), qr = q.get(r);
        hk4.x = fmaf(x[r].x, kr, hk4.x); hk4.y = fmaf(x[r].y, kr, hk4.y);
        hk4.z = fmaf(x[r].z, kr, hk4.z); hk4.w = fmaf(x[r].w, kr, hk4.w);
        hq4.x = fmaf(x[r].x, qr, hq4.x); hq4.y = fmaf(x[r].y, qr, hq4.y);
        hq4.z = fmaf(x[r].z, qr, hq4.z); hq4.w = fmaf(x[r].w, qr, hq4.w);
        kk = fmaf(kr, kr, kk); qq = fmaf(qr, qr, qq); kq = fmaf(kr, qr, kq);
    }
    sums[0][group][quad] = hk4;
    sums[1][group][quad] = hq4;
    if (quad == 0) { dots[0][group] = kk; dots[1][group] = qq; dots[2][group] = kq; }
    __syncthreads();
    kk = qq = kq = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) { kk += dots[0][g]; qq += dots[1][g]; kq += dots[2][g]; }
    const float kn = p.qk_norm ? 1.f / sqrtf(kk + p.qk_eps) : 1.f, qn = p.qk_norm ? 1.f / sqrtf(qq + p.qk_eps) : 1.f;
    auto total = [&](int i) {
        float4 y = sums[i][0][quad];
#pragma unroll
        for (int g = 1; g < kGroups; ++g) {
            const float4 z = sums[i][g][quad];
            y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
        }
        return y;
    };
    const float4 w = total(0);
    const float u[4] = {be * (v[0] - a * (kn * w.x)), be * (v[1] - a * (kn * w.y)), be * (v[2] - a * (kn * w.z)),
                        be * (v[3] - a * (kn * w.w))};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float kr = k.get(r) * kn;
        __stcg(hp + r * pitch, make_float4(fmaf(kr, u[0], a * x[r].x), fmaf(kr, u[1], a * x[r].y),
                                           fmaf(kr, u[2], a * x[r].z), fmaf(kr, u[3], a * x[r].w)));
    }
    if (group == 0) {
        const float4 y = total(1);
        const float b = kq * kn * qn, aq = a * qn;
        store_o(p, oi, fmaf(b, u[0], aq * y.x));
        store_o(p, oi + 1, fmaf(b, u[1], aq * y.y));
        store_o(p, oi + 2, fmaf(b, u[2], aq * y.z));
        store_o(p, oi + 3, fmaf(b, u[3], aq * y.w));
    }
}

template <int R, bool BF16, bool VEC>
__global__ void __launch_bounds__(256, 2) recurrent_step_kernel(const PoolParams p, int slices) {
    if (p.early) { grid_next(); grid_wait(); }
    const int slice = blockIdx.x % slices, sh = blockIdx.x / slices, s = sh / p.H, h = sh % p.H;
    int slot, t, end;
    if (!sequence(p, s, &slot, &t, &end)) return;
    if (slot < 0) {                      // no sequence: a zero row of o
        const int wide = p.dv / slices;
        if ((int)threadIdx.x < wide) store_o(p, ((int64_t)t * p.H + h) * p.dv + slice * wide + threadIdx.x, 0.f);
        return;
    }
    __shared__ StepShared<32> shared;
    step<R, BF16, VEC>(p, slot, t, h, slice, slices, shared);
}

__device__ __forceinline__ float xor_add(float x, int mask) { return x + __shfl_xor_sync(~0u, x, mask); }

constexpr int kCols = 16;       // value columns a warp
constexpr int kFour = 4;        // tokens a step of the ragged kernel takes at once

// The sequence of rank `rank` when those with more tokens come first, to within the
// power of two of their tokens: blocks start in order, and a long sequence that
// starts last leaves the device to itself.  Each block counts for itself.
template <int THREADS>
__device__ __forceinline__ int longest_first(const PoolParams &p, int rank) {
    __shared__ int count[33], found;
    auto bucket = [&](int s) {           // 32: none, else leading zeros of the tokens
        const int n = p.cu_seqlens[s + 1] - p.cu_seqlens[s];
        return n > 0 ? __clz(n) : 32;
    };
    if (threadIdx.x < 33) count[threadIdx.x] = 0;
    if (threadIdx.x == 0) found = rank;      // (a sequence whatever happens to cu_seqlens meanwhile)
    __syncthreads();
    for (int s = threadIdx.x; s < p.seqs; s += THREADS) atomicAdd(&count[bucket(s)], 1);
    __syncthreads();
    int mine = 0;
    for (; rank >= count[mine]; ++mine) rank -= count[mine];
    // the rank-th of that bucket, in order
    for (int first = 0; first < p.seqs; first += THREADS) {
        const int s = first + threadIdx.x;
        const bool is = s < p.seqs && bucket(s) == mine;
        const unsigned votes = __ballot_sync(~0u, is);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) count[threadIdx.x >> 5] = __popc(votes);
        __syncthreads();
        int before = __popc(votes & ((1u << (threadIdx.x & 31)) - 1)), all = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < (int)(threadIdx.x >> 5)) before += count[w];
            all += count[w];
        }
        if (is && before == rank) found = s;
        if (rank < all) break;
        rank -= all;
    }
    __syncthreads();
    return found;
}

template <int N>
__device__ __forceinline__ void store_few(float *p, const float (&x)[N]) {
    if constexpr (N == 4) *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else if constexpr (N == 2) *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
    else p[0] = x[0];
}

// Ragged sequences.  Columns of h never meet: a block takes one sequence, head and
// W NQ 16 columns, and each warp 16 NQ of them through all tokens, with h in registers.
// Lane = row group (8) x column quad (4), R = d_k / 8 rows by 4 columns NQ times, as
// pairs of rows for the two-float fma.
//
// The chain p -> u -> h would cost a token two exchanges over d_k, one after the
// other, so tokens go in fours, by forward substitution: with h = A g (A the product
// of the decays), P_i = g^T k_i and Q_i = g^T q_i of the four from the old g, and the
// dot products of the four's keys and queries,
//
//   u'_i = beta_i v_i / A_i - beta_i (P_i + sum_{j<i} (k_j . k_i) u'_j)
//   o_i  = A_i (Q_i + sum_{j<=i} (k_j . q_i) u'_j),     g <- g + sum_i k_i u'_i,
//
// which is the same recurrence in fp32 and has one exchange for the four.  Bound by
// its fma's, 3 for each of the d_k d_v cells of a token, two in an instruction.  A
// goes into g before it leaves [2^-32, 2^32]; a decay that would take it past
// [2^-64, 2^64] within four tokens ends the four early.
//
// The warps bring the tokens after next into shared memory, as fp32 and normalised,
// and form the next ones' dot products, beside the present ones.  A group's rows
// are interleaved, so that the groups' 16-byte reads of k and q meet in no bank.
// LONG: two fours between barriers, twice the registers, and the longest sequences
// first.  NQ = 2 reads a token's k and q once for twice the columns, at 8 warps a SM
// either way; at d_k 128 it spills a little of its 255 registers (132 bytes a thread in
// bf16, 644 in fp32).  48 sequences of 0 to 600 tokens (5155 in all), 32 heads of
// 128 x 128: 542 us (NQ = 1: 648); the fma's alone would take 225 (an f32x2 takes two
// cycles of its pipe).
template <int R, bool BF16, int W, bool LONG, int NQ>
__global__ void __launch_bounds__(W * 32, R < 16 ? 1 : LONG ? 8 / W : 12 / W) recurrent_ragged_kernel(const PoolParams p) {
    if (p.early) { grid_next(); grid_wait(); }
    constexpr int kBring = LONG ? 2 * kFour : kFour; // tokens between two barriers
    constexpr int kDk = R * kGroups, kThreads = W * 32, kWide = W * NQ * kCols;
    constexpr int kRun = R < 4 ? R : 4;              // consecutive rows
    constexpr int kMine = kBring / W;                // tokens of those a warp brings
    constexpr int kPer = (kDk + 31) / 32, kPerV = kWide / 32;   // numbers of k, v a lane brings
    constexpr int kDot = kThreads / (4 * kBring);    // threads that share a dot product
    constexpr int kParts = kDk / 4 < 8 ? kDk / 4 : 8;           // sums that a dot product is made of, whoever forms them
    constexpr int kDotParts = kParts < kDot ? 1 : kParts / kDot;
    static_assert(kDk / 4 % kParts == 0 && (kParts % kDot == 0 || kParts < kDot), "every product is a whole row's");
    __shared__ __align__(16) float ks[3][kBring][kDk], qs[3][kBring][kDk], vs[3][kBring][kWide];
    __shared__ __align__(16) float alphas[3][kBring], betas[3][kBring], kk[2][kBring][kFour], kq[2][kBring][kFour];
    __shared__ StepShared<W * 4> one;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slices = p.dv / kWide;
    const int slice = blockIdx.x % slices, h = blockIdx.x / slices % p.H;
    int s = blockIdx.x / slices / p.H;
    if (LONG && p.seqs <= 512) s = longest_first<kThreads>(p, s);     // (of more, the last is a small part)
    int slot, begin, end;
    if (!sequence(p, s, &slot, &begin, &end)) return;
    if (slot < 0) {                      // no sequence: zero rows of o
        for (int64_t t = begin; t < end; ++t)
            if (threadIdx.x < kWide) store_o(p, (t * p.H + h) * p.dv + slice * kWide + threadIdx.x, 0.f);
        return;
    }
    // A single token as in the kernel above, which has no tokens to bring (256 such sequences of 16
    // heads, 37 of them idle: 80 us, the other way 105); the block has the shape of a step's, NQ
    // times.  Here and in the order of the products' sums the variants agree, so that what a
    // sequence gives does not depend on the batch that chose the variant.
    if (end - begin == 1) {
#pragma unroll 1
        for (int z = 0; z < NQ; ++z) {
            if (z) __syncthreads();
            if (p.vec) step<R, BF16, true>(p, slot, begin, h, slice * NQ + z, slices * NQ, one);
            else step<R, BF16, false>(p, slot, begin, h, slice * NQ + z, slices * NQ, one);
        }
        return;
    }
    const int group = lane >> 2, quad = lane & 3, hk = h / (p.H / p.Hk);
    auto row_of = [&](int r) { return (group + kGroups * (r / kRun)) * kRun + r % kRun; };
    const int col0 = slice * kWide + warp * NQ * kCols;
    float4 *hp = reinterpret_cast<float4 *>(p.state + ((int64_t)slot * p.H + h) * p.dk * p.dv + col0) + quad;
    const int pitch = p.dv / 4;          // float4 a row
    F2 g[NQ][R / 2][4];

    // this warp's tokens of a bring, from memory (zeros behind the end): kPer consecutive
    // numbers of q and k a lane, kPerV of v
    Raw<kPer, BF16> kr[kMine], qr[kMine];
    Raw<kPerV, BF16> vr[kMine];
    float ar[kMine], br[kMine];
    const int in_row = lane * kPer, in_v = lane * kPerV;
    const int64_t ko = (int64_t)hk * p.k_head + in_row, qo = (int64_t)hk * p.q_head + in_row;
    const int64_t vo = (int64_t)h * p.v_head + slice * kWide + in_v;
    auto fetch = [&](int n) {
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const int64_t t = (int64_t)begin + n * kBring + warp + m * W;
            kr[m].zero(); qr[m].zero(); vr[m].zero();
            ar[m] = br[m] = 1.f;
            if (t < end) {
                if (in_row < kDk) {
                    if (p.vec) {
                        kr[m].template load<true>(p.k, t * p.k_row + ko);
                        qr[m].template load<true>(p.q, t * p.q_row + qo);
                    } else {
                        kr[m].template load<false>(p.k, t * p.k_row + ko);
                        qr[m].template load<false>(p.q, t * p.q_row + qo);
                    }
                }
                if (p.vec) vr[m].template load<true>(p.v, t * p.v_row + vo);
                else vr[m].template load<false>(p.v, t * p.v_row + vo);
                if (p.alpha) ar[m] = plain(p.alpha + t * p.alpha_row + h);
                if (p.beta) br[m] = plain(p.beta + t * p.beta_row + h);
            }
        }
    };
    auto keep = [&](int b) {
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const int i0 = warp + m * W;
            float k[kPer], q[kPer], v[kPerV];
#pragma unroll
            for (int i = 0; i < kPer; ++i) { k[i] = kr[m].get(i); q[i] = qr[m].get(i); }
#pragma unroll
            for (int i = 0; i < kPerV; ++i) v[i] = vr[m].get(i);
            if (p.qk_norm) {
                float x = 0.f, y = 0.f;
#pragma unroll
                for (int i = 0; i < kPer; ++i) { x = fmaf(k[i], k[i], x); y = fmaf(q[i], q[i], y); }
#pragma unroll
                for (int z = 1; z < 32; z *= 2) { x = xor_add(x, z); y = xor_add(y, z); }
                x = 1.f / sqrtf(x + p.qk_eps);
                y = 1.f / sqrtf(y + p.qk_eps);
#pragma unroll
                for (int i = 0; i < kPer; ++i) { k[i] *= x; q[i] *= y; }
            }
            if (in_row < kDk) {
                store_few<kPer>(&ks[b][i0][in_row], k);
                store_few<kPer>(&qs[b][i0][in_row], q);
            }
            store_few<kPerV>(&vs[b][i0][in_v], v);
            if (lane == 0) { alphas[b][i0] = ar[m]; betas[b][i0] = br[m]; }
        }
    };
    // for each four of a bring, 6 products k_i . k_j (j < i) and 10 q_i . k_j (j <= i), kDot threads each
    const int dot = threadIdx.x / kDot % 16, four = threadIdx.x / kDot / 16 * kFour, part = threadIdx.x % kDot;
    const int de = dot < 6 ? dot : dot - 6, dot_i0 = de < 1 ? 0 : de < 3 ? 1 : de < 6 ? 2 : 3;
    const int dot_j = de - dot_i0 * (dot_i0 + 1) / 2, dot_i = four + (dot < 6 ? dot_i0 + 1 : dot_i0);
    auto dots = [&](int b, int to) {
        const float4 *x = reinterpret_cast<const float4 *>(dot < 6 ? ks[b][dot_i] : qs[b][dot_i]) + part;
        const float4 *y = reinterpret_cast<const float4 *>(ks[b][four + dot_j]) + part;
        // kParts sums of every kParts-th four, joined by halves: the same order in every variant
        float sum[kDotParts];
#pragma unroll
        for (int i = 0; i < kDotParts; ++i) {
            sum[i] = 0.f;
            if (kParts < kDot && part >= kParts) break;
#pragma unroll
            for (int m = 0; m < kDk / 4 / kParts; ++m) {
                const float4 u = x[m * kParts + i * kDot], v = y[m * kParts + i * kDot];
                sum[i] = fmaf(u.x, v.x, fmaf(u.y, v.y, fmaf(u.z, v.z, fmaf(u.w, v.w, sum[i]))));
            }
        }
#pragma unroll
        for (int w = kDotParts / 2; w; w /= 2)
#pragma unroll
            for (int i = 0; i < w; ++i) sum[i] += sum[i + w];
#pragma unroll
        for (int m = kDot / 2; m; m /= 2) sum[0] = xor_add(sum[0], m);
        if (part == 0) (dot < 6 ? kk : kq)[to][dot_i][dot_j] = sum[0];
    };
    auto rows_at = [&](const float *x, F2 (&y)[R / 2]) {
#pragma unroll
        for (int r = 0; r < R; r += kRun) {
            if constexpr (kRun == 4) {
                const float4 z = *reinterpret_cast<const float4 *>(x + row_of(r));
                y[r / 2] = pack(z.x, z.y);
                y[r / 2 + 1] = pack(z.z, z.w);
            } else {
                const float2 z = *reinterpret_cast<const float2 *>(x + row_of(r));
                y[r / 2] = pack(z.x, z.y);
            }
        }
    };
    // this lane's sums over its rows of g with one token's numbers, by column
    auto partial = [&](const float *x, float (&y)[NQ][4]) {
        F2 xp[R / 2];
        rows_at(x, xp);
#pragma unroll
        for (int z = 0; z < NQ; ++z) {
            F2 acc[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[c] = mul2(g[z][0][c], xp[0]);
#pragma unroll
            for (int r = 1; r < R / 2; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[c] = fma2(g[z][r][c], xp[r], acc[c]);
#pragma unroll
            for (int c = 0; c < 4; ++c) y[z][c] = both(acc[c]);
        }
    };
    // halving exchange over bits 4 and 3: the sum of column 2 (bit 4) + (bit 3)
    const bool hi = lane & 16, odd = lane & 8, is_q = lane & 4;
    auto halve = [&](const float (&y)[4]) {
        const float a = (hi ? y[2] : y[0]) + __shfl_xor_sync(~0u, hi ? y[0] : y[2], 16);
        const float c = (hi ? y[3] : y[1]) + __shfl_xor_sync(~0u, hi ? y[1] : y[3], 16);
        return (odd ? c : a) + __shfl_xor_sync(~0u, odd ? a : c, 8);
    };

    const int mine = warp * NQ * kCols + quad * 4 + 2 * hi + odd; // the lane's (first) column after it
    const int64_t o_row = (int64_t)p.H * p.dv;
    int64_t oi = ((int64_t)begin * p.H + h) * p.dv + slice * kWide + mine;
    float A = 1.f;

    // `cnt` tokens from token i0 of the four that starts at token f of the bring in buffer b,
    // with products in buffer d; Ai: the decays up to each of them.  ALL: cnt = 4, i0 = 0.
    auto advance = [&](auto all, int b, int d, int f, int i0, int cnt, const float (&Ai)[kFour]) {
        constexpr bool ALL = decltype(all)::value;
        if (ALL) i0 = 0;
        const int at = f + i0;
        auto has = [&](int i) { return ALL || i < cnt; };
        float sum[NQ][kFour], u[NQ][kFour];      // P in the lanes with bit 2 clear, Q in those with it set
#pragma unroll
        for (int i = 0; i < kFour; ++i) {
            float P[NQ][4], Q[NQ][4];
            if (has(i)) {
                partial(ks[b][at + i], P);
                partial(qs[b][at + i], Q);
            } else {
#pragma unroll
                for (int z = 0; z < NQ; ++z)
#pragma unroll
                    for (int c = 0; c < 4; ++c) P[z][c] = Q[z][c] = 0.f;
            }
#pragma unroll
            for (int z = 0; z < NQ; ++z) {
                const float x = halve(P[z]), y = halve(Q[z]);
                sum[z][i] = (is_q ? y : x) + __shfl_xor_sync(~0u, is_q ? x : y, 4);
            }
        }
        // u' where P is, then across to where Q is
#pragma unroll
        for (int z = 0; z < NQ; ++z) {
#pragma unroll
            for (int i = 0; i < kFour; ++i) {
                float y = sum[z][i];
#pragma unroll
                for (int j = 0; j < i; ++j)
                    if (has(i)) y = fmaf(kk[d][at + i][i0 + j], u[z][j], y);
                u[z][i] = has(i) ? betas[b][at + i] * (__fdividef(vs[b][at + i][mine + z * kCols], Ai[i]) - y) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kFour; ++i) {
                const float y = __shfl_xor_sync(~0u, u[z][i], 4);
                if (is_q) u[z][i] = y;
            }
        }
#pragma unroll
        for (int i = 0; i < kFour; ++i)
            if (has(i)) {
#pragma unroll
                for (int z = 0; z < NQ; ++z) {
                    float y = sum[z][i];
#pragma unroll
                    for (int j = 0; j <= i; ++j) y = fmaf(kq[d][at + i][i0 + j], u[z][j], y);
                    if (is_q) store_o(p, oi + z * kCols, Ai[i] * y);
                }
                oi += o_row;
            }
#pragma unroll
        for (int i = 0; i < kFour; ++i) {
            float y[NQ][4];
#pragma unroll
            for (int z = 0; z < NQ; ++z) {
                const float un = __shfl_xor_sync(~0u, u[z][i], 8);
                const float u0 = odd ? un : u[z][i], u1 = odd ? u[z][i] : un;
                const float w0 = __shfl_xor_sync(~0u, u0, 16), w1 = __shfl_xor_sync(~0u, u1, 16);
                y[z][0] = hi ? w0 : u0; y[z][1] = hi ? w1 : u1; y[z][2] = hi ? u0 : w0; y[z][3] = hi ? u1 : w1;
            }
            if (has(i)) {
                F2 kp[R / 2];
                rows_at(ks[b][at + i], kp);
#pragma unroll
                for (int z = 0; z < NQ; ++z)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const F2 uu = pack(y[z][c], y[z][c]);
#pragma unroll
                        for (int r = 0; r < R / 2; ++r) g[z][r][c] = fma2(kp[r], uu, g[z][r][c]);
                    }
            }
        }
    };
    auto in = [](float x, float lo, float hi) { return x > lo && x < hi; };
    auto into_g = [&](float x) {
        const F2 f = pack(x, x);
#pragma unroll
        for (int z = 0; z < NQ; ++z)
#pragma unroll
            for (int r = 0; r < R / 2; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) g[z][r][c] = mul2(g[z][r][c], f);
    };

    const int brings = (end - begin - 1) / kBring + 1;
    fetch(0);                            // before the state: it is needed first
    float4 rows[NQ][R];
#pragma unroll
    for (int z = 0; z < NQ; ++z)
#pragma unroll
        for (int r = 0; r < R; ++r) rows[z][r] = __ldcg(hp + row_of(r) * pitch + z * (kCols / 4));
    keep(0);
    if (brings > 1) { fetch(1); keep(1); }
    if (brings > 2) fetch(2);
#pragma unroll
    for (int z = 0; z < NQ; ++z)
#pragma unroll
        for (int r = 0; r < R; r += 2) {
            const float4 x = rows[z][r], y = rows[z][r + 1];
            g[z][r / 2][0] = pack(x.x, y.x); g[z][r / 2][1] = pack(x.y, y.y);
            g[z][r / 2][2] = pack(x.z, y.z); g[z][r / 2][3] = pack(x.w, y.w);
        }
    __syncthreads();
    dots(0, 0);
    __syncthreads();
    int b = 0;                           // n % 3
    for (int n = 0; n < brings; ++n) {
        const int next = b == 2 ? 0 : b + 1, after = next == 2 ? 0 : next + 1;
        // bring n + 2, fetched one bring ago, takes the place of bring n - 1
        if (n + 2 < brings) keep(after);
        if (n + 3 < brings) fetch(n + 3);
#pragma unroll 1
        for (int f = 0; f < kBring; f += kFour) {
            const int tokens = min(kFour, end - begin - n * kBring - f);
            if (tokens <= 0) break;
            constexpr float kLo = 2.3283064e-10f, kHi = 4.2949673e9f, kLo2 = 5.4210109e-20f, kHi2 = 1.8446744e19f;   // 2^-+32, 2^-+64
            const float4 al = *reinterpret_cast<const float4 *>(&alphas[b][f]);
            float Ai[kFour];
            Ai[0] = A * al.x; Ai[1] = Ai[0] * al.y; Ai[2] = Ai[1] * al.z; Ai[3] = Ai[2] * al.w;
            if (tokens == kFour && in(Ai[0], kLo, kHi) && in(Ai[1], kLo2, kHi2) && in(Ai[2], kLo2, kHi2) && in(Ai[3], kLo2, kHi2)) {
                advance(std::true_type(), b, n & 1, f, 0, kFour, Ai);
                A = Ai[3];
            } else {
                for (int i0 = 0, cnt; i0 < tokens; i0 += cnt) {
                    Ai[0] = A * alphas[b][f + i0];
                    if (!in(Ai[0], kLo, kHi)) { into_g(Ai[0]); Ai[0] = 1.f; }
                    A = Ai[0];
                    cnt = 1;
#pragma unroll
                    for (int i = 1; i < kFour; ++i) {
                        Ai[i] = 1.f;
                        if (cnt == i && i0 + i < tokens) {
                            const float x = Ai[i - 1] * alphas[b][f + i0 + i];
                            if (in(x, kLo2, kHi2)) { Ai[i] = A = x; cnt = i + 1; }
                        }
                    }
                    advance(std::false_type(), b, n & 1, f, i0, cnt, Ai);
                }
            }
        }
        if (n + 1 < brings) dots(next, (n + 1) & 1);
        __syncthreads();
        b = next;
    }
#pragma unroll
    for (int z = 0; z < NQ; ++z)
#pragma unroll
        for (int r = 0; r < R; r += 2) {
            float x[4], y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) unpack(g[z][r / 2][c], &x[c], &y[c]);
            __stcg(hp + row_of(r) * pitch + z * (kCols / 4), make_float4(A * x[0], A * x[1], A * x[2], A * x[3]));
            __stcg(hp + row_of(r + 1) * pitch + z * (kCols / 4), make_float4(A * y[0], A * y[1], A * y[2], A * y[3]));
        }
}

template <typename... A, typename... B>
cudaError_t launch_blocks(bool early, void (*kernel)(PoolParams, A...), unsigned blocks, int threads, cudaStream_t stream, PoolParams p,
                          B... args) {
    p.early = early;
    return launch(p.early, kernel, dim3(blocks), dim3(threads), 0, stream, 1, p, args...);
}
template <int R, bool BF16, int W>
cudaError_t launch_ragged(const PoolParams &p, bool is_long, unsigned blocks, cudaStream_t stream) {
    return launch_blocks(is_early(blocks), is_long ? recurrent_ragged_kernel<R, BF16, W, true, 1> : recurrent_ragged_kernel<R, BF16, W, false, 1>,
                         blocks, W * 32, stream, p);
}
template <int R, bool BF16>
cudaError_t launch_r(const PoolParams &p, cudaStream_t stream) {
    const unsigned blocks = (unsigned)p.seqs * (unsigned)p.H;
    if (p.cu_seqlens) {
        // LONG where sequences have 16 tokens and more on average: 600 tokens of 16 heads 213 us
        // (288 the other way); 200 sequences of 1 to 8 tokens, 16 heads, 115 us (128).
        const bool is_long = p.rows / 16 >= p.seqs;
        // Two column quads a lane where whole heads still fill the SMs twice (48 sequences x 32
        // heads 545 us, with one 648); fewer are quicker on more blocks.
        if (is_long && p.dv == 128 && blocks >= 296)
            return launch_blocks(is_early(blocks), recurrent_ragged_kernel<R, BF16, 4, true, 2>, blocks, 128, stream, p);
        if (p.dv % 64 == 0) return launch_ragged<R, BF16, 4>(p, is_long, blocks * (p.dv / 64), stream);
        return launch_ragged<R, BF16, 2>(p, is_long, blocks * (p.dv / 32), stream);
    }
    // 64 columns a block (256 x 16 heads of 128 x 128: 86 us; 128 columns 90, 32 columns 90);
    // where the heads are fewer than two a SM, 32, so that more SMs take part (16 heads: 2.8 us,
    // with 64 columns 3.2, with 128 4.2).
    const int slices = blocks < 296 ? p.dv / 32 : p.dv % 64 ? 1 : p.dv / 64, threads = p.dv / 4 / slices * kGroups;
    // Begun early at every size: equal blocks have no order to lose (32 x 16 heads 14.7 us, 15.5
    // without; 128 x 32 heads 84.9, 85.8; 256 x 32 heads of 16 x 32 12.6, 13.0).
    return launch_blocks(true, p.vec ? recurrent_step_kernel<R, BF16, true> : recurrent_step_kernel<R, BF16, false>, blocks * slices, threads,
                         stream, p, slices);
}
template <int R>
cudaError_t launch_io(const PoolParams &p, cudaStream_t stream) {
    return p.io_bf16 ? launch_r<R, true>(p, stream) : launch_r<R, false>(p, stream);
}

}  // namespace

cudaError_t launch_recurrent_pool(const PoolParams &p, cudaStream_t stream) {
    switch (p.dk / kGroups) {
        case 2: return launch_io<2>(p, stream);
        case 4: return launch_io<4>(p, stream);
        case 8: return launch_io<8>(p, stream);
        case 16: return launch_io<16>(p, stream);
    }
    return cudaErrorInvalidValue;
}

unsigned int pool_read_and_clear_error(cudaError_t *err) {
    unsigned int v = 0, zero = 0;
    *err = cudaMemcpyFromSymbol(&v, g_pool_error, sizeof(v));
    if (*err == cudaSuccess && v) *err = cudaMemcpyToSymbol(g_pool_error, &zero, sizeof(zero));
    return v;
}

}  // namespace gdn
