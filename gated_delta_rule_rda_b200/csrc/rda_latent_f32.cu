// Latent attention on the fp32 pipes: the expanded form (forward and
// gradients) and the absorbed form over a paged cache.
//
//   s_ij = scale (q_i . k_j + q~_i . k~_j),  p = softmax_j s,  o_i = sum_j p_ij v_j
//   ds_ij = p_ij (do_i . v_j - do_i . o_i),  dq = scale ds k,  dk = scale ds^T q,  dv = p^T do
//
// fp32 inputs are held to fp32 accuracy, which one product of 16- or 19-bit
// tensor-core operands does not give.  Operands split in two or three terms would
// (rda_decode_tokens does so), at three to six products each; these kernels are
// the simpler form, on FMAs: register tiles of 4 x 4 scores and 4 x (D / 16)
// outputs a thread, operands as fp32 rows in shared memory (a row stride of D + 4
// floats keeps the 128-bit reads of eight consecutive rows on different banks).
// Bound by the reads of shared memory that feed the FMAs, at a quarter to two
// fifths of the FMA rate (74 TFLOP/s).
//
// Measured, 16 heads of 128 + 64 and 128, causal: T = 1100 in 247 us, T = 2000 in 678
// us (25 and 30 TFLOP/s), gradients of T = 900 in 621 us (17); two heads, T = 256: 7.9
// us and 3.9 us for the join.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "rda_io.cuh"
#include "rda_latent.h"
#include "sm100_ptx.cuh"

namespace rda {
namespace {

constexpr int kTile = 64;         // query rows and keys per tile
constexpr int kThreads = 256;
constexpr int kLdP = kTile + 4;

// Rows [row0, row0 + n) of head h as fp32 into dst[64][ld]: `part` ([rows, H, D0])
// and behind it `shared` ([rows, Hs, D1], the same for every head if Hs = 1).
// Rows from n on are zero, whatever lies behind a sequence.
template <typename T, int ROWS = kTile, int NT = kThreads>
__device__ __forceinline__ void load_rows(float *dst, int ld, const T *part, int D0, const T *shared, int D1, int Hs,
                                          long row0, int n, int H, int h) {
    // 16 threads a row
    const int r0 = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * 4;
#pragma unroll
    for (int r = r0; r < ROWS; r += NT / 16) {
        const size_t row = (size_t)(row0 + r);
#pragma unroll 3
        for (int c = c0; c < D0 + D1; c += 64) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < n)
                x = c < D0 ? Io<T>::ld4(part + (row * H + h) * D0 + c)
                           : Io<T>::ld4(shared + (row * Hs + (Hs == 1 ? 0 : h)) * D1 + (c - D0));
            *reinterpret_cast<float4 *>(dst + r * ld + c) = x;
        }
    }
}

// The same copied asynchronously (fp32).
template <int ROWS, int NT>
__device__ __forceinline__ void copy_rows(float *dst, int ld, const float *part, int D0, const float *shared, int D1, int Hs,
                                          long row0, int n, int H, int h) {
    const int r0 = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * 4;
#pragma unroll
    for (int r = r0; r < ROWS; r += NT / 16) {
        const size_t row = (size_t)(row0 + min(r, n - 1));
        for (int c = c0; c < D0 + D1; c += 64)
            cp_async16_or_zero((uint32_t)__cvta_generic_to_shared(dst + r * ld + c),
                               c < D0 ? part + (row * H + h) * D0 + c : shared + (row * Hs + (Hs == 1 ? 0 : h)) * D1 + (c - D0),
                               r < n ? 16 : 0);
    }
}

// acc[i][j] += a[RI ty + i] . b[tx + 16 j] over D
template <int RI>
__device__ __forceinline__ void dot(float (&acc)[RI][4], const float *a, int lda, const float *b, int ldb, int D) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float *ar = a + RI * ty * lda, *br = b + tx * ldb;
#pragma unroll(RI == 1 ? 8 : 2)
    for (int d = 0; d < D; d += 4) {
        float4 x[RI], y[4];
#pragma unroll
        for (int i = 0; i < RI; ++i) x[i] = *reinterpret_cast<const float4 *>(ar + i * lda + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = *reinterpret_cast<const float4 *>(br + 16 * i * ldb + d);
#pragma unroll
        for (int i = 0; i < RI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, acc[i][j]))));
    }
}

// acc[i][4 c ..] += sum_j w[RI ty + i][j] b[j][64 c + 4 tx ..]   (w row-major)
template <int RI, int NC>
__device__ __forceinline__ void rows_times(float (&acc)[RI][NC][4], const float *w, const float *b, int ldb) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll(RI == 1 ? 4 : 1)
    for (int j = 0; j < kTile; j += 4) {
        float4 x[RI];
#pragma unroll
        for (int i = 0; i < RI; ++i) x[i] = *reinterpret_cast<const float4 *>(w + (RI * ty + i) * kLdP + j);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const float4 y = *reinterpret_cast<const float4 *>(b + (j + u) * ldb + 64 * c + 4 * tx);
#pragma unroll
                for (int i = 0; i < RI; ++i) {
                    const float p = u == 0 ? x[i].x : u == 1 ? x[i].y : u == 2 ? x[i].z : x[i].w;
                    acc[i][c][0] = fmaf(p, y.x, acc[i][c][0]);
                    acc[i][c][1] = fmaf(p, y.y, acc[i][c][1]);
                    acc[i][c][2] = fmaf(p, y.z, acc[i][c][2]);
                    acc[i][c][3] = fmaf(p, y.w, acc[i][c][3]);
                }
            }
    }
}
// Columns [64 c, 64 c + 64) of 64 rows to out ([rows, H, D0]) or, from column
// D0 on, to shared ([rows, H, D1]).
template <typename T, typename U, int RI, int NC>
__device__ __forceinline__ void store_rows(const float (&acc)[RI][NC][4], float f, T *out, int D0, U *shared, int D1,
                                           long row0, int n, int H, int h) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        if (RI * ty + i >= n) continue;
        const size_t row = (size_t)(row0 + RI * ty + i) * H + h;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = 64 * c + 4 * tx;
            const float4 x = make_float4(f * acc[i][c][0], f * acc[i][c][1], f * acc[i][c][2], f * acc[i][c][3]);
            if (col < D0) Io<T>::st4(out + row * D0 + col, x);
            else Io<U>::st4(shared + row * D1 + (col - D0), x);
        }
    }
}

__device__ __forceinline__ bool seen(const LatentArgs &a, int i, int j, int lq, int lk) {
    return i < lq && j < lk && (!a.causal || j <= i + lk - lq);
}

// ---------------------------------------------------------------------------
// Forward: one CTA per (RI NT / 16 query rows, head), online softmax over key
// tiles.  RI = 4 with 512 threads (128 rows) or 256 (64) reads each operand for four
// products; RI = 1 with 256 threads (16 rows) makes eight times
// as many CTAs, for calls that would leave SMs empty, copies the next key tile
// while it works on one, and may split the keys over `splits` CTAs (blockIdx.z),
// whose results a second kernel joins.  Two heads of 256 queries: 22.5 us with 16
// rows, 7.9 + 3.9 us with split keys; three heads of 100, 300 and 77: 139 -> 69 us.
// ---------------------------------------------------------------------------
template <typename T, int NDV, int RI, int NT>
__global__ void __launch_bounds__(NT) latent_forward_f32_kernel(LatentArgs a, int splits) {
    extern __shared__ __align__(16) float smem[];
    constexpr int M = RI * NT / 16;
    const int D = a.Dk + a.Ds, ld = D + 4, ldv = 64 * NDV + 4;
    constexpr int BUF = RI == 1 ? 2 : 1;
    float *Qs = smem, *Ps = Qs + M * ld, *KV = Ps + M * kLdP;
    int t;
    // the last tiles of a sequence see the most keys: start with them
    const int n = find_tile(a.cu_q, a.num_seqs, a.total_q, M, (int)((gridDim.x - 1 - blockIdx.x) / a.H), &t);
    const SeqSpan sq = seq_span(a.cu_q, n, a.total_q), sk = seq_span(a.cu_k, n, a.total_k);
    const int h = blockIdx.x % a.H, r0 = t * M;
    const int rows = min(M, sq.len - r0);
    if (rows <= 0) return;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    load_rows<T, M, NT>(Qs, ld, (const T *)a.q, a.Dk, (const T *)a.q_shared, a.Ds, a.H, sq.start + r0, rows, a.H, h);
    float o[RI][NDV][4] = {}, m[RI], l[RI];
#pragma unroll
    for (int i = 0; i < RI; ++i) m[i] = -INFINITY, l[i] = 0.f;
    const int kend = a.causal ? min(sk.len, r0 + rows + sk.len - sq.len) : sk.len;
    auto copy = [&](int k0) {
        float *Ks = KV + (k0 / kTile % BUF) * kTile * (ld + ldv), *Vs = Ks + kTile * ld;
        const int n = min(kTile, sk.len - k0);
        copy_rows<kTile, NT>(Ks, ld, (const float *)a.k, a.Dk, (const float *)a.k_shared, a.Ds, 1, sk.start + k0, n, a.H, h);
        copy_rows<kTile, NT>(Vs, ldv, (const float *)a.v, 64 * NDV, (const float *)nullptr, 0, 1, sk.start + k0, n, a.H, h);
        cp_async_commit();
    };
    const int all = kend > 0 ? (kend + kTile - 1) / kTile : 0;
    const int k_lo = RI == 1 ? all * (int)blockIdx.z / splits * kTile : 0;
    const int k_hi = RI == 1 ? min(kend, all * ((int)blockIdx.z + 1) / splits * kTile) : kend;
    if (BUF == 2 && k_lo < k_hi) copy(k_lo);
    for (int k0 = k_lo; k0 < k_hi; k0 += kTile) {
        float *Ks = KV + (k0 / kTile % BUF) * kTile * (ld + ldv), *Vs = Ks + kTile * ld;
        if (BUF == 1) {
            __syncthreads();
            copy(k0);
        }
        cp_async_wait_all();
        __syncthreads();
        if (BUF == 2 && k0 + kTile < k_hi) copy(k0 + kTile);
        float s[RI][4] = {};
        dot<RI>(s, Qs, ld, Ks, ld, D);
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            const int r = r0 + RI * ty + i;
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = seen(a, r, k0 + tx + 16 * j, sq.len, sk.len) ? s[i][j] * a.scale : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int off = 8; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float base = top == -INFINITY ? 0.f : top;    // nothing seen so far: every p is e^-inf
            const float keep = expf(m[i] - base);
            m[i] = top;
            l[i] *= keep;
#pragma unroll
            for (int c = 0; c < NDV; ++c)
#pragma unroll
                for (int u = 0; u < 4; ++u) o[i][c][u] *= keep;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = expf(s[i][j] - base);
                l[i] += p;
                Ps[(RI * ty + i) * kLdP + tx + 16 * j] = p;
            }
        }
        __syncthreads();
        rows_times<RI, NDV>(o, Ps, Vs, ldv);
    }
#pragma unroll
    for (int i = 0; i < RI; ++i) {
#pragma unroll
        for (int off = 8; off; off >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
        const int r = r0 + RI * ty + i;
        if (tx == 0 && RI * ty + i < rows) {
            const size_t at = (size_t)(sq.start + r) * a.H + h;
            const float lse = l[i] > 0.f ? m[i] + logf(l[i]) : -INFINITY;
            if (RI == 1 && splits > 1) a.delta[at * splits + blockIdx.z] = lse;
            else if (a.lse) a.lse[at] = lse;
        }
        const float f = l[i] > 0.f ? 1.f / l[i] : 0.f;
#pragma unroll
        for (int c = 0; c < NDV; ++c)
#pragma unroll
            for (int u = 0; u < 4; ++u) o[i][c][u] *= f;
    }
    if (RI == 1 && splits > 1) {
        // a part: [row][split][Dv] behind the log-sum-exps
        const size_t rows_all = (size_t)a.total_q * a.H, at = ((size_t)(sq.start + r0 + ty) * a.H + h) * splits + blockIdx.z;
        float *po = a.delta + ((rows_all * splits + 3) & ~(size_t)3) + at * (64 * NDV);
        if (ty < rows)
#pragma unroll
            for (int c = 0; c < NDV; ++c)
                *reinterpret_cast<float4 *>(po + 64 * c + 4 * tx) = make_float4(o[0][c][0], o[0][c][1], o[0][c][2], o[0][c][3]);
        return;
    }
    store_rows<T, T, RI, NDV>(o, 1.f, (T *)a.out, 64 * NDV, (T *)nullptr, 0, sq.start + r0, rows, a.H, h);
}

// ---------------------------------------------------------------------------
// Gradients.  One kernel for both sides: a CTA owns 16 RI rows of the one side
// (keys: dk, dv; or query rows: dq) with their sums in registers, and walks over
// the other side's rows that they meet, 32 at a time, the next 32 copied
// meanwhile.  No sum depends on the order of atomics; the price is that the
// scores and do . v are formed twice.
//
//   w[own][other] = ds (and p for keys):  acc[own] += w[own][..] other's rows
//
// 4 x 8 lanes a warp: with RI = 4 a thread's products over four columns read six
// 128-byte rows of shared memory for 32 FMAs a lane, its sums 16 for 192.  RI = 2
// makes twice the CTAs, where 64 rows each would leave SMs empty (80 tiles of 64: 177
// us against 231; 120: 470 and 614; but 240 of them: 821 and 620).
// Measured (16 heads of 128 + 64 and 128, T = 900, causal): 621 us for both sides, 899
// with a head's tiles side by side instead of the heads (an SM idle for half the
// time), 997 without the copies meanwhile and with 2 x 16 lanes a warp.
// ---------------------------------------------------------------------------
constexpr int kMov = 32, kLdW = 40;

// acc[i][j] = a[16 i] . b[16 j], rows of ld floats, over D
template <int RI>
__device__ __forceinline__ void dot_rows(float (&acc)[RI][2], const float *a, const float *b, int ld, int D) {
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
        float4 x[RI], y[2];
#pragma unroll
        for (int i = 0; i < RI; ++i) x[i] = *reinterpret_cast<const float4 *>(a + 16 * i * ld + d);
#pragma unroll
        for (int j = 0; j < 2; ++j) y[j] = *reinterpret_cast<const float4 *>(b + 16 * j * ld + d);
#pragma unroll
        for (int i = 0; i < RI; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, acc[i][j]))));
    }
}

// acc[i][c] += sum_m w[16 i][m] b[m][64 c ..]
template <int RI, int NC>
__device__ __forceinline__ void add_rows(float (&acc)[RI][NC][4], const float *w, const float *b, int ldb) {
#pragma unroll 2
    for (int m = 0; m < kMov; m += 4) {
        float4 x[RI];
#pragma unroll
        for (int i = 0; i < RI; ++i) x[i] = *reinterpret_cast<const float4 *>(w + 16 * i * kLdW + m);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const float4 y = *reinterpret_cast<const float4 *>(b + (m + u) * ldb + 64 * c);
#pragma unroll
                for (int i = 0; i < RI; ++i) {
                    const float p = u == 0 ? x[i].x : u == 1 ? x[i].y : u == 2 ? x[i].z : x[i].w;
                    acc[i][c][0] = fmaf(p, y.x, acc[i][c][0]);
                    acc[i][c][1] = fmaf(p, y.y, acc[i][c][1]);
                    acc[i][c][2] = fmaf(p, y.z, acc[i][c][2]);
                    acc[i][c][3] = fmaf(p, y.w, acc[i][c][3]);
                }
            }
    }
}

constexpr size_t grad_smem(int ND, int NDV, int RI, bool keys) {
    return sizeof(float) * ((16 * RI + 2 * kMov) * (64 * ND + 4 + 64 * NDV + 4) + (keys ? 2 : 1) * 16 * RI * kLdW +
                            (keys ? 4 * kMov : 32 * RI));
}

template <int ND, int NDV, int RI, bool KEYS>
__global__ void __launch_bounds__(kThreads) latent_grad_f32_kernel(LatentArgs a) {
    extern __shared__ __align__(16) float smem[];
    constexpr int OWN = 16 * RI, D = 64 * ND, ld = D + 4, Dv = 64 * NDV, ldv = Dv + 4;
    float *A1 = smem, *A2 = A1 + OWN * ld, *B1 = A2 + OWN * ldv, *B2 = B1 + 2 * kMov * ld, *W1 = B2 + 2 * kMov * ldv,
          *W2 = W1 + OWN * kLdW, *stat = W2 + (KEYS ? OWN * kLdW : 0);      // lse, delta: of the rows walked over, or my own
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tx = (warp & 1) * 8 + (lane & 7), ty = (warp >> 1) * 4 + (lane >> 3);
    const int h = blockIdx.x % a.H, slot = blockIdx.x / a.H, slots = gridDim.x / a.H;
    int t;
    // the first keys are seen by the most queries, the last queries see the most keys
    const int n = KEYS ? find_tile(a.cu_k, a.num_seqs, a.total_k, OWN, slot, &t)
                       : find_tile(a.cu_q, a.num_seqs, a.total_q, OWN, slots - 1 - slot, &t);
    const SeqSpan sq = seq_span(a.cu_q, n, a.total_q), sk = seq_span(a.cu_k, n, a.total_k);
    const SeqSpan own = KEYS ? sk : sq, mov = KEYS ? sq : sk;
    const int o0 = t * OWN, count = min(OWN, own.len - o0), more = sk.len - sq.len;
    if (count <= 0) return;
    const int lo = KEYS && a.causal ? max(0, o0 - more) / kMov * kMov : 0;
    const int hi = KEYS || !a.causal ? mov.len : min(mov.len, o0 + count + more);
    const float *q = (const float *)a.q, *qs = (const float *)a.q_shared, *k = (const float *)a.k, *ks = (const float *)a.k_shared;
    copy_rows<OWN, kThreads>(A1, ld, KEYS ? k : q, a.Dk, KEYS ? ks : qs, a.Ds, KEYS ? 1 : a.H, own.start + o0, count, a.H, h);
    copy_rows<OWN, kThreads>(A2, ldv, (const float *)(KEYS ? a.v : a.d_out), Dv, (const float *)nullptr, 0, 1, own.start + o0,
                             count, a.H, h);
    auto copy = [&](int m0) {
        const int c = min(kMov, mov.len - m0), buf = (m0 / kMov) & 1;
        copy_rows<kMov, kThreads>(B1 + buf * kMov * ld, ld, KEYS ? q : k, a.Dk, KEYS ? qs : ks, a.Ds, KEYS ? a.H : 1,
                                  mov.start + m0, c, a.H, h);
        copy_rows<kMov, kThreads>(B2 + buf * kMov * ldv, ldv, (const float *)(KEYS ? a.d_out : a.v), Dv, (const float *)nullptr,
                                  0, 1, mov.start + m0, c, a.H, h);
        if (KEYS && tid < 2 * kMov) {
            const int r = tid % kMov;
            const size_t at = (size_t)(mov.start + m0 + r) * a.H + h;
            stat[buf * 2 * kMov + tid] = r < c ? (tid < kMov ? a.lse : a.delta)[at] : 0.f;
        }
    };
    if (!KEYS && tid < 2 * OWN) {
        const int r = tid % OWN;
        const size_t at = (size_t)(own.start + o0 + r) * a.H + h;
        stat[tid] = r < count ? (tid < OWN ? a.lse : a.delta)[at] : 0.f;
    }
    if (lo < hi) copy(lo);
    cp_async_commit();
    float acc1[RI][ND][4] = {}, acc2[RI][NDV][4] = {};
    for (int m0 = lo; m0 < hi; m0 += kMov) {
        const int buf = (m0 / kMov) & 1;
        const float *b1 = B1 + buf * kMov * ld, *b2 = B2 + buf * kMov * ldv, *st = stat + (KEYS ? buf * 2 * kMov : 0);
        cp_async_wait_all();
        __syncthreads();                              // these rows are here, the last ones used up
        if (m0 + kMov < hi) copy(m0 + kMov);
        cp_async_commit();
        float s[RI][2] = {}, dp[RI][2] = {};
        dot_rows<RI>(s, A1 + ty * ld, b1 + tx * ld, ld, D);
        dot_rows<RI>(dp, A2 + ty * ldv, b2 + tx * ldv, ldv, Dv);
#pragma unroll
        for (int i = 0; i < RI; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int o = ty + 16 * i, m = tx + 16 * j;
                const bool on = KEYS ? seen(a, m0 + m, o0 + o, sq.len, sk.len) : seen(a, o0 + o, m0 + m, sq.len, sk.len);
                const float lse = KEYS ? st[m] : st[o], delta = KEYS ? st[kMov + m] : st[OWN + o];
                const float p = on ? expf(s[i][j] * a.scale - lse) : 0.f;
                if (KEYS) W2[o * kLdW + m] = p;
                W1[o * kLdW + m] = on ? p * (dp[i][j] - delta) : 0.f;
            }
        __syncthreads();
        add_rows<RI, ND>(acc1, W1 + ty * kLdW, b1 + 4 * tx, ld);
        if (KEYS) add_rows<RI, NDV>(acc2, W2 + ty * kLdW, b2 + 4 * tx, ldv);
    }
    cp_async_wait_all();                              // nothing lands after the CTA has left
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        if (ty + 16 * i >= count) continue;
        const size_t row = (size_t)(own.start + o0 + ty + 16 * i) * a.H + h;
#pragma unroll
        for (int c = 0; c < ND; ++c) {
            const int col = 64 * c + 4 * tx;
            const float f = a.scale, *x = acc1[i][c];
            float *to = col < a.Dk ? (float *)(KEYS ? a.dk : a.dq) + row * a.Dk + col
                                   : (KEYS ? a.dks_heads : (float *)a.dq_shared) + row * a.Ds + (col - a.Dk);
            *reinterpret_cast<float4 *>(to) = make_float4(f * x[0], f * x[1], f * x[2], f * x[3]);
        }
        if (KEYS)
#pragma unroll
            for (int c = 0; c < NDV; ++c) {
                const float *x = acc2[i][c];
                *reinterpret_cast<float4 *>((float *)a.dv + row * Dv + 64 * c + 4 * tx) = make_float4(x[0], x[1], x[2], x[3]);
            }
    }
}

// delta_i = d_out_i . out_i: one warp per (row, head).
template <typename T>
__global__ void __launch_bounds__(256) latent_delta_kernel(const T *out, const T *d_out, float *delta, long rows, int Dv) {
    const long r = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (r >= rows) return;
    float x = 0.f;
    for (int c = 4 * lane; c < Dv; c += 128) {
        const float4 o = Io<T>::ld4(out + r * Dv + c), d = Io<T>::ld4(d_out + r * Dv + c);
        x = fmaf(o.x, d.x, fmaf(o.y, d.y, fmaf(o.z, d.z, fmaf(o.w, d.w, x))));
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if (lane == 0) delta[r] = x;
}

// dk_shared[row] = sum over heads of its per-head parts, heads in order.  Rows
// that belong to no sequence are left as they were.
template <typename T>
__global__ void __launch_bounds__(256) latent_shared_sum_kernel(const float *parts, T *out, const int32_t *cu_k,
                                                                int num_seqs, long rows, int H, int Ds) {
    ptx::pdl_launch_dependents();
    ptx::pdl_wait_primary();
    const long e = ((long)blockIdx.x * 256 + threadIdx.x) * 4;
    const long row = e / Ds;
    if (row >= rows || row < cu_k[0] || row >= cu_k[num_seqs]) return;
    const int c = (int)(e % Ds);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int h = 0; h < H; ++h) {
        const float4 y = *reinterpret_cast<const float4 *>(parts + ((size_t)row * H + h) * Ds + c);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    Io<T>::st4(out + row * Ds + c, x);
}

// Fewer tiles of 64 rows than SMs: smaller tiles; in the forward pass of 16, and the keys split until two CTAs per
// SM have work (8 at most).
bool few_tiles(int total, int H) { return (long)(total / kTile + 1) * H < kSms; }
int forward_splits(int total_q, int total_k, int H) {
    if (!few_tiles(total_q, H)) return 1;
    const long ctas = (long)(total_q / 16 + 1) * H, want = 2 * kSms / ctas, tiles = (total_k + kTile - 1) / kTile;
    return (int)std::max(1L, std::min({want, tiles, 8L}));
}

__global__ void latent_join_kernel(LatentDecodeArgs a, int splits, const int32_t *cu, int num_seqs);

template <typename T, int NDV, int RI, int NT> cudaError_t forward_ri(const LatentArgs &a, int splits, cudaStream_t s) {
    constexpr int M = RI * NT / 16;
    constexpr int BUF = RI == 1 ? 2 : 1;
    constexpr size_t most = sizeof(float) * (M * (192 + 4 + kLdP) + BUF * kTile * ((192 + 4) + (64 * NDV + 4)));
    cudaError_t e = allow_smem<latent_forward_f32_kernel<T, NDV, RI, NT>>(most);
    if (e != cudaSuccess) return e;
    const int ld = a.Dk + a.Ds + 4;
    const size_t bytes = sizeof(float) * (M * (ld + kLdP) + BUF * kTile * (ld + (64 * NDV + 4)));
    const dim3 grid(tile_slots(a.total_q, a.num_seqs, M) * a.H, 1, splits);
    latent_forward_f32_kernel<T, NDV, RI, NT><<<grid, NT, bytes, s>>>(a, splits);
    if ((e = cudaGetLastError()) != cudaSuccess || splits == 1) return e;
    LatentDecodeArgs j{};
    j.B = a.total_q, j.T = 1, j.H = a.H, j.Dl = 64 * NDV;
    j.out = a.out, j.lse = a.lse, j.part = a.delta;
    latent_join_kernel<<<a.total_q * a.H, 128, 0, s>>>(j, splits, a.cu_q, a.num_seqs);
    return cudaGetLastError();
}
template <typename T, int NDV> cudaError_t forward_nv(const LatentArgs &a, cudaStream_t s) {
    // 128 rows a CTA, unless 64 balance better: up to one and a half waves of them (16 heads of 1100 queries: 247 us
    // with 64 rows, 385 with 128; of 1500: 445 and 510; of 2000: 735 and 678).
    if (!few_tiles(a.total_q, a.H))
        return (long)(a.total_q / 128 + 1) * a.H < kSms * 3 / 2 ? forward_ri<T, NDV, 4, 256>(a, 1, s) : forward_ri<T, NDV, 4, 512>(a, 1, s);
    return forward_ri<T, NDV, 1, 256>(a, forward_splits(a.total_q, a.total_k, a.H), s);
}

template <int ND, int NDV, int RI, bool KEYS> cudaError_t grad_ri(const LatentArgs &a, cudaStream_t s) {
    constexpr size_t bytes = grad_smem(ND, NDV, RI, KEYS);
    const cudaError_t e = allow_smem<latent_grad_f32_kernel<ND, NDV, RI, KEYS>>(bytes);
    if (e != cudaSuccess) return e;
    const int grid = tile_slots(KEYS ? a.total_k : a.total_q, a.num_seqs, 16 * RI) * a.H;      // heads side by side
    latent_grad_f32_kernel<ND, NDV, RI, KEYS><<<grid, kThreads, bytes, s>>>(a);
    return cudaGetLastError();
}
template <int ND, int NDV, bool KEYS> cudaError_t grad(const LatentArgs &a, cudaStream_t s) {
    const int total = KEYS ? a.total_k : a.total_q;
    if (total == 0) return cudaSuccess;
    return few_tiles(total, a.H) ? grad_ri<ND, NDV, 2, KEYS>(a, s) : grad_ri<ND, NDV, 4, KEYS>(a, s);
}
template <int ND, int NDV> cudaError_t backward_nd(const LatentArgs &a, cudaStream_t s) {
    const cudaError_t e = grad<ND, NDV, true>(a, s);
    return e == cudaSuccess ? grad<ND, NDV, false>(a, s) : e;
}

// ---------------------------------------------------------------------------
// Absorbed form over pages.  One CTA per (split of a sequence, 16 query rows);
// the splits' outputs and log-sum-exps are joined by a second kernel.
// ---------------------------------------------------------------------------
constexpr int kDecTok = 32;

// ROWS = 16 or 32 query rows a CTA, 16 threads each: 32 halve the reads of the
// cache where there are that many.  The next tile's rows are copied (cp.async)
// while this one is worked on.
template <int NL, int ROWS>      // Dl = 128 NL
__global__ void __launch_bounds__(16 * ROWS) latent_decode_f32_kernel(LatentDecodeArgs a, int splits) {
    extern __shared__ __align__(16) float smem[];
    using T = float;
    constexpr int kThreads = 16 * ROWS;
    __shared__ const T *row_s[2][kDecTok];
    constexpr int Dl = 128 * NL, LP = kDecTok + 4;
    const int D = Dl + a.Ds, ld = D + 4;
    float *Qs = smem, *Cs0 = Qs + ROWS * ld, *Ps = Cs0 + 2 * kDecTok * ld, *stat = Ps + ROWS * LP;
    // stat: rescaling factors of the tile [ROWS]
    const int b = blockIdx.x / splits, sp = blockIdx.x % splits, R = a.T * a.H, row0 = blockIdx.y * ROWS;
    const int rows = min(ROWS, R - row0), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long most = (long)a.table_width * a.page_size;
    const int given = a.lens[b];
    const int len = (int)min((long)max(given, 0), most);
    if ((given < 0 || given > most) && tid == 0) atomicCAS(a.err, 0, (int32_t)RDA_ERR_INVALID_ARG);
    const int tiles = (len + kDecTok - 1) / kDecTok;
    const int t_lo = (int)((long)tiles * sp / splits), t_hi = (int)((long)tiles * (sp + 1) / splits);
    for (int r = warp; r < ROWS; r += kThreads / 32)
        for (int c = 4 * lane; c < D; c += 128) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const size_t row = (size_t)b * R + row0 + r;
                x = c < Dl ? Io<T>::ld4((const T *)a.q + row * Dl + c) : Io<T>::ld4((const T *)a.q_shared + row * a.Ds + c - Dl);
            }
            *reinterpret_cast<float4 *>(Qs + r * ld + c) = x;
        }
    // scores: thread = 4 rows x 4 tokens over one of SL slices of the columns
    constexpr int SL = kThreads / (ROWS / 4 * (kDecTok / 4));
    const int slice = lane % SL, blk = warp * (32 / SL) + lane / SL, br = blk % (ROWS / 4) * 4, bt = blk / (ROWS / 4) * 4;
    // softmax: PR threads a row, U tokens each
    constexpr int PR = kThreads / ROWS, U = kDecTok / PR;
    float m = -INFINITY, l = 0.f;
    const int srow = tid / PR, sc = tid % PR;
    // outputs: thread = rows RO (tid / 128) .., columns tid % 128 + 128 c
    constexpr int RO = 8;
    const int og = tid >> 7, oc = tid & 127;
    float o[RO][NL] = {};
    // where each token of tile t lies (null: not cached, or on a page outside the cache)
    auto find = [&](int t) {
        if (tid < kDecTok) {
            const int j = t * kDecTok + tid;
            const T *p = nullptr;
            if (t < t_hi && j < len) {
                const int page = a.table[(size_t)b * a.table_width + j / a.page_size];
                if (page >= 0 && page < a.num_pages)
                    p = (const T *)a.pages + ((size_t)page * a.page_size + j % a.page_size) * D;
                else
                    atomicCAS(a.err, 0, (int32_t)RDA_ERR_INVALID_ARG);
            }
            row_s[t & 1][tid] = p;
        }
    };
    auto fetch = [&](int t) {
        float *Cs = Cs0 + (t & 1) * kDecTok * ld;
        for (int r = warp; r < kDecTok; r += kThreads / 32) {
            const T *p = row_s[t & 1][r];
            for (int c = 4 * lane; c < D; c += 128) {
                if (p) cp_async16((uint32_t)__cvta_generic_to_shared(Cs + r * ld + c), p + c);
                else *reinterpret_cast<float4 *>(Cs + r * ld + c) = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        cp_async_commit();
    };
    find(t_lo);
    __syncthreads();
    if (t_lo < t_hi) fetch(t_lo);
    for (int t = t_lo; t < t_hi; ++t) {
        const int j0 = t * kDecTok;
        const float *Cs = Cs0 + (t & 1) * kDecTok * ld;
        find(t + 1);
        cp_async_wait_all();
        __syncthreads();
        if (t + 1 < t_hi) fetch(t + 1);
        {
            float s[4][4] = {};
            for (int c = 4 * slice; c < D; c += 4 * SL) {
                float4 x[4], y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = *reinterpret_cast<const float4 *>(Qs + (br + i) * ld + c);
                    y[i] = *reinterpret_cast<const float4 *>(Cs + (bt + i) * ld + c);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, s[i][j]))));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
#pragma unroll
                    for (int off = SL / 2; off; off >>= 1) s[i][j] += __shfl_xor_sync(0xffffffffu, s[i][j], off);
                    if (slice == 0) Ps[(br + i) * LP + bt + j] = s[i][j];
                }
        }
        __syncthreads();
        {
            const int last = len - a.T + (row0 + srow) / a.H;     // the last token this row sees
            float x[U], top = m;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = sc + PR * u, j = j0 + i;
                x[u] = j <= last && srow < rows && row_s[t & 1][i] ? Ps[srow * LP + i] * a.scale : -INFINITY;
                top = fmaxf(top, x[u]);
            }
#pragma unroll
            for (int off = PR / 2; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float base = top == -INFINITY ? 0.f : top;
            const float keep = expf(m - base);
            m = top;
            l *= keep;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float p = expf(x[u] - base);
                l += p;
                Ps[srow * LP + sc + PR * u] = p;
            }
            if (sc == 0) stat[srow] = keep;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RO; ++i) {
            const float keep = stat[RO * og + i];
#pragma unroll
            for (int c = 0; c < NL; ++c) o[i][c] *= keep;
        }
#pragma unroll 1
        for (int j = 0; j < kDecTok; j += 4) {
            float y[4][NL];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int c = 0; c < NL; ++c) y[u][c] = Cs[(j + u) * ld + oc + 128 * c];
#pragma unroll
            for (int i = 0; i < RO; ++i) {
                const float4 p = *reinterpret_cast<const float4 *>(Ps + (RO * og + i) * LP + j);
#pragma unroll
                for (int c = 0; c < NL; ++c)
                    o[i][c] = fmaf(p.x, y[0][c], fmaf(p.y, y[1][c], fmaf(p.z, y[2][c], fmaf(p.w, y[3][c], o[i][c]))));
            }
        }
    }
#pragma unroll
    for (int off = PR / 2; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    __syncthreads();
    if (sc == 0) {
        stat[srow] = l > 0.f ? 1.f / l : 0.f;
        const float lse = l > 0.f ? m + logf(l) : -INFINITY;
        if (srow < rows) {
            const size_t row = (size_t)b * R + row0 + srow;
            if (splits > 1) a.part[row * splits + sp] = lse;
            else if (a.lse) a.lse[row] = lse;
        }
    }
    __syncthreads();
    float *po = a.part + (((size_t)a.B * R * splits + 3) & ~(size_t)3);
#pragma unroll
    for (int i = 0; i < RO; ++i) {
        if (RO * og + i >= rows) continue;
        const size_t row = (size_t)b * R + row0 + RO * og + i;
        const float f = stat[RO * og + i];
#pragma unroll
        for (int c = 0; c < NL; ++c) {
            if (splits > 1) po[(row * splits + sp) * Dl + oc + 128 * c] = o[i][c] * f;
            else static_cast<float *>(a.out)[row * Dl + oc + 128 * c] = o[i][c] * f;
        }
    }
}

// out = sum_s e^{lse_s - lse} o_s, lse = log sum_s e^{lse_s}: one CTA per row.
// Rows of tokens outside the sequences of `cu` (where given) are left as they were.
__global__ void __launch_bounds__(128) latent_join_kernel(LatentDecodeArgs a, int splits, const int32_t *cu, int num_seqs) {
    const size_t row = blockIdx.x;
    if (cu && ((long)(row / a.H) < (long)cu[0] || (long)(row / a.H) >= (long)cu[num_seqs])) return;
    const float *ls = a.part + row * splits;
    const float *po = a.part + (((size_t)a.B * a.T * a.H * splits + 3) & ~(size_t)3) + row * splits * a.Dl;
    float top = -INFINITY, sum = 0.f;
    for (int s = 0; s < splits; ++s) top = fmaxf(top, ls[s]);
    const float base = top == -INFINITY ? 0.f : top;
    for (int s = 0; s < splits; ++s) sum += expf(ls[s] - base);
    const float f = sum > 0.f ? 1.f / sum : 0.f;
    for (int c = threadIdx.x * 4; c < a.Dl; c += 512) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < splits; ++s) {
            const float w = expf(ls[s] - base) * f;
            const float4 y = *reinterpret_cast<const float4 *>(po + (size_t)s * a.Dl + c);
            x.x = fmaf(w, y.x, x.x), x.y = fmaf(w, y.y, x.y), x.z = fmaf(w, y.z, x.z), x.w = fmaf(w, y.w, x.w);
        }
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * a.Dl + c) = x;
    }
    if (threadIdx.x == 0 && a.lse) a.lse[row] = sum > 0.f ? base + logf(sum) : -INFINITY;
}

int decode_rows(int rows) { return rows > 16 ? 32 : 16; }
// Enough splits that two CTAs per SM have work, at most 64.
int decode_splits(int B, int rows) {
    const int tile = decode_rows(rows);
    const long units = (long)B * ((rows + tile - 1) / tile);
    const long want = (2 * kSms + units - 1) / units;
    return (int)(want < 1 ? 1 : want > 64 ? 64 : want);
}

template <int NL, int ROWS> cudaError_t decode_rows_nl(const LatentDecodeArgs &a, cudaStream_t s) {
    constexpr size_t extra = ROWS * (kDecTok + 4) + ROWS;
    constexpr size_t most = sizeof(float) * ((ROWS + 2 * kDecTok) * (128 * NL + 64 + 4) + extra);
    cudaError_t e = allow_smem<latent_decode_f32_kernel<NL, ROWS>>(most);
    if (e != cudaSuccess) return e;
    const int R = a.T * a.H, splits = decode_splits(a.B, R);
    const size_t bytes = sizeof(float) * ((ROWS + 2 * kDecTok) * (128 * NL + a.Ds + 4) + extra);
    latent_decode_f32_kernel<NL, ROWS><<<dim3(splits * a.B, (R + ROWS - 1) / ROWS), 16 * ROWS, bytes, s>>>(a, splits);
    if ((e = cudaGetLastError()) != cudaSuccess || splits == 1) return e;
    latent_join_kernel<<<a.B * R, 128, 0, s>>>(a, splits, nullptr, 0);
    return cudaGetLastError();
}
template <int NL> cudaError_t decode_nl(const LatentDecodeArgs &a, cudaStream_t s) {
    return decode_rows(a.T * a.H) == 32 ? decode_rows_nl<NL, 32>(a, s) : decode_rows_nl<NL, 16>(a, s);
}

}  // namespace

cudaError_t launch_latent_forward_f32(const LatentArgs &a, cudaStream_t s) {
    return a.Dv == 64 ? forward_nv<float, 1>(a, s) : forward_nv<float, 2>(a, s);
}

cudaError_t launch_latent_delta(const LatentArgs &a, cudaStream_t s) {
    const long rows = (long)a.total_q * a.H;
    const unsigned grid = (unsigned)((rows + 7) / 8);
    if (!grid) return cudaSuccess;
    latent_delta_kernel<float><<<grid, 256, 0, s>>>((const float *)a.out, (const float *)a.d_out, a.delta, rows, a.Dv);
    return cudaGetLastError();
}

cudaError_t launch_latent_shared_sum(const LatentArgs &a, cudaStream_t s) {
    const long n = (long)a.total_k * a.Ds / 4;
    const unsigned grid = (unsigned)((n + 255) / 256);
    if (!grid) return cudaSuccess;
    if (a.dtype == RDA_F32)
        latent_shared_sum_kernel<float><<<grid, 256, 0, s>>>(a.dks_heads, (float *)a.dk_shared, a.cu_k, a.num_seqs,
                                                             a.total_k, a.H, a.Ds);
    else
        return launch_after(latent_shared_sum_kernel<__nv_bfloat16>, grid, 256, 0, s, (const float *)a.dks_heads,
                            (__nv_bfloat16 *)a.dk_shared, a.cu_k, a.num_seqs, (long)a.total_k, a.H, a.Ds);
    return cudaGetLastError();
}

cudaError_t launch_latent_backward_f32(const LatentArgs &a, cudaStream_t s) {
    const int nd = (a.Dk + a.Ds) / 64;
    if (a.Dv == 64) return nd == 1 ? backward_nd<1, 1>(a, s) : nd == 2 ? backward_nd<2, 1>(a, s) : backward_nd<3, 1>(a, s);
    return nd == 1 ? backward_nd<1, 2>(a, s) : nd == 2 ? backward_nd<2, 2>(a, s) : backward_nd<3, 2>(a, s);
}

cudaError_t launch_latent_decode_f32(const LatentDecodeArgs &a, cudaStream_t s) {
    switch (a.Dl / 128) {
        case 1: return decode_nl<1>(a, s);
        case 2: return decode_nl<2>(a, s);
        case 3: return decode_nl<3>(a, s);
        default: return decode_nl<4>(a, s);
    }
}

size_t latent_backward_scratch_bytes(int total_q, int total_k, int H, int Ds) {
    const size_t d = ((size_t)total_q * H * sizeof(float) + 255) / 256 * 256;
    return d + (size_t)total_k * H * Ds * sizeof(float);
}

size_t latent_forward_f32_scratch_bytes(int total_q, int total_k, int H, int Dv) {
    const int splits = forward_splits(total_q, total_k, H);
    return splits == 1 ? 0 : ((size_t)total_q * H * splits * (Dv + 1) + 4) * sizeof(float);
}

size_t latent_decode_scratch_bytes(int B, int T, int H, int Dl) {
    const int splits = decode_splits(B, T * H);
    return splits == 1 ? 0 : ((size_t)B * T * H * splits * (Dl + 1) + 4) * sizeof(float);
}

}  // namespace rda
