// Verification of drafted tokens against the target's probabilities, from
// given random numbers (speculative sampling).
//
// For one sequence with drafts x_0 .. x_{n-1}: draft t is kept iff all before
// it were and u_t q_t(x_t) < p_t(x_t).  With k kept, the next token is drawn by
// inverse CDF with the last uniform from
//   w_i = max(p_k(i) - q_k(i), 0)   (k < n: the residual at the first refusal)
//   w_i = p_n(i)                    (k = n)
// as the first i with w_0 + .. + w_i > u (w_0 + .. + w_{V-1}).
//
// Bound by memory: two rows of V floats a sequence (one when every draft is
// kept).  Sums and the comparison with u are in fp64: float products and
// differences are exact there, and a choice then hangs on the order of the sum
// only where u lies within ~1e-14 of a border.
//
// Two kernels.  sums: a warp per 1024-token slice, all its loads in flight at
// once, one fp64 sum a slice.  pick: a CTA per sequence scans the slices' sums,
// re-reads the one slice that u falls into (from L2) and scans it.
// Sums run in a fixed order: results do not depend on timing.
//
// Measured: 64 sequences, V = 259,840: sums 22.7 us (5.9 TB/s, 89% of a copy's rate),
// both kernels 27.2 us; one sequence, V = 32,000: 15 us, of which the host's two
// launches are most (2.8 and 3.7 us on the device).
#include <cuda_runtime.h>

#include "rda_latent.h"
#include "sm100_ptx.cuh"

namespace rda {
namespace {

constexpr int kSlice = 1024;      // tokens a warp sums at once: 8 float4 of each row per lane
constexpr int kWarps = 8;
constexpr int kPick = 256;

__host__ __device__ constexpr int slices_of(int V) { return (V + kSlice - 1) / kSlice; }

// Kept drafts of sequence b (the same in every lane), and how many there are.
__device__ __forceinline__ int kept_drafts(const VerifyArgs &a, int b, int lane, int *n_out) {
    const int n = a.num_drafts ? min(max(a.num_drafts[b], 0), a.T) : a.T;
    *n_out = n;
    bool keep = false;
    if (lane < n) {
        const int x = a.draft[(size_t)b * a.T + lane];
        if (x >= 0 && x < a.V) {       // a token outside the vocabulary is refused
            const double p = a.target_probs[((size_t)b * (a.T + 1) + lane) * a.V + x];
            const double q = a.draft_probs ? a.draft_probs[((size_t)b * a.T + lane) * a.V + x] : 1.0;
            keep = (double)a.uniforms[(size_t)b * (a.T + 1) + lane] * q < p;
        }
    }
    const unsigned refused = ~__ballot_sync(0xffffffffu, keep);     // lanes from n on refuse
    return refused ? __ffs(refused) - 1 : 32;
}

// The weights' rows of a sequence.
struct Rows {
    const float *p, *q;        // q null: no residual, or the draft is a point mass
    int x;                     // point mass at x (-1: none)
};
__device__ __forceinline__ Rows weight_rows(const VerifyArgs &a, int b, int k, int n) {
    Rows r;
    r.p = a.target_probs + ((size_t)b * (a.T + 1) + k) * a.V;
    r.q = k < n && a.draft_probs ? a.draft_probs + ((size_t)b * a.T + k) * a.V : nullptr;
    r.x = k < n && !a.draft_probs ? a.draft[(size_t)b * a.T + k] : -1;
    return r;
}
// A token's weight: max(p - q, 0), exact in fp64.  Without q the target's own; 0 at the point mass.  A comparison of
// the floats decides, so that NaN weighs nothing and only what counts is converted.
__device__ __forceinline__ double weight(float p, float q, bool at_x) {
    return p > q && !at_x ? (double)p - (double)q : 0.0;
}
// Sum of slice s by a warp (every lane gets it), all its loads in flight at once.
template <bool VEC> __device__ __forceinline__ double slice_sum(const Rows &r, int s, int V, int lane) {
    const int i0 = s * kSlice;
    double sum = 0.0;
    if (VEC) {
        float4 p[8], q[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + 128 * u + 4 * lane;
            p[u] = q[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < V) {
                p[u] = __ldg(reinterpret_cast<const float4 *>(r.p + i));
                if (r.q) q[u] = __ldg(reinterpret_cast<const float4 *>(r.q + i));
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + 128 * u + 4 * lane;
            sum += weight(p[u].x, q[u].x, i == r.x);
            sum += weight(p[u].y, q[u].y, i + 1 == r.x);
            sum += weight(p[u].z, q[u].z, i + 2 == r.x);
            sum += weight(p[u].w, q[u].w, i + 3 == r.x);
        }
    } else {
        // rows of a vocabulary that is no multiple of 4 start anywhere: single floats
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            float p[16], q[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const int i = i0 + 512 * half + 32 * u + lane;
                p[u] = i < V ? __ldg(r.p + i) : 0.f;
                q[u] = r.q && i < V ? __ldg(r.q + i) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < 16; ++u) sum += weight(p[u], q[u], i0 + 512 * half + 32 * u + lane == r.x);
        }
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    return sum;
}

template <bool VEC>
__global__ void __launch_bounds__(32 * kWarps) verify_sums_kernel(VerifyArgs a) {
    const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ptx::pdl_launch_dependents();
    ptx::pdl_wait_primary();
    int n;
    const int k = kept_drafts(a, b, lane, &n);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.num_accepted[b] = k;
    const Rows r = weight_rows(a, b, k, n);
    const int ns = slices_of(a.V);
    for (int s = blockIdx.x * kWarps + warp; s < ns; s += gridDim.x * kWarps) {
        const double sum = slice_sum<VEC>(r, s, a.V, lane);
        if (lane == 0) a.part[(size_t)b * ns + s] = sum;
    }
}

// Inclusive sums over the CTA's threads; *total gets the sum of all.
__device__ __forceinline__ double block_scan(double x, double *warp_s, double *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_s[warp] = x;
    __syncthreads();
    double before = 0.0, sum = 0.0;
#pragma unroll
    for (int w = 0; w < kPick / 32; ++w) {
        if (w == warp) before = sum;
        sum += warp_s[w];
    }
    *total = sum;
    return before + x;
}

__global__ void __launch_bounds__(kPick) verify_pick_kernel(VerifyArgs a) {
    __shared__ double warp_s[kPick / 32], start_s;
    __shared__ int slice_s, last_s, token_s, tail_s;
    const int b = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) slice_s = token_s = 0x7fffffff, last_s = tail_s = -1, start_s = 0.0;
    const int ns = slices_of(a.V);
    double *part = a.part + (size_t)b * ns;
    ptx::pdl_launch_dependents();
    ptx::pdl_wait_primary();
    const int n = a.num_drafts ? min(max(a.num_drafts[b], 0), a.T) : a.T;
    const double u = a.uniforms[(size_t)b * (a.T + 1) + a.T];
    const int k = a.num_accepted[b];
    Rows r = weight_rows(a, b, k, n);
    // each thread's slices are consecutive: one scan gives every slice's start
    const int per = (ns + kPick - 1) / kPick, s0 = min(ns, tid * per), s1 = min(ns, s0 + per);
    double mine, end, total;
    for (int pass = 0;; ++pass) {
        mine = 0.0;
        for (int s = s0; s < s1; ++s) mine += part[s];
        end = block_scan(mine, warp_s, &total);
        if (total > 0.0 || pass || (!r.q && r.x < 0)) break;
        // a residual of nothing (the target nowhere above the draft): the target itself
        r.q = nullptr;
        r.x = -1;
        for (int s = tid >> 5; s < ns; s += kPick / 32) {
            const double sum = slice_sum<false>(r, s, a.V, tid & 31);
            if ((tid & 31) == 0) part[s] = sum;
        }
        __syncthreads();
    }
    const double goal = u * total;
    double upto = end - mine;
    // the first slice whose end passes the goal
    for (int s = s0; s < s1; ++s) {
        const double w = part[s];
        upto += w;
        if (w > 0.0) {
            if (upto > goal) atomicMin(&slice_s, s);
            atomicMax(&last_s, s);
        }
    }
    __syncthreads();
    // none passes it (u next to 1, and rounding): the last one that weighs anything
    const bool past = slice_s == 0x7fffffff;
    const int slice = past ? last_s : slice_s;
    if (slice >= s0 && slice < s1) {
        double start = end - mine;
        for (int s = s0; s < slice; ++s) start += part[s];
        start_s = start;
    }
    double w[4] = {0.0, 0.0, 0.0, 0.0};
    const int i0 = slice * kSlice + 4 * tid;
    if (slice >= 0) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int i = i0 + v;
            if (i < a.V) w[v] = weight(r.p[i], r.q ? r.q[i] : 0.f, i == r.x);
        }
    }
    const double four = w[0] + w[1] + w[2] + w[3];
    double sum;
    double at = block_scan(four, warp_s, &sum) - four + start_s;      // its barriers publish start_s
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        at += w[v];
        if (w[v] > 0.0) {
            if (!past && at > goal) atomicMin(&token_s, i0 + v);
            atomicMax(&tail_s, i0 + v);
        }
    }
    __syncthreads();
    const int next = token_s != 0x7fffffff ? token_s : tail_s;
    if (tid <= a.T)
        a.tokens[(size_t)b * (a.T + 1) + tid] = tid < k ? a.draft[(size_t)b * a.T + tid] : tid == k ? next : -1;
}

}  // namespace

size_t verify_scratch_bytes(int B, int V) { return (size_t)B * slices_of(V) * sizeof(double); }

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t s) {
    // at most one wave of CTAs (8 per SM), every warp with as many slices as the others
    const int need = (slices_of(a.V) + kWarps - 1) / kWarps, wave = (148 * 8 + a.B - 1) / a.B;
    const int rounds = (need + wave - 1) / wave;
    const dim3 grid((need + rounds - 1) / rounds, a.B);
    const bool vec = a.V % 4 == 0 && (uintptr_t)a.target_probs % 16 == 0 && (uintptr_t)a.draft_probs % 16 == 0;
    const cudaError_t e = launch_after(vec ? verify_sums_kernel<true> : verify_sums_kernel<false>, grid, 32 * kWarps, 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_after(verify_pick_kernel, a.B, kPick, 0, s, a);
}

}  // namespace rda
