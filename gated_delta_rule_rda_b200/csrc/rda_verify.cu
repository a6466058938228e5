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
// Sums: a warp per 1024-token slice, all its loads in flight at once, one fp64 sum a
// slice.  Draw: one CTA a sequence scans the slices' sums, re-reads the one slice
// that u falls into (from L2) and scans it.  One kernel, a cluster per sequence, or
// two (see the launch).
// Sums run in a fixed order: results do not depend on timing.
//
// Measured: 64 sequences, V = 259,840: sums 22.7 us (5.9 TB/s, 89% of a copy's rate),
// both kernels 26 us; one sequence, V = 32,000: 5.2 us, 12.7 with the host's part.
#include <cuda_runtime.h>

#include "rda_latent.h"
#include "sm100_ptx.cuh"

namespace rda {
namespace {

constexpr int kSlice = 1024;      // tokens a warp sums at once: 8 float4 of each row per lane
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kMostCtas = 8;      // of a sequence (the portable size of a cluster)

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

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
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) before = sum;
        sum += warp_s[w];
    }
    *total = sum;
    return before + x;
}

// The token of sequence b after its k kept drafts of n, from the slices' sums: by one CTA, which saw them written.
__device__ __forceinline__ void draw(const VerifyArgs &a, int b, int k, int n, double *part) {
    __shared__ double warp_s[kWarps], start_s;
    __shared__ int slice_s, last_s, token_s, tail_s;
    const int tid = threadIdx.x, ns = slices_of(a.V);
    if (tid == 0) slice_s = token_s = 0x7fffffff, last_s = tail_s = -1, start_s = 0.0;
    const double u = a.uniforms[(size_t)b * (a.T + 1) + a.T];
    Rows r = weight_rows(a, b, k, n);
    // each thread's slices are consecutive: one scan gives every slice's start
    const int per = (ns + kThreads - 1) / kThreads, s0 = min(ns, tid * per), s1 = min(ns, s0 + per);
    double mine, end, total;
    for (int pass = 0;; ++pass) {
        mine = 0.0;
        for (int s = s0; s < s1; ++s) mine += part[s];
        end = block_scan(mine, warp_s, &total);
        if (total > 0.0 || pass || (!r.q && r.x < 0)) break;
        // a residual of nothing (the target nowhere above the draft): the target itself
        r.q = nullptr;
        r.x = -1;
        for (int s = tid >> 5; s < ns; s += kThreads / 32) {
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
    const double upto4 = block_scan(four, warp_s, &sum);
    double at = upto4 - four + start_s;      // read behind the scan, whose barriers publish it
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

// The slices' sums of one sequence by `warps` warps, of which this is number w.
template <bool VEC> __device__ __forceinline__ void sums(const VerifyArgs &a, const Rows &r, int w, int warps, double *part) {
    const int ns = slices_of(a.V), lane = threadIdx.x & 31;
    for (int s = w; s < ns; s += warps) {
        const double sum = slice_sum<VEC>(r, s, a.V, lane);
        if (lane == 0) part[s] = sum;
    }
}

// A sequence by a cluster.
template <bool VEC> __global__ void __launch_bounds__(kThreads) verify_kernel(VerifyArgs a) {
    const int b = blockIdx.y, rank = blockIdx.x;
    double *part = a.part + (size_t)b * slices_of(a.V);
    ptx::pdl_launch_dependents();
    ptx::pdl_wait_primary();
    int n;
    const int k = kept_drafts(a, b, threadIdx.x & 31, &n);
    sums<VEC>(a, weight_rows(a, b, k, n), rank * kWarps + (threadIdx.x >> 5), gridDim.x * kWarps, part);
    // the sequence's sums are written, and seen by its first CTA
    if (gridDim.x > 1) cluster_barrier();
    else __syncthreads();
    if (rank > 0) return;
    if (threadIdx.x == 0) a.num_accepted[b] = k;
    draw(a, b, k, n, part);
}

// The same in two kernels, sums and draw.
template <bool VEC> __global__ void __launch_bounds__(kThreads) verify_sums_kernel(VerifyArgs a) {
    const int b = blockIdx.y;
    ptx::pdl_launch_dependents();
    ptx::pdl_wait_primary();
    int n;
    const int k = kept_drafts(a, b, threadIdx.x & 31, &n);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.num_accepted[b] = k;
    sums<VEC>(a, weight_rows(a, b, k, n), blockIdx.x * kWarps + (threadIdx.x >> 5), gridDim.x * kWarps,
              a.part + (size_t)b * slices_of(a.V));
}
__global__ void __launch_bounds__(kThreads) verify_draw_kernel(VerifyArgs a) {
    const int b = blockIdx.x;
    ptx::pdl_launch_dependents();
    ptx::pdl_wait_primary();
    const int n = a.num_drafts ? min(max(a.num_drafts[b], 0), a.T) : a.T;
    draw(a, b, a.num_accepted[b], n, a.part + (size_t)b * slices_of(a.V));
}

}  // namespace

size_t verify_scratch_bytes(int B, int V) { return (size_t)B * slices_of(V) * sizeof(double); }

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t s) {
    const int ns = slices_of(a.V);
    const bool vec = a.V % 4 == 0 && (uintptr_t)a.target_probs % 16 == 0 && (uintptr_t)a.draft_probs % 16 == 0;
    // One launch while the warps of a cluster have two slices each at most.  Called one by one (host included) and on
    // the device, us: 1 sequence of V = 32,000 12.7 and 5.2, against 14.7 and 6.0 by two kernels; 8 of 100,003 12.7 and
    // 8.2 against 14.7 and 7.5; 250 of 4096 12.7 and 5.9 against 14.7 and 8.6.  Beyond, more SMs count: 1 of 259,840
    // would take 9.3 on the device against 6.2 by two kernels, 64 of them 27.8 against 25.5.
    if (ns <= 2 * kMostCtas * kWarps) {
        // CTAs of a sequence: until every warp has one slice at most, or every SM two CTAs
        int ctas = 1;
        while (ctas < kMostCtas && ctas * kWarps < ns && (long)a.B * ctas < 2 * kSms) ctas *= 2;
        return launch_clusters_after(vec ? verify_kernel<true> : verify_kernel<false>, ctas, dim3(ctas, a.B), kThreads, 0, s, a);
    }
    // At most 8 CTAs an SM, every warp with as many slices as the others.  80 registers let 3 of them run at once (4
    // without 128-bit loads), in two to three waves; a grid of 3 or 4 an SM is no faster on the whole, us on the device: 64 sequences
    // of 259,840 23.5 either way, of 200,003 23.2 against 21.8, 16 of 259,840 9.2 against 10.7, 250 of 140,000 40
    // against 51.
    const int need = (ns + kWarps - 1) / kWarps, wave = (kSms * 8 + a.B - 1) / a.B;
    const int rounds = (need + wave - 1) / wave;
    const dim3 grid((need + rounds - 1) / rounds, a.B);
    const cudaError_t e = launch_after(vec ? verify_sums_kernel<true> : verify_sums_kernel<false>, grid, kThreads, 0, s, a);
    return e == cudaSuccess ? launch_after(verify_draw_kernel, a.B, kThreads, 0, s, a) : e;
}

}  // namespace rda
