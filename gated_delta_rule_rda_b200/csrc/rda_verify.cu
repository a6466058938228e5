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
// (residual weight, weight of the target alone); written so that NaN weighs nothing
__device__ __forceinline__ double2 weight(float p, float q, bool at_x) {
    const double d = (double)p - (double)q;
    return make_double2(!at_x && d > 0.0 ? d : 0.0, p > 0.f ? (double)p : 0.0);
}

template <bool VEC>
__global__ void __launch_bounds__(32 * kWarps) verify_sums_kernel(VerifyArgs a) {
    const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ptx::pdl_launch_dependents();
    int n;
    int k = kept_drafts(a, b, lane, &n);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.num_accepted[b] = k;
    const Rows r = weight_rows(a, b, k, n);
    const int ns = slices_of(a.V);
    for (int s = blockIdx.x * kWarps + warp; s < ns; s += gridDim.x * kWarps) {
        const int i0 = s * kSlice;
        double rest = 0.0, all = 0.0;
        if (VEC) {
            float4 p[8], q[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int i = i0 + 128 * u + 4 * lane;
                const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                p[u] = i < a.V ? __ldg(reinterpret_cast<const float4 *>(r.p + i)) : z;
                q[u] = r.q && i < a.V ? __ldg(reinterpret_cast<const float4 *>(r.q + i)) : z;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int i = i0 + 128 * u + 4 * lane;
                const float ps[4] = {p[u].x, p[u].y, p[u].z, p[u].w}, qs[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const double2 w = weight(ps[v], qs[v], i + v == r.x);
                    rest += w.x;
                    all += w.y;
                }
            }
        } else {
            // rows of a vocabulary that is no multiple of 4 start anywhere: single floats
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float p[16], q[16];
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    const int i = i0 + 512 * half + 32 * u + lane;
                    p[u] = i < a.V ? __ldg(r.p + i) : 0.f;
                    q[u] = r.q && i < a.V ? __ldg(r.q + i) : 0.f;
                }
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    const double2 w = weight(p[u], q[u], i0 + 512 * half + 32 * u + lane == r.x);
                    rest += w.x;
                    all += w.y;
                }
            }
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) {
            rest += __shfl_xor_sync(0xffffffffu, rest, off);
            all += __shfl_xor_sync(0xffffffffu, all, off);
        }
        if (lane == 0) a.part[(size_t)b * ns + s] = make_double2(rest, all);
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
    __shared__ int slice_s, last_s, token_s;
    const int b = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) slice_s = 0x7fffffff, last_s = -1, token_s = 0x7fffffff, start_s = 0.0;
    const int n = a.num_drafts ? min(max(a.num_drafts[b], 0), a.T) : a.T;
    const double u = a.uniforms[(size_t)b * (a.T + 1) + a.T];
    const int ns = slices_of(a.V);
    const double2 *part = a.part + (size_t)b * ns;
    ptx::pdl_wait_primary();
    const int k = a.num_accepted[b];
    const Rows r = weight_rows(a, b, k, n);
    // the residual's sum, the target's
    double rest = 0.0, all = 0.0;
    for (int s = tid; s < ns; s += kPick) {
        const double2 w = part[s];
        rest += w.x;
        all += w.y;
    }
    double total_rest, total_all;
    block_scan(rest, warp_s, &total_rest);
    block_scan(all, warp_s, &total_all);
    // a residual of nothing (the target nowhere above the draft): the target itself
    const bool residual = k < n && total_rest > 0.0;
    const double goal = u * (residual ? total_rest : total_all);
    // the first slice whose end passes the goal
    double done = 0.0;
    for (int s0 = 0; s0 < ns; s0 += kPick) {
        const int s = s0 + tid;
        const double2 w2 = s < ns ? part[s] : make_double2(0.0, 0.0);
        const double w = residual ? w2.x : w2.y;
        double sum;
        const double upto = done + block_scan(w, warp_s, &sum);
        if (w > 0.0) {
            if (upto > goal) atomicMin(&slice_s, s);
            atomicMax(&last_s, s);
        }
        __syncthreads();
        if (s == slice_s) start_s = upto - w;
        done += sum;
        __syncthreads();
        if (slice_s != 0x7fffffff) break;
    }
    // none passes it (u next to 1, and rounding): the last one that weighs anything
    const bool past = slice_s == 0x7fffffff;
    const int slice = past ? last_s : slice_s;
    const double start = start_s;
    __syncthreads();
    if (tid == 0) last_s = -1;
    double w[4] = {0.0, 0.0, 0.0, 0.0};
    const int i0 = slice * kSlice + 4 * tid;
    if (slice >= 0) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int i = i0 + v;
            if (i < a.V) {
                const double2 x = weight(r.p[i], r.q ? r.q[i] : 0.f, i == r.x);
                w[v] = residual ? x.x : x.y;
            }
        }
    }
    double sum;
    double upto = start + block_scan(w[0] + w[1] + w[2] + w[3], warp_s, &sum) - (w[0] + w[1] + w[2] + w[3]);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        upto += w[v];
        if (w[v] > 0.0) {
            if (!past && upto > goal) atomicMin(&token_s, i0 + v);
            atomicMax(&last_s, i0 + v);
        }
    }
    __syncthreads();
    const int next = token_s != 0x7fffffff ? token_s : last_s;
    if (tid <= a.T)
        a.tokens[(size_t)b * (a.T + 1) + tid] = tid < k ? a.draft[(size_t)b * a.T + tid] : tid == k ? next : -1;
}

}  // namespace

size_t verify_scratch_bytes(int B, int V) { return (size_t)B * slices_of(V) * sizeof(double2); }

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t s) {
    // CTAs for one wave (8 per SM); each warp takes slice after slice
    const int need = (slices_of(a.V) + kWarps - 1) / kWarps, wave = (148 * 8 + a.B - 1) / a.B;
    const dim3 grid(need < wave ? need : wave, a.B);
    const bool vec = a.V % 4 == 0 && (uintptr_t)a.target_probs % 16 == 0 && (uintptr_t)a.draft_probs % 16 == 0;
    if (vec) verify_sums_kernel<true><<<grid, 32 * kWarps, 0, s>>>(a);
    else verify_sums_kernel<false><<<grid, 32 * kWarps, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.B);
    cfg.blockDim = dim3(kPick);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_pick_kernel, a);
}

}  // namespace rda
