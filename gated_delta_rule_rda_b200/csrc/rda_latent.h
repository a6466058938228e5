// Launch interface of the latent-attention kernels and of draft verification.
// Not installed; the public interface is include/rda.h.
#pragma once

#include <atomic>
#include <utility>

#include "rda_internal.h"

namespace rda {

constexpr int kSms = 148;      // streaming multiprocessors of a B200

// Lets kernel K have `bytes` of dynamic shared memory, once per device (the
// attribute belongs to the device's copy of the kernel).
template <auto K> cudaError_t allow_smem(size_t bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// Arguments of the expanded form (packed sequences) and of its gradients.
struct LatentArgs {
    const void *q, *q_shared, *k, *k_shared, *v;   // q_shared, k_shared: null exactly when Ds = 0
    const int32_t *cu_q, *cu_k;
    int num_seqs, total_q, total_k;
    int H, Dk, Ds, Dv;
    float scale;
    int causal;
    rda_dtype_t dtype;
    void *out;                   // forward: written; backward: read
    float *lse;                  // forward: written (or null); backward: read
    int32_t *err;                // device error word
    uint64_t wait_ns;            // bound of every device-side wait
    int debug_drop;              // fault injection (tests only): tiles from this one on are never filled; -1 = off
    const int2 *order;           // tiles by work (TileOrder), or null: by their places
    // backward only
    const void *d_out;
    void *dq, *dq_shared, *dk, *dk_shared, *dv;
    float *delta;                // workspace: sum_d d_out out, [total_q, H] (fp32 forward: parts of split rows)
    float *dks_heads;            // workspace: the shared key part's gradient per head, [total_k, H, Ds]
};

// Arguments of the absorbed form over a paged cache.
struct LatentDecodeArgs {
    const void *q, *q_shared, *pages;
    const int32_t *table, *lens;
    int num_pages, page_size, table_width;
    int B, T, H, Dl, Ds;
    float scale;
    rda_dtype_t dtype;
    void *out;
    float *lse;
    int32_t *err;
    uint64_t wait_ns;
    int debug_drop;              // as above
    float *part;                 // workspace: partial outputs and their log-sum-exps
};

struct VerifyArgs {
    const int32_t *draft;        // [B, T]
    const float *draft_probs;    // [B, T, V] or null
    const float *target_probs;   // [B, T + 1, V]
    const float *uniforms;       // [B, T + 1]
    const int32_t *num_drafts;   // [B] or null
    int32_t *tokens, *num_accepted;
    int B, T, V;
    double *part;                // workspace: sums of the weights per slice
};

// Most drafted tokens one verification takes per sequence (one warp lane each).
constexpr int kMaxDrafts = 32;

// Tokens of sequence n in a packed batch, with whatever the device array holds
// kept inside [0, total].
struct SeqSpan {
    int start, len;
};
__device__ __forceinline__ int clamped(const int32_t *cu, int n, int total) { return min(max(cu[n], 0), total); }
__device__ __forceinline__ SeqSpan seq_span(const int32_t *cu, int n, int total) {
    const int s = clamped(cu, n, total);
    return SeqSpan{s, max(clamped(cu, n + 1, total) - s, 0)};
}
// Tiles of `tile` rows over packed sequences without a prefix sum: sequence n
// owns the slots from floor(cu[n] / tile) + n on, which are as many as its
// rows need or one more, since ceil(len / tile) <= floor((c + len) / tile) -
// floor(c / tile) + 1.  Returns the sequence that owns `slot` and the tile in it.
__device__ __forceinline__ int find_tile(const int32_t *cu, int num_seqs, int total, int tile, int slot, int *t) {
    int lo = 0, hi = num_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (clamped(cu, mid, total) / tile + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    *t = slot - (clamped(cu, lo, total) / tile + lo);
    if (*t < 0) *t = 0x3fffffff / tile;           // before the first sequence: behind every end
    return lo;
}
__host__ __device__ inline int tile_slots(int total, int num_seqs, int tile) { return total / tile + num_seqs; }

// The tiles of a packed batch in the order of their work, most first, so that
// the last CTAs are short.  Tiles are of query rows (work: units of keys that they
// see) or of keys (units of query rows that see them).
struct TileOrder {
    int keys, tile, unit;
    int2 *out;                   // [slots]: {sequence, tile}, then {-1, -1}
};
size_t order_bytes(int total, int num_seqs, int tile);
// One CTA makes the order, whatever the number of heads that use it.  With two heads or more it is worth that for any
// batch (two heads, 2000 sequences of 1 to 300: gradients 1226 -> 1195 us; 100,000 of 0 to 4: 22.3 -> 21.8 ms).  With one
// head it is for 500 sequences (gradients 170.3 -> 168.8 us) and no longer for 1000 (324.7 -> 332.0).
inline bool worth_order(const LatentArgs &a) { return a.num_seqs > 1 && (a.H > 1 || a.num_seqs <= 512); }

// A launch that may overlap the end of the kernel before it on the stream,
// whosever that is.  Every CTA of a kernel launched so waits (griddepcontrol.wait)
// before it reads or writes global memory and before its first exit, so that
// whatever comes next finds both done; it lets its own dependents go at once.
// Measured in calls one after the other: 22.6 -> 19.2 us for one sequence of
// 4096 tokens decoded, 71.5 -> 64.6 us for the gradients of a packed batch.
// `cluster` CTAs along x form a cluster.
template <typename... P, typename... A>
cudaError_t launch_clusters_after(void (*kernel)(P...), int cluster, dim3 grid, int threads, size_t smem, cudaStream_t s, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A &&...args) {
    return launch_clusters_after(kernel, 1, grid, threads, smem, s, std::forward<A>(args)...);
}

cudaError_t launch_latent_forward_f32(const LatentArgs &a, cudaStream_t s);
cudaError_t launch_latent_backward_f32(const LatentArgs &a, cudaStream_t s);
// shared steps of the gradients: delta before, the sum over heads after
cudaError_t launch_latent_delta(const LatentArgs &a, cudaStream_t s);
cudaError_t launch_latent_shared_sum(const LatentArgs &a, cudaStream_t s);
cudaError_t launch_latent_decode_f32(const LatentDecodeArgs &a, cudaStream_t s);
// bf16: tensor cores
cudaError_t launch_latent_backward_tc(const LatentArgs &a, void *scratch, cudaStream_t s);
size_t latent_backward_tc_scratch_bytes(int total_q, int total_k, int num_seqs, int H, int Ds);
cudaError_t launch_latent_forward_tc(const LatentArgs &a, void *scratch, cudaStream_t s);
size_t latent_prefill_scratch_bytes(int total_q, int num_seqs);
cudaError_t launch_latent_decode_tc(const LatentDecodeArgs &a, cudaStream_t s);
cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t s);

size_t latent_backward_scratch_bytes(int total_q, int total_k, int H, int Ds);
size_t latent_forward_f32_scratch_bytes(int total_q, int total_k, int H, int Dv);
size_t latent_decode_scratch_bytes(int B, int T, int H, int Dl);
size_t latent_decode_tc_scratch_bytes(int T, int H, int Dl, int Ds);
size_t verify_scratch_bytes(int B, int V);

}  // namespace rda
