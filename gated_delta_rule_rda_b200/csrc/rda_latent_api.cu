// C-ABI entry points of latent attention and draft verification
// (include/rda.h): argument validation on the host, then dispatch on the
// caller's stream.  Nothing here allocates device memory.
#include <algorithm>

#include "rda_latent.h"

using namespace rda;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kMaxHeads = 1024;
constexpr int kMaxBatch = 65535;      // grid dimension

bool head_dims_ok(int Dk, int Ds, int Dv) {
    return (Dk == 64 || Dk == 128) && (Ds == 0 || Ds == 64) && (Dv == 64 || Dv == 128);
}

// Checks shared by the expanded form and its gradients.
rda_status_t check_packed(const void *q, const void *q_shared, const void *k, const void *k_shared, const void *v,
                          const int32_t *cu_q, const int32_t *cu_k, int num_seqs, int total_q, int total_k,
                          rda_dtype_t dtype, int H, int Dk, int Ds, int Dv) {
    if (dtype != RDA_F32 && dtype != RDA_BF16) return RDA_ERR_UNSUPPORTED;
    if (num_seqs < 0 || total_q < 0 || total_k < 0 || H <= 0) return RDA_ERR_INVALID_ARG;
    if (!head_dims_ok(Dk, Ds, Dv) || H > kMaxHeads) return RDA_ERR_UNSUPPORTED;
    if ((long long)std::max(total_q, total_k) * H * (Dk + Ds) >= (1LL << 31)) return RDA_ERR_INVALID_ARG;
    if (((long long)std::max(total_q, total_k) + num_seqs) * H >= (1LL << 31)) return RDA_ERR_INVALID_ARG;      // CTAs
    if ((q_shared == nullptr && total_q > 0) != (Ds == 0 && total_q > 0)) return RDA_ERR_INVALID_ARG;
    if ((k_shared == nullptr && total_k > 0) != (Ds == 0 && total_k > 0)) return RDA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!cu_q || !cu_k)) return RDA_ERR_INVALID_ARG;
    if (total_q > 0 && !q) return RDA_ERR_INVALID_ARG;
    if (total_k > 0 && (!k || !v)) return RDA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(q_shared, 16) || !aligned(k, 16) || !aligned(k_shared, 16) || !aligned(v, 16) ||
        !aligned(cu_q, 4) || !aligned(cu_k, 4))
        return RDA_ERR_MISALIGNED;
    return RDA_OK;
}

rda_status_t check_workspace(const void *workspace, size_t given, size_t need) {
    if (!workspace || given < need) return RDA_ERR_WORKSPACE;
    return aligned(workspace, 256) ? RDA_OK : RDA_ERR_MISALIGNED;
}

rda_status_t done(cudaError_t e) { return e == cudaSuccess ? RDA_OK : RDA_ERR_CUDA; }

}  // namespace

extern "C" {

size_t rda_latent_prefill_workspace_bytes(int total_q, int total_k, int H, int Dk, int Ds, int Dv, int num_seqs) {
    if (total_q < 0 || total_k < 0 || H <= 0 || H > kMaxHeads || num_seqs < 0 || !head_dims_ok(Dk, Ds, Dv)) return 0;
    return kErrorWordBytes + std::max(latent_prefill_scratch_bytes(total_q, num_seqs),
                                      latent_forward_f32_scratch_bytes(total_q, total_k, H, Dv));
}

rda_status_t rda_latent_prefill(const void *q, const void *q_shared, const void *k, const void *k_shared, const void *v,
                                const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                int num_seqs, int total_q, int total_k, void *out, float *lse,
                                rda_dtype_t dtype, int H, int Dk, int Ds, int Dv, float scale, int causal,
                                void *workspace, size_t workspace_bytes, void *stream) {
    rda_status_t st = check_packed(q, q_shared, k, k_shared, v, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                                   dtype, H, Dk, Ds, Dv);
    if (st != RDA_OK) return st;
    if (total_q > 0 && !out) return RDA_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(lse, 4)) return RDA_ERR_MISALIGNED;
    st = check_workspace(workspace, workspace_bytes,
                         rda_latent_prefill_workspace_bytes(total_q, total_k, H, Dk, Ds, Dv, num_seqs));
    if (st != RDA_OK) return st;
    if (num_seqs == 0 || total_q == 0) return RDA_OK;
    LatentArgs a{};
    a.q = q; a.q_shared = q_shared; a.k = k; a.k_shared = k_shared; a.v = v;
    a.cu_q = cu_seqlens_q; a.cu_k = cu_seqlens_k;
    a.num_seqs = num_seqs; a.total_q = total_q; a.total_k = total_k;
    a.H = H; a.Dk = Dk; a.Ds = Ds; a.Dv = Dv; a.scale = scale; a.causal = causal != 0; a.dtype = dtype;
    a.out = out; a.lse = lse;
    a.err = static_cast<int32_t *>(workspace);
    const WaitSettings ws = wait_settings();
    a.wait_ns = ws.wait_ns;
    a.debug_drop = ws.drop_chunk;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.delta = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kErrorWordBytes);
    return done(dtype == RDA_BF16 ? launch_latent_forward_tc(a, static_cast<uint8_t *>(workspace) + kErrorWordBytes, s)
                                  : launch_latent_forward_f32(a, s));
}

size_t rda_latent_backward_workspace_bytes(int total_q, int total_k, int H, int Dk, int Ds, int Dv, int num_seqs) {
    if (total_q < 0 || total_k < 0 || H <= 0 || H > kMaxHeads || num_seqs < 0 || !head_dims_ok(Dk, Ds, Dv)) return 0;
    return kErrorWordBytes + std::max(latent_backward_scratch_bytes(total_q, total_k, H, Ds),
                                      latent_backward_tc_scratch_bytes(total_q, total_k, num_seqs, H, Ds));
}

rda_status_t rda_latent_backward(const void *q, const void *q_shared, const void *k, const void *k_shared, const void *v,
                                 const void *out, const float *lse, const void *d_out,
                                 const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                 int num_seqs, int total_q, int total_k,
                                 void *dq, void *dq_shared, void *dk, void *dk_shared, void *dv,
                                 rda_dtype_t dtype, int H, int Dk, int Ds, int Dv, float scale, int causal,
                                 void *workspace, size_t workspace_bytes, void *stream) {
    rda_status_t st = check_packed(q, q_shared, k, k_shared, v, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q, total_k,
                                   dtype, H, Dk, Ds, Dv);
    if (st != RDA_OK) return st;
    if (total_q > 0 && (!out || !lse || !d_out || !dq || (Ds && !dq_shared))) return RDA_ERR_INVALID_ARG;
    if (total_k > 0 && (!dk || !dv || (Ds && !dk_shared))) return RDA_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(d_out, 16) || !aligned(dq, 16) || !aligned(dq_shared, 16) ||
        !aligned(dk, 16) || !aligned(dk_shared, 16) || !aligned(dv, 16))
        return RDA_ERR_MISALIGNED;
    st = check_workspace(workspace, workspace_bytes,
                         rda_latent_backward_workspace_bytes(total_q, total_k, H, Dk, Ds, Dv, num_seqs));
    if (st != RDA_OK) return st;
    if (num_seqs == 0 || (total_q == 0 && total_k == 0)) return RDA_OK;
    LatentArgs a{};
    a.q = q; a.q_shared = q_shared; a.k = k; a.k_shared = k_shared; a.v = v;
    a.cu_q = cu_seqlens_q; a.cu_k = cu_seqlens_k;
    a.num_seqs = num_seqs; a.total_q = total_q; a.total_k = total_k;
    a.H = H; a.Dk = Dk; a.Ds = Ds; a.Dv = Dv; a.scale = scale; a.causal = causal != 0; a.dtype = dtype;
    a.out = const_cast<void *>(out); a.lse = const_cast<float *>(lse); a.d_out = d_out;
    a.dq = dq; a.dq_shared = dq_shared; a.dk = dk; a.dk_shared = dk_shared; a.dv = dv;
    a.err = static_cast<int32_t *>(workspace);
    const WaitSettings ws = wait_settings();
    a.wait_ns = ws.wait_ns;
    a.debug_drop = ws.drop_chunk;
    uint8_t *scratch = static_cast<uint8_t *>(workspace) + kErrorWordBytes;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == RDA_BF16) return done(launch_latent_backward_tc(a, scratch, s));
    a.delta = reinterpret_cast<float *>(scratch);
    a.dks_heads = reinterpret_cast<float *>(scratch + latent_backward_scratch_bytes(total_q, 0, H, Ds));
    cudaError_t e = launch_latent_delta(a, s);
    if (e == cudaSuccess) e = launch_latent_backward_f32(a, s);
    if (e == cudaSuccess && Ds) e = launch_latent_shared_sum(a, s);
    return done(e);
}

size_t rda_latent_decode_workspace_bytes(int B, int T, int H, int Dl, int Ds) {
    if (B < 0 || T < 0 || T > kMaxDecodeTokens || H <= 0 || H > kMaxHeads || Dl <= 0 || Dl > 512 || Dl % 128 ||
        (Ds != 0 && Ds != 64))
        return 0;
    if (!B || !T) return kErrorWordBytes;
    return kErrorWordBytes + std::max(latent_decode_scratch_bytes(B, T, H, Dl), latent_decode_tc_scratch_bytes(T, H, Dl, Ds));
}

rda_status_t rda_latent_decode(const void *q, const void *q_shared, const void *pages, const int32_t *block_table,
                               const int32_t *seq_lens, void *out, float *lse, rda_dtype_t dtype,
                               int B, int T, int H, int Dl, int Ds, int num_pages, int page_size, int table_width,
                               float scale, void *workspace, size_t workspace_bytes, void *stream) {
    if (dtype != RDA_F32 && dtype != RDA_BF16) return RDA_ERR_UNSUPPORTED;
    if (B < 0 || T < 0 || H <= 0 || num_pages < 0 || page_size <= 0 || table_width < 0) return RDA_ERR_INVALID_ARG;
    if (T > kMaxDecodeTokens || B > kMaxBatch || H > kMaxHeads || Dl <= 0 || Dl > 512 || Dl % 128 || (Ds != 0 && Ds != 64) ||
        page_size % 16)
        return RDA_ERR_UNSUPPORTED;
    if ((long long)B * T * H * (Dl + Ds) >= (1LL << 31) || (long long)num_pages * page_size >= (1LL << 31) ||
        (long long)table_width * page_size >= (1LL << 31) - 1024)     // tokens are counted in int, tiles rounded up
        return RDA_ERR_INVALID_ARG;
    if (B > 0 && T > 0) {
        if (!q || (q_shared == nullptr) != (Ds == 0) || !seq_lens || !out) return RDA_ERR_INVALID_ARG;
        if ((table_width > 0 && !block_table) || (num_pages > 0 && !pages)) return RDA_ERR_INVALID_ARG;
    }
    if (!aligned(q, 16) || !aligned(q_shared, 16) || !aligned(pages, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(block_table, 4) || !aligned(seq_lens, 4))
        return RDA_ERR_MISALIGNED;
    const rda_status_t st = check_workspace(workspace, workspace_bytes, rda_latent_decode_workspace_bytes(B, T, H, Dl, Ds));
    if (st != RDA_OK) return st;
    if (B == 0 || T == 0) return RDA_OK;
    LatentDecodeArgs a{};
    a.q = q; a.q_shared = q_shared; a.pages = pages; a.table = block_table; a.lens = seq_lens;
    a.num_pages = num_pages; a.page_size = page_size; a.table_width = table_width;
    a.B = B; a.T = T; a.H = H; a.Dl = Dl; a.Ds = Ds; a.scale = scale; a.dtype = dtype;
    a.out = out; a.lse = lse;
    a.err = static_cast<int32_t *>(workspace);
    const WaitSettings ws = wait_settings();
    a.wait_ns = ws.wait_ns;
    a.debug_drop = ws.drop_chunk;
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kErrorWordBytes);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return done(dtype == RDA_BF16 ? launch_latent_decode_tc(a, s) : launch_latent_decode_f32(a, s));
}

size_t rda_verify_drafts_workspace_bytes(int B, int T, int V) {
    if (B < 0 || T < 0 || T > kMaxDrafts || V <= 0) return 0;
    return kErrorWordBytes + verify_scratch_bytes(B, V);
}

rda_status_t rda_verify_drafts(const int32_t *draft_tokens, const float *draft_probs, const float *target_probs,
                               const float *uniforms, const int32_t *num_drafts, int32_t *tokens, int32_t *num_accepted,
                               int B, int T, int V, void *workspace, size_t workspace_bytes, void *stream) {
    if (B < 0 || T < 0 || V <= 0) return RDA_ERR_INVALID_ARG;
    if (T > kMaxDrafts || B > kMaxBatch || V > (1 << 30)) return RDA_ERR_UNSUPPORTED;
    if (B > 0 && (!target_probs || !uniforms || !tokens || !num_accepted || (T > 0 && !draft_tokens)))
        return RDA_ERR_INVALID_ARG;
    if (!aligned(draft_tokens, 4) || !aligned(draft_probs, 4) || !aligned(target_probs, 4) || !aligned(uniforms, 4) ||
        !aligned(num_drafts, 4) || !aligned(tokens, 4) || !aligned(num_accepted, 4))
        return RDA_ERR_MISALIGNED;
    const rda_status_t st = check_workspace(workspace, workspace_bytes, rda_verify_drafts_workspace_bytes(B, T, V));
    if (st != RDA_OK) return st;
    if (B == 0) return RDA_OK;
    VerifyArgs a{};
    a.draft = draft_tokens; a.draft_probs = draft_probs; a.target_probs = target_probs; a.uniforms = uniforms;
    a.num_drafts = num_drafts; a.tokens = tokens; a.num_accepted = num_accepted;
    a.B = B; a.T = T; a.V = V;
    a.part = reinterpret_cast<double *>(static_cast<uint8_t *>(workspace) + kErrorWordBytes);
    return done(launch_verify(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
