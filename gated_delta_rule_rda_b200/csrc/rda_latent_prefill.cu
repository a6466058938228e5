// Latent attention in its expanded form over packed sequences (bf16): forward.
//
//   s_ij = scale (q_i . k_j + q~_i . k~_j),  o_i = sum_j softmax_j(s_i) v_j,  lse_i = log sum_j e^{s_ij}
//
// Bound by the tensor cores: 2 (Dk + Ds + Dv) flops per visible pair and head,
// against Dk + Dv + Ds / H values a key.  The key part that the heads share is
// read as it lies ([total, Ds]): it is the third column chunk of a key tile.
//
// One CTA per 256 query rows (two tiles of 128) and head; both tiles use every
// key tile that is brought in.  One pass over the keys with the running maximum
// and sum:
//   S_t  [128 x 80]   = Q_t K^T      (both from shared memory; accumulator in TMEM)
//   P_t               = 2^(S_t scale log2 e - m), bf16, written to TMEM
//   O_t  [128 x Dv]  += P_t V        (P from TMEM, V from shared memory)
// 80 keys a tile: S (80 columns) and P (40) of both tiles fit beside the two O
// (128 each) in the 512 columns of TMEM, so that the scores of the next key
// tile can be formed while this one's P is still being computed; a product of N
// = 80 columns from shared memory costs 52 cycles against 40 of arithmetic, one
// of 64 costs 48 against 32.
//
//   warp 0       producer: Q, then K and V tiles by TMA (two stages each)
//   warp 1       one thread issues the scores' MMAs, one of warp 10 those of P: each
//                waits for its own operands only, and neither for the other's
//   warps 2..9   softmax: one thread per query row (no shuffles); O is rescaled
//                only when a row's maximum has grown by more than 2^8
//
// P is rounded to bf16 for its product (relative error 2^-8 at most); sums and
// statistics are fp32.
//
// Measured, 16 heads of 128 + 64 and 128, causal: T = 8192 in 285 us (1.2 PFLOP/s of
// the visible pairs, 73% of what a library's plain product reaches; 335 us in a loop
// under the power cap), T = 4096 in 80 us.  The two products of a step take 1,900
// cycles of tensor pipe (288 of them reread Q), a step 2,600: the rest is what the
// chain of scores, softmax and values leaves exposed, 1,280 cycles of exponentials
// in it.  A pair of CTAs that share the keys
// (cta_group::2, half the reads) measured 389 us against 302 then: its barriers between CTAs cost more
// than the reads.
#include <cmath>
#include <cstring>

#include "rda_latent.h"
#include "rda_latent_order.cuh"
#include "sm100_pipe.cuh"

namespace rda {
namespace {

using namespace ptx;

constexpr int kBM = 128, kQ = 2;             // rows of a query tile, tiles of a CTA
constexpr int kBN = 80;                      // keys of a tile
constexpr int kStages = 2;
constexpr int kSoftWarp = 2;                 // first softmax warp
constexpr int kThreads = 32 * (kSoftWarp + 4 * kQ + 1);
constexpr uint32_t kQChunk = kBM * 128, kKChunk = kBN * 128;      // 64 columns of a tile
constexpr uint32_t kCols = 512;
constexpr uint32_t kTO = 0, kTS = 256, kTP = kTS + 2 * kBN;       // TMEM columns: O (128 each), S (80), P (40)
constexpr float kGrow = 8.f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
static_assert(kTP + 2 * (kBN / 2) <= kCols, "TMEM");

struct Maps {
    CUtensorMap q, q_shared, k, k_shared, v;
};

struct Bars {
    uint64_t q_full[kQ], k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t s_ready[kQ], s_free[kQ], p_ready[kQ], pv_done[kQ];
    uint32_t tmem;
    volatile int abort;
};

__host__ __device__ inline uint32_t smem_bytes(int nk, int nv) {
    return kQ * nk * kQChunk + kStages * (nk + nv) * kKChunk + sizeof(Bars) + 1024;
}

__global__ void __launch_bounds__(kThreads, 1) latent_prefill_kernel(const __grid_constant__ Maps maps, const LatentArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = align_1024(smem_raw);
    const int nd = a.Dk / 64, nk = (a.Dk + a.Ds) / 64, nv = a.Dv / 64;        // 64-column chunks
    uint8_t *q_s = sm, *k_s = q_s + kQ * nk * kQChunk, *v_s = k_s + kStages * nk * kKChunk;
    Bars &B = *reinterpret_cast<Bars *>(v_s + kStages * nv * kKChunk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Waiter w{&B.abort, a.err, a.wait_ns};

    // heads side by side, tiles with the most work first
    pdl_launch_dependents();
    pdl_wait_primary();
    const int h = blockIdx.x % a.H;
    int t;
    const int n = tile_at(a, false, kQ * kBM, blockIdx.x / a.H, gridDim.x / a.H, &t);
    if (n < 0) return;
    const SeqSpan sq = seq_span(a.cu_q, n, a.total_q), sk = seq_span(a.cu_k, n, a.total_k);
    const int r0 = t * kQ * kBM;
    if (r0 >= sq.len) return;
    const int more = sk.len - sq.len;                       // keys before the first query's own
    auto rows_of = [&](int q) { return max(0, min(kBM, sq.len - r0 - q * kBM)); };
    auto tiles_of = [&](int q) {
        const int rows = rows_of(q);
        const int end = a.causal ? min(sk.len, r0 + q * kBM + rows + more) : sk.len;
        return rows > 0 && end > 0 ? (end + kBN - 1) / kBN : 0;
    };
    const int n0 = tiles_of(0), n1 = tiles_of(1), nt = max(n0, n1);

    if (warp == 0) {
        tmem_alloc(&B.tmem, kCols);
        tmem_relinquish();
    }
    if (tid == 32) {
        mbar_init(&B.q_full[0], 1);
        mbar_init(&B.q_full[1], 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&B.k_full[i], 1);
            mbar_init(&B.k_empty[i], 1);
            mbar_init(&B.v_full[i], 1);
            mbar_init(&B.v_empty[i], 1);
        }
        for (int q = 0; q < kQ; ++q) {
            mbar_init(&B.s_ready[q], 1);
            mbar_init(&B.s_free[q], 128);
            mbar_init(&B.p_ready[q], 128);
            mbar_init(&B.pv_done[q], 1);
        }
        B.abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&maps.q);
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B.tmem;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (elect_one() && nt > 0) {
            // in the order of use: the first tile's queries, K, the second tile's queries, V
            auto queries = [&](int q) {
                mbar_arrive_expect_tx(&B.q_full[q], nk * kQChunk);
                for (int c = 0; c < nk; ++c)
                    tma_load_3d(q_s + (q * nk + c) * kQChunk, c < nd ? &maps.q : &maps.q_shared, &B.q_full[q],
                                (c < nd ? c : c - nd) * 64, h, sq.start + r0 + q * kBM);
            };
            if (n0 > 0) queries(0);
            RingPos p;
            bool go = true;
            int loaded_k = 0, loaded_v = 0;
            for (int j = 0; j < nt; ++j) {
                if (j == a.debug_drop) break;
                const int row = sk.start + j * kBN;
                if (j >= kStages) go = go && w.wait(&B.k_empty[p.slot], p.phase ^ 1);
                if (!go) break;
                mbar_arrive_expect_tx(&B.k_full[p.slot], nk * kKChunk);
                for (int c = 0; c < nk; ++c)
                    tma_load_3d(k_s + (p.slot * nk + c) * kKChunk, c < nd ? &maps.k : &maps.k_shared, &B.k_full[p.slot],
                                (c < nd ? c : c - nd) * 64, c < nd ? h : 0, row);
                ++loaded_k;
                if (j == 0 && n1 > 0) queries(1);
                if (j >= kStages) go = go && w.wait(&B.v_empty[p.slot], p.phase ^ 1);
                if (!go) break;
                mbar_arrive_expect_tx(&B.v_full[p.slot], nv * kKChunk);
                for (int c = 0; c < nv; ++c)
                    tma_load_3d(v_s + (p.slot * nv + c) * kKChunk, &maps.v, &B.v_full[p.slot], c * 64, h, row);
                ++loaded_v;
                p.next(kStages);
            }
            if (B.abort) {
                // copies in flight land before the CTA leaves: the last ones of each stage
                const uint64_t t0 = Waiter::now();
                if (n0 > 0) w.drain(&B.q_full[0], 0, t0);
                if (n1 > 0) w.drain(&B.q_full[1], 0, t0);
                for (int i = max(0, loaded_k - kStages); i < loaded_k; ++i)
                    w.drain(&B.k_full[i % kStages], (i / kStages) & 1, t0);
                for (int i = max(0, loaded_v - kStages); i < loaded_v; ++i)
                    w.drain(&B.v_full[i % kStages], (i / kStages) & 1, t0);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs of the scores
        if (elect_one() && nt > 0) {
            const uint32_t idS = idesc_bf16(kBM, kBN, 0, 0);
            const uint64_t dq = smem_desc(smem_u32(q_s), 16, 1024, kSw128), dk = smem_desc(smem_u32(k_s), 16, 1024, kSw128);
            bool ok = true;
            RingPos ks;
            for (int j = 0; j < nt; ++j) {
                ok = w.wait(&B.k_full[ks.slot], ks.phase) && ok;
                for (int q = 0; q < kQ; ++q) {
                    if (j >= (q ? n1 : n0)) continue;
                    ok = (j > 0 ? w.wait(&B.s_free[q], (j - 1) & 1) : w.wait(&B.q_full[q], 0)) && ok;
                    tc_fence_after();
                    if (ok)
                        for (int c = 0; c < nk; ++c) {
                            const uint64_t da = dq + (q * nk + c) * (kQChunk / 16), db = dk + (ks.slot * nk + c) * (kKChunk / 16);
#pragma unroll
                            for (int k = 0; k < 4; ++k) mma_bf16(tmem + kTS + q * kBN, da + 2 * k, db + 2 * k, idS, c > 0 || k > 0);
                        }
                    mma_commit(&B.s_ready[q]);
                }
                mma_commit(&B.k_empty[ks.slot]);
                ks.next(kStages);
            }
            // everything issued has completed with the last commit
            if (B.abort) w.drain(&B.k_empty[(nt - 1) % kStages], ((nt - 1) / kStages) & 1, Waiter::now());
        }
        __syncwarp();
    } else if (warp == kSoftWarp + 8) {
        // ------------------------------------------------------------ MMAs of the values
        if (elect_one() && nt > 0) {
            const uint32_t idO = idesc_bf16(kBM, a.Dv, 0, 1);
            const uint64_t dv = smem_desc(smem_u32(v_s), kKChunk, 1024, kSw128);
            bool ok = true;
            RingPos vs;
            for (int j = 0; j < nt; ++j) {
                ok = w.wait(&B.v_full[vs.slot], vs.phase) && ok;
                for (int q = 0; q < kQ; ++q) {
                    if (j >= (q ? n1 : n0)) continue;
                    ok = w.wait(&B.p_ready[q], j & 1) && ok;
                    tc_fence_after();
                    if (ok) {
                        const uint64_t db = dv + vs.slot * nv * (kKChunk / 16);
#pragma unroll
                        for (int k = 0; k < kBN / 16; ++k)
                            mma_bf16_ta(tmem + kTO + q * 128, tmem + kTP + q * (kBN / 2) + 8 * k, db + 128 * k, idO, j > 0 || k > 0);
                    }
                    mma_commit(&B.pv_done[q]);
                }
                mma_commit(&B.v_empty[vs.slot]);
                vs.next(kStages);
            }
            if (B.abort) w.drain(&B.v_empty[(nt - 1) % kStages], ((nt - 1) / kStages) & 1, Waiter::now());
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax: my row of my tile
        const int q = warp >= 6, quad = warp & 3, rows = rows_of(q), tiles = q ? n1 : n0;
        const int r = 32 * quad + lane;
        const int row = r0 + q * kBM + r;                          // in the sequence
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        const uint32_t t_s = tmem + kTS + q * kBN + lanes, t_p = tmem + kTP + q * (kBN / 2) + lanes,
                       t_o = tmem + kTO + q * 128 + lanes;
        const bool flip = a.scale < 0.f;                           // the maximum is taken of -s then
        const float sc = fabsf(a.scale) * kLog2e;
        const int limit = r >= rows ? 0 : a.causal ? min(sk.len, row + more + 1) : sk.len;     // keys that my row sees
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < tiles; ++j) {
            float s[kBN];
            w.wait(&B.s_ready[q], j & 1);
            tc_fence_after();
            tmem_ld32(t_s, s);
            tmem_ld32(t_s + 32, s + 32);
            tmem_ld16(t_s + 64, s + 64);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&B.s_free[q]);
            if (flip) {
#pragma unroll
                for (int i = 0; i < kBN; ++i) s[i] = -s[i];
            }
            const int left = limit - j * kBN;                      // keys of this tile that I see
            const bool masked = __any_sync(0xffffffffu, left < kBN);
            if (masked) {
#pragma unroll
                for (int i = 0; i < kBN; ++i) s[i] = i < left ? s[i] : -INFINITY;
            }
            float t0 = s[0], t1 = s[1], t2 = s[2], t3 = s[3];
#pragma unroll
            for (int i = 4; i < kBN; i += 4) {
                t0 = fmaxf(t0, s[i]);
                t1 = fmaxf(t1, s[i + 1]);
                t2 = fmaxf(t2, s[i + 2]);
                t3 = fmaxf(t3, s[i + 3]);
            }
            const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3));
            float f = 1.f;
            const bool grown = (top - m) * sc > kGrow || (m == -INFINITY && top > -INFINITY);
            if (grown) {
                f = m == -INFINITY ? 0.f : ex2((m - top) * sc);
                m = top;
            }
            const float base = m == -INFINITY ? 0.f : m * sc;
            // probabilities, and their sums in four chains (a branch inside would keep the exponentials in lockstep)
            float p0 = 0.f, p1 = 0.f, p2 = 0.f, p3 = 0.f;
            uint32_t pk[kBN / 2];
            if (masked) {
#pragma unroll
                for (int i = 0; i < kBN; ++i) s[i] = i < left ? ex2(fmaf(s[i], sc, -base)) : 0.f;     // also for a scale of 0
            } else {
#pragma unroll
                for (int i = 0; i < kBN; ++i) s[i] = ex2(fmaf(s[i], sc, -base));
            }
#pragma unroll
            for (int i = 0; i < kBN; i += 4) {
                p0 += s[i];
                p1 += s[i + 1];
                p2 += s[i + 2];
                p3 += s[i + 3];
                pk[i / 2] = pack2(s[i], s[i + 1]);
                pk[i / 2 + 1] = pack2(s[i + 2], s[i + 3]);
            }
            l = fmaf(l, f, (p0 + p1) + (p2 + p3));
            if (j > 0) w.wait(&B.pv_done[q], (j - 1) & 1);           // P and O are free
            tc_fence_after();
            if (__any_sync(0xffffffffu, grown) && j > 0) {
#pragma unroll 1
                for (int c = 0; c < a.Dv; c += 32) {
                    float o[32];
                    tmem_ld32(t_o + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= f;
                    tmem_st16f(t_o + c, o);
                    tmem_st16f(t_o + c + 16, o + 16);
                }
            }
            tmem_st16(t_p, pk);
            tmem_st16(t_p + 16, pk + 16);
            tmem_st8(t_p + 32, pk + 32);
            // the last keys' rows of V behind the sequence may hold anything: 0 x NaN must not reach O
            const int keys = sk.len - j * kBN;
            if (keys < kBN) {
                w.wait(&B.v_full[j % kStages], (j / kStages) & 1);
                for (int e = tid - 64 - 128 * q; e < (kBN - keys) * nv * 8; e += 128) {
                    const int c = (e >> 3) % nv, kr = keys + (e >> 3) / nv;
                    *reinterpret_cast<uint4 *>(v_s + ((j % kStages) * nv + c) * kKChunk + sw128(kr, e & 7)) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&B.p_ready[q]);
        }
        if (tiles > 0) {
            w.wait(&B.pv_done[q], (tiles - 1) & 1);
            tc_fence_after();
        }
        const float f = l > 0.f ? 1.f / l : 0.f;
        if (r < rows && a.lse) a.lse[(size_t)(sq.start + row) * a.H + h] = l > 0.f ? (m * sc + lg2(l)) * kLn2 : -INFINITY;
        // through the tile's own query rows, which no product reads any more
        uint8_t *buf = q_s + q * nk * kQChunk + quad * 4096;
        auto *out = static_cast<__nv_bfloat16 *>(a.out) + ((size_t)(sq.start + r0 + q * kBM + 32 * quad) * a.H + h) * a.Dv;
#pragma unroll 1
        for (int c = 0; c < nv; ++c) {
            uint4 x[8];
            tmem_row_bf16(t_o + 64 * c, f, tiles > 0, x);
            store_rows_128(buf, x, out + 64 * c, (size_t)a.H * a.Dv * 2, rows - 32 * quad);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

__global__ void __launch_bounds__(512) latent_order_kernel(const LatentArgs a, const TileOrder o) {
    pdl_launch_dependents();
    pdl_wait_primary();
    order_tiles(a, o);
}

}  // namespace

size_t order_bytes(int total, int num_seqs, int tile) { return (size_t)tile_slots(total, num_seqs, tile) * sizeof(int2); }

size_t latent_prefill_scratch_bytes(int total_q, int num_seqs) { return order_bytes(total_q, num_seqs, kQ * kBM); }

cudaError_t launch_latent_forward_tc(const LatentArgs &a0, void *scratch, cudaStream_t s) {
    LatentArgs a = a0;
    cudaError_t e = allow_smem<latent_prefill_kernel>(232448);
    if (e != cudaSuccess) return e;
    Maps m;
    std::memset(&m, 0, sizeof(m));
    if (!make_map_heads(&m.q, a.q, a.Dk, a.H, a.total_q, kBM, a.q) || !make_map_heads(&m.k, a.k, a.Dk, a.H, a.total_k, kBN, a.q) ||
        !make_map_heads(&m.v, a.v, a.Dv, a.H, a.total_k, kBN, a.q) ||
        (a.Ds && (!make_map_heads(&m.q_shared, a.q_shared, a.Ds, a.H, a.total_q, kBM, a.q) ||
                  !make_map_heads(&m.k_shared, a.k_shared, a.Ds, 1, a.total_k, kBN, a.q))))
        return cudaErrorInvalidValue;
    const uint32_t bytes = smem_bytes((a.Dk + a.Ds) / 64, a.Dv / 64);
    const int slots = tile_slots(a.total_q, a.num_seqs, kQ * kBM);
    // Where the CTAs need more than one wave and sequences may differ, the order is worth a small kernel whose
    // launch and run mostly hide: 8 sequences of 0 to 2048 queries take 82.3 us by their places and 79.9 us in
    // order; a single wave, or one sequence, has nothing to gain.
    const bool sorted = worth_order(a) && (long)slots * a.H > kSms;
    if (sorted) {
        TileOrder o{0, kQ * kBM, kBN, static_cast<int2 *>(scratch)};
        if ((e = launch_after(latent_order_kernel, 1, 512, 0, s, a, o)) != cudaSuccess) return e;
        a.order = o.out;
    }
    return launch_after(latent_prefill_kernel, slots * a.H, kThreads, bytes, s, m, a);
}

}  // namespace rda
