// Gradients of latent attention in its expanded form (bf16), packed sequences.
//
//   p_ij = e^{s_ij - lse_i},  dp_ij = do_i . v_j,  delta_i = do_i . o_i,  ds_ij = p_ij (dp_ij - delta_i)
//   dv_j = sum_i p_ij do_i,   dk_j = scale sum_i ds_ij q_i,   dq_i = scale sum_j ds_ij k_j
//
// Bound by the tensor cores.  Two kernels, each with the sums that its CTA owns
// in TMEM: one over keys (dv, dk), one over query rows (dq).  The scores and dp
// are formed in both, seven products instead of five; in exchange no sum is
// shared between CTAs: nothing depends on the order of atomics, and no fp32
// copy of dq is written, cleared and converted.
//
//   keys    128 keys x 64 query rows a step:  S^T = K Q^T,  dP^T = V dO^T  (shared memory),
//           then dV += P^T dO and dK += dS^T Q with P^T, dS^T as TMEM operands
//   rows    128 query rows x 80 keys a step:  S = Q K^T,  dP = dO V^T,  then dQ += dS K
//
// In both, one thread issues the first two products and another those that P and
// dS go into, each as soon as its own operands are there, so that the tensor pipe
// and the eight element-wise warps (a lane per key, or per query row; two warps
// share the columns of a lane) work at the same time.  P and dS are rounded to
// bf16 for their products; p, dp, delta and all sums are fp32.
//
// Measured, 16 heads of 128 + 64 and 128, T = 4096, causal: dQ 122 us, dK and dV 146
// us, statistics 10 us, the sum 7 us (335 us a call in a loop under the power cap).  A
// step of the keys kernel takes 1,980 cycles, its MMAs 1,620; one of the rows kernel
// 2,030 and 1,530.  96 keys a step in two stages measured 181 us for dQ: the third
// stage of K is worth more than the longer step.
//
// The key part that all heads share gets its gradient from every head: the
// heads' parts are written in fp32 and summed in a fixed order afterwards.
#include <cmath>
#include <cstring>

#include "rda_latent.h"
#include "rda_latent_order.cuh"
#include "sm100_pipe.cuh"

namespace rda {
namespace {

using namespace ptx;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kElemWarp = 2;                    // first element-wise warp
constexpr int kThreads = 32 * (kElemWarp + 8 + 1);
constexpr uint32_t kCols = 512;
constexpr int kStat = 64;                       // query rows of a block of statistics
constexpr uint32_t kBig = 128 * 128;            // 128 rows x 64 columns

// keys kernel
constexpr int kRows = 64, kStagesA = 3;         // query rows of a step
constexpr uint32_t kSmall = kRows * 128;        // 64 rows x 64 columns
constexpr uint32_t kTdV = 0, kTdK = 128, kTS = 320, kTdP = 384, kTP = 448, kTdS = 480;
// rows kernel
constexpr int kKeys = 80, kStK = 3, kStV = 2;   // keys of a step; V is free again before K
constexpr uint32_t kMid = kKeys * 128;          // 80 rows x 64 columns
constexpr uint32_t kUdQ = 0, kUS = 192, kUdP = kUS + kKeys, kUdS = kUdP + kKeys;

struct Maps {
    CUtensorMap q, q_shared, k, k_shared, v, d_out;
};

// ---------------------------------------------------------------------------
// Statistics of 64 query rows of a head, ready for the exponent: lse log2 e and
// delta, [head][block][2][64].  Rows behind the sequence's end, and rows that
// saw no key, get +inf: their p is 2^-inf = 0.
// ---------------------------------------------------------------------------
// Two more CTAs (of the row behind the heads) put the tiles of the other kernels in order.
__global__ void __launch_bounds__(256) latent_stats_kernel(const LatentArgs a, float *stats, const TileOrder rows,
                                                           const TileOrder keys) {
    pdl_launch_dependents();
    pdl_wait_primary();
    if (blockIdx.y == a.H) {
        if (blockIdx.x < 2) order_tiles(a, blockIdx.x ? keys : rows);
        return;
    }
    int t;
    const int n = find_tile(a.cu_q, a.num_seqs, a.total_q, kStat, blockIdx.x, &t);
    const SeqSpan sq = seq_span(a.cu_q, n, a.total_q);
    const int h = blockIdx.y;
    // a lane per 16 bytes of a row: 16 or 8 lanes a row, all loads of a warp's 8 rows in flight at once
    const int lanes = a.Dv / 8, per = 32 / lanes, lane = threadIdx.x & 31, part = lane % lanes;
    const int first = (threadIdx.x >> 5) * 8 + lane / lanes;
    uint4 u[4], v[4];
    float lse[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = t * kStat + first + i * per;
        u[i] = v[i] = make_uint4(0, 0, 0, 0);
        lse[i] = -INFINITY;
        if (i * per < 8 && row < sq.len) {
            const size_t at = (size_t)(sq.start + row) * a.H + h;
            u[i] = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.out) + at * a.Dv)[part];
            v[i] = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.d_out) + at * a.Dv)[part];
            lse[i] = a.lse[at];
        }
    }
    float *s = stats + ((size_t)h * gridDim.x + blockIdx.x) * 2 * kStat;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i * per >= 8) break;
        float x = 0.f;
        const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&u[i]);
        const __nv_bfloat162 *q = reinterpret_cast<const __nv_bfloat162 *>(&v[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = __bfloat1622float2(p[k]), g = __bfloat1622float2(q[k]);
            x = fmaf(f.x, g.x, fmaf(f.y, g.y, x));
        }
        for (int off = lanes / 2; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        if (part == 0) {
            s[first + i * per] = lse[i] == -INFINITY ? INFINITY : lse[i] * kLog2e;
            s[kStat + first + i * per] = x;
        }
    }
}

__device__ __forceinline__ int stat_block(const LatentArgs &a, int n, int row) {
    return clamped(a.cu_q, n, a.total_q) / kStat + n + row / kStat;
}

// 16-byte chunks [0, 8) of rows [from, to) of `chunks` tiles of 128-byte rows, zeroed by 256 threads.
__device__ __forceinline__ void zero_rows(uint8_t *tile, uint32_t tile_bytes, int chunks, int from, int to) {
    const int n = (to - from) * 8;
    for (int c = 0; c < chunks; ++c)
        for (int e = threadIdx.x - 64; e < n; e += 256)
            *reinterpret_cast<uint4 *>(tile + c * tile_bytes + sw128(from + (e >> 3), e & 7)) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// dK and dV: one CTA per (128 keys, head).
// ---------------------------------------------------------------------------
struct BarsA {
    uint64_t kv_full, q_full[kStagesA], q_empty[kStagesA];
    uint64_t s_ready, s_free, p_ready, dv_done, dp_ready, dp_free, ds_ready, dk_done;
    uint32_t tmem;
    volatile int abort;
};
__host__ __device__ inline uint32_t stage_a(int nk, int nv) { return (nk + nv) * kSmall + 1024; }
inline uint32_t smem_a(int nk, int nv) { return (nk + nv) * kBig + kStagesA * stage_a(nk, nv) + sizeof(BarsA) + 1024; }

__global__ void __launch_bounds__(kThreads, 1)
    latent_dkv_kernel(const __grid_constant__ Maps maps, const LatentArgs a, const float *stats, int stat_blocks) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = align_1024(smem_raw);
    const int nd = a.Dk / 64, nk = (a.Dk + a.Ds) / 64, nv = a.Dv / 64;
    const uint32_t stage = stage_a(nk, nv);
    uint8_t *k_s = sm, *v_s = k_s + nk * kBig, *st_s = v_s + nv * kBig;       // a stage: Q, dO, statistics
    BarsA &B = *reinterpret_cast<BarsA *>(st_s + kStagesA * stage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Waiter w{&B.abort, a.err, a.wait_ns};

    // heads side by side, tiles with the most work first
    const int h = blockIdx.x % a.H;
    pdl_launch_dependents();
    pdl_wait_primary();
    int t;
    const int n = tile_at(a, true, 128, blockIdx.x / a.H, gridDim.x / a.H, &t);
    if (n < 0) return;
    const SeqSpan sq = seq_span(a.cu_q, n, a.total_q), sk = seq_span(a.cu_k, n, a.total_k);
    const int k0 = t * 128, more = sk.len - sq.len;
    if (k0 >= sk.len) return;
    const int first = a.causal ? max(0, k0 - more) / kRows : 0;               // the first step with a query that sees key k0
    const int steps = max(0, (sq.len + kRows - 1) / kRows - first);

    if (warp == 0) {
        tmem_alloc(&B.tmem, kCols);
        tmem_relinquish();
    }
    if (tid == 32) {
        mbar_init(&B.kv_full, 1);
        for (int i = 0; i < kStagesA; ++i) mbar_init(&B.q_full[i], 1), mbar_init(&B.q_empty[i], 1);
        mbar_init(&B.s_ready, 1);
        mbar_init(&B.dp_ready, 1);
        mbar_init(&B.dv_done, 1);
        mbar_init(&B.dk_done, 1);
        mbar_init(&B.s_free, 256);
        mbar_init(&B.p_ready, 256);
        mbar_init(&B.dp_free, 256);
        mbar_init(&B.ds_ready, 256);
        B.abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.q);
        prefetch_tensormap(&maps.d_out);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B.tmem;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (elect_one() && steps > 0) {
            mbar_arrive_expect_tx(&B.kv_full, (nk + nv) * kBig);
            for (int c = 0; c < nk; ++c)
                tma_load_3d(k_s + c * kBig, c < nd ? &maps.k : &maps.k_shared, &B.kv_full, (c < nd ? c : c - nd) * 64,
                            c < nd ? h : 0, sk.start + k0);
            for (int c = 0; c < nv; ++c) tma_load_3d(v_s + c * kBig, &maps.v, &B.kv_full, c * 64, h, sk.start + k0);
            RingPos p;
            int loaded = 0;
            for (; loaded < steps; ++loaded) {
                if (loaded == a.debug_drop) break;
                const int row = (first + loaded) * kRows;
                if (loaded >= kStagesA && !w.wait(&B.q_empty[p.slot], p.phase ^ 1)) break;
                uint8_t *dst = st_s + p.slot * stage;
                mbar_arrive_expect_tx(&B.q_full[p.slot], (nk + nv) * kSmall + 2 * kStat * 4);
                for (int c = 0; c < nk; ++c)
                    tma_load_3d(dst + c * kSmall, c < nd ? &maps.q : &maps.q_shared, &B.q_full[p.slot],
                                (c < nd ? c : c - nd) * 64, h, sq.start + row);
                for (int c = 0; c < nv; ++c)
                    tma_load_3d(dst + (nk + c) * kSmall, &maps.d_out, &B.q_full[p.slot], c * 64, h, sq.start + row);
                bulk_load(dst + (nk + nv) * kSmall, stats + ((size_t)h * stat_blocks + stat_block(a, n, row)) * 2 * kStat,
                          2 * kStat * 4, &B.q_full[p.slot]);
                p.next(kStagesA);
            }
            if (B.abort) {
                const uint64_t t0 = Waiter::now();
                w.drain(&B.kv_full, 0, t0);
                for (int i = max(0, loaded - kStagesA); i < loaded; ++i)
                    w.drain(&B.q_full[i % kStagesA], (i / kStagesA) & 1, t0);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs of S^T and dP^T
        if (elect_one() && steps > 0) {
            const uint32_t id = idesc_bf16(128, kRows, 0, 0);
            const uint64_t dk = smem_desc(smem_u32(k_s), 16, 1024, kSw128), dv = smem_desc(smem_u32(v_s), 16, 1024, kSw128);
            const uint64_t ds = smem_desc(smem_u32(st_s), 16, 1024, kSw128);          // K-major
            bool ok = w.wait(&B.kv_full, 0);
            // `chunks` of 64 columns of the stationary tile against the stage's
            auto product = [&](uint32_t d, uint64_t da, uint64_t db, int chunks) {
                for (int c = 0; c < chunks; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(d, da + c * (kBig / 16) + 2 * k, db + c * (kSmall / 16) + 2 * k, id, c > 0 || k > 0);
            };
            RingPos p;
            for (int i = 0; i < steps; ++i) {
                const uint64_t off = p.slot * (stage / 16);
                ok = w.wait(&B.q_full[p.slot], p.phase) && ok;
                if (i > 0) ok = w.wait(&B.s_free, (i - 1) & 1) && ok;
                tc_fence_after();
                if (ok) product(tmem + kTS, dk, ds + off, nk);
                mma_commit(&B.s_ready);
                if (i > 0) ok = w.wait(&B.dp_free, (i - 1) & 1) && ok;
                tc_fence_after();
                if (ok) product(tmem + kTdP, dv, ds + off + nk * (kSmall / 16), nv);
                mma_commit(&B.dp_ready);
                p.next(kStagesA);
            }
            // everything issued has completed with the last commit
            if (B.abort) w.drain(&B.dp_ready, (steps - 1) & 1, Waiter::now());
        }
        __syncwarp();
    } else if (warp == kElemWarp + 8) {
        // ------------------------------------------------------------ MMAs of dV and dK
        if (elect_one() && steps > 0) {
            const uint32_t idV = idesc_bf16(128, a.Dv, 0, 1), idK = idesc_bf16(128, 64 * nk, 0, 1);
            const uint64_t dm = smem_desc(smem_u32(st_s), kSmall, 1024, kSw128);      // MN-major
            bool ok = true;
            RingPos p;
            for (int i = 0; i < steps; ++i) {
                const uint64_t off = p.slot * (stage / 16);
                ok = w.wait(&B.p_ready, i & 1) && ok;
                tc_fence_after();
                if (ok) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16_ta(tmem + kTdV, tmem + kTP + 8 * k, dm + off + nk * (kSmall / 16) + 128 * k, idV, i > 0 || k > 0);
                }
                mma_commit(&B.dv_done);
                ok = w.wait(&B.ds_ready, i & 1) && ok;
                tc_fence_after();
                if (ok) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16_ta(tmem + kTdK, tmem + kTdS + 8 * k, dm + off + 128 * k, idK, i > 0 || k > 0);
                }
                mma_commit(&B.q_empty[p.slot]);
                mma_commit(&B.dk_done);
                p.next(kStagesA);
            }
            if (B.abort) w.drain(&B.dk_done, (steps - 1) & 1, Waiter::now());
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ element-wise: my key, half of the query rows
        const int quad = warp & 3, half = warp >= 6, key = k0 + 32 * quad + lane;
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        const uint32_t t_s = tmem + kTS + 32 * half + lanes, t_dp = tmem + kTdP + 32 * half + lanes,
                       t_p = tmem + kTP + 16 * half + lanes, t_ds = tmem + kTdS + 16 * half + lanes;
        const float sc = a.scale * kLog2e;
        RingPos p;
        for (int i = 0; i < steps; ++i) {
            const int row0 = (first + i) * kRows;
            const float *st = reinterpret_cast<const float *>(st_s + p.slot * stage + (nk + nv) * kSmall) + 32 * half;
            const int rows = sq.len - row0;                        // query rows of this step that exist
            // my first visible query among my 32
            const int from = a.causal ? key - more - row0 - 32 * half : 0, to = rows - 32 * half;
            const bool masked = __any_sync(0xffffffffu, from > 0 || to < 32);
            float x[32], y[32];
            w.wait(&B.s_ready, i & 1);
            tc_fence_after();
            tmem_ld32(t_s, x);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&B.s_free);
            w.wait(&B.q_full[p.slot], p.phase);                    // the statistics, written by the copy
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
                const float4 lse = *reinterpret_cast<const float4 *>(st + c);
                x[c] = ex2(fmaf(x[c], sc, -lse.x));
                x[c + 1] = ex2(fmaf(x[c + 1], sc, -lse.y));
                x[c + 2] = ex2(fmaf(x[c + 2], sc, -lse.z));
                x[c + 3] = ex2(fmaf(x[c + 3], sc, -lse.w));
            }
            if (masked) {
#pragma unroll
                for (int c = 0; c < 32; ++c) x[c] = c >= from && c < to ? x[c] : 0.f;
            }
#pragma unroll
            for (int c = 0; c < 32; c += 2) pk[c / 2] = pack2(x[c], x[c + 1]);
            if (i > 0) w.wait(&B.dv_done, (i - 1) & 1);
            tc_fence_after();
            tmem_st16(t_p, pk);
            if (rows < kRows) {
                // rows behind the sequence may hold anything: 0 x NaN must not reach the sums
                zero_rows(st_s + p.slot * stage, kSmall, nk + nv, rows, kRows);
                fence_proxy_async_smem();
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&B.p_ready);
            w.wait(&B.dp_ready, i & 1);
            tc_fence_after();
            tmem_ld32(t_dp, y);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&B.dp_free);
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
                const float4 d = *reinterpret_cast<const float4 *>(st + kStat + c);
                y[c] = x[c] * (y[c] - d.x);
                y[c + 1] = x[c + 1] * (y[c + 1] - d.y);
                y[c + 2] = x[c + 2] * (y[c + 2] - d.z);
                y[c + 3] = x[c + 3] * (y[c + 3] - d.w);
            }
            if (rows < kRows) {
#pragma unroll
                for (int c = 0; c < 32; ++c) y[c] = c < to ? y[c] : 0.f;
            }
#pragma unroll
            for (int c = 0; c < 32; c += 2) pk[c / 2] = pack2(y[c], y[c + 1]);
            if (i > 0) w.wait(&B.dk_done, (i - 1) & 1);
            tc_fence_after();
            tmem_st16(t_ds, pk);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&B.ds_ready);
            p.next(kStagesA);
        }
        if (steps > 0) {
            w.wait(&B.dk_done, (steps - 1) & 1);
            tc_fence_after();
        }
        // through the stages, which no product reads any more
        const int rows = sk.len - k0 - 32 * quad;
        const bool any = steps > 0;
        uint8_t *buf = st_s + (warp - kElemWarp) * 4096;
        const size_t at = (size_t)(sk.start + k0 + 32 * quad) * a.H + h;
        uint4 x[8];
#pragma unroll 1
        for (int c = 0; c < (half ? nd : nv); ++c) {
            const int D = half ? a.Dk : a.Dv;
            tmem_row_bf16(tmem + (half ? kTdK : kTdV) + 64 * c + lanes, half ? a.scale : 1.f, any, x);
            store_rows_128(buf, x, static_cast<__nv_bfloat16 *>(half ? a.dk : a.dv) + at * D + 64 * c, (size_t)a.H * D * 2, rows);
        }
        if (a.Ds) {
            // the shared part: 32 of its 64 columns each
            tmem_row_f32(tmem + kTdK + a.Dk + 32 * half + lanes, a.scale, any, x);
            store_rows_128(buf, x, a.dks_heads + at * a.Ds + 32 * half, (size_t)a.H * a.Ds * 4, rows);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// ---------------------------------------------------------------------------
// dQ: one CTA per (128 query rows, head).
//
// delta from the stored result carries that result's rounding to bf16, an error
// of up to 2^-8 sum |do o| that all ds of a row share.  Over many keys the result
// is an average and small; over few it is as large as v, and with one visible key
// ds should vanish.  Tiles that see at most two steps of keys therefore run a
// pass ahead: sum_j p_ij (dp_ij - delta_i) is what delta lacks, and delta is
// corrected before it is used, here and (through the statistics) for dK.
// ---------------------------------------------------------------------------
constexpr int kExactSteps = 2;
struct BarsB {
    uint64_t q_full, k_full[kStK], k_empty[kStK], v_full[kStV], v_empty[kStV];
    uint64_t s_ready, s_free, dp_ready, dp_free, ds_ready, dq_done;
    float lack[2][128];                          // sum of ds of a row, by half of the columns
    uint32_t tmem;
    volatile int abort;
};
inline uint32_t smem_b(int nk, int nv) {
    return (nk + nv) * kBig + (kStK * nk + kStV * nv) * kMid + sizeof(BarsB) + 1024;
}

__global__ void __launch_bounds__(kThreads, 1)
    latent_dq_kernel(const __grid_constant__ Maps maps, const LatentArgs a, float *stats, int stat_blocks) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = align_1024(smem_raw);
    const int nd = a.Dk / 64, nk = (a.Dk + a.Ds) / 64, nv = a.Dv / 64;
    uint8_t *q_s = sm, *o_s = q_s + nk * kBig, *k_s = o_s + nv * kBig, *v_s = k_s + kStK * nk * kMid;
    BarsB &B = *reinterpret_cast<BarsB *>(v_s + kStV * nv * kMid);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Waiter w{&B.abort, a.err, a.wait_ns};

    const int h = blockIdx.x % a.H;
    pdl_launch_dependents();
    pdl_wait_primary();
    int t;
    const int n = tile_at(a, false, 128, blockIdx.x / a.H, gridDim.x / a.H, &t);
    if (n < 0) return;
    const SeqSpan sq = seq_span(a.cu_q, n, a.total_q), sk = seq_span(a.cu_k, n, a.total_k);
    const int r0 = t * 128, more = sk.len - sq.len;
    const int rows = min(128, sq.len - r0);
    if (rows <= 0) return;
    const int end = a.causal ? min(sk.len, r0 + rows + more) : sk.len;
    const int tiles = end > 0 ? (end + kKeys - 1) / kKeys : 0;
    const int ahead = tiles <= kExactSteps ? tiles : 0, steps = ahead + tiles;      // steps before the first that counts

    if (warp == 0) {
        tmem_alloc(&B.tmem, kCols);
        tmem_relinquish();
    }
    if (tid == 32) {
        mbar_init(&B.q_full, 1);
        for (int i = 0; i < kStK; ++i) mbar_init(&B.k_full[i], 1), mbar_init(&B.k_empty[i], 1);
        for (int i = 0; i < kStV; ++i) mbar_init(&B.v_full[i], 1), mbar_init(&B.v_empty[i], 1);
        mbar_init(&B.s_ready, 1);
        mbar_init(&B.dp_ready, 1);
        mbar_init(&B.dq_done, 1);
        mbar_init(&B.s_free, 256);
        mbar_init(&B.dp_free, 256);
        mbar_init(&B.ds_ready, 256);
        B.abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.q);
        prefetch_tensormap(&maps.d_out);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B.tmem;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (elect_one() && steps > 0) {
            mbar_arrive_expect_tx(&B.q_full, (nk + nv) * kBig);
            for (int c = 0; c < nk; ++c)
                tma_load_3d(q_s + c * kBig, c < nd ? &maps.q : &maps.q_shared, &B.q_full, (c < nd ? c : c - nd) * 64, h,
                            sq.start + r0);
            for (int c = 0; c < nv; ++c) tma_load_3d(o_s + c * kBig, &maps.d_out, &B.q_full, c * 64, h, sq.start + r0);
            RingPos pk, pv;
            int loaded_k = 0, loaded_v = 0;
            for (int i = 0; i < steps; ++i) {
                if (i == a.debug_drop) break;
                const int row = sk.start + (i < ahead ? i : i - ahead) * kKeys;
                if (i >= kStK && !w.wait(&B.k_empty[pk.slot], pk.phase ^ 1)) break;
                mbar_arrive_expect_tx(&B.k_full[pk.slot], nk * kMid);
                for (int c = 0; c < nk; ++c)
                    tma_load_3d(k_s + (pk.slot * nk + c) * kMid, c < nd ? &maps.k : &maps.k_shared, &B.k_full[pk.slot],
                                (c < nd ? c : c - nd) * 64, c < nd ? h : 0, row);
                pk.next(kStK);
                ++loaded_k;
                if (i >= kStV && !w.wait(&B.v_empty[pv.slot], pv.phase ^ 1)) break;
                mbar_arrive_expect_tx(&B.v_full[pv.slot], nv * kMid);
                for (int c = 0; c < nv; ++c)
                    tma_load_3d(v_s + (pv.slot * nv + c) * kMid, &maps.v, &B.v_full[pv.slot], c * 64, h, row);
                pv.next(kStV);
                ++loaded_v;
            }
            if (B.abort) {
                const uint64_t t0 = Waiter::now();
                w.drain(&B.q_full, 0, t0);
                for (int i = max(0, loaded_k - kStK); i < loaded_k; ++i) w.drain(&B.k_full[i % kStK], (i / kStK) & 1, t0);
                for (int i = max(0, loaded_v - kStV); i < loaded_v; ++i) w.drain(&B.v_full[i % kStV], (i / kStV) & 1, t0);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs of S and dP
        if (elect_one() && steps > 0) {
            const uint32_t id = idesc_bf16(128, kKeys, 0, 0);
            const uint64_t dq = smem_desc(smem_u32(q_s), 16, 1024, kSw128), dO = smem_desc(smem_u32(o_s), 16, 1024, kSw128);
            const uint64_t dk = smem_desc(smem_u32(k_s), 16, 1024, kSw128), dv = smem_desc(smem_u32(v_s), 16, 1024, kSw128);
            bool ok = w.wait(&B.q_full, 0);
            auto product = [&](uint32_t d, uint64_t da, uint64_t db, int chunks) {
                for (int c = 0; c < chunks; ++c)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(d, da + c * (kBig / 16) + 2 * k, db + c * (kMid / 16) + 2 * k, id, c > 0 || k > 0);
            };
            RingPos ks, vs;
            for (int i = 0; i < steps; ++i) {
                ok = w.wait(&B.k_full[ks.slot], ks.phase) && ok;
                if (i > 0) ok = w.wait(&B.s_free, (i - 1) & 1) && ok;
                tc_fence_after();
                if (ok) product(tmem + kUS, dq, dk + ks.slot * nk * (kMid / 16), nk);
                mma_commit(&B.s_ready);
                ks.next(kStK);
                ok = w.wait(&B.v_full[vs.slot], vs.phase) && ok;
                if (i > 0) ok = w.wait(&B.dp_free, (i - 1) & 1) && ok;
                tc_fence_after();
                if (ok) product(tmem + kUdP, dO, dv + vs.slot * nv * (kMid / 16), nv);
                mma_commit(&B.v_empty[vs.slot]);
                mma_commit(&B.dp_ready);
                vs.next(kStV);
            }
            // everything issued has completed with the last commit
            if (B.abort) w.drain(&B.dp_ready, (steps - 1) & 1, Waiter::now());
        }
        __syncwarp();
    } else if (warp == kElemWarp + 8) {
        // ------------------------------------------------------------ MMAs of dQ
        if (elect_one() && steps > 0) {
            const uint32_t id = idesc_bf16(128, 64 * nk, 0, 1);
            const uint64_t dm = smem_desc(smem_u32(k_s), kMid, 1024, kSw128);         // K, MN-major
            bool ok = true;
            RingPos p;
            for (int i = 0; i < steps; ++i) {
                ok = w.wait(&B.ds_ready, i & 1) && ok;
                tc_fence_after();
                if (ok && i >= ahead) {
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        mma_bf16_ta(tmem + kUdQ, tmem + kUdS + 8 * k, dm + p.slot * nk * (kMid / 16) + 128 * k, id, i > ahead || k > 0);
                }
                mma_commit(&B.k_empty[p.slot]);
                mma_commit(&B.dq_done);
                p.next(kStK);
            }
            if (B.abort) w.drain(&B.dq_done, (steps - 1) & 1, Waiter::now());
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ element-wise: my query row, half of the keys
        constexpr int C = kKeys / 2;
        static_assert(C == 40, "loads of 32 + 8 columns");
        const int quad = warp & 3, half = warp >= 6, r = 32 * quad + lane, row = r0 + r;
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        const uint32_t t_s = tmem + kUS + C * half + lanes, t_dp = tmem + kUdP + C * half + lanes,
                       t_ds = tmem + kUdS + C / 2 * half + lanes;
        const float sc = a.scale * kLog2e;
        const int limit = r >= rows ? 0 : a.causal ? min(sk.len, row + more + 1) : sk.len;      // keys that my row sees
        float lse = INFINITY, delta = 0.f, lack = 0.f;
        float *st = stats + ((size_t)h * stat_blocks + stat_block(a, n, row)) * 2 * kStat + row % kStat;
        if (r < rows) {
            lse = st[0];
            delta = st[kStat];
        }
        RingPos p;
        for (int i = 0; i < steps; ++i) {
            float x[C];
            uint32_t pk[C / 2];
            const int k0 = (i < ahead ? i : i - ahead) * kKeys, left = limit - k0 - C * half;
            const bool masked = __any_sync(0xffffffffu, left < C);
            w.wait(&B.s_ready, i & 1);
            tc_fence_after();
            tmem_ld32(t_s, x);
            tmem_ld8(t_s + 32, x + 32);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&B.s_free);
#pragma unroll
            for (int c = 0; c < C; ++c) x[c] = ex2(fmaf(x[c], sc, -lse));
            const int keys = sk.len - k0;
            if (keys < kKeys) {
                // keys behind the sequence may hold anything: 0 x NaN must not reach the sums
                w.wait(&B.k_full[p.slot], p.phase);
                zero_rows(k_s + p.slot * nk * kMid, kMid, nk, keys, kKeys);
                fence_proxy_async_smem();
            }
            w.wait(&B.dp_ready, i & 1);
            tc_fence_after();
            float y[C];
            tmem_ld32(t_dp, y);
            tmem_ld8(t_dp + 32, y + 32);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&B.dp_free);
#pragma unroll
            for (int c = 0; c < C; ++c) x[c] *= y[c] - delta;
            if (masked) {
#pragma unroll
                for (int c = 0; c < C; ++c) x[c] = c < left ? x[c] : 0.f;
            }
            if (i < ahead) {
#pragma unroll
                for (int c = 0; c < C; ++c) lack += x[c];
                if (i == ahead - 1) {
                    B.lack[half][r] = lack;
                    named_bar_sync(1, 256);
                    delta += B.lack[0][r] + B.lack[1][r];
                    if (half == 0 && r < rows) st[kStat] = delta;
                }
                // not two phases ahead of the thread that waits for them: it tells them apart by parity alone
                if (i > 0) w.wait(&B.dq_done, (i - 1) & 1);
                mbar_arrive(&B.ds_ready);
                p.next(kStK);
                continue;
            }
#pragma unroll
            for (int c = 0; c < C; c += 2) pk[c / 2] = pack2(x[c], x[c + 1]);
            if (i > 0) w.wait(&B.dq_done, (i - 1) & 1);
            tc_fence_after();
            tmem_st16(t_ds, pk);
            tmem_st4(t_ds + 16, pk + 16);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&B.ds_ready);
            p.next(kStK);
        }
        if (steps > 0) {
            w.wait(&B.dq_done, (steps - 1) & 1);
            tc_fence_after();
        }
        // through the stages, which no product reads any more; chunks of 64 columns in turn
        uint8_t *buf = k_s + (warp - kElemWarp) * 4096;
        const size_t at = (size_t)(sq.start + r0 + 32 * quad) * a.H + h;
#pragma unroll 1
        for (int c = half; c < nk; c += 2) {
            uint4 x[8];
            tmem_row_bf16(tmem + kUdQ + 64 * c + lanes, a.scale, steps > 0, x);
            if (c < nd)
                store_rows_128(buf, x, static_cast<__nv_bfloat16 *>(a.dq) + at * a.Dk + 64 * c, (size_t)a.H * a.Dk * 2, rows - 32 * quad);
            else
                store_rows_128(buf, x, static_cast<__nv_bfloat16 *>(a.dq_shared) + at * a.Ds, (size_t)a.H * a.Ds * 2, rows - 32 * quad);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

size_t stats_bytes(int total_q, int num_seqs, int H) {
    return (size_t)tile_slots(total_q, num_seqs, kStat) * H * 2 * kStat * sizeof(float);
}

bool make_maps(Maps *m, const LatentArgs &a, uint32_t box_q, uint32_t box_k) {
    std::memset(m, 0, sizeof(*m));
    const void *any = a.total_q ? a.q : a.k;
    return make_map_heads(&m->q, a.q, a.Dk, a.H, a.total_q, box_q, any) && make_map_heads(&m->k, a.k, a.Dk, a.H, a.total_k, box_k, any) &&
           make_map_heads(&m->v, a.v, a.Dv, a.H, a.total_k, box_k, any) &&
           make_map_heads(&m->d_out, a.d_out, a.Dv, a.H, a.total_q, box_q, any) &&
           (!a.Ds || (make_map_heads(&m->q_shared, a.q_shared, a.Ds, a.H, a.total_q, box_q, any) &&
                      make_map_heads(&m->k_shared, a.k_shared, a.Ds, 1, a.total_k, box_k, any)));
}

}  // namespace

// statistics, the shared key part's gradients by head, and the two orders
size_t latent_backward_tc_scratch_bytes(int total_q, int total_k, int num_seqs, int H, int Ds) {
    return stats_bytes(total_q, num_seqs, H) + (size_t)total_k * H * Ds * sizeof(float) + order_bytes(total_q, num_seqs, 128) +
           order_bytes(total_k, num_seqs, 128);
}

cudaError_t launch_latent_backward_tc(const LatentArgs &a0, void *scratch, cudaStream_t s) {
    LatentArgs a = a0;
    float *stats = static_cast<float *>(scratch);
    a.dks_heads = reinterpret_cast<float *>(static_cast<uint8_t *>(scratch) + stats_bytes(a.total_q, a.num_seqs, a.H));
    cudaError_t e = allow_smem<latent_dkv_kernel>(232448);
    if (e == cudaSuccess) e = allow_smem<latent_dq_kernel>(232448);
    if (e != cudaSuccess) return e;
    const int blocks = tile_slots(a.total_q, a.num_seqs, kStat), nk = (a.Dk + a.Ds) / 64, nv = a.Dv / 64;
    TileOrder rows{0, 128, kKeys, nullptr}, keys{1, 128, kRows, nullptr};
    rows.out = reinterpret_cast<int2 *>(a.dks_heads + (size_t)a.total_k * a.H * a.Ds);
    keys.out = rows.out + tile_slots(a.total_q, a.num_seqs, 128);
    const bool sorted = worth_order(a);           // two CTAs beside the others (blocks >= num_seqs >= 2)
    if (a.total_q > 0 || sorted) {
        e = launch_after(latent_stats_kernel, dim3(blocks, a.H + sorted), 256, 0, s, a, stats, rows, keys);
        if (e != cudaSuccess) return e;
    }
    Maps m;
    // dQ first: it corrects the statistics that dK uses
    if (a.total_q > 0) {
        if (!make_maps(&m, a, 128, kKeys)) return cudaErrorInvalidValue;
        a.order = sorted ? rows.out : nullptr;
        e = launch_after(latent_dq_kernel, tile_slots(a.total_q, a.num_seqs, 128) * a.H, kThreads, smem_b(nk, nv), s, m, a,
                         stats, blocks);
        if (e != cudaSuccess) return e;
    }
    if (a.total_k > 0) {
        if (!make_maps(&m, a, kRows, 128)) return cudaErrorInvalidValue;
        a.order = sorted ? keys.out : nullptr;
        e = launch_after(latent_dkv_kernel, tile_slots(a.total_k, a.num_seqs, 128) * a.H, kThreads, smem_a(nk, nv), s, m, a,
                         stats, blocks);
        if (e != cudaSuccess) return e;
    }
    return a.Ds ? launch_latent_shared_sum(a, s) : cudaSuccess;
}

}  // namespace rda
