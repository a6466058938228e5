// Latent attention in its absorbed form over a paged cache (bf16), for 1..8 new
// tokens a sequence.
//
//   s_rj = scale (q_r . l_j + q~_r . k~_j),  o_r = sum_j softmax_j(s_r) l_j
//
// for the R = T H rows r of a sequence against its cached vectors c_j =
// [l_j, k~_j].  Every cached vector is read once and serves as key and as value:
// 2 (Dl + Ds) bytes and 2 R (2 Dl + Ds) flops a token, so HBM bounds it up to
// about R = 100 rows.
//
// The few rows are the N of the tensor-core products, the cache their M:
//   S^T [64 tokens x N]  = C [64 x D] Q^T            (C K-major, rows as they lie in a page)
//   O^T [Dl x N]        += L^T [Dl x 64] P^T          (the same tile, MN-major)
// so that 16 rows cost 16 columns and not a padded tile of 128.  Tiles are 64
// tokens: with the latents as 16 KiB pairs of chunks (64 tokens x 128 columns) the
// ring holds two to three tiles next to Q, and copies go on while one is worked on.
// More than 64 rows go to several CTAs, each of which reads the cache (the later
// ones from L2).
//
// Work is split evenly whatever the lengths: the tiles of all sequences, laid
// end to end, are cut into one contiguous range per CTA (persistent, one CTA per
// SM).  A sequence that lies in one range is finished there; the others leave
// partial results (normalised, with their log-sum-exp), which a second kernel
// joins in a fixed order.
//
//   warp 0      one thread issues the MMAs: whatever can go next, a slot's share of
//               the next tile's scores or this tile's values, so that the tensor
//               pipe works while softmax runs
//   warps 1..4  copies: 16 tokens of a tile each, 512 bytes of a row at a time
//               (cp.async; pages are multiples of 16 tokens, so a warp's tokens lie
//               on one page); the tile after that is asked into L2 meanwhile
//   warps 5..   softmax, four warps (16 rows) or eight (each four take half of the
//               rows): running maximum and sum per row (a column of S^T: over
//               lanes by shuffles, over warps through shared memory); P^T goes to
//               shared memory; O^T stays in TMEM and is rescaled only when a
//               maximum has grown by more than 2^8
//   last warp   Q of each sequence by TMA
//
// P is rounded to bf16 for its product (its scale is that of the running
// maximum, its relative error 2^-8 at most); sums and statistics are fp32.
//
// Measured (Dl + Ds = 512 + 64, 16 heads; this kernel, without the join):
//   256 sequences of up to 4096 tokens, 16 rows     106 to 109 us, 5.7 TB/s (87% of a copy's
//               rate); a call, which joins the parts too, 111 on the device
//   32 of up to 8192, 8 tokens: 128 rows, two CTAs   78 to 82 us; what bounds it is how long a
//               tile stays in the ring, which holds two beside 64 rows of Q: 3,300 cycles a
//               tile, of which the MMAs take 1,950
// Copies by TMA took one box per page and chunk, ~200 cycles each whatever its size:
// 110 us instead of 95 at that time for pages of 32.  Slots of one pair instead of two
// cost the issuing thread twice the waits (158 us instead of 115 for 256 sequences),
// slots of four leave no copy in flight; eight copying warps measured 134 us against
// 115 for four; 65 to 80 rows as one tile of 80 (less than two tiles fit beside it)
// 60 us against 52 as two of 40.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "rda_io.cuh"
#include "rda_latent.h"
#include "sm100_pipe.cuh"

namespace rda {
namespace {

using namespace ptx;

constexpr int kTok = 64;                 // tokens per tile
constexpr int kCtas = kSms;              // one CTA per SM
constexpr int kScan = 128;               // threads that sum up the lengths
constexpr uint32_t kPair = 16384;        // 64 tokens x 128 latent columns; a slot is one or two of them
constexpr uint32_t kBox = 8192;          // 64 tokens x 64 columns
constexpr int kMaxSlots = 12, kMaxShared = 2;
constexpr int kLens = 256;               // batches up to this keep their lengths in shared memory
constexpr int kInfo = 16;                // tiles whose masks are kept (the ring holds at most kMaxSlots)
constexpr float kGrow = 8.f;             // rescale O when a maximum has grown by more (log2)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Columns of S^T (rows of the result) that the first four softmax warps take; four more take the rest.
__host__ __device__ constexpr int split_cols(int nt) { return nt == 16 ? 16 : nt == 48 ? 32 : nt / 2; }
__host__ __device__ constexpr int softmax_warps(int nt) { return nt == 16 ? 4 : 8; }
// Warp 0 issues the MMAs, warps 1..4 copy the cache, then the softmax warps, the last one brings Q.
constexpr int kCopyWarps = 4, kSoftWarp = 1 + kCopyWarps;
__host__ __device__ constexpr int threads_of(int nt) { return 32 * (kSoftWarp + softmax_warps(nt) + 1); }

// Shared memory behind the operand areas.
template <int NT> struct Small {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t q_full, q_empty, s_full[2], p_ready, pv_done, o_empty, drained;
    alignas(8) uint16_t seen[kInfo][kCopyWarps];    // which of a tile's tokens are cached, 16 by each copying warp
    union {
        long long sums[kScan];           // before the roles part
        float wmax[4][NT];               // within a tile
        float lsum[4][NT];               // at a segment's end
    };
    float factor[NT];
    long long total, lo, hi;
    int first_b, first_off;
    int lens[kLens];
    uint32_t tmem;
    volatile int abort;
};

struct Geometry {
    int rt, rows, nt;                    // row tiles, rows of a tile, columns of its MMAs
    int groups;                          // CTAs along the tiles
    int slots, sp, shared;               // ring slots, pairs of a slot, slots of shared columns
    uint32_t smem;
};

struct Maps {
    CUtensorMap q, q_shared;
};

__host__ __device__ inline uint32_t operand_bytes(int nt, int D, int pairs, int shared) {
    return (uint32_t)(D / 64) * nt * 128 + nt * 128 + pairs * kPair + shared * kBox;
}

// Partial results: [group][row tile][first or last segment][column] -> Dl floats,
// then their log-sum-exps, then the sequences that are left in parts: a record per
// sequence where there are no more of them than groups, per group otherwise (a
// group leaves one at most).
struct Parts {
    float *o, *lse;
    int4 *rec;                           // {sequence or -1, last group, slot of the first part, first group}
};
__host__ __device__ inline size_t part_slots(const Geometry &g) { return (size_t)g.groups * g.rt * 2; }
__host__ __device__ inline Parts parts_of(float *base, const Geometry &g, int Dl) {
    Parts p;
    p.o = base;
    p.lse = base + part_slots(g) * g.nt * Dl;
    p.rec = reinterpret_cast<int4 *>(p.lse + part_slots(g) * g.nt);
    return p;
}

struct Args {
    LatentDecodeArgs a;
    Geometry g;
};

// Tokens of sequence b (cut to what its table can hold).
__device__ __forceinline__ int seq_len(const LatentDecodeArgs &a, int b) {
    return max(0, min(a.lens[b], a.table_width * a.page_size));
}
// Tiles of a sequence; an empty one has one (fully masked), so that its rows are written.
__device__ __forceinline__ int seq_tiles(int len) { return max(1, (len + kTok - 1) / kTok); }

// The segments (runs of tiles of one sequence) of a CTA's range; every role walks them by itself.
struct Walk {
    long long pos, hi;
    int b, off;                          // next sequence, tiles of it already behind
    int len, tiles, t0, t1;              // the current segment: tiles [t0, t1) of sequence `seq`
    int seq;
    const int *lens;                     // all of them in shared memory, or null
    __device__ __forceinline__ bool next(const LatentDecodeArgs &a) {
        if (pos >= hi) return false;
        seq = b;
        len = lens ? lens[b] : seq_len(a, b);
        tiles = seq_tiles(len);
        t0 = off;
        t1 = (int)min((long long)tiles, off + (hi - pos));
        pos += t1 - t0;
        off = 0;
        ++b;
        return true;
    }
};

// Rows 0 .. rows - 1 of O (columns of O^T in TMEM), times their factors: out[r][128 p + lane ..].
template <int NT, int NC, typename T, typename F>
__device__ __forceinline__ void store_result(uint32_t t_o, int NP, int rows, const float *factor, T *out, int stride, F conv) {
#pragma unroll 1
    for (int c = 0; c < NC; c += 16) {
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = factor[c + i];
#pragma unroll 1
        for (int p = 0; p < NP; ++p) {
            float x[16];
            tmem_ld16(t_o + p * NT + c, x);
            tmem_wait_ld();
            T *o = out + c * stride + 128 * p;
            if (c + 16 <= rows) {
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i * stride] = conv(x[i] * f[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < rows) o[i * stride] = conv(x[i] * f[i]);
            }
        }
    }
}


template <int NT> struct SoftmaxCtx {
    Small<NT> &S;
    const Args &args;
    Walk walk;
    Waiter w;
    uint8_t *p_s;
    uint32_t tmem;
    int rt, grp, rows, row0;
    long long hi, total;
};

// Four warps on the columns [c0, c0 + NC) of S^T and O^T, c0 = 0 or split_cols(NT) (half 0 or 1).
template <int NT, int NC>
__device__ __forceinline__ void softmax(const SoftmaxCtx<NT> &x_, int half) {
    Small<NT> &S = x_.S;
    const Args &args = x_.args;
    const LatentDecodeArgs &a = args.a;
    const Geometry &g = args.g;
    const Waiter w = x_.w;
    Walk walk = x_.walk;
    uint8_t *p_s = x_.p_s;
    const int NP = a.Dl / 128, NS = NP / g.sp, R = a.T * a.H;
    const int rt = x_.rt, grp = x_.grp, row0 = x_.row0, rows = x_.rows;
    const long long hi = x_.hi, total = x_.total;
    const int c0 = half ? split_cols(NT) : 0, bar = 1 + half;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t t_o = x_.tmem + c0, t_s = x_.tmem + 4 * NT + c0;
    const int quad = warp & 3;                       // tokens 16 quad .. + 15 of a tile
    const int tok = lane >> 2, col = 2 * (lane & 3); // my tokens: tok, tok + 8; my columns: 8 c + col, + 1
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const float sc = a.scale * kLog2e;
    constexpr int C = NC / 8;
    uint32_t it = 0;
    RingPos ring;                                    // a tile's first slot
    const Parts parts = parts_of(a.part, g, a.Dl);
    bool first_segment = true;
    while (walk.next(a)) {
        float m[C][2], l[C][2];
        int last[C][2];                              // last token that my columns see
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                m[c][u] = -INFINITY;
                l[c][u] = 0.f;
                const int r = c0 + 8 * c + col + u;
                last[c][u] = r < rows ? walk.len - a.T + (row0 + r) / a.H : -1;
            }
        const int all_see = rows > 0 ? walk.len - a.T + row0 / a.H : -1;     // what every row sees
        for (int t = walk.t0; t < walk.t1; ++t, ++it) {
            w.wait(&S.s_full[it & 1], (it >> 1) & 1);
            tc_fence_after();
            float v[C][4];
#pragma unroll
            for (int c = 0; c < C; c += 2) tmem_ld_16x256b_x2(t_s + (it & 1) * NT + 8 * c + lanes, &v[c][0]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int u = 0; u < 4; ++u) v[c][u] *= sc;       // log2 units; sc may be negative
            w.wait(&S.full[ring.slot], ring.phase);             // the masks, written beside the copies
            const uint2 seen = *reinterpret_cast<const uint2 *>(S.seen[it % kInfo]);
            ring.skip(NS, g.slots);
            const int j0 = t * kTok + 16 * quad + tok;
            const bool whole = (seen.x & seen.y) == 0xffffffffu && t * kTok + kTok - 1 <= all_see;
            if (!whole) {
                const uint32_t mine = (quad & 2 ? seen.y : seen.x) >> (16 * (quad & 1) + tok);
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        if (!(mine & 1) || j0 > last[c][u]) v[c][u] = -INFINITY;
                        if (!(mine >> 8 & 1) || j0 + 8 > last[c][u]) v[c][2 + u] = -INFINITY;
                    }
            }
            // The rows' maxima are only looked for when some score passes the one in use by more than 2^kGrow: P
            // stays in range, and a tile costs one barrier and no exchange.
            bool above = false;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int u = 0; u < 4; ++u) above |= v[c][u] - m[c][u & 1] > kGrow;
            float f[C][2];
#pragma unroll
            for (int c = 0; c < C; ++c) f[c][0] = f[c][1] = 1.f;
            const bool grown = named_bar_any(bar, 128, above);
            if (grown) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float x = fmaxf(v[c][u], v[c][2 + u]);
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        if (lane < 4) S.wmax[quad][c0 + 8 * c + col + u] = x;
                    }
                named_bar_sync(bar, 128);
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int r = c0 + 8 * c + col + u;
                        const float now = fmaxf(fmaxf(S.wmax[0][r], S.wmax[1][r]), fmaxf(S.wmax[2][r], S.wmax[3][r]));
                        if (now > m[c][u]) {
                            f[c][u] = ex2(m[c][u] - now);
                            m[c][u] = now;
                        }
                    }
            }
            const bool rescale = grown && t != walk.t0;
            // P^T, and my part of the sums
            uint32_t pk[C][2];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float p[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) p[u] = m[c][u & 1] == -INFINITY ? 0.f : ex2(v[c][u] - m[c][u & 1]);
                l[c][0] = fmaf(l[c][0], f[c][0], p[0] + p[2]);
                l[c][1] = fmaf(l[c][1], f[c][1], p[1] + p[3]);
                pk[c][0] = pack2(p[0], p[1]);
                pk[c][1] = pack2(p[2], p[3]);
            }
            if (it > 0) w.wait(&S.pv_done, (it - 1) & 1);       // P and O^T are free
            tc_fence_after();
            if (rescale) {
                if (quad == 0 && lane < 4)
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        S.factor[c0 + 8 * c + col] = f[c][0];
                        S.factor[c0 + 8 * c + col + 1] = f[c][1];
                    }
                named_bar_sync(bar, 128);
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int c = 0; c < NC; c += 16) {
                        float x[16];
                        tmem_ld16(t_o + p * NT + c + lanes, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] *= S.factor[c0 + c + i];
                        tmem_st16f(t_o + p * NT + c + lanes, x);
                    }
                tmem_wait_st();
                named_bar_sync(bar, 128);                          // factors read by all
            }
#pragma unroll
            for (int c = 0; c < C; c += 2) {
                // matrices: (block c, tokens 0-7), (c, 8-15), (c + 1, 0-7), (c + 1, 8-15) of my warp's 16
                const int r = c0 + 8 * (c + (lane >> 4)) + (lane & 7), ch = 2 * quad + ((lane >> 3) & 1);
                stsm_x4_t(smem_u32(p_s) + sw128(r, ch), pk[c][0], pk[c][1], pk[c + 1][0], pk[c + 1][1]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(&S.p_ready);
        }
        // the segment's result: whole, or one part of a sequence
        const bool done = walk.t0 == 0 && walk.t1 == walk.tiles;
        named_bar_sync(bar, 128);                    // the last maxima are read, lsum takes their place
        const size_t slot = ((size_t)grp * g.rt + rt) * 2 + (first_segment ? 0 : 1);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float x = l[c][u];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (lane < 4) S.lsum[quad][c0 + 8 * c + col + u] = x;
            }
        named_bar_sync(bar, 128);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = c0 + 8 * c + col + u;
                const float x = (S.lsum[0][r] + S.lsum[1][r]) + (S.lsum[2][r] + S.lsum[3][r]);
                if (quad == 0 && lane < 4) {
                    S.factor[r] = x > 0.f ? 1.f / x : 0.f;
                    const float lse = x > 0.f ? (m[c][u] + lg2(x)) * kLn2 : -INFINITY;
                    if (r < rows) {
                        if (!done) parts.lse[slot * NT + r] = lse;
                        else if (a.lse) a.lse[(size_t)walk.seq * R + row0 + r] = lse;
                    }
                }
            }
        w.wait(&S.pv_done, (it - 1) & 1);
        tc_fence_after();
        named_bar_sync(bar, 128);
        if (done) {
            auto *o = static_cast<__nv_bfloat16 *>(a.out) + ((size_t)walk.seq * R + row0 + c0) * a.Dl + 32 * quad + lane;
            store_result<NT, NC>(t_o + lanes, NP, rows - c0, S.factor + c0, o, a.Dl,
                             [](float x) { return __float2bfloat16_rn(x); });
        } else {
            store_result<NT, NC>(t_o + lanes, NP, rows - c0, S.factor + c0, parts.o + (slot * NT + c0) * a.Dl + 32 * quad + lane, a.Dl,
                             [](float x) { return x; });
        }
        tc_fence_before();
        mbar_arrive(&S.o_empty);
        named_bar_sync(bar, 128);                                  // factors are free again
        const bool by_seq = a.B <= g.groups;
        if (rt == 0 && threadIdx.x == 32 * kSoftWarp && (by_seq ? walk.t0 == 0 : walk.pos >= hi)) {
            // does a sequence begin here and go on in other groups?
            int4 rec = make_int4(-1, 0, 0, 0);
            if (!done && walk.t0 == 0) {
                const long long groups = min((long long)g.groups, total);
                const long long end = hi - walk.t1 + walk.tiles - 1;      // the sequence's last tile
                long long gl = min(groups - 1, end * groups / total);     // the group that holds it
                while (gl + 1 < groups && total * (gl + 1) / groups <= end) ++gl;
                while (total * gl / groups > end) --gl;
                rec = make_int4(walk.seq, (int)gl, first_segment ? 0 : 1, grp);
            }
            parts.rec[by_seq ? walk.seq : grp] = rec;
        }
        first_segment = false;
    }
}

template <int NT>
__global__ void __launch_bounds__(threads_of(NT), 1) latent_decode_kernel(const __grid_constant__ Maps maps, const Args args) {
    extern __shared__ __align__(1024) uint8_t sm[];      // no room to spare for aligning it here
    const LatentDecodeArgs &a = args.a;
    const Geometry &g = args.g;
    const int NP = a.Dl / 128, NB = (a.Dl + a.Ds) / 64, NS = NP / g.sp;    // pairs, boxes, slots of a tile
    uint8_t *q_s = sm, *p_s = q_s + NB * NT * 128, *pair_s = p_s + NT * 128, *shared_s = pair_s + g.slots * g.sp * kPair;
    Small<NT> &S = *reinterpret_cast<Small<NT> *>(shared_s + (a.Ds ? g.shared * kBox : 0));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rt = blockIdx.x % g.rt, grp = blockIdx.x / g.rt;
    const int R = a.T * a.H, row0 = rt * g.rows, rows = min(g.rows, R - row0);
    const Waiter w{&S.abort, a.err, a.wait_ns};
    pdl_launch_dependents();
    if (smem_u32(sm) & 1023) {                           // the swizzled operands need it
        pdl_wait_primary();
        if (tid == 0) atomicCAS(a.err, 0, (int32_t)RDA_ERR_CUDA);
        return;
    }
    constexpr uint32_t kCols = NT <= 16 ? 128 : NT <= 32 ? 256 : 512;      // 4 NT for O^T, 2 NT for S^T

    // Ahead of the wait below: TMEM cannot run short between this kernel and one before it that still has to allocate
    // its own, as their CTAs (74 KB of shared memory at least) do not fit on an SM beside one of this kernel's (200 KB).
    if (warp == 0) {
        tmem_alloc(&S.tmem, kCols);
        tmem_relinquish();
    }
    if (tid == 32) {
        for (int i = 0; i < g.slots; ++i) mbar_init(&S.full[i], 33 * kCopyWarps), mbar_init(&S.empty[i], 1);
        mbar_init(&S.q_full, 1);
        mbar_init(&S.q_empty, 1);
        mbar_init(&S.s_full[0], 1);
        mbar_init(&S.s_full[1], 1);
        mbar_init(&S.p_ready, 32 * softmax_warps(NT));
        mbar_init(&S.pv_done, 1);
        mbar_init(&S.drained, 1);
        mbar_init(&S.o_empty, 32 * softmax_warps(NT));
        S.abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&maps.q);
    }
    pdl_wait_primary();                                  // nothing above reads what another kernel may still write
    // this group's range of the tiles of all sequences
    const int per = (a.B + kScan - 1) / kScan, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    {
        long long x = 0;
        for (int b = b0; b < b1; ++b) {
            const int given = a.lens[b], len = max(0, min(given, a.table_width * a.page_size));
            if (given != len && blockIdx.x == 0) atomicCAS(a.err, 0, (int32_t)RDA_ERR_INVALID_ARG);
            if (a.B <= kLens) S.lens[b] = len;
            x += seq_tiles(len);
        }
        if (tid < kScan) S.sums[tid] = x;
    }
    __syncthreads();
    if (warp == 0) {
        long long part[kScan / 32], x = 0;
#pragma unroll
        for (int i = 0; i < kScan / 32; ++i) part[i] = S.sums[lane * (kScan / 32) + i], x += part[i];
        long long incl = x;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        long long before = incl - x;
#pragma unroll
        for (int i = 0; i < kScan / 32; ++i) {
            S.sums[lane * (kScan / 32) + i] = before;
            before += part[i];
        }
        if (lane == 31) {
            const long long groups = min((long long)g.groups, incl);
            S.total = incl;
            S.lo = grp < groups ? incl * grp / groups : 0;
            S.hi = grp < groups ? incl * (grp + 1) / groups : 0;
        }
    }
    __syncthreads();
    const long long lo = S.lo, hi = S.hi, total = S.total;
    if (lo < hi && tid < kScan && lo >= S.sums[tid]) {
        // the thread whose sequences hold tile lo looks for it
        long long at = S.sums[tid];
        for (int b = b0; b < b1; ++b) {
            const int n = seq_tiles(a.B <= kLens ? S.lens[b] : seq_len(a, b));
            if (lo < at + n) {
                S.first_b = b;
                S.first_off = (int)(lo - at);
                break;
            }
            at += n;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    const uint32_t t_o = tmem, t_s = tmem + 4 * NT;
    Walk walk{lo, hi, lo < hi ? S.first_b : 0, lo < hi ? S.first_off : 0, 0, 0, 0, 0, 0,
              a.B <= kLens ? S.lens : nullptr};

    if (warp == 0) {
        // ------------------------------------------------------------ MMAs
        if (elect_one()) {
            // One loop that issues whatever can go next: a slot's share of the scores once its copy has landed, a
            // tile's values once softmax has left P.  Each is written out once and in short loops: the code of all
            // roles has to stay in the instruction caches for the MMAs to be issued as fast as they run.
            constexpr uint32_t idS = idesc_bf16(kTok, NT, 0, 0), idO = idesc_bf16(128, NT, 1, 0);
            // descriptors count in units of 16 bytes: offsets are added to the first slot's
            const uint32_t dq = (uint32_t)smem_desc(smem_u32(q_s), 16, 1024, kSw128), dp = (uint32_t)smem_desc(smem_u32(p_s), 16, 1024, kSw128);
            const uint32_t dc = (uint32_t)smem_desc(smem_u32(pair_s), 16, 1024, kSw128);
            const uint32_t dv = (uint32_t)smem_desc(smem_u32(pair_s), kBox, 1024, kSw128);
            const uint32_t ds = (uint32_t)smem_desc(smem_u32(shared_s), 16, 1024, kSw128);
            const uint32_t high = (uint32_t)(smem_desc(0, 0, 1024, kSw128) >> 32);
            constexpr uint32_t kQBox = NT * 8, kPairD = kPair / 16, kBoxD = kBox / 16;
            const uint32_t slot_d = g.sp * kPairD;
            RingPos qk_p, pv_p;
            int qk_shared = 0, part = 0;                 // slot of the shared columns; slots of the tile already issued
            Walk ahead = walk;                           // the scores run up to one tile ahead of the values
            bool more = ahead.next(a), left = walk.next(a);
            int at = ahead.t0, t = walk.t0;
            uint32_t qk_it = 0, qk_seg = 0, it = 0, seg = 0;
            uint64_t since = 0;
            uint32_t idle = 0;
            while (left) {
                if (qk_it > it && mbar_test(&S.p_ready, it & 1) && (t != walk.t0 || seg == 0 || mbar_test(&S.o_empty, (seg - 1) & 1))) {
                    // O^T += L^T P^T of tile t
                    tc_fence_after();
                    for (int n = 0; n < NS; ++n) {
                        for (int p = 0; p < g.sp; ++p) {
                            const uint32_t da = dv + (pv_p.slot * slot_d + p * kPairD);
                            const uint32_t d = t_o + (n * g.sp + p) * NT;
#pragma unroll
                            for (int k = 0; k < 4; ++k) mma_bf16_low(d, da + k * 128, dp + k * 2, high, idO, t != walk.t0 || k > 0);
                        }
                        mma_commit(&S.empty[pv_p.slot]);
                        pv_p.next(g.slots);
                    }
                    mma_commit(&S.pv_done);
                    ++it;
                    if (++t == walk.t1) {
                        ++seg;
                        left = walk.next(a);
                        t = walk.t0;
                    }
                    idle = 0;
                } else if (more && qk_it < it + 2 && mbar_test(&S.full[qk_p.slot], qk_p.phase) &&
                           (part > 0 || at != ahead.t0 || mbar_test(&S.q_full, qk_seg & 1))) {
                    // S^T of tile `at` of the segment `ahead`: the columns of one slot
                    fence_proxy_async_smem();            // the copies wrote through the generic proxy
                    tc_fence_after();
                    const uint32_t d = t_s + (qk_it & 1) * NT;
                    const uint32_t da = dc + qk_p.slot * slot_d, db = dq + part * 2 * g.sp * kQBox;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c >= 2 * g.sp) break;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16_low(d, da + (c * kBoxD + k * 2), db + (c * kQBox + k * 2), high, idS, part > 0 || c > 0 || k > 0);
                    }
                    qk_p.next(g.slots);
                    if (++part == NS) {
                        if (a.Ds) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_bf16_low(d, ds + (qk_shared * kBoxD + k * 2), dq + (2 * NP * kQBox + k * 2), high, idS, 1);
                            if (++qk_shared == g.shared) qk_shared = 0;
                        }
                        mma_commit(&S.s_full[qk_it & 1]);
                        part = 0;
                        ++qk_it;
                        if (++at == ahead.t1) {
                            mma_commit(&S.q_empty);
                            ++qk_seg;
                            more = ahead.next(a);
                            at = ahead.t0;
                        }
                    }
                    idle = 0;
                } else if ((++idle & 255) == 0) {
                    // nothing for a while: give up when another role has, or after the limit
                    if (S.abort) break;
                    if (idle == 256) since = Waiter::now();
                    else if (Waiter::now() - since > a.wait_ns) {
                        S.abort = 1;
                        atomicCAS(a.err, 0, (int32_t)RDA_ERR_TIMEOUT);
                    }
                }
            }
            if (S.abort) {
                // what was issued completes before the CTA leaves
                mma_commit(&S.drained);
                w.drain(&S.drained, 0, Waiter::now());
            }
        }
        __syncwarp();
    } else if (warp < kSoftWarp) {
        // ------------------------------------------------------------ copies: 16 tokens of a tile each
        // (pages are multiples of 16 tokens: a warp's tokens of a tile lie on one page)
        const int mine = warp - 1;
        RingPos pr;
        int sr = 0;
        uint32_t it = 0;
        bool go = true;
        auto page_of = [&](const Walk &x, int t) {
            const int j = t * kTok + 16 * mine;
            return j < x.len ? a.table[(size_t)x.seq * a.table_width + j / a.page_size] : -1;
        };
        bool more = walk.next(a);
        int page_next = more ? page_of(walk, walk.t0) : -1;
        const __nv_bfloat16 *pages = static_cast<const __nv_bfloat16 *>(a.pages);
        const int D = a.Dl + a.Ds;
        while (more) {
            Walk after = walk;
            const bool another = after.next(a);
            for (int t = walk.t0; t < walk.t1; ++t, ++it) {
                if (it == (uint32_t)a.debug_drop) {
                    more = false;
                    break;
                }
                const int j = t * kTok + 16 * mine, page = page_next;
                const bool ok = page >= 0 && page < a.num_pages;
                if (t + 1 < walk.t1) page_next = page_of(walk, t + 1);
                else if (another) page_next = page_of(after, after.t0);
                // tokens behind the end, or on a page outside the cache: zeros, whatever the cache holds there
                const int have = ok ? min(16, walk.len - j) : 0;
                if (lane == 0) {
                    if (!ok && j < walk.len) atomicCAS(a.err, 0, (int32_t)RDA_ERR_INVALID_ARG);
                    S.seen[it % kInfo][mine] = (uint16_t)((1u << max(have, 0)) - 1);
                }
                const __nv_bfloat16 *src = ok ? pages + ((size_t)page * a.page_size + j % a.page_size) * D : static_cast<const __nv_bfloat16 *>(a.q);
                for (int n = 0; n < NS; ++n) {
                    // The shared columns come with the tile's last slot; theirs is free once the scores that read it
                    // last are done.
                    const bool with = n == NS - 1 && a.Ds;
                    if (with && it >= (uint32_t)g.shared)
                        go = w.wait(&S.s_full[(it - g.shared) & 1], ((it - g.shared) >> 1) & 1) && go;
                    if (it * NS + n >= (uint32_t)g.slots) go = w.wait(&S.empty[pr.slot], pr.phase ^ 1) && go;
                    const uint32_t dst = smem_u32(pair_s) + pr.slot * g.sp * kPair;
                    if (g.sp == 2) {
                        // 512 bytes of a row at a time
                        const __nv_bfloat16 *x = src + n * 256 + lane * 8;
                        const uint32_t to = dst + (lane >> 3) * kBox + 16 * mine * 128;
                        if (have == 16) {
#pragma unroll 8
                            for (int r = 0; r < 16; ++r, x += D) cp_async16_row(to + sw128(r, lane & 7), x);
                        } else {
#pragma unroll 4
                            for (int r = 0; r < 16; ++r, x += r < have ? D : 0)
                                cp_async16_or_zero(to + sw128(r, lane & 7), x, r < have ? 16 : 0);
                        }
                    } else {
                        const int half = lane >> 4, y = lane & 15;
                        const __nv_bfloat16 *x = src + half * D + n * 128 + y * 8;
                        const uint32_t to = dst + (y >> 3) * kBox + 16 * mine * 128;
                        if (have == 16) {
#pragma unroll
                            for (int r = 0; r < 16; r += 2, x += 2 * D) cp_async16_row(to + sw128(r + half, y & 7), x);
                        } else {
                            for (int r = half; r < 16; r += 2)
                                cp_async16_or_zero(to + sw128(r, y & 7), src + (size_t)min(r, max(have - 1, 0)) * D + n * 128 + y * 8,
                                                   r < have ? 16 : 0);
                        }
                    }
                    if (with) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = 4 * i + (lane >> 3);
                            cp_async16_or_zero(smem_u32(shared_s) + sr * kBox + sw128(16 * mine + r, lane & 7),
                                               src + (size_t)min(r, max(have - 1, 0)) * D + a.Dl + (lane & 7) * 8, r < have ? 16 : 0);
                        }
                        if (++sr == g.shared) sr = 0;
                    }
                    cp_async_arrive(smem_u32(&S.full[pr.slot]));
                    // that arrival stands for copies alone: what lane 0 has written to `seen` is published by one of its own
                    if (lane == 0) mbar_arrive(&S.full[pr.slot]);
                    pr.next(g.slots);
                }
                // the next tile's tokens come as far as L2 while this warp waits for room
                const Walk &then = t + 1 < walk.t1 ? walk : after;
                const int j1 = (t + 1 < walk.t1 ? t + 1 : after.t0) * kTok + 16 * mine, have1 = min(16, then.len - j1);
                if ((t + 1 < walk.t1 || another) && lane == 0 && have1 > 0 && page_next >= 0 && page_next < a.num_pages)
                    prefetch_l2(pages + ((size_t)page_next * a.page_size + j1 % a.page_size) * D, have1 * D * 2);
            }
            walk = after;
            more = more && another;
        }
        cp_async_wait_all();                                // nothing lands after the CTA has left
    } else if (warp == kSoftWarp + softmax_warps(NT)) {
        // ------------------------------------------------------------ Q of each segment, once the one before is used up
        if (elect_one()) {
            uint32_t seg = 0;
            while (walk.next(a)) {
                if (seg > 0 && !w.wait(&S.q_empty, (seg - 1) & 1)) break;
                mbar_arrive_expect_tx(&S.q_full, NB * NT * 128);
                const int r = walk.seq * R + row0;
                for (int c = 0; c < a.Dl / 64; ++c) tma_load_3d(q_s + c * NT * 128, &maps.q, &S.q_full, c * 64, r, 0);
                if (a.Ds) tma_load_3d(q_s + (NB - 1) * NT * 128, &maps.q_shared, &S.q_full, 0, r, 0);
                ++seg;
            }
            if (S.abort && seg > 0) w.drain(&S.q_full, (seg - 1) & 1, Waiter::now());
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const SoftmaxCtx<NT> x{S, args, walk, w, p_s, tmem, rt, grp, rows, row0, hi, total};
        if (warp < kSoftWarp + 4) softmax<NT, split_cols(NT)>(x, 0);
        else if constexpr (NT > 16) softmax<NT, NT - split_cols(NT)>(x, 1);
        if (rt == 0 && tid == 32 * kSoftWarp && lo >= hi && a.B > g.groups) parts_of(a.part, g, a.Dl).rec[grp] = make_int4(-1, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// Joins the parts of the sequence of record blockIdx.x: out = sum_i e^{lse_i - lse} o_i.
// MANY: a CTA per row and 128 columns, each of its 16 warps takes every 16th part;
// otherwise four rows a CTA, 128 threads each.  The parts come from L2; what counts
// is how few loads wait for one another: the record, then log-sum-exps and the
// first parts at once.  4 us for one sequence of 16 rows, 8 for 256, 13 for 32 of 128
// rows (28 MB of parts); rows walked over in one wave of CTAs were no faster.
constexpr int kJoin = 512, kMostParts = 160;
static_assert(kMostParts >= kCtas && kMostParts % 32 == 0, "parts of a sequence");
template <bool MANY> __global__ void __launch_bounds__(kJoin) latent_join_bf16_kernel(const Args args) {
    constexpr int SHARES = MANY ? kJoin / 32 : 1;
    __shared__ float4 acc_s[SHARES][32];
    __shared__ float w_s[kJoin / 32][kMostParts];
    const LatentDecodeArgs &a = args.a;
    const Geometry &g = args.g;
    const Parts parts = parts_of(a.part, g, a.Dl);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int share = MANY ? warp : 0, c = MANY ? blockIdx.z * 128 + lane * 4 : (tid & 127) * 4;
    const int at = MANY ? blockIdx.y : blockIdx.y * 4 + (tid >> 7);       // row, by tile
    const int rt = at / g.rows, r = at % g.rows, R = a.T * a.H;
    const bool on = at < g.rt * g.rows && rt * g.rows + r < R;
    pdl_launch_dependents();
    pdl_wait_primary();
    const int4 rec = parts.rec[blockIdx.x];
    if (rec.x < 0 || !on) return;
    if (rec.x >= a.B || rec.w < 0 || rec.y < rec.w || rec.y >= g.groups) return;      // never written
    const int n = rec.y - rec.w + 1;
    auto slot = [&](int i) { return (((size_t)(rec.w + i) * g.rt + rt) * 2 + (i == 0 ? rec.z : 0)) * g.nt + r; };
    auto part = [&](int i) {
        return i < n && c < a.Dl ? *reinterpret_cast<const float4 *>(parts.o + slot(i) * a.Dl + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) y[u] = part(share + u * SHARES);
    float l[kMostParts / 32], top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kMostParts / 32; ++j) {
        l[j] = 32 * j + lane < n ? parts.lse[slot(32 * j + lane)] : -INFINITY;
        top = fmaxf(top, l[j]);
    }
    // every warp computes the common maximum and sum
#pragma unroll
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < kMostParts / 32; ++j) {
        l[j] = expf(l[j] - base);
        sum += l[j];
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const float f = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int j = 0; j < kMostParts / 32; ++j) w_s[warp][32 * j + lane] = l[j] * f;
    __syncwarp();
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = share; i < n; i += 4 * SHARES) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = i + u * SHARES;
            const float w = k < n ? w_s[warp][k] : 0.f;
            x.x = fmaf(w, y[u].x, x.x), x.y = fmaf(w, y[u].y, x.y), x.z = fmaf(w, y[u].z, x.z), x.w = fmaf(w, y[u].w, x.w);
            y[u] = part(k + 4 * SHARES);
        }
    }
    if (MANY) {
        acc_s[share][lane] = x;
        __syncthreads();
        if (share) return;
#pragma unroll
        for (int i = 1; i < SHARES; ++i) {
            const float4 z = acc_s[i][lane];
            x.x += z.x, x.y += z.y, x.z += z.z, x.w += z.w;
        }
    }
    const size_t row = (size_t)rec.x * R + rt * g.rows + r;
    if (c < a.Dl)
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + row * a.Dl + c) =
            make_uint2(pack2(x.x, x.y), pack2(x.z, x.w));
    if (c == 0 && a.lse) a.lse[row] = sum > 0.f ? base + logf(sum) : -INFINITY;
}

template <int NT> uint32_t small_bytes() { return (uint32_t)sizeof(Small<NT>); }

Geometry geometry(int T, int H, int Dl, int Ds) {
    Geometry g{};
    const int R = T * H;
    g.rt = (R + 63) / 64;
    g.rows = (R + g.rt - 1) / g.rt;
    g.nt = (g.rows + 15) / 16 * 16;
    g.groups = std::max(1, kCtas / g.rt);
    const uint32_t small = g.nt == 16 ? small_bytes<16>() : g.nt == 32 ? small_bytes<32>() : g.nt == 48 ? small_bytes<48>() : small_bytes<64>();
    const uint32_t most = 232448 - small;
    const int D = Dl + Ds, NP = Dl / 128;
    // slots of two pairs where the latents have an even number: half the waits for the issuing thread
    g.sp = NP % 2 == 0 ? 2 : 1;
    // the scores run a tile ahead of the values: two tiles of latents at least; one slot for the
    // shared columns if two do not fit beside them
    g.shared = Ds ? 2 : 1;
    if (Ds && operand_bytes(g.nt, D, 2 * NP, 2) > most) g.shared = 1;
    const uint32_t beside = operand_bytes(g.nt, D, 0, Ds ? g.shared : 0);
    g.slots = std::min<int>(kMaxSlots, (int)((most - beside) / (g.sp * kPair)));
    g.smem = beside + g.slots * g.sp * kPair + small;
    return g;
}
static_assert(sizeof(Small<64>) % 8 == 0, "barriers are 8-byte aligned");

template <int NT> cudaError_t launch(const Maps &maps, const Args &args, cudaStream_t s) {
    cudaError_t e = allow_smem<latent_decode_kernel<NT>>(232448);
    if (e != cudaSuccess) return e;
    return launch_after(latent_decode_kernel<NT>, args.g.rt * args.g.groups, threads_of(NT), args.g.smem, s, maps, args);
}

}  // namespace

size_t latent_decode_tc_scratch_bytes(int T, int H, int Dl, int Ds) {
    const Geometry g = geometry(T, H, Dl, Ds);
    return part_slots(g) * g.nt * (size_t)(Dl + 1) * sizeof(float) + (size_t)g.groups * sizeof(int4);
}

cudaError_t launch_latent_decode_tc(const LatentDecodeArgs &a, cudaStream_t s) {
    Args args{};
    args.a = a;
    args.g = geometry(a.T, a.H, a.Dl, a.Ds);
    const int R = a.T * a.H;
    if (args.g.slots * args.g.sp < 2 * (a.Dl / 128)) return cudaErrorInvalidConfiguration;
    Maps maps;
    std::memset(&maps, 0, sizeof(maps));
    if (!make_map_3d(&maps.q, a.q, a.Dl, (uint64_t)a.B * R, 1, a.Dl, (uint64_t)a.B * R * a.Dl, args.g.nt, 1) ||
        (a.Ds && !make_map_3d(&maps.q_shared, a.q_shared, a.Ds, (uint64_t)a.B * R, 1, a.Ds, (uint64_t)a.B * R * a.Ds,
                              args.g.nt, 1)))
        return cudaErrorInvalidValue;
    cudaError_t e;
    switch (args.g.nt) {
        case 16: e = launch<16>(maps, args, s); break;
        case 32: e = launch<32>(maps, args, s); break;
        case 48: e = launch<48>(maps, args, s); break;
        default: e = launch<64>(maps, args, s); break;
    }
    if (e != cudaSuccess || args.g.groups == 1) return e;
    // Parts per sequence: about groups / B.  From 16 on 16 warps share a row: 64 parts of 16 rows take 3.8 us so,
    // 13.3 with four warps a row.
    const bool many = args.g.groups >= 16 * a.B;
    const int at = args.g.rt * args.g.rows, records = std::min(a.B, args.g.groups);
    return many ? launch_after(latent_join_bf16_kernel<true>, dim3(records, at, a.Dl / 128), kJoin, 0, s, args)
                : launch_after(latent_join_bf16_kernel<false>, dim3(records, (at + 3) / 4), kJoin, 0, s, args);
}

}  // namespace rda
