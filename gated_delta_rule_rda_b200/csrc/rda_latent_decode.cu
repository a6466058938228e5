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
//   S^T [64 tokens x N]  = C [64 x D] Q^T            (C K-major, as TMA brings it)
//   O^T [Dl x N]        += L^T [Dl x 64] P^T          (the same tile, MN-major)
// so that 16 rows cost 16 columns and not a padded tile of 128.  Tiles are 64
// tokens: with the latents as 16 KiB slots (64 tokens x 128 columns) the ring
// holds two to three tiles next to Q, and loads go on while one is worked on.
//
// Work is split evenly whatever the lengths: the tiles of all sequences, laid
// end to end, are cut into one contiguous range per CTA (persistent, one CTA per
// SM).  A sequence that lies in one range is finished there; the others leave
// partial results (normalised, with their log-sum-exp), which a second kernel
// joins in a fixed order.
//
//   warp 0      producer: pages by TMA (one box per 16..64 rows of a page), Q
//   warp 1      one thread issues the MMAs: the next tile's scores before this
//               tile's values, so that the tensor pipe works while softmax runs
//   warps 2..5  softmax: running maximum and sum per row (a column of S^T: over
//               lanes by shuffles, over warps through shared memory); P^T goes to
//               shared memory; O^T stays in TMEM and is rescaled only when a
//               maximum has grown by more than 2^8
//
// P is rounded to bf16 for its product (its scale is that of the running
// maximum, its relative error 2^-8 at most); sums and statistics are fp32.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "rda_latent.h"
#include "sm100_pipe.cuh"

namespace rda {
namespace {

using namespace ptx;

constexpr int kTok = 64;                 // tokens per tile
constexpr int kCtas = 148;               // one CTA per SM
constexpr int kThreads = 192;
constexpr uint32_t kPair = 16384;        // slot: 64 tokens x 128 latent columns
constexpr uint32_t kBox = 8192;          // 64 tokens x 64 columns
constexpr int kMaxPairs = 12, kMaxShared = 2;
constexpr int kInfo = 16;                // tiles whose masks are kept (the ring holds at most kMaxPairs)
constexpr float kGrow = 8.f;             // rescale O when a maximum has grown by more (log2)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Shared memory behind the operand areas.
template <int NT> struct Small {
    uint64_t full[kMaxPairs], empty[kMaxPairs], sfull[kMaxShared], sempty[kMaxShared];
    uint64_t q_full, q_empty, s_full[2], p_ready, pv_done, o_empty;
    uint64_t info[kInfo];
    float wmax[2][4][NT];
    float lsum[4][NT];
    float factor[NT];
    long long sums[kThreads];
    long long total, lo, hi;
    int first_b, first_off;
    uint32_t tmem;
    volatile int abort;
};

struct Geometry {
    int rt, rows, nt;                    // row tiles, rows of a tile, columns of its MMAs
    int groups;                          // CTAs along the tiles
    int pairs, shared;                   // ring slots
    uint32_t smem;
};

struct Maps {
    CUtensorMap pages, q, q_shared;
};

__host__ __device__ inline uint32_t operand_bytes(int nt, int D, int pairs, int shared) {
    return (uint32_t)(D / 64) * nt * 128 + nt * 128 + pairs * kPair + shared * kBox;
}

// Partial results: [group][row tile][first or last segment][column] -> Dl floats,
// then their log-sum-exps, then what each group leaves unfinished.
struct Parts {
    float *o, *lse;
    int4 *rec;                           // {sequence or -1, last group, slot of the first part, -}
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
    int box_rows;
    int pages_bound;                     // first page coordinate outside the map
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
    __device__ __forceinline__ bool next(const LatentDecodeArgs &a) {
        if (pos >= hi) return false;
        seq = b;
        len = seq_len(a, b);
        tiles = seq_tiles(len);
        t0 = off;
        t1 = (int)min((long long)tiles, off + (hi - pos));
        pos += t1 - t0;
        off = 0;
        ++b;
        return true;
    }
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) latent_decode_kernel(const __grid_constant__ Maps maps, const Args args) {
    extern __shared__ uint8_t smem_raw[];
    const LatentDecodeArgs &a = args.a;
    const Geometry &g = args.g;
    uint8_t *sm = align_1024(smem_raw);
    const int NP = a.Dl / 128, NB = (a.Dl + a.Ds) / 64;
    uint8_t *q_s = sm, *p_s = q_s + NB * NT * 128, *pair_s = p_s + NT * 128, *shared_s = pair_s + g.pairs * kPair;
    Small<NT> &S = *reinterpret_cast<Small<NT> *>(shared_s + g.shared * kBox);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rt = blockIdx.x % g.rt, grp = blockIdx.x / g.rt;
    const int R = a.T * a.H, row0 = rt * g.rows, rows = min(g.rows, R - row0);
    const Waiter w{&S.abort, a.err, a.wait_ns};
    pdl_launch_dependents();
    constexpr uint32_t kCols = NT <= 16 ? 128 : NT <= 32 ? 256 : 512;      // 4 NT for O^T, 2 NT for S^T

    if (warp == 0) {
        tmem_alloc(&S.tmem, kCols);
        tmem_relinquish();
    }
    if (tid == 32) {
        for (int i = 0; i < g.pairs; ++i) mbar_init(&S.full[i], 1), mbar_init(&S.empty[i], 1);
        for (int i = 0; i < g.shared; ++i) mbar_init(&S.sfull[i], 1), mbar_init(&S.sempty[i], 1);
        mbar_init(&S.q_full, 1);
        mbar_init(&S.q_empty, 1);
        mbar_init(&S.s_full[0], 1);
        mbar_init(&S.s_full[1], 1);
        mbar_init(&S.p_ready, 128);
        mbar_init(&S.pv_done, 1);
        mbar_init(&S.o_empty, 128);
        S.abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&maps.pages);
        prefetch_tensormap(&maps.q);
    }
    // this group's range of the tiles of all sequences
    const int per = (a.B + kThreads - 1) / kThreads, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    {
        long long x = 0;
        for (int b = b0; b < b1; ++b) x += seq_tiles(seq_len(a, b));
        S.sums[tid] = x;
    }
    __syncthreads();
    if (warp == 0) {
        long long part[kThreads / 32], x = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) part[i] = S.sums[lane * (kThreads / 32) + i], x += part[i];
        long long incl = x;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        long long before = incl - x;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            S.sums[lane * (kThreads / 32) + i] = before;
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
    if (lo < hi && lo >= S.sums[tid]) {
        // the thread whose sequences hold tile lo looks for it
        long long at = S.sums[tid];
        for (int b = b0; b < b1; ++b) {
            const int n = seq_tiles(seq_len(a, b));
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
    Walk walk{lo, hi, lo < hi ? S.first_b : 0, lo < hi ? S.first_off : 0, 0, 0, 0, 0, 0};

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        RingPos pr, sr;
        uint32_t seg = 0, it = 0;
        const int ng = kTok / args.box_rows;           // row boxes of a tile
        const int mine = lane % ng;
        const long long most = (long long)a.table_width * a.page_size;
        while (walk.next(a)) {
            if (rt == 0 && walk.t0 == 0 && lane == 0) {
                const int given = a.lens[walk.seq];
                if (given < 0 || given > most) atomicCAS(a.err, 0, (int32_t)RDA_ERR_INVALID_ARG);
            }
            const int32_t *table = a.table + (size_t)walk.seq * a.table_width;
            // my row box of tile t: its page, or one outside the map (zeros)
            auto page_of = [&](int t) {
                const int j = t * kTok + mine * args.box_rows;
                return t < walk.t1 && j < walk.len ? table[j / a.page_size] : -1;
            };
            int page = page_of(walk.t0);
            // lane 0 waits for room and announces the bytes; false once the CTA has given up
            auto room = [&](uint64_t *empty, uint32_t parity, bool used, uint64_t *full, uint32_t bytes) {
                bool go = true;
                if (lane == 0) {
                    go = (!used || w.wait(empty, parity)) && !S.abort;
                    if (go) mbar_arrive_expect_tx(full, bytes);
                }
                return __shfl_sync(0xffffffffu, go, 0) != 0;
            };
            if (room(&S.q_empty, (seg - 1) & 1, seg > 0, &S.q_full, NB * NT * 128)) {
                if (lane < NB) {
                    const int c = lane * 64, r = walk.seq * R + row0;
                    if (c < a.Dl) tma_load_3d(q_s + lane * NT * 128, &maps.q, &S.q_full, c, r, 0);
                    else tma_load_3d(q_s + lane * NT * 128, &maps.q_shared, &S.q_full, c - a.Dl, r, 0);
                }
                ++seg;
            }
            for (int t = walk.t0; t < walk.t1; ++t, ++it) {
                const int j = t * kTok + mine * args.box_rows;
                const bool ok = page >= 0 && page < a.num_pages;
                if (!ok && j < walk.len && lane < ng) atomicCAS(a.err, 0, (int32_t)RDA_ERR_INVALID_ARG);
                const unsigned good = __ballot_sync(0xffffffffu, ok && lane < ng);
                const int px = ok ? page : args.pages_bound, row = j % a.page_size;
                page = page_of(t + 1);
                if (lane == 0) {
                    uint64_t m = 0;
                    for (int i = 0; i < ng; ++i)
                        if (good >> i & 1)
                            m |= (args.box_rows == 64 ? ~0ull : (1ull << args.box_rows) - 1) << (i * args.box_rows);
                    const int left = walk.len - t * kTok;
                    if (left < kTok) m &= left <= 0 ? 0ull : (1ull << left) - 1;
                    S.info[it % kInfo] = m;
                }
                for (int p = 0; p < NP; ++p) {
                    if (!room(&S.empty[pr.slot], pr.phase ^ 1, it * NP + p >= (uint32_t)g.pairs, &S.full[pr.slot], kPair))
                        break;
                    if (lane < 2 * ng)
                        tma_load_3d(pair_s + pr.slot * kPair + (lane / ng) * kBox + mine * args.box_rows * 128,
                                    &maps.pages, &S.full[pr.slot], p * 128 + (lane / ng) * 64, row, px);
                    pr.next(g.pairs);
                }
                if (a.Ds && room(&S.sempty[sr.slot], sr.phase ^ 1, it >= (uint32_t)g.shared, &S.sfull[sr.slot], kBox)) {
                    if (lane < ng)
                        tma_load_3d(shared_s + sr.slot * kBox + lane * args.box_rows * 128, &maps.pages,
                                    &S.sfull[sr.slot], a.Dl, row, px);
                    sr.next(g.shared);
                }
            }
        }
        if (S.abort && lane == 0) {
            // copies in flight land before the CTA leaves: the last phase of every slot that was filled
            // (one that never was counts as complete)
            const uint64_t t0 = Waiter::now();
            for (int i = 0; i < g.pairs; ++i) w.drain(&S.full[i], (i < pr.slot ? pr.phase : pr.phase ^ 1), t0);
            for (int i = 0; i < g.shared; ++i) w.drain(&S.sfull[i], (i < sr.slot ? sr.phase : sr.phase ^ 1), t0);
            if (seg > 0) w.drain(&S.q_full, (seg - 1) & 1, t0);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        if (lane == 0) {
            RingPos qk_p, qk_s, pv_p;
            constexpr uint32_t idS = idesc_bf16(kTok, NT, 0, 0), idO = idesc_bf16(128, NT, 1, 0);
            const uint32_t qa = smem_u32(q_s), pa = smem_u32(p_s), ca = smem_u32(pair_s), sa = smem_u32(shared_s);
            Walk ahead = walk;                    // the scores run one tile ahead
            bool more = ahead.next(a);
            int at = more ? ahead.t0 : 0;
            uint32_t qk_seg = 0, pv_seg = 0, it = 0, qk_it = 0;
            auto scores = [&]() {
                // S^T of tile `at` of the segment `ahead`
                bool ok = at != ahead.t0 || w.wait(&S.q_full, qk_seg & 1);
                const uint32_t d = t_s + (qk_it & 1) * NT;
                uint32_t acc = 0;
                tc_fence_after();
                for (int p = 0; p < NP; ++p) {
                    ok = w.wait(&S.full[qk_p.slot], qk_p.phase) && ok;
                    if (ok && !S.abort) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            mma_bf16(d, smem_desc(ca + qk_p.slot * kPair + (k >> 2) * kBox + (k & 3) * 32, 16, 1024, kSw128),
                                     smem_desc(qa + (2 * p + (k >> 2)) * NT * 128 + (k & 3) * 32, 16, 1024, kSw128), idS, acc);
                            acc = 1;
                        }
                    }
                    qk_p.next(g.pairs);
                }
                if (a.Ds) {
                    ok = w.wait(&S.sfull[qk_s.slot], qk_s.phase) && ok;
                    if (ok && !S.abort) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16(d, smem_desc(sa + qk_s.slot * kBox + k * 32, 16, 1024, kSw128),
                                     smem_desc(qa + 2 * NP * NT * 128 + k * 32, 16, 1024, kSw128), idS, 1);
                        mma_commit(&S.sempty[qk_s.slot]);
                    }
                    qk_s.next(g.shared);
                }
                mma_commit(&S.s_full[qk_it & 1]);
                ++qk_it;
                if (++at == ahead.t1) {
                    mma_commit(&S.q_empty);
                    ++qk_seg;
                    more = ahead.next(a);
                    at = ahead.t0;
                }
            };
            if (more) scores();
            while (walk.next(a)) {
                for (int t = walk.t0; t < walk.t1; ++t, ++it) {
                    if (more) scores();
                    bool ok = w.wait(&S.p_ready, it & 1);
                    if (t == walk.t0 && pv_seg > 0) ok = w.wait(&S.o_empty, (pv_seg - 1) & 1) && ok;
                    tc_fence_after();
                    for (int p = 0; p < NP; ++p) {
                        if (ok && !S.abort) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_bf16(t_o + p * NT, smem_desc(ca + pv_p.slot * kPair + k * 2048, kBox, 1024, kSw128),
                                         smem_desc(pa + k * 32, 16, 1024, kSw128), idO, t != walk.t0 || k > 0);
                            mma_commit(&S.empty[pv_p.slot]);
                        }
                        pv_p.next(g.pairs);
                    }
                    mma_commit(&S.pv_done);
                }
                ++pv_seg;
            }
            // every MMA has completed when pv_done has (the softmax warps wait for it, or below)
            if (S.abort && it > 0) w.drain(&S.pv_done, (it - 1) & 1, Waiter::now());
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int quad = warp & 3;                       // tokens 16 quad .. + 15 of a tile
        const int tok = lane >> 2, col = 2 * (lane & 3); // my tokens: tok, tok + 8; my columns: 8 c + col, + 1
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        const float sc = a.scale * kLog2e;
        constexpr int C = NT / 8;
        uint32_t it = 0;
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
                    const int r = 8 * c + col + u;
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
                const uint64_t valid = S.info[it % kInfo];
                const int j0 = t * kTok + 16 * quad + tok;
                const bool whole = valid == ~0ull && t * kTok + kTok - 1 <= all_see;
                if (!whole) {
                    const bool v0 = valid >> (16 * quad + tok) & 1, v1 = valid >> (16 * quad + tok + 8) & 1;
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            if (!v0 || j0 > last[c][u]) v[c][u] = -INFINITY;
                            if (!v1 || j0 + 8 > last[c][u]) v[c][2 + u] = -INFINITY;
                        }
                    // rows behind the sequence's end in a page may hold anything: 0 x NaN must not reach O
                    const int left = walk.len - t * kTok;
                    if (left < kTok) {
                        const int end = min(kTok, (max(left, 0) + args.box_rows - 1) / args.box_rows * args.box_rows);
                        for (int e = tid - 64; e < (end - max(left, 0)) * 8 * 2 * NP; e += 128) {
                            const int r = max(left, 0) + e / (16 * NP), x = e % (16 * NP);
                            const int slot = (int)(((long long)it * NP + (x >> 4)) % g.pairs);
                            *reinterpret_cast<uint4 *>(pair_s + slot * kPair + ((x >> 3) & 1) * kBox + sw128(r, x & 7)) =
                                make_uint4(0, 0, 0, 0);
                        }
                    }
                }
                // the tile's maximum of each of my columns
                float top[C][2];
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float x = fmaxf(v[c][u], v[c][2 + u]);
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        top[c][u] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    }
                if (lane < 4)
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        *reinterpret_cast<float2 *>(&S.wmax[it & 1][quad][8 * c + col]) = make_float2(top[c][0], top[c][1]);
                named_bar_sync(1, 128);
                bool grown = false;
                float f[C][2];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float2 x[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) x[q] = *reinterpret_cast<float2 *>(&S.wmax[it & 1][q][8 * c + col]);
                    top[c][0] = fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x));
                    top[c][1] = fmaxf(fmaxf(x[0].y, x[1].y), fmaxf(x[2].y, x[3].y));
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float now = top[c][u];
                        f[c][u] = 1.f;
                        if (now > m[c][u] + kGrow || (m[c][u] == -INFINITY && now > -INFINITY)) {
                            f[c][u] = ex2(m[c][u] - now);
                            m[c][u] = now;
                            grown = true;
                        }
                    }
                }
                const bool rescale = __any_sync(0xffffffffu, grown) && t != walk.t0;
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
                            S.factor[8 * c + col] = f[c][0];
                            S.factor[8 * c + col + 1] = f[c][1];
                        }
                    named_bar_sync(2, 128);
                    for (int p = 0; p < NP; ++p)
#pragma unroll
                        for (int c = 0; c < NT; c += 16) {
                            float x[16];
                            tmem_ld16(t_o + p * NT + c + lanes, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) x[i] *= S.factor[c + i];
                            tmem_st16f(t_o + p * NT + c + lanes, x);
                        }
                    tmem_wait_st();
                    named_bar_sync(2, 128);                          // factors read by all
                }
#pragma unroll
                for (int c = 0; c < C; c += 2) {
                    // matrices: (block c, tokens 0-7), (c, 8-15), (c + 1, 0-7), (c + 1, 8-15) of my warp's 16
                    const int r = 8 * (c + (lane >> 4)) + (lane & 7), ch = 2 * quad + ((lane >> 3) & 1);
                    stsm_x4_t(smem_u32(p_s) + sw128(r, ch), pk[c][0], pk[c][1], pk[c + 1][0], pk[c + 1][1]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&S.p_ready);
            }
            // the segment's result: whole, or one part of a sequence
            const bool done = walk.t0 == 0 && walk.t1 == walk.tiles;
            const size_t slot = ((size_t)grp * g.rt + rt) * 2 + (first_segment ? 0 : 1);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float x = l[c][u];
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    if (lane < 4) S.lsum[quad][8 * c + col + u] = x;
                }
            named_bar_sync(1, 128);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int r = 8 * c + col + u;
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
            named_bar_sync(1, 128);
            for (int p = 0; p < NP; ++p) {
                const int d = p * 128 + 32 * quad + lane;
#pragma unroll
                for (int c = 0; c < NT; c += 16) {
                    float x[16];
                    tmem_ld16(t_o + p * NT + c + lanes, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int r = c + i;
                        if (r >= rows) continue;
                        const float y = x[i] * S.factor[r];
                        if (!done) parts.o[(slot * NT + r) * a.Dl + d] = y;
                        else
                            static_cast<__nv_bfloat16 *>(a.out)[((size_t)walk.seq * R + row0 + r) * a.Dl + d] =
                                __float2bfloat16_rn(y);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(&S.o_empty);
            named_bar_sync(1, 128);                                  // factors are free again
            if (rt == 0 && tid == 64 && walk.pos >= hi) {
                // this group's last segment: does its sequence begin here and go on in others?
                int4 rec = make_int4(-1, 0, 0, 0);
                if (!done && walk.t0 == 0) {
                    const long long groups = min((long long)g.groups, total);
                    const long long end = hi - walk.t1 + walk.tiles - 1;      // the sequence's last tile
                    long long gl = min(groups - 1, end * groups / total);     // the group that holds it
                    while (gl + 1 < groups && total * (gl + 1) / groups <= end) ++gl;
                    while (total * gl / groups > end) --gl;
                    rec = make_int4(walk.seq, (int)gl, first_segment ? 0 : 1, 0);
                }
                parts.rec[grp] = rec;
            }
            first_segment = false;
        }
        if (rt == 0 && tid == 64 && lo >= hi) parts.rec[grp] = make_int4(-1, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// Joins the parts of the sequence that begins in group blockIdx.x and goes on in
// others: out = sum_i e^{lse_i - lse} o_i.  One CTA per row; four quarters of
// the CTA take every fourth part.
constexpr int kJoin = 512;
__global__ void __launch_bounds__(kJoin) latent_join_bf16_kernel(const Args args) {
    __shared__ float4 acc_s[3][128];
    __shared__ float w_s[kCtas];
    const LatentDecodeArgs &a = args.a;
    const Geometry &g = args.g;
    const Parts parts = parts_of(a.part, g, a.Dl);
    const int grp = blockIdx.x, rt = blockIdx.y / g.rows, r = blockIdx.y % g.rows, R = a.T * a.H;
    const int tid = threadIdx.x, lane = tid & 31, part = tid >> 7, c = (tid & 127) * 4;
    if (rt * g.rows + r >= R) return;
    pdl_wait_primary();
    const int4 rec = parts.rec[grp];
    if (rec.x < 0) return;
    const int n = rec.y - grp + 1;
    auto slot = [&](int i) { return (((size_t)(grp + i) * g.rt + rt) * 2 + (i == 0 ? rec.z : 0)) * g.nt + r; };
    // weights: every warp computes the common maximum and sum
    float top = -INFINITY;
    for (int i = lane; i < n; i += 32) top = fmaxf(top, parts.lse[slot(i)]);
#pragma unroll
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int i = lane; i < n; i += 32) {
        const float x = expf(parts.lse[slot(i)] - base);
        sum += x;
        if (tid < 32) w_s[i] = x;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    __syncthreads();
    const float f = sum > 0.f ? 1.f / sum : 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < a.Dl) {
#pragma unroll 4
        for (int i = part; i < n; i += 4) {
            const float4 y = *reinterpret_cast<const float4 *>(parts.o + slot(i) * a.Dl + c);
            const float wi = w_s[i] * f;
            x.x = fmaf(wi, y.x, x.x), x.y = fmaf(wi, y.y, x.y), x.z = fmaf(wi, y.z, x.z), x.w = fmaf(wi, y.w, x.w);
        }
    }
    if (part) acc_s[part - 1][tid & 127] = x;
    __syncthreads();
    const size_t row = (size_t)rec.x * R + rt * g.rows + r;
    if (part == 0 && c < a.Dl) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const float4 y = acc_s[i][tid];
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        uint2 h = make_uint2(pack2(x.x, x.y), pack2(x.z, x.w));
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + row * a.Dl + c) = h;
    }
    if (tid == 0 && a.lse) a.lse[row] = sum > 0.f ? base + logf(sum) : -INFINITY;
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
    const uint32_t most = 232448 - 1024 - small;
    const int D = Dl + Ds, NP = Dl / 128;
    // the scores run a tile ahead of the values: two tiles of latents at least; one slot for the
    // shared columns if two do not fit beside them
    g.shared = Ds ? 2 : 0;
    if (Ds && operand_bytes(g.nt, D, 2 * NP, 2) > most) g.shared = 1;
    g.pairs = std::min<int>(kMaxPairs, (int)((most - operand_bytes(g.nt, D, 0, g.shared)) / kPair));
    g.smem = operand_bytes(g.nt, D, g.pairs, g.shared) + small + 1024;
    return g;
}
static_assert(sizeof(Small<64>) % 8 == 0, "barriers are 8-byte aligned");

template <int NT> cudaError_t launch(const Maps &maps, const Args &args, cudaStream_t s) {
    cudaError_t e = allow_smem<latent_decode_kernel<NT>>(232448);
    if (e != cudaSuccess) return e;
    latent_decode_kernel<NT><<<args.g.rt * args.g.groups, kThreads, args.g.smem, s>>>(maps, args);
    return cudaGetLastError();
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
    args.box_rows = std::min(kTok, a.page_size & -a.page_size);
    const int D = a.Dl + a.Ds, R = a.T * a.H;
    if (args.g.pairs < 2 * (a.Dl / 128)) return cudaErrorInvalidConfiguration;
    Maps maps;
    std::memset(&maps, 0, sizeof(maps));
    // without a page the map is never read inside its bounds; any aligned base will do
    const int pages = std::max(1, a.num_pages);
    args.pages_bound = pages;
    if (!make_map_3d(&maps.pages, a.num_pages ? a.pages : a.q, D, a.page_size, pages, D, (uint64_t)a.page_size * D,
                     args.box_rows, 1) ||
        !make_map_3d(&maps.q, a.q, a.Dl, (uint64_t)a.B * R, 1, a.Dl, (uint64_t)a.B * R * a.Dl, args.g.nt, 1) ||
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(args.g.groups, args.g.rt * args.g.rows);
    cfg.blockDim = dim3(kJoin);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, latent_join_bf16_kernel, args);
}

}  // namespace rda
