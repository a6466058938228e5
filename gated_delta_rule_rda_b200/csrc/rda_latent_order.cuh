// Orders the tiles of a packed batch by their work (device side).
#pragma once

#include "rda_latent.h"

namespace rda {

__device__ __forceinline__ int tile_work(const LatentArgs &a, const TileOrder &o, int n, int t) {
    const int lq = seq_span(a.cu_q, n, a.total_q).len, lk = seq_span(a.cu_k, n, a.total_k).len, more = lk - lq;
    if (o.keys) {
        if (t * o.tile >= lk) return -1;
        return max(0, (lq + o.unit - 1) / o.unit - (a.causal ? max(0, t * o.tile - more) / o.unit : 0));
    }
    if (t * o.tile >= lq) return -1;
    const int end = a.causal ? min(lk, min((t + 1) * o.tile, lq) + more) : lk;
    return end > 0 ? (end + o.unit - 1) / o.unit : 0;
}

// By the threads of one CTA: a counting sort over 512 classes of work.  The order
// inside a class is that of the atomics: it decides which CTA takes which tile
// and nothing else.
static __device__ void order_tiles(const LatentArgs &a0, const TileOrder &o) {
    constexpr int kClasses = 512, kSeqs = 1024;
    __shared__ int count_s[kClasses], most_s, total_s;
    __shared__ int32_t cu_s[2][kSeqs + 1];
    const int tid = threadIdx.x, nt = blockDim.x;
    LatentArgs a = a0;
    if (a.num_seqs <= kSeqs) {
        // the offsets are read over and over
        for (int n = tid; n <= a.num_seqs; n += nt) cu_s[0][n] = a0.cu_q[n], cu_s[1][n] = a0.cu_k[n];
        a.cu_q = cu_s[0];
        a.cu_k = cu_s[1];
    }
    for (int c = tid; c < kClasses; c += nt) count_s[c] = 0;
    if (tid == 0) most_s = 0, total_s = 0;
    __syncthreads();
    const int32_t *cu = o.keys ? a.cu_k : a.cu_q;
    const int total = o.keys ? a.total_k : a.total_q, slots = tile_slots(total, a.num_seqs, o.tile);
    // this thread's first place is kept, more are looked up again
    int n0 = 0, t0 = 0, w0 = -1;
    auto look = [&](int s, int *n, int *t) {
        if (s == tid) {
            *n = n0;
            *t = t0;
            return w0;
        }
        *n = find_tile(cu, a.num_seqs, total, o.tile, s, t);
        return tile_work(a, o, *n, *t);
    };
    if (tid < slots) {
        n0 = find_tile(cu, a.num_seqs, total, o.tile, tid, &t0);
        w0 = tile_work(a, o, n0, t0);
    }
    int most = w0, n, t;
    for (int s = tid + nt; s < slots; s += nt) most = max(most, look(s, &n, &t));
    atomicMax(&most_s, most);
    __syncthreads();
    most = most_s + 1;
    auto cls = [&](int w) { return kClasses - 1 - (int)((long long)w * kClasses / most); };       // the most work in class 0
    for (int s = tid; s < slots; s += nt) {
        const int w = look(s, &n, &t);
        if (w >= 0) atomicAdd(&count_s[cls(w)], 1);
    }
    __syncthreads();
    if (tid < 32) {
        // exclusive sums: 16 classes a lane
        int x = 0;
        for (int i = 0; i < kClasses / 32; ++i) x += count_s[tid * (kClasses / 32) + i];
        int upto = x;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, off);
            if (tid >= off) upto += y;
        }
        if (tid == 31) total_s = upto;
        int before = upto - x;
        for (int i = 0; i < kClasses / 32; ++i) {
            const int y = count_s[tid * (kClasses / 32) + i];
            count_s[tid * (kClasses / 32) + i] = before;
            before += y;
        }
    }
    __syncthreads();
    for (int s = tid; s < slots; s += nt) {
        const int w = look(s, &n, &t);
        if (w >= 0) o.out[atomicAdd(&count_s[cls(w)], 1)] = make_int2(n, t);
        if (s >= total_s) o.out[s] = make_int2(-1, -1);
    }
}

// Sequence and tile of place `slot`, most work first; -1 where there is none.  Without an order, places
// run from the batch's last tile (the sequences' last query tiles see the most keys) or, for keys, its first.
__device__ __forceinline__ int tile_at(const LatentArgs &a, bool keys, int tile, int slot, int slots, int *t) {
    if (a.order) {
        const int2 x = a.order[slot];
        *t = x.y;
        return x.x;
    }
    return keys ? find_tile(a.cu_k, a.num_seqs, a.total_k, tile, slot, t)
                : find_tile(a.cu_q, a.num_seqs, a.total_q, tile, slots - 1 - slot, t);
}

}  // namespace rda
