// What the latent-attention kernels share besides sm100_ptx.cuh: bounded waits,
// the remaining tcgen05 forms, swizzled addressing and small conversions.
#pragma once

#include <cuda_bf16.h>

#include "rda.h"
#include "sm100_ptx.cuh"

namespace rda {
namespace ptx {

// Bounded mbarrier waits of one CTA.  `abort` is a word of shared memory: a
// wait that runs out records RDA_ERR_TIMEOUT in *err and sets it; from then on
// every wait of the CTA that would block returns at once.  All threads run their
// loops to the end either way (no thread leaves a named barrier short); MMAs and
// copies are issued only after waits that succeeded.
struct Waiter {
    volatile int *abort;
    int32_t *err;
    uint64_t limit_ns;

    static __device__ __forceinline__ uint64_t now() {
        uint64_t t;
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        return t;
    }
    __device__ __noinline__ bool slow(uint64_t *bar, uint32_t parity) const {
        const uint64_t t0 = now();
        for (;;) {
            if (*abort) return false;
            for (int i = 0; i < 8; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (now() - t0 > limit_ns) {
                *abort = 1;
                atomicCAS(err, 0, (int32_t)RDA_ERR_TIMEOUT);
                return false;
            }
        }
    }
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) const {
        return mbar_try_wait(bar, parity) || slow(bar, parity);
    }
    // ignores the abort word: lets what is in flight land before the CTA leaves (bounded from t0 on)
    __device__ __noinline__ void drain(uint64_t *bar, uint32_t parity, uint64_t t0) const {
        while (!mbar_try_wait(bar, parity))
            if (now() - t0 > limit_ns) return;
    }
};

// An MMA whose operands' descriptors are given by their low words (address and leading offset); the high words (stride
// and swizzle) are the same constant.  Half the arithmetic per MMA for a thread that issues them one after the other.
__device__ __forceinline__ void mma_bf16_low(uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(high), "r"(idesc), "r"(acc)
        : "memory");
}

// `bytes` (a multiple of 16) from a 16-byte boundary on come into L2.
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(__cvta_generic_to_global(p)), "r"(bytes) : "memory");
}

// One lane of a converged warp.  The MMA issuers branch on it (and not on the
// lane's number): the compiler then knows that one thread runs the branch and
// keeps descriptors in uniform registers.  An unrolled chain of M = 64, N = 16
// products issues every 24 cycles this way, every 51 behind `lane == 0`.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// A slot of a ring and the parity of its next phase.
struct RingPos {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++slot == n) slot = 0, phase ^= 1;
    }
    // `by` slots on, n of them at most
    __device__ __forceinline__ void skip(int by, int n) {
        if ((slot += by) >= n) slot -= n, phase ^= 1;
    }
};

// D[tmem] (+)= A[tmem] * B[smem], bf16 inputs, fp32 accumulate (A: one row per lane, two values a column).
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 lanes x 16 columns: thread l gets lanes l/4 and l/4 + 8 at columns 2(l%4), + 1 of both 8-column blocks.
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, float *v) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// 32 lanes x 32 bits, 32 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float *v) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0,%1,%2,%3};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16f(uint32_t taddr, const float *v) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    tmem_st16(taddr, r);
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four 8x8 matrices of 16-bit values, each stored transposed: row r of matrix m at the address that lane
// 8 m + r gives; register m holds (row l/4, columns 2(l%4), + 1) of the untransposed matrix.
__device__ __forceinline__ void stsm_x4_t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r0), "r"(r1),
                 "r"(r2), "r"(r3)
                 : "memory");
}

// Named barrier that also tells every thread whether `mine` holds in any of them.
__device__ __forceinline__ bool named_bar_any(uint32_t id, uint32_t nthreads, bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(nthreads), "r"((uint32_t)mine)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}

// Byte offset of 16-byte chunk `c` (0..7) of row `row` in a tile of 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t c) { return row * 128 + ((c ^ (row & 7)) << 4); }

// 128 bytes of each of a warp's 32 rows (lane = row) to global memory, rows `stride` bytes apart, the first `rows`
// of them.  Through 4 KiB of shared memory, so that a store covers four whole rows: straight from the lanes each
// store touches 32 lines (9,700 cycles for 128 rows of 384 columns, 3,000 this way).
__device__ __forceinline__ void store_rows_128(uint8_t *buf, const uint4 (&x)[8], void *out, size_t stride, int rows) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(buf + sw128(lane, c)) = x[c];
    __syncwarp();
    uint8_t *to = static_cast<uint8_t *>(out) + (lane >> 3) * stride + (lane & 7) * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i, to += 4 * stride) {
        const int r = 4 * i + (lane >> 3);
        if (r < rows) *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(buf + sw128(r, lane & 7));
    }
    __syncwarp();
}
// 64 columns of an accumulator times f, as bf16 (zeros where there is no accumulator).
__device__ __forceinline__ void tmem_row_bf16(uint32_t t, float f, bool any, uint4 (&x)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float v[32];
        if (any) {
            tmem_ld32(t + 32 * h, v);
            tmem_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = any ? v[i] * f : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[4 * h + i] = make_uint4(pack2(v[8 * i], v[8 * i + 1]), pack2(v[8 * i + 2], v[8 * i + 3]),
                                      pack2(v[8 * i + 4], v[8 * i + 5]), pack2(v[8 * i + 6], v[8 * i + 7]));
    }
}
// 32 columns times f, as fp32.
__device__ __forceinline__ void tmem_row_f32(uint32_t t, float f, bool any, uint4 (&x)[8]) {
    float v[32];
    if (any) {
        tmem_ld32(t, v);
        tmem_wait_ld();
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = any ? v[i] * f : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                          __float_as_uint(v[4 * i + 3]));
}

// The dynamic shared memory rounded up to 1024 bytes, as shared memory.
__device__ __forceinline__ uint8_t *align_1024(uint8_t *raw) { return raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u); }

}  // namespace ptx

// A bf16 tensor [d2][d1][d0] (contiguous rows of d0, strides in elements) as a
// TMA map with boxes of 64 x box1 x box2, 128-byte swizzle, zeros outside.
bool make_map_3d(CUtensorMap *map, const void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t stride1,
                 uint64_t stride2, uint32_t box1, uint32_t box2);
// [rows, H, D]: boxes of 64 columns of one head x `box` rows; where there are no rows the map is only read outside
// its bounds, and `any` is its base.
bool make_map_heads(CUtensorMap *map, const void *base, int D, int H, long rows, uint32_t box, const void *any);

}  // namespace rda
