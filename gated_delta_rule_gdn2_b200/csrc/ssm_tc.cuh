// Pieces shared by the tensor-core kernels of the selective state space scan:
// tensor maps of strided token tensors, tile addressing, 32-lane tensor-memory
// accesses, the product whose left operand lies in tensor memory, and the
// decay factors of a chunk.
//
// Tiles are [rows][64] bf16 blocks of 128-byte rows, their 16-byte pieces
// permuted by row mod 8 (the 128-byte swizzle): a [R][D] tile is D / 64 such
// blocks of R rows, one after the other.
#pragma once

#include "gdn2.h"
#include "ssm.h"
#include "tc.cuh"
#include "tc_tiles.cuh"
#include "tma_host.h"

namespace gdn2 {
namespace ssm {

constexpr int kCT = 128;   // tokens of a chunk of the tensor-core kernels
constexpr int kNT = 512;   // their threads: four warps per tensor-memory sub-partition

// [B][T] rows, ld elements apart, of `heads` heads of D channels, in boxes of
// 128 tokens x 64 channels of one head: coordinates (0, token, channel / 64, head, batch).
inline bool scan_tile_map(CUtensorMap *m, const void *base, long long ld, int B, int T, int heads, int D) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[5] = {64, (cuuint64_t)T, (cuuint64_t)(D / 64), (cuuint64_t)heads, (cuuint64_t)B};
    const cuuint64_t strides[4] = {(cuuint64_t)ld * 2, 128, (cuuint64_t)D * 2, (cuuint64_t)T * (cuuint64_t)ld * 2};
    const cuuint32_t box[5] = {64, (cuuint32_t)kCT, 1, 1, 1};
    const cuuint32_t unit[5] = {1, 1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims, strides, box, unit,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

typedef __nv_bfloat16 bf16;

__device__ __forceinline__ void tma_store_5d(const void *map, const void *src, int y, int z, int w, int v) {
    asm volatile("cp.async.bulk.tensor.5d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4, %5}], [%6];\n" ::"l"(map),
                 "r"(0), "r"(y), "r"(z), "r"(w), "r"(v), "r"(tc::smem_addr(src))
                 : "memory");
}

// e^x by the fast base-2 exponential, results below 2^-126 taken as 0 (2
// instructions; x = -inf gives 0).
__device__ __forceinline__ float exp_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// What a block's bounded waits share (in shared memory).
struct alignas(8) Waits {
    uint32_t dead;   // one has run out
    uint32_t limit;  // iterations of a wait
};
__device__ __forceinline__ void waits_init(Waits &w, uint32_t limit) {
    w.dead = 0;
    w.limit = limit ? limit : tc::kWaitLimit;
}
// A bounded wait for the phase `parity` of a barrier: false when it ran out
// here, or (w->dead) in any thread of the block.  Kept to a dozen
// instructions: the kernels hold dozens of waits, and their code has to stay
// within the instruction cache.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, Waits *w) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\n.reg .u32 n, d, l;\nmov.u32 n, 0;\n"
        "AGAIN:\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "@p bra DONE;\n"
        "ld.volatile.shared.v2.u32 {d, l}, [%3];\n"
        "add.u32 n, n, 1;\n"
        "setp.ge.u32 p, n, l;\n"
        "@p mov.u32 d, 1;\n"
        "setp.eq.u32 p, d, 0;\n"
        "@p bra AGAIN;\n"
        "st.volatile.shared.u32 [%3], d;\n"
        "setp.ne.u32 p, d, d;\n"
        "DONE:\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(tc::smem_addr(bar)), "r"(parity), "r"(tc::smem_addr(w))
        : "memory");
    return ok != 0;
}
// One lane of a converged warp (products and copies are issued by the warp
// that runs their loop as a whole: its operands stay uniform).
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n.reg .pred q;\nelect.sync _|q, 0xffffffff;\nselp.b32 %0, 1, 0, q;\n}\n" : "=r"(p));
    return p != 0;
}

// D (+)= A B with A [128][K] bf16 in tensor memory (two values a column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1 : 0));
}

__device__ __forceinline__ void ld16(uint32_t t, float (&v)[16]) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t));
}
__device__ __forceinline__ void st16(uint32_t t, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
__device__ __forceinline__ void ld8(uint32_t t, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t));
}
__device__ __forceinline__ void st8(uint32_t t, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(t), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}
__device__ __forceinline__ void ld8(uint32_t t, float (&v)[8]) { ld8(t, reinterpret_cast<uint32_t(&)[8]>(v)); }
__device__ __forceinline__ void ld4(uint32_t t, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(t));
}
__device__ __forceinline__ void st4(uint32_t t, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]));
}
// 16 or 32 consecutive columns of this thread's lane
template <int W>
__device__ __forceinline__ void ldw(uint32_t t, float (&v)[W]) {
    if constexpr (W == 16) ld16(t, v);
    else tc::ld_32x32b_x32(t, v);
}
template <int W>
__device__ __forceinline__ void stw(uint32_t t, const float (&v)[W]) {
    if constexpr (W == 16) st16(t, reinterpret_cast<const uint32_t(&)[16]>(v));
    else tc::st_32x32b_x32(t, v);
}

// Byte offset of piece `p8` (8 channels) of row r in a [R][.] tile.
__device__ __forceinline__ uint32_t piece(int R, int r, int p8) {
    return (uint32_t)((p8 >> 3) * (R * 128) + r * 128 + (((p8 & 7) ^ (r & 7)) << 4));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&x);
}
__device__ __forceinline__ float2 unpack2(uint32_t u) { return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u)); }

// W consecutive fp32 values of row r from column c0 on, rounded to bf16, into a tile.
template <int W>
__device__ __forceinline__ void put_row(unsigned char *tile, int R, int r, int c0, const float (&v)[W]) {
#pragma unroll
    for (int i = 0; i < W / 8; ++i)
        *reinterpret_cast<uint4 *>(tile + piece(R, r, c0 / 8 + i)) =
            make_uint4(pack2(v[8 * i], v[8 * i + 1]), pack2(v[8 * i + 2], v[8 * i + 3]), pack2(v[8 * i + 4], v[8 * i + 5]),
                       pack2(v[8 * i + 6], v[8 * i + 7]));
}

// Decay factors of a chunk, by blocks of 32 tokens (one warp each): exponents
// of products across blocks are sums of terms <= 0, so none overflows and none
// is a difference of long sums.
//   l    log decay from the block's start through the token
//   cf   e^{log decay from behind the token to the block's end} (FWD: times dt)
//   er   e^{log decay from the chunk's start through the token}
//   wt   e^{log decay from behind the token to the chunk's end} (FWD: times dt)
//   ld   l less the log of the step size (so e^{l_i - ld_j} holds dt_j)
struct alignas(16) Gates {  // (read in 16-byte pieces, two side by side)
    float l[kCT], cf[kCT], er[kCT], wt[kCT], ld[kCT];
    float bs[4];    // the blocks' log decays
    float gamma;    // the chunk's decay
};
// Formed by one warp, four tokens a lane, from token t0 of a sequence of len
// tokens whose values lie `stride` elements apart from `first` on (dt ==
// nullptr: 1); `carry` is a log decay that er and wt hold besides.  Returns the
// chunk's log decay.
__device__ __forceinline__ float form_gates_warp(Gates &g, const void *la, const void *dt, size_t first, int stride, int t0,
                                                 int len, int lane, float carry) {
    float x[4], d[4], up[4], dn[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int t = t0 + 4 * lane + e;
        const size_t r = first + (size_t)t * stride;
        x[e] = t < len ? bounded_log(__bfloat162float(static_cast<const bf16 *>(la)[r])) : 0.f;
        d[e] = t >= len ? 0.f : dt ? __bfloat162float(static_cast<const bf16 *>(dt)[r]) : 1.f;
    }
    up[0] = x[0];
    dn[3] = x[3];
#pragma unroll
    for (int e = 1; e < 4; ++e) {
        up[e] = up[e - 1] + x[e];
        dn[3 - e] = dn[4 - e] + x[3 - e];
    }
    // within the blocks of 32 tokens (8 lanes), then across them
    float a = up[3], c = dn[0];
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, a, m, 8), z = __shfl_down_sync(0xffffffffu, c, m, 8);
        if ((lane & 7) >= m) a += y;
        if ((lane & 7) + m < 8) c += z;
    }
    float before = __shfl_up_sync(0xffffffffu, a, 1, 8), behind = __shfl_down_sync(0xffffffffu, c, 1, 8);
    if ((lane & 7) == 0) before = 0.f;
    if ((lane & 7) == 7) behind = 0.f;
    const float b0 = __shfl_sync(0xffffffffu, a, 7), b1 = __shfl_sync(0xffffffffu, a, 15), b2 = __shfl_sync(0xffffffffu, a, 23),
                b3 = __shfl_sync(0xffffffffu, a, 31);
    const int w = lane >> 3;
    const float pre = w == 0 ? 0.f : w == 1 ? b0 : w == 2 ? b0 + b1 : b0 + b1 + b2;
    const float post = w == 3 ? 0.f : w == 2 ? b3 : w == 1 ? b2 + b3 : b1 + b2 + b3;
    float l[4], cf[4], er[4], wt[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float s = behind + (e < 3 ? dn[e + 1] : 0.f);
        l[e] = before + up[e];
        cf[e] = exp_ftz(s) * d[e];
        er[e] = exp_ftz(pre + l[e] + carry);
        wt[e] = exp_ftz(s + post + carry) * d[e];
    }
    *reinterpret_cast<float4 *>(&g.l[4 * lane]) = make_float4(l[0], l[1], l[2], l[3]);
    *reinterpret_cast<float4 *>(&g.cf[4 * lane]) = make_float4(cf[0], cf[1], cf[2], cf[3]);
    *reinterpret_cast<float4 *>(&g.er[4 * lane]) = make_float4(er[0], er[1], er[2], er[3]);
    *reinterpret_cast<float4 *>(&g.wt[4 * lane]) = make_float4(wt[0], wt[1], wt[2], wt[3]);
    // (a step of zero: ld = inf, a factor of 0; a negative one does not occur)
    *reinterpret_cast<float4 *>(&g.ld[4 * lane]) =
        make_float4(l[0] - __logf(d[0]), l[1] - __logf(d[1]), l[2] - __logf(d[2]), l[3] - __logf(d[3]));
    if ((lane & 7) == 7) g.bs[w] = a;
    const float all = b0 + b1 + b2 + b3;
    if (lane == 0) g.gamma = exp_ftz(all);
    return all;
}
// log decay of the blocks strictly between block a and block b > a
__device__ __forceinline__ float between(const Gates &g, int a, int b) {
    float s = 0.f;
    if (a < 1 && b > 1) s += g.bs[1];
    if (a < 2 && b > 2) s += g.bs[2];
    return s;
}

// Rows [len, 128) of a [128][64 nblk] tile set to zero (the last chunk of a
// packed sequence, whose box reaches into the next one).
__device__ __forceinline__ void zero_tail(unsigned char *tile, int nblk, int len, int tid, int nt) {
    const int n = (kCT - len) * 8;
    for (int i = tid; i < n * nblk; i += nt) {
        const int blk = i / n, x = i % n;
        *reinterpret_cast<uint4 *>(tile + blk * (kCT * 128) + (len + x / 8) * 128 + (x % 8) * 16) = make_uint4(0, 0, 0, 0);
    }
}

// Rows r0 .. r0 + ROWS - 1 of a [128][D] tile scaled by f[row], in two bf16
// parts whose sum carries 16 bits: the parts of the first go in place, of the
// rest to the [ROWS][D] tile `lo`.  Rows from len on become zero whatever they hold.
template <int D, int NT, int ROWS>
__device__ __forceinline__ void scale_hi_lo(unsigned char *hi, unsigned char *lo, const float *f, int r0, int len, int tid) {
    // eight consecutive lanes take the eight pieces of one 128-byte row; up to
    // four pieces of a thread are loaded ahead of their use
    constexpr int PER = ROWS * (D / 8) / NT, U = PER % 4 == 0 ? 4 : 2;
    static_assert(PER % U == 0 && ROWS % 8 == 0, "pieces of a thread");
    const bool whole = len == kCT;
#pragma unroll 1
    for (int i0 = 0; i0 < PER; i0 += U) {
        uint4 x[U];
        float w[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int id = tid + (i0 + i) * NT, blk = id / (ROWS * 8), r = r0 + (id / 8) % ROWS;
            x[i] = *reinterpret_cast<const uint4 *>(hi + blk * (kCT * 128) + r * 128 + (id % 8) * 16);
            w[i] = f[r];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int id = tid + (i0 + i) * NT, blk = id / (ROWS * 8), r = r0 + (id / 8) % ROWS;
            uint4 y;
            uint32_t *xe = reinterpret_cast<uint32_t *>(&x[i]), *ye = reinterpret_cast<uint32_t *>(&y);
            const float2 w2 = make_float2(w[i], w[i]);
            const bool keep = whole || r < len;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = unpack2(xe[e]), t = __fmul2_rn(v, w2);
                const uint32_t h = pack2(t.x, t.y);
                const float2 hf = unpack2(h), d = __ffma2_rn(hf, make_float2(-1.f, -1.f), t);
                xe[e] = keep ? h : 0u;
                ye[e] = keep ? pack2(d.x, d.y) : 0u;
            }
            *reinterpret_cast<uint4 *>(hi + blk * (kCT * 128) + r * 128 + (id % 8) * 16) = x[i];
            *reinterpret_cast<uint4 *>(lo + id * 16) = y;
        }
    }
}

}  // namespace ssm
}  // namespace gdn2
