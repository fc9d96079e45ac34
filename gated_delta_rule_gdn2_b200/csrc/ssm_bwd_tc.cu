// The selective state space scan's gradients of a chunk, for bf16 tokens on
// the fifth-generation tensor cores.
//
// A CTA takes one chunk of 128 tokens of one group (or of a run of its heads)
// and goes through the heads, 64 value columns at a time ("a unit": v, dO and
// the matching columns of the state S at the chunk's start and of the gradient
// E at its end, 64 KB, double buffered).  With the factors of ssm_scan.cu,
// G = q k^T kept once per CTA and D_ij the decay from j to i, a head is
//     X = v dO^T            -> W = G D X: sums for dla and ddt; Z += D X dt
// over both of its units, and a unit
//     R = q S               -> u_i += e^{L_i} R_i . dO_i
//     Y = k E               -> r_j += w_j Y_j . v_j; Y scaled by w_j
//     Y += (G D)^T dO       -> dv = dt Y + skip dO
//     dq += (e^L dO) S^T
//     dk += (dt w v) E^T
// and behind the last head dq += Z k, dk += Z^T q, so that both are summed over
// the heads before they are rounded.  Rows of X, Y are tokens j (lanes of
// tensor memory), columns i, so that (G D)^T is written back to tensor memory
// as the left operand of the third product; the sums over j of W's columns are
// a transposing reduction within each warp.  (u_i is also q_i . (what the head
// adds to dq_i), but as a difference of sums over the heads it would have the
// rounding of the largest of them.)  Operands rounded to bf16: G, G D,
// e^L dO, dt w v, and the images of S and E, all of them factors of gradients that
// are rounded to bf16 themselves (dq and dk are 1.7e-3 of their norms from exact,
// dv, dla and ddt 2.0e-3 to 2.3e-3, and that last rounding alone is 1.7e-3), and Z
// in two parts; sums are fp32, in a fixed order.
//
// Bound: 64 KB in and 16 KB out a unit at dk = 128 (3500 cycles of an SM's share
// of HBM) against 1500 cycles of tensor pipe.  Measured 8700 cycles a unit (8 x
// 4096 tokens, 16 heads of 128: 302 us; 256 blocks, so a wave and three
// quarters), with 46% of the issue slots, 19% of the tensor pipe and a quarter of
// HBM in use: what bounds it is that the warps meet twice a unit and wait for
// the longest stretch between.  That is X's elementwise part, for its rows j <= i lie four blocks deep in the first sub-partition
// of tensor memory and one deep in the last, and only a sub-partition's own
// warps can read it.  Kept on measurement (same case): waits of a dozen
// instructions and products issued by a converged warp 501 -> 436 us; the
// diagonal block without branches 393; no registers spilled 369; dq in tensor
// memory, which frees 32 registers a thread, 331; X and u once a head 295; no
// warp waits for the next head's decays as they are loaded 281; u from R 299
// (with <E, S> ahead of R 310; Y's part ahead of X's 322); Z in two parts 301.
#include "common.cuh"
#include "ssm_tc.cuh"

namespace gdn2 {
namespace ssm {
namespace {

using tct::mma_tiles;

// Warps 3 and 7 (last sub-partition, first token blocks) have no part in X:
// one issues the products, the other the copies, and writes a head's dla and ddt.
constexpr int kIssuer = 3, kFinisher = 7;

struct BwdMaps {
    CUtensorMap q, k, v, dO, dv;
};

// As Gates, but without dt in cf and wt, and with lf = e^l.
struct alignas(16) BwdGates {
    float l[kCT], lf[kCT], cf[kCT], er[kCT], wt[kCT], dt[kCT];
    float bs[4];
    float gamma;
};
__device__ __forceinline__ void form_bwd_gates(BwdGates &g, float la, float dt, int t) {
    const int lane = t & 31, w = t >> 5;
    float up = la, dn = la;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, up, m), z = __shfl_down_sync(0xffffffffu, dn, m);
        if (lane >= m) up += y;
        if (lane + m < 32) dn += z;
    }
    const float behind = __shfl_down_sync(0xffffffffu, dn, 1), s = lane < 31 ? behind : 0.f;
    g.l[t] = up;
    g.lf[t] = exp_ftz(up);
    g.cf[t] = exp_ftz(s);
    g.dt[t] = dt;
    if (lane == 31) g.bs[w] = up;
    asm volatile("bar.sync 1, 128;\n" ::: "memory");
    const float b0 = g.bs[0], b1 = g.bs[1], b2 = g.bs[2], b3 = g.bs[3];
    const float pre = w == 0 ? 0.f : w == 1 ? b0 : w == 2 ? b0 + b1 : b0 + b1 + b2;
    const float post = w == 3 ? 0.f : w == 2 ? b3 : w == 1 ? b2 + b3 : b1 + b2 + b3;
    g.er[t] = exp_ftz(pre + up);
    g.wt[t] = exp_ftz(s + post);
    if (t == 0) g.gamma = exp_ftz(b0 + b1 + b2 + b3);
}

// Sums over the 32 lanes of 16 values a lane: lanes 2 c and 2 c + 1 end with
// the sum of value c (each step keeps the upper half where the lane's bit m is set).
__device__ __forceinline__ float lane_sums16(float (&v)[16], int lane) {
#pragma unroll
    for (int n = 8, m = 16; n >= 1; n >>= 1, m >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

template <int N>
struct BwdTcSmem {
    static constexpr int QB = kCT * N * 2, VB = kCT * 64 * 2, SB = N * 64 * 2, STAGE = 2 * VB + 2 * SB;
    static constexpr int K = 0, Q = QB, ST0 = 2 * QB, STG = ST0 + 2 * STAGE, G = STG + VB,
                         ROWP = G + 2 * (int)sizeof(BwdGates), COLP = ROWP + 4 * kCT * 4, RP = COLP + 4 * kCT * 4,
                         UP = RP + 4 * kCT * 4, CD = UP + 4 * kCT * 4, RED = CD + kCT * 4, FIN = RED + 2 * 16 * 4, END = FIN + 3 * kCT * 4;
    static constexpr int BYTES = END + 1024;
    static_assert(BYTES + 1024 <= 232448, "shared memory of an SM");
};

template <int N, int P>
__global__ void __launch_bounds__(kNT, 1) bwd_kernel(ScanBwdArgs a, const __grid_constant__ BwdMaps maps) {
    using L = BwdTcSmem<N>;
    constexpr int NX = P / 64, WN = N / 4;  // units a head; a thread's columns of an N-column row
    constexpr uint32_t cX = 0, cDQ = 128, cY = 256, cDK = 320, cG = 448;  // ((G D)^T lies over X)
    constexpr uint32_t idX = tc::idesc_bf16(128, 128, false, false), idY = tc::idesc_bf16(128, 64, false, true),
                       idN = tc::idesc_bf16(128, N, false, false), idZk = tc::idesc_bf16(128, N, false, true),
                       idZq = tc::idesc_bf16(128, N, true, true);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (tc::smem_addr(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t ld_qk, ldx[2], ld[2], b_x, b_q, r_q, b_y, b_c, b_d, b_z;
    __shared__ uint32_t tmem_slot;
    __shared__ Waits waits;
    BwdGates *gates = reinterpret_cast<BwdGates *>(sm + L::G);
    float(*rowp)[kCT] = reinterpret_cast<float(*)[kCT]>(sm + L::ROWP), (*colp)[kCT] = reinterpret_cast<float(*)[kCT]>(sm + L::COLP);
    float(*rp)[kCT] = reinterpret_cast<float(*)[kCT]>(sm + L::RP), (*up)[kCT] = reinterpret_cast<float(*)[kCT]>(sm + L::UP);
    float *cd = reinterpret_cast<float *>(sm + L::CD), *red = reinterpret_cast<float *>(sm + L::RED),
          *fin = reinterpret_cast<float *>(sm + L::FIN);
    const ScanArgs &f = a.f;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, p = warp & 3, qc = warp >> 2, row = 32 * p + lane;
    const int hpg = f.H / f.G, per = (hpg + a.splits - 1) / a.splits;
    const int sp = blockIdx.x % a.splits, g = (blockIdx.x / a.splits) % f.G;
    const long long slot = blockIdx.x / (a.splits * f.G);
    const int h_lo = g * hpg + min(sp * per, hpg), nh = g * hpg + min((sp + 1) * per, hpg) - h_lo, nu = nh * NX;
    int b, n;
    Seq sq;
    if (!find_slot(f.cu, f.B, f.T, kCT, slot, b, n, sq)) {
        if (a.dskip_part)
            for (int i = tid; i < nh; i += kNT) a.dskip_part[slot * f.H + h_lo + i] = 0.f;
        return;
    }
    const int t0 = n * kCT, len = min(kCT, sq.len - t0);
    const size_t grow = (size_t)(sq.row0 + t0);  // the chunk's first row
    const int mb = f.cu ? 0 : b, mt = (f.cu ? (int)sq.row0 : 0) + t0;
    const bool tail = f.cu && len < kCT;

    if (warp == kIssuer) tc::tmem_alloc(&tmem_slot, 512);
    if (tid == 0) {
        uint64_t *bars[] = {&ld_qk, &ldx[0], &ldx[1], &ld[0], &ld[1], &b_x, &b_q, &b_y, &b_c, &b_d, &b_z};
        for (uint64_t *x : bars) tc::mbar_init(x, 1);
        tc::mbar_init(&r_q, kNT / 32);
        tc::fence_mbar_init();
        waits_init(waits, a.f.wait_limit);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = tmem_slot, tl = tm + ((uint32_t)(32 * p) << 16);

    int nl = 0;
    auto load = [&](int u) {
        ++nl;
        if (!elect()) return;
        const int s = u & 1, h = h_lo + u / NX, x = u % NX;
        unsigned char *st = sm + L::ST0 + s * L::STAGE;
        tc::mbar_expect_tx(&ldx[s], 2 * L::VB);
        tc::tma_load_5d(st, &maps.v, 0, mt, x, h, mb, &ldx[s]);
        tc::tma_load_5d(st + L::VB, &maps.dO, 0, mt, x, h, mb, &ldx[s]);
        tc::mbar_expect_tx(&ld[s], 2 * L::SB);
        const size_t img = ((size_t)slot * f.H + h) * (N * P * 2) + (size_t)x * L::SB;
        tc::bulk_load(st + 2 * L::VB, static_cast<const unsigned char *>(a.grads) + img, L::SB, &ld[s]);
        tc::bulk_load(st + 2 * L::VB + L::SB, static_cast<const unsigned char *>(f.states) + img, L::SB, &ld[s]);
    };
    bool bad = false, aborted = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!wait_bar(bar, parity, &waits)) bad = true;
        __syncwarp();
    };
    auto handoff = [&]() {
        tc::fence_async_smem();
        tc::fence_before();
        aborted = __syncthreads_or(bad);
        tc::fence_after();
    };
    if (warp == kFinisher) {
        if (elect()) {
            tc::mbar_expect_tx(&ld_qk, 2 * L::QB);
            for (int x = 0; x < N / 64; ++x) {
                tc::tma_load_5d(sm + L::K + x * kCT * 128, &maps.k, 0, mt, x, g, mb, &ld_qk);
                tc::tma_load_5d(sm + L::Q + x * kCT * 128, &maps.q, 0, mt, x, g, mb, &ld_qk);
            }
        }
        if (nu > 0) load(0);
        if (nu > 1) load(1);
    }
    // the warps of the last sub-partition, which have the least of X, form the
    // decay factors, one head ahead
    bf16 g_la, g_dt;  // as loaded: nothing waits for them before they are used
    const int gt = p == 3 ? 32 * qc + lane : -1;
    auto load_gates = [&](int i) {
        g_la = g_dt = __ushort_as_bfloat16(0);
        if (i < nh && gt < len) {
            const size_t r = (grow + gt) * f.H + h_lo + i;
            g_la = static_cast<const bf16 *>(f.la)[r];
            g_dt = static_cast<const bf16 *>(f.dt)[r];
        }
    };
    if (gt >= 0) {
        load_gates(0);
        form_bwd_gates(gates[0], bounded_log(__bfloat162float(g_la)), __bfloat162float(g_dt), gt);
        load_gates(1);
    }
    for (int i = tid; i < 8 * kCT; i += kNT) (&rowp[0][0])[i] = 0.f;  // (rowp and colp: those of masked blocks stay zero)

    // ---- G^T = k q^T, kept as bf16 pairs in tensor memory
    wait(&ld_qk, 0);
    if (tail) {
        zero_tail(sm + L::K, N / 64, len, tid, kNT);
        zero_tail(sm + L::Q, N / 64, len, tid, kNT);
    }
    handoff();
    if (warp == kIssuer && elect()) {
        mma_tiles<true, true>(tm + cX, sm + L::K, kCT, sm + L::Q, kCT, N / 16, idX, false);
        tc::commit(&b_z);
    }
    wait(&b_z, 0);
    tc::fence_after();
    {
        float x[32];
        uint32_t u[16];
        tc::ld_32x32b_x32(tl + cX + 32 * qc, x);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = pack2(x[2 * i], x[2 * i + 1]);
        st16(tl + cG + 16 * qc, u);
        tc::wait_st();
    }
    handoff();

    float Z[32], es = 0.f, dsk = 0.f, rs = 0.f, us = 0.f;  // rs, us: r and u of the token `row`
#pragma unroll
    for (int i = 0; i < 32; ++i) Z[i] = 0.f;

    // dla_t = sum_{i >= t} (u_i + rowsum_i - dt_i colsum_i) + sum_{j < t} dt_j r_j + e^{L_end} <E, S>,
    // ddt_t = r_t + colsum_t + the diagonal, of head h_lo + hh: one warp, four tokens a lane
    float eall = 0.f, dall = 0.f;  // (kFinisher) e^{L_end} <E, S> and dskip's sum
    auto finish = [&](int hh) {
        const float4 x4 = *reinterpret_cast<const float4 *>(&fin[4 * lane]), y4 = *reinterpret_cast<const float4 *>(&fin[kCT + 4 * lane]);
        const float4 d4 = *reinterpret_cast<const float4 *>(&fin[2 * kCT + 4 * lane]);
        float sx = (x4.x + x4.y) + (x4.z + x4.w), sy = (y4.x + y4.y) + (y4.z + y4.w);
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const float px = __shfl_down_sync(0xffffffffu, sx, m), py = __shfl_up_sync(0xffffffffu, sy, m);
            if (lane + m < 32) sx += px;
            if (lane >= m) sy += py;
        }
        if (lane == 0 && a.dskip_part) a.dskip_part[slot * f.H + h_lo + hh] = dall;
        float after = __shfl_down_sync(0xffffffffu, sx, 1), before = __shfl_up_sync(0xffffffffu, sy, 1);
        if (lane == 31) after = 0.f;
        before = (lane == 0 ? 0.f : before) + eall;
        const float r3 = after + x4.w, r2 = r3 + x4.z, r1 = r2 + x4.y, r0 = r1 + x4.x;
        const float la[4] = {r0 + before, r1 + (before + y4.x), r2 + (before + y4.x + y4.y), r3 + (before + y4.x + y4.y + y4.z)};
        const float dd[4] = {d4.x, d4.y, d4.z, d4.w};
        const size_t at = (grow + 4 * lane) * f.H + h_lo + hh;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (4 * lane + e < len) {
                static_cast<bf16 *>(a.dla)[at + (size_t)e * f.H] = __float2bfloat16_rn(la[e]);
                static_cast<bf16 *>(a.ddt)[at + (size_t)e * f.H] = __float2bfloat16_rn(dd[e]);
            }
    };
    // X of a head, summed over its units (whose v and dO have landed)
    auto product_X = [&](int u) {
        if (!elect()) return;
        const unsigned char *v = sm + L::ST0 + (u & 1) * L::STAGE;
        mma_tiles<true, true>(tm + cX, v, kCT, v + L::VB, kCT, 4, idX, u % NX > 0);
        if (u % NX == NX - 1) tc::commit(&b_x);
    };
    auto product_R = [&](int u) {  // (lies where Y comes next)
        wait(&ld[u & 1], (uint32_t)(u >> 1) & 1u);
        if (!elect()) return;
        mma_tiles<true, false>(tm + cY, sm + L::Q, kCT, sm + L::ST0 + (u & 1) * L::STAGE + 2 * L::VB + L::SB, N, N / 16, idY, false);
        tc::commit(&b_q);
    };
    auto product_Y = [&](int u) {
        if (!elect()) return;
        mma_tiles<true, false>(tm + cY, sm + L::K, kCT, sm + L::ST0 + (u & 1) * L::STAGE + 2 * L::VB, N, N / 16, idY, false);
        tc::commit(&b_y);
    };
    if (warp == kIssuer && nu > 0) {
        if (!tail) {
            wait(&ldx[0], 0);
            product_X(0);
        }
        product_R(0);
    }
    for (int u = 0; u < nu && !aborted; ++u) {
        const int s = u & 1, hh = u / NX, x = u % NX, h = h_lo + hh;
        const uint32_t ph = u & 1, ph2 = (u >> 1) & 1;
        const BwdGates &G = gates[hh & 1];
        unsigned char *sV = sm + L::ST0 + s * L::STAGE, *sO = sV + L::VB, *sE = sO + L::VB, *sS = sE + L::SB;
        wait(&ldx[s], ph2);
        if (tail && x == 0) {
            if (NX > 1) wait(&ldx[1], ph2);
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                unsigned char *v = sm + L::ST0 + ((s + i) & 1) * L::STAGE;
                zero_tail(v, 1, len, tid, kNT);
                zero_tail(v + L::VB, 1, len, tid, kNT);
            }
            handoff();
            if (aborted) break;
            if (warp == kIssuer)
#pragma unroll
                for (int i = 0; i < NX; ++i) product_X(u + i);
        }
        wait(&ld[s], ph2);
        const float dtj = G.dt[row];
        if (x == 0 && u > 0) {  // the head before is summed up; its parts may be overwritten
            if (NX == 1) asm volatile("bar.sync 2, 512;\n" ::: "memory");
            else if (p == 3) asm volatile("bar.sync 1, 128;\n" ::: "memory");  // (the other warps wait for X, which comes after)
            if (warp == kFinisher) finish(hh - 1);  // (this warp has no part in X below)
        }
        if (!tail && NX > 1 && x == 0 && warp == kIssuer) {  // the rest of X
            wait(&ldx[1], ph2);
            product_X(u + 1);
        }
        // ---- R: token i = row, value columns 16 qc ..
        wait(&b_q, ph);
        tc::fence_after();
        {
            float r[16];
            ld16(tl + cY + 16 * qc, r);
            const float er = G.er[row];
            float d = 0.f;
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 o = *reinterpret_cast<const uint4 *>(sO + piece(kCT, row, 2 * qc + i));
                const uint32_t oe[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 oo = unpack2(oe[e]);
                    d = fmaf(r[8 * i + 2 * e], oo.x, fmaf(r[8 * i + 2 * e + 1], oo.y, d));
                }
            }
            us = fmaf(er, d, us);
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0 && u != f.withheld) tc::mbar_arrive(&r_q);
        if (warp == kIssuer) {  // (every warp has read R)
            wait(&r_q, ph);
            tc::fence_after();
            product_Y(u);
        }
        // <E, S> (the two images have one layout), by the warps with the least of X
        if (p >= 2) {
            const int t = (warp >> 2) * 64 + (p & 1) * 32 + lane;  // 0 .. 255
#pragma unroll 2
            for (int i = 0; i < L::SB / 16 / 256; ++i) {
                const uint4 e = reinterpret_cast<const uint4 *>(sE)[t + i * 256], y4 = reinterpret_cast<const uint4 *>(sS)[t + i * 256];
                const uint32_t ee[4] = {e.x, e.y, e.z, e.w}, tt[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 y = unpack2(ee[c]), z = unpack2(tt[c]);
                    es = fmaf(y.x, z.x, fmaf(y.y, z.y, es));
                }
            }
        }
        // ---- X of the head: token j = row, tokens i = 32 qc ..; (G D)^T over the columns read
        if (x == 0) {
            wait(&b_x, hh & 1);
            tc::fence_after();
        }
        if (x > 0) {
        } else if (qc < p) {
            const uint32_t z[16] = {0};
            st16(tl + cX + 32 * qc, z);
        } else {
            const bool dg = qc == p;  // the block on the diagonal
            const float lj = G.l[row];
            const float fj = dg ? 0.f : G.cf[row] * exp_ftz(qc - p == 1 ? 0.f : qc - p == 3 ? G.bs[1] + G.bs[2] : G.bs[p + 1]);
            const float *src = dg ? &G.l[32 * qc] : &G.lf[32 * qc];
            float2 col2 = make_float2(0.f, 0.f);
            float diag = 0.f;
            const float2 dt2 = make_float2(dtj, dtj);
#pragma unroll
            for (int c0 = 0; c0 < 32; c0 += 16) {
                float X[16], c[16];
                uint32_t gp[8];
#pragma unroll
                for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(&c[i]) = *reinterpret_cast<const float4 *>(src + c0 + i);
                ld16(tl + cX + 32 * qc + c0, X);
                ld8(tl + cG + 16 * qc + c0 / 2, gp);
                const int d = lane - c0;  // the diagonal's column
                if (dg) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) c[i] = exp_ftz(i >= d ? c[i] - lj : -INFINITY);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 t = __fmul2_rn(make_float2(c[i], c[i + 1]), make_float2(fj, fj));
                        c[i] = t.x;
                        c[i + 1] = t.y;
                    }
                }
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 gg = unpack2(gp[i / 2]), cc = make_float2(c[i], c[i + 1]);
                    const float2 x2 = __fmul2_rn(make_float2(X[i], X[i + 1]), cc), m = __fmul2_rn(gg, cc), w = __fmul2_rn(gg, x2);
                    const float2 z = __ffma2_rn(x2, dt2, make_float2(Z[c0 + i], Z[c0 + i + 1]));
                    Z[c0 + i] = z.x;
                    Z[c0 + i + 1] = z.y;
                    gp[i / 2] = pack2(m.x, m.y);
                    X[i] = w.x;
                    X[i + 1] = w.y;
                }
                st8(tl + cX + 32 * qc + c0 / 2, gp);
                if (dg) {  // the diagonal apart: it is in ddt, not in dla
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        diag += i == d ? X[i] : 0.f;
                        X[i] = i == d ? 0.f : X[i];
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float2 w = make_float2(X[i], X[i + 1]), t = __fmul2_rn(w, dt2);
                    col2 = __fadd2_rn(col2, w);
                    X[i] = t.x;
                    X[i + 1] = t.y;
                }
                const float sum = lane_sums16(X, lane);
                if ((lane & 1) == 0) rowp[p][32 * qc + c0 + (lane >> 1)] = sum;
            }
            colp[qc][row] = col2.x + col2.y;
            if (dg) cd[row] = diag;
        }
        {  // e^{L_i} dO_i, for dq: beside (G D)^T, over columns of X that this warp has read
            const float er = G.er[row];
            uint32_t eo[8];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 o = *reinterpret_cast<const uint4 *>(sO + piece(kCT, row, 2 * qc + i));
                const uint32_t oe[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 oo = unpack2(oe[e]);
                    eo[4 * i + e] = pack2(oo.x * er, oo.y * er);
                }
            }
            st8(tl + cX + 32 * qc + 16, eo);
        }
        // ---- Y: token j = row, value columns 16 qc ..  (v is overwritten: X, which has read it, was waited for above)
        wait(&b_y, ph);
        tc::fence_after();
        {
            float y[16];
            ld16(tl + cY + 16 * qc, y);
            const float w = G.wt[row], wd = w * dtj;
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t at = piece(kCT, row, 2 * qc + i);
                const uint4 v = *reinterpret_cast<const uint4 *>(sV + at), o = *reinterpret_cast<const uint4 *>(sO + at);
                uint32_t ve[4] = {v.x, v.y, v.z, v.w};
                const uint32_t oe[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 vv = unpack2(ve[e]), oo = unpack2(oe[e]);
                    const int c = 8 * i + 2 * e;
                    dsk = fmaf(vv.x, oo.x, fmaf(vv.y, oo.y, dsk));
                    y[c] *= w;
                    y[c + 1] *= w;
                    rs = fmaf(y[c], vv.x, fmaf(y[c + 1], vv.y, rs));
                    ve[e] = pack2(vv.x * wd, vv.y * wd);
                }
                *reinterpret_cast<uint4 *>(sV + at) = make_uint4(ve[0], ve[1], ve[2], ve[3]);
            }
            stw<16>(tl + cY + 16 * qc, y);
        }
        tc::wait_st();
        if (x == NX - 1) {
            const float e2 = warp_sum(es), d2 = warp_sum(dsk);
            if (lane == 0) {
                red[warp] = e2;
                red[16 + warp] = d2;
            }
            rp[qc][row] = rs;
            up[qc][row] = us;
            es = dsk = rs = us = 0.f;
        }
        if (x == 0 && gt >= 0) {
            form_bwd_gates(gates[(hh + 1) & 1], bounded_log(__bfloat162float(g_la)), __bfloat162float(g_dt), gt);
            load_gates(hh + 2);
        }
        if (warp == kFinisher && elect()) tc::bulk_wait_read();  // the dv tile of the unit before
        handoff();
        if (aborted) break;
        if (warp == kIssuer && elect()) {
            const uint64_t o0 = tct::mnmaj(sO, kCT, 0);
#pragma unroll
            for (int i = 0; i < kCT / 16; ++i)
                mma_ts(tm + cY, tm + cX + 32 * (i >> 1) + 8 * (i & 1), o0 + (tct::kstep_bytes<false>(kCT, i) >> 4), idY, true);
            tc::commit(&b_c);
            mma_tiles<true, true>(tm + cDK, sV, kCT, sE, N, 4, idN, u > 0);
            const uint64_t s0 = tct::kmaj(sS, N, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mma_ts(tm + cDQ, tm + cX + 32 * i + 16, s0 + (tct::kstep_bytes<true>(N, i) >> 4), idN, u > 0 || i > 0);
            tc::commit(&b_d);
        }
        wait(&b_c, ph);
        tc::fence_after();
        {  // dv
            float y[16];
            ld16(tl + cY + 16 * qc, y);
            const float skip = f.skip ? f.skip[h] : 0.f;
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t at = piece(kCT, row, 2 * qc + i);
                const uint4 o = *reinterpret_cast<const uint4 *>(sO + at);
                uint32_t oe[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 oo = unpack2(oe[e]);
                    const int c = 8 * i + 2 * e;
                    oe[e] = pack2(fmaf(dtj, y[c], skip * oo.x), fmaf(dtj, y[c + 1], skip * oo.y));
                }
                *reinterpret_cast<uint4 *>(sm + L::STG + at) = make_uint4(oe[0], oe[1], oe[2], oe[3]);
            }
        }
        if (warp == kIssuer) {
            wait(&b_d, ph);
            if (!tail && x == NX - 1 && u + 1 < nu) {  // the next X (the products that read (G D)^T and e^L dO are done)
                wait(&ldx[s ^ 1], (uint32_t)((u + 1) >> 1) & 1u);
                product_X(u + 1);
            }
        }
        handoff();
        if (aborted) break;
        if (warp == kIssuer && u + 1 < nu) product_R(u + 1);
        if (warp == kFinisher) {
            if (u + 2 < nu) load(u + 2);  // (the stage's products and reads are done)
            if (!tail && elect()) {
                tma_store_5d(&maps.dv, sm + L::STG, mt, x, h, mb);
                tc::bulk_commit();
            }
        }
        if (tail) {
            bf16 *dv = static_cast<bf16 *>(a.dv) + grow * f.ldv + (size_t)h * P + 64 * x;
            for (int i = tid; i < len * 8; i += kNT)
                *reinterpret_cast<uint4 *>(dv + (size_t)(i / 8) * f.ldv + 8 * (i % 8)) =
                    *reinterpret_cast<const uint4 *>(sm + L::STG + piece(kCT, i / 8, i % 8));
        }
        if (x == NX - 1 && p == 3) {  // the head's sums of token 32 qc + lane
            const int t = 32 * qc + lane;
            auto take = [&](const float(*part)[kCT]) { return (part[0][t] + part[1][t]) + (part[2][t] + part[3][t]); };
            const float ro = take(rowp), co = take(colp), r = take(rp), uu = take(up), dt = G.dt[t];
            fin[t] = uu + ro - dt * co;
            fin[kCT + t] = dt * r;
            fin[2 * kCT + t] = r + co + cd[t];
            if (warp == kFinisher) {
                eall = warp_sum(lane < 16 ? red[lane] : 0.f) * G.gamma;
                dall = warp_sum(lane < 16 ? red[16 + lane] : 0.f);
            }
        }
    }
    __syncthreads();
    if (!aborted && nu > 0 && warp == kFinisher) finish(nh - 1);

    // ---- dq += Z k, dk += Z^T q, and out.  Z in two bf16 parts: where the heads
    // of a group are cut into runs, each rounds its own Z, which may be far larger
    // than what the group's sum is (one part: dq off by a tenth of its norm where
    // pairs of heads cancel to a thirtieth).
    unsigned char *Zhi = sm + L::ST0, *Zlo = Zhi + kCT * kCT * 2;
    static_assert(2 * L::STAGE >= 2 * kCT * kCT * 2, "Z's parts lie over the stages");
    if (!aborted) {
        put_row<32>(Zhi, kCT, row, 32 * qc, Z);
#pragma unroll
        for (int i = 0; i < 32; ++i) Z[i] -= __bfloat162float(__float2bfloat16_rn(Z[i]));
        put_row<32>(Zlo, kCT, row, 32 * qc, Z);
    }
    handoff();
    if (!aborted) {
        if (warp == kIssuer && elect()) {
            mma_tiles<true, false>(tm + cDK, Zhi, kCT, sm + L::Q, kCT, kCT / 16, idZk, nu > 0);
            mma_tiles<true, false>(tm + cDK, Zlo, kCT, sm + L::Q, kCT, kCT / 16, idZk, true);
            mma_tiles<false, false>(tm + cDQ, Zhi, kCT, sm + L::K, kCT, kCT / 16, idZq, nu > 0);
            mma_tiles<false, false>(tm + cDQ, Zlo, kCT, sm + L::K, kCT, kCT / 16, idZq, true);
            tc::commit(&b_z);
        }
        wait(&b_z, 1);
        tc::fence_after();
        const size_t rows = f.cu ? (size_t)f.T : (size_t)f.B * f.T;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float t[WN];
            ldw<WN>(tl + (which ? cDK : cDQ) + WN * qc, t);
            tc::wait_ld();
            if (row < len) {
                if (a.splits == 1) {
                    bf16 *dst = which ? static_cast<bf16 *>(a.dk) + (grow + row) * f.ldk + (size_t)g * N + WN * qc
                                      : static_cast<bf16 *>(a.dq) + (grow + row) * f.ldq + (size_t)g * N + WN * qc;
#pragma unroll
                    for (int i = 0; i < WN; i += 8)
                        *reinterpret_cast<uint4 *>(dst + i) = make_uint4(pack2(t[i], t[i + 1]), pack2(t[i + 2], t[i + 3]),
                                                                         pack2(t[i + 4], t[i + 5]), pack2(t[i + 6], t[i + 7]));
                } else {
                    float *dst = a.dqk_part + (((size_t)(which * a.splits + sp) * rows + grow + row) * f.G + g) * N + WN * qc;
#pragma unroll
                    for (int i = 0; i < WN; i += 4)
                        *reinterpret_cast<float4 *>(dst + i) = make_float4(t[i], t[i + 1], t[i + 2], t[i + 3]);
                }
            }
        }
    }
    if (aborted && warp == kIssuer) {  // nothing is left in flight
        if (elect()) tc::commit(&b_z);
        (void)tc::mbar_wait(&b_z, 1);
    }
    if (warp == kFinisher) {
        if (elect()) tc::bulk_wait();
        for (int i = 0; i < 2 && i < nl; ++i) {
            (void)tc::mbar_wait(&ldx[i], ((nl - 1 - i) >> 1) & 1);
            (void)tc::mbar_wait(&ld[i], ((nl - 1 - i) >> 1) & 1);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (tid == 0 && waits.dead) record_status(f.status, GDN2_ERR_TIMEOUT);
    if (warp == kIssuer) {
        tc::fence_after();
        tc::tmem_dealloc(tm, 512);
    }
}

template <int N, int P>
cudaError_t bwd_np(const ScanBwdArgs &a, cudaStream_t s) {
    const ScanArgs &f = a.f;
    BwdMaps m;
    const int MB = f.cu ? 1 : f.B;
    if (!scan_tile_map(&m.q, f.q, f.ldq, MB, f.T, f.G, N) || !scan_tile_map(&m.k, f.k, f.ldk, MB, f.T, f.G, N) ||
        !scan_tile_map(&m.v, f.v, f.ldv, MB, f.T, f.H, P) || !scan_tile_map(&m.dv, a.dv, f.ldv, MB, f.T, f.H, P) ||
        !scan_tile_map(&m.dO, a.dO, (long long)f.H * P, MB, f.T, f.H, P))
        return cudaErrorInvalidValue;
    auto kernel = bwd_kernel<N, P>;
    constexpr int bytes = BwdTcSmem<N>::BYTES;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(slot_count(f.cu, f.B, f.T, kCT) * f.G * a.splits), kNT, bytes, s>>>(a, m);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan_bwd_tc(const ScanBwdArgs &a, int dk, int dv, cudaStream_t s) {
    cudaError_t e = launch_scan_grads_tc(a, dk, dv, s);
    if (e != cudaSuccess) return e;
    if (dk == 128) e = dv == 128 ? bwd_np<128, 128>(a, s) : bwd_np<128, 64>(a, s);
    else e = dv == 128 ? bwd_np<64, 128>(a, s) : bwd_np<64, 64>(a, s);
    return e != cudaSuccess ? e : launch_grad_sums(a, dk, true, kCT, s);
}

}  // namespace ssm
}  // namespace gdn2
