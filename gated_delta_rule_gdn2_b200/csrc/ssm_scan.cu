// The selective state space scan and its backward in fp32 arithmetic.
//
// Forward: S_t = a_t S_{t-1} + dt_t k_t v_t^T, o_t = S_t^T q_t + skip v_t
// (a_t = e^{la_t}).  Backward: with E_t the gradient that reaches S_t from the
// tokens after t,
//     dS_t = E_t + q_t do_t^T,  E_{t-1} = a_t dS_t,
// and in a chunk of 64 tokens, L_i = la_0 + .. + la_i from its start, S the
// state at its start, E the gradient at its end, w_j = e^{L_end - L_j},
// D_ij = e^{L_i - L_j} (i >= j, else 0), Z_ij = (do_i . v_j) D_ij dt_j,
//     dv_j = dt_j (w_j E^T k_j + sum_i (q_i . k_j) D_ij do_i) + skip do_j
//     dk_j = dt_j w_j E v_j + sum_i Z_ij q_i     (summed over the group's heads)
//     dq_i = e^{L_i} S do_i + sum_j Z_ij k_j     (summed over the group's heads)
//     ddt_j = w_j k_j . E v_j + sum_i (q_i . k_j) Z_ij / dt_j
//     dla_t = sum_{i >= t} e^{L_i} q_i . S do_i + sum_{i >= t > j} (q_i . k_j) Z_ij
//             + sum_{j < t} dt_j w_j k_j . E v_j + e^{L_end} <E, S>.
// The double sum over i >= t > j is the running sum from the chunk's end of
// (row sum - column sum) of the strictly lower part: both sums are taken from
// the same fp32 products, so their difference loses nothing to rounding of
// operands.
//
// Two kernels.  The recurrent one walks tokens with the state in registers (a
// warp holds all dk rows of 16 value columns, 8 x 4 lanes of (dk / 8) x 4
// entries; q, k, v of 16 tokens at a time in shared memory, loaded one step
// ahead) and serves the forward and, run from the end, the chain of E.  It is
// bound by the fp32 pipe: 3 dk dv operations per token and head (2 on packed
// pairs).  Few long sequences are cut into parts that run side by side: a
// first launch leaves each part's state from zero, the second starts each
// part from those before it.  The chunk kernel takes one chunk of one group,
// heads one after the other, so that dq and dk are summed over the heads in
// registers, in a fixed order.
#include "common.cuh"
#include "gdn2.h"
#include "ssm.h"

namespace gdn2 {
namespace ssm {
namespace {

constexpr int kTok = 16;  // tokens staged at a time by the recurrent kernel

__device__ __forceinline__ void cp16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// REV == false: forward; true: the chain of E (k = q, v = dO, dt = 1, no o),
// walked from the end.  LOCAL: a part's state from zero, to part_state.
struct RecArgs {
    const float *q, *k, *v, *la, *dt, *skip;
    const float *start;       // state before the first token walked ([B][H][N][P] or nullptr)
    float *o, *end, *states;  // end: the state after the last token walked
    long long ldq, ldk, ldv;
    int ldh;                  // elements between the heads of v
    const int *cu;
    int B, T, H, G, parts;
    float *part_state, *part_decay;
    int *status;
};

template <int N, int P, bool REV, bool LOCAL>
__global__ void __launch_bounds__(128) rec_kernel(RecArgs a) {
    constexpr int U = N / 32;  // blocks of 32 state rows, 4 of each in this thread
    __shared__ __align__(16) float s_k[2][kTok][N], s_q[2][REV || LOCAL ? 1 : kTok][N], s_v[2][kTok][64];
    __shared__ float s_a[2][kTok], s_d[2][kTok];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ng = lane >> 2, pg = lane & 3;
    const int np = LOCAL ? a.parts - 1 : a.parts;
    const int bh = blockIdx.x / np, part = blockIdx.x % np + (LOCAL && REV ? 1 : 0);
    const int b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G), c0 = blockIdx.y * 64, pc = c0 + warp * 16 + pg * 4;
    const Seq sq = seq_of(a.cu, b, a.T, kC);
    if (!sq.ok) {
        if (tid == 0) record_status(a.status, GDN2_ERR_INVALID_ARG);
        return;
    }
    const int cpp = (sq.nchunks + a.parts - 1) / a.parts;
    const int t_lo = min(part * cpp * kC, sq.len), t_hi = min((part + 1) * cpp * kC, sq.len);
    constexpr size_t SE = (size_t)N * P;

    float2 S[U * 4][2];
    auto rowoff = [&](int i) { return (size_t)(32 * (i >> 2) + 4 * ng + (i & 3)) * P + pc; };
    if (LOCAL || !a.start) {
#pragma unroll
        for (int i = 0; i < U * 4; ++i) S[i][0] = S[i][1] = make_float2(0.f, 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < U * 4; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(a.start + bh * SE + rowoff(i));
            S[i][0] = make_float2(x.x, x.y);
            S[i][1] = make_float2(x.z, x.w);
        }
    }
    if (!LOCAL) {  // the parts walked before this one
        for (int s = REV ? a.parts - 1 : 0; s != part; s += REV ? -1 : 1) {
            const size_t at = (size_t)bh * (a.parts - 1) + (REV ? s - 1 : s);
            const float d = a.part_decay[at];
            const float2 d2 = make_float2(d, d);
#pragma unroll
            for (int i = 0; i < U * 4; ++i) {
                const float4 x = *reinterpret_cast<const float4 *>(a.part_state + at * SE + rowoff(i));
                S[i][0] = __ffma2_rn(S[i][0], d2, make_float2(x.x, x.y));
                S[i][1] = __ffma2_rn(S[i][1], d2, make_float2(x.z, x.w));
            }
        }
    }

    const int ntile = (t_hi - t_lo + kTok - 1) / kTok;
    const float *kb = a.k + sq.row0 * a.ldk + (size_t)g * N, *vb = a.v + sq.row0 * a.ldv + (size_t)h * a.ldh + c0;
    const float *qb = REV || LOCAL ? nullptr : a.q + sq.row0 * a.ldq + (size_t)g * N;
    auto load = [&](int it) {  // tile `it` of the walk (tokens past the end are not read)
        const int tile = REV ? ntile - 1 - it : it, t0 = t_lo + tile * kTok, n = min(kTok, t_hi - t0), st = it & 1;
        for (int i = tid; i < n * (N / 4); i += 128) {
            const int t = i / (N / 4), c = (i % (N / 4)) * 4;
            cp16(&s_k[st][t][c], kb + (t0 + t) * a.ldk + c);
            if (!REV && !LOCAL) cp16(&s_q[st][t][c], qb + (t0 + t) * a.ldq + c);
        }
        for (int i = tid; i < n * 16; i += 128) {
            const int t = i / 16, c = (i % 16) * 4;
            cp16(&s_v[st][t][c], vb + (t0 + t) * a.ldv + c);
        }
        if (tid < n) {
            const size_t r = (size_t)(sq.row0 + t0 + tid) * a.H + h;
            s_a[st][tid] = a.la[r];
            s_d[st][tid] = REV ? 1.f : a.dt[r];
        }
        cp_commit();
    };
    double sum_la = 0.;  // (LOCAL: the part's decay)
    const float skip = !REV && !LOCAL && a.skip ? a.skip[h] : 0.f;
    if (ntile > 0) load(0);
    for (int it = 0; it < ntile; ++it) {
        if (it + 1 < ntile) {
            load(it + 1);
            cp_wait<1>();
        } else {
            cp_wait<0>();
        }
        __syncthreads();
        const int st = it & 1, tile = REV ? ntile - 1 - it : it, t0 = t_lo + tile * kTok, n = min(kTok, t_hi - t0);
        // a chunk's first token (REV: its last) comes next: keep the state
        const int edge = REV ? (t0 + n) % kC == 0 || t0 + n == sq.len : t0 % kC == 0;
        if (!LOCAL && a.states && edge) {
            float *dst = a.states + ((size_t)(sq.slot + (REV ? (t0 + n - 1) / kC : t0 / kC)) * a.H + h) * SE;
#pragma unroll
            for (int i = 0; i < U * 4; ++i)
                *reinterpret_cast<float4 *>(dst + rowoff(i)) = make_float4(S[i][0].x, S[i][0].y, S[i][1].x, S[i][1].y);
        }
        // (tokens side by side, as far as the registers go: 2 x 1000 tokens, 8 heads of
        // 64, in parts of 64 tokens: 32 -> 27 us with o, 20 -> 19 the gradients' chain)
#pragma unroll(REV || LOCAL ? 4 : 2)
        for (int x = 0; x < n; ++x) {
            const int t = REV ? n - 1 - x : x;
            const float la = s_a[st][t], al = expf(la), dt = s_d[st][t];
            const float2 a2 = make_float2(al, al);
            const float4 v = *reinterpret_cast<const float4 *>(&s_v[st][t][warp * 16 + pg * 4]);
            const float2 v0 = make_float2(v.x * dt, v.y * dt), v1 = make_float2(v.z * dt, v.w * dt);
            if (LOCAL) sum_la += la;
            float2 y0 = make_float2(0.f, 0.f), y1 = y0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float4 k4 = *reinterpret_cast<const float4 *>(&s_k[st][t][32 * u + 4 * ng]);
                float4 q4 = make_float4(0.f, 0.f, 0.f, 0.f);
                if (!REV && !LOCAL) q4 = *reinterpret_cast<const float4 *>(&s_q[st][t][32 * u + 4 * ng]);
                const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 *s = S[4 * u + e];
                    const float2 k2 = make_float2(kk[e], kk[e]), q2 = make_float2(qq[e], qq[e]);
                    if (REV) {
                        s[0] = __fmul2_rn(__ffma2_rn(k2, v0, s[0]), a2);
                        s[1] = __fmul2_rn(__ffma2_rn(k2, v1, s[1]), a2);
                    } else {
                        s[0] = __ffma2_rn(s[0], a2, __fmul2_rn(k2, v0));
                        s[1] = __ffma2_rn(s[1], a2, __fmul2_rn(k2, v1));
                        if (!LOCAL) {
                            y0 = __ffma2_rn(q2, s[0], y0);
                            y1 = __ffma2_rn(q2, s[1], y1);
                        }
                    }
                }
            }
            if (!REV && !LOCAL && a.o) {
#pragma unroll
                for (int m = 4; m < 32; m <<= 1) {
                    y0.x += __shfl_xor_sync(0xffffffffu, y0.x, m);
                    y0.y += __shfl_xor_sync(0xffffffffu, y0.y, m);
                    y1.x += __shfl_xor_sync(0xffffffffu, y1.x, m);
                    y1.y += __shfl_xor_sync(0xffffffffu, y1.y, m);
                }
                if (ng == 0)
                    *reinterpret_cast<float4 *>(a.o + ((size_t)(sq.row0 + t0 + t) * a.H + h) * P + pc) =
                        make_float4(fmaf(skip, v.x, y0.x), fmaf(skip, v.y, y0.y), fmaf(skip, v.z, y1.x),
                                    fmaf(skip, v.w, y1.y));
            }
        }
        __syncthreads();
    }

    const bool last = REV ? part == 0 : part == a.parts - 1;
    float *dst = LOCAL ? a.part_state + ((size_t)bh * (a.parts - 1) + (REV ? part - 1 : part)) * SE
                       : (last && a.end ? a.end + bh * SE : nullptr);
    if (dst)
#pragma unroll
        for (int i = 0; i < U * 4; ++i)
            *reinterpret_cast<float4 *>(dst + rowoff(i)) = make_float4(S[i][0].x, S[i][0].y, S[i][1].x, S[i][1].y);
    if (LOCAL && tid == 0 && blockIdx.y == 0)
        a.part_decay[(size_t)bh * (a.parts - 1) + (REV ? part - 1 : part)] = (float)exp(sum_la);
}

template <bool REV>
cudaError_t launch_rec(const RecArgs &a, int dk, int dv, cudaStream_t s) {
    auto go = [&](auto n, auto p) {
        constexpr int N = decltype(n)::value, P = decltype(p)::value;
        const unsigned bh = (unsigned)(a.B * a.H);
        if (a.parts > 1) rec_kernel<N, P, REV, true><<<dim3(bh * (a.parts - 1), P / 64), 128, 0, s>>>(a);
        rec_kernel<N, P, REV, false><<<dim3(bh * a.parts, P / 64), 128, 0, s>>>(a);
        return cudaGetLastError();
    };
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    if (dk == 128) return dv == 128 ? go(I128{}, I128{}) : go(I128{}, I64{});
    return dv == 128 ? go(I64{}, I128{}) : go(I64{}, I64{});
}

// ---------------------------------------------------------------------------
// One chunk of one group, head after head.  256 threads as 16 x 16: thread
// (ti, tj) holds rows ti + 16 r (r < 4) and, of a 64-column Gram matrix,
// columns tj + 16 c; of a D-column product, columns 4 tj + 64 u .. + 3.
// Shared rows are padded by four floats, so that 16-byte reads of consecutive
// rows fall on different banks.

template <int N, int P>
struct BwdSmem {
    static constexpr int LN = N + 4, LP = P + 4, LG = 68;
    static constexpr int Q = 0, K = Q + 64 * LN, V = K + 64 * LN, O = V + 64 * LP, S = O + 64 * LP, M = S + N * LP,
                         LAM = M + 64 * LG, LML = LAM + 64, LSU = LML + 64, BS = LSU + 64, DT = BS + 4, RS = DT + 64, CSP = RS + 64, R = CSP + 8 * 64, UU = R + 64,
                         CD = UU + 64, RED = CD + 64, END = RED + 16;
    static constexpr size_t BYTES = sizeof(float) * END;
};

__device__ __forceinline__ float dot4(float4 a, float4 b, float acc) {
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, acc))));
}
__device__ __forceinline__ float half_sum(float x) {  // over the 16 lanes of one ti
#pragma unroll
    for (int m = 8; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// acc[r][c] (+)= A[ti + 16 r] . B[tj + 16 c] over D columns
template <int D>
__device__ __forceinline__ void gram(const float *A, const float *B, int ti, int tj, float (&acc)[4][4]) {
    constexpr int L = D + 4;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = 0.f;
#pragma unroll 2
    for (int d = 0; d < D; d += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            x[r] = *reinterpret_cast<const float4 *>(A + (ti + 16 * r) * L + d);
            y[r] = *reinterpret_cast<const float4 *>(B + (tj + 16 * r) * L + d);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[r][c] = dot4(x[r], y[c], acc[r][c]);
    }
}

// acc[r][4 u + e] += sum_x A(x, row) B[x][4 tj + 64 u + e], x < X.  TRANS:
// A(x, row) = A[x][row], else A[row][x].
template <int X, int D, bool TRANS, int LA>
__device__ __forceinline__ void prod(const float *A, const float *B, int ti, int tj, float (&acc)[4][D / 16]) {
    constexpr int LB = D + 4;
#pragma unroll 2
    for (int x0 = 0; x0 < X; x0 += 4) {
        float w[4][4];  // [r][x]
        if (!TRANS) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 t = *reinterpret_cast<const float4 *>(A + (ti + 16 * r) * LA + x0);
                w[r][0] = t.x; w[r][1] = t.y; w[r][2] = t.z; w[r][3] = t.w;
            }
        } else {
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int r = 0; r < 4; ++r) w[r][x] = A[(x0 + x) * LA + ti + 16 * r];
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                const float4 y = *reinterpret_cast<const float4 *>(B + (x0 + x) * LB + 4 * tj + 64 * u);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    acc[r][4 * u] = fmaf(w[r][x], y.x, acc[r][4 * u]);
                    acc[r][4 * u + 1] = fmaf(w[r][x], y.y, acc[r][4 * u + 1]);
                    acc[r][4 * u + 2] = fmaf(w[r][x], y.z, acc[r][4 * u + 2]);
                    acc[r][4 * u + 3] = fmaf(w[r][x], y.w, acc[r][4 * u + 3]);
                }
            }
    }
}

// acc[r][4 u + e] = A[ti + 16 r] . B[4 tj + 64 u + e] over X columns (both
// operands' rows along the sum; B's rows are 4 tj + e, so their banks repeat
// every second tj: half rate, taken for the simpler output layout)
template <int X, int D>
__device__ __forceinline__ void prod_nt(const float *A, const float *B, int ti, int tj, float (&acc)[4][D / 16]) {
    constexpr int L = X + 4;
#pragma unroll 1
    for (int d = 0; d < X; d += 4) {
        float4 x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = *reinterpret_cast<const float4 *>(A + (ti + 16 * r) * L + d);
#pragma unroll
        for (int u = 0; u < D / 64; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 y = *reinterpret_cast<const float4 *>(B + (4 * tj + 64 * u + e) * L + d);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r][4 * u + e] = dot4(x[r], y, acc[r][4 * u + e]);
            }
    }
}

// (dk = dv = 64: two blocks an SM, at 128 registers a thread instead of 214; 8 x
// 4096 tokens, 16 heads: 1763 -> 1242 us.  The larger ones' tiles fill an SM.)
template <int N, int P>
__global__ void __launch_bounds__(256, N + P == 128 ? 2 : 1) chunk_bwd_kernel(ScanBwdArgs a) {
    using L = BwdSmem<N, P>;
    extern __shared__ __align__(16) float sm[];
    float *sQ = sm + L::Q, *sK = sm + L::K, *sV = sm + L::V, *sO = sm + L::O, *sS = sm + L::S, *sM = sm + L::M;
    float *lam = sm + L::LAM, *lml = sm + L::LML, *lsu = sm + L::LSU, *bs = sm + L::BS, *sdt = sm + L::DT, *rs = sm + L::RS, *csp = sm + L::CSP, *sr = sm + L::R, *su = sm + L::UU,
          *cd = sm + L::CD, *red = sm + L::RED;
    const ScanArgs &f = a.f;
    const int tid = threadIdx.x, ti = tid >> 4, tj = tid & 15, warp = tid >> 5;
    const int hpg = f.H / f.G, per = (hpg + a.splits - 1) / a.splits;
    const int sp = blockIdx.x % a.splits, g = (blockIdx.x / a.splits) % f.G;
    const long long slot = blockIdx.x / ((long long)a.splits * f.G);
    const int h_lo = g * hpg + min(sp * per, hpg), h_hi = g * hpg + min((sp + 1) * per, hpg);
    int b, n;
    Seq sq;
    if (!find_slot(f.cu, f.B, f.T, kC, slot, b, n, sq)) {
        if (a.dskip_part)
            for (int h = h_lo + tid; h < h_hi; h += 256) a.dskip_part[slot * f.H + h] = 0.f;
        return;
    }
    const int t0 = n * kC, len = min(kC, sq.len - t0);
    const size_t row = (size_t)(sq.row0 + t0);
    constexpr size_t SE = (size_t)N * P;
    auto load = [&](float *dst, const float *src, long long ld, int D) {  // rows past the chunk's end read as zero
        for (int i = tid; i < 64 * (D / 4); i += 256) {
            const int t = i / (D / 4), c = (i % (D / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < len) x = *reinterpret_cast<const float4 *>(src + (size_t)t * ld + c);
            *reinterpret_cast<float4 *>(dst + t * (D + 4) + c) = x;
        }
    };
    load(sQ, static_cast<const float *>(f.q) + row * f.ldq + (size_t)g * N, f.ldq, N);
    load(sK, static_cast<const float *>(f.k) + row * f.ldk + (size_t)g * N, f.ldk, N);
    __syncthreads();
    float G[4][4], Z[4][4];
    gram<N>(sQ, sK, ti, tj, G);
    float dq[4][N / 16], dk[4][N / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int c = 0; c < 4; ++c) Z[r][c] = 0.f;
#pragma unroll
        for (int c = 0; c < N / 16; ++c) dq[r][c] = dk[r][c] = 0.f;
    }

    for (int h = h_lo; h < h_hi; ++h) {
        load(sV, static_cast<const float *>(f.v) + row * f.ldv + (size_t)h * P, f.ldv, P);
        load(sO, static_cast<const float *>(a.dO) + (row * f.H + h) * P, (long long)f.H * P, P);
        const float *E = static_cast<const float *>(a.grads) + ((size_t)slot * f.H + h) * SE;
        const float *S = static_cast<const float *>(f.states) + ((size_t)slot * f.H + h) * SE;
        for (int i = tid; i < N * (P / 4); i += 256)
            *reinterpret_cast<float4 *>(sS + i / (P / 4) * L::LP + (i % (P / 4)) * 4) =
                reinterpret_cast<const float4 *>(E)[i];
        if (tid < 32) {
            // log decays by blocks of 16 tokens, two tokens a lane: lam = the sum
            // from the block's start through the token, lsu = from behind it to the
            // block's end, bs = the block's.  An exponent L_i - L_j across blocks
            // is then a sum of terms <= 0, which loses nothing where a chunk
            // decays far.  Within a block it is a difference of prefix sums, and
            // behind a run of resets (kLogMin each) both are in the thousands: the
            // prefix sums are formed in 64 bits and kept in two parts, lam + lml.
            const int t = 2 * tid;
            const size_t r = (row + t) * f.H + h;
            const float *la = static_cast<const float *>(f.la), *dt = static_cast<const float *>(f.dt);
            const float x0 = t < len ? bounded_log(la[r]) : 0.f, x1 = t + 1 < len ? bounded_log(la[r + f.H]) : 0.f;
            double up = (double)x0 + x1;
            float dn = x0 + x1;
#pragma unroll
            for (int m = 1; m < 8; m <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, up, m, 8);
                const float z = __shfl_down_sync(0xffffffffu, dn, m, 8);
                if ((tid & 7) >= m) up += y;
                if ((tid & 7) + m < 8) dn += z;
            }
            const float after = __shfl_down_sync(0xffffffffu, dn, 1, 8);
            const double before = __shfl_up_sync(0xffffffffu, up, 1, 8), first = ((tid & 7) ? before : 0.) + x0;
            lam[t] = (float)first;
            lml[t] = (float)(first - lam[t]);
            lam[t + 1] = (float)up;
            lml[t + 1] = (float)(up - lam[t + 1]);
            lsu[t + 1] = (tid & 7) < 7 ? after : 0.f;
            lsu[t] = lsu[t + 1] + x1;
            if ((tid & 7) == 7) bs[tid >> 3] = (float)up;
            sdt[t] = t < len ? dt[r] : 0.f;
            sdt[t + 1] = t + 1 < len ? dt[r + f.H] : 0.f;
        }
        __syncthreads();
        // per block of 16: the log decay before it and behind it
        const float b0 = bs[0], b1 = bs[1], b2 = bs[2], b3 = bs[3];
        const float pre[4] = {0.f, b0, b0 + b1, b0 + b1 + b2}, post[4] = {b1 + b2 + b3, b2 + b3, b3, 0.f};
        const float Lend = b0 + post[0], skip = f.skip ? f.skip[h] : 0.f;

        // A_ij = (q_i . k_j) D_ij to shared memory; Z; row and column sums of W_ij = A_ij (do_i . v_j) dt_j
        {
            float X[4][4];
            gram<P>(sO, sV, ti, tj, X);
            float rsum[4] = {0.f, 0.f, 0.f, 0.f}, csum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int i = ti + 16 * r, j = tj + 16 * c;
                    // (r, c: the blocks of i and j)
                    const float mid = r == 2 && c == 0 ? b1 : r == 3 && c == 1 ? b2 : r == 3 && c == 0 ? b1 + b2 : 0.f;
                    const float D = r > c ? expf(lam[i] + mid + lsu[j]) : r == c && i >= j ? expf((lam[i] - lam[j]) + (lml[i] - lml[j])) : 0.f;
                    const float x = X[r][c] * D, dtj = sdt[j], w = G[r][c] * x;
                    sM[i * L::LG + j] = G[r][c] * D;
                    Z[r][c] = fmaf(x, dtj, Z[r][c]);
                    if (i > j) {
                        rsum[r] = fmaf(w, dtj, rsum[r]);
                        csum[c] += w;
                    }
                }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                rsum[r] = half_sum(rsum[r]);
                if (tj == 0) rs[ti + 16 * r] = rsum[r];
                // columns (without dt): the two ti of a warp, then the warps in order below
                csum[r] += __shfl_xor_sync(0xffffffffu, csum[r], 16);
                if ((tid & 16) == 0) csp[warp * 64 + tj + 16 * r] = csum[r];
            }
            // the diagonal of A_ij (do_i . v_j): thread ti == tj holds entries (ti + 16 r, ti + 16 r)
            if (ti == tj)
#pragma unroll
                for (int r = 0; r < 4; ++r) cd[ti + 16 * r] = G[r][r] * X[r][r];
        }
        __syncthreads();

        // dv_j and r_j = w_j k_j . E v_j
        {
            float acc[4][P / 16];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < P / 16; ++c) acc[r][c] = 0.f;
            prod<N, P, false, L::LN>(sK, sS, ti, tj, acc);
            float dsk = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = ti + 16 * r;
                const float w = expf(lsu[j] + post[r]);
                float d = 0.f;
#pragma unroll
                for (int u = 0; u < P / 64; ++u) {
                    const float4 v = *reinterpret_cast<const float4 *>(sV + j * L::LP + 4 * tj + 64 * u);
                    const float4 o = *reinterpret_cast<const float4 *>(sO + j * L::LP + 4 * tj + 64 * u);
                    dsk = dot4(v, o, dsk);
                    acc[r][4 * u] *= w; acc[r][4 * u + 1] *= w; acc[r][4 * u + 2] *= w; acc[r][4 * u + 3] *= w;
                    d = dot4(v, make_float4(acc[r][4 * u], acc[r][4 * u + 1], acc[r][4 * u + 2], acc[r][4 * u + 3]), d);
                }
                d = half_sum(d);
                if (tj == 0) sr[j] = d;
            }
            dsk = warp_sum(dsk);
            if ((tid & 31) == 0) red[warp] = dsk;
            prod<64, P, true, L::LG>(sM, sO, ti, tj, acc);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = ti + 16 * r;
                if (j >= len) continue;
                const float dtj = sdt[j];
                float *dst = static_cast<float *>(a.dv) + (row + j) * f.ldv + (size_t)h * P;
#pragma unroll
                for (int u = 0; u < P / 64; ++u) {
                    const float4 o = *reinterpret_cast<const float4 *>(sO + j * L::LP + 4 * tj + 64 * u);
                    *reinterpret_cast<float4 *>(dst + 4 * tj + 64 * u) =
                        make_float4(fmaf(dtj, acc[r][4 * u], skip * o.x), fmaf(dtj, acc[r][4 * u + 1], skip * o.y),
                                    fmaf(dtj, acc[r][4 * u + 2], skip * o.z), fmaf(dtj, acc[r][4 * u + 3], skip * o.w));
                }
            }
        }
        // dk_j += dt_j w_j E v_j
        {
            float acc[4][N / 16];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < N / 16; ++c) acc[r][c] = 0.f;
            prod_nt<P, N>(sV, sS, ti, tj, acc);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = ti + 16 * r;
                const float w = sdt[j] * expf(lsu[j] + post[r]);
#pragma unroll
                for (int c = 0; c < N / 16; ++c) dk[r][c] = fmaf(w, acc[r][c], dk[r][c]);
            }
        }
        __syncthreads();
        if (tid == 0 && a.dskip_part) {
            float s = 0.f;
            for (int w = 0; w < 8; ++w) s += red[w];
            a.dskip_part[slot * f.H + h] = s;
        }
        // <E, S>, and S over E in shared memory
        float es = 0.f;
        for (int i = tid; i < N * (P / 4); i += 256) {
            float4 *p = reinterpret_cast<float4 *>(sS + i / (P / 4) * L::LP + (i % (P / 4)) * 4);
            const float4 s = reinterpret_cast<const float4 *>(S)[i];
            es = dot4(*p, s, es);
            *p = s;
        }
        es = warp_sum(es);
        if ((tid & 31) == 0) red[8 + warp] = es;
        __syncthreads();
        // dq_i += e^{L_i} S do_i and u_i = e^{L_i} q_i . S do_i
        {
            float acc[4][N / 16];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < N / 16; ++c) acc[r][c] = 0.f;
            prod_nt<P, N>(sO, sS, ti, tj, acc);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = ti + 16 * r;
                const float w = expf(pre[r] + lam[i]);
                float d = 0.f;
#pragma unroll
                for (int u = 0; u < N / 64; ++u) {
                    const float4 q = *reinterpret_cast<const float4 *>(sQ + i * L::LN + 4 * tj + 64 * u);
                    d = dot4(q, make_float4(acc[r][4 * u], acc[r][4 * u + 1], acc[r][4 * u + 2], acc[r][4 * u + 3]), d);
                }
                d = half_sum(d);
                if (tj == 0) su[i] = w * d;
#pragma unroll
                for (int c = 0; c < N / 16; ++c) dq[r][c] = fmaf(w, acc[r][c], dq[r][c]);
            }
        }
        __syncthreads();
        if (tid < 32) {
            // dla_t = sum_{i >= t} (u_i + rowsum_i - dt_i colsum_i) + sum_{j < t} dt_j r_j + e^{L_end} <E, S>:
            // lane l takes tokens 2 l, 2 l + 1
            float es_all = 0.f;
            for (int w = 0; w < 8; ++w) es_all += red[8 + w];
            es_all *= expf(Lend);
            float col[2], x[2], y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * tid + e;
                col[e] = 0.f;
                for (int w = 0; w < 8; ++w) col[e] += csp[w * 64 + t];
                x[e] = su[t] + rs[t] - sdt[t] * col[e];
                y[e] = sdt[t] * sr[t];
            }
            float sx = x[0] + x[1], sy = y[0] + y[1];
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const float px = __shfl_down_sync(0xffffffffu, sx, m), py = __shfl_up_sync(0xffffffffu, sy, m);
                if (tid + m < 32) sx += px;
                if (tid >= m) sy += py;
            }
            const float before = sy - y[0] - y[1];
            const size_t r = (row + 2 * tid) * f.H + h;
            float *dla = static_cast<float *>(a.dla), *ddt = static_cast<float *>(a.ddt);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * tid + e;
                if (t >= len) continue;
                dla[r + e * f.H] = (e ? sx - x[0] : sx) + (e ? before + y[0] : before) + es_all;
                ddt[r + e * f.H] = sr[t] + col[e] + cd[t];
            }
        }
        __syncthreads();
    }

    // the Gram terms of dq and dk
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) sM[(ti + 16 * r) * L::LG + tj + 16 * c] = Z[r][c];
    __syncthreads();
    prod<64, N, false, L::LG>(sM, sK, ti, tj, dq);
    prod<64, N, true, L::LG>(sM, sQ, ti, tj, dk);
    const size_t rows = f.cu ? (size_t)f.T : (size_t)f.B * f.T;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = ti + 16 * r;
        if (i >= len) continue;
        float *oq, *ok;
        if (a.splits == 1) {
            oq = static_cast<float *>(a.dq) + (row + i) * f.ldq + (size_t)g * N;
            ok = static_cast<float *>(a.dk) + (row + i) * f.ldk + (size_t)g * N;
        } else {
            oq = a.dqk_part + (((size_t)sp * rows + row + i) * f.G + g) * N;
            ok = oq + (size_t)a.splits * rows * f.G * N;
        }
#pragma unroll
        for (int u = 0; u < N / 64; ++u) {
            *reinterpret_cast<float4 *>(oq + 4 * tj + 64 * u) =
                make_float4(dq[r][4 * u], dq[r][4 * u + 1], dq[r][4 * u + 2], dq[r][4 * u + 3]);
            *reinterpret_cast<float4 *>(ok + 4 * tj + 64 * u) =
                make_float4(dk[r][4 * u], dk[r][4 * u + 1], dk[r][4 * u + 2], dk[r][4 * u + 3]);
        }
    }
}

// dq, dk from the splits' sums, added in order; one row a block.
template <typename T>
__global__ void qk_reduce_kernel(ScanBwdArgs a, int N) {
    const ScanArgs &f = a.f;
    const long long row = blockIdx.x;
    const size_t rows = gridDim.x, W = (size_t)f.G * N;
    if (f.cu) {  // rows of no sequence are left as they are
        int lo = 0, hi = f.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (f.cu[mid] <= row) lo = mid; else hi = mid - 1;
        }
        const Seq s = seq_of(f.cu, lo, f.T, 1);
        if (!s.ok || row < s.row0 || row >= s.row0 + s.len) return;
    }
    for (int c = threadIdx.x; c < 2 * (int)W; c += blockDim.x) {
        const int which = c >= (int)W, x = which ? c - (int)W : c;
        const float *p = a.dqk_part + ((size_t)which * a.splits * rows + row) * W + x;
        float s = 0.f;
        for (int i = 0; i < a.splits; ++i) s += p[(size_t)i * rows * W];
        (which ? static_cast<T *>(a.dk) + row * f.ldk : static_cast<T *>(a.dq) + row * f.ldq)[x] = from_f32<T>(s);
    }
}

// dskip[h] = the sum over the slots, by one block a head.
__global__ void dskip_reduce_kernel(const float *part, long long slots, int H, float *dskip) {
    __shared__ float red[256];
    const int h = blockIdx.x;
    float s = 0.f;
    for (long long i = threadIdx.x; i < slots; i += 256) s += part[i * H + h];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int m = 128; m > 0; m >>= 1) {
        if (threadIdx.x < m) red[threadIdx.x] += red[threadIdx.x + m];
        __syncthreads();
    }
    if (threadIdx.x == 0) dskip[h] = red[0];
}

}  // namespace

cudaError_t launch_scan_fwd_f32(const ScanArgs &a, int dk, int dv, cudaStream_t s) {
    RecArgs r{static_cast<const float *>(a.q), static_cast<const float *>(a.k), static_cast<const float *>(a.v),
              static_cast<const float *>(a.la), static_cast<const float *>(a.dt), a.skip, a.S0,
              static_cast<float *>(a.o), a.S_T, static_cast<float *>(a.states), a.ldq, a.ldk, a.ldv, dv, a.cu,
              a.B, a.T, a.H, a.G, a.parts, a.part_state, a.part_decay, a.status};
    return launch_rec<false>(r, dk, dv, s);
}

cudaError_t launch_scan_bwd_f32(const ScanBwdArgs &a, int dk, int dv, cudaStream_t s) {
    const ScanArgs &f = a.f;
    // the chain of E: rows q (k's place) and dO (v's)
    RecArgs r{nullptr, static_cast<const float *>(f.q), static_cast<const float *>(a.dO),
              static_cast<const float *>(f.la), nullptr, nullptr, a.dS_T, nullptr, a.dS0,
              static_cast<float *>(a.grads), 0, f.ldq, (long long)f.H * dv, dv, f.cu, f.B, f.T, f.H, f.G,
              f.parts, f.part_state, f.part_decay, f.status};
    cudaError_t e = launch_rec<true>(r, dk, dv, s);
    if (e != cudaSuccess) return e;
    const long long slots = slot_count(f.cu, f.B, f.T, kC);
    auto go = [&](auto n, auto p) {
        constexpr int N = decltype(n)::value, P = decltype(p)::value;
        auto kernel = chunk_bwd_kernel<N, P>;
        cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)BwdSmem<N, P>::BYTES);
        if (err != cudaSuccess) return err;
        kernel<<<(unsigned)(slots * f.G * a.splits), 256, BwdSmem<N, P>::BYTES, s>>>(a);
        return cudaGetLastError();
    };
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    if (dk == 128) e = dv == 128 ? go(I128{}, I128{}) : go(I128{}, I64{});
    else e = dv == 128 ? go(I64{}, I128{}) : go(I64{}, I64{});
    return e != cudaSuccess ? e : launch_grad_sums(a, dk, false, kC, s);
}

cudaError_t launch_grad_sums(const ScanBwdArgs &a, int dk, bool bf16, int chunk, cudaStream_t s) {
    const ScanArgs &f = a.f;
    cudaError_t e = cudaSuccess;
    if (a.splits > 1) {
        const unsigned rows = (unsigned)(f.cu ? (long long)f.T : (long long)f.B * f.T);
        if (bf16) qk_reduce_kernel<__nv_bfloat16><<<rows, 256, 0, s>>>(a, dk);
        else qk_reduce_kernel<float><<<rows, 256, 0, s>>>(a, dk);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (a.dskip) {
        dskip_reduce_kernel<<<f.H, 256, 0, s>>>(a.dskip_part, slot_count(f.cu, f.B, f.T, chunk), f.H, a.dskip);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace ssm
}  // namespace gdn2
