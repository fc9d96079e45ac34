// The selective state space scan for bf16 tokens on the fifth-generation
// tensor cores: the forward, the chain of states (or of their gradients) that
// the backward reads, and the end states of a sequence's parts.
//
// A CTA of 16 warps takes one (sequence, head) -- or one part of it -- and
// walks its chunks of 128 tokens with the fp32 state S [dk][dv] in tensor
// memory.  In a chunk, with L_i the log decay from its start through token i,
//     o_i = e^{L_i} S^T q_i + sum_{j <= i} (q_i . k_j) e^{L_i - L_j} dt_j v_j + skip v_i,
//     S  <- e^{L_end} S + sum_j e^{L_end - L_j} dt_j k_j v_j^T,
// as four products: G = q k^T; q S (S rounded to bf16); M v, with M = G masked,
// decayed and rounded to bf16, written back to tensor memory as the left
// operand; and the state's, whose left operand k e^{L_end - L_j} dt_j is taken
// as two bf16 parts, so that S and S_T carry 16 bits of every factor.  The
// chain of gradients E <- e^{L_end} E + sum_i e^{L_i} q_i do_i^T has the same
// form, walked from the end.
//
// Bounds: the forward reads q, k (shared by the group's heads, so mostly from
// L2) and v and writes o once; its chunk costs 2560 cycles of tensor pipe at
// dk = dv = 128 against 2800 of memory at full rate.  The products and the
// read-backs of one chunk overlap (the state's product runs under M's
// construction, M v under the state's read-back); tiles of the next chunk
// arrive meanwhile: k two ahead, q as soon as this chunk's products have read
// it, v at the chunk's end.  Every wait is bounded: where one runs out the
// kernel records GDN2_ERR_TIMEOUT, lets its copies land, frees its tensor
// memory and returns.
#include "common.cuh"
#include "ssm_tc.cuh"

namespace gdn2 {
namespace ssm {
namespace {

using tct::mma_tiles;

struct Maps {
    CUtensorMap q, k, v, o;
};

// The state (or gradient) that reaches part `part`, W columns of row r.
template <int N, int P, int W, bool REV>
__device__ __forceinline__ void start_state(const float *first, const float *part_state, const float *part_decay,
                                            int parts, int part, int bh, int r, int c0, float (&S)[W]) {
    constexpr size_t SE = (size_t)N * P;
#pragma unroll
    for (int i = 0; i < W; ++i) S[i] = 0.f;
    if (r >= N) return;
    const size_t at = (size_t)r * P + c0;
    if (first)
#pragma unroll
        for (int i = 0; i < W; i += 4) *reinterpret_cast<float4 *>(&S[i]) = *reinterpret_cast<const float4 *>(first + bh * SE + at + i);
    for (int s = REV ? parts - 1 : 0; s != part; s += REV ? -1 : 1) {
        const size_t idx = (size_t)bh * (parts - 1) + (REV ? s - 1 : s);
        const float d = part_decay[idx];
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(part_state + idx * SE + at + i);
            S[i] = fmaf(S[i], d, x.x);
            S[i + 1] = fmaf(S[i + 1], d, x.y);
            S[i + 2] = fmaf(S[i + 2], d, x.z);
            S[i + 3] = fmaf(S[i + 3], d, x.w);
        }
    }
}

__device__ __forceinline__ float token(const void *p, size_t i) { return __bfloat162float(static_cast<const bf16 *>(p)[i]); }

// ---------------------------------------------------------------------------
// Forward

template <int N, int P>
struct FwdSmem {
    static constexpr int QB = kCT * N * 2, VB = kCT * P * 2;
    // lo: the second part of the scaled k, and later the o tile.  (At N = 64 the
    // state's product reads 128 rows of its left operand; the upper 64 are
    // whatever block follows, and go to rows of S that nothing reads.)
    static constexpr int LO = 0, K0 = (QB > VB ? QB : VB), K1 = K0 + QB, Q = K1 + QB, V = Q + QB, S16 = V + VB,
                         G = S16 + N * P * 2, END = G + 2 * (int)sizeof(Gates);
    static constexpr int BYTES = END + 1024;
};

template <int N, int P>
__global__ void __launch_bounds__(kNT, 1) fwd_kernel(ScanArgs a, const __grid_constant__ Maps maps) {
    using L = FwdSmem<N, P>;
    constexpr int W = P / 4;  // columns of a thread in a P-column row
    constexpr uint32_t cS = 0, cG = 128, cY = 256, cM = 384;  // tensor-memory columns
    constexpr uint32_t idG = tc::idesc_bf16(128, 128, false, false), idY = tc::idesc_bf16(128, P, false, true),
                       idS = tc::idesc_bf16(128, P, true, true);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (tc::smem_addr(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t ld_q, ld_k[2], ld_v, b_g, b_y1, b_s, b_y2, b_fin;
    __shared__ uint32_t tmem_slot;
    Gates *gates = reinterpret_cast<Gates *>(sm + L::G);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, p = warp & 3, qc = warp >> 2, row = 32 * p + lane;
    const int part = blockIdx.x % a.parts, bh = blockIdx.x / a.parts, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
    const Seq sq = seq_of(a.cu, b, a.T, kCT);
    if (!sq.ok) {
        if (tid == 0) record_status(a.status, GDN2_ERR_INVALID_ARG);
        return;
    }
    const int cpp = (sq.nchunks + a.parts - 1) / a.parts, c_lo = min(part * cpp, sq.nchunks),
              n_chunks = min((part + 1) * cpp, sq.nchunks) - c_lo;
    const bool last_part = part == a.parts - 1;
    const float skip = a.skip ? a.skip[h] : 0.f;
    const int mb = a.cu ? 0 : b, mt = (a.cu ? (int)sq.row0 : 0) + c_lo * kCT;  // coordinates of the part's first row

    if (warp == 0) tc::tmem_alloc(&tmem_slot, 512);
    if (tid == 0) {
        uint64_t *bars[] = {&ld_q, &ld_k[0], &ld_k[1], &ld_v, &b_g, &b_y1, &b_s, &b_y2, &b_fin};
        for (uint64_t *x : bars) tc::mbar_init(x, 1);
        tc::fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = tmem_slot, tl = tm + ((uint32_t)(32 * p) << 16);

    int nq = 0, nk[2] = {0, 0}, nv = 0;  // (thread 0) loads issued
    auto load_q = [&](int m) {
        tc::mbar_expect_tx(&ld_q, L::QB);
        for (int x = 0; x < N / 64; ++x) tc::tma_load_5d(sm + L::Q + x * kCT * 128, &maps.q, 0, mt + m * kCT, x, g, mb, &ld_q);
        ++nq;
    };
    auto load_k = [&](int m) {
        const int s = m & 1;
        tc::mbar_expect_tx(&ld_k[s], L::QB);
        for (int x = 0; x < N / 64; ++x)
            tc::tma_load_5d(sm + (s ? L::K1 : L::K0) + x * kCT * 128, &maps.k, 0, mt + m * kCT, x, g, mb, &ld_k[s]);
        ++nk[s];
    };
    auto load_v = [&](int m) {
        tc::mbar_expect_tx(&ld_v, L::VB);
        for (int x = 0; x < P / 64; ++x) tc::tma_load_5d(sm + L::V + x * kCT * 128, &maps.v, 0, mt + m * kCT, x, h, mb, &ld_v);
        ++nv;
    };
    bool bad = false, aborted = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!tc::mbar_wait(bar, parity)) {
            bad = true;
            record_status(a.status, GDN2_ERR_TIMEOUT);
        }
    };
    // what the threads wrote becomes visible to the tensor cores and copies; a
    // wait that ran out in one thread ends the walk for all of them together
    auto handoff = [&]() {
        tc::fence_async_smem();
        tc::fence_before();
        aborted = __syncthreads_or(bad);
        tc::fence_after();
    };
    if (tid == 0 && n_chunks > 0) {
        load_q(0);
        load_k(0);
        load_v(0);
        if (n_chunks > 1) load_k(1);
    }
    // the last four warps form the decay factors, one chunk ahead, from values loaded two ahead
    float g_la = 0.f, g_dt = 0.f;
    const int gt = tid - (kNT - kCT);
    auto load_gates = [&](int m) {
        const int t = (c_lo + m) * kCT + gt;
        g_la = g_dt = 0.f;
        if (m < n_chunks && t < sq.len) {
            const size_t r = (size_t)(sq.row0 + t) * a.H + h;
            g_la = fmaxf(token(a.la, r), kLogMin);
            g_dt = token(a.dt, r);
        }
    };
    if (gt >= 0) {
        load_gates(0);
        form_gates(gates[0], g_la, g_dt, gt, 1, 0.f);
        load_gates(1);
    }
    float S[W];
    start_state<N, P, W, false>(a.S0, a.part_state, a.part_decay, a.parts, part, bh, row, W * qc, S);
    if (n_chunks > 0 && row < N) put_row<W>(sm + L::S16, N, row, W * qc, S);
    __syncthreads();
    if (n_chunks > 0) {
        const float gm = gates[0].gamma;
        float t[W];
#pragma unroll
        for (int i = 0; i < W; ++i) t[i] = S[i] * gm;
        stw<W>(tl + cS + W * qc, t);
        tc::wait_st();
    }
    handoff();

    for (int m = 0; m < n_chunks; ++m) {
        const int s = m & 1, len = min(kCT, sq.len - (c_lo + m) * kCT);
        const uint32_t ph = m & 1, ph2 = (m >> 1) & 1;
        const Gates &G = gates[s];
        unsigned char *K = sm + (s ? L::K1 : L::K0);
        if (tid == 0) {
            tc::bulk_wait_read();  // the o tile of the chunk before
            wait(&ld_q, ph);
            wait(&ld_k[s], ph2);
            mma_tiles<true, true>(tm + cG, sm + L::Q, kCT, K, kCT, N / 16, idG, false);
            tc::commit(&b_g);
            mma_tiles<true, false>(tm + cY, sm + L::Q, kCT, sm + L::S16, N, N / 16, idY, false);
            tc::commit(&b_y1);
            if (a.states) {  // the state at the chunk's start, as it lies here
                tc::bulk_store(static_cast<unsigned char *>(a.states) +
                                   ((size_t)(sq.slot + c_lo + m) * a.H + h) * (N * P * 2),
                               sm + L::S16, N * P * 2);
                tc::bulk_commit();
            }
        }
        wait(&b_g, ph);
        tc::fence_after();
        scale_hi_lo<N>(K, sm + L::LO, G.wt, len, tid);
        if (a.cu && len < kCT) {
            wait(&ld_v, ph);
            zero_tail(sm + L::V, P / 64, len, tid, kNT);
        }
        handoff();
        if (aborted) break;
        if (tid == 0) {
            wait(&ld_v, ph);
            mma_tiles<false, false>(tm + cS, K, kCT, sm + L::V, kCT, kCT / 16, idS, true);
            mma_tiles<false, false>(tm + cS, sm + L::LO, kCT, sm + L::V, kCT, kCT / 16, idS, true);
            tc::commit(&b_s);
        }
        // M = G masked and decayed: this thread's row i = row, columns 32 qc ..
        {
            uint32_t u[16];
            if (qc > p) {
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = 0u;
            } else {
                float x[32];
                tc::ld_32x32b_x32(tl + cG + 32 * qc, x);
                const float li = G.l[row];
                const float f = qc < p ? __expf(li + between(G, qc, p)) : 0.f;
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    float c[4];
                    if (qc < p) {
                        const float4 cf = *reinterpret_cast<const float4 *>(&G.cf[32 * qc + i]);
                        c[0] = f * cf.x; c[1] = f * cf.y; c[2] = f * cf.z; c[3] = f * cf.w;
                    } else {
                        const float4 l4 = *reinterpret_cast<const float4 *>(&G.l[32 * qc + i]);
                        const float4 d4 = *reinterpret_cast<const float4 *>(&G.dt[32 * qc + i]);
                        c[0] = __expf(li - l4.x) * d4.x; c[1] = __expf(li - l4.y) * d4.y;
                        c[2] = __expf(li - l4.z) * d4.z; c[3] = __expf(li - l4.w) * d4.w;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[i + e] = qc < p || i + e <= lane ? x[i + e] * c[e] : 0.f;
                    u[i / 2] = pack2(x[i], x[i + 1]);
                    u[i / 2 + 1] = pack2(x[i + 2], x[i + 3]);
                }
            }
            st16(tl + cM + 16 * qc, u);
            tc::wait_st();
        }
        if (gt >= 0) {
            form_gates(gates[s ^ 1], g_la, g_dt, gt, 1, 0.f);
            load_gates(m + 2);
        }
        if (tid == 0) tc::bulk_wait_read();  // S16 has been read
        handoff();
        if (aborted) break;
        if (tid == 0) {
            const uint64_t dv0 = tct::mnmaj(sm + L::V, kCT, 0);
#pragma unroll
            for (int x = 0; x < kCT / 16; ++x)
                mma_ts(tm + cG, tm + cM + 8 * x, dv0 + (tct::kstep_bytes<false>(kCT, x) >> 4), idY, x > 0);
            tc::commit(&b_y2);
        }
        wait(&b_y1, ph);
        if (tid == 0 && m + 1 < n_chunks) load_q(m + 1);
        // the state behind this chunk: its bf16 copy, and decayed for the next
        wait(&b_s, ph);
        tc::fence_after();
        if (tid == 0 && m + 2 < n_chunks) load_k(m + 2);
        {
            ldw<W>(tl + cS + W * qc, S);
            tc::wait_ld();
            if (m + 1 < n_chunks) {
                if (row < N) put_row<W>(sm + L::S16, N, row, W * qc, S);
                const float gm = gates[s ^ 1].gamma;
                float t[W];
#pragma unroll
                for (int i = 0; i < W; ++i) t[i] = S[i] * gm;
                stw<W>(tl + cS + W * qc, t);
                tc::wait_st();
            }
        }
        wait(&b_y2, ph);
        tc::fence_after();
        if (a.o) {
            float y[W], z[W];
            ldw<W>(tl + cY + W * qc, y);
            ldw<W>(tl + cG + W * qc, z);
            const float er = G.er[row];
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < W / 8; ++i) {
                const uint32_t at = piece(kCT, row, W / 8 * qc + i);
                const uint4 v = *reinterpret_cast<const uint4 *>(sm + L::V + at);
                const uint32_t ve[4] = {v.x, v.y, v.z, v.w};
                uint32_t u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack2(ve[e]);
                    const int c = 8 * i + 2 * e;
                    u[e] = pack2(fmaf(er, y[c], fmaf(skip, f.x, z[c])), fmaf(er, y[c + 1], fmaf(skip, f.y, z[c + 1])));
                }
                *reinterpret_cast<uint4 *>(sm + L::LO + at) = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
        handoff();
        if (aborted) break;
        if (tid == 0) {
            if (a.o && (!a.cu || len == kCT)) {
                for (int x = 0; x < P / 64; ++x) tma_store_5d(&maps.o, sm + L::LO + x * kCT * 128, mt + m * kCT, x, h, mb);
                tc::bulk_commit();
            }
            if (m + 1 < n_chunks) load_v(m + 1);
        }
        if (a.o && a.cu && len < kCT) {  // a packed sequence's end: row by row (no chunk follows)
            bf16 *o = static_cast<bf16 *>(a.o) + ((size_t)(sq.row0 + (c_lo + m) * kCT) * a.H + h) * P;
            for (int i = tid; i < len * (P / 8); i += kNT) {
                const int r = i / (P / 8), c = i % (P / 8);
                *reinterpret_cast<uint4 *>(o + (size_t)r * a.H * P + 8 * c) =
                    *reinterpret_cast<const uint4 *>(sm + L::LO + piece(kCT, r, c));
            }
        }
    }
    if (last_part && a.S_T && !aborted && row < N) {
        float *dst = a.S_T + (size_t)bh * N * P + (size_t)row * P + W * qc;
#pragma unroll
        for (int i = 0; i < W; i += 4) *reinterpret_cast<float4 *>(dst + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
    }
    if (tid == 0) {  // nothing is left in flight
        tc::commit(&b_fin);
        (void)tc::mbar_wait(&b_fin, 0);
        if (nq) (void)tc::mbar_wait(&ld_q, (nq - 1) & 1);
        if (nv) (void)tc::mbar_wait(&ld_v, (nv - 1) & 1);
        for (int s = 0; s < 2; ++s)
            if (nk[s]) (void)tc::mbar_wait(&ld_k[s], (nk[s] - 1) & 1);
        tc::bulk_wait();
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after();
        tc::tmem_dealloc(tm, 512);
    }
}

// ---------------------------------------------------------------------------
// The chain: states at the chunks' starts (k, v), or REV the gradients at
// their ends (q, dO, walked from the end), as bf16 tile images, and the value
// behind the last chunk walked in fp32.  LOCAL: only a part's value from zero,
// walked against the chain's direction, so that each chunk's weights hold the
// whole way to the part's end and the accumulator is never rescaled.

struct ChainArgs {
    const void *la, *dt;
    const float *first;     // [B][H][N][P] or nullptr
    float *last;            // or nullptr
    unsigned char *images;
    const int *cu;
    int B, T, H, G, parts;
    float *part_state, *part_decay;
    int *status;
};

struct ChainMaps {
    CUtensorMap a, x;  // k and v, or q and dO
};

template <int N, int P, bool LOCAL>
struct ChainSmem {
    static constexpr int AB = kCT * N * 2, XB = kCT * P * 2;
    static constexpr int LO0 = 0, LO1 = LO0 + (LOCAL ? AB : 0), A0 = LO1 + AB, A1 = A0 + AB, X0 = A1 + AB, X1 = X0 + XB,
                         S16 = X1 + XB, G = S16 + (LOCAL ? 0 : N * P * 2), END = G + 2 * (int)sizeof(Gates);
    static constexpr int BYTES = END + 1024;
};

template <int N, int P, bool REV, bool LOCAL>
__global__ void __launch_bounds__(kNT, 1) chain_kernel(ChainArgs a, const __grid_constant__ ChainMaps maps) {
    using L = ChainSmem<N, P, LOCAL>;
    constexpr int W = P / 4;
    constexpr uint32_t idS = tc::idesc_bf16(128, P, true, true);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (tc::smem_addr(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t ld[2], b_s[2], b_fin;
    __shared__ uint32_t tmem_slot;
    Gates *gates = reinterpret_cast<Gates *>(sm + L::G);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, p = warp & 3, qc = warp >> 2, row = 32 * p + lane;
    const int np = LOCAL ? a.parts - 1 : a.parts;
    const int part = blockIdx.x % np + (LOCAL && REV ? 1 : 0), bh = blockIdx.x / np, b = bh / a.H, h = bh % a.H,
              g = h / (a.H / a.G);
    const Seq sq = seq_of(a.cu, b, a.T, kCT);
    if (!sq.ok) {
        if (tid == 0) record_status(a.status, GDN2_ERR_INVALID_ARG);
        return;
    }
    const int cpp = (sq.nchunks + a.parts - 1) / a.parts, c_lo = min(part * cpp, sq.nchunks),
              c_hi = min((part + 1) * cpp, sq.nchunks), n_chunks = c_hi - c_lo;
    constexpr bool DOWN = REV != LOCAL;  // chunks from the last to the first
    auto chunk_of = [&](int m) { return DOWN ? c_hi - 1 - m : c_lo + m; };
    const int mb = a.cu ? 0 : b, mt = a.cu ? (int)sq.row0 : 0;

    if (warp == 0) tc::tmem_alloc(&tmem_slot, 128);
    if (tid == 0) {
        uint64_t *bars[] = {&ld[0], &ld[1], &b_s[0], &b_s[1], &b_fin};
        for (uint64_t *x : bars) tc::mbar_init(x, 1);
        tc::fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = tmem_slot, tl = tm + ((uint32_t)(32 * p) << 16);

    int nl[2] = {0, 0};
    auto load = [&](int m) {
        const int s = m & 1, t = mt + chunk_of(m) * kCT;
        tc::mbar_expect_tx(&ld[s], L::AB + L::XB);
        for (int x = 0; x < N / 64; ++x)
            tc::tma_load_5d(sm + (s ? L::A1 : L::A0) + x * kCT * 128, &maps.a, 0, t, x, g, mb, &ld[s]);
        for (int x = 0; x < P / 64; ++x)
            tc::tma_load_5d(sm + (s ? L::X1 : L::X0) + x * kCT * 128, &maps.x, 0, t, x, h, mb, &ld[s]);
        ++nl[s];
    };
    bool bad = false, aborted = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!tc::mbar_wait(bar, parity)) {
            bad = true;
            record_status(a.status, GDN2_ERR_TIMEOUT);
        }
    };
    auto handoff = [&]() {
        tc::fence_async_smem();
        tc::fence_before();
        aborted = __syncthreads_or(bad);
        tc::fence_after();
    };
    if (tid == 0) {
        if (n_chunks > 0) load(0);
        if (n_chunks > 1) load(1);
    }
    float g_la = 0.f, g_dt = 0.f, carry = 0.f;  // carry (LOCAL): the log decay of the chunks walked
    const int gt = tid - (kNT - kCT);
    auto load_gates = [&](int m) {
        const int t = chunk_of(m) * kCT + gt;
        g_la = g_dt = 0.f;
        if (m < n_chunks && t < sq.len) {
            const size_t r = (size_t)(sq.row0 + t) * a.H + h;
            g_la = fmaxf(token(a.la, r), kLogMin);
            g_dt = REV ? 1.f : token(a.dt, r);
        }
    };
    // (REV weights e^{L_i}: er, with the carry where the walk is LOCAL)
    auto gates_of = [&](int m) {
        Gates &G = gates[m & 1];
        form_gates(G, g_la, g_dt, gt, 1, LOCAL && !REV ? carry : 0.f);
        if (LOCAL) {
            if (REV) G.er[gt] *= __expf(carry);
            asm volatile("bar.sync 1, 128;\n" ::: "memory");
            carry = fmaxf(carry + G.total, 2.f * kLogMin);  // (as good as -inf; kept finite)
        }
        load_gates(m + 1);
    };
    if (gt >= 0) {
        load_gates(0);
        gates_of(0);
    }
    float S[W];
    constexpr int IMG = N * P * 2;
    if (!LOCAL) {
        start_state<N, P, W, REV>(a.first, a.part_state, a.part_decay, a.parts, part, bh, row, W * qc, S);
        if (n_chunks > 0 && row < N) put_row<W>(sm + L::S16, N, row, W * qc, S);
    }
    __syncthreads();
    if (!LOCAL && n_chunks > 0) {
        const float gm = gates[0].gamma;
        float t[W];
#pragma unroll
        for (int i = 0; i < W; ++i) t[i] = S[i] * gm;
        stw<W>(tl + W * qc, t);
        tc::wait_st();
    }
    handoff();
    for (int m = 0; m < n_chunks; ++m) {
        const int s = m & 1, len = min(kCT, sq.len - chunk_of(m) * kCT);
        const uint32_t ph2 = (m >> 1) & 1;
        unsigned char *A = sm + (s ? L::A1 : L::A0), *X = sm + (s ? L::X1 : L::X0),
                      *LOW = sm + (LOCAL && s ? L::LO1 : L::LO0);
        if (!LOCAL && tid == 0) {
            tc::bulk_store(a.images + ((size_t)(sq.slot + chunk_of(m)) * a.H + h) * IMG, sm + L::S16, IMG);
            tc::bulk_commit();
        }
        wait(&ld[s], ph2);
        if (a.cu && len < kCT) zero_tail(X, P / 64, len, tid, kNT);
        scale_hi_lo<N>(A, LOW, REV ? gates[s].er : gates[s].wt, len, tid);
        if (gt >= 0 && m + 1 < n_chunks) gates_of(m + 1);
        if (!LOCAL && tid == 0) tc::bulk_wait_read();
        handoff();
        if (aborted) break;
        if (tid == 0) {
            mma_tiles<false, false>(tm, A, kCT, X, kCT, kCT / 16, idS, !LOCAL || m > 0);
            mma_tiles<false, false>(tm, LOW, kCT, X, kCT, kCT / 16, idS, true);
            tc::commit(&b_s[s]);
        }
        if (LOCAL) {  // the product runs under the next chunk's scaling; its tiles are free when it is done
            if (m > 0) {
                wait(&b_s[s ^ 1], ((m - 1) >> 1) & 1);
                if (tid == 0 && m + 1 < n_chunks) load(m + 1);
            }
            continue;
        }
        wait(&b_s[s], ph2);
        tc::fence_after();
        if (tid == 0 && m + 2 < n_chunks) load(m + 2);
        ldw<W>(tl + W * qc, S);
        tc::wait_ld();
        if (m + 1 < n_chunks) {
            if (row < N) put_row<W>(sm + L::S16, N, row, W * qc, S);
            const float gm = gates[s ^ 1].gamma;
            float t[W];
#pragma unroll
            for (int i = 0; i < W; ++i) t[i] = S[i] * gm;
            stw<W>(tl + W * qc, t);
            tc::wait_st();
        }
        handoff();
    }
    if (LOCAL) {
#pragma unroll
        for (int i = 0; i < W; ++i) S[i] = 0.f;
        if (n_chunks > 0 && !aborted) {
            wait(&b_s[(n_chunks - 1) & 1], ((n_chunks - 1) >> 1) & 1);
            tc::fence_after();
            ldw<W>(tl + W * qc, S);
            tc::wait_ld();
        }
    }
    float *dst = nullptr;
    if (LOCAL) dst = a.part_state + ((size_t)bh * (a.parts - 1) + (REV ? part - 1 : part)) * N * P;
    else if (part == (REV ? 0 : a.parts - 1) && a.last) dst = a.last + (size_t)bh * N * P;
    if (dst && !aborted && row < N) {
        dst += (size_t)row * P + W * qc;
#pragma unroll
        for (int i = 0; i < W; i += 4) *reinterpret_cast<float4 *>(dst + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
    }
    if (LOCAL && gt == 0) a.part_decay[(size_t)bh * (a.parts - 1) + (REV ? part - 1 : part)] = __expf(carry);
    if (tid == 0) {
        tc::commit(&b_fin);
        (void)tc::mbar_wait(&b_fin, 0);
        for (int s = 0; s < 2; ++s)
            if (nl[s]) (void)tc::mbar_wait(&ld[s], (nl[s] - 1) & 1);
        tc::bulk_wait();
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after();
        tc::tmem_dealloc(tm, 128);
    }
}

template <typename K>
cudaError_t big_smem(K kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int N, int P, bool REV, bool LOCAL>
cudaError_t go_chain(const ChainArgs &c, const ChainMaps &m, cudaStream_t s) {
    auto kernel = chain_kernel<N, P, REV, LOCAL>;
    constexpr int bytes = ChainSmem<N, P, LOCAL>::BYTES;
    const cudaError_t e = big_smem(kernel, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(c.B * c.H * (LOCAL ? c.parts - 1 : c.parts)), kNT, bytes, s>>>(c, m);
    return cudaGetLastError();
}

ChainArgs chain_args(const ScanArgs &a) {
    return ChainArgs{a.la, a.dt, nullptr, nullptr, nullptr, a.cu, a.B, a.T, a.H, a.G, a.parts, a.part_state, a.part_decay,
                     a.status};
}

template <int N, int P>
cudaError_t fwd_np(const ScanArgs &a, cudaStream_t s) {
    Maps m;
    ChainMaps cm;
    const int MB = a.cu ? 1 : a.B;
    if (!scan_tile_map(&m.q, a.q, a.ldq, MB, a.T, a.G, N) || !scan_tile_map(&m.k, a.k, a.ldk, MB, a.T, a.G, N) ||
        !scan_tile_map(&m.v, a.v, a.ldv, MB, a.T, a.H, P) ||
        (a.o && !scan_tile_map(&m.o, a.o, (long long)a.H * P, MB, a.T, a.H, P)))
        return cudaErrorInvalidValue;
    cudaError_t e;
    cm.a = m.k;
    cm.x = m.v;
    if (a.parts > 1 && (e = go_chain<N, P, false, true>(chain_args(a), cm, s)) != cudaSuccess) return e;
    if (!a.o) {  // only the states at the chunks' starts
        ChainArgs c = chain_args(a);
        c.first = a.S0;
        c.last = a.S_T;
        c.images = static_cast<unsigned char *>(a.states);
        return go_chain<N, P, false, false>(c, cm, s);
    }
    auto kernel = fwd_kernel<N, P>;
    constexpr int bytes = FwdSmem<N, P>::BYTES;
    if ((e = big_smem(kernel, bytes)) != cudaSuccess) return e;
    kernel<<<(unsigned)(a.B * a.H * a.parts), kNT, bytes, s>>>(a, m);
    return cudaGetLastError();
}

template <int N, int P>
cudaError_t grads_np(const ScanBwdArgs &a, cudaStream_t s) {
    const ScanArgs &f = a.f;
    ChainMaps cm;
    const int MB = f.cu ? 1 : f.B;
    if (!scan_tile_map(&cm.a, f.q, f.ldq, MB, f.T, f.G, N) ||
        !scan_tile_map(&cm.x, a.dO, (long long)f.H * P, MB, f.T, f.H, P))
        return cudaErrorInvalidValue;
    cudaError_t e;
    if (f.parts > 1 && (e = go_chain<N, P, true, true>(chain_args(f), cm, s)) != cudaSuccess) return e;
    ChainArgs c = chain_args(f);
    c.first = a.dS_T;
    c.last = a.dS0;
    c.images = static_cast<unsigned char *>(a.grads);
    return go_chain<N, P, true, false>(c, cm, s);
}

}  // namespace

cudaError_t launch_scan_fwd_tc(const ScanArgs &a, int dk, int dv, cudaStream_t s) {
    if (dk == 128) return dv == 128 ? fwd_np<128, 128>(a, s) : fwd_np<128, 64>(a, s);
    return dv == 128 ? fwd_np<64, 128>(a, s) : fwd_np<64, 64>(a, s);
}

cudaError_t launch_scan_grads_tc(const ScanBwdArgs &a, int dk, int dv, cudaStream_t s) {
    if (dk == 128) return dv == 128 ? grads_np<128, 128>(a, s) : grads_np<128, 64>(a, s);
    return dv == 128 ? grads_np<64, 128>(a, s) : grads_np<64, 64>(a, s);
}

}  // namespace ssm
}  // namespace gdn2
