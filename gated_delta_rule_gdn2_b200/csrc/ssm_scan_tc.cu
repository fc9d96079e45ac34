// The selective state space scan for bf16 tokens on the fifth-generation
// tensor cores: the forward, the chain of states (or of their gradients) that
// the backward reads, and the end states of a sequence's parts.
//
// A CTA takes one (sequence, head) -- or one part of it -- and walks its chunks
// of 128 tokens with the fp32 state S [dk][dv] in tensor memory.  In a chunk,
// with L_i the log decay from its start through token i,
//     o_i = e^{L_i} S^T q_i + sum_{j <= i} M_ij v_j + skip v_i,
//     M_ij = (q_i . k_j) e^{L_i - L_j} dt_j,
//     S  <- e^{L_end} S + sum_j e^{L_end - L_j} dt_j k_j v_j^T,
// as four products: G = q k^T; q S (S rounded to bf16); M v, with M formed from
// G, rounded to bf16 and written over it in tensor memory as the left operand;
// and the state's, whose left operand k e^{L_end - L_j} dt_j is taken as two
// bf16 parts, so that S and S_T carry 16 bits of every factor (measured: S_T
// 2e-6 from the exact state).  The chain of gradients
// E <- e^{L_end} E + sum_i e^{L_i} q_i do_i^T has the same form, walked from the
// end.
//
// What is rounded to bf16 is so because an operand beside v or k, which are bf16,
// has to be: M and the state's copy, which are factors of o alone.  o is rounded
// to bf16 itself, which puts it 1.66e-3 of its norm from the exact one; with these
// two it is 1.88e-3.  The state is not rounded; S_T is 1.3e-6 to 1.9e-6 of its norm
// from exact by what the two parts leave out (fp32 products: 5e-8), and a third
// part would be half as much again of the state's products and of the scaling.
// The decay factors come from the fast base-2 exponential and logarithm: 2^-21.
//
// Bounds, at dk = dv = 128 and for a chunk: 64 KB of HBM traffic (v in, o out; q
// and k come from L2, shared by the group's heads) take 2800 cycles of an SM's
// share; the products take 2560 cycles of the tensor pipe, and read 256 KB of
// operands from shared memory at its full 128 bytes a cycle; the warps and the
// copies move another 350 KB through it.  So shared memory, at about 4800
// cycles, is the nearest limit; measured 7800 (8 x 4096 tokens, 16 heads: 130 to
// 139 us, by the GPU, against 46 for the bytes at the rate of a plain copy), the
// rest being the hand-overs between the roles.  What made the
// difference on the way (same case, on the fastest GPU): all warps in step 208 us; roles that meet
// through mbarriers, without local memory 174; waits of a dozen instructions
// and products issued by a converged warp (the code had outgrown the
// instruction cache) 150; separate accumulators for q S and M v, o's tile over
// q, the copies' waits off the issuer's path 125.  Every wait is bounded: where
// one runs out the kernel records GDN2_ERR_TIMEOUT, lets its copies land, frees
// its tensor memory and returns.
#include "common.cuh"
#include "ssm_tc.cuh"

namespace gdn2 {
namespace ssm {
namespace {

using tct::mma_tiles;

struct Maps {
    CUtensorMap q, k, v, o;
};

// A packed batch with more blocks than SMs gives its blocks out longest sequence
// first, so that none of the long walks begins behind the short ones (12
// sequences of 9001 tokens in all, 32 heads of 64: 96 us against 109 in the
// batch's order, over eight draws of their lengths).  Up to 64 sequences: with more of them the order matters less,
// and each warp finds the sequence by counting.
constexpr int kSortMost = 64;
bool by_length(const int *cu, int B, int H, int parts) {
    return cu && B > 1 && B <= kSortMost && parts == 1 && (long long)B * H > device_sm_count();
}
// The sequence that `rank` others come before (by a whole warp).
__device__ __forceinline__ int sequence_of_rank(const int *cu, int B, int T, int rank) {
    const int lane = threadIdx.x & 31;
    int len[2], before[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int b = lane + 32 * i;
        len[i] = b < B ? seq_of(cu, b, T, kCT).len : -1;
    }
    for (int j = 0; j < B; ++j) {
        const int x = __shfl_sync(0xffffffffu, j < 32 ? len[0] : len[1], j & 31);
#pragma unroll
        for (int i = 0; i < 2; ++i) before[i] += x > len[i] || (x == len[i] && j < lane + 32 * i);
    }
    const uint32_t lo = __ballot_sync(0xffffffffu, len[0] >= 0 && before[0] == rank),
                   hi = __ballot_sync(0xffffffffu, len[1] >= 0 && before[1] == rank);
    return lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
}

// Tensor memory gives a thread 32 columns of its own row, which in the fp32
// states of global memory lie a row apart from its neighbours': 32 lines an
// access.  So a warp's 32 x 32 tile is read and written four rows at a time
// (piece lane >> 2 of row 4 i + (lane & 3) in v[4 i ..]) and turned in registers:
// three exchanges between lanes whose numbers differ in one of the upper three
// bits swap those with the piece's index (200 tokens of one sequence, 16
// heads of 128: 15.6 -> 14.1 us; 32768 tokens in nine parts, which read up to
// eight states: 136 -> 129).
__device__ __forceinline__ void turn(float (&v)[32], int lane) {
#pragma unroll
    for (int b = 0; b < 3; ++b) {
        const int m = 1 << b;
        const bool up = lane & (4 << b);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & m))
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float &lo = v[4 * i + e], &hi = v[4 * (i + m) + e];
                    const float got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, 4 << b);
                    if (up) lo = got;
                    else hi = got;
                }
    }
}
template <int P>
__device__ __forceinline__ void put_tile(float *tile, int lane, float (&S)[32]) {  // (S is turned)
    turn(S, lane);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float4 *>(tile + (size_t)(4 * i + (lane & 3)) * P + 4 * (lane >> 2)) =
            make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
}

// The state (or gradient) that reaches part `part`: columns c0 .. c0 + 31 of
// row r0 + lane (by a whole warp).
template <int N, int P, bool REV>
__device__ __forceinline__ void start_state(const float *first, const float *part_state, const float *part_decay,
                                            int parts, int part, int bh, int r0, int c0, int lane, float (&S)[32]) {
    constexpr size_t SE = (size_t)N * P;
#pragma unroll
    for (int i = 0; i < 32; ++i) S[i] = 0.f;
    if (r0 >= N) return;
    const size_t at = (size_t)(r0 + (lane & 3)) * P + c0 + 4 * (lane >> 2);
    if (first)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4 *>(&S[4 * i]) = *reinterpret_cast<const float4 *>(first + bh * SE + at + 4 * i * P);
    for (int s = REV ? parts - 1 : 0; s != part; s += REV ? -1 : 1) {
        const size_t idx = (size_t)bh * (parts - 1) + (REV ? s - 1 : s);
        const float d = part_decay[idx];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(part_state + idx * SE + at + 4 * i * P);
            S[4 * i] = fmaf(S[4 * i], d, x.x);
            S[4 * i + 1] = fmaf(S[4 * i + 1], d, x.y);
            S[4 * i + 2] = fmaf(S[4 * i + 2], d, x.z);
            S[4 * i + 3] = fmaf(S[4 * i + 3], d, x.w);
        }
    }
    turn(S, lane);
}

// ---------------------------------------------------------------------------
// Forward.  Four roles: warp 16 issues the copies and the products, warp 17
// forms the decay factors up to four chunks ahead, and the other sixteen work
// in two groups that meet only through mbarriers, so that the state-free half
// of chunk m + 1 runs beside the state's half of chunk m:
//   A (warps 0..7)   the two parts of the scaled k in shared memory (64 tokens
//                    at a time: the second part's tile is half a chunk's); M
//   B (warps 8..15)  o from q S and M v; the state's bf16 copy and its decay
// A thread of either group owns a row (token or key channel) of tensor memory
// and half of its columns.

constexpr int kFwdThreads = 18 * 32, kRing = 4;

template <int N, int P>
struct FwdSmem {
    static constexpr int QB = kCT * N * 2, VB = kCT * P * 2;
    // (At N = 64 the state's product reads 128 rows of its left operand; the
    // upper 64 are whatever block follows, and go to rows of S that nothing reads.)
    // The o tile is written over this chunk's q (at N = 64 it may be larger, and has its own place).
    static constexpr bool OVER_Q = QB >= VB;
    static constexpr int LO = 0, K = QB / 2, Q = K + 2 * QB, V = Q + 2 * QB, S16 = V + VB, O = S16 + N * P * 2,
                         G = O + (OVER_Q ? 0 : VB), END = G + kRing * (int)sizeof(Gates);
    static constexpr int BYTES = END + 1024;
};

template <int N, int P>
__global__ void __launch_bounds__(kFwdThreads, 1) fwd_kernel(ScanArgs a, const __grid_constant__ Maps maps) {
    using L = FwdSmem<N, P>;
    constexpr int HP = P / 2;  // columns of a thread in a P-column row
    constexpr uint32_t cS = 0, cG = 128, cY = 256, cY2 = 384;  // tensor-memory columns (M lies over G)
    constexpr uint32_t idG = tc::idesc_bf16(128, 128, false, false), idY = tc::idesc_bf16(128, P, false, true),
                       idS = tc::idesc_bf16(128, P, true, true);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (tc::smem_addr(smem_raw) & 1023u)) & 1023u);
    // tiles landed; products done; hand-overs of the groups (one arrival a warp)
    __shared__ uint64_t ld_qk[2], ld_v, d_g, d_yi, d_s1, d_s, d_y, r_hl, r_hl2, r_m, r_st, r_o, r_y2, r_tail, r_gate[kRing], r_gfree[kRing], d_fin;
    __shared__ uint32_t tmem_slot;
    __shared__ Waits waits;
    Gates *gates = reinterpret_cast<Gates *>(sm + L::G);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, p = warp & 3, half = (warp >> 2) & 1, row = 32 * p + lane;
    const int part = blockIdx.x % a.parts, i = blockIdx.x / a.parts, h = i % a.H, g = h / (a.H / a.G),
              b = a.sorted ? sequence_of_rank(a.cu, a.B, a.T, i / a.H) : i / a.H, bh = b * a.H + h;
    const Seq sq = seq_of(a.cu, b, a.T, kCT);
    if (!sq.ok) {
        if (tid == 0) record_status(a.status, GDN2_ERR_INVALID_ARG);
        return;
    }
    const int cpp = (sq.nchunks + a.parts - 1) / a.parts, c_lo = min(part * cpp, sq.nchunks),
              n_chunks = min((part + 1) * cpp, sq.nchunks) - c_lo;
    const bool last_part = part == a.parts - 1;
    const int mb = a.cu ? 0 : b, mt = (a.cu ? (int)sq.row0 : 0) + c_lo * kCT;  // coordinates of the part's first row

    if (warp == 16) tc::tmem_alloc(&tmem_slot, 512);
    if (tid == 0) {
        uint64_t *one[] = {&ld_qk[0], &ld_qk[1], &ld_v, &d_g, &d_yi, &d_s1, &d_s, &d_y, &d_fin};
        for (uint64_t *x : one) tc::mbar_init(x, 1);
        uint64_t *eight[] = {&r_hl, &r_hl2, &r_m, &r_st, &r_o, &r_y2, &r_tail};
        for (uint64_t *x : eight) tc::mbar_init(x, 8);
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(&r_gate[i], 1);
            tc::mbar_init(&r_gfree[i], 16);
        }
        tc::fence_mbar_init();
        waits_init(waits, a.wait_limit);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = tmem_slot, tl = tm + ((uint32_t)(32 * p) << 16);

    // a bounded wait by a whole warp, with one answer for all its lanes
    auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_bar(bar, parity, &waits)) != 0; };
    // what this warp wrote, and read, handed over
    auto give = [&](uint64_t *bar, bool comes = true) {
        tc::fence_async_smem();
        tc::fence_before();
        __syncwarp();
        if (lane == 0 && comes) tc::mbar_arrive(bar);
    };
    auto tile_o = [&](int m) { return sm + (L::OVER_Q ? L::Q + (m & 1) * L::QB : L::O); };
    // chunk m's parity on a barrier that completes once a chunk, or once in R chunks
    auto par = [](int m, int R) { return (uint32_t)(m / R) & 1u; };

    if (warp == 16) {
        if (n_chunks > 0) {
            int nqk = 0, nv = 0;  // loads issued
            auto load_qk = [&](int m) {
                ++nqk;
                if (!elect()) return;
                uint64_t *bar = &ld_qk[m & 1];
                unsigned char *q = sm + L::Q + (m & 1) * L::QB, *k = sm + L::K + (m & 1) * L::QB;
                tc::mbar_expect_tx(bar, 2 * L::QB);
#pragma unroll
                for (int x = 0; x < N / 64; ++x) {
                    tc::tma_load_5d(q + x * kCT * 128, &maps.q, 0, mt + m * kCT, x, g, mb, bar);
                    tc::tma_load_5d(k + x * kCT * 128, &maps.k, 0, mt + m * kCT, x, g, mb, bar);
                }
            };
            auto load_v = [&](int m) {
                ++nv;
                if (!elect()) return;
                tc::mbar_expect_tx(&ld_v, L::VB);
#pragma unroll
                for (int x = 0; x < P / 64; ++x) tc::tma_load_5d(sm + L::V + x * kCT * 128, &maps.v, 0, mt + m * kCT, x, h, mb, &ld_v);
            };
            auto product_G = [&](int m) {
                if (!elect()) return;
                mma_tiles<true, true>(tm + cG, sm + L::Q + (m & 1) * L::QB, kCT, sm + L::K + (m & 1) * L::QB, kCT, N / 16, idG, false);
                tc::commit(&d_g);
            };
            // half x of the state's product: 64 tokens
            auto product_S = [&](int m, int x, uint64_t *done) {
                if (!elect()) return;
                const unsigned char *k = sm + L::K + (m & 1) * L::QB + x * 64 * 128, *v = sm + L::V + x * 64 * 128;
                mma_tiles<false, false>(tm + cS, k, kCT, v, kCT, 4, idS, true);
                mma_tiles<false, false>(tm + cS, sm + L::LO, 64, v, kCT, 4, idS, true);
                if (x) tc::bulk_wait_read();  // (S16's image has been read: the commit lets group B overwrite it)
                tc::commit(done);
            };
            load_qk(0);
            load_v(0);
            if (n_chunks > 1) load_qk(1);
            bool ok = wait(&ld_qk[0], 0);
            if (ok) product_G(0);
            for (int m = 0; ok && m < n_chunks; ++m) {
                const uint32_t ph = m & 1;
                const bool more = m + 1 < n_chunks;
                if (!(ok = wait(&r_st, ph) && wait(&r_hl, ph) && wait(&ld_v, ph))) break;
                tc::fence_after();
                product_S(m, 0, &d_s1);
                if (elect()) {
                    mma_tiles<true, false>(tm + cY, sm + L::Q + (m & 1) * L::QB, kCT, sm + L::S16, N, N / 16, idY, false);
                    tc::commit(&d_yi);
                    if (a.states) {  // the state at the chunk's start, as it lies here
                        tc::bulk_store(static_cast<unsigned char *>(a.states) +
                                           ((size_t)(sq.slot + c_lo + m) * a.H + h) * (N * P * 2),
                                       sm + L::S16, N * P * 2);
                        tc::bulk_commit();
                    }
                }
                if (m > 0) {
                    // the chunk before: its o has been read out of its tile, which this chunk's
                    // o goes to once M v is done (N < P: every chunk has the one tile), or the next q
                    if (elect()) tc::bulk_wait_read();
                    __syncwarp();
                    if (more) load_qk(m + 1);
                }
                if (!(ok = wait(&r_m, ph) && wait(&r_y2, ph))) break;
                tc::fence_after();
                if (elect()) {
                    const uint64_t v0 = tct::mnmaj(sm + L::V, kCT, 0);
#pragma unroll
                    for (int x = 0; x < kCT / 16; ++x)
                        mma_ts(tm + cY2, tm + cG + 8 * x + (x < 4 ? 0 : 32), v0 + (tct::kstep_bytes<false>(kCT, x) >> 4), idY, true);
                    tc::commit(&d_y);
                }
                if (!(ok = wait(&r_hl2, ph))) break;
                tc::fence_after();
                product_S(m, 1, &d_s);
                if (more) {
                    if (!(ok = wait(&ld_qk[ph ^ 1], par(m + 1, 2)))) break;
                    product_G(m + 1);  // (behind M v, which reads M where G goes)
                    if (!(ok = wait(&d_s, ph))) break;
                    load_v(m + 1);
                }
                if (!(ok = wait(&r_o, ph))) break;
                if (elect()) {  // (a packed sequence's end is stored row by row)
                    if (!a.cu || sq.len - (c_lo + m) * kCT >= kCT)
#pragma unroll
                        for (int x = 0; x < P / 64; ++x)
                            tma_store_5d(&maps.o, tile_o(m) + x * kCT * 128, mt + m * kCT, x, h, mb);
                    tc::bulk_commit();
                }
            }
            if (elect()) {  // nothing is left in flight
                tc::commit(&d_fin);
                tc::bulk_wait();
            }
            (void)tc::mbar_wait(&d_fin, 0);
            (void)tc::mbar_wait(&ld_v, (nv - 1) & 1);
            (void)tc::mbar_wait(&ld_qk[0], ((nqk - 1) >> 1) & 1);
            if (nqk > 1) (void)tc::mbar_wait(&ld_qk[1], ((nqk - 2) >> 1) & 1);
        }
        __syncwarp();
    } else if (warp == 17) {
        for (int m = 0; m < n_chunks; ++m) {
            if (m >= kRing && !wait(&r_gfree[m % kRing], par(m - kRing, kRing))) break;
            (void)form_gates_warp(gates[m % kRing], a.la, a.dt, (size_t)sq.row0 * a.H + h, a.H, (c_lo + m) * kCT, sq.len, lane, 0.f);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&r_gate[m % kRing]);
        }
    } else if (warp < 8) {
        const int gt = tid;  // 0 .. 255
        for (int m = 0; m < n_chunks; ++m) {
            const uint32_t ph = m & 1;
            const int len = min(kCT, sq.len - (c_lo + m) * kCT);
            const Gates &G = gates[m % kRing];
            // (the second part's tile was last read by the state's product before)
            if (!wait(&r_gate[m % kRing], par(m, kRing)) || !wait(&d_g, ph) || (m > 0 && !wait(&d_s, ph ^ 1))) break;
            unsigned char *K = sm + L::K + (m & 1) * L::QB;
            scale_hi_lo<N, 256, 64>(K, sm + L::LO, G.wt, 0, len, gt);
            if (a.cu && len < kCT) {
                if (!wait(&ld_v, ph)) break;
                zero_tail(sm + L::V, P / 64, len, gt, 256);
            }
            give(&r_hl);
            // M = G masked and decayed: row i = row, columns 64 half .., written over the columns of G that this thread
            // has read (64 half + 0 .. 31).  (Column factors are fetched whole before the
            // tile's values: a shared load takes hundreds of cycles while the
            // products stream their operands.)
            tc::fence_after();
            const float li = G.l[row];
#pragma unroll 1
            for (int c0 = 64 * half; c0 < 64 * half + 64; c0 += 16) {
                const int blk = c0 >> 5;
                float c[16], x[16];
                const float *src = blk < p ? &G.cf[c0] : &G.ld[c0];
#pragma unroll
                for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(&c[i]) = *reinterpret_cast<const float4 *>(src + i);
                ld16(tl + cG + c0, x);
                tc::wait_ld();
                uint32_t u[8];
                if (blk > p) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] = 0u;
                } else if (blk < p) {
                    const float f = exp_ftz(li + between(G, blk, p));
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] = pack2(x[2 * i] * (f * c[2 * i]), x[2 * i + 1] * (f * c[2 * i + 1]));
                } else {
                    // (without branches: e^{-inf} above the diagonal, and the value
                    // there, which may be anything, replaced)
                    const int d = lane - (c0 & 31);  // the column on the diagonal
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float e = exp_ftz(i <= d ? li - c[i] : -INFINITY);
                        x[i] = i <= d ? x[i] * e : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[i] = pack2(x[2 * i], x[2 * i + 1]);
                }
                st8(tl + cG + 64 * half + (c0 & 63) / 2, u);
            }
            tc::wait_st();
            give(&r_m);
            if (!wait(&d_s1, ph)) break;  // the first half's second part has been read
            scale_hi_lo<N, 256, 64>(K, sm + L::LO, G.wt, 64, len, gt);
            give(&r_hl2);
            if (lane == 0) tc::mbar_arrive(&r_gfree[m % kRing]);
        }
    } else {
        // the state that reaches this part: its bf16 copy, and decayed for the first chunk
        bool ok = true;
        if (n_chunks > 0) ok = wait(&r_gate[0], 0);
#pragma unroll 1
        for (int x = 0; x < HP / 32; ++x) {
            const int c0 = HP * half + 32 * x;
            float S[32];
            start_state<N, P, false>(a.S0, a.part_state, a.part_decay, a.parts, part, bh, 32 * p, c0, lane, S);
            if (n_chunks == 0) {
                if (last_part && a.S_T && row < N) put_tile<P>(a.S_T + (size_t)bh * N * P + 32 * p * P + c0, lane, S);
            } else {
                if (row < N) put_row<32>(sm + L::S16, N, row, c0, S);
                const float gm = gates[0].gamma;
#pragma unroll
                for (int i = 0; i < 32; ++i) S[i] *= gm;
                tc::st_32x32b_x32(tl + cS + c0, S);
            }
        }
        // M v is added to skip v in fp32 (as part of M's diagonal the term would
        // be rounded to bf16 once more: o's error 1.8e-3 -> 2.3e-3)
        const float skip = a.skip ? a.skip[h] : 0.f;
        auto start_y2 = [&]() {
#pragma unroll 1
            for (int x = 0; x < HP / 16; ++x) {
                const int c0 = HP * half + 16 * x;
                float y[16];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(sm + L::V + piece(kCT, row, c0 / 8 + i));
                    const uint32_t ve[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = unpack2(ve[e]);
                        y[8 * i + 2 * e] = skip * f.x;
                        y[8 * i + 2 * e + 1] = skip * f.y;
                    }
                }
                stw<16>(tl + cY2 + c0, y);
            }
            tc::wait_st();
        };
        tc::wait_st();
        if (n_chunks > 0) {
            give(&r_st);
            ok = ok && wait(&ld_v, 0);
            if (ok) start_y2();
            give(&r_y2, a.withheld != 0);
        }
        for (int m = 0; ok && m < n_chunks; ++m) {
            const uint32_t ph = m & 1;
            const int len = min(kCT, sq.len - (c_lo + m) * kCT);
            const Gates &G = gates[m % kRing];
            const bool more = m + 1 < n_chunks;
            if (!wait(&r_gate[m % kRing], par(m, kRing)) || !wait(&d_yi, ph) || !wait(&d_y, ph)) break;
            tc::fence_after();
            unsigned char *O = tile_o(m);
            const float er = G.er[row];
#pragma unroll 1
            for (int x = 0; x < HP / 16; ++x) {  // o
                const int c0 = HP * half + 16 * x;
                float y[16], z[16];
                ld16(tl + cY + c0, y);
                ld16(tl + cY2 + c0, z);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = fmaf(er, y[i], z[i]);
                put_row<16>(O, kCT, row, c0, y);
            }
            if (a.cu && len < kCT) {  // a packed sequence's end: row by row
                give(&r_tail);
                if (!wait(&r_tail, 0)) break;
                bf16 *o = static_cast<bf16 *>(a.o) + ((size_t)(sq.row0 + (c_lo + m) * kCT) * a.H + h) * P;
                for (int i = tid - 256; i < len * (P / 8); i += 256) {
                    const int r = i / (P / 8), c = i % (P / 8);
                    *reinterpret_cast<uint4 *>(o + (size_t)r * a.H * P + 8 * c) = *reinterpret_cast<const uint4 *>(O + piece(kCT, r, c));
                }
            }
            give(&r_o);
            if (lane == 0) tc::mbar_arrive(&r_gfree[m % kRing]);
            // the state behind this chunk
            if ((more && !wait(&r_gate[(m + 1) % kRing], par(m + 1, kRing))) || !wait(&d_s, ph)) break;
            tc::fence_after();
            if (more) {
                const float gm = gates[(m + 1) % kRing].gamma;
#pragma unroll 1
                for (int x = 0; x < HP / 32; ++x) {
                    float S[32];
                    const int c0 = HP * half + 32 * x;
                    tc::ld_32x32b_x32(tl + cS + c0, S);
                    tc::wait_ld();
                    if (row < N) put_row<32>(sm + L::S16, N, row, c0, S);
#pragma unroll
                    for (int i = 0; i < 32; ++i) S[i] *= gm;
                    tc::st_32x32b_x32(tl + cS + c0, S);
                }
                tc::wait_st();
                give(&r_st);
                if (!wait(&ld_v, ph ^ 1)) break;
                start_y2();
                give(&r_y2, a.withheld != m + 1);
            } else if (last_part && a.S_T) {
#pragma unroll 1
                for (int x = 0; x < HP / 32; ++x) {
                    float S[32];
                    const int c0 = HP * half + 32 * x;
                    tc::ld_32x32b_x32(tl + cS + c0, S);
                    tc::wait_ld();
                    if (row < N) put_tile<P>(a.S_T + (size_t)bh * N * P + 32 * p * P + c0, lane, S);
                }
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (tid == 0 && waits.dead) record_status(a.status, GDN2_ERR_TIMEOUT);
    if (warp == 16) {
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
    bool sorted;
    uint32_t wait_limit;
    int withheld;
};

struct ChainMaps {
    CUtensorMap a, x;  // k and v, or q and dO
};

template <int N, int P, bool LOCAL>
struct ChainSmem {
    static constexpr int AB = kCT * N * 2, XB = kCT * P * 2;
    static constexpr int LO = 0, A = AB, X = A + 2 * AB, S16 = X + 2 * XB, G = S16 + (LOCAL ? 0 : N * P * 2),
                         END = G + kRing * (int)sizeof(Gates);
    static constexpr int BYTES = END + 1024;
};

// Roles as in the forward: group A scales, group B (the chain only) keeps the
// value's bf16 copy and decays it, one warp issues, one forms the factors.
template <int N, int P, bool REV, bool LOCAL>
__global__ void __launch_bounds__(kFwdThreads, 1) chain_kernel(ChainArgs a, const __grid_constant__ ChainMaps maps) {
    using L = ChainSmem<N, P, LOCAL>;
    constexpr int HP = P / 2, IMG = N * P * 2;
    constexpr uint32_t idS = tc::idesc_bf16(128, P, true, true);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (tc::smem_addr(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t ld[2], d_s1, d_s, r_hl, r_hl2, r_st, r_gate[kRing], r_gfree[kRing], d_fin;
    __shared__ uint32_t tmem_slot;
    __shared__ Waits waits;
    Gates *gates = reinterpret_cast<Gates *>(sm + L::G);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, p = warp & 3, half = (warp >> 2) & 1, row = 32 * p + lane;
    const int np = LOCAL ? a.parts - 1 : a.parts;
    const int part = blockIdx.x % np + (LOCAL && REV ? 1 : 0), i = blockIdx.x / np, h = i % a.H, g = h / (a.H / a.G),
              b = a.sorted ? sequence_of_rank(a.cu, a.B, a.T, i / a.H) : i / a.H, bh = b * a.H + h;
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

    if (warp == 16) tc::tmem_alloc(&tmem_slot, 128);
    if (tid == 0) {
        uint64_t *one[] = {&ld[0], &ld[1], &d_s1, &d_s, &d_fin};
        for (uint64_t *x : one) tc::mbar_init(x, 1);
        uint64_t *eight[] = {&r_hl, &r_hl2, &r_st};
        for (uint64_t *x : eight) tc::mbar_init(x, 8);
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(&r_gate[i], 1);
            tc::mbar_init(&r_gfree[i], LOCAL ? 8 : 16);
        }
        tc::fence_mbar_init();
        waits_init(waits, a.wait_limit);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = tmem_slot, tl = tm + ((uint32_t)(32 * p) << 16);
    auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_bar(bar, parity, &waits)) != 0; };
    auto give = [&](uint64_t *bar, bool comes = true) {
        tc::fence_async_smem();
        tc::fence_before();
        __syncwarp();
        if (lane == 0 && comes) tc::mbar_arrive(bar);
    };
    auto par = [](int m, int R) { return (uint32_t)(m / R) & 1u; };

    if (warp == 16) {
        if (n_chunks > 0) {
            auto load = [&](int m) {
                if (!elect()) return;
                const int s = m & 1, t = mt + chunk_of(m) * kCT;
                tc::mbar_expect_tx(&ld[s], L::AB + L::XB);
#pragma unroll
                for (int x = 0; x < N / 64; ++x)
                    tc::tma_load_5d(sm + L::A + s * L::AB + x * kCT * 128, &maps.a, 0, t, x, g, mb, &ld[s]);
#pragma unroll
                for (int x = 0; x < P / 64; ++x)
                    tc::tma_load_5d(sm + L::X + s * L::XB + x * kCT * 128, &maps.x, 0, t, x, h, mb, &ld[s]);
            };
            auto product = [&](int m, int x, uint64_t *done) {
                if (!elect()) return;
                const unsigned char *k = sm + L::A + (m & 1) * L::AB + x * 64 * 128, *v = sm + L::X + (m & 1) * L::XB + x * 64 * 128;
                mma_tiles<false, false>(tm, k, kCT, v, kCT, 4, idS, !LOCAL || m > 0 || x > 0);
                mma_tiles<false, false>(tm, sm + L::LO + x * (L::AB / 2), 64, v, kCT, 4, idS, true);
                if (!LOCAL && x) tc::bulk_wait_read();  // (S16's image has been read: the commit lets group B overwrite it)
                tc::commit(done);
            };
            int nl = 1;  // loads issued
            load(0);
            if (n_chunks > 1) {
                load(1);
                nl = 2;
            }
            for (int m = 0; m < n_chunks; ++m) {
                const uint32_t ph = m & 1;
                if (!wait(&r_hl, ph) || (!LOCAL && !wait(&r_st, ph))) break;
                tc::fence_after();
                if (!LOCAL && elect()) {
                    tc::bulk_store(a.images + ((size_t)(sq.slot + chunk_of(m)) * a.H + h) * IMG, sm + L::S16, IMG);
                    tc::bulk_commit();
                }
                __syncwarp();
                product(m, 0, &d_s1);
                if (!wait(&r_hl2, ph)) break;
                tc::fence_after();
                product(m, 1, &d_s);
                if (m + 2 < n_chunks) {
                    if (!wait(&d_s, ph)) break;
                    load(m + 2);
                    ++nl;
                }
            }
            if (elect()) {  // nothing is left in flight
                tc::commit(&d_fin);
                tc::bulk_wait();
            }
            (void)tc::mbar_wait(&d_fin, 0);
            (void)tc::mbar_wait(&ld[0], ((nl - 1) >> 1) & 1);
            if (nl > 1) (void)tc::mbar_wait(&ld[1], ((nl - 2) >> 1) & 1);
        }
        __syncwarp();
    } else if (warp == 17) {
        float carry = 0.f;  // LOCAL: the log decay of the chunks walked
        for (int m = 0; m < n_chunks; ++m) {
            if (m >= kRing && !wait(&r_gfree[m % kRing], par(m - kRing, kRing))) break;
            const float all = form_gates_warp(gates[m % kRing], a.la, REV ? nullptr : a.dt, (size_t)sq.row0 * a.H + h, a.H,
                                              chunk_of(m) * kCT, sq.len, lane, carry);
            if (LOCAL) carry = carry + all < 2.f * kLogMin ? 2.f * kLogMin : carry + all;  // (as good as -inf; kept finite)
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&r_gate[m % kRing]);
        }
        if (LOCAL && lane == 0)
            a.part_decay[(size_t)bh * (a.parts - 1) + (REV ? part - 1 : part)] = exp_ftz(carry);
    } else if (warp < 8) {
        for (int m = 0; m < n_chunks; ++m) {
            const uint32_t ph = m & 1;
            const int len = min(kCT, sq.len - chunk_of(m) * kCT);
            const Gates &G = gates[m % kRing];
            const float *f = REV ? G.er : G.wt;
            unsigned char *A = sm + L::A + (m & 1) * L::AB;
            if (!wait(&r_gate[m % kRing], par(m, kRing)) || !wait(&ld[m & 1], par(m, 2)) || (m > 0 && !wait(&d_s1, ph ^ 1))) break;
            scale_hi_lo<N, 256, 64>(A, sm + L::LO, f, 0, len, tid);
            if (a.cu && len < kCT) zero_tail(sm + L::X + (m & 1) * L::XB, P / 64, len, tid, 256);
            give(&r_hl);
            if (m > 0 && !wait(&d_s, ph ^ 1)) break;
            scale_hi_lo<N, 256, 64>(A, sm + L::LO + L::AB / 2, f, 64, len, tid);
            give(&r_hl2, a.withheld != m);
            if (lane == 0) tc::mbar_arrive(&r_gfree[m % kRing]);
        }
    } else {
        // the value after chunk m - 1 (m = 0: the one that reaches this part): its
        // bf16 copy, and decayed for chunk m; behind the last chunk, out
        float *dst = nullptr;
        if (LOCAL) dst = a.part_state + ((size_t)bh * (a.parts - 1) + (REV ? part - 1 : part)) * N * P;
        else if (part == (REV ? 0 : a.parts - 1) && a.last) dst = a.last + (size_t)bh * N * P;
        for (int m = LOCAL ? n_chunks : 0; m <= n_chunks; ++m) {
            const bool more = m < n_chunks;
            // (LOCAL: the issuer's last commit, for this group has not followed the chunks' barrier)
            if ((more && !wait(&r_gate[m % kRing], par(m, kRing))) ||
                (m > 0 && !(LOCAL ? wait(&d_fin, 0) : wait(&d_s, (m - 1) & 1))))
                break;
            tc::fence_after();
            const float gm = more ? gates[m % kRing].gamma : 0.f;
#pragma unroll 1
            for (int x = 0; x < HP / 32; ++x) {
                const int c0 = HP * half + 32 * x;
                float S[32];
                if (m > 0) {
                    tc::ld_32x32b_x32(tl + c0, S);
                    tc::wait_ld();
                } else {  // (LOCAL with no chunk: zero)
                    start_state<N, P, REV>(LOCAL ? nullptr : a.first, a.part_state, a.part_decay, LOCAL ? 1 : a.parts,
                                           LOCAL ? 0 : part, bh, 32 * p, c0, lane, S);
                }
                if (more) {
                    if (row < N) put_row<32>(sm + L::S16, N, row, c0, S);
#pragma unroll
                    for (int i = 0; i < 32; ++i) S[i] *= gm;
                    tc::st_32x32b_x32(tl + c0, S);
                } else if (dst && row < N) {
                    put_tile<P>(dst + 32 * p * P + c0, lane, S);
                }
            }
            if (more) {
                tc::wait_st();
                give(&r_st);
                if (lane == 0) tc::mbar_arrive(&r_gfree[m % kRing]);
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (tid == 0 && waits.dead) record_status(a.status, GDN2_ERR_TIMEOUT);
    if (warp == 16) {
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
    kernel<<<(unsigned)(c.B * c.H * (LOCAL ? c.parts - 1 : c.parts)), kFwdThreads, bytes, s>>>(c, m);
    return cudaGetLastError();
}

ChainArgs chain_args(const ScanArgs &a) {
    return ChainArgs{a.la, a.dt, nullptr, nullptr, nullptr, a.cu, a.B, a.T, a.H, a.G, a.parts, a.part_state, a.part_decay,
                     a.status, by_length(a.cu, a.B, a.H, a.parts), a.wait_limit, a.withheld};
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
    ScanArgs f = a;
    f.sorted = by_length(a.cu, a.B, a.H, a.parts);
    kernel<<<(unsigned)(a.B * a.H * a.parts), kFwdThreads, bytes, s>>>(f, m);
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
