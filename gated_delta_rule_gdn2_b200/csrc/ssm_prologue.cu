// The prologue of a selective state space layer: a depthwise causal
// convolution over K <= 4 taps with bias and SiLU on C channels, and per head
// the step size and log decay,
//     u[t, c] = bias[c] + sum_{j<K} W[c][j] x[t - (K-1) + j, c],  y = u sigmoid(u),
//     dt = log(1 + e^{xdt + dt_bias}),  log_alpha = -e^{A_log} dt,
// for prompts (fixed-length or packed; each sequence starts from the K - 1
// inputs of its window, or zeros, and leaves its own), their backward, and the
// single token, whose window is rolled in place.
//
// Forward and single token read each input and write each output once and are
// bound by memory.  A thread owns four channels and walks a strip of rows
// with the last K - 1 inputs in registers, 16 rows' loads in flight;
// the strip re-reads K - 1 rows before it (they come from L2).  The backward
// recomputes u of its strip and of the K - 1 rows behind it, carries the K
// rows of dx that are still open, and sums the filters' gradients of the strip
// in registers; a block adds its strips', and a second kernel the blocks', in a
// fixed order.
#include <type_traits>

#include "common.cuh"
#include "gdn2.h"
#include "ssm.h"

namespace gdn2 {
namespace ssm {
namespace {

constexpr int kMaxTaps = 4;

template <typename T, int V>
struct Raw;  // V elements as loaded
template <> struct Raw<__nv_bfloat16, 4> { uint2 r; };
template <> struct Raw<float, 4> { float4 r; };

template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V> &raw, float (&v)[V]) {
    if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&raw.r);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 f = __bfloat1622float2(p[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
        v[0] = raw.r.x; v[1] = raw.r.y; v[2] = raw.r.z; v[3] = raw.r.w;
    }
}
// VEC: the address is aligned to the V elements; else element by element.
template <typename T, int V, bool VEC>
__device__ __forceinline__ Raw<T, V> load_raw(const T *p) {
    Raw<T, V> x;
    if constexpr (VEC) {
        x.r = *reinterpret_cast<const decltype(x.r) *>(p);
    } else {
        T *e = reinterpret_cast<T *>(&x.r);
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = p[i];
    }
    return x;
}
template <typename T, int V>
__device__ __forceinline__ void store(T *p, const float (&v)[V]) {
    Raw<T, V> x;
    if constexpr (sizeof(T) == 2) {
        __nv_bfloat162 *e = reinterpret_cast<__nv_bfloat162 *>(&x.r);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) e[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    } else {
        x.r = make_float4(v[0], v[1], v[2], v[3]);
    }
    *reinterpret_cast<decltype(x.r) *>(p) = x.r;
}

// 1 / (1 + e^{-x}): 0 and 1 at the ends (e^{-x} = inf divides to 0)
__device__ __forceinline__ float sigm(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
// Of two values.  (One reciprocal of the product of both denominators would have
// to keep e^{-x} below 2^64, where a sigmoid is far from 0 against an x of 1e15;
// a branch around it costs the forward 6%.)  rest: 1 - sigmoid, which for large x
// is not the difference: s is rounded, and the derivative multiplies what is left
// by x.  Where s is 0 it is of no account, but must not be a NaN.
__device__ __forceinline__ float2 sigm2(float2 x, float2 &rest) {
    const float2 t = __fmul2_rn(x, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    float2 e, s;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e.y) : "f"(t.y));
    const float2 a = __fadd2_rn(e, make_float2(1.f, 1.f));
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(s.x) : "f"(a.x));
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(s.y) : "f"(a.y));
    rest = __fmul2_rn(make_float2(fminf(e.x, 3e38f), fminf(e.y, 3e38f)), s);
    return s;
}
__device__ __forceinline__ float2 sigm2(float2 x) {
    float2 rest;
    return sigm2(x, rest);
}
// log(1 + e^x) without cancellation or overflow
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(__expf(-fabsf(x))); }

// Rows on their way: each thread copies its own channels of the next rows to a
// ring of its own in shared memory (S groups of four rows) and reads them back
// itself, so nothing but its own copies' completion is waited for.  Held in
// registers instead, a third as many bytes were in flight and the forward took
// 93 us where it now takes 64 (8 x 4096 rows of 2304 bf16 channels; 46 at the
// rate of a plain copy).
template <typename T, int V>
__device__ __forceinline__ void copy_async(Raw<T, V> *dst, const T *src) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (sizeof(Raw<T, V>) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(d), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(d), "l"(src) : "memory");
}
template <typename T, int V, bool VEC>
__device__ __forceinline__ void fetch_row(Raw<T, V> *dst, const T *src) {
    if constexpr (VEC) copy_async<T, V>(dst, src);
    else *dst = load_raw<T, V, false>(src);
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

// The sequence that holds row r, searched once, then followed forward.
struct Cursor {
    const int *cu;
    int B, T, b;
    long long start, end;  // rows of sequence b (end <= r: r lies in no sequence)
    __device__ __forceinline__ void take(int i) {
        const Seq s = seq_of(cu, i, T, 1);
        b = i;
        start = s.row0;
        end = s.ok ? s.row0 + s.len : s.row0;
    }
    __device__ __forceinline__ void seek(long long r) {
        if (!cu) {
            b = (int)(r / T);
            start = (long long)b * T;
            end = start + T;
            return;
        }
        int lo = 0, hi = B - 1;  // the last sequence that starts at or before r
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cu[mid] <= r) lo = mid; else hi = mid - 1;
        }
        take(lo);
    }
};

struct ProArgs {
    const void *x;
    long long ldx;
    const float *W, *bias;
    int K, C;
    const void *xdt;
    long long ldt;
    const float *dt_bias, *A_log;
    int H;
    const void *init;  // [B][K-1][C] or nullptr
    void *y, *dt, *la, *window;
    const int *cu;
    int B, T;
    long long rows;
    int strip;
    // backward
    const void *dy, *ddt, *dla;
    void *dx, *dxdt, *dinit;
    float *dW, *dbias, *ddt_bias, *dA_log;
    float *part;  // [blocks][C * (K + 1) + 2 H]
    int nblk;
    int *status;
};

constexpr int kFwdThreads = 128, kFwdRing = 4, kBwdRing = 2;
constexpr int kLanes = 64, kStrips = 4;  // backward: a block's lanes of four channels, and strips

// y rows of one thread's strip; ring[group][row][thread].
template <typename T, int V, int K, bool VEC>
__device__ __forceinline__ void conv_strip(const ProArgs &a, int c, long long r0, long long r1,
                                           Raw<T, V> (*ring)[4][kFwdThreads]) {
    const T *x = static_cast<const T *>(a.x) + c;
    T *y = static_cast<T *>(a.y) + c;
    float w[K][V], bias[V], win[K + 3][V];  // win: the last K - 1 inputs, then four rows
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bias[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][i] = a.W[(size_t)(c + i) * K + j];
    }
    Cursor cur{a.cu, a.B, a.T};
    cur.seek(r0);
    long long r = r0;
    while (r < r1) {
        if (r >= cur.end) {  // the next sequence, or rows of none
            if (a.cu) {
                if (cur.b + 1 >= a.B) return;
                cur.take(cur.b + 1);
                if (cur.start > r) r = cur.start;
            } else {
                cur.seek(r);
            }
            continue;
        }
        if (r < cur.start) { r = cur.start; continue; }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {  // the inputs before row r
            const long long rr = r - (K - 1) + j;
            if (rr >= cur.start) {
                unpack<T, V>(load_raw<T, V, VEC>(x + rr * a.ldx), win[j]);
            } else if (a.init) {
                unpack<T, V>(load_raw<T, V, true>(static_cast<const T *>(a.init) +
                                                  ((size_t)cur.b * (K - 1) + (rr - cur.start + K - 1)) * a.C + c),
                             win[j]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) win[j][i] = 0.f;
            }
        }
        const long long stop = r1 < cur.end ? r1 : cur.end;
        const T *px = x + r * a.ldx;
        T *py = y + r * a.C;
        int left = (int)(stop - r), ahead = left, at = 0;
        auto fetch = [&](int g) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < ahead) fetch_row<T, V, VEC>(&ring[g][i][threadIdx.x], px + i * a.ldx);
            copies_commit();
            px += 4 * a.ldx;
            ahead -= 4;
        };
#pragma unroll
        for (int g = 0; g < kFwdRing; ++g) fetch(g);
        for (; left > 0; left -= 4) {
            copies_wait<kFwdRing - 1>();
#pragma unroll
            for (int i = 0; i < 4; ++i) unpack<T, V>(ring[at][i][threadIdx.x], win[K - 1 + i]);
            fetch(at);
            at = at + 1 == kFwdRing ? 0 : at + 1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i >= left) break;
                float o[V];
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    float2 u = make_float2(bias[e], bias[e + 1]);
#pragma unroll
                    for (int j = 0; j < K; ++j)
                        u = __ffma2_rn(make_float2(w[j][e], w[j][e + 1]), make_float2(win[i + j][e], win[i + j][e + 1]), u);
                    const float2 s = __fmul2_rn(u, sigm2(u));
                    o[e] = s.x;
                    o[e + 1] = s.y;
                }
                store<T, V>(py + (size_t)i * a.C, o);
            }
            py += 4 * (size_t)a.C;
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) win[j][e] = win[j + 4][e];
        }
        r = stop;
    }
}

// Is row r inside a sequence?
__device__ __forceinline__ bool in_sequence(const ProArgs &a, long long r) {
    if (!a.cu) return true;
    Cursor cur{a.cu, a.B, a.T};
    cur.seek(r);
    return r >= cur.start && r < cur.end;
}

// Blocks (x): strips, then one per sequence for the windows; (y): runs of
// channels, and last the step sizes.
template <typename T, int K, bool VEC>
__global__ void __launch_bounds__(128) prologue_fwd_kernel(ProArgs a, unsigned nstrip) {
    constexpr int V = 4;
    const int nc = (a.C / V + 127) / 128;
    if (blockIdx.x >= nstrip) {  // the window behind sequence b, and its check
        const int b = blockIdx.x - nstrip;
        const Seq s = seq_of(a.cu, b, a.T, 1);
        if (!s.ok) {
            if (threadIdx.x == 0) record_status(a.status, GDN2_ERR_INVALID_ARG);
            return;
        }
        const int c = ((int)blockIdx.y * 128 + threadIdx.x) * V;
        if ((int)blockIdx.y >= nc || c >= a.C || !a.window) return;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int t = s.len - (K - 1) + j;  // token of the window's row j
            float v[V];
            if (t >= 0) {
                unpack<T, V>(load_raw<T, V, VEC>(static_cast<const T *>(a.x) + (s.row0 + t) * a.ldx + c), v);
            } else if (a.init) {
                unpack<T, V>(load_raw<T, V, true>(static_cast<const T *>(a.init) +
                                                  ((size_t)b * (K - 1) + t + K - 1) * a.C + c), v);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = 0.f;
            }
            store<T, V>(static_cast<T *>(a.window) + ((size_t)b * (K - 1) + j) * a.C + c, v);
        }
        return;
    }
    const long long r0 = (long long)blockIdx.x * a.strip, r1 = min(r0 + a.strip, a.rows);
    if ((int)blockIdx.y < nc) {
        const int c = ((int)blockIdx.y * 128 + threadIdx.x) * V;
        __shared__ Raw<T, V> ring[kFwdRing][4][kFwdThreads];
        if (c < a.C) conv_strip<T, V, K, VEC>(a, c, r0, r1, ring);
        return;
    }
    const int n = (int)(r1 - r0) * a.H;  // step sizes
    for (int i = threadIdx.x; i < n; i += 128) {
        const long long r = r0 + i / a.H;
        const int h = i % a.H;
        if (!in_sequence(a, r)) continue;
        const float z = to_f32(static_cast<const T *>(a.xdt)[r * a.ldt + h]) + (a.dt_bias ? a.dt_bias[h] : 0.f);
        const float dt = softplus(z);
        static_cast<T *>(a.dt)[r * a.H + h] = from_f32<T>(dt);
        static_cast<T *>(a.la)[r * a.H + h] = from_f32<T>(-expf(a.A_log[h]) * dt);
    }
}

// ---------------------------------------------------------------------------
// Backward.  64 lanes of four channels x 4 strips a block.

template <typename T, int K, bool VEC>
__device__ __forceinline__ void conv_strip_bwd(const ProArgs &a, int c, long long r0, long long r1, float (&gw)[K + 1][4],
                                               Raw<T, 4> (*ring)[2][4][kLanes * kStrips]) {
    constexpr int V = 4;
    const T *x = static_cast<const T *>(a.x) + c, *dy = static_cast<const T *>(a.dy) + c;
    T *dx = static_cast<T *>(a.dx) + c;
    float w[K][V], bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bias[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][i] = a.W[(size_t)(c + i) * K + j];
    }
    Cursor cur{a.cu, a.B, a.T};
    cur.seek(r0);
    long long r = r0;
    while (r < r1) {
        if (r >= cur.end) {
            if (a.cu) {
                if (cur.b + 1 >= a.B) return;
                cur.take(cur.b + 1);
                if (cur.start > r) r = cur.start;
            } else {
                cur.seek(r);
            }
            continue;
        }
        if (r < cur.start) { r = cur.start; continue; }
        // rows [r, own) of this sequence are this strip's; du of the K - 1
        // rows behind them reaches into them too
        const long long first = r, own = r1 < cur.end ? r1 : cur.end, stop = min(own + K - 1, cur.end);
        float win[K][V], pend[K][V];  // pend[j]: dx of row r - (K - 1) + j, so far
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) pend[j][i] = win[j][i] = 0.f;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const long long rr = r - (K - 1) + j;
            if (rr >= cur.start) {
                unpack<T, V>(load_raw<T, V, VEC>(x + rr * a.ldx), win[j]);
            } else if (a.init) {
                unpack<T, V>(load_raw<T, V, true>(static_cast<const T *>(a.init) +
                                                  ((size_t)cur.b * (K - 1) + (rr - cur.start + K - 1)) * a.C + c),
                             win[j]);
            }
        }
        // dx of a row, or of a row of the window before the sequence
        auto put = [&](long long at, const float (&v)[V]) {
            if (at >= first) {
                if (at < own) store<T, V>(dx + at * a.C, v);
            } else if (at < cur.start && first == cur.start && a.dinit) {
                store<T, V>(static_cast<T *>(a.dinit) + ((size_t)cur.b * (K - 1) + (at - cur.start + K - 1)) * a.C + c, v);
            }
        };
        auto row = [&](const Raw<T, V> &rx, const Raw<T, V> &ry, long long at, auto inside) {
            float g[V], du[V];
            unpack<T, V>(rx, win[K - 1]);
            unpack<T, V>(ry, g);
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                float2 u = make_float2(bias[i], bias[i + 1]);
#pragma unroll
                for (int j = 0; j < K; ++j)
                    u = __ffma2_rn(make_float2(w[j][i], w[j][i + 1]), make_float2(win[j][i], win[j][i + 1]), u);
                float2 n;
                const float2 s = sigm2(u, n);
                du[i] = g[i] * s.x * fmaf(u.x, n.x, 1.f);
                du[i + 1] = g[i + 1] * s.y * fmaf(u.y, n.y, 1.f);
            }
            const float own_row = decltype(inside)::value || at < own ? 1.f : 0.f;
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const float2 d = make_float2(du[i], du[i + 1]), m = decltype(inside)::value ? d : make_float2(own_row * du[i], own_row * du[i + 1]);
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    const float2 t = __ffma2_rn(m, make_float2(win[j][i], win[j][i + 1]), make_float2(gw[j][i], gw[j][i + 1]));
                    gw[j][i] = t.x;
                    gw[j][i + 1] = t.y;
                    const float2 q = __ffma2_rn(make_float2(w[j][i], w[j][i + 1]), d, make_float2(pend[j][i], pend[j][i + 1]));
                    pend[j][i] = q.x;
                    pend[j][i + 1] = q.y;
                }
                gw[K][i] += m.x;
                gw[K][i + 1] += m.y;
            }
            put(at - (K - 1), pend[0]);
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    pend[j][i] = pend[j + 1][i];
                    win[j][i] = win[j + 1][i];
                }
#pragma unroll
            for (int i = 0; i < V; ++i) pend[K - 1][i] = 0.f;
        };
        const T *px = x + r * a.ldx, *py = dy + r * a.C;
        int ahead = (int)(stop - r), at = 0;
        auto fetch = [&](int g) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < ahead) {
                    fetch_row<T, V, VEC>(&ring[g][0][i][threadIdx.x], px + i * a.ldx);
                    copy_async<T, V>(&ring[g][1][i][threadIdx.x], py + (size_t)i * a.C);
                }
            copies_commit();
            px += 4 * a.ldx;
            py += 4 * (size_t)a.C;
            ahead -= 4;
        };
#pragma unroll
        for (int g = 0; g < kBwdRing; ++g) fetch(g);
        while (r < stop) {
            copies_wait<kBwdRing - 1>();
            Raw<T, V> rx[4], ry[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                rx[i] = ring[at][0][i][threadIdx.x];
                ry[i] = ring[at][1][i][threadIdx.x];
            }
            fetch(at);
            at = at + 1 == kBwdRing ? 0 : at + 1;
            // (four rows of this strip's own without a branch between them: the
            // windows' shifts are then renamings)
            if (r + 4 <= own) {
#pragma unroll
                for (int i = 0; i < 4; ++i) row(rx[i], ry[i], r + i, std::true_type{});
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (r + i < stop) row(rx[i], ry[i], r + i, std::false_type{});
            }
            r = min(r + 4, stop);
        }
        // the rows still open (nothing behind them reaches in any more)
#pragma unroll
        for (int j = 0; j < K - 1; ++j) put(r - (K - 1) + j, pend[j]);
        r = own;
    }
}

template <typename T, int K, bool VEC>
__global__ void __launch_bounds__(kLanes *kStrips) prologue_bwd_kernel(ProArgs a) {
    constexpr int V = 4;
    extern __shared__ __align__(16) unsigned char shared[];  // the rings; then the strips' sums
    auto ring = reinterpret_cast<Raw<T, V>(*)[2][4][kLanes * kStrips]>(shared);
    auto red = reinterpret_cast<float(*)[K + 1][V][kLanes]>(shared);
    const int lane = threadIdx.x % kLanes, st = threadIdx.x / kLanes, nc = (a.C / V + kLanes - 1) / kLanes;
    const size_t W = (size_t)a.C * (K + 1) + 2 * a.H;
    if ((int)blockIdx.x >= a.nblk) {  // a sequence without tokens: nothing reaches its window
        const int b = blockIdx.x - a.nblk;
        const Seq s = seq_of(a.cu, b, a.T, 1);
        if (!s.ok) {
            if (threadIdx.x == 0) record_status(a.status, GDN2_ERR_INVALID_ARG);
            return;
        }
        if (s.len > 0 || !a.dinit || (int)blockIdx.y >= nc) return;
        const int c = ((int)blockIdx.y * kLanes + lane) * V;
        const float z[V] = {0.f, 0.f, 0.f, 0.f};
        if (c < a.C)
            for (int j = st; j < K - 1; j += kStrips)
                store<T, V>(static_cast<T *>(a.dinit) + ((size_t)b * (K - 1) + j) * a.C + c, z);
        return;
    }
    if ((int)blockIdx.y < nc) {
        const int c = ((int)blockIdx.y * kLanes + lane) * V;
        const long long r0 = min(((long long)blockIdx.x * kStrips + st) * a.strip, a.rows), r1 = min(r0 + a.strip, a.rows);
        float gw[K + 1][V];
#pragma unroll
        for (int j = 0; j <= K; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) gw[j][i] = 0.f;
        if (c < a.C && r0 < r1) conv_strip_bwd<T, K, VEC>(a, c, r0, r1, gw, ring);
        __syncthreads();  // every ring is done with
#pragma unroll
        for (int j = 0; j <= K; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) red[st][j][i][lane] = gw[j][i];
        __syncthreads();
        float *out = a.part + blockIdx.x * W;
        const int cb = (int)blockIdx.y * kLanes * V;
        for (int x = threadIdx.x; x < (K + 1) * V * kLanes; x += kLanes * kStrips) {
            const int j = x / (V * kLanes), ch = x % (V * kLanes);  // ch = V lane + i
            if (cb + ch >= a.C) continue;
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < kStrips; ++q) s += red[q][j][ch % V][ch / V];
            out[j < K ? (size_t)(cb + ch) * K + j : (size_t)a.C * K + cb + ch] = s;
        }
        return;
    }
    // step sizes: lanes over the heads, threads over the rows
    float *r2 = reinterpret_cast<float *>(shared);  // [256][2]
    const long long r0 = min((long long)blockIdx.x * kStrips * a.strip, a.rows), r1 = min(r0 + kStrips * a.strip, a.rows);
    const int HB = a.H < 256 ? a.H : 256, per = 256 / HB, hl = threadIdx.x % HB, rl = threadIdx.x / HB;
    for (int h0 = 0; h0 < a.H; h0 += HB) {
        const int h = h0 + hl;
        float sb = 0.f, sA = 0.f;
        if (h < a.H && rl < per) {
            const float A = -expf(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f;
            for (long long r = r0 + rl; r < r1; r += per) {
                if (!in_sequence(a, r)) continue;
                const float z = to_f32(static_cast<const T *>(a.xdt)[r * a.ldt + h]) + bias;
                const float gt = to_f32(static_cast<const T *>(a.ddt)[r * a.H + h]);
                const float gl = to_f32(static_cast<const T *>(a.dla)[r * a.H + h]);
                const float d = fmaf(A, gl, gt) * sigm(z);
                sb += d;
                sA = fmaf(A * softplus(z), gl, sA);
                static_cast<T *>(a.dxdt)[r * a.H + h] = from_f32<T>(d);
            }
        }
        r2[2 * threadIdx.x] = sb;
        r2[2 * threadIdx.x + 1] = sA;
        __syncthreads();
        if (threadIdx.x < HB && h0 + (int)threadIdx.x < a.H) {
            float s0 = 0.f, s1 = 0.f;
            for (int q = 0; q < per; ++q) {
                s0 += r2[2 * (q * HB + threadIdx.x)];
                s1 += r2[2 * (q * HB + threadIdx.x) + 1];
            }
            float *out = a.part + blockIdx.x * W + (size_t)a.C * (K + 1);
            out[h0 + threadIdx.x] = s0;
            out[a.H + h0 + threadIdx.x] = s1;
        }
        __syncthreads();
    }
}

// The parameters' gradients: the blocks' sums, 8 runs of them a column, each
// in order, then the runs in order.
__global__ void __launch_bounds__(256) prologue_reduce_kernel(ProArgs a) {
    __shared__ float red[8][32];
    const size_t nW = (size_t)a.C * a.K, W = nW + a.C + 2 * a.H;
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const size_t i = (size_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (i < W) {
        const int per = (a.nblk + 7) / 8, hi = min((q + 1) * per, a.nblk);
        for (int b = q * per; b < hi; ++b) s += a.part[(size_t)b * W + i];
    }
    red[q][lane] = s;
    __syncthreads();
    if (q != 0 || i >= W) return;
    s = 0.f;
#pragma unroll
    for (int x = 0; x < 8; ++x) s += red[x][lane];
    if (i < nW) a.dW[i] = s;
    else if (i < nW + a.C) { if (a.dbias) a.dbias[i - nW] = s; }
    else if (i < nW + a.C + a.H) { if (a.ddt_bias) a.ddt_bias[i - nW - a.C] = s; }
    else a.dA_log[i - nW - a.C - a.H] = s;
}

// ---------------------------------------------------------------------------
// One token per sequence; a thread owns a column of the window.
template <typename T, int K, bool VEC>
__global__ void __launch_bounds__(128) prologue_step_kernel(ProArgs a) {
    constexpr int V = 4;
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x, nconv = (long long)a.B * (a.C / V);
    if (i < nconv) {
        const int b = (int)(i / (a.C / V)), c = (int)(i % (a.C / V)) * V;
        T *win = static_cast<T *>(a.window) + (size_t)b * (K - 1) * a.C + c;
        Raw<T, V> raw[K];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) raw[j] = load_raw<T, V, true>(win + (size_t)j * a.C);
        raw[K - 1] = load_raw<T, V, VEC>(static_cast<const T *>(a.x) + b * a.ldx + c);
        float u[V], x[V];
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] = a.bias ? a.bias[c + e] : 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            unpack<T, V>(raw[j], x);
#pragma unroll
            for (int e = 0; e < V; ++e) u[e] = fmaf(a.W[(size_t)(c + e) * K + j], x[e], u[e]);
        }
#pragma unroll
        for (int e = 0; e < V; e += 2) {  // (as a prompt's rows)
            const float2 s = sigm2(make_float2(u[e], u[e + 1]));
            u[e] *= s.x;
            u[e + 1] *= s.y;
        }
        store<T, V>(static_cast<T *>(a.y) + (size_t)b * a.C + c, u);
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            *reinterpret_cast<decltype(raw[0].r) *>(win + (size_t)j * a.C) = raw[j + 1].r;
        return;
    }
    const long long n = i - nconv;
    if (n >= (long long)a.B * a.H) return;
    const int b = (int)(n / a.H), h = (int)(n % a.H);
    const float dt = softplus(to_f32(static_cast<const T *>(a.xdt)[b * a.ldt + h]) + (a.dt_bias ? a.dt_bias[h] : 0.f));
    static_cast<T *>(a.dt)[n] = from_f32<T>(dt);
    static_cast<T *>(a.la)[n] = from_f32<T>(-expf(a.A_log[h]) * dt);
}

enum { kFwd, kBwd, kStep };

template <typename T, int K, bool VEC>
cudaError_t launch_k(const ProArgs &a, int what, cudaStream_t s) {
    constexpr int V = 4;
    const unsigned gates = a.H > 0 ? 1 : 0;
    if (what == kFwd) {
        const unsigned nstrip = (unsigned)((a.rows + a.strip - 1) / a.strip);
        const unsigned tail = a.window || a.cu ? (unsigned)a.B : 0u;  // (windows; the offsets' check)
        prologue_fwd_kernel<T, K, VEC><<<dim3(nstrip + tail, (a.C / V + 127) / 128 + gates), 128, 0, s>>>(a, nstrip);
    } else if (what == kBwd) {
        const unsigned tail = a.dinit || a.cu ? (unsigned)a.B : 0u;
        constexpr int rings = kBwdRing * 8 * kLanes * kStrips * (int)sizeof(Raw<T, 4>), sums = kStrips * (K + 1) * 4 * kLanes * 4;
        constexpr int smem = rings > sums ? rings : sums;
        const cudaError_t e = cudaFuncSetAttribute(prologue_bwd_kernel<T, K, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        prologue_bwd_kernel<T, K, VEC>
            <<<dim3(a.nblk + tail, (a.C / 4 + kLanes - 1) / kLanes + gates), kLanes * kStrips, smem, s>>>(a);
    } else {
        const long long n = (long long)a.B * (a.C / V + a.H);
        prologue_step_kernel<T, K, VEC><<<(unsigned)((n + 127) / 128), 128, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const ProArgs &a, int what, bool vec, cudaStream_t s) {
    switch (a.K) {
        case 1: return vec ? launch_k<T, 1, true>(a, what, s) : launch_k<T, 1, false>(a, what, s);
        case 2: return vec ? launch_k<T, 2, true>(a, what, s) : launch_k<T, 2, false>(a, what, s);
        case 3: return vec ? launch_k<T, 3, true>(a, what, s) : launch_k<T, 3, false>(a, what, s);
        default: return vec ? launch_k<T, 4, true>(a, what, s) : launch_k<T, 4, false>(a, what, s);
    }
}

int launch(const ProArgs &a, int what, int dtype, cudaStream_t s) {
    const int e = dtype == GDN2_BF16 ? 2 : 4, v = 4;
    const bool vec = (reinterpret_cast<uintptr_t>(a.x) % (v * e)) == 0 && a.ldx % v == 0;
    const cudaError_t err = dtype == GDN2_BF16 ? launch_t<__nv_bfloat16>(a, what, vec, s) : launch_t<float>(a, what, vec, s);
    if (err != cudaSuccess) {
        (void)cudaGetLastError();
        return GDN2_ERR_CUDA;
    }
    return GDN2_OK;
}

bool a16(const void *p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool o16(const void *p) { return p == nullptr || a16(p); }
bool ae(const void *p, int dtype) {  // an element's alignment
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (dtype == GDN2_BF16 ? 1u : 3u)) == 0;
}
bool f4(const void *p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool of4(const void *p) { return p == nullptr || f4(p); }

int check(int B, int T, int C, int K, int H, int dtype, long long ldx, long long ldt) {
    if (B < 0 || T < 0 || C < 0 || H < 0 || (long long)B * T > 0x7fffffffLL) return GDN2_ERR_INVALID_ARG;
    if (dtype != GDN2_BF16 && dtype != GDN2_FP32) return GDN2_ERR_UNSUPPORTED;
    if (K < 1 || K > kMaxTaps || C % 8 != 0 || C > (1 << 20) || H > (1 << 16)) return GDN2_ERR_UNSUPPORTED;
    if (ldx < C || (H > 0 && ldt < H)) return GDN2_ERR_INVALID_ARG;
    return GDN2_OK;
}

// Rows a thread walks: long strips re-read and re-form less at their ends,
// short ones keep small calls spread over the GPU (about 512 threads an SM).
int strip_rows(long long rows, long long threads_per_row, int most, int least) {
    int s = most;
    while (s > least && (rows + s - 1) / s * threads_per_row < (long long)device_sm_count() * 512) s /= 2;
    return s;
}
int bwd_strip(long long rows, int C) { return strip_rows(rows, (C + 3) / 4, 64, 8); }
int bwd_blocks(long long rows, int C) {
    const long long per = (long long)kStrips * bwd_strip(rows, C);
    return (int)((rows + per - 1) / per);
}

}  // namespace
}  // namespace ssm
}  // namespace gdn2

using namespace gdn2;
using namespace gdn2::ssm;

extern "C" {

int gdn2_ssm_prologue_fwd(const void *x, const float *W, const float *bias, int K, const void *xdt,
                          const float *dt_bias, const float *A_log, const void *init, void *y, void *dt,
                          void *log_alpha, void *window, const int *cu_seqlens, long long ldx, long long ldt, int B,
                          int T, int C, int H, int dtype, cudaStream_t stream) {
    const int st = check(B, T, C, K, H, dtype, ldx, ldt);
    if (st != GDN2_OK) return st;
    const long long rows = cu_seqlens ? (long long)T : (long long)B * T;
    if (B == 0 || (C == 0 && H == 0)) return GDN2_OK;
    if (K == 1) init = window = nullptr;
    if (C > 0 && (!f4(W) || !of4(bias) || !o16(init) || !o16(window))) return GDN2_ERR_INVALID_ARG;
    if (C > 0 && rows > 0 && (!ae(x, dtype) || !a16(y))) return GDN2_ERR_INVALID_ARG;
    if (H > 0 && rows > 0 &&
        (!ae(xdt, dtype) || !of4(dt_bias) || !f4(A_log) || !ae(dt, dtype) || !ae(log_alpha, dtype)))
        return GDN2_ERR_INVALID_ARG;
    if (cu_seqlens && (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return GDN2_ERR_INVALID_ARG;
    ProArgs a{};
    a.x = x; a.ldx = ldx; a.W = W; a.bias = bias; a.K = K; a.C = C; a.xdt = xdt; a.ldt = ldt; a.dt_bias = dt_bias;
    a.A_log = A_log; a.H = H; a.init = init; a.y = y; a.dt = dt; a.la = log_alpha; a.window = window;
    a.cu = cu_seqlens; a.B = B; a.T = T; a.rows = rows;
    if (rows == 0 && !window) return GDN2_OK;
    if (!(a.status = device_status_ptr())) return GDN2_ERR_CUDA;
    a.strip = strip_rows(rows, C / 4 + 1, 64, 4);
    return launch(a, kFwd, dtype, stream);
}

size_t gdn2_ssm_prologue_bwd_workspace(int B, int T, int C, int K, int H, int packed) {
    if (B <= 0 || T <= 0 || C < 0 || H < 0 || K < 1 || K > kMaxTaps || C + H == 0) return 0;
    const long long rows = packed ? (long long)T : (long long)B * T;
    return (size_t)bwd_blocks(rows, C) * ((size_t)C * (K + 1) + 2 * (size_t)H) * sizeof(float);
}

int gdn2_ssm_prologue_bwd(const void *x, const float *W, const float *bias, int K, const void *xdt,
                          const float *dt_bias, const float *A_log, const void *init, const void *dy, const void *ddt,
                          const void *dlog_alpha, void *dx, float *dW, float *dbias, void *dxdt, float *ddt_bias,
                          float *dA_log, void *dinit, const int *cu_seqlens, long long ldx, long long ldt, int B,
                          int T, int C, int H, int dtype, void *ws, size_t ws_bytes, cudaStream_t stream) {
    const int st = check(B, T, C, K, H, dtype, ldx, ldt);
    if (st != GDN2_OK) return st;
    const long long rows = cu_seqlens ? (long long)T : (long long)B * T;
    if (C == 0 && H == 0) return GDN2_OK;
    if (K == 1) init = dinit = nullptr;
    if (C > 0 && (!f4(W) || !of4(bias) || !o16(init) || !o16(dinit) || !f4(dW) || !of4(dbias))) return GDN2_ERR_INVALID_ARG;
    if (H > 0 && (!of4(dt_bias) || !f4(A_log) || !of4(ddt_bias) || !f4(dA_log))) return GDN2_ERR_INVALID_ARG;
    if (C > 0 && rows > 0 && (!ae(x, dtype) || !a16(dy) || !a16(dx))) return GDN2_ERR_INVALID_ARG;
    if (H > 0 && rows > 0 && (!ae(xdt, dtype) || !ae(ddt, dtype) || !ae(dlog_alpha, dtype) || !ae(dxdt, dtype)))
        return GDN2_ERR_INVALID_ARG;
    if (cu_seqlens && (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return GDN2_ERR_INVALID_ARG;
    if (ws_bytes < gdn2_ssm_prologue_bwd_workspace(B, T, C, K, H, cu_seqlens != nullptr) ||
        (B > 0 && rows > 0 && !a16(ws)))
        return GDN2_ERR_WORKSPACE;
    ProArgs a{};
    a.x = x; a.ldx = ldx; a.W = W; a.bias = bias; a.K = K; a.C = C; a.xdt = xdt; a.ldt = ldt; a.dt_bias = dt_bias;
    a.A_log = A_log; a.H = H; a.init = init; a.cu = cu_seqlens; a.B = B; a.T = T; a.rows = rows;
    a.dy = dy; a.ddt = ddt; a.dla = dlog_alpha; a.dx = dx; a.dxdt = dxdt; a.dinit = dinit;
    a.dW = dW; a.dbias = dbias; a.ddt_bias = ddt_bias; a.dA_log = dA_log;
    a.part = static_cast<float *>(ws);
    if (!(a.status = device_status_ptr())) return GDN2_ERR_CUDA;
    if (B > 0 && rows > 0) {
        a.strip = bwd_strip(rows, C);
        a.nblk = bwd_blocks(rows, C);
        const int e = launch(a, kBwd, dtype, stream);
        if (e != GDN2_OK) return e;
    } else if (B > 0 && dinit) {  // every sequence is empty
        const int e = launch(a, kBwd, dtype, stream);
        if (e != GDN2_OK) return e;
    }
    const size_t W_ = (size_t)C * (K + 1) + 2 * (size_t)H;
    prologue_reduce_kernel<<<(unsigned)((W_ + 31) / 32), 256, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return GDN2_ERR_CUDA;
    return GDN2_OK;
}

int gdn2_ssm_prologue_step(const void *x, const float *W, const float *bias, int K, const void *xdt,
                           const float *dt_bias, const float *A_log, void *window, void *y, void *dt, void *log_alpha,
                           long long ldx, long long ldt, int B, int C, int H, int dtype, cudaStream_t stream) {
    const int st = check(B, 1, C, K, H, dtype, ldx, ldt);
    if (st != GDN2_OK) return st;
    if (B == 0 || (C == 0 && H == 0)) return GDN2_OK;
    if (C > 0 && (!f4(W) || !of4(bias) || (K > 1 && !a16(window)) || !ae(x, dtype) || !a16(y)))
        return GDN2_ERR_INVALID_ARG;
    if (H > 0 && (!ae(xdt, dtype) || !of4(dt_bias) || !f4(A_log) || !ae(dt, dtype) || !ae(log_alpha, dtype)))
        return GDN2_ERR_INVALID_ARG;
    ProArgs a{};
    a.x = x; a.ldx = ldx; a.W = W; a.bias = bias; a.K = K; a.C = C; a.xdt = xdt; a.ldt = ldt; a.dt_bias = dt_bias;
    a.A_log = A_log; a.H = H; a.window = window; a.y = y; a.dt = dt; a.la = log_alpha; a.B = B; a.T = 1; a.rows = B;
    return launch(a, kStep, dtype, stream);
}

}  // extern "C"
