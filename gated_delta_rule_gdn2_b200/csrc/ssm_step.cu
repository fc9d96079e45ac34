// One token per sequence of the selective state space scan, on fp32 states
// updated in place: S <- e^{la} S + (dt k) v^T, o = S^T q + skip v.
//
// Bound by the state's two passes over memory (8 bytes an entry against 5
// operations): a warp covers whole rows (or runs of them) with 16-byte
// accesses, all of a thread's entries are loaded before the first is used, and
// each is read once and written once, around L1.  The sum over the key axis is
// a thread's own rows, then the warps' in order.  A state is cut into blocks
// of CB value columns, each a block of its own, so that a few sequences still
// reach every SM.
#include "common.cuh"
#include "ssm.h"

namespace gdn2 {
namespace ssm {
namespace {

constexpr int kThreads = 256, kWarps = 8;

template <typename T>
__device__ __forceinline__ float4 load4(const T *p) {
    if constexpr (sizeof(T) == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
        return make_float4(a.x, a.y, b.x, b.y);
    } else {
        return *reinterpret_cast<const float4 *>(p);
    }
}

template <typename T, int N, int P, int CB>
__global__ void __launch_bounds__(kThreads) step_kernel(StepArgs a) {
    constexpr int LPR = CB / 4, RPW = 32 / LPR, RT = N / (kWarps * RPW);  // lanes a row, rows a warp, rows a thread
    static_assert(RT >= 1 && N % (kWarps * RPW) == 0, "state layout");
    __shared__ float s_q[N], s_k[N];
    __shared__ __align__(16) float s_red[kWarps][CB];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cl = (lane % LPR) * 4;
    const int cb = blockIdx.x % (P / CB), bh = blockIdx.x / (P / CB), b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
    float4 *S = reinterpret_cast<float4 *>(a.S + (size_t)bh * N * P + cb * CB + cl);
    float4 x[RT];
    int row[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        row[i] = (i * kWarps + warp) * RPW + lane / LPR;
        x[i] = ld_stream(S + (size_t)row[i] * (P / 4));
    }
    const float al = __expf(to_f32(static_cast<const T *>(a.la)[bh])), dt = to_f32(static_cast<const T *>(a.dt)[bh]);
    if (tid < N) {
        s_q[tid] = to_f32(static_cast<const T *>(a.q)[b * a.ldq + (size_t)g * N + tid]);
        s_k[tid] = dt * to_f32(static_cast<const T *>(a.k)[b * a.ldk + (size_t)g * N + tid]);
    }
    const float4 v = load4(static_cast<const T *>(a.v) + b * a.ldv + (size_t)h * P + cb * CB + cl);
    __syncthreads();
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const float k = s_k[row[i]], q = s_q[row[i]];
        x[i].x = fmaf(al, x[i].x, k * v.x);
        x[i].y = fmaf(al, x[i].y, k * v.y);
        x[i].z = fmaf(al, x[i].z, k * v.z);
        x[i].w = fmaf(al, x[i].w, k * v.w);
        st_stream(S + (size_t)row[i] * (P / 4), x[i]);
        y.x = fmaf(q, x[i].x, y.x);
        y.y = fmaf(q, x[i].y, y.y);
        y.z = fmaf(q, x[i].z, y.z);
        y.w = fmaf(q, x[i].w, y.w);
    }
#pragma unroll
    for (int m = LPR; m < 32; m <<= 1) {
        y.x += __shfl_xor_sync(0xffffffffu, y.x, m);
        y.y += __shfl_xor_sync(0xffffffffu, y.y, m);
        y.z += __shfl_xor_sync(0xffffffffu, y.z, m);
        y.w += __shfl_xor_sync(0xffffffffu, y.w, m);
    }
    if (lane < LPR) *reinterpret_cast<float4 *>(&s_red[warp][cl]) = y;
    __syncthreads();
    if (tid < CB) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += s_red[w][tid];
        const float vj = to_f32(static_cast<const T *>(a.v)[b * a.ldv + (size_t)h * P + cb * CB + tid]);
        if (a.skip) s = fmaf(a.skip[h], vj, s);
        static_cast<T *>(a.o)[(size_t)bh * P + cb * CB + tid] = from_f32<T>(s);
    }
}

template <typename T, int N, int P>
cudaError_t go(const StepArgs &a, cudaStream_t s) {
    // whole rows where the states alone fill the GPU, else 32 columns a block
    const int bh = a.B * a.H;
    if (bh >= 2 * device_sm_count()) step_kernel<T, N, P, P><<<(unsigned)bh, kThreads, 0, s>>>(a);
    else step_kernel<T, N, P, 32><<<(unsigned)bh * (P / 32), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t go_t(const StepArgs &a, int dk, int dv, cudaStream_t s) {
    if (dk == 128) return dv == 128 ? go<T, 128, 128>(a, s) : go<T, 128, 64>(a, s);
    return dv == 128 ? go<T, 64, 128>(a, s) : go<T, 64, 64>(a, s);
}

}  // namespace

cudaError_t launch_step(const StepArgs &a, int dk, int dv, bool bf16, cudaStream_t s) {
    return bf16 ? go_t<__nv_bfloat16>(a, dk, dv, s) : go_t<float>(a, dk, dv, s);
}

}  // namespace ssm
}  // namespace gdn2
