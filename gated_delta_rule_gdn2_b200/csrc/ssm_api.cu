// C ABI of the selective state space scan: argument checks, buffer sizes and
// dispatch.  The contract of every entry point is in include/gdn2.h.
#include "gdn2.h"

#include <algorithm>
#include <cmath>

#include "ssm.h"

namespace gdn2 {

int device_sm_count() {
    constexpr int kMaxDevices = 64;
    static int count[kMaxDevices] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)cudaGetLastError();
        return 148;
    }
    if (!count[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();
            return 148;
        }
        count[dev] = n;
    }
    return count[dev];
}

namespace ssm {
namespace {

bool a16(const void *p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool o16(const void *p) { return p == nullptr || a16(p); }
bool ae(const void *p, int dtype) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (dtype == GDN2_BF16 ? 1u : 3u)) == 0;
}
bool of4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check(int B, int T, int H, int G, int dk, int dv, int dtype) {
    if (B < 0 || T < 0 || H < 0) return GDN2_ERR_INVALID_ARG;
    if (dtype != GDN2_BF16 && dtype != GDN2_FP32) return GDN2_ERR_UNSUPPORTED;
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return GDN2_ERR_UNSUPPORTED;
    if (H > 0 && (G < 1 || H % G != 0)) return GDN2_ERR_INVALID_ARG;
    // grids, rows' widths and slot numbers stay within 31 bits
    if (H > (1 << 16) || (long long)B * H > (1LL << 24) || (long long)B * T > 0x7fffffffLL) return GDN2_ERR_INVALID_ARG;
    return GDN2_OK;
}
// row strides: whole rows, and every row 16-byte aligned
bool ld_ok(long long ld, int width, int dtype) { return ld >= width && ld % (dtype == GDN2_BF16 ? 8 : 4) == 0; }

size_t r256(size_t x) { return (x + 255) / 256 * 256; }
long long rows_of(const void *cu, int B, int T) { return cu ? (long long)T : (long long)B * T; }

int chunk_of(int dtype) { return dtype == GDN2_BF16 ? 128 : kC; }

// Parts a sequence is cut into: as many as fill the SMs (bf16: a block of the
// walk takes a whole SM; fp32: four of its 64-column blocks share one).  A
// part costs its tokens once more for its end state, and the parts before it
// are added up at its start, so bf16 parts are at least four chunks long; the
// fp32 walk goes token by token, and one chunk repays the cut (B2 T1000 H8
// d64: 91 us for parts of four chunks, 39 us for parts of one).
int part_count(const void *cu, int B, int T, int H, int dv, int dtype) {
    if (B == 0 || H == 0) return 1;
    const bool bf16 = dtype == GDN2_BF16;
    const long long room = (long long)device_sm_count() * (bf16 ? 1 : 4);
    const long long blocks = (long long)B * H * (bf16 ? 1 : dv / 64);
    const long long chunks = ((cu ? T / B : T) + chunk_of(dtype) - 1) / chunk_of(dtype);
    const long long p = std::min(room / std::max(1LL, blocks), chunks / (bf16 ? 4 : 1));
    return (int)std::max(1LL, std::min(p, 64LL));
}

struct Plan {
    int parts, splits;
    size_t part_state, part_decay, grads, states, dqk, dskip, total;  // byte offsets into the workspace
};

Plan plan(const void *cu, int B, int T, int H, int G, int dk, int dv, int dtype, bool bwd, bool own_states) {
    Plan p{};
    const size_t SE = (size_t)dk * dv, img = SE * (dtype == GDN2_BF16 ? 2 : 4);
    const int chunk = chunk_of(dtype);
    const long long slots = slot_count(cu, B, T, chunk), rows = rows_of(cu, B, T);
    p.parts = part_count(cu, B, T, H, dv, dtype);
    size_t at = 0;
    p.part_state = at; at += r256((size_t)B * H * (p.parts - 1) * SE * 4);
    p.part_decay = at; at += r256((size_t)B * H * (p.parts - 1) * 4);
    p.splits = 1;
    if (bwd) {
        const int hpg = H / G;
        // heads of a group in one block after another, unless the blocks then
        // leave a fifth of the GPU idle (several runs' sums cost a pass over
        // dq and dk in fp32)
        // (two of the fp32 kernel's blocks share an SM at dk = dv = 64)
        const double sms = device_sm_count() * (dtype == GDN2_FP32 && dk + dv == 128 ? 2 : 1);
        auto cost = [&](int n) { return std::ceil(slots * G * n / sms) * ((hpg + n - 1) / n); };
        for (int n = 2; n <= hpg; n *= 2)
            if (cost(n) < 0.8 * cost(p.splits)) p.splits = n;
        p.grads = at; at += r256((size_t)slots * H * img);
        p.states = at; at += own_states ? r256((size_t)slots * H * img) : 0;
        p.dqk = at; at += p.splits > 1 ? r256((size_t)2 * p.splits * rows * G * dk * 4) : 0;
        p.dskip = at; at += r256((size_t)slots * H * 4);
    }
    p.total = at;
    return p;
}

int launch_status(cudaError_t e) {
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return GDN2_ERR_CUDA;
    }
    return GDN2_OK;
}

int copy_state(float *dst, const float *src, size_t n, cudaStream_t s) {
    if (!dst) return GDN2_OK;
    return launch_status(src ? cudaMemcpyAsync(dst, src, n * 4, cudaMemcpyDeviceToDevice, s)
                             : cudaMemsetAsync(dst, 0, n * 4, s));
}

const int *packed_mark(int packed) { return packed ? reinterpret_cast<const int *>(16) : nullptr; }

}  // namespace
}  // namespace ssm
}  // namespace gdn2

using namespace gdn2;
using namespace gdn2::ssm;

extern "C" {

size_t gdn2_ssm_states_bytes(int B, int T, int H, int dk, int dv, int dtype, int packed) {
    if (check(B, T, H, 1, dk, dv, dtype) != GDN2_OK || B == 0 || T == 0 || H == 0) return 0;
    return (size_t)slot_count(packed_mark(packed), B, T, chunk_of(dtype)) * H * dk * dv * (dtype == GDN2_BF16 ? 2 : 4);
}

size_t gdn2_ssm_fwd_workspace(int B, int T, int H, int G, int dk, int dv, int dtype, int packed) {
    if (check(B, T, H, G, dk, dv, dtype) != GDN2_OK || B == 0 || T == 0 || H == 0) return 0;
    return plan(packed_mark(packed), B, T, H, G, dk, dv, dtype, false, false).total;
}

size_t gdn2_ssm_bwd_workspace(int B, int T, int H, int G, int dk, int dv, int dtype, int packed, int states_given) {
    if (check(B, T, H, G, dk, dv, dtype) != GDN2_OK || B == 0 || T == 0 || H == 0) return 0;
    return plan(packed_mark(packed), B, T, H, G, dk, dv, dtype, true, !states_given).total;
}

int gdn2_ssm_fwd(const void *q, const void *k, const void *v, const void *log_alpha, const void *dt,
                 const float *skip, const float *S0, void *o, float *S_T, void *states, const int *cu_seqlens,
                 long long ldq, long long ldk, long long ldv, int B, int T, int H, int G, int dk, int dv, int dtype,
                 void *ws, size_t ws_bytes, cudaStream_t stream) {
    const int st = check(B, T, H, G, dk, dv, dtype);
    if (st != GDN2_OK) return st;
    if (!o16(S0) || !o16(S_T) || !o16(states) || !o16(ws) || !of4(skip) || !of4(cu_seqlens)) return GDN2_ERR_INVALID_ARG;
    if (B == 0 || H == 0) return GDN2_OK;
    if (T == 0) return copy_state(S_T, S0, (size_t)B * H * dk * dv, stream);
    if (!a16(q) || !a16(k) || !a16(v) || !ae(log_alpha, dtype) || !ae(dt, dtype) || !a16(o)) return GDN2_ERR_INVALID_ARG;
    if (!ld_ok(ldq, G * dk, dtype) || !ld_ok(ldk, G * dk, dtype) || !ld_ok(ldv, H * dv, dtype)) return GDN2_ERR_INVALID_ARG;
    const Plan p = plan(cu_seqlens, B, T, H, G, dk, dv, dtype, false, false);
    if (ws_bytes < p.total || (p.total && !ws)) return GDN2_ERR_WORKSPACE;
    ScanArgs a{q, k, v, log_alpha, dt, skip, S0, o, S_T, states, ldq, ldk, ldv, cu_seqlens, B, T, H, G,
               device_status_ptr(), p.parts};
    a.wait_limit = debug_wait_limit();
    a.withheld = debug_withheld();
    if (!a.status) return GDN2_ERR_CUDA;
    unsigned char *w = static_cast<unsigned char *>(ws);
    a.part_state = reinterpret_cast<float *>(w + p.part_state);
    a.part_decay = reinterpret_cast<float *>(w + p.part_decay);
    return launch_status(dtype == GDN2_BF16 ? launch_scan_fwd_tc(a, dk, dv, stream) : launch_scan_fwd_f32(a, dk, dv, stream));
}

int gdn2_ssm_bwd(const void *q, const void *k, const void *v, const void *log_alpha, const void *dt,
                 const float *skip, const float *S0, const void *dO, const float *dS_T, const void *states, void *dq,
                 void *dk_, void *dv_, void *dlog_alpha, void *ddt, float *dskip, float *dS0, const int *cu_seqlens,
                 long long ldq, long long ldk, long long ldv, int B, int T, int H, int G, int dk, int dv, int dtype,
                 void *ws, size_t ws_bytes, cudaStream_t stream) {
    const int st = check(B, T, H, G, dk, dv, dtype);
    if (st != GDN2_OK) return st;
    if (!o16(S0) || !o16(dS_T) || !o16(dS0) || !o16(states) || !o16(ws) || !of4(skip) || !of4(dskip) || !of4(cu_seqlens))
        return GDN2_ERR_INVALID_ARG;
    // (the gradients of q and k are sums over heads, and there is none to write them)
    if (H == 0 && B > 0 && T > 0) return GDN2_ERR_INVALID_ARG;
    if (B == 0 || H == 0 || T == 0) {
        if (dskip && H > 0) {
            const int e = launch_status(cudaMemsetAsync(dskip, 0, (size_t)H * 4, stream));
            if (e != GDN2_OK) return e;
        }
        return B == 0 || H == 0 ? GDN2_OK : copy_state(dS0, dS_T, (size_t)B * H * dk * dv, stream);
    }
    if (!a16(q) || !a16(k) || !a16(v) || !ae(log_alpha, dtype) || !ae(dt, dtype) || !a16(dO) || !a16(dq) || !a16(dk_) ||
        !a16(dv_) || !ae(dlog_alpha, dtype) || !ae(ddt, dtype))
        return GDN2_ERR_INVALID_ARG;
    if (!ld_ok(ldq, G * dk, dtype) || !ld_ok(ldk, G * dk, dtype) || !ld_ok(ldv, H * dv, dtype)) return GDN2_ERR_INVALID_ARG;
    const Plan p = plan(cu_seqlens, B, T, H, G, dk, dv, dtype, true, !states);
    if (ws_bytes < p.total || !ws) return GDN2_ERR_WORKSPACE;
    unsigned char *w = static_cast<unsigned char *>(ws);
    ScanBwdArgs a{};
    a.f = ScanArgs{q, k, v, log_alpha, dt, skip, S0, nullptr, nullptr, states ? const_cast<void *>(states) : w + p.states,
                   ldq, ldk, ldv, cu_seqlens, B, T, H, G, device_status_ptr(), p.parts,
                   reinterpret_cast<float *>(w + p.part_state), reinterpret_cast<float *>(w + p.part_decay)};
    if (!a.f.status) return GDN2_ERR_CUDA;
    a.f.wait_limit = debug_wait_limit();
    a.f.withheld = debug_withheld();
    a.dO = dO; a.dS_T = dS_T; a.dq = dq; a.dk = dk_; a.dv = dv_; a.dla = dlog_alpha; a.ddt = ddt;
    a.dskip = dskip; a.dS0 = dS0; a.grads = w + p.grads; a.splits = p.splits;
    a.dqk_part = reinterpret_cast<float *>(w + p.dqk);
    a.dskip_part = reinterpret_cast<float *>(w + p.dskip);
    if (!states) {  // the states at the chunks' starts, without o
        const cudaError_t e = dtype == GDN2_BF16 ? launch_scan_fwd_tc(a.f, dk, dv, stream) : launch_scan_fwd_f32(a.f, dk, dv, stream);
        if (e != cudaSuccess) return launch_status(e);
    }
    return launch_status(dtype == GDN2_BF16 ? launch_scan_bwd_tc(a, dk, dv, stream) : launch_scan_bwd_f32(a, dk, dv, stream));
}

int gdn2_ssm_step(const void *q, const void *k, const void *v, const void *log_alpha, const void *dt,
                  const float *skip, float *S, void *o, long long ldq, long long ldk, long long ldv, int B, int H,
                  int G, int dk, int dv, int dtype, cudaStream_t stream) {
    const int st = check(B, 1, H, G, dk, dv, dtype);
    if (st != GDN2_OK) return st;
    if (B == 0 || H == 0) return GDN2_OK;
    if (!a16(q) || !a16(k) || !a16(v) || !ae(log_alpha, dtype) || !ae(dt, dtype) || !a16(S) || !a16(o) || !of4(skip))
        return GDN2_ERR_INVALID_ARG;
    if (!ld_ok(ldq, G * dk, dtype) || !ld_ok(ldk, G * dk, dtype) || !ld_ok(ldv, H * dv, dtype)) return GDN2_ERR_INVALID_ARG;
    const StepArgs a{q, k, v, log_alpha, dt, skip, S, o, ldq, ldk, ldv, B, H, G};
    return launch_status(launch_step(a, dk, dv, dtype == GDN2_BF16, stream));
}

}  // extern "C"
