// Internal interface of the selective state space operators (ssm_*.cu): the
// scan S_t = e^{la_t} S_{t-1} + dt_t k_t v_t^T, o_t = S_t^T q_t + skip_h v_t
// with a scalar decay per token and head and q, k shared by the H / G heads of
// a group, its backward and single-token step, and the layer prologue (short
// causal convolution, step size and decay).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn2 {

int *device_status_ptr();  // (api.cu) the status word of the current device, nullptr on failure
int device_sm_count();     // SMs of the current device
uint32_t debug_wait_limit();  // (api.cu) the test knobs' values: iterations of a wait (0: the default),
int debug_withheld();         // and the chunk whose hand-over does not come (-1: none)

namespace ssm {

constexpr int kC = 64;  // tokens of a chunk of the fp32 kernels (the bf16 ones: 128)

// A log decay as the chunks' sums take it: e^{-104} is 0 in fp32, so a stronger
// decay changes nothing, and differences of the sums stay finite (-inf - -inf
// would not).  A NaN stays one.
constexpr float kLogMin = -104.f;
__device__ __forceinline__ float bounded_log(float x) { return x < kLogMin ? kLogMin : x; }

// Where sequence b's tokens lie; chunks of CH tokens.  Fixed length (cu ==
// nullptr): rows b*T .. ; packed: rows cu[b] .. cu[b+1] - 1 of T rows in all.
// `slot`: the per-chunk slot of its chunk 0.  A packed batch reserves slots
// floor(cu[b] / CH) + b on: sequence b needs at most floor(cu[b+1] / CH) -
// floor(cu[b] / CH) + 1 of them, so sequences never overlap and floor(T / CH)
// + B slots hold them all.
struct Seq {
    long long row0;
    int len, nchunks;
    long long slot;
    bool ok;
};
__device__ __forceinline__ Seq seq_of(const int *cu, int b, int T, int CH) {
    Seq s;
    if (!cu) {
        s.row0 = (long long)b * T;
        s.len = T;
        s.nchunks = (T + CH - 1) / CH;
        s.slot = (long long)b * s.nchunks;
        s.ok = true;
        return s;
    }
    const int r0 = cu[b], r1 = cu[b + 1];
    s.ok = r0 >= 0 && r0 <= r1 && r1 <= T;
    s.row0 = s.ok ? r0 : 0;
    s.len = s.ok ? r1 - r0 : 0;
    s.nchunks = (s.len + CH - 1) / CH;
    s.slot = s.ok ? (long long)(r0 / CH) + b : 0;
    return s;
}
inline long long slot_count(const void *cu, int B, int T, int CH) {
    return cu ? (long long)(T / CH) + B : (long long)B * ((T + CH - 1) / CH);
}
// The sequence and chunk of a slot (false: an unused slot).
__device__ __forceinline__ bool find_slot(const int *cu, int B, int T, int CH, long long slot, int &b, int &n, Seq &s) {
    if (!cu) {
        const int nch = (T + CH - 1) / CH;
        b = (int)(slot / nch);
        n = (int)(slot % nch);
        s = seq_of(cu, b, T, CH);
        return true;
    }
    int lo = 0, hi = B - 1;  // the last b whose first slot is <= slot
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((long long)(cu[mid] / CH) + mid <= slot) lo = mid; else hi = mid - 1;
    }
    b = lo;
    s = seq_of(cu, b, T, CH);
    n = (int)(slot - s.slot);
    return s.ok && n >= 0 && n < s.nchunks;
}

// Token tensors of the scan.  Rows of q, k, v (and of dq, dk, dv, which have
// their layout) are ldq, ldk, ldv elements apart; o, dO are [rows][H][dv],
// log_alpha and dt (and their gradients) [rows][H].
struct ScanArgs {
    const void *q, *k, *v, *la, *dt;
    const float *skip;  // [H] or nullptr
    const float *S0;    // [B][H][dk][dv] or nullptr (zero)
    void *o;            // nullptr: not wanted
    float *S_T;
    void *states;       // per slot and head, the state at the chunk's start
    long long ldq, ldk, ldv;
    const int *cu;
    int B, T, H, G;
    int *status;
    // sequence parts: each sequence is cut into `parts` runs of whole chunks;
    // part_state / part_decay: [B][H][parts - 1] end states (from zero) and decays
    int parts;
    float *part_state, *part_decay;
    bool sorted;        // (bf16) blocks take the sequences by length, longest first
    uint32_t wait_limit;  // (bf16) the test knobs
    int withheld;
};

struct ScanBwdArgs {
    ScanArgs f;          // inputs; states: the forward's
    const void *dO;
    const float *dS_T;
    void *dq, *dk, *dv, *dla, *ddt;
    float *dskip, *dS0;
    void *grads;         // per slot and head, the gradient of the state at the chunk's end
    int splits;          // the heads of a group are cut into this many runs ...
    float *dqk_part;     // ... whose sums of dq and dk go here, [2][splits][rows][G][dk] (splits > 1)
    float *dskip_part;   // [slots][H]
};

// ssm_scan_tc.cu, ssm_bwd_tc.cu (bf16); grads: the chain of a.grads alone
cudaError_t launch_scan_fwd_tc(const ScanArgs &a, int dk, int dv, cudaStream_t s);
cudaError_t launch_scan_grads_tc(const ScanBwdArgs &a, int dk, int dv, cudaStream_t s);
cudaError_t launch_scan_bwd_tc(const ScanBwdArgs &a, int dk, int dv, cudaStream_t s);

// ssm_scan.cu (fp32); sums: dq, dk from the splits' and dskip from the chunks'
cudaError_t launch_grad_sums(const ScanBwdArgs &a, int dk, bool bf16, int chunk, cudaStream_t s);
cudaError_t launch_scan_fwd_f32(const ScanArgs &a, int dk, int dv, cudaStream_t s);
cudaError_t launch_scan_bwd_f32(const ScanBwdArgs &a, int dk, int dv, cudaStream_t s);

// ssm_step.cu
struct StepArgs {
    const void *q, *k, *v, *la, *dt;
    const float *skip;
    float *S;
    void *o;
    long long ldq, ldk, ldv;
    int B, H, G;
};
cudaError_t launch_step(const StepArgs &a, int dk, int dv, bool bf16, cudaStream_t s);

}  // namespace ssm
}  // namespace gdn2
