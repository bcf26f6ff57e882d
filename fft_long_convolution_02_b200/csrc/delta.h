// delta.h -- what the gated delta rule's translation units share: the launch
// arguments and the launchers.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace hyena {

constexpr int kDeltaMaxDk = 128;
constexpr int kDeltaMaxDv = 256;
constexpr float kDeltaNormEps = 1e-6f;

// A [B, H d, L] operand: element strides of batch, channel and time.
struct DeltaView {
    int64_t sb, sc, st;
};

struct DeltaArgs {
    int64_t B, L;
    int Hk, Hv, dk, dv;
    int l2norm;
    float scale;
    const void *q, *k, *v;
    void* o;
    const float *g, *beta;               // nullptr: 0 and 1
    DeltaView qs, ks, vs, os, gs, bs;
    const float* state_in;               // nullptr: 0
    float* state_out;                    // nullptr: not wanted
    const int32_t* lengths;              // nullptr: L
};

// Token by token (delta.cu): any strides, either storage type.
cudaError_t launch_delta_seq(const DeltaArgs& a, int dtype, cudaStream_t s);
// In chunks of 64 tokens (delta_chunk.cu): bf16 storage, any strides, with a workspace of delta_chunk_workspace().
size_t delta_chunk_workspace(int64_t B, int64_t L, int Hv);
// The scans' waits give up after budget_ns; `hold` (a test's) is the chunk whose stage is never freed, -1 for none.
cudaError_t launch_delta_chunk(const DeltaArgs& a, void* workspace, uint32_t* status, uint64_t budget_ns, int64_t hold,
                               cudaStream_t s);
// One token, states in place (delta.cu).
cudaError_t launch_delta_step(const DeltaArgs& a, int dtype, float* states, int64_t n_states, const int32_t* slots,
                              uint32_t* status, cudaStream_t s);

}  // namespace hyena
