// Internal interface of the linear attention with one decay per head (not part of the C ABI).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {
namespace lin {

struct Params {
    const __nv_bfloat16 *q, *k, *v;
    int64_t qs, ks, vs;  // elements from one token to the next
    const float *g;
    int32_t g_per_token;
    const int32_t *cu;  // NULL: every sequence has `steps` tokens
    int32_t steps;
    int32_t N;
    int64_t T;
    int64_t longest;  // with cu: sequences of more tokens are left out (the recurrence), of no more (chunks; negative: none is)
    int32_t H, rep;  // value heads; value heads per query/key head
    const float *s0;
    float scale;
    __nv_bfloat16 *o;
    float *sT;
    int32_t *status;
};

// A log decay below this counts as -inf: e^-138 is below 2^-126 times any finite bf16 ratio that could show
constexpr float G_FLOOR = -138.f;

constexpr int CHUNK = 128;  // tokens

// For tests of the failure detection: in each pass, the number of the chunk of each CTA whose v~ does not get its decays (-1: none).
struct Withhold {
    int32_t states = -1, outputs = -1;
};

// A part of a sequence that one CTA walks: tokens t0 .. t0 + len - 1 of sequence seq, its index-th of count segments; slot: where
// its state goes, if the sequence is cut.
struct Segment {
    int32_t t0, len, seq, index, count, slot;
};

// the recurrence, token after token (few tokens per sequence)
cudaError_t launch_recurrent(const Params &p, cudaStream_t stream);

// chunk by chunk on the tensor cores; the recurrence where sequences are short
cudaError_t launch_chunked(const Params &p, void *workspace, cudaStream_t stream, Withhold withhold);
size_t chunked_workspace_bytes(int64_t N, int64_t T, int64_t H);

}  // namespace lin
}  // namespace kda
