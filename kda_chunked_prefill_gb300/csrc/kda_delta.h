// Internal interface of the delta rule with one decay per head (not part of the C ABI).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {
namespace delta {

constexpr int CHUNK = 64;  // tokens of a chunk

struct Params {
    const __nv_bfloat16 *q, *k, *v;
    int64_t qs, ks, vs;  // elements from one token to the next
    const float *g, *beta;
    const int32_t *cu;  // NULL: every sequence has `steps` tokens
    int32_t steps;
    int32_t N;
    int64_t T;
    int64_t longest;  // the recurrence with cu: sequences of more tokens are left out (negative: none is), but listed:
    int32_t *listed;  // [0] their chunks (of CHUNK tokens) in all, [1] 1 where some bounds are not in order, else 0
    int2 *list;       // the sequence and number of each of these chunks, a sequence's one after the other
    int64_t most;     // that there is room for (enough, where bounds are in order)
    int32_t H, rep;  // value heads; value heads per query/key head
    const float *s0;
    float scale;
    __nv_bfloat16 *o;
    float *sT;
    int32_t *status;
};

// the recurrence, token after token (few tokens per sequence)
cudaError_t launch_recurrent(const Params &p, cudaStream_t stream);

// chunk by chunk on the tensor cores; withhold, for tests of the failure detection: the number of the chunk of each CTA whose operand
// is not handed on to the tensor cores (-1: none)
cudaError_t launch_chunked(const Params &p, void *workspace, cudaStream_t stream, int withhold);
size_t chunked_workspace_bytes(int64_t N, int64_t T, int64_t H);

}  // namespace delta
}  // namespace kda
