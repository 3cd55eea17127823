// damp_prompt.h -- arguments and launchers of the batch plan, the decay-rule
// step and the prompt prefill.
#pragma once
#include "damp_internal.h"

namespace damp {

// Test hooks of the prefill's block kernels (DAMP_HOOK_FAIL_HALF, DAMP_HOOK_HOLD_FIRST_KERNEL,
// DAMP_HOOK_NO_TENSOR_MAPS).
constexpr uint32_t kHookFailHalf = 2u;
constexpr uint32_t kHookHoldFirstKernel = 4u;
constexpr uint32_t kHookNoTensorMaps = 8u;

// Arguments of the batch-plan kernel (damp_plan.cu).
struct PlanArgs {
    const int32_t* lengths;
    const int32_t* past;       // may be NULL: no request has tokens in its state yet
    const int32_t* slot_idx;
    int n, n_slots, max_tokens, max_blocks;
    int32_t* cu_seqlens;       // [n + 1]
    int32_t* load_slot;        // [n]
    int32_t* store_slot;       // [n]
    int32_t* block_table;      // [max_blocks][4]
    int32_t* token_slot;       // [max_tokens] (both token maps or neither)
    int32_t* token_pos;        // [max_tokens]
    int32_t* totals;           // [4]
    int32_t* order;            // [n] or NULL
};

// Arguments of the prefill kernels (damp_prefill.cu, damp_prefill_chunk.cu).
// States are FP32 [d_k][d_v]: state (r, h) at state + index*state_stride +
// h*d_k*d_v*4 bytes, where index is the request's slot (FP32 pools, read and
// written in place) or r itself (state = workspace, filled by unpack).
struct PrefillArgs {
    const int32_t* cu_seqlens;
    const int32_t* load_slot;
    const int32_t* store_slot;
    const int32_t* block_table;
    const int32_t* order;      // [n] requests in the order in which they are started; NULL: as they come
    const void* q;
    const void* k;
    const void* v;
    long long q_stride, k_stride, v_stride;   // elements between token rows
    const float* alpha;        // [max_tokens][H]
    const float* beta;         // [max_tokens][H]; NULL for the decay rule
    void* out;                 // [max_tokens][H][d_v], type of q
    uint8_t* state;
    unsigned long long state_stride;   // bytes between two indices
    int state_by_slot;         // 1: index = slot, 0: index = request
    uint32_t* status;
    int n, max_tokens, H, H_qk, d_k, d_v, n_slots;
    int delta;                 // 1: gated delta rule, 0: decay rule
    int bf16;
    unsigned long long wait_ns;
    uint32_t hooks;            // test hooks (kHook...)
    uint8_t* work;             // chunk kernels' workspace
    int max_blocks;
};

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t stream);
// One token of the decay rule on the pool's blocks, every shape and format
// (damp_decay_step.cu); a.beta is not read.
cudaError_t launch_decay_step(const StepArgs& a, int in_dtype, int H_qk, cudaStream_t stream);
// Prompts, token by token (damp_prefill.cu): every shape and input type.
cudaError_t launch_prefill_tokens(const PrefillArgs& a, cudaStream_t stream);
// Prompts in blocks of 64 tokens on the tensor cores (damp_prefill_chunk.cu):
// bf16 inputs, 128 x 128 states.  prepare_prefill looks up the driver's tensor-
// map encoder and sets the kernels' attributes (damp_pool_create calls it ahead of
// the first prefill, whose launch asks again and reports what is missing).
cudaError_t prepare_prefill(uint32_t hooks);
bool prefill_chunk_fits(int d_k, int d_v, int bf16);
size_t prefill_chunk_bytes(int n, int H, int max_tokens, int max_blocks, int delta);
cudaError_t launch_prefill_chunk(const PrefillArgs& a, cudaStream_t stream);

}  // namespace damp
