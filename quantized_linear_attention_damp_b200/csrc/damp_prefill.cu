// damp_prefill.cu -- prompts of a ragged batch through a decayed ("decay") or
// gated delta rule ("delta") layer, token by token: every d_k x d_v, bf16 or
// FP32 inputs, FP32 arithmetic throughout.
//
//   decay:  S <- alpha_t S + k_t v_t^T
//   delta:  S <- alpha_t S;  S <- S + beta_t k_t (v_t - S^T k_t)^T
//   out_t = S^T q_t
//
// The columns of S never meet, so a CTA takes one (request, head) and a group
// of columns and walks the tokens with the state in registers: NL lanes share
// a column, each holding 32 of its (up to 256) key rows; lane p of a column
// holds rows 4p + 4 NL i + (0..3), which makes the lanes' 16-byte reads of k
// and q adjacent.  A tile of tokens is staged in shared memory as FP32.
//
// What bounds it: the latency of one token's chain (k^T S, its shuffles, the
// update, q^T S), not bytes.  The bf16 128 x 128 layers take the chunked
// kernels instead (damp_prefill_chunk.cu).
#include <cuda_runtime.h>

#include <algorithm>

#include "damp.h"
#include "damp_device.cuh"

namespace damp {
namespace {

constexpr int kTokThreads = 128;
constexpr int kTile = 16;      // tokens staged at a time
constexpr int kRows = 32;      // key rows a lane holds

__device__ __forceinline__ float row_in(const void* base, long long i, bool bf16) {
    return bf16 ? __uint_as_float(
                      static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(base) + i)) << 16)
                : __ldg(static_cast<const float*>(base) + i);
}

template <int NL, bool DELTA>
__global__ void __launch_bounds__(kTokThreads) prefill_tokens_kernel(const PrefillArgs a) {
    constexpr int DK = NL * kRows;              // key rows with padding
    constexpr int CPC = kTokThreads / NL;       // columns a CTA owns
    __shared__ __align__(16) float s_k[kTile][DK];
    __shared__ __align__(16) float s_q[kTile][DK];
    __shared__ float s_v[kTile][CPC];
    __shared__ float s_al[kTile], s_be[kTile];
    const int tid = threadIdx.x, p = tid % NL, col = tid / NL;
    const int r = blockIdx.x, h = blockIdx.y;
    const int j = blockIdx.z * CPC + col;       // this thread's value column
    const bool bf16 = a.bf16;
    const int end = min(max(__ldg(a.cu_seqlens + r + 1), 0), a.max_tokens);
    const int start = min(max(__ldg(a.cu_seqlens + r), 0), end);
    if (start == end) return;
    const int slot = __ldg(a.store_slot + r), from = __ldg(a.load_slot + r);
    auto put = [&](int t, float x) {
        const size_t at = ((size_t)t * a.H + h) * a.d_v + j;
        if (bf16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(x);
        else static_cast<float*>(a.out)[at] = x;
    };
    if (slot < 0 || slot >= a.n_slots) {        // no state to leave: the rows read out zeros
        if (slot >= a.n_slots && tid == 0 && blockIdx.y == 0 && blockIdx.z == 0)
            atomicOr(a.status, DAMP_EFLAG_SLOT_RANGE);
        if (p == 0 && j < a.d_v)
            for (int t = start; t < end; ++t) put(t, 0.f);
        return;
    }
    const size_t unit = (size_t)h * a.d_k * a.d_v * 4;
    float* st = reinterpret_cast<float*>(
        a.state + (size_t)(a.state_by_slot ? slot : r) * a.state_stride + unit);
    const bool has = from >= 0 && from < a.n_slots;
    const float* ld = reinterpret_cast<const float*>(
        a.state + (size_t)(a.state_by_slot ? (has ? from : slot) : r) * a.state_stride + unit);
    auto row = [&](int i) { return 4 * p + 4 * NL * (i >> 2) + (i & 3); };
    float S[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        S[i] = has && row(i) < a.d_k && j < a.d_v ? ld[(size_t)row(i) * a.d_v + j] : 0.f;
    const int hq = h / (a.H / a.H_qk);

    for (int t0 = start; t0 < end; t0 += kTile) {
        const int nt = min(kTile, end - t0);
        __syncthreads();
        for (int e = tid; e < nt * DK; e += kTokThreads) {
            const int t = e / DK, i = e % DK;
            const bool in = i < a.d_k;
            s_k[t][i] = in ? row_in(a.k, (t0 + t) * a.k_stride + (long long)hq * a.d_k + i, bf16) : 0.f;
            s_q[t][i] = in ? row_in(a.q, (t0 + t) * a.q_stride + (long long)hq * a.d_k + i, bf16) : 0.f;
        }
        for (int e = tid; e < nt * CPC; e += kTokThreads) {
            const int t = e / CPC, c = blockIdx.z * CPC + e % CPC;
            s_v[t][e % CPC] =
                c < a.d_v ? row_in(a.v, (t0 + t) * a.v_stride + (long long)h * a.d_v + c, bf16) : 0.f;
        }
        if (tid < nt) {
            s_al[tid] = __ldg(a.alpha + (size_t)(t0 + tid) * a.H + h);
            if (DELTA) s_be[tid] = __ldg(a.beta + (size_t)(t0 + tid) * a.H + h);
        }
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            const float al = s_al[t];
            float4 k[kRows / 4];
#pragma unroll
            for (int i = 0; i < kRows / 4; ++i)
                k[i] = *reinterpret_cast<const float4*>(&s_k[t][4 * p + 4 * NL * i]);
            float d = s_v[t][col];
            if (DELTA) {
                float u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < kRows / 4; ++i) {
                    S[4 * i] *= al;
                    S[4 * i + 1] *= al;
                    S[4 * i + 2] *= al;
                    S[4 * i + 3] *= al;
                    u[0] = __fmaf_rn(k[i].x, S[4 * i], u[0]);
                    u[1] = __fmaf_rn(k[i].y, S[4 * i + 1], u[1]);
                    u[2] = __fmaf_rn(k[i].z, S[4 * i + 2], u[2]);
                    u[3] = __fmaf_rn(k[i].w, S[4 * i + 3], u[3]);
                }
                float s = (u[0] + u[1]) + (u[2] + u[3]);
#pragma unroll
                for (int off = NL / 2; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
                d = s_be[t] * (d - s);
            }
            float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kRows / 4; ++i) {
                const float4 q = *reinterpret_cast<const float4*>(&s_q[t][4 * p + 4 * NL * i]);
                if (!DELTA) {
                    S[4 * i] *= al;
                    S[4 * i + 1] *= al;
                    S[4 * i + 2] *= al;
                    S[4 * i + 3] *= al;
                }
                S[4 * i] = __fmaf_rn(k[i].x, d, S[4 * i]);
                S[4 * i + 1] = __fmaf_rn(k[i].y, d, S[4 * i + 1]);
                S[4 * i + 2] = __fmaf_rn(k[i].z, d, S[4 * i + 2]);
                S[4 * i + 3] = __fmaf_rn(k[i].w, d, S[4 * i + 3]);
                o[0] = __fmaf_rn(q.x, S[4 * i], o[0]);
                o[1] = __fmaf_rn(q.y, S[4 * i + 1], o[1]);
                o[2] = __fmaf_rn(q.z, S[4 * i + 2], o[2]);
                o[3] = __fmaf_rn(q.w, S[4 * i + 3], o[3]);
            }
            float s = (o[0] + o[1]) + (o[2] + o[3]);
#pragma unroll
            for (int off = NL / 2; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            if (p == 0 && j < a.d_v) put(t0 + t, s);
        }
    }
    if (j < a.d_v) {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (row(i) < a.d_k) st[(size_t)row(i) * a.d_v + j] = S[i];
    }
}

template <int NL>
cudaError_t launch_nl(const PrefillArgs& a, cudaStream_t s) {
    constexpr int CPC = kTokThreads / NL;
    const dim3 grid(a.n, a.H, (a.d_v + CPC - 1) / CPC);
    if (a.delta) prefill_tokens_kernel<NL, true><<<grid, kTokThreads, 0, s>>>(a);
    else prefill_tokens_kernel<NL, false><<<grid, kTokThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_tokens(const PrefillArgs& a, cudaStream_t s) {
    if (a.d_k <= 32) return launch_nl<1>(a, s);
    if (a.d_k <= 64) return launch_nl<2>(a, s);
    if (a.d_k <= 128) return launch_nl<4>(a, s);
    return launch_nl<8>(a, s);
}

}  // namespace damp
