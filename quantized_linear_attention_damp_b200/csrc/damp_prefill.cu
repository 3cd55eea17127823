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
// a column, each holding 32 or 16 of its (up to 256) key rows; lane p of a column
// holds rows 4p + 4 NL i + (0..3), which makes the lanes' 16-byte reads of k
// and q adjacent.  Tiles of 8 tokens come in by asynchronous copies, three
// tiles ahead, and are spread out as FP32 for the walk.
//
// What bounds it: the latency of one token's chain (k^T S, its shuffles, the
// update, q^T S), not bytes.  The bf16 128 x 128 layers take the chunked
// kernels instead (damp_prefill_chunk.cu).
#include <cuda_runtime.h>

#include <algorithm>

#include "damp.h"
#include "damp_device.cuh"
#include "damp_prompt.h"

namespace damp {
namespace {

constexpr int kTokThreads = 128;
constexpr int kTile = 8;       // tokens staged at a time
constexpr int kAhead = 3;      // tiles on their way while one is worked on

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Shared memory: FP32 tiles (k, q, v), then a ring of raw tiles: k, q and v rows
// as they are in memory, alpha and beta.
struct TokSmem {
    int k, q, v, raw, rk, rv, ra, raw_bytes, bytes;
    __host__ __device__ TokSmem(int NL, int kRows, int d_k, int esz) {
        const int DK = NL * kRows, CPC = kTokThreads / NL;
        k = 0;
        q = kTile * DK * 4;
        v = 2 * q;
        raw = v + kTile * CPC * 4;
        rk = d_k * esz;                 // a token's k or q row
        rv = CPC * esz;                 // its columns of v
        ra = kTile * (2 * rk + rv);     // offset of alpha, beta in a raw tile
        raw_bytes = ra + kTile * 8;
        bytes = raw + (kAhead + 1) * raw_bytes;
    }
};

template <int NL, int kRows, bool DELTA>
__global__ void __launch_bounds__(kTokThreads) prefill_tokens_kernel(const PrefillArgs a) {
    constexpr int DK = NL * kRows;              // key rows with padding
    constexpr int CPC = kTokThreads / NL;       // columns a CTA owns
    extern __shared__ __align__(16) uint8_t sm[];
    const int tid = threadIdx.x, p = tid % NL, col = tid / NL;
    const int r = a.order ? __ldg(a.order + blockIdx.x) : blockIdx.x, h = blockIdx.y;
    if (r < 0 || r >= a.n) return;
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
    float2 S[kRows / 2];
    auto from_state = [&](int i) {
        return has && row(i) < a.d_k && j < a.d_v ? ld[(size_t)row(i) * a.d_v + j] : 0.f;
    };
#pragma unroll
    for (int i = 0; i < kRows / 2; ++i) S[i] = make_float2(from_state(2 * i), from_state(2 * i + 1));
    const int hq = h / (a.H / a.H_qk), esz = bf16 ? 2 : 4;
    const TokSmem L(NL, kRows, a.d_k, esz);
    float (*s_k)[DK] = reinterpret_cast<float (*)[DK]>(sm + L.k);
    float (*s_q)[DK] = reinterpret_cast<float (*)[DK]>(sm + L.q);
    float (*s_v)[CPC] = reinterpret_cast<float (*)[CPC]>(sm + L.v);
    const int cols = min(CPC, a.d_v - (int)blockIdx.z * CPC);       // > 0: the grid covers d_v
    const uint8_t* kg = static_cast<const uint8_t*>(a.k) + (size_t)hq * a.d_k * esz;
    const uint8_t* qg = static_cast<const uint8_t*>(a.q) + (size_t)hq * a.d_k * esz;
    const uint8_t* vg = static_cast<const uint8_t*>(a.v) + ((size_t)h * a.d_v + (size_t)blockIdx.z * CPC) * esz;
    auto fetch = [&](int t0, int buf) {
        if (t0 < end) {
            const int nt = min(kTile, end - t0), nk = L.rk / 16, nv = cols * esz / 16;
            const uint32_t dst = smem_u32(sm + L.raw + buf * L.raw_bytes);
            for (int e = tid; e < nt * nk; e += kTokThreads) {
                const int t = e / nk, i = e % nk * 16;
                copy16(dst + t * L.rk + i, kg + (size_t)(t0 + t) * a.k_stride * esz + i);
                copy16(dst + (kTile + t) * L.rk + i, qg + (size_t)(t0 + t) * a.q_stride * esz + i);
            }
            for (int e = tid; e < nt * nv; e += kTokThreads) {
                const int t = e / nv, i = e % nv * 16;
                copy16(dst + 2 * kTile * L.rk + t * L.rv + i, vg + (size_t)(t0 + t) * a.v_stride * esz + i);
            }
            if (tid < nt) {
                copy4(dst + L.ra + 4 * tid, a.alpha + (size_t)(t0 + tid) * a.H + h);
                if (DELTA) copy4(dst + L.ra + 4 * (kTile + tid), a.beta + (size_t)(t0 + tid) * a.H + h);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // rows of `n` values to FP32 rows of `width`, four values at a time
    auto spread = [&](float* to, int width, const uint8_t* from, int row, int n, int nt) {
        const int n4 = n / 4;
        for (int e = tid; e < nt * n4; e += kTokThreads) {
            const int t = e / n4, i = e % n4;
            float4 f;
            if (bf16) {
                const uint2 w = *reinterpret_cast<const uint2*>(from + t * row + i * 8);
                f = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                                __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
            } else {
                f = *reinterpret_cast<const float4*>(from + t * row + i * 16);
            }
            *reinterpret_cast<float4*>(to + t * width + i * 4) = f;
        }
    };
    // key rows behind d_k stay zero
    for (int e = tid; e < 2 * kTile * (DK - a.d_k); e += kTokThreads)
        s_k[0][e / (DK - a.d_k) * DK + a.d_k + e % (DK - a.d_k)] = 0.f;   // (q follows k)
    for (int i = 0; i < kAhead; ++i) fetch(start + i * kTile, i);
    int buf = 0;

    for (int t0 = start; t0 < end; t0 += kTile, buf = (buf + 1) % (kAhead + 1)) {
        const int nt = min(kTile, end - t0);
        fetch(t0 + kAhead * kTile, (buf + kAhead) % (kAhead + 1));
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
        __syncthreads();
        const uint8_t* raw = sm + L.raw + buf * L.raw_bytes;
        spread(&s_k[0][0], DK, raw, L.rk, a.d_k, nt);
        spread(&s_q[0][0], DK, raw + kTile * L.rk, L.rk, a.d_k, nt);
        spread(&s_v[0][0], CPC, raw + 2 * kTile * L.rk, L.rv, cols, nt);
        const float* s_al = reinterpret_cast<const float*>(raw + L.ra);
        const float* s_be = s_al + kTile;
        __syncthreads();
        // one token; returns this lane's part of its readout
        auto step = [&](int t) -> float {
            const float2 al = make_float2(s_al[t], s_al[t]);
            float2 k[kRows / 2];
#pragma unroll
            for (int i = 0; i < kRows / 4; ++i) {
                const float4 f = *reinterpret_cast<const float4*>(&s_k[t][4 * p + 4 * NL * i]);
                k[2 * i] = make_float2(f.x, f.y);
                k[2 * i + 1] = make_float2(f.z, f.w);
            }
            float d = s_v[t][col];
#pragma unroll
            for (int i = 0; i < kRows / 2; ++i) S[i] = __fmul2_rn(al, S[i]);
            if (DELTA) {
                float2 u[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int i = 0; i < kRows / 2; ++i) u[i & 1] = __ffma2_rn(k[i], S[i], u[i & 1]);
                float s = (u[0].x + u[0].y) + (u[1].x + u[1].y);
#pragma unroll
                for (int off = NL / 2; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
                d = s_be[t] * (d - s);
            }
            const float2 d2 = make_float2(d, d);
            float2 o[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int i = 0; i < kRows / 4; ++i) {
                const float4 q = *reinterpret_cast<const float4*>(&s_q[t][4 * p + 4 * NL * i]);
                S[2 * i] = __ffma2_rn(k[2 * i], d2, S[2 * i]);
                S[2 * i + 1] = __ffma2_rn(k[2 * i + 1], d2, S[2 * i + 1]);
                o[0] = __ffma2_rn(make_float2(q.x, q.y), S[2 * i], o[0]);
                o[1] = __ffma2_rn(make_float2(q.z, q.w), S[2 * i + 1], o[1]);
            }
            return (o[0].x + o[0].y) + (o[1].x + o[1].y);
        };
        // the readouts' sums over lanes come behind the tile's last token: eight
        // independent ones, and none of them in a token's chain
        float o[kTile];
        if (nt == kTile) {
#pragma unroll
            for (int t = 0; t < kTile; ++t) o[t] = step(t);
        } else {
#pragma unroll
            for (int t = 0; t < kTile; ++t) o[t] = t < nt ? step(t) : 0.f;
        }
#pragma unroll
        for (int off = NL / 2; off >= 1; off >>= 1)
#pragma unroll
            for (int t = 0; t < kTile; ++t) o[t] += __shfl_xor_sync(0xffffffffu, o[t], off);
#pragma unroll
        for (int t = 0; t < kTile; ++t)
            if (p == t % NL && t < nt && j < a.d_v) put(t0 + t, o[t]);
        __syncthreads();
    }
    if (j < a.d_v) {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (row(i) < a.d_k) st[(size_t)row(i) * a.d_v + j] = i & 1 ? S[i / 2].y : S[i / 2].x;
    }
}

template <int NL, int R>
cudaError_t launch_nl(const PrefillArgs& a, cudaStream_t s) {
    constexpr int CPC = kTokThreads / NL;
    const dim3 grid(a.n, a.H, (a.d_v + CPC - 1) / CPC);
    const auto f = a.delta ? prefill_tokens_kernel<NL, R, true> : prefill_tokens_kernel<NL, R, false>;
    const int smem = TokSmem(NL, R, a.d_k, a.bf16 ? 2 : 4).bytes;
    // (the kernel's most, not this call's: another thread may be launching it too)
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               TokSmem(NL, R, NL * R, 4).bytes);
    if (e != cudaSuccess) return e;
    f<<<grid, kTokThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_tokens(const PrefillArgs& a, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    // 32 rows a lane give the fewest instructions; where that leaves less than
    // three CTAs an SM, one token's latency counts, and 16 rows a lane halve its
    // chain (2048 tokens x 16 heads: 96 x 160 decay rule 470 -> 410 us)
    const int nl32 = a.d_k <= 32 ? 1 : a.d_k <= 64 ? 2 : a.d_k <= 128 ? 4 : 8;
    const long long ctas = (long long)a.n * a.H * ((a.d_v * nl32 + kTokThreads - 1) / kTokThreads);
    if (ctas >= 3 * sms) switch (nl32) {
        case 1: return launch_nl<1, 32>(a, s);
        case 2: return launch_nl<2, 32>(a, s);
        case 4: return launch_nl<4, 32>(a, s);
        default: return launch_nl<8, 32>(a, s);
    }
    if (a.d_k <= 16) return launch_nl<1, 16>(a, s);
    if (a.d_k <= 32) return launch_nl<2, 16>(a, s);
    if (a.d_k <= 64) return launch_nl<4, 16>(a, s);
    if (a.d_k <= 128) return launch_nl<8, 16>(a, s);
    return launch_nl<16, 16>(a, s);
}

}  // namespace damp
