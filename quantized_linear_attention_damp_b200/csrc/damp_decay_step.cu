// damp_decay_step.cu -- one token of a decayed linear-attention layer without
// the delta rule, on the pool's compressed states (damp_decay_step):
//   S'_ij = fl(alpha S^_ij);  X_ij = fma(k_i, v_j, S'_ij);  out_j = sum_i q_i X_ij
// with X stored back in the pool's format.  The rounding points, the row
// formats and the quantizer are the decode step's (damp_device.cuh).
//
// What bounds it: HBM, each block read once and written once (4 flops per
// state value).  Without the delta rule no row needs another row's value
// before it is updated, so a thread keeps its tile in registers from the load
// to the store and the only exchange between warps is the readout's sum.
#include <cuda_runtime.h>

#include <algorithm>

#include "damp.h"
#include "damp_device.cuh"

namespace damp {
namespace {

constexpr int kDecayThreads = 256;

__device__ __forceinline__ float step_in(const void* base, size_t i, bool bf16) {
    return bf16 ? __uint_as_float(
                      static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(base) + i)) << 16)
                : __ldg(static_cast<const float*>(base) + i);
}

// Square d in {16, 32, 64, 128}: the codec's thread tile (d/8 rows x 4 columns
// a thread, 128/d units a CTA), so a row maximum stays inside a warp.
template <int D, bool QUANT, bool FP8>
__global__ void __launch_bounds__(kDecayThreads) decay_step_kernel(const StepArgs a, int H_qk,
                                                                   int bf16) {
    using G = Geo<D>;
    constexpr int RPT = G::RPT, UPI = G::UPI, LPR = G::LPR;
    __shared__ float rowbuf_all[UPI * 8 * 2 * RPT];
    __shared__ float s_out[UPI][8][D];
    const int tid = threadIdx.x;
    const int ui = tid / G::TPU, tu = tid % G::TPU;
    const int cg = tu % LPR, rg = tu / LPR, r0 = rg * RPT;
    float* rowbuf = rowbuf_all + (ui * 8 + rg) * 2 * RPT;
    const int u = blockIdx.x * UPI + ui;
    const bool live = u < a.n * a.H;   // uniform over a unit's threads (2d: whole warps)
    const int b = live ? u / a.H : 0, h = live ? u % a.H : 0;
    const int slot = live ? __ldg(a.slot_idx + b) : -1;
    const bool ok = slot >= 0 && slot < a.n_slots;
    if (slot >= a.n_slots && tu == 0) atomicOr(a.status, DAMP_EFLAG_SLOT_RANGE);
    if (ok) {
        const uint4 hb = __ldg(a.heads + h);
        uint8_t* blk = a.blocks + (size_t)slot * a.slot_stride + hb.x;
        uint32_t bits = 0;
        int rank16 = 0;
        float2 x[RPT][2];
        if constexpr (QUANT) {
            const uint4 mw = __ldg(reinterpret_cast<const uint4*>(a.masks + (size_t)h * kMaskWords));
            row_formats<D>(mw, r0, bits, rank16);
            load_tile_mask<D, FP8>(blk, hb.z, hb.w, bits, rank16, r0, cg, x);
        } else {
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float4 f = *reinterpret_cast<const float4*>(
                    blk + ((size_t)(r0 + i) * D + 4 * cg) * 4);
                x[i][0] = make_float2(f.x, f.y);
                x[i][1] = make_float2(f.z, f.w);
            }
        }
        const size_t qk = ((size_t)b * H_qk + h / (a.H / H_qk)) * D + r0;
        const float al = __ldg(a.alpha + u);
        float v[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = step_in(a.v, (size_t)u * D + 4 * cg + c, bf16);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float k = step_in(a.k, qk + i, bf16), q = step_in(a.q, qk + i, bf16);
            x[i][0].x = __fmaf_rn(k, v[0], __fmul_rn(al, x[i][0].x));
            x[i][0].y = __fmaf_rn(k, v[1], __fmul_rn(al, x[i][0].y));
            x[i][1].x = __fmaf_rn(k, v[2], __fmul_rn(al, x[i][1].x));
            x[i][1].y = __fmaf_rn(k, v[3], __fmul_rn(al, x[i][1].y));
            o[0] = __fmaf_rn(q, x[i][0].x, o[0]);
            o[1] = __fmaf_rn(q, x[i][0].y, o[1]);
            o[2] = __fmaf_rn(q, x[i][1].x, o[2]);
            o[3] = __fmaf_rn(q, x[i][1].y, o[3]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) s_out[ui][rg][4 * cg + c] = o[c];
        if constexpr (QUANT) {
            store_quant_tile<D, FP8>(blk, hb.z, hb.w, bits, rank16, r0, cg, x, rowbuf);
        } else {
#pragma unroll
            for (int i = 0; i < RPT; ++i)
                *reinterpret_cast<float4*>(blk + ((size_t)(r0 + i) * D + 4 * cg) * 4) =
                    make_float4(x[i][0].x, x[i][0].y, x[i][1].x, x[i][1].y);
        }
    }
    __syncthreads();
    if (live && tu < D) {   // the readout of 8 row groups, in a fixed order
        float s = 0.f;
        if (ok) {
#pragma unroll
            for (int g = 0; g < 8; ++g) s = __fadd_rn(s, s_out[ui][g][tu]);
        }
        a.out[(size_t)u * D + tu] = s;
    }
}

// Every other d_k x d_v: one CTA per unit, warp w takes key rows w, w + 8, ...;
// lane l holds columns l, l + 32, ... of its row.
constexpr int kWarps = kDecayThreads / 32;
constexpr int kCols = kMaxDim / 32;

__global__ void __launch_bounds__(kDecayThreads) decay_step_any_kernel(const StepArgs a, int codec,
                                                                       int H_qk, int bf16) {
    __shared__ float s_out[kWarps][kMaxDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d_k = a.d_k, d_v = a.d_v;
    const long long u = blockIdx.x;
    const int b = (int)(u / a.H), h = (int)(u % a.H);
    const int slot = __ldg(a.slot_idx + b);
    const bool ok = slot >= 0 && slot < a.n_slots;
    if (slot >= a.n_slots && threadIdx.x == 0) atomicOr(a.status, DAMP_EFLAG_SLOT_RANGE);
    float o[kCols] = {};
    if (ok) {
        const uint4 hb = __ldg(a.heads + h);
        uint8_t* blk = a.blocks + (size_t)slot * a.slot_stride + hb.x;
        const size_t qk = ((size_t)b * H_qk + h / (a.H / H_qk)) * d_k;
        const float al = __ldg(a.alpha + u);
        float v[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
            const int j = lane + 32 * c;
            v[c] = j < d_v ? step_in(a.v, (size_t)u * d_v + j, bf16) : 0.f;
        }
        for (int i = warp; i < d_k; i += kWarps) {
            const uint32_t e = codec ? __ldg(a.dir + (size_t)h * d_k + i) : 0u;
            const bool byte_row = codec && !(e >> 31);
            float* scale_at = reinterpret_cast<float*>(blk + dir_scale(e));
            const float s = byte_row ? *scale_at : 1.f;
            const float k = step_in(a.k, qk + i, bf16), q = step_in(a.q, qk + i, bf16);
            uint8_t* row = codec ? blk + dir_row(e) : blk + (size_t)i * d_v * 4;
            float x[kCols], m = 0.f;
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const int j = lane + 32 * c;
                if (j >= d_v) break;
                float f;
                if (!codec) f = reinterpret_cast<const float*>(row)[j];
                else if (!byte_row) f = __half2float(*reinterpret_cast<const __half*>(row + f16_pos(j, d_v)));
                else if (codec == 2) f = __fmul_rn(e4m3_value(row[j]), s);
                else f = __fmul_rn((float)(int8_t)row[j], s);
                x[c] = __fmaf_rn(k, v[c], __fmul_rn(al, f));
                o[c] = __fmaf_rn(q, x[c], o[c]);
                m = fmaxf(m, fabsf(x[c]));
            }
            float sc = 0.f, inv = 0.f;
            if (byte_row) {   // the warp has read the whole row (and its scale) before it writes
                m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
                if (codec == 2) row_scale<true>(m, sc, inv);
                else row_scale<false>(m, sc, inv);
                if (lane == 0) *scale_at = sc;
            }
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const int j = lane + 32 * c;
                if (j >= d_v) break;
                if (!codec) reinterpret_cast<float*>(row)[j] = x[c];
                else if (!byte_row) *reinterpret_cast<__half*>(row + f16_pos(j, d_v)) = __float2half_rn(x[c]);
                else if (codec == 2) row[j] = inv == 0.f ? 0 : e4m3_code(__fmul_rn(x[c], inv));
                else row[j] = (uint8_t)(__float_as_uint(__fmaf_rn(x[c], inv, 12582912.0f)) & 0xffu);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < kCols; ++c) s_out[warp][lane + 32 * c] = o[c];
    __syncthreads();
    for (int j = threadIdx.x; j < d_v; j += kDecayThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s = __fadd_rn(s, s_out[w][j]);
        a.out[(size_t)u * d_v + j] = s;
    }
}

template <int D>
cudaError_t launch_square(const StepArgs& a, int H_qk, int bf16, cudaStream_t s) {
    const int units = a.n * a.H, grid = (units + Geo<D>::UPI - 1) / Geo<D>::UPI;
    if (a.format == DAMP_FMT_FP32) decay_step_kernel<D, false, false><<<grid, kDecayThreads, 0, s>>>(a, H_qk, bf16);
    else if (a.format == DAMP_FMT_FP8_ROW) decay_step_kernel<D, true, true><<<grid, kDecayThreads, 0, s>>>(a, H_qk, bf16);
    else decay_step_kernel<D, true, false><<<grid, kDecayThreads, 0, s>>>(a, H_qk, bf16);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_step(const StepArgs& a, int in_dtype, int H_qk, cudaStream_t s) {
    const int bf16 = in_dtype == DAMP_DTYPE_BF16;
    if (a.d_k == a.d_v) switch (a.d_k) {
        case 16: return launch_square<16>(a, H_qk, bf16, s);
        case 32: return launch_square<32>(a, H_qk, bf16, s);
        case 64: return launch_square<64>(a, H_qk, bf16, s);
        case 128: return launch_square<128>(a, H_qk, bf16, s);
        default: break;
    }
    const int codec = a.format == DAMP_FMT_FP32 ? 0 : a.format == DAMP_FMT_FP8_ROW ? 2 : 1;
    decay_step_any_kernel<<<a.n * a.H, kDecayThreads, 0, s>>>(a, codec, H_qk, bf16);
    return cudaGetLastError();
}

}  // namespace damp
