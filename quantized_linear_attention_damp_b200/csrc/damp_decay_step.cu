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
#include <type_traits>

#include "damp.h"
#include "damp_device.cuh"
#include "damp_prompt.h"

namespace damp {
namespace {

constexpr int kDecayThreads = 256;

__device__ __forceinline__ float step_in(const void* base, size_t i, bool bf16) {
    return bf16 ? __uint_as_float(
                      static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(base) + i)) << 16)
                : __ldg(static_cast<const float*>(base) + i);
}

// Square d in {16, 32, 64}, and FP32 d = 128: the codec's thread tile (d/8 rows x 4 columns
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

// Every other shape, and quantized d = 128.  A block's rows need not be taken
// in key order (nothing passes from row to row), so they are taken as they are
// stored: first the byte rows, then the FP16 rows, in batches of 8 rows of one
// format (4 of FP32 states) and no test per row; q and k are put into that order
// once per unit.  A batch is one run of bytes: the warp copies it into its own
// ring in shared memory by asynchronous 16-byte copies, two batches ahead (one for
// d_v > 128) and across units (one batch ahead in registers kept 16 KB an SM in
// flight and reached 3 TB/s).  Lane l holds the column groups (of 4) l and, for d_v > 128
// (G = 2), l + 32.  One lane per row computes the row's scale: one division for
// 8 rows, not 8 by every lane.
//   SOLO: a warp owns a unit and all its batches; no barrier, no sum over
//   warps.  Otherwise the 8 warps of a CTA share a unit.
// Measured at 512 x 48 states of 128 x 128: mixed 227 us (4.5 TB/s, 69 % of the
// copy rate), INT8 225, FP8 233; the tile kernel above took 894 (one CTA an SM
// at 134 registers).  Of its limits issue is the nearest: dequantizing, two
// roundings and requantizing cost about 55 instructions a row of 128 values, and
// 71 % of the issue slots are used (256 x 32 states; DRAM 34 %).
//
// KIND: 0 FP32, 1 INT8 (and FP16) rows, 2 FP8 rows.  ALL: every lane holds
// columns (d_v = 128 G).
template <int G>
struct Ring {
    static constexpr int stages = G == 1 ? 3 : 2;
    static constexpr int slot = G * 2048 + 32;           // a batch and its scales
    static constexpr int bytes = kDecayThreads / 32 * stages * slot;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <int KIND, int G, bool SOLO, bool ALL>
__global__ void __launch_bounds__(kDecayThreads, G == 1 ? 3 : 2)
    decay_step_rows_kernel(const StepArgs a, int H_qk, int bf16) {
    constexpr bool F32 = KIND == 0, FP8 = KIND == 2;
    constexpr int B = F32 ? 4 : 8;         // rows of a batch: 512 G bytes of FP32, 128 G of codes, 256 G of FP16
    constexpr int kWarps = kDecayThreads / 32, kTeams = SOLO ? kWarps : 1, kTeam = kWarps / kTeams;
    constexpr int S = Ring<G>::stages;
    extern __shared__ __align__(16) uint8_t s_ring[];
    __shared__ __align__(16) float s_out[SOLO ? 1 : kWarps][SOLO ? 4 : G * 128];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int member = SOLO ? 0 : warp, mtid = SOLO ? lane : tid;   // this warp's and thread's place in its team
    const int d_k = a.d_k, d_v = ALL ? G * 128 : a.d_v, units = a.n * a.H;
    uint8_t* ring = s_ring + warp * S * Ring<G>::slot;
    // (q, q, k, k) of a row: the packed operations take pairs
    float4* s_qk = reinterpret_cast<float4*>(s_ring + Ring<G>::bytes) + (SOLO ? warp * d_k : 0);
    const int stride = gridDim.x * kTeams;
    const bool in[2] = {ALL || 4 * lane < d_v, G == 2 && (ALL || 4 * (lane + 32) < d_v)};

    struct Unit {
        uint8_t* blk;              // NULL: no block to step
        uint32_t f16, i8;          // offsets of the FP16 and of the byte rows
        int r8, batches;           // byte rows, all batches
        __device__ int b8() const { return (r8 + B - 1) / B; }   // batches of byte rows
    };
    auto find = [&](int u) -> Unit {
        Unit x{nullptr, 0, 0, 0, 0};
        if (u < units) {
            const int slot = __ldg(a.slot_idx + u / a.H);
            if (slot >= 0 && slot < a.n_slots) {
                const uint4 hb = __ldg(a.heads + u % a.H);
                x.blk = a.blocks + (size_t)slot * a.slot_stride + hb.x;
                x.f16 = hb.z;
                x.i8 = hb.w;
                const int r16 = F32 ? 0 : (int)(hb.w - hb.z) / (2 * d_v);
                x.r8 = d_k - r16;
                x.batches = x.b8() + (r16 + B - 1) / B;
            } else if (slot >= a.n_slots && mtid == 0) {
                atomicOr(a.status, DAMP_EFLAG_SLOT_RANGE);
            }
        }
        return x;
    };
    // ---- copies: the batches of this warp's units in the order in which they are worked on
    const int u0 = blockIdx.x * kTeams + (SOLO ? warp : 0);
    int pu = u0, pb = member, pslot = 0;
    Unit px = find(pu);
    auto issue = [&]() {
        while (pu < units && pb >= px.batches) {       // (a unit without a block has no batches)
            pu += stride;
            px = find(pu);
            pb = member;
        }
        if (pu < units) {
            const uint32_t dst = smem_u32(ring + pslot * Ring<G>::slot);
            const uint8_t* src;
            int bytes;
            if (F32) {
                src = px.blk + (size_t)pb * B * d_v * 4;
                bytes = B * d_v * 4;
            } else if (pb < px.b8()) {
                const int r0 = pb * B, rows = min(B, px.r8 - r0);
                src = px.blk + px.i8 + r0 * d_v;
                bytes = rows * d_v;
                if (lane < rows) copy4(dst + G * 2048 + lane * 4, px.blk + (r0 + lane) * 4);
            } else {
                const int r0 = (pb - px.b8()) * B, rows = min(B, d_k - px.r8 - r0);
                src = px.blk + px.f16 + r0 * d_v * 2;
                bytes = rows * d_v * 2;
            }
#pragma unroll
            for (int i = 0; i < G * 4; ++i) {
                const int at = (i * 32 + lane) * 16;
                if (at < bytes) copy16(dst + at, src + at);
            }
            pb += kTeam;
        }
        pslot = pslot + 1 == S ? 0 : pslot + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue();

    int u = u0, slot = 0;
    Unit x = find(u);
    while (u < units) {
        float* out = a.out + (size_t)u * d_v;
        if (!x.blk) {
            for (int j = mtid; j < d_v; j += kTeam * 32) out[j] = 0.f;
        } else {
            const int h = u % a.H;
            const size_t qk = ((size_t)(u / a.H) * H_qk + h / (a.H / H_qk)) * d_k;
            for (int i = mtid; i < d_k; i += kTeam * 32) {
                int at = i;                    // key row i's place in the stored order
                if (!F32 && x.r8 < d_k) {
                    const uint32_t* mask = a.masks + (size_t)h * kMaskWords;
                    int rank = 0;
                    for (int w = 0; w < i >> 5; ++w) rank += __popc(__ldg(mask + w));
                    const uint32_t m = __ldg(mask + (i >> 5));
                    rank += __popc(m & ((1u << (i & 31)) - 1u));
                    at = (m >> (i & 31)) & 1u ? x.r8 + rank : i - rank;
                }
                const float qi = step_in(a.q, qk + i, bf16), ki = step_in(a.k, qk + i, bf16);
                s_qk[at] = make_float4(qi, qi, ki, ki);
            }
            const float al = __ldg(a.alpha + u);
            float2 v[G][2], o[G][2];
#pragma unroll
            for (int c = 0; c < G; ++c) {
                const size_t at = (size_t)u * d_v + 4 * (lane + 32 * c);
                v[c][0] = v[c][1] = o[c][0] = o[c][1] = make_float2(0.f, 0.f);
                if (in[c]) {
                    v[c][0] = make_float2(step_in(a.v, at, bf16), step_in(a.v, at + 1, bf16));
                    v[c][1] = make_float2(step_in(a.v, at + 2, bf16), step_in(a.v, at + 3, bf16));
                }
            }
            if (SOLO) __syncwarp();
            else __syncthreads();
            for (int bi = member; bi < x.batches; bi += kTeam) {
                const bool byte = F32 || bi < x.b8();
                // rows of the stored order, and how many of the batch there are
                const int p0 = byte ? bi * B : x.r8 + (bi - x.b8()) * B, rows = min(B, (byte ? x.r8 : d_k) - p0);
                asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
                __syncwarp();
                const uint8_t* sl = ring + slot * Ring<G>::slot;
                slot = slot + 1 == S ? 0 : slot + 1;
                const float2 al2 = make_float2(al, al);
                issue();                       // into the slot of the batch before
                // N rows from row i0 of the batch: BYTE codes or FP16 (or FP32) values
                auto work = [&](auto byte_c, auto n_c, int i0) {
                    constexpr bool BYTE = decltype(byte_c)::value;
                    constexpr int N = decltype(n_c)::value;
                    float2 y[N][G][2];
                    float mine = 0.f;          // lane i: row i's largest magnitude
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        [[maybe_unused]] const float s =
                            BYTE ? reinterpret_cast<const float*>(sl + G * 2048)[i0 + i] : 0.f;
#pragma unroll
                        for (int c = 0; c < G; ++c) {
                            y[i][c][0] = y[i][c][1] = make_float2(0.f, 0.f);
                            if (!in[c]) continue;
                            if constexpr (F32) {
                                const float4 f =
                                    reinterpret_cast<const float4*>(sl)[(i0 + i) * (d_v / 4) + lane + 32 * c];
                                y[i][c][0] = make_float2(f.x, f.y);
                                y[i][c][1] = make_float2(f.z, f.w);
                            } else if constexpr (BYTE) {
                                const uint32_t w =
                                    reinterpret_cast<const uint32_t*>(sl)[(i0 + i) * (d_v / 4) + lane + 32 * c];
                                if (FP8) dequant_e4m3x4(w, s, y[i][c][0], y[i][c][1]);
                                else dequant_int8x4_packed(w, s, y[i][c][0], y[i][c][1]);
                            } else {
                                const uint32_t* row = reinterpret_cast<const uint32_t*>(sl) + (i0 + i) * (d_v / 2);
                                dequant_fp16x4(make_uint2(row[lane + 32 * c], row[d_v / 4 + lane + 32 * c]),
                                               y[i][c][0], y[i][c][1]);
                            }
                        }
                        const float4 qk4 = s_qk[p0 + i0 + i];
                        const float2 q2 = make_float2(qk4.x, qk4.y), k2 = make_float2(qk4.z, qk4.w);
                        float m = 0.f;
#pragma unroll
                        for (int c = 0; c < G; ++c) {
                            const float2 lo = __ffma2_rn(k2, v[c][0], __fmul2_rn(al2, y[i][c][0]));
                            const float2 hi = __ffma2_rn(k2, v[c][1], __fmul2_rn(al2, y[i][c][1]));
                            o[c][0] = __ffma2_rn(q2, lo, o[c][0]);
                            o[c][1] = __ffma2_rn(q2, hi, o[c][1]);
                            y[i][c][0] = lo;
                            y[i][c][1] = hi;
                            if (BYTE && in[c]) m = fmaxf(m, absmax4(lo, hi));
                        }
                        if (BYTE) {
                            m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
                            if (lane == i) mine = m;
                        }
                    }
                    float scale = 0.f, inv = 0.f;
                    if (BYTE && lane < N) {
                        row_scale<FP8>(mine, scale, inv);
                        reinterpret_cast<float*>(x.blk)[p0 + i0 + lane] = scale;
                    }
                    const int r = p0 + i0;
                    uint32_t* row = F32    ? reinterpret_cast<uint32_t*>(x.blk) + (size_t)r * d_v + 4 * lane
                                    : BYTE ? reinterpret_cast<uint32_t*>(x.blk + x.i8) + r * (d_v / 4) + lane
                                           : reinterpret_cast<uint32_t*>(x.blk + x.f16) + (r - x.r8) * (d_v / 2) + lane;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float iv = BYTE ? __shfl_sync(0xffffffffu, inv, i) : 0.f;
#pragma unroll
                        for (int c = 0; c < G; ++c) {
                            if (!in[c]) continue;
                            const float2 lo = y[i][c][0], hi = y[i][c][1];
                            if constexpr (F32) {
                                __stcs(reinterpret_cast<float4*>(row + (size_t)i * d_v + 128 * c),
                                       make_float4(lo.x, lo.y, hi.x, hi.y));
                            } else if constexpr (BYTE) {
                                __stcs(row + i * (d_v / 4) + 32 * c,
                                       FP8 ? quant_e4m3x4(lo, hi, iv) : quant_int8x4(lo, hi, iv));
                            } else {
                                const uint2 q = quant_fp16x4(lo, hi);
                                __stcs(row + i * (d_v / 2) + 32 * c, q.x);
                                __stcs(row + i * (d_v / 2) + d_v / 4 + 32 * c, q.y);
                            }
                        }
                    }
                };
                using Byte = std::true_type;
                using Value = std::false_type;
                using Full = std::integral_constant<int, B>;
                using One = std::integral_constant<int, 1>;
                if constexpr (F32) {
                    work(Value{}, Full{}, 0);
                } else if (byte) {
                    if (rows == B) work(Byte{}, Full{}, 0);
                    else
#pragma unroll 1
                        for (int i = 0; i < rows; ++i) work(Byte{}, One{}, i);
                } else if (KIND == 1) {
                    if (rows == B) work(Value{}, Full{}, 0);
                    else
#pragma unroll 1
                        for (int i = 0; i < rows; ++i) work(Value{}, One{}, i);
                }
            }
            if (SOLO) {
#pragma unroll
                for (int c = 0; c < G; ++c)
                    if (in[c])
                        reinterpret_cast<float4*>(out)[lane + 32 * c] =
                            make_float4(o[c][0].x, o[c][0].y, o[c][1].x, o[c][1].y);
                __syncwarp();                  // s_qk may be written again
            } else {
#pragma unroll
                for (int c = 0; c < G; ++c)
                    *reinterpret_cast<float4*>(&s_out[warp][4 * (lane + 32 * c)]) =
                        make_float4(o[c][0].x, o[c][0].y, o[c][1].x, o[c][1].y);
                __syncthreads();
                for (int j = tid; j < d_v; j += kDecayThreads) {
                    float s = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) s = __fadd_rn(s, s_out[w][j]);
                    out[j] = s;
                }
                __syncthreads();
            }
        }
        u += stride;
        x = find(u);
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

template <int KIND, int G, bool SOLO, bool ALL>
cudaError_t launch_rows_f(const StepArgs& a, int ctas, int H_qk, int bf16, cudaStream_t s) {
    const auto f = decay_step_rows_kernel<KIND, G, SOLO, ALL>;
    constexpr int base = Ring<G>::bytes, per_row = (SOLO ? kDecayThreads / 32 : 1) * 16;
    const int smem = base + per_row * a.d_k;
    // (the kernel's most, not this call's: another thread may be launching it too)
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               base + per_row * kMaxDim);
    if (e != cudaSuccess) return e;
    f<<<ctas, kDecayThreads, smem, s>>>(a, H_qk, bf16);
    return cudaGetLastError();
}

template <int KIND, int G>
cudaError_t launch_rows_t(const StepArgs& a, int H_qk, int bf16, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const int units = a.n * a.H, ctas = sms * (G == 1 ? 3 : 2), warps = kDecayThreads / 32;
    const bool all = a.d_v == 128 * G;
    // A warp per unit once two thirds of the warps have one (128 x 32 mixed d = 128 states 48.0 us
    // against 57.4 for a CTA per unit, 64 x 32: 35.7 against 32.3).
    if (units * 3ll >= 2ll * ctas * warps)
        return all ? launch_rows_f<KIND, G, true, true>(a, ctas, H_qk, bf16, s)
                   : launch_rows_f<KIND, G, true, false>(a, ctas, H_qk, bf16, s);
    return all ? launch_rows_f<KIND, G, false, true>(a, std::min(units, ctas), H_qk, bf16, s)
               : launch_rows_f<KIND, G, false, false>(a, std::min(units, ctas), H_qk, bf16, s);
}

template <int G>
cudaError_t launch_rows(const StepArgs& a, int H_qk, int bf16, cudaStream_t s) {
    switch (a.format) {
        case DAMP_FMT_FP32: return launch_rows_t<0, G>(a, H_qk, bf16, s);
        case DAMP_FMT_FP8_ROW: return launch_rows_t<2, G>(a, H_qk, bf16, s);
        default: return launch_rows_t<1, G>(a, H_qk, bf16, s);
    }
}

}  // namespace

cudaError_t launch_decay_step(const StepArgs& a, int in_dtype, int H_qk, cudaStream_t s) {
    const int bf16 = in_dtype == DAMP_DTYPE_BF16;
    if (a.d_k == a.d_v) switch (a.d_k) {
        case 16: return launch_square<16>(a, H_qk, bf16, s);
        case 32: return launch_square<32>(a, H_qk, bf16, s);
        case 64: return launch_square<64>(a, H_qk, bf16, s);
        case 128:
            if (a.format != DAMP_FMT_FP32) break;
            decay_step_kernel<128, false, false><<<a.n * a.H, kDecayThreads, 0, s>>>(a, H_qk, bf16);
            return cudaGetLastError();
        default: break;
    }
    return a.d_v > 128 ? launch_rows<2>(a, H_qk, bf16, s) : launch_rows<1>(a, H_qk, bf16, s);
}

}  // namespace damp
