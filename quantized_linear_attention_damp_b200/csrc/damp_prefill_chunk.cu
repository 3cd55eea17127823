// damp_prefill_chunk.cu -- prompts in blocks of 64 tokens on the 5th-generation
// tensor cores (bf16 inputs, d_k = d_v = 128), both rules.
//
// With gamma_t the product of a block's decays up to token t, Gamma_ts =
// gamma_t / gamma_s, and S the state before the block (rows of Q, K, V are
// tokens):
//   delta rule:  (I + A) U = diag(beta) (V - diag(gamma) K S),
//                A_ts = beta_t Gamma_ts k_t.k_s  (s < t)
//                O  = diag(gamma) Q S + (Q K^T o Gamma) U       (s <= t)
//                S <- gamma_C S + K^T diag(gamma_C / gamma) U
//   decay rule:  the same with U = V.
// delta: two kernels.
//   prepare (one CTA per block and head, no order between blocks): what does not
//     depend on S: T' = (I + A)^-1 diag(beta) and P = Q K^T o Gamma, so that with
//     R = V - diag(gamma) K S and U = T' R:  O = diag(gamma) Q S + P U and
//     S <- gamma_C S + K^T diag(gamma_C / gamma) U.
//   chain (one CTA per request and head, blocks in order): the products with
//     S, transposed so that the 128 value columns are the M dimension of every
//     matrix instruction and S^T, R^T and U^T are A operands in TMEM.
// decay: one kernel, a chain likewise, that forms its operands itself.
// S itself stays in the state warps' registers in FP32 from the first block to
// the last: a block's part comes out of TMEM and is added with one rounding
// (accumulating in TMEM over all blocks would let the tensor core's truncated
// sums drift).
//
// Precision: Q, K and V enter as the bf16 they are, accumulation is FP32.  The
// FP32 operands of whatever a state is made of (S in K S, T' and R in T' R,
// diag(w) U; diag(w) V of the decay rule) enter as three bf16 terms, which hold
// all their bits; the product of two such keeps every pair of terms down to
// 2^-18 (6 of 9).  Pairs are not enough there: with equal keys T' alternates in
// sign, T' R cancels, and what the pairs had lost came to 1e-3 of the state
// (beta |k|^2 = 1.9, where the recurrence is stable and FP32 sums of the same
// form keep 2e-5); values that cancel under a slow decay lost 3e-4.
// What only a readout is made of (P and U in P U, P V, S in Q S) enters as a
// pair, hi + mid, which leaves 2^-17 of it: a readout is rounded to bf16 (2^-8)
// afterwards.  (As G R with G = P T', which needs no U, the readout would cancel
// as T' R does: 1.4e-3 of it lost with equal keys.)
//
// Decays are running products, never quotients or exponentials of sums: a
// decay of zero inside a block, or products that underflow, need no care.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "damp.h"
#include "damp_tcgen05.cuh"
#include "damp_prompt.h"

namespace damp {
namespace {

constexpr int C = DAMP_PLAN_BLOCK;     // tokens of a block
constexpr int D = 128;                 // d_k = d_v
constexpr int kSms = 148;              // of a B200: how work is cut, not how it is launched
static_assert(C == 64, "the kernels' tiles are 64 tokens");

constexpr int kMat = C * C * 2;                                  // 8192
__device__ __forceinline__ uint32_t swz(int row, int byte) {     // byte in 0..127 of a 128-byte row
    return (uint32_t)(row * 128 + (byte ^ ((row & 7) << 4)));
}

struct ChunkArgs {
    PrefillArgs p;
    int32_t* first_block;      // [n] index of each request's first block
    uint8_t* records;          // [max_blocks][H] DRec
};

// ------------------------------------------------------------------ shared

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
constexpr int kPrepThreads = 128;

constexpr int kTile = C * D * 2;       // bytes of a Q, K or V tile: two halves of 64 channels
constexpr int kHalf = kTile / 2;

// Products of a block's decays up to each of a lane's two tokens, and behind them (a warp; lane l:
// tokens 2 l and 2 l + 1).  In 64 bits, rounded once: gamma_C multiplies every element of a state, so an
// error of it is the same for all of them, and where a head's decay does not change it is the same in
// every block.  (As FP32 products 4096 tokens of such a head came out 7e-5 off, a rounding a block is 2e-6.)
__device__ __forceinline__ void decay_products(float a0, float a1, int lane, float2& upto, float2& behind) {
    double up = (double)a0 * a1, down = up;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double u = __shfl_up_sync(0xffffffffu, up, off), d = __shfl_down_sync(0xffffffffu, down, off);
        if (lane >= off) up = u * up;
        if (lane + off < 32) down = down * d;
    }
    double before = __shfl_up_sync(0xffffffffu, up, 1), rest = __shfl_down_sync(0xffffffffu, down, 1);
    if (lane == 0) before = 1.0;
    if (lane == 31) rest = 1.0;
    upto = make_float2((float)(before * a0), (float)up);
    behind = make_float2((float)(a1 * rest), (float)rest);
}

// Waits for a phase of an mbarrier, at most wait_ns; gives up at once where
// another warp gave up.  A patient waiter (the loader, whose waits are long
// and not on the chain) sleeps between its looks: polling takes shared-memory
// bandwidth from everyone else.
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, uint64_t wait_ns,
                                             volatile int* abort, bool patient) {
    uint64_t began = 0;
    for (uint32_t n = 1; !mbar_try_wait_short(bar, parity); ++n) {
        if (patient) __nanosleep(200);
        if (n & 255u) continue;                // (the timer is slow to read)
        if (*abort) return false;
        const uint64_t now = global_ns();
        if (!began) began = now;
        if (now - began > wait_ns) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

// ------------------------------------------------------------------ delta: prepare
//
// 128 threads a (block, head), four CTAs an SM: the steps are short and each waits
// for the one before, so it is the number of resident CTAs that keeps the SM busy.
// [Q; K] K^T is one tensor-core product of 128 rows; a thread then has one row of
// Q K^T (warps 0, 1) or K K^T (warps 2, 3) and multiplies the decays up along it.
// The inverse is FP32 arithmetic of the ordinary kind: an error of it is an error
// of the state.  Q and K share their 32 KB with A and T (FP32) and then with T'.
// (8672 units: 157 us, 38 % of the issue slots, DRAM 44 %, tensor pipe 5 %.)

// The record of one (block, head): C x C bf16 matrices with 128-byte rows
// (K-major, 128-byte swizzle) as the chain's products take them, gamma_t
// and gamma_C / gamma_t, and a word that says whether the record is there: a
// prepare that gives up at a wait leaves kMissing in it, and the chain then
// leaves its state as it was.
constexpr uint32_t kThere = 1u, kMissing = 0u;
struct DRec {
    static constexpr int th = 0, tm = kMat, tl = 2 * kMat;   // T' hi, mid, lo
    static constexpr int ph = 3 * kMat, pm = 4 * kMat;       // P hi, mid
    static constexpr int gam = 5 * kMat, w = gam + 4 * C, there = w + 4 * C;
    static constexpr int bytes = there + 16;
};

constexpr int kFA = C + 4;             // floats of a row of A and T
struct DPrep {
    static constexpr int qk = 0;                       // Q0 K0 Q1 K1: halves of 64 channels
    static constexpr int a = 0, t = C * kFA * 4;       // over Q and K
    static constexpr int img = 0;                      // T', over A and T
    static constexpr int end = 2 * C * kFA * 4;        // the record from P on
    static constexpr int vec = end + DRec::bytes - DRec::ph;           // alpha, beta
    static constexpr int bytes = vec + 2 * C * 4 + 1024;
    static_assert(2 * kTile <= end && DRec::ph <= end && vec % 16 == 0, "Q and K, and T', fit over A and T");
    static constexpr uint32_t cols = 64;               // TMEM: [Q; K] K^T
};

__global__ void __launch_bounds__(kPrepThreads, 4)
    delta_prepare_kernel(const ChunkArgs ca, const __grid_constant__ CUtensorMap mq,
                         const __grid_constant__ CUtensorMap mk) {
    const PrefillArgs& a = ca.p;
    extern __shared__ __align__(1024) uint8_t sm_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ __align__(8) uint64_t s_bar[3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // heads of a block run side by side: their rows of Q and K are neighbours in memory
    const int blk = blockIdx.x / a.H, h = blockIdx.x % a.H;
    const int4 row = __ldg(reinterpret_cast<const int4*>(a.block_table) + blk);
    const int req = row.x, t0 = row.y, len = row.z;
    if (req < 0 || req >= a.n || t0 < 0 || len < 1 || len > C || t0 > a.max_tokens - len) return;
    if (h == 0 && row.w == 0 && tid == 0) ca.first_block[req] = blk;
    const int slot = __ldg(a.store_slot + req);
    if (slot < 0 || slot >= a.n_slots) return;
    const uint32_t base = (smem_u32(sm_raw) + 1023u) & ~1023u;
    uint8_t* sm = sm_raw + (base - smem_u32(sm_raw));
    float* s_al = reinterpret_cast<float*>(sm + DPrep::vec);
    float* s_be = s_al + C;
    uint8_t* img = sm + DPrep::img;
    uint8_t* img2 = sm + DPrep::end - DRec::ph;        // the record's places from P on
    float* s_ga = reinterpret_cast<float*>(img2 + DRec::gam);
    float* s_w = reinterpret_cast<float*>(img2 + DRec::w);
    const uint32_t bar_in = smem_u32(&s_bar[0]), bar_mma = smem_u32(&s_bar[1]), bar_drain = smem_u32(&s_bar[2]);

    if (warp == 0) {
        if (elect_one()) {
            mbar_init(bar_in, 1);
            mbar_init(bar_mma, 1);
            mbar_init(bar_drain, 1);
            fence_mbar_init();
            s_abort = 0;
            const int hq = h / (a.H / a.H_qk);
            if (!(a.hooks & (kHookHoldFirstItem | kHookHoldFirstKernel))) {
                mbar_arrive_expect_tx(bar_in, 2 * kTile);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    tma_load_3d(base + DPrep::qk + half * kTile, &mq, half * 64, hq, t0, bar_in);
                    tma_load_3d(base + DPrep::qk + half * kTile + kHalf, &mk, half * 64, hq, t0, bar_in);
                }
            }
        }
        __syncwarp();
        tmem_alloc(smem_u32(&s_tmem), DPrep::cols);
    } else if (warp == 1) {
        // decays, two tokens a lane: as they are, their products up to each token and behind it
        const float* al = a.alpha + (size_t)t0 * a.H + h;
        const float* be = a.beta + (size_t)t0 * a.H + h;
        const int i = 2 * lane;
        const float a0 = i < len ? __ldg(al + (size_t)i * a.H) : 1.f;
        const float a1 = i + 1 < len ? __ldg(al + (size_t)(i + 1) * a.H) : 1.f;
        const float b0 = i < len ? __ldg(be + (size_t)i * a.H) : 0.f;
        const float b1 = i + 1 < len ? __ldg(be + (size_t)(i + 1) * a.H) : 0.f;
        reinterpret_cast<float2*>(s_al)[lane] = make_float2(a0, a1);
        reinterpret_cast<float2*>(s_be)[lane] = make_float2(b0, b1);
        decay_products(a0, a1, lane, reinterpret_cast<float2*>(s_ga)[lane], reinterpret_cast<float2*>(s_w)[lane]);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem, lanes = tm + ((uint32_t)(warp * 32) << 16);

    // ---- [Q; K] K^T
    bool ok = true;
    if (warp == 0) {
        ok = __all_sync(0xffffffffu, bounded_wait(bar_in, 0, a.wait_ns, &s_abort, false));
        if (ok && len < C) {
            // rows behind the request's end hold another request's keys, NaN for all we know
            for (int e = lane; e < (C - len) * 16; e += 32)
                *reinterpret_cast<uint4*>(sm + DPrep::qk + (e & 8 ? kTile : 0) + kHalf + (len + e / 16) * 128 +
                                          (e & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
        }
        if (ok && elect_one()) {
            constexpr uint32_t id = mma_idesc(128, 64, false, false);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint32_t at = base + DPrep::qk + (ks >> 2) * kTile + (ks & 3) * 32;
                mma_ss(tm, desc_k_major(at), desc_k_major(at + kHalf), id, ks > 0);
            }
            tc_commit(bar_mma);
        }
        // one warp polls, the others wait at the barrier: polling takes shared-memory bandwidth
        ok = ok && __all_sync(0xffffffffu, bounded_wait(bar_mma, 0, a.wait_ns, &s_abort, false));
    }
    const bool fine = __syncthreads_and(ok);       // (a wait that ran out: nothing more is done)
    tc_fence_after();
    float* s_a = reinterpret_cast<float*>(sm + DPrep::a);
    float* s_t = reinterpret_cast<float*>(sm + DPrep::t);
    const int r0 = warp * 16;
    if (fine) {
        // ---- row t of P (as a pair) or of A = diag(beta) K K^T o Gamma below the diagonal
        const int t = (warp & 1) * 32 + lane;
        const bool is_p = warp < 2;
        // gamma_t / gamma_s from s = t down (times beta_t for A), zero above; rows of P behind the
        // request's end are used by no one
        const float first = is_p ? 1.f : s_be[t];
        float x = 0.f, above = 1.f;                // above: alpha_{s + 1}
#pragma unroll
        for (int part = 1; part >= 0; --part) {
            if (part > (warp & 1)) {               // above the diagonal: P is zero, A is not read
                if (is_p)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        *reinterpret_cast<uint4*>(img2 + DRec::ph + swz(t, part * 64 + j * 16)) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4*>(img2 + DRec::pm + swz(t, part * 64 + j * 16)) = make_uint4(0, 0, 0, 0);
                    }
                continue;
            }
            uint32_t y[32];
            tmem_ld32(lanes + part * 32, y);
            tmem_wait_ld();
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                const float4 a1 = *reinterpret_cast<const float4*>(s_al + part * 32 + j * 8 + 4);
                const float4 a0 = *reinterpret_cast<const float4*>(s_al + part * 32 + j * 8);
                const float as[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
                float f[8];
#pragma unroll
                for (int i = 7; i >= 0; --i) {
                    const float z = x * above;
                    x = part * 32 + j * 8 + i == t ? first : z;
                    above = as[i];
                    f[i] = (is_p ? x : z) * __uint_as_float(y[j * 8 + i]);     // A: zero on the diagonal
                }
                if (is_p) {
                    uint4 hi, mid;
                    split_bf16(f[0], f[1], hi.x, mid.x);
                    split_bf16(f[2], f[3], hi.y, mid.y);
                    split_bf16(f[4], f[5], hi.z, mid.z);
                    split_bf16(f[6], f[7], hi.w, mid.w);
                    *reinterpret_cast<uint4*>(img2 + DRec::ph + swz(t, part * 64 + j * 16)) = hi;
                    *reinterpret_cast<uint4*>(img2 + DRec::pm + swz(t, part * 64 + j * 16)) = mid;
                } else {
                    float4* to = reinterpret_cast<float4*>(s_a + t * kFA + part * 32 + j * 8);
                    to[0] = make_float4(f[0], f[1], f[2], f[3]);
                    to[1] = make_float4(f[4], f[5], f[6], f[7]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (fine) {
    // ---- T = (I + A)^-1, lower triangle: the four 16 x 16 diagonal blocks by
    // substitution (a lane a column), then pairs of blocks, then halves: the
    // block below the diagonal is -T22 (A21 T11).  The unused upper blocks of
    // T hold A21 T11.
    if (lane < 16) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v0 = i == lane ? 1.f : 0.f, v1 = 0.f;
            const float* ar = s_a + (r0 + i) * kFA + r0;
#pragma unroll
            for (int k = 0; k < i; k += 4) {
                const float4 av = *reinterpret_cast<const float4*>(ar + k);
                v0 = __fmaf_rn(-av.x, x[k], v0);
                if (k + 1 < i) v1 = __fmaf_rn(-av.y, x[k + 1], v1);
                if (k + 2 < i) v0 = __fmaf_rn(-av.z, x[k + 2], v0);
                if (k + 3 < i) v1 = __fmaf_rn(-av.w, x[k + 3], v1);
            }
            x[i] = v0 + v1;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) s_t[(r0 + i) * kFA + r0 + lane] = x[i];
    }
    __syncthreads();
    {
        // blocks (1, 0) and (3, 2), two warps each
        const int m = (tid >> 6) * 32, i = (tid & 63) >> 2, j = (tid & 3) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        auto product = [&](const float* lhs, const float* rhs) {      // rows of 16, steps of 4
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
                const float4 av = *reinterpret_cast<const float4*>(lhs + k);
                const float l[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const float4 tv = *reinterpret_cast<const float4*>(rhs + (k + kk) * kFA);
                    r.x = __fmaf_rn(l[kk], tv.x, r.x);
                    r.y = __fmaf_rn(l[kk], tv.y, r.y);
                    r.z = __fmaf_rn(l[kk], tv.z, r.z);
                    r.w = __fmaf_rn(l[kk], tv.w, r.w);
                }
            }
            return r;
        };
        x = product(s_a + (m + 16 + i) * kFA + m, s_t + m * kFA + m + j);
        *reinterpret_cast<float4*>(&s_t[(m + i) * kFA + m + 16 + j]) = x;
        __syncthreads();
        const float4 y = product(s_t + (m + 16 + i) * kFA + m + 16, s_t + m * kFA + m + 16 + j);
        __syncthreads();
        *reinterpret_cast<float4*>(&s_t[(m + 16 + i) * kFA + m + j]) = make_float4(-y.x, -y.y, -y.z, -y.w);
        *reinterpret_cast<float4*>(&s_t[(m + i) * kFA + m + 16 + j]) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    {
        // the lower left 32 x 32 block: 2 rows x 4 columns a thread; a warp's
        // columns (first product) or rows (second) bound the triangle it needs
        float x[2][4] = {}, y[2][4] = {};
        auto product = [&](float (&r)[2][4], const float* l0, const float* rhs, int k0, int k1) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                if (k < k0 || k >= k1) continue;      // the same for the whole warp
                const float4 a0 = *reinterpret_cast<const float4*>(l0 + k);
                const float4 a1 = *reinterpret_cast<const float4*>(l0 + kFA + k);
                const float l[2][4] = {{a0.x, a0.y, a0.z, a0.w}, {a1.x, a1.y, a1.z, a1.w}};
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const float4 tv = *reinterpret_cast<const float4*>(rhs + (k + kk) * kFA);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        r[i][0] = __fmaf_rn(l[i][kk], tv.x, r[i][0]);
                        r[i][1] = __fmaf_rn(l[i][kk], tv.y, r[i][1]);
                        r[i][2] = __fmaf_rn(l[i][kk], tv.z, r[i][2]);
                        r[i][3] = __fmaf_rn(l[i][kk], tv.w, r[i][3]);
                    }
                }
            }
        };
        {
            const int i = (lane >> 1) * 2, j = warp * 8 + (lane & 1) * 4;       // columns by warp
            product(x, s_a + (32 + i) * kFA, s_t + j, warp * 8, 32);
            *reinterpret_cast<float4*>(&s_t[i * kFA + 32 + j]) = make_float4(x[0][0], x[0][1], x[0][2], x[0][3]);
            *reinterpret_cast<float4*>(&s_t[(i + 1) * kFA + 32 + j]) = make_float4(x[1][0], x[1][1], x[1][2], x[1][3]);
        }
        __syncthreads();
        {
            const int i = warp * 8 + (lane >> 3) * 2, j = (lane & 7) * 4;       // rows by warp
            product(y, s_t + (32 + i) * kFA + 32, s_t + 32 + j, 0, warp * 8 + 8);
            *reinterpret_cast<float4*>(&s_t[(32 + i) * kFA + j]) = make_float4(-y[0][0], -y[0][1], -y[0][2], -y[0][3]);
            *reinterpret_cast<float4*>(&s_t[(33 + i) * kFA + j]) = make_float4(-y[1][0], -y[1][1], -y[1][2], -y[1][3]);
        }
    }
    __syncthreads();
    // ---- T' = T diag(beta) as three bf16 terms in the record's image (over A and T: through registers).
    // Behind the request's end beta is zero, so those columns vanish, and A has no such rows.
    {
        const int s = (tid & 15) * 4, r = tid >> 4;       // 4 columns, rows r, r + 8, ...
        const float4 be = *reinterpret_cast<const float4*>(s_be + s);
        uint2 hi[C / 8], mid[C / 8], lo[C / 8];
#pragma unroll
        for (int i = 0; i < C / 8; ++i) {
            const int t = r + 8 * i;
            const float4 tv = *reinterpret_cast<const float4*>(&s_t[t * kFA + s]);
            split3_bf16(make_float2(s <= t ? tv.x * be.x : 0.f, s + 1 <= t ? tv.y * be.y : 0.f), hi[i].x, mid[i].x,
                        lo[i].x);
            split3_bf16(make_float2(s + 2 <= t ? tv.z * be.z : 0.f, s + 3 <= t ? tv.w * be.w : 0.f), hi[i].y,
                        mid[i].y, lo[i].y);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < C / 8; ++i) {
            *reinterpret_cast<uint2*>(img + DRec::th + swz(r + 8 * i, s * 2)) = hi[i];
            *reinterpret_cast<uint2*>(img + DRec::tm + swz(r + 8 * i, s * 2)) = mid[i];
            *reinterpret_cast<uint2*>(img + DRec::tl + swz(r + 8 * i, s * 2)) = lo[i];
        }
    }
    if (tid == 0) *reinterpret_cast<uint32_t*>(img2 + DRec::there) = kThere;
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        if (s_abort) {
            // nothing in flight when TMEM and shared memory are given back
            mbar_wait_bounded(bar_in, 0, a.wait_ns);
            if (elect_one()) tc_commit(bar_drain);
            mbar_wait_bounded(bar_drain, 0, a.wait_ns);
        }
        tmem_free(tm, DPrep::cols);
        uint8_t* record = ca.records + ((size_t)blk * a.H + h) * DRec::bytes;
        if (s_abort) {
            if (lane == 0) {
                *reinterpret_cast<uint32_t*>(record + DRec::there) = kMissing;
                atomicOr(a.status, DAMP_EFLAG_TIMEOUT);
            }
        } else if (elect_one()) {
            bulk_s2g(record, smem_u32(img), DRec::ph);
            bulk_s2g(record + DRec::ph, smem_u32(img2 + DRec::ph), DRec::bytes - DRec::ph);
            bulk_commit();
            bulk_wait_read<0>();
        }
    }
}

// ------------------------------------------------------------------ delta: chain

// One CTA of 22 warps a (request, head): 16 keep the state and form the A
// operands (warp w: TMEM lanes of w & 3, a quarter of the columns), 4 form U's
// pair and write the readout, one loads, one issues the matrix instructions.
//
// What bounds it is the chain of one block after another: S as three terms -> K S
// -> R as terms -> U -> U as terms -> the block's part of S -> S.  So Q S and P U
// are products of their own behind the ones the chain waits for (K and Q as one
// operand of 128 rows cost less, but the chain waits for all of them), and S's
// update and K S go by halves of the key channels: one half's product runs while
// the other half's state is split.
struct DChain {
    static constexpr int kWarps = 16, kOut = 4;              // state warps, readout warps
    static constexpr int kStages = 2;
    static constexpr int threads = 32 * (kWarps + kOut + 2);
    static constexpr int kq = 0, v = 2 * kTile, rec = 3 * kTile;   // K, Q by halves of 64 channels: K0 Q0 K1 Q1
    static constexpr int stage = (rec + DRec::bytes + 1023) / 1024 * 1024;
    static constexpr int out = kStages * stage;              // readout rows, 16 bytes apart in banks
    static constexpr int out_row = D * 2 + 16;
    static constexpr int bar = out + C * out_row;
    static constexpr int bytes = bar + 256 + 1024;
    // TMEM columns
    static constexpr uint32_t dS = 0;       // the block's part of S^T, FP32 [128 v][128 k]
    static constexpr uint32_t S = 128;      // S^T hi, mid, lo (64 columns each)
    static constexpr uint32_t R = 0;        // R^T hi, mid, lo (32 each), while dS is not needed
    static constexpr uint32_t U = 160;      // (diag(w) U)^T hi, mid, lo (64 apart), over S's terms of the channels'
                                            // second half: the first half's next terms are written while the
                                            // second half's product still reads U
    static constexpr uint32_t KS = 320;     // (K S)^T, FP32 [128][64], then U^T in its place: R is formed, and
                                            // K S with it read, before T' R is issued.  Then U^T hi and mid for
                                            // P U: 16 tokens' 8 + 8 columns over the 16 they were read from
    static constexpr uint32_t QS = 384, PU = 448;   // (Q S)^T, (P U)^T
    // Barriers.  B*: a product is done (KS; U; Q S and P U; S's two halves).  C*: the state warps have
    // left an operand in TMEM (S's halves, R, diag(w) U), the readout's U; CO: the readout is out of TMEM.
    enum { Full = 0, Empty = kStages, BK = 2 * kStages, BU, BO, BS, CS = BS + 2, CR = CS + 2, CU, CV, CO, Drain };
};

__global__ void __launch_bounds__(DChain::threads, 1)
    delta_chain_kernel(const ChunkArgs ca, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using X = DChain;
    const PrefillArgs& a = ca.p;
    extern __shared__ __align__(1024) uint8_t sm_raw[];
    const uint32_t base = (smem_u32(sm_raw) + 1023u) & ~1023u;
    uint8_t* sm = sm_raw + (base - smem_u32(sm_raw));
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int at = blockIdx.x / a.H, h = blockIdx.x % a.H, req = a.order ? __ldg(a.order + at) : at;
    if (req < 0 || req >= a.n) return;
    const int cu0 = __ldg(a.cu_seqlens + req), cu1 = __ldg(a.cu_seqlens + req + 1);
    const int slot = __ldg(a.store_slot + req), from = __ldg(a.load_slot + req), block0 = ca.first_block[req];
    const int end = min(max(cu1, 0), a.max_tokens), start = min(max(cu0, 0), end), len = end - start;
    if (len == 0) return;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((size_t)start * a.H + h) * D;
    if (slot < 0 || slot >= a.n_slots) {
        if (slot >= a.n_slots && tid == 0 && h == 0) atomicOr(a.status, DAMP_EFLAG_SLOT_RANGE);
        for (long long e = tid; e < (long long)len * (D / 8); e += X::threads)
            reinterpret_cast<uint4*>(out + (e / (D / 8)) * (size_t)a.H * D)[e % (D / 8)] =
                make_uint4(0, 0, 0, 0);
        return;
    }
    const int nc = (len + C - 1) / C;
    // a plan's first_block + nc always fits; anything else is kept inside the workspace
    const int fb = min(max(block0, 0), max(a.max_blocks - nc, 0));
    auto bar = [&](int i) { return base + X::bar + 8 * i; };

    constexpr int wLoad = X::kWarps + X::kOut, wMma = wLoad + 1;
    auto load = [&](int c) {                           // one lane: block c into its stage
        const int hq = h / (a.H / a.H_qk), t = start + c * C;
        const uint32_t st = base + c % X::kStages * X::stage, f = bar(X::Full + c % X::kStages);
        mbar_arrive_expect_tx(f, 3 * kTile + DRec::bytes);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            tma_load_3d(st + X::kq + half * kTile, &mk, half * 64, hq, t, f);
            tma_load_3d(st + X::kq + half * kTile + kHalf, &mq, half * 64, hq, t, f);
            tma_load_3d(st + X::v + half * kHalf, &mv, half * 64, h, t, f);
        }
        bulk_g2s(st + X::rec, ca.records + ((size_t)(fb + c) * a.H + h) * DRec::bytes, DRec::bytes, f);
        // a stage is not free early enough to cover DRAM's latency: the next blocks come to L2
        // ahead of their turn
        const int n = c + X::kStages, tn = start + n * C;
        if (n < nc) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                tma_prefetch_3d(&mk, half * 64, hq, tn);
                tma_prefetch_3d(&mq, half * 64, hq, tn);
                tma_prefetch_3d(&mv, half * 64, h, tn);
            }
            bulk_prefetch(ca.records + ((size_t)(fb + n) * a.H + h) * DRec::bytes, DRec::bytes);
        }
    };
    if (warp == wLoad) {
        if (elect_one()) {
            for (int i = 0; i < X::kStages; ++i) {
                mbar_init(bar(X::Full + i), 1);
                mbar_init(bar(X::Empty + i), X::kWarps / 2 + X::kOut);
            }
            for (int i = X::BK; i < X::CS; ++i) mbar_init(bar(i), 1);
            mbar_init(bar(X::CS), X::kWarps / 2);
            mbar_init(bar(X::CS + 1), X::kWarps / 2);
            mbar_init(bar(X::CR), X::kWarps);
            mbar_init(bar(X::CU), X::kWarps);
            mbar_init(bar(X::CV), X::kOut);
            mbar_init(bar(X::CO), X::kOut);
            mbar_init(bar(X::Drain), 1);
            fence_mbar_init();
            s_abort = 0;
            // the first blocks are on their way before the rest of the CTA is ready
            for (int c = a.hooks & kHookHoldFirstItem ? 1 : 0; c < min(nc, X::kStages); ++c) load(c);
        }
        __syncwarp();
    } else if (warp == wMma) {
        tmem_alloc(smem_u32(&s_tmem), 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;

    auto wait_all = [&](int i, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, bounded_wait(bar(i), parity, a.wait_ns, &s_abort,
                                                    warp == X::kWarps + X::kOut));
    };
    // A group of warps waits by one of them polling and the others at a hardware
    // barrier: 20 polling warps would take the shared-memory pipe from the matrix
    // instructions' operands.  All of the group get the same answer.
    auto wait_group = [&](bool polls, int i, uint32_t parity, int id, int threads, bool go = true) -> bool {
        const bool ok = go && (!polls || wait_all(i, parity));
        return !bar_red_or(id, threads, !ok);
    };
    auto arrive = [&](int i) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(i));
    };
    const int quad = warp & 3;
    const uint32_t lanes = tm + ((uint32_t)(quad * 32) << 16);
    const int vcol = quad * 32 + lane;                 // a state or readout thread's value column

    if (warp < X::kWarps) {
        // ---------------------------------------------------------- state
        const int part = warp >> 2;                    // key channels [32 part, +32), tokens [16 part, +16)
        const size_t unit = (size_t)h * D * D * 4;
        const bool has = from >= 0 && from < a.n_slots;
        float S[32];
        {
            const float* in = reinterpret_cast<const float*>(
                a.state + (size_t)(a.state_by_slot ? (has ? from : slot) : req) * a.state_stride + unit);
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = has ? in[(size_t)(part * 32 + i) * D + vcol] : 0.f;
        }
        // The warps of one half of the channels wait for their own half alone.  A wait that runs out in one
        // half need not run out in the other, so it is carried (good) to the next wait of all state warps:
        // they leave the loop together, and no half is left at a barrier that the other will not reach.
        bool ok = true, good = true;
        auto wait_half = [&](int i, uint32_t parity) -> bool {
            const bool polls = quad + (part & 1) == 0;
            bool fine = !polls || wait_all(i, parity);
            if (polls && (a.hooks & kHookFailHalf) && part / 2 == (h & 1)) {
                s_abort = 1;
                fine = false;
            }
            return !bar_red_or(2 + part / 2, X::kWarps * 16, !fine);
        };
        for (int c = 0; c < nc; ++c) {
            const uint32_t ph = c & 1;
            uint8_t* st = sm + (c % X::kStages) * X::stage;
            const float* gam = reinterpret_cast<const float*>(st + X::rec + DRec::gam);
            const float* w = reinterpret_cast<const float*>(st + X::rec + DRec::w);
            // ---- the state before block c as three terms
            uint32_t h8[8], m8[8], l8[8];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    split3_bf16(make_float2(S[16 * j + 2 * i], S[16 * j + 2 * i + 1]), h8[i], m8[i], l8[i]);
                tmem_st8(lanes + X::S + part * 16 + j * 8, h8);
                tmem_st8(lanes + X::S + 64 + part * 16 + j * 8, m8);
                tmem_st8(lanes + X::S + 128 + part * 16 + j * 8, l8);
            }
            const int live = min(C, len - c * C);         // tokens of block c
            if (live < C) {
                // rows behind the request's end hold another request's keys and values:
                // they must not enter the sums over tokens
                good = good && wait_half(X::Full + c % X::kStages, (c / X::kStages) & 1);
                if (good) {
                    // (a half of the channels by the warps that hand over that half)
                    for (int e = tid % (X::kWarps * 16); e < (C - live) * 8; e += X::kWarps * 16) {
                        const int at = (live + e / 8) * 128 + (e % 8) * 16;
                        *reinterpret_cast<uint4*>(st + X::kq + part / 2 * kTile + at) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4*>(st + X::v + part / 2 * kHalf + at) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
            }
            tmem_wait_st();
            if (good) arrive(X::CS + part / 2);
            // ---- R = V - diag(gamma) K S
            if (!(ok = wait_group(warp == 0, X::Full + c % X::kStages, (c / X::kStages) & 1, 4, X::kWarps * 32,
                                  good)))
                break;
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int t = part * 16 + i;
                const uint16_t b = *reinterpret_cast<const uint16_t*>(
                    st + X::v + (vcol >> 6) * kHalf + swz(t, (vcol & 63) * 2));
                v[i] = __uint_as_float((uint32_t)b << 16);
            }
            uint32_t x[16];
            // (the decays of R behind the wait, the factors of U ahead of theirs, as measured: with both
            // ahead a thread's registers do not suffice, 579 us against 551 for 8192 tokens x 32 heads)
            if (!(ok = wait_group(warp == 0, X::BK, ph, 4, X::kWarps * 32))) break;
            tc_fence_after();
            tmem_ld16(lanes + X::KS + part * 16, x);
            float g[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = reinterpret_cast<const float4*>(gam + part * 16)[i];
                g[4 * i] = f.x, g[4 * i + 1] = f.y, g[4 * i + 2] = f.z, g[4 * i + 3] = f.w;
            }
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                split3_bf16(make_float2(__fmaf_rn(-g[2 * i], __uint_as_float(x[2 * i]), v[2 * i]),
                                        __fmaf_rn(-g[2 * i + 1], __uint_as_float(x[2 * i + 1]), v[2 * i + 1])),
                            h8[i], m8[i], l8[i]);
            tmem_st8(lanes + X::R + part * 8, h8);
            tmem_st8(lanes + X::R + 32 + part * 8, m8);
            tmem_st8(lanes + X::R + 64 + part * 8, l8);
            tmem_wait_st();
            arrive(X::CR);
            // ---- diag(w) U as three terms
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = reinterpret_cast<const float4*>(w + part * 16)[i];
                g[4 * i] = f.x, g[4 * i + 1] = f.y, g[4 * i + 2] = f.z, g[4 * i + 3] = f.w;
            }
            if (!(ok = wait_group(warp == 0, X::BU, ph, 4, X::kWarps * 32))) break;
            tc_fence_after();
            tmem_ld16(lanes + X::KS + part * 16, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                split3_bf16(make_float2(g[2 * i] * __uint_as_float(x[2 * i]),
                                        g[2 * i + 1] * __uint_as_float(x[2 * i + 1])),
                            h8[i], m8[i], l8[i]);
            tmem_st8(lanes + X::U + part * 8, h8);
            tmem_st8(lanes + X::U + 64 + part * 8, m8);
            tmem_st8(lanes + X::U + 128 + part * 8, l8);
            const float gc = gam[C - 1];
            const bool there = *reinterpret_cast<const uint32_t*>(st + X::rec + DRec::there) == kThere;
            tmem_wait_st();
            arrive(X::CU);
            // ---- S <- gamma_C S + the block's part
            good = wait_half(X::BS + part / 2, ph);
            if (!there) s_abort = 1;           // (for every thread, or none)
            good = good && there;
            if (!good) continue;               // (to the next wait of all, or the last one below)
            tc_fence_after();
            uint32_t y[32];
            tmem_ld32(lanes + X::dS + part * 32, y);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = __fmaf_rn(gc, S[i], __uint_as_float(y[i]));
            // Of the state's side the stage is used up: every state warp had its values out before the
            // second half's product was issued.  (P U is the readout's.)
            if (part >= 2 && lane == 0) mbar_arrive(bar(X::Empty + c % X::kStages));
        }
        // (all state warps are here, or none: the waits that leave the loop are waits of all)
        if (ok) ok = !bar_red_or(4, X::kWarps * 32, !good);
        if (ok) {
            float* to = reinterpret_cast<float*>(
                a.state + (size_t)(a.state_by_slot ? slot : req) * a.state_stride + unit);
#pragma unroll
            for (int i = 0; i < 32; ++i) to[(size_t)(part * 32 + i) * D + vcol] = S[i];
        }
    } else if (warp < X::kWarps + X::kOut) {
        // ---------------------------------------------------------- readout
        const int wt = tid - X::kWarps * 32;
        uint8_t* so = sm + X::out;
        for (int c = 0; c < nc; ++c) {
            const float* gam = reinterpret_cast<const float*>(sm + (c % X::kStages) * X::stage + X::rec + DRec::gam);
            // U as a pair for P U, once the state warps have read it (8192 tokens x 32 heads: 50 us more where
            // they form it themselves)
            if (!wait_group(warp == X::kWarps, X::CU, c & 1, 1, X::kOut * 32)) break;
            tc_fence_after();
#pragma unroll 1
            for (int part = 0; part < 4; ++part) {
                uint32_t x[16], u[16];
                tmem_ld16(lanes + X::KS + part * 16, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    split_bf16(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]), u[i], u[8 + i]);
                tmem_st16(lanes + X::KS + part * 16, u);
            }
            tmem_wait_st();
            arrive(X::CV);
            if (!wait_group(warp == X::kWarps, X::BO, c & 1, 1, X::kOut * 32)) break;
            tc_fence_after();
            // out of TMEM first: the next block's Q S waits for that
#pragma unroll
            for (int part = 0; part < 4; ++part) {
                uint32_t o1[16], o2[16];
                tmem_ld16(lanes + X::QS + part * 16, o1);
                tmem_ld16(lanes + X::PU + part * 16, o2);
                float2 gt[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) gt[i] = *reinterpret_cast<const float2*>(gam + part * 16 + 2 * i);
                tmem_wait_ld();
                if (part == 3) {
                    arrive(X::CO);
                    if (lane == 0) mbar_arrive(bar(X::Empty + c % X::kStages));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t o = pack_bf16(
                        __fmaf_rn(gt[i].x, __uint_as_float(o1[2 * i]), __uint_as_float(o2[2 * i])),
                        __fmaf_rn(gt[i].y, __uint_as_float(o1[2 * i + 1]), __uint_as_float(o2[2 * i + 1])));
                    uint8_t* to = so + (part * 16 + 2 * i) * X::out_row + vcol * 2;
                    *reinterpret_cast<uint16_t*>(to) = (uint16_t)o;
                    *reinterpret_cast<uint16_t*>(to + X::out_row) = (uint16_t)(o >> 16);
                }
            }
            bar_sync(1, X::kOut * 32);
            const int live = min(C, len - c * C);
#pragma unroll
            for (int i = 0; i < C * 16 / (X::kOut * 32); ++i) {
                const int r = (wt >> 4) + i * (X::kOut * 2), u = wt & 15;
                if (r < live)
                    *reinterpret_cast<uint4*>(out + (size_t)(c * C + r) * a.H * D + u * 8) =
                        *reinterpret_cast<const uint4*>(so + r * X::out_row + u * 16);
            }
            bar_sync(1, X::kOut * 32);
        }
    } else if (warp == wLoad) {
        // ---------------------------------------------------------- loads
        int issued = min(nc, X::kStages);
        for (int c = X::kStages; c < nc; ++c) {
            if (!wait_all(X::Empty + c % X::kStages, (c / X::kStages - 1) & 1)) break;
            if (elect_one()) load(c);
            issued = c + 1;
        }
        // copies in flight end before the CTA does
        for (int c = max(0, issued - X::kStages); c < issued; ++c)
            mbar_wait_bounded(bar(X::Full + c % X::kStages), (c / X::kStages) & 1, a.wait_ns);
    } else {
        // ---------------------------------------------------------- matrix instructions
        // One at a time in order; what the state warps wait for goes first, the
        // readout's products run while they work on its result.
        constexpr uint32_t idk = mma_idesc(128, 64, false, false), idmn = mma_idesc(128, 64, false, true);
        for (int c = 0; c < nc; ++c) {
            const uint32_t st = base + (c % X::kStages) * X::stage, rec = st + X::rec;
            const uint32_t ph = c & 1;
            if (!wait_all(X::Full + c % X::kStages, (c / X::kStages) & 1)) break;
            if (c > 0 && !wait_all(X::BO, ph ^ 1)) break;     // (P U read the columns that K S is written to)
            // (K S)^T, the channels' first half as soon as it is there.  Small terms go first here and
            // below: the tensor core truncates its sums, the less the smaller they are.
            bool ok = true;
#pragma unroll
            for (int half = 0; half < 2 && ok; ++half) {
                if (!(ok = wait_all(X::CS + half, ph))) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 12; ++ks)
                        mma_ts(tm + X::KS, tm + X::S + (2 - (ks >> 2)) * 64 + half * 32 + (ks & 3) * 8,
                               desc_k_major(st + X::kq + half * kTile + (ks & 3) * 32), idk, half + ks > 0);
                    if (half == 1) tc_commit(bar(X::BK));
                }
            }
            if (!ok) break;
            // (Q S)^T, hi and mid, while the state warps work on R
            if (c > 0 && !wait_all(X::CO, ph ^ 1)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 16; ++ks)
                    mma_ts(tm + X::QS, tm + X::S + 8 * ks,
                           desc_k_major(st + X::kq + ((ks >> 2) & 1) * kTile + kHalf + (ks & 3) * 32), idk, ks > 0);
            }
            // U^T = (T' R)^T in six products of terms
            if (!wait_all(X::CR, ph)) break;
            tc_fence_after();
            if (elect_one()) {
                constexpr int r[6] = {2, 1, 0, 1, 0, 0}, t[6] = {0, 1, 2, 0, 1, 0};    // terms of R and of T'
#pragma unroll
                for (int ks = 0; ks < 24; ++ks)
                    mma_ts(tm + X::KS, tm + X::R + r[ks >> 2] * 32 + 8 * (ks & 3),
                           desc_k_major(rec + t[ks >> 2] * kMat + (ks & 3) * 32), idk, ks > 0);
                tc_commit(bar(X::BU));
            }
            // the block's part of S^T, by halves of its channels
            if (!wait_all(X::CU, ph)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int ks = 0; ks < 12; ++ks)
                        mma_ts(tm + X::dS + half * 64, tm + X::U + (2 - (ks >> 2)) * 64 + 8 * (ks & 3),
                               desc_mn_major(st + X::kq + half * kTile + (ks & 3) * 2048, kTile), idmn, ks > 0);
                    tc_commit(bar(X::BS + half));
                }
            }
            // (P U)^T: mid * hi, hi * mid, hi * hi, while the state warps work on S
            if (!wait_all(X::CV, ph)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 12; ++ks)
                    mma_ts(tm + X::PU, tm + X::KS + (ks & 3) * 16 + (ks < 4 ? 8 : 0),
                           desc_k_major(rec + (ks >> 2 == 1 ? DRec::pm : DRec::ph) + (ks & 3) * 32), idk, ks > 0);
                tc_commit(bar(X::BO));
            }
        }
        // nothing in flight when TMEM and shared memory are given back
        if (elect_one()) tc_commit(bar(X::Drain));
        mbar_wait_bounded(bar(X::Drain), 0, a.wait_ns);
    }
    tc_fence_before();
    __syncthreads();
    if (s_abort && tid == 0) atomicOr(a.status, DAMP_EFLAG_TIMEOUT);
    if (warp == wMma) {
        tc_fence_after();
        tmem_free(tm, 512);
    }
}

// ------------------------------------------------------------------ decay

// One CTA of 26 warps a (request, head, segment): 16 keep the state, 4 form
// diag(w) V and P = Q K^T o Gamma, 4 write the readout, one loads (and
// multiplies the decays up), one issues the matrix instructions.  Without the
// delta rule a block's part of S does not depend on S, so operands are formed
// ahead and the tensor core always has a product to work on (cycles a block):
//   dS = (diag(w) V)^T K   A hi and mid in TMEM, lo in shared memory (TMEM is full)   1088
//   S^T Q^T                A pair in TMEM                                    768
//   Q K^T                  of the next block, as two products of 32 columns
//                          whose tokens lie in lanes 0..63 and 64..127: all
//                          four warps (and schedulers) share what follows   1024
//   V^T P^T                A from V's tile as it is, B pair in shared memory 640
// (Q K^T by mma.sync, in the warps that form the operands, took 2800.)
// A request's blocks may be cut into segments that run side by side (few
// chains would leave SMs idle): a first pass (SUM) leaves each segment's sum
// and decay, and the segments of the second start from what those add up to.
struct EChain {
    static constexpr int kWarps = 16, kForm = 4, kOut = 4;
    static constexpr int wOut = kWarps + kForm, wLoad = wOut + kOut, wMma = wLoad + 1;
    static constexpr int threads = 32 * (wMma + 1);
    static constexpr int kStages = 3;
    static constexpr int k = 0, v = kTile, q = 2 * kTile, stage = 3 * kTile;
    static constexpr int p = kStages * stage;                 // P pair [2][hi, mid]
    static constexpr int lo = p + 2 * 2 * kMat;               // (diag(w) V)^T lo of two blocks, K-major [128 v][64 t]
    static constexpr int out = lo + 2 * kTile;                // half a block's readout rows, 16 bytes apart in banks
    static constexpr int out_row = D * 2 + 16;
    static constexpr int ring = out + C / 2 * out_row;        // alpha, gamma, w, mid of four blocks
    static constexpr int bar = ring + 4 * 4 * C * 4;
    static constexpr int bytes = bar + 256 + 1024;
    // TMEM columns.  dS's first 64 hold the next block's Q K^T between two uses.
    static constexpr uint32_t dS = 0, Sh = 128, O1 = 256, O2 = 320, V = 384;   // V: hi, mid of two blocks, 64 each
    // Barriers.  Full: a block's tiles and decays are there.  BD, BQ, BP: dS, S^T Q^T, Q K^T done; BO:
    // V^T P^T too.  CV, CP: diag(w) V, P are there; CD, CP0: dS, Q K^T are out of TMEM; CS: S's pair is
    // there; CO: the readout is out of TMEM.  Where a waiter can be a block behind there are two.
    enum { Full = 0, Empty = kStages, BD = 2 * kStages, BQ = BD + 2, BP, BO, CV = BO + 2, CP = CV + 2, CD = CP + 2,
           CP0, CS, CO, Drain };
};

struct SegArgs {
    int segs;                  // segments of a request (at most: short ones have fewer)
    float* part;               // [n][H][segs][128][128]: state behind segment 0, sums of the others;
                               // the last entry keeps the request's first state
    float* decay;              // [n][H][segs] product of a segment's decays
    uint32_t* there;           // [n][H][segs] kThere: the first pass left the segment's sum; kMissing: it gave up
};

template <bool SUM>
__global__ void __launch_bounds__(EChain::threads, 1)
    decay_chain_kernel(const ChunkArgs ca, const SegArgs sa, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using X = EChain;
    const PrefillArgs& a = ca.p;
    extern __shared__ __align__(1024) uint8_t sm_raw[];
    const uint32_t base = (smem_u32(sm_raw) + 1023u) & ~1023u;
    uint8_t* sm = sm_raw + (base - smem_u32(sm_raw));
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seg = blockIdx.x % sa.segs, place = blockIdx.x / sa.segs, h = place % a.H;
    const int req = a.order ? __ldg(a.order + place / a.H) : place / a.H;
    if (req < 0 || req >= a.n) return;
    const int unit = req * a.H + h;
    const int cu0 = __ldg(a.cu_seqlens + req), cu1 = __ldg(a.cu_seqlens + req + 1);
    const int slot = __ldg(a.store_slot + req), from = __ldg(a.load_slot + req);
    const int end = min(max(cu1, 0), a.max_tokens), first = min(max(cu0, 0), end);
    if (first == end) return;
    const int blocks = (end - first + C - 1) / C, per = (blocks + sa.segs - 1) / sa.segs;
    if (seg * per >= blocks || (SUM && (seg + 1) * per >= blocks)) return;   // nothing, or no one to hand on to
    const bool last = (seg + 1) * per >= blocks;
    const int start = first + seg * per * C, len = min(end - start, per * C), nc = (len + C - 1) / C;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((size_t)start * a.H + h) * D;
    if (slot < 0 || slot >= a.n_slots) {
        if (SUM) return;
        if (slot >= a.n_slots && tid == 0 && h == 0) atomicOr(a.status, DAMP_EFLAG_SLOT_RANGE);
        for (long long e = tid; e < (long long)len * (D / 8); e += X::threads)
            reinterpret_cast<uint4*>(out + (e / (D / 8)) * (size_t)a.H * D)[e % (D / 8)] =
                make_uint4(0, 0, 0, 0);
        return;
    }
    auto bar = [&](int i) { return base + X::bar + 8 * i; };

    auto load = [&](int c) {                           // one lane: block c into its stage
        const int hq = h / (a.H / a.H_qk), t = start + c * C;
        const uint32_t st = base + c % X::kStages * X::stage, f = bar(X::Full + c % X::kStages);
        mbar_arrive_expect_tx(f, (SUM ? 2 : 3) * kTile);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            tma_load_3d(st + X::v + half * kHalf, &mv, half * 64, h, t, f);
            tma_load_3d(st + X::k + half * kHalf, &mk, half * 64, hq, t, f);
            if (!SUM) tma_load_3d(st + X::q + half * kHalf, &mq, half * 64, hq, t, f);
        }
    };
    if (warp == X::wLoad) {
        if (elect_one()) {
            for (int i = 0; i < X::kStages; ++i) {
                mbar_init(bar(X::Full + i), 2);
                mbar_init(bar(X::Empty + i), 1 + X::kForm);
            }
            for (int i = X::BD; i < X::CV; ++i) mbar_init(bar(i), 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(bar(X::CV + i), X::kForm);
                mbar_init(bar(X::CP + i), X::kForm);
            }
            mbar_init(bar(X::CD), X::kWarps);
            mbar_init(bar(X::CP0), X::kForm);
            mbar_init(bar(X::CS), X::kWarps);
            mbar_init(bar(X::CO), X::kOut);
            mbar_init(bar(X::Drain), 1);
            fence_mbar_init();
            s_abort = 0;
            // the first blocks are on their way before the rest of the CTA is ready
            constexpr uint32_t hold = kHookHoldFirstItem | (SUM ? kHookHoldFirstKernel : 0u);
            for (int c = a.hooks & hold ? 1 : 0; c < min(nc, X::kStages); ++c) load(c);
        }
        __syncwarp();
    } else if (warp == X::wMma) {
        tmem_alloc(smem_u32(&s_tmem), 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s_tmem;

    auto wait_all = [&](int i, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, bounded_wait(bar(i), parity, a.wait_ns, &s_abort, warp == X::wLoad));
    };
    auto wait_group = [&](bool polls, int i, uint32_t parity, int id, int threads) -> bool {
        const bool ok = !polls || wait_all(i, parity);
        return !bar_red_or(id, threads, !ok);
    };
    auto arrive = [&](int i) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(i));
    };
    const int quad = warp & 3;
    const uint32_t lanes = tm + ((uint32_t)(quad * 32) << 16);
    const int vcol = quad * 32 + lane;                 // a state or readout thread's value column
    // alpha_t, gamma_t, gamma_C / gamma_t and (t >= 32) gamma_t / gamma_31 of block c
    auto ring = [&](int c) { return reinterpret_cast<float*>(sm + X::ring) + (c & 3) * 4 * C; };

    if (warp < X::kWarps) {
        // ---------------------------------------------------------- state
        const int part = warp >> 2;                    // key channels [32 part, +32)
        const size_t at = (size_t)(part * 32) * D + vcol;
        uint8_t* states = a.state + (size_t)h * D * D * 4;
        float* parts = sa.part + (size_t)unit * sa.segs * D * D + at;
        const bool has = from >= 0 && from < a.n_slots;
        float S[32];
        bool ok = true;
        if (seg == 0) {
            // the second pass may find the slot's new state in its place already
            const float* in = !SUM && !last
                ? parts + (size_t)(sa.segs - 1) * D * D
                : reinterpret_cast<const float*>(states + (size_t)(a.state_by_slot ? (has ? from : slot) : req) *
                                                              a.state_stride) + at;
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = has ? in[(size_t)i * D] : 0.f;
            if (SUM)
#pragma unroll
                for (int i = 0; i < 32; ++i) parts[(size_t)(sa.segs - 1) * D * D + (size_t)i * D] = S[i];
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = SUM ? 0.f : parts[(size_t)i * D];
            if (!SUM)
                for (int j = 0; j < seg; ++j) ok = ok && sa.there[(size_t)unit * sa.segs + j] == kThere;
            if (!ok) s_abort = 1;              // (for every thread, or none; the state stays as it was)
            if (!SUM)
                for (int j = 1; j < seg; ++j) {
                    const float g = sa.decay[(size_t)unit * sa.segs + j];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        S[i] = __fmaf_rn(g, S[i], parts[(size_t)j * D * D + (size_t)i * D]);
                }
        }
        double total = 1.0;
        for (int c = 0; c < nc && ok; ++c) {
            const uint32_t ph = c & 1;
            if (!SUM) {
                // ---- the state before block c as a pair
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) split_bf16(S[2 * i], S[2 * i + 1], hi[i], lo[i]);
                if (c > 0 && !(ok = wait_group(warp == 0, X::BQ, ph ^ 1, 4, X::kWarps * 32))) break;
                tc_fence_after();
                tmem_st16(lanes + X::Sh + part * 16, hi);
                tmem_st16(lanes + X::Sh + 64 + part * 16, lo);
                tmem_wait_st();
                arrive(X::CS);
            }
            // ---- S <- gamma_C S + the block's part
            if (!(ok = wait_group(warp == 0, X::BD + ph, (c >> 1) & 1, 4, X::kWarps * 32))) break;
            tc_fence_after();
            const float gc = ring(c)[2 * C - 1];
            uint32_t y[32];
            tmem_ld32(lanes + X::dS + part * 32, y);
            tmem_wait_ld();
            arrive(X::CD);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 s = __ffma2_rn(make_float2(gc, gc), make_float2(S[2 * i], S[2 * i + 1]),
                                            make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])));
                S[2 * i] = s.x;
                S[2 * i + 1] = s.y;
            }
            total *= gc;
        }
        if (SUM && tid == 0) sa.there[(size_t)unit * sa.segs + seg] = ok ? kThere : kMissing;
        if (ok) {
            if (SUM) {
#pragma unroll
                for (int i = 0; i < 32; ++i) parts[(size_t)seg * D * D + (size_t)i * D] = S[i];
                if (tid == 0) sa.decay[(size_t)unit * sa.segs + seg] = (float)total;
            } else if (last) {
                float* to = reinterpret_cast<float*>(
                    states + (size_t)(a.state_by_slot ? slot : req) * a.state_stride) + at;
#pragma unroll
                for (int i = 0; i < 32; ++i) to[(size_t)i * D] = S[i];
            }
        }
    } else if (warp < (SUM ? X::wLoad : X::wOut)) {
        // ---------------------------------------------------------- operands
        // (in a first pass the readout's warps have every other block's)
        constexpr int kN = X::kForm * 32;
        const int group = (warp - X::kWarps) / X::kForm, kId = 2 + group, lead = X::kWarps + group * X::kForm;
        const int ft = tid - lead * 32, c2 = (lane & 3) * 2;
        // diag(w) V of block c as three terms, hi and mid in TMEM
        auto form_v = [&](int c) -> bool {
            const uint32_t st = base + c % X::kStages * X::stage, buf = c & 1;
            const int live = min(C, len - c * C);
            if (!wait_group(warp == lead, X::Full + c % X::kStages, (c / X::kStages) & 1, kId, kN)) return false;
            if (live < C) {
                // rows behind the end hold another request's keys and values: they must not
                // enter the sums over tokens
                uint8_t* stp = sm + c % X::kStages * X::stage;
                for (int e = ft; e < (C - live) * 16; e += kN) {
                    const int to = (e & 8 ? kHalf : 0) + (live + e / 16) * 128 + (e & 7) * 16;
                    *reinterpret_cast<uint4*>(stp + X::k + to) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(stp + X::v + to) = make_uint4(0, 0, 0, 0);
                }
            }
            // the block before last has used these terms up
            if (!wait_group(c >= 2 && warp == lead, X::BD + buf, ((c >> 1) - 1) & 1, kId, kN)) return false;
            tc_fence_after();
            const float* w = ring(c) + 2 * C;
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {   // 16 value columns (TMEM lanes) each, transposed by ldmatrix
                uint32_t hi[16], mid[16];
                const int col = quad * 32 + hf * 16;
                uint8_t* lop = sm + X::lo + buf * kTile;
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // 16 tokens each
                    uint32_t v[4];
                    const int row = j * 16 + (lane & 7) + (lane >> 4) * 8;
                    ldsm4t(v, st + X::v + (col >> 6) * kHalf +
                                  swz(row, (col & 63) * 2 + ((lane >> 3) & 1) * 16));
                    const float2 w0 = *reinterpret_cast<const float2*>(w + j * 16 + c2);
                    const float2 w1 = *reinterpret_cast<const float2*>(w + j * 16 + 8 + c2);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = make_float2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u));
                        uint32_t lo;               // of column l / 4 + 8 (i & 1), tokens 16 j + 8 (i / 2) + 2 (l % 4), + 1
                        split3_bf16(__fmul2_rn(x, i < 2 ? w0 : w1), hi[4 * j + i], mid[4 * j + i], lo);
                        *reinterpret_cast<uint32_t*>(lop + swz(col + (lane >> 2) + 8 * (i & 1),
                                                               j * 32 + (i >> 1) * 16 + c2 * 2)) = lo;
                    }
                }
                const uint32_t to = lanes + ((uint32_t)(hf * 16) << 16) + X::V + buf * 64;
                tmem_st_16x128(to, hi);
                tmem_st_16x128(to + 32, mid);
            }
            fence_proxy_async_smem();
            tmem_wait_st();
            arrive(X::CV + buf);
            if (lane == 0) mbar_arrive(bar(X::Empty + c % X::kStages));
            return true;
        };
        bool ok = true;
        // this thread's token and its 32 columns of P (TMEM lanes 0..63: 0..31, 64..127: 32..63)
        const int t = (quad & 1) * 32 + lane, s0 = (quad >> 1) * 32;
        // P of block c, and diag(w) V two blocks ahead (a first pass: that alone, every other block)
        for (int c = SUM ? group - 2 : -2; c < nc && ok; c += SUM ? 2 : 1) {
            if (!SUM && c >= 0) {
                uint8_t* pm = sm + X::p + (c & 1) * 2 * kMat;
                if (!(ok = wait_group(warp == lead, X::BP, c & 1, kId, kN))) break;
                tc_fence_after();
                uint32_t y[32];
                tmem_ld32(lanes + X::dS + s0, y);
                tmem_wait_ld();
                arrive(X::CP0);
                const float* al = ring(c);
                const bool row_live = t < min(C, len - c * C);
                // gamma_t / gamma_s for s downwards; it starts at s = t, or from the columns above
                float x = row_live && t >= s0 + 32 ? al[3 * C + t] : 0.f, above = 1.f;   // above: alpha_{s + 1}
#pragma unroll
                for (int j = 3; j >= 0; --j) {
                    float f[8];
                    const float4 a1 = *reinterpret_cast<const float4*>(al + s0 + j * 8 + 4);
                    const float4 a0 = *reinterpret_cast<const float4*>(al + s0 + j * 8);
                    const float as[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
                    for (int i = 7; i >= 0; --i) {
                        x = s0 + j * 8 + i == t && row_live ? 1.f : x * above;
                        above = as[i];
                        f[i] = x == 0.f ? 0.f : x * __uint_as_float(y[j * 8 + i]);
                    }
                    uint4 hi, lo;
                    split_bf16(f[0], f[1], hi.x, lo.x);
                    split_bf16(f[2], f[3], hi.y, lo.y);
                    split_bf16(f[4], f[5], hi.z, lo.z);
                    split_bf16(f[6], f[7], hi.w, lo.w);
                    const uint32_t to = swz(t, (s0 + j * 8) * 2);
                    *reinterpret_cast<uint4*>(pm + to) = hi;
                    *reinterpret_cast<uint4*>(pm + kMat + to) = lo;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(X::CP + (c & 1)));
            }
            if (c + 2 < nc) ok = form_v(c + 2);
        }
    } else if (warp < X::wLoad) {
        // ---------------------------------------------------------- readout
        const int wt = tid - X::wOut * 32;
        uint8_t* so = sm + X::out;
        for (int c = 0; c < nc; ++c) {
            const float* gam = ring(c) + C;
            if (!wait_group(warp == X::wOut, X::BO + (c & 1), (c >> 1) & 1, 1, X::kOut * 32)) break;
            tc_fence_after();
            const int live = min(C, len - c * C);
            // (Not unrolled, as other long loops of this kernel are not: while all of them were, its warps were
            // stalled for want of an instruction 2.1 times an issue, now 0.5 times, and the 16 requests took 5 %
            // longer.  Unrolling this one alone makes no difference, 127 and 128 us.)
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
#pragma unroll 1
                for (int part = 2 * half; part < 2 * half + 2; ++part) {
                    uint32_t o1[16], o2[16];
                    tmem_ld16(lanes + X::O1 + part * 16, o1);
                    tmem_ld16(lanes + X::O2 + part * 16, o2);
                    float2 gt[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) gt[i] = *reinterpret_cast<const float2*>(gam + part * 16 + 2 * i);
                    tmem_wait_ld();
                    // (the loader may write over these decays once the block after next is loaded, which
                    // this arrival lets happen: they are read before it)
                    if (part == 3) arrive(X::CO);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t o = pack_bf16(
                            __fmaf_rn(gt[i].x, __uint_as_float(o1[2 * i]), __uint_as_float(o2[2 * i])),
                            __fmaf_rn(gt[i].y, __uint_as_float(o1[2 * i + 1]), __uint_as_float(o2[2 * i + 1])));
                        uint8_t* to = so + ((part & 1) * 16 + 2 * i) * X::out_row + vcol * 2;
                        *reinterpret_cast<uint16_t*>(to) = (uint16_t)o;
                        *reinterpret_cast<uint16_t*>(to + X::out_row) = (uint16_t)(o >> 16);
                    }
                }
                // (rows of 256 bytes from shared memory: a warp's own 64 bytes of each, as they come, took 157 us
                // for the 16 requests against 126)
                bar_sync(1, X::kOut * 32);
#pragma unroll
                for (int i = 0; i < C / 2 * 16 / (X::kOut * 32); ++i) {
                    const int r = (wt >> 4) + i * (X::kOut * 2), u = wt & 15, t = half * (C / 2) + r;
                    if (t < live)
                        *reinterpret_cast<uint4*>(out + (size_t)(c * C + t) * a.H * D + u * 8) =
                            *reinterpret_cast<const uint4*>(so + r * X::out_row + u * 16);
                }
                bar_sync(1, X::kOut * 32);
            }
        }
    } else if (warp == X::wLoad) {
        // ---------------------------------------------------------- loads
        int issued = min(nc, X::kStages);
        auto alpha_of = [&](int t) {
            return t < len ? __ldg(a.alpha + (size_t)(start + t) * a.H + h) : 1.f;
        };
        float a0 = alpha_of(2 * lane), a1 = alpha_of(2 * lane + 1);    // of this lane's two tokens
        for (int c = 0; c < nc; ++c) {
            const uint32_t f = bar(X::Full + c % X::kStages);
            // the products first: they take their time while the stage is still in use
            float2 upto, behind;
            decay_products(a0, a1, lane, upto, behind);
            float mid = a0 * a1;               // from token 32 on
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, mid, off);
                if (lane >= 16 + off) mid = u * mid;
            }
            float mid0 = __shfl_up_sync(0xffffffffu, mid, 1);
            mid0 = lane == 16 ? a0 : mid0 * a0;
            const float2 al = make_float2(a0, a1);
            a0 = alpha_of((c + 1) * C + 2 * lane);
            a1 = alpha_of((c + 1) * C + 2 * lane + 1);
            if (c >= X::kStages) {
                if (!wait_all(X::Empty + c % X::kStages, (c / X::kStages - 1) & 1)) break;
                if (elect_one()) load(c);
                issued = c + 1;
            }
            float2* r = reinterpret_cast<float2*>(ring(c)) + lane;
            r[0] = al;
            r[C / 2] = upto;
            r[C] = behind;
            r[3 * C / 2] = make_float2(mid0, mid);
            __syncwarp();
            if (lane == 0) mbar_arrive(f);
        }
        // copies in flight end before the CTA does
        for (int c = max(0, issued - X::kStages); c < issued; ++c)
            mbar_wait_bounded(bar(X::Full + c % X::kStages), (c / X::kStages) & 1, a.wait_ns);
    } else {
        // ---------------------------------------------------------- matrix instructions
        constexpr uint32_t ids = mma_idesc(128, 128, false, true), idk = mma_idesc(128, 64, false, false),
                           idv = mma_idesc(128, 64, true, false), idp = mma_idesc(128, 32, false, false);
        auto scores = [&](int c) -> bool {           // Q K^T of block c
            const uint32_t st = base + c % X::kStages * X::stage;
            if (!wait_all(X::Full + c % X::kStages, (c / X::kStages) & 1)) return false;
            if (elect_one()) {
#pragma unroll 1
                for (int half = 0; half < 2; ++half)     // columns; rows of M that are not Q's are not used
#pragma unroll 4
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ss(tm + X::dS + half * 32,
                               desc_k_major(st + X::q - half * kHalf + (ks >> 2) * kHalf + (ks & 3) * 32),
                               desc_k_major(st + X::k + (ks >> 2) * kHalf + half * (kHalf / 2) + (ks & 3) * 32), idp,
                               ks > 0);
                tc_commit(bar(X::BP));
            }
            return true;
        };
        bool ok = SUM || scores(0);
        for (int c = 0; c < nc && ok; ++c) {
            const uint32_t st = base + c % X::kStages * X::stage, ph = c & 1;
            if (!(ok = wait_all(X::CV + ph, (c >> 1) & 1))) break;     // (its writers saw the stage full)
            if (SUM && c > 0 && !(ok = wait_all(X::CD, ph ^ 1))) break;
            if (!SUM && !(ok = wait_all(X::CP0, ph))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll 4
                for (int ks = 0; ks < 4; ++ks)       // lo, then mid and hi
                    mma_ss(tm + X::dS, desc_k_major(base + X::lo + ph * kTile + ks * 32),
                           desc_mn_major(st + X::k + ks * 2048, kHalf), ids, ks > 0);
#pragma unroll 4
                for (int ks = 7; ks >= 0; --ks)
                    mma_ts(tm + X::dS, tm + X::V + ph * 64 + 8 * ks,
                           desc_mn_major(st + X::k + (ks & 3) * 2048, kHalf), ids, 1);
                tc_commit(bar(X::BD + ph));
                if (SUM) tc_commit(bar(X::Empty + c % X::kStages));
            }
            if (SUM) continue;
            if (c > 0 && !(ok = wait_all(X::CO, ph ^ 1))) break;
            if (!(ok = wait_all(X::CS, ph))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll 4
                for (int ks = 0; ks < 16; ++ks)
                    mma_ts(tm + X::O1, tm + X::Sh + 8 * ks,
                           desc_k_major(st + X::q + ((ks >> 2) & 1) * kHalf + (ks & 3) * 32), idk, ks > 0);
                tc_commit(bar(X::BQ));
            }
            if (c + 1 < nc) {
                if (!(ok = wait_all(X::CD, ph))) break;
                tc_fence_after();
                if (!(ok = scores(c + 1))) break;
            }
            if (!(ok = wait_all(X::CP + ph, (c >> 1) & 1))) break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t pm = base + X::p + ph * 2 * kMat;
#pragma unroll 4
                for (int ks = 0; ks < 8; ++ks)
                    mma_ss(tm + X::O2, desc_mn_major(st + X::v + (ks & 3) * 2048, kHalf),
                           desc_k_major(pm + (ks >> 2) * kMat + (ks & 3) * 32), idv, ks > 0);
                tc_commit(bar(X::BO + ph));
                tc_commit(bar(X::Empty + c % X::kStages));
            }
        }
        // nothing in flight when TMEM and shared memory are given back
        if (elect_one()) tc_commit(bar(X::Drain));
        mbar_wait_bounded(bar(X::Drain), 0, a.wait_ns);
    }
    tc_fence_before();
    __syncthreads();
    if (s_abort && tid == 0) atomicOr(a.status, DAMP_EFLAG_TIMEOUT);
    if (warp == X::wMma) {
        tc_fence_after();
        tmem_free(tm, 512);
    }
}

// ------------------------------------------------------------------ host

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                 CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);
std::atomic<EncodeTiled> g_encode{nullptr};

// Token rows of `heads` heads of 128 bf16 channels, in boxes of 64 rows of one
// head's 64 channels, 128-byte swizzle; rows behind the last read as zeros.
cudaError_t token_map(CUtensorMap* m, const void* p, int heads, long long rows, long long stride) {
    EncodeTiled f = g_encode.load(std::memory_order_relaxed);
    if (!f) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)C}, step[3] = {1, 1, 1};
    const CUresult r = f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box,
                         step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Segments of a request for the decay rule: as many as the SMs have room for,
// none shorter (on average) than 4 blocks; a batch whose (request, head) pairs
// take more than half of the SMs stays whole (the first pass reads K and V once
// more).  One prompt of 4096 tokens x 32 heads: 89 us in 4 segments, 145 in 2,
// 185 whole.
int decay_segments(int n, int H, int max_tokens, int sms) {
    const long long chains = (long long)n * H;
    if (chains * 2 > sms) return 1;
    const long long blocks = max_tokens / ((long long)C * n);
    return (int)std::max(1ll, std::min((long long)sms / chains, blocks / 4));
}

size_t first_block_bytes(int n) { return ((size_t)n * 4 + 255) / 256 * 256; }

}  // namespace

// The driver's encoder and the kernels' attributes, once per device (the
// current one).
cudaError_t prepare_prefill(uint32_t hooks) {
    if (hooks & kHookNoTensorMaps) return cudaErrorNotSupported;
    static std::atomic<uint64_t> ready{0};             // a bit per device below 64
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (ready.load() >> dev & 1)) return cudaSuccess;
    if (!g_encode.load()) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess) return e != cudaSuccess ? e : cudaErrorNotSupported;
        g_encode.store(reinterpret_cast<EncodeTiled>(f));
    }
    constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    if ((e = cudaFuncSetAttribute(delta_prepare_kernel, attr, DPrep::bytes)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(delta_chain_kernel, attr, DChain::bytes)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(decay_chain_kernel<false>, attr, EChain::bytes)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(decay_chain_kernel<true>, attr, EChain::bytes)) != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev);
    return cudaSuccess;
}

bool prefill_chunk_fits(int d_k, int d_v, int bf16) { return bf16 && d_k == D && d_v == D; }

size_t prefill_chunk_bytes(int n, int H, int max_tokens, int max_blocks, int delta) {
    if (delta) return first_block_bytes(n) + (size_t)max_blocks * H * DRec::bytes;
    const int segs = decay_segments(n, H, max_tokens, kSms);
    return segs == 1 ? 0 : (size_t)n * H * segs * (D * D + 2) * 4;
}

cudaError_t launch_prefill_chunk(const PrefillArgs& a, cudaStream_t s) {
    CUtensorMap mq, mk, mv;
    cudaError_t e = prepare_prefill(a.hooks);
    if (e == cudaSuccess) e = token_map(&mq, a.q, a.H_qk, a.max_tokens, a.q_stride);
    if (e == cudaSuccess) e = token_map(&mk, a.k, a.H_qk, a.max_tokens, a.k_stride);
    if (e == cudaSuccess) e = token_map(&mv, a.v, a.H, a.max_tokens, a.v_stride);
    if (e != cudaSuccess) return e;
    ChunkArgs ca{a, nullptr, nullptr};
    if (!a.delta) {
        SegArgs sa{decay_segments(a.n, a.H, a.max_tokens, kSms), reinterpret_cast<float*>(a.work), nullptr,
                   nullptr};
        sa.decay = sa.part + (size_t)a.n * a.H * sa.segs * D * D;
        sa.there = reinterpret_cast<uint32_t*>(sa.decay + (size_t)a.n * a.H * sa.segs);
        const int grid = a.n * a.H * sa.segs;
        if (sa.segs > 1) {
            decay_chain_kernel<true><<<grid, EChain::threads, EChain::bytes, s>>>(ca, sa, mq, mk, mv);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
        }
        decay_chain_kernel<false><<<grid, EChain::threads, EChain::bytes, s>>>(ca, sa, mq, mk, mv);
        return cudaGetLastError();
    }
    ca.first_block = reinterpret_cast<int32_t*>(a.work);
    ca.records = a.work + first_block_bytes(a.n);
    delta_prepare_kernel<<<a.max_blocks * a.H, kPrepThreads, DPrep::bytes, s>>>(ca, mq, mk);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    delta_chain_kernel<<<a.n * a.H, DChain::threads, DChain::bytes, s>>>(ca, mq, mk, mv);
    return cudaGetLastError();
}

}  // namespace damp
