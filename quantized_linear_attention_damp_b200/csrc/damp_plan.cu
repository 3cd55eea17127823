// damp_plan.cu -- index arrays of a ragged batch, built on the GPU from the
// requests' lengths (damp_batch_plan): row offsets, the slots each request's
// state is loaded from and stored to, the table of 64-token blocks, and the
// slot and position of every token row.
//
// One launch, no workspace, no atomics.  Every CTA scans all n lengths into
// its shared memory (n <= 16,384: 4 KB .. 128 KB) and then writes its own
// slice of every output, locating rows by a binary search in the scanned
// offsets.  The redundant scan costs each CTA one read of the lengths out of
// L2; a scan that the CTAs share would need a second launch or a chain of
// waits between CTAs, either of which takes longer than the scan.
//
// What bounds it: the launch and the scan's latency for small batches, the
// 8 bytes stored per token row for large ones.
#include <cuda_runtime.h>
#include <limits.h>

#include <algorithm>

#include "damp.h"
#include "damp_internal.h"
#include "damp_prompt.h"

namespace damp {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kRowsPerCta = 4 * kPlanThreads;   // token rows one CTA is given at least
constexpr int kB = DAMP_PLAN_BLOCK;
constexpr int kSorted = 1024;                   // requests up to which the order is by length

// Smallest r with end[r] > x; `end` ascends and end[n - 1] > x.
__device__ __forceinline__ int owner(const int* end, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (end[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
    extern __shared__ int s_dyn[];
    int* s_end = s_dyn;          // [n] row behind each request's last, dropped requests clipped
    int* s_bend = s_dyn + a.n;   // [n] likewise in blocks
    __shared__ long long s_wt[kPlanWarps];
    __shared__ long long s_wb[kPlanWarps];
    __shared__ int s_top[kPlanWarps], s_btop[kPlanWarps], s_long[kPlanWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = a.n;
    const long long limit = a.max_tokens;

    // ---- inclusive scan of lengths and block counts; each thread takes a run
    // of consecutive requests.  64-bit sums: n lengths can pass 2^31.
    const int per = (n + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(n, tid * per), r1 = min(n, r0 + per);
    long long t = 0, b = 0;
    int bad = 0;
    for (int r = r0; r < r1; ++r) {
        const int len = __ldg(a.lengths + r);
        if (len < 0 || (a.past && __ldg(a.past + r) < 0)) bad |= DAMP_PLAN_EFLAG_VALUE;
        if (__ldg(a.slot_idx + r) >= a.n_slots) bad |= DAMP_PLAN_EFLAG_SLOT;
        t += max(len, 0);
        b += (max(len, 0) + (long long)kB - 1) / kB;
    }
    long long ti = t, bi = b;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long tu = __shfl_up_sync(0xffffffffu, ti, off);
        const long long bu = __shfl_up_sync(0xffffffffu, bi, off);
        if (lane >= off) {
            ti += tu;
            bi += bu;
        }
    }
    if (lane == 31) {
        s_wt[warp] = ti;
        s_wb[warp] = bi;
    }
    __syncthreads();
    long long te = ti - t, be = bi - b;   // exclusive prefix
    for (int w = 0; w < warp; ++w) {
        te += s_wt[w];
        be += s_wb[w];
    }
    // ---- ends; a request whose end lies behind max_tokens is dropped, and
    // with it every later request that has rows (ends ascend).  top = rows of
    // the kept requests.
    int top = 0, btop = 0, longest = 0;
    for (int r = r0; r < r1; ++r) {
        const int len = max(__ldg(a.lengths + r), 0);
        te += len;
        be += ((long long)len + kB - 1) / kB;
        if (te <= limit) {
            top = (int)te;
            btop = (int)be;
            longest = max(longest, len);
        } else if (len > 0) {
            bad |= DAMP_PLAN_EFLAG_TOKENS;
        }
        s_end[r] = te <= limit ? (int)te : -1;
        s_bend[r] = (int)min(be, (long long)INT_MAX);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    btop = __reduce_max_sync(0xffffffffu, btop);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) {
        s_top[warp] = top;
        s_btop[warp] = btop;
        s_long[warp] = longest;
    }
    // (the OR is needed by CTA 0 alone, but the barrier by all)
    bad = __syncthreads_or(bad & DAMP_PLAN_EFLAG_VALUE ? 1 : 0) * DAMP_PLAN_EFLAG_VALUE |
          __syncthreads_or(bad & DAMP_PLAN_EFLAG_TOKENS ? 1 : 0) * DAMP_PLAN_EFLAG_TOKENS |
          __syncthreads_or(bad & DAMP_PLAN_EFLAG_SLOT ? 1 : 0) * DAMP_PLAN_EFLAG_SLOT;
    for (int w = 0; w < kPlanWarps; ++w) {
        top = max(top, s_top[w]);
        btop = max(btop, s_btop[w]);
        longest = max(longest, s_long[w]);
    }
    for (int r = r0; r < r1; ++r)
        if (s_end[r] < 0) {
            s_end[r] = top;
            s_bend[r] = btop;
        }
    __syncthreads();

    const int gtid = blockIdx.x * kPlanThreads + tid, gsize = gridDim.x * kPlanThreads;
    // ---- per request
    for (int r = gtid; r < n; r += gsize) {
        const int start = r ? s_end[r - 1] : 0, len = s_end[r] - start;
        const int slot = __ldg(a.slot_idx + r);
        const int st = len > 0 && slot >= 0 && slot < a.n_slots ? slot : -1;
        a.cu_seqlens[r + 1] = s_end[r];
        a.store_slot[r] = st;
        a.load_slot[r] = a.past && __ldg(a.past + r) > 0 ? st : -1;
    }
    if (gtid == 0) {
        a.cu_seqlens[0] = 0;
        a.totals[0] = top;
        a.totals[1] = btop;
        a.totals[2] = longest;
        a.totals[3] = bad;
    }
    // ---- order: longest first, so that a long prompt is not what a launch ends with.  n compares for
    // each request; more requests than kSorted balance themselves and are taken as they come.
    if (a.order) {
        __shared__ __align__(16) int s_len[kSorted];
        if (n <= kSorted) {
            for (int r = tid; r < kSorted; r += kPlanThreads)
                s_len[r] = r < n ? s_end[r] - (r ? s_end[r - 1] : 0) : -1;
            __syncthreads();
        }
        for (int r = gtid; r < n; r += gsize) {
            int rank = r;
            if (n <= kSorted) {
                const int mine = s_len[r];
                rank = 0;
                for (int j = 0; j < n; j += 4) {
                    const int4 l = *reinterpret_cast<const int4*>(s_len + j);
                    rank += (l.x > mine || (l.x == mine && j < r)) + (l.y > mine || (l.y == mine && j + 1 < r)) +
                            (l.z > mine || (l.z == mine && j + 2 < r)) + (l.w > mine || (l.w == mine && j + 3 < r));
                }
            }
            a.order[rank] = r;
        }
    }
    // ---- per block
    for (int i = gtid; i < a.max_blocks; i += gsize) {
        int4 row = make_int4(-1, -1, -1, -1);
        if (i < btop) {
            const int r = owner(s_bend, n, i);
            const int first = i - (r ? s_bend[r - 1] : 0);
            const int at = (r ? s_end[r - 1] : 0) + first * kB;
            row = make_int4(r, at, min(kB, s_end[r] - at), first);
        }
        reinterpret_cast<int4*>(a.block_table)[i] = row;
    }
    // ---- per token row: 4 rows a thread, one search for the first
    if (!a.token_slot) return;
    for (long long i0 = (long long)gtid * 4; i0 < a.max_tokens; i0 += (long long)gsize * 4) {
        int slots[4], poss[4];
        int r = i0 < top ? owner(s_end, n, (int)i0) : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = (int)i0 + j;
            slots[j] = poss[j] = -1;
            if (i < top) {
                while (s_end[r] <= i) ++r;   // ends within n: i < top = the last end
                const int slot = __ldg(a.slot_idx + r);
                slots[j] = slot >= 0 && slot < a.n_slots ? slot : -1;
                poss[j] = (a.past ? max(__ldg(a.past + r), 0) : 0) + i - (r ? s_end[r - 1] : 0);
            }
        }
        if (i0 + 4 <= a.max_tokens) {
            *reinterpret_cast<int4*>(a.token_slot + i0) =
                make_int4(slots[0], slots[1], slots[2], slots[3]);
            *reinterpret_cast<int4*>(a.token_pos + i0) = make_int4(poss[0], poss[1], poss[2], poss[3]);
        } else {
            for (int j = 0; j < 4; ++j)
                if (i0 + j < a.max_tokens) {
                    a.token_slot[i0 + j] = slots[j];
                    a.token_pos[i0 + j] = poss[j];
                }
        }
    }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    const size_t smem = (size_t)a.n * 8;
    // (beside 5 KB of static shared memory)
    if (smem > 40 * 1024 && (e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                      DAMP_PLAN_MAX_REQUESTS * 8)) != cudaSuccess)
        return e;
    const long long rows = std::max((long long)a.max_tokens, (long long)a.max_blocks);
    const int grid = (int)std::max(1ll, std::min((long long)sms, (rows + kRowsPerCta - 1) / kRowsPerCta));
    plan_kernel<<<grid, kPlanThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace damp
