// plan_kernel.cu -- the bookkeeping of a step over the paged cache, from the lengths of its
// requests: pages for the new tokens, their places in block_table, and each token's slot.
//
// Sequence b holds c tokens and gets t more: o = ceil(c / page_size) pages are its own already, pages
// o .. ceil((c + t) / page_size) - 1 come off the end of the free list, the sequences' one after the
// other.  Every new page starts with a new token, so one thread a token does all of it: the token at
// position p with p % page_size == 0 also writes the page into the table.  The offsets (of tokens and
// of pages) are scans over the sequences, done by one CTA before.
#include "ptx.cuh"
#include "step_kernels.h"

namespace attn {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanTokenThreads = 256;

struct PlanSeq {
    int c, t, o, n;  // tokens held and new, pages held and new
    bool bad;
};

__device__ __forceinline__ PlanSeq plan_seq(const PlanParams& p, int b) {
    PlanSeq s;
    s.c = p.cache_seqlens[b];
    s.t = p.new_lens[b];
    const long long keys = static_cast<long long>(s.c) + s.t;
    s.bad = s.c < 0 || s.t < 0 || s.t > p.total_q ||
            keys > static_cast<long long>(p.max_pages) * p.page_size;
    if (s.bad) s.t = 0, s.c = 0;
    s.o = (s.c + p.page_size - 1) / p.page_size;  // (the host keeps table widths below 2^30)
    s.n = (s.c + s.t + p.page_size - 1) / p.page_size - s.o;
    return s;
}

struct Pair {
    long long t, n;
};

// Exclusive scan of one pair a thread over the block, and its total.
__device__ Pair plan_scan(Pair v, Pair* warp_sum, Pair& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Pair x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long yt = __shfl_up_sync(0xffffffffu, x.t, o);
        const long long yn = __shfl_up_sync(0xffffffffu, x.n, o);
        if (lane >= o) x.t += yt, x.n += yn;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
        Pair w = warp_sum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long yt = __shfl_up_sync(0xffffffffu, w.t, o);
            const long long yn = __shfl_up_sync(0xffffffffu, w.n, o);
            if (lane >= o) w.t += yt, w.n += yn;
        }
        warp_sum[lane] = w;
    }
    __syncthreads();
    total = warp_sum[31];
    Pair before = {x.t - v.t, x.n - v.n};
    if (warp > 0) before.t += warp_sum[warp - 1].t, before.n += warp_sum[warp - 1].n;
    __syncthreads();
    return before;
}

// All that goes by sequence, and the offsets.
__device__ __forceinline__ void plan_sequences(const PlanParams& p, int* page_off, Pair* warp_sum) {
    const int tid = threadIdx.x;
    const int count = *p.free_count;
    // What cannot be met as a whole changes nothing: the sums come first.
    Pair sum = {0, 0};
    bool bad = false;
    for (int b = tid; b < p.batch; b += kPlanThreads) {
        const PlanSeq s = plan_seq(p, b);
        sum.t += s.t;
        sum.n += s.n;
        bad |= s.bad;
    }
    Pair all;
    plan_scan(sum, warp_sum, all);
    bad = __syncthreads_or(bad) || all.t > p.total_q || count < 0 || count > p.num_free || all.n > count;
    Pair carry = {0, 0};
    for (int base = 0; base < p.batch; base += kPlanThreads) {
        const int b = base + tid;
        PlanSeq s = {0, 0, 0, 0, false};
        int held = 0;
        if (b < p.batch) {
            s = plan_seq(p, b);
            held = p.cache_seqlens[b];
        }
        if (bad) s.t = s.n = 0;
        Pair total;
        const Pair at = plan_scan({s.t, s.n}, warp_sum, total);
        if (b < p.batch) {
            p.cu_seqlens_q[b] = static_cast<int>(carry.t + at.t);
            page_off[b] = static_cast<int>(carry.n + at.n);
            p.seqlens_after[b] = held + s.t;  // (may be cache_seqlens: this thread has read its entry)
        }
        carry.t += total.t;
        carry.n += total.n;
    }
    if (tid == 0) {
        if (bad) atomicOr(p.status, kStatusBounds);
        p.cu_seqlens_q[p.batch] = static_cast<int>(carry.t);
        page_off[p.batch] = count;
        *p.free_left = count - static_cast<int>(carry.n);  // (may be free_count)
    }
}

// Token t's position and slot, and the page that begins with it.
__device__ __forceinline__ void plan_token(const PlanParams& p, const int* page_off, int t) {
    int pos = 0, slot = -1;
    if (t < p.cu_seqlens_q[p.batch]) {
        int lo = 0, hi = p.batch - 1;  // the last sequence that starts at t or before
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.cu_seqlens_q[mid] <= t) lo = mid; else hi = mid - 1;
        }
        const int b = lo, q0 = p.cu_seqlens_q[b];
        const int c = p.seqlens_after[b] - (p.cu_seqlens_q[b + 1] - q0);
        pos = c + (t - q0);
        const int j = pos / p.page_size, in = pos - j * p.page_size;
        const int held = (c + p.page_size - 1) / p.page_size;
        int* entry = p.block_table + static_cast<size_t>(b) * p.max_pages + j;
        const int page = j >= held
                             ? p.free_pages[page_off[p.batch] - 1 - (page_off[b] + j - held)]
                             : *entry;
        const bool ok = page >= 0 && page < p.num_pages;
        if (!ok) atomicOr(p.status, kStatusBounds);
        if (j >= held && in == 0) *entry = ok ? page : -1;
        if (ok) slot = page * p.page_size + in;
    }
    p.positions[t] = pos;
    p.slot_map[t] = slot;
}

__global__ void __launch_bounds__(kPlanThreads) plan_scan_kernel(const PlanParams p) {
    __shared__ Pair warp_sum[32];
    griddep_launch_dependents();
    plan_sequences(p, p.page_off, warp_sum);
}

__global__ void __launch_bounds__(kPlanTokenThreads) plan_tokens_kernel(const PlanParams p) {
    const int t = blockIdx.x * kPlanTokenThreads + threadIdx.x;
    griddep_wait();
    if (t < p.total_q) plan_token(p, p.page_off, t);
}

// Few tokens: both in one launch, by one block (which sees its own writes behind the barrier).
__global__ void __launch_bounds__(kPlanThreads) plan_small_kernel(const PlanParams p) {
    __shared__ Pair warp_sum[32];
    __shared__ int page_off[kPlanSmall + 1];
    plan_sequences(p, page_off, warp_sum);
    __syncthreads();
    for (int t = threadIdx.x; t < p.total_q; t += kPlanThreads) plan_token(p, page_off, t);
}

}  // namespace

cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream) {
    if (p.page_off == nullptr) {
        plan_small_kernel<<<1, kPlanThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    plan_scan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.total_q == 0) return e;  // (no tokens: no pages either, and a grid may not be empty)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((static_cast<unsigned>(p.total_q) + kPlanTokenThreads - 1) / kPlanTokenThreads);
    cfg.blockDim = dim3(kPlanTokenThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, plan_tokens_kernel, p);
}

}  // namespace attn
