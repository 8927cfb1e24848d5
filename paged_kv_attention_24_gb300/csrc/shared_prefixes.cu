// Groups of neighbouring requests whose page tables begin with the same pages.
//
// "Mini-SGLang 实战指南", §6.5 "Radix Cache": requests with a common prefix are
// given the same pages.  m_b is the length that rows b-1 and b have in common;
// row b joins the group of b-1 when m_b reaches min_shared, and a group shares
// the least m of its joined rows (the common prefix of a run of rows is the
// least of its neighbours' common prefixes).
//
// Bound by latency (a batch's tables are at most a few megabytes).  Small tables take one launch
// (small_prefixes_kernel).  Others take two: one block per row compares it with the row before, 4096
// columns a round, done at the first round with a difference; one block then finds each group's start
// and least m by a scan over the rows.  m travels in shared_lens, which the scan overwrites, so the
// call needs no scratch.  64 requests: 3.1 us up to 1024 columns, 5 us for 16384 equal ones.  Slower:
// blocks of 256 threads (+2 us at 16384 columns) or of 1024 (+2.7 us for 1024 requests).
#include <limits.h>

#include "kernels.h"

namespace msgl {

namespace {

constexpr int kThreads = 512;
constexpr int kPerThread = 8;

__device__ __forceinline__ bool row_ok(const SharedPrefixesArgs &a, int s) {
    return s >= 1 && s <= a.max_seq_len && ((s - 1) >> a.log2_ps) < a.pages.width;
}

__global__ void __launch_bounds__(kThreads) row_match_kernel(const SharedPrefixesArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x;
    const int s1 = __ldg(a.seq_lens + b), s0 = b > 0 ? __ldg(a.seq_lens + b - 1) : 0;
    if (threadIdx.x == 0) {
        if (s1 < 1 || s1 > a.max_seq_len) report(a.status, MSGL_DEVERR_LENGTH);
        else if (!row_ok(a, s1)) report(a.status, MSGL_DEVERR_PAGE_RANGE);
    }
    int m = 0;
    if (b > 0 && row_ok(a, s0) && row_ok(a, s1)) {
        const int both = min(s0, s1);
        const int n = ((both - 1) >> a.log2_ps) + 1;
        const int32_t *x = a.pages.ids + (long long)(b - 1) * a.pages.stride, *y = x + a.pages.stride;
        __shared__ int first;
        if (threadIdx.x == 0) first = n;
        __syncthreads();
        for (int c0 = 0; c0 < n; c0 += kThreads * kPerThread) {
            int far = INT_MAX;
#pragma unroll
            for (int u = kPerThread - 1; u >= 0; --u) {
                const int p = c0 + u * kThreads + (int)threadIdx.x;
                if (p < n && __ldg(x + p) != __ldg(y + p)) far = p;
            }
            if (__syncthreads_or(far != INT_MAX)) {
                if (far != INT_MAX) atomicMin(&first, far);
                __syncthreads();
                break;
            }
        }
        m = (int)min((long long)first << a.log2_ps, (long long)both);
    }
    if (threadIdx.x == 0) a.shared_lens[b] = m;
}

// One block.  A row's group starts at the last row up to it that did not join (a max scan).
// Up to 1024 rows, one a thread, the least m of a group is gathered in shared memory: 3.0 us a call
// for 64 rows, against 4.4 in the global memory that larger batches use.  Those are taken 1024
// rows at a time, and a group's least m by atomicMin on its start row's entry, which holds no m of
// its own (1000 rows: 5.4 us; 1025: 7.7; 2048: 10.2).
constexpr int kScanThreads = 1024;

// Row threadIdx.x of at most one a thread, which has m in common with the row before.  warp_max: 32
// and least: blockDim.x entries of shared memory.
__device__ __forceinline__ void group_row(const SharedPrefixesArgs &a, int m, int *warp_max, int *least) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = threadIdx.x;
    const bool joined = b > 0 && b < a.num_reqs && m >= a.min_shared;
    const uint32_t starts = __ballot_sync(0xffffffffu, !joined);
    least[b] = INT_MAX;
    if (lane == 0) warp_max[warp] = starts ? b + 31 - __clz(starts) : 0;
    __syncthreads();
    const int before = (int)__reduce_max_sync(0xffffffffu, lane < warp ? (uint32_t)warp_max[lane] : 0u);
    const uint32_t mine = starts & (0xffffffffu >> (31 - lane));
    const int start = mine ? b - lane + 31 - __clz(mine) : before;
    if (joined) atomicMin(&least[start], m);
    __syncthreads();
    if (b < a.num_reqs) {
        const int shared = least[start];
        a.group_start[b] = start;
        a.shared_lens[b] = shared == INT_MAX ? 0 : shared;
    }
}

__global__ void __launch_bounds__(kScanThreads) row_groups_kernel(const SharedPrefixesArgs a) {
    __shared__ int warp_max[32];
    __shared__ int carry;
    __shared__ int least[kScanThreads];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) carry = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (a.num_reqs <= kScanThreads) {
        const int b = threadIdx.x;
        group_row(a, b < a.num_reqs ? __ldcg(a.shared_lens + b) : 0, warp_max, least);
        return;
    }
    __syncthreads();
    for (int c0 = 0; c0 < a.num_reqs; c0 += kScanThreads) {
        const int b = c0 + threadIdx.x;
        const int m = b < a.num_reqs ? __ldcg(a.shared_lens + b) : 0;
        const bool joined = b > 0 && m >= a.min_shared;
        int start = b < a.num_reqs && !joined ? b : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, start, o);
            if (lane >= o) start = max(start, u);
        }
        if (lane == 31) warp_max[warp] = start;
        __syncthreads();
        int before = carry;
        for (int w = 0; w < warp; ++w) before = max(before, warp_max[w]);
        start = max(start, before);
        if (b < a.num_reqs) {
            a.group_start[b] = start;
            if (!joined) a.shared_lens[b] = INT_MAX;   // no m of its own: gathers the group's
        }
        __syncthreads();
        if (threadIdx.x == kScanThreads - 1) carry = start;
        if (b < a.num_reqs && joined) atomicMin(a.shared_lens + start, m);
        __syncthreads();
    }
    // (read past L1: the atomics above worked in L2)
    for (int b = threadIdx.x; b < a.num_reqs; b += kScanThreads) {
        const int start = a.group_start[b];
        if (start != b) a.shared_lens[b] = __ldcg(a.shared_lens + start);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < a.num_reqs; b += kScanThreads)
        if (__ldcg(a.shared_lens + b) == INT_MAX) a.shared_lens[b] = 0;
}

// Both steps in one launch, for small tables: a cluster of 8 blocks, one warp for each row and one
// round of loads for all its columns; m goes into the first block's shared memory.  64 rows of 128
// columns: 2.7 us in a graph and 4.1 launched one by one (two kernels: 3.1 and 5.5); 512 columns in two
// rounds took 4.0 and 6.2 (3.1 and 5.4), 256 rows in two 3.4 and 5.2 (3.2 and 5.2).
constexpr int kCluster = 8, kSmallRows = kCluster * kThreads / 32, kSmallColumns = 32 * kPerThread;

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    small_prefixes_kernel(const SharedPrefixesArgs a) {
    __shared__ int warp_max[32];
    __shared__ int least[kThreads], common[kSmallRows];
    const int lane = threadIdx.x & 31, b = blockIdx.x + kCluster * (int)(threadIdx.x >> 5);
    uint32_t first_block;   // the first block's `common`
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(first_block) : "r"((uint32_t)__cvta_generic_to_shared(common)));
    // (the first block has to be running before another writes into its shared memory)
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    int m = 0;
    if (b < a.num_reqs) {
        const int s1 = __ldg(a.seq_lens + b), s0 = b > 0 ? __ldg(a.seq_lens + b - 1) : 0;
        if (lane == 0) {
            if (s1 < 1 || s1 > a.max_seq_len) report(a.status, MSGL_DEVERR_LENGTH);
            else if (!row_ok(a, s1)) report(a.status, MSGL_DEVERR_PAGE_RANGE);
        }
        if (b > 0 && row_ok(a, s0) && row_ok(a, s1)) {
            const int both = min(s0, s1);
            const int n = ((both - 1) >> a.log2_ps) + 1;   // at most kSmallColumns
            const int32_t *x = a.pages.ids + (long long)(b - 1) * a.pages.stride, *y = x + a.pages.stride;
            int far = n;
#pragma unroll
            for (int u = kPerThread - 1; u >= 0; --u) {
                const int p = u * 32 + lane;
                if (p < n && __ldg(x + p) != __ldg(y + p)) far = p;
            }
            far = __reduce_min_sync(0xffffffffu, far);
            m = (int)min((long long)far << a.log2_ps, (long long)both);
        }
    }
    asm volatile("barrier.cluster.wait;" ::: "memory");
    if (lane == 0) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(first_block + 4 * b), "r"(m) : "memory");
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (blockIdx.x == 0) group_row(a, threadIdx.x < kSmallRows ? common[threadIdx.x] : 0, warp_max, least);
}

}  // namespace

cudaError_t launch_shared_prefixes(const SharedPrefixesArgs &a, cudaStream_t stream) {
    if (a.num_reqs <= kSmallRows && min(a.pages.width, ((a.max_seq_len - 1) >> a.log2_ps) + 1) <= kSmallColumns) {
        small_prefixes_kernel<<<kCluster, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    row_match_kernel<<<a.num_reqs, kThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kScanThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, row_groups_kernel, a);
}

}  // namespace msgl
