// Drafted tokens accepted or replaced by the target's probabilities.
//
// A draft x_i, drawn from q, stands when u_i q(x_i) < p(x_i), p being the target's
// probabilities of its place; the first one that does not stand is replaced by a
// token drawn from max(p - q, 0), and a request whose drafts all stand gets one more
// token drawn from p ("Mini-SGLang 实战指南", §6.4: a decode step is a launch of
// fixed shape, so nothing of this may wait for the host).  The result is
// distributed as if every token had been drawn from p.
//
// Drawing takes the first token at which the running sum of the weights passes
// u times their total.  Tokens are whole numbers, so the sums are kept to about 48
// bits (pairs of 32-bit numbers for a lane's own, 64 bits where lanes join): with
// 32 bits one draw in some hundred would fall on a neighbour.
//
// Bound by HBM for large batches (one row of p, and of q where a draft was refused,
// is read once), by latency for small ones.  A cluster of blocks takes a request,
// so that a row is read by many SMs; each warp sums a run of neighbouring tokens,
// the blocks exchange their warps' sums, and only the run in which the draw falls
// is read again (out of L2).
#include "kernels.h"

namespace msgl {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }

// max(p - q, 0); what is no number counts nothing.
__device__ __forceinline__ float weight(float p, float q) { return p > q ? p - q : 0.f; }

// (hi, lo) += x, with the rounding error of the sum kept in lo (Knuth's two-sum).
__device__ __forceinline__ void add(float &hi, float &lo, float x) {
    const float s = hi + x, b = s - hi;
    lo += (hi - (s - b)) + (x - b);
    hi = s;
}

// What is left to draw from: row p, less row q (NULL: none) or less all of token `without`.
template <class T>
struct Row {
    const T *p, *q;
    int without;
    __device__ __forceinline__ float at(int i) const {
        return weight(value(p[i]), q ? value(q[i]) : i == without ? INFINITY : 0.f);
    }
};

struct Shared {
    double sums[kWarps];
    double warp[kWarps];
    double draw, before;             // u * total; the weights in front of the drawn run
    int drafts, accepted, run, drawn, last;
    bool bad;
};

// Sum of the weights of tokens [i0, i1).
template <class T>
__device__ __forceinline__ double run_sum(const Row<T> &r, int i0, int i1) {
    const int lane = threadIdx.x & 31;
    float hi = 0.f, lo = 0.f;
#pragma unroll 8
    for (int i = i0 + lane; i < i1; i += 32) add(hi, lo, r.at(i));
    double sum = (double)hi + (double)lo;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// How many drafts stand: the first one that does not, or all.
template <class T>
__device__ __forceinline__ int standing(const VerifyArgs &a, int first, int drafts, bool &bad_token) {
    const int lane = threadIdx.x & 31;
    const T *p = static_cast<const T *>(a.target), *q = static_cast<const T *>(a.draft);
    for (int i0 = 0; i0 < drafts; i0 += 32) {
        const int i = i0 + lane;
        bool ok = true, bad = false;
        if (i < drafts) {
            const int64_t row = first + i;
            const int x = __ldg(a.tokens + row + 1);
            bad = x < 0 || x >= a.vocab;
            ok = false;
            if (!bad) {
                const double u = __ldg(a.accept_u + row);
                const double qx = q ? (double)value(q[row * a.draft_stride + x]) : 1.0;
                ok = u * qx < (double)value(p[row * a.target_stride + x]);
            }
        }
        bad_token |= __any_sync(0xffffffffu, bad);
        const uint32_t fails = ~__ballot_sync(0xffffffffu, ok);
        if (fails) return i0 + __ffs(fails) - 1;
    }
    return drafts;
}

template <class T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a, int cluster) {
    __shared__ Shared s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = cluster_rank(), b = blockIdx.x / cluster;
    const int first = __ldg(a.cu_ext + b), end = __ldg(a.cu_ext + b + 1);
    const bool ok = first >= 0 && first <= end && end <= a.total_tokens;
    if (!ok || first == end) {
        // no rows of its own: nothing drafted, nothing drawn
        if (rank == 0 && threadIdx.x == 0) {
            a.accepted[b] = 0;
            a.kv_lens[b] = a.cached_lens ? __ldg(a.cached_lens + b) : 0;
            if (!ok) report(a.status, MSGL_DEVERR_LENGTH);
        }
        return;
    }
    const int drafts = end - first - 1;
    if (warp == 0) {
        bool bad = false;
        const int n = standing<T>(a, first, drafts, bad);
        if (lane == 0) {
            s.accepted = n;
            s.drawn = INT32_MAX;
            s.last = -1;
            if (bad && rank == 0) report(a.status, MSGL_DEVERR_TOKEN);
        }
    }
    __syncthreads();
    const int taken = s.accepted, row = first + taken;
    const bool refused = taken < drafts;
    Row<T> r{static_cast<const T *>(a.target) + row * a.target_stride,
             refused && a.draft ? static_cast<const T *>(a.draft) + row * a.draft_stride : nullptr,
             refused && !a.draft ? __ldg(a.tokens + row + 1) : -1};
    if (rank == 0)
        for (int i = threadIdx.x; i <= drafts; i += kThreads)
            if (i != taken) a.out_tokens[first + i] = i < taken ? __ldg(a.tokens + first + i + 1) : -1;
    if (rank == 0 && threadIdx.x == 0) {
        a.accepted[b] = taken;
        a.kv_lens[b] = (a.cached_lens ? __ldg(a.cached_lens + b) : 0) + taken + 1;
    }
    const int runs = cluster * kWarps, length = (a.vocab + runs - 1) / runs;
    const int mine = rank * kWarps + warp;
    for (int pass = 0;; ++pass) {
        const int i0 = min((int64_t)mine * length, (int64_t)a.vocab), i1 = min((int64_t)i0 + length, (int64_t)a.vocab);
        const double sum = run_sum(r, i0, i1);
        if (lane == 0) s.sums[warp] = sum;
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        // every block goes through all runs' sums in the same order and so comes to the same end
        if (warp == 0) {
            constexpr int kEach = kMaxCluster * kWarps / 32;
            double x[kEach], upto[kEach], sum = 0;
            const int each = runs / 32 > 0 ? runs / 32 : 1;    // runs of a lane
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int i = lane * each + k;
                x[k] = 0;
                if (k < each && i < runs) {
                    uint32_t at;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;"
                        : "=r"(at)
                        : "r"((uint32_t)__cvta_generic_to_shared(&s.sums[i % kWarps])), "r"(i / kWarps));
                    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(x[k]) : "r"(at) : "memory");
                }
                sum += x[k];
                upto[k] = sum;
            }
            double scan = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, scan, o);
                if (lane >= o) scan += y;
            }
            const double total = __shfl_sync(0xffffffffu, scan, 31);
            double lower = __shfl_up_sync(0xffffffffu, scan, 1);
            if (lane == 0) lower = 0;
            const double draw = (double)__ldg(a.sample_u + b) * total;
            // the first run at which the sum passes the draw, else the last one with any weight
            int run = INT32_MAX, heavy = -1;
#pragma unroll
            for (int k = kEach - 1; k >= 0; --k) {
                if (k < each && lower + upto[k] > draw && x[k] > 0) run = lane * each + k;
                if (k < each && x[k] > 0 && heavy < 0) heavy = lane * each + k;
            }
            const int found = __reduce_min_sync(0xffffffffu, run), final = __reduce_max_sync(0xffffffffu, heavy);
            const int chosen = found != INT32_MAX ? found : final;
#pragma unroll
            for (int k = 0; k < kEach; ++k)
                if (k < each && lane * each + k == chosen) s.before = lower + upto[k] - x[k];
            if (lane == 0) {
                s.draw = draw;
                s.run = chosen;
                s.bad = !(total > 0 && total <= 3.4e38);
            }
        }
        __syncthreads();
        // nothing left over (p nowhere above q): the target's own row
        const bool again = s.bad && pass == 0 && refused;
        // (no block leaves, or sums anew, while another may still read its sums)
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        if (!again) break;
        r.q = nullptr;
        r.without = -1;
    }
    if (s.bad) {
        if (rank == 0 && threadIdx.x == 0) {
            a.out_tokens[row] = -1;
            report(a.status, MSGL_DEVERR_PROBS);
        }
        return;
    }
    if (s.run / kWarps != rank) return;
    // the token within the run
    const int i0 = s.run * length, i1 = min(i0 + length, a.vocab);
    double before = s.before;
    for (int t = i0; t < i1; t += kThreads) {
        const int i = t + threadIdx.x;
        const float w = i < i1 ? r.at(i) : 0.f;
        double scan = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += y;
        }
        if (lane == 31) s.warp[warp] = scan;
        __syncthreads();
        double lower = before, all = before;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            if (k < warp) lower += s.warp[k];
            all += s.warp[k];
        }
        if (w > 0 && lower + scan > s.draw) atomicMin(&s.drawn, i);
        if (w > 0) atomicMax(&s.last, i);
        before = all;
        __syncthreads();
        if (s.drawn != INT32_MAX) break;
    }
    if (threadIdx.x == 0) a.out_tokens[row] = s.drawn != INT32_MAX ? s.drawn : s.last;
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs &a, cudaStream_t stream) {
    int cluster = kMaxCluster;
    while (cluster > 1 && a.vocab < cluster * 2048) cluster /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.num_reqs * cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.bf16 ? cudaLaunchKernelEx(&cfg, verify_kernel<__nv_bfloat16>, a, cluster)
                  : cudaLaunchKernelEx(&cfg, verify_kernel<float>, a, cluster);
}

}  // namespace msgl
