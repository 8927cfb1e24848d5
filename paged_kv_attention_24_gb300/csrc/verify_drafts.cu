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
// u times their total.  Tokens are whole numbers, so the sums are kept to about 46
// bits, as unevaluated pairs of 32-bit numbers (Knuth's two-sum; with 32 bits one
// draw of some hundred from a flat row falls on a neighbour, and this GPU adds 64-bit
// numbers at a sixty-fourth of the rate).
//
// Bound by HBM for large batches (one row of p, and of q where a draft was refused,
// is read once), by latency for small ones.  A cluster of blocks takes a request,
// so that a row is read by many SMs; each warp sums a run of neighbouring tokens,
// the blocks exchange their warps' sums, and only the run in which the draw falls
// is read again (out of L2).  128 requests over 131072 tokens of fp32: 27 us (the rows alone
// 18 us at the copy rate; lookups in front, exchange and draw behind take the rest); 4 over
// 50001 of bf16: 6.8 us.  With 64-bit sums: 72 and 14 us.
#include "kernels.h"

namespace msgl {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// hi + lo, |lo| at most half a unit of hi's last place.
struct Sum {
    float hi, lo;
};

// The exact error of s = a + b, in whichever order of size.
__device__ __forceinline__ float two_sum_error(float a, float b, float s) {
    const float t = s - a;
    return (a - (s - t)) + (b - t);
}

__device__ __forceinline__ Sum settled(float hi, float lo) {
    const float s = hi + lo;
    return Sum{s, lo - (s - hi)};
}

__device__ __forceinline__ Sum operator+(const Sum &a, const Sum &b) {
    const float s = a.hi + b.hi;
    return settled(s, two_sum_error(a.hi, b.hi, s) + (a.lo + b.lo));
}

__device__ __forceinline__ Sum times(float u, const Sum &a) {
    const float p = u * a.hi;
    return settled(p, fmaf(u, a.lo, fmaf(u, a.hi, -p)));
}

__device__ __forceinline__ bool operator>(const Sum &a, const Sum &b) {
    return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}

__device__ __forceinline__ Sum shfl(const Sum &a, int lane) {
    return Sum{__shfl_sync(0xffffffffu, a.hi, lane), __shfl_sync(0xffffffffu, a.lo, lane)};
}

// Sums over the warp's lanes before this one (before) and up to this one (returned).
__device__ __forceinline__ Sum warp_scan(Sum x, Sum &before) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum y{__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
        if (lane >= o) x = y + x;
    }
    before = Sum{__shfl_up_sync(0xffffffffu, x.hi, 1), __shfl_up_sync(0xffffffffu, x.lo, 1)};
    if (lane == 0) before = Sum{0.f, 0.f};
    return x;
}

// The first lane with any weight x at which the running sum `upto` passes the draw, else the last one with any; -1
// when there is none.
__device__ __forceinline__ int drawn_lane(const Sum &x, const Sum &upto, const Sum &draw) {
    const uint32_t heavy = __ballot_sync(0xffffffffu, x.hi > 0), over = __ballot_sync(0xffffffffu, x.hi > 0 && upto > draw);
    return over ? __ffs(over) - 1 : 31 - __clz(heavy);
}

// max(p - q, 0); what is no number counts nothing.
__device__ __forceinline__ float weight(float p, float q) { return p > q ? p - q : 0.f; }

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }

// 16 bytes of a row.
template <class T>
struct Vec {
    static constexpr int kN = 16 / sizeof(T);
    uint4 r;
    __device__ __forceinline__ float operator[](int k) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        if constexpr (kN == 4) return __uint_as_float(w[k]);
        else return k % 2 ? bf16_hi(w[k / 2]) : bf16_lo(w[k / 2]);
    }
};

// Tokens i .. i + kN - 1 of a row; zeros outside [0, vocab).  aligned: the address is a multiple of 16.
template <class T>
__device__ __forceinline__ Vec<T> fetch(const T *row, int i, int vocab, bool aligned) {
    constexpr int kN = Vec<T>::kN;
    Vec<T> v;
    if (aligned && i >= 0 && i + kN <= vocab) {
        v.r = ld_stream_16(row + i);
        return v;
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        if (i + k < 0 || i + k >= vocab) continue;
        if constexpr (kN == 4) w[k] = __ldg(reinterpret_cast<const uint32_t *>(row) + i + k);
        else w[k / 2] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(row) + i + k) << (16 * (k % 2));
    }
    v.r = make_uint4(w[0], w[1], w[2], w[3]);
    return v;
}

// What is left to draw from: row p, less row q (NULL: none) or less all of token `without`.  Tokens are
// taken in vectors whose p is aligned: vector n holds tokens n * kN - shift onwards.
template <class T>
struct Row {
    const T *p, *q;
    int without, shift, vocab;
    bool q_aligned;

    __device__ __forceinline__ void set(const T *p_, const T *q_, int without_, int vocab_) {
        constexpr int kN = Vec<T>::kN;
        p = p_;
        q = q_;
        without = without_;
        vocab = vocab_;
        shift = (int)(reinterpret_cast<uintptr_t>(p) / sizeof(T) % kN);
        q_aligned = (reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(q)) % 16 == 0;
    }
    __device__ __forceinline__ int vectors() const { return (int)(((int64_t)vocab + shift + Vec<T>::kN - 1) / Vec<T>::kN); }
    __device__ __forceinline__ int token(int vector) const { return vector * Vec<T>::kN - shift; }
    __device__ __forceinline__ Vec<T> target(int vector) const { return fetch(p, token(vector), vocab, true); }
    __device__ __forceinline__ Vec<T> draft(int vector) const {
        return q ? fetch(q, token(vector), vocab, q_aligned) : Vec<T>{make_uint4(0, 0, 0, 0)};
    }
    __device__ __forceinline__ float at(int vector, int k, const Vec<T> &x, const Vec<T> &y) const {
        const float w = weight(x[k], y[k]);
        return token(vector) + k == without ? 0.f : w;
    }
    __device__ __forceinline__ float at(int i) const {   // token i, by itself
        return i < 0 || i >= vocab || i == without ? 0.f : weight(value(p[i]), q ? value(q[i]) : 0.f);
    }
};

struct Shared {
    Sum sums[kWarps], total;         // of this block's runs, and of the block
    Sum warp[kWarps];
    Sum draw, before;                // u * total; the weights in front of the drawn run
    int accepted, run, drawn, last;  // run: of this block's, -1 when the draw is in another block
    bool bad;
};

// Sum of the weights of vectors [n0, n1).
template <class T>
__device__ __forceinline__ Sum run_sum(const Row<T> &r, int n0, int n1) {
    constexpr int kN = Vec<T>::kN, kUnroll = 4;
    const int lane = threadIdx.x & 31;
    // (four sums, so that one does not wait for the last; as two pairs, by the instructions that add two floats at once,
    // 39 us in place of 27 for 128 requests)
    float hi[4] = {}, lo[4] = {};
    for (int n = n0 + lane; n < n1; n += 32 * kUnroll) {
        Vec<T> x[kUnroll], y[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (n + 32 * u < n1) {
                x[u] = r.target(n + 32 * u);
                y[u] = r.draft(n + 32 * u);
            }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (n + 32 * u < n1)
#pragma unroll
                for (int k = 0; k < kN; ++k) {
                    const float w = r.at(n + 32 * u, k, x[u], y[u]), s = hi[k % 4] + w;
                    lo[k % 4] += two_sum_error(hi[k % 4], w, s);
                    hi[k % 4] = s;
                }
    }
    Sum sum = (settled(hi[0], lo[0]) + settled(hi[1], lo[1])) + (settled(hi[2], lo[2]) + settled(hi[3], lo[3]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum = sum + Sum{__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)};
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
            const float u = __ldg(a.accept_u + row);
            bad = x < 0 || x >= a.vocab;
            ok = false;
            if (!bad) {
                // (the product of two 24-bit numbers is exact in 64 bits)
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
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyArgs a, int log2_cluster) {
    const int cluster = 1 << log2_cluster, log2_runs = log2_cluster + 4;
    static_assert(kWarps == 16, "a block of 16 runs");
    __shared__ Shared s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = cluster_rank(), b = blockIdx.x >> log2_cluster;
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
    const float sample = __ldg(a.sample_u + b);
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
    const T *p = static_cast<const T *>(a.target) + row * a.target_stride;
    Row<T> r;
    r.set(p, refused && a.draft ? static_cast<const T *>(a.draft) + row * a.draft_stride : nullptr,
          refused && !a.draft ? __ldg(a.tokens + row + 1) : -1, a.vocab);
    const int vectors = r.vectors();
    const int length = ((vectors - 1) >> log2_runs) / 32 * 32 + 32;       // whole rounds of a warp
    const int mine = rank * kWarps + warp;
    for (bool second = false;; second = true) {
        const int n0 = (int)min((int64_t)mine * length, (int64_t)vectors), n1 = min(n0 + length, vectors);
        const Sum sum = run_sum(r, n0, n1);
        if (lane == 0) s.sums[warp] = sum;
        __syncthreads();
        Sum x{0.f, 0.f}, upto, lower;
        if (warp == 0) {
            if (lane < kWarps) x = s.sums[lane];
            upto = warp_scan(x, lower);
            if (lane == 31) s.total = upto;
        }
        cluster_arrive();
        if (rank == 0 && !second) {
            // (written here, where the block waits anyway)
            for (int i = threadIdx.x; i <= drafts; i += kThreads)
                if (i != taken) a.out_tokens[first + i] = i < taken ? __ldg(a.tokens + first + i + 1) : -1;
            if (threadIdx.x == kThreads - 1) {
                a.accepted[b] = taken;
                a.kv_lens[b] = (a.cached_lens ? __ldg(a.cached_lens + b) : 0) + taken + 1;
            }
        }
        cluster_wait();
        // Every block goes through all blocks' sums in the same order and so comes to the same end; the one that
        // the draw falls into goes on to its runs.  (One warp over all runs' sums at once, four a lane, was more
        // code than it was worth: 7.2 against 6.8 us for 4 requests.  Rolled scans: 8.0.)
        if (warp == 0) {
            Sum y{0.f, 0.f}, ahead;
            if (lane < cluster) {
                uint32_t at;
                asm("mapa.shared::cluster.u32 %0, %1, %2;"
                    : "=r"(at)
                    : "r"((uint32_t)__cvta_generic_to_shared(&s.total)), "r"(lane));
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(y.hi), "=f"(y.lo) : "r"(at) : "memory");
            }
            const Sum blocks = warp_scan(y, ahead), total = shfl(blocks, 31), draw = times(sample, total);
            const bool bad = !(total.hi > 0 && total.hi <= 3.4e38f);
            int run = -1;
            if (!bad && drawn_lane(y, blocks, draw) == rank) {
                const Sum base = shfl(ahead, rank);
                run = drawn_lane(x, base + upto, draw);
                if (lane == run) s.before = base + lower;
            }
            if (lane == 0) {
                s.draw = draw;
                s.run = run;
                s.bad = bad;
            }
        }
        // (no block leaves, or sums anew, while another may still read its sums)
        cluster_arrive();
        __syncthreads();
        // nothing left over (p nowhere above q): the target's own row
        if (second || !s.bad || !refused) break;
        cluster_wait();
        r.set(p, nullptr, -1, a.vocab);
    }
    if (s.bad) {
        if (rank == 0 && threadIdx.x == 0) {
            a.out_tokens[row] = -1;
            report(a.status, MSGL_DEVERR_PROBS);
        }
    } else if (s.run >= 0) {
        // the token within the run: four a thread
        constexpr int kEach = 4;
        const int n0 = (rank * kWarps + s.run) * length, i1 = r.token(min(n0 + length, vectors));
        Sum before = s.before;
        for (int t = r.token(n0); t < i1; t += kEach * kThreads) {
            const int i = t + kEach * (int)threadIdx.x;
            float w[kEach];
            Sum own{0.f, 0.f}, lower, ahead;
#pragma unroll
            for (int k = 0; k < kEach; ++k) w[k] = i + k < i1 ? r.at(i + k) : 0.f;
#pragma unroll
            for (int k = 0; k < kEach; ++k) own = own + Sum{w[k], 0.f};
            const Sum upto = warp_scan(own, lower);
            if (lane == 31) s.warp[warp] = upto;
            __syncthreads();
            const Sum warps = warp_scan(lane < kWarps ? s.warp[lane] : Sum{0.f, 0.f}, ahead);
            Sum sum = (before + shfl(ahead, warp)) + lower;
            before = before + shfl(warps, 31);
            if (own.hi > 0) {
                int drawn = INT32_MAX, last = -1;
#pragma unroll
                for (int k = 0; k < kEach; ++k) {
                    sum = sum + Sum{w[k], 0.f};
                    if (w[k] > 0) last = i + k;
                    if (w[k] > 0 && drawn == INT32_MAX && sum > s.draw) drawn = i + k;
                }
                if (drawn != INT32_MAX) atomicMin(&s.drawn, drawn);
                atomicMax(&s.last, last);
            }
            __syncthreads();
            if (s.drawn != INT32_MAX) break;
        }
        if (threadIdx.x == 0) a.out_tokens[row] = s.drawn != INT32_MAX ? s.drawn : s.last;
    }
    cluster_wait();
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs &a, cudaStream_t stream) {
    // As many blocks a request as all run at once, so that none begins its chain of lookups behind another's
    // row: two blocks an SM, in GPCs of 19 SMs on average, which hold 4 clusters of 8 blocks, 9 of 4 or 19 of 2;
    // and at least 2048 tokens a block.  131072 tokens, us with 1, 2, 4, 8 blocks: 16 requests 33.6, 20.2, 13.5,
    // 12.0; 64 (bf16) 24.2, 15.7, 14.7, 20.2; 128 36.6, 27.9, 31.2, 41.8; 37 (100003 tokens) 28.8, 18.7, 15.0, 18.0.
    // Blocks of 256 threads, four an SM, are at most 3% ahead (small batches) and up to 18% behind.
    const int sms = sm_count(), n = a.num_reqs;
    int log2_cluster = n <= sms * 4 / 19 ? 3 : n <= sms * 9 / 19 ? 2 : n <= sms ? 1 : 0;
    while (log2_cluster > 0 && a.vocab < 2048 << log2_cluster) --log2_cluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.num_reqs << log2_cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << log2_cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.bf16 ? cudaLaunchKernelEx(&cfg, verify_kernel<__nv_bfloat16>, a, log2_cluster)
                  : cudaLaunchKernelEx(&cfg, verify_kernel<float>, a, log2_cluster);
}

}  // namespace msgl
