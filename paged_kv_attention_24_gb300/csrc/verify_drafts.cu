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
// so that a row is read by many SMs; each warp sums a run of neighbouring tokens and
// writes its sum into the shared memory of all the cluster's blocks, each of which
// then finds the run in which the draw falls; only that one is read again (out of L2), by
// the block that summed it, or, where runs are short, not even that one.  128 requests
// over 131072 tokens of fp32: 24.6 us (the rows alone 18 us at the copy rate; lookups in
// front, exchange and draw behind take the rest); 4 over 50001 of bf16: 4.9 us.  With
// 64-bit sums: 72 and 14 us.  Sums sent by st.async and waited for by one warp, in place
// of the cluster's barrier: 25.8 us, and 0.25 less for 4 requests.
#include "cluster.cuh"
#include "kernels.h"

namespace msgl {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;

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

// The same without settling (lo a few units of hi's last place), for sums of a few that settle at the end: a third
// fewer instructions in the chains behind the rows (6.0 -> 5.5 us for 4 requests).
__device__ __forceinline__ Sum loose(const Sum &a, const Sum &b) {
    const float s = a.hi + b.hi;
    return Sum{s, two_sum_error(a.hi, b.hi, s) + (a.lo + b.lo)};
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

// Sum over the warp's lanes up to this one.
__device__ __forceinline__ Sum warp_scan(Sum x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum y{__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
        if (lane >= o) x = loose(y, x);
    }
    return settled(x.hi, x.lo);
}

// The sum up to the lane before, from the sums up to each lane.
__device__ __forceinline__ Sum lane_before(const Sum &upto) {
    const Sum x{__shfl_up_sync(0xffffffffu, upto.hi, 1), __shfl_up_sync(0xffffffffu, upto.lo, 1)};
    return threadIdx.x & 31 ? x : Sum{0.f, 0.f};
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
    Sum runs[8 * kWarps];            // the sums of all the cluster's runs
    Sum warp[kWarps];
    Sum draw, before;                // u * total; the weights in front of the drawn run
    int first, drafts;               // the request's first row, its drafts
    int accepted, refused;           // drafts that stand, the token of the one that does not
    float sample;
    int run, last;                   // the drawn run; the last token with any weight in the tiles gone by
    bool bad;
};

// Four sums, and all lanes' of them, as one.
__device__ __forceinline__ Sum warp_sum(const float (&hi)[4], const float (&lo)[4]) {
    Sum sum = loose(loose(Sum{hi[0], lo[0]}, Sum{hi[1], lo[1]}), loose(Sum{hi[2], lo[2]}, Sum{hi[3], lo[3]}));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum = loose(sum, Sum{__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)});
    return settled(sum.hi, sum.lo);
}

constexpr int kUnroll = 4;           // vectors of a row that a lane has on the way

// Sum of the weights of vectors [n0, n1).
template <class T>
__device__ __forceinline__ Sum run_sum(const Row<T> &r, int n0, int n1) {
    constexpr int kN = Vec<T>::kN;
    const int lane = threadIdx.x & 31;
    // (four sums, so that one does not wait for the last; as two pairs, by the instructions that add two floats at once,
    // 39 us in place of 27 for 128 requests)
    float hi[4] = {}, lo[4] = {};
    // (four vectors of each row on the way; 128 requests: three 25.2 us, two 26.6, six, which spill, 29.2)
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
    return warp_sum(hi, lo);
}

// Vectors a lane of a short run: as many weights as a lane has registers for (four of fp32 are spilled).
template <class T>
constexpr int kShortRun = sizeof(T) == 4 ? 3 : 2;

// The same of a short run, whose weights stay in w.
template <class T>
__device__ __forceinline__ Sum run_sum(const Row<T> &r, int n0, int n1, float (&w)[kShortRun<T>][Vec<T>::kN]) {
    constexpr int kN = Vec<T>::kN, kUnroll = kShortRun<T>;
    const int n = n0 + (threadIdx.x & 31);
    float hi[4] = {}, lo[4] = {};
    Vec<T> x[kUnroll], y[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        if (n + 32 * u < n1) {
            x[u] = r.target(n + 32 * u);
            y[u] = r.draft(n + 32 * u);
        }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            w[u][k] = n + 32 * u < n1 ? r.at(n + 32 * u, k, x[u], y[u]) : 0.f;
            const float s = hi[k % 4] + w[u][k];
            lo[k % 4] += two_sum_error(hi[k % 4], w[u][k], s);
            hi[k % 4] = s;
        }
    return warp_sum(hi, lo);
}

// The token (of the run's vectors, from n0 on) at which the running sum passes the draw; where rounding lets none pass, the
// last one with any weight.  By the warp that has the run's weights.
template <class T>
__device__ __forceinline__ void draw_token(const Row<T> &r, int n0, const float (&w)[kShortRun<T>][Vec<T>::kN],
                                           Sum before, const Sum &draw, int32_t *out) {
    constexpr int kN = Vec<T>::kN, kUnroll = kShortRun<T>;
    const int lane = threadIdx.x & 31;
    Sum upto[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        Sum own{w[u][0], 0.f};
#pragma unroll
        for (int k = 1; k < kN; ++k) own = loose(own, Sum{w[u][k], 0.f});
        upto[u] = warp_scan(own);
    }
    float drawn[kN] = {};                                        // the lane's weights of the drawn round
    Sum ahead{0.f, 0.f};
    int round = -1, owner = 0;
    bool passed = false;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        bool any = false;
#pragma unroll
        for (int k = 0; k < kN; ++k) any |= w[u][k] > 0;
        const uint32_t heavy = __ballot_sync(0xffffffffu, any),
                       over = __ballot_sync(0xffffffffu, any && before + upto[u] > draw);
        if (heavy && !passed) {
            passed = over;
            round = u;
            owner = over ? __ffs(over) - 1 : 31 - __clz(heavy);
            ahead = before + lane_before(upto[u]);
#pragma unroll
            for (int k = 0; k < kN; ++k) drawn[k] = w[u][k];
        }
        before = before + shfl(upto[u], 31);
    }
    if (lane != owner || round < 0) return;
    int token = -1;
    passed = false;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        ahead = ahead + Sum{drawn[k], 0.f};
        if (drawn[k] > 0 && !passed) {
            token = r.token(n0 + lane + 32 * round) + k;
            passed = ahead > draw;
        }
    }
    *out = token;
}

// How many drafts stand: the first one that does not (its token in `refused`), or all.
template <class T>
__device__ __forceinline__ int standing(const VerifyArgs &a, int first, int drafts, int &refused, bool &bad_token) {
    const int lane = threadIdx.x & 31;
    const T *p = static_cast<const T *>(a.target), *q = static_cast<const T *>(a.draft);
    for (int i0 = 0; i0 < drafts; i0 += 32) {
        const int i = i0 + lane;
        bool ok = true, bad = false;
        int x = -1;
        if (i < drafts) {
            const int64_t row = first + i;
            x = __ldg(a.tokens + row + 1);
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
        if (fails) {
            refused = __shfl_sync(0xffffffffu, x, __ffs(fails) - 1);
            return i0 + __ffs(fails) - 1;
        }
    }
    refused = -1;
    return drafts;
}

// The token at which the running sum passes the draw, of tokens [i0, i1) of the drawn run, E a thread in each tile:
// the block's warps scan a tile, and the warp that the draw falls into goes on to its lanes.  By the whole block.
template <int E, class T>
__device__ __forceinline__ void draw_token(const Row<T> &r, Shared &s, int i0, int i1, int32_t *out) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Sum draw = s.draw;
    Sum before = s.before;
    for (int t = i0;; t += E * kThreads) {
        const int i = t + E * (int)threadIdx.x;
        float w[E];
        Sum own{0.f, 0.f};
#pragma unroll
        for (int k = 0; k < E; ++k) w[k] = i + k < i1 ? r.at(i + k) : 0.f;
#pragma unroll
        for (int k = 0; k < E; ++k) own = loose(own, Sum{w[k], 0.f});
        const Sum upto = warp_scan(own), lower = lane_before(upto);
        if (lane == 31) s.warp[warp] = upto;
        __syncthreads();
        const Sum x = lane < kWarps ? s.warp[lane] : Sum{0.f, 0.f}, warps = warp_scan(x), ahead = lane_before(warps);
        // (where rounding lets no token pass, the last one with any weight counts)
        const int chosen = drawn_lane(x, before + warps, draw);
        const bool passes = __any_sync(0xffffffffu, x.hi > 0 && before + warps > draw), ends = t + E * kThreads >= i1;
        if (warp == chosen) {
            const Sum base = before + shfl(ahead, warp);
            if (lane == drawn_lane(own, base + upto, draw)) {
                Sum sum = base + lower;
                int drawn = -1, last = -1;
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    sum = sum + Sum{w[k], 0.f};
                    if (w[k] > 0) last = i + k;
                    if (w[k] > 0 && drawn < 0 && sum > draw) drawn = i + k;
                }
                if (passes || ends) *out = drawn >= 0 ? drawn : last;
                else s.last = last;
            }
        } else if (chosen < 0 && ends && threadIdx.x == 0) {
            *out = s.last;
        }
        if (passes || ends) return;
        before = before + shfl(warps, 31);
        __syncthreads();
    }
}

// kShort: runs are short, and the drawn one's weights are still in its warp's registers (4 requests over 50001 tokens of
// bf16: read again 5.5 us, else 5.0; one over 32000 of fp32 5.1 and 4.6; 300 over 8000 of bf16 8.2 and 7.5).
template <class T, bool kShort>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyArgs a, int log2_cluster) {
    const int cluster = 1 << log2_cluster, log2_runs = log2_cluster + 4;
    static_assert(kWarps == 16, "a block of 16 runs");
    __shared__ Shared s;
    // (the others have to be running before this block writes into their shared memory)
    cluster_started();
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
    if (warp == 0) {
        const float sample = __ldg(a.sample_u + b);
        bool bad = false;
        int token;
        const int n = standing<T>(a, first, end - first - 1, token, bad);
        if (lane == 0) {
            s.first = first;
            s.drafts = end - first - 1;
            s.accepted = n;
            s.refused = token;
            s.sample = sample;
            s.last = -1;
            if (bad && rank == 0) report(a.status, MSGL_DEVERR_TOKEN);
        }
    }
    __syncthreads();
    // What a request is about is looked up in shared memory where it is needed: kept in registers over the sums it was
    // spilled, and the spilled registers came back out of L2, 700 cycles each.
    auto row_of = [&](bool residual) {
        const int taken = s.accepted, row = s.first + taken;
        const bool refused = residual && taken < s.drafts;
        Row<T> r;
        r.set(static_cast<const T *>(a.target) + row * a.target_stride,
              refused && a.draft ? static_cast<const T *>(a.draft) + row * a.draft_stride : nullptr,
              refused && !a.draft ? s.refused : -1, a.vocab);
        return r;
    };
    auto length_of = [&](int vectors) { return ((vectors - 1) >> log2_runs) / 32 * 32 + 32; };   // whole rounds of a warp
    bool second = false;
    float w[kShortRun<T>][Vec<T>::kN];
    for (;; second = true) {
        const Row<T> r = row_of(!second);
        const int vectors = r.vectors(), length = length_of(vectors), mine = rank * kWarps + warp;
        const int n0 = (int)min((int64_t)mine * length, (int64_t)vectors), n1 = min(n0 + length, vectors);
        Sum sum;
        if constexpr (kShort) sum = run_sum(r, n0, n1, w);
        else sum = run_sum(r, n0, n1);
        // every block gets every run's sum
        if (!second) cluster_wait();
        if (lane < cluster)
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(peer_address(&s.runs[mine], lane)), "f"(sum.hi),
                         "f"(sum.lo)
                         : "memory");
        cluster_arrive();
        if (rank == 0 && !second) {
            // (written here, where the block waits anyway)
            const int first = s.first, taken = s.accepted, drafts = s.drafts;
            for (int i = threadIdx.x; i <= drafts; i += kThreads)
                if (i != taken) a.out_tokens[first + i] = i < taken ? __ldg(a.tokens + first + i + 1) : -1;
            if (threadIdx.x == kThreads - 1) {
                a.accepted[b] = taken;
                a.kv_lens[b] = (a.cached_lens ? __ldg(a.cached_lens + b) : 0) + taken + 1;
            }
        }
        cluster_wait();
        // every block goes through them in the same order and so comes to the same end: up to four neighbours a lane
        if (warp == 0) {
            const int log2_each = max(log2_runs - 5, 0), i0 = lane << log2_each;
            Sum x[4], sum{0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[k] = Sum{0.f, 0.f};
                if (k < 1 << log2_each && i0 + k < 1 << log2_runs) x[k] = s.runs[i0 + k];
                if (k < 1 << log2_each) sum = loose(sum, x[k]);
            }
            const Sum upto = warp_scan(sum), total = shfl(upto, 31), draw = times(s.sample, total);
            const int chosen = drawn_lane(sum, upto, draw);
            Sum lower = lane_before(upto);
            if (lane == max(chosen, 0)) {
                int run = -1;
                bool passed = false;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const Sum with = lower + x[k];
                    if (x[k].hi > 0 && !passed) {
                        run = i0 + k;
                        s.before = lower;
                        passed = with > draw;
                    }
                    lower = with;
                }
                s.draw = draw;
                s.run = run;
                s.bad = !(total.hi > 0 && total.hi <= 3.4e38f);
            }
        }
        __syncthreads();
        // nothing left over (p nowhere above q): the target's own row
        if (second || !s.bad || s.accepted == s.drafts) break;
        // (no block sums anew while another may still look at its sums)
        cluster_arrive();
        cluster_wait();
    }
    int32_t *out = a.out_tokens + s.first + s.accepted;
    if (s.bad) {
        if (rank == 0 && threadIdx.x == 0) {
            *out = -1;
            report(a.status, MSGL_DEVERR_PROBS);
        }
    } else if (s.run / kWarps == rank) {
        if (kShort && warp != s.run % kWarps) return;
        const Row<T> r = row_of(!second);
        const int vectors = r.vectors(), length = length_of(vectors), n0 = s.run * length;
        if constexpr (kShort) {
            draw_token(r, n0, w, s.before, s.draw, out);
            return;
        }
        const int i0 = max(r.token(n0), 0), i1 = min(r.token(min(n0 + length, vectors)), a.vocab);
        if (i1 - i0 <= kThreads) draw_token<1>(r, s, i0, i1, out);
        else if (i1 - i0 <= 2 * kThreads) draw_token<2>(r, s, i0, i1, out);
        else draw_token<8>(r, s, i0, i1, out);
    }
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs &a, cudaStream_t stream) {
    // As many blocks a request as all run at once, so that none begins its chain of lookups behind another's
    // row: two blocks an SM, in GPCs of 19 SMs on average, which hold 4 clusters of 8 blocks, 9 of 4 or 19 of 2;
    // and at least 2048 tokens a block.  131072 tokens, us with 1, 2, 4, 8 blocks: 16 requests 29.5, 17.4, 11.5, 9.4;
    // 37 (100003 tokens) 25.0, 15.8, 13.5, 13.7; 64 (bf16) 22.4, 13.7, 12.8, 15.3; 128 32.2, 24.6, 27.4, 32.5; 300
    // (32000 tokens) 16.2, 19.6, 27.9, 45.9.
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
    // (a row's shift may add a vector to it)
    const int64_t per = a.bf16 ? 8 : 4, most = a.bf16 ? kShortRun<__nv_bfloat16> : kShortRun<float>;
    const bool brief = (a.vocab + per - 1) / per + 1 <= (kWarps * 32 * most) << log2_cluster;
    auto kernel = a.bf16 ? (brief ? verify_kernel<__nv_bfloat16, true> : verify_kernel<__nv_bfloat16, false>)
                         : (brief ? verify_kernel<float, true> : verify_kernel<float, false>);
    return cudaLaunchKernelEx(&cfg, kernel, a, log2_cluster);
}

}  // namespace msgl
