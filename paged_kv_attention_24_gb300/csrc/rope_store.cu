// Rotary positions and the store step in one pass over the new tokens.
//
// "不懂SGLang？从miniSGLang开始", §1.3 items 1 and 3: the positions of the new tokens
// are an input of the forward, and the new K/V rows become part of the pool.  The
// rotation stands between the projection and the store, so that a pass of its
// own would read and write q and k once more.
//
// A head's pairs (x_j, y_j) turn by angle_j = pos[axis_j] * f_j:
//   x' = x cos - y sin,  y' = y cos + x sin   (times `factor`),
// after an optional norm of the head, x * w / sqrt(mean(x^2) + eps).  The frequency
// comes as a 64-bit fraction of a whole turn, so that the product with an integer
// position modulo 2^64 is the angle modulo a turn with nothing lost, however far the
// position; rounded to 32 bits (by 2^-24 of the angle at most, so that the slow pairs'
// small angles keep their digits) it goes through sincospif.
// Everything is in 32 bits up to the one rounding to bf16.
//
// Bound by HBM for many tokens, by latency for few.  A warp takes a token, or a part
// of its heads where tokens are few, 4 heads a turn: 8 lanes hold a head, so that
// both halves of every pair are in one lane, and a lane's part of the rotation
// (the weights of the norm multiplied in) stays in its registers from head to head.
// Heads come 5 turns ahead by cp.async into the lane's own places in shared memory, so
// that no thread waits for another.  8256 tokens of 64/8 heads, normed: 54.7 us (6.2 TB/s of
// the 338 MB; ncu: DRAM 68% busy, 28% of the warps), 4 tokens of 16/8 heads 2.3 us.  Slower:
// angles shared by a block through shared memory, cosines, sines and weights read
// again for every head (370 instructions a turn in place of 200: 70 us); heads ahead in
// registers, 2 to 5 turns (66 to 72 us); 4 turns ahead, or 24 or 28 warps an SM (56 to 59).  Blocks
// of 128 threads and 6 turns ahead: 54.7 too, 64 tokens 3.2 in place of 3.0, 8192 of 8/8 heads 20.0
// in place of 19.2.
#include "kernels.h"

namespace msgl {

namespace {

constexpr int kThreads = 64, kWarps = kThreads / 32;
constexpr int kLanes = 8;                          // lanes of a head: two 16-byte chunks each
constexpr int kHeads = 32 / kLanes;                // heads of a warp's turn
constexpr int kAhead = 5;                          // turns whose heads are on their way
constexpr int kBlocks = 10;                         // blocks an SM

// Two floats, for the instructions that take both at once.
struct Two {
    uint64_t v;
    __device__ __forceinline__ float lo() const { return __uint_as_float((uint32_t)v); }
    __device__ __forceinline__ float hi() const { return __uint_as_float((uint32_t)(v >> 32)); }
};
__device__ __forceinline__ Two two(uint32_t lo, uint32_t hi) { return Two{(uint64_t)hi << 32 | lo}; }
__device__ __forceinline__ Two two(float lo, float hi) { return two(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ Two swapped(Two a) { return Two{a.v << 32 | a.v >> 32}; }
__device__ __forceinline__ Two operator*(Two a, Two b) {
    Two d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}

// 8 bf16 as four pairs of floats, and back.
__device__ __forceinline__ void unpack8(const uint4 &r, Two (&x)[4]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = two(w[i] << 16, w[i] & 0xffff0000u);
}
__device__ __forceinline__ uint4 pack8(const Two (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[i].hi()), "f"(x[i].lo()));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes into the lane's own place in shared memory, past L1 (not the read-only path: q may be turned in place).
// behind: what was read from that place before, so that the copy is not issued until it has arrived.
__device__ __forceinline__ void copy16(void *to, const void *from, uint32_t behind) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
                 "r"(behind)
                 : "memory");
}
__device__ __forceinline__ void end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_group() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// What a lane does to its chunks x and y: x' = x * a + other(x) * b, y' = y * c + other(y) * d, where the
// other of x is y (and of y x), or, for adjacent pairs, the chunk with its neighbours exchanged.
struct Rotation {
    Two a[4], b[4], c[4], d[4];
};

// kind: 0 for q, 1 for k.
template <bool kAdjacent>
__device__ __forceinline__ void rotation_of(const RopeStoreArgs &args, int kind, const float *cosines, const float *sines,
                                            int c0, int c1, bool turns, Rotation &r) {
    const __nv_bfloat16 *weight = kind == 0 ? args.q_norm : args.k_norm;
    Two wx[4], wy[4];
    if (weight) {
        unpack8(__ldg(reinterpret_cast<const uint4 *>(weight) + c0), wx);
        unpack8(__ldg(reinterpret_cast<const uint4 *>(weight) + c1), wy);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) wx[i] = wy[i] = two(1.f, 1.f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (!turns) {
            r.a[i] = wx[i];
            r.c[i] = wy[i];
            r.b[i] = r.d[i] = two(0.f, 0.f);
        } else if (kAdjacent) {
            const float cx = cosines[4 * c0 + i], sx = sines[4 * c0 + i], cy = cosines[4 * c1 + i], sy = sines[4 * c1 + i];
            r.a[i] = wx[i] * two(cx, cx);
            r.b[i] = swapped(wx[i]) * two(-sx, sx);
            r.c[i] = wy[i] * two(cy, cy);
            r.d[i] = swapped(wy[i]) * two(-sy, sy);
        } else {
            const float2 co = *reinterpret_cast<const float2 *>(cosines + 8 * c0 + 2 * i);
            const float2 si = *reinterpret_cast<const float2 *>(sines + 8 * c0 + 2 * i);
            r.a[i] = wx[i] * two(co.x, co.y);
            r.b[i] = wy[i] * two(-si.x, -si.y);
            r.c[i] = wy[i] * two(co.x, co.y);
            r.d[i] = wx[i] * two(si.x, si.y);
        }
    }
}

template <bool kAdjacent, bool kNorm>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_store_kernel(const __grid_constant__ RopeStoreArgs a, int parts) {
    __shared__ __align__(16) float angles[kWarps][2][kHeadDim / 2];
    __shared__ uint4 places[kWarps][kAhead][2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x % kLanes, head0 = (threadIdx.x & 31) / kLanes;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + warp, t = unit / parts;
    if (t >= a.n_tokens) return;
    const int part = (int)(unit - t * parts);
    // the lane's two chunks of 8 dims: a pair's halves where it turns, neighbours behind the turned dims
    const int turning = a.pairs / 8;
    const bool turns = lane < turning;
    const int c0 = turns ? lane : 2 * lane, c1 = turns ? lane + turning : 2 * lane + 1;
    const int hkv = a.pool.hkv, heads = a.hq + 2 * hkv;
    const __nv_bfloat16 *q = a.q + t * a.q_stride, *k = a.k + t * a.k_stride - a.hq * kHeadDim,
                        *v = a.v + t * a.v_stride - (a.hq + hkv) * kHeadDim;
    const int64_t slot = __ldg(a.out_loc + t);
    const int step = parts * kHeads;
    uint4 (*place)[2][32] = places[warp];
    // (read before the slot is known, whatever that says: one wait less)
    auto load = [&](int h, int at, uint32_t behind0, uint32_t behind1) {
        if (h < heads) {
            const __nv_bfloat16 *row = (h < a.hq ? q : h < a.hq + hkv ? k : v) + h * kHeadDim;
            copy16(&place[at][0][threadIdx.x & 31], row + 8 * c0, behind0);
            copy16(&place[at][1][threadIdx.x & 31], row + 8 * c1, behind1);
        }
        end_group();
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(part * kHeads + head0 + u * step, u, 0, 0);
    // the token's angles, two a lane
    float *cosines = angles[warp][0], *sines = angles[warp][1];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = threadIdx.x % 32 + 32 * i;
        if (j >= a.pairs) break;
        // (all four words are there for every lane: an index of its own would be read lane by lane)
        const uint32_t bits = j % 32 < 16 ? a.axis_bits[2 * i] : a.axis_bits[2 * i + 1];
        const int axis = bits >> (2 * (j % 16)) & 3;
        const int64_t pos = __ldg(a.positions + axis * a.axis_stride + t);
        const int64_t turn = (int64_t)(__ldg(a.turns + j) * (uint64_t)pos);
        float s, c;
        sincospif((float)turn * 0x1p-63f, &s, &c);
        cosines[j] = c * a.factor;
        sines[j] = s * a.factor;
    }
    if (slot == -1) {
        wait_group<0>();
        return;                                    // not a token: a bucket's padding
    }
    if (part == 0 && threadIdx.x % 32 == 0 && (slot < 0 || slot >= a.pool.num_slots))
        report(a.status, MSGL_DEVERR_SLOT_RANGE);
    __syncwarp();
    Rotation rotation;
    int kind = -1;
    int at = 0;
    for (int h = part * kHeads + head0; h - head0 < heads; h += step) {
            const bool live = h < heads, is_q = h < a.hq, is_k = !is_q && h < a.hq + hkv;
            wait_group<kAhead - 1>();
            uint4 r0 = place[at][0][threadIdx.x & 31], r1 = place[at][1][threadIdx.x & 31];
            load(h + step * kAhead, at, r0.x, r1.x);
            at = at + 1 == kAhead ? 0 : at + 1;
            if (h - head0 < a.hq + hkv) {          // (else the whole turn is v's, or behind it)
                const int now = is_q || !kNorm ? 0 : 1;
                if (now != kind) {
                    rotation_of<kAdjacent>(a, now, cosines, sines, c0, c1, turns, rotation);
                    kind = now;
                }
                Two x[4], y[4];
                unpack8(r0, x);
                unpack8(r1, y);
                float scale = 1.f;
                if (kNorm) {
                    Two sum = two(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum = fma2(y[i], y[i], fma2(x[i], x[i], sum));
                    float all = sum.lo() + sum.hi();
#pragma unroll
                    for (int o = 1; o < kLanes; o <<= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
                    // (rsqrtf is off by two units of the last place at most; a root and a division: 55.3 us)
                    if (is_q ? a.q_norm : a.k_norm) scale = rsqrtf(all * (1.f / kHeadDim) + a.eps);
                }
                if (is_q || is_k) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const Two xo = kAdjacent ? swapped(x[i]) : y[i], yo = kAdjacent ? swapped(y[i]) : x[i];
                        Two p = x[i] * rotation.a[i], q = y[i] * rotation.c[i];
                        if (turns) {               // (what does not turn takes nothing of the other chunk, infinities neither)
                            p = fma2(xo, rotation.b[i], p);
                            q = fma2(yo, rotation.d[i], q);
                        }
                        x[i] = kNorm ? p * two(scale, scale) : p;
                        y[i] = kNorm ? q * two(scale, scale) : q;
                    }
                    r0 = pack8(x);
                    r1 = pack8(y);
                }
            }
            if (live && (is_q || (slot >= 0 && slot < a.pool.num_slots))) {
                __nv_bfloat16 *row = is_q   ? a.q_out + t * a.out_stride + h * kHeadDim
                                     : is_k ? a.k_pool + (slot * hkv + h - a.hq) * kHeadDim
                                            : a.v_pool + (slot * hkv + h - a.hq - hkv) * kHeadDim;
                *reinterpret_cast<uint4 *>(row + 8 * c0) = r0;
                *reinterpret_cast<uint4 *>(row + 8 * c1) = r1;
            }
    }
    wait_group<0>();
}

}  // namespace

cudaError_t launch_rope_store(const RopeStoreArgs &a, cudaStream_t stream) {
    const int turns = (a.hq + 2 * a.pool.hkv + kHeads - 1) / kHeads;
    // As many warps as the GPU holds at once (10 blocks of 2 an SM): a token's heads in parts where tokens are
    // few, whole tokens where they are enough (64/8 heads, us with 1, 2, 4, 10, 20 parts: 64 tokens 11.0, 6.9, 5.2,
    // 4.1, 3.3; 256 tokens 11.4, 7.2, 5.7, 4.7, 6.0; 4096 tokens 33.7, 34.1, 39.6, 49.9, 71).
    const int64_t fit = (int64_t)sm_count() * kBlocks * kWarps / a.n_tokens;
    const int parts = (int)(fit < 1 ? 1 : fit < turns ? fit : turns);
    const unsigned blocks = (unsigned)(((int64_t)a.n_tokens * parts + kWarps - 1) / kWarps);
    auto kernel = a.q_norm || a.k_norm ? (a.adjacent ? rope_store_kernel<true, true> : rope_store_kernel<false, true>)
                                       : (a.adjacent ? rope_store_kernel<true, false> : rope_store_kernel<false, false>);
    kernel<<<blocks, kThreads, 0, stream>>>(a, parts);
    return cudaGetLastError();
}

}  // namespace msgl
