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
// position; its upper 32 bits go through sincospif (an error of 2^-25 of the angle).
// Everything is in 32 bits up to the one rounding to bf16.
//
// Bound by HBM for many tokens, by latency for few.  One block per token: a thread's
// loads of its heads are issued first, the angles are computed once a token under
// them, and 8 lanes hold a head so that both halves of every pair are in one lane.
#include "kernels.h"

namespace msgl {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;                          // lanes of a head: two 16-byte chunks each
constexpr int kHeadsPerPass = kThreads / kLanes;
constexpr int kUnroll = 3;                         // passes whose loads are issued together

__device__ __forceinline__ void unpack8(const uint4 &r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(kThreads) rope_store_kernel(const __grid_constant__ RopeStoreArgs a) {
    __shared__ float cosines[kHeadDim / 2], sines[kHeadDim / 2];
    const int64_t t = blockIdx.x;
    const int64_t slot = __ldg(a.out_loc + t);
    if (slot == -1) return;                        // not a token: a bucket's padding
    const bool stored = slot >= 0 && slot < a.pool.num_slots;
    if (!stored && threadIdx.x == 0) report(a.status, MSGL_DEVERR_SLOT_RANGE);
    const int lane = threadIdx.x % kLanes, head0 = threadIdx.x / kLanes;
    // the lane's two chunks of 8 dims: a pair's halves where it turns, neighbours behind the turned dims
    const int turning = a.pairs / 8;
    const bool turns = lane < turning;
    const int c0 = turns ? lane : 2 * lane, c1 = turns ? lane + turning : 2 * lane + 1;
    const int hkv = a.pool.hkv, heads = a.hq + 2 * hkv;
    bool ready = false;
    for (int h0 = 0; h0 < heads; h0 += kHeadsPerPass * kUnroll) {
        uint4 r[kUnroll][2];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u * kHeadsPerPass + head0;
            if (h >= heads) continue;
            const __nv_bfloat16 *row = h < a.hq         ? a.q + t * a.q_stride + h * kHeadDim
                                       : h < a.hq + hkv ? a.k + t * a.k_stride + (h - a.hq) * kHeadDim
                                                        : a.v + t * a.v_stride + (h - a.hq - hkv) * kHeadDim;
            r[u][0] = *reinterpret_cast<const uint4 *>(row + 8 * c0);
            r[u][1] = *reinterpret_cast<const uint4 *>(row + 8 * c1);
        }
        if (!ready) {
            if (threadIdx.x < a.pairs) {
                const int j = threadIdx.x, axis = a.axis_bits[j / 16] >> (2 * (j % 16)) & 3;
                const int64_t pos = __ldg(a.positions + axis * a.axis_stride + t);
                const uint64_t turn = a.turns[j] * (uint64_t)pos;
                float s, c;
                sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
                cosines[j] = c * a.factor;
                sines[j] = s * a.factor;
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u * kHeadsPerPass + head0;
            // (a head's 8 lanes go the same way, but the shuffles below take the whole warp)
            const bool is_q = h < a.hq, is_k = !is_q && h < a.hq + hkv, live = h < heads;
            float x[8], y[8];
            unpack8(r[u][0], x);
            unpack8(r[u][1], y);
            const __nv_bfloat16 *weight = is_q ? a.q_norm : is_k ? a.k_norm : nullptr;
            if (a.q_norm || a.k_norm) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += x[i] * x[i] + y[i] * y[i];
#pragma unroll
                for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (live && weight) {
                    const float scale = 1.f / sqrtf(sum * (1.f / kHeadDim) + a.eps);
                    float wx[8], wy[8];
                    unpack8(__ldg(reinterpret_cast<const uint4 *>(weight) + c0), wx);
                    unpack8(__ldg(reinterpret_cast<const uint4 *>(weight) + c1), wy);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] *= scale * wx[i];
                        y[i] *= scale * wy[i];
                    }
                }
            }
            if (!live) continue;
            if (is_q || is_k) {
                if (turns && !a.adjacent) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float c = cosines[8 * c0 + i], s = sines[8 * c0 + i];
                        const float p = x[i] * c - y[i] * s, q = y[i] * c + x[i] * s;
                        x[i] = p;
                        y[i] = q;
                    }
                } else if (turns) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float cx = cosines[4 * c0 + i / 2], sx = sines[4 * c0 + i / 2];
                        const float cy = cosines[4 * c1 + i / 2], sy = sines[4 * c1 + i / 2];
                        const float p = x[i] * cx - x[i + 1] * sx, q = x[i + 1] * cx + x[i] * sx;
                        const float v = y[i] * cy - y[i + 1] * sy, w = y[i + 1] * cy + y[i] * sy;
                        x[i] = p;
                        x[i + 1] = q;
                        y[i] = v;
                        y[i + 1] = w;
                    }
                }
                r[u][0] = pack8(x);
                r[u][1] = pack8(y);
            }
            if (!is_q && !stored) continue;
            __nv_bfloat16 *row = is_q   ? a.q_out + t * a.out_stride + h * kHeadDim
                                 : is_k ? a.k_pool + (slot * hkv + h - a.hq) * kHeadDim
                                        : a.v_pool + (slot * hkv + h - a.hq - hkv) * kHeadDim;
            *reinterpret_cast<uint4 *>(row + 8 * c0) = r[u][0];
            *reinterpret_cast<uint4 *>(row + 8 * c1) = r[u][1];
        }
    }
}

}  // namespace

cudaError_t launch_rope_store(const RopeStoreArgs &a, cudaStream_t stream) {
    rope_store_kernel<<<a.n_tokens, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace msgl
