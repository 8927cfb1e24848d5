// Shared-prefix decode of short requests: one launch, nothing to merge.
//
// Below a few hundred keys a decode is all latency, and the split kernel's scan
// over the batch, its partials and the merge behind it are most of it.  Here a
// block owns one request and 8 of the q heads of one kv head: its warps take
// the request's 16-key tiles in turn, each with its own running maximum and sum,
// and join through shared memory.  A block looks at its own request only.
//
// A key's page id is looked up by the lane that will load it (shared keys through
// the group's first request), its 256-byte K and V rows arrive by 16-byte
// cp.async at a pitch that keeps ldmatrix free of bank conflicts, two tiles in
// flight a warp; the products are the decode's (S^T = K Q^T with M = 16 keys and
// N = 8 q heads, O^T = V^T P^T).
//
// Bound by latency: lengths, page ids, keys, joins, each waiting for the one
// before.  4 requests of 145 to 200 keys (16 q heads over 8): 7.5 us, against 12
// to 14 for the split and its merge.
#include <math.h>

#include "kernels.h"
#include "ptx.cuh"

namespace msgl {

namespace {

constexpr int kTileKeys = 16;
constexpr int kPitch = 256 + 16;
constexpr int kTileBytes = 2 * kTileKeys * kPitch;   // K, then V
constexpr int kStages = 2;
constexpr int smem_bytes(int warps) { return warps * kStages * kTileBytes; }
static_assert(8 * kHeadDim * 4 <= kStages * kTileBytes, "a warp's sums fit where its tiles were");

struct ShortArgs {
    PoolView pool;
    PageView pages;
    GroupRows rows;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    float *lse;
    int32_t hq, group, slices;   // q heads; per kv head; blocks of 8 of those
    float scale_log2;
    uint32_t *status;
};

template <int kWarps>
__global__ void __launch_bounds__(32 * kWarps) decode_short_kernel(const ShortArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[kWarps][8], s_l[kWarps][8];
    __shared__ int s_bad;
    __shared__ uint32_t s_err;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y, g = blockIdx.x / a.slices, hoff = (blockIdx.x - g * a.slices) * 8;
    const int G = a.group, Gs = min(8, G - hoff);   // q heads of this block (slots past them are empty)
    int from;                                       // first key of the row's own pages
    const GroupRow row = group_row_at(a.rows, b);
    const int n = through_keys(a.rows, row, from), lead = row.lead;
    if (threadIdx.x == 0) s_bad = 0;

    // Q^T fragments: head slot lane / 4
    const int qh = lane >> 2;
    const __nv_bfloat16 *qp = a.q + ((long long)b * a.hq + (long long)g * G + hoff + qh) * kHeadDim + 2 * (lane & 3);
    uint32_t qf[8][2];
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        qf[ks][0] = qh < Gs ? *reinterpret_cast<const uint32_t *>(qp + 16 * ks) : 0u;
        qf[ks][1] = qh < Gs ? *reinterpret_cast<const uint32_t *>(qp + 16 * ks + 8) : 0u;
    }
    __syncthreads();

    const int tiles = (n + kTileKeys - 1) / kTileKeys;
    uint8_t *mine = smem + warp * kStages * kTileBytes;
    // loads tile i into the warp's stage; bit k of the result: key k is there
    auto load = [&](int i, int stage) -> uint32_t {
        const int key = i * kTileKeys + lane;
        long long slot = -1;
        bool bad = false;
        if (lane < kTileKeys && key < n) slot = slot_of(a.pool, a.pages, key < from ? lead : b, key, bad);
        if (bad) s_bad = 1;
        const uint32_t mask = __ballot_sync(0xffffffffu, slot >= 0);
        const uint32_t dst = ptx::smem_u32(mine + stage * kTileBytes);
        const int c = lane & 15;
#pragma unroll
        for (int x = 0; x < kTileKeys / 2; ++x) {
            const int r = 2 * x + (lane >> 4);
            const long long s = __shfl_sync(0xffffffffu, slot, r);
            const long long off = s >= 0 ? (s * a.pool.hkv + g) * kHeadDim + 8 * c : 0;
            const uint32_t bytes = s >= 0 ? 16u : 0u;   // (rows that are not there read as zeros)
            ptx::cp_async_16(dst + r * kPitch + 16 * c, a.pool.k + off, bytes);
            ptx::cp_async_16(dst + kTileKeys * kPitch + r * kPitch + 16 * c, a.pool.v + off, bytes);
        }
        return mask;
    };

    float acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    float m2[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    uint32_t masks[kStages] = {0u, 0u};
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
        if (warp + s * kWarps < tiles) masks[s] = load(warp + s * kWarps, s);
        ptx::cp_async_commit();
    }
    // (the group rules are looked up while the first tiles are on their way)
    if (threadIdx.x == 0) {
        int start, pair;
        s_err = group_row_errors(a.rows, row, start, pair);
    }
    const int krow = (lane & 7) + 8 * ((lane >> 3) & 1), kcol = 8 * (lane >> 4);
    const int vrow = (lane & 7) + 8 * (lane >> 4), vcol = 8 * ((lane >> 3) & 1);
    const int k0 = lane >> 2, k1 = k0 + 8;   // keys of this lane's S^T elements
    for (int i = warp, it = 0; i < tiles; i += kWarps, ++it) {
        const int stage = it & 1;
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        const uint32_t base = ptx::smem_u32(mine + stage * kTileBytes);
        const uint32_t mask = stage ? masks[1] : masks[0];
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            uint32_t kf[4];
            ptx::ldsm_x4(base + krow * kPitch + (16 * ks + kcol) * 2, kf[0], kf[1], kf[2], kf[3]);
            ptx::mma_bf16_16816(ks & 1 ? s2 : s, kf, qf[ks][0], qf[ks][1]);
        }
        const bool v0 = (mask >> k0) & 1u, v1 = (mask >> k1) & 1u;
        const float x00 = v0 ? (s[0] + s2[0]) * a.scale_log2 : -INFINITY;
        const float x01 = v0 ? (s[1] + s2[1]) * a.scale_log2 : -INFINITY;
        const float x10 = v1 ? (s[2] + s2[2]) * a.scale_log2 : -INFINITY;
        const float x11 = v1 ? (s[3] + s2[3]) * a.scale_log2 : -INFINITY;
        float mx0 = fmaxf(x00, x10), mx1 = fmaxf(x01, x11);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
        }
        const float mn0 = fmaxf(m2[0], mx0), mn1 = fmaxf(m2[1], mx1);
        const float al0 = mn0 == -INFINITY ? 1.f : ptx::ex2(m2[0] - mn0);
        const float al1 = mn1 == -INFINITY ? 1.f : ptx::ex2(m2[1] - mn1);
        const float p00 = x00 == -INFINITY ? 0.f : ptx::ex2(x00 - mn0);
        const float p01 = x01 == -INFINITY ? 0.f : ptx::ex2(x01 - mn1);
        const float p10 = x10 == -INFINITY ? 0.f : ptx::ex2(x10 - mn0);
        const float p11 = x11 == -INFINITY ? 0.f : ptx::ex2(x11 - mn1);
        m2[0] = mn0;
        m2[1] = mn1;
        l[0] = l[0] * al0 + p00 + p10;
        l[1] = l[1] * al1 + p01 + p11;
        // P is rounded to bf16 for the product (at most 2^-8 of each weight); the sums are not
        const uint32_t pb0 = ptx::movmatrix_t(ptx::pack_bf16(p00, p01));
        const uint32_t pb1 = ptx::movmatrix_t(ptx::pack_bf16(p10, p11));
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            uint32_t vf[4];
            ptx::ldsm_x4_t(base + (kTileKeys + vrow) * kPitch + (16 * d + vcol) * 2, vf[0], vf[1], vf[2], vf[3]);
            acc[d][0] *= al0;
            acc[d][1] *= al1;
            acc[d][2] *= al0;
            acc[d][3] *= al1;
            ptx::mma_bf16_16816(acc[d], vf, pb0, pb1);
        }
        __syncwarp();   // every lane has read the stage
        const int next = i + kStages * kWarps;
        if (next < tiles) {
            const uint32_t fresh = load(next, stage);
            if (stage) masks[1] = fresh;
            else masks[0] = fresh;
        }
        ptx::cp_async_commit();
    }
    ptx::cp_async_wait_all();
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
        l[1] += __shfl_xor_sync(0xffffffffu, l[1], o);
    }
    __syncthreads();   // the tiles' memory is free
    float *sums = reinterpret_cast<float *>(smem) + warp * 8 * kHeadDim;
    const int h0 = 2 * (lane & 3), h1 = h0 + 1;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
        const int d0 = 16 * d + (lane >> 2), d1 = d0 + 8;
        sums[h0 * kHeadDim + d0] = acc[d][0];
        sums[h0 * kHeadDim + d1] = acc[d][2];
        sums[h1 * kHeadDim + d0] = acc[d][1];
        sums[h1 * kHeadDim + d1] = acc[d][3];
    }
    if (lane < 4) {
        s_m[warp][h0] = m2[0];
        s_m[warp][h1] = m2[1];
        s_l[warp][h0] = l[0];
        s_l[warp][h1] = l[1];
    }
    __syncthreads();
    // warp w joins head slots w, w + kWarps, ...: each lane 4 of the 128 dims
    for (int h = warp; h < Gs; h += kWarps) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
        float L = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = s_m[w][h] == -INFINITY ? 0.f : ptx::ex2(s_m[w][h] - M);
            const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem) +
                                                               (w * 8 + h) * kHeadDim + 4 * lane);
            L += f * s_l[w][h];
            o0 += f * v.x;
            o1 += f * v.y;
            o2 += f * v.z;
            o3 += f * v.w;
        }
        const uint32_t err = s_err;
        const bool zero = err || s_bad || !(L > 0.f);
        const float inv = zero ? 0.f : 1.f / L;
        const long long row = (long long)b * a.hq + (long long)g * G + hoff + h;
        *reinterpret_cast<uint2 *>(a.o + row * kHeadDim + 4 * lane) =
            zero ? make_uint2(0u, 0u)
                 : make_uint2(ptx::pack_bf16(o0 * inv, o1 * inv), ptx::pack_bf16(o2 * inv, o3 * inv));
        if (lane == 0) {
            a.lse[row] = zero ? -INFINITY : (M + log2f(L)) * kLn2;
            if (h == 0 && (err || s_bad)) report(a.status, err ? err : MSGL_DEVERR_PAGE_RANGE);
        }
    }
}

template <int kWarps>
cudaError_t launch(const ShortArgs &a, cudaStream_t stream) {
    static bool attr_set[64];   // per device; idempotent, racing setters write the same value
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        cudaError_t e = cudaFuncSetAttribute(decode_short_kernel<kWarps>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             smem_bytes(kWarps));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    decode_short_kernel<kWarps><<<dim3(a.pool.hkv * a.slices, a.rows.num_reqs), 32 * kWarps, smem_bytes(kWarps),
                                  stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_short(const DecodeArgs &d, cudaStream_t stream) {
    ShortArgs a{};
    a.pool = d.pool;
    a.pages = d.pages;
    a.rows = GroupRows{d.seq_lens, d.group_start, d.shared_lens, d.num_reqs, d.max_seq_len, d.pair_rows};
    a.q = d.q;
    a.o = d.o;
    a.lse = d.lse;
    a.hq = d.hq;
    a.group = d.hq / d.pool.hkv;
    a.slices = (a.group + 7) / 8;
    a.scale_log2 = d.scale * kLog2e;
    a.status = d.status;
    // At most two tiles a warp, so that all of a request's keys are on their way at once, and no
    // more warps than that, so that more requests fit an SM: three blocks of 4 warps, one of 8.  When
    // there are more blocks than SMs, 4 warps also serve longer requests (512 keys, 32 requests of 8 kv
    // heads: 12.7 against 15.0 us; 8 requests: 9.2 against 8.2).
    const long long blocks = (long long)d.num_reqs * d.pool.hkv * a.slices;
    if (d.max_seq_len <= 2 * 2 * kTileKeys) return launch<2>(a, stream);
    if (d.max_seq_len <= 4 * 2 * kTileKeys || blocks > sm_count()) return launch<4>(a, stream);
    return launch<8>(a, stream);
}

}  // namespace msgl
