// Shared-prefix decode: one query row per request, groups of requests over one prefix.
#include <math.h>

#include "kernels.h"

namespace msgl {

namespace {

// One warp per (request, q head): keys below the shared length at the slots of the
// group's first row, the others at the row's own; running maximum and sum in fp32.
__global__ void __launch_bounds__(128) decode_shared_simple_kernel(const DecodeSharedArgs a) {
    const DecodeArgs &d = a.dec;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y, h = blockIdx.x * 4 + warp;
    if (h >= d.hq) return;
    const int g = h / (d.hq / d.pool.hkv);
    const int seq = __ldg(d.seq_lens + b), lead = __ldg(a.group_start + b);
    int shared = __ldg(a.shared_lens + b);
    const long long row = (long long)b * d.hq + h;
    uint32_t err = 0;
    if (seq < 1 || seq > d.max_seq_len) err |= MSGL_DEVERR_LENGTH;
    else if (lead != b ? (b == 0 || lead < 0 || lead > b || __ldg(a.group_start + b - 1) != lead ||
                          __ldg(a.group_start + lead) != lead || __ldg(a.shared_lens + lead) != shared ||
                          shared < 0 || shared > seq)
                       : (b + 1 < d.num_reqs && __ldg(a.group_start + b + 1) == b && (shared < 0 || shared > seq)))
        err |= MSGL_DEVERR_GROUP;
    const __nv_bfloat16 *qp = d.q + row * kHeadDim + lane * 4;
    const uint2 qv = *reinterpret_cast<const uint2 *>(qp);
    const float q0 = bf16_lo(qv.x), q1 = bf16_hi(qv.x), q2 = bf16_lo(qv.y), q3 = bf16_hi(qv.y);
    float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
    for (int j = 0; j < seq && !err; ++j) {
        bool bad = false;
        const long long slot = slot_of(d.pool, d.pages, j < shared ? lead : b, j, bad);
        if (bad) { err |= MSGL_DEVERR_PAGE_RANGE; break; }
        const long long at = (slot * d.pool.hkv + g) * kHeadDim + lane * 4;
        const uint2 kv = *reinterpret_cast<const uint2 *>(d.pool.k + at);
        const uint2 vv = *reinterpret_cast<const uint2 *>(d.pool.v + at);
        const float s = warp_sum(q0 * bf16_lo(kv.x) + q1 * bf16_hi(kv.x) + q2 * bf16_lo(kv.y) + q3 * bf16_hi(kv.y)) *
                        d.scale;
        const float mn = fmaxf(m, s), al = expf(m - mn), p = expf(s - mn);
        l = l * al + p;
        o0 = o0 * al + p * bf16_lo(vv.x);
        o1 = o1 * al + p * bf16_hi(vv.x);
        o2 = o2 * al + p * bf16_lo(vv.y);
        o3 = o3 * al + p * bf16_hi(vv.y);
        m = mn;
    }
    if (err && lane == 0) report(d.status, err);
    const float inv = err ? 0.f : 1.f / l;
    __nv_bfloat162 *op = reinterpret_cast<__nv_bfloat162 *>(d.o + row * kHeadDim + lane * 4);
    op[0] = err ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(o0 * inv, o1 * inv);
    op[1] = err ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(o2 * inv, o3 * inv);
    if (lane == 0) d.lse[row] = err ? -INFINITY : m + logf(l);
}

}  // namespace

size_t decode_shared_workspace_bytes(int32_t num_reqs, int32_t hq, int32_t hkv) {
    return plan_decode(num_reqs, hq, hkv, 1).workspace;
}

cudaError_t launch_decode_shared(const DecodeSharedArgs &a, cudaStream_t stream) {
    decode_shared_simple_kernel<<<dim3((a.dec.hq + 3) / 4, a.dec.num_reqs), 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace msgl
