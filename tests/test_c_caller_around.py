"""The calls around a step from a C program, with plain pointers and row pitches beyond the width: free pages, forks and
their page copies, the rotary store, the verification of drafts, a compaction and its copies."""
import os
import subprocess

import numpy as np
import pytest
import torch

from paged_kv_attention_24_gb300 import build as cuda_build
from paged_kv_attention_24_gb300 import ops
from tests import step_reference as ref
from tests.step_reference import assert_rounded, rope_rows
from tests.test_c_caller import ROOT, _compiler, _i32, _u16

pytestmark = pytest.mark.gpu

PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include <stdint.h>
#include <cuda_runtime.h>
#include "msgl_attn.h"

#define CK(x) do { cudaError_t e_ = (x); if (e_ != cudaSuccess) { \
    fprintf(stderr, "%s: %s\n", #x, cudaGetErrorString(e_)); return 2; } } while (0)
#define MK(x) do { msgl_status s_ = (x); if (s_ != MSGL_OK) { \
    fprintf(stderr, "%s: %s (%s)\n", #x, msgl_status_string(s_), msgl_last_error()); return 3; } } while (0)

static void *to_device(FILE *f, size_t n) {
    void *h = malloc(n ? n : 1), *d = NULL;
    if (n && fread(h, 1, n, f) != n) { fprintf(stderr, "short read\n"); exit(4); }
    if (cudaMalloc(&d, n ? n : 16) != cudaSuccess) exit(5);
    if (n && cudaMemcpy(d, h, n, cudaMemcpyHostToDevice) != cudaSuccess) exit(5);
    free(h);
    return d;
}

static void *filled(size_t n, int byte) {
    void *d = NULL;
    if (cudaMalloc(&d, n) != cudaSuccess || cudaMemset(d, byte, n) != cudaSuccess) exit(5);
    return d;
}

static int put(FILE *o, const void *d, size_t n) {
    void *h = malloc(n);
    int bad = cudaMemcpy(h, d, n, cudaMemcpyDeviceToHost) != cudaSuccess || fwrite(h, 1, n, o) != n;
    free(h);
    return bad;
}

int main(int argc, char **argv) {
    if (argc != 3) return 1;
    FILE *f = fopen(argv[1], "rb");
    if (!f) return 1;
    int32_t hdr[11];
    if (fread(hdr, sizeof hdr, 1, f) != 1) return 4;
    const int32_t slots = hdr[0], ps = hdr[1], hkv = hdr[2], hq = hdr[3], rows = hdr[4], width = hdr[5], stride = hdr[6];
    const int32_t B = hdr[7], N = hdr[8], T = hdr[9], V = hdr[10], np = slots / ps, heads = hq + 2 * hkv;
    const size_t pool_bytes = (size_t)slots * hkv * 256;
    uint8_t axes[64];
    if (fread(axes, 1, 64, f) != 64) return 4;
    void *k[2], *v[2];
    for (int i = 0; i < 2; ++i) {
        k[i] = to_device(f, pool_bytes);
        v[i] = to_device(f, pool_bytes);
    }
    char *qkv = to_device(f, (size_t)T * heads * 256);
    uint64_t *turns = to_device(f, 64 * 8);
    int32_t *pos = to_device(f, (size_t)3 * (T + 2) * 4), *loc = to_device(f, T * 4);
    int32_t *table = to_device(f, (size_t)rows * stride * 4), *req_rows = to_device(f, B * 4), *lens = to_device(f, B * 4);
    uint8_t *held = to_device(f, np);
    int32_t *parents = to_device(f, N * 4), *children = to_device(f, N * 4), *flens = to_device(f, N * 4);
    int32_t *all_rows = to_device(f, (B + N) * 4), *all_lens = to_device(f, (B + N) * 4);
    float *p = to_device(f, (size_t)T * (V + 3) * 4), *d = to_device(f, (size_t)T * V * 4);
    int32_t *tokens = to_device(f, T * 4), *cu = to_device(f, (B + 1) * 4);
    float *au = to_device(f, T * 4), *su = to_device(f, B * 4);
    fclose(f);

    int32_t *free_ids = filled((size_t)np * 4, 0), *num_free = filled(4, 0);
    msgl_fork_out forked = {filled(N * 4, 0), filled(N * 4, 0), filled(N * 4, 0), filled(4, 0)};
    void *turned = filled((size_t)T * (hq + 1) * 256, 0x11);
    int32_t *accepted = filled(B * 4, 0), *out_tokens = filled(T * 4, 0xff), *kv_lens = filled(B * 4, 0);
    msgl_compact_out com = {filled((size_t)rows * (width + 1) * 4, 0xff), width + 1, filled((size_t)np * 4, 0),
                            filled((size_t)np / 2 * 4, 0), filled((size_t)np / 2 * 4, 0), filled(4, 0), filled(4, 0)};
    uint32_t *status = filled(4, 0), flags = 0;
    const size_t bytes = msgl_page_map_workspace_size(slots, ps);
    void *ws = filled(bytes, 0x5a);
    cudaStream_t st;
    CK(cudaStreamCreate(&st));
    CK(cudaDeviceSynchronize());

    const msgl_kv_pool pools[2] = {{k[0], v[0], slots, ps, hkv, 128}, {k[1], v[1], slots, ps, hkv, 128}};
    MK(msgl_free_pages(slots, ps, table, rows, stride, width, req_rows, lens, B, held, free_ids, num_free, ws, bytes, status, st));
    MK(msgl_fork_requests(slots, ps, table, rows, stride, width, parents, children, flens, N, free_ids, np, &forked, status, st));
    MK(msgl_copy_pages(pools, 2, forked.copy_src, forked.copy_dst, forked.copy_tokens, N, NULL, status, st));
    const msgl_rope rope = {turns, axes, 64, 3, 1, 0.5f};
    const msgl_new_tokens tok = {qkv, qkv + (size_t)hq * 256, qkv + (size_t)(hq + hkv) * 256, turned, (int64_t)heads * 128,
                                 (int64_t)heads * 128, (int64_t)heads * 128, (int64_t)(hq + 1) * 128, pos, T + 2, loc, T, hq};
    MK(msgl_rope_store_kv(&pools[1], &tok, &rope, NULL, NULL, 0.f, status, st));
    const msgl_draft_batch batch = {p, d, V + 3, V, V, 0, tokens, cu, au, su, lens, B, T, accepted, out_tokens, kv_lens};
    MK(msgl_verify_drafts(&batch, status, st));
    MK(msgl_compact_pages(slots, ps, table, rows, stride, width, all_rows, all_lens, B + N, held, &com, ws, bytes, status, st));
    MK(msgl_copy_pages(pools, 2, com.src, com.dst, NULL, np / 2, com.num_moves, status, st));
    MK(msgl_read_status(status, &flags, st));
    FILE *w = fopen(argv[2], "wb");
    if (!w) return 1;
    if (fwrite(&flags, 4, 1, w) != 1 || put(w, free_ids, (size_t)np * 4) || put(w, num_free, 4) || put(w, forked.copy_src, N * 4) ||
        put(w, forked.copy_dst, N * 4) || put(w, forked.copy_tokens, N * 4) || put(w, forked.pages_taken, 4) ||
        put(w, table, (size_t)rows * stride * 4) || put(w, accepted, B * 4) || put(w, out_tokens, T * 4) || put(w, kv_lens, B * 4) ||
        put(w, com.page_ids, (size_t)rows * (width + 1) * 4) || put(w, com.remap, (size_t)np * 4) ||
        put(w, com.src, (size_t)np / 2 * 4) || put(w, com.dst, (size_t)np / 2 * 4) || put(w, com.num_moves, 4) ||
        put(w, com.num_used, 4) || put(w, turned, (size_t)T * (hq + 1) * 256))
        return 6;
    for (int i = 0; i < 2; ++i)
        if (put(w, k[i], pool_bytes) || put(w, v[i], pool_bytes)) return 6;
    return fclose(w);
}
"""


def test_c_program_runs_the_calls_around_a_step(tmp_path):
    lib = cuda_build.build()
    rng, g = np.random.default_rng(5), torch.Generator().manual_seed(5)
    ps, hkv, hq, np_, rows, width, stride, B, N, T, V = 8, 4, 8, 91, 12, 6, 9, 4, 5, 11, 333
    slots = np_ * ps
    normal = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    pools = [[normal(slots, hkv, 128) for _ in range(2)] for _ in range(2)]
    qkv = normal(T, hq + 2 * hkv, 128)
    axes = [j % 3 for j in range(64)]
    freq = [1e4 ** (-j / 64) for j in range(64)]
    pos = rng.integers(0, 900, (3, T + 2)).astype(np.int32)
    order = rng.permutation(np_).astype(np.int32)
    table = rng.integers(0, np_, (rows, stride)).astype(np.int32)
    where = rng.permutation(rows)
    lens = np.array([48, 1, 29, 16], np.int32)
    table[where[:B], :width] = order[:B * width].reshape(B, width)
    held = np.zeros(np_, np.uint8)
    held[order[B * width:B * width + 20]] = 7
    free_slots = [int(x) for x in order[-3:]]                     # (the last free pages are not handed out: see below)
    loc = np.array([free_slots[t // 5] * ps + t % 5 for t in range(T)], np.int32)
    loc[7] = -1
    parents, children = where[[0, 2, 2, 3, 1]].astype(np.int32), where[B:B + N].astype(np.int32)
    flens = np.array([48, 29, 13, 16, 0], np.int32)
    cu = np.array([0, 3, 4, 8, 11], np.int32)
    z = 3 * torch.randn(T, V, generator=g)
    p, d = torch.softmax(z, -1), torch.softmax(z + 0.3 * torch.randn(T, V, generator=g), -1)
    drawn = torch.multinomial(d, 1, generator=g)[:, 0].int()
    tokens = torch.cat([drawn[:1], drawn[:-1]])
    au, su = torch.rand(T, generator=g), torch.rand(B, generator=g)
    wide = torch.full((T, V + 3), float("nan"))
    wide[:, :V] = p
    src, exe, inp, outp = (tmp_path / n for n in ("around.c", "around", "in.bin", "out.bin"))
    src.write_text(PROGRAM)
    i32 = lambda x: np.ascontiguousarray(x, dtype=np.int32).tobytes()
    all_rows, all_lens = np.concatenate([where[:B], children]), np.concatenate([lens, flens])
    with open(inp, "wb") as f:
        f.write(i32([slots, ps, hkv, hq, rows, width, stride, B, N, T, V]) + bytes(axes))
        for t in (*pools[0], *pools[1], qkv):
            f.write(_u16(t))
        f.write(ops.Rope(freq, axes, device="cpu").turns.numpy().tobytes())
        for x in (pos, loc, table, where[:B], lens):
            f.write(i32(x))
        f.write(held.tobytes())
        for x in (parents, children, flens, all_rows, all_lens):
            f.write(i32(x))
        f.write(wide.numpy().tobytes() + d.numpy().tobytes())
        f.write(_i32(tokens) + i32(cu) + au.numpy().tobytes() + su.numpy().tobytes())
    subprocess.run([_compiler(), "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src), lib,
                    "-Xlinker", f"-rpath={os.path.dirname(lib)}"], check=True)
    r = subprocess.run([str(exe), str(inp), str(outp)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    raw = open(outp, "rb").read()
    at = 0

    def take(n, *shape):
        nonlocal at
        x = np.frombuffer(raw, np.int32, n, at).reshape(shape or (n,))
        at += 4 * n
        return x
    assert take(1)[0] == 0
    used = ref.held_by(table[:, :width], where[:B], lens, np_, ps) | (held != 0)
    free = np.nonzero(~used)[0].tolist()
    assert take(np_).tolist() == free + [-1] * (np_ - len(free)) and take(1)[0] == len(free)
    want, s, n, m, taken = ref.fork(table[:, :width], parents.tolist(), children.tolist(), flens.tolist(), free, np_, ps)
    assert (take(N).tolist(), take(N).tolist(), take(N).tolist(), take(1)[0]) == (s, n, m, taken)
    after = take(rows * stride, rows, stride)
    assert np.array_equal(after[:, :width], want) and np.array_equal(after[:, width:], table[:, width:])
    ver = ref.verify(p, d, tokens.tolist(), cu.tolist(), au.tolist(), su.tolist(), lens.tolist(), [-1] * T)
    for x, k in zip(ver, (B, T, B)):
        assert take(k).tolist() == x.tolist()
    blank = np.full((rows, width), -1, np.int32)
    c = ref.compact(want, all_rows.tolist(), all_lens.tolist(), held, np_, ps, into=blank)
    ids = take(rows * (width + 1), rows, width + 1)
    assert np.array_equal(ids[:, :width], c[0]) and (ids[:, width] == -1).all()
    assert take(np_).tolist() == c[1].tolist() and take(np_ // 2).tolist() == c[2] and take(np_ // 2).tolist() == c[3]
    assert (take(1)[0], take(1)[0]) == (c[4], c[5]) and c[4] > 0
    bf = lambda n, *shape: torch.frombuffer(bytearray(raw[at:at + 2 * n]), dtype=torch.bfloat16).reshape(shape)
    turned = bf(T * (hq + 1) * 128, T, hq + 1, 128)
    at += T * (hq + 1) * 256
    live = [t for t in range(T) if loc[t] >= 0]
    args = (pos[:, :T][:, live].tolist(), freq, axes, True, 0.5, None, 0)
    assert_rounded(turned[live][:, :hq], *rope_rows(qkv[live][:, :hq], *args))
    assert (turned[:, hq].view(torch.int16) == 0x1111).all() and (turned[7].view(torch.int16) == 0x1111).all()
    # the pools: the forks' copies, the tokens' K and V in the second layer, the compaction's copies
    for i, (k0, v0) in enumerate(pools):
        got = []
        for _ in range(2):
            got.append(bf(slots * hkv * 128, slots, hkv, 128))
            at += slots * hkv * 256
        for x, is_k in zip((k0, v0), (True, False)):
            x = x.clone()
            stored = torch.zeros(slots, dtype=torch.bool)
            for a, b, k in zip(s, n, m):
                if a >= 0:
                    x[b * ps:b * ps + k] = x[a * ps:a * ps + k]
            if i == 1:
                x[loc[live]] = got[0 if is_k else 1][loc[live]]
                stored[loc[live]] = True
            for a, b in zip(c[2][:c[4]], c[3][:c[4]]):
                x[b * ps:(b + 1) * ps] = x[a * ps:(a + 1) * ps]
            assert torch.equal(got[0 if is_k else 1].view(torch.int16), x.view(torch.int16)), (i, is_k)
        if i == 1:
            slots_of = [int(x) for x in loc[live]]
            assert_rounded(got[0][slots_of], *rope_rows(qkv[live][:, hq:hq + hkv], *args))
            assert torch.equal(got[1][slots_of], qkv[live][:, hq + hkv:])
    assert at == len(raw)
