"""A decode step from a C program: tables, store, prefix groups and shared-prefix decode, with plain pointers.

The program gets the pool as it stood before the step's tokens, the tables as
they stood before its pages were handed out, and a list of free pages; Python
compares what it writes with the whole batch's fp64 reference.
"""
import os
import subprocess

import numpy as np
import pytest
import torch

from paged_kv_attention_24_gb300 import build as cuda_build
from tests import shared_batch
from tests.parity import assert_lse_close, assert_o_close
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
    int32_t hdr[8];
    float scale;
    if (fread(hdr, sizeof hdr, 1, f) != 1 || fread(&scale, sizeof scale, 1, f) != 1) return 4;
    const int32_t slots = hdr[0], ps = hdr[1], hkv = hdr[2], hq = hdr[3], B = hdr[4], W = hdr[5], nfree = hdr[6];
    const int32_t max_seq = hdr[7];
    const size_t row = (size_t)hkv * 256;
    void *k = to_device(f, slots * row), *v = to_device(f, slots * row);
    void *kn = to_device(f, B * row), *vn = to_device(f, B * row), *q = to_device(f, (size_t)B * hq * 256);
    int32_t *table = to_device(f, (size_t)B * W * 4), *cached = to_device(f, B * 4);
    int32_t *free_pages = to_device(f, nfree * 4);
    fclose(f);

    int32_t *ints;   /* every int32 output in one block */
    const size_t n = (size_t)B * W + 6 * B + 2;
    CK(cudaMalloc((void **)&ints, n * 4));
    CK(cudaMemset(ints, 0, n * 4));
    msgl_step_out out = {ints, W, W, ints + B * W, 0, 0, 0, 0, B};
    out.cu_ext = out.seq_lens + B;
    out.positions = out.cu_ext + B + 1;
    out.out_loc = out.positions + B;
    int32_t *first = out.out_loc + B, *shared = first + B;
    out.pages_taken = shared + B;
    void *o, *lse, *ws;
    uint32_t *status, flags = 0;
    CK(cudaMalloc(&o, (size_t)B * hq * 256));
    CK(cudaMalloc(&lse, (size_t)B * hq * 4));
    CK(cudaMalloc((void **)&status, 4));
    CK(cudaMemset(status, 0, 4));
    const size_t bytes = msgl_decode_shared_workspace_size(B, hq, hkv, 128, max_seq);
    CK(cudaMalloc(&ws, bytes));
    cudaStream_t st;
    CK(cudaStreamCreate(&st));

    msgl_kv_pool pool = {k, v, slots, ps, hkv, 128};
    msgl_page_table pages = {out.page_ids, W, W};
    MK(msgl_step_tables(slots, ps, table, B, W, W, NULL, cached, NULL, B, free_pages, nfree, &out, status, st));
    MK(msgl_store_kv(&pool, kn, vn, out.out_loc, B, status, st));
    MK(msgl_shared_prefixes(&pages, out.seq_lens, B, ps, max_seq, ps, first, shared, status, st));
    MK(msgl_attn_decode_shared(&pool, &pages, q, hq, first, shared, out.seq_lens, B, max_seq, MSGL_SHARE_AUTO, scale,
                               o, (float *)lse, ws, bytes, status, st));
    MK(msgl_read_status(status, &flags, st));
    FILE *w = fopen(argv[2], "wb");
    if (!w) return 1;
    if (fwrite(&flags, 4, 1, w) != 1 || put(w, ints, n * 4) || put(w, o, (size_t)B * hq * 256) ||
        put(w, lse, (size_t)B * hq * 4)) return 6;
    return fclose(w);
}
"""


@pytest.mark.parametrize("ps,groups", [(16, [(160, [1, 40, 17]), (0, [33]), (64, [5, 16, 1, 300])]),
                                       (1, [(90, [3, 1]), (700, [20, 21, 22])])])
def test_c_program_runs_a_decode_step(tmp_path, ps, groups):
    lib = cuda_build.build()
    b = shared_batch.make(40, 8, ps, groups, seed=70 + ps)
    ref_o, ref_l, ref_a = b.reference()
    B, W = b.table.shape
    cached = b.seq - 1
    table, k, v = b.table.clone(), b.k.clone(), b.v.clone()
    k_new, v_new, loc, fresh = [], [], [], []
    for i, at in enumerate(cached.tolist()):
        page = int(b.table[i, at // ps])
        loc.append(page * ps + at % ps)
        k_new.append(b.k[loc[-1]].clone()), v_new.append(b.v[loc[-1]].clone())
        k[loc[-1]] = v[loc[-1]] = float("nan")
        if at % ps == 0:
            fresh.append(page)
            table[i, at // ps] = -1
    taken = len(fresh)
    free = torch.tensor(fresh + [0, 0], dtype=torch.int32)
    src, exe, inp, outp = (tmp_path / n for n in ("step.c", "step", "in.bin", "out.bin"))
    src.write_text(PROGRAM)
    with open(inp, "wb") as f:
        f.write(np.array([k.shape[0], ps, 8, 40, B, W, len(free), b.max_seq], dtype=np.int32).tobytes())
        f.write(np.float32(b.scale).tobytes())
        for t in (k, v, torch.stack(k_new), torch.stack(v_new), b.q):
            f.write(_u16(t))
        for t in (table, cached, free):
            f.write(_i32(t))
    subprocess.run([_compiler(), "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src), lib,
                    "-Xlinker", f"-rpath={os.path.dirname(lib)}"], check=True)
    r = subprocess.run([str(exe), str(inp), str(outp)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    raw = np.fromfile(outp, dtype=np.int32)
    assert raw[0] == 0
    ids, raw = raw[1:1 + B * W].reshape(B, W), raw[1 + B * W:]
    seq, cu, pos, got_loc, first, shared = np.split(raw[:6 * B + 1], np.cumsum([B, B + 1, B, B, B]))
    for i in range(B):
        used = -(-int(b.seq[i]) // ps)
        assert ids[i, :used].tolist() == b.table[i, :used].tolist()
    assert seq.tolist() == b.seq.tolist() and cu.tolist() == list(range(B + 1)) and pos.tolist() == cached.tolist()
    assert got_loc.tolist() == loc and raw[6 * B + 1] == taken
    for i in range(B):   # whole shared pages are found; where the requests went on from there is their own
        if int(b.first[i]) != i:
            assert first[i] == b.first[i] and shared[i] >= int(b.shared[i]) // ps * ps
    rest = raw[6 * B + 2:].tobytes()
    o = torch.frombuffer(bytearray(rest[:B * 40 * 256]), dtype=torch.bfloat16).reshape(B, 40, 128)
    lse = torch.frombuffer(bytearray(rest[B * 40 * 256:]), dtype=torch.float32).reshape(B, 40)
    assert_o_close(o, ref_o, abs_ref=ref_a)
    assert_lse_close(lse, ref_l)
