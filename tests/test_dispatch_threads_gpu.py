"""moe_dispatch from several host threads at once, with geometries whose routing needs different amounts of
shared memory."""
import ctypes
import shutil
import subprocess

import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
from oracle import grouped as og
from test_grouped_gpu import BF, F32, I32, built, draw_ids  # noqa: F401

pytestmark = pytest.mark.gpu

THREADS = r"""
#include <pthread.h>
#include "moe.h"
typedef int (*dispatch_fn)(const moe_geom *, const void *, const void *, int, const float *, const int32_t *, void *, size_t,
                           moe_handle *, void *);
typedef struct { dispatch_fn f; moe_geom g; void *x, *ids, *w, *workspace; size_t bytes; moe_handle *h; void *stream;
                 int calls, refused, code; } job;
static void *run(void *p) {
    job *j = p;
    for (int i = 0; i < j->calls; ++i) {
        const int rc = j->f(&j->g, j->x, j->ids, MOE_IDS_INT64, j->w, NULL, j->workspace, j->bytes, j->h, j->stream);
        if (rc) { j->refused += 1; j->code = rc; }
    }
    return NULL;
}
int run_jobs(job *jobs, int n) {
    pthread_t t[8];
    int made = 0;
    while (made < n && made < 8 && !pthread_create(t + made, NULL, run, jobs + made)) ++made;
    for (int i = 0; i < made; ++i) pthread_join(t[i], NULL);
    return made;
}
"""


class Job(ctypes.Structure):
    _fields_ = ([("f", ctypes.c_void_p), ("g", moe.MoeGeom)] +
                [(n, ctypes.c_void_p) for n in ("x", "ids", "w", "workspace")] + [("bytes", ctypes.c_size_t)] +
                [(n, ctypes.c_void_p) for n in ("h", "stream")] + [(n, ctypes.c_int) for n in ("calls", "refused", "code")])


# experts and ranks: 65.6, 51.2 and 8 KB for the picks' places; 49.7 KB in one block, and under 48
@pytest.mark.parametrize("worlds", [((2048, 1), (1600, 1), (256, 1)), ((64, 64), (64, 32), (32, 4))])
def test_threads_with_different_geometries(tmp_path, worlds):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    (tmp_path / "threads.c").write_text(THREADS)
    subprocess.run([cc, "-O2", "-shared", "-fPIC", "-I", moe.__path__[0] + "/../include", str(tmp_path / "threads.c"), "-o",
                    str(tmp_path / "threads.so"), "-lpthread"], check=True)
    run_jobs = ctypes.CDLL(str(tmp_path / "threads.so")).run_jobs
    T, k, H = 64, 4, 128
    dispatch, held, jobs = ctypes.cast(moe.lib().moe_dispatch, ctypes.c_void_p).value, [], (Job * len(worlds))()
    for i, (E, W) in enumerate(worlds):
        layer = moe.MoELayer1GPU(W, T // W, T, H, E, k, 128, "FLAT", "HT")
        x, ids = torch.randn((T, H), device="cuda").to(BF), draw_ids(T, k, E, 0.1, i)
        t = [x, torch.tensor(ids).cuda(), torch.rand((T, k), device="cuda"), layer.workspace]
        held.append((layer, ids, t, torch.cuda.Stream()))
        jobs[i] = Job(dispatch, layer.geom, *[v.data_ptr() for v in t], layer.workspace.numel(), ctypes.addressof(layer.handle),
                      held[i][3].cuda_stream, 2000)
    torch.cuda.synchronize()
    assert run_jobs(jobs, len(worlds)) == len(worlds)
    torch.cuda.synchronize()
    assert [(j.refused, j.code) for j in jobs] == [(0, 0)] * len(worlds)
    for (E, W), (layer, ids, _, _) in zip(worlds, held):
        offsets, position, _ = og.order(ids, E)
        np.testing.assert_array_equal(layer.view("offsets", (E + 1,), I32).cpu().numpy(), offsets)
        np.testing.assert_array_equal(layer.view("pick_pos", (T, k), I32).cpu().numpy(), position)
        assert layer.status() == 0
