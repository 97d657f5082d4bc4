"""moe_sort_picks from two host threads at once, and its workspace of exactly the size asked for."""
import ctypes
import shutil
import subprocess

import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
from oracle import grouped as og
from test_grouped_gpu import I32, built, draw_ids  # noqa: F401

pytestmark = pytest.mark.gpu

# Host threads in C, so that no lock of the interpreter parts their calls.
THREADS = r"""
#include <pthread.h>
#include "moe_grouped.h"
typedef int (*sort_fn)(const moe_sort *, const void *, int, int32_t *, int32_t *, int32_t *, int32_t *, void *, size_t, void *);
typedef struct { sort_fn f; moe_sort g; void *ids, *offsets, *position, *workspace; size_t bytes; void *stream; int calls, refused, code; } job;
static void *run(void *p) {
    job *j = p;
    for (int i = 0; i < j->calls; ++i) {
        const int rc = j->f(&j->g, j->ids, MOE_IDS_INT64, j->offsets, j->position, NULL, NULL, j->workspace, j->bytes, j->stream);
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
    _fields_ = ([("f", ctypes.c_void_p), ("g", moe.MoeSort)] +
                [(n, ctypes.c_void_p) for n in ("ids", "offsets", "position", "workspace")] +
                [("bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p)] +
                [(n, ctypes.c_int) for n in ("calls", "refused", "code")])


def test_threads_with_different_expert_counts(tmp_path):
    """Each thread's calls need another amount of shared memory (80, 51 and 27 KB) and have a stream, a workspace and
    outputs of their own: none is refused, and all are right."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    (tmp_path / "threads.c").write_text(THREADS)
    subprocess.run([cc, "-O2", "-shared", "-fPIC", "-I", moe.__path__[0] + "/../include", str(tmp_path / "threads.c"), "-o",
                    str(tmp_path / "threads.so"), "-lpthread"], check=True)
    run_jobs = ctypes.CDLL(str(tmp_path / "threads.so")).run_jobs
    T, k, experts = 600, 8, (2048, 1300, 700)
    sort, held, jobs = ctypes.cast(moe.lib().moe_sort_picks, ctypes.c_void_p).value, [], (Job * len(experts))()
    for i, E in enumerate(experts):
        t = [torch.tensor(draw_ids(T, k, E, 0.1, i)).cuda(), torch.empty(E + 1, dtype=I32, device="cuda"),
             torch.empty((T, k), dtype=I32, device="cuda"),
             torch.empty(moe.moe_sort_picks_workspace_size(T, k, E), dtype=torch.uint8, device="cuda"), torch.cuda.Stream()]
        held.append(t)
        jobs[i] = Job(sort, moe.MoeSort(T, E, k), *[v.data_ptr() for v in t[:4]], t[3].numel(), t[4].cuda_stream, 2000)
    torch.cuda.synchronize()
    assert run_jobs(jobs, len(experts)) == len(experts)
    torch.cuda.synchronize()
    assert [(j.refused, j.code) for j in jobs] == [(0, 0)] * len(experts)
    for E, (ids, offsets, position, _, _) in zip(experts, held):
        want = og.order(ids.cpu().numpy(), E)
        np.testing.assert_array_equal(offsets.cpu().numpy(), want[0])
        np.testing.assert_array_equal(position.cpu().numpy(), want[1])
