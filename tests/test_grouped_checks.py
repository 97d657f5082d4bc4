"""The operators on expert-grouped rows: what they refuse, on the host, before anything is queued
(the C codes and the binding's exceptions); the binding's structs against the header; their oracle."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
from oracle import grouped as og

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(1 << 20)          # never dereferenced: every call here fails before a launch
ODD = ctypes.c_void_p((1 << 20) + 1)
OFF8 = ctypes.c_void_p((1 << 20) + 8)
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        moe.build()
    return moe.lib()


def changed(s, kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), -1), (dict(num_experts=0), -1), (dict(top_k=0), -6), (dict(top_k=33), -6),
    (dict(num_experts=2049), -13), (dict(num_tokens=1 << 30), -13)])
def test_sort_rules(lib, kw, code):
    g = changed(moe.MoeSort(64, 256, 8), kw)
    size = ctypes.c_size_t()
    assert lib.moe_sort_picks_workspace_size(g, ctypes.byref(size)) == code
    assert lib.moe_sort_picks(g, P, 1, P, P, P, P, P, 1 << 40, None) == code


def test_sort_pointers(lib):
    g = moe.MoeSort(64, 256, 8)
    f = lib.moe_sort_picks
    assert f(None, P, 1, P, P, P, P, P, 1 << 40, None) == -1
    for missing in (0, 1, 2, 5):      # ids, offsets, position, workspace
        args = [P] * 6
        args[missing] = None
        assert f(g, args[0], 1, *args[1:], 1 << 40, None) == -1, missing
    for odd in range(6):
        args = [P] * 6
        args[odd] = ODD
        assert f(g, args[0], 1, *args[1:], 1 << 40, None) == -9, odd
    assert f(g, P, 2, P, P, P, P, P, 1 << 40, None) == -7
    assert f(g, P, 1, P, P, P, P, P, 16, None) == -8
    assert f(g, P, 1, P, P, P, P, OFF8, 1 << 40, None) == -9


@pytest.mark.parametrize("T,k,E", [(0, 1, 1), (1, 8, 256), (512, 8, 64), (513, 8, 64), (32768, 8, 256),
                                   (32768, 8, 2048), ((1 << 31) // 8 - 128, 8, 2048)])
def test_sort_workspace(lib, T, k, E):
    """The counts of all blocks, at most 152 * 256 of them, and a word for each block."""
    n = moe.moe_sort_picks_workspace_size(T, k, E)
    assert 4 * (E + 1) <= n <= 4 * (152 * 256 + 152 + 4) or T * k <= 4096 and n <= 4 * (E + 1) + 16


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), -1), (dict(num_rows=-1), -1), (dict(hidden=0), -1), (dict(rows_dtype=4), -1),
    (dict(rows_stride=255), -1), (dict(tokens_stride=-256), -1), (dict(top_k=0), -6), (dict(top_k=33), -6),
    (dict(hidden=65537), -13)])
def test_rows_rules(lib, kw, code):
    g = changed(moe.MoeRows(4, 2, 256, 8, 0, 0), kw)
    assert lib.moe_sort_rows(g, P, None, P, P, None, None) == code
    assert lib.moe_sort_rows_backward(g, P, P, P, None) == code
    assert lib.moe_unsort_rows(g, P, P, P, P, None) == code
    assert lib.moe_unsort_rows_backward(g, P, P, P, P, P, P, None) == code


def test_rows_pointers(lib):
    g, q = moe.MoeRows(4, 2, 256, 8, 0, 0), moe.MoeRows(4, 2, 256, 8, 2, 0)
    s, u, b = lib.moe_sort_rows, lib.moe_unsort_rows, lib.moe_unsort_rows_backward
    assert s(None, P, None, P, P, None, None) == -1 and u(None, P, P, P, P, None) == -1
    assert lib.moe_sort_rows_backward(None, P, P, P, None) == -1 and b(None, P, P, P, P, P, P, None) == -1
    for args in ((None, None, P, P, None), (P, None, None, P, None), (P, None, P, None, None),
                 (P, P, P, P, None), (P, None, P, P, P)):            # bf16 rows have no scales
        assert s(g, *args, None) == -1
    for args in ((P, None, P, P, P), (P, P, P, P, None)):             # codes have
        assert s(q, *args, None) == -1
    assert s(changed(moe.MoeRows(4, 2, 200, 8, 2, 0), {}), P, P, P, P, P, None) == -3
    for kw in (dict(tokens_stride=512), dict(rows_stride=512)):       # and are packed
        assert s(changed(moe.MoeRows(4, 2, 256, 8, 2, 0), kw), P, P, P, P, P, None) == -1
    assert s(q, OFF8, P, P, P, P, None) == -9 and s(q, P, P, P, OFF8, P, None) == -9
    assert s(q, P, ODD, P, P, P, None) == -9 and s(q, P, P, P, P, ODD, None) == -9
    for odd in (0, 2, 3):
        args = [P, None, P, P, None]
        args[odd] = ODD
        assert s(g, *args, None) == -9, odd
    for missing in (0, 2, 3):
        args = [P] * 4
        args[missing] = None
        assert u(g, *args, None) == -1, missing
    for odd in range(4):
        args = [P] * 4
        args[odd] = ODD
        assert u(g, *args, None) == -9, odd
    assert u(moe.MoeRows(4, 2, 256, 8, 2, 0), P, P, P, P, None) == -1    # codes are not summed
    assert u(moe.MoeRows(4, 2, 256, 8, 0, 2), P, P, P, P, None) == -1
    assert lib.moe_sort_rows_backward(moe.MoeRows(4, 2, 256, 8, 2, 0), P, P, P, None) == -1
    assert b(g, None, P, P, P, P, P, None) == -1 and b(g, P, P, P, None, P, P, None) == -1
    assert b(g, P, None, P, P, P, P, None) == -1                      # dweights need rows
    assert b(g, P, P, P, P, None, None, None) == -1
    assert b(changed(moe.MoeRows(4, 2, 256, 8, 0, 0), dict(drows_stride=100)), P, P, P, P, P, P, None) == -1
    for odd in range(6):
        args = [P] * 6
        args[odd] = ODD
        assert b(g, *args, None) == -9, odd


@pytest.mark.parametrize("kw,code", [
    (dict(matrices=0), -1), (dict(num_rows=-1), -1), (dict(cols=0), -1), (dict(block_rows=64), -1),
    (dict(x_dtype=2), -1), (dict(x_stride=255), -1), (dict(cols=200), -3), (dict(cols=65536 + 128), -13)])
def test_quantize_rules(lib, kw, code):
    q = changed(moe.MoeQuantize(1, 4, 256, 1, 0, 0), kw)
    assert lib.moe_quantize_fp8(q, P, None, P, P, None) == code
    assert lib.moe_swiglu_fp8(q, P, None, P, P, None) == code


def test_quantize_pointers(lib):
    q = moe.MoeQuantize(1, 4, 256, 1, 0, 0)
    for f in (lib.moe_quantize_fp8, lib.moe_swiglu_fp8):
        assert f(None, P, None, P, P, None) == -1
        for missing in (0, 2, 3):
            args = [P] * 4
            args[missing] = None
            assert f(q, *args, None) == -1, missing
        for odd in range(4):
            args = [P] * 4
            args[odd] = ODD
            assert f(q, *args, None) == -9, odd
        assert f(q, P, None, OFF8, P, None) == -9
        assert f(moe.MoeQuantize(2, 4, 256, 1, 0, 0), P, P, P, P, None) == -1     # live rows of several matrices
    assert lib.moe_quantize_fp8(moe.MoeQuantize(1, 4, 256, 128, 0, 0), P, P, P, P, None) == -1
    assert lib.moe_swiglu_fp8(moe.MoeQuantize(1, 4, 256, 128, 0, 0), P, None, P, P, None) == -1
    assert lib.moe_swiglu_fp8(moe.MoeQuantize(1, 4, 256, 1, 0, 511), P, None, P, P, None) == -1   # two halves to a row


@pytest.mark.parametrize("kw,code", [
    (dict(num_rows=-1), -1), (dict(n=0), -1), (dict(k=0), -1), (dict(groups=-1), -1), (dict(out_dtype=2), -1),
    (dict(a_stride=240), -1), (dict(out_stride=255), -1), (dict(k=200), -3), (dict(k=65536 + 128), -13),
    (dict(n=65537), -13), (dict(groups=2049), -13), (dict(a_stride=264), -9), (dict(a_stride=1 << 40), -13)])
def test_product_rules(lib, kw, code):
    p = changed(moe.MoeProduct(4, 256, 256, 2, 0, 0, 0), kw)
    assert lib.moe_product_fp8(p, P, P, P, P, P, P, P, None) == code


def test_product_pointers(lib):
    f, p = lib.moe_product_fp8, moe.MoeProduct(4, 256, 256, 2, 0, 0, 0)
    assert f(None, P, P, P, P, P, P, P, None) == -1
    for missing in range(6):
        args = [P] * 6
        args[missing] = None
        assert f(p, *args, None, None) == -1, missing
    for odd in range(7):
        args = [P] * 7
        args[odd] = ODD
        assert f(p, *args, None) == -9, odd
    assert f(p, OFF8, P, P, P, P, P, P, None) == -9 and f(p, P, P, OFF8, P, P, P, P, None) == -9
    assert f(moe.MoeProduct(4, 256, 256, 0, 0, 0, 0), P, P, P, P, P, P, P, None) == -1    # offsets without groups


def test_structs_match_the_header(tmp_path):
    """Sizes and field offsets of the binding's structs are those that a C compiler gives the header's."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"moe_sort": moe.MoeSort, "moe_rows": moe.MoeRows, "moe_quantize": moe.MoeQuantize,
               "moe_product": moe.MoeProduct}
    lines = []
    for name, cls in structs.items():
        lines.append('printf("%%zu\\n", sizeof(%s));' % name)
        lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (name, f[0]) for f in cls._fields_]
    src = tmp_path / "s.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"moe_grouped.h\"\nint main(void) {\n%s\nreturn 0; }"
                   % "\n".join(lines))
    subprocess.run([cc, str(src), "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "s")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True).stdout.split()]
    want = []
    for cls in structs.values():
        want += [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]
    assert got == want


# ---- the binding ---------------------------------------------------------------------------------

def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def refused(call, good, cases):
    for kw, err in cases:
        with pytest.raises(err):
            call(**{**good, **kw})
    with pytest.raises(ValueError, match="host memory"):     # nothing else is wrong with `good`
        call(**good)


def test_sort_picks_binding(lib):
    good = dict(topk_ids=z(3, 4, dtype=torch.int64), num_experts=8, offsets=z(9, dtype=I32), position=z(3, 4, dtype=I32),
                workspace=z(64, dtype=U8), source=z(12, dtype=I32), status=z(1, dtype=I32))
    refused(moe.moe_sort_picks, good, [
        (dict(topk_ids=z(3, 4, dtype=torch.int16)), TypeError), (dict(topk_ids=z(12, dtype=I32)), ValueError),
        (dict(topk_ids=z(4, 3, dtype=I32).t()), ValueError), (dict(offsets=z(8, dtype=I32)), ValueError),
        (dict(offsets=None), ValueError), (dict(position=z(3, 4, dtype=torch.int64)), TypeError),
        (dict(position=None), ValueError), (dict(workspace=z(64)), TypeError), (dict(workspace=None), ValueError),
        (dict(source=z(11, dtype=I32)), ValueError), (dict(status=z(2, dtype=I32)), ValueError)])
    with pytest.raises(moe.MoeError):
        moe.moe_sort_picks_workspace_size(4, 33, 8)


def test_rows_binding(lib):
    pos, w = z(3, 2, dtype=I32), z(3, 2, dtype=F32)
    good = dict(x=z(3, 256), position=pos, rows=z(6, 256))
    refused(moe.moe_sort_rows, good, [
        (dict(x=z(3, 256, dtype=torch.float16)), TypeError), (dict(rows=z(6, 256, dtype=F32)), TypeError),
        (dict(rows=z(6, 255)), ValueError), (dict(rows=None), ValueError), (dict(position=z(2, 3, dtype=I32)), ValueError),
        (dict(position=z(3, 2, dtype=torch.int64)), TypeError), (dict(rows_scales=z(6, 2, dtype=F32)), ValueError),
        (dict(x=z(3, 256, dtype=U8), rows=z(6, 256, dtype=U8)), ValueError),
        (dict(rows=z(1, 256).expand(6, 256)), ValueError)])
    codes = dict(x=z(3, 256, dtype=U8), position=pos, rows=z(6, 256, dtype=torch.float8_e4m3fn),
                 x_scales=z(3, 2, dtype=F32), rows_scales=z(6, 2, dtype=F32))
    refused(moe.moe_sort_rows, codes, [(dict(x_scales=z(2, 3, dtype=F32)), ValueError), (dict(rows_scales=None), ValueError),
                                       (dict(x=z(3, 512, dtype=U8)[:, :256]), ValueError), (dict(rows=z(6, 256)), TypeError)])
    refused(moe.moe_sort_rows_backward, dict(drows=z(6, 256), position=pos, dx=z(3, 256)),
            [(dict(dx=z(3, 256, dtype=F32)), TypeError), (dict(dx=None), ValueError), (dict(drows=z(6, 256, dtype=U8)), TypeError),
             (dict(dx=z(4, 256)), ValueError)])
    refused(moe.moe_unsort_rows, dict(rows=z(6, 256), weights=w, position=pos, out=z(3, 256, dtype=F32)),
            [(dict(weights=z(3, 2)), TypeError), (dict(weights=z(3, 3, dtype=F32)), ValueError), (dict(out=None), ValueError),
             (dict(out=z(3, 128)), ValueError), (dict(rows=z(6, 256, dtype=U8)), TypeError)])
    back = dict(dout=z(3, 256), rows=z(6, 256, dtype=F32), weights=w, position=pos, drows=z(6, 256, dtype=F32), dweights=w)
    refused(moe.moe_unsort_rows_backward, back,
            [(dict(drows=z(6, 256)), TypeError), (dict(rows=None), ValueError), (dict(drows=None, dweights=None), ValueError),
             (dict(dweights=z(3, 2)), TypeError), (dict(dout=z(3, 200)), ValueError), (dict(drows=z(5, 256, dtype=F32)), ValueError)])


def test_quantize_binding(lib):
    good = dict(x=z(4, 256), codes=z(4, 256, dtype=U8), scales=z(4, 2, dtype=F32))
    refused(moe.moe_quantize_fp8, good, [
        (dict(x=z(4, 256, dtype=torch.float16)), TypeError), (dict(x=z(256)), ValueError), (dict(block_rows=32), ValueError),
        (dict(codes=z(4, 256)), TypeError), (dict(codes=None), ValueError), (dict(scales=z(4, 1, dtype=F32)), ValueError),
        (dict(scales=z(4, 2, dtype=F32), block_rows=128), ValueError), (dict(live_rows=z(2, dtype=I32)), ValueError),
        (dict(x=z(2, 4, 512)[:, :, :256], codes=z(2, 4, 256, dtype=U8), scales=z(2, 4, 2, dtype=F32)), ValueError)])
    refused(moe.moe_swiglu_fp8, dict(gate_up=z(4, 512), codes=good["codes"], scales=good["scales"]),
            [(dict(gate_up=z(4, 511)), ValueError), (dict(gate_up=z(4, 256)), ValueError), (dict(scales=None), ValueError)])


def test_product_binding(lib):
    good = dict(a=z(4, 256, dtype=U8), a_scales=z(4, 2, dtype=F32), b=z(200, 256, dtype=U8), b_scales=z(2, 2, dtype=F32),
                out=z(4, 200))
    refused(moe.moe_product_fp8, good, [
        (dict(a=z(4, 256)), TypeError), (dict(a=z(256, 4, dtype=U8).t()), ValueError), (dict(b=z(200, 128, dtype=U8)), ValueError),
        (dict(b=z(1, 200, 256, dtype=U8)), ValueError), (dict(b_scales=z(1, 2, dtype=F32)), ValueError),
        (dict(a_scales=None), ValueError), (dict(b_scales=None), ValueError), (dict(out=None), ValueError),
        (dict(out=z(4, 201)), ValueError), (dict(out=z(4, 200, dtype=torch.float16)), TypeError),
        (dict(offsets=z(2, dtype=I32)), ValueError), (dict(status=z(1)), TypeError)])
    many = dict(good, b=z(3, 200, 256, dtype=U8), b_scales=z(3, 2, 2, dtype=F32), offsets=z(4, dtype=I32))
    refused(moe.moe_product_fp8, many, [(dict(offsets=z(3, dtype=I32)), ValueError), (dict(offsets=z(4, dtype=torch.int64)), TypeError),
                                        (dict(b=z(3, 400, 256, dtype=U8)[:, ::2]), ValueError),
                                        (dict(b=z(0, 200, 256, dtype=U8), b_scales=z(0, 2, 2, dtype=F32), offsets=z(1, dtype=I32)),
                                         ValueError)])


# ---- the oracle ----------------------------------------------------------------------------------

def test_oracle_order_by_hand():
    offsets, position, source = og.order(np.array([[2, 0], [-1, 2], [0, 0], [7, 2]]), 3)
    assert offsets.tolist() == [0, 3, 3, 6]
    assert position.tolist() == [[3, 0], [-1, 4], [1, 2], [-1, 5]]
    assert source.tolist() == [1, 4, 5, 0, 3, 7, -1, -1]


def test_oracle_gradients_by_differences():
    rng = np.random.default_rng(0)
    position = og.order(np.array([[1, 0, -1], [0, 1, 1]]), 2)[1]
    rows, w, dout = rng.normal(size=(6, 4)), rng.normal(size=(2, 3)), rng.normal(size=(2, 4))
    drows, dw, _ = og.unsort_rows_backward(dout, rows, w, position, np.zeros((6, 4)))
    loss = lambda r, v: (og.unsort_rows(r, v, position)[0] * dout).sum()  # noqa: E731
    for v, g in ((rows, drows), (w, dw)):
        for i in np.ndindex(v.shape):
            keep, d = v[i], []
            for h in (1e-3, -1e-3):
                v[i] = keep + h
                d.append(loss(rows, w))
            v[i] = keep
            np.testing.assert_allclose((d[0] - d[1]) / 2e-3, g[i], atol=1e-9)
