"""The operators around the expert layer: what they refuse, on the host, before anything is
queued (the C codes and the binding's exceptions); the binding's structs against the header."""
import ctypes
import os

import pytest
import torch

import combine_topk_ids_gb300 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(1 << 20)          # never dereferenced: every call here fails before a launch
ODD = ctypes.c_void_p((1 << 20) + 1)
OFF8 = ctypes.c_void_p((1 << 20) + 8)
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        moe.build()
    return moe.lib()


def norm(**kw):
    n = moe.MoeNorm(4, 256, 0, 0, 1e-6)
    for k, v in kw.items():
        setattr(n, k, v)
    return n


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), -1), (dict(hidden=0), -1), (dict(residual_dtype=2), -1), (dict(weight_dtype=-1), -1),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(x_stride=255), -1), (dict(out_stride=-256), -1),
    (dict(hidden=65537), -13)])
def test_norm_rules(lib, kw, code):
    n = norm(**kw)
    assert lib.moe_add_rmsnorm(n, P, P, P, P, P, None, None, None, None) == code
    assert lib.moe_add_rmsnorm_backward(n, P, P, P, P, P, P, P, P, 1 << 40, None) == code
    size = ctypes.c_size_t()
    assert lib.moe_add_rmsnorm_workspace_size(n, ctypes.byref(size)) == code


def test_norm_pointers(lib):
    f = lib.moe_add_rmsnorm
    n = norm()
    assert f(None, P, P, P, P, P, P, P, P, None) == -1
    assert f(n, None, P, P, P, P, P, P, P, None) == -1
    assert f(n, P, P, None, P, P, P, P, P, None) == -1
    assert f(n, P, P, P, P, None, None, None, P, None) == -1       # no output
    assert f(n, P, P, P, P, None, P, None, P, None) == -1          # codes without scales
    assert f(n, P, P, P, P, P, None, P, P, None) == -1             # scales without codes
    assert f(norm(hidden=200), P, P, P, P, None, P, P, P, None) == -3
    for i in range(1, 9):
        args = [P] * 8
        args[i - 1] = ODD
        assert f(n, *args, None) == -9, i
    assert f(n, P, P, P, P, P, OFF8, P, P, None) == -9
    b = lib.moe_add_rmsnorm_backward
    assert b(n, P, P, P, P, P, P, P, P, 16, None) == -8
    assert b(n, P, P, P, P, None, P, None, P, 1 << 40, None) == -1
    assert b(n, P, P, P, P, P, P, P, None, 1 << 40, None) == -1
    assert b(n, P, None, P, P, P, P, P, P, 1 << 40, None) == -1
    assert b(n, P, P, P, P, P, P, P, OFF8, 1 << 40, None) == -9


def router(**kw):
    r = moe.make_router(64, 4, "sigmoid", 8, 2, "top2")
    for k, v in kw.items():
        setattr(r, k, v)
    return r


@pytest.mark.parametrize("kw,code", [
    (dict(num_experts=0), -1), (dict(groups=0), -1), (dict(groups=7), -1), (dict(top_groups=0), -1),
    (dict(top_groups=9), -1), (dict(score=2), -1), (dict(group_score=-1), -1), (dict(logits_dtype=3), -1),
    (dict(logits_stride=63), -1), (dict(num_experts=2056), -13), (dict(groups=64), -13), (dict(top_k=0), -6),
    (dict(top_k=17), -6), (dict(top_k=33, top_groups=8), -6)])
def test_router_rules(lib, kw, code):
    assert lib.moe_route_topk(router(**kw), 4, P, P, P, 1, P, None) == code
    assert lib.moe_route_topk_backward(router(**kw), 4, P, P, 1, P, P, None) == code


def test_router_pointers(lib):
    f, b, r = lib.moe_route_topk, lib.moe_route_topk_backward, router()
    assert f(r, -1, P, P, P, 1, P, None) == -1
    assert f(r, 4, None, P, P, 1, P, None) == -1 and f(r, 4, P, P, None, 1, P, None) == -1
    assert f(r, 4, P, P, P, 1, None, None) == -1 and f(r, 4, P, P, P, 2, P, None) == -7
    assert f(r, 4, ODD, P, P, 1, P, None) == -9 and f(r, 4, P, ODD, P, 1, P, None) == -9
    assert f(r, 4, P, P, ctypes.c_void_p((1 << 20) + 4), 1, P, None) == -9
    assert b(r, 4, P, P, 1, P, None, None) == -1 and b(r, 4, P, P, 1, P, ODD, None) == -9
    assert b(r, 4, P, P, 5, P, P, None) == -7 and b(r, 4, P, P, 1, None, P, None) == -1


def w4(**kw):
    g = moe.make_w4_geom(4, 256, 8, 2, 512, 64)
    for k, v in kw.items():
        setattr(g, k, v)
    return g


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), -1), (dict(group=16), -1), (dict(group=96), -1), (dict(num_experts=0), -1),
    (dict(top_k=0), -6), (dict(top_k=33), -6), (dict(hidden=192), -3), (dict(intermediate=64), -4),
    (dict(num_experts=2049), -13), (dict(hidden=65664), -13), (dict(num_tokens=1 << 30), -13)])
def test_w4_rules(lib, kw, code):
    g, size = w4(**kw), ctypes.c_size_t()
    assert lib.moe_forward_w4_workspace_size(g, ctypes.byref(size)) == code
    assert lib.moe_forward_w4(g, P, P, 1, P, P, P, P, P, P, P, P, 1 << 60, None) == code
    assert lib.moe_prepare_weights_w4(g, *[P] * 8, None) == code


def test_w4_pointers(lib):
    f, g = lib.moe_forward_w4, w4()
    assert f(g, P, P, 3, P, P, P, P, P, P, P, P, 1 << 60, None) == -7
    assert f(g, P, P, 1, P, P, P, P, P, P, P, P, 16, None) == -8
    for i in range(10):     # every array is needed, and none may lie anywhere
        args = [P] * 10
        args[i] = None
        assert f(g, *args[:2], 1, *args[2:], 1 << 60, None) == -1, i
        args[i] = ODD
        assert f(g, *args[:2], 1, *args[2:], 1 << 60, None) == -9, i
    q = [ctypes.c_void_p((1 << 20) * (i + 1)) for i in range(8)]
    assert lib.moe_prepare_weights_w4(g, *q[:4], q[0], *q[5:], None) == -1      # in place
    assert lib.moe_prepare_weights_w4(g, *q[:7], ODD, None) == -9
    assert lib.moe_prepare_weights_w4(g, *q[:7], None, None) == -1
    z = lib.moe_quantize_w4
    assert z(4, 96, 64, P, P, P, None) == -1 and z(4, 64, 48, P, P, P, None) == -1 and z(-1, 64, 64, P, P, P, None) == -1
    assert z(1 << 60, 64, 64, P, P, P, None) == -1 and z(4, 64, 64, None, P, P, None) == -1
    assert z(4, 64, 64, ODD, P, P, None) == -9 and z(1 << 45, 64, 64, P, P, P, None) == -13


def test_structs_match_the_header(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    classes = {"moe_norm": moe.MoeNorm, "moe_router": moe.MoeRouter, "moe_w4_geom": moe.MoeW4Geom}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "moe_block.h"', "int main(void) {"]
    for st, cls in classes.items():
        lines.append('printf("%s sizeof %%zu\\n", sizeof(%s));' % (st, st))
        lines += ['printf("%s %s %%zu\\n", offsetof(%s, %s));' % (st, n, st, n) for n, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        st, n, v = line.split()
        cls = classes[st]
        assert int(v) == (ctypes.sizeof(cls) if n == "sizeof" else getattr(cls, n).offset), line


# ---- the binding ---------------------------------------------------------------------------------

def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("kw,err", [
    (dict(x=z(4, 256, dtype=F32)), TypeError), (dict(x=z(256)), ValueError), (dict(x=[1.0]), TypeError),
    (dict(residual=z(4, 256, dtype=torch.float16)), TypeError), (dict(residual=z(5, 256)), ValueError),
    (dict(sum_out=z(4, 256, dtype=F32)), TypeError),                 # not the residual's type
    (dict(weight=z(255)), ValueError), (dict(weight=None), ValueError), (dict(out=z(256, 4).t()), ValueError),
    (dict(out=z(1, 256).expand(4, 256)), ValueError), (dict(out=None), ValueError),
    (dict(out_fp8=z(4, 256, dtype=torch.uint8)), ValueError),        # codes without scales
    (dict(scales=z(4, 2, dtype=F32)), ValueError),
    (dict(out_fp8=z(4, 256, dtype=torch.uint8), scales=z(2, 4, dtype=F32)), ValueError),
    (dict(rstd=z(4)), TypeError), (dict(rstd=z(8, dtype=F32)[::2]), ValueError)])
def test_norm_binding(lib, kw, err):
    args = dict(x=z(4, 256), residual=z(4, 256), weight=z(256), eps=1e-6, out=z(4, 256))
    args.update(kw)
    with pytest.raises(err):
        moe.moe_add_rmsnorm(**args)


def test_norm_backward_binding(lib):
    good = dict(dout=z(4, 256), h=z(4, 256), weight=z(256), rstd=z(4, dtype=F32), dx=z(4, 256),
                dweight=z(256, dtype=F32), workspace=z(64, dtype=torch.uint8))
    for kw, err in ((dict(dout=z(4, 256, dtype=F32)), TypeError), (dict(h=z(4, 128)), ValueError),
                    (dict(dx=z(4, 256, dtype=F32)), TypeError), (dict(dsum=z(4, 256, dtype=F32)), TypeError),
                    (dict(dweight=z(256)), TypeError), (dict(rstd=None), ValueError), (dict(dx=None), ValueError),
                    (dict(workspace=z(64)), TypeError)):
        with pytest.raises(err):
            moe.moe_add_rmsnorm_backward(**{**good, **kw})


def test_router_binding(lib):
    r = moe.make_router(64, 4)
    good = dict(logits=z(3, 64), bias=None, topk_ids=z(3, 4, dtype=torch.int64), topk_weights=z(3, 4, dtype=F32))
    for kw, err in ((dict(logits=z(3, 63)), ValueError), (dict(logits=z(3, 64, dtype=torch.float64)), TypeError),
                    (dict(logits=z(64, 3).t()), ValueError), (dict(bias=z(64)), TypeError),
                    (dict(topk_ids=z(3, 4, dtype=torch.int16)), TypeError), (dict(topk_ids=None), ValueError),
                    (dict(topk_weights=z(3, 5, dtype=F32)), ValueError)):
        with pytest.raises(err):
            moe.moe_route_topk(r, **{**good, **kw})
    with pytest.raises(TypeError):
        moe.moe_route_topk_backward(r, z(3, 64), good["topk_ids"], good["topk_weights"], z(3, 64, dtype=F32))
    for kw in (dict(score="relu"), dict(group_score="sum")):
        with pytest.raises(KeyError):
            moe.make_router(64, 4, **kw)


def test_w4_binding(lib):
    layer = moe.MoELayerW4(4, 256, 8, 2, 512, 64, device="cpu")
    x, ids, w = z(4, 256), z(4, 2, dtype=torch.int64), z(4, 2, dtype=F32)
    with pytest.raises(RuntimeError, match="set_weights"):
        layer.forward(x, ids, w)
    w1, s1, w2, s2 = z(8, 1024, 128, dtype=torch.uint8), z(8, 1024, 4), z(8, 256, 256, dtype=torch.uint8), z(8, 256, 8)
    for bad in ((w1[:4], s1, w2, s2), (w1, s1.float(), w2, s2), (w1, s1, w2.to(torch.int8), s2), (w1, s1, w2, None)):
        with pytest.raises((TypeError, ValueError)):
            layer.set_weights(*bad)
    layer.weights = []      # past the check: the tensors are looked at next
    for args in ((z(5, 256), z(5, 2, dtype=torch.int64), z(5, 2, dtype=F32)), (x.float(), ids, w), (x, ids.short(), w),
                 (x, ids, w.double()), (x, ids[:, :1], w), (x, None, w), (z(256), ids, w)):
        with pytest.raises((TypeError, ValueError)):
            layer.forward(*args)
    for g in (dict(group=48), dict(hidden=200)):
        with pytest.raises(moe.MoeError):
            moe.MoELayerW4(**{**dict(max_tokens=4, hidden=256, num_experts=8, top_k=2, intermediate=512, device="cpu"), **g})
    with pytest.raises(ValueError):
        moe.moe_quantize_w4(z(4, 96), 64, z(4, 48, dtype=torch.uint8), z(4, 1))
    with pytest.raises(TypeError):
        moe.moe_quantize_w4(z(4, 128, dtype=F32), 64, z(4, 64, dtype=torch.uint8), z(4, 2))
