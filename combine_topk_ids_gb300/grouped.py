"""Python binding of the operators on expert-grouped rows (include/moe_grouped.h).

moe_sort_picks, moe_sort_rows and moe_unsort_rows with their gradients, moe_quantize_fp8,
moe_swiglu_fp8 and moe_product_fp8.  Argument checks and marshalling only; results go to the
caller's tensors, on the current stream or the one given.

Row matrices of bf16 and float32 may have any row stride, and the codes of a product's rows one
that is a multiple of 16; every other tensor is contiguous.  A tensor of another type raises
TypeError, one of another shape, layout or device ValueError, and what the library refuses MoeError.
"""
import ctypes

import torch

from .block import _BF16, _BYTE, _E4M3, _F32, _IDS, _P, _ROW, DTYPE, _call, _lib, _packed, _rows, _stream, _typed

_I32 = (torch.int32,)
_DTYPE = {**DTYPE, torch.float8_e4m3fn: 2, torch.uint8: 2}


class MoeSort(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_tokens", "num_experts", "top_k")]


class MoeRows(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("num_tokens", "top_k", "hidden", "num_rows", "rows_dtype",
                                               "tokens_dtype")] +
                [(n, ctypes.c_int64) for n in ("rows_stride", "drows_stride", "tokens_stride")])


class MoeQuantize(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("matrices", "num_rows", "cols", "block_rows", "x_dtype")] +
                [("x_stride", ctypes.c_int64)])


class MoeProduct(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("num_rows", "n", "k", "groups", "out_dtype")] +
                [(n, ctypes.c_int64) for n in ("a_stride", "out_stride")])


def bind(L):
    """Argument types of the library's entry points of this header."""
    S, R, Q, M = (ctypes.POINTER(t) for t in (MoeSort, MoeRows, MoeQuantize, MoeProduct))
    size, out = ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
    L.moe_sort_picks_workspace_size.argtypes = [S, out]
    L.moe_sort_picks.argtypes = [S, _P, ctypes.c_int] + [_P] * 5 + [size, _P]
    L.moe_sort_rows.argtypes = [R] + [_P] * 6
    L.moe_sort_rows_backward.argtypes = [R] + [_P] * 4
    L.moe_unsort_rows.argtypes = [R] + [_P] * 5
    L.moe_unsort_rows_backward.argtypes = [R] + [_P] * 7
    L.moe_quantize_fp8.argtypes = [Q] + [_P] * 5
    L.moe_swiglu_fp8.argtypes = [Q] + [_P] * 5
    L.moe_product_fp8.argtypes = [M] + [_P] * 8
    for f in ("moe_sort_picks_workspace_size", "moe_sort_picks", "moe_sort_rows", "moe_sort_rows_backward",
              "moe_unsort_rows", "moe_unsort_rows_backward", "moe_quantize_fp8", "moe_swiglu_fp8", "moe_product_fp8"):
        getattr(L, f).restype = ctypes.c_int


def _matrix(t, name, dtypes):
    """(rows, columns), device of a matrix."""
    _typed(t, name, dtypes)
    if t.dim() != 2:
        raise ValueError("%s: shape %s, expected a matrix" % (name, tuple(t.shape)))
    return t.shape, t.get_device()


def _needed(**tensors):
    missing = [n for n, t in tensors.items() if t is None]
    if missing:
        raise ValueError("%s must be given" % " and ".join(missing))


def moe_sort_picks_workspace_size(tokens, top_k, num_experts):
    """Bytes of the workspace of moe_sort_picks."""
    size = ctypes.c_size_t()
    _call(_lib().moe_sort_picks_workspace_size(MoeSort(tokens, num_experts, top_k), ctypes.byref(size)),
          "moe_sort_picks_workspace_size")
    return size.value


def moe_sort_picks(topk_ids, num_experts, offsets, position, workspace, source=None, status=None, stream=None):
    """The order of the picks topk_ids (int32 or int64 [T, k], -1: masked) by (expert, token, pick):
    offsets int32 [num_experts + 1], the first row of each expert; position int32 [T, k], each pick's
    row or -1; source int32 [T * k], the pick t * k + j of each row, -1 behind the last one; status
    int32 [1], MOE_STATUS_* bits (an id outside [-1, num_experts) is dropped).  workspace: uint8, of
    moe_sort_picks_workspace_size bytes."""
    _needed(offsets=offsets, position=position, workspace=workspace)
    shape, dev = _matrix(topk_ids, "topk_ids", _IDS)
    T, k = shape
    _typed(workspace, "workspace", _BYTE)
    pi = _packed(topk_ids, "topk_ids", _IDS, shape, dev)
    po = _packed(offsets, "offsets", _I32, (num_experts + 1,), dev)
    pp = _packed(position, "position", _I32, shape, dev)
    ps = _packed(source, "source", _I32, (T * k,), dev)
    pt = _packed(status, "status", _I32, (1,), dev)
    pw = _packed(workspace, "workspace", _BYTE, workspace.shape, dev)
    _call(_lib().moe_sort_picks(MoeSort(T, num_experts, k), pi, _IDS[topk_ids.dtype], po, pp, ps, pt, pw,
                                workspace.numel(), _stream(stream, dev)), "moe_sort_picks")


def _positions(position, T, dev):
    """The address of position [T, k], and k."""
    _typed(position, "position", _I32)
    if position.dim() != 2 or position.shape[0] != T:
        raise ValueError("position: shape %s, expected [%d, top_k]" % (tuple(position.shape), T))
    return _packed(position, "position", _I32, position.shape, dev), position.shape[1]


def moe_sort_rows(x, position, rows, x_scales=None, rows_scales=None, stream=None):
    """rows[position[t, j]] = x[t] for every pick that has a row.  x [T, H] and rows [R, H] bf16,
    float32, or e4m3 codes (float8_e4m3fn or uint8) with x_scales float32 [T, H / 128] and rows_scales
    [R, H / 128]."""
    _needed(rows=rows)
    (T, H), dev = _matrix(x, "x", _ROW + _E4M3)
    (R, _), _ = _matrix(rows, "rows", _ROW + _E4M3)
    codes = _DTYPE[x.dtype] == 2
    if codes:
        _needed(x_scales=x_scales, rows_scales=rows_scales)
        px, xs = _packed(x, "x", _E4M3, (T, H), dev), 0
        pr, rs = _packed(rows, "rows", _E4M3, (R, H), dev), 0
        pc = _packed(x_scales, "x_scales", _F32, (T, H // 128), dev)
        pd = _packed(rows_scales, "rows_scales", _F32, (R, H // 128), dev)
    else:
        if x_scales is not None or rows_scales is not None:
            raise ValueError("x_scales and rows_scales belong to codes")
        px, xs = _rows(x, "x", _ROW, (T, H), dev)
        pr, rs = _rows(rows, "rows", (x.dtype,), (R, H), dev)
        pc = pd = None
    pp, k = _positions(position, T, dev)
    g = MoeRows(T, k, H, R, _DTYPE[x.dtype], 0, rs, 0, xs)
    _call(_lib().moe_sort_rows(g, px, pc, pp, pr, pd, _stream(stream, dev)), "moe_sort_rows")


def moe_sort_rows_backward(drows, position, dx, stream=None):
    """dx[t] = sum of drows[position[t, j]] over the token's picks (bf16 or float32 alike)."""
    _needed(dx=dx)
    (R, H), dev = _matrix(drows, "drows", _ROW)
    (T, _), _ = _matrix(dx, "dx", _ROW)
    pr, rs = _rows(drows, "drows", _ROW, (R, H), dev)
    px, xs = _rows(dx, "dx", (drows.dtype,), (T, H), dev)
    pp, k = _positions(position, T, dev)
    g = MoeRows(T, k, H, R, DTYPE[drows.dtype], DTYPE[drows.dtype], rs, 0, xs)
    _call(_lib().moe_sort_rows_backward(g, pr, pp, px, _stream(stream, dev)), "moe_sort_rows_backward")


def moe_unsort_rows(rows, weights, position, out, stream=None):
    """out[t] = sum over the token's picks of weights[t, j] * rows[position[t, j]], in their order;
    weights float32 [T, k], or None: all 1.  rows [R, H] and out [T, H] bf16 or float32 each."""
    _needed(out=out)
    (R, H), dev = _matrix(rows, "rows", _ROW)
    (T, _), _ = _matrix(out, "out", _ROW)
    pr, rs = _rows(rows, "rows", _ROW, (R, H), dev)
    po, os = _rows(out, "out", _ROW, (T, H), dev)
    pp, k = _positions(position, T, dev)
    pw = _packed(weights, "weights", _F32, (T, k), dev)
    g = MoeRows(T, k, H, R, DTYPE[rows.dtype], DTYPE[out.dtype], rs, 0, os)
    _call(_lib().moe_unsort_rows(g, pr, pw, pp, po, _stream(stream, dev)), "moe_unsort_rows")


def moe_unsort_rows_backward(dout, rows, weights, position, drows, dweights, stream=None):
    """Gradient of moe_unsort_rows: drows[position[t, j]] = weights[t, j] * dout[t] (of rows' type and
    shape) and dweights[t, j] = <dout[t], rows[position[t, j]]> (float32, 0 for masked picks); either
    may be None.  Rows that no pick has are left as they were in drows."""
    (T, H), dev = _matrix(dout, "dout", _ROW)
    if drows is None and dweights is None:
        raise ValueError("drows or dweights must be given")
    if dweights is not None:
        _needed(rows=rows)
    like = rows if rows is not None else drows
    (R, _), _ = _matrix(like, "rows" if rows is not None else "drows", _ROW)
    pg, gs = _rows(dout, "dout", _ROW, (T, H), dev)
    pr, rs = _rows(rows, "rows", _ROW, (R, H), dev)
    pd, ds = _rows(drows, "drows", (like.dtype,), (R, H), dev)
    pp, k = _positions(position, T, dev)
    pw = _packed(weights, "weights", _F32, (T, k), dev)
    pv = _packed(dweights, "dweights", _F32, (T, k), dev)
    g = MoeRows(T, k, H, R, DTYPE[like.dtype], DTYPE[dout.dtype], rs, ds, gs)
    _call(_lib().moe_unsort_rows_backward(g, pg, pr, pw, pp, pd, pv, _stream(stream, dev)),
          "moe_unsort_rows_backward")


def moe_quantize_fp8(x, codes, scales, block_rows=1, live_rows=None, stream=None):
    """x bf16 or float32 [R, C] (rows) or [.., R, C] (contiguous) to e4m3 codes of its shape
    (float8_e4m3fn or uint8) and float32 scales [.., R, C / 128], or [.., ceil(R / 128), C / 128] with
    block_rows=128.  live_rows: int32 [1], only the first that many rows are taken (a matrix, block_rows=1)."""
    _typed(x, "x", _ROW)
    if x.dim() < 2 or block_rows not in (1, 128):
        raise ValueError("x: shape %s, expected rows, and block_rows 1 or 128" % (tuple(x.shape),))
    _needed(codes=codes, scales=scales)
    lead, (R, C), dev = x.shape[:-2], x.shape[-2:], x.get_device()
    n = lead.numel()
    px, xs = _rows(x, "x", _ROW, x.shape, dev) if not lead else (_packed(x, "x", _ROW, x.shape, dev), 0)
    pc = _packed(codes, "codes", _E4M3, x.shape, dev)
    ps = _packed(scales, "scales", _F32, lead + (-(-R // block_rows), C // 128), dev)
    pl = _packed(live_rows, "live_rows", _I32, (1,), dev)
    stream = _stream(stream, dev)
    if n == 0:
        return
    _call(_lib().moe_quantize_fp8(MoeQuantize(n, R, C, block_rows, DTYPE[x.dtype], xs), px, pl, pc, ps, stream),
          "moe_quantize_fp8")


def moe_swiglu_fp8(gate_up, codes, scales, live_rows=None, stream=None):
    """silu(gate) * up of gate_up bf16 or float32 [R, 2 C] (gate: the first C columns), as e4m3 codes
    [R, C] and float32 scales [R, C / 128].  live_rows as in moe_quantize_fp8."""
    _needed(codes=codes, scales=scales)
    (R, W), dev = _matrix(gate_up, "gate_up", _ROW)
    if W % 2:
        raise ValueError("gate_up: shape %s, expected [rows, 2 * columns]" % (tuple(gate_up.shape),))
    C = W // 2
    px, xs = _rows(gate_up, "gate_up", _ROW, (R, W), dev)
    pc = _packed(codes, "codes", _E4M3, (R, C), dev)
    ps = _packed(scales, "scales", _F32, (R, C // 128), dev)
    pl = _packed(live_rows, "live_rows", _I32, (1,), dev)
    _call(_lib().moe_swiglu_fp8(MoeQuantize(1, R, C, 1, DTYPE[gate_up.dtype], xs), px, pl, pc, ps,
                                _stream(stream, dev)), "moe_swiglu_fp8")


def moe_product_fp8(a, a_scales, b, b_scales, out, offsets=None, status=None, stream=None):
    """out[m] = a[m] b^T for e4m3 rows a [M, K] (float32 scales [M, K / 128]) and e4m3 weights b [N, K]
    (scales [ceil(N / 128), K / 128]), or, with offsets int32 [G + 1] as moe_sort_picks writes them,
    b [G, N, K] (scales [G, ..]) of which rows offsets[g] to offsets[g + 1] take matrix g; rows of no
    group are left as they were.  out [M, N] bf16 or float32.  status: int32 [1], into which
    MOE_STATUS_TIMEOUT is or-ed where a wait of the kernel gave up."""
    _needed(out=out)
    (M, K), dev = _matrix(a, "a", _E4M3)
    _typed(b, "b", _E4M3)
    if b.dim() != (2 if offsets is None else 3):
        raise ValueError("b: shape %s, expected %s" % (tuple(b.shape), "[N, K]" if offsets is None else "[G, N, K]"))
    lead, N = b.shape[:-2], b.shape[-2]
    pa, sa = _rows(a, "a", _E4M3, (M, K), dev)
    pb = _packed(b, "b", _E4M3, lead + (N, K), dev)
    ps = _packed(a_scales, "a_scales", _F32, (M, K // 128), dev)
    pt = _packed(b_scales, "b_scales", _F32, lead + (-(-N // 128), K // 128), dev)
    _needed(a_scales=a_scales, b_scales=b_scales)
    po, so = _rows(out, "out", _ROW, (M, N), dev)
    pf = _packed(offsets, "offsets", _I32, tuple(n + 1 for n in lead), dev)
    px = _packed(status, "status", _I32, (1,), dev)
    if pf is not None and not lead[0]:
        raise ValueError("b: no matrix for the rows")
    p = MoeProduct(M, N, K, lead[0] if lead else 0, DTYPE[out.dtype], sa, so)
    _call(_lib().moe_product_fp8(p, pa, ps, pb, pt, pf, po, px, _stream(stream, dev)), "moe_product_fp8")
