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

from .block import (_BYTE, _E4M3, _F32, _IDS, _P, _ROW, DTYPE, _call, _lib, _packed, _rows, _stream, _too_large,
                    _typed)

_I32 = (torch.int32,)
_ROWS_CODES = _ROW + _E4M3
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


# Small calls take as long as their checks do on the host: a tensor is looked at once, and what is
# right is found out first.

def _matrix(t, name, dtypes):
    """(rows, columns), device, address and row stride of a matrix with packed columns whose shape
    is the call's to find out."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.dim() == 2 and t.is_contiguous():
        return t.shape, t.get_device(), t.data_ptr(), 0
    _typed(t, name, dtypes)
    if t.dim() != 2:
        raise ValueError("%s: shape %s, expected a matrix" % (name, tuple(t.shape)))
    dev = t.get_device()
    return (t.shape, dev, *_rows(t, name, dtypes, t.shape, dev))


def _packed_matrix(t, name, dtypes):
    """(rows, columns), device and address of a contiguous matrix."""
    shape, dev, p, stride = _matrix(t, name, dtypes)
    if stride:
        raise ValueError("%s: strides %s; must be contiguous" % (name, t.stride()))
    return shape, dev, p


def _missing(names, *addresses):
    """Raises for the first of the names whose address is None."""
    raise ValueError("%s must be given" % names.split()[addresses.index(None)])


def moe_sort_picks_workspace_size(tokens, top_k, num_experts):
    """Bytes of the workspace of moe_sort_picks."""
    size = ctypes.c_size_t()
    if max(tokens, top_k, num_experts) >> 31:
        _too_large("moe_sort_picks_workspace_size")
    _call(_lib().moe_sort_picks_workspace_size(MoeSort(tokens, num_experts, top_k), ctypes.byref(size)),
          "moe_sort_picks_workspace_size")
    return size.value


def moe_sort_picks(topk_ids, num_experts, offsets, position, workspace, source=None, status=None, stream=None):
    """The order of the picks topk_ids (int32 or int64 [T, k], -1: masked) by (expert, token, pick):
    offsets int32 [num_experts + 1], the first row of each expert; position int32 [T, k], each pick's
    row or -1; source int32 [T * k], the pick t * k + j of each row, -1 behind the last one; status
    int32 [1], MOE_STATUS_* bits (an id outside [-1, num_experts) is dropped).  workspace: uint8, of
    moe_sort_picks_workspace_size bytes."""
    (T, k), dev, pi = _packed_matrix(topk_ids, "topk_ids", _IDS)
    if (T | k | num_experts) >> 31 > 0:
        _too_large("moe_sort_picks")
    po = _packed(offsets, "offsets", _I32, (num_experts + 1,), dev)
    pp = _packed(position, "position", _I32, (T, k), dev)
    if workspace is not None:
        _typed(workspace, "workspace", _BYTE)
    pw = None if workspace is None else _packed(workspace, "workspace", _BYTE, workspace.shape, dev)
    ps = _packed(source, "source", _I32, (T * k,), dev)
    pt = _packed(status, "status", _I32, (1,), dev)
    if po is None or pp is None or pw is None:
        _missing("offsets position workspace", po, pp, pw)
    _call(_lib().moe_sort_picks(MoeSort(T, num_experts, k), pi, _IDS[topk_ids.dtype], po, pp, ps, pt, pw,
                                workspace.numel(), _stream(stream, dev)), "moe_sort_picks")


def moe_sort_rows(x, position, rows, x_scales=None, rows_scales=None, stream=None):
    """rows[position[t, j]] = x[t] for every pick that has a row.  x [T, H] and rows [R, H] bf16,
    float32, or e4m3 codes (float8_e4m3fn or uint8) with x_scales float32 [T, H / 128] and rows_scales
    [R, H / 128]."""
    if rows is None:
        _missing("rows", None)
    (T, H), dev, px, xs = _matrix(x, "x", _ROWS_CODES)
    (R, _), _, pr, rs = _matrix(rows, "rows", _ROWS_CODES)
    (t, k), _, pp = _packed_matrix(position, "position", _I32)
    if (T | H | R | k) >> 31:
        _too_large("moe_sort_rows")
    dtype, shape = _DTYPE[x.dtype], (R, H)
    if t != T or rows.shape != shape or rows.get_device() != dev or position.get_device() != dev or \
            _DTYPE[rows.dtype] != dtype:
        _typed(rows, "rows", _E4M3 if dtype == 2 else (x.dtype,))
        _rows(rows, "rows", _ROWS_CODES, shape, dev)
        _packed(position, "position", _I32, (T, k), dev)
    pc = _packed(x_scales, "x_scales", _F32, (T, H // 128), dev)
    pd = _packed(rows_scales, "rows_scales", _F32, (R, H // 128), dev)
    if dtype == 2:
        if pc is None or pd is None:
            _missing("x_scales rows_scales", pc, pd)
        if xs or rs:
            raise ValueError("x and rows: codes must be contiguous")
    elif pc is not None or pd is not None:
        raise ValueError("x_scales and rows_scales belong to codes")
    _call(_lib().moe_sort_rows(MoeRows(T, k, H, R, dtype, 0, rs, 0, xs), px, pc, pp, pr, pd, _stream(stream, dev)),
          "moe_sort_rows")


def moe_sort_rows_backward(drows, position, dx, stream=None):
    """dx[t] = sum of drows[position[t, j]] over the token's picks (bf16 or float32 alike)."""
    (T, k), dev, pp = _packed_matrix(position, "position", _I32)
    (R, H), _, pr, rs = _matrix(drows, "drows", _ROW)
    if (T | k | R | H) >> 31:
        _too_large("moe_sort_rows_backward")
    if drows.get_device() != dev:
        _rows(drows, "drows", _ROW, drows.shape, dev)
    px, xs = _rows(dx, "dx", (drows.dtype,), (T, H), dev)
    if px is None:
        _missing("dx", px)
    dtype = DTYPE[drows.dtype]
    _call(_lib().moe_sort_rows_backward(MoeRows(T, k, H, R, dtype, dtype, rs, 0, xs), pr, pp, px, _stream(stream, dev)),
          "moe_sort_rows_backward")


def moe_unsort_rows(rows, weights, position, out, stream=None):
    """out[t] = sum over the token's picks of weights[t, j] * rows[position[t, j]], in their order;
    weights float32 [T, k], or None: all 1.  rows [R, H] and out [T, H] bf16 or float32 each."""
    (T, k), dev, pp = _packed_matrix(position, "position", _I32)
    (R, H), _, pr, rs = _matrix(rows, "rows", _ROW)
    if (T | k | R | H) >> 31:
        _too_large("moe_unsort_rows")
    if rows.get_device() != dev:
        _rows(rows, "rows", _ROW, rows.shape, dev)
    po, os = _rows(out, "out", _ROW, (T, H), dev)
    pw = _packed(weights, "weights", _F32, (T, k), dev)
    if po is None:
        _missing("out", po)
    g = MoeRows(T, k, H, R, DTYPE[rows.dtype], DTYPE[out.dtype], rs, 0, os)
    _call(_lib().moe_unsort_rows(g, pr, pw, pp, po, _stream(stream, dev)), "moe_unsort_rows")


def moe_unsort_rows_backward(dout, rows, weights, position, drows, dweights, stream=None):
    """Gradient of moe_unsort_rows: drows[position[t, j]] = weights[t, j] * dout[t] (of rows' type and
    shape) and dweights[t, j] = <dout[t], rows[position[t, j]]> (float32, 0 for masked picks); either
    may be None.  Rows that no pick has are left as they were in drows."""
    (T, k), dev, pp = _packed_matrix(position, "position", _I32)
    (t, H), _, pg, gs = _matrix(dout, "dout", _ROW)
    if t != T or dout.get_device() != dev:
        _rows(dout, "dout", _ROW, (T, H), dev)
    like = drows if rows is None else rows
    if like is None:
        raise ValueError("rows or drows must be given")
    if drows is None and dweights is None:
        raise ValueError("drows or dweights must be given")
    R = _matrix(like, "drows" if rows is None else "rows", _ROW)[0][0]
    if (T | k | R | H) >> 31:
        _too_large("moe_unsort_rows_backward")
    pr, rs = _rows(rows, "rows", _ROW, (R, H), dev)
    pd, ds = _rows(drows, "drows", (like.dtype,), (R, H), dev)
    pw = _packed(weights, "weights", _F32, (T, k), dev)
    pv = _packed(dweights, "dweights", _F32, (T, k), dev)
    if rows is None and dweights is not None:
        _missing("rows", None)
    g = MoeRows(T, k, H, R, DTYPE[like.dtype], DTYPE[dout.dtype], rs, ds, gs)
    _call(_lib().moe_unsort_rows_backward(g, pg, pr, pw, pp, pd, pv, _stream(stream, dev)),
          "moe_unsort_rows_backward")


def moe_quantize_fp8(x, codes, scales, block_rows=1, live_rows=None, stream=None):
    """x bf16 or float32 [R, C] (rows) or [.., R, C] (contiguous) to e4m3 codes of its shape
    (float8_e4m3fn or uint8) and float32 scales [.., R, C / 128], or [.., ceil(R / 128), C / 128] with
    block_rows=128.  live_rows: int32 [1], only the first that many rows are taken (a matrix, block_rows=1)."""
    if isinstance(x, torch.Tensor) and x.dim() == 2:
        (R, C), dev, px, xs = _matrix(x, "x", _ROW)
        lead, n = (), 1
    else:
        _typed(x, "x", _ROW)
        if x.dim() < 2:
            raise ValueError("x: shape %s, expected rows" % (tuple(x.shape),))
        lead, (R, C), dev = x.shape[:-2], x.shape[-2:], x.get_device()
        px, xs, n = _packed(x, "x", _ROW, x.shape, dev), 0, lead.numel()
    if (n | R | C) >> 31:
        _too_large("moe_quantize_fp8")
    if block_rows not in (1, 128):
        raise ValueError("block_rows: %r, expected 1 or 128" % (block_rows,))
    pc = _packed(codes, "codes", _E4M3, x.shape, dev)
    ps = _packed(scales, "scales", _F32, (*lead, -(-R // block_rows), C // 128), dev)
    pl = _packed(live_rows, "live_rows", _I32, (1,), dev)
    if pc is None or ps is None:
        _missing("codes scales", pc, ps)
    stream = _stream(stream, dev)
    if n:
        _call(_lib().moe_quantize_fp8(MoeQuantize(n, R, C, block_rows, DTYPE[x.dtype], xs), px, pl, pc, ps, stream),
              "moe_quantize_fp8")


def moe_swiglu_fp8(gate_up, codes, scales, live_rows=None, stream=None):
    """silu(gate) * up of gate_up bf16 or float32 [R, 2 C] (gate: the first C columns), as e4m3 codes
    [R, C] and float32 scales [R, C / 128].  live_rows as in moe_quantize_fp8."""
    (R, W), dev, px, xs = _matrix(gate_up, "gate_up", _ROW)
    if W % 2:
        raise ValueError("gate_up: shape %s, expected [rows, 2 * columns]" % (tuple(gate_up.shape),))
    C = W // 2
    if (R | C) >> 31:
        _too_large("moe_swiglu_fp8")
    pc = _packed(codes, "codes", _E4M3, (R, C), dev)
    ps = _packed(scales, "scales", _F32, (R, C // 128), dev)
    pl = _packed(live_rows, "live_rows", _I32, (1,), dev)
    if pc is None or ps is None:
        _missing("codes scales", pc, ps)
    _call(_lib().moe_swiglu_fp8(MoeQuantize(1, R, C, 1, DTYPE[gate_up.dtype], xs), px, pl, pc, ps,
                                _stream(stream, dev)), "moe_swiglu_fp8")


def moe_product_fp8(a, a_scales, b, b_scales, out, offsets=None, status=None, stream=None):
    """out[m] = a[m] b^T for e4m3 rows a [M, K] (float32 scales [M, K / 128]) and e4m3 weights b [N, K]
    (scales [ceil(N / 128), K / 128]), or, with offsets int32 [G + 1] as moe_sort_picks writes them,
    b [G, N, K] (scales [G, ..]) of which rows offsets[g] to offsets[g + 1] take matrix g; rows of no
    group are left as they were.  out [M, N] bf16 or float32.  status: int32 [1], into which
    MOE_STATUS_TIMEOUT is or-ed where a wait of the kernel gave up, and out is not valid; without it that
    cannot be seen.  The caller clears the word: moe_sort_picks with the same word does."""
    (M, K), dev, pa, sa = _matrix(a, "a", _E4M3)
    _typed(b, "b", _E4M3)
    lead = b.shape[:-2]
    if b.dim() != (2 if offsets is None else 3):
        raise ValueError("b: shape %s, expected %s" % (tuple(b.shape), "[N, K]" if offsets is None else "[G, N, K]"))
    N, G = b.shape[-2], lead[0] if lead else 0
    if (M | K | N | G) >> 31:
        _too_large("moe_product_fp8")
    pb = _packed(b, "b", _E4M3, (*lead, N, K), dev)
    ps = _packed(a_scales, "a_scales", _F32, (M, K // 128), dev)
    pt = _packed(b_scales, "b_scales", _F32, (*lead, -(-N // 128), K // 128), dev)
    po, so = _rows(out, "out", _ROW, (M, N), dev)
    pf = _packed(offsets, "offsets", _I32, (G + 1,), dev)
    px = _packed(status, "status", _I32, (1,), dev)
    if ps is None or pt is None or po is None:
        _missing("a_scales b_scales out", ps, pt, po)
    if lead and not G:
        raise ValueError("b: no matrix for the rows")
    _call(_lib().moe_product_fp8(MoeProduct(M, N, K, G, DTYPE[out.dtype], sa, so), pa, ps, pb, pt, pf, po, px,
                                 _stream(stream, dev)), "moe_product_fp8")
