"""Python binding of the operators around the expert layer (include/moe_block.h).

moe_add_rmsnorm / moe_add_rmsnorm_backward, moe_route_topk / moe_route_topk_backward and the
4-bit expert FFN: moe_quantize_w4, moe_prepare_weights_w4, moe_forward_w4 and MoELayerW4,
which owns one layer's weights and buffers.  Argument checks and marshalling only; results
go to the caller's tensors, on the current stream or the one given.

The norm's row matrices and the router's logits may have any row stride (their columns are
packed); every other tensor is contiguous.  A tensor of another type raises TypeError, one of another shape, layout or
device ValueError, and what the library refuses MoeError.
"""
import ctypes

import torch

DTYPE = {torch.bfloat16: 0, torch.float32: 1}
SCORE = {"softmax": 0, "sigmoid": 1}
GROUP_SCORE = {"max": 0, "top2": 1}
_IDS = {torch.int32: 0, torch.int64: 1}
_P = ctypes.c_void_p


class MoeNorm(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("residual_dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64),
                ("residual_stride", ctypes.c_int64), ("sum_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]


class MoeRouter(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("num_experts", "top_k", "score", "groups", "top_groups", "group_score",
                                               "renormalize", "logits_dtype")] +
                [("scale", ctypes.c_float), ("logits_stride", ctypes.c_int64)])


class MoeW4Geom(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_tokens", "hidden", "num_experts", "top_k", "intermediate", "group")]


def bind(L):
    """Argument types of the library's entry points of this header."""
    N, R, W = ctypes.POINTER(MoeNorm), ctypes.POINTER(MoeRouter), ctypes.POINTER(MoeW4Geom)
    i32, i64, size, out = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
    L.moe_add_rmsnorm.argtypes = [N] + [_P] * 9
    L.moe_add_rmsnorm_workspace_size.argtypes = [N, out]
    L.moe_add_rmsnorm_backward.argtypes = [N] + [_P] * 8 + [size, _P]
    L.moe_route_topk.argtypes = [R, i32, _P, _P, _P, ctypes.c_int, _P, _P]
    L.moe_route_topk_backward.argtypes = [R, i32, _P, _P, ctypes.c_int, _P, _P, _P]
    L.moe_quantize_w4.argtypes = [i64, i64, i32] + [_P] * 4
    L.moe_prepare_weights_w4.argtypes = [W] + [_P] * 9
    L.moe_forward_w4_workspace_size.argtypes = [W, out]
    L.moe_forward_w4.argtypes = [W, _P, _P, ctypes.c_int] + [_P] * 8 + [size, _P]
    for f in ("moe_add_rmsnorm", "moe_add_rmsnorm_workspace_size", "moe_add_rmsnorm_backward", "moe_route_topk",
              "moe_route_topk_backward", "moe_quantize_w4", "moe_prepare_weights_w4",
              "moe_forward_w4_workspace_size", "moe_forward_w4"):
        getattr(L, f).restype = ctypes.c_int


_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        from . import lib
        _loaded = lib()
    return _loaded


def _call(rc, where):
    if rc != 0:
        from . import MoeError
        raise MoeError(rc, where)


def _typed(t, name, dtypes):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor, got %s" % (name, type(t).__name__))
    if t.dtype not in dtypes:
        raise TypeError("%s: dtype %s, expected %s" % (name, t.dtype, " or ".join(str(d) for d in dtypes)))


def _refuse(t, name, dtypes, shape, dev, layout):
    """Raises for what _packed or _rows found wrong."""
    _typed(t, name, dtypes)
    if t.shape != shape:
        raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.get_device() != dev:
        raise ValueError("%s is on %s; expected device %d" % (name, t.device, dev))
    raise ValueError("%s: strides %s; %s" % (name, t.stride(), layout))


def _too_large(where):
    """Raises for a size that the C structs' 32-bit fields do not hold: ctypes would cut it off without a word."""
    _call(-13, where)   # MOE_ERR_LIMIT


# Small calls take as long as their checks do on the host, so what is right is found out first.

def _packed(t, name, dtypes, shape, dev):
    """The address of a contiguous tensor of one of `dtypes`, of `shape` and on device `dev`;
    None stays None."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.is_contiguous() \
            and t.get_device() == dev:
        return t.data_ptr()
    _refuse(t, name, dtypes, shape, dev, "must be contiguous")


def _rows(t, name, dtypes, shape, dev):
    """(address, row stride) of a matrix with packed columns."""
    if t is None:
        return None, 0
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == dev:
        if t.is_contiguous():
            return t.data_ptr(), 0
        row, col = t.stride()
        if (col == 1 or shape[1] <= 1) and (row >= shape[1] or shape[0] <= 1):
            return t.data_ptr(), row if shape[0] > 1 else 0
    _refuse(t, name, dtypes, shape, dev, "rows may lie apart, but not overlap, and columns are packed")


def _stream(stream, dev):
    """The handle of the stream given, or of the current one, of device `dev`."""
    if dev < 0:
        raise ValueError("the tensors are in host memory; expected a CUDA device")
    if stream is None:
        if torch._C._cuda_getDevice() != dev:
            raise ValueError("the tensors are on cuda:%d, and the current device is cuda:%d"
                             % (dev, torch.cuda.current_device()))
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError("the tensors are on cuda:%d, and the stream is on cuda:%d" % (dev, stream.device_index))
    return stream.cuda_stream


_BF16, _F32, _ROW = (torch.bfloat16,), (torch.float32,), (torch.bfloat16, torch.float32)
_E4M3, _BYTE = (torch.float8_e4m3fn, torch.uint8), (torch.uint8,)


def moe_add_rmsnorm(x, residual, weight, eps, sum_out=None, out=None, out_fp8=None, scales=None, rstd=None,
                    stream=None):
    """h = x + residual (None: h = x) and y = h / sqrt(mean(h^2) + eps) * weight, row by row.

    x bf16 [T, H]; residual and sum_out (h) bf16 or float32 alike; weight bf16 or float32 [H].
    Writes those of out (bf16 y), out_fp8 with scales (y as float8_e4m3fn or uint8 codes [T, H]
    and float32 [T, H / 128]; what moe_dispatch_fp8 takes), sum_out and rstd (float32 [T], for
    the gradient) that are given.  sum_out may be residual, and out may be x."""
    _typed(x, "x", _BF16)
    if x.dim() != 2:
        raise ValueError("x: shape %s, expected [tokens, hidden]" % (tuple(x.shape),))
    if weight is None or (out is None and out_fp8 is None) or (out_fp8 is None) != (scales is None):
        raise ValueError("weight, and out or out_fp8 with scales, must be given")
    shape, dev = x.shape, x.get_device()
    T, H = shape
    if (T | H) >> 31:
        _too_large("moe_add_rmsnorm")
    px, xs = _rows(x, "x", _BF16, shape, dev)
    pr, rs = _rows(residual, "residual", _ROW, shape, dev)
    ps, ss = _rows(sum_out, "sum_out", _ROW if residual is None else (residual.dtype,), shape, dev)
    po, os = _rows(out, "out", _BF16, shape, dev)
    pw = _packed(weight, "weight", _ROW, (H,), dev)
    pq = _packed(out_fp8, "out_fp8", _E4M3, shape, dev)
    pc = _packed(scales, "scales", _F32, (T, H // 128), dev)
    pd = _packed(rstd, "rstd", _F32, (T,), dev)
    h = sum_out if residual is None else residual
    n = MoeNorm(T, H, 0 if h is None else DTYPE[h.dtype], DTYPE[weight.dtype], eps, xs, rs, ss, os)
    _call(_lib().moe_add_rmsnorm(n, px, pr, pw, ps, po, pq, pc, pd, _stream(stream, dev)), "moe_add_rmsnorm")


def moe_add_rmsnorm_workspace_size(tokens, hidden):
    """Bytes of the workspace of moe_add_rmsnorm_backward."""
    size = ctypes.c_size_t()
    if max(tokens, hidden) >> 31:
        _too_large("moe_add_rmsnorm_workspace_size")
    _call(_lib().moe_add_rmsnorm_workspace_size(MoeNorm(tokens, hidden), ctypes.byref(size)),
          "moe_add_rmsnorm_workspace_size")
    return size.value


def moe_add_rmsnorm_backward(dout, h, weight, rstd, dx, dweight, workspace, dsum=None, stream=None):
    """Gradient of moe_add_rmsnorm at the saved h (sum_out) and rstd: dx for x and residual
    alike, with dsum (the gradient that reaches h from the residual stream) added, and dweight
    (float32).  dout bf16; h, dsum and dx bf16 or float32 alike; dx may be dsum."""
    _typed(dout, "dout", _BF16)
    if dout.dim() != 2:
        raise ValueError("dout: shape %s, expected [tokens, hidden]" % (tuple(dout.shape),))
    _typed(h, "h", _ROW)
    _typed(workspace, "workspace", _BYTE)
    shape, dev, same = dout.shape, dout.get_device(), (h.dtype,)
    T, H = shape
    if (T | H) >> 31:
        _too_large("moe_add_rmsnorm_backward")
    pg, gs = _rows(dout, "dout", _BF16, shape, dev)
    ph, hs = _rows(h, "h", same, shape, dev)
    ps, ss = _rows(dsum, "dsum", same, shape, dev)
    px, xs = _rows(dx, "dx", same, shape, dev)
    pw = _packed(weight, "weight", _ROW, (H,), dev)
    pr = _packed(rstd, "rstd", _F32, (T,), dev)
    pd = _packed(dweight, "dweight", _F32, (H,), dev)
    pk = _packed(workspace, "workspace", _BYTE, workspace.shape, dev)
    if None in (pw, pr, pd, px):
        raise ValueError("weight, rstd, dx and dweight must be given")
    n = MoeNorm(T, H, DTYPE[h.dtype], DTYPE[weight.dtype], 0.0, gs, hs, ss, xs)
    _call(_lib().moe_add_rmsnorm_backward(n, pg, ph, pw, pr, ps, px, pd, pk, workspace.numel(), _stream(stream, dev)),
          "moe_add_rmsnorm_backward")


def make_router(num_experts, top_k, score="softmax", groups=1, top_groups=None, group_score="max",
                renormalize=True, scale=1.0):
    """The router's rule.  score: "softmax" or "sigmoid"; groups: equal runs of experts, of which
    the top_groups best (all by default) take part, by their largest key ("max") or the sum of
    their two largest ("top2"); renormalize: the picked scores are divided by their sum."""
    return MoeRouter(num_experts, top_k, SCORE[score], groups, groups if top_groups is None else top_groups,
                     GROUP_SCORE[group_score], int(renormalize), 0, scale, 0)


def _route(r, logits):
    """The rule for these logits, their address, shape [T, k] of the picks and device."""
    _typed(logits, "logits", _ROW)
    if logits.dim() != 2 or logits.shape[1] != r.num_experts:
        raise ValueError("logits: shape %s, expected [tokens, %d]" % (tuple(logits.shape), r.num_experts))
    if logits.shape[0] >> 31:
        _too_large("moe_route_topk")
    dev = logits.get_device()
    p, stride = _rows(logits, "logits", _ROW, logits.shape, dev)
    dtype = DTYPE[logits.dtype]
    if r.logits_dtype != dtype or r.logits_stride != stride:
        r = MoeRouter.from_buffer_copy(r)   # the caller's rule stays as it is
        r.logits_dtype, r.logits_stride = dtype, stride
    return r, p, (logits.shape[0], r.top_k), dev


def moe_route_topk(r, logits, bias, topk_ids, topk_weights, stream=None):
    """Expert ids (int32 or int64 [T, k], -1 where no expert is left) and routing weights
    (float32 [T, k]) from the gate's logits (bf16 or float32 [T, E]) by the rule `r`
    (make_router).  bias: float32 [E], added to the scores for the picking alone, or None."""
    r, pl, picks, dev = _route(r, logits)
    pb = _packed(bias, "bias", _F32, (r.num_experts,), dev)
    pi = _packed(topk_ids, "topk_ids", _IDS, picks, dev)
    pw = _packed(topk_weights, "topk_weights", _F32, picks, dev)
    if pi is None or pw is None:
        raise ValueError("topk_ids and topk_weights must be given")
    _call(_lib().moe_route_topk(r, picks[0], pl, pb, pi, _IDS[topk_ids.dtype], pw, _stream(stream, dev)),
          "moe_route_topk")


def moe_route_topk_backward(r, logits, topk_ids, dweights, dlogits, stream=None):
    """dlogits (contiguous, of the logits' type) from dweights, the picks held fixed."""
    r, pl, picks, dev = _route(r, logits)
    pi = _packed(topk_ids, "topk_ids", _IDS, picks, dev)
    pw = _packed(dweights, "dweights", _F32, picks, dev)
    pd = _packed(dlogits, "dlogits", (logits.dtype,), logits.shape, dev)
    if None in (pi, pw, pd):
        raise ValueError("topk_ids, dweights and dlogits must be given")
    _call(_lib().moe_route_topk_backward(r, picks[0], pl, pi, _IDS[topk_ids.dtype], pw, pd, _stream(stream, dev)),
          "moe_route_topk_backward")


def moe_quantize_w4(w, group, codes, scales, stream=None):
    """bf16 w [..., cols] to 4-bit codes (uint8 [..., cols / 2], the even column in the low half)
    and bf16 scales [..., cols / group]; a weight is (code - 8) * scale."""
    _typed(w, "w", _BF16)
    if w.dim() < 1 or group not in (32, 64, 128) or w.shape[-1] % group:
        raise ValueError("w: shape %s, expected whole groups of 32, 64 or 128 columns" % (tuple(w.shape),))
    cols, dev = w.shape[-1], w.get_device()
    pw = _packed(w, "w", _BF16, w.shape, dev)
    pc = _packed(codes, "codes", _BYTE, w.shape[:-1] + (cols // 2,), dev)
    ps = _packed(scales, "scales", _BF16, w.shape[:-1] + (cols // group,), dev)
    if pc is None or ps is None:
        raise ValueError("codes and scales must be given")
    _call(_lib().moe_quantize_w4(w.numel() // max(cols, 1), cols, group, pw, pc, ps, _stream(stream, dev)),
          "moe_quantize_w4")


def make_w4_geom(tokens, hidden, experts, k, intermediate, group):
    return MoeW4Geom(tokens, hidden, experts, k, intermediate, group)


def moe_forward_w4_workspace_size(g):
    size = ctypes.c_size_t()
    _call(_lib().moe_forward_w4_workspace_size(g, ctypes.byref(size)), "moe_forward_w4_workspace_size")
    return size.value


class MoELayerW4:
    """The routed experts of one layer with 4-bit weights, for batches of up to `max_tokens`.

    forward(x, topk_ids, topk_weights) -> out [T, H] bf16, the function of MoELayer1GPU.forward
    with the activation in the eleven bits of f16 (there by default a pair of bf16), on the
    current stream and with no host synchronisation.  group: inputs per scale (32, 64 or 128).  The buffers (out among them) are the layer's own and are written by every call.
    """

    def __init__(self, max_tokens, hidden, num_experts, top_k, intermediate, group=128, device="cuda"):
        self.geom = make_w4_geom(max_tokens, hidden, num_experts, top_k, intermediate, group)
        self.device = torch.device(device)
        self.max_tokens = max_tokens
        self.workspace = torch.empty(moe_forward_w4_workspace_size(self.geom), dtype=torch.uint8, device=self.device)
        self.out = torch.empty((max_tokens, hidden), dtype=torch.bfloat16, device=self.device)
        self.status_word = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.weights = None
        self._addresses = None
        self._buffers = (self.out.data_ptr(), self.status_word.data_ptr(), self.workspace.data_ptr(),
                         self.workspace.numel())

    def set_weights(self, w1, s1, w2, s2):
        """Codes w1 uint8 [E, 2I, H / 2] (gate rows, then up rows) and w2 [E, H, I / 2] with bf16
        scales s1 [E, 2I, H / group] and s2 [E, H, I / group]; put in the kernels' order once here."""
        g = self.geom
        E, H, I, G = g.num_experts, g.hidden, g.intermediate, g.group
        given = [(w1, "w1", _BYTE, (E, 2 * I, H // 2)), (s1, "s1", _BF16, (E, 2 * I, H // G)),
                 (w2, "w2", _BYTE, (E, H, I // 2)), (s2, "s2", _BF16, (E, H, I // G))]
        dev = self.out.get_device()
        natural = [_packed(*one, dev) for one in given]
        if None in natural:
            raise ValueError("w1, s1, w2 and s2 must be given")
        s = _stream(None, dev)
        weights = [torch.empty_like(t) for t, _, _, _ in given]
        addresses = [t.data_ptr() for t in weights]
        _call(_lib().moe_prepare_weights_w4(g, *natural, *addresses, s), "moe_prepare_weights_w4")
        self.weights, self._addresses = weights, addresses   # (the old ones stay where the call was refused)

    def quantize_weights(self, w1, w2):
        """set_weights from bf16 w1 [E, 2I, H] and w2 [E, H, I]."""
        g = self.geom
        E, H, I, G = g.num_experts, g.hidden, g.intermediate, g.group
        given = []
        for w, name, shape in ((w1, "w1", (E, 2 * I, H)), (w2, "w2", (E, H, I))):
            if _packed(w, name, _BF16, shape, self.out.get_device()) is None:
                raise ValueError("%s must be given" % name)
            codes = torch.empty(shape[:2] + (shape[2] // 2,), dtype=torch.uint8, device=w.device)
            scales = torch.empty(shape[:2] + (shape[2] // G,), dtype=torch.bfloat16, device=w.device)
            moe_quantize_w4(w, G, codes, scales)
            given += [codes, scales]
        self.set_weights(*given)

    def forward(self, x, topk_ids, topk_weights, stream=None):
        if self.weights is None:
            raise RuntimeError("set_weights() has not been called")
        g = self.geom
        _typed(x, "x", _BF16)
        T, dev = x.shape[0] if x.dim() else 0, self.out.get_device()
        if T > self.max_tokens:
            raise ValueError("x: %d tokens, at most %d" % (T, self.max_tokens))
        px = _packed(x, "x", _BF16, (T, g.hidden), dev)
        pi = _packed(topk_ids, "topk_ids", _IDS, (T, g.top_k), dev)
        pw = _packed(topk_weights, "topk_weights", _F32, (T, g.top_k), dev)
        if pi is None or pw is None:
            raise ValueError("topk_ids and topk_weights must be given")
        if T != self.max_tokens:
            g = make_w4_geom(T, g.hidden, g.num_experts, g.top_k, g.intermediate, g.group)
        _call(_lib().moe_forward_w4(g, px, pi, _IDS[topk_ids.dtype], pw, *self._addresses, *self._buffers,
                                    _stream(stream, dev)), "moe_forward_w4")
        return self.out if T == self.max_tokens else self.out[:T]

    def status(self):
        """MOE_STATUS_* bits of the last forward (synchronises)."""
        return int(self.status_word.item())
