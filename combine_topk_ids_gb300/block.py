"""Python binding of the operators around the expert layer (include/moe_block.h).

moe_add_rmsnorm / moe_add_rmsnorm_backward, moe_route_topk / moe_route_topk_backward and the
4-bit expert FFN: moe_quantize_w4, moe_prepare_weights_w4, moe_forward_w4 and MoELayerW4,
which owns one layer's weights and buffers.  Argument checks and marshalling only; results
go to the caller's tensors, on the current stream or the one given.

A row matrix may have any row stride (its columns are packed); every other tensor is
contiguous.  A tensor of another type raises TypeError, one of another shape, layout or
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


def _packed(t, name, dtypes, shape):
    """The address of a contiguous tensor of one of `dtypes` and of `shape`; None stays None."""
    if t is None:
        return None
    _typed(t, name, dtypes)
    if t.shape != shape:
        raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _rows(t, name, dtypes, shape):
    """(address, row stride) of a matrix with packed columns."""
    if t is None:
        return None, 0
    _typed(t, name, dtypes)
    if t.shape != shape:
        raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    row, col = t.stride()
    if (col != 1 and shape[1] > 1) or (row < shape[1] and shape[0] > 1):
        raise ValueError("%s: strides %s; rows may lie apart, but not overlap, and columns are packed"
                         % (name, t.stride()))
    return t.data_ptr(), row if shape[0] > 1 else 0


def _launch(stream, tensors):
    """The stream's handle, after a look that every tensor is on its device."""
    s = torch.cuda.current_stream() if stream is None else stream
    dev = s.device_index
    for name, t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("%s is on %s; expected cuda:%d" % (name, t.device, dev))
    return s.cuda_stream


_BF16, _F32, _ROW = (torch.bfloat16,), (torch.float32,), (torch.bfloat16, torch.float32)


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
    shape = x.shape
    T, H = shape
    n = MoeNorm(T, H, 0, 0, eps)
    px, n.x_stride = _rows(x, "x", _BF16, shape)
    pr, n.residual_stride = _rows(residual, "residual", _ROW, shape)
    ps, n.sum_stride = _rows(sum_out, "sum_out", _ROW if residual is None else (residual.dtype,), shape)
    po, n.out_stride = _rows(out, "out", _BF16, shape)
    pq = _packed(out_fp8, "out_fp8", (torch.float8_e4m3fn, torch.uint8), shape)
    pc = _packed(scales, "scales", _F32, (T, H // 128))
    pw = _packed(weight, "weight", _ROW, (H,))
    pd = _packed(rstd, "rstd", _F32, (T,))
    if pw is None or (out is None and out_fp8 is None) or (out_fp8 is None) != (scales is None):
        raise ValueError("weight, and out or out_fp8 with scales, must be given")
    stream_of = residual if residual is not None else sum_out
    n.residual_dtype = 0 if stream_of is None else DTYPE[stream_of.dtype]
    n.weight_dtype = DTYPE[weight.dtype]
    s = _launch(stream, (("x", x), ("residual", residual), ("weight", weight), ("sum_out", sum_out), ("out", out),
                         ("out_fp8", out_fp8), ("scales", scales), ("rstd", rstd)))
    _call(_lib().moe_add_rmsnorm(n, px, pr, pw, ps, po, pq, pc, pd, s), "moe_add_rmsnorm")


def moe_add_rmsnorm_workspace_size(tokens, hidden):
    """Bytes of the workspace of moe_add_rmsnorm_backward."""
    size = ctypes.c_size_t()
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
    shape = dout.shape
    T, H = shape
    _typed(h, "h", _ROW)
    n = MoeNorm(T, H, DTYPE[h.dtype], 0, 0.0)
    pg, n.x_stride = _rows(dout, "dout", _BF16, shape)
    ph, n.residual_stride = _rows(h, "h", _ROW, shape)
    ps, n.sum_stride = _rows(dsum, "dsum", (h.dtype,), shape)
    px, n.out_stride = _rows(dx, "dx", (h.dtype,), shape)
    pw = _packed(weight, "weight", _ROW, (H,))
    pr = _packed(rstd, "rstd", _F32, (T,))
    pd = _packed(dweight, "dweight", _F32, (H,))
    _typed(workspace, "workspace", (torch.uint8,))
    if None in (pw, pr, pd, px) or not workspace.is_contiguous():
        raise ValueError("weight, rstd, dx, dweight and a contiguous workspace must be given")
    n.weight_dtype = DTYPE[weight.dtype]
    s = _launch(stream, (("dout", dout), ("h", h), ("weight", weight), ("rstd", rstd), ("dsum", dsum), ("dx", dx),
                         ("dweight", dweight), ("workspace", workspace)))
    _call(_lib().moe_add_rmsnorm_backward(n, pg, ph, pw, pr, ps, px, pd, workspace.data_ptr(), workspace.numel(), s),
          "moe_add_rmsnorm_backward")


def make_router(num_experts, top_k, score="softmax", groups=1, top_groups=None, group_score="max",
                renormalize=True, scale=1.0):
    """The router's rule.  score: "softmax" or "sigmoid"; groups: equal runs of experts, of which
    the top_groups best (all by default) take part, by their largest key ("max") or the sum of
    their two largest ("top2"); renormalize: the picked scores are divided by their sum."""
    return MoeRouter(num_experts, top_k, SCORE[score], groups, groups if top_groups is None else top_groups,
                     GROUP_SCORE[group_score], int(renormalize), 0, scale, 0)


def _route(r, logits):
    _typed(logits, "logits", _ROW)
    if logits.dim() != 2 or logits.shape[1] != r.num_experts:
        raise ValueError("logits: shape %s, expected [tokens, %d]" % (tuple(logits.shape), r.num_experts))
    p, stride = _rows(logits, "logits", _ROW, logits.shape)
    rule = MoeRouter.from_buffer_copy(r)   # the caller's rule stays as it is
    rule.logits_dtype, rule.logits_stride = DTYPE[logits.dtype], stride
    return rule, p, logits.shape[0]


def moe_route_topk(r, logits, bias, topk_ids, topk_weights, stream=None):
    """Expert ids (int32 or int64 [T, k], -1 where no expert is left) and routing weights
    (float32 [T, k]) from the gate's logits (bf16 or float32 [T, E]) by the rule `r`
    (make_router).  bias: float32 [E], added to the scores for the picking alone, or None."""
    rule, pl, T = _route(r, logits)
    pb = _packed(bias, "bias", _F32, (r.num_experts,))
    pi = _packed(topk_ids, "topk_ids", tuple(_IDS), (T, r.top_k))
    pw = _packed(topk_weights, "topk_weights", _F32, (T, r.top_k))
    if pi is None or pw is None:
        raise ValueError("topk_ids and topk_weights must be given")
    s = _launch(stream, (("logits", logits), ("bias", bias), ("topk_ids", topk_ids), ("topk_weights", topk_weights)))
    _call(_lib().moe_route_topk(rule, T, pl, pb, pi, _IDS[topk_ids.dtype], pw, s), "moe_route_topk")


def moe_route_topk_backward(r, logits, topk_ids, dweights, dlogits, stream=None):
    """dlogits (contiguous, of the logits' type) from dweights, the picks held fixed."""
    rule, pl, T = _route(r, logits)
    pi = _packed(topk_ids, "topk_ids", tuple(_IDS), (T, r.top_k))
    pw = _packed(dweights, "dweights", _F32, (T, r.top_k))
    pd = _packed(dlogits, "dlogits", (logits.dtype,), logits.shape)
    if None in (pi, pw, pd):
        raise ValueError("topk_ids, dweights and dlogits must be given")
    s = _launch(stream, (("logits", logits), ("topk_ids", topk_ids), ("dweights", dweights), ("dlogits", dlogits)))
    _call(_lib().moe_route_topk_backward(rule, T, pl, pi, _IDS[topk_ids.dtype], pw, pd, s),
          "moe_route_topk_backward")


def moe_quantize_w4(w, group, codes, scales, stream=None):
    """bf16 w [..., cols] to 4-bit codes (uint8 [..., cols / 2], the even column in the low half)
    and bf16 scales [..., cols / group]; a weight is (code - 8) * scale."""
    _typed(w, "w", _BF16)
    if w.dim() < 1 or group not in (32, 64, 128) or w.shape[-1] % group:
        raise ValueError("w: shape %s, expected whole groups of 32, 64 or 128 columns" % (tuple(w.shape),))
    cols = w.shape[-1]
    pw = _packed(w, "w", _BF16, w.shape)
    pc = _packed(codes, "codes", (torch.uint8,), w.shape[:-1] + (cols // 2,))
    ps = _packed(scales, "scales", _BF16, w.shape[:-1] + (cols // group,))
    if pc is None or ps is None:
        raise ValueError("codes and scales must be given")
    s = _launch(stream, (("w", w), ("codes", codes), ("scales", scales)))
    _call(_lib().moe_quantize_w4(w.numel() // max(cols, 1), cols, group, pw, pc, ps, s), "moe_quantize_w4")


def make_w4_geom(tokens, hidden, experts, k, intermediate, group):
    return MoeW4Geom(tokens, hidden, experts, k, intermediate, group)


def moe_forward_w4_workspace_size(g):
    size = ctypes.c_size_t()
    _call(_lib().moe_forward_w4_workspace_size(g, ctypes.byref(size)), "moe_forward_w4_workspace_size")
    return size.value


class MoELayerW4:
    """The routed experts of one layer with 4-bit weights, for batches of up to `max_tokens`.

    forward(x, topk_ids, topk_weights) -> out [T, H] bf16, the function of MoELayer1GPU.forward,
    on the current stream and with no host synchronisation.  group: inputs per scale (32, 64
    or 128).  The buffers (out among them) are the layer's own and are written by every call.
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

    def set_weights(self, w1, s1, w2, s2):
        """Codes w1 uint8 [E, 2I, H / 2] (gate rows, then up rows) and w2 [E, H, I / 2] with bf16
        scales s1 [E, 2I, H / group] and s2 [E, H, I / group]; put in the kernels' order once here."""
        g = self.geom
        E, H, I, G = g.num_experts, g.hidden, g.intermediate, g.group
        given = [(w1, "w1", (torch.uint8,), (E, 2 * I, H // 2)), (s1, "s1", _BF16, (E, 2 * I, H // G)),
                 (w2, "w2", (torch.uint8,), (E, H, I // 2)), (s2, "s2", _BF16, (E, H, I // G))]
        for t, name, dtypes, shape in given:
            if _packed(t, name, dtypes, shape) is None:
                raise ValueError("%s must be given" % name)
        s = _launch(None, [(name, t) for t, name, _, _ in given])
        self.weights = [torch.empty_like(t) for t, _, _, _ in given]
        self._addresses = [t.data_ptr() for t in self.weights]
        _call(_lib().moe_prepare_weights_w4(g, *(t.data_ptr() for t, _, _, _ in given), *self._addresses, s),
              "moe_prepare_weights_w4")

    def quantize_weights(self, w1, w2):
        """set_weights from bf16 w1 [E, 2I, H] and w2 [E, H, I]."""
        g = self.geom
        E, H, I, G = g.num_experts, g.hidden, g.intermediate, g.group
        given = []
        for w, name, shape in ((w1, "w1", (E, 2 * I, H)), (w2, "w2", (E, H, I))):
            if _packed(w, name, _BF16, shape) is None:
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
        T = x.shape[0] if x.dim() else 0
        if T > self.max_tokens:
            raise ValueError("x: %d tokens, at most %d" % (T, self.max_tokens))
        px = _packed(x, "x", _BF16, (T, g.hidden))
        pi = _packed(topk_ids, "topk_ids", tuple(_IDS), (T, g.top_k))
        pw = _packed(topk_weights, "topk_weights", _F32, (T, g.top_k))
        if pi is None or pw is None:
            raise ValueError("topk_ids and topk_weights must be given")
        s = _launch(stream, (("x", x), ("topk_ids", topk_ids), ("topk_weights", topk_weights), ("the layer", self.out)))
        call = g if T == self.max_tokens else make_w4_geom(T, g.hidden, g.num_experts, g.top_k, g.intermediate, g.group)
        _call(_lib().moe_forward_w4(call, px, pi, _IDS[topk_ids.dtype], pw, *self._addresses, self.out.data_ptr(),
                                    self.status_word.data_ptr(), self.workspace.data_ptr(), self.workspace.numel(), s),
              "moe_forward_w4")
        return self.out if T == self.max_tokens else self.out[:T]

    def status(self):
        """MOE_STATUS_* bits of the last forward (synchronises)."""
        return int(self.status_word.item())
