"""Python binding of libmoe (include/moe.h): argument marshalling only.

Each function has the name of the C entry point it calls and takes plain
integers for device pointers and streams.  Every step of the layer runs in
the HIP kernels of libmoe; there is no other implementation to fall back to,
so a missing library raises instead of computing anything.

`Layer` is a convenience owner of one plan plus a workspace tensor allocated
with torch (PyTorch supplies device memory and streams, nothing else).
"""
from __future__ import annotations

import ctypes
import math
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_STATE = -4
MOE_ERR_HIP = -5
MOE_ERR_ROUTING = -6
MOE_ERR_TOO_LARGE = -7
MOE_STATIC_SCRATCH_BYTES = 32 << 20

MOE_BF16 = 0
MOE_MXFP8_E4M3 = 1
MOE_MXFP4 = 2
MOE_FP8_BLOCK128 = 3

MOE_PATH_AUTO = 0
MOE_PATH_PREFILL = 1
MOE_PATH_DECODE = 2

MOE_DEV_ID_OUT_OF_RANGE = 1
MOE_DEV_ID_DUPLICATE = 2
MOE_DEV_BAD_INDPTR = 4
MOE_ACT_SWIGLU, MOE_ACT_GEGLU, MOE_ACT_REGLU = 0, 1, 2
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN = 0, 1, 2

# every symbol include/moe.h declares
EXPORTS = ("moe_plan", "moe_workspace_bytes", "moe_bind_workspace", "moe_plan_destroy",
           "moe_dispatch", "moe_quantize_mxfp8", "moe_prepare_weights", "moe_prepare_weights_backward",
           "moe_forward", "moe_forward_static",
           "moe_forward_routed",
           "moe_backward", "moe_get_status", "moe_status_string", "moe_profile", "moe_plan_explain",
           "moe_profile_read", "moe_expand_weights",
           "moe_router_workspace_bytes", "moe_router_forward", "moe_router_backward",
           "moe_norm_workspace_bytes", "moe_norm_forward", "moe_norm_backward",
           "moe_quantize_block128", "moe_product_workspace_bytes", "moe_product_prepare_weights",
           "moe_product_expand_weights", "moe_product_forward", "moe_product_backward")

STAGES = ("dispatch", "quant_x", "w13", "w2", "combine", "score_grad", "dgrad_w2", "wgrad_w2",
          "dgrad_w13", "wgrad_w13", "dx_combine", "decode_w13", "decode_w2", "wgrad_rows", "recompute_h",
          "mega", "quant_do", "act_bwd", "quant_t")


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (%d)" % (where, status_string(status), status))


class MoeConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("precision", ctypes.c_int32),
                ("training", ctypes.c_int32), ("path", ctypes.c_int32),
                ("wgrad_accumulate", ctypes.c_int32), ("recompute_h", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("mega", ctypes.c_int32)]


class MoeWeights(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("w13_scale", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p),
                ("w13t", ctypes.c_void_p), ("w13t_scale", ctypes.c_void_p),
                ("w2t", ctypes.c_void_p), ("w2t_scale", ctypes.c_void_p)]


class RouterConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("score", ctypes.c_int32), ("normalize", ctypes.c_int32), ("logits_f32", ctypes.c_int32),
                ("scale", ctypes.c_float), ("balance_coef", ctypes.c_float),
                ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32)]


class NormConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("residual_f32", ctypes.c_int32), ("eps", ctypes.c_float),
                ("residual_scale", ctypes.c_float)]


class ProductConfig(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("E", ctypes.c_int32),
                ("training", ctypes.c_int32), ("wgrad_accumulate", ctypes.c_int32)]


_lib = None


def lib():
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmoe.so is not built (run __graft_entry__.build()); "
                               "there is no fallback implementation")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.moe_plan.argtypes = [ctypes.POINTER(MoeConfig), ctypes.POINTER(vp)]
        L.moe_plan.restype = ctypes.c_int
        L.moe_workspace_bytes.argtypes = [vp]
        L.moe_workspace_bytes.restype = ctypes.c_size_t
        L.moe_plan_explain.argtypes = [vp, ctypes.c_char_p, ctypes.c_size_t]
        L.moe_plan_explain.restype = ctypes.c_size_t
        L.moe_bind_workspace.argtypes = [vp, vp, ctypes.c_size_t]
        L.moe_bind_workspace.restype = ctypes.c_int
        L.moe_plan_destroy.argtypes = [vp]
        L.moe_plan_destroy.restype = ctypes.c_int
        L.moe_dispatch.argtypes = [vp] * 8
        L.moe_dispatch.restype = ctypes.c_int
        L.moe_quantize_mxfp8.argtypes = [vp, i64, i32, vp, vp, vp]
        L.moe_quantize_mxfp8.restype = ctypes.c_int
        L.moe_prepare_weights.argtypes = [vp] * 8
        L.moe_prepare_weights_backward.argtypes = [vp] * 8
        L.moe_prepare_weights_backward.restype = ctypes.c_int
        L.moe_prepare_weights.restype = ctypes.c_int
        L.moe_forward.argtypes = [vp, vp, vp, vp, ctypes.POINTER(MoeWeights), vp, vp]
        L.moe_forward.restype = ctypes.c_int
        L.moe_forward_static.argtypes = [vp, vp, vp, vp, ctypes.POINTER(MoeWeights), vp, vp]
        L.moe_forward_static.restype = ctypes.c_int
        L.moe_forward_routed.argtypes = [vp, vp, vp, ctypes.POINTER(MoeWeights), vp, vp]
        L.moe_forward_routed.restype = ctypes.c_int
        L.moe_backward.argtypes = [vp, vp, vp, ctypes.POINTER(MoeWeights), vp, vp, vp, vp, vp]
        L.moe_backward.restype = ctypes.c_int
        L.moe_expand_weights.argtypes = [vp, ctypes.POINTER(MoeWeights), vp, vp, vp]
        L.moe_expand_weights.restype = ctypes.c_int
        sz, router, norm = ctypes.c_size_t, ctypes.POINTER(RouterConfig), ctypes.POINTER(NormConfig)
        L.moe_router_workspace_bytes.argtypes = [router]
        L.moe_router_workspace_bytes.restype = sz
        L.moe_router_forward.argtypes = [router] + [vp] * 9 + [sz, vp]
        L.moe_router_forward.restype = ctypes.c_int
        L.moe_router_backward.argtypes = [router] + [vp] * 8
        L.moe_router_backward.restype = ctypes.c_int
        L.moe_norm_workspace_bytes.argtypes = [norm]
        L.moe_norm_workspace_bytes.restype = sz
        L.moe_norm_forward.argtypes = [norm] + [vp] * 8
        L.moe_norm_forward.restype = ctypes.c_int
        L.moe_norm_backward.argtypes = [norm] + [vp] * 13 + [sz, vp]
        L.moe_norm_backward.restype = ctypes.c_int
        product = ctypes.POINTER(ProductConfig)
        L.moe_quantize_block128.argtypes = [vp, i64, i32, vp, vp, vp]
        L.moe_quantize_block128.restype = ctypes.c_int
        L.moe_product_workspace_bytes.argtypes = [product]
        L.moe_product_workspace_bytes.restype = sz
        L.moe_product_prepare_weights.argtypes = [product] + [vp] * 4
        L.moe_product_prepare_weights.restype = ctypes.c_int
        L.moe_product_expand_weights.argtypes = [product] + [vp] * 4
        L.moe_product_expand_weights.restype = ctypes.c_int
        L.moe_product_forward.argtypes = [product] + [vp] * 7 + [sz, vp]
        L.moe_product_forward.restype = ctypes.c_int
        L.moe_product_backward.argtypes = [product] + [vp] * 9 + [sz, vp]
        L.moe_product_backward.restype = ctypes.c_int
        L.moe_get_status.argtypes = [vp, ctypes.POINTER(i32), i32, vp]
        L.moe_get_status.restype = ctypes.c_int
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_profile.argtypes = [vp, i32]
        L.moe_profile.restype = ctypes.c_int
        L.moe_profile_read.argtypes = [vp, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(i32), i32]
        L.moe_profile_read.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().moe_status_string(int(status)).decode()
    except Exception:  # library not loadable: describe the code ourselves
        return "status %d" % status


def _ok(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def moe_plan(T, d, I, E, k, precision=MOE_BF16, training=0, path=MOE_PATH_AUTO,
             wgrad_accumulate=0, recompute_h=0, activation=MOE_ACT_SWIGLU, mega=0) -> int:
    cfg = MoeConfig(T, d, I, E, k, precision, training, path, wgrad_accumulate, recompute_h, activation, mega)
    h = ctypes.c_void_p()
    _ok(lib().moe_plan(ctypes.byref(cfg), ctypes.byref(h)), "moe_plan")
    return h.value


def moe_workspace_bytes(plan: int) -> int:
    return int(lib().moe_workspace_bytes(plan))


def moe_plan_explain(plan: int) -> str:
    n = int(lib().moe_plan_explain(plan, None, 0))
    buf = ctypes.create_string_buffer(n + 1)
    lib().moe_plan_explain(plan, buf, n + 1)
    return buf.value.decode()


def moe_bind_workspace(plan: int, ptr: int, nbytes: int):
    _ok(lib().moe_bind_workspace(plan, ptr, nbytes), "moe_bind_workspace")


def moe_plan_destroy(plan: int):
    _ok(lib().moe_plan_destroy(plan), "moe_plan_destroy")


def moe_dispatch(plan, ids, scores, m_indptr, gather, slots, probs, stream=0):
    _ok(lib().moe_dispatch(plan, ids, scores, m_indptr, gather, slots, probs, stream), "moe_dispatch")


def moe_quantize_mxfp8(v, rows, K, codes, scales, stream=0):
    _ok(lib().moe_quantize_mxfp8(v, rows, K, codes, scales, stream), "moe_quantize_mxfp8")


def moe_prepare_weights(plan, w13, w2, w13_q, w13_s, w2_q, w2_s, stream=0):
    _ok(lib().moe_prepare_weights(plan, w13, w2, w13_q, w13_s, w2_q, w2_s, stream),
        "moe_prepare_weights")


def moe_prepare_weights_backward(plan, w13, w2, w13t_q, w13t_s, w2t_q, w2t_s, stream=0):
    _ok(lib().moe_prepare_weights_backward(plan, w13, w2, w13t_q, w13t_s, w2t_q, w2t_s, stream),
        "moe_prepare_weights_backward")


def weights(w13, w2, w13_scale=0, w2_scale=0, w13t=0, w13t_scale=0, w2t=0, w2t_scale=0) -> MoeWeights:
    return MoeWeights(w13, w2, w13_scale or None, w2_scale or None, w13t or None, w13t_scale or None,
                      w2t or None, w2t_scale or None)


def moe_forward(plan, x, ids, scores, w: MoeWeights, y, stream=0):
    _ok(lib().moe_forward(plan, x, ids, scores, ctypes.byref(w), y, stream), "moe_forward")


def moe_forward_static(plan, x, ids, scores, w: MoeWeights, y, stream=0):
    _ok(lib().moe_forward_static(plan, x, ids, scores, ctypes.byref(w), y, stream), "moe_forward_static")


def moe_forward_routed(plan, x_rows, m_indptr, w: MoeWeights, out, stream=0):
    _ok(lib().moe_forward_routed(plan, x_rows, m_indptr, ctypes.byref(w), out, stream),
        "moe_forward_routed")


def moe_backward(plan, dy, x, w: MoeWeights, dx, dw13, dw2, dscores, stream=0):
    _ok(lib().moe_backward(plan, dy, x, ctypes.byref(w), dx, dw13, dw2, dscores, stream),
        "moe_backward")


def moe_expand_weights(plan, w: MoeWeights, w13, w2, stream=0):
    _ok(lib().moe_expand_weights(plan, ctypes.byref(w), w13, w2, stream), "moe_expand_weights")


def moe_router_workspace_bytes(cfg: RouterConfig) -> int:
    return int(lib().moe_router_workspace_bytes(ctypes.byref(cfg)))


def moe_router_forward(cfg: RouterConfig, logits, bias, mask, ids, scores, counts, prob_sums, loss, workspace,
                       workspace_bytes, stream=0):
    _ok(lib().moe_router_forward(ctypes.byref(cfg), logits, bias, mask, ids, scores, counts, prob_sums, loss,
                                 workspace, workspace_bytes, stream), "moe_router_forward")


def moe_router_backward(cfg: RouterConfig, dscores, logits, mask, ids, counts, dloss, dlogits, stream=0):
    _ok(lib().moe_router_backward(ctypes.byref(cfg), dscores, logits, mask, ids, counts, dloss, dlogits, stream),
        "moe_router_backward")


def moe_norm_workspace_bytes(cfg: NormConfig) -> int:
    return int(lib().moe_norm_workspace_bytes(ctypes.byref(cfg)))


def moe_norm_forward(cfg: NormConfig, x, y, w_post, gate, w_pre, z, h, stream=0):
    _ok(lib().moe_norm_forward(ctypes.byref(cfg), x, y, w_post, gate, w_pre, z, h, stream), "moe_norm_forward")


def moe_norm_backward(cfg: NormConfig, dz, dh, z, y, w_post, gate, w_pre, dx, dy, dw_post, dgate, dw_pre, workspace,
                      workspace_bytes, stream=0):
    _ok(lib().moe_norm_backward(ctypes.byref(cfg), dz, dh, z, y, w_post, gate, w_pre, dx, dy, dw_post, dgate, dw_pre,
                                workspace, workspace_bytes, stream), "moe_norm_backward")


def moe_quantize_block128(v, rows, K, codes, scales, stream=0):
    _ok(lib().moe_quantize_block128(v, rows, K, codes, scales, stream), "moe_quantize_block128")


def moe_product_workspace_bytes(cfg: ProductConfig) -> int:
    return int(lib().moe_product_workspace_bytes(ctypes.byref(cfg)))


def moe_product_prepare_weights(cfg: ProductConfig, w, w_q, w_s, stream=0):
    _ok(lib().moe_product_prepare_weights(ctypes.byref(cfg), w, w_q, w_s, stream), "moe_product_prepare_weights")


def moe_product_expand_weights(cfg: ProductConfig, w_q, w_s, w, stream=0):
    _ok(lib().moe_product_expand_weights(ctypes.byref(cfg), w_q, w_s, w, stream), "moe_product_expand_weights")


def moe_product_forward(cfg: ProductConfig, x, m_indptr, w_q, w_s, y, status, workspace, workspace_bytes, stream=0):
    _ok(lib().moe_product_forward(ctypes.byref(cfg), x, m_indptr, w_q, w_s, y, status, workspace, workspace_bytes, stream),
        "moe_product_forward")


def moe_product_backward(cfg: ProductConfig, dy, x, m_indptr, w_q, w_s, dx, dw, status, workspace, workspace_bytes,
                         stream=0):
    _ok(lib().moe_product_backward(ctypes.byref(cfg), dy, x, m_indptr, w_q, w_s, dx, dw, status, workspace,
                                   workspace_bytes, stream), "moe_product_backward")


def moe_get_status(plan, clear=True, stream=0):
    """Returns (status, device_flags); synchronises the stream."""
    flags = ctypes.c_int32(0)
    st = lib().moe_get_status(plan, ctypes.byref(flags), 1 if clear else 0, stream)
    if st not in (MOE_OK, MOE_ERR_ROUTING):
        raise MoeError(st, "moe_get_status")
    return st, flags.value


def moe_profile(plan, enable: bool):
    _ok(lib().moe_profile(plan, 1 if enable else 0), "moe_profile")


def moe_profile_read(plan) -> dict:
    """{stage name: (total ms, launches)} for the stages recorded since the last read."""
    n = len(STAGES)
    ms = (ctypes.c_float * n)()
    cnt = (ctypes.c_int32 * n)()
    _ok(lib().moe_profile_read(plan, ms, cnt, n), "moe_profile_read")
    return {STAGES[i]: (float(ms[i]), int(cnt[i])) for i in range(n) if cnt[i] > 0}


# ---------------------------------------------------------------- torch plumbing

def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


_raw_stream = None


def _current_stream(index: int) -> int:
    """The current stream of device `index` as an integer (by the raw lookup where torch has
    one: 0.1 us, against 2.7 us by way of a Stream object)."""
    global _raw_stream
    import torch
    if _raw_stream is None:
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda i: torch.cuda.current_stream(i).cuda_stream)
    return int(_raw_stream(index))


def _stream(stream) -> int:
    import torch
    if stream is None:
        return _current_stream(torch.cuda.current_device())
    return int(stream.cuda_stream)


class Layer:
    """One plan plus its torch-allocated workspace; all compute goes through libmoe.  Tensors that a
    call makes come from the memory of the stream that writes them (`stream`, else the current one)."""

    _block128 = None                   # shapes of the weights' scales, with MOE_FP8_BLOCK128
    _forward_args = _routed_args = None  # and what _check_rows takes of a call's other tensors

    def __init__(self, T, d, I, E, k, precision=MOE_BF16, training=False, path=MOE_PATH_AUTO,
                 device="cuda", wgrad_accumulate=False, recompute_h=False, activation=MOE_ACT_SWIGLU,
                 mega=False):
        import torch
        self.T, self.d, self.I, self.E, self.k = T, d, I, E, k
        self.precision = precision
        self._rows = _dense(T, d)
        self.plan = moe_plan(T, d, I, E, k, precision, int(bool(training)), path,
                             int(bool(wgrad_accumulate)), int(bool(recompute_h)), int(activation),
                             int(bool(mega)))
        # shapes and strides of W13 and W2, and with MXFP4 of their (codes, scales)
        self._weights = _dense(E, 2 * I, d), _dense(E, d, I)
        self._mxfp4 = None
        if precision == MOE_MXFP4:
            self._mxfp4 = ((_dense(E, I * d), _dense(E, 2 * I // 16, (d + 511) // 512, 64, 4)),
                           (_dense(E, d * I // 2), _dense(E, d // 16, (I + 511) // 512, 64, 4)))
            self._mxfp4_sizes = tuple(math.prod(shape) for shape, _ in sum(self._mxfp4, ()))
        if precision == MOE_FP8_BLOCK128:
            self._set_block128()
        nbytes = moe_workspace_bytes(self.plan)
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        moe_bind_workspace(self.plan, _ptr(self.workspace), self.workspace.numel())

    def _set_block128(self):
        import torch
        T, d, I, E, k, bf16, i32 = self.T, self.d, self.I, self.E, self.k, torch.bfloat16, torch.int32
        self._block128 = (E, 2 * I // 128, d // 128), (E, d // 128, I // 128)
        row, per_choice = (bf16, (T, d), T * d), (T, k)
        self._forward_args = (("x", *row), ("ids", i32, per_choice, T * k), ("scores", torch.float32, per_choice, T * k),
                              ("y", *row))
        # x_rows and out may end with the last segment's rows
        rows = bf16, (T * k, d), None
        self._routed_args = ("x_rows", *rows), ("m_indptr", i32, (E + 1,), E + 1), ("out", *rows)

    def explain(self) -> str:
        return moe_plan_explain(self.plan)

    def close(self):
        if self.plan:
            moe_plan_destroy(self.plan)
            self.plan = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def dispatch(self, ids, scores, stream=None):
        import torch
        dev, i32 = ids.device, torch.int32
        R = self.T * self.k
        m_indptr = _new(_dense(self.E + 1), i32, dev, stream)
        gather = _new(_dense(max(R, 1)), i32, dev, stream)
        slots = _new(_dense(self.T, self.k), i32, dev, stream)
        probs = _new(_dense(max(R, 1)), torch.float32, dev, stream)
        moe_dispatch(self.plan, _ptr(ids), _ptr(scores), _ptr(m_indptr), _ptr(gather),
                     _ptr(slots), _ptr(probs), _stream(stream))
        return m_indptr, gather[:R], slots, probs[:R]

    def forward(self, x, ids, scores, w13, w2, w13_scale=None, w2_scale=None, y=None, stream=None):
        import torch
        if y is None:
            y = _new(self._rows, torch.bfloat16, x.device, stream)
        if self._mxfp4 is not None:
            self._check_mxfp4(w13, w13_scale, w2, w2_scale, x, ids, scores, y, stream)
        if self._block128 is not None:
            self._check_block128(w13, w13_scale, w2, w2_scale, (x, ids, scores, y), self._forward_args, stream)
        w = weights(_ptr(w13), _ptr(w2), _ptr(w13_scale), _ptr(w2_scale))
        moe_forward(self.plan, _ptr(x), _ptr(ids), _ptr(scores), w, _ptr(y), _stream(stream))
        return y

    def forward_routed(self, x_rows, m_indptr, w13, w2, w13_scale=None, w2_scale=None, out=None,
                       stream=None):
        """Expert outputs of rows already in expert order (int32 m_indptr [E+1] on the
        device); out BF16 [T*k, d], of which rows m_indptr[E].. are not written.  MXFP8
        plans take the prepared weights and their scales."""
        import torch
        if out is None:
            out = _new(_dense(self.T * self.k, self.d), torch.bfloat16, x_rows.device, stream)
        if self._mxfp4 is not None:
            self._check_mxfp4(w13, w13_scale, w2, w2_scale, x_rows, m_indptr, out, out, stream)
        if self._block128 is not None:
            self._check_block128(w13, w13_scale, w2, w2_scale, (x_rows, m_indptr, out), self._routed_args, stream)
        w = weights(_ptr(w13), _ptr(w2), _ptr(w13_scale), _ptr(w2_scale))
        moe_forward_routed(self.plan, _ptr(x_rows), _ptr(m_indptr), w, _ptr(out), _stream(stream))
        return out

    def backward(self, dy, x, w13, w2, dx=None, dw13=None, dw2=None, dscores=None, stream=None,
                 w13_scale=None, w13t=None, w13t_scale=None, w2t=None, w2t_scale=None):
        """BF16 plans take the BF16 weights; MXFP8 plans the tensors of
        prepare_weights_backward (w13t, w13t_scale, w2t, w2t_scale) and, with
        recompute_h, the forward's prepared w13 and w13_scale (w2 unused)."""
        import torch
        dev = dy.device
        if dx is None:
            dx = _new(self._rows, torch.bfloat16, dev, stream)
        if dw13 is None:
            dw13 = _new(self._weights[0], torch.bfloat16, dev, stream)
        if dw2 is None:
            dw2 = _new(self._weights[1], torch.bfloat16, dev, stream)
        if dscores is None:
            dscores = _new(_dense(self.T, self.k), torch.float32, dev, stream)
        w = weights(_ptr(w13), _ptr(w2), _ptr(w13_scale), 0, _ptr(w13t), _ptr(w13t_scale), _ptr(w2t),
                    _ptr(w2t_scale))
        moe_backward(self.plan, _ptr(dy), _ptr(x), w, _ptr(dx), _ptr(dw13), _ptr(dw2), _ptr(dscores),
                     _stream(stream))
        return dx, dw13, dw2, dscores

    def prepare_weights(self, w13, w2, stream=None):
        """BF16 weights -> (w13_q, w13_s, w2_q, w2_s): MXFP8 codes and scales, or on an
        MXFP4 layer MXFP4 ones in the decode kernels' tile layout, or with MOE_FP8_BLOCK128 codes and the
        FP32 scales of their 128 x 128 squares."""
        import torch
        dev = w13.device
        E, I, d = self.E, self.I, self.d
        if self.precision == MOE_MXFP4:
            n13, n2 = self._mxfp4
            dev = torch.device("cuda", torch.cuda.current_device())
            if stream is not None:
                _check_stream(stream, dev.index)
            _check("w13", w13, (E, 2 * I, d), torch.bfloat16, dev)
            _check("w2", w2, (E, d, I), torch.bfloat16, dev)
            w13_q, w13_s, w2_q, w2_s = (_new(n, torch.uint8, dev, stream) for n in n13 + n2)
            moe_prepare_weights(self.plan, w13.data_ptr(), w2.data_ptr(), w13_q.data_ptr(), w13_s.data_ptr(),
                                w2_q.data_ptr(), w2_s.data_ptr(), _stream(stream))
            return w13_q, w13_s, w2_q, w2_s
        if self._block128 is not None:
            dev = torch.device("cuda", torch.cuda.current_device())
            if stream is not None:
                _check_stream(stream, dev.index)
            _check("w13", w13, (E, 2 * I, d), torch.bfloat16, dev)
            _check("w2", w2, (E, d, I), torch.bfloat16, dev)
            w13_q, w2_q = (_new(n, torch.uint8, dev, stream) for n in self._weights)
            w13_s, w2_s = (_new(_dense(*n), torch.float32, dev, stream) for n in self._block128)
            moe_prepare_weights(self.plan, w13.data_ptr(), w2.data_ptr(), w13_q.data_ptr(), w13_s.data_ptr(),
                                w2_q.data_ptr(), w2_s.data_ptr(), _stream(stream))
            return w13_q, w13_s, w2_q, w2_s
        w13_q = _new(self._weights[0], torch.uint8, dev, stream)
        # scales block-major: [K/128, rows, 4] (see moe_prepare_weights in include/moe.h)
        w13_s = _new(_dense(d // 128, E * 2 * I, 4), torch.uint8, dev, stream)
        w2_q = _new(self._weights[1], torch.uint8, dev, stream)
        w2_s = _new(_dense(I // 128, E * d, 4), torch.uint8, dev, stream)
        moe_prepare_weights(self.plan, _ptr(w13), _ptr(w2), _ptr(w13_q), _ptr(w13_s), _ptr(w2_q),
                            _ptr(w2_s), _stream(stream))
        return w13_q, w13_s, w2_q, w2_s

    def _check_mxfp4(self, w13_q, w13_s, w2_q, w2_s, a, b, c, d, stream):
        """Prepared weights of this layer's sizes, they, the four other tensors and the stream on the
        current device, or ValueError (a missing tensor is left to the call, which refuses it): the
        kernels address them by the plan's sizes."""
        import torch
        index = torch.cuda.current_device()
        if stream is not None:
            _check_stream(stream, index)
        try:
            if ((w13_q.numel(), w13_s.numel(), w2_q.numel(), w2_s.numel()) == self._mxfp4_sizes
                    and w13_q.is_contiguous() and w13_s.is_contiguous() and w2_q.is_contiguous() and w2_s.is_contiguous()
                    and index == w13_q.get_device() == w13_s.get_device() == w2_q.get_device() == w2_s.get_device()
                    == a.get_device() == b.get_device() == c.get_device() == d.get_device()):
                return
        except AttributeError:
            return
        dev, layout = torch.device("cuda", index), sum(self._mxfp4, ())
        for name, t, (shape, _) in zip(("w13_q", "w13_s", "w2_q", "w2_s"), (w13_q, w13_s, w2_q, w2_s), layout):
            _check(name, t, shape, torch.uint8, dev)
        raise ValueError("the current device is %s; x, ids, scores or the output is elsewhere" % dev)

    def _check_block128(self, w13_q, w13_s, w2_q, w2_s, others, args, stream):
        """Codes and scales of this layer's sizes, the other tensors as args says, they and the stream on the
        current device, or ValueError (a missing tensor is left to the call, which refuses it)."""
        import torch
        index = torch.cuda.current_device()
        if stream is not None:
            _check_stream(stream, index)
        if w13_q is None or w13_s is None or w2_q is None or w2_s is None:
            return
        (n13, n2), (s13, s2) = self._weights, self._block128
        if not (w13_q.shape == n13[0] and w2_q.shape == n2[0] and w13_s.shape == s13 and w2_s.shape == s2
                and w13_q.dtype in _codes8() and w2_q.dtype in _codes8()
                and w13_s.dtype is torch.float32 and w2_s.dtype is torch.float32
                and w13_q.is_contiguous() and w2_q.is_contiguous() and w13_s.is_contiguous() and w2_s.is_contiguous()
                and index == w13_q.get_device() == w2_q.get_device() == w13_s.get_device() == w2_s.get_device()):
            dev = torch.device("cuda", index)
            _check_codes("w13_q", w13_q, n13[0], dev)
            _check("w13_s", w13_s, s13, torch.float32, dev)
            _check_codes("w2_q", w2_q, n2[0], dev)
            _check("w2_s", w2_s, s2, torch.float32, dev)
        for t, arg in zip(others, args or _no_args):
            if t is not None:
                if t.get_device() != index:
                    raise ValueError("the current device is cuda:%d; x, ids, scores or the output is elsewhere" % index)
                if arg is not None and not (t.dtype is arg[1] and t.shape == arg[2] and t.is_contiguous()):
                    _check_rows(t, *arg)

    def expand_weights(self, w13_q, w13_s, w2_q, w2_s, stream=None):
        """The BF16 weights (w13, w2) that the prepared weights of an MXFP4 or MOE_FP8_BLOCK128 layer
        stand for."""
        import torch
        if self._block128 is not None:
            self._check_block128(w13_q, w13_s, w2_q, w2_s, (), None, stream)
        if self._mxfp4 is not None:
            self._check_mxfp4(w13_q, w13_s, w2_q, w2_s, w13_q, w13_s, w2_q, w2_s, stream)
        w13, w2 = (_new(n, torch.bfloat16, w13_q.device, stream) for n in self._weights)
        w = weights(_ptr(w13_q), _ptr(w2_q), _ptr(w13_s), _ptr(w2_s))
        moe_expand_weights(self.plan, w, _ptr(w13), _ptr(w2), _stream(stream))
        return w13, w2

    def prepare_weights_backward(self, w13, w2, stream=None):
        """(w13t, w13t_scale, w2t, w2t_scale) for the MXFP8 backward: W13_e^T [d, 2I] and
        W2_e^T [I, d] quantized along their last dimension, scales block-major."""
        import torch
        dev = w13.device
        E, I, d = self.E, self.I, self.d
        w13t = _new(_dense(E, d, 2 * I), torch.uint8, dev, stream)
        w13t_s = _new(_dense(2 * I // 128, E * d, 4), torch.uint8, dev, stream)
        w2t = _new(_dense(E, I, d), torch.uint8, dev, stream)
        w2t_s = _new(_dense(d // 128, E * I, 4), torch.uint8, dev, stream)
        moe_prepare_weights_backward(self.plan, _ptr(w13), _ptr(w2), _ptr(w13t), _ptr(w13t_s), _ptr(w2t),
                                     _ptr(w2t_s), _stream(stream))
        return w13t, w13t_s, w2t, w2t_s

    def status(self, clear=True, stream=None):
        return moe_get_status(self.plan, clear, _stream(stream))


# ---------------------------------------------------------------- around the layer

def _dense(*shape):
    """(shape, strides) of a row-major tensor."""
    strides, n = [], 1
    for size in reversed(shape):
        strides.append(n)
        n *= max(size, 1)
    return shape, tuple(reversed(strides))


def _new(rows, dtype, device, stream=None):
    """An uninitialised tensor of _dense's shape and strides (1.2 us a call, torch.empty 1.6), from the
    memory of `stream` where it is given: a block of the current stream's may still be in use there by
    work that was enqueued before its last owner let it go, and `stream` does not wait for that."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return torch.empty_strided(*rows, dtype=dtype, device=device)
    return torch.empty_strided(*rows, dtype=dtype, device=device)


def _check_stream(stream, index):
    """A stream of device `index`, or ValueError."""
    if stream.device.index != index:
        raise ValueError("a stream of cuda:%d is needed, got one of %s" % (index, stream.device))


def _check(name, t, shape, dtype, device):
    """A dense tensor of this shape and type on this device, or ValueError."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    raise ValueError("%s: a contiguous %s tensor of shape %s on %s is needed, got %s %s on %s%s" % (
        name, dtype, tuple(shape), device, t.dtype, tuple(t.shape), t.device,
        "" if t.is_contiguous() else ", not contiguous"))


_no_args = (None,) * 4


def _check_rows(t, name, dtype, shape, numel):
    """A dense tensor of this type, of rows as long as the shape's (or flat), `numel` elements in all unless that is
    None, or ValueError: the kernels address it by the plan's sizes."""
    if (t.dtype is dtype and t.is_contiguous() and (numel is None or t.numel() == numel)
            and (t.dim() == 1 or t.shape[-1:] == shape[-1:])):
        return
    raise ValueError("%s: a contiguous %s tensor of shape %s is needed, got %s %s%s" % (
        name, dtype, shape, t.dtype, tuple(t.shape), "" if t.is_contiguous() else ", not contiguous"))


_codes = None


def _codes8():
    """The types that hold E4M3 codes."""
    global _codes
    if _codes is None:
        import torch
        _codes = torch.uint8, torch.float8_e4m3fn
    return _codes


def _check_codes(name, t, shape, device):
    """_check for E4M3 codes."""
    import torch
    _check(name, t, shape, t.dtype if t.dtype in _codes8() else torch.uint8, device)


class _OnDevice:
    """What Router, BlockNorm and Product share: their device, a workspace there, and calls made with
    that device current and their outputs allocated on the stream that writes them.  The workspace
    belongs to the stream that the object was made on.  Calls on other streams, and captured ones, take
    one of their own from their stream's (the graph's) memory, so that calls of one object may overlap."""

    def __init__(self, device, workspace_bytes):
        import torch
        device = torch.device(device)
        if device.index is None:
            device = torch.device(device.type, torch.cuda.current_device())
        self.device, self._index = device, device.index
        self._workspace_bytes = max(workspace_bytes, 16)
        with torch.cuda.device(device):
            self.workspace = torch.empty(self._workspace_bytes, dtype=torch.uint8, device=device)
            # a graph's memory is not kept for other calls: no stream is the object's own then
            self._own = None if torch.cuda.is_current_stream_capturing() else _current_stream(self._index)

    def _room(self, s):
        """The workspace of a call on raw stream s.  (0, the default stream, is never captured.)"""
        import torch
        if s == self._own and not (s and torch.cuda.is_current_stream_capturing()):
            return self.workspace
        return torch.empty(self._workspace_bytes, dtype=torch.uint8, device=self.device)

    def _call(self, f, stream, *args):
        """f(raw stream, *args) with this object's device current and `stream` its current stream."""
        import torch
        if stream is not None:
            _check_stream(stream, self._index)
            with torch.cuda.stream(stream):            # also makes the stream's device current
                return f(int(stream.cuda_stream), *args)
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self.device):
                return f(_current_stream(self._index), *args)
        return f(_current_stream(self._index), *args)


class Router(_OnDevice):
    """Logits [T, E] (FP32 or BF16) -> ids, scores, per-expert counts and the balance loss, and
    the gradient; see the router section of include/moe.h for the formulas.  With groups, only experts of
    the top_groups groups whose group_top largest keys have the largest sum are chosen."""

    def __init__(self, T, E, k, score=MOE_SCORE_SOFTMAX, normalize=True, scale=1.0, balance_coef=0.0, device="cuda",
                 groups=0, top_groups=0, group_top=0):
        self.T, self.E, self.k = T, E, k
        self._per_choice, self._per_expert = _dense(T, k), _dense(E)
        self._cfg = {f32: RouterConfig(T, E, k, int(score), int(bool(normalize)), int(f32), scale, balance_coef,
                                       int(groups), int(top_groups), int(group_top))
                     for f32 in (False, True)}
        nbytes = moe_router_workspace_bytes(self._cfg[True])
        if not nbytes:                                 # the reason, from the call that names it
            moe_router_forward(self._cfg[True], 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
        super().__init__(device, nbytes)

    def _logits_cfg(self, logits):
        import torch
        f32 = logits.dtype == torch.float32
        _check("logits", logits, (self.T, self.E), torch.float32 if f32 else torch.bfloat16, self.device)
        return self._cfg[f32]

    def _check_mask(self, mask):
        import torch
        if mask is not None:
            _check("mask", mask, (self.T,), torch.bool if mask.dtype == torch.bool else torch.uint8, self.device)

    def forward(self, logits, bias=None, mask=None, stats=True, stream=None):
        """(ids int32 [T, k], scores f32 [T, k], counts int32 [E], prob_sums f32 [E], loss f32 []);
        without `stats` the last three are None and not computed."""
        import torch
        cfg = self._logits_cfg(logits)
        if bias is not None:
            _check("bias", bias, (self.E,), torch.float32, self.device)
        self._check_mask(mask)

        return self._call(self._forward, stream, cfg, logits, bias, mask, stats)

    def _forward(self, s, cfg, logits, bias, mask, stats):
        import torch
        dev, f32, i32 = self.device, torch.float32, torch.int32
        ids, scores = _new(self._per_choice, i32, dev), _new(self._per_choice, f32, dev)
        counts = sums = loss = room = None
        if stats:
            room = self._room(s)
            counts, sums = _new(self._per_expert, i32, dev), _new(self._per_expert, f32, dev)
            loss = _new(((), ()), f32, dev)
        moe_router_forward(cfg, logits.data_ptr(), _ptr(bias), _ptr(mask), ids.data_ptr(), scores.data_ptr(),
                           _ptr(counts), _ptr(sums), _ptr(loss), _ptr(room), self._workspace_bytes, s)
        return ids, scores, counts, sums, loss

    def backward(self, dscores, logits, ids, counts=None, dloss=None, mask=None, dlogits=None, stream=None):
        """dlogits [T, E] from dscores f32 [T, k] (None: zeros) and dloss f32 [] or [1] (None: the
        loss has no gradient; else counts are needed)."""
        import torch
        cfg, dev = self._logits_cfg(logits), self.device
        _check("ids", ids, (self.T, self.k), torch.int32, dev)
        if dscores is not None:
            _check("dscores", dscores, (self.T, self.k), torch.float32, dev)
        if counts is not None:
            _check("counts", counts, (self.E,), torch.int32, dev)
        if dloss is not None:
            _check("dloss", dloss, dloss.shape if dloss.numel() == 1 else (), torch.float32, dev)
        if dlogits is not None:
            _check("dlogits", dlogits, (self.T, self.E), logits.dtype, dev)
        self._check_mask(mask)

        return self._call(self._backward, stream, cfg, dscores, logits, ids, counts, dloss, mask, dlogits)

    def _backward(self, s, cfg, dscores, logits, ids, counts, dloss, mask, dlogits):
        import torch
        out = torch.empty_like(logits) if dlogits is None else dlogits
        moe_router_backward(cfg, _ptr(dscores), logits.data_ptr(), _ptr(mask), ids.data_ptr(), _ptr(counts),
                            _ptr(dloss), out.data_ptr(), s)
        return out


class BlockNorm(_OnDevice):
    """The norms before and after the layer with its gate and residual:
    z = x + residual_scale * gate * rms(y; w_post), h = rms(z; w_pre); see include/moe.h."""

    def __init__(self, T, d, eps=1e-6, residual_scale=1.0, gate=MOE_GATE_NONE, residual_f32=False, device="cuda"):
        self.T, self.d, self.gate = T, d, gate
        self.residual_f32 = bool(residual_f32)
        self._rows = _dense(T, d)
        self._shape, self._channels = (T, d), (d,)
        self._cfg = NormConfig(T, d, int(gate), int(self.residual_f32), eps, residual_scale)
        nbytes = moe_norm_workspace_bytes(self._cfg)
        if not nbytes:
            moe_norm_forward(self._cfg, 0, 0, 0, 0, 0, 0, 0)
        super().__init__(device, nbytes)

    def _check_args(self, y, w_post, gate, w_pre):
        """The arguments that both directions take."""
        import torch
        dev, f32 = self.device, torch.float32
        if y is not None:
            _check("y", y, self._shape, torch.bfloat16, dev)
        if w_post is not None:
            _check("w_post", w_post, self._channels, f32, dev)
        if gate is not None:
            _check("gate", gate, (self.T,) if self.gate == MOE_GATE_TOKEN else self._channels, f32, dev)
        if w_pre is not None:
            _check("w_pre", w_pre, self._channels, f32, dev)
        return f32 if self.residual_f32 else torch.bfloat16

    def forward(self, x, y=None, w_post=None, gate=None, w_pre=None, z=None, stream=None):
        """(z, h); h is None without w_pre.  Without y, z is x itself.  z may be given (also x)."""
        res = self._check_args(y, w_post, gate, w_pre)
        _check("x", x, self._shape, res, self.device)
        if z is not None:
            _check("z", z, self._shape, res, self.device)
        return self._call(self._forward, stream, res, x, y, w_post, gate, w_pre, z)

    def _forward(self, s, res, x, y, w_post, gate, w_pre, z):
        import torch
        if z is None and y is not None:
            z = _new(self._rows, res, self.device)
        h = None if w_pre is None else _new(self._rows, torch.bfloat16, self.device)
        moe_norm_forward(self._cfg, x.data_ptr(), _ptr(y), _ptr(w_post), _ptr(gate), _ptr(w_pre), _ptr(z), _ptr(h), s)
        return x if y is None else z, h

    def backward(self, dz, dh, z, y=None, w_post=None, gate=None, w_pre=None, dx=None, stream=None):
        """(dx, dy, dw_post, dgate, dw_pre), None where there is no such input.  dz None: the stream
        has no gradient but h's.  dx may be given (also dz)."""
        import torch
        res = self._check_args(y, w_post, gate, w_pre)
        for name, t in (("dz", dz), ("z", z), ("dx", dx)):
            if t is not None:
                _check(name, t, self._shape, res, self.device)
        if dh is not None:
            _check("dh", dh, self._shape, torch.bfloat16, self.device)
        return self._call(self._backward, stream, res, dz, dh, z, y, w_post, gate, w_pre, dx)

    def _backward(self, s, res, dz, dh, z, y, w_post, gate, w_pre, dx):
        import torch
        like = torch.empty_like
        if dx is None:
            dx = _new(self._rows, res, self.device)
        dy = None if y is None else like(y)
        dw_post = None if w_post is None else like(w_post)
        dgate = None if gate is None else like(gate)
        dw_pre = None if w_pre is None else like(w_pre)
        room = self._room(s)
        moe_norm_backward(self._cfg, _ptr(dz), _ptr(dh), _ptr(z), _ptr(y), _ptr(w_post), _ptr(gate), _ptr(w_pre),
                          dx.data_ptr(), _ptr(dy), _ptr(dw_post), _ptr(dgate), _ptr(dw_pre), room.data_ptr(),
                          self._workspace_bytes, s)
        return dx, dy, dw_post, dgate, dw_pre


class Product(_OnDevice):
    """Rows [R, K] in BF16 times weights [E, N, K] in E4M3 with one FP32 scale per 128 x 128: one matrix, or
    with m_indptr (int32 [E+1] on the device) the matrix of each segment of the rows.  See the section on
    products in include/moe.h.  Weights are codes (uint8 or float8_e4m3fn) [E, N, K] and scales f32
    [E, N/128, K/128], from prepare_weights or from a checkpoint that holds them so.  Calls may be captured; the
    object is made before."""

    def __init__(self, R, N, K, E=1, training=False, wgrad_accumulate=False, device="cuda"):
        import torch
        self.R, self.N, self.K, self.E = R, N, K, E
        self._in, self._out, self._weights = _dense(R, K), _dense(R, N), _dense(E, N, K)
        self._scales = _dense(E, N // 128, K // 128)
        self._cfg = ProductConfig(R, N, K, E, int(bool(training)), int(bool(wgrad_accumulate)))
        nbytes = moe_product_workspace_bytes(self._cfg)
        if not nbytes:                                 # the reason, from the call that names it
            moe_product_forward(self._cfg, 0, 0, 0, 0, 0, 0, 0, 0)
        super().__init__(device, nbytes)
        if self._own is None:
            raise RuntimeError("a Product is made before a capture, not in it: its status word would be cleared by each replay")
        self._status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._wait()

    def _wait(self):
        """The status word is cleared: calls on any stream may set it from now on."""
        import torch
        torch.cuda.current_stream(self.device).synchronize()

    def _check_args(self, w_q, w_s, m_indptr):
        import torch
        if w_q is not None:
            _check_codes("w_q", w_q, self._weights[0], self.device)
        if w_s is not None:
            _check("w_s", w_s, self._scales[0], torch.float32, self.device)
        if m_indptr is not None:
            _check("m_indptr", m_indptr, (self.E + 1,), torch.int32, self.device)

    def prepare_weights(self, w, stream=None):
        """BF16 weights [E, N, K] -> (codes uint8, scales f32)."""
        import torch
        _check("w", w, self._weights[0], torch.bfloat16, self.device)
        return self._call(self._prepare, stream, w)

    def _prepare(self, s, w):
        import torch
        w_q, w_s = _new(self._weights, torch.uint8, self.device), _new(self._scales, torch.float32, self.device)
        moe_product_prepare_weights(self._cfg, w.data_ptr(), w_q.data_ptr(), w_s.data_ptr(), s)
        return w_q, w_s

    def expand_weights(self, w_q, w_s, stream=None):
        """The BF16 weights that codes and scales stand for."""
        self._check_args(w_q, w_s, None)
        return self._call(self._expand, stream, w_q, w_s)

    def _expand(self, s, w_q, w_s):
        import torch
        w = _new(self._weights, torch.bfloat16, self.device)
        moe_product_expand_weights(self._cfg, w_q.data_ptr(), w_s.data_ptr(), w.data_ptr(), s)
        return w

    def forward(self, x, w_q, w_s, m_indptr=None, y=None, stream=None):
        """y BF16 [R, N]; rows behind m_indptr[E] are not written."""
        import torch
        _check("x", x, self._in[0], torch.bfloat16, self.device)
        self._check_args(w_q, w_s, m_indptr)
        if y is not None:
            _check("y", y, self._out[0], torch.bfloat16, self.device)
        return self._call(self._forward, stream, x, w_q, w_s, m_indptr, y)

    def _forward(self, s, x, w_q, w_s, m_indptr, y):
        import torch
        if y is None:
            y = _new(self._out, torch.bfloat16, self.device)
        room = self._room(s)
        moe_product_forward(self._cfg, x.data_ptr(), _ptr(m_indptr), _ptr(w_q), _ptr(w_s), y.data_ptr(),
                            self._status.data_ptr(), room.data_ptr(), self._workspace_bytes, s)
        return y

    def backward(self, dy, x, w_q, w_s, m_indptr=None, dx=None, dw=None, need_dx=True, need_dw=True, stream=None):
        """(dx BF16 [R, K], dw BF16 [E, N, K]), None where it is not needed; x may be None without dw,
        the weights without dx.  dx and dw may be given (with wgrad_accumulate dw has to be)."""
        import torch
        _check("dy", dy, self._out[0], torch.bfloat16, self.device)
        if x is not None:
            _check("x", x, self._in[0], torch.bfloat16, self.device)
        self._check_args(w_q, w_s, m_indptr)
        for name, t, shape in (("dx", dx, self._in[0]), ("dw", dw, self._weights[0])):
            if t is not None:
                _check(name, t, shape, torch.bfloat16, self.device)
        if need_dw and dw is None and self._cfg.wgrad_accumulate:
            raise ValueError("dw: the gradients to add to are needed")
        return self._call(self._backward, stream, dy, x, w_q, w_s, m_indptr, dx, dw, need_dx, need_dw)

    def _backward(self, s, dy, x, w_q, w_s, m_indptr, dx, dw, need_dx, need_dw):
        import torch
        bf16 = torch.bfloat16
        dx = None if not need_dx else _new(self._in, bf16, self.device) if dx is None else dx
        dw = None if not need_dw else _new(self._weights, bf16, self.device) if dw is None else dw
        room = self._room(s)
        moe_product_backward(self._cfg, dy.data_ptr(), _ptr(x), _ptr(m_indptr), _ptr(w_q), _ptr(w_s), _ptr(dx), _ptr(dw),
                             self._status.data_ptr(), room.data_ptr(), self._workspace_bytes, s)
        return dx, dw

    def status(self, clear=True):
        """(status, device flags) of the calls so far; waits for the device's work."""
        import torch
        torch.cuda.synchronize(self.device)
        flags = int(self._status.item())
        if clear and flags:
            self._status.zero_()
            self._wait()
        return (MOE_ERR_ROUTING if flags else MOE_OK), flags
