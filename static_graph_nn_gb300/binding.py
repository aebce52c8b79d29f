"""Thin ctypes binding of libmg.so: the C ABI of include/mg.h under the same
names, plus a small ``Plan`` wrapper that marshals torch tensors into pointers.

Argument marshalling only: every step of the training step runs in the
library's CUDA kernels.  If the library is missing the import of the binding
fails loudly; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmg.so")

MG_OK, MG_ERR_INVALID_ARG, MG_ERR_UNSUPPORTED, MG_ERR_SHAPE, MG_ERR_ALIGN = 0, -1, -2, -3, -4
MG_ERR_OOM, MG_ERR_CUDA, MG_ERR_NONFINITE, MG_ERR_TIMEOUT, MG_ERR_INTERNAL = -5, -6, -7, -8, -9
STATUS_NAMES = {0: "MG_OK", -1: "MG_ERR_INVALID_ARG", -2: "MG_ERR_UNSUPPORTED", -3: "MG_ERR_SHAPE",
                -4: "MG_ERR_ALIGN", -5: "MG_ERR_OOM", -6: "MG_ERR_CUDA", -7: "MG_ERR_NONFINITE",
                -8: "MG_ERR_TIMEOUT", -9: "MG_ERR_INTERNAL"}

OPS = {"linear": 0, "relu": 1, "gelu_tanh": 2, "rmsnorm": 3, "residual_begin": 4,
       "residual_end": 5, "causal_attention": 6, "embedding": 7, "grouped_linear": 8}
LOSSES = {"ce_dense": 0, "ce_index": 1, "mse": 2}
PRECISIONS = {"strict": 0, "bf16": 1}
OPTIMIZERS = {"sgd": 0, "adam": 1, "laprop": 2, "sgd_momentum": 3}


class mg_layer(ctypes.Structure):
    _fields_ = [("op", ctypes.c_int), ("d_in", ctypes.c_int), ("d_out", ctypes.c_int),
                ("has_bias", ctypes.c_int), ("eps", ctypes.c_float), ("n_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("seq_len", ctypes.c_int)]


class mg_graph_desc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("n_layers", ctypes.c_int),
                ("layers", ctypes.POINTER(mg_layer)), ("loss", ctypes.c_int),
                ("precision", ctypes.c_int), ("optimizer", ctypes.c_int),
                ("beta1", ctypes.c_float), ("beta2", ctypes.c_float), ("adam_eps", ctypes.c_float)]


_P = ctypes.c_void_p
_SIGS = {
    "mg_step_plan_create": (ctypes.c_int, [ctypes.POINTER(mg_graph_desc), ctypes.POINTER(_P)]),
    "mg_step_plan_destroy": (None, [_P]),
    "mg_param_count": (ctypes.c_size_t, [_P]),
    "mg_param_tensor_count": (ctypes.c_int, [_P]),
    "mg_param_info": (ctypes.c_int, [_P, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t),
                                     ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    "mg_workspace_bytes": (ctypes.c_size_t, [_P]),
    "mg_forward": (ctypes.c_int, [_P, _P, _P, _P, _P]),
    "mg_train_step": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, ctypes.c_float, ctypes.c_int, _P]),
    "mg_loss": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_float), _P]),
    "mg_set_row_groups": (ctypes.c_int, [_P, _P]),
    "mg_set_grad_clip": (ctypes.c_int, [_P, ctypes.c_float]),
    "mg_grad_norm_device_ptr": (_P, [_P]),
    "mg_grad_norm": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_float), _P]),
    "mg_loss_device_ptr": (_P, [_P]),
    "mg_loss_async": (ctypes.c_int, [_P, ctypes.c_void_p, _P]),
    "mg_refresh_params": (ctypes.c_int, [_P, _P, _P]),
    "mg_plan_dump": (ctypes.c_size_t, [_P, ctypes.c_char_p, ctypes.c_size_t]),
    "mg_last_error": (ctypes.c_char_p, [_P]),
    "mg_debug_check_finite": (ctypes.c_int, [_P, _P, ctypes.c_size_t,
                                             ctypes.POINTER(ctypes.c_longlong), _P]),
    "mg_last_launch_count": (ctypes.c_int, [_P]),
    "mg_graph_replays": (ctypes.c_longlong, [_P]),
    "mg_profile_begin": (ctypes.c_int, [_P, ctypes.c_int]),
    "mg_profile_end": (ctypes.c_int, [_P]),
    "mg_profile_entries": (ctypes.c_int, [_P]),
    "mg_ffma_peak": (ctypes.c_int, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double),
                                    _P]),
    "mg_softmax_ce_noalloc": (ctypes.c_int, [ctypes.c_int, _P, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_int, _P, _P, _P, _P]),
    "mg_checkpoint_bytes": (ctypes.c_size_t, [_P, ctypes.c_int, ctypes.c_int]),
    "mg_checkpoint_save": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_void_p, ctypes.c_size_t,
                                          ctypes.POINTER(ctypes.c_size_t), _P]),
    "mg_checkpoint_load": (ctypes.c_int, [_P, ctypes.c_void_p, ctypes.c_size_t, _P, _P, _P, _P]),
    "mg_profile_entry": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_char_p, ctypes.c_size_t,
                                        ctypes.POINTER(ctypes.c_int),
                                        ctypes.POINTER(ctypes.c_double),
                                        ctypes.POINTER(ctypes.c_double),
                                        ctypes.POINTER(ctypes.c_double)]),
    "mg_embedding_workspace_bytes": (ctypes.c_size_t, [ctypes.c_longlong, ctypes.c_int, ctypes.c_int]),
    "mg_embedding_forward": (ctypes.c_int, [ctypes.c_int, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                            _P, ctypes.c_longlong, ctypes.c_float, ctypes.c_int, _P,
                                            _P]),
    "mg_embedding_backward": (ctypes.c_int, [ctypes.c_int, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                             _P, ctypes.c_longlong, ctypes.c_float, _P, _P,
                                             ctypes.c_size_t, _P]),
    "mg_grouped_linear_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 4),
    "mg_grouped_linear_forward": (ctypes.c_int, [ctypes.c_int, _P, _P] + [ctypes.c_int] * 4
                                  + [_P, _P, _P, ctypes.c_size_t, _P]),
    "mg_grouped_linear_backward_input": (ctypes.c_int, [ctypes.c_int, _P, _P] + [ctypes.c_int] * 4
                                         + [_P, _P, _P, ctypes.c_size_t, _P]),
    "mg_grouped_linear_backward_weight": (ctypes.c_int, [ctypes.c_int, _P, _P, _P] + [ctypes.c_int] * 4
                                          + [_P, _P, ctypes.c_size_t, _P]),
    "mg_grouped_linear_status": (ctypes.c_int, [_P, _P]),
    "mg_grad_list_create": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(_P), ctypes.POINTER(_P),
                                           ctypes.POINTER(ctypes.c_size_t),
                                           ctypes.POINTER(ctypes.c_int), ctypes.POINTER(_P)]),
    "mg_grad_list_destroy": (None, [_P]),
    "mg_grad_list_clip": (ctypes.c_int, [_P, ctypes.c_float, _P, _P]),
}

_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmg.so (built by build.py / __graft_entry__.build()).  Raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libmg.so not built at {path}; run __graft_entry__.build() first")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def exported_symbols() -> list[str]:
    return list(_SIGS)


class MGError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_INT_MAX = 2 ** 31 - 1     # sizes in the C ABI; ctypes would keep a larger one's low bits


def layer_struct(l: dict) -> mg_layer:
    for name, v in l.items():
        if isinstance(v, int) and abs(v) > _INT_MAX:
            raise MGError(MG_ERR_SHAPE, f"{l['op']}: {name} = {v} is beyond 32 bits")
    s = mg_layer()
    s.op = OPS[l["op"]]
    if l["op"] == "linear":
        s.d_in, s.d_out, s.has_bias = l["d_in"], l["d_out"], int(l["bias"])
    elif l["op"] == "rmsnorm":
        s.d_in, s.eps = l["d"], l["eps"]
    elif l["op"] == "causal_attention":
        s.n_heads, s.head_dim, s.seq_len = l["n_heads"], l["head_dim"], l["seq_len"]
    elif l["op"] == "embedding":
        s.d_in, s.d_out, s.eps = l["vocab"], l["dim"], l["scale"]
    elif l["op"] == "grouped_linear":
        s.d_in, s.d_out, s.n_heads = l["d_in"], l["d_out"], l["groups"]
    return s


class Plan:
    """A step plan for one graph; owns the library's workspace until close()."""

    def __init__(self, layers: list[dict], batch: int, loss: str, precision: str,
                 optimizer: str, beta1: float = 0.9, beta2: float = 0.999,
                 adam_eps: float = 1e-8):
        self.lib = load()
        arr = (mg_layer * len(layers))(*[layer_struct(l) for l in layers])
        d = mg_graph_desc()
        d.batch, d.n_layers, d.layers = batch, len(layers), arr
        d.loss, d.precision, d.optimizer = LOSSES[loss], PRECISIONS[precision], OPTIMIZERS[optimizer]
        d.beta1, d.beta2, d.adam_eps = beta1, beta2, adam_eps
        h = _P()
        st = self.lib.mg_step_plan_create(ctypes.byref(d), ctypes.byref(h))
        if st != MG_OK:
            raise MGError(st, self.lib.mg_last_error(None).decode())
        self.h = h
        self.batch, self.precision, self.loss_kind = batch, precision, loss
        self.layers = list(layers)
        self._takes_ids = bool(layers) and layers[0]["op"] == "embedding"

    @classmethod
    def for_workload(cls, w, precision: str):
        return cls(w.layers, w.batch, w.loss, precision, w.optimizer, w.beta1, w.beta2,
                   w.adam_eps)

    def _check(self, st: int):
        if st != MG_OK:
            raise MGError(st, self.lib.mg_last_error(self.h).decode())

    def close(self):
        if getattr(self, "h", None):
            self.lib.mg_step_plan_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def param_count(self) -> int:
        return self.lib.mg_param_count(self.h)

    @property
    def workspace_bytes(self) -> int:
        return self.lib.mg_workspace_bytes(self.h)

    def param_info(self) -> list[tuple[int, int, int]]:
        out = []
        for i in range(self.lib.mg_param_tensor_count(self.h)):
            o, r, c = ctypes.c_size_t(), ctypes.c_int(), ctypes.c_int()
            self._check(self.lib.mg_param_info(self.h, i, ctypes.byref(o), ctypes.byref(r),
                                               ctypes.byref(c)))
            out.append((o.value, r.value, c.value))
        return out

    def _check_ids(self, x):
        # the library reads batch int32 ids; a tensor says whether it holds them
        if self._takes_ids and x is not None and not isinstance(x, int):
            if x.dtype != _type_tables()[3]:
                _refuse(f"ids must be int32, not {x.dtype}")
            if x.numel() != self.batch:
                _refuse(f"{x.numel()} ids for a batch of {self.batch}", MG_ERR_SHAPE)
            _dense(x, "ids")

    def forward(self, params, x, out, stream=None):
        self._check_ids(x)
        self._check(self.lib.mg_forward(self.h, _ptr(params), _ptr(x), _ptr(out), _stream(stream)))

    def train_step(self, params, grads, adam_m, adam_v, x, labels, lr: float, step: int,
                   stream=None):
        self._check_ids(x)
        self._check(self.lib.mg_train_step(self.h, _ptr(params), _ptr(grads), _ptr(adam_m),
                                           _ptr(adam_v), _ptr(x), _ptr(labels), float(lr),
                                           int(step), _stream(stream)))

    def set_row_groups(self, offsets):
        """Row groups of the grouped_linear layers: int32 offsets [groups + 1] on the
        device (kept; its values are read by every later forward and train_step)."""
        if not isinstance(offsets, int):
            groups = next((l["groups"] for l in self.layers if l["op"] == "grouped_linear"), 0)
            if offsets.dtype != _type_tables()[3]:
                _refuse("offsets must be int32")
            _dense(offsets, "offsets", (groups + 1,))
        self._check(self.lib.mg_set_row_groups(self.h, _ptr(offsets)))
        self.row_groups = offsets

    def set_grad_clip(self, max_norm: float):
        """Clip every later step's gradients to this global norm (inf: measure only;
        0: off)."""
        if max_norm > 0 and ctypes.c_float(max_norm).value == 0:
            _refuse(f"max_norm = {max_norm} is 0 in fp32, which would turn clipping off")
        self._check(self.lib.mg_set_grad_clip(self.h, max_norm))

    def grad_norm(self, stream=None) -> tuple[float, float]:
        """(norm, factor) of the last clipped step; waits for it."""
        v = (ctypes.c_float * 2)()
        self._check(self.lib.mg_grad_norm(self.h, v, _stream(stream)))
        return v[0], v[1]

    def grad_norm_device_ptr(self) -> int | None:
        return self.lib.mg_grad_norm_device_ptr(self.h)

    def loss(self, stream=None) -> float:
        v = ctypes.c_float()
        self._check(self.lib.mg_loss(self.h, ctypes.byref(v), _stream(stream)))
        return v.value

    def loss_async(self, host_dst, stream=None):
        """Enqueue the copy of this step's (loss, timed_out) pair into 8 bytes of
        host memory (a pinned tensor or an address); no wait."""
        self._check(self.lib.mg_loss_async(self.h, _ptr(host_dst), _stream(stream)))

    def loss_device_ptr(self) -> int:
        return self.lib.mg_loss_device_ptr(self.h)

    def refresh_params(self, params, stream=None):
        self._check(self.lib.mg_refresh_params(self.h, _ptr(params), _stream(stream)))

    def checkpoint_save(self, params, m=None, v=None, stream=None) -> bytes:
        """The checkpoint image of params (and moments when given) as bytes."""
        n = self.lib.mg_checkpoint_bytes(self.h, int(m is not None), int(v is not None))
        buf = ctypes.create_string_buffer(n)
        written = ctypes.c_size_t()
        self._check(self.lib.mg_checkpoint_save(self.h, _ptr(params), _ptr(m), _ptr(v), buf, n,
                                                ctypes.byref(written), _stream(stream)))
        return buf.raw[:written.value]

    def checkpoint_load(self, image: bytes, params, m=None, v=None, stream=None):
        """Restore params (and moments when given) from a checkpoint image; the
        image is checked in full first and nothing changes if it fails."""
        buf = ctypes.create_string_buffer(bytes(image), len(image))
        self._check(self.lib.mg_checkpoint_load(self.h, buf, len(image), _ptr(params), _ptr(m),
                                                _ptr(v), _stream(stream)))

    def dump(self) -> str:
        n = self.lib.mg_plan_dump(self.h, None, 0)
        buf = ctypes.create_string_buffer(n + 1)
        self.lib.mg_plan_dump(self.h, buf, n + 1)
        return buf.value.decode()

    def check_finite(self, data, n: int, stream=None) -> int:
        """-1 if all finite, else the first bad index."""
        idx = ctypes.c_longlong()
        st = self.lib.mg_debug_check_finite(self.h, _ptr(data), n, ctypes.byref(idx),
                                            _stream(stream))
        if st not in (MG_OK, MG_ERR_NONFINITE):
            self._check(st)
        return idx.value

    def last_launch_count(self) -> int:
        return self.lib.mg_last_launch_count(self.h)

    def graph_replays(self) -> int:
        return self.lib.mg_graph_replays(self.h)

    def profile_begin(self, max_calls: int):
        self._check(self.lib.mg_profile_begin(self.h, max_calls))

    def profile_end(self) -> list[dict]:
        self._check(self.lib.mg_profile_end(self.h))
        out = []
        for i in range(self.lib.mg_profile_entries(self.h)):
            name = ctypes.create_string_buffer(256)
            n, ms, fl, by = ctypes.c_int(), ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
            self._check(self.lib.mg_profile_entry(self.h, i, name, 256, ctypes.byref(n),
                                                  ctypes.byref(ms), ctypes.byref(fl),
                                                  ctypes.byref(by)))
            out.append({"name": name.value.decode(), "launches": n.value, "total_ms": ms.value,
                        "flops": fl.value, "bytes": by.value})
        return out


def ffma_peak(stream=None) -> tuple[float, float]:
    """Measured FP32 FFMA rate of the current device: (TFLOP/s, flop per clock
    per SM), the strict path's roofline denominator."""
    lib = load()
    t, c = ctypes.c_double(), ctypes.c_double()
    st = lib.mg_ffma_peak(ctypes.byref(t), ctypes.byref(c), _stream(stream))
    if st != MG_OK:
        raise MGError(st, lib.mg_last_error(None).decode())
    return t.value, c.value


# ---- language-model operators (no plan) ---------------------------------------
# Tensors are dense torch tensors on the current device; shapes and types are
# checked here and refused with an MGError before the library is called.

_types = None


def _type_tables():
    """(dtype codes, id kinds, float32, int32), by torch's dtype objects; torch is
    imported on first use."""
    global _types
    if _types is None:
        import torch
        _types = ({torch.float32: 0, torch.bfloat16: 1}, {torch.int32: 0, torch.int64: 1}, torch.float32,
                  torch.int32)
    return _types


def _refuse(msg: str, status: int = MG_ERR_INVALID_ARG):
    raise MGError(status, msg)


def _code(t, name: str, table: dict | None = None) -> int:
    if table is None:
        table = _type_tables()[0]
    k = table.get(t.dtype)
    if k is None:
        _refuse(f"{name} must be one of {', '.join(sorted(map(str, table)))}, not {t.dtype}")
    return k


def _dense(t, name: str, shape: tuple | None = None):
    # (memory that is not this device's is refused by the library)
    if not t.is_contiguous():
        _refuse(f"{name} must be contiguous (strides {tuple(t.stride())})")
    if shape is not None and t.shape != shape:
        _refuse(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}", MG_ERR_SHAPE)


def _fits(*sizes: int):
    if max(sizes) > _INT_MAX:
        _refuse(f"a size is beyond 32 bits: {sizes}", MG_ERR_SHAPE)


def _status(st: int):
    if st != MG_OK:
        raise MGError(st, load().mg_last_error(None).decode())


def embedding_workspace_bytes(n: int, vocab: int, dim: int) -> int:
    """Bytes of workspace that embedding_backward needs for n ids (0: refused sizes)."""
    if max(vocab, dim) > _INT_MAX or n >= 2 ** 63:
        return 0
    return load().mg_embedding_workspace_bytes(n, vocab, dim)


def embedding_forward(table, ids, out, scale: float = 1.0, stream=None):
    """out[i] = scale * table[ids[i]]; zeros for an id outside [0, vocab).

    table [vocab, dim] and out [*ids.shape, dim] fp32 or bf16 (each its own
    type), ids int32 or int64 of any shape."""
    if table.dim() != 2:
        _refuse("table must be [vocab, dim]", MG_ERR_SHAPE)
    v, d = table.shape
    _fits(v, d)
    _dense(table, "table")
    _dense(ids, "ids")
    _dense(out, "out", ids.shape + (d,))
    _status(load().mg_embedding_forward(_code(table, "table"), _ptr(table), v, d,
                                        _code(ids, "ids", _type_tables()[1]), _ptr(ids), ids.numel(), scale,
                                        _code(out, "out"), _ptr(out), _stream(stream)))


def embedding_backward(dout, ids, dtable, workspace, scale: float = 1.0, stream=None):
    """dtable[v] = scale * sum of dout[i] over ids[i] == v; every row of dtable is
    written.  dout [*ids.shape, dim] fp32 or bf16, dtable [vocab, dim] fp32,
    workspace a byte tensor of embedding_workspace_bytes."""
    if dtable.dim() != 2 or dtable.dtype != _type_tables()[2]:
        _refuse("dtable must be [vocab, dim] float32", MG_ERR_SHAPE)
    v, d = dtable.shape
    _fits(v, d)
    _dense(dtable, "dtable")
    _dense(ids, "ids")
    _dense(dout, "dout", ids.shape + (d,))
    _dense(workspace, "workspace")
    _status(load().mg_embedding_backward(_code(dout, "dout"), _ptr(dout), v, d,
                                         _code(ids, "ids", _type_tables()[1]), _ptr(ids), ids.numel(), scale,
                                         _ptr(dtable), _ptr(workspace),
                                         workspace.nbytes,
                                         _stream(stream)))


def grouped_linear_workspace_bytes(rows: int, groups: int, d_in: int, d_out: int) -> int:
    """Bytes of workspace for the grouped products of these sizes (zero it once; 0:
    refused sizes)."""
    if max(rows, groups, d_in, d_out) > _INT_MAX:
        return 0
    return load().mg_grouped_linear_workspace_bytes(rows, groups, d_in, d_out)


def _grouped_args(rows_t, name, offsets, weights, workspace):
    if rows_t.dim() != 2:
        _refuse(f"{name} must be two-dimensional", MG_ERR_SHAPE)
    _fits(*rows_t.shape, *weights)
    _dense(rows_t, name)
    if offsets.dtype != _type_tables()[3]:
        _refuse("offsets must be int32")
    _dense(offsets, "offsets", (weights[0] + 1,))
    _dense(workspace, "workspace")
    return workspace.nbytes


def _same_type(a, an, b, bn):
    if a.dtype != b.dtype:
        _refuse(f"{an} and {bn} must have one type, not {a.dtype} and {b.dtype}")


def grouped_linear_forward(x, offsets, w, y, workspace, stream=None):
    """y[r] = x[r] @ w[e] for the rows offsets[e] <= r < offsets[e + 1] of each
    group e; other rows of y are left as they were.  x [rows, d_in], w [groups,
    d_in, d_out], y [rows, d_out], all fp32 or all bf16; offsets int32 on the
    device."""
    if w.dim() != 3:
        _refuse("w must be [groups, d_in, d_out]", MG_ERR_SHAPE)
    e, k, n = w.shape
    nb = _grouped_args(x, "x", offsets, (e, k, n), workspace)
    _dense(x, "x", (x.shape[0], k))
    _dense(w, "w")
    _dense(y, "y", (x.shape[0], n))
    _same_type(x, "x", w, "w")
    _same_type(x, "x", y, "y")
    _status(load().mg_grouped_linear_forward(_code(x, "x"), _ptr(x), _ptr(offsets), x.shape[0], e, k, n,
                                             _ptr(w), _ptr(y), _ptr(workspace), nb, _stream(stream)))


def grouped_linear_backward_input(dy, offsets, w, dx, workspace, stream=None):
    """dx[r] = dy[r] @ w[e].T; shapes and types as grouped_linear_forward's."""
    if w.dim() != 3:
        _refuse("w must be [groups, d_in, d_out]", MG_ERR_SHAPE)
    e, k, n = w.shape
    nb = _grouped_args(dy, "dy", offsets, (e, k, n), workspace)
    _dense(dy, "dy", (dy.shape[0], n))
    _dense(w, "w")
    _dense(dx, "dx", (dy.shape[0], k))
    _same_type(dy, "dy", w, "w")
    _same_type(dy, "dy", dx, "dx")
    _status(load().mg_grouped_linear_backward_input(_code(dy, "dy"), _ptr(dy), _ptr(offsets),
                                                    dy.shape[0], e, k, n, _ptr(w), _ptr(dx),
                                                    _ptr(workspace), nb, _stream(stream)))


def grouped_linear_backward_weight(x, dy, offsets, dw, workspace, stream=None):
    """dw[e] = x_e.T @ dy_e (fp32; zeros for a group without rows)."""
    if dw.dim() != 3 or dw.dtype != _type_tables()[2]:
        _refuse("dw must be [groups, d_in, d_out] float32", MG_ERR_SHAPE)
    e, k, n = dw.shape
    nb = _grouped_args(x, "x", offsets, (e, k, n), workspace)
    _dense(x, "x", (x.shape[0], k))
    _dense(dy, "dy", (x.shape[0], n))
    _dense(dw, "dw")
    _same_type(x, "x", dy, "dy")
    _status(load().mg_grouped_linear_backward_weight(_code(x, "x"), _ptr(x), _ptr(dy), _ptr(offsets),
                                                     x.shape[0], e, k, n, _ptr(dw), _ptr(workspace), nb,
                                                     _stream(stream)))


def grouped_linear_status(workspace, stream=None):
    """Waits for the stream; raises an MGError (MG_ERR_TIMEOUT) if a device-side wait
    gave up in an earlier call with this workspace, whose results are then invalid."""
    _dense(workspace, "workspace")
    _status(load().mg_grouped_linear_status(_ptr(workspace), _stream(stream)))


class GradList:
    """Gradient tensors (fp32 or bf16, contiguous) whose global norm is taken and
    that are scaled by it together, in place or into ``out``.  Keeps the tensors
    alive; the table lives on the device until close()."""

    def __init__(self, grads, out=None):
        self.h = None
        self.lib = load()
        grads = list(grads)
        out = None if out is None else list(out)
        if out is not None and len(out) != len(grads):
            _refuse(f"{len(grads)} gradients but {len(out)} outputs")
        for i, g in enumerate(grads):
            _dense(g, f"gradient {i}")
            if out is not None:
                _dense(out[i], f"output {i}", g.shape)
                _same_type(g, f"gradient {i}", out[i], f"output {i}")
        n = len(grads)
        pg = (_P * max(1, n))(*[_ptr(g) for g in grads])
        po = (_P * max(1, n))(*[_ptr(o) for o in out]) if out is not None else None
        counts = (ctypes.c_size_t * max(1, n))(*[g.numel() for g in grads])
        types = (ctypes.c_int * max(1, n))(*[_code(g, f"gradient {i}") for i, g in enumerate(grads)])
        h = _P()
        _status(self.lib.mg_grad_list_create(n, pg, po, counts, types, ctypes.byref(h)))
        self.h, self.tensors = h, (grads, out)

    def clip(self, max_norm: float, stats, stream=None):
        """stats[0] = the norm, stats[1] = the factor (fp32 [2] on the device);
        the gradients times the factor to their outputs."""
        if stats.dtype != _type_tables()[2]:
            _refuse("stats must be float32")
        _dense(stats, "stats", (2,))
        _status(self.lib.mg_grad_list_clip(self.h, max_norm, _ptr(stats), _stream(stream)))

    def close(self):
        if getattr(self, "h", None):
            self.lib.mg_grad_list_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
