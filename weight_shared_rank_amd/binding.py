"""ctypes binding of the C ABI in include/weightless.h.

Argument marshalling only: every step of the weightless linear runs in the
HIP library.  torch supplies device memory (arena, workspace, x, y) and the
current HIP stream.  There is no fallback: if libweightless.so is missing or
fails to load, every entry point raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Dict, Iterable, NamedTuple, Optional, Sequence, Tuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIBPATH = os.path.join(HERE, "libweightless.so")

FAMILIES = ("q", "k", "v", "o", "gate", "up", "down")
FAMILY = {f: i for i, f in enumerate(FAMILIES)}
STACKS = {"qkv": 0, "gate_up": 1}
ACTS = {"gelu_tanh": 0, "silu": 1, "gelu": 2}
W0_FORMATS = {"bf16": 0, "fp8": 1, "mxfp4": 2}
WL_DTYPE_BF16, WL_DTYPE_F32 = 0, 1
WL_SRC_W0, WL_SRC_S, WL_SRC_U, WL_SRC_V = 0, 1, 2, 3
SRC_KIND = {"w0": WL_SRC_W0, "s": WL_SRC_S, "u": WL_SRC_U, "v": WL_SRC_V}
STATUS = {0: "WL_OK", -1: "WL_EINVAL", -2: "WL_ESHAPE", -3: "WL_EDTYPE", -4: "WL_ERANGE",
          -5: "WL_ENOSPACE", -6: "WL_EHIP"}
MAX_TYPES = 2
DECODE_MAX_T = 16
NOALLOC_WORKSPACE_BYTES = 64 << 20    # WL_NOALLOC_WORKSPACE_BYTES

# every symbol include/weightless.h declares
EXPORTS = ("theta_bundle_arena_bytes", "theta_bundle_load", "theta_bundle_free",
           "weightless_workspace_bytes",
           "weightless_linear", "weightless_linear_noalloc", "weightless_stacked_linear", "weightless_out_dim", "wl_last_error",
           "weightless_materialize_workspace_bytes", "weightless_materialize", "weightless_gate_up_act",
           "weightless_decompose_workspace_bytes", "weightless_decompose",
           "weightless_decompose_als_workspace_bytes", "weightless_decompose_als",
           "weightless_act_code_bytes", "weightless_weight_code_bytes", "weightless_act_encode",
           "weightless_act_expand", "weightless_weight_encode",
           "weightless_coded_linear_workspace_bytes", "weightless_coded_linear",
           "weightless_backward_workspace_bytes", "weightless_linear_backward", "weightless_stacked_backward",
           "weightless_norm", "weightless_norm_backward_workspace_bytes", "weightless_norm_backward",
           "weightless_adapters_workspace_bytes", "weightless_adapters_add",
           "weightless_adapters_backward_workspace_bytes", "weightless_adapters_backward")


class WlBundleSpec(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("num_bands", ctypes.c_int32),
                ("num_layer_types", ctypes.c_int32), ("layer_type", ctypes.POINTER(ctypes.c_int8)),
                ("out_dim", (ctypes.c_int32 * 7) * MAX_TYPES), ("in_dim", (ctypes.c_int32 * 7) * MAX_TYPES),
                ("rank", (ctypes.c_int32 * 7) * MAX_TYPES), ("k_eq_v_type_mask", ctypes.c_uint32),
                ("w0_format", ctypes.c_int32)]


class WlSrc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("index", ctypes.c_int32), ("layer_type", ctypes.c_int32),
                ("family", ctypes.c_int32), ("dtype", ctypes.c_int32), ("on_device", ctypes.c_int32),
                ("ptr", ctypes.c_void_p)]


class WlGrads(ctypes.Structure):
    _fields_ = [("dx", ctypes.c_void_p), ("ds", ctypes.c_void_p), ("du", ctypes.c_void_p * 3),
                ("dv", ctypes.c_void_p * 3), ("dw0", ctypes.c_void_p), ("accumulate_dw0", ctypes.c_int32)]


class WlAdapters(ctypes.Structure):
    _fields_ = [("num_slots", ctypes.c_int32), ("rank", ctypes.c_int32), ("in_dim", ctypes.c_int32),
                ("num_children", ctypes.c_int32), ("out_dim", ctypes.c_int32 * 3),
                ("d_vt", ctypes.c_void_p), ("d_u", ctypes.c_void_p), ("d_scale", ctypes.c_void_p),
                ("d_rank", ctypes.c_void_p)]


class WlAdapterGrads(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("dx", ctypes.c_void_p), ("du", ctypes.c_void_p), ("dv", ctypes.c_void_p)]


class Grads(NamedTuple):
    """Gradients of one call (None: not asked for).  du, dv: tensors, or for a
    stacked call tuples over its children."""
    dx: object = None
    ds: object = None
    du: object = None
    dv: object = None
    dw0: object = None


class WlError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None


def lib():
    """Load libweightless.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBPATH):
        raise RuntimeError(f"{LIBPATH} is not built; run `python -m weight_shared_rank_amd.build`")
    # torch's HIP runtime must be the process's only one: loaded first, it
    # satisfies the library's libamdhip64 dependency.  Loaded the other way
    # round, the library pulls in the system runtime beside torch's, and that
    # second runtime finds no device.
    import torch  # noqa: F401
    L = ctypes.CDLL(LIBPATH)
    vp, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    sig = {
        "theta_bundle_arena_bytes": (sz, [ctypes.POINTER(WlBundleSpec)]),
        "theta_bundle_load": (i32, [ctypes.POINTER(WlBundleSpec), ctypes.POINTER(WlSrc), sz, vp, sz, vp,
                                    ctypes.POINTER(vp)]),
        "theta_bundle_free": (i32, [vp]),
        "weightless_workspace_bytes": (sz, [vp, i32]),
        "weightless_linear": (i32, [vp, i32, i32, vp, i32, vp, vp, sz, vp]),
        "weightless_linear_noalloc": (i32, [vp, i32, i32, vp, i32, vp, vp]),
        "weightless_stacked_linear": (i32, [vp, i32, i32, vp, i32, vp, vp, sz, vp]),
        "weightless_out_dim": (i32, [vp, i32, i32, i32]),
        "wl_last_error": (ctypes.c_char_p, []),
        "weightless_materialize_workspace_bytes": (sz, [vp]),
        "weightless_materialize": (i32, [vp, i32, i32, vp, vp, sz, vp]),
        "weightless_gate_up_act": (i32, [vp, i32, i32, vp, i32, vp, vp, sz, vp]),
        "weightless_decompose_workspace_bytes": (sz, [i32, i32, i32, i32]),
        "weightless_decompose": (i32, [vp, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
        "weightless_decompose_als_workspace_bytes": (sz, [i32, i32, i32, i32]),
        "weightless_decompose_als": (i32, [vp, i32, i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
        "weightless_act_code_bytes": (sz, [i32, i32]),
        "weightless_weight_code_bytes": (sz, [i32, i32]),
        "weightless_act_encode": (i32, [vp, i32, i32, vp, sz, vp]),
        "weightless_act_expand": (i32, [vp, sz, i32, i32, vp, vp]),
        "weightless_weight_encode": (i32, [vp, i32, i32, vp, sz, vp]),
        "weightless_coded_linear_workspace_bytes": (sz, [i32, i32, i32]),
        "weightless_coded_linear": (i32, [vp, sz, i32, i32, vp, vp, sz, i32, vp, vp, sz, vp]),
        "weightless_backward_workspace_bytes": (sz, [vp, i32]),
        "weightless_linear_backward": (i32, [vp, i32, i32, vp, sz, vp, i32, ctypes.POINTER(WlGrads), vp, sz, vp]),
        "weightless_stacked_backward": (i32, [vp, i32, i32, vp, sz, vp, i32, ctypes.POINTER(WlGrads), vp, sz, vp]),
        "weightless_norm": (i32, [vp, vp, i32, i32, vp, i32, f32, f32, vp, vp, vp, sz, vp, vp]),
        "weightless_norm_backward_workspace_bytes": (sz, [i32, i32]),
        "weightless_adapters_workspace_bytes": (sz, [ctypes.POINTER(WlAdapters), i32]),
        "weightless_adapters_add": (i32, [ctypes.POINTER(WlAdapters), vp, vp, i32, vp, vp, vp, sz, vp]),
        "weightless_adapters_backward_workspace_bytes": (sz, [ctypes.POINTER(WlAdapters), i32]),
        "weightless_adapters_backward": (i32, [ctypes.POINTER(WlAdapters), vp, sz, vp, vp, i32,
                                               ctypes.POINTER(WlAdapterGrads), vp, sz, vp]),
        "weightless_norm_backward": (i32, [vp, vp, vp, vp, i32, i32, vp, i32, f32, vp, vp, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def last_error() -> str:
    return lib().wl_last_error().decode()


def _check(st: int):
    if st != 0:
        raise WlError(st, last_error())


def make_spec(num_layers: int, num_bands: int, dims: Dict[Tuple[int, str], Tuple[int, int]],
              ranks: Dict[Tuple[int, str], int], layer_types: Optional[Sequence[int]] = None,
              k_eq_v_types: Iterable[int] = (), w0_format: str = "bf16") -> WlBundleSpec:
    """Spec from Python dicts: dims[(type, family)] = (N, K), ranks[(type, family)] = r;
    w0_format "bf16" or "fp8" (E4M3 codes with a power-of-two scale per W0 row)."""
    sp = WlBundleSpec()
    sp.num_layers = num_layers
    sp.num_bands = num_bands
    nt = (max(layer_types) + 1) if layer_types else 1
    nt = max(nt, max([t for t, _ in dims] + [0]) + 1)
    sp.num_layer_types = nt
    if layer_types is not None:
        arr = (ctypes.c_int8 * len(layer_types))(*layer_types)
        sp.layer_type = ctypes.cast(arr, ctypes.POINTER(ctypes.c_int8))
        sp._keep = arr  # keep the array alive with the struct
    for (t, f), (n, k) in dims.items():
        sp.out_dim[t][FAMILY[f]] = n
        sp.in_dim[t][FAMILY[f]] = k
        sp.rank[t][FAMILY[f]] = ranks.get((t, f), 0)
    mask = 0
    for t in k_eq_v_types:
        mask |= 1 << t
    sp.k_eq_v_type_mask = mask
    sp.w0_format = W0_FORMATS[w0_format]
    return sp


def _stream_ptr(stream) -> ctypes.c_void_p:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def theta_bundle_arena_bytes(spec: WlBundleSpec) -> int:
    n = lib().theta_bundle_arena_bytes(ctypes.byref(spec))
    if n == 0:
        raise WlError(-1, last_error())
    return n


class ThetaBundle:
    """A theta bundle resident in a torch-allocated device arena."""

    def __init__(self, spec: WlBundleSpec, sources, device="cuda", stream=None, arena=None):
        """sources: iterable of (kind, index, layer_type, family, tensor) with
        kind in {"w0", "s", "u", "v"}; tensors may live on the host or the
        device (bf16 for w0/u/v, float32 for s, contiguous)."""
        import torch
        self.spec = spec
        need = theta_bundle_arena_bytes(spec)
        self.arena = arena if arena is not None else torch.empty(need, dtype=torch.uint8, device=device)
        if self.arena.numel() < need:
            raise WlError(-5, f"arena has {self.arena.numel()} bytes, bundle needs {need}")
        keep = []
        srcs = (WlSrc * max(1, len(sources)))()
        for i, (kind, index, ltype, fam, t) in enumerate(sources):
            if not t.is_contiguous():
                t = t.contiguous()
            keep.append(t)
            srcs[i].kind = SRC_KIND[kind]
            srcs[i].index = index
            srcs[i].layer_type = ltype
            srcs[i].family = FAMILY[fam]
            srcs[i].dtype = WL_DTYPE_F32 if t.dtype == torch.float32 else (WL_DTYPE_BF16 if t.dtype == torch.bfloat16 else 99)
            srcs[i].on_device = 1 if t.is_cuda else 0
            srcs[i].ptr = t.data_ptr()
        h = ctypes.c_void_p()
        _check(lib().theta_bundle_load(ctypes.byref(spec), srcs, len(sources), self.arena.data_ptr(),
                                       self.arena.numel(), _stream_ptr(stream), ctypes.byref(h)))
        self.handle = h
        self._keep_until_sync = keep
        # the load is asynchronous: the handle (which owns the host-side V^T
        # copies) is freed only once the stream has passed this event
        self._loaded = torch.cuda.Event()
        self._loaded.record(stream if stream is not None else torch.cuda.current_stream())
        self._ws = {}
        self._backward_need = {}   # T -> workspace bytes

    def close(self):
        if getattr(self, "handle", None):
            self._loaded.synchronize()
            lib().theta_bundle_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def out_dim(self, layer: int, family: Optional[str] = None, stack: Optional[str] = None) -> int:
        n = lib().weightless_out_dim(self.handle, layer, FAMILY[family] if family else -1,
                                     STACKS[stack] if stack else -1)
        if n == 0:
            raise WlError(-4, last_error())
        return n

    def workspace_bytes(self, T: int) -> int:
        n = lib().weightless_workspace_bytes(self.handle, T)
        if n == 0:
            raise WlError(-1, last_error())
        return n

    def workspace(self, T: int, stream=None):
        """A workspace large enough for T tokens."""
        import torch
        return torch.empty(self.workspace_bytes(T), dtype=torch.uint8, device=self.arena.device)

    def _ws_for(self, T, stream):
        need = self.workspace_bytes(T)
        key = "prefill" if T > DECODE_MAX_T else "decode"
        ws = self._ws.get(key)
        if ws is None or ws.numel() < need:
            ws = self.workspace(T, stream)
            self._ws[key] = ws
        return ws

    def _call(self, fn, layer, code, x, y, ws, stream, width):
        import torch
        T = x.shape[0]
        if y is None:
            y = torch.empty((T, width), dtype=torch.bfloat16, device=x.device)
        if ws is None:
            ws = self._ws_for(T, stream)
        _check(fn(self.handle, layer, code, x.data_ptr(), T, y.data_ptr(), ws.data_ptr(), ws.numel(),
                  _stream_ptr(stream)))
        return y

    def linear(self, layer: int, family: str, x, y=None, ws=None, stream=None):
        """y = s*(W0 x) + U (V^T x) for one family; x bf16 [T, K] on the device."""
        return self._call(lib().weightless_linear, layer, FAMILY[family], x, y, ws, stream,
                          self.out_dim(layer, family=family))

    def linear_noalloc(self, layer: int, family: str, x, y=None, stream=None):
        """weightless_linear on the library's fixed device workspace (no
        caller workspace); y is allocated here only if not given."""
        import torch
        T = x.shape[0]
        if y is None:
            y = torch.empty((T, self.out_dim(layer, family=family)), dtype=torch.bfloat16, device=x.device)
        _check(lib().weightless_linear_noalloc(self.handle, layer, FAMILY[family], x.data_ptr(), T, y.data_ptr(),
                                               _stream_ptr(stream)))
        return y

    def stacked(self, layer: int, stack: str, x, y=None, ws=None, stream=None):
        """The stacked q|k|v or gate|up call over one x."""
        return self._call(lib().weightless_stacked_linear, layer, STACKS[stack], x, y, ws, stream,
                          self.out_dim(layer, stack=stack))

    def gate_up_act(self, layer: int, act: str, x, h=None, ws=None, stream=None):
        """h = act(gate) * up of one layer's gate|up stack, bf16 [T, N_gate]."""
        return self._call(lambda hd, l, code, *rest: lib().weightless_gate_up_act(hd, l, ACTS[act], *rest),
                          layer, 0, x, h, ws, stream, self.out_dim(layer, family="gate"))

    def _children(self, layer: int, families):
        """(N, K, r) of the bundles behind these families of a layer (a tied
        type's v is k's and no child of its own in a stack)."""
        t = self.spec.layer_type[layer] if self.spec.layer_type else 0
        tied = (self.spec.k_eq_v_type_mask >> t) & 1
        fams = ["k" if f == "v" and tied else f for f in families]
        fams = [f for i, f in enumerate(fams) if f not in fams[:i]]
        return [(self.spec.out_dim[t][FAMILY[f]], self.spec.in_dim[t][FAMILY[f]], self.spec.rank[t][FAMILY[f]])
                for f in fams]

    def _backward(self, fn, layer, code, width, families, stacked, x, dy, want, dw0, accumulate, ws, stream):
        import torch
        dev = self.arena.device
        unknown = set(want) - {"dx", "ds", "du", "dv", "dw0"}
        if unknown:
            raise WlError(-1, f"unknown gradients {sorted(unknown)}")
        kids = self._children(layer, families)
        rows, K = sum(n for n, _, _ in kids), kids[0][1]
        if not isinstance(x, ActCode) or x.K != K or x.buf.device != dev:
            raise WlError(-1, f"x must be an ActCode of K = {K} on {dev}")
        T = x.T
        with _scope(dev, stream):
            _check_tensor(dy, "dy", (T, width), torch.bfloat16, dev)
            g, bf = WlGrads(), dict(dtype=torch.bfloat16, device=dev)
            out = {}
            if "dx" in want:
                out["dx"] = torch.empty((T, K), **bf)
                g.dx = out["dx"].data_ptr()
            if "ds" in want:
                out["ds"] = torch.empty((rows,), dtype=torch.float32, device=dev)
                g.ds = out["ds"].data_ptr()
            for name, arr in (("du", g.du), ("dv", g.dv)):
                if name in want:
                    ts = tuple(torch.empty((n if name == "du" else K, r), **bf) for n, _, r in kids)
                    for i, t in enumerate(ts):
                        arr[i] = t.data_ptr() or None
                    out[name] = ts if stacked else ts[0]
            if "dw0" in want:
                if dw0 is None:
                    if accumulate:
                        raise WlError(-1, "accumulate needs a dw0 to add to")
                    dw0 = torch.empty((rows, K), dtype=torch.float32, device=dev)
                _check_tensor(dw0, "dw0", (rows, K), torch.float32, dev)
                out["dw0"] = dw0
                g.dw0 = dw0.data_ptr()
                g.accumulate_dw0 = 1 if accumulate else 0
            elif dw0 is not None or accumulate:
                raise WlError(-1, "dw0 is given but not wanted")
            if ws is None:
                need = self._backward_need.get(T)
                if need is None:
                    need = lib().weightless_backward_workspace_bytes(self.handle, T)
                    if need == 0:
                        raise WlError(-1, last_error())
                    self._backward_need[T] = need
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
            else:
                _check_tensor(ws, "ws", (None,), torch.uint8, dev)
            _check(fn(self.handle, layer, code, x.buf.data_ptr(), x.buf.numel(), dy.data_ptr(), T, ctypes.byref(g),
                      ws.data_ptr(), ws.numel(), _raw_stream(dev)))
        return Grads(**out)

    def linear_backward(self, layer: int, family: str, x, dy, want=("dx", "ds", "du", "dv"), dw0=None,
                        accumulate: bool = False, ws=None, stream=None) -> Grads:
        """Gradients of linear() (weightless_linear_backward).

        x: the ActCode checkpoint of the call's input; dy: bf16 [T, N];
        want: which of dx, ds, du, dv, dw0.  dw0: float32 [N, K] to write (or,
        with accumulate, to add to); allocated if not given."""
        return self._backward(lib().weightless_linear_backward, layer, FAMILY[family],
                              self.out_dim(layer, family=family), (family,), False, x, dy, want, dw0, accumulate, ws,
                              stream)

    def stacked_backward(self, layer: int, stack: str, x, dy, want=("dx", "ds", "du", "dv"), dw0=None,
                         accumulate: bool = False, ws=None, stream=None) -> Grads:
        """Gradients of stacked() (weightless_stacked_backward): dy with the
        stacked call's columns; ds and dw0 over the children's rows, du and dv
        one per child."""
        return self._backward(lib().weightless_stacked_backward, layer, STACKS[stack],
                              self.out_dim(layer, stack=stack), ("q", "k", "v") if stack == "qkv" else ("gate", "up"),
                              True, x, dy, want, dw0, accumulate, ws, stream)

    def in_dim(self, layer: int, family: str) -> int:
        """K of one family of one layer (from the spec)."""
        t = self.spec.layer_type[layer] if self.spec.layer_type else 0
        f = FAMILY[family]
        if family == "v" and (self.spec.k_eq_v_type_mask >> t) & 1:
            f = FAMILY["k"]
        return self.spec.in_dim[t][f]

    def materialize(self, layer: int, family: str, out=None, ws=None, stream=None):
        """W_eff = diag(s) W0 + U V^T of one family, bf16 [N, K] on the device."""
        import torch
        n, k = self.out_dim(layer, family=family), self.in_dim(layer, family)
        if out is None:
            out = torch.empty((n, k), dtype=torch.bfloat16, device=self.arena.device)
        if ws is None:
            need = lib().weightless_materialize_workspace_bytes(self.handle)
            if need == 0:
                raise WlError(-1, last_error())
            ws = torch.empty(need, dtype=torch.uint8, device=self.arena.device)
        _check(lib().weightless_materialize(self.handle, layer, FAMILY[family], out.data_ptr(), ws.data_ptr(),
                                            ws.numel(), _stream_ptr(stream)))
        return out


def sketch_columns(N: int, K: int, rank: int, oversample: int) -> int:
    """Columns l of the test matrix weightless_decompose takes: min(rank + oversample, N, K)."""
    return min(rank + oversample, N, K)


def decompose(w, rank: int, omega=None, oversample: int = 16, power_iters: int = 4, stream=None,
              als_sweeps: int = None):
    """Decompose one band of one family on the GPU.

    w: bf16 [m, N, K] device tensor (the band's layers in layer order);
    omega: fp32 [K, l] device test matrix, l = sketch_columns(N, K, rank, oversample)
    (required when rank > 0).  als_sweeps: None calls weightless_decompose;
    an integer calls weightless_decompose_als with that many ALS sweeps.
    Returns (W0 bf16 [N, K], s fp32 [m, N], U bf16 [m, N, rank], V bf16
    [m, K, rank]), the layouts theta_bundle_load takes."""
    import torch
    if w.dim() != 3 or w.dtype != torch.bfloat16 or not w.is_cuda or not w.is_contiguous():
        raise WlError(-1, "w must be a contiguous bf16 [m, N, K] device tensor")
    m, n, k = w.shape
    dev = w.device
    l = sketch_columns(n, k, rank, oversample)
    if rank > 0:
        if omega is None or tuple(omega.shape) != (k, l) or omega.dtype != torch.float32 \
                or not omega.is_contiguous() or omega.device != dev:
            raise WlError(-1, f"omega must be a contiguous fp32 [{k}, {l}] tensor on {dev}")
    als = als_sweeps is not None
    need = (lib().weightless_decompose_als_workspace_bytes if als else lib().weightless_decompose_workspace_bytes)(
        n, k, rank, oversample)
    if need == 0:
        raise WlError(-1, "decomposition workspace size: arguments out of range")
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    w0 = torch.empty((n, k), dtype=torch.bfloat16, device=dev)
    s = torch.empty((m, n), dtype=torch.float32, device=dev)
    u = torch.empty((m, n, rank), dtype=torch.bfloat16, device=dev)
    v = torch.empty((m, k, rank), dtype=torch.bfloat16, device=dev)
    lead = (w.data_ptr(), m, n, k, rank, oversample, power_iters) + ((als_sweeps,) if als else ())
    fn = lib().weightless_decompose_als if als else lib().weightless_decompose
    _check(fn(*lead, omega.data_ptr() if rank > 0 else None, w0.data_ptr(), s.data_ptr(),
              u.data_ptr() if rank > 0 else None, v.data_ptr() if rank > 0 else None,
              ws.data_ptr(), ws.numel(), _stream_ptr(stream)))
    return w0, s, u, v


# ---- 8-bit coded operands -------------------------------------------------

CODE_BLOCK = 128


_HERE = contextlib.nullcontext()


def _scope(device, stream):
    """The device and stream a call runs on: the given stream, or the current
    stream of the tensors' device.  Everything the call allocates is then
    allocated on that stream."""
    import torch
    if stream is not None:
        if stream.device != device:
            raise WlError(-1, f"stream is on {stream.device}, the tensors are on {device}")
        return torch.cuda.stream(stream)
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _raw_stream(device) -> int:
    """The current stream of `device` as a hipStream_t (inside its _scope)."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


def _check_tensor(t, name, shape, dtype, device=None):
    """A contiguous device tensor of this shape (None: any extent) and dtype."""
    if t.shape == shape and t.dtype == dtype and t.is_cuda and t.is_contiguous() and (device is None or t.device == device):
        return  # (what nearly every call finds, at a third of the time)
    if not t.is_cuda or t.dtype != dtype or t.dim() != len(shape) or not t.is_contiguous() \
            or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        want = ", ".join("*" if w is None else str(w) for w in shape)
        raise WlError(-1, f"{name} must be a contiguous {dtype} [{want}] device tensor, got {t.dtype} "
                          f"{list(t.shape)} on {t.device}")
    if device is not None and t.device != device:
        raise WlError(-1, f"{name} is on {t.device}, expected {device}")


class _Code:
    """A coded buffer and its shape (rows R by K); layout in include/weightless.h."""

    _rows_per_scale, _run_multiple, _bytes = 1, 16, "weightless_act_code_bytes"

    def __init__(self, rows: int, K: int, device="cuda", buf=None):
        import torch
        self.rows, self.K = rows, K
        need = getattr(lib(), self._bytes)(rows, K)
        if need == 0:
            raise WlError(-2, last_error())
        if buf is None:
            buf = torch.empty(need, dtype=torch.uint8, device=device)
        else:
            _check_tensor(buf, "code buffer", (None,), torch.uint8)
            if buf.numel() < need:
                raise WlError(-5, f"code buffer has {buf.numel()} bytes, needs {need}")
        self.buf = buf

    @property
    def blocks(self) -> int:
        return -(-self.K // CODE_BLOCK)

    @property
    def codes(self):
        """The E4M3 codes [rows, K] (a view)."""
        import torch
        return self.buf.view(torch.float8_e4m3fn).as_strided((self.rows, self.K), (self.blocks * CODE_BLOCK, 1), self.buf.storage_offset())

    @property
    def scales(self):
        """The scale bytes e + 127, [rows (or 128-row blocks), blocks of K] (a view)."""
        n = -(-self.rows // self._rows_per_scale)
        run = -(-n // self._run_multiple) * self._run_multiple
        at = -(-self.rows * self.blocks * CODE_BLOCK // 256) * 256
        return self.buf.as_strided((n, self.blocks), (1, run), self.buf.storage_offset() + at)


class ActCode(_Code):
    """8-bit activations [T, K]: one scale per token and 128 k.  The coded
    operand of coded_linear and the checkpoint of the backward calls."""

    @property
    def T(self) -> int:
        return self.rows

    def expand(self, out=None, stream=None):
        """The bf16 values [T, K] the codes stand for."""
        import torch
        with _scope(self.buf.device, stream):
            if out is None:
                out = torch.empty((self.rows, self.K), dtype=torch.bfloat16, device=self.buf.device)
            _check_tensor(out, "out", (self.rows, self.K), torch.bfloat16, self.buf.device)
            _check(lib().weightless_act_expand(self.buf.data_ptr(), self.buf.numel(), self.rows, self.K,
                                               out.data_ptr(), _raw_stream(self.buf.device)))
        return out


class WeightCode(_Code):
    """8-bit weight [N, K]: one scale per 128 x 128 block."""

    _rows_per_scale, _run_multiple, _bytes = CODE_BLOCK, 4, "weightless_weight_code_bytes"

    def __init__(self, rows: int, K: int, device="cuda", buf=None):
        super().__init__(rows, K, device, buf)
        self._linear_need = {}   # T -> workspace bytes

    @property
    def N(self) -> int:
        return self.rows

    def workspace_bytes(self, T: int) -> int:
        """Workspace bytes of coded_linear with T tokens (0: none needed)."""
        need = self._linear_need.get(T)
        if need is None:
            need = lib().weightless_coded_linear_workspace_bytes(self.rows, self.K, T)
            self._linear_need[T] = need
        return need


def _code_out(cls, rows, K, device, out):
    if out is None:
        return cls(rows, K, device)
    if not isinstance(out, cls) or (out.rows, out.K) != (rows, K) or out.buf.device != device:
        raise WlError(-1, f"out must be a {cls.__name__} of {rows} x {K} on {device}")
    return out


def encode_act(x, out: Optional[ActCode] = None, stream=None) -> ActCode:
    """Code activations x bf16 [T, K] (weightless_act_encode)."""
    import torch
    _check_tensor(x, "x", (None, None), torch.bfloat16)
    with _scope(x.device, stream):
        out = _code_out(ActCode, x.shape[0], x.shape[1], x.device, out)
        _check(lib().weightless_act_encode(x.data_ptr(), out.rows, out.K, out.buf.data_ptr(), out.buf.numel(),
                                           _raw_stream(x.device)))
    return out


def encode_weight(w, out: Optional[WeightCode] = None, stream=None) -> WeightCode:
    """Code a weight w bf16 [N, K] (weightless_weight_encode)."""
    import torch
    _check_tensor(w, "w", (None, None), torch.bfloat16)
    with _scope(w.device, stream):
        out = _code_out(WeightCode, w.shape[0], w.shape[1], w.device, out)
        _check(lib().weightless_weight_encode(w.data_ptr(), out.rows, out.K, out.buf.data_ptr(), out.buf.numel(),
                                              _raw_stream(w.device)))
    return out


def coded_linear(w: WeightCode, x, y=None, code: Optional[ActCode] = None, ws=None, stream=None):
    """y = x w^T in 8 bits, bf16 [T, N] (weightless_coded_linear).

    x: bf16 [T, K], coded first (into `code`, if given: the checkpoint to
    keep), or an ActCode that already holds the coded activations."""
    import torch
    if not isinstance(w, WeightCode):
        raise WlError(-1, "w must be a WeightCode")
    dev = w.buf.device
    with _scope(dev, stream):
        if isinstance(x, ActCode):
            if code is not None:
                raise WlError(-1, "code is only for a bf16 x")
            if x.K != w.K or x.buf.device != dev:
                raise WlError(-1, f"x is coded as [{x.T}, {x.K}] on {x.buf.device}, the weight is "
                                  f"[{w.N}, {w.K}] on {dev}")
            code, src = x, None
        else:
            _check_tensor(x, "x", (None, w.K), torch.bfloat16, dev)
            code, src = _code_out(ActCode, x.shape[0], w.K, dev, code), x.data_ptr()
        T = code.rows
        if y is None:
            y = torch.empty((T, w.rows), dtype=torch.bfloat16, device=dev)
        else:
            _check_tensor(y, "y", (T, w.rows), torch.bfloat16, dev)
        if ws is not None:
            _check_tensor(ws, "ws", (None,), torch.uint8, dev)
        elif w.workspace_bytes(T):
            ws = torch.empty(w.workspace_bytes(T), dtype=torch.uint8, device=dev)
        _check(lib().weightless_coded_linear(w.buf.data_ptr(), w.buf.numel(), w.rows, w.K, src, code.buf.data_ptr(),
                                             code.buf.numel(), T, y.data_ptr(),
                                             ws.data_ptr() if ws is not None else None,
                                             ws.numel() if ws is not None else 0, _raw_stream(dev)))
    return y


# ---- norm before a projection ----------------------------------------------

class Normed(NamedTuple):
    """Outputs of norm_act (None: not asked for)."""
    y: object = None
    code: object = None
    h: object = None
    rstd: object = None


class NormGrads(NamedTuple):
    """Gradients of norm_act (None: not asked for)."""
    dx: object = None
    dw: object = None


def _norm_weight(w, K, dev):
    import torch
    _check_tensor(w, "weight", (K,), torch.float32 if w.dtype == torch.float32 else torch.bfloat16, dev)
    return w.data_ptr(), WL_DTYPE_F32 if w.dtype == torch.float32 else WL_DTYPE_BF16


def _output(t, name, shape, dtype, dev, like=None):
    """The caller's tensor for an output, or a new one (like: a tensor of that kind)."""
    import torch
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev) if like is None else torch.empty_like(like)
    _check_tensor(t, name, shape, dtype, dev)
    return t


def _only_wanted(want, known, given):
    unknown = [name for name in want if name not in known]
    if unknown or not want:
        raise WlError(-1, f"unknown outputs {sorted(unknown)}" if unknown else "no output is asked for")
    for name, t in given.items():
        if t is not None and name not in want:
            raise WlError(-1, f"{name} is given but not wanted")


def norm_act(x, weight, eps: float = 1e-6, residual=None, offset: float = 0.0, want=("y",), y=None,
             code: Optional[ActCode] = None, h=None, rstd=None, stream=None) -> Normed:
    """Root-mean-square norm of x (+ residual), bf16 [T, K], contiguous (weightless_norm).

    weight: bf16 or float32 [K], added to `offset`.  want: which of y (bf16),
    code (ActCode of y: coded_linear's operand and the backward calls'
    checkpoint), h (bf16, x + residual) and rstd (float32 [T]); y, code, h and
    rstd are written if given, allocated otherwise.  h may be x or residual."""
    import torch
    _check_tensor(x, "x", (None, None), torch.bfloat16)
    dev, (T, K) = x.device, x.shape
    _only_wanted(want, Normed._fields, {"y": y, "code": code, "h": h, "rstd": rstd})
    with _scope(dev, stream):
        if residual is not None:
            _check_tensor(residual, "residual", (T, K), torch.bfloat16, dev)
        w, wt = _norm_weight(weight, K, dev)
        y = _output(y, "y", (T, K), torch.bfloat16, dev, x) if "y" in want else None
        code = _code_out(ActCode, T, K, dev, code) if "code" in want else None
        h = _output(h, "h", (T, K), torch.bfloat16, dev, x) if "h" in want else None
        rstd = _output(rstd, "rstd", (T,), torch.float32, dev) if "rstd" in want else None
        _check(lib().weightless_norm(x.data_ptr(), None if residual is None else residual.data_ptr(), T, K, w, wt,
                                     offset, eps, None if h is None else h.data_ptr(),
                                     None if y is None else y.data_ptr(), None if code is None else code.buf.data_ptr(),
                                     0 if code is None else code.buf.numel(),
                                     None if rstd is None else rstd.data_ptr(), _raw_stream(dev)))
    return Normed(y, code, h, rstd)


def norm_backward(dy, h, rstd, weight, offset: float = 0.0, dh=None, want=("dx", "dw"), dx=None, dw=None, ws=None,
                  stream=None) -> NormGrads:
    """Gradients of norm_act (weightless_norm_backward).

    dy: bf16 [T, K], the gradient of y; h, rstd: norm_act's; dh: the gradient
    that reaches h past the norm, or None.  dx is the gradient of x and of the
    residual alike, bf16 (may be given as dy or dh); dw float32 [K]."""
    import torch
    _check_tensor(dy, "dy", (None, None), torch.bfloat16)
    dev, (T, K) = dy.device, dy.shape
    _only_wanted(want, NormGrads._fields, {"dx": dx, "dw": dw})
    with _scope(dev, stream):
        _check_tensor(h, "h", (T, K), torch.bfloat16, dev)
        _check_tensor(rstd, "rstd", (T,), torch.float32, dev)
        if dh is not None:
            _check_tensor(dh, "dh", (T, K), torch.bfloat16, dev)
        w, wt = _norm_weight(weight, K, dev)
        dx = _output(dx, "dx", (T, K), torch.bfloat16, dev, dy) if "dx" in want else None
        dw = _output(dw, "dw", (K,), torch.float32, dev) if "dw" in want else None
        if ws is not None:
            _check_tensor(ws, "ws", (None,), torch.uint8, dev)
        elif dw is not None:
            need = lib().weightless_norm_backward_workspace_bytes(T, K)
            if need == 0:
                raise WlError(-2, last_error())
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
        _check(lib().weightless_norm_backward(dy.data_ptr(), h.data_ptr(), rstd.data_ptr(),
                                              None if dh is None else dh.data_ptr(), T, K, w, wt, offset,
                                              None if dx is None else dx.data_ptr(),
                                              None if dw is None else dw.data_ptr(),
                                              None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(),
                                              _raw_stream(dev)))
    return NormGrads(dx, dw)


# ---- low-rank adapters of many requests -------------------------------------

class AdapterGrads(NamedTuple):
    """Gradients of AdapterPool.add (None: not asked for)."""
    dx: object = None
    du: object = None
    dv: object = None


class AdapterPool:
    """Slots of low-rank adapters beside one projection or one stacked call
    (wl_adapters): y[t] = base[t] + scale U (V^T x[t]) with the slot index[t].

    vt: bf16 [slots, children * rank, K], the children's V^T rows one after the
    other; u: bf16 [slots, sum of out_dims, rank]; scale: float32 [slots]; rank:
    int32 [slots], the ranks in use, or None for all of them (what vt and u hold
    from a slot's rank on is not used).  The pool keeps these tensors and reads
    what they hold when a call runs."""

    def __init__(self, vt, u, scale, out_dims: Sequence[int], rank=None):
        import torch
        _check_tensor(vt, "vt", (None, None, None), torch.bfloat16)
        dev, n, kids = vt.device, vt.shape[0], len(out_dims)
        if not 1 <= kids <= 3 or vt.shape[1] % kids:
            raise WlError(-2, f"{vt.shape[1]} rows of vt for {kids} children")
        room = vt.shape[1] // kids
        _check_tensor(u, "u", (n, sum(out_dims), room), torch.bfloat16, dev)
        _check_tensor(scale, "scale", (n,), torch.float32, dev)
        if rank is not None:
            _check_tensor(rank, "rank", (n,), torch.int32, dev)
        self.vt, self.u, self.scale, self.rank, self.out_dims = vt, u, scale, rank, tuple(out_dims)
        self.device, self.slots, self.room, self.K, self.width = dev, n, room, vt.shape[2], sum(out_dims)
        self.spec = WlAdapters(n, room, self.K, kids, (ctypes.c_int32 * 3)(*out_dims), vt.data_ptr(), u.data_ptr(),
                               scale.data_ptr(), None if rank is None else rank.data_ptr())
        self._ref = ctypes.byref(self.spec)
        self._need = {}          # T -> workspace bytes
        self._backward_need = {}
        self.workspace_bytes(1)  # refuses dimensions the library does not take

    @classmethod
    def empty(cls, slots: int, rank: int, K: int, out_dims: Sequence[int], device="cuda") -> "AdapterPool":
        """A pool whose slots are all free (rank 0): tokens sent to them run
        without an adapter until load() fills them."""
        import torch
        dev = torch.device(device)
        return cls(torch.zeros((slots, len(out_dims) * rank, K), dtype=torch.bfloat16, device=dev),
                   torch.zeros((slots, sum(out_dims), rank), dtype=torch.bfloat16, device=dev),
                   torch.zeros((slots,), dtype=torch.float32, device=dev), out_dims,
                   torch.zeros((slots,), dtype=torch.int32, device=dev))

    def load(self, slot: int, down, up, scale: float = 1.0):
        """Fill a slot on the current stream.  down: per child [r, K] (V^T); up:
        per child [N, r] (U); one rank r <= the pool's for all children."""
        kids = len(self.out_dims)
        r = down[0].shape[0] if len(down) else 0
        if not 0 <= slot < self.slots or len(down) != kids or len(up) != kids or not 1 <= r <= self.room \
                or any(tuple(a.shape) != (r, self.K) or tuple(b.shape) != (n, r) for a, b, n in zip(down, up, self.out_dims)):
            raise WlError(-1, f"slot {slot} takes {kids} pairs of [r, {self.K}] and [N, r], N = {self.out_dims}, r <= {self.room}")
        if self.rank is None and r != self.room:
            raise WlError(-1, f"this pool has no ranks: every slot takes rank {self.room}")
        at = 0
        for c, (a, b, n) in enumerate(zip(down, up, self.out_dims)):
            self.vt[slot, c * self.room:c * self.room + r].copy_(a)
            self.u[slot, at:at + n, :r].copy_(b)
            at += n
        self.scale[slot] = scale
        if self.rank is not None:
            self.rank[slot] = r

    def clear(self, slot: int):
        """Free a slot: tokens sent to it run without an adapter."""
        if self.rank is None or not 0 <= slot < self.slots:
            raise WlError(-1, f"slot {slot} of a pool with{'' if self.rank is not None else 'out'} ranks cannot be cleared")
        self.rank[slot] = 0

    def workspace_bytes(self, T: int) -> int:
        """Workspace bytes of add() with T tokens (fewer can need more)."""
        need = self._need.get(T)
        if need is None:
            need = lib().weightless_adapters_workspace_bytes(self._ref, T)
            if need == 0:
                raise WlError(-2, last_error())
            self._need[T] = need
        return need

    def add(self, x, index, base, y=None, ws=None, stream=None):
        """y[t] = base[t] + scale U (V^T x[t]), bf16 [T, N] (weightless_adapters_add).

        x: bf16 [T, K]; index: int32 [T], each token's slot (outside the pool:
        none); base: bf16 [T, N], the shared projection's output; y may be base."""
        import torch
        dev = self.device
        _check_tensor(x, "x", (None, self.K), torch.bfloat16, dev)
        T = x.shape[0]
        with _scope(dev, stream):
            _check_tensor(index, "index", (T,), torch.int32, dev)
            _check_tensor(base, "base", (T, self.width), torch.bfloat16, dev)
            y = _output(y, "y", (T, self.width), torch.bfloat16, dev, base)
            if ws is None:
                ws = torch.empty(self.workspace_bytes(T), dtype=torch.uint8, device=dev)
            else:
                _check_tensor(ws, "ws", (None,), torch.uint8, dev)
            _check(lib().weightless_adapters_add(self._ref, x.data_ptr(), index.data_ptr(), T, base.data_ptr(),
                                                 y.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(dev)))
        return y

    def backward_workspace_bytes(self, T: int) -> int:
        """Workspace bytes of backward() with T tokens (fewer can need more)."""
        need = self._backward_need.get(T)
        if need is None:
            need = lib().weightless_adapters_backward_workspace_bytes(self._ref, T)
            if need == 0:
                raise WlError(-2, last_error())
            self._backward_need[T] = need
        return need

    def backward(self, x: ActCode, dy, index, base=None, want=("dx", "du", "dv"), dx=None, du=None, dv=None, ws=None,
                 stream=None) -> AdapterGrads:
        """Gradients of add() (weightless_adapters_backward).

        x: the ActCode checkpoint of the call's input; dy: bf16 [T, N]; base: bf16
        [T, K], the shared projection's dx, which dx adds to (dx may be base).
        du and dv have u's and vt's shapes, bf16, written for every slot; outputs are
        allocated if not given."""
        import torch
        dev = self.device
        if not isinstance(x, ActCode) or x.K != self.K or x.buf.device != dev:
            raise WlError(-1, f"x must be an ActCode of K = {self.K} on {dev}")
        T = x.T
        _only_wanted(want, AdapterGrads._fields, {"dx": dx, "du": du, "dv": dv})
        if (base is not None) != ("dx" in want):
            raise WlError(-1, "base goes with dx")
        with _scope(dev, stream):
            _check_tensor(dy, "dy", (T, self.width), torch.bfloat16, dev)
            _check_tensor(index, "index", (T,), torch.int32, dev)
            g = WlAdapterGrads()
            if "dx" in want:
                _check_tensor(base, "base", (T, self.K), torch.bfloat16, dev)
                dx = _output(dx, "dx", (T, self.K), torch.bfloat16, dev, base)
                g.base, g.dx = base.data_ptr(), dx.data_ptr()
            if "du" in want:
                du = _output(du, "du", tuple(self.u.shape), torch.bfloat16, dev, self.u)
                g.du = du.data_ptr()
            if "dv" in want:
                dv = _output(dv, "dv", tuple(self.vt.shape), torch.bfloat16, dev, self.vt)
                g.dv = dv.data_ptr()
            if ws is None:
                ws = torch.empty(self.backward_workspace_bytes(T), dtype=torch.uint8, device=dev)
            else:
                _check_tensor(ws, "ws", (None,), torch.uint8, dev)
            _check(lib().weightless_adapters_backward(self._ref, x.buf.data_ptr(), x.buf.numel(), dy.data_ptr(),
                                                      index.data_ptr(), T, ctypes.byref(g), ws.data_ptr(), ws.numel(),
                                                      _raw_stream(dev)))
        return AdapterGrads(dx, du, dv)
