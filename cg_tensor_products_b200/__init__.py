"""Python binding of libetp.so, the B200 edge-wise equivariant tensor product library.

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels (see include/etp.h for the operation, layouts and conventions).
PyTorch supplies device memory and the current stream. There is no CPU path:
tensors must live on a CUDA device, and a missing library raises.

    plan = Plan("0..3", 3, "0..3", C=128)
    out = forward(plan, row_ptr, src, r, x, w)
    rev_ptr, rev_perm, dst = build_reverse_csr(N, row_ptr, src)
    gx, gw, gr = backward(plan, row_ptr, src, rev_ptr, rev_perm, dst, r, x, w, grad_out)

A call given stream=s runs on s and allocates there what it creates; results may be used on s, or on the caller's
current stream once that waits for s. Inputs have to be ready on s and alive until it has passed the call.

The dense row operators (include/etp_dense.h) need no plan; they read blocks of node features in place:

    h, mean, rstd = layer_norm_forward(x[:, :1], weight, bias)
    out, z = linear_forward(h, W, b, activation="silu", residual=x[:, :1], save_z=True)
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libetp.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "etp.h")
DENSE_HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "etp_dense.h")

ETP_OK, ETP_ERR_INVALID_ARG, ETP_ERR_UNSUPPORTED, ETP_ERR_BAD_CSR = 0, 1, 2, 3
ETP_ERR_CUDA, ETP_ERR_ALLOC, ETP_ERR_WORKSPACE, ETP_ERR_TOO_LARGE = 4, 5, 6, 7
STATIC_MAX_NODES = STATIC_MAX_EDGES = 1 << 18
FRAME_FLOATS = 88  # floats of one edge frame record (ETP_FRAME_FLOATS)
ETP_F32, ETP_BF16 = 0, 1
ACT_NONE, ACT_SILU = 0, 1
LINEAR_MAX_CHANNELS, NORM_MAX_CHANNELS = 65536, 8192
CSR_BAD_ENDPOINTS, CSR_NOT_MONOTONE, CSR_SRC_RANGE = 1, 2, 4

_lib = None


class EtpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _load().etp_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: {msg} (status {status})")


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m cg_tensor_products_b200.build` "
                           "(or __graft_entry__.build()); there is no fallback implementation")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sig = {
        "etp_plan_create": [ctypes.POINTER(vp), ctypes.c_char_p, i32, ctypes.c_char_p, i32, i32],
        "etp_plan_info": [vp, vp, vp, vp, vp, vp],
        "etp_plan_couplings": [vp, vp, vp, vp, vp, vp, vp],
        "etp_plan_destroy": [vp],
        "etp_plan_frames_advised": [vp, i32, ctypes.POINTER(i32)],
        "etp_edge_frames": [vp, i32, vp, vp, vp],
        "etp_tp_workspace_size": [vp, i32, i32, i32, ctypes.POINTER(sz)],
        "etp_forward": [vp, i32, i32] + [vp] * 7 + [vp, sz, vp],
        "etp_backward": [vp, i32, i32] + [vp] * 13 + [vp, sz, vp],
        "etp_double_backward": [vp, i32, i32] + [vp] * 16 + [vp, sz, vp],
        "etp_cart_forward": [vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "etp_cart_backward": [vp, i32, i32] + [vp] * 12 + [vp, sz, vp],
        "etp_assemble_forces": [i32, i32, vp, vp, vp, vp, vp, vp, vp, vp],
        "etp_node_product": [vp, i32, i32, i32, vp, vp, vp, vp],
        "etp_node_product_ops": [vp, i32, ctypes.POINTER(i32)],
        "etp_radial_workspace_size": [vp, i32, i32, i32, ctypes.POINTER(sz)],
        "etp_radial_forward": [vp, i32, i32, i32, ctypes.c_float, vp, vp, vp, vp, vp, sz, vp],
        "etp_radial_backward": [vp, i32, i32, i32, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "etp_fused_workspace_size": [vp, i32, i32, i32, ctypes.POINTER(sz)],
        "etp_fused_forward": [vp, i32, i32, vp, vp, vp, vp, i32, i32, ctypes.c_float, vp, vp, vp, vp, sz, vp],
        "etp_reverse_csr_workspace_size": [i32, i32, ctypes.POINTER(sz)],
        "etp_build_reverse_csr": [i32, i32, vp, vp, vp, vp, vp, vp, sz, vp],
        "etp_build_reverse_csr_static": [i32, i32, vp, vp, vp, vp, vp, vp],
        "etp_validate_csr": [i32, i32, vp, vp, vp, vp],
        "etp_locality_schedule_workspace_size": [i32, i32, ctypes.POINTER(sz)],
        "etp_build_locality_schedule": [i32, i32, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "etp_forward_ordered": [vp, i32, i32] + [vp] * 10 + [sz, vp],
        "etp_backward_ordered": [vp, i32, i32] + [vp] * 13 + [sz, vp],
        "etp_linear_forward": [i32] * 5 + [vp, vp, vp, i32, vp, vp, vp, vp, sz, vp],
        "etp_linear_workspace_size": [i32] * 6 + [ctypes.POINTER(sz)],
        "etp_linear_backward": [i32] * 5 + [vp, vp, i32] + [vp] * 6 + [sz, vp],
        "etp_layer_norm_forward": [i32] * 4 + [ctypes.c_float] + [vp] * 7,
        "etp_layer_norm_workspace_size": [i32] * 4 + [ctypes.POINTER(sz)],
        "etp_layer_norm_backward": [i32] * 4 + [vp] * 9 + [sz, vp],
        "etp_device_fault": [vp],
        "etp_status_string": [i32],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name == "etp_status_string" else ctypes.c_int
    _lib = lib
    return lib


def declared_symbols(header: str = HEADER_PATH) -> list:
    """Function names declared in include/etp.h (or in another of the library's headers)."""
    with open(header) as f:
        txt = f.read()
    return re.findall(r"ETP_API\s+[\w\s\*]+?\b(etp_\w+)\s*\(", txt)


def _check(status: int, where: str):
    if status != ETP_OK:
        raise EtpError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need_cuda(*ts):
    """The one CUDA device all given tensors live on (None entries are skipped)."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors: this library has no CPU path")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on different devices ({dev}, {t.device})")
    return dev


def _tensors(v):
    """The tensors of an argument or a result: a tensor, a tuple or dict of them, a schedule."""
    if isinstance(v, Schedule):
        v = v.tensors()
    elif isinstance(v, dict):
        v = tuple(v.values())
    return [t for t in (v if isinstance(v, tuple) else (v,)) if hasattr(t, "record_stream")]


def _on_stream(stream, t, fn, *args):
    """fn(*args) with `stream`, which must belong to t's device, as the current one: the tensors that it allocates are
    that stream's. What it returns of them may be used on the caller's current stream too, so their memory is not
    given to later work before that stream has passed the point where they are dropped."""
    import torch

    if stream.device != t.device:
        raise ValueError(f"{fn.__name__}: stream on {stream.device}, tensors on {t.device}")
    caller = torch.cuda.current_stream(t.device)
    if caller == stream:
        return fn(*args)
    with torch.cuda.stream(stream):
        result = fn(*args)
    own = {id(u) for a in args for u in _tensors(a)}
    for r in _tensors(result):
        if id(r) not in own:
            r.record_stream(caller)
    return result


def _launch(dev, where: str, fn, *args):
    """Call library function `fn(*args, stream)` with the tensors' device current, on torch's current stream of it."""
    import torch

    with torch.cuda.device(dev):
        _check(fn(*args, ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)), where)


def _expect(t, name: str, dtype: str, shape: tuple):
    """Raise ValueError unless t (if given) has the dtype ('float32' / 'int32' / 'uint8') and the
    shape (None entries match any size); checked before anything is launched."""
    if t is None:
        return
    if str(t.dtype) != "torch." + dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(want is not None and got != want for got, want in zip(t.shape, shape)):
        raise ValueError(f"{name}: expected shape {tuple('*' if v is None else v for v in shape)}, "
                         f"got {tuple(t.shape)}")


def _check_graph(row_ptr, src, N: int, E: int):
    _expect(row_ptr, "row_ptr", "int32", (N + 1,))
    _expect(src, "src", "int32", (E,))


class Plan:
    """A tensor-product plan: irreps in x harmonics 0..sh_lmax -> irreps out, C channels, fp32."""

    def __init__(self, irreps_in: str, sh_lmax: int, irreps_out: str, C: int):
        lib = _load()
        h = ctypes.c_void_p()
        _check(lib.etp_plan_create(ctypes.byref(h), irreps_in.encode(), int(sh_lmax), irreps_out.encode(),
                                   int(C), ETP_F32), "etp_plan_create")
        self._h = h
        self.C = int(C)
        n_paths, d_in, d_sh, d_out = (ctypes.c_int() for _ in range(4))
        _check(lib.etp_plan_info(h, ctypes.byref(n_paths), ctypes.byref(d_in), ctypes.byref(d_sh),
                                 ctypes.byref(d_out), None), "etp_plan_info")
        self.n_paths, self.dim_in, self.dim_sh, self.dim_out = n_paths.value, d_in.value, d_sh.value, d_out.value
        arr = (ctypes.c_int * (3 * self.n_paths))()
        _check(lib.etp_plan_info(h, None, None, None, None, arr), "etp_plan_info")
        self.paths = [tuple(arr[3 * p:3 * p + 3]) for p in range(self.n_paths)]

    @property
    def handle(self):
        return self._h

    def couplings(self):
        """(path_off, m1, m2, m3, val) of the coefficients compiled into the kernels."""
        lib = _load()
        nnz = ctypes.c_int()
        _check(lib.etp_plan_couplings(self._h, ctypes.byref(nnz), None, None, None, None, None), "couplings")
        n = nnz.value
        off = (ctypes.c_int * (self.n_paths + 1))()
        m1, m2, m3 = ((ctypes.c_int * n)() for _ in range(3))
        val = (ctypes.c_double * n)()
        _check(lib.etp_plan_couplings(self._h, ctypes.byref(nnz), off, m1, m2, m3, val), "couplings")
        return list(off), list(m1), list(m2), list(m3), list(val)

    def frames_advised(self, E: int) -> bool:
        """Whether precomputed edge frame records pay for E edges (etp_plan_frames_advised)."""
        v = ctypes.c_int()
        _check(_load().etp_plan_frames_advised(self._h, int(E), ctypes.byref(v)), "etp_plan_frames_advised")
        return bool(v.value)

    def close(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.etp_plan_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def edge_frames(plan: Plan, r, frames=None, stream=None):
    """Per-edge frame records [E][FRAME_FLOATS] for r (launches etp_edge_frames)."""
    import torch

    if stream is not None:
        return _on_stream(stream, r, edge_frames, plan, r, frames)
    _expect(r, "r", "float32", (None, 3))
    E = r.shape[0]
    if frames is None:
        frames = torch.empty((E, FRAME_FLOATS), device=r.device, dtype=torch.float32)
    _expect(frames, "frames", "float32", (E, FRAME_FLOATS))
    dev = _need_cuda(r, frames)
    _launch(dev, "etp_edge_frames", _load().etp_edge_frames, plan.handle, E, _ptr(r), _ptr(frames))
    return frames


def tp_workspace_size(plan: Plan, N: int, E: int, ordered: bool = False, device=None) -> int:
    """Bytes of partial-row workspace forward/backward (ordered: their schedule variants) need
    (etp_tp_workspace_size, answered for `device`, default the current one)."""
    import torch

    b = ctypes.c_size_t()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _check(_load().etp_tp_workspace_size(plan.handle, int(N), int(E), int(bool(ordered)), ctypes.byref(b)),
               "tp_workspace_size")
    return b.value


def _tp_workspace(plan, N, E, ordered, workspace, dev):
    """The caller's workspace (checked), or a new one of the needed size on dev."""
    import torch

    if workspace is None:
        n = tp_workspace_size(plan, N, E, ordered, dev)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    _expect(workspace, "workspace", "uint8", (None,))
    return workspace


def forward(plan: Plan, row_ptr, src, r, x, w, out=None, frames=None, workspace=None, stream=None):
    """out[i] = sum over row i of the weighted tensor products (launches etp_forward).
    frames: None, or edge_frames(plan, r) (then the kernel reads those instead of building them).
    workspace: uint8 device tensor of tp_workspace_size bytes (allocated when None)."""
    import torch

    if stream is not None:
        return _on_stream(stream, row_ptr, forward, plan, row_ptr, src, r, x, w, out, frames, workspace)
    N, E = row_ptr.numel() - 1, src.numel()
    _check_graph(row_ptr, src, N, E)
    _expect(r, "r", "float32", (E, 3))
    _expect(frames, "frames", "float32", (E, FRAME_FLOATS))
    _expect(x, "x", "float32", (N, plan.dim_in, plan.C))
    _expect(w, "w", "float32", (E, plan.n_paths, plan.C))
    if out is None:
        out = torch.empty((N, plan.dim_out, plan.C), device=x.device, dtype=torch.float32)
    _expect(out, "out", "float32", (N, plan.dim_out, plan.C))
    dev = _need_cuda(row_ptr, src, r, frames, x, w, out)
    workspace = _tp_workspace(plan, N, E, False, workspace, dev)
    _need_cuda(out, workspace)
    _launch(dev, "etp_forward", _load().etp_forward, plan.handle, N, E, _ptr(row_ptr), _ptr(src), _ptr(r),
            _ptr(frames), _ptr(x), _ptr(w), _ptr(out), _ptr(workspace), workspace.numel())
    return out


def backward(plan: Plan, row_ptr, src, rev_ptr, rev_perm, dst, r, x, w, grad_out,
             want=("x", "w", "r"), grad_x=None, grad_w=None, grad_r=None, frames=None, workspace=None, stream=None):
    """(grad_x, grad_w, grad_r) for the cotangent grad_out (launches etp_backward); unwanted ones are None."""
    import torch

    if stream is not None:
        return _on_stream(stream, row_ptr, backward, plan, row_ptr, src, rev_ptr, rev_perm, dst, r, x, w, grad_out,
                          want, grad_x, grad_w, grad_r, frames, workspace)
    N, E = row_ptr.numel() - 1, src.numel()
    _check_graph(row_ptr, src, N, E)
    _expect(rev_ptr, "rev_ptr", "int32", (N + 1,))
    _expect(rev_perm, "rev_perm", "int32", (E,))
    _expect(dst, "dst", "int32", (E,))
    _expect(r, "r", "float32", (E, 3))
    _expect(frames, "frames", "float32", (E, FRAME_FLOATS))
    _expect(x, "x", "float32", (N, plan.dim_in, plan.C))
    _expect(w, "w", "float32", (E, plan.n_paths, plan.C))
    _expect(grad_out, "grad_out", "float32", (N, plan.dim_out, plan.C))
    dev = x.device
    if "x" in want and grad_x is None:
        grad_x = torch.empty((N, plan.dim_in, plan.C), device=dev, dtype=torch.float32)
    if "w" in want and grad_w is None:
        grad_w = torch.empty((E, plan.n_paths, plan.C), device=dev, dtype=torch.float32)
    if "r" in want and grad_r is None:
        grad_r = torch.empty((E, 3), device=dev, dtype=torch.float32)
    _expect(grad_x, "grad_x", "float32", (N, plan.dim_in, plan.C))
    _expect(grad_w, "grad_w", "float32", (E, plan.n_paths, plan.C))
    _expect(grad_r, "grad_r", "float32", (E, 3))
    dev = _need_cuda(row_ptr, src, rev_ptr, rev_perm, dst, r, frames, x, w, grad_out, grad_x, grad_w, grad_r)
    workspace = _tp_workspace(plan, N, E, False, workspace, dev)
    _need_cuda(x, workspace)
    _launch(dev, "etp_backward", _load().etp_backward, plan.handle, N, E, _ptr(row_ptr), _ptr(src), _ptr(rev_ptr),
            _ptr(rev_perm), _ptr(dst), _ptr(r), _ptr(frames), _ptr(x), _ptr(w), _ptr(grad_out), _ptr(grad_x),
            _ptr(grad_w), _ptr(grad_r), _ptr(workspace), workspace.numel())
    return grad_x, grad_w, grad_r


def cart_forward(plan: Plan, row_ptr, src, r, x, w, out=None, workspace=None, stream=None):
    """Cartesian edge convolution (launches etp_cart_forward): x and out in independent STF components."""
    import torch

    if stream is not None:
        return _on_stream(stream, row_ptr, cart_forward, plan, row_ptr, src, r, x, w, out, workspace)
    N, E = row_ptr.numel() - 1, src.numel()
    _check_graph(row_ptr, src, N, E)
    _expect(r, "r", "float32", (E, 3))
    _expect(x, "x", "float32", (N, plan.dim_in, plan.C))
    _expect(w, "w", "float32", (E, plan.n_paths, plan.C))
    if out is None:
        out = torch.empty((N, plan.dim_out, plan.C), device=x.device, dtype=torch.float32)
    _expect(out, "out", "float32", (N, plan.dim_out, plan.C))
    dev = _need_cuda(row_ptr, src, r, x, w, out)
    workspace = _tp_workspace(plan, N, E, False, workspace, dev)
    _need_cuda(out, workspace)
    _launch(dev, "etp_cart_forward", _load().etp_cart_forward, plan.handle, N, E, _ptr(row_ptr), _ptr(src), _ptr(r),
            _ptr(x), _ptr(w), _ptr(out), _ptr(workspace), workspace.numel())
    return out


def node_product(plan: Plan, x, w, K=None, cartesian=False, out=None, stream=None):
    """Node-local product of correlation order K (launches etp_node_product): out = B(K) with
    B(1) = x, B(k+1) = sum_p w[k-1, p] couple_p(B(k), x). x [N, D, C]; w [K-1, P, C] (K defaults
    to w.shape[0] + 1; w may be None for K = 1); spherical or Cartesian (independent STF
    components) couplings."""
    import torch

    if stream is not None:
        return _on_stream(stream, x, node_product, plan, x, w, K, cartesian, out)
    N = x.shape[0] if x.dim() == 3 else -1
    _expect(x, "x", "float32", (N, plan.dim_in, plan.C))
    if K is None:
        if w is None:
            raise ValueError("give K or w")
        K = w.shape[0] + 1
    if K < 1:
        raise ValueError(f"K must be >= 1, got {K}")
    if K > 1:
        if w is None:
            raise ValueError("w is required for K > 1")
        _expect(w, "w", "float32", (K - 1, plan.n_paths, plan.C))
    if out is None:
        out = torch.empty((N, plan.dim_out, plan.C), device=x.device, dtype=torch.float32)
    _expect(out, "out", "float32", (N, plan.dim_out, plan.C))
    for t in (x, w if K > 1 else None):
        if t is not None and t.numel() and out.numel() and \
                out.data_ptr() < t.data_ptr() + 4 * t.numel() and t.data_ptr() < out.data_ptr() + 4 * out.numel():
            raise ValueError("out must not overlap x or w")
    dev = _need_cuda(x, out, *([w] if K > 1 else []))
    _launch(dev, "etp_node_product", _load().etp_node_product, plan.handle, N, int(K), int(bool(cartesian)),
            _ptr(x), _ptr(w) if K > 1 else None, _ptr(out))
    return out


def node_product_ops(plan: Plan, cartesian=False) -> int:
    """FP32 operations per node, channel and step of the node-local product kernel."""
    n = ctypes.c_int()
    _check(_load().etp_node_product_ops(plan.handle, int(bool(cartesian)), ctypes.byref(n)), "node product ops")
    return n.value


def cart_backward(plan: Plan, row_ptr, src, rev_ptr, rev_perm, dst, r, x, w, grad_out, want=("x", "w", "r"),
                  workspace=None, stream=None):
    """VJP of cart_forward (launches etp_cart_backward): (grad_x, grad_w, grad_r), unwanted ones None."""
    import torch

    if stream is not None:
        return _on_stream(stream, row_ptr, cart_backward, plan, row_ptr, src, rev_ptr, rev_perm, dst, r, x, w,
                          grad_out, want, workspace)
    N, E = row_ptr.numel() - 1, src.numel()
    _check_graph(row_ptr, src, N, E)
    _expect(rev_ptr, "rev_ptr", "int32", (N + 1,))
    _expect(rev_perm, "rev_perm", "int32", (E,))
    _expect(dst, "dst", "int32", (E,))
    _expect(r, "r", "float32", (E, 3))
    _expect(x, "x", "float32", (N, plan.dim_in, plan.C))
    _expect(w, "w", "float32", (E, plan.n_paths, plan.C))
    _expect(grad_out, "grad_out", "float32", (N, plan.dim_out, plan.C))
    dev = x.device
    gx = torch.empty((N, plan.dim_in, plan.C), device=dev, dtype=torch.float32) if "x" in want else None
    gw = torch.empty((E, plan.n_paths, plan.C), device=dev, dtype=torch.float32) if "w" in want else None
    gr = torch.empty((E, 3), device=dev, dtype=torch.float32) if "r" in want else None
    dev = _need_cuda(row_ptr, src, rev_ptr, rev_perm, dst, r, x, w, grad_out, gx, gw, gr)
    workspace = _tp_workspace(plan, N, E, False, workspace, dev)
    _need_cuda(x, workspace)
    _launch(dev, "etp_cart_backward", _load().etp_cart_backward, plan.handle, N, E, _ptr(row_ptr), _ptr(src),
            _ptr(rev_ptr), _ptr(rev_perm), _ptr(dst), _ptr(r), _ptr(x), _ptr(w), _ptr(grad_out), _ptr(gx), _ptr(gw),
            _ptr(gr), _ptr(workspace), workspace.numel())
    return gx, gw, gr


def double_backward(plan: Plan, row_ptr, src, rev_ptr, rev_perm, dst, r, x, w, grad_out, gg_x=None, gg_w=None,
                    gg_r=None, want=("g", "x", "w", "r"), out=None, workspace=None, stream=None):
    """VJP of the VJP (launches etp_double_backward): dict with 'grad_g', 'grad_x', 'grad_w', 'grad_r'
    (the wanted ones) of <gg_x, grad_x> + <gg_w, grad_w> + <gg_r, grad_r>; None cotangents are zero."""
    import torch

    if stream is not None:
        return _on_stream(stream, row_ptr, double_backward, plan, row_ptr, src, rev_ptr, rev_perm, dst, r, x, w,
                          grad_out, gg_x, gg_w, gg_r, want, out, workspace)
    N, E = row_ptr.numel() - 1, src.numel()
    _check_graph(row_ptr, src, N, E)
    _expect(rev_ptr, "rev_ptr", "int32", (N + 1,))
    _expect(rev_perm, "rev_perm", "int32", (E,))
    _expect(dst, "dst", "int32", (E,))
    _expect(r, "r", "float32", (E, 3))
    for t, name in ((x, "x"), (gg_x, "gg_x")):
        _expect(t, name, "float32", (N, plan.dim_in, plan.C))
    for t, name in ((w, "w"), (gg_w, "gg_w")):
        _expect(t, name, "float32", (E, plan.n_paths, plan.C))
    _expect(grad_out, "grad_out", "float32", (N, plan.dim_out, plan.C))
    _expect(gg_r, "gg_r", "float32", (E, 3))
    shapes = {"g": (N, plan.dim_out, plan.C), "x": (N, plan.dim_in, plan.C), "w": (E, plan.n_paths, plan.C),
              "r": (E, 3)}
    out = dict(out or {})
    for k in "gxwr":
        key = "grad_" + k
        if k in want and out.get(key) is None:
            out[key] = torch.empty(shapes[k], device=x.device, dtype=torch.float32)
        _expect(out.get(key), key, "float32", shapes[k])
    dev = _need_cuda(row_ptr, src, rev_ptr, rev_perm, dst, r, x, w, grad_out, gg_x, gg_w, gg_r, *out.values())
    workspace = _tp_workspace(plan, N, E, False, workspace, dev)
    _need_cuda(x, workspace)
    _launch(dev, "etp_double_backward", _load().etp_double_backward, plan.handle, N, E, _ptr(row_ptr), _ptr(src),
            _ptr(rev_ptr), _ptr(rev_perm), _ptr(dst), _ptr(r), _ptr(x), _ptr(w), _ptr(grad_out), _ptr(gg_x),
            _ptr(gg_w), _ptr(gg_r), _ptr(out.get("grad_g")), _ptr(out.get("grad_x")), _ptr(out.get("grad_w")),
            _ptr(out.get("grad_r")), _ptr(workspace), workspace.numel())
    return out


class _Rows(ctypes.Structure):
    """etp_rows: rows of channels at data + group * group_stride + row * row_stride."""
    _fields_ = [("data", ctypes.c_void_p), ("group_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64)]


_INT_MAX = 2**31 - 1
_DENSE_TYPES = {"torch.float32": ETP_F32, "torch.bfloat16": ETP_BF16}
_ACTIVATIONS = {None: ACT_NONE, "none": ACT_NONE, "silu": ACT_SILU}


def _dense_lead(x, channels=None):
    """(leading sizes, C) of x [M, C] or [groups, rows, C]; channels: the C it must have."""
    shape = tuple(x.shape)
    if len(shape) != 2 and len(shape) != 3:
        raise ValueError(f"x: expected [rows, channels] or [groups, rows, channels], got {shape}")
    if channels is not None and shape[-1] != channels:
        raise ValueError(f"x: expected {channels} channels, got {shape[-1]}")
    if max(shape) > _INT_MAX:  # the C call's sizes are ints
        raise EtpError(ETP_ERR_TOO_LARGE, "x")
    return shape[:-1], shape[-1]


def _dense_rows(t, name: str, dtype, lead, C: int):
    """etp_rows of a tensor of the given dtype and sizes (*lead, C) whose channels are contiguous (None for None)."""
    if t is None:
        return None
    st = t.stride()
    if t.dtype is not dtype or t.shape != (*lead, C) or (st[-1] != 1 and C > 1):
        shape = tuple(t.shape)
        if t.dtype is not dtype:
            raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
        if shape[:-1] != lead:
            raise ValueError(f"{name}: expected leading sizes {lead}, got {shape[:-1]}")
        if shape[-1] != C:
            raise ValueError(f"{name}: expected {C} channels, got {shape[-1]}")
        raise ValueError(f"{name}: channels must be contiguous (stride {st[-1]})")
    return ctypes.byref(_Rows(t.data_ptr(), st[0], st[1] if len(st) == 3 else 0))


def _dense_new(x, lead, C: int):
    """(a new contiguous tensor of sizes (*lead, C) like x, its etp_rows)."""
    import torch

    t = torch.empty_like(x) if x.shape[-1] == C and x.is_contiguous() else x.new_empty((*lead, C))
    return t, ctypes.byref(_Rows(t.data_ptr(), C if len(lead) == 1 else lead[1] * C, C))


def _dense_code(dtype):
    """etp_dtype of a torch dtype or its name."""
    code = _DENSE_TYPES.get("torch." + str(dtype).replace("torch.", ""))
    if code is None:
        raise ValueError(f"dtype: expected float32 or bfloat16, got {dtype}")
    return code


def _dense_index(device):
    """Index of a CUDA device (None, or one without an index: the current one)."""
    import torch

    index = None if device is None else torch.device(device).index
    return torch.cuda.current_device() if index is None else index


def _dense_type(x):
    code = _DENSE_TYPES.get(str(x.dtype))
    if code is None:
        raise ValueError(f"x: expected float32 or bfloat16, got {x.dtype}")
    return code


def _dense_vector(t, name: str, dtype, *shape):
    """Address of a contiguous tensor of the given dtype and shape (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} of shape {shape}, got {t.dtype} of shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _dense_device(x, *ts):
    """Index of the CUDA device of x, which the other tensors (None entries are skipped) must share."""
    index = x.get_device()
    for t in ts:
        if t is not None and t.get_device() != index or index < 0:
            if index < 0 or t.get_device() < 0:
                raise ValueError("tensors must be CUDA tensors: this library has no CPU path")
            raise ValueError(f"tensors on different devices ({x.device}, {t.device})")
    return index


def _dense_call(index: int, where: str, fn, *args):
    """fn(*args, stream) with device `index` current, on torch's current stream of it."""
    import torch

    raw = torch._C._cuda_getCurrentRawStream(index)
    if torch.cuda.current_device() == index:  # switching costs more than a small launch
        status = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            status = fn(*args, raw)
    if status != ETP_OK:
        raise EtpError(status, where)


@functools.lru_cache(maxsize=1024)
def _dense_bytes(index: int, name: str, *args) -> int:
    """Bytes that the size function `name` answers for these sizes on device `index` (they depend on nothing else)."""
    import torch

    if max(args) > _INT_MAX or min(args) < -_INT_MAX:
        raise EtpError(ETP_ERR_TOO_LARGE, name)
    b = ctypes.c_size_t()
    with torch.cuda.device(index):
        _check(getattr(_load(), name)(*args, ctypes.byref(b)), name)
    return b.value


def _dense_workspace(index: int, workspace, name: str, *args):
    """(workspace or None, its bytes): the caller's, checked, or a new one when the call needs any."""
    if workspace is not None:
        _expect(workspace, "workspace", "uint8", (None,))
        if not workspace.is_contiguous():
            raise ValueError("workspace: must be contiguous")
        return workspace, workspace.numel()
    n = _dense_bytes(index, name, *args)
    if n == 0:
        return None, 0
    import torch

    return torch.empty(n, dtype=torch.uint8, device=torch.device("cuda", index)), n


def _boxes_meet(d: int, dims) -> bool:
    """Whether two boxes of elements share one. Box a starts at 0, box b at d; dims, from the outermost in: (stride,
    a's size, b's size), the last of stride 1. A stride that does not clear what lies inside it: True (they may)."""
    s, na, nb = dims[0]
    if len(dims) == 1:
        return -nb < d < na
    inside = [1 + sum((n[i] - 1) * n[0] for n in dims[1:]) for i in (1, 2)]
    if s < max(inside):
        return True
    q, r = divmod(d, s)  # b's slot of index j is a's slot q + j, shifted by r, and reaches into the next
    return any(-nb < k < na and _boxes_meet(e, dims[1:]) for k, e in ((q, r), (q + 1, r - s)))


def _overlap(a, b) -> bool:
    """Whether the tensors may share memory: not where their address ranges are apart, nor two views of one feature
    tensor that have no element in common, such as other ranks or other channels of the same nodes."""
    if a is None or b is None or not a.numel() or not b.numel():
        return False
    pa, pb, es = a.data_ptr(), b.data_ptr(), a.element_size()
    end = lambda t: t.data_ptr() + (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))) * t.element_size()
    if end(a) <= pb or end(b) <= pa:
        return False
    if es != b.element_size() or (pb - pa) % es:
        return True
    dims = {1: [1, 1]}  # stride: a's and b's sizes along it
    for i, t in enumerate((a, b)):
        for s, n in zip(t.stride(), t.shape):
            if s and n > 1:
                dims.setdefault(s, [1, 1])[i] += n - 1
    dims = sorted(((s, *n) for s, n in dims.items()), reverse=True)
    return _boxes_meet((pb - pa) // es, dims)


def _same_rows(a, b) -> bool:
    return b is not None and a.data_ptr() == b.data_ptr() and a.stride() == b.stride()


def _dense_outputs(outs, ins, in_place=()):
    """Raise ValueError when a caller's output overlaps an input or another output. in_place: (output, input)
    names that may be the very same tensor."""
    outs = [(n, t) for n, t in outs if t is not None]
    for i, (n, t) in enumerate(outs):
        for m, u in list(ins) + outs[:i]:
            if _overlap(t, u) and not ((n, m) in in_place and _same_rows(t, u)):
                raise ValueError(f"{n} must not overlap {m}")


def _dense_want(want, *names):
    """The gradients asked for (names, or one name), each of which must be one of `names`."""
    want = (want,) if isinstance(want, str) else tuple(want)
    for w in want:
        if w not in names:
            raise ValueError(f"want: expected some of {names}, got {w!r}")
    return want


def _check_linear(x, W, activation):
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation: expected 'none' or 'silu', got {activation!r}")
    if W.dim() != 2 or not 1 <= W.shape[0] <= LINEAR_MAX_CHANNELS or not 1 <= W.shape[1] <= LINEAR_MAX_CHANNELS:
        raise ValueError(f"W: expected [K, N] with 1 <= K, N <= {LINEAR_MAX_CHANNELS}, got {tuple(W.shape)}")
    return _ACTIVATIONS[activation]


def linear_workspace_size(M: int, K: int, N: int, dtype="float32", backward: bool = False, device=None) -> int:
    """Bytes of workspace linear_forward (linear_backward) needs for M rows (etp_linear_workspace_size on `device`)."""
    index = _dense_index(device)
    return _dense_bytes(index, "etp_linear_workspace_size", _dense_code(dtype),
                        int(M), 1, int(K), int(N), int(bool(backward)))


def linear_forward(x, W, bias=None, activation="none", residual=None, save_z=False, z=None, out=None,
                   workspace=None, stream=None):
    """out = act(x W + bias) + residual (launches etp_linear_forward). x [M, K] or [groups, rows, K], rows at any
    stride (a block x[:, l*l:(l+1)**2] of node features is read in place); W [K, N]; float32 or bfloat16, one type
    for all. activation: 'none' or 'silu'. save_z=True (or z given) also keeps z = x W + bias for linear_backward:
    returns (out, z). out may be residual itself. workspace: uint8 device tensor of linear_workspace_size bytes
    (allocated when None)."""
    if stream is not None:
        return _on_stream(stream, x, linear_forward, x, W, bias, activation, residual, save_z, z, out, workspace)
    code = _dense_type(x)
    act = _check_linear(x, W, activation)
    K, N = W.shape
    dtype, (lead, _) = x.dtype, _dense_lead(x, K)
    xr = _dense_rows(x, "x", dtype, lead, K)
    Wp, bp = _dense_vector(W, "W", dtype, K, N), _dense_vector(bias, "bias", dtype, N)
    rr = _dense_rows(residual, "residual", dtype, lead, N)
    if out is not None or z is not None:
        _dense_outputs([("out", out), ("z", z)], [("x", x), ("W", W), ("bias", bias), ("residual", residual)],
                       {("out", "residual")})
    out, orow = (out, _dense_rows(out, "out", dtype, lead, N)) if out is not None else _dense_new(x, lead, N)
    z, zr = (z, _dense_rows(z, "z", dtype, lead, N)) if z is not None or not save_z else _dense_new(x, lead, N)
    index = _dense_device(x, W, bias, residual, z, out, workspace)
    groups, per = lead if len(lead) == 2 else (lead[0], 1)
    workspace, nbytes = _dense_workspace(index, workspace, "etp_linear_workspace_size", code, groups, per, K, N, 0)
    _dense_call(index, "etp_linear_forward", _load().etp_linear_forward, code, groups, per, K, N, xr, Wp, bp, act, rr,
                zr, orow, _ptr(workspace), nbytes)
    return out if z is None else (out, z)


def linear_backward(x, W, grad_out, z=None, activation="none", want=("x", "W", "bias"), grad_x=None, grad_W=None,
                    grad_bias=None, workspace=None, stream=None):
    """(grad_x, grad_W, grad_bias) of linear_forward for the cotangent grad_out (launches etp_linear_backward);
    unwanted ones are None. z: what linear_forward kept (needed for 'silu'). The residual's gradient is grad_out."""
    if stream is not None:
        return _on_stream(stream, x, linear_backward, x, W, grad_out, z, activation, want, grad_x, grad_W, grad_bias,
                          workspace)
    code = _dense_type(x)
    act = _check_linear(x, W, activation)
    want = _dense_want(want, "x", "W", "bias")
    K, N = W.shape
    dtype, (lead, _) = x.dtype, _dense_lead(x, K)
    if act == ACT_NONE:
        z = None
    elif z is None:
        raise ValueError("z: the forward's pre-activation is needed for this activation")
    xr, Wp = _dense_rows(x, "x", dtype, lead, K), _dense_vector(W, "W", dtype, K, N)
    gr, zr = _dense_rows(grad_out, "grad_out", dtype, lead, N), _dense_rows(z, "z", dtype, lead, N)
    if grad_x is not None or grad_W is not None or grad_bias is not None:
        _dense_outputs([("grad_x", grad_x), ("grad_W", grad_W), ("grad_bias", grad_bias)],
                       [("x", x), ("W", W), ("grad_out", grad_out), ("z", z)])
    gxr = _dense_rows(grad_x, "grad_x", dtype, lead, K)
    if "x" in want and grad_x is None:
        grad_x, gxr = _dense_new(x, lead, K)
    if "W" in want and grad_W is None:
        grad_W = x.new_empty((K, N))
    if "bias" in want and grad_bias is None:
        grad_bias = x.new_empty(N)
    gWp, gbp = _dense_vector(grad_W, "grad_W", dtype, K, N), _dense_vector(grad_bias, "grad_bias", dtype, N)
    index = _dense_device(x, W, grad_out, z, grad_x, grad_W, grad_bias, workspace)
    groups, per = lead if len(lead) == 2 else (lead[0], 1)
    workspace, nbytes = _dense_workspace(index, workspace, "etp_linear_workspace_size", code, groups, per, K, N, 1)
    _dense_call(index, "etp_linear_backward", _load().etp_linear_backward, code, groups, per, K, N, xr, Wp, act, zr, gr,
                gxr, gWp, gbp, _ptr(workspace), nbytes)
    return grad_x, grad_W, grad_bias


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5, out=None, mean=None, rstd=None, stream=None):
    """(out, mean, rstd): each row of x normalised over its channels, times weight, plus bias (launches
    etp_layer_norm_forward). x [M, C] or [groups, rows, C], rows at any stride; mean, rstd float32 [M] or
    [groups, rows]. out may be x itself."""
    import torch

    if stream is not None:
        return _on_stream(stream, x, layer_norm_forward, x, weight, bias, eps, out, mean, rstd)
    code = _dense_type(x)
    dtype, (lead, C) = x.dtype, _dense_lead(x)
    xr = _dense_rows(x, "x", dtype, lead, C)
    wp, bp = _dense_vector(weight, "weight", dtype, C), _dense_vector(bias, "bias", dtype, C)
    if out is not None or mean is not None or rstd is not None:
        _dense_outputs([("out", out), ("mean", mean), ("rstd", rstd)], [("x", x), ("weight", weight), ("bias", bias)],
                       {("out", "x")})
    out, orow = (out, _dense_rows(out, "out", dtype, lead, C)) if out is not None else _dense_new(x, lead, C)
    if mean is None:
        mean = x.new_empty(lead, dtype=torch.float32)
    if rstd is None:
        rstd = torch.empty_like(mean) if mean.is_contiguous() else x.new_empty(lead, dtype=torch.float32)
    mp, rp = _dense_vector(mean, "mean", torch.float32, *lead), _dense_vector(rstd, "rstd", torch.float32, *lead)
    index = _dense_device(x, weight, bias, out, mean, rstd)
    groups, per = lead if len(lead) == 2 else (lead[0], 1)
    _dense_call(index, "etp_layer_norm_forward", _load().etp_layer_norm_forward, code, groups, per, C, float(eps), xr,
                wp, bp, orow, mp, rp)
    return out, mean, rstd


def layer_norm_workspace_size(M: int, C: int, dtype="float32", device=None) -> int:
    """Bytes of workspace layer_norm_backward needs for M rows (etp_layer_norm_workspace_size on `device`)."""
    index = _dense_index(device)
    return _dense_bytes(index, "etp_layer_norm_workspace_size",
                        _dense_code(dtype), int(M), 1, int(C))


def layer_norm_backward(x, weight, mean, rstd, grad_out, want=("x", "weight", "bias"), grad_x=None, grad_weight=None,
                        grad_bias=None, workspace=None, stream=None):
    """(grad_x, grad_weight, grad_bias) of layer_norm_forward for the cotangent grad_out (launches
    etp_layer_norm_backward); unwanted ones are None. weight: as in the forward (None: ones); mean, rstd: what it
    returned. grad_x may be grad_out or x itself."""
    import torch

    if stream is not None:
        return _on_stream(stream, x, layer_norm_backward, x, weight, mean, rstd, grad_out, want, grad_x, grad_weight,
                          grad_bias, workspace)
    code = _dense_type(x)
    want = _dense_want(want, "x", "weight", "bias")
    dtype, (lead, C) = x.dtype, _dense_lead(x)
    xr, gr = _dense_rows(x, "x", dtype, lead, C), _dense_rows(grad_out, "grad_out", dtype, lead, C)
    wp = _dense_vector(weight, "weight", dtype, C)
    mp, rp = _dense_vector(mean, "mean", torch.float32, *lead), _dense_vector(rstd, "rstd", torch.float32, *lead)
    if grad_x is not None or grad_weight is not None or grad_bias is not None:
        _dense_outputs([("grad_x", grad_x), ("grad_weight", grad_weight), ("grad_bias", grad_bias)],
                       [("x", x), ("weight", weight), ("mean", mean), ("rstd", rstd), ("grad_out", grad_out)],
                       {("grad_x", "x"), ("grad_x", "grad_out")})
    gxr = _dense_rows(grad_x, "grad_x", dtype, lead, C)
    if "x" in want and grad_x is None:
        grad_x, gxr = _dense_new(x, lead, C)
    if "weight" in want and grad_weight is None:
        grad_weight = x.new_empty(C) if weight is None else torch.empty_like(weight)
    if "bias" in want and grad_bias is None:
        grad_bias = x.new_empty(C) if grad_weight is None else torch.empty_like(grad_weight)
    gwp, gbp = _dense_vector(grad_weight, "grad_weight", dtype, C), _dense_vector(grad_bias, "grad_bias", dtype, C)
    index = _dense_device(x, weight, mean, rstd, grad_out, grad_x, grad_weight, grad_bias, workspace)
    groups, per = lead if len(lead) == 2 else (lead[0], 1)
    nbytes = 0
    if grad_weight is not None or grad_bias is not None:
        workspace, nbytes = _dense_workspace(index, workspace, "etp_layer_norm_workspace_size", code, groups, per, C)
    _dense_call(index, "etp_layer_norm_backward", _load().etp_layer_norm_backward, code, groups, per, C, xr, wp,
                mp, rp, gr, gxr, gwp, gbp, _ptr(workspace) if nbytes else None, nbytes)
    return grad_x, grad_weight, grad_bias


def assemble_forces(N: int, row_ptr, rev_ptr, rev_perm, grad_r, r=None, forces=None, virial=None, stream=None):
    """(forces [N, 3], virial [N, 3, 3] or None) from grad_r = dE/dr (etp_assemble_forces).
    The per-atom virial is computed when r is given."""
    import torch

    if stream is not None:
        return _on_stream(stream, grad_r, assemble_forces, N, row_ptr, rev_ptr, rev_perm, grad_r, r, forces, virial)
    _expect(grad_r, "grad_r", "float32", (None, 3))
    E = grad_r.shape[0]
    _expect(row_ptr, "row_ptr", "int32", (N + 1,))
    _expect(rev_ptr, "rev_ptr", "int32", (N + 1,))
    _expect(rev_perm, "rev_perm", "int32", (E,))
    _expect(r, "r", "float32", (E, 3))
    dev = grad_r.device
    if forces is None:
        forces = torch.empty((N, 3), device=dev, dtype=torch.float32)
    if r is not None and virial is None:
        virial = torch.empty((N, 3, 3), device=dev, dtype=torch.float32)
    _expect(forces, "forces", "float32", (N, 3))
    if virial is not None and (str(virial.dtype) != "torch.float32" or virial.numel() != 9 * N):
        raise ValueError("virial: expected float32 with N*9 elements")
    dev = _need_cuda(row_ptr, rev_ptr, rev_perm, grad_r, r, forces, virial)
    _launch(dev, "etp_assemble_forces", _load().etp_assemble_forces, int(N), int(E), _ptr(row_ptr), _ptr(rev_ptr),
            _ptr(rev_perm), _ptr(r), _ptr(grad_r), _ptr(forces), _ptr(virial))
    return forces, virial


def radial_workspace_size(plan: Plan, E: int, n_basis: int, hidden: int) -> int:
    b = ctypes.c_size_t()
    _check(_load().etp_radial_workspace_size(plan.handle, int(E), int(n_basis), int(hidden), ctypes.byref(b)),
           "etp_radial_workspace_size")
    return b.value


def _radial_ws(plan, E, W1, workspace):
    import torch

    nbytes = radial_workspace_size(plan, E, W1.shape[0], W1.shape[1])
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=W1.device)
    _expect(workspace, "workspace", "uint8", (None,))
    return workspace


def radial_forward(plan: Plan, r, W1, W2, r_cut: float, w=None, workspace=None, stream=None):
    """w [E, P, C] = SiLU(bessel(|r|) W1) W2 (etp_radial_forward)."""
    import torch

    if stream is not None:
        return _on_stream(stream, r, radial_forward, plan, r, W1, W2, r_cut, w, workspace)
    _expect(r, "r", "float32", (None, 3))
    E = r.shape[0]
    _expect(W1, "W1", "float32", (None, None))
    _expect(W2, "W2", "float32", (W1.shape[1], plan.n_paths * plan.C))
    if w is None:
        w = torch.empty((E, plan.n_paths, plan.C), device=r.device, dtype=torch.float32)
    _expect(w, "w", "float32", (E, plan.n_paths, plan.C))
    workspace = _radial_ws(plan, E, W1, workspace)
    dev = _need_cuda(r, W1, W2, w, workspace)
    _launch(dev, "etp_radial_forward", _load().etp_radial_forward, plan.handle, E, W1.shape[0], W1.shape[1],
            float(r_cut), _ptr(r), _ptr(W1), _ptr(W2), _ptr(w), _ptr(workspace), workspace.numel())
    return w


def radial_backward(plan: Plan, r, W1, W2, r_cut: float, grad_w, grad_r, grad_W1=None, grad_W2=None,
                    workspace=None, stream=None):
    """(grad_W1, grad_W2); adds the derivative through |r| to grad_r in place (etp_radial_backward)."""
    import torch

    if stream is not None:
        return _on_stream(stream, r, radial_backward, plan, r, W1, W2, r_cut, grad_w, grad_r, grad_W1, grad_W2,
                          workspace)
    _expect(r, "r", "float32", (None, 3))
    E = r.shape[0]
    _expect(W1, "W1", "float32", (None, None))
    _expect(W2, "W2", "float32", (W1.shape[1], plan.n_paths * plan.C))
    _expect(grad_w, "grad_w", "float32", (E, plan.n_paths, plan.C))
    _expect(grad_r, "grad_r", "float32", (E, 3))
    if grad_W1 is None:
        grad_W1 = torch.empty_like(W1)
    if grad_W2 is None:
        grad_W2 = torch.empty_like(W2)
    _expect(grad_W1, "grad_W1", "float32", tuple(W1.shape))
    _expect(grad_W2, "grad_W2", "float32", tuple(W2.shape))
    workspace = _radial_ws(plan, E, W1, workspace)
    dev = _need_cuda(r, W1, W2, grad_w, grad_r, grad_W1, grad_W2, workspace)
    _launch(dev, "etp_radial_backward", _load().etp_radial_backward, plan.handle, E, W1.shape[0], W1.shape[1],
            float(r_cut), _ptr(r), _ptr(W1), _ptr(W2), _ptr(grad_w), _ptr(grad_W1), _ptr(grad_W2), _ptr(grad_r),
            _ptr(workspace), workspace.numel())
    return grad_W1, grad_W2


def fused_workspace_size(plan: Plan, E: int, n_basis: int = 8, hidden: int = 64) -> int:
    b = ctypes.c_size_t()
    _check(_load().etp_fused_workspace_size(plan.handle, int(E), int(n_basis), int(hidden), ctypes.byref(b)),
           "etp_fused_workspace_size")
    return b.value


def fused_forward(plan: Plan, row_ptr, src, r, x, W1, W2, r_cut: float, out=None, workspace=None, stream=None):
    """out [N, D, C] = forward(plan, ..., w = radial_forward(plan, r, W1, W2, r_cut)) without storing w
    (launches etp_fused_forward)."""
    import torch

    if stream is not None:
        return _on_stream(stream, row_ptr, fused_forward, plan, row_ptr, src, r, x, W1, W2, r_cut, out, workspace)
    N, E = row_ptr.numel() - 1, src.numel()
    _check_graph(row_ptr, src, N, E)
    _expect(r, "r", "float32", (E, 3))
    _expect(x, "x", "float32", (N, plan.dim_in, plan.C))
    _expect(W1, "W1", "float32", (None, None))
    _expect(W2, "W2", "float32", (W1.shape[1], plan.n_paths * plan.C))
    if out is None:
        out = torch.empty((N, plan.dim_out, plan.C), device=x.device, dtype=torch.float32)
    _expect(out, "out", "float32", (N, plan.dim_out, plan.C))
    nbytes = fused_workspace_size(plan, E, W1.shape[0], W1.shape[1])
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    _expect(workspace, "workspace", "uint8", (None,))
    dev = _need_cuda(row_ptr, src, r, x, W1, W2, out, workspace)
    _launch(dev, "etp_fused_forward", _load().etp_fused_forward, plan.handle, N, E, _ptr(row_ptr), _ptr(src),
            _ptr(r), _ptr(x), W1.shape[0], W1.shape[1], float(r_cut), _ptr(W1), _ptr(W2), _ptr(out),
            _ptr(workspace), workspace.numel())
    return out


def reverse_csr_workspace_size(N: int, E: int) -> int:
    b = ctypes.c_size_t()
    _check(_load().etp_reverse_csr_workspace_size(int(N), int(E), ctypes.byref(b)), "workspace_size")
    return b.value


def build_reverse_csr(N: int, row_ptr, src, with_dst=True, workspace=None, stream=None):
    """(rev_ptr [N+1], rev_perm [E], dst [E] or None), all int32 on the device (etp_build_reverse_csr)."""
    import torch

    if stream is not None:
        return _on_stream(stream, row_ptr, build_reverse_csr, N, row_ptr, src, with_dst, workspace)
    E = src.numel()
    _check_graph(row_ptr, src, N, E)
    dev = row_ptr.device
    rev_ptr = torch.empty(N + 1, dtype=torch.int32, device=dev)
    rev_perm = torch.empty(E, dtype=torch.int32, device=dev)
    dst = torch.empty(E, dtype=torch.int32, device=dev) if with_dst else None
    nbytes = reverse_csr_workspace_size(N, E)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    _expect(workspace, "workspace", "uint8", (None,))
    dev = _need_cuda(row_ptr, src, rev_ptr, rev_perm, dst, workspace)
    _launch(dev, "etp_build_reverse_csr", _load().etp_build_reverse_csr, N, E, _ptr(row_ptr), _ptr(src),
            _ptr(rev_ptr), _ptr(rev_perm), _ptr(dst), _ptr(workspace), workspace.numel())
    return rev_ptr, rev_perm, dst


def build_reverse_csr_static(N: int, row_ptr, src, with_dst=True, stream=None):
    """As build_reverse_csr, with the library's fixed device scratch instead of a workspace
    (etp_build_reverse_csr_static; N, E <= 2^18; calls that overlap on the GPU race)."""
    import torch

    if stream is not None:
        return _on_stream(stream, row_ptr, build_reverse_csr_static, N, row_ptr, src, with_dst)
    E = src.numel()
    _check_graph(row_ptr, src, N, E)
    dev = row_ptr.device
    rev_ptr = torch.empty(N + 1, dtype=torch.int32, device=dev)
    rev_perm = torch.empty(E, dtype=torch.int32, device=dev)
    dst = torch.empty(E, dtype=torch.int32, device=dev) if with_dst else None
    dev = _need_cuda(row_ptr, src, rev_ptr, rev_perm, dst)
    _launch(dev, "etp_build_reverse_csr_static", _load().etp_build_reverse_csr_static, N, E, _ptr(row_ptr),
            _ptr(src), _ptr(rev_ptr), _ptr(rev_perm), _ptr(dst))
    return rev_ptr, rev_perm, dst


class Schedule:
    """Locality schedule of a CSR graph (etp_build_locality_schedule): node order, the
    forward CSR over that order (ord_ptr, ord_edge), the reverse CSR over that order
    (rev_ptr, rev_perm) and the destination of every edge, all int32 on the device."""

    def __init__(self, N, E, order, ord_ptr, ord_edge, rev_ptr, rev_perm, dst):
        self.N, self.E = N, E
        self.order, self.ord_ptr, self.ord_edge = order, ord_ptr, ord_edge
        self.rev_ptr, self.rev_perm, self.dst = rev_ptr, rev_perm, dst

    def tensors(self):
        return self.order, self.ord_ptr, self.ord_edge, self.rev_ptr, self.rev_perm, self.dst


def locality_schedule_workspace_size(N: int, E: int) -> int:
    b = ctypes.c_size_t()
    _check(_load().etp_locality_schedule_workspace_size(int(N), int(E), ctypes.byref(b)), "workspace_size")
    return b.value


def locality_schedule(N: int, row_ptr, src, pos, cell: float, out: Schedule = None, workspace=None, stream=None):
    """Schedule whose rows follow the Morton order of the nodes' cells (side `cell`) of pos [N, 3]
    (etp_build_locality_schedule). out: a Schedule of the same sizes to overwrite."""
    import torch

    if stream is not None:
        return _on_stream(stream, row_ptr, locality_schedule, N, row_ptr, src, pos, cell, out, workspace)
    E = src.numel()
    _check_graph(row_ptr, src, N, E)
    _expect(pos, "pos", "float32", (N, 3))
    dev = row_ptr.device
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = Schedule(N, E, torch.empty(N, **i32), torch.empty(N + 1, **i32), torch.empty(E, **i32),
                       torch.empty(N + 1, **i32), torch.empty(E, **i32), torch.empty(E, **i32))
    if (out.N, out.E) != (N, E):
        raise ValueError(f"schedule for (N, E) = {(out.N, out.E)}, graph has {(N, E)}")
    nbytes = locality_schedule_workspace_size(N, E)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    _expect(workspace, "workspace", "uint8", (None,))
    dev = _need_cuda(row_ptr, src, pos, workspace, *out.tensors())
    _launch(dev, "etp_build_locality_schedule", _load().etp_build_locality_schedule, N, E, _ptr(row_ptr), _ptr(src),
            _ptr(pos), float(cell), *[_ptr(t) for t in out.tensors()], _ptr(workspace), workspace.numel())
    return out


def forward_ordered(plan: Plan, sched: Schedule, src, r, x, w, out=None, frames=None, workspace=None, stream=None):
    """forward() on a locality schedule (etp_forward_ordered): the same out, rows visited in schedule order."""
    import torch

    if stream is not None:
        return _on_stream(stream, x, forward_ordered, plan, sched, src, r, x, w, out, frames, workspace)
    N, E = sched.N, sched.E
    _expect(src, "src", "int32", (E,))
    _expect(r, "r", "float32", (E, 3))
    _expect(frames, "frames", "float32", (E, FRAME_FLOATS))
    _expect(x, "x", "float32", (N, plan.dim_in, plan.C))
    _expect(w, "w", "float32", (E, plan.n_paths, plan.C))
    if out is None:
        out = torch.empty((N, plan.dim_out, plan.C), device=x.device, dtype=torch.float32)
    _expect(out, "out", "float32", (N, plan.dim_out, plan.C))
    dev = _need_cuda(sched.order, sched.ord_ptr, sched.ord_edge, src, r, frames, x, w, out)
    workspace = _tp_workspace(plan, N, E, True, workspace, dev)
    _need_cuda(out, workspace)
    _launch(dev, "etp_forward_ordered", _load().etp_forward_ordered, plan.handle, N, E, _ptr(sched.order),
            _ptr(sched.ord_ptr), _ptr(sched.ord_edge), _ptr(src), _ptr(r), _ptr(frames), _ptr(x), _ptr(w),
            _ptr(out), _ptr(workspace), workspace.numel())
    return out


def backward_ordered(plan: Plan, sched: Schedule, r, x, w, grad_out, want=("x", "w", "r"), grad_x=None,
                     grad_w=None, grad_r=None, frames=None, workspace=None, stream=None):
    """backward() on a locality schedule (etp_backward_ordered): the same (grad_x, grad_w, grad_r)."""
    import torch

    if stream is not None:
        return _on_stream(stream, x, backward_ordered, plan, sched, r, x, w, grad_out, want, grad_x, grad_w, grad_r,
                          frames, workspace)
    N, E = sched.N, sched.E
    _expect(r, "r", "float32", (E, 3))
    _expect(frames, "frames", "float32", (E, FRAME_FLOATS))
    _expect(x, "x", "float32", (N, plan.dim_in, plan.C))
    _expect(w, "w", "float32", (E, plan.n_paths, plan.C))
    _expect(grad_out, "grad_out", "float32", (N, plan.dim_out, plan.C))
    dev = x.device
    if "x" in want and grad_x is None:
        grad_x = torch.empty((N, plan.dim_in, plan.C), device=dev, dtype=torch.float32)
    if "w" in want and grad_w is None:
        grad_w = torch.empty((E, plan.n_paths, plan.C), device=dev, dtype=torch.float32)
    if "r" in want and grad_r is None:
        grad_r = torch.empty((E, 3), device=dev, dtype=torch.float32)
    _expect(grad_x, "grad_x", "float32", (N, plan.dim_in, plan.C))
    _expect(grad_w, "grad_w", "float32", (E, plan.n_paths, plan.C))
    _expect(grad_r, "grad_r", "float32", (E, 3))
    dev = _need_cuda(sched.order, sched.rev_ptr, sched.rev_perm, sched.dst, r, frames, x, w, grad_out, grad_x,
                     grad_w, grad_r)
    workspace = _tp_workspace(plan, N, E, True, workspace, dev)
    _need_cuda(x, workspace)
    _launch(dev, "etp_backward_ordered", _load().etp_backward_ordered, plan.handle, N, E, _ptr(sched.order),
            _ptr(sched.rev_ptr), _ptr(sched.rev_perm), _ptr(sched.dst), _ptr(r), _ptr(frames), _ptr(x), _ptr(w),
            _ptr(grad_out), _ptr(grad_x), _ptr(grad_w), _ptr(grad_r), _ptr(workspace), workspace.numel())
    return grad_x, grad_w, grad_r


def device_fault() -> int:
    """1 if a bounded wait inside a kernel ran out since the last call (never expected); clears it."""
    f = ctypes.c_int()
    _check(_load().etp_device_fault(ctypes.byref(f)), "etp_device_fault")
    return f.value


def validate_csr(N: int, row_ptr, src, stream=None) -> int:
    """The ETP_CSR_* bits of every problem found in the CSR (0 = valid). Synchronises the stream."""
    import torch

    if stream is not None:
        return _on_stream(stream, row_ptr, validate_csr, N, row_ptr, src)
    _check_graph(row_ptr, src, N, src.numel())
    flag = torch.empty(1, dtype=torch.int32, device=row_ptr.device)
    dev = _need_cuda(row_ptr, src, flag)
    _launch(dev, "etp_validate_csr", _load().etp_validate_csr, N, src.numel(), _ptr(row_ptr), _ptr(src),
            _ptr(flag))
    return int(flag.item())
