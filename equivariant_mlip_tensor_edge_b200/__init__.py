"""B200-native equivariant edge tensor-product convolution: Python binding of libetp.so.

Argument marshalling only. Every step of the path (neighbour list, CSR, spherical harmonics,
radial basis and projection, Clebsch-Gordan contraction, segmented sums, backward, forces)
runs in the CUDA kernels of ``libetp.so``; PyTorch provides device memory and streams. There
is no CPU fallback: without the built library, or without a CUDA device, calls raise.

The C ABI is documented in ``include/etp.h``.
"""
import ctypes
import functools
import os
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libetp.so")

ETP_OK = 0
STATUS_NAMES = {0: "ETP_OK", 1: "ETP_ERR_INVALID_ARG", 2: "ETP_ERR_IRREPS", 3: "ETP_ERR_UNSUPPORTED",
                4: "ETP_ERR_BAD_GRAPH", 5: "ETP_ERR_CUDA", 6: "ETP_ERR_CAPACITY"}

# exported symbols and their C signatures (restype, argtypes)
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll = ctypes.c_longlong
_ip = ctypes.POINTER(ctypes.c_int)
_dp = ctypes.POINTER(ctypes.c_double)


class EtpInfo(ctypes.Structure):
    _fields_ = [("lmax", ctypes.c_int), ("channels", ctypes.c_int), ("dim_in", ctypes.c_int),
                ("dim_out", ctypes.c_int), ("n_paths", ctypes.c_int), ("n_basis", ctypes.c_int),
                ("weight_numel", ctypes.c_int), ("cg_nnz", ctypes.c_int), ("sum_2l3p1", ctypes.c_int),
                ("r_cut", ctypes.c_float), ("general", ctypes.c_int), ("flop_fwd", ctypes.c_int),
                ("flop_bwd", ctypes.c_int)]


SIGNATURES = {
    "etp_create": (_i, [ctypes.c_char_p, _i, ctypes.c_char_p, _i, _f, ctypes.POINTER(_vp)]),
    "etp_destroy": (_i, [_vp]),
    "etp_get_info": (_i, [_vp, ctypes.POINTER(EtpInfo)]),
    "etp_get_paths": (_i, [_vp, _ip, _i]),
    "etp_status_string": (ctypes.c_char_p, [_i]),
    "etp_last_error": (ctypes.c_char_p, []),
    "etp_workspace_bytes": (_sz, [_vp, _i, _i]),
    "etp_forward": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "etp_forward_noalloc": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "etp_backward": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "etp_backward_weights": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "etp_forward_masked": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "etp_backward_masked": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                 _vp]),
    "etp_radial_weights": (_i, [_vp, _i, _vp, _vp, _vp, _vp]),
    "etp_node_ladder": (_i, [_i, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "etp_node_ladder_full_step_floats": (_sz, [_i, _i]),
    "etp_node_ladder_full_workspace_bytes": (_sz, [_i, _i, _i]),
    "etp_node_ladder_full": (_i, [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "etp_checkpoint_store": (_i, [_i, _i, _ll, _i, _vp, _vp, _vp, _vp]),
    "etp_checkpoint_restore": (_i, [_i, _i, _ll, _i, _vp, _vp, _vp, _vp]),
    "etp_group_norm_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "etp_group_norm": (_i, [_i, _i, _i, _i, _i, _vp, _i, _vp, _vp, _vp, _f, _i, _i, _vp, _vp, _i, _vp, _vp, _vp, _sz, _vp]),
    "etp_group_norm_backward": (_i, [_i, _i, _i, _i, _i, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _vp,
                                     _vp, _vp, _sz, _vp]),
    "etp_group_norm_status": (_i, [_vp, _ip]),
    "etp_group_norm_status_word": (_ip, []),
    "etp_forces": (_i, [_i, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "etp_graph_workspace_bytes": (_sz, [_i, _i]),
    "etp_neighbors": (_i, [_vp, _i, _dp, _ip, _f, _i, _ip, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "etp_build_csr": (_i, [_i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "etp_get_status": (_i, [_vp, _vp, _ip]),
    "etp_status_word": (_ip, [_vp]),
}

_lib = None


def load_library(path=LIB_PATH):
    """Load libetp.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m equivariant_mlip_tensor_edge_b200.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


class EtpError(RuntimeError):
    def __init__(self, status, where):
        lib = load_library()
        msg = lib.etp_last_error().decode()
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def _check(status, where):
    if status != ETP_OK:
        raise EtpError(status, where)


@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need_cuda(*tensors):
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError("libetp operates on CUDA tensors only (no CPU fallback)")


def _i32(t):
    torch = _torch()
    return t if t.dtype == torch.int32 and t.is_contiguous() else t.to(torch.int32).contiguous()


def _f32(t):
    torch = _torch()
    return t if t.dtype == torch.float32 and t.is_contiguous() else t.to(torch.float32).contiguous()


@dataclass
class Graph:
    """Receiver-sorted CSR edge layout plus the transposed (sender-sorted) order (device tensors)."""
    n_nodes: int
    n_edges: int
    row_ptr: object
    sender: object
    edge_vec: object
    t_row_ptr: object
    t_perm: object
    shift: object = None
    perm: object = None


def graph_workspace_bytes(n_nodes, max_edges):
    return load_library().etp_graph_workspace_bytes(n_nodes, max_edges)


def neighbors(pos, r_cut, cell=None, pbc=(False, False, False), max_edges=None, with_shift=True):
    """Neighbour list + canonical CSR on the GPU. pos: [N,3] float32 CUDA tensor; cell: 3x3 (host)."""
    torch = _torch()
    lib = load_library()
    _need_cuda(pos)
    pos = _f32(pos)
    n = pos.shape[0]
    dev = pos.device
    if max_edges is None:
        max_edges = max(1024, n * 128)
    cell_arr = None
    if cell is not None:
        vals = [float(v) for row in cell for v in row]
        cell_arr = (ctypes.c_double * 9)(*vals)
    pbc_arr = (ctypes.c_int * 3)(*[int(bool(p)) for p in pbc])
    while True:
        row_ptr = torch.empty(n + 1, dtype=torch.int32, device=dev)
        t_row_ptr = torch.empty(n + 1, dtype=torch.int32, device=dev)
        sender = torch.empty(max(max_edges, 1), dtype=torch.int32, device=dev)
        edge_vec = torch.empty((max(max_edges, 1), 3), dtype=torch.float32, device=dev)
        shift = torch.empty((max(max_edges, 1), 3), dtype=torch.int32, device=dev) if with_shift else None
        t_perm = torch.empty(max(max_edges, 1), dtype=torch.int32, device=dev)
        ws_bytes = lib.etp_graph_workspace_bytes(n, max_edges)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        n_edges = ctypes.c_int(0)
        st = lib.etp_neighbors(_ptr(pos), n, ctypes.cast(cell_arr, _dp) if cell_arr is not None else None, pbc_arr,
                               float(r_cut), max_edges, ctypes.byref(n_edges), _ptr(row_ptr), _ptr(sender),
                               _ptr(edge_vec), _ptr(shift), _ptr(t_row_ptr), _ptr(t_perm), _ptr(ws), ws_bytes,
                               _stream(dev))
        if st == 6:  # capacity: retry with the reported count
            max_edges = n_edges.value
            continue
        _check(st, "etp_neighbors")
        e = n_edges.value
        return Graph(n, e, row_ptr, sender[:e], edge_vec[:e], t_row_ptr, t_perm[:e],
                     shift[:e] if shift is not None else None)


def build_csr(n_nodes, receiver, sender, edge_vec):
    """Canonical CSR of a given edge list (any order), on the GPU."""
    torch = _torch()
    lib = load_library()
    _need_cuda(receiver, sender, edge_vec)
    receiver, sender, edge_vec = _i32(receiver), _i32(sender), _f32(edge_vec)
    e = receiver.shape[0]
    dev = receiver.device
    row_ptr = torch.empty(n_nodes + 1, dtype=torch.int32, device=dev)
    t_row_ptr = torch.empty(n_nodes + 1, dtype=torch.int32, device=dev)
    s_out = torch.empty(max(e, 1), dtype=torch.int32, device=dev)
    v_out = torch.empty((max(e, 1), 3), dtype=torch.float32, device=dev)
    perm = torch.empty(max(e, 1), dtype=torch.int32, device=dev)
    t_perm = torch.empty(max(e, 1), dtype=torch.int32, device=dev)
    ws_bytes = lib.etp_graph_workspace_bytes(n_nodes, e)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _check(lib.etp_build_csr(n_nodes, e, _ptr(receiver), _ptr(sender), _ptr(edge_vec), _ptr(row_ptr),
                             _ptr(s_out), _ptr(v_out), _ptr(perm), _ptr(t_row_ptr), _ptr(t_perm), _ptr(ws),
                             ws_bytes, _stream(dev)), "etp_build_csr")
    return Graph(n_nodes, e, row_ptr, s_out[:e], v_out[:e], t_row_ptr, t_perm[:e], None, perm[:e])


def forces(graph, grad_edge_vec, out=None):
    torch = _torch()
    lib = load_library()
    _need_cuda(grad_edge_vec)
    if out is None:
        out = torch.empty((graph.n_nodes, 3), dtype=torch.float32, device=grad_edge_vec.device)
    _check(lib.etp_forces(graph.n_nodes, graph.n_edges, _ptr(graph.row_ptr), _ptr(graph.t_row_ptr),
                          _ptr(graph.t_perm), _ptr(_f32(grad_edge_vec)), _ptr(out), _stream(out.device)),
           "etp_forces")
    return out


class EdgeConv:
    """Handle for one convolution configuration (irreps, SH lmax, radial basis, cutoff).

    Uniform irreps (C x (0e + 1o + ... + Le), SH lmax L <= 3) run on the tensor-core kernels;
    anything else the library supports (per-block multiplicities, both parities, rank <= 4) on the
    general kernels (``info["general"] == 1``), whose W is [n_basis, cols] in ``paths`` order.
    """

    def __init__(self, irreps_in, sh_lmax, irreps_out, n_basis=8, r_cut=5.0):
        lib = load_library()
        h = ctypes.c_void_p()
        _check(lib.etp_create(irreps_in.encode(), int(sh_lmax), irreps_out.encode(), int(n_basis),
                              float(r_cut), ctypes.byref(h)), "etp_create")
        self._h = h
        info = EtpInfo()
        _check(lib.etp_get_info(h, ctypes.byref(info)), "etp_get_info")
        self.info = {k: getattr(info, k) for k, _ in EtpInfo._fields_}
        self.r_cut = float(r_cut)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.etp_destroy(h)
            self._h = None

    @property
    def n_paths(self):
        return self.info["n_paths"]

    @property
    def paths(self):
        """[(input block, l2, output block)] in W's column order."""
        n = self.n_paths
        buf = (ctypes.c_int * (3 * n))()
        _check(load_library().etp_get_paths(self._h, buf, n), "etp_get_paths")
        return [tuple(buf[3 * p:3 * p + 3]) for p in range(n)]

    def workspace_bytes(self, n_nodes, n_edges):
        return load_library().etp_workspace_bytes(self._h, n_nodes, n_edges)

    def check_status(self, device=None):
        """Synchronise the current stream and raise if a kernel of an earlier call on this handle
        gave up a bounded pipeline wait (the code is cleared)."""
        code = ctypes.c_int(0)
        stream = _stream(device) if device is not None else None
        _check(load_library().etp_get_status(self._h, stream, ctypes.byref(code)), "etp_get_status")

    def _features(self, x):
        """Node features as float32: a tensor's, or those that a Checkpoint8 holds."""
        return x.restore(dtype=_torch().float32) if isinstance(x, Checkpoint8) else _f32(x)

    def _workspace(self, n_nodes, n_edges, device, workspace):
        torch = _torch()
        nb = self.workspace_bytes(n_nodes, n_edges)
        if workspace is None or workspace.numel() < nb:
            workspace = torch.empty(max(nb, 1), dtype=torch.uint8, device=device)
        return workspace, nb

    def forward(self, graph, x, W, out=None, workspace=None, path_mask=None):
        """path_mask: optional int32 CUDA tensor [n_edges] (canonical order), bit p = path p on."""
        torch = _torch()
        _need_cuda(x, W, graph.row_ptr)
        x, W = _f32(x), _f32(W)
        if out is None:
            out = torch.empty((graph.n_nodes, self.info["dim_out"]), dtype=torch.float32, device=x.device)
        ws, nb = self._workspace(graph.n_nodes, graph.n_edges, x.device, workspace)
        lib = load_library()
        if path_mask is None:
            _check(lib.etp_forward(self._h, graph.n_nodes, graph.n_edges, _ptr(graph.row_ptr),
                                   _ptr(graph.sender), _ptr(graph.edge_vec), _ptr(x), _ptr(W), _ptr(out),
                                   _ptr(ws), nb, _stream(x.device)), "etp_forward")
        else:
            _need_cuda(path_mask)
            m = _i32(path_mask)
            _check(lib.etp_forward_masked(self._h, graph.n_nodes, graph.n_edges, _ptr(graph.row_ptr),
                                          _ptr(graph.sender), _ptr(graph.edge_vec), _ptr(x), _ptr(W), _ptr(m),
                                          _ptr(out), _ptr(ws), nb, _stream(x.device)), "etp_forward_masked")
        return out

    def backward(self, graph, x, W, grad_out, want_grad_x=True, want_grad_vec=True, grad_x=None,
                 grad_vec=None, workspace=None, path_mask=None):
        """x: the forward's node features, or their Checkpoint8 (restored to float32 for the call)."""
        torch = _torch()
        _need_cuda(x.q if isinstance(x, Checkpoint8) else x, W, grad_out)
        x, W, grad_out = self._features(x), _f32(W), _f32(grad_out)
        dev = x.device
        if want_grad_x and grad_x is None:
            grad_x = torch.empty((graph.n_nodes, self.info["dim_in"]), dtype=torch.float32, device=dev)
        if want_grad_vec and grad_vec is None:
            grad_vec = torch.empty((max(graph.n_edges, 1), 3), dtype=torch.float32, device=dev)[:graph.n_edges]
        ws, nb = self._workspace(graph.n_nodes, graph.n_edges, dev, workspace)
        gx_p = _ptr(grad_x) if want_grad_x else None
        gv_p = _ptr(grad_vec) if want_grad_vec else None
        if path_mask is None:
            _check(load_library().etp_backward(
                self._h, graph.n_nodes, graph.n_edges, _ptr(graph.row_ptr), _ptr(graph.sender), _ptr(graph.edge_vec),
                _ptr(graph.t_row_ptr), _ptr(graph.t_perm), _ptr(x), _ptr(W), _ptr(grad_out), gx_p, gv_p, _ptr(ws), nb,
                _stream(dev)), "etp_backward")
        else:
            _need_cuda(path_mask)
            m = _i32(path_mask)
            _check(load_library().etp_backward_masked(
                self._h, graph.n_nodes, graph.n_edges, _ptr(graph.row_ptr), _ptr(graph.sender), _ptr(graph.edge_vec),
                _ptr(graph.t_row_ptr), _ptr(graph.t_perm), _ptr(x), _ptr(W), _ptr(m), _ptr(grad_out), gx_p, gv_p,
                _ptr(ws), nb, _stream(dev)), "etp_backward_masked")
        return (grad_x if want_grad_x else None), (grad_vec if want_grad_vec else None)

    def backward_weights(self, graph, x, grad_out, grad_W=None, workspace=None):
        """dL/dW for L = <grad_out, forward(graph, x, W)>: [n_basis, n_paths, C], or [n_basis, cols] for
        a general irreps handle. x: the forward's node features, or their Checkpoint8 (restored to
        float32 for the call)."""
        torch = _torch()
        _need_cuda(x.q if isinstance(x, Checkpoint8) else x, grad_out)
        x, grad_out = self._features(x), _f32(grad_out)
        if grad_W is None:
            shape = ((self.info["n_basis"], self.info["n_paths"], self.info["channels"]) if not self.info["general"]
                     else (self.info["n_basis"], self.info["weight_numel"] // self.info["n_basis"]))
            grad_W = torch.empty(shape, dtype=torch.float32, device=x.device)
        ws, nb = self._workspace(graph.n_nodes, graph.n_edges, x.device, workspace)
        _check(load_library().etp_backward_weights(
            self._h, graph.n_nodes, graph.n_edges, _ptr(graph.row_ptr), _ptr(graph.sender), _ptr(graph.edge_vec),
            _ptr(x), _ptr(grad_out), _ptr(grad_W), _ptr(ws), nb, _stream(x.device)), "etp_backward_weights")
        return grad_W

    def radial_weights(self, edge_vec, W):
        torch = _torch()
        _need_cuda(edge_vec, W)
        edge_vec, W = _f32(edge_vec), _f32(W)
        e = edge_vec.shape[0]
        out = torch.empty((max(e, 1), self.n_paths, self.info["channels"]), dtype=torch.float32,
                          device=edge_vec.device)[:e]
        _check(load_library().etp_radial_weights(self._h, e, _ptr(edge_vec), _ptr(W), _ptr(out),
                                                 _stream(edge_vec.device)), "etp_radial_weights")
        return out


def node_ladder(A, Ws, lmax, out=None):
    """Node-local product ladder: out = B_1 + ... + B_nu with B_1 = A and B_{q+1} = P(B_q, A; Ws[q-1]).

    A: [N, C (lmax+1)^2] float32 CUDA tensor (node-row layout); Ws: [nu - 1, n_paths, C] (nu - 1 may
    be 0). Returns out like A.
    """
    torch = _torch()
    _need_cuda(A, Ws)
    A, Ws = _f32(A), _f32(Ws)
    n, dim = A.shape
    c = dim // ((lmax + 1) ** 2)
    nu = Ws.shape[0] + 1
    if out is None:
        out = torch.empty_like(A)
    _check(load_library().etp_node_ladder(int(lmax), c, n, nu, _ptr(A), _ptr(Ws) if nu > 1 else None, _ptr(out),
                                          _stream(A.device)), "etp_node_ladder")
    return out


def node_ladder_full_step_floats(lmax, channels):
    """Floats of one step of full-ladder weights (the per-rank matrices [C][P_l3 C], l3 = 0..lmax)."""
    return int(load_library().etp_node_ladder_full_step_floats(int(lmax), int(channels)))


def node_ladder_full(A, Ws, lmax, out=None, workspace=None):
    """The full product ladder: out = B_1 + ... + B_nu, B_1 = A, and each step the per-path products
    of B_q and A compressed by that step's per-rank matrices (paths and channels mixed; the mixing
    runs on the tensor cores).

    A: [N, C (lmax+1)^2] float32 CUDA tensor (node-row layout, C in 32, 64, 96, 128);
    Ws: [nu - 1, node_ladder_full_step_floats(lmax, C)] (nu - 1 may be 0). Returns out like A.
    """
    torch = _torch()
    _need_cuda(A, Ws)
    A, Ws = _f32(A), _f32(Ws)
    n, dim = A.shape
    c = dim // ((lmax + 1) ** 2)
    nu = Ws.shape[0] + 1
    lib = load_library()
    if out is None:
        out = torch.empty_like(A)
    need = int(lib.etp_node_ladder_full_workspace_bytes(int(lmax), c, n))
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=A.device)
    _check(lib.etp_node_ladder_full(int(lmax), c, n, nu, _ptr(A), _ptr(Ws) if nu > 1 else None, _ptr(out),
                                    _ptr(workspace), workspace.numel(), _stream(A.device)), "etp_node_ladder_full")
    return out


# ---- between two convolutions: 8-bit checkpoints, group norm with an activation

CKPT_FORMATS = {None: 0, "none": 0, "int8": 1, "e4m3": 2}
ACTIVATIONS = {None: 0, "none": 0, "silu": 1}
CKPT_BLOCK = 32   # values of a row that share a checkpoint scale


@functools.lru_cache(maxsize=None)
def _dtype_codes():
    torch = _torch()
    return {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _dtype_code(dtype):
    code = _dtype_codes().get(dtype)
    if code is None:
        raise ValueError(f"float32, bfloat16 or float16 values expected, got {dtype}")
    return code


def _named(table, name, what):
    code = table.get(name)
    if code is None:
        raise ValueError(f"{what} must be one of {[k for k in table if k]} or None, got {name!r}")
    return code


def _fit_int(**sizes):
    """Refuses sizes that a C int does not hold (ctypes would cut off their upper bits)."""
    for what, v in sizes.items():
        if not -1 << 31 <= v < 1 << 31:
            raise ValueError(f"{what} must be below 2^31, got {v}")


def _rows(t):
    """t contiguous and 16-byte aligned (a copy where it is not)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _call(index, where, fn, *args):
    """Calls a library function on the current stream of device ``index``, which is made current for it."""
    torch = _torch()
    if torch.cuda.current_device() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != ETP_OK:
        raise EtpError(st, where)


def _addr(t):
    return None if t is None else t.data_ptr()


def _one_device(x, *others):
    """Index of the CUDA device that all of the tensors are on."""
    index = x.get_device()
    if index < 0:
        raise ValueError("libetp operates on CUDA tensors only (no CPU fallback)")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on {x.device} and {t.device} in one call")
    return index


@dataclass
class Checkpoint8:
    """Activations kept in 8 bits: 1 + 1/32 byte a value.

    q: codes in the shape of the activations, int8 or float8_e4m3fn; scale: uint8 [..., ceil(cols / 32)],
    32 values of a row share the scale 2^(byte - 127) (255: the run held a NaN or an infinity and
    restores as NaN); dtype: type of the activations.
    """
    q: object
    scale: object
    dtype: object

    @property
    def shape(self):
        return self.q.shape

    @property
    def format(self):
        return "int8" if self.q.dtype == _torch().int8 else "e4m3"

    @property
    def nbytes(self):
        return self.q.numel() + self.scale.numel()

    def _checked(self):
        """(format code, codes, scales) for the library."""
        torch = _torch()
        q, scale = self.q, self.scale
        fmt = 1 if q.dtype == torch.int8 else 2 if q.dtype == torch.float8_e4m3fn else 0
        if fmt == 0 or scale.dtype != torch.uint8:
            raise ValueError("a checkpoint has int8 or float8_e4m3fn codes and uint8 scales")
        shape = q.shape
        if scale.shape != shape[:-1] + (-(-shape[-1] // CKPT_BLOCK),):
            raise ValueError(f"scales of shape {tuple(scale.shape)} do not fit codes of shape {tuple(shape)}")
        return fmt, _rows(q), _rows(scale)

    def restore(self, dtype=None, out=None):
        """The values the checkpoint stands for, in ``dtype`` (default: that of the activations)."""
        fmt, q, scale = self._checked()
        shape = q.shape
        _fit_int(columns=shape[-1])
        if out is None:
            out = q.new_empty(shape, dtype=dtype or self.dtype)
        elif out.shape != shape or not out.is_contiguous() or (dtype is not None and out.dtype != dtype):
            raise ValueError("out must be contiguous, of the checkpoint's shape and the dtype asked for")
        cols = shape[-1]
        _call(_one_device(q, scale, out), "etp_checkpoint_restore", load_library().etp_checkpoint_restore, fmt,
              _dtype_code(out.dtype), q.numel() // max(cols, 1), cols, q.data_ptr(), scale.data_ptr(), out.data_ptr())
        return out


def _empty_checkpoint(x, fmt):
    torch = _torch()
    shape = x.shape
    return Checkpoint8(x.new_empty(shape, dtype=torch.int8 if fmt == 1 else torch.float8_e4m3fn),
                       x.new_empty(shape[:-1] + (-(-shape[-1] // CKPT_BLOCK),), dtype=torch.uint8), x.dtype)


def checkpoint8(x, fmt="int8"):
    """8-bit checkpoint of x [..., cols] (float32, bfloat16 or float16 CUDA tensor): a Checkpoint8.

    fmt "int8": values within half a step of max|x| / 63.5 of their run of 32 (or 2^-126) at most; "e4m3": within
    2^-4 of each value, or 2^-10 of the scale. EdgeConv.backward, EdgeConv.backward_weights and
    group_norm_backward take a Checkpoint8 in the place of x.
    """
    code = _named(CKPT_FORMATS, fmt, "fmt")
    if code == 0:
        raise ValueError("fmt must be 'int8' or 'e4m3'")
    index = _one_device(x)
    if x.dim() < 1:
        raise ValueError("x needs at least one dimension")
    _fit_int(columns=x.shape[-1])
    dtype = _dtype_code(x.dtype)
    x = x.contiguous()
    ck = _empty_checkpoint(x, code)
    cols = x.shape[-1]
    _call(index, "etp_checkpoint_store", load_library().etp_checkpoint_store, code, dtype, x.numel() // max(cols, 1),
          cols, x.data_ptr(), ck.q.data_ptr(), ck.scale.data_ptr())
    return ck


@functools.lru_cache(maxsize=256)
def group_norm_workspace_bytes(lmax, channels, groups, n_structs=1, backward=False):
    return load_library().etp_group_norm_workspace_bytes(int(lmax), int(channels), int(groups), int(n_structs), int(backward))


def _norm_shape(shape, lmax, groups, node_ptr, weight, bias):
    """(rows, channels, structures) of the checked arguments."""
    if len(shape) != 2:
        raise ValueError("node rows are [n_nodes, channels (lmax + 1)^2]")
    n, dim = shape
    comps = (lmax + 1) ** 2
    if lmax < 0 or dim % comps or dim == 0:
        raise ValueError(f"rows of {dim} values do not hold (lmax + 1)^2 = {comps} components")
    c = dim // comps
    if node_ptr is not None and (node_ptr.dim() != 1 or node_ptr.numel() < 1):
        raise ValueError("node_ptr is a vector of n_structs + 1 row numbers")
    if weight is not None and weight.shape != (lmax + 1, c):
        raise ValueError(f"weight must be [{lmax + 1}, {c}], got {tuple(weight.shape)}")
    if bias is not None and bias.shape != (c,):
        raise ValueError(f"bias must be [{c}], got {tuple(bias.shape)}")
    s = 1 if node_ptr is None else node_ptr.numel() - 1
    _fit_int(rows=n, channels=c, groups=groups, structures=s)
    return n, c, s


def _norm_workspace(lmax, c, groups, s, backward, x, workspace):
    nb = group_norm_workspace_bytes(lmax, c, groups, s, backward)
    if workspace is None or workspace.numel() * workspace.element_size() < nb:
        workspace = x.new_empty(max(nb, 1), dtype=_torch().uint8)
    elif workspace.get_device() != x.get_device():
        raise ValueError(f"workspace on {workspace.device}, tensors on {x.device}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, nb


def _into(out, shape, dtype, x, what):
    """(tensor to write, whether the library made it)"""
    if out is None:
        return x.new_empty(shape, dtype=dtype), True
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype or out.device != x.device or not out.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {x.device}")
    return out, False


def group_norm(x, weight, bias, lmax, groups, node_ptr=None, eps=1e-5, activation="silu", checkpoint=None, out=None,
               stats=None, workspace=None):
    """Group norm with an activation on node rows: (out, stats, checkpoint).

    x: [N, C (lmax+1)^2] CUDA tensor in the uniform node-row layout (float32, bfloat16, float16);
    weight [lmax+1, C], bias [C] (float32, or None); node_ptr: int32 [S + 1] starts of the structures'
    rows (None: one structure). Statistics per structure, rank and group of C / groups channels: mean and
    variance for l = 0, mean square for l > 0. activation "silu": SiLU on l = 0, the same channel's
    logistic gate on l > 0. stats: [S, lmax + 2, groups] (mean; 1 / deviation of every rank), for the
    backward. checkpoint "int8" or "e4m3": also returns the Checkpoint8 of x (else None), in the same
    pass when C % 32 == 0. Rows of no structure: untouched in a given ``out``, zero in a new one.
    """
    index = _one_device(x, weight, bias, node_ptr)
    dtype = _dtype_code(x.dtype)
    n, c, s = _norm_shape(x.shape, lmax, groups, node_ptr, weight, bias)
    act, fmt = _named(ACTIVATIONS, activation, "activation"), _named(CKPT_FORMATS, checkpoint, "checkpoint")
    x = _rows(x)
    weight = None if weight is None else _f32(weight)
    bias = None if bias is None else _f32(bias)
    node_ptr = None if node_ptr is None else _i32(node_ptr)
    out, made = _into(out, x.shape, x.dtype, x, "out")
    stats, _ = _into(stats, (s, lmax + 2, groups), _torch().float32, x, "stats")
    ck = _empty_checkpoint(x, fmt) if fmt else None
    ws, nb = _norm_workspace(lmax, c, groups, s, False, x, workspace)
    _call(index, "etp_group_norm", load_library().etp_group_norm, lmax, c, groups, n, s, _addr(node_ptr), dtype,
          x.data_ptr(), _addr(weight), _addr(bias), eps, act, made, out.data_ptr(), stats.data_ptr(), fmt,
          ck.q.data_ptr() if ck else None, ck.scale.data_ptr() if ck else None, ws.data_ptr(), nb)
    return out, stats, ck


def group_norm_backward(x, stats, weight, bias, grad_out, lmax, groups, node_ptr=None, activation="silu",
                        want_grad_x=True, want_grad_affine=True, grad_x=None, workspace=None):
    """(grad_x, grad_weight, grad_bias) for the cotangent grad_out of group_norm's out.

    x: group_norm's input or its Checkpoint8, whose codes are read directly; stats: from group_norm.
    grad_weight [lmax+1, C] and grad_bias [C] are float32 sums over all structures (None when
    want_grad_affine is false). Rows of no structure: untouched in a given ``grad_x``, zero in a new one.
    """
    kept = isinstance(x, Checkpoint8)
    index = _one_device(grad_out, x.q if kept else x, stats, weight, bias, node_ptr)
    dtype = _dtype_code(grad_out.dtype)
    n, c, s = _norm_shape(x.shape, lmax, groups, node_ptr, weight, bias)
    act = _named(ACTIVATIONS, activation, "activation")
    if grad_out.shape != x.shape or (not kept and grad_out.dtype != x.dtype):
        raise ValueError(f"grad_out must have x's shape and type, got {tuple(grad_out.shape)} {grad_out.dtype}")
    if stats.shape != (s, lmax + 2, groups):
        raise ValueError(f"stats must be [{s}, {lmax + 2}, {groups}], got {tuple(stats.shape)}")
    if not (want_grad_x or want_grad_affine):
        return None, None, None
    grad_out, stats = _rows(grad_out), _f32(stats)
    fmt, q, scale = x._checked() if kept else (0, None, None)
    if kept:
        _one_device(grad_out, scale)
    else:
        x = _rows(x)
    weight = None if weight is None else _f32(weight)
    bias = None if bias is None else _f32(bias)
    node_ptr = None if node_ptr is None else _i32(node_ptr)
    made = False
    if want_grad_x:
        grad_x, made = _into(grad_x, grad_out.shape, grad_out.dtype, grad_out, "grad_x")
    gw = grad_out.new_empty((lmax + 1, c), dtype=_torch().float32) if want_grad_affine else None
    gb = grad_out.new_empty(c, dtype=_torch().float32) if want_grad_affine else None
    ws, nb = _norm_workspace(lmax, c, groups, s, True, grad_out, workspace)
    _call(index, "etp_group_norm_backward", load_library().etp_group_norm_backward, lmax, c, groups, n, s,
          _addr(node_ptr), dtype, None if kept else x.data_ptr(), fmt, _addr(q),
          _addr(scale), stats.data_ptr(), _addr(weight), _addr(bias), act, grad_out.data_ptr(), made,
          grad_x.data_ptr() if want_grad_x else None, _addr(gw), _addr(gb), ws.data_ptr(), nb)
    return (grad_x if want_grad_x else None), gw, gb


def group_norm_check_status(device=None):
    """Synchronise the current stream (of ``device``) and raise if a kernel of an earlier group_norm or
    group_norm_backward call gave up a bounded pipeline wait (the code is cleared). Until then later calls raise."""
    code = ctypes.c_int(0)
    stream = _stream(device) if _torch().cuda.is_available() else None
    _check(load_library().etp_group_norm_status(stream, ctypes.byref(code)), "etp_group_norm_status")


def group_norm_function(checkpoint=None):
    """torch.autograd.Function: out = group_norm(x, weight, bias, lmax, groups, node_ptr, eps, activation);
    gradients for x, weight and bias. checkpoint "int8" or "e4m3": the input is kept for the backward in
    8 bits, and the gradients are taken at the kept values.
    """
    torch = _torch()
    _named(CKPT_FORMATS, checkpoint, "checkpoint")

    class _GroupNormFn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, lmax, groups, node_ptr=None, eps=1e-5, activation="silu"):
            out, stats, ck = group_norm(x.detach(), None if weight is None else weight.detach(),
                                        None if bias is None else bias.detach(), lmax, groups, node_ptr, eps, activation,
                                        checkpoint)
            ctx.args = (lmax, groups, activation)
            ctx.kept_dtype = ck.dtype if ck else None
            ctx.save_for_backward(*((ck.q, ck.scale) if ck else (x, None)), stats, weight, bias, node_ptr)
            return out

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, grad_out):
            x, scale, stats, weight, bias, node_ptr = ctx.saved_tensors
            if ctx.kept_dtype is not None:
                x = Checkpoint8(x, scale, ctx.kept_dtype)
            lmax, groups, activation = ctx.args
            need = ctx.needs_input_grad
            gx, gw, gb = group_norm_backward(x, stats, weight, bias, grad_out, lmax, groups, node_ptr, activation,
                                             need[0], need[1] or need[2])
            return (gx, gw.to(weight.dtype) if need[1] else None, gb.to(bias.dtype) if need[2] else None, None, None,
                    None, None, None)

    return _GroupNormFn


def edge_conv_function(checkpoint=None):
    """torch.autograd.Function: out = conv(x, edge_vec, W); gradients for x, edge_vec and W.

    checkpoint "int8" or "e4m3": the node features are kept for the backward in 8 bits instead of
    float32, and restored to a float32 copy by the backward; the gradients for edge_vec and W are taken at
    the kept values (that for x does not depend on x).
    """
    torch = _torch()
    _named(CKPT_FORMATS, checkpoint, "checkpoint")
    keep = CKPT_FORMATS[checkpoint] != 0

    class _EdgeConvFn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, conv, graph, x, edge_vec, W):
            g = Graph(graph.n_nodes, graph.n_edges, graph.row_ptr, graph.sender, edge_vec.detach(),
                      graph.t_row_ptr, graph.t_perm)
            ctx.conv, ctx.graph = conv, g
            if keep:
                ck = checkpoint8(x.detach(), checkpoint)
                ctx.kept_dtype = ck.dtype
                ctx.save_for_backward(ck.q, ck.scale, W)
            else:
                ctx.save_for_backward(x, W)
            return conv.forward(g, x.detach(), W.detach())

        @staticmethod
        def backward(ctx, grad_out):
            if keep:
                q, scale, W = ctx.saved_tensors
                x = Checkpoint8(q, scale, ctx.kept_dtype).restore(dtype=torch.float32)
            else:
                x, W = ctx.saved_tensors
            go = grad_out.contiguous()
            gx = gv = gW = None
            if ctx.needs_input_grad[2] or ctx.needs_input_grad[3]:
                gx, gv = ctx.conv.backward(ctx.graph, x.detach(), W.detach(), go, ctx.needs_input_grad[2],
                                           ctx.needs_input_grad[3])
            if ctx.needs_input_grad[4]:
                gW = ctx.conv.backward_weights(ctx.graph, x.detach(), go).reshape(W.shape)
            return None, None, gx, gv, gW

    return _EdgeConvFn
