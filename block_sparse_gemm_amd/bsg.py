"""Thin ctypes binding of ``include/bsg.h`` (libbsg.so).

Each function has the name of its C entry point without the ``bsg_``
prefix and only marshals arguments: torch tensors in, raw device pointers,
sizes and the current HIP stream out.  Every step of the layer runs in the
library's gfx950 kernels; there is no fallback of any kind: if the library
is missing this module raises on first use.
"""
from __future__ import annotations

import array
import ctypes as C
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libbsg.so")

OK, EINVAL, EUNSUPPORTED, EHIP = 0, -1, -2, -3
F32, BF16, E4M3 = 0, 1, 2
EPI_NONE, EPI_GELU, EPI_SILU_MUL, EPI_GELU_BWD, EPI_SILU_MUL_BWD = 0, 1, 2, 3, 4
BLOCK = 128
MAX_EXPERTS = 1024
MAX_TOPK = 32
ROUTE_SCRATCH_BYTES = 4 << 20   # BSG_ROUTE_SCRATCH_BYTES

EPILOGUES = {"none": EPI_NONE, "gelu": EPI_GELU, "silu_mul": EPI_SILU_MUL,
             "gelu_bwd": EPI_GELU_BWD, "silu_mul_bwd": EPI_SILU_MUL_BWD}

# Every symbol include/bsg.h declares.
SYMBOLS = ("bsg_max_padded_rows", "bsg_topology_sizes", "bsg_route_workspace_bytes", "bsg_route",
           "bsg_route_noalloc",
           "bsg_route_backward", "bsg_permute_pad", "bsg_permute_pad_gate_backward",
           "bsg_build_topology", "bsg_route_topology", "bsg_route_permute_topology", "bsg_sdd", "bsg_dsd", "bsg_dsd_workspace_bytes",
           "bsg_dsd_combine_top1", "bsg_dstd",
           "bsg_unpermute_combine", "bsg_rms_norm", "bsg_rms_norm_backward",
           "bsg_rms_norm_backward_workspace_bytes", "bsg_grouped_gemm",
           "bsg_grouped_gemm_workspace_bytes", "bsg_grouped_wgrad",
           "bsg_grouped_wgrad_workspace_bytes", "bsg_grad_norm",
           "bsg_grad_norm_workspace_bytes", "bsg_grad_clip", "bsg_stream_copy", "bsg_status_string", "bsg_last_error")


class BsgError(RuntimeError):
    def __init__(self, call, status, detail):
        super().__init__(f"{call}: status {status} ({detail})")
        self.status = status


class TopoSizes(C.Structure):
    _fields_ = [("row_blocks_max", C.c_int64), ("nnz_max", C.c_int64), ("n_cols", C.c_int64),
                ("row_tiles_max", C.c_int64)]


class TopologyStruct(C.Structure):
    _fields_ = [("row_ptr", C.c_void_p), ("col_idx", C.c_void_p), ("row_idx", C.c_void_p),
                ("col_ptr", C.c_void_p), ("trans_idx", C.c_void_p), ("row_tiles", C.c_void_p),
                ("expert_order", C.c_void_p), ("meta", C.c_void_p),
                ("E", C.c_int32), ("F", C.c_int32), ("block_rows", C.c_int32),
                ("Tp_max", C.c_int64)]


_lib = None


def lib():
    """Load libbsg.so (built by ``python -m block_sparse_gemm_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run python -m block_sparse_gemm_amd.build")
        L = C.CDLL(LIB_PATH)
        vp, i64, i32, sz = C.c_void_p, C.c_int64, C.c_int, C.c_size_t
        L.bsg_max_padded_rows.restype = i64
        L.bsg_max_padded_rows.argtypes = [i64, i32, i32, i32]
        L.bsg_topology_sizes.restype = i32
        L.bsg_topology_sizes.argtypes = [i64, i32, i32, i32, C.POINTER(TopoSizes)]
        L.bsg_route_workspace_bytes.restype = sz
        L.bsg_route_workspace_bytes.argtypes = [i64, i32, i32]
        L.bsg_route.restype = i32
        L.bsg_route.argtypes = [vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
        L.bsg_stream_copy.restype = i32
        L.bsg_stream_copy.argtypes = [vp, vp, sz, vp]
        L.bsg_route_noalloc.restype = i32
        L.bsg_route_noalloc.argtypes = [vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
        L.bsg_route_backward.restype = i32
        L.bsg_route_backward.argtypes = [vp, i64, i32, i32, i32, vp, vp, vp, i32, i32, vp, i32,
                                         i64, vp, vp]
        L.bsg_permute_pad.restype = i32
        L.bsg_permute_pad.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp, vp, i32, i32, i64, vp, vp,
                                      vp]
        L.bsg_permute_pad_gate_backward.restype = i32
        L.bsg_permute_pad_gate_backward.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp, vp, i32,
                                                    i32, i64, vp, vp, vp, i32, vp, vp, i32, i64,
                                                    vp, vp]
        L.bsg_build_topology.restype = i32
        L.bsg_build_topology.argtypes = [vp, i32, i32, i64, C.POINTER(TopologyStruct), vp]
        L.bsg_route_topology.restype = i32
        L.bsg_route_topology.argtypes = [vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz,
                                         i32, i64, C.POINTER(TopologyStruct), vp]
        L.bsg_route_permute_topology.restype = i32
        L.bsg_route_permute_topology.argtypes = [vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp,
                                                 vp, sz, vp, i32, i32, i64, vp, vp, i32,
                                                 C.POINTER(TopologyStruct), vp]
        L.bsg_sdd.restype = i32
        L.bsg_sdd.argtypes = [vp, i64, vp, vp, i64, i32, i32, C.POINTER(TopologyStruct), i32, vp,
                              vp, vp, i32, vp]
        L.bsg_dsd.restype = i32
        L.bsg_dsd.argtypes = [vp, vp, C.POINTER(TopologyStruct), vp, vp, i64, i32, i32, vp, i64,
                              i32, i32, vp, sz, vp]
        L.bsg_dsd_workspace_bytes.restype = i32
        L.bsg_dsd_workspace_bytes.argtypes = [vp, C.POINTER(i64)]
        L.bsg_dsd_combine_top1.restype = i32
        L.bsg_dsd_combine_top1.argtypes = [vp, C.POINTER(TopologyStruct), vp, i64, i32, i32, vp,
                                           i64, vp, vp, vp, i64, i32, vp]
        L.bsg_dstd.restype = i32
        L.bsg_dstd.argtypes = [vp, C.POINTER(TopologyStruct), vp, i64, i32, vp, i64, i32, i32,
                               vp]
        L.bsg_unpermute_combine.restype = i32
        L.bsg_unpermute_combine.argtypes = [vp, i32, i64, vp, vp, i64, i32, i32, vp, i32, vp]
        f32 = C.c_float
        L.bsg_rms_norm.restype = i32
        L.bsg_rms_norm.argtypes = [vp, i64, vp, i64, vp, f32, i64, i32, i32, vp, i64, vp, i64,
                                   i32, vp, vp, vp]
        L.bsg_rms_norm_backward_workspace_bytes.restype = sz
        L.bsg_rms_norm_backward_workspace_bytes.argtypes = [i64, i32]
        L.bsg_rms_norm_backward.restype = i32
        L.bsg_rms_norm_backward.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, i64, i32, i32, vp,
                                            i64, vp, vp, sz, vp]
        L.bsg_grouped_gemm_workspace_bytes.restype = sz
        L.bsg_grouped_gemm_workspace_bytes.argtypes = [i64, i32, i32, i32, i32]
        L.bsg_grouped_gemm.restype = i32
        L.bsg_grouped_gemm.argtypes = [vp, vp, i64, vp, vp, vp, i64, i64, vp, i32, vp, i32, i64,
                                       i32, i32, i32, vp, vp, i64, i32, vp, i32, vp, sz, vp]
        L.bsg_grouped_wgrad.restype = i32
        L.bsg_grouped_wgrad.argtypes = [vp, i64, vp, i64, vp, i32, i64, i32, i32, vp, i64, i64,
                                        i32, i32, vp, sz, vp]
        L.bsg_grouped_wgrad_workspace_bytes.restype = sz
        L.bsg_grouped_wgrad_workspace_bytes.argtypes = [i64, i32, i32, i32]
        L.bsg_grad_norm_workspace_bytes.restype = sz
        L.bsg_grad_norm_workspace_bytes.argtypes = []
        L.bsg_grad_norm.restype = i32
        L.bsg_grad_norm.argtypes = [vp, vp, vp, i32, vp, vp, sz, vp]
        L.bsg_grad_clip.restype = i32
        L.bsg_grad_clip.argtypes = [vp, vp, vp, vp, i32, vp, f32, vp]
        L.bsg_status_string.restype = C.c_char_p
        L.bsg_status_string.argtypes = [i32]
        L.bsg_last_error.restype = C.c_char_p
        L.bsg_last_error.argtypes = []
        _lib = L
    return _lib


def _check(call: str, status: int) -> None:
    if status != OK:
        raise BsgError(call, status, lib().bsg_last_error().decode())


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream():
    if torch.cuda.is_available():
        return C.c_void_p(torch.cuda.current_stream().cuda_stream)
    return None


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def torch_dtype(code: int):
    return torch.bfloat16 if code == BF16 else torch.float32


def _ld(t: torch.Tensor) -> int:
    assert t.dim() == 2 and t.stride(1) == 1, "operands must be row-major 2-D views"
    return t.stride(0)


# ------------------------------------------------------------- size queries

def max_padded_rows(T: int, k: int, E: int, bin_rows: int = BLOCK) -> int:
    return int(lib().bsg_max_padded_rows(T, k, E, bin_rows))


def topology_sizes(Tp_max: int, E: int, f: int, block_rows: int = BLOCK) -> TopoSizes:
    out = TopoSizes()
    _check("topology_sizes", lib().bsg_topology_sizes(Tp_max, E, f, block_rows, C.byref(out)))
    return out


def route_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(lib().bsg_route_workspace_bytes(T, k, E))


# ------------------------------------------------------------------ topology

class Topology:
    """Device buffers of one hybrid BCSR-COO topology (capacity for Tp_max),
    in blocks of block_rows (128, or 64 for bins of 64 rows) x 128."""

    def __init__(self, Tp_max: int, E: int, f: int, device="cuda", block_rows: int = BLOCK):
        sz = topology_sizes(Tp_max, E, f, block_rows)
        i32 = dict(dtype=torch.int32, device=device)
        self.E, self.F, self.f, self.Tp_max = E, f // BLOCK, f, Tp_max
        self.block_rows = block_rows
        self.row_blocks_max, self.nnz_max = int(sz.row_blocks_max), int(sz.nnz_max)
        self.row_ptr = torch.zeros(self.row_blocks_max + 1, **i32)
        self.col_idx = torch.zeros(self.nnz_max, **i32)
        self.row_idx = torch.zeros(self.nnz_max, **i32)
        self.col_ptr = torch.zeros(E * self.F + 1, **i32)
        self.trans_idx = torch.zeros(self.nnz_max, **i32)
        self.row_tiles_max = int(sz.row_tiles_max)
        self.row_tiles = torch.zeros(self.row_tiles_max, **i32)
        self.expert_order = torch.zeros(E, **i32)
        self.meta = torch.zeros(4, **i32)
        self.struct = TopologyStruct(self.row_ptr.data_ptr(), self.col_idx.data_ptr(),
                                     self.row_idx.data_ptr(), self.col_ptr.data_ptr(),
                                     self.trans_idx.data_ptr(), self.row_tiles.data_ptr(),
                                     self.expert_order.data_ptr(), self.meta.data_ptr(), E,
                                     self.F, block_rows, Tp_max)


# ------------------------------------------------------------------- calls

def route(logits, k, renorm, expert_idx, gate, dest_row, counts, bin_offsets, workspace,
          bin_rows=BLOCK):
    T, E = logits.shape
    _check("route", lib().bsg_route(_ptr(logits), T, E, k, int(bool(renorm)), bin_rows,
                                    _ptr(expert_idx),
                                    _ptr(gate), _ptr(dest_row), _ptr(counts), _ptr(bin_offsets),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream()))


def route_noalloc(logits, k, renorm, expert_idx, gate, dest_row, counts, bin_offsets,
                  bin_rows=BLOCK):
    T, E = logits.shape
    _check("route_noalloc", lib().bsg_route_noalloc(
        _ptr(logits), T, E, k, int(bool(renorm)), bin_rows, _ptr(expert_idx), _ptr(gate),
        _ptr(dest_row), _ptr(counts), _ptr(bin_offsets), _stream()))


def route_backward(logits, k, renorm, expert_idx, dest_row, dy, yp, dlogits):
    T, E = logits.shape
    _check("route_backward", lib().bsg_route_backward(
        _ptr(logits), T, E, k, int(bool(renorm)), _ptr(expert_idx), _ptr(dest_row), _ptr(dy),
        dtype_code(dy), dy.shape[1], _ptr(yp), dtype_code(yp), _ld(yp), _ptr(dlogits),
        _stream()))


def permute_pad(x, k, dest_row, scale, counts, bin_offsets, E, Tp_max, row_src, xp,
                bin_rows=BLOCK):
    T, d = x.shape
    _check("permute_pad", lib().bsg_permute_pad(_ptr(x), dtype_code(x), T, d, k, _ptr(dest_row),
                                                _ptr(scale), _ptr(counts), _ptr(bin_offsets), E,
                                                bin_rows, Tp_max, _ptr(row_src), _ptr(xp),
                                                _stream()))


def permute_pad_gate_backward(dy, k, dest_row, gate, counts, bin_offsets, E, Tp_max, row_src,
                              dyp, logits, renorm, expert_idx, yp, dlogits, bin_rows=BLOCK):
    T, d = dy.shape
    _check("permute_pad_gate_backward", lib().bsg_permute_pad_gate_backward(
        _ptr(dy), dtype_code(dy), T, d, k, _ptr(dest_row), _ptr(gate), _ptr(counts),
        _ptr(bin_offsets), E, bin_rows, Tp_max, _ptr(row_src), _ptr(dyp), _ptr(logits),
        int(bool(renorm)), _ptr(expert_idx), _ptr(yp), dtype_code(yp), _ld(yp), _ptr(dlogits),
        _stream()))


def build_topology(bin_offsets, E, f, Tp_max, topo: Topology):
    _check("build_topology", lib().bsg_build_topology(_ptr(bin_offsets), E, f, Tp_max,
                                                      C.byref(topo.struct), _stream()))


def route_topology(logits, k, renorm, expert_idx, gate, dest_row, counts, bin_offsets, workspace,
                   f, Tp_max, topo: Topology, bin_rows=BLOCK):
    """route + build_topology, the topology written by the routing's own launch."""
    T, E = logits.shape
    _check("route_topology", lib().bsg_route_topology(
        _ptr(logits), T, E, k, int(bool(renorm)), bin_rows, _ptr(expert_idx), _ptr(gate),
        _ptr(dest_row), _ptr(counts), _ptr(bin_offsets), _ptr(workspace),
        workspace.numel() * workspace.element_size(), f, Tp_max, C.byref(topo.struct),
        _stream()))


def route_permute_topology(logits, k, renorm, expert_idx, gate, dest_row, counts, bin_offsets,
                           workspace, x, Tp_max, row_src, xp, f=0, topo: Topology = None,
                           bin_rows=BLOCK):
    """route + permute_pad (no scale) + build_topology (topo may be None) in
    the routing's two launches."""
    T, E = logits.shape
    _check("route_permute_topology", lib().bsg_route_permute_topology(
        _ptr(logits), T, E, k, int(bool(renorm)), bin_rows, _ptr(expert_idx), _ptr(gate),
        _ptr(dest_row), _ptr(counts), _ptr(bin_offsets), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(x), dtype_code(x), x.shape[1],
        Tp_max, _ptr(row_src), _ptr(xp), f, C.byref(topo.struct) if topo is not None else None,
        _stream()))


def sdd(a, b, K, topo: Topology, epilogue, out_blocks, b2=None, trans_b=False, aux_in=None,
        aux_out=None):
    epi = EPILOGUES[epilogue] if isinstance(epilogue, str) else int(epilogue)
    _check("sdd", lib().bsg_sdd(_ptr(a), _ld(a), _ptr(b), _ptr(b2), _ld(b), int(bool(trans_b)),
                                K, C.byref(topo.struct), epi, _ptr(aux_in), _ptr(out_blocks),
                                _ptr(aux_out), dtype_code(a), _stream()))


def dsd(blocks, topo: Topology, b, N, c, trans_b=False, blocks2=None, b2=None, workspace=None):
    """bsg_dsd; workspace (a device tensor, or None) lets the product split
    its last round (see dsd_workspace_bytes)."""
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("dsd", lib().bsg_dsd(_ptr(blocks), _ptr(blocks2), C.byref(topo.struct), _ptr(b),
                                _ptr(b2), _ld(b), int(bool(trans_b)), N, _ptr(c), _ld(c),
                                dtype_code(c), dtype_code(blocks), _ptr(workspace), nbytes,
                                _stream()))


def dsd_workspace_bytes() -> int:
    """Bytes of a bsg_dsd workspace that allows every split of its last round
    on the current device (one 256 KiB share per compute unit)."""
    out = C.c_int64(0)
    _check("dsd_workspace_bytes", lib().bsg_dsd_workspace_bytes(_stream(), C.byref(out)))
    return int(out.value)


def dsd_combine_top1(blocks, topo: Topology, b, N, c, row_src, gate, y, trans_b=False):
    """bsg_dsd + bsg_unpermute_combine for top-1 routing in one launch (c may
    be None: only y is written)."""
    _check("dsd_combine_top1", lib().bsg_dsd_combine_top1(
        _ptr(blocks), C.byref(topo.struct), _ptr(b), _ld(b), int(bool(trans_b)), N, _ptr(c),
        _ld(c) if c is not None else 0, _ptr(row_src), _ptr(gate), _ptr(y), _ld(y),
        dtype_code(blocks), _stream()))


def dstd(blocks, topo: Topology, dmat, N, c, trans_c=False):
    _check("dstd", lib().bsg_dstd(_ptr(blocks), C.byref(topo.struct), _ptr(dmat), _ld(dmat), N,
                                  _ptr(c), _ld(c), int(bool(trans_c)), dtype_code(blocks),
                                  _stream()))


def unpermute_combine(yp, dest_row, gate, T, k, d, y):
    _check("unpermute_combine", lib().bsg_unpermute_combine(
        _ptr(yp), dtype_code(yp), _ld(yp), _ptr(dest_row), _ptr(gate), T, k, d, _ptr(y),
        dtype_code(y), _stream()))


# ------------------------------------------- norm, ragged products, clipping
#
# These take their sizes from the tensors, so what the C call cannot see (that
# the tensors agree, and lie on the current device) is checked here.  The
# checks are written to cost little: a small call takes about as long here as
# on the GPU.

_F8 = torch.float8_e4m3fn
_CODES = {torch.float32: F32, torch.bfloat16: BF16, _F8: E4M3}


def _fail(call, what):
    raise ValueError(f"{call}: {what}")


def _current(call, tensors):
    """The current stream, if every tensor (or None) is on the current GPU."""
    devices = {t.get_device() for t in tensors if t is not None}
    dev = devices.pop()
    if devices or dev < 0 or dev != torch.cuda.current_device():
        _fail(call, "tensors must be on the current GPU")
    return torch._C._cuda_getCurrentRawStream(dev)


def _address(t):
    return None if t is None else t.data_ptr()


def _rows(call, name, t, shape, dtype):
    """The leading dimension of a row-major [T, d] tensor."""
    if t.shape != shape or t.dtype != dtype or shape[1] >> 31:
        _fail(call, f"{name} must be a {list(shape)} tensor of {dtype}, under 2^31 wide")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1 and shape[0]:
        _fail(call, f"{name} must be row-major")
    return ld if shape[0] > 1 else shape[1]   # one row has no stride to speak of


def _vector(call, name, t, n, dtype):
    if t.dim() != 1 or t.numel() != n or t.dtype != dtype or not t.is_contiguous():
        _fail(call, f"{name} must be a contiguous vector of {n} {dtype}")


def _nbytes(call, t):
    if t is None:
        return 0
    if not t.is_contiguous():
        _fail(call, "the workspace must be contiguous")
    return t.numel() * t.element_size()


def rms_norm(x, weight, eps, y, h=None, residual=None, y_scale=None, rstd=None):
    """y = rms_norm(x + residual) * weight; y in x's type, or in
    torch.float8_e4m3fn with y_scale [T]; h (with a residual) takes the sum."""
    c = "rms_norm"
    stream = _current(c, (x, weight, y, h, residual, y_scale, rstd))
    shape, dt = x.shape, x.dtype
    if len(shape) != 2:
        _fail(c, "x must be a [T, d] tensor")
    T, d = shape
    code = dtype_code(x)
    ycode = E4M3 if y.dtype == _F8 else code
    ldx = _rows(c, "x", x, shape, dt)
    ldy = _rows(c, "y", y, shape, _F8 if ycode == E4M3 else dt)
    ldr = _rows(c, "residual", residual, shape, dt) if residual is not None else 0
    ldh = _rows(c, "h", h, shape, dt) if h is not None else 0
    _vector(c, "weight", weight, d, dt)
    if y_scale is not None:
        _vector(c, "y_scale", y_scale, T, torch.float32)
    if rstd is not None:
        _vector(c, "rstd", rstd, T, torch.float32)
    _check(c, lib().bsg_rms_norm(
        x.data_ptr(), ldx, _address(residual), ldr, weight.data_ptr(), eps, T, d, code,
        _address(h), ldh, y.data_ptr(), ldy, ycode, _address(y_scale), _address(rstd), stream))


def rms_norm_backward_workspace_bytes(T: int, d: int) -> int:
    return int(lib().bsg_rms_norm_backward_workspace_bytes(T, d))


def rms_norm_backward(dy, h, weight, rstd, dx, dweight, workspace, dh=None):
    """dx (of x and of the residual alike) and dweight (fp32) from dy and,
    when given, the gradient dh that reaches h along the residual stream."""
    c = "rms_norm_backward"
    stream = _current(c, (dy, h, weight, rstd, dx, dweight, workspace, dh))
    shape, dt = dy.shape, dy.dtype
    if len(shape) != 2:
        _fail(c, "dy must be a [T, d] tensor")
    T, d = shape
    lddy = _rows(c, "dy", dy, shape, dt)
    ldh = _rows(c, "h", h, shape, dt)
    lddx = _rows(c, "dx", dx, shape, dt)
    lddh = _rows(c, "dh", dh, shape, dt) if dh is not None else 0
    _vector(c, "weight", weight, d, dt)
    _vector(c, "rstd", rstd, T, torch.float32)
    _vector(c, "dweight", dweight, d, torch.float32)
    _check(c, lib().bsg_rms_norm_backward(
        dy.data_ptr(), lddy, _address(dh), lddh, h.data_ptr(), ldh, weight.data_ptr(),
        rstd.data_ptr(), T, d, dtype_code(dy), dx.data_ptr(), lddx, dweight.data_ptr(),
        workspace.data_ptr(), _nbytes(c, workspace), stream))


def _operand_code(t):
    return E4M3 if t.dtype == _F8 else dtype_code(t)


def _matrices(call, name, t, shape, dtype):
    """(ld, stride) of one matrix an expert, [E, rows, cols] with contiguous rows."""
    if t.shape != shape or t.dtype != dtype or max(shape) >> 31:
        _fail(call, f"{name} must be a {list(shape)} tensor of {dtype}, sizes under 2^31")
    stride, ld, one = t.stride()
    if one != 1 and shape[2] > 1:
        _fail(call, f"{name} must have contiguous rows")
    return ld if shape[1] > 1 else shape[2], stride if shape[0] > 1 else 16


def _code_of(epilogue):
    return EPILOGUES[epilogue] if isinstance(epilogue, str) else int(epilogue)


def grouped_gemm_workspace_bytes(M: int, K: int, N: int, E: int, epilogue="none") -> int:
    """Bytes of a workspace that lets grouped_gemm split few-row products (0:
    it never splits this one)."""
    return int(lib().bsg_grouped_gemm_workspace_bytes(M, K, N, E, _code_of(epilogue)))


def grouped_gemm(a, row_offsets, b, c, epilogue="none", trans_b=False, a2=None, b2=None,
                 a_scale=None, b_scale=None, aux_in=None, aux_out=None, workspace=None):
    """c[r] = epilogue(a[r] @ b[e]) for the rows r of expert e, row_offsets[e]
    <= r < row_offsets[e + 1].  b is [E, K, N], or [E, N, K] with trans_b, a
    view with contiguous rows (the layer's W1 [d, E f]: W1.view(d, E,
    f).permute(1, 0, 2)); a, b of bf16, fp32 or float8_e4m3fn (with a_scale
    [M], b_scale [E, N], or [2, E, N] with b2).  c is [M, N]; two-plane
    arrays (silu_mul's aux_out, silu_mul_bwd's aux_in and c) [2, M, N]."""
    call = "grouped_gemm"
    stream = _current(call, (a, row_offsets, b, c, a2, b2, a_scale, b_scale, aux_in, aux_out,
                             workspace))
    epi = _code_of(epilogue)
    if a.dim() != 2 or b.dim() != 3:
        _fail(call, "a is [M, K], b one matrix an expert")
    M, K = a.shape
    E, N = b.shape[0], b.shape[1 if trans_b else 2]
    lda = _rows(call, "a", a, a.shape, a.dtype)
    ldb, stride = _matrices(call, "b", b, (E, N, K) if trans_b else (E, K, N), a.dtype)
    _vector(call, "row_offsets", row_offsets, E + 1, torch.int32)
    if a2 is not None and _rows(call, "a2", a2, a.shape, a.dtype) != lda:
        _fail(call, "a2 must be laid out as a")
    if b2 is not None and _matrices(call, "b2", b2, b.shape, a.dtype) != (ldb, stride):
        _fail(call, "b2 must be laid out as b")
    if a_scale is not None:
        _vector(call, "a_scale", a_scale, M, torch.float32)
    if b_scale is not None:
        n = (2 if b2 is not None else 1) * E * N
        if b_scale.numel() != n or b_scale.dtype != torch.float32 or not b_scale.is_contiguous():
            _fail(call, f"b_scale must be {n} contiguous fp32 values")

    def planes(name, t, two, ld=None):
        if t.dim() != (3 if two else 2) or (two and t.shape[0] != 2):
            _fail(call, f"{name} must be a [{'2, ' if two else ''}{M}, {N}] tensor")
        got = _rows(call, name, t[0] if two else t, (M, N), c.dtype)
        if ld is not None and got != ld:
            _fail(call, f"{name} must be laid out as c")
        if two and M and t.stride(0) != M * got:
            _fail(call, f"the second plane of {name} must follow the first")
        return got

    ldc = planes("c", c, epi == EPI_SILU_MUL_BWD)
    if aux_in is not None:
        planes("aux_in", aux_in, epi == EPI_SILU_MUL_BWD, ldc)
    if aux_out is not None:
        planes("aux_out", aux_out, epi == EPI_SILU_MUL, ldc)
    _check(call, lib().bsg_grouped_gemm(
        a.data_ptr(), _address(a2), lda, _address(a_scale), b.data_ptr(), _address(b2), ldb,
        stride, _address(b_scale), int(bool(trans_b)), row_offsets.data_ptr(), E, M, K, N, epi,
        _address(aux_in), c.data_ptr(), ldc, dtype_code(c), _address(aux_out), _operand_code(a),
        _address(workspace), _nbytes(call, workspace), stream))


def grouped_wgrad_workspace_bytes(M: int, K: int, N: int, E: int) -> int:
    """Bytes of a workspace that lets grouped_wgrad split long groups (0: it
    never splits this one)."""
    return int(lib().bsg_grouped_wgrad_workspace_bytes(M, K, N, E))


def grouped_wgrad(a, dmat, row_offsets, c, workspace=None):
    """c[e] = a[rows of e]^T @ dmat[rows of e]: c is an [E, K, N] view with
    contiguous rows, of a's type or fp32."""
    call = "grouped_wgrad"
    stream = _current(call, (a, dmat, row_offsets, c, workspace))
    if a.dim() != 2 or dmat.dim() != 2 or c.dim() != 3:
        _fail(call, "a is [M, K], dmat [M, N], c one matrix an expert")
    M, K = a.shape
    N, E = dmat.shape[1], c.shape[0]
    lda = _rows(call, "a", a, a.shape, a.dtype)
    ldd = _rows(call, "dmat", dmat, (M, N), a.dtype)
    ldc, stride = _matrices(call, "c", c, (E, K, N), c.dtype)
    _vector(call, "row_offsets", row_offsets, E + 1, torch.int32)
    _check(call, lib().bsg_grouped_wgrad(
        a.data_ptr(), lda, dmat.data_ptr(), ldd, row_offsets.data_ptr(), E, M, K, N, c.data_ptr(),
        ldc, stride, dtype_code(c), dtype_code(a), _address(workspace), _nbytes(call, workspace),
        stream))


def _tensor_list(call, name, tensors):
    """Addresses, sizes and type codes of a list of gradients, as C arrays."""
    T = torch.Tensor
    if not all(map(T.is_contiguous, tensors)):
        _fail(call, f"{name} must be contiguous")
    try:
        codes = [_CODES[t.dtype] for t in tensors]
    except KeyError as e:
        raise TypeError(f"{call}: unsupported dtype {e}") from None
    return (array.array("Q", map(T.data_ptr, tensors)), array.array("q", map(T.numel, tensors)),
            array.array("i", codes))


def _start(a):
    return a.buffer_info()[0] if a else None


def grad_norm_workspace_bytes() -> int:
    return int(lib().bsg_grad_norm_workspace_bytes())


def grad_norm(grads, norm, workspace):
    """norm (one fp32) = the 2-norm over all values of the tensors in grads."""
    c = "grad_norm"
    stream = _current(c, (norm, workspace, *grads))
    if norm.numel() != 1 or norm.dtype != torch.float32:
        _fail(c, "norm must be one fp32 value")
    ptrs, counts, dtypes = _tensor_list(c, "grads", grads)
    _check(c, lib().bsg_grad_norm(_start(ptrs), _start(counts), _start(dtypes), len(grads),
                                  norm.data_ptr(), workspace.data_ptr(), _nbytes(c, workspace),
                                  stream))


def grad_clip(grads, norm, max_norm, out=None):
    """Scale grads by min(1, max_norm / norm), in place or into out."""
    c = "grad_clip"
    stream = _current(c, (norm, *grads, *(out or ())))
    if norm.numel() != 1 or norm.dtype != torch.float32:
        _fail(c, "norm must be one fp32 value")
    ptrs, counts, dtypes = _tensor_list(c, "grads", grads)
    to = None
    if out is not None:
        to, out_counts, out_dtypes = _tensor_list(c, "out", out)
        if out_counts != counts or out_dtypes != dtypes:
            _fail(c, "out must have the sizes and types of grads")
    _check(c, lib().bsg_grad_clip(_start(ptrs), _start(to) if to else None, _start(counts),
                                  _start(dtypes), len(grads), norm.data_ptr(), max_norm, stream))


def stream_copy(src, dst, nbytes=None):
    """Copy nbytes (default: all of src) from src to dst with the library's
    streaming copy (a measurement ceiling, not a step of the layer)."""
    n = src.numel() * src.element_size() if nbytes is None else int(nbytes)
    _check("stream_copy", lib().bsg_stream_copy(_ptr(src), _ptr(dst), n, _stream()))
