"""MI355X (gfx950) compressed-MLP matmul: Python binding of libunweight.

Argument marshalling only: every step runs in libunweight's host code or
gfx950 kernels.  PyTorch provides device memory and the current HIP stream.
The names follow include/unweight.h without the ``uw_`` prefix.

Method: Cloudflare, "Unweight: how we compressed an LLM 22% without
sacrificing quality" -- lossless BF16 exponent compression of MLP weights with
four pipelines ("Four ways to use compressed weights") and a reconstructive
matmul ("How the reconstructive matmul works").
"""
from __future__ import annotations

import ctypes as ct
from typing import NamedTuple

import numpy as np

from ._capi import (  # noqa: F401
    SECTION_NAMES, UW_KERNEL_AUTO, UW_KERNEL_GEMV, UW_KERNEL_MFMA, UW_KERNEL_SKINNY, UW_NUM_SECTIONS,
    UW_ACT_GELU, UW_ACT_GELU_TANH, UW_ACT_NONE, UW_ACT_RELU, UW_ACT_SILU, UW_BF16, UW_F32,
    UW_PIPE_AUTO, UW_PIPE_BF16, UW_PIPE_DIRECT, UW_PIPE_EXP, UW_PIPE_FULL, UW_PIPE_HUFF, UW_PIPE_PAL,
    UW_SEC_BITMAP, UW_SEC_DLUT, UW_SEC_GLEN, UW_SEC_MLUT, UW_SEC_NIB, UW_SEC_SM, UW_SEC_STREAM,
    UW_SEC_TILE_OFF, UW_SEC_TILE_VBASE, UW_SEC_VEXP, UW_EUNSUPPORTED, UW_EINVAL, UW_STATIC_SCRATCH_BYTES,
    UnweightError, check, lib,
    uw_dmat, uw_info,
    uw_opts,
)

PIPELINES = {"full": UW_PIPE_FULL, "exp": UW_PIPE_EXP, "pal": UW_PIPE_PAL, "direct": UW_PIPE_DIRECT}
ACTIVATIONS = {"none": UW_ACT_NONE, "relu": UW_ACT_RELU, "silu": UW_ACT_SILU, "gelu": UW_ACT_GELU,
               "gelu_tanh": UW_ACT_GELU_TANH}
KERNELS = {"auto": UW_KERNEL_AUTO, "gemv": UW_KERNEL_GEMV, "mfma": UW_KERNEL_MFMA, "skinny": UW_KERNEL_SKINNY}

# sections each use reads on the device
DECODE_SECTIONS = ("sm", "stream", "glen", "tile_off", "tile_vbase", "vexp", "bitmap", "dlut", "mlut")
DIRECT_SECTIONS = ("sm", "nib", "vexp", "bitmap", "tile_vbase")
SECTION_DTYPES = {"sm": np.uint8, "stream": np.uint8, "glen": np.uint8, "tile_off": np.uint32,
                  "tile_vbase": np.uint32, "vexp": np.uint8, "bitmap": np.uint64, "nib": np.uint8,
                  "dlut": np.uint8, "mlut": np.uint32}


def _torch():
    import torch
    return torch


def _stream(stream):
    if stream is not None:
        return ct.c_void_p(stream)
    return ct.c_void_p(_torch().cuda.current_stream().cuda_stream)


def _ptr(t):
    return ct.c_void_p(0 if t is None else t.data_ptr())


# ------------------------------------------------------------------ host blob
class Blob:
    """A compressed matrix on the host (owns a uw_blob*)."""

    def __init__(self, handle: ct.c_void_p):
        self._h = handle

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and h.value:
            lib().uw_blob_free(h)
            self._h = None

    @property
    def handle(self):
        return self._h

    def info(self) -> uw_info:
        inf = uw_info()
        check(lib().uw_blob_info(self._h, ct.byref(inf)), "uw_blob_info")
        return inf

    def section(self, name) -> np.ndarray:
        """Copy of a section as a numpy array of its on-disk dtype."""
        idx = SECTION_NAMES.index(name)
        p, n = ct.c_void_p(), ct.c_uint64()
        check(lib().uw_blob_section(self._h, idx, ct.byref(p), ct.byref(n)), "uw_blob_section")
        if n.value == 0:
            return np.zeros(0, dtype=SECTION_DTYPES[name])
        raw = np.ctypeslib.as_array(ct.cast(p, ct.POINTER(ct.c_uint8)), shape=(n.value,)).copy()
        return raw.view(SECTION_DTYPES[name])

    def validate(self):
        check(lib().uw_validate(self._h), "uw_validate")

    def add_palette(self):
        check(lib().uw_blob_add_palette(self._h), "uw_blob_add_palette")

    def serialize(self) -> bytes:
        need = ct.c_uint64()
        check(lib().uw_blob_serialize(self._h, None, 0, ct.byref(need)), "uw_blob_serialize")
        buf = (ct.c_uint8 * need.value)()
        check(lib().uw_blob_serialize(self._h, buf, need.value, ct.byref(need)), "uw_blob_serialize")
        return bytes(buf)

    @staticmethod
    def deserialize(data: bytes) -> "Blob":
        h = ct.c_void_p()
        buf = (ct.c_uint8 * len(data)).from_buffer_copy(data)
        check(lib().uw_blob_deserialize(buf, len(data), ct.byref(h)), "uw_blob_deserialize")
        return Blob(h)

    def to_device(self, sections=DECODE_SECTIONS + ("nib",), device="cuda") -> "DeviceMatrix":
        return DeviceMatrix(self, sections, device)


def compress(w, emit_palette: bool = True, threads: int = 0) -> Blob:
    """uw_compress on a host [rows, cols] array of bf16 bit patterns."""
    a = np.ascontiguousarray(np.asarray(w).view(np.uint16))
    if a.ndim != 2:
        raise ValueError("w must be 2-D [rows, cols]")
    h = ct.c_void_p()
    opts = uw_opts(1 if emit_palette else 0, int(threads))
    check(lib().uw_compress(a.ctypes.data_as(ct.c_void_p), a.shape[0], a.shape[1], ct.byref(opts),
                            ct.byref(h)), "uw_compress")
    return Blob(h)


# ---------------------------------------------------------- device matrices
class DeviceMatrix:
    """A compressed matrix with the chosen sections copied to device memory
    (torch uint8 buffers, 16-byte padded) and its uw_dmat descriptor."""

    requires_grad = False              # as a tensor's

    def __init__(self, blob: Blob, sections, device="cuda"):
        torch = _torch()
        self.info = blob.info()
        self.buffers = {}
        ptrs = (ct.c_void_p * UW_NUM_SECTIONS)()
        for name in sections:
            host = blob.section(name)
            if host.nbytes == 0:
                continue
            raw = host.view(np.uint8)
            pad = (-raw.size) % 16 + 16
            t = torch.zeros(raw.size + pad, dtype=torch.uint8, device=device)
            t[:raw.size].copy_(torch.from_numpy(raw))
            self.buffers[name] = t
            ptrs[SECTION_NAMES.index(name)] = t.data_ptr()
        self.dmat = uw_dmat()
        check(lib().uw_dmat_init(ct.byref(self.dmat), ct.byref(self.info), ptrs), "uw_dmat_init")

    @classmethod
    def from_sections(cls, rows, cols, palette, verbatim_groups, sections) -> "DeviceMatrix":
        """A matrix whose direct-palette sections are on the device already:
        uint8 tensors of the SM, NIB, VEXP, BITMAP and TILE_VBASE bytes, and
        the palette's exponents in index order."""
        torch = _torch()
        rows, cols, verbatim_groups, palette = int(rows), int(cols), int(verbatim_groups), bytes(palette)
        if rows < 0 or cols < 0 or cols % 64 or len(palette) > 16 or not 0 <= verbatim_groups <= rows * cols // 64:
            raise ValueError("bad shape, palette or number of verbatim groups")
        inf = uw_info(rows=rows, cols=cols, groups=rows * cols // 64, verbatim_groups=verbatim_groups,
                      palette_size=len(palette), has_palette=1)
        inf.tiles = (inf.groups + 63) // 64
        inf.palette[:len(palette)] = palette
        need = {"sm": rows * cols, "nib": rows * cols // 2, "vexp": 64 * verbatim_groups, "bitmap": 8 * inf.tiles,
                "tile_vbase": 4 * (inf.tiles + 1)}
        if set(sections) - set(need):
            raise ValueError(f"sections of the direct-palette form are {sorted(need)}")
        ptrs = (ct.c_void_p * UW_NUM_SECTIONS)()
        devices = set()
        for name, n in need.items():
            t = sections.get(name)
            if t is None:
                if n:
                    raise ValueError(f"section {name} is missing")
                continue
            if t.dtype != torch.uint8 or not t.is_contiguous() or not t.is_cuda or t.numel() < n:
                raise ValueError(f"section {name}: a contiguous uint8 device tensor of at least {n} bytes is needed")
            devices.add(t.device)
            inf.section_bytes[SECTION_NAMES.index(name)] = n
            ptrs[SECTION_NAMES.index(name)] = t.data_ptr()
        if len(devices) > 1:
            raise ValueError("the sections are on more than one device")
        dm = cls.__new__(cls)
        dm.info, dm.buffers, dm.dmat = inf, dict(sections), uw_dmat()
        check(lib().uw_dmat_init(ct.byref(dm.dmat), ct.byref(inf), ptrs), "uw_dmat_init")
        return dm

    @property
    def device(self):
        """The device of the sections (None without any)."""
        return next((t.device for t in self.buffers.values()), None)

    @property
    def rows(self):
        return self.info.rows

    @property
    def cols(self):
        return self.info.cols

    def device_bytes(self):
        return sum(int(self.info.section_bytes[SECTION_NAMES.index(n)]) for n in self.buffers)


# ---------------------------------------------------------------- operations
def decode_full(dm: DeviceMatrix, out=None, stream=None):
    torch = _torch()
    if out is None:
        out = torch.empty((dm.rows, dm.cols), dtype=torch.bfloat16, device="cuda")
    check(lib().uw_decode_full(ct.byref(dm.dmat), _ptr(out), _stream(stream)), "uw_decode_full")
    return out


def decode_exponents(dm: DeviceMatrix, out=None, stream=None):
    torch = _torch()
    if out is None:
        out = torch.empty((dm.rows, dm.cols), dtype=torch.uint8, device="cuda")
    check(lib().uw_decode_exponents(ct.byref(dm.dmat), _ptr(out), _stream(stream)), "uw_decode_exponents")
    return out


def transcode_palette(dm: DeviceMatrix, out=None, stream=None):
    torch = _torch()
    if out is None:
        out = torch.empty((dm.rows * dm.cols // 2,), dtype=torch.uint8, device="cuda")
    check(lib().uw_transcode_palette(ct.byref(dm.dmat), _ptr(out), _stream(stream)), "uw_transcode_palette")
    return out


def _y(Y, batch, rows):
    if Y is None:
        Y = _torch().empty((batch, rows), dtype=_torch().float32, device="cuda")
    return Y


def _scratch_args(scratch):
    if scratch is None:
        return ct.c_void_p(0), 0
    return _ptr(scratch), scratch.numel() * scratch.element_size()


def gemm_bf16(W, X, Y=None, kernel=UW_KERNEL_AUTO, split_k=1, scratch=None, stream=None):
    rows, cols = W.shape
    batch = X.shape[0]
    Y = _y(Y, batch, rows)
    sp, sb = _scratch_args(scratch)
    check(lib().uw_gemm_bf16(_ptr(W), rows, cols, _ptr(X), batch, _ptr(Y), kernel, split_k, sp, sb,
                             _stream(stream)), "uw_gemm_bf16")
    return Y


def gemm_recon_exp(dm: DeviceMatrix, e, X, Y=None, kernel=UW_KERNEL_AUTO, split_k=1, scratch=None, stream=None):
    batch = X.shape[0]
    Y = _y(Y, batch, dm.rows)
    sp, sb = _scratch_args(scratch)
    check(lib().uw_gemm_recon_exp(ct.byref(dm.dmat), _ptr(e), _ptr(X), batch, _ptr(Y), kernel, split_k, sp, sb,
                                  _stream(stream)), "uw_gemm_recon_exp")
    return Y


def gemm_recon_pal(dm: DeviceMatrix, nib, X, Y=None, kernel=UW_KERNEL_AUTO, split_k=1, scratch=None,
                   stream=None):
    batch = X.shape[0]
    Y = _y(Y, batch, dm.rows)
    sp, sb = _scratch_args(scratch)
    nibp = _ptr(nib) if nib is not None else ct.c_void_p(dm.dmat.nib)
    check(lib().uw_gemm_recon_pal(ct.byref(dm.dmat), nibp, _ptr(X), batch, _ptr(Y), kernel, split_k, sp, sb,
                                  _stream(stream)), "uw_gemm_recon_pal")
    return Y


def gemm_recon_pal_static(dm: DeviceMatrix, nib, X, Y=None, kernel=UW_KERNEL_AUTO, split_k=0, stream=None):
    """uw_gemm_recon_pal_static: the palette-source matmul with its split-K
    partials in the library's static device array (no caller scratch)."""
    batch = X.shape[0]
    Y = _y(Y, batch, dm.rows)
    nibp = _ptr(nib) if nib is not None else ct.c_void_p(dm.dmat.nib)
    check(lib().uw_gemm_recon_pal_static(ct.byref(dm.dmat), nibp, _ptr(X), batch, _ptr(Y), kernel, split_k,
                                         _stream(stream)), "uw_gemm_recon_pal_static")
    return Y


def scratch_bytes(pipeline, rows, cols, batch, split_k=1) -> int:
    n = lib().uw_scratch_bytes(pipeline, rows, cols, batch, split_k)
    if n < 0:
        check(int(n), "uw_scratch_bytes")
    return int(n)


def alloc_scratch(pipeline, rows, cols, batch, split_k=1):
    n = scratch_bytes(pipeline, rows, cols, batch, split_k)
    return _torch().empty(max(n, 16), dtype=_torch().uint8, device="cuda")


def matmul(dm: DeviceMatrix, X, pipeline=UW_PIPE_AUTO, kernel=UW_KERNEL_AUTO, split_k=1, Y=None, scratch=None,
           stream=None):
    batch = X.shape[0]
    Y = _y(Y, batch, dm.rows)
    sp, sb = _scratch_args(scratch)
    check(lib().uw_matmul(ct.byref(dm.dmat), pipeline, kernel, split_k, _ptr(X), batch, _ptr(Y), sp, sb,
                          _stream(stream)), "uw_matmul")
    return Y


def mlp_gate_up(gate: DeviceMatrix, up: DeviceMatrix, X, h=None, g=None, u=None, stream=None):
    """h = bf16(SiLU(X.gate^T) * (X.up^T)) in one fused launch (direct-palette
    form, batch 1..16, and 17..32 on matrices of at least 48 rows per compute
    unit); g and u (fp32) are also written when given."""
    torch = _torch()
    batch = X.shape[0]
    if h is None:
        h = torch.empty((batch, gate.rows), dtype=torch.bfloat16, device="cuda")
    check(lib().uw_mlp_gate_up(ct.byref(gate.dmat), ct.byref(up.dmat), _ptr(X), batch, _ptr(h),
                               _ptr(g) if g is not None else None, _ptr(u) if u is not None else None,
                               _stream(stream)), "uw_mlp_gate_up")
    return h


def mlp_scratch_bytes(pipeline, rows, cols, batch) -> int:
    n = lib().uw_mlp_scratch_bytes(pipeline, rows, cols, batch)
    if n < 0:
        check(int(n), "uw_mlp_scratch_bytes")
    return int(n)


def mlp_layer(gate: DeviceMatrix, up: DeviceMatrix, down: DeviceMatrix, X, pipeline=UW_PIPE_DIRECT, y=None,
              scratch=None, stream=None, aux_stream=None):
    """y = down . bf16(SiLU(X.gate^T) * (X.up^T)) through one pipeline; with an
    aux_stream the decodes overlap the matmuls (uw_mlp_layer)."""
    torch = _torch()
    batch = X.shape[0]
    if y is None:
        y = torch.empty((batch, down.rows), dtype=torch.float32, device="cuda")
    if scratch is None:
        scratch = torch.empty(max(mlp_scratch_bytes(pipeline, gate.rows, gate.cols, batch), 16), dtype=torch.uint8,
                              device="cuda")
    aux = ct.c_void_p(aux_stream) if aux_stream is not None else None
    check(lib().uw_mlp_layer(ct.byref(gate.dmat), ct.byref(up.dmat), ct.byref(down.dmat), pipeline, _ptr(X), batch,
                             _ptr(y), _ptr(scratch), scratch.numel(), _stream(stream), aux), "uw_mlp_layer")
    return y


def silu_mul_bf16(g, u, h=None, stream=None):
    torch = _torch()
    if h is None:
        h = torch.empty(g.shape, dtype=torch.bfloat16, device="cuda")
    check(lib().uw_silu_mul_bf16(_ptr(g), _ptr(u), g.numel(), _ptr(h), _stream(stream)), "uw_silu_mul_bf16")
    return h


# ------------------------------- matmul with an epilogue, mixture of experts
# A weight is a contiguous bf16 tensor or a DeviceMatrix with the sections of
# the direct-palette form.  Tensors of a call are on one device, which need
# not be the current one; the call runs on that device's current stream, or on
# `stream` (a raw handle), where its outputs are allocated too.  There is no
# backward pass: tensors that require a gradient are refused outside
# torch.no_grad().
class Routing(NamedTuple):
    """What moe_route returns: the experts and weights of every token, and its
    slots grouped by expert (uw_moe_route)."""
    ids: "object"
    weights: "object"
    offsets: "object"
    order: "object"
    place: "object"


def _value_type(t, name):
    torch = _torch()
    if t.dtype == torch.float32:
        return UW_F32
    if t.dtype == torch.bfloat16:
        return UW_BF16
    raise ValueError(f"{name} must be float32 or bfloat16, not {t.dtype}")


def _matrix_arg(t, name, rows=None, cols=None):
    """Row stride of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must be [{'rows' if rows is None else rows}, {'cols' if cols is None else cols}], "
                         f"not {list(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _x_arg(X, cols=None):
    if X.dtype != _torch().bfloat16:
        raise ValueError(f"X must be bfloat16, not {X.dtype}")
    ld = _matrix_arg(X, "X", None, cols)
    return ld if X.shape[0] > 1 else (X.shape[1] + 7) // 8 * 8


def _index_arg(t, name, shape):
    if t.dtype != _torch().int32 or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)}")


def _weight_arg(W, experts, name="W"):
    """(bf16 pointer, descriptor, rows, cols) of one expert's matrix."""
    if isinstance(W, DeviceMatrix):
        n = experts or 1
        if W.rows % n:
            raise ValueError(f"{name}: {W.rows} rows are not {n} experts' matrices")
        return None, ct.byref(W.dmat), W.rows // n, W.cols
    if W.dtype != _torch().bfloat16 or not W.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bfloat16 tensor or a DeviceMatrix")
    if W.dim() != (2 if experts is None else 3) or (experts is not None and W.shape[0] != experts):
        raise ValueError(f"{name} must be " + ("[rows, cols]" if experts is None else f"[{experts}, rows, cols]") +
                         f", not {list(W.shape)}")
    return W.data_ptr(), None, W.shape[-2], W.shape[-1]


def _one_device(first, *others):
    """The device all of them are on (None entries are left out).  None of them
    may ask for a gradient: there is no backward pass."""
    dev = first.device
    if dev.type != "cuda":
        raise ValueError("the tensors must be on a GPU")
    grad = first.requires_grad
    for t in others:
        if t is None:
            continue
        if t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}: a call takes one device")
        grad = grad or t.requires_grad
    if grad and _torch().is_grad_enabled():
        raise ValueError("a tensor requires a gradient and there is no backward pass: call under torch.no_grad()")
    return dev


def _current_stream(dev):
    """Raw handle of the device's current stream (without the Stream object
    that torch.cuda.current_stream makes: 2.7 us a call)."""
    return _torch()._C._cuda_getCurrentRawStream(dev.index)


def _elsewhere(dev, stream):
    """None where the call runs as it stands, else the context that makes
    `dev` and `stream` the current ones."""
    torch = _torch()
    if stream is None:
        return None if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)
    with torch.cuda.device(dev):
        return torch.cuda.stream(torch.cuda.ExternalStream(stream, dev) if stream else torch.cuda.default_stream(dev))


def _new_scratch(need, least, dev):
    """`need` bytes, or where memory has no room for them the `least` that the
    call runs with (None: none)."""
    torch = _torch()
    if need > 0:
        try:
            return torch.empty(need, dtype=torch.uint8, device=dev)
        except torch.cuda.OutOfMemoryError:
            if need == least:
                raise
    return torch.empty(least, dtype=torch.uint8, device=dev) if least else None


def _scratch_arg(scratch):
    """(its pointer, its bytes)"""
    if scratch is None:
        return None, 0
    if not scratch.is_contiguous():
        raise ValueError("scratch must be contiguous")
    return scratch.data_ptr() or None, scratch.numel() * scratch.element_size()


def _new_matrix(rows, cols, dtype, dev):
    """An empty tensor (by its strides: 1.2 us a call against torch.empty's 1.6)."""
    return _torch().empty_strided((rows, cols), (max(cols, 1), 1), dtype=dtype, device=dev)


def _out_arg(out, rows, cols, dtype, dev):
    """(out, row stride, type), allocated where it is None."""
    torch = _torch()
    if out is None:
        dtype = dtype or torch.float32
        out = _new_matrix(rows, cols, dtype, dev)
        return out, max(cols, 1), _value_type(out, "out")
    if dtype is not None and out.dtype != dtype:
        raise ValueError(f"out is {out.dtype}, out_dtype {dtype}")
    return out, _matrix_arg(out, "out", rows, cols), _value_type(out, "out")


def _residual_arg(residual, rows, cols):
    if residual is None:
        return None, UW_F32, 0
    return residual.data_ptr(), _value_type(residual, "residual"), _matrix_arg(residual, "residual", rows, cols)


def linear(W, X, bias=None, act="none", residual=None, out=None, out_dtype=None, scratch=None, stream=None):
    """uw_linear: act(X . W^T + bias) + residual in one matmul.  W [rows, cols],
    X bf16 [batch, cols] (any row stride that is a multiple of 8), bias [rows]
    and residual [batch, rows] fp32 or bf16; `out` (out_dtype, fp32 by default)
    may be the residual itself.  `scratch` (None: allocated where it helps) is a
    tensor of any size: for large batches of compressed weights it holds the
    matrix as bf16 (2 bytes a weight), sums of K-slices for others; an empty one
    saves that memory and is slower."""
    dev = _one_device(X, W, bias, residual, out, scratch)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return linear(W, X, bias, act, residual, out, out_dtype, scratch)
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    w, d, rows, cols = _weight_arg(W, None)
    ldx, batch = _x_arg(X, cols), X.shape[0]
    if bias is not None and (bias.dim() != 1 or bias.shape[0] != rows or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous [{rows}] tensor")
    res, res_type, ldr = _residual_arg(residual, batch, rows)
    out, ldo, out_type = _out_arg(out, batch, rows, out_dtype, dev)
    if scratch is None and batch > 2:                        # never any through 2 rows
        need = lib().uw_linear_scratch_bytes(0 if d is None else 1, rows, cols, batch)
        scratch = _new_scratch(need, 0, dev)
    sp, sb = _scratch_arg(scratch)
    check(lib().uw_linear(w, d, rows, cols, X.data_ptr(), ldx, batch, None if bias is None else bias.data_ptr(),
                          UW_F32 if bias is None else _value_type(bias, "bias"), ACTIVATIONS[act], res, res_type, ldr,
                          out.data_ptr(), out_type, ldo, sp, sb, _current_stream(dev)), "uw_linear")
    return out


def moe_route(logits, top_k, renormalize=True, scratch=None, stream=None) -> Routing:
    """uw_moe_route: the top_k experts of every token (logits [tokens, experts],
    fp32 or bf16), their softmax weights, and the slots grouped by expert."""
    dev = _one_device(logits, scratch)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return moe_route(logits, top_k, renormalize, scratch)
    torch = _torch()
    ld, kind = _matrix_arg(logits, "logits"), _value_type(logits, "logits")
    tokens, experts = logits.shape
    need = lib().uw_moe_route_scratch_bytes(tokens, experts, top_k)
    if need < 0:
        check(int(need), "uw_moe_route")
    if scratch is None and need:
        scratch = torch.empty(need, dtype=torch.uint8, device=dev)
    i32 = torch.int32
    r = Routing(_new_matrix(tokens, top_k, i32, dev), _new_matrix(tokens, top_k, torch.float32, dev),
                torch.empty_strided((experts + 1,), (1,), dtype=i32, device=dev),
                torch.empty_strided((tokens * top_k,), (1,), dtype=i32, device=dev),
                _new_matrix(tokens, top_k, i32, dev))
    sp, sb = _scratch_arg(scratch)
    check(lib().uw_moe_route(logits.data_ptr(), kind, ld, tokens, experts, top_k, 1 if renormalize else 0,
                             r.ids.data_ptr(), r.weights.data_ptr(), r.offsets.data_ptr(), r.order.data_ptr(),
                             r.place.data_ptr(), sp, sb, _current_stream(dev)), "uw_moe_route")
    return r


def _group_args(X, offsets, order):
    """(experts, rows): the groups of a grouped matmul over X."""
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be [experts + 1]")
    _index_arg(offsets, "offsets", (offsets.shape[0],))
    if order is None:
        return offsets.shape[0] - 1, X.shape[0]
    _index_arg(order, "order", (order.numel(),))
    return offsets.shape[0] - 1, order.shape[0]


def _grouped_scratch(scratch, d, pair, experts, rows, cols, n, dev):
    """(the tensor, its pointer, its bytes)"""
    if scratch is None and d is not None and n > 64:         # below, none is taken
        need = lib().uw_grouped_scratch_bytes(1, pair, experts, rows, cols, n)
        if need < 0:
            check(int(need), "uw_grouped_scratch_bytes")
        scratch = _new_scratch(need, 0, dev)
    return (scratch, *_scratch_arg(scratch))


def gemm_grouped(W, X, offsets, order=None, top_k=1, out=None, out_dtype=None, scratch=None,
                 stream=None):
    """uw_gemm_grouped: rows offsets[e] .. offsets[e+1]-1 of the result are
    X's rows (order[s] // top_k where order is given, else s) times expert e's
    matrix.  W [experts, rows, cols] or a DeviceMatrix of experts*rows rows.
    `scratch` (None: allocated where it helps) is a tensor of any size; for
    compressed weights of experts with hundreds of rows it holds every expert's
    matrix as bf16 (2 bytes a weight; the pair of moe_gate_up both matrices), an
    empty one saves that memory and is slower."""
    dev = _one_device(X, W, offsets, order, out, scratch)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return gemm_grouped(W, X, offsets, order, top_k, out, out_dtype, scratch)
    experts, n = _group_args(X, offsets, order)
    w, d, rows, cols = _weight_arg(W, experts)
    ldx = _x_arg(X, cols)
    out, ldo, out_type = _out_arg(out, n, rows, out_dtype, dev)
    scratch, sp, sb = _grouped_scratch(scratch, d, 0, experts, rows, cols, n, dev)
    check(lib().uw_gemm_grouped(w, d, experts, rows, cols, X.data_ptr(), X.shape[0], ldx, offsets.data_ptr(),
                                None if order is None else order.data_ptr(), top_k, n, out.data_ptr(), out_type, ldo,
                                sp, sb, _current_stream(dev)), "uw_gemm_grouped")
    return out


def moe_gate_up(gate, up, X, offsets, order=None, top_k=1, h=None, scratch=None, stream=None):
    """uw_moe_gate_up: h = bf16(SiLU(x . gate_e^T) * (x . up_e^T)), rows,
    inputs and scratch as gemm_grouped's."""
    dev = _one_device(X, gate, up, offsets, order, h, scratch)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return moe_gate_up(gate, up, X, offsets, order, top_k, h, scratch)
    experts, n = _group_args(X, offsets, order)
    gw, gd, rows, cols = _weight_arg(gate, experts, "gate")
    uw_, ud, urows, ucols = _weight_arg(up, experts, "up")
    if (urows, ucols) != (rows, cols):
        raise ValueError("gate and up must have the same shape")
    ldx = _x_arg(X, cols)
    h, ldh, kind = _out_arg(h, n, rows, _torch().bfloat16, dev)
    scratch, sp, sb = _grouped_scratch(scratch, gd, 1, experts, rows, cols, n, dev)
    check(lib().uw_moe_gate_up(gw, gd, uw_, ud, experts, rows, cols, X.data_ptr(), X.shape[0], ldx, offsets.data_ptr(),
                               None if order is None else order.data_ptr(), top_k, n, h.data_ptr(), ldh,
                               sp, sb, _current_stream(dev)), "uw_moe_gate_up")
    return h


def moe_combine(Y, place, weights, residual=None, out=None, out_dtype=None, stream=None):
    """uw_moe_combine: sum_j weights[t, j] * Y[place[t, j]] (+ residual)."""
    dev = _one_device(Y, place, weights, residual, out)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return moe_combine(Y, place, weights, residual, out, out_dtype)
    torch = _torch()
    if Y.dtype != torch.float32 or Y.dim() != 2 or not Y.is_contiguous():
        raise ValueError("Y must be a contiguous float32 [rows, cols] tensor")
    if place.dim() != 2:
        raise ValueError("place must be [tokens, top_k]")
    _index_arg(place, "place", place.shape)
    if weights.dtype != torch.float32 or weights.shape != place.shape or not weights.is_contiguous():
        raise ValueError("weights must be a contiguous float32 tensor of place's shape")
    (tokens, top_k), (n, cols) = place.shape, Y.shape
    res, res_type, ldr = _residual_arg(residual, tokens, cols)
    out, ldo, out_type = _out_arg(out, tokens, cols, out_dtype, dev)
    check(lib().uw_moe_combine(Y.data_ptr(), n, cols, place.data_ptr(), weights.data_ptr(), tokens, top_k, res,
                               res_type, ldr, out.data_ptr(), out_type, ldo, _current_stream(dev)), "uw_moe_combine")
    return out


def moe_scratch_bytes(tokens, experts, top_k, rows, cols, compressed=False) -> int:
    n = lib().uw_moe_scratch_bytes(1 if compressed else 0, tokens, experts, top_k, rows, cols)
    if n < 0:
        check(int(n), "uw_moe_scratch_bytes")
    return int(n)


def moe_layer(gate, up, down, X, logits, top_k, renormalize=True, residual=None, out=None, out_dtype=None,
              scratch=None, stream=None):
    """uw_moe_layer: sum_j w_j down_e(SiLU(gate_e x) * up_e x) over each token's
    top_k experts (+ residual), the experts chosen by `logits`
    [tokens, experts].  gate, up [experts, F, H] and down [experts, H, F], or
    DeviceMatrix of experts*F and experts*H rows; `out` may be X or the
    residual.  h, between up and down, is rounded to bf16.  `scratch` (None:
    allocated) needs moe_scratch_bytes() bytes; with compressed=True, which None
    takes where memory has room, they hold gate and up of all experts as bf16
    (2 bytes a weight each) for prompts."""
    dev = _one_device(X, gate, up, down, logits, residual, out, scratch)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return moe_layer(gate, up, down, X, logits, top_k, renormalize, residual, out, out_dtype, scratch)
    tokens, experts = X.shape[0], logits.shape[-1]
    ldl, kind = _matrix_arg(logits, "logits", tokens), _value_type(logits, "logits")
    gw, gd, F, H = _weight_arg(gate, experts, "gate")
    uw_, ud, urows, ucols = _weight_arg(up, experts, "up")
    dw, dd, drows, dcols = _weight_arg(down, experts, "down")
    if (urows, ucols) != (F, H) or (drows, dcols) != (H, F):
        raise ValueError("gate and up must be [experts, F, H] and down [experts, H, F]")
    ldx = _x_arg(X, H)
    res, res_type, ldr = _residual_arg(residual, tokens, H)
    out, ldo, out_type = _out_arg(out, tokens, H, out_dtype, dev)
    if scratch is None:
        least = moe_scratch_bytes(tokens, experts, top_k, F, H)
        need = moe_scratch_bytes(tokens, experts, top_k, F, H, True) if gd or dd else least
        scratch = _new_scratch(need, least, dev)
    sp, sb = _scratch_arg(scratch)
    check(lib().uw_moe_layer(gw, gd, uw_, ud, dw, dd, experts, F, H, X.data_ptr(), ldx, tokens, logits.data_ptr(), kind,
                             ldl, top_k, 1 if renormalize else 0, res, res_type, ldr, out.data_ptr(), out_type, ldo,
                             sp, sb, _current_stream(dev)), "uw_moe_layer")
    return out


class KernelTimer:
    """Context manager: durations (ms) of the matmul kernels launched inside it,
    recorded by the launches themselves (uw_kernel_timer_*)."""

    def __init__(self, capacity=4096):
        self.capacity = capacity
        self.ms = []

    def __enter__(self):
        check(lib().uw_kernel_timer_enable(self.capacity), "uw_kernel_timer_enable")
        return self

    def __exit__(self, *exc):
        lib().uw_kernel_timer_disable()
        n = ct.c_int()
        buf = (ct.c_float * self.capacity)()
        check(lib().uw_kernel_timer_read(buf, self.capacity, ct.byref(n)), "uw_kernel_timer_read")
        self.ms = [buf[i] for i in range(min(n.value, self.capacity))]
        return False


def plan_set(rows, cols, batch, pipeline, kernel=UW_KERNEL_AUTO, split_k=1):
    check(lib().uw_plan_set(rows, cols, batch, pipeline, kernel, split_k), "uw_plan_set")


def plan_lookup(rows, cols, batch):
    p, k, s = ct.c_int(), ct.c_int(), ct.c_int()
    rc = lib().uw_plan_lookup(rows, cols, batch, ct.byref(p), ct.byref(k), ct.byref(s))
    return (p.value, k.value, s.value) if rc == 0 else None


def plan_clear():
    check(lib().uw_plan_clear(), "uw_plan_clear")


def plan_count() -> int:
    return int(lib().uw_plan_count())


def plan_save(path):
    check(lib().uw_plan_save(str(path).encode()), "uw_plan_save")


def plan_load(path):
    check(lib().uw_plan_load(str(path).encode()), "uw_plan_load")
