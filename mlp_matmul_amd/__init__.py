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
    UW_FORM_BF16, UW_FORM_COMPRESSED, UW_FORM_MX4, UW_SCORE_SIGMOID, UW_SCORE_SOFTMAX,
    UnweightError, check, lib,
    uw_dmat, uw_info, uw_mx4,
    uw_opts,
)

PIPELINES = {"full": UW_PIPE_FULL, "exp": UW_PIPE_EXP, "pal": UW_PIPE_PAL, "direct": UW_PIPE_DIRECT}
ACTIVATIONS = {"none": UW_ACT_NONE, "relu": UW_ACT_RELU, "silu": UW_ACT_SILU, "gelu": UW_ACT_GELU,
               "gelu_tanh": UW_ACT_GELU_TANH}
SCORES = {"sigmoid": UW_SCORE_SIGMOID, "softmax": UW_SCORE_SOFTMAX}
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


class Mx4Matrix:
    """A matrix of microscaled 4-bit numbers on the device (uw_mx4): codes uint8
    [rows, cols/2] and scales uint8 [rows, cols/32], the rows of each contiguous
    and a multiple of 16 bytes apart.  The matrices of a layer's experts are one
    matrix of experts*rows rows.  The tensors are kept, not copied; their addresses are
    taken once, so they are not to be resized or moved.  Scales of other rows, as of
    1408 columns, go into such ones first: with n = scales.shape[1],
    torch.nn.functional.pad(scales, (0, -n % 16))[:, :n]."""

    requires_grad = False              # as a tensor's

    def __init__(self, codes, scales):
        torch = _torch()
        for t, name in ((codes, "codes"), (scales, "scales")):
            if t.dtype != torch.uint8 or t.dim() != 2:
                raise ValueError(f"{name} must be a 2-D uint8 tensor")
            if t.shape[1] > 1 and t.stride(1) != 1:
                raise ValueError(f"the rows of {name} must be contiguous")
            if t.shape[0] > 1 and t.stride(0) % 16 or t.data_ptr() % 16:
                raise ValueError(f"the rows of {name} must lie at multiples of 16 bytes")
        if scales.shape[0] != codes.shape[0] or codes.shape[1] != 16 * scales.shape[1]:
            raise ValueError(f"codes [rows, cols/2] and scales [rows, cols/32] do not match: {list(codes.shape)}, "
                             f"{list(scales.shape)}")
        if codes.device != scales.device:
            raise ValueError(f"codes on {codes.device} and scales on {scales.device}")

        def stride(t):
            return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 15) // 16 * 16

        self._hold(codes, scales, codes.device, codes.shape[0], codes.shape[1] * 2, stride(codes), stride(scales))

    def _hold(self, codes, scales, dev, rows, cols, ldc, lds):
        self.codes, self.scales, self.device, self.rows, self.cols, self.shape = codes, scales, dev, rows, cols, (rows, cols)
        self.mx4 = uw_mx4(rows, cols, codes.data_ptr(), scales.data_ptr(), ldc, lds)

    @classmethod
    def _empty(cls, rows, cols, dev):
        """A new one, without __init__'s checks: a call of mx4_quantize takes 8.1 us on the host, 10.3 with them.  Rows
        of codes longer than 1 KB start at multiples of 128 bytes, the lines that the products load: 14336 x 4000
        with 4096 rows on 128x128 tiles takes 170 us so, 197 with rows of 2000 bytes."""
        u8, half, blocks, room = _torch().uint8, cols // 2, cols // 32, (cols // 32 + 15) // 16 * 16
        ldc = (half + 127) // 128 * 128 if half > 1024 else half
        empty, m = _torch().empty_strided, cls.__new__(cls)
        m._hold(empty((rows, half), (ldc, 1), dtype=u8, device=dev), empty((rows, blocks), (room, 1), dtype=u8, device=dev),
                dev, rows, cols, ldc, room)
        return m

    def device_bytes(self):
        return self.codes.numel() + self.scales.numel()


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
# A weight is a contiguous bf16 tensor, a DeviceMatrix with the sections of the
# direct-palette form, or an Mx4Matrix, whose products take an Mx4Matrix of the
# same format as X too.  Tensors of a call are on one device, which need
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
    kind = getattr(t, "dtype", None)                         # a compressed or 4-bit matrix has none
    if kind == torch.float32:
        return UW_F32
    if kind == torch.bfloat16:
        return UW_BF16
    raise ValueError(f"{name} must be float32 or bfloat16, not {kind or type(t).__name__}")


def _matrix_arg(t, name, rows=None, cols=None):
    """Row stride of a 2-D tensor whose rows are contiguous (its type is checked before: no other matrix comes here)."""
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must be [{'rows' if rows is None else rows}, {'cols' if cols is None else cols}], "
                         f"not {list(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _x_arg(X, cols=None):
    if getattr(X, "dtype", None) != _torch().bfloat16:
        if isinstance(X, Mx4Matrix):
            raise ValueError("X must be bfloat16: only products with Mx4Matrix weights, but moe_experts, take it as an Mx4Matrix")
        raise ValueError(f"X must be bfloat16, not {getattr(X, 'dtype', type(X).__name__)}")
    ld = _matrix_arg(X, "X", None, cols)
    return ld if X.shape[0] > 1 else (X.shape[1] + 7) // 8 * 8


def _mx4_rows(X, cols):
    """(bf16 pointer, row stride, descriptor, rows) of what 4-bit weights are multiplied with."""
    if isinstance(X, Mx4Matrix):
        if X.cols != cols:
            raise ValueError(f"X must be [rows, {cols}], not {list(X.shape)}")
        return None, 0, ct.byref(X.mx4), X.rows
    ld = _x_arg(X, cols)
    return X.data_ptr(), ld, None, X.shape[0]


def _mx4_weight(W, experts, name="W"):
    """Rows of one expert's matrix."""
    if not isinstance(W, Mx4Matrix):
        raise ValueError(f"{name} must be an Mx4Matrix as the other weights are")
    if W.rows % experts:
        raise ValueError(f"{name}: {W.rows} rows are not {experts} experts' matrices")
    return W.rows // experts


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
    if getattr(W, "dtype", None) != _torch().bfloat16 or not W.is_contiguous():
        if isinstance(W, Mx4Matrix):
            raise ValueError(f"{name} is an Mx4Matrix and the other weights are not")
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
    kind = _value_type(out, "out")
    if dtype is not None and out.dtype != dtype:
        raise ValueError(f"out is {out.dtype}, out_dtype {dtype}")
    return out, _matrix_arg(out, "out", rows, cols), kind


def _residual_arg(residual, rows, cols):
    if residual is None:
        return None, UW_F32, 0
    kind = _value_type(residual, "residual")
    return residual.data_ptr(), kind, _matrix_arg(residual, "residual", rows, cols)


def linear(W, X, bias=None, act="none", residual=None, out=None, out_dtype=None, scratch=None, stream=None):
    """uw_linear: act(X . W^T + bias) + residual in one matmul.  W [rows, cols],
    X bf16 [batch, cols] (any row stride that is a multiple of 8), bias [rows]
    and residual [batch, rows] fp32 or bf16; `out` (out_dtype, fp32 by default)
    may be the residual itself.  `scratch` (None: allocated where it helps) is a
    tensor of any size: for large batches of compressed weights it holds the
    matrix as bf16 (2 bytes a weight), sums of K-slices for others; an empty one
    saves that memory and is slower.  With an Mx4Matrix W (uw_mx4_linear) X may be
    one too, and no scratch is taken."""
    dev = _one_device(X, W, bias, residual, out, scratch)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return linear(W, X, bias, act, residual, out, out_dtype, scratch)
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    mx4 = isinstance(W, Mx4Matrix)
    if mx4:
        rows, cols = W.rows, W.cols
        xp, ldx, x4, batch = _mx4_rows(X, cols)
    else:
        w, d, rows, cols = _weight_arg(W, None)
        ldx, batch = _x_arg(X, cols), X.shape[0]
    bias_type = UW_F32 if bias is None else _value_type(bias, "bias")
    if bias is not None and (bias.dim() != 1 or bias.shape[0] != rows or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous [{rows}] tensor")
    res, res_type, ldr = _residual_arg(residual, batch, rows)
    out, ldo, out_type = _out_arg(out, batch, rows, out_dtype, dev)
    if mx4:
        check(lib().uw_mx4_linear(ct.byref(W.mx4), xp, ldx, x4, batch, None if bias is None else bias.data_ptr(),
                                  bias_type, ACTIVATIONS[act], res, res_type, ldr, out.data_ptr(), out_type, ldo,
                                  _current_stream(dev)), "uw_mx4_linear")
        return out
    if scratch is None and batch > 2:                        # never any through 2 rows
        need = lib().uw_linear_scratch_bytes(0 if d is None else 1, rows, cols, batch)
        scratch = _new_scratch(need, 0, dev)
    sp, sb = _scratch_arg(scratch)
    check(lib().uw_linear(w, d, rows, cols, X.data_ptr(), ldx, batch, None if bias is None else bias.data_ptr(),
                          bias_type, ACTIVATIONS[act], res, res_type, ldr,
                          out.data_ptr(), out_type, ldo, sp, sb, _current_stream(dev)), "uw_linear")
    return out


def _routing(tokens, experts, top_k, scratch, dev):
    """(a Routing's tensors, the scratch that a routing call needs)"""
    torch = _torch()
    need = lib().uw_moe_route_scratch_bytes(tokens, experts, top_k)
    if need < 0:
        check(int(need), "uw_moe_route")
    if scratch is None and need:
        scratch = torch.empty(need, dtype=torch.uint8, device=dev)
    i32 = torch.int32
    return Routing(_new_matrix(tokens, top_k, i32, dev), _new_matrix(tokens, top_k, torch.float32, dev),
                   torch.empty_strided((experts + 1,), (1,), dtype=i32, device=dev),
                   torch.empty_strided((tokens * top_k,), (1,), dtype=i32, device=dev),
                   _new_matrix(tokens, top_k, i32, dev)), scratch


def moe_route(logits, top_k, renormalize=True, scratch=None, stream=None) -> Routing:
    """uw_moe_route: the top_k experts of every token (logits [tokens, experts],
    fp32 or bf16), their softmax weights, and the slots grouped by expert."""
    dev = _one_device(logits, scratch)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return moe_route(logits, top_k, renormalize, scratch)
    kind, ld = _value_type(logits, "logits"), _matrix_arg(logits, "logits")
    tokens, experts = logits.shape
    r, scratch = _routing(tokens, experts, top_k, scratch, dev)
    sp, sb = _scratch_arg(scratch)
    check(lib().uw_moe_route(logits.data_ptr(), kind, ld, tokens, experts, top_k, 1 if renormalize else 0,
                             r.ids.data_ptr(), r.weights.data_ptr(), r.offsets.data_ptr(), r.order.data_ptr(),
                             r.place.data_ptr(), sp, sb, _current_stream(dev)), "uw_moe_route")
    return r


def moe_route_scored(logits, top_k, score="sigmoid", bias=None, groups=1, top_groups=1, group_top=2, renormalize=True,
                     scale=1.0, scratch=None, stream=None) -> Routing:
    """uw_moe_route_scored: the top_k experts of every token by their scores
    ("sigmoid" or "softmax" of logits [tokens, experts], fp32 or bf16) plus
    `bias` (fp32 [experts], for the choice alone), among the experts of the
    top_groups of `groups` groups of neighbours with the largest sums of their
    group_top best; the weights are the chosen scores, renormalised and scaled.
    The Routing is moe_route's."""
    dev = _one_device(logits, bias, scratch)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return moe_route_scored(logits, top_k, score, bias, groups, top_groups, group_top, renormalize, scale, scratch)
    torch = _torch()
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}")
    kind, ld = _value_type(logits, "logits"), _matrix_arg(logits, "logits")
    tokens, experts = logits.shape
    if bias is not None and (getattr(bias, "dtype", None) != torch.float32 or tuple(bias.shape) != (experts,) or
                             not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous float32 [{experts}] tensor")
    r, scratch = _routing(tokens, experts, top_k, scratch, dev)
    sp, sb = _scratch_arg(scratch)
    check(lib().uw_moe_route_scored(logits.data_ptr(), kind, ld, tokens, experts, top_k, SCORES[score],
                                    None if bias is None else bias.data_ptr(), groups, top_groups, group_top,
                                    1 if renormalize else 0, scale, r.ids.data_ptr(), r.weights.data_ptr(),
                                    r.offsets.data_ptr(), r.order.data_ptr(), r.place.data_ptr(), sp, sb,
                                    _current_stream(dev)), "uw_moe_route_scored")
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
    empty one saves that memory and is slower.  With an Mx4Matrix W
    (uw_mx4_gemm_grouped) X may be one too, and no scratch is taken."""
    dev = _one_device(X, W, offsets, order, out, scratch)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return gemm_grouped(W, X, offsets, order, top_k, out, out_dtype, scratch)
    experts, n = _group_args(X, offsets, order)
    if isinstance(W, Mx4Matrix):
        rows = _mx4_weight(W, experts)
        xp, ldx, x4, x_rows = _mx4_rows(X, W.cols)
        out, ldo, out_type = _out_arg(out, n, rows, out_dtype, dev)
        check(lib().uw_mx4_gemm_grouped(ct.byref(W.mx4), experts, xp, x_rows, ldx, x4, offsets.data_ptr(),
                                        None if order is None else order.data_ptr(), top_k, n, out.data_ptr(), out_type,
                                        ldo, _current_stream(dev)), "uw_mx4_gemm_grouped")
        return out
    w, d, rows, cols = _weight_arg(W, experts)
    ldx = _x_arg(X, cols)
    out, ldo, out_type = _out_arg(out, n, rows, out_dtype, dev)
    scratch, sp, sb = _grouped_scratch(scratch, d, 0, experts, rows, cols, n, dev)
    check(lib().uw_gemm_grouped(w, d, experts, rows, cols, X.data_ptr(), X.shape[0], ldx, offsets.data_ptr(),
                                None if order is None else order.data_ptr(), top_k, n, out.data_ptr(), out_type, ldo,
                                sp, sb, _current_stream(dev)), "uw_gemm_grouped")
    return out


def moe_gate_up(gate, up, X, offsets, order=None, top_k=1, h=None, scratch=None, stream=None):
    """uw_moe_gate_up (uw_mx4_gate_up): h = bf16(SiLU(x . gate_e^T) * (x . up_e^T)),
    rows, inputs and scratch as gemm_grouped's."""
    dev = _one_device(X, gate, up, offsets, order, h, scratch)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return moe_gate_up(gate, up, X, offsets, order, top_k, h, scratch)
    experts, n = _group_args(X, offsets, order)
    if isinstance(gate, Mx4Matrix):
        rows = _mx4_weight(gate, experts, "gate")
        _mx4_weight(up, experts, "up")
        if up.shape != gate.shape:
            raise ValueError("gate and up must have the same shape")
        xp, ldx, x4, x_rows = _mx4_rows(X, gate.cols)
        h, ldh, kind = _out_arg(h, n, rows, _torch().bfloat16, dev)
        check(lib().uw_mx4_gate_up(ct.byref(gate.mx4), ct.byref(up.mx4), experts, xp, x_rows, ldx, x4,
                                   offsets.data_ptr(), None if order is None else order.data_ptr(), top_k, n,
                                   h.data_ptr(), ldh, _current_stream(dev)), "uw_mx4_gate_up")
        return h
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
    if getattr(Y, "dtype", None) != torch.float32 or Y.dim() != 2 or not Y.is_contiguous():
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
    if isinstance(gate, Mx4Matrix):
        raise ValueError("moe_layer takes no Mx4Matrix: moe_route and moe_experts do its work with them")
    tokens, experts = X.shape[0], logits.shape[-1]
    kind, ldl = _value_type(logits, "logits"), _matrix_arg(logits, "logits", tokens)
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


def moe_experts_scratch_bytes(form, tokens, experts, top_k, rows, cols) -> int:
    n = lib().uw_moe_experts_scratch_bytes(form, tokens, experts, top_k, rows, cols)
    if n < 0:
        check(int(n), "uw_moe_experts_scratch_bytes")
    return int(n)


def moe_experts(gate, up, down, X, routing, residual=None, out=None, out_dtype=None, scratch=None, stream=None):
    """uw_moe_experts: moe_layer's sum over each token's experts (+ residual) on
    a Routing that moe_route or moe_route_scored returned.  gate, up and down as
    moe_layer's, or all three Mx4Matrix of experts*F, experts*F and experts*H
    rows; `out` may be X or the residual.  h, between up and down, is rounded to
    bf16.  `scratch` (None: allocated) needs moe_experts_scratch_bytes() bytes; for
    DeviceMatrix weights those of UW_FORM_BF16 do too, and prompts are slower."""
    ids, weights, offsets, order, place = routing
    dev = _one_device(X, gate, up, down, weights, offsets, order, place, residual, out, scratch)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return moe_experts(gate, up, down, X, routing, residual, out, out_dtype, scratch)
    if place.dim() != 2 or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("place must be [tokens, top_k] and offsets [experts + 1]")
    (tokens, top_k), experts = place.shape, offsets.shape[0] - 1
    _index_arg(place, "place", (X.shape[0], top_k))
    _index_arg(order, "order", (tokens * top_k,))
    _index_arg(offsets, "offsets", (experts + 1,))
    if weights.dtype != _torch().float32 or weights.shape != place.shape or not weights.is_contiguous():
        raise ValueError("weights must be a contiguous float32 tensor of place's shape")
    least_form = UW_FORM_BF16
    if isinstance(gate, Mx4Matrix):
        form = least_form = UW_FORM_MX4
        F, H = _mx4_weight(gate, experts, "gate"), gate.cols
        shapes = (_mx4_weight(up, experts, "up"), up.cols), (_mx4_weight(down, experts, "down"), down.cols)
        ws = [ct.byref(m.mx4) for m in (gate, up, down)]
    else:
        parts = [_weight_arg(m, experts, name) for m, name in ((gate, "gate"), (up, "up"), (down, "down"))]
        form = UW_FORM_BF16 if parts[0][1] is None else UW_FORM_COMPRESSED
        if any((p[1] is None) != (parts[0][1] is None) for p in parts):
            raise ValueError("gate, up and down must be of one form")
        F, H = parts[0][2:]
        shapes = parts[1][2:], parts[2][2:]
        ws = [p[0] if p[1] is None else p[1] for p in parts]
    if shapes != ((F, H), (H, F)):
        raise ValueError("gate and up must be [experts, F, H] and down [experts, H, F]")
    ldx = _x_arg(X, H)
    res, res_type, ldr = _residual_arg(residual, tokens, H)
    out, ldo, out_type = _out_arg(out, tokens, H, out_dtype, dev)
    if scratch is None:
        need = moe_experts_scratch_bytes(form, tokens, experts, top_k, F, H)
        least = need if form == least_form else moe_experts_scratch_bytes(least_form, tokens, experts, top_k, F, H)
        scratch = _new_scratch(need, least, dev)
    sp, sb = _scratch_arg(scratch)
    check(lib().uw_moe_experts(form, *ws, experts, F, H, X.data_ptr(), ldx, tokens, top_k, weights.data_ptr(),
                               offsets.data_ptr(), order.data_ptr(), place.data_ptr(), res, res_type, ldr,
                               out.data_ptr(), out_type, ldo, sp, sb, _current_stream(dev)), "uw_moe_experts")
    return out


# ------------------------------------------------- microscaled 4-bit numbers
def mx4_quantize(X, out=None, stream=None) -> Mx4Matrix:
    """uw_mx4_quantize: X [rows, cols] (bf16 or fp32, cols a multiple of 32) as
    microscaled 4-bit numbers, in a new Mx4Matrix or in `out`.  The rows of a new
    one may lie further apart than their bytes."""
    dev = _one_device(X, out)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return mx4_quantize(X, out)
    kind, ld = _value_type(X, "X"), _matrix_arg(X, "X")
    rows, cols = X.shape
    if cols % 32:
        raise ValueError(f"X must have a multiple of 32 columns, not {cols}")
    if out is None:
        out = Mx4Matrix._empty(rows, cols, dev)
    elif not isinstance(out, Mx4Matrix):
        raise ValueError(f"out must be an Mx4Matrix, not {type(out).__name__}")
    elif out.shape != (rows, cols):
        raise ValueError(f"out must be [{rows}, {cols}], not {list(out.shape)}")
    m = out.mx4
    check(lib().uw_mx4_quantize(X.data_ptr(), kind, ld, rows, cols, m.codes, m.ldc, m.scales, m.lds,
                                _current_stream(dev)), "uw_mx4_quantize")
    return out


def mx4_dequantize(M: Mx4Matrix, out=None, out_dtype=None, stream=None):
    """uw_mx4_dequantize: the numbers of M, fp32 by default or bf16."""
    dev = _one_device(M, out)
    ctx = _elsewhere(dev, stream)
    if ctx is not None:
        with ctx:
            return mx4_dequantize(M, out, out_dtype)
    if not isinstance(M, Mx4Matrix):
        raise ValueError("M must be an Mx4Matrix")
    out, ldo, kind = _out_arg(out, M.rows, M.cols, out_dtype, dev)
    check(lib().uw_mx4_dequantize(ct.byref(M.mx4), out.data_ptr(), kind, ldo, _current_stream(dev)), "uw_mx4_dequantize")
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
