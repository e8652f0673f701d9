"""Python binding of the C ABI, with the same names.

Tensors are PyTorch CUDA tensors (device memory and streams only); each call
hands raw pointers and the current stream to libattnmask.  The binding does
no arithmetic of the method.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _native

ATTN_OK = 0
(ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_WORKSPACE_TOO_SMALL, ATTN_ERR_MASK_MISMATCH,
 ATTN_ERR_CUDA, ATTN_ERR_DEVICE_TIMEOUT, ATTN_ERR_DEVICE_INVALID_INPUT) = range(1, 8)
STATUS = {
    0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED",
    3: "ATTN_ERR_WORKSPACE_TOO_SMALL", 4: "ATTN_ERR_MASK_MISMATCH", 5: "ATTN_ERR_CUDA",
    6: "ATTN_ERR_DEVICE_TIMEOUT", 7: "ATTN_ERR_DEVICE_INVALID_INPUT",
}
MASK_KINDS = {"causal": 0, "causal_document": 1, "shared_prefix": 2, "strip_thinking": 3,
              "strip_thinking_dup": 4, "none": 5, "dense": 6}
DTYPES = {torch.bfloat16: 0, torch.float32: 1}
TILE_EMPTY, TILE_PARTIAL, TILE_FULL = 0, 1, 2
BLOCK_M = BLOCK_N = 128


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {STATUS.get(status, status)} ({attn_status_string(status)})"
        if status == 5:
            msg += f": {attn_last_error_message()}"
        super().__init__(msg)


def _check(status: int, where: str) -> None:
    if status != ATTN_OK:
        raise AttnError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, name: str, where: str, dtypes=None, shape=None, device=None) -> None:
    """Refuse, before any library call, a tensor the C side would misread: not
    on a CUDA device (a host pointer would reach a kernel), on another device
    than the rest, not contiguous (the layouts are dense row-major), of the
    wrong element type or shape."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise AttnError(1, f"{where}: {name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise AttnError(1, f"{where}: {name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise AttnError(1, f"{where}: {name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise AttnError(1, f"{where}: {name} has dtype {t.dtype}, expected one of {dtypes}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise AttnError(1, f"{where}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _need_meta(where, cu_seqlens, seg_id, role, turn, dense_bits, dense_offsets, device=None):
    """cu_seqlens int32; seg_id / turn int32, role int8 (one value per token);
    the dense kind's words (32-bit) and int64 offsets."""
    _need(cu_seqlens, "cu_seqlens", where, (torch.int32,), device=device)
    dev = cu_seqlens.device
    _need(seg_id, "seg_id", where, (torch.int32,), device=dev)
    _need(role, "role", where, (torch.int8, torch.uint8), device=dev)
    _need(turn, "turn", where, (torch.int32,), device=dev)
    _need(dense_bits, "dense_bits", where, _WORD_DTYPES, device=dev)
    _need(dense_offsets, "dense_offsets", where, (torch.int64,), device=dev)


_WORD_DTYPES = (torch.int32,) + ((torch.uint32,) if hasattr(torch, "uint32") else ())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _kind(kind) -> int:
    return MASK_KINDS[kind] if isinstance(kind, str) else int(kind)


def attn_status_string(status: int) -> str:
    return _native.lib().attn_status_string(int(status)).decode()


def attn_last_error_message() -> str:
    return _native.lib().attn_last_error_message().decode()


def attn_version() -> int:
    return int(_native.lib().attn_version())


def attn_block_mask_workspace_size(batch: int, total_tokens: int, max_seqlen: int,
                                   block_m: int = BLOCK_M, block_n: int = BLOCK_N) -> int:
    out = ctypes.c_size_t(0)
    _check(_native.lib().attn_block_mask_workspace_size(batch, total_tokens, max_seqlen, block_m,
                                                        block_n, ctypes.byref(out)),
           "attn_block_mask_workspace_size")
    return int(out.value)


class BlockMask:
    """A built block mask: the C struct plus the tensors it points into."""

    # arrays attn_block_mask_build_noalloc keeps in its own scratch and does not
    # write to the workspace
    NOALLOC_UNWRITTEN = ("labels", "qt_off", "pair_off")

    def __init__(self, struct: _native.AttnBlockMask, workspace: torch.Tensor, keep: tuple,
                 noalloc: bool = False):
        self.struct = struct
        self.workspace = workspace
        self._keep = keep  # metadata tensors must outlive the mask
        self.noalloc = noalloc

    # -- read-back helpers (copy device arrays to the host; synchronising) --
    def _array(self, off: int, count: int, dtype) -> torch.Tensor:
        nbytes = count * torch.empty((), dtype=dtype).element_size()
        raw = self.workspace[off: off + nbytes]
        return raw.view(dtype).cpu()

    def header(self) -> torch.Tensor:
        return self._array(self.struct.off_header, 16, torch.int32)

    @property
    def n_qtiles(self) -> int:
        return int(self.header()[0])

    def lists(self) -> dict:
        """Device arrays copied back: q-tile descriptors, labels, CSR lists, order.
        A mask from the no-allocation builder has no ``labels``, ``qt_off`` or
        ``pair_off`` (never written to its workspace); they are left out."""
        s = self.struct
        n = self.n_qtiles
        hdr = self.header()
        nent = int(hdr[1])
        koff = self._array(s.off_koff, n + 1, torch.int32)
        out = {
            "header": hdr,
            "qt_seq": self._array(s.off_qt_seq, n, torch.int32),
            "qt_idx": self._array(s.off_qt_idx, n, torch.int32),
            "labels": self._array(s.off_labels, s.max_qtiles * s.max_ktiles, torch.uint8)
                          .view(s.max_qtiles, s.max_ktiles)[:n],
            "kcount": self._array(s.off_kcount, n, torch.int32),
            "koff": koff,
            "kidx": self._array(s.off_kidx, nent, torch.int32),
            "klabel": self._array(s.off_klabel, nent, torch.uint8),
            "order": self._array(s.off_order, n, torch.int32),
            "qt_off": self._array(s.off_qt_off, s.batch + 1, torch.int32),
            "pair_off": self._array(s.off_pair_off, s.batch + 1, torch.int32),
            "pair_q0": self._array(s.off_pair_q0, int(hdr[3]), torch.int32),
            "pair_order": self._array(s.off_pair_order, int(hdr[3]), torch.int32),
            "qcount": self._array(s.off_qcount, n, torch.int32),
            "qoff": self._array(s.off_qoff, n + 1, torch.int32),
            "qidx": self._array(s.off_qidx, nent, torch.int32),
            "qlabel": self._array(s.off_qlabel, nent, torch.uint8),
            "korder": self._array(s.off_korder, n, torch.int32),
        }
        if self.noalloc:
            for name in self.NOALLOC_UNWRITTEN:
                del out[name]
        return out


def _params(role_think: int, dense_bits, dense_offsets) -> "_native.AttnMaskParams":
    return _native.AttnMaskParams(role_think, _ptr(dense_bits), _ptr(dense_offsets))


def attn_block_mask_build(kind, cu_seqlens: torch.Tensor, total_tokens: int, max_seqlen: int,
                          seg_id: Optional[torch.Tensor] = None, role: Optional[torch.Tensor] = None,
                          turn: Optional[torch.Tensor] = None, role_think: int = 1,
                          workspace: Optional[torch.Tensor] = None, stream=None,
                          dense_bits: Optional[torch.Tensor] = None,
                          dense_offsets: Optional[torch.Tensor] = None) -> BlockMask:
    """Build the block mask on the device (asynchronous on ``stream``)."""
    _need_meta("attn_block_mask_build", cu_seqlens, seg_id, role, turn, dense_bits, dense_offsets)
    _need(workspace, "workspace", "attn_block_mask_build", device=cu_seqlens.device)
    batch = cu_seqlens.numel() - 1
    need = attn_block_mask_workspace_size(batch, total_tokens, max_seqlen)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=cu_seqlens.device)
    params = _params(role_think, dense_bits, dense_offsets)
    out = _native.AttnBlockMask()
    _check(_native.lib().attn_block_mask_build(
        _kind(kind), ctypes.byref(params), _ptr(cu_seqlens), batch, total_tokens, max_seqlen,
        _ptr(seg_id), _ptr(role), _ptr(turn), BLOCK_M, BLOCK_N, _ptr(workspace),
        workspace.numel() * workspace.element_size(), ctypes.byref(out), _stream(stream)),
        "attn_block_mask_build")
    return BlockMask(out, workspace, (cu_seqlens, seg_id, role, turn, dense_bits, dense_offsets))


def attn_block_mask_build_noalloc(kind, cu_seqlens: torch.Tensor, total_tokens: int,
                                  max_seqlen: int, workspace: torch.Tensor,
                                  seg_id: Optional[torch.Tensor] = None,
                                  role: Optional[torch.Tensor] = None,
                                  turn: Optional[torch.Tensor] = None, role_think: int = 1,
                                  stream=None, dense_bits: Optional[torch.Tensor] = None,
                                  dense_offsets: Optional[torch.Tensor] = None) -> BlockMask:
    """Block-mask build that allocates nothing, for callers that cannot.

    The caller passes the output buffer ``workspace`` (at least
    ``attn_block_mask_workspace_size`` bytes); the builder's temporaries use a
    fixed 4 MiB array inside the library, shared by every call on the device,
    so calls must not overlap on the GPU.  The first call on a device does a
    one-time address lookup and should come before any stream capture.  Only
    the arrays the forward and backward read are stored (``labels``, ``qt_off``
    and ``pair_off`` are not).  The scratch serves up to 259,968 tokens in
    one sequence (2031 tiles); larger problems are refused.
    """
    _need_meta("attn_block_mask_build_noalloc", cu_seqlens, seg_id, role, turn, dense_bits,
               dense_offsets)
    _need(workspace, "workspace", "attn_block_mask_build_noalloc", device=cu_seqlens.device)
    batch = cu_seqlens.numel() - 1
    params = _params(role_think, dense_bits, dense_offsets)
    out = _native.AttnBlockMask()
    _check(_native.lib().attn_block_mask_build_noalloc(
        _kind(kind), ctypes.byref(params), _ptr(cu_seqlens), batch, total_tokens, max_seqlen,
        _ptr(seg_id), _ptr(role), _ptr(turn), BLOCK_M, BLOCK_N, _ptr(workspace),
        workspace.numel() * workspace.element_size(), ctypes.byref(out), _stream(stream)),
        "attn_block_mask_build_noalloc")
    return BlockMask(out, workspace, (cu_seqlens, seg_id, role, turn, dense_bits, dense_offsets),
                     noalloc=True)


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, bm: BlockMask, kind,
             cu_seqlens: torch.Tensor, max_seqlen: int, seg_id=None, role=None, turn=None,
             role_think: int = 1, scale: float = 0.0, out: Optional[torch.Tensor] = None,
             lse: Optional[torch.Tensor] = None, stream=None,
             dense_bits: Optional[torch.Tensor] = None, dense_offsets: Optional[torch.Tensor] = None):
    """Masked attention forward; returns (O [T, H, D], LSE [H, T] fp32)."""
    where = "attn_fwd"
    _need(q, "q", where, tuple(DTYPES))
    if q.dim() != 3:
        raise AttnError(1, f"{where}: q must be [T, H, D]")
    T, H, D = q.shape
    for name, t in (("k", k), ("v", v), ("out", out)):
        _need(t, name, where, (q.dtype,), q.shape, q.device)
    _need(lse, "lse", where, (torch.float32,), (H, T), q.device)
    _need_meta(where, cu_seqlens, seg_id, role, turn, dense_bits, dense_offsets, q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    params = _params(role_think, dense_bits, dense_offsets)
    _check(_native.lib().attn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), DTYPES[q.dtype], T, H, D, float(scale),
        _ptr(cu_seqlens), cu_seqlens.numel() - 1, max_seqlen, _kind(kind), ctypes.byref(params),
        _ptr(seg_id), _ptr(role), _ptr(turn), ctypes.byref(bm.struct), _stream(stream)),
        "attn_fwd")
    return out, lse


def attn_bwd_workspace_size(bm: BlockMask, num_heads: int, head_dim: int) -> int:
    """Bytes of device workspace attn_bwd needs: D and ||dO_i|| per row and
    head, per-sequence bound words and the int32 fixed-point dQ accumulator,
    O(T H D)."""
    out = ctypes.c_size_t()
    _check(_native.lib().attn_bwd_workspace_size(ctypes.byref(bm.struct), num_heads, head_dim,
                                                 ctypes.byref(out)), "attn_bwd_workspace_size")
    return int(out.value)


def attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
             lse: torch.Tensor, dout: torch.Tensor, bm: BlockMask, kind, cu_seqlens: torch.Tensor,
             max_seqlen: int, seg_id=None, role=None, turn=None, role_think: int = 1,
             scale: float = 0.0, dq: Optional[torch.Tensor] = None,
             dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, stream=None,
             dense_bits: Optional[torch.Tensor] = None, dense_offsets: Optional[torch.Tensor] = None):
    """Masked attention backward (bf16); returns (dQ, dK, dV), each [T, H, D].

    ``workspace`` (uint8, device) defaults to a fresh buffer of
    attn_bwd_workspace_size(bm, H, D) bytes.
    """
    where = "attn_bwd"
    _need(q, "q", where, tuple(DTYPES))
    if q.dim() != 3:
        raise AttnError(1, f"{where}: q must be [T, H, D]")
    T, H, D = q.shape
    if q.dtype != torch.bfloat16:
        raise AttnError(2, "attn_bwd: dtype must be bfloat16")
    for name, t in (("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq), ("dk", dk), ("dv", dv)):
        _need(t, name, where, (q.dtype,), q.shape, q.device)
    if o is None or dout is None or lse is None:
        raise AttnError(1, f"{where}: o, lse and dout are required")
    _need(lse, "lse", where, (torch.float32,), (H, T), q.device)
    _need(workspace, "workspace", where, device=q.device)
    _need_meta(where, cu_seqlens, seg_id, role, turn, dense_bits, dense_offsets, q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = torch.empty(attn_bwd_workspace_size(bm, H, D), dtype=torch.uint8, device=q.device)
    params = _params(role_think, dense_bits, dense_offsets)
    _check(_native.lib().attn_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
        DTYPES[q.dtype], T, H, D, float(scale), _ptr(cu_seqlens), cu_seqlens.numel() - 1,
        max_seqlen, _kind(kind), ctypes.byref(params), _ptr(seg_id), _ptr(role), _ptr(turn),
        ctypes.byref(bm.struct), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)),
        "attn_bwd")
    return dq, dk, dv


def attn_get_status(bm: BlockMask, stream=None) -> int:
    """Synchronise and return the device status code of the mask's error word."""
    return int(_native.lib().attn_get_status(ctypes.byref(bm.struct), _stream(stream)))


# ---------------------------------------------------------------------------
# Rotary positions and the 8-bit key / value cache (include/attn_cache.h)
# ---------------------------------------------------------------------------

ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "ramp": 3}


class _Launch:
    """Where a call runs when its device is not the current one or it names a
    stream: the device made current, new tensors allocated for that stream."""

    def __init__(self, device: torch.device, stream):
        self._guards = [torch.cuda.device(device)]
        self._stream, self._device = stream, device

    def __enter__(self):
        self._guards[0].__enter__()
        s = self._stream
        if s is None:
            return torch.cuda.current_stream().cuda_stream
        if not hasattr(s, "cuda_stream"):
            s = torch.cuda.ExternalStream(int(s), device=self._device)
        g = torch.cuda.stream(s)
        g.__enter__()
        self._guards.append(g)
        return s.cuda_stream

    def __exit__(self, *exc):
        # (also called without arguments, behind a plain try)
        exc = exc or (None, None, None)
        while self._guards:
            self._guards.pop().__exit__(*exc)


_Tensor = torch.Tensor
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_ROW_DTYPES = tuple(DTYPES)


def _raw_stream(index: int) -> int:
    # (looked up when called: a PyTorch without CUDA has none, and imports this module)
    return torch._C._cuda_getCurrentRawStream(index)


def _elsewhere(device: torch.device, stream):
    """None in the usual case, where a call runs on the current device and its
    current stream; otherwise the context it runs in."""
    if stream is None and device.index == torch._C._cuda_getDevice():
        return None
    return _Launch(device, stream)


def _fits(t, dtype, shape, index: int) -> bool:
    """The quick form of _need: a contiguous CUDA tensor of this type and shape on
    device `index`.  Where it is False, _need says what is wrong."""
    return (type(t) is _Tensor and t.dtype is dtype and t.get_device() == index and t.shape == shape
            and t.is_contiguous())


def _need_rows(t, name: str, where: str, dtypes, index: int = -1) -> int:
    """[tokens, heads, dim] with dense heads, tokens any distance apart (a slice
    of a wider projection); returns that distance in elements."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise AttnError(1, f"{where}: {name} must be a CUDA tensor")
    if index >= 0 and t.get_device() != index:
        raise AttnError(1, f"{where}: {name} is on {t.device}, expected cuda:{index}")
    if t.dtype not in dtypes:
        raise AttnError(1, f"{where}: {name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != 3:
        raise AttnError(1, f"{where}: {name} must be [tokens, heads, dim]")
    n, h, d = t.shape
    if t.is_contiguous():
        return h * d
    if (d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d):
        raise AttnError(1, f"{where}: the heads of {name} must be dense")
    if n > 1 and t.stride(0) < h * d:
        raise AttnError(1, f"{where}: the tokens of {name} overlap")
    return t.stride(0) if n > 1 else h * d


class RopePlan:
    """A prepared rotation (see ``attn_rope_plan``)."""

    def __init__(self, struct: _native.AttnRopePlan):
        self.struct = struct
        self._ref = ctypes.byref(struct)
        self.rotary_dim = int(struct.rotary_dim)


def attn_rope_plan(rotary_dim: int, base: float = 10000.0, interleaved: bool = False,
                   scaling: str = "none", factor: float = 1.0, original_context: float = 0.0,
                   alpha: float = 1.0, beta: float = 32.0, result_factor: float = 0.0) -> RopePlan:
    """Prepare a rotation of the first ``rotary_dim`` dimensions of each head:
    pairs (i, i + rotary_dim / 2), or neighbours when ``interleaved``.

    ``scaling`` stretches the angles theta_i = base^(-2 i / rotary_dim) to
    contexts ``factor`` times longer: "linear" divides them, "ntk" raises the
    base, "ramp" divides only those of pairs that turn less than ``alpha``
    times in ``original_context`` tokens, blending up to ``beta`` turns.
    ``result_factor`` multiplies the rotated dimensions (0: 1, or
    0.1 ln(factor) + 1 for "ramp")."""
    if scaling not in ROPE_SCALINGS:
        raise AttnError(1, f"attn_rope_plan: scaling must be one of {sorted(ROPE_SCALINGS)}")
    out = _native.AttnRopePlan()
    _check(_native.lib().attn_rope_plan_init(
        ctypes.byref(out), int(rotary_dim), int(bool(interleaved)), float(base), ROPE_SCALINGS[scaling],
        float(factor), float(original_context), float(alpha), float(beta), float(result_factor)),
        "attn_rope_plan")
    return RopePlan(out)


def attn_rope(q: torch.Tensor, k: Optional[torch.Tensor], plan: RopePlan,
              positions: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
              seq_lens: Optional[torch.Tensor] = None, inverse: bool = False,
              q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotate q [T, Hq, D] and k [T, Hk, D] (or None) by their positions;
    returns (q_out, k_out).

    Positions are ``positions`` (int32 [T]), or follow from ``cu_seqlens``
    (int32 [B + 1]): the place in the own sequence, behind the
    ``seq_lens[b] - n`` earlier tokens where ``seq_lens`` (int32 [B]) is given (as
    long as no eviction has shortened the sequence).
    ``inverse`` turns back: applied to the gradients of the rotated q and k it
    gives those of q and k.  bf16 or fp32; the tokens of q and k may be apart
    (slices of one projection).  ``q_out=q`` rotates in place."""
    where = "attn_rope"
    qs = _need_rows(q, "q", where, _ROW_DTYPES)
    T, H, D = q.shape
    dtype, dev = q.dtype, q.device
    index = dev.index
    ks = kos = Hk = 0
    if k is not None:
        ks = _need_rows(k, "k", where, (dtype,), index)
        n, Hk, d = k.shape
        if n != T or d != D:
            raise AttnError(1, f"{where}: k has shape {tuple(k.shape)}, expected [{T}, heads, {D}]")
    elif k_out is not None:
        raise AttnError(1, f"{where}: k_out without k")
    if not isinstance(plan, RopePlan):
        raise AttnError(1, f"{where}: plan must come from attn_rope_plan")
    batch = 0
    if positions is not None:
        if cu_seqlens is not None or seq_lens is not None:
            raise AttnError(1, f"{where}: positions, or cu_seqlens and seq_lens, not both")
        if not _fits(positions, _I32, (T,), index):
            _need(positions, "positions", where, (_I32,), (T,), dev)
    elif cu_seqlens is None:
        raise AttnError(1, f"{where}: positions or cu_seqlens is required")
    else:
        if not (isinstance(cu_seqlens, _Tensor) and _fits(cu_seqlens, _I32, cu_seqlens.shape, index)):
            _need(cu_seqlens, "cu_seqlens", where, (_I32,), device=dev)
        batch = cu_seqlens.numel() - 1
        if seq_lens is not None and not _fits(seq_lens, _I32, (batch,), index):
            _need(seq_lens, "seq_lens", where, (_I32,), (batch,), dev)
    at = _elsewhere(dev, stream)
    s = _raw_stream(index) if at is None else at.__enter__()
    try:
        if q_out is None:
            q_out, qos = torch.empty((T, H, D), dtype=dtype, device=dev), H * D
        else:
            qos = _need_rows(q_out, "q_out", where, (dtype,), index)
            if q_out.shape != q.shape:
                raise AttnError(1, f"{where}: q_out has shape {tuple(q_out.shape)}, expected {tuple(q.shape)}")
        if k is not None:
            if k_out is None:
                k_out, kos = torch.empty((T, Hk, D), dtype=dtype, device=dev), Hk * D
            else:
                kos = _need_rows(k_out, "k_out", where, (dtype,), index)
                if k_out.shape != k.shape:
                    raise AttnError(1, f"{where}: k_out has shape {tuple(k_out.shape)}, expected {tuple(k.shape)}")
        _check(_native.lib().attn_rope(
            q.data_ptr(), q_out.data_ptr(), qs, qos, H, k.data_ptr() if Hk else None,
            k_out.data_ptr() if Hk else None, ks, kos, Hk, DTYPES[dtype], T, D,
            None if positions is None else positions.data_ptr(),
            None if cu_seqlens is None else cu_seqlens.data_ptr(),
            None if seq_lens is None else seq_lens.data_ptr(), batch, plan._ref, 1 if inverse else 0, s), where)
    finally:
        if at is not None:
            at.__exit__()
    return q_out, k_out


class KVCache:
    """A paged key / value cache in e4m3 with one power-of-two scale per page
    and head: the C struct and the tensors it points into.

    k_pages, v_pages: uint8 or float8_e4m3fn [num_pages, heads, page_size, dim];
    k_scale, v_scale: fp32 [num_pages, heads]; page_table: int32
    [batch, max_pages].  The caller owns them, and the sequence lengths;
    the table may be rewritten between calls."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor, page_table: torch.Tensor, status: Optional[torch.Tensor] = None):
        where = "KVCache"
        codes = (torch.uint8, torch.float8_e4m3fn)
        _need(k_pages, "k_pages", where, codes)
        if k_pages is None or k_pages.dim() != 4:
            raise AttnError(1, f"{where}: k_pages must be [num_pages, heads, page_size, dim]")
        dev = k_pages.device
        P, H, ps, D = k_pages.shape
        for name, t, dt, shape in (("v_pages", v_pages, codes, (P, H, ps, D)),
                                   ("k_scale", k_scale, (torch.float32,), (P, H)),
                                   ("v_scale", v_scale, (torch.float32,), (P, H)),
                                   ("page_table", page_table, (torch.int32,), None)):
            if t is None:
                raise AttnError(1, f"{where}: {name} is required")
            _need(t, name, where, dt, shape, dev)
        if page_table.dim() != 2:
            raise AttnError(1, f"{where}: page_table must be [batch, max_pages]")
        _need(status, "status", where, (torch.int32,), (1,), dev)
        if status is None:
            status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.page_table, self.status = page_table, status
        self.device, self.index, self.num_kv_heads, self.head_dim = dev, dev.index, H, D
        self.batch, self.max_pages = page_table.shape
        self.page_size, self.num_pages = ps, P
        self.struct = _native.AttnKVCache(
            k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            page_table.data_ptr(), status.data_ptr(), P, H, ps, D, self.batch, self.max_pages)
        self._ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, num_pages: int, num_kv_heads: int, head_dim: int, page_table: torch.Tensor,
              page_size: int = 64) -> "KVCache":
        """A cache with new pages (codes 0, scales 1) on the table's device."""
        dev = page_table.device
        shape = (num_pages, num_kv_heads, page_size, head_dim)
        codes = [torch.zeros(shape, dtype=torch.uint8, device=dev) for _ in range(2)]
        scales = [torch.ones(shape[:2], dtype=torch.float32, device=dev) for _ in range(2)]
        return cls(*codes, *scales, page_table)


def _need_cache(cache, where: str) -> KVCache:
    if not isinstance(cache, KVCache):
        raise AttnError(1, f"{where}: cache must be a KVCache")
    return cache


def _need_seqs(cache: KVCache, cu_seqlens, seq_lens, where: str) -> None:
    if seq_lens is None or cu_seqlens is None:
        raise AttnError(1, f"{where}: cu_seqlens and seq_lens are required")
    if not (_fits(cu_seqlens, _I32, (cache.batch + 1,), cache.index)
            and _fits(seq_lens, _I32, (cache.batch,), cache.index)):
        _need(cu_seqlens, "cu_seqlens", where, (torch.int32,), (cache.batch + 1,), cache.device)
        _need(seq_lens, "seq_lens", where, (torch.int32,), (cache.batch,), cache.device)


def attn_cache_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, cu_seqlens: torch.Tensor,
                      seq_lens: torch.Tensor, max_new: int, stream=None) -> None:
    """Quantise the new tokens' keys and values [T, Hk, D] (bf16 or fp32) into
    the cache.  Sequence b's new tokens are rows cu_seqlens[b] ..
    cu_seqlens[b + 1] - 1 and become its last ones: ``seq_lens`` counts them in.
    ``max_new`` bounds each sequence's number of new tokens.  Their pages must
    belong to the sequence alone."""
    where = "attn_cache_append"
    _need_cache(cache, where)
    ks = _need_rows(k, "k", where, _ROW_DTYPES, cache.index)
    vs = _need_rows(v, "v", where, (k.dtype,), cache.index)
    T, h, d = k.shape
    if k.shape != v.shape or h != cache.num_kv_heads or d != cache.head_dim:
        raise AttnError(1, f"{where}: k and v must be [tokens, {cache.num_kv_heads}, {cache.head_dim}], got "
                           f"{tuple(k.shape)} and {tuple(v.shape)}")
    _need_seqs(cache, cu_seqlens, seq_lens, where)
    at = _elsewhere(cache.device, stream)
    s = _raw_stream(cache.index) if at is None else at.__enter__()
    try:
        _check(_native.lib().attn_cache_append(
            k.data_ptr(), v.data_ptr(), ks, vs, DTYPES[k.dtype], T, cu_seqlens.data_ptr(),
            seq_lens.data_ptr(), max_new, cache._ref, s), where)
    finally:
        if at is not None:
            at.__exit__()


def _need_queries(q, cache, where: str):
    _need_cache(cache, where)
    if q is None:
        raise AttnError(1, f"{where}: q is required")
    if not (isinstance(q, _Tensor) and _fits(q, _BF16, q.shape, cache.index)):
        _need(q, "q", where, _ROW_DTYPES, device=cache.device)
        if q.dtype != _BF16:
            raise AttnError(2, f"{where}: dtype must be bfloat16")
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.head_dim or shape[1] % cache.num_kv_heads:
        raise AttnError(1, f"{where}: q has shape {tuple(shape)}, expected [tokens, a multiple of "
                           f"{cache.num_kv_heads}, {cache.head_dim}]")
    return shape


def attn_cache_fwd_workspace_size(cache: KVCache, total_tokens: int, num_heads: int, max_new: int,
                                  max_seqlen: int) -> int:
    """Bytes of device workspace ``attn_cache_fwd`` needs at these sizes."""
    _need_cache(cache, "attn_cache_fwd_workspace_size")
    out = ctypes.c_size_t()
    _check(_native.lib().attn_cache_fwd_workspace_size(cache._ref, total_tokens, num_heads, max_new,
                                                       max_seqlen, ctypes.byref(out)),
           "attn_cache_fwd_workspace_size")
    return int(out.value)


def attn_cache_fwd(q: torch.Tensor, cache: KVCache, cu_seqlens: torch.Tensor, seq_lens: torch.Tensor,
                   max_new: int, max_seqlen: int, kind="causal", scale: float = 0.0,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of the new tokens' queries q [T, H, D] (bf16) over the cache,
    which holds their keys and values already (``attn_cache_append``); returns
    (O [T, H, D], LSE [H, T] fp32).

    ``kind`` is "causal" (a query sees the tokens up to its own) or "none" (all
    of its sequence's).  ``max_new`` and ``max_seqlen`` bound the new tokens and
    the length of every sequence.  Rows behind the last sequence keep what
    ``out`` and ``lse`` held.  ``workspace`` (uint8) defaults to a new buffer of
    ``attn_cache_fwd_workspace_size`` bytes; calls that may overlap need one each."""
    where = "attn_cache_fwd"
    T, H, D = _need_queries(q, cache, where)
    dev = cache.device
    if out is not None and not _fits(out, _BF16, q.shape, cache.index):
        _need(out, "out", where, (q.dtype,), q.shape, dev)
    if lse is not None and not _fits(lse, _F32, (H, T), cache.index):
        _need(lse, "lse", where, (torch.float32,), (H, T), dev)
    _need(workspace, "workspace", where, device=dev)
    _need_seqs(cache, cu_seqlens, seq_lens, where)
    at = _elsewhere(dev, stream)
    s = _raw_stream(cache.index) if at is None else at.__enter__()
    try:
        if out is None:
            out = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((H, T), dtype=torch.float32, device=dev)
        own = None
        if workspace is not None:
            ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        else:
            ws, nbytes = None, attn_cache_fwd_workspace_size(cache, T, H, max_new, max_seqlen)
            if nbytes:
                # what torch.empty draws on, without a tensor around it (a fifth of its time)
                ws = own = torch._C._cuda_cudaCachingAllocator_raw_alloc(nbytes, s)
        try:
            _check(_native.lib().attn_cache_fwd(
                q.data_ptr(), out.data_ptr(), lse.data_ptr(), 0, T, H, scale, cu_seqlens.data_ptr(), max_new,
                seq_lens.data_ptr(), max_seqlen, _kind(kind), cache._ref, ws, nbytes, s), where)
        finally:
            if own is not None:  # reused in the order of the stream
                torch._C._cuda_cudaCachingAllocator_raw_delete(own)
    finally:
        if at is not None:
            at.__exit__()
    return out, lse


def attn_cache_weights(q: torch.Tensor, lse: torch.Tensor, cache: KVCache, cu_seqlens: torch.Tensor,
                       seq_lens: torch.Tensor, max_new: int, max_seqlen: int, kind="causal",
                       scale: float = 0.0, prev: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The attention weight that each cached token receives from the queries of
    an ``attn_cache_fwd`` call (its q and LSE, the same kind and scale), summed over
    the queries and the query heads of each key / value head and added to
    ``prev``: fp32 [batch, heads, width], width >= max_seqlen.  ``out=prev``
    adds in place.  Entries behind a sequence's tokens keep what ``out`` held
    (0 in a new one)."""
    where = "attn_cache_weights"
    T, H, D = _need_queries(q, cache, where)
    dev = cache.device
    if lse is None:
        raise AttnError(1, f"{where}: lse is required")
    if not _fits(lse, torch.float32, (H, T), cache.index):
        _need(lse, "lse", where, (torch.float32,), (H, T), dev)
    _need_seqs(cache, cu_seqlens, seq_lens, where)
    like = out if out is not None else prev
    shape = (cache.batch, cache.num_kv_heads, int(max_seqlen)) if like is None else tuple(like.shape)
    if len(shape) != 3 or shape[:2] != (cache.batch, cache.num_kv_heads):
        raise AttnError(1, f"{where}: weights must be [{cache.batch}, {cache.num_kv_heads}, width], got {shape}")
    for name, t in (("prev", prev), ("out", out)):
        if t is not None and not _fits(t, torch.float32, shape, cache.index):
            _need(t, name, where, (torch.float32,), shape, dev)
    at = _elsewhere(dev, stream)
    s = _raw_stream(cache.index) if at is None else at.__enter__()
    try:
        if out is None:
            out = torch.zeros(shape, dtype=torch.float32, device=dev)
        _check(_native.lib().attn_cache_weights(
            q.data_ptr(), lse.data_ptr(), DTYPES[q.dtype], T, H, float(scale), cu_seqlens.data_ptr(),
            int(max_new), seq_lens.data_ptr(), int(max_seqlen), _kind(kind), cache._ref,
            None if prev is None else prev.data_ptr(), out.data_ptr(), shape[2], s), where)
    finally:
        if at is not None:
            at.__exit__()
    return out


def _need_weights(t, name: str, cache: KVCache, where: str) -> None:
    """fp32 [batch, heads, width], any width."""
    B, H = cache.batch, cache.num_kv_heads
    if not (isinstance(t, _Tensor) and t.dim() == 3 and _fits(t, _F32, (B, H, t.shape[2]), cache.index)):
        _need(t, name, where, (_F32,), device=cache.device)
        if t.dim() != 3 or tuple(t.shape[:2]) != (B, H):
            raise AttnError(1, f"{where}: {name} must be [{B}, {H}, width], got {tuple(t.shape)}")


def attn_cache_evict(weights: torch.Tensor, cache: KVCache, dst: KVCache, seq_lens: torch.Tensor,
                     budgets: torch.Tensor, recent: int, max_seqlen: int, max_keep: int,
                     kept: Optional[torch.Tensor] = None, new_weights: Optional[torch.Tensor] = None,
                     new_lens: Optional[torch.Tensor] = None, stream=None):
    """Keep min(seq_lens[b], budgets[b]) tokens of each sequence, for every head
    by itself: the last ``recent`` ones and, of the others, those with the
    largest ``weights`` (fp32 [batch, heads, width]; ties to the lower index,
    -inf first to go), and copy them in order into ``dst``'s pages (a KVCache
    with a page table of its own; the pools may be the same, the pages not).
    Keys stay as they were rotated, so that later tokens of a shortened sequence take
    ``attn_rope``'s ``positions`` (their place in the whole text), not its ``seq_lens``.

    Returns (kept int32 [batch, heads, max_keep] with -1 behind the last,
    new_weights [batch, heads, max_keep or wider] with 0 behind the last,
    new_lens int32 [batch])."""
    where = "attn_cache_evict"
    _need_cache(cache, where)
    _need_cache(dst, where)
    dev, B, H = cache.device, cache.batch, cache.num_kv_heads
    if dst.device != dev:
        raise AttnError(1, f"{where}: dst is on {dst.device}, expected {dev}")
    max_keep = int(max_keep)
    if weights is None or seq_lens is None or budgets is None:
        raise AttnError(1, f"{where}: weights, seq_lens and budgets are required")
    index = cache.index
    if not (_fits(seq_lens, _I32, (B,), index) and _fits(budgets, _I32, (B,), index)
            and (kept is None or _fits(kept, _I32, (B, H, max_keep), index))
            and (new_lens is None or _fits(new_lens, _I32, (B,), index))):
        for name, t, shape in (("seq_lens", seq_lens, (B,)), ("budgets", budgets, (B,)),
                               ("kept", kept, (B, H, max_keep)), ("new_lens", new_lens, (B,))):
            _need(t, name, where, (_I32,), shape, dev)
    _need_weights(weights, "weights", cache, where)
    if new_weights is not None:
        _need_weights(new_weights, "new_weights", cache, where)
    if max_keep < 0:
        raise AttnError(1, f"{where}: max_keep is negative")
    at = _elsewhere(dev, stream)
    s = _raw_stream(cache.index) if at is None else at.__enter__()
    try:
        if kept is None:
            kept = torch.empty((B, H, max_keep), dtype=torch.int32, device=dev)
        if new_weights is None:
            new_weights = torch.empty((B, H, max_keep), dtype=torch.float32, device=dev)
        if new_lens is None:
            new_lens = torch.empty(B, dtype=torch.int32, device=dev)
        _check(_native.lib().attn_cache_evict(
            weights.data_ptr(), weights.shape[2], seq_lens.data_ptr(), budgets.data_ptr(), int(recent),
            int(max_seqlen), max_keep, cache._ref, dst._ref, kept.data_ptr(), new_weights.data_ptr(),
            new_weights.shape[2], new_lens.data_ptr(), s), where)
    finally:
        if at is not None:
            at.__exit__()
    return kept, new_weights, new_lens


def attn_cache_get_status(cache: KVCache, stream=None) -> int:
    """Synchronise, then return and clear the cache's device status code."""
    _need_cache(cache, "attn_cache_get_status")
    at = _elsewhere(cache.device, stream)
    s = _raw_stream(cache.index) if at is None else at.__enter__()
    try:
        return int(_native.lib().attn_cache_get_status(cache._ref, s))
    finally:
        if at is not None:
            at.__exit__()
