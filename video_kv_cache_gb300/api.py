"""Convenience layer over the C ABI: allocates the compressed cache and the workspace as
torch CUDA tensors and passes their pointers and the current stream to libqvg.

torch is used here only for device memory and streams; the computation is entirely in
libqvg's kernels (video_kv_cache_gb300.qvg is the ctypes binding).
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from fractions import Fraction

import torch

from . import qvg as _c

_DT = {torch.float16: _c.QVG_F16, torch.bfloat16: _c.QVG_BF16, torch.float32: _c.QVG_F32}
D = 128


@dataclass
class CompressedKV:
    """The compressed cache of H tensors (layouts as in include/qvg.h)."""
    codes: torch.Tensor      # uint8 [H][cap][d*bits/8]
    scales: torch.Tensor     # uint8 [H][cap][d/group], E4M3 bit patterns
    pi: torch.Tensor         # uint8 [H][T][cap]
    centroids: torch.Tensor  # fp32  [H][n_tables][T][C][d]
    C: int
    T: int
    bits: int
    group: int
    qscheme: int = 0         # qvg_qscheme of the codes (set by quantize)
    centroid_format: int = 0  # qvg_centroid_format of the stored centroids (set by quantize)

    @property
    def H(self):
        return self.codes.shape[0]

    @property
    def capacity(self):
        return self.codes.shape[1]

    @property
    def n_tables(self):
        return self.centroids.shape[1]

    def buffers(self) -> _c.qvg_buffers:
        return _c.qvg_buffers(self.codes.data_ptr(), self.scales.data_ptr(),
                              self.pi.data_ptr() if self.pi.numel() else None,
                              self.centroids.data_ptr() if self.centroids.numel() else None)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.codes, self.scales, self.pi, self.centroids))


def allocate(H: int, capacity: int, C: int, T: int, bits: int, group: int, n_tables: int = 1,
             device="cuda") -> CompressedKV:
    dev = torch.device(device)
    return CompressedKV(
        codes=torch.empty((H, capacity, D * bits // 8), dtype=torch.uint8, device=dev),
        scales=torch.empty((H, capacity, D // group), dtype=torch.uint8, device=dev),
        pi=torch.empty((H, T, capacity), dtype=torch.uint8, device=dev),
        centroids=torch.empty((H, n_tables, T, C if T > 0 else 0, D), dtype=torch.float32,
                              device=dev),
        C=C, T=T, bits=bits, group=group)


def quant_params(H, N, C, T, bits, group, iters, dtype, seed=0, tensor_id_base=0, x_stride=0,
                 token_offset=0, token_capacity=0, table_index=0, n_tables=0, warm_stride=0,
                 qscheme=0, centroid_format=0):
    return _c.qvg_quant_params(n_tensors=H, d=D, N=N, C=C, T=T, bits=bits, group=group,
                               iters=iters, in_dtype=_DT[dtype], seed=seed & (2 ** 64 - 1),
                               tensor_id_base=tensor_id_base, x_stride=x_stride,
                               token_offset=token_offset, token_capacity=token_capacity,
                               table_index=table_index, n_tables=n_tables,
                               warm_stride=warm_stride, qscheme=qscheme,
                               centroid_format=centroid_format)


def workspace_bytes(H: int, N: int, C: int, T: int, bits: int = 2, group: int = 32) -> int:
    return _c.qvg_quantize_workspace_bytes(
        quant_params(H, N, C, T, bits, group, 1, torch.bfloat16))


def new_workspace(H: int, N: int, C: int, T: int, device="cuda") -> torch.Tensor:
    n = workspace_bytes(H, N, C, T)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _stream_handle(stream):
    if stream is not None:
        return stream.cuda_stream
    # the raw handle of the current stream, without the Stream object around it
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def quantize(X: torch.Tensor, C: int, T: int, bits: int, group: int, iters: int, seed: int = 0,
             *, warm: torch.Tensor | None = None, warm_stride: int = 0,
             out: CompressedKV | None = None, token_offset: int = 0, table_index: int = 0,
             workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
             tensor_id_base: int = 0, stream=None, qscheme: int = 0,
             centroid_format: int = 0) -> CompressedKV:
    """Compress X [H][N][128] (fp16 / bf16 / fp32 CUDA tensor; tensor stride may be larger
    than N*128).  With ``out`` given, writes tokens [token_offset, token_offset + N) and
    centroid table ``table_index`` of it; ``warm`` (fp32 [H][T][C][128] or a view with tensor
    stride ``warm_stride``) replaces the seeded cold start.  ``qscheme`` picks the integer
    grid of the codes (qvg.QVG_QSCHEME_*) and ``centroid_format`` the value format of the
    stored centroids (qvg.QVG_CENTROIDS_*); both are recorded in the returned cache."""
    assert X.is_cuda and X.dim() == 3 and X.shape[2] == D
    assert X.stride(2) == 1 and X.stride(1) == D
    H, N, _ = X.shape
    if out is None:
        out = allocate(H, N, C, T, bits, group, 1, X.device)
    if workspace is None:
        workspace = new_workspace(H, N, C, T, X.device)
    prm = quant_params(H, N, C, T, bits, group, iters, X.dtype, seed, tensor_id_base,
                       X.stride(0), token_offset, out.capacity, table_index, out.n_tables,
                       warm_stride, qscheme, centroid_format)
    rc = _c.qvg_quantize(prm, X.data_ptr(), warm.data_ptr() if warm is not None else None,
                         out.buffers(), workspace.data_ptr(), workspace.numel(),
                         status.data_ptr() if status is not None else None,
                         _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_quantize")
    out.qscheme = qscheme
    out.centroid_format = centroid_format
    return out


def reassign(X: torch.Tensor, ckv: CompressedKV, iters: int, workspace: torch.Tensor,
             seed: int = 0, *, token_offset: int = 0, table_index: int = 0,
             status: torch.Tensor | None = None, tensor_id_base: int = 0, stream=None,
             steps: int | None = None):
    """Re-run the last stage's assignment against the stored centroids (see qvg_reassign);
    the arguments must match the preceding quantize call.  ``steps``: a mask of
    QVG_STEP_PLANES / QVG_STEP_GEMM / QVG_STEP_REFINE (qvg_reassign_steps); all by default."""
    H, N, _ = X.shape
    prm = quant_params(H, N, ckv.C, ckv.T, ckv.bits, ckv.group, iters, X.dtype, seed,
                       tensor_id_base, X.stride(0), token_offset, ckv.capacity, table_index,
                       ckv.n_tables)
    st = status.data_ptr() if status is not None else None
    if steps is None:
        rc = _c.qvg_reassign(prm, X.data_ptr(), ckv.buffers(), workspace.data_ptr(),
                             workspace.numel(), st, _stream_handle(stream))
    else:
        rc = _c.qvg_reassign_steps(prm, X.data_ptr(), ckv.buffers(), workspace.data_ptr(),
                                   workspace.numel(), steps, st, _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_reassign")


def dequantize(ckv: CompressedKV, N: int | None = None, out_dtype=torch.bfloat16,
               chunk_len: int = 0, out: torch.Tensor | None = None,
               status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Reconstruct tokens [0, N) of every tensor into ``out`` [H][N][128] (tensor stride
    may be larger); token i uses centroid table i // chunk_len (0 = one table)."""
    N = ckv.capacity if N is None else N
    if out is None:
        out = torch.empty((ckv.H, N, D), dtype=out_dtype, device=ckv.codes.device)
    assert out.stride(2) == 1 and out.stride(1) == D
    prm = _c.qvg_dequant_params(n_tensors=ckv.H, d=D, N=N, C=ckv.C if ckv.T > 0 else 0, T=ckv.T,
                                bits=ckv.bits, group=ckv.group, out_dtype=_DT[out.dtype],
                                chunk_len=chunk_len, token_capacity=ckv.capacity,
                                n_tables=ckv.n_tables, out_stride=out.stride(0),
                                qscheme=ckv.qscheme)
    rc = _c.qvg_dequantize(prm, ckv.buffers(), out.data_ptr(),
                           status.data_ptr() if status is not None else None,
                           _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_dequantize")
    return out


def attention_params(ckv: CompressedKV, H: int, M: int, N: int, q_dtype, out_dtype, scale: float,
                     chunk_len: int = 0, k_first: int = 0, v_first: int = 0,
                     tensor_step: int = 1):
    return _c.qvg_attention_params(
        n_heads=H, d=D, M=M, N=N, C=ckv.C if ckv.T > 0 else 0, T=ckv.T, bits=ckv.bits,
        group=ckv.group, qscheme=ckv.qscheme, chunk_len=chunk_len,
        token_capacity=ckv.capacity, n_tables=ckv.n_tables, q_dtype=_DT[q_dtype],
        out_dtype=_DT[out_dtype], scale=scale, k_first=k_first, v_first=v_first,
        tensor_step=tensor_step)


def attention_layout(one_cache: bool, k_first=None, v_first=None, tensor_step=None):
    """(k_first, v_first, tensor_step) with the defaults of ``attention`` filled in: keys and
    values interleaved in one cache (0, 1, 2), or tensor h of each of two caches (0, 0, 1)."""
    return (0 if k_first is None else k_first,
            (1 if one_cache else 0) if v_first is None else v_first,
            (2 if one_cache else 1) if tensor_step is None else tensor_step)


def attention(Q: torch.Tensor, k_cache: CompressedKV, v_cache: CompressedKV | None = None,
              scale: float | None = None, N: int | None = None, *, out_dtype=torch.float32,
              chunk_len: int = 0, k_first: int | None = None, v_first: int | None = None,
              tensor_step: int | None = None, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """Softmax attention of Q [H][M][128] over tokens [0, N) of compressed keys and values
    (qvg_attention): head h reads key tensor k_first + h * tensor_step of ``k_cache`` and
    value tensor v_first + h * tensor_step of ``v_cache``.  With one cache (``v_cache``
    omitted) the default layout is keys and values interleaved, tensors 2h and 2h + 1; with
    two caches it is tensor h of each.  ``scale`` defaults to 1 / sqrt(128)."""
    k_first, v_first, tensor_step = attention_layout(v_cache is None, k_first, v_first,
                                                     tensor_step)
    v_cache = k_cache if v_cache is None else v_cache
    assert Q.is_cuda and Q.dim() == 3 and Q.shape[2] == D and Q.is_contiguous()
    H, M, _ = Q.shape
    N = k_cache.capacity if N is None else N
    scale = D ** -0.5 if scale is None else scale
    if out is None:
        out = torch.empty((H, M, D), dtype=out_dtype, device=Q.device)
    assert out.is_contiguous() and out.shape == (H, M, D)
    prm = attention_params(k_cache, H, M, N, Q.dtype, out.dtype, scale, chunk_len, k_first,
                           v_first, tensor_step)
    need = _c.qvg_attention_workspace_bytes(prm)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=Q.device)
    rc = _c.qvg_attention(prm, Q.data_ptr(), k_cache.buffers(), v_cache.buffers(),
                          out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                          status.data_ptr() if status is not None else None,
                          _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_attention")
    return out


# ------------------------------------------------------------------------------------
# The paged cache of recent tokens: rotary positions, writing, reading, attention
# ------------------------------------------------------------------------------------

_PAGE_FORMAT = {torch.float16: _c.QVG_PAGE_F16, torch.bfloat16: _c.QVG_PAGE_BF16,
                torch.float8_e4m3fn: _c.QVG_PAGE_E4M3, torch.int8: _c.QVG_PAGE_INT8,
                torch.float4_e2m1fn_x2: _c.QVG_PAGE_E2M1, torch.uint8: _c.QVG_PAGE_INT4}
_WIDE = (torch.float16, torch.bfloat16)
_FOUR = (torch.float4_e2m1fn_x2, torch.uint8)  # two codes an element
GROUP = 16  # channels that share a scale in a 4-bit row


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _gpu(x: torch.Tensor, what: str) -> int:
    """The GPU that x is on, which is the one that the call launches on: the current one."""
    dev = x.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError("%s must be on the current GPU" % what)
    return dev


def _rows(x: torch.Tensor, what: str, dev: int):
    """(tokens, heads, token stride, head stride) of rows [tokens][heads][128] of contiguous
    channels; a stride is 0 where there is one row only, whose stride says nothing."""
    shape, stride = x.shape, x.stride()
    if not (x.get_device() == dev and len(shape) == 3 and shape[2] == D and stride[2] == 1 and x.dtype in _DT):
        _need(x.get_device() == dev and len(shape) == 3 and shape[2] == D and (stride[2] == 1 or x.numel() == 0),
              "%s must be a tensor [tokens][heads][128] on the call's GPU, with contiguous channels" % what)
        _need(x.dtype in _DT, "%s must be fp16, bf16 or fp32" % what)
    return (shape[0], shape[1], stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0)


def _index(x: torch.Tensor, dtype, shape, what: str, dev: int | None = None):
    if not (x.dtype == dtype and x.shape == shape and x.is_contiguous()
            and (x.is_cuda if dev is None else x.get_device() == dev)):
        raise ValueError("%s must be a contiguous tensor %s of %s on the call's GPU" % (what, list(shape), dtype))


def _check_scratch(status, workspace, dev: int):
    if status is not None and not (status.get_device() == dev and status.dtype == torch.int32 and status.numel() >= 1):
        raise ValueError("status must be an int32 tensor on the call's GPU")
    if workspace is not None and not (workspace.get_device() == dev and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the call's GPU")


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to the stream that the call uses."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_as(X, shape, dtype, stream):
    """A new tensor beside X; one that is just like it takes less time to make."""
    if stream is None and dtype is X.dtype and X.is_contiguous():
        return torch.empty_like(X)
    return _empty(shape, dtype, X.device, stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


@dataclass(frozen=True)
class RopeTable:
    """Frequencies and layout of a rotary position code (see qvg_rotary)."""
    freqs: torch.Tensor       # int64 [rot_dim / 2]: turns per position as 64-bit fractions
    rot_dim: int
    sections: tuple           # pairs of each position axis
    interleaved: bool = False
    mscale: float = 1.0

    def __post_init__(self):
        sections = tuple(int(s) for s in self.sections)
        object.__setattr__(self, "sections", sections)
        _need(1 <= len(sections) <= 4 and sum(sections) == self.rot_dim // 2,
              "1 to 4 sections must add up to rot_dim / 2 pairs")
        _index(self.freqs, torch.int64, (self.rot_dim // 2,), "freqs")
        axes = len(sections)
        object.__setattr__(self, "_fixed", _c.qvg_rotary(
            self.rot_dim, int(self.interleaved), axes, (*sections, *(0,) * (4 - axes)),
            self.mscale, 0, None, self.freqs.data_ptr()))

    def __reduce__(self):  # a copy describes its own tensor's memory
        return RopeTable, (self.freqs, self.rot_dim, self.sections, self.interleaved, self.mscale)

    def rotary(self, positions: torch.Tensor, n: int) -> _c.qvg_rotary:
        dev = self.freqs.get_device()
        axes, shape, stride = len(self.sections), positions.shape, positions.stride()
        if len(shape) == 1:
            shape, stride = (1, shape[0]), (n, stride[0])
        if not (positions.get_device() == dev and positions.dtype == torch.int64 and shape == (axes, n)
                and (n <= 1 or stride[1] == 1) and (axes == 1 or stride[0] >= n)):
            raise ValueError("positions must be int64 [%d][%d] on the table's GPU, each axis contiguous" % (axes, n))
        r = _c.qvg_rotary.from_buffer_copy(self._fixed)
        r.pos_stride = stride[0]
        r.positions = positions.data_ptr()
        return r


def rope_frequencies(rot_dim: int, base: float = 10000.0, sections=None, scaling: str = "none",
                     factor: float = 1.0, original_len: int = 4096, fast_turns: float = 32.0,
                     slow_turns: float = 1.0):
    """(radians per position of each pair, mscale): pair i of an axis with n pairs turns
    base ** (-i / n) a position.  ``scaling`` fits longer contexts by ``factor``:
      * "linear": every frequency divided by the factor (position interpolation);
      * "stretched": a larger base, which slows the slowest pair by the factor and leaves the
        fastest as it is;
      * "by_parts" (YaRN, arXiv 2309.00071): pairs that turn more than ``fast_turns`` times in
        ``original_len`` positions stay, those below ``slow_turns`` are divided by the factor,
        a linear ramp between; mscale is 0.1 ln(factor) + 1."""
    _need(scaling in ("none", "linear", "stretched", "by_parts"), "unknown scaling %r" % (scaling,))
    _need(rot_dim >= 2 and rot_dim % 2 == 0 and base > 0 and factor >= 1,
          "rot_dim must be even, base positive and factor at least 1")
    _need(fast_turns > slow_turns and original_len > 0,
          "fast_turns must be above slow_turns, and original_len positive")
    sections = (rot_dim // 2,) if sections is None else tuple(sections)
    _need(sum(sections) == rot_dim // 2, "sections must add up to rot_dim / 2")
    out, mscale = [], 1.0
    for n in sections:
        b = base * factor ** (n / (n - 1.0)) if scaling == "stretched" and n > 1 else base
        out += [b ** (-i / n) for i in range(n)]
    if scaling == "linear":
        out = [f / factor for f in out]
    elif scaling == "by_parts":
        turns = [original_len * f / (2 * math.pi) for f in out]
        keep = [min(1.0, max(0.0, (t - slow_turns) / (fast_turns - slow_turns))) for t in turns]
        out = [f * k + f / factor * (1 - k) for f, k in zip(out, keep)]
        mscale = 0.1 * math.log(factor) + 1.0
    return torch.tensor(out, dtype=torch.float64), mscale


def rope_table(rot_dim: int = D, *, freqs=None, sections=None, interleaved: bool = False,
               mscale: float | None = None, device="cuda", **kw) -> RopeTable:
    """A rotary table on the device, from given radians per position of each pair or from
    ``rope_frequencies(rot_dim, sections=sections, **kw)``.  ``sections`` gives the pairs of
    each position axis (frame, row and column of a video token, say); one axis by default."""
    if freqs is None:
        freqs, made = rope_frequencies(rot_dim, sections=sections, **kw)
        mscale = made if mscale is None else mscale
    else:
        _need(not kw, "freqs are given: %s would have no effect" % ", ".join(kw))
    turns = torch.as_tensor(freqs, dtype=torch.float64).cpu() / (2 * math.pi)
    _need(turns.shape == (rot_dim // 2,) and bool(torch.isfinite(turns).all()),
          "freqs must be rot_dim / 2 finite numbers")
    words = [round(Fraction(f) * 2 ** 64) % 2 ** 64 for f in turns.tolist()]
    words = torch.tensor([w - 2 ** 64 if w >= 2 ** 63 else w for w in words], dtype=torch.int64)
    return RopeTable(words.to(device), rot_dim, (rot_dim // 2,) if sections is None else sections,
                     bool(interleaved), 1.0 if mscale is None else float(mscale))


def rope(X: torch.Tensor, positions: torch.Tensor, table: RopeTable, *,
         out: torch.Tensor | None = None, backward: bool = False, stream=None) -> torch.Tensor:
    """Turn X [n][heads][128] (fp16 / bf16 / fp32, any token and head strides) by its positions
    (int64 [n], or [axes][n] for a table with several axes).  ``out`` may be X itself.
    ``backward`` gives the gradient of X from that of the result.  Autograd does not record the
    call, so an X whose gradient it would have to carry is refused: call it under
    ``torch.no_grad()`` or from a ``torch.autograd.Function``, whose backward is
    ``backward=True``."""
    dev = _gpu(X, "X")
    _need(not (X.requires_grad and torch.is_grad_enabled()),
          "autograd would lose X's gradient here: call rope without gradient recording, and backward=True for it")
    n, heads, xt, xh = _rows(X, "X", dev)
    _need(table.freqs.get_device() == dev, "the table must be on the GPU of X")
    if out is None:
        out = _empty_as(X, (n, heads, D), X.dtype, stream)
        yt, yh = heads * D, D
    else:
        on, oh, yt, yh = _rows(out, "out", dev)
        _need(on == n and oh == heads and out.dtype == X.dtype, "out must have the shape and type of X")
    prm = _c.qvg_rope_params(n, heads, D, _DT[X.dtype], 1 if backward else 0, xt, xh, yt, yh)
    rc = _c.qvg_rope(prm, table.rotary(positions, n), X.data_ptr(), out.data_ptr(),
                     _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_rope")
    return out


@dataclass(frozen=True)
class PagedKV:
    """Pages of recent keys and values (layouts as in include/qvg.h).  The type of ``k`` and
    ``v`` is the page format: fp16, bf16, float8_e4m3fn or int8, or, with two 4-bit codes an
    element, float4_e2m1fn_x2 (E2M1) or uint8 (INT4).  8-bit and 4-bit pages have a scale for
    each row, 4-bit ones another for each group of 16 channels."""
    k: torch.Tensor                        # [pages][heads][page_tokens][128], 4 bits: [..][64]
    v: torch.Tensor
    k_scale: torch.Tensor | None = None    # fp32 [pages][heads][page_tokens]
    v_scale: torch.Tensor | None = None
    k_group: torch.Tensor | None = None    # float8_e4m3fn [pages][heads][page_tokens][8]
    v_group: torch.Tensor | None = None

    def __post_init__(self):
        shape = self.k.shape
        four = self.k.dtype in _FOUR
        _need(len(shape) == 4 and shape[3] == (D // 2 if four else D) and self.k.dtype in _PAGE_FORMAT,
              "pages are [pages][heads][page_tokens][128] of fp16, bf16, float8_e4m3fn or int8, "
              "or [pages][heads][page_tokens][64] of float4_e2m1fn_x2 or uint8 (INT4)")
        dev = self.k.get_device()
        for t in (self.k, self.v):
            _index(t, self.k.dtype, shape, "k and v")
            _need(t.get_device() == dev, "k and v must be on one GPU")
        for t in (self.k_scale, self.v_scale):
            if self.k.dtype in _WIDE:
                _need(t is None, "16-bit pages have no scales")
            else:
                _need(t is not None, "8-bit and 4-bit pages need k_scale and v_scale")
                _index(t, torch.float32, shape[:3], "scales", dev)
        for t in (self.k_group, self.v_group):
            if four:
                _need(t is not None, "4-bit pages need k_group and v_group")
                _index(t, torch.float8_e4m3fn, (*shape[:3], D // GROUP), "group scales", dev)
            else:
                _need(t is None, "only 4-bit pages have group scales")
        for name, value in (("gpu", dev), ("n_pages", shape[0]), ("heads", shape[1]), ("page_tokens", shape[2]),
                            ("format", _PAGE_FORMAT[self.k.dtype]),
                            ("_buffers", _c.qvg_pages(self.k.data_ptr(), self.v.data_ptr(),
                                                      _ptr(self.k_scale), _ptr(self.v_scale),
                                                      _ptr(self.k_group), _ptr(self.v_group)))):
            object.__setattr__(self, name, value)
        object.__setattr__(self, "_copy_params", _c.qvg_page_table_params(
            1, self.heads, D, self.page_tokens, self.format, 1, self.n_pages, 0, 0))

    def __reduce__(self):  # a copy describes its own tensors' memory
        parts = (self.k, self.v, self.k_scale, self.v_scale, self.k_group, self.v_group)
        # (torch does not pickle tensors of 8-bit and 4-bit floats: their bytes go, and their type)
        odd = (torch.float8_e4m3fn, torch.float4_e2m1fn_x2)
        return _pages_of, tuple((t.dtype, t.view(torch.uint8)) if t is not None and t.dtype in odd else (None, t) for t in parts)

    def buffers(self) -> _c.qvg_pages:
        return self._buffers

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.k, self.v, self.k_scale, self.v_scale, self.k_group, self.v_group) if t is not None)


def _pages_of(*parts):
    return PagedKV(*(t if dtype is None else t.view(dtype) for dtype, t in parts))


def allocate_pages(n_pages: int, heads: int, page_tokens: int = 64, dtype=torch.bfloat16,
                   device="cuda") -> PagedKV:
    """An empty paged cache; ``dtype`` picks the page format."""
    _need(dtype in _PAGE_FORMAT, "pages are fp16, bf16, float8_e4m3fn, int8, float4_e2m1fn_x2 or uint8 (INT4)")
    shape = (n_pages, heads, page_tokens)
    four = dtype in _FOUR

    def codes():
        return torch.empty((*shape, D // 2 if four else D), dtype=dtype, device=device)

    def scales():
        return None if dtype in _WIDE else torch.empty(shape, dtype=torch.float32, device=device)

    def groups():
        return torch.empty((*shape, D // GROUP), dtype=torch.float8_e4m3fn, device=device) if four else None
    return PagedKV(codes(), codes(), scales(), scales(), groups(), groups())


def page_write(kv: PagedKV, K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, *,
               rope: RopeTable | None = None, positions: torch.Tensor | None = None,
               status: torch.Tensor | None = None, stream=None) -> None:
    """Store new tokens K and V [n][heads][128] at ``slots`` (int64 [n]: page * page_tokens +
    row; negative: skipped), rounded to the pages' format; with ``rope`` the keys are first
    turned by their positions."""
    dev = _gpu(K, "K")
    n, heads, kt, kh = _rows(K, "K", dev)
    vn, v_heads, vt, vh = _rows(V, "V", dev)
    _need(kv.gpu == dev, "the pages must be on the GPU of K and V")
    _need(vn == n and v_heads == heads == kv.heads and K.dtype == V.dtype,
          "K and V must be [n][heads][128] of one type, with the heads of the pages")
    _index(slots, torch.int64, (n,), "slots", dev)
    _need((rope is None) == (positions is None), "rope and positions go together")
    _need(rope is None or rope.freqs.get_device() == dev, "the table must be on the GPU of K and V")
    _check_scratch(status, None, dev)
    prm = _c.qvg_page_write_params(n, heads, D, kv.page_tokens, kv.format, kv.n_pages,
                                   _DT[K.dtype], kt, kh, vt, vh)
    rc = _c.qvg_page_write(prm, K.data_ptr(), V.data_ptr(), slots.data_ptr(),
                           None if rope is None else rope.rotary(positions, n), kv._buffers,
                           _ptr(status), _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_page_write")


def _tables(page_table, seq_lens, dev: int):
    shape = page_table.shape
    _need(len(shape) == 2 and shape[0] > 0 and shape[1] > 0, "page_table must be [sequences][pages], one of each at least")
    _index(page_table, torch.int32, shape, "page_table", dev)
    _index(seq_lens, torch.int32, shape[:1], "seq_lens", dev)
    return shape[0], shape[1]


def page_read(kv: PagedKV, page_table: torch.Tensor, seq_lens: torch.Tensor, count: int, *,
              first: int = 0, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
              status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Tokens [first, first + count) of every sequence as [sequences][2 * heads][count][128],
    keys and values interleaved: ``out[b]`` is an X of ``quantize``.  Rows past a sequence's
    length are zeros.  ``out`` may have larger sequence and tensor strides."""
    dev = _gpu(kv.k, "pages")
    n_seqs, max_pages = _tables(page_table, seq_lens, dev)
    _check_scratch(status, None, dev)
    shape = (n_seqs, 2 * kv.heads, count, D)
    if out is None:
        _need(out_dtype in _DT, "out_dtype must be fp16, bf16 or fp32")
        out = _empty(shape, out_dtype, kv.k.device, stream)
        stride = (2 * kv.heads * count * D, count * D)
    else:
        stride = out.stride()
        _need(out.get_device() == dev and out.shape == shape and out.dtype in _DT and
              (count == 0 or (stride[3] == 1 and (count == 1 or stride[2] == D))),
              "out must be [sequences][2 * heads][count][128] on the pages' GPU, with contiguous tokens")
    prm = _c.qvg_page_read_params(n_seqs, kv.heads, D, kv.page_tokens, kv.format, _DT[out.dtype],
                                  kv.n_pages, max_pages, first, count,
                                  stride[0] if n_seqs > 1 else 0, stride[1])
    rc = _c.qvg_page_read(prm, kv._buffers, page_table.data_ptr(), seq_lens.data_ptr(),
                          out.data_ptr(), _ptr(status), _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_page_read")
    return out


def page_attention(Q: torch.Tensor, kv: PagedKV, page_table: torch.Tensor,
                   seq_lens: torch.Tensor, *, cu_q: torch.Tensor | None = None,
                   max_q: int | None = None, max_kv: int | None = None, causal: bool = True,
                   window: int = 0, scale: float | None = None, out_dtype=None,
                   out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                   return_lse: bool = False, workspace: torch.Tensor | None = None,
                   status: torch.Tensor | None = None, stream=None):
    """Attention of new tokens Q [total_q][q_heads][128] (fp16 / bf16) over the pages
    (qvg_page_attention).  ``seq_lens`` counts each sequence's cached tokens, the queries' own
    among them; ``cu_q`` (int32 [sequences + 1]) holds where each one's queries start, and
    ``max_q`` a bound on their number; without ``cu_q`` every sequence has total_q / sequences.
    ``max_kv`` (about the longest sequence, the page table's capacity by default) sizes the
    split of the work.  Returns the output, and with ``return_lse`` the fp32 log-sum-exp
    [total_q][q_heads] beside it."""
    dev = _gpu(Q, "Q")
    total, q_heads, qt, qh = _rows(Q, "Q", dev)
    n_seqs, max_pages = _tables(page_table, seq_lens, dev)
    _need(kv.gpu == dev, "the pages must be on the GPU of Q")
    _check_scratch(status, workspace, dev)
    if cu_q is None:
        _need(total % n_seqs == 0 and (max_q is None or max_q == total // n_seqs),
              "without cu_q every sequence has total_q / sequences queries")
        max_q = total // n_seqs
    else:
        _index(cu_q, torch.int32, (n_seqs + 1,), "cu_q", dev)
        max_q = total if max_q is None else max_q
    if out is None:
        out = _empty_as(Q, (total, q_heads, D), Q.dtype if out_dtype is None else out_dtype, stream)
        ot, oh = q_heads * D, D
    else:
        on, o_heads, ot, oh = _rows(out, "out", dev)
        _need(on == total and o_heads == q_heads, "out must have the shape of Q")
    if lse is None and return_lse:
        lse = _empty((total, q_heads), torch.float32, Q.device, stream)
    elif lse is not None:
        _index(lse, torch.float32, (total, q_heads), "lse", dev)
    prm = _c.qvg_page_attention_params(
        n_seqs, q_heads, kv.heads, D, kv.page_tokens, kv.format, _DT[Q.dtype], _DT[out.dtype],
        kv.n_pages, max_pages, 1 if causal else 0, window, total, max_q,
        max_pages * kv.page_tokens if max_kv is None else max_kv,
        D ** -0.5 if scale is None else scale, qt, qh, ot, oh)
    if workspace is None:
        need = _c.qvg_page_attention_workspace_bytes(prm)
        if need:
            workspace = _empty((need,), torch.uint8, Q.device, stream)
    rc = _c.qvg_page_attention(prm, Q.data_ptr(), kv._buffers, page_table.data_ptr(),
                               seq_lens.data_ptr(), _ptr(cu_q), out.data_ptr(), _ptr(lse),
                               _ptr(workspace), 0 if workspace is None else workspace.numel(),
                               _ptr(status), _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_page_attention")
    return (out, lse) if return_lse else out


# ------------------------------------------------------------------------------------
# The pages of sequences.  refs (int32 [pages]) counts the table entries that name a page, 0 is
# free; refs, page_table and seq_lens change on the device, in stream order.  Pages are taken in
# ascending order, for sequences in order: every run has the same outcome.  Where first tokens are
# dropped (a sliding window), ``starts`` (int64 [sequences], zeros at first) goes into page_append,
# page_fork and page_free: the position of each sequence's first token, from which new ones count on.
# ------------------------------------------------------------------------------------

def _book(kv: PagedKV, refs, page_table, seq_lens, status, workspace, total: int = 0, out_pages: int = 0, starts=None):
    """(GPU, sequences, entries of a row, parameters) of a call on the pages of sequences."""
    dev, shape = kv.gpu, page_table.shape
    # (one condition for what is as it should be, the checks one by one for what is not)
    if not (dev >= 0 and dev == torch._C._cuda_getDevice() and len(shape) == 2 and seq_lens.dim() == refs.dim() == 1
            and len(seq_lens) == shape[0] > 0 < shape[1] and len(refs) == kv.n_pages
            and page_table.dtype is torch.int32 is seq_lens.dtype is refs.dtype
            and page_table.get_device() == seq_lens.get_device() == refs.get_device() == dev
            and page_table.is_contiguous() and seq_lens.is_contiguous() and refs.is_contiguous()):
        dev = _gpu(kv.k, "pages")
        _tables(page_table, seq_lens, dev)
        _index(refs, torch.int32, (kv.n_pages,), "refs", dev)
    _check_scratch(status, workspace, dev)
    n_seqs, max_pages = shape
    if starts is not None:
        _index(starts, torch.int64, shape[:1], "starts", dev)
    return dev, n_seqs, max_pages, _c.qvg_page_table_params(n_seqs, kv.heads, D, kv.page_tokens, kv.format, max_pages,
                                                            kv.n_pages, total, out_pages, _ptr(starts))


def _book_workspace(prm, kv: PagedKV, workspace, stream):
    """The workspace, which has to live as long as the call, its address and its bytes."""
    if workspace is None:
        if prm.n_seqs <= _c.QVG_FEW_SEQS and not prm.out_pages:
            return None, None, 0
        need = _c.qvg_page_table_workspace_bytes(prm)
        if not need:
            return None, None, 0
        workspace = _empty((need,), torch.uint8, kv.k.device, stream)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _same_pages(kv: PagedKV, out: PagedKV, dev: int):
    _need(out.gpu == dev and out.heads == kv.heads and out.page_tokens == kv.page_tokens and out.format == kv.format,
          "out must be pages of the same heads, page_tokens and format, on the same GPU")


def page_copy(kv: PagedKV, src: torch.Tensor, dst: torch.Tensor, *, rows: torch.Tensor | None = None,
              out: PagedKV | None = None, status: torch.Tensor | None = None, stream=None) -> None:
    """Copy pages ``src`` to ``dst`` (int32 [n]; negative: skipped), of all heads, keys and values
    with their scales, the first ``rows`` tokens of each (int32 [n]) or all.  ``out`` is the pool of
    ``dst``, ``kv`` itself by default.  No page may be written twice, nor, in one pool, be written and
    read."""
    dev = _gpu(kv.k, "pages")
    n = src.shape[0] if src.dim() == 1 else -1
    _index(src, torch.int32, (n,), "src", dev)
    _index(dst, torch.int32, (n,), "dst", dev)
    if rows is not None:
        _index(rows, torch.int32, (n,), "rows", dev)
    if out is None:
        out = kv
    else:
        _same_pages(kv, out, dev)
    if status is not None:
        _check_scratch(status, None, dev)
    rc = _c.qvg_page_copy(kv._copy_params, n, kv._buffers, src.data_ptr(), dst.data_ptr(), _ptr(rows), out._buffers,
                          out.n_pages, _ptr(status), _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_page_copy")


def page_append(kv: PagedKV, refs: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                counts: torch.Tensor, total: int, *, starts: torch.Tensor | None = None, copies: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None):
    """Let sequence b grow by ``counts[b]`` tokens (int32 [sequences]), ``total`` in all, taking free
    pages where its own are full (qvg_page_append).  Returns the new tokens' slots and positions
    (int64 [total], sequence after sequence) for ``page_write`` and ``rope``.  Positions count from
    ``starts``; without it they are places in the sequence, which are none to turn by once first tokens
    were dropped.  A part-filled last page
    that others share is replaced by a copy first, recorded in ``copies`` (int32 [3][sequences]: source,
    destination, rows) if given, with which ``page_copy`` does the same for another layer's pages.  A
    sequence for which pages do not suffice stays as it is, its slots are -1 and ``status`` gets
    QVG_DEV_NO_PAGES."""
    dev, n_seqs, _, prm = _book(kv, refs, page_table, seq_lens, status, workspace, total=total, starts=starts)
    _index(counts, torch.int32, (n_seqs,), "counts", dev)
    _need(total >= 0, "total must not be negative")
    if copies is not None:
        _index(copies, torch.int32, (3, n_seqs), "copies", dev)
    workspace, scratch, size = _book_workspace(prm, kv, workspace, stream)
    slots, positions = (_empty((total,), torch.int64, kv.k.device, stream) for _ in range(2))
    rc = _c.qvg_page_append(prm, kv._buffers, refs.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
                            counts.data_ptr(), slots.data_ptr(), positions.data_ptr(), _ptr(copies),
                            scratch, size, _ptr(status), _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_page_append")
    return slots, positions


def page_fork(kv: PagedKV, refs: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
              parents: torch.Tensor, *, starts: torch.Tensor | None = None, copies: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Let the empty sequence b begin as a fork of sequence ``parents[b]`` (int32 [sequences],
    negative: none): whole pages are shared, a part-filled last one is copied, ``starts[b]`` becomes
    the parent's (qvg_page_fork).
    Returns the copies made (int32 [4][sequences]: source, destination, rows, and whole pages shared, -1
    where there is no fork), with which ``page_copy`` does the same for another layer's pages."""
    dev, n_seqs, _, prm = _book(kv, refs, page_table, seq_lens, status, workspace, starts=starts)
    _index(parents, torch.int32, (n_seqs,), "parents", dev)
    if copies is None:
        copies = _empty((4, n_seqs), torch.int32, kv.k.device, stream)
    else:
        _index(copies, torch.int32, (4, n_seqs), "copies", dev)
    workspace, scratch, size = _book_workspace(prm, kv, workspace, stream)
    rc = _c.qvg_page_fork(prm, kv._buffers, refs.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
                          parents.data_ptr(), copies.data_ptr(), scratch, size, _ptr(status),
                          _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_page_fork")
    return copies


def page_free(kv: PagedKV, refs: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor, *,
              first: torch.Tensor | None = None, last: torch.Tensor | None = None,
              starts: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> None:
    """Sequence b gives up its ``first[b]`` oldest tokens, as far as they fill whole pages, and its
    ``last[b]`` newest (int32 [sequences] each; past the length: all), and the pages that hold
    nothing else of it (qvg_page_free).  Its entries move to the front of its row, and ``starts[b]``
    grows by the first tokens given up, or becomes 0 where all that it has goes as its newest."""
    dev, n_seqs, _, prm = _book(kv, refs, page_table, seq_lens, status, None, starts=starts)
    _need(first is not None or last is not None, "first or last says how many tokens go")
    for t, what in ((first, "first"), (last, "last")):
        if t is not None:
            _index(t, torch.int32, (n_seqs,), what, dev)
    rc = _c.qvg_page_free(prm, refs.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), _ptr(first), _ptr(last),
                          _ptr(status), _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_page_free")


def page_compact(kv: PagedKV, refs: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                 out: PagedKV, *, workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                 stream=None):
    """Copy the pages in use to the front of another pool ``out``, in order (qvg_page_compact).
    Returns the page table and the refs for it, and the number of pages in use (int32 [1]).  The first
    pool with its table and refs stays as it is; what ``out`` has no room for is left out, with
    QVG_DEV_NO_PAGES."""
    dev, n_seqs, max_pages, prm = _book(kv, refs, page_table, seq_lens, status, workspace, out_pages=out.n_pages)
    _same_pages(kv, out, dev)
    workspace, scratch, size = _book_workspace(prm, kv, workspace, stream)
    table = _empty_as(page_table, (n_seqs, max_pages), torch.int32, stream)
    new_refs = _empty((out.n_pages,), torch.int32, kv.k.device, stream)
    live = _empty((1,), torch.int32, kv.k.device, stream)
    rc = _c.qvg_page_compact(prm, kv._buffers, refs.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), out._buffers,
                             table.data_ptr(), new_refs.data_ptr(), live.data_ptr(), scratch, size,
                             _ptr(status), _stream_handle(stream))
    if rc != _c.QVG_OK:
        raise _c.QVGError(rc, "qvg_page_compact")
    return table, new_refs, live
