"""Convenience wrapper over the C ABI: a KV cache whose device buffers are torch allocations.

Next to it, the operators around the attention: rotary positions of q and k (AxisRope), layer norm with
modulation (layer_norm, layer_norm_backward) and the linear layers with INT8 and 4-bit weights.

Only allocation (torch), stream selection and argument marshalling happen here; the quantise-append,
mask build, attention and these operators all run in libnomas's kernels.

No call records an autograd graph, whatever its inputs require: results carry no gradient function, and a
tensor written through out= keeps its version.  Gradients are calls of their own: layer_norm_backward, and
AxisRope with inverse=True.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence, Tuple

import torch

from . import _nomas as N


def _stream_handle(stream: Optional[torch.cuda.Stream]) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _bf16_strides(t: torch.Tensor) -> Tuple[int, int]:
    if t.dtype != torch.bfloat16 or t.dim() != 3 or t.stride(2) != 1:
        raise ValueError("expected a bf16 [tokens, heads, head_dim] tensor with contiguous head_dim")
    return t.stride(0), t.stride(1)


_DTYPES = {torch.float32: N.NOMAS_DTYPE_F32, torch.bfloat16: N.NOMAS_DTYPE_BF16}


_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _pitch(t: torch.Tensor) -> int:
    """Row pitch of a matrix; a single row's own stride says nothing."""
    return t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 8) * 8


def _split_rows(t: torch.Tensor) -> bool:
    """Whether a matrix' rows are not contiguous; a single column's stride says nothing."""
    return t.stride(1) != 1 and t.shape[1] != 1


def _same_device(ref: torch.Tensor, *others: Optional[torch.Tensor]) -> None:
    index = ref.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on {ref.device} and {t.device}: expected one device")


class _on:
    """Runs a call on the device of `ref`, on `stream` (allocations then belong to it) or the device's current
    stream; _stream_on skips it where neither has to change."""

    __slots__ = ("guards",)

    def __init__(self, ref: torch.Tensor, stream: Optional[torch.cuda.Stream]):
        if stream is not None and stream.device != ref.device:
            raise ValueError(f"a stream of {stream.device} for tensors on {ref.device}")
        self.guards = (torch.cuda.device(ref.device),) + ((torch.cuda.stream(stream),) if stream is not None else ())

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _stream_on(ref: torch.Tensor, stream: Optional[torch.cuda.Stream]) -> Optional[int]:
    """The current stream of `ref`'s device as an address, or None when a call needs _on first."""
    index = ref.get_device()
    if index < 0 or not ref.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {ref.device}")
    if stream is not None or index != _current_device():
        return None
    return _raw_stream(index)


def segment_text(n_frames: int, head_len: int, tails: Sequence[Tuple[int, int, int]] = ()):
    return N.make_segment_text(n_frames, head_len, [tuple(t) for t in tails])


def segment_text_of(seg) -> "N.nomas_segment_text":
    """From a workloads.SegmentText."""
    return segment_text(seg.n_frames, seg.head_len, [(t.len, t.f0, t.f1) for t in seg.tails])


class KVCache:
    """INT8 history ring + description-head store on one device (see include/nomas.h)."""

    def __init__(self, heads: int, head_dim: int, tokens_per_frame: int, window_frames: int,
                 capacity_frames: int, head_store_tokens: int, device="cuda", stream=None):
        self.dims = N.make_dims(heads, head_dim, tokens_per_frame, window_frames, capacity_frames,
                                head_store_tokens)
        total, sizes = N.nomas_kv_cache_bytes(self.dims)
        if total == 0:
            raise ValueError("invalid cache dimensions")
        self.device = torch.device(device)
        self.sizes = sizes
        self.bufs = [torch.empty(max(s, 16), dtype=torch.uint8, device=self.device) for s in sizes]
        self.handle = N.nomas_kv_cache_init(self.dims, [b.data_ptr() for b in self.bufs], _stream_handle(stream))
        self.H, self.D, self.T = heads, head_dim, tokens_per_frame
        self.C, self.HS = capacity_frames, head_store_tokens

    @classmethod
    def for_config(cls, cfg, device="cuda"):
        return cls(cfg.heads, cfg.head_dim, cfg.tokens_per_frame, cfg.window_frames, cfg.capacity_frames,
                   cfg.head_store_tokens, device)

    def __del__(self, _destroy=N.nomas_kv_cache_destroy):
        # the destroy function is bound at definition time: module globals may already be gone when
        # the interpreter shuts down
        h = getattr(self, "handle", None)
        if h:
            _destroy(h)
            self.handle = None

    # ---- raw buffer views (for tests and diagnostics) -----------------------------------------
    def _view(self, i, dtype, shape):
        n = math.prod(shape) * torch.tensor([], dtype=dtype).element_size()
        return self.bufs[i][:n].view(dtype).view(*shape)

    def ring_k8(self):
        return self._view(N.NOMAS_BUF_K8, torch.int8, (self.H, self.C * self.T, self.D))

    def ring_v8(self):
        return self._view(N.NOMAS_BUF_V8, torch.int8, (self.H, self.C * self.T, self.D))

    def ring_ks(self):
        return self._view(N.NOMAS_BUF_KS, torch.float32, (self.H, self.C * self.T))

    def ring_vs(self):
        return self._view(N.NOMAS_BUF_VS, torch.float32, (self.H, self.C * self.T))

    def head_k8(self):
        return self._view(N.NOMAS_BUF_HK8, torch.int8, (self.H, self.HS, self.D))

    def head_v8(self):
        return self._view(N.NOMAS_BUF_HV8, torch.int8, (self.H, self.HS, self.D))

    def head_ks(self):
        return self._view(N.NOMAS_BUF_HKS, torch.float32, (self.H, self.HS))

    def head_vs(self):
        return self._view(N.NOMAS_BUF_HVS, torch.float32, (self.H, self.HS))

    # ---- operations ------------------------------------------------------------------------------
    def state(self):
        return N.nomas_kv_cache_state(self.handle)

    def append(self, k: Optional[torch.Tensor], v: Optional[torch.Tensor], n_frames: int,
               head_k: Optional[torch.Tensor] = None, head_v: Optional[torch.Tensor] = None, stream=None):
        ref = k if k is not None else head_k
        ts, hs = _bf16_strides(ref)
        for t in (v, head_k, head_v):
            if t is not None and _bf16_strides(t) != (ts, hs):
                raise ValueError("all K/V tensors of one append must share strides")
        head_len = 0 if head_k is None else head_k.shape[0]
        rc = N.nomas_kv_append(self.handle, k.data_ptr() if k is not None else 0,
                               v.data_ptr() if v is not None else 0, ts, hs, n_frames,
                               head_k.data_ptr() if head_k is not None else 0,
                               head_v.data_ptr() if head_v is not None else 0, head_len, _stream_handle(stream))
        N._check(rc, "nomas_kv_append")

    def mask_layout(self, seg, mode=N.NOMAS_MODE_DENSE, keep_frac=0.25):
        return N.nomas_mask_layout_query(self.handle, seg, mode, keep_frac)

    def build_mask(self, seg, mode=N.NOMAS_MODE_DENSE, keep_frac=0.25, q=None, kcur=None, mask_buf=None,
                   stream=None):
        lay = self.mask_layout(seg, mode, keep_frac)
        if mask_buf is None:
            mask_buf = torch.empty(lay["total_bytes"], dtype=torch.uint8, device=self.device)
        ts = hs = 8
        if mode == N.NOMAS_MODE_SPARSE:
            ts, hs = _bf16_strides(q)
            if _bf16_strides(kcur) != (ts, hs):
                raise ValueError("q and kcur must share strides")
        rc = N.nomas_mask_build(self.handle, seg, mode, keep_frac, q.data_ptr() if q is not None else 0,
                                kcur.data_ptr() if kcur is not None else 0, ts, hs, mask_buf.data_ptr(),
                                _stream_handle(stream))
        N._check(rc, "nomas_mask_build")
        return mask_buf, lay

    def workspace(self, seg):
        """A device buffer of the size nomas_attn_fwd needs for this segment (torch-allocated)."""
        n = N.nomas_attn_workspace_bytes(self.handle, seg)
        if n == 0:
            raise ValueError("invalid segment text")
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def attention(self, seg, mask_buf, q, kcur, vcur, ktxt, vtxt, softmax_scale=None, mode=N.NOMAS_MODE_DENSE,
                  keep_frac=0.25, out=None, lse=None, want_lse=False, workspace=None, stream=None):
        ts, hs = _bf16_strides(q)
        for t in (kcur, vcur) + ((ktxt, vtxt) if ktxt is not None and ktxt.shape[0] else ()):
            if _bf16_strides(t) != (ts, hs):
                raise ValueError("all bf16 inputs of one attention call must share strides")
        nq, H, D = q.shape
        if out is None:
            out = torch.empty((nq, H, D), dtype=torch.float32, device=self.device)
        if lse is None and want_lse:
            lse = torch.empty((H, nq), dtype=torch.float32, device=self.device)
        scale = softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(D)
        has_txt = ktxt is not None and ktxt.shape[0] > 0
        if workspace is None:
            workspace = self.workspace(seg)
        rc = N.nomas_attn_fwd(self.handle, seg, mode, keep_frac, mask_buf.data_ptr(), q.data_ptr(),
                              kcur.data_ptr(), vcur.data_ptr(), ktxt.data_ptr() if has_txt else 0,
                              vtxt.data_ptr() if has_txt else 0, ts, hs, scale, out.data_ptr(),
                              lse.data_ptr() if lse is not None else 0, workspace.data_ptr(),
                              _stream_handle(stream))
        N._check(rc, "nomas_attn_fwd")
        return out, lse

    # ---- archive of evicted frames and selection of the retained history ------------------------
    def record_bytes(self) -> int:
        return N.nomas_kv_frame_record_bytes(self.dims)

    def retained(self):
        return N.nomas_kv_retained(self.handle)

    def evicted_by(self, n_frames: int):
        return N.nomas_kv_evicted_by(self.handle, n_frames)

    def archive(self, frame: int, record: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Copy retained `frame` into a host record (a pinned uint8 tensor, allocated when not given)."""
        if record is None:
            record = torch.empty(self.record_bytes(), dtype=torch.uint8).pin_memory()
        N._check(N.nomas_kv_archive(self.handle, frame, record.data_ptr(), _stream_handle(stream)), "nomas_kv_archive")
        return record

    def select(self, frames, records: Optional[dict] = None, stream=None):
        """Make `frames` the retained history (age order); records: frame -> host record for frames that
        are not retained now."""
        recs = None if records is None else [records[f].data_ptr() if f in records else 0 for f in frames]
        N._check(N.nomas_kv_select(self.handle, list(frames), recs, _stream_handle(stream)), "nomas_kv_select")

    def dequant(self, stream=None):
        st = self.state()
        n = st["history_tokens"]
        k = torch.empty((n, self.H, self.D), dtype=torch.float32, device=self.device)
        v = torch.empty_like(k)
        N._check(N.nomas_kv_dequant(self.handle, k.data_ptr(), v.data_ptr(), _stream_handle(stream)),
                 "nomas_kv_dequant")
        return k, v

    def status(self, stream=None) -> int:
        return N.nomas_device_status(self.handle, _stream_handle(stream))


def mask_views(mask_buf: torch.Tensor, lay: dict):
    """Class map, kept candidates and scores inside a mask buffer (device tensors)."""
    nqb, nt, H, keep, nc = lay["n_qblocks"], lay["n_tiles"], lay["heads"], lay["keep"], lay["n_cand"]
    cls = mask_buf[lay["off_class"]:lay["off_class"] + nqb * nt].view(torch.int8).view(nqb, nt)
    out = {"class": cls}
    if lay["mode"] == N.NOMAS_MODE_SPARSE:
        out["sel"] = mask_buf[lay["off_sel"]:lay["off_sel"] + H * nqb * keep * 4].view(torch.int32).view(H, nqb, keep)
        out["score"] = mask_buf[lay["off_score"]:lay["off_score"] + H * nqb * nc * 4].view(torch.float32).view(
            H, nqb, nc)
    nl, cap = lay["n_lists"], lay["list_cap"]
    out["count"] = mask_buf[lay["off_count"]:lay["off_count"] + nl * 4].view(torch.int32)
    out["list"] = mask_buf[lay["off_list"]:lay["off_list"] + nl * cap * 16].view(torch.int32).view(nl, cap, 4)
    return out


class Int8Linear:
    """A DiT linear layer with INT8 weights and float scales per output channel, computed in BF16
    (include/nomas.h): codes int8 [N][K] and scales fp32 [N] stay resident; every call dequantises the
    codes into a transient bf16 workspace and runs the tensor-core GEMM y = x W^T."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dtype != torch.int8 or codes.dim() != 2 or not codes.is_contiguous():
            raise ValueError("codes: contiguous int8 [N, K]")
        if scales.dtype != torch.float32 or scales.shape != (codes.shape[0],):
            raise ValueError("scales: float32 [N]")
        self.codes, self.scales = codes, scales
        self.n_out, self.k_in = codes.shape
        self.workspace = torch.empty(N.nomas_w8a16_workspace_bytes(self.n_out, self.k_in), dtype=torch.uint8,
                                     device=codes.device)
        self.status_word = torch.zeros(4, dtype=torch.int32, device=codes.device)

    @classmethod
    def from_weights(cls, w: torch.Tensor, stream=None) -> "Int8Linear":
        """Quantise bf16 weights [N, K] on the device."""
        if w.dtype != torch.bfloat16 or w.dim() != 2 or w.stride(1) != 1:
            raise ValueError("w: bf16 [N, K] with contiguous rows")
        n, k = w.shape
        codes = torch.empty((n, k), dtype=torch.int8, device=w.device)
        scales = torch.empty(n, dtype=torch.float32, device=w.device)
        N._check(N.nomas_w8_quantize(w.data_ptr(), n, k, w.stride(0), codes.data_ptr(), scales.data_ptr(),
                                     _stream_handle(stream)), "nomas_w8_quantize")
        return cls(codes, scales)

    def dequantized(self, stream=None) -> torch.Tensor:
        w = torch.empty((self.n_out, self.k_in), dtype=torch.bfloat16, device=self.codes.device)
        N._check(N.nomas_w8_dequant(self.codes.data_ptr(), self.scales.data_ptr(), self.n_out, self.k_in,
                                    w.data_ptr(), _stream_handle(stream)), "nomas_w8_dequant")
        return w

    def __call__(self, x: torch.Tensor, out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1 or x.shape[1] != self.k_in:
            raise ValueError("x: bf16 [M, K] with contiguous rows")
        m = x.shape[0]
        if out is None:
            out = torch.empty((m, self.n_out), dtype=out_dtype, device=x.device)
        dt = N.NOMAS_DTYPE_BF16 if out.dtype == torch.bfloat16 else N.NOMAS_DTYPE_F32
        N._check(N.nomas_w8a16_linear(x.data_ptr(), m, self.k_in, x.stride(0), self.codes.data_ptr(),
                                      self.scales.data_ptr(), self.n_out, out.data_ptr(), out.stride(0), dt,
                                      self.workspace.data_ptr(), self.status_word.data_ptr(),
                                      _stream_handle(stream)), "nomas_w8a16_linear")
        return out

    def status(self, stream=None) -> int:
        return N.nomas_status_read(self.status_word.data_ptr(), _stream_handle(stream))


class Int4Linear:
    """A linear layer with 4-bit weights and bf16 group scales, computed in BF16 (include/nomas.h): codes
    uint8 [N][K / 2] (even column in the low half, stored + 8) and scales bf16 [N][ceil(K / group)] stay
    resident.  Few rows of x read every code once and widen it in registers; more rows dequantise into a
    transient bf16 workspace (allocated by the call) and run the tensor-core GEMM."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, group: int = 64):
        if codes.dtype != torch.uint8 or codes.dim() != 2 or not codes.is_contiguous() or codes.shape[1] % 16:
            raise ValueError("codes: contiguous uint8 [N, K / 2], K a multiple of 32")
        self.n_out, self.k_in = codes.shape[0], 2 * codes.shape[1]
        if group not in (32, 64, 128):
            raise ValueError("group: 32, 64 or 128")
        if scales.dtype != torch.bfloat16 or scales.shape != (self.n_out, -(-self.k_in // group)) or \
                not scales.is_contiguous() or scales.device != codes.device:
            raise ValueError("scales: contiguous bfloat16 [N, ceil(K / group)] on the device of codes")
        self.codes, self.scales, self.group = codes, scales, group
        self.status_word = torch.zeros(4, dtype=torch.int32, device=codes.device)

    @classmethod
    def from_weights(cls, w: torch.Tensor, group: int = 64, stream=None) -> "Int4Linear":
        """Quantise bf16 weights [N, K] on the device."""
        if w.dtype != torch.bfloat16 or w.dim() != 2 or w.stride(1) != 1 or w.shape[1] % 32 or group not in (32, 64, 128):
            raise ValueError("w: bf16 [N, K] with contiguous rows, K a multiple of 32; group: 32, 64 or 128")
        st = _stream_on(w, stream)
        if st is None:
            with _on(w, stream):
                return cls.from_weights(w, group)
        n, k = w.shape
        codes = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((n, -(-k // group)), dtype=torch.bfloat16, device=w.device)
        # a single row's own stride says nothing
        N._check(N.nomas_w4_quantize(w.data_ptr(), n, k, w.stride(0) if n > 1 else k, group, codes.data_ptr(),
                                     scales.data_ptr(), st), "nomas_w4_quantize")
        return cls(codes, scales, group)

    def dequantized(self, stream=None) -> torch.Tensor:
        st = _stream_on(self.codes, stream)
        if st is None:
            with _on(self.codes, stream):
                return self.dequantized()
        w = torch.empty((self.n_out, self.k_in), dtype=torch.bfloat16, device=self.codes.device)
        N._check(N.nomas_w4_dequant(self.codes.data_ptr(), self.scales.data_ptr(), self.group, self.n_out, self.k_in,
                                    w.data_ptr(), st), "nomas_w4_dequant")
        return w

    def __call__(self, x: torch.Tensor, out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        st = _stream_on(self.codes, stream)
        if st is None:
            with _on(self.codes, stream):
                return self(x, out_dtype, out)
        codes, n, k, shape, strides = self.codes, self.n_out, self.k_in, x.shape, x.stride()
        if x.dtype is not torch.bfloat16 or len(shape) != 2 or shape[1] != k or strides[1] != 1:
            raise ValueError("x: bf16 [M, K] with contiguous rows")
        m = shape[0]
        _same_device(codes, x, out)
        dtype = _DTYPES.get(out_dtype if out is None else out.dtype)
        if dtype is None or (out is not None and (out.shape != (m, n) or _split_rows(out))):
            raise ValueError("out: bf16 or fp32 [M, N] with contiguous rows")
        if out is None:
            out, ldy = x.new_empty((m, n), dtype=out_dtype), n
        else:
            ldy = _pitch(out)
        if m:
            ws = 0
            if m > N.NOMAS_W4_FEW_ROWS:
                need = N.nomas_w4a16_workspace_bytes(m, n, k, dtype)
                if need:
                    keep = x.new_empty(need, dtype=torch.uint8)
                    ws = keep.data_ptr()
            # a single row's own stride says nothing
            rc = N.lib.nomas_w4a16_linear(x.data_ptr(), m, k, strides[0] if m > 1 else k, codes.data_ptr(), self.scales.data_ptr(),
                                          self.group, n, out.data_ptr(), ldy, dtype, ws, self.status_word.data_ptr(), st)
            if rc:
                N._check(rc, "nomas_w4a16_linear")
        return out

    def status(self, stream=None) -> int:
        st = _stream_on(self.codes, stream)
        if st is None:
            with _on(self.codes, stream):
                return self.status()
        return N.nomas_status_read(self.status_word.data_ptr(), st)


# ------------------------------------------------------------------------------------------------
# rotary positions
# ------------------------------------------------------------------------------------------------

def rope_grid(grid_h: int, grid_w: int, origin=(0.0, 0.0, 0.0), step=(1.0, 1.0, 1.0)) -> "N.nomas_rope_grid":
    """Positions of video tokens in memory order: token n is frame n // (grid_h * grid_w), then row, then
    column, at origin + step * index on the time, height and width axes."""
    return N.make_rope_grid(grid_h, grid_w, tuple(origin), tuple(step))


class AxisRope:
    """Rotary positions over (time, height, width) for q and k (include/nomas.h).  axis_dims: channels of a
    head that each axis turns; the channels behind them pass through."""

    def __init__(self, head_dim: int, axis_dims: Sequence[int], theta: float = 10000.0, pairing: str = "interleaved"):
        if pairing not in ("interleaved", "halves"):
            raise ValueError("pairing: 'interleaved' or 'halves'")
        if len(axis_dims) != 3:
            raise ValueError("axis_dims: channels of time, height and width")
        self.head_dim = head_dim
        self.spec = N.make_rope_spec(head_dim, axis_dims, theta,
                                     N.NOMAS_ROPE_HALVES if pairing == "halves" else N.NOMAS_ROPE_INTERLEAVED)
        self._spec = ctypes.byref(self.spec)

    def __call__(self, tensors, grid=None, positions: Optional[torch.Tensor] = None, inverse: bool = False, out=None,
                 stream=None):
        """Rotate one [tokens, heads, head_dim] tensor (bf16 or fp32) or a sequence of them (q and k: one
        launch), at the positions of `grid` (rope_grid) or `positions` (fp32 [tokens, 3]).  inverse: the
        inverse rotation, which is also the gradient.  out: tensors to write (x itself: in place)."""
        single = isinstance(tensors, torch.Tensor)
        xs = (tensors,) if single else tuple(tensors)
        if not 1 <= len(xs) <= N.NOMAS_ROPE_MAX_TENSORS:
            raise ValueError(f"1 to {N.NOMAS_ROPE_MAX_TENSORS} tensors")
        ref = xs[0]
        st = _stream_on(ref, stream)
        if st is None:
            with _on(ref, stream):
                return self(tensors, grid, positions, inverse, out)
        dtype = ref.dtype
        if ref.dim() != 3 or dtype not in _DTYPES:
            raise ValueError("expected bf16 or fp32 [tokens, heads, head_dim] tensors with contiguous head_dim")
        if (grid is None) == (positions is None):
            raise ValueError("give either grid or positions")
        t = ref.shape[0]
        if positions is not None:
            if positions.dtype != torch.float32 or positions.shape != (t, 3) or not positions.is_contiguous():
                raise ValueError("positions: contiguous fp32 [tokens, 3]")
            _same_device(ref, positions)
        index, d = ref.get_device(), self.head_dim
        args, ys = [], []
        given = (None,) * len(xs) if out is None else (out,) if isinstance(out, torch.Tensor) else tuple(out)
        if len(given) != len(xs):
            raise ValueError("out: one tensor for each input")
        for x, y in zip(xs, given):
            shape, sx = x.shape, x.stride()
            if len(shape) != 3 or shape[0] != t or shape[2] != d or x.dtype != dtype or sx[2] != 1 or x.get_device() != index:
                raise ValueError("expected tensors [tokens, heads, head_dim] of one device, type and token count with "
                                 "contiguous head_dim")
            h = shape[1]
            if y is None:
                y = torch.empty_like(x, memory_format=torch.contiguous_format)
                sy = (h * d, d)
            else:
                sy = y.stride()
                if y.shape != shape or y.dtype != dtype or sy[2] != 1 or y.get_device() != index:
                    raise ValueError("out: tensors of the inputs' shape, type and device with contiguous head_dim")
            ys.append(y)
            if h:                          # a tensor without heads has nothing to turn
                # a single token's or head's stride says nothing
                args += (x.data_ptr(), y.data_ptr(), sx[0] if t > 1 else 0, sx[1] if h > 1 else 0, sy[0] if t > 1 else 0,
                         sy[1] if h > 1 else 0, h, 0)
        if t and args:
            N._check(N.lib.nomas_rope(self._spec, None if grid is None else ctypes.byref(grid),
                                      None if positions is None else positions.data_ptr(), t, N.pack_rope_tensors(args),
                                      len(args) // 8, _DTYPES[dtype], inverse, st), "nomas_rope")
        return ys[0] if single else tuple(ys)


# ------------------------------------------------------------------------------------------------
# layer norm
# ------------------------------------------------------------------------------------------------

def _norm_params(x, weight, bias, rows_per_group):
    """(pitch, type, groups) of a layer norm's parameters: [C], or [groups, C]."""
    if x.dim() != 2 or x.dtype not in _DTYPES or _split_rows(x):
        raise ValueError("x: bf16 or fp32 [rows, C] with contiguous rows")
    rows, cols = x.shape
    if rows_per_group < 0:
        raise ValueError("rows_per_group: at least 0")
    if weight is None and bias is None:
        return cols, N.NOMAS_DTYPE_F32, -(-rows // rows_per_group) if rows_per_group else 1
    groups = -(-rows // rows_per_group) if rows_per_group else 1
    pitch = dtype = None
    for p in (weight, bias):
        if p is None:
            continue
        shape, strides = p.shape, p.stride()
        if len(shape) == 1:
            shape, strides = (1, *shape), (cols, *strides)
        if shape != (groups, cols) or p.dtype not in _DTYPES or (strides[1] != 1 and cols != 1):
            raise ValueError("weight, bias: bf16 or fp32 [groups, C] ([C] for one group) with contiguous rows")
        at = strides[0] if groups > 1 else cols
        if at < cols:
            raise ValueError("weight, bias: a row of its own for every group, not an expanded or overlapping one")
        if dtype is not None and (at != pitch or p.dtype != dtype):
            raise ValueError("weight and bias must share their type and strides")
        pitch, dtype = at, p.dtype
    return pitch, _DTYPES[dtype], groups


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-6, rows_per_group: int = 0, unit_offset: bool = False, out_dtype=None,
               out: Optional[torch.Tensor] = None, want_stats: bool = False, stream=None):
    """Layer norm of the rows of x [rows, C] (include/nomas.h): xhat * weight + bias, or with unit_offset
    xhat * (1 + weight) + bias (modulation).  rows_per_group: rows that share a row of weight and bias
    ([groups, C], every row its own memory, so no expanded one); 0: one weight and bias [C] for all.  Returns y, or (y, mean, rstd) with want_stats, which
    layer_norm_backward takes."""
    st = _stream_on(x, stream)
    if st is None:
        with _on(x, stream):
            return layer_norm(x, weight, bias, eps, rows_per_group, unit_offset, out_dtype, out, want_stats)
    pitch, p_dtype, _ = _norm_params(x, weight, bias, rows_per_group)
    rows, cols = x.shape
    _same_device(x, weight, bias, out)
    if ((out_dtype or x.dtype) if out is None else out.dtype) not in _DTYPES:
        raise ValueError("out: bf16 or fp32 [rows, C] with contiguous rows")
    if out is None:
        out = torch.empty_like(x, dtype=out_dtype, memory_format=torch.contiguous_format)
    elif out.shape != x.shape or _split_rows(out):
        raise ValueError("out: bf16 or fp32 [rows, C] with contiguous rows")
    mean = rstd = None
    if want_stats:
        mean = x.new_empty(rows, dtype=torch.float32)
        rstd = torch.empty_like(mean)
    if rows:
        N._check(N.lib.nomas_layernorm_fwd(x.data_ptr(), rows, cols, _pitch(x), _DTYPES[x.dtype], _ptr(weight), _ptr(bias),
                                           pitch, p_dtype, rows_per_group, unit_offset, eps, out.data_ptr(), _pitch(out),
                                           _DTYPES[out.dtype], _ptr(mean), _ptr(rstd), st), "nomas_layernorm_fwd")
    return (out, mean, rstd) if want_stats else out


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None, rows_per_group: int = 0, unit_offset: bool = False,
                        want_dx: bool = True, want_params: bool = True, stream=None):
    """Gradients of layer_norm: (dx of x's type, dweight fp32 [groups, C], dbias fp32 [groups, C]); what is not
    wanted is None.  mean and rstd are layer_norm's."""
    st = _stream_on(x, stream)
    if st is None:
        with _on(x, stream):
            return layer_norm_backward(dy, x, mean, rstd, weight, rows_per_group, unit_offset, want_dx, want_params)
    pitch, p_dtype, groups = _norm_params(x, weight, None, rows_per_group)
    rows, cols = x.shape
    if dy.shape != x.shape or dy.dtype not in _DTYPES or _split_rows(dy):
        raise ValueError("dy: bf16 or fp32 [rows, C] with contiguous rows")
    for s in (mean, rstd):
        if s.dtype != torch.float32 or s.shape != (rows,) or not s.is_contiguous():
            raise ValueError("mean, rstd: contiguous fp32 [rows]")
    _same_device(x, dy, mean, rstd, weight)
    dx = torch.empty_like(x, memory_format=torch.contiguous_format) if want_dx else None
    dw = db = ws = None
    if want_params:
        dw = x.new_empty((groups, cols), dtype=torch.float32)
        db = torch.empty_like(dw)
        need = N.lib.nomas_layernorm_workspace_bytes(rows, cols, rows_per_group)
        if need > 16:                                         # 16: nothing to add up across shares
            ws = x.new_empty(need, dtype=torch.uint8)
    if rows and (want_dx or want_params):
        N._check(N.lib.nomas_layernorm_bwd(dy.data_ptr(), _pitch(dy), _DTYPES[dy.dtype], x.data_ptr(), _pitch(x),
                                           _DTYPES[x.dtype], rows, cols, _ptr(weight), pitch, p_dtype, rows_per_group,
                                           unit_offset, mean.data_ptr(), rstd.data_ptr(), _ptr(dx), cols, _ptr(dw),
                                           _ptr(db), cols, _ptr(ws), st), "nomas_layernorm_bwd")
    elif want_params:
        dw.zero_()
        db.zero_()
    return dx, dw, db
