"""Device-resident synthetic layers: torch owns the memory, libmoe does the work.

``DeviceLayer`` draws a layer with ``synth`` (in pinned host chunks, copied
to HBM), opens it through the C ABI and owns a zero-initialised workspace.
Its ``decode`` / ``prefill`` methods only allocate outputs and marshal
pointers to ``moe_decode`` / ``moe_prefill_chunk``.
"""
from __future__ import annotations

import numpy as np
import torch

from . import moe, synth


def bf16_tensor(bits: np.ndarray, device) -> torch.Tensor:
    """bf16 bit patterns (uint16) -> torch.bfloat16 tensor on `device`."""
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)
    return t.to(device)


def bf16_bits(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


_ELEM_TYPE = {torch.bfloat16: moe.MOE_BF16, torch.float16: moe.MOE_F16, torch.float32: moe.MOE_F32}


def _stream(device, stream):
    """`stream`, or the device's current one (the raw handle: building a
    torch.cuda.Stream takes as long as the call itself)."""
    if stream is not None:
        return stream
    return torch._C._cuda_getCurrentRawStream(device.index if device.index is not None else torch.cuda.current_device())


# Calls with stream= run on that stream, given as a raw handle.  The caller has
# it wait for the inputs, keeps them until the work is done, and waits before it
# reads the outputs.  What a wrapper allocates is safe on both streams:

def _other(device, stream):
    """The stream given to a call as torch has it; None if it is the current one."""
    if stream is None or stream == _stream(device, None):
        return None
    return torch.cuda.ExternalStream(stream, device)


def _empty(device, other, dtype, *shape) -> torch.Tensor:
    """Memory that a call on the stream `other` writes.  It is that stream's, as
    work queued on the current one may still use what the current one would
    reuse; and the current one's too, so that it is not reused once freed
    before work queued there by then is done."""
    if other is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(other):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _refuse(where: str, what: str):
    raise moe.MoEError(moe.MOE_ERR_ARG, where, what)


def _type(dtype: torch.dtype, where: str) -> int:
    """The element type's code."""
    code = _ELEM_TYPE.get(dtype)
    if code is None:
        _refuse(where, f"elements of type {dtype}")
    return code


def _matrix(t: torch.Tensor, shape, where: str, name: str) -> None:
    """The library gets addresses only, so shapes are compared here."""
    if t.shape != shape:
        _refuse(where, f"{name} has the shape {tuple(t.shape)}, not {tuple(shape)}")


def _on_gpu(where: str, index: int, *tensors) -> None:
    """All of them (None: no tensor) on the GPU `index`, and that the current
    device, on which the library launches."""
    for t in tensors:
        if t is not None and (index < 0 or t.get_device() != index):
            _refuse(where, f"a tensor is on {t.device}; all must be on the same GPU")
    if index != torch.cuda.current_device():
        _refuse(where, f"the tensors' device {index} must be the current device")


def _ld(t: torch.Tensor, rows: int, cols: int, where: str) -> int:
    """Leading dimension of a [rows][cols] matrix whose rows are contiguous."""
    ld, step = t.stride()
    if step != 1 and cols != 1:
        _refuse(where, f"rows must be contiguous, their elements are {step} apart")
    return ld if rows > 1 else max(ld, cols)


def block_norm(y=None, h=None, gate=None, w_post=None, w_pre=None, post_norm=True, pre_norm=True, w_add=0.0,
               eps=1e-6, residual_scale=1.0, h_out=None, x_out=None, x_type=torch.bfloat16, stream=None):
    """moe_block_norm of device tensors: y and h [rows][hidden] (either may be
    None); gate a tensor that broadcasts to [rows][hidden]; weights
    [hidden].  Returns (h', x), allocated unless given."""
    me = "block_norm"
    like = h if h is not None else y
    if like is None or like.dim() != 2:
        _refuse(me, "y or h must be given, a matrix [rows][hidden]")
    shape = rows, hidden = like.shape
    dev, index = like.device, like.get_device()
    a = moe.moe_block_norm_args()
    a.rows, a.hidden, a.h_type = rows, hidden, _type(like.dtype if h_out is None else h_out.dtype, me)
    a.x_type = _type(x_type if x_out is None else x_out.dtype, me)
    if y is not None:
        _matrix(y, shape, me, "y")
        a.y, a.ld_y, a.y_type = y.data_ptr(), _ld(y, rows, hidden, me), _type(y.dtype, me)
    if h is not None:
        if h_out is not None and h.dtype != h_out.dtype:
            _refuse(me, f"h is of type {h.dtype}, h_out of {h_out.dtype}")
        a.h, a.ld_h = h.data_ptr(), _ld(h, rows, hidden, me)
    if gate is not None:
        try:
            g = gate.expand(rows, hidden)
        except RuntimeError as e:
            _refuse(me, f"gate: {e}")
        a.gate, a.gate_type = g.data_ptr(), _type(g.dtype, me)
        a.ld_gate_row, a.ld_gate_col = (g.stride(0) if rows > 1 else 0), (g.stride(1) if hidden > 1 else 0)
    for name, w in (("w_post", w_post), ("w_pre", w_pre)):
        if w is not None:
            _matrix(w, (hidden,), me, name)
            if not w.is_contiguous():
                _refuse(me, f"{name} must be contiguous")
            setattr(a, name, w.data_ptr())
            a.w_type = _type(w.dtype, me)
    if w_post is not None and w_pre is not None and w_post.dtype != w_pre.dtype:
        _refuse(me, f"w_post is of type {w_post.dtype}, w_pre of {w_pre.dtype}")
    a.post_norm, a.pre_norm = int(post_norm), int(pre_norm)
    a.w_add, a.eps, a.residual_scale = w_add, eps, residual_scale
    for name, t in (("h_out", h_out), ("x_out", x_out)):
        if t is not None:
            _matrix(t, shape, me, name)
            _ld(t, rows, hidden, me)
    _on_gpu(me, index, like, y, gate, w_post, w_pre, h_out, x_out)
    if h_out is None or x_out is None:
        other = _other(dev, stream)
        h_out = _empty(dev, other, like.dtype, rows, hidden) if h_out is None else h_out
        x_out = _empty(dev, other, x_type, rows, hidden) if x_out is None else x_out
    a.h_out, a.ld_h_out = h_out.data_ptr(), _ld(h_out, rows, hidden, me)
    a.x_out, a.ld_x_out = x_out.data_ptr(), _ld(x_out, rows, hidden, me)
    moe.moe_block_norm(a, _stream(dev, stream))
    return h_out, x_out


def token_logprobs(logits: torch.Tensor, targets=None, top_n: int = 0, scale: float = 1.0, ranks: bool = True,
                   stream=None) -> dict:
    """moe_token_logprobs of device logits [rows][vocab]; targets int32 [rows]
    or [rows][n_targets].  Returns device tensors: lse, entropy [rows];
    logprob and rank in the targets' shape; top_ids, top_logprobs
    [rows][top_n]."""
    me = "token_logprobs"
    if logits.dim() != 2:
        _refuse(me, "logits must be a matrix [rows][vocab]")
    rows, vocab = logits.shape
    dev, index = logits.device, logits.get_device()
    a = moe.moe_token_logprobs_args()
    a.logits, a.ld_logits, a.logits_type = logits.data_ptr(), _ld(logits, rows, vocab, me), _type(logits.dtype, me)
    a.rows, a.vocab, a.top_n, a.scale = rows, vocab, top_n, scale
    if targets is not None:
        if targets.dtype != torch.int32 or not targets.is_contiguous() or targets.dim() < 1 or targets.shape[0] != rows:
            _refuse(me, f"targets must be contiguous int32, {rows} or {rows} x n_targets of them")
    _on_gpu(me, index, logits, targets)
    other = _other(dev, stream)
    out = {"lse": _empty(dev, other, torch.float32, rows), "entropy": _empty(dev, other, torch.float32, rows)}
    a.lse, a.entropy = out["lse"].data_ptr(), out["entropy"].data_ptr()
    if targets is not None:
        a.targets, a.n_targets = targets.data_ptr(), targets.numel() // max(rows, 1)
        out["logprob"] = _empty(dev, other, torch.float32, *targets.shape)
        a.target_logprobs = out["logprob"].data_ptr()
        if ranks:
            out["rank"] = _empty(dev, other, torch.int32, *targets.shape)
            a.target_ranks = out["rank"].data_ptr()
    if top_n:
        out["top_ids"] = _empty(dev, other, torch.int32, rows, top_n)
        out["top_logprobs"] = _empty(dev, other, torch.float32, rows, top_n)
        a.top_ids, a.top_logprobs = out["top_ids"].data_ptr(), out["top_logprobs"].data_ptr()
    moe.moe_token_logprobs(a, _stream(dev, stream))
    return out


class Fp8Linear:
    """A linear layer in 8-bit floating point (moe_fp8_*): codes uint8
    [n][ld] with ld a multiple of 16 (e4m3, k of each row used), scales float
    [ceil(n/128)][ceil(k/128)].  Owns the handle and a workspace for up to
    max_rows rows."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, k: int, max_rows: int, stream=None):
        me = "Fp8Linear"
        self.handle = None
        if codes.dim() != 2 or codes.element_size() != 1 or codes.shape[1] < k:
            _refuse(me, f"codes must be bytes [n][at least {k}]")
        self.codes, self.scales, self.k, self.n = codes, scales, k, codes.shape[0]
        self.max_rows = max_rows
        _matrix(scales, (-(-self.n // 128), -(-k // 128)), me, "scales")
        if not scales.is_contiguous() or scales.dtype != torch.float32:
            _refuse(me, "scales must be contiguous float32")
        self.index = codes.get_device()
        _on_gpu(me, self.index, codes, scales)
        self.handle = moe.moe_fp8_open(self.n, k, codes.data_ptr(), _ld(codes, self.n, codes.shape[1], me), scales.data_ptr())
        self.ws_bytes = moe.moe_fp8_workspace_bytes(self.handle, max_rows)
        self.ws = _empty(codes.device, _other(codes.device, stream), torch.uint8, self.ws_bytes)
        self.ws_ptr = self.ws.data_ptr()
        moe.moe_fp8_workspace_init(self.handle, self.ws_ptr, self.ws_bytes, _stream(codes.device, stream))

    @classmethod
    def from_weights(cls, weights: torch.Tensor, max_rows: int, stream=None):
        """Quantises device weights [n][k] (moe_fp8_quantize_weights)."""
        me = "Fp8Linear.from_weights"
        if weights.dim() != 2:
            _refuse(me, "weights must be a matrix [n][k]")
        n, k = weights.shape
        ld = -(-k // 16) * 16
        w_type, ld_w, index = _type(weights.dtype, me), _ld(weights, n, k, me), weights.get_device()
        _on_gpu(me, index, weights)
        dev, other = weights.device, _other(weights.device, stream)
        codes = _empty(dev, other, torch.uint8, n, ld)
        scales = _empty(dev, other, torch.float32, -(-n // 128), -(-k // 128))
        moe.moe_fp8_quantize_weights(weights.data_ptr(), w_type, ld_w, n, k, codes.data_ptr(), ld, scales.data_ptr(),
                                     _stream(dev, stream))
        return cls(codes, scales, k, max_rows, stream)

    def __call__(self, x: torch.Tensor, out: torch.Tensor | None = None, out_type=torch.bfloat16, stream=None):
        """x [rows][k] -> [rows][n]."""
        me = "Fp8Linear"
        shape, n = x.shape, self.n
        if len(shape) != 2 or shape[1] != self.k:
            _refuse(me, f"x has the shape {tuple(shape)}, not [rows][{self.k}]")
        rows, k = shape
        x_type, ld_x = _type(x.dtype, me), _ld(x, rows, k, me)
        if x.get_device() != self.index or out is not None and out.get_device() != self.index:
            _on_gpu(me, self.index, x, out)
        other = None if stream is None else _other(x.device, stream)
        if other is not None:
            for t in (self.ws, self.codes, self.scales):
                t.record_stream(other)
        if out is None:
            out = _empty(x.device, other, out_type, rows, n)
        elif out.shape != (rows, n):
            _refuse(me, f"out has the shape {tuple(out.shape)}, not {rows, n}")
        moe.moe_fp8_linear(self.handle, x.data_ptr(), x_type, ld_x, rows, out.data_ptr(),
                           _type(out.dtype, me), _ld(out, rows, n, me), self.ws_ptr, self.ws_bytes, _stream(x.device, stream))
        return out

    def check(self, stream=None) -> int:
        return moe.moe_fp8_check(self.handle, self.ws_ptr, _stream(self.codes.device, stream))

    def close(self):
        if self.handle:
            moe.moe_fp8_close(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class DeviceLayer:
    def __init__(self, shape: synth.Shape, weight_seed: int, layer: int = 0, beta=None,
                 max_tokens: int = 16, device="cuda:0", chunk_records: int = 32,
                 host_records: np.ndarray | None = None, host_shared: np.ndarray | None = None,
                 router=None, resident: bool = True, rvq: bool = False, codebooks=None):
        """rvq: the experts are 3-bit residual-VQ records (wbits = 3) with the
        layer's codebooks (synth.rvq_codebooks unless given)."""
        self.shape = s = shape
        self.device = torch.device(device)
        self.max_tokens = max_tokens
        self.rvq = rvq
        stride_of = synth.rvq_record_stride if rvq else synth.record_stride
        fill = synth.fill_rvq_records if rvq else synth.fill_records
        one = synth.rvq_expert_record if rvq else synth.expert_record
        self.stride = stride_of(s.H, s.F)
        if resident:
            self.records = torch.empty(s.E * self.stride, dtype=torch.uint8, device=self.device)
            if host_records is not None:
                self.records.copy_(torch.from_numpy(np.ascontiguousarray(host_records).reshape(-1)))
            else:
                n = min(chunk_records, s.E)
                pinned = torch.empty(n * self.stride, dtype=torch.uint8, pin_memory=True)
                view = pinned.numpy()
                for e0 in range(0, s.E, n):
                    cnt = min(n, s.E - e0)
                    fill(weight_seed, layer, range(e0, e0 + cnt), s.H, s.F, view)
                    self.records[e0 * self.stride:(e0 + cnt) * self.stride].copy_(
                        pinned[:cnt * self.stride])
        else:
            self.records = None
        if s.Fs:
            sh = host_shared if host_shared is not None else one(weight_seed, layer, s.E, s.H, s.Fs)
            self.shared = torch.from_numpy(np.ascontiguousarray(sh)).to(self.device)
        else:
            self.shared = None
        rc, rsb = router if router is not None else synth.router(weight_seed, layer, s.E, s.H)
        self.router_codes = torch.from_numpy(np.ascontiguousarray(rc)).to(self.device)
        self.router_sb = torch.from_numpy(np.ascontiguousarray(rsb).view(np.int32)).to(self.device)
        self.beta = None if beta is None else torch.from_numpy(
            np.ascontiguousarray(beta, np.float32)).to(self.device)
        self.codebooks = None
        if rvq:
            cb = codebooks if codebooks is not None else synth.rvq_codebooks(weight_seed, layer)
            self.codebooks = torch.from_numpy(np.ascontiguousarray(cb, np.uint16).view(np.int16)).to(self.device)
        self.desc = moe.desc(s.H, s.E, s.k, s.F, s.Fs, max_tokens=max_tokens, wbits=3 if rvq else 4)
        self.weights = moe.moe_layer_weights(
            self.records.data_ptr() if self.records is not None else None,
            self.shared.data_ptr() if self.shared is not None else None,
            self.router_codes.data_ptr(), self.router_sb.data_ptr(),
            self.beta.data_ptr() if self.beta is not None else None,
            self.codebooks.data_ptr() if self.codebooks is not None else None)
        self.handle = moe.moe_open(self.desc, self.weights)
        self.ws_bytes = moe.moe_workspace_bytes(self.handle, max_tokens)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        moe.moe_workspace_init(self.handle, self.ws.data_ptr(), self.ws_bytes,
                               torch.cuda.current_stream(self.device).cuda_stream)

    def outputs(self, T: int):
        s, dev = self.shape, self.device
        return (torch.empty(T, s.H, dtype=torch.bfloat16, device=dev),
                torch.empty(T, s.H, dtype=torch.float32, device=dev),
                torch.empty(T, s.k, dtype=torch.int32, device=dev),
                torch.empty(T, s.k, dtype=torch.float32, device=dev))

    def _call(self, fn, x: torch.Tensor, outs, stream):
        ob, of, ids, w = outs
        T = x.shape[0]
        st = stream if stream is not None else torch.cuda.current_stream(self.device).cuda_stream
        fn(self.handle, x.data_ptr(), T, ob.data_ptr(), of.data_ptr() if of is not None else None,
           ids.data_ptr(), w.data_ptr(), self.ws.data_ptr(), self.ws_bytes, st)
        return ob, of, ids, w

    def decode(self, x: torch.Tensor, outs=None, stream=None):
        return self._call(moe.moe_decode, x, outs or self.outputs(x.shape[0]), stream)

    def prefill(self, x: torch.Tensor, outs=None, stream=None):
        return self._call(moe.moe_prefill_chunk, x, outs or self.outputs(x.shape[0]), stream)

    def check(self, stream=None) -> int:
        st = stream if stream is not None else torch.cuda.current_stream(self.device).cuda_stream
        return moe.moe_check(self.handle, self.ws.data_ptr(), st)

    def close(self):
        if self.handle:
            moe.moe_close(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def pinned_records(shape: synth.Shape, weight_seed: int, layer: int = 0,
                   host_records: np.ndarray | None = None, rvq: bool = False) -> torch.Tensor:
    """All E expert records of a layer in page-locked host memory (3-bit
    residual-VQ records when rvq)."""
    stride = (synth.rvq_record_stride if rvq else synth.record_stride)(shape.H, shape.F)
    t = torch.empty(shape.E * stride, dtype=torch.uint8, pin_memory=True)
    if host_records is not None:
        t.copy_(torch.from_numpy(np.ascontiguousarray(host_records).reshape(-1)))
    else:
        fill = synth.fill_rvq_records if rvq else synth.fill_records
        fill(weight_seed, layer, range(shape.E), shape.H, shape.F, t.numpy())
    return t


class CachedLayer:
    """A layer whose routed experts are read through the HBM expert cache
    (moe_residency_*): host records pinned, n_slots record slots on the GPU."""

    def __init__(self, dl: DeviceLayer, host_records: torch.Tensor, n_slots: int):
        self.dl = dl
        self.host = host_records
        self.n_slots = n_slots
        self.pool_bytes = moe.moe_residency_pool_bytes(dl.handle, n_slots)
        self.pool = torch.empty(self.pool_bytes, dtype=torch.uint8, device=dl.device)
        self.handle = moe.moe_residency_open(dl.handle, host_records.data_ptr(), n_slots,
                                             self.pool.data_ptr(), self.pool_bytes)
        self.copy_stream = torch.cuda.Stream(dl.device)
        self.ahead_ws = None

    def decode(self, x: torch.Tensor, outs=None, stream=None):
        ob, of, ids, w = outs or self.dl.outputs(x.shape[0])
        st = stream if stream is not None else torch.cuda.current_stream(self.dl.device).cuda_stream
        moe.moe_residency_decode(self.handle, x.data_ptr(), x.shape[0], ob.data_ptr(),
                                 of.data_ptr() if of is not None else None, ids.data_ptr(),
                                 w.data_ptr(), self.dl.ws.data_ptr(), self.dl.ws_bytes, st,
                                 self.copy_stream.cuda_stream)
        return ob, of, ids, w

    def lookahead(self, x: torch.Tensor, n_ahead: int, stream=None, copy_stream=None):
        """Runs this layer's router on an earlier hidden state x and reads the
        first n_ahead experts of each token's predicted ranking into the
        cache (moe_residency_lookahead).  Uses a workspace of its own, so it
        may run on another stream than the layer's steps.  Returns the
        predicted (ids, weights) [B][k] on the device."""
        dl = self.dl
        st = stream if stream is not None else torch.cuda.current_stream(dl.device).cuda_stream
        self.prepare_lookahead(st)
        B = x.shape[0]
        moe.moe_residency_lookahead(self.handle, x.data_ptr(), B, n_ahead, self.ahead_ids.data_ptr(),
                                    self.ahead_w.data_ptr(), self.ahead_ws.data_ptr(), dl.ws_bytes,
                                    st, (copy_stream or self.copy_stream).cuda_stream)
        return self.ahead_ids[:B], self.ahead_w[:B]

    def prepare_lookahead(self, stream) -> None:
        """Allocates the lookahead's workspace and predicted-routing buffers
        (once); stream orders the workspace initialisation."""
        if self.ahead_ws is None:
            dl = self.dl
            self.ahead_ws = torch.empty(dl.ws_bytes, dtype=torch.uint8, device=dl.device)
            moe.moe_workspace_init(dl.handle, self.ahead_ws.data_ptr(), dl.ws_bytes, stream)
            _, _, self.ahead_ids, self.ahead_w = dl.outputs(dl.desc.max_tokens)

    def check_lookahead(self, stream=None) -> int:
        """moe_check of the lookahead workspace (0 if none was made)."""
        if self.ahead_ws is None:
            return moe.MOE_OK
        st = stream if stream is not None else torch.cuda.current_stream(self.dl.device).cuda_stream
        return moe.moe_check(self.dl.handle, self.ahead_ws.data_ptr(), st)

    def stats(self) -> dict:
        return moe.moe_residency_stats(self.handle)

    def slots(self):
        return moe.moe_residency_slots(self.handle, self.n_slots)

    def set_fault(self, mode: int) -> None:
        moe.moe_residency_set_fault(self.handle, mode)

    def close(self):
        if self.handle:
            moe.moe_residency_close(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
