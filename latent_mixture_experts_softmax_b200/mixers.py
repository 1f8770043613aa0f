"""The token mixers of the hybrid layers, held as torch tensors with thin
calls into the C ABI (include/lmoe.h), beside `layer.DeviceLayer`: the 8-bit
paged KV cache with the attention over it, and the gated delta rule with its
states.  torch provides the memory and the stream; all arithmetic runs in
liblmoe.so.

    kv = PagedKV(n_heads=20, n_kv_heads=4, head_dim=128, page_size=64, n_pages=4096)
    ws = kv.workspace()
    batch = kv.batch(q_start, kv_len, page_table, n_tokens, max_new)   # once a step, for every layer's cache
    kv.append(k, v, batch, ws)
    y = kv.attend(q, batch, ws)

Arguments are checked for type, shape, strides and device; what a call finds
wrong on the device (lengths, pages, states) is read with
`binding.lmoe_last_device_status(ws)`.  A call runs on the current stream of
its tensors' device (or on `stream`: a stream or its handle, whose memory the
results then are), and a workspace serves one call at a time: calls on
different streams, and graphs replayed side by side, need their own.  A
workspace is cleared on the stream that is current where it is made."""
from __future__ import annotations

import torch

from . import binding as B

_KV = {"int8": (B.LMOE_KV_INT8, torch.int8), "e4m3": (B.LMOE_KV_E4M3, torch.float8_e4m3fn)}


# The current stream's handle and the current device, by torch's own short ways where it has them
# (torch.cuda.current_stream builds an object, a third of a small call's time).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_of(device, stream):
    return _raw_stream(device.index) if stream is None else stream


def _empty(shape, device, stream):
    """A bf16 result in the memory of the stream that writes it: memory of another may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=device)
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=device)):
        return torch.empty(shape, dtype=torch.bfloat16, device=device)


def _run(device, call, *args):
    """One call with its tensors' device current."""
    now = _current_device()
    if now == device.index:
        return call(*args)
    torch.cuda.set_device(device)
    try:
        return call(*args)
    finally:
        torch.cuda.set_device(now)


def _device(device):
    d = torch.device(device)
    if d.type != "cuda":
        raise ValueError(f"the mixers run on CUDA devices, not on {d}")
    return torch.device("cuda", torch.cuda.current_device()) if d.index is None else d


def _zeroed(n, device):
    if n == 0:
        raise B.LmoeError(B.LMOE_ERR_UNSUPPORTED, "workspace of this shape")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:4096].zero_()
    return ws


def _ints(t, n, name, device):
    if t.dtype != torch.int32 or not t.is_contiguous() or t.device != device or t.shape != n:
        raise ValueError(f"{name}: an int32 tensor of shape {tuple(n)}, contiguous, on {device}")
    return t.data_ptr()


def _rows(t, shape, name, device):
    """A bf16 tensor [tokens, heads, dim] whose heads lie one after the other; its stride between tokens."""
    if t.dtype != torch.bfloat16 or t.shape != shape or t.device != device:
        raise ValueError(f"{name}: a bfloat16 tensor of shape {tuple(shape)} on {device}")
    s = t.stride()
    if s[2] != 1 or (s[1] != shape[2] and shape[1] > 1):
        raise ValueError(f"{name}: heads have to lie one after the other (only the stride between tokens is free)")
    return max(s[0], shape[1] * shape[2]) if shape[0] <= 1 else s[0]


def _whole(t, shape, dtype, name, device):
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: a {dtype} tensor of shape {tuple(shape)}, contiguous, on {device}")
    return t


class KVBatch:
    """lmoe_kv_batch with the tensors it points to (lmoe_kv_batch in include/lmoe.h)."""

    def __init__(self, q_start, kv_len, page_table, n_tokens, max_new):
        device = q_start.device
        if kv_len.dim() != 1 or page_table.dim() != 2:
            raise ValueError("kv_len: [sequences]; page_table: [sequences, pages]")
        n = kv_len.shape[0]
        self.device, self.n_tokens, self.n_seqs = device, n_tokens, n
        self.tensors = (q_start, kv_len, page_table)
        self.c = B.lmoe_kv_batch(_ints(q_start, (n + 1,), "q_start", device), _ints(kv_len, (n,), "kv_len", device),
                                 _ints(page_table, (n, page_table.shape[1]), "page_table", device), n,
                                 page_table.shape[1], n_tokens, max_new)


class PagedKV:
    """One layer's paged cache of 8-bit keys and values, and the attention over it.

    kv_fmt: "int8" or "e4m3".  buffers: (k, v, k_scale, v_scale) that exist already, else zeros are allocated:
    codes [n_pages, n_kv_heads, page_size, head_dim], scales fp32 [n_pages, n_kv_heads, page_size]."""

    def __init__(self, n_heads, n_kv_heads, head_dim, page_size, n_pages=None, kv_fmt="int8", device="cuda", buffers=None):
        fmt, dtype = _KV[kv_fmt]
        self.cfg = B.lmoe_attn_cfg(n_heads, n_kv_heads, head_dim, page_size, fmt)
        status = B.lmoe_attn_cfg_check(self.cfg)
        if status != B.LMOE_OK:
            raise B.LmoeError(status, "lmoe_attn_cfg_check")
        if buffers is None:
            self.device = _device(device)
            rows = (n_pages, n_kv_heads, page_size)
            self.k, self.v = (torch.zeros(*rows, head_dim, dtype=dtype, device=self.device) for _ in "kv")
            self.k_scale, self.v_scale = (torch.ones(rows, dtype=torch.float32, device=self.device) for _ in "kv")
        else:
            self.device = buffers[0].device
            rows = (buffers[0].shape[0], n_kv_heads, page_size)
            self.k, self.v = (_whole(t, (*rows, head_dim), dtype, "codes", self.device) for t in buffers[:2])
            self.k_scale, self.v_scale = (_whole(t, rows, torch.float32, "scales", self.device) for t in buffers[2:])
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, n_kv_heads, head_dim
        self.c = B.lmoe_kv_cache(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
                                 rows[0])

    def workspace(self) -> torch.Tensor:
        """A workspace for batches of any size, its status word cleared."""
        return _zeroed(B.lmoe_attn_workspace_bytes(self.cfg), self.device)

    @staticmethod
    def batch(q_start, kv_len, page_table, n_tokens, max_new) -> KVBatch:
        """Describes the new tokens of a step (device tensors, int32; lmoe_kv_batch)."""
        return KVBatch(q_start, kv_len, page_table, n_tokens, max_new)

    def _same_device(self, batch, ws):
        if batch.device != self.device or ws.device != self.device:
            raise ValueError(f"the batch and the workspace have to be on {self.device}")

    def append(self, k, v, batch, ws, stream=None):
        """Quantise k, v (bf16 [n_tokens, n_kv_heads, head_dim]) into the cache at the batch's places."""
        self._same_device(batch, ws)
        shape = (batch.n_tokens, self.n_kv_heads, self.head_dim)
        ks, vs = _rows(k, shape, "k", self.device), _rows(v, shape, "v", self.device)
        _run(self.device, B.lmoe_kv_append, self.cfg, self.c, batch.c, k, v, ks, vs, ws, _stream_of(self.device, stream))

    def read(self, batch, ws, out=None, stream=None):
        """(k, v) of the batch's tokens as bf16 values; out: a pair of tensors to write."""
        self._same_device(batch, ws)
        shape = (batch.n_tokens, self.n_kv_heads, self.head_dim)
        k, v = out if out is not None else (_empty(shape, self.device, stream) for _ in "kv")
        ks, vs = _rows(k, shape, "k", self.device), _rows(v, shape, "v", self.device)
        _run(self.device, B.lmoe_kv_read, self.cfg, self.c, batch.c, k, v, ks, vs, ws, _stream_of(self.device, stream))
        return k, v

    def attend(self, q, batch, ws, scale=None, causal=True, window=0, out=None, lse=None, stream=None):
        """softmax(scale q k') v of q (bf16 [n_tokens, n_heads, head_dim]) over the cache; scale: head_dim ** -0.5.
        lse: an fp32 [n_tokens, n_heads] tensor for the log-sums of exponentials."""
        self._same_device(batch, ws)
        shape = (batch.n_tokens, self.n_heads, self.head_dim)
        qs = _rows(q, shape, "q", self.device)
        out = _empty(shape, self.device, stream) if out is None else _whole(out, shape, torch.bfloat16, "out", self.device)
        if lse is not None:
            _whole(lse, shape[:2], torch.float32, "lse", self.device)
        _run(self.device, B.lmoe_attend, self.cfg, self.c, batch.c, q, qs,
             self.head_dim ** -0.5 if scale is None else scale, causal, window, out, lse, ws,
             _stream_of(self.device, stream))
        return out


class DeltaBatch:
    """lmoe_delta_batch with the tensors it points to."""

    def __init__(self, q_start, src, dst, n_states, n_tokens, max_new):
        device = q_start.device
        if src.dim() != 1:
            raise ValueError("src, dst: [sequences]")
        n = src.shape[0]
        self.device, self.n_tokens, self.n_seqs = device, n_tokens, n
        self.tensors = (q_start, src, dst)
        self.c = B.lmoe_delta_batch(_ints(q_start, (n + 1,), "q_start", device), _ints(src, (n,), "src", device),
                                    _ints(dst, (n,), "dst", device), n, n_states, n_tokens, max_new)


class DeltaStates:
    """One layer's gated-delta states, fp32 [n_states, n_heads, head_k, head_v], and the rule that moves them on.

    l2norm: q and k rows are normalised by the call."""

    def __init__(self, n_heads, n_qk_heads, head_k, head_v, n_states=None, l2norm=False, device="cuda", state=None):
        self.cfg = B.lmoe_delta_cfg(n_heads, n_qk_heads, head_k, head_v, int(l2norm))
        status = B.lmoe_delta_cfg_check(self.cfg)
        if status != B.LMOE_OK:
            raise B.LmoeError(status, "lmoe_delta_cfg_check")
        if state is None:
            state = torch.zeros(n_states, n_heads, head_k, head_v, device=_device(device))
        self.device = state.device
        self.state = _whole(state, (state.shape[0], n_heads, head_k, head_v), torch.float32, "state", self.device)
        self.n_heads, self.n_qk_heads, self.head_k, self.head_v = n_heads, n_qk_heads, head_k, head_v

    def workspace(self, n_tokens, n_seqs, max_new) -> torch.Tensor:
        """A workspace for batches up to these sizes, its status word cleared."""
        return _zeroed(B.lmoe_delta_workspace_bytes(self.cfg, n_tokens, n_seqs, max_new), self.device)

    def batch(self, q_start, src, dst, n_tokens, max_new) -> DeltaBatch:
        """Describes a step: sequence s starts from state src[s] (-1: zeros) and leaves state dst[s] (lmoe_delta_batch)."""
        return DeltaBatch(q_start, src, dst, self.state.shape[0], n_tokens, max_new)

    def forward(self, q, k, v, log_decay, beta, batch, ws, scale=None, out=None, stream=None):
        """The rule over q, k (bf16 [n_tokens, n_qk_heads, head_k]), v (bf16 [n_tokens, n_heads, head_v]) and the gates
        (fp32 [n_tokens, n_heads]); scale: head_k ** -0.5.  Returns out, bf16 [n_tokens, n_heads, head_v]."""
        d, T = self.device, batch.n_tokens
        if batch.device != d or ws.device != d:
            raise ValueError(f"the batch and the workspace have to be on {d}")
        if batch.c.n_states != self.state.shape[0]:
            raise ValueError("the batch is of other states")
        shape = (T, self.n_heads, self.head_v)
        qs, ks = (_rows(t, (T, self.n_qk_heads, self.head_k), n, d) for t, n in ((q, "q"), (k, "k")))
        vs = _rows(v, shape, "v", d)
        for t, n in ((log_decay, "log_decay"), (beta, "beta")):
            _whole(t, shape[:2], torch.float32, n, d)
        out = _empty(shape, d, stream) if out is None else _whole(out, shape, torch.bfloat16, "out", d)
        _run(d, B.lmoe_delta_rule, self.cfg, batch.c, q, k, v, qs, ks, vs, log_decay, beta,
             self.head_k ** -0.5 if scale is None else scale, self.state, out, ws, _stream_of(d, stream))
        return out
