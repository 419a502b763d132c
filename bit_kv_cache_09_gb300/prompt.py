"""Attention of whole prompts packed one behind the other (PyTorch allocates, libkvq computes).

The prompt's own attention next to the caches: the caches store a prompt's keys and values
and answer single-token queries; ``PromptAttention`` computes the outputs of the prompt's
tokens from the 16-bit rows before they are quantized.
"""

from __future__ import annotations

import ctypes

import torch

from . import kvq
from .paged import _code, _ints, _launch, _rows


class PromptAttention:
    """Causal (or full) attention with grouped heads over packed sequences.

    Holds the workspace of its calls (about 20 MB): calls that may overlap, on several streams or in
    graphs replayed at the same time, need an object each."""

    def __init__(self, *, n_kv_heads, gqa_ratio, d_head=128, dtype=torch.float16, device="cuda"):
        self.n_kv, self.n_q, self.gqa, self.d_head = n_kv_heads, n_kv_heads * gqa_ratio, gqa_ratio, d_head
        self.dtype, self._dtype_code = dtype, _code(dtype)
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("the prompt attention runs on a CUDA device")
        self.device = torch.device("cuda", torch.cuda.current_device() if device.index is None else device.index)
        self.ws = torch.zeros(kvq.kvq_prompt_workspace_size(), dtype=torch.uint8, device=self.device)
        self._ws, self._ws_bytes = self.ws.data_ptr(), self.ws.numel()

    def __call__(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor, *,
                 softmax_scale: float, kv_start: torch.Tensor = None, causal: bool = True, out: torch.Tensor = None,
                 return_lse: bool = False, flags: int = 0):
        """q: [tokens][n_q][d_head]; k, v: [tokens][n_kv][d_head] (row strides are free: views of
        a fused projection); q_start, kv_start: int32 [sequences + 1] on the device, the first row of
        each sequence and the end of the last (kv_start None: the same as q_start). With causal the
        last query of a sequence sees its last key. Returns out [tokens][n_q][d_head] and, with
        return_lse, the natural logarithm of each row's sum of exponentials, float32 [tokens][n_q]
        (rows of no sequence: zeros and -inf; an `out` that was passed without return_lse keeps
        what it held there). `out` must not overlap q, k or v. flags: extra bits (PROMPT_ZERO_WAIT_LIMIT)."""
        qs = _rows("q", q, self.device, self.dtype, self.n_q, self.d_head)
        ks = _rows("k", k, self.device, self.dtype, self.n_kv, self.d_head)
        vs = _rows("v", v, self.device, self.dtype, self.n_kv, self.d_head)
        if k.shape[0] != v.shape[0]:
            raise ValueError(f"k has {k.shape[0]} rows, v {v.shape[0]}")
        qp = _ints("q_start", q_start, self.device)
        if q_start.numel() < 2:
            raise ValueError("q_start needs one entry per sequence and one for the end")
        kp = qp if kv_start is None else _ints("kv_start", kv_start, self.device, q_start.numel())
        fresh = out is None
        if fresh:
            out = torch.empty(q.shape, dtype=self.dtype, device=self.device)
        elif out.shape != q.shape:
            raise ValueError(f"out must be {tuple(q.shape)}, not {tuple(out.shape)}")
        os = _rows("out", out, self.device, self.dtype, self.n_q, self.d_head)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=self.device) if return_lse else None
        args = kvq.kvq_prompt_args(self.n_kv, self.gqa, self.d_head, self._dtype_code, q_start.numel() - 1, causal,
                                   (kvq.PROMPT_ZERO_REST if fresh or return_lse else 0) | flags, q.shape[0],
                                   k.shape[0], q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, os, qp, kp, softmax_scale, out.data_ptr(),
                                   lse.data_ptr() if return_lse else None)
        _launch(self.device, "kvq_prompt_attention", ctypes.byref(args), self._ws, self._ws_bytes)
        return (out, lse) if return_lse else out

    def check_errors(self) -> None:
        """Raise KVQDeviceError if a call since the last check recorded an error on the device
        (a bounded wait that ran out); clears it. Synchronizes the current stream."""
        with torch.cuda.device(self.device):
            word = kvq.kvq_decode_error(self.ws.data_ptr(), self.ws.numel(),
                                        torch.cuda.current_stream(self.device).cuda_stream)
        if word:
            raise kvq.KVQDeviceError(word)
