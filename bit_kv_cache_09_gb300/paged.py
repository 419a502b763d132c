"""Paged 8-bit cache for requests of different lengths: PyTorch allocates, libkvq computes.

A serving step is ``cache.step(new)`` once (new tokens of each request row, on the
device), then per layer ``cache.append(layer, k, v)`` with the step's packed rows and
``cache.attention(layer, q, scale)`` for the newest token of every request in the step.
Nothing synchronizes or copies to the host, so a step can be captured in a CUDA graph.

Every call runs on the current stream of the cache's device. The cache's own tensors
(tables, workspace) are written by its calls: calls of one cache object must be ordered,
on one stream or by events.

``attention`` reads the tables while the kernel before it on the stream finishes, unless that
kernel is this object's ``step``. A kernel that writes ``tables.lens``, ``tables.tile_start`` or
``block_table`` outside this object must therefore not directly precede ``attention`` on the same
stream; pass ``early=False`` after one.
"""

from __future__ import annotations

import ctypes

import torch

from . import kvq

_DTYPES = {torch.float16: kvq.F16, torch.bfloat16: kvq.BF16}


def _code(dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be float16 or bfloat16, not {dtype}")
    return _DTYPES[dtype]


def _rows(name: str, x: torch.Tensor, device, dtype, heads: int, d_head: int) -> int:
    """Checks [rows][heads][d_head] rows (heads contiguous inside a row); returns the row stride in elements."""
    shape, stride = x.shape, x.stride()
    if (x.device == device and x.dtype == dtype and len(shape) == 3 and shape[1] == heads and shape[2] == d_head
            and stride[2] == 1 and (heads == 1 or stride[1] == d_head)):
        if shape[0] <= 1:
            return heads * d_head
        if stride[0] % 8 == 0:
            return stride[0]
        raise ValueError(f"{name}: the row stride must be a multiple of 8 elements, not {stride[0]}")
    if x.device != device:
        raise ValueError(f"{name} is on {x.device}, expected {device}")
    if x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {x.dtype}")
    if len(shape) != 3 or shape[1] != heads or shape[2] != d_head:
        raise ValueError(f"{name} must be [rows][{heads}][{d_head}], not {tuple(shape)}")
    raise ValueError(f"{name}: the heads of a row must lie behind one another (strides {stride})")


def _ints(name: str, x: torch.Tensor, device, n=None) -> int:
    if x.device != device or x.dtype != torch.int32 or x.dim() != 1 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 vector on {device}")
    if n is not None and x.numel() != n:
        raise ValueError(f"{name} must have {n} entries, not {x.numel()}")
    return x.data_ptr()


def _launch(device, name: str, *args) -> None:
    """Calls entry point `name` with `args` and the current stream of `device`, that device being current."""
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            return _launch(device, name, *args)
    status = getattr(kvq.load(), name)(*args, _stream(device))
    if status:
        raise kvq.KVQError(name, status, kvq.kvq_status_string(status))


def _stream(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


class StepTables:
    """What one step wrote (int32 tensors on the device, reused by the cache's next step)."""

    def __init__(self, cfg: kvq.kvq_paged_config, device):
        units = cfg.max_new // cfg.block_tokens + cfg.n_requests
        sizes = (("lens", cfg.n_requests), ("free_count", 1), ("q_start", cfg.n_requests + 1),
                 ("positions", cfg.max_new), ("slots", cfg.max_new), ("units", 4 * units),
                 ("tile_start", cfg.n_requests + 1), ("status", 4))
        for name, n in sizes:
            setattr(self, name, torch.zeros(n, dtype=torch.int32, device=device))
        self.ptrs = kvq.kvq_paged_step(*[getattr(self, name).data_ptr() for name, _ in sizes])


class PagedKVCache:
    """Blocks of ``block_tokens`` tokens in 8 bits (``fmt`` "int8" or "e4m3") with one scale
    per block, kv head and tensor; the tokens of unfinished blocks stay ``dtype``.

    State tensors (int32, on the device): ``lens`` [n_requests], ``block_table``
    [n_requests][max_blocks], ``free_list`` [n_blocks] and ``free_count`` [1].
    """

    def __init__(self, *, n_layers, n_kv_heads, gqa_ratio, d_head, n_blocks, block_tokens, n_requests, max_blocks,
                 max_new, fmt="int8", dtype=torch.float16, device="cuda"):
        if fmt not in kvq.PAGED_FORMATS:
            raise ValueError(f"fmt must be one of {sorted(kvq.PAGED_FORMATS)}, not {fmt!r}")
        self.cfg = kvq.make_paged_config(n_layers=n_layers, n_kv_heads=n_kv_heads, gqa_ratio=gqa_ratio, d_head=d_head,
                                         n_blocks=n_blocks, block_tokens=block_tokens, n_requests=n_requests,
                                         max_blocks=max_blocks, max_new=max_new, fmt=fmt, dtype=_code(dtype))
        sizes = kvq.kvq_paged_buffer_sizes(self.cfg)  # raises on an unsupported configuration, before any allocation
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("the paged cache lives on a CUDA device")
        self.device = torch.device("cuda", torch.cuda.current_device() if device.index is None else device.index)
        self.dtype = dtype
        self.n_q = n_kv_heads * gqa_ratio
        with torch.cuda.device(self.device):
            self.buffers = [torch.zeros(max(n, 256), dtype=torch.uint8, device=self.device) for n in sizes]
            self.bufs = kvq.kvq_paged_buffers(*[b.data_ptr() for b in self.buffers])
            new = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=self.device)  # noqa: E731
            self.lens, self.block_table = new(n_requests), new(n_requests, max_blocks)
            # a stack: block 0 on top
            self.free_list = torch.arange(n_blocks - 1, -1, -1, dtype=torch.int32, device=self.device)
            self.free_count = torch.full((1,), n_blocks, dtype=torch.int32, device=self.device)
            self.state = kvq.kvq_paged_state(self.lens.data_ptr(), self.block_table.data_ptr(),
                                             self.free_list.data_ptr(), self.free_count.data_ptr())
            self.tables = StepTables(self.cfg, self.device)
            self.ws = torch.zeros(max(kvq.kvq_paged_workspace_size(self.cfg), 256), dtype=torch.uint8,
                                  device=self.device)
        self._tables_on = None  # the stream of a step() that no other call of this object has followed
        # the arguments that never change
        self._cfg, self._bufs, self._state, self._step = (ctypes.byref(x) for x in (self.cfg, self.bufs, self.state,
                                                                                    self.tables.ptrs))
        self._table, self._ws = self.block_table.data_ptr(), self.ws.data_ptr()

    def _call(self, name: str, *args) -> None:
        """lib.name(*args, stream) with the cache's device current."""
        _launch(self.device, name, *args)

    def step(self, new_tokens: torch.Tensor, commit: bool = True) -> StepTables:
        """Builds the tables of a step that adds new_tokens[i] tokens to request i (int32
        [n_requests] on the device; -1 releases the request). With commit=False lens and
        free_count stay as they were, so the step can be built again."""
        ptr = _ints("new_tokens", new_tokens, self.device, self.cfg.n_requests)
        self._call("kvq_paged_step_tables", self._cfg, self._state, ptr, self._step, int(commit))
        self._tables_on = _stream(self.device)
        return self.tables

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor) -> None:
        """k, v: [rows][n_kv_heads][d_head], the step's new tokens in packed order (rows behind
        them are not read). Row strides are free (views of a fused projection)."""
        c = self.cfg
        ks = _rows("k", k, self.device, self.dtype, c.n_kv_heads, c.d_head)
        vs = _rows("v", v, self.device, self.dtype, c.n_kv_heads, c.d_head)
        if k.shape[0] != v.shape[0]:
            raise ValueError(f"k has {k.shape[0]} rows, v {v.shape[0]}")
        self._call("kvq_paged_append", self._cfg, self._bufs, self._table, self._step, layer, k.shape[0], k.data_ptr(), ks,
                   v.data_ptr(), vs)
        self._tables_on = None

    def dequantize(self, layer: int, slots: torch.Tensor):
        """Keys and values kept at `slots` (int32, as in StepTables.slots): two float32
        [len(slots)][n_kv_heads][d_head] tensors."""
        c = self.cfg
        ptr, n = _ints("slots", slots, self.device), slots.numel()
        k = torch.empty((n, c.n_kv_heads, c.d_head), dtype=torch.float32, device=self.device)
        v = torch.empty_like(k)
        self._call("kvq_paged_dequantize", self._cfg, self._bufs, layer, n, ptr, k.data_ptr(), v.data_ptr())
        return k, v

    def _flags(self, fresh: bool, early) -> int:
        """Flag bits of an attention call (see the module's docstring)."""
        if early is None:
            early = self._tables_on is None or self._tables_on != _stream(self.device)
        return (kvq.PAGED_ZERO_REST if fresh else 0) | (kvq.PAGED_EARLY_TABLES if early else 0)

    def attention(self, layer: int, q: torch.Tensor, softmax_scale: float, out: torch.Tensor = None,
                  early=None, flags: int = 0) -> torch.Tensor:
        """Attention of the newest token of every request in the step. q: [n_requests][n_q][d_head];
        returns out of the same shape. Rows of requests without new tokens keep what `out` held
        (a new `out` holds zeros there). flags: extra bits (PAGED_ZERO_WAIT_LIMIT)."""
        c = self.cfg
        qs = _rows("q", q, self.device, self.dtype, self.n_q, c.d_head)
        if q.shape[0] != c.n_requests:
            raise ValueError(f"q must have {c.n_requests} rows, not {q.shape[0]}")
        fresh = out is None
        if fresh:
            out = torch.empty(q.shape, dtype=self.dtype, device=self.device)
        elif out.shape != q.shape or out.dtype != self.dtype or out.device != self.device or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous {self.dtype} tensor of shape {tuple(q.shape)} on {self.device}")
        self._call("kvq_paged_decode_attention", self._cfg, self._bufs, self._table, self._step, layer, q.data_ptr(), qs,
                   softmax_scale, out.data_ptr(), self._flags(fresh, early) | flags, self._ws, self.ws.numel())
        self._tables_on = None
        return out

    def check_errors(self) -> None:
        """Raise KVQStepError / KVQDeviceError if a call since the last check recorded an error
        on the device; clears it. Synchronizes the current stream."""
        with torch.cuda.device(self.device):
            bits = int(self.tables.status[0].item())
            if bits:
                self.tables.status[0].zero_()
            word = kvq.kvq_decode_error(self._ws, self.ws.numel(), torch.cuda.current_stream().cuda_stream)
        if bits:
            raise kvq.KVQStepError(bits)
        if word:
            raise kvq.KVQDeviceError(word)
