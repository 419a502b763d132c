"""The paged cache and the prompt attention without a GPU: sizes, refusals on the host before
any launch, the layout inside a tile, and the checks of the Python callers."""

import ctypes

import numpy as np
import pytest
import torch

from bit_kv_cache_09_gb300 import build as kvq_build
from bit_kv_cache_09_gb300 import kvq, paged
from paged_reference import Tables, block_values, e4m3

B = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    kvq_build.build()
    return kvq.load()


def cfg(**kw):
    base = dict(n_layers=2, n_kv_heads=2, gqa_ratio=4, d_head=128, n_blocks=20, block_tokens=64, n_requests=3,
                max_blocks=9, max_new=500, fmt="int8", dtype=kvq.F16)
    base.update(kw)
    return kvq.make_paged_config(**base)


def test_buffer_sizes(lib):
    """Two bytes per token, head and channel (key and value code), 8 bytes of scales per block and
    head, and one unfinished block of 16-bit rows per request and head."""
    for bt in (32, 64, 128):
        L, H, nb, R = 2, 3, 11, 5
        sizes = kvq.kvq_paged_buffer_sizes(cfg(n_kv_heads=H, n_blocks=nb, n_requests=R, block_tokens=bt))
        assert sizes == [L * nb * H * bt * 256, L * nb * H * 8, L * R * H * bt * 512]
    assert kvq.kvq_paged_workspace_size(cfg()) >= 256


@pytest.mark.parametrize("kw,status", [
    (dict(d_head=64), 2), (dict(gqa_ratio=9), 2), (dict(gqa_ratio=0), 1), (dict(n_kv_heads=256), 2),
    (dict(block_tokens=16), 2), (dict(block_tokens=48), 2), (dict(n_requests=8193), 2), (dict(n_requests=0), 1),
    (dict(n_blocks=0), 1), (dict(max_blocks=0), 1), (dict(max_new=0), 1), (dict(fmt=2), 1), (dict(dtype=2), 1),
    (dict(n_blocks=2 ** 25), 2), (dict(max_blocks=2 ** 25), 2), (dict(max_new=2 ** 31 - 1), 2), (dict(n_layers=0), 1),
    (dict(block_tokens=-64), 1),
])
def test_bad_configs_are_rejected(lib, kw, status):
    sizes = (ctypes.c_size_t * 3)()
    assert lib.kvq_paged_buffer_sizes(B(cfg(**kw)), sizes) == status
    assert kvq.kvq_paged_workspace_size(cfg(**kw)) == 0
    assert lib.kvq_paged_buffer_sizes(None, sizes) == 1 and lib.kvq_paged_buffer_sizes(B(cfg()), None) == 1


def _bufs(p=4096):
    return kvq.kvq_paged_buffers(p, p, p)


def _state(**kw):
    f = dict(lens=4096, block_table=8192, free_list=12288, free_count=16384)
    f.update(kw)
    return kvq.kvq_paged_state(*f.values())


def _step(**kw):
    f = dict(lens=65536, free_count=65792, q_start=66048, positions=66304, slots=66560, units=66816, tile_start=67072,
             status=67328)
    f.update(kw)
    return kvq.kvq_paged_step(*f.values())


def test_step_tables_refusals(lib):
    call = lambda c=None, st=None, new=20480, sp=None, commit=1: lib.kvq_paged_step_tables(  # noqa: E731
        B(c or cfg()), B(st or _state()), new, B(sp or _step()), commit, None)
    assert call(c=cfg(block_tokens=40)) == 2
    for name in ("lens", "block_table", "free_list", "free_count"):
        assert call(st=_state(**{name: None})) == 1 and call(st=_state(**{name: 4098})) == 1
    for name in ("lens", "free_count", "q_start", "positions", "slots", "units", "tile_start", "status"):
        assert call(sp=_step(**{name: None})) == 1 and call(sp=_step(**{name: 65538})) == 1
    assert call(sp=_step(units=66824)) == 1  # entries of the work list are 16-byte aligned
    assert call(new=None) == 1 and call(new=4098) == 1 and call(commit=2) == 1
    # the state is read while the step is written
    assert call(sp=_step(lens=4096)) == 1 and call(sp=_step(free_count=16384)) == 1 and call(new=65536) == 1
    assert lib.kvq_paged_step_tables(B(cfg()), None, 20480, B(_step()), 1, None) == 1
    assert lib.kvq_paged_step_tables(B(cfg()), B(_state()), 20480, None, 1, None) == 1


def test_append_and_dequantize_refusals(lib):
    app = lambda c=None, b=None, table=8192, sp=None, layer=0, n=10, k=4096, ks=256, v=4096, vs=256: (  # noqa: E731
        lib.kvq_paged_append(B(c or cfg()), B(b or _bufs()), table, B(sp or _step()), layer, n, k, ks, v, vs, None))
    assert app(c=cfg(gqa_ratio=12)) == 2 and app(b=_bufs(4112)) == 1 and app(table=None) == 1
    assert app(sp=_step(units=None)) == 1 and app(layer=2) == 1 and app(layer=-1) == 1
    assert app(n=-1) == 1 and app(n=2 ** 31) == 1
    assert app(k=None) == 1 and app(k=4104) == 1 and app(v=4098) == 1
    assert app(ks=252) == 1 and app(vs=-256) == 1 and app(ks=2 ** 31) == 1
    deq = lambda c=None, b=None, layer=0, n=5, slots=4096, k=4096, v=4096: lib.kvq_paged_dequantize(  # noqa: E731
        B(c or cfg()), B(b or _bufs()), layer, n, slots, k, v, None)
    assert deq(c=cfg(fmt=5)) == 1 and deq(b=_bufs(4100)) == 1 and deq(layer=2) == 1 and deq(n=-1) == 1
    assert deq(slots=None) == 1 and deq(slots=4097) == 1 and deq(k=4104) == 1 and deq(v=None) == 1
    assert deq(n=0, slots=None, k=None, v=None) == 0  # nothing to read


def test_decode_refusals(lib):
    need = kvq.kvq_paged_workspace_size(cfg())
    dec = lambda c=None, b=None, table=8192, sp=None, layer=0, q=4096, qs=1024, scale=0.1, out=4096, ws=4096, n=need, flags=0: (  # noqa: E731
        lib.kvq_paged_decode_attention(B(c or cfg()), B(b or _bufs()), table, B(sp or _step()), layer, q, qs,
                                       ctypes.c_float(scale), out, flags, ws, n, None))
    assert dec(c=cfg(block_tokens=256)) == 2 and dec(b=_bufs(None)) == 1 and dec(table=4097) == 1
    assert dec(sp=_step(tile_start=None)) == 1 and dec(layer=7) == 1 and dec(q=4104) == 1 and dec(out=None) == 1
    assert dec(qs=1020) == 1 and dec(scale=float("nan")) == 1 and dec(scale=float("inf")) == 1 and dec(scale=3e38) == 1
    assert dec(flags=8) == 1 and dec(flags=2 ** 31) == 1
    assert dec(ws=None) == 4 and dec(ws=4112) == 4 and dec(n=need - 1) == 4


def test_prompt_refusals(lib):
    need = kvq.kvq_prompt_workspace_size()
    assert need > 1024

    def call(ws=4096, n=need, **kw):
        f = dict(n_kv_heads=2, gqa_ratio=4, d_head=128, dtype=0, n_seqs=1, causal=1, flags=0, n_q=10, n_kv=10,
                 q=4096, k=4096, v=4096, q_stride=1024, k_stride=256, v_stride=256, out_stride=1024, q_start=4096,
                 kv_start=4096, softmax_scale=0.1, out=65536, lse=None)
        f.update(kw)
        return lib.kvq_prompt_attention(B(kvq.kvq_prompt_args(*f.values())), ws, n, None)

    assert call(d_head=64) == 2 and call(gqa_ratio=9) == 2 and call(n_kv_heads=0) == 1 and call(n_kv_heads=256) == 2
    assert call(flags=4) == 1 and call(flags=2 ** 31) == 1
    assert call(dtype=3) == 1 and call(causal=2) == 1 and call(n_seqs=0) == 1 and call(n_seqs=65536) == 2
    assert call(n_q=-1) == 1 and call(n_kv=2 ** 31) == 2 and call(softmax_scale=-0.1) == 1
    assert call(softmax_scale=float("nan")) == 1 and call(softmax_scale=float("inf")) == 1
    assert call(softmax_scale=3e38) == 1
    assert call(q_start=None) == 1 and call(kv_start=4098) == 1
    for name in ("q", "k", "v", "out"):
        assert call(**{name: None}) == 1 and call(**{name: 4104}) == 1
        assert call(**{name + "_stride": 1028}) == 1 and call(**{name + "_stride": -1024}) == 1
    assert call(q_stride=1016) == 1 and call(out_stride=512) == 1 and call(k_stride=128) == 1  # rows would overlap
    assert call(out=4096) == 1 and call(q=8192, k=65536) == 1 and call(v=65536) == 1  # out is one of the inputs
    assert call(lse=4097) == 1 and call(ws=None) == 4 and call(ws=4104) == 4 and call(n=need - 1) == 4
    assert lib.kvq_prompt_attention(None, 4096, need, None) == 1
    assert call(n_q=0, q=None, out=None) == 0  # nothing to compute


def test_tables_are_read_early_unless_a_step_was_the_last_call(monkeypatch):
    """Host logic of the early-tables flag."""
    now = [5]
    monkeypatch.setattr(paged, "_stream", lambda device: now[0])
    c = paged.PagedKVCache.__new__(paged.PagedKVCache)
    c.device, c._tables_on = None, None
    Z, E = kvq.PAGED_ZERO_REST, kvq.PAGED_EARLY_TABLES
    assert c._flags(True, None) == Z | E and c._flags(False, None) == E
    c._tables_on = 5  # a step on this stream
    assert c._flags(False, None) == 0 and c._flags(True, None) == Z and c._flags(False, True) == E
    now[0] = 6        # another stream waits for the step by an event
    assert c._flags(False, None) == E and c._flags(False, False) == 0


def test_python_callers_check_their_tensors():
    cpu = torch.device("cpu")
    x = torch.zeros(5, 2, 128, dtype=torch.float16)
    assert paged._rows("x", x, cpu, torch.float16, 2, 128) == 256
    fused = torch.zeros(5, 6, 128, dtype=torch.float16)
    assert paged._rows("x", fused[:, 2:4], cpu, torch.float16, 2, 128) == 768
    with pytest.raises(TypeError):
        paged._rows("x", x.float(), cpu, torch.float16, 2, 128)
    for bad in (x[:, :1], x[0], x.transpose(0, 1), torch.zeros(5, 128, 2, dtype=torch.float16).transpose(1, 2),
                torch.zeros(5, 2 * 128 + 4, dtype=torch.float16)[:, :256].unflatten(1, (2, 128))):
        with pytest.raises(ValueError):
            paged._rows("x", bad, cpu, torch.float16, 2, 128)
    with pytest.raises(ValueError):
        paged._rows("x", x, torch.device("cuda", 0), torch.float16, 2, 128)
    for bad in (torch.zeros(4), torch.zeros(4, dtype=torch.int64), torch.zeros(8, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            paged._ints("n", bad, cpu)
    with pytest.raises(ValueError):
        paged._ints("n", torch.zeros(4, dtype=torch.int32), cpu, 5)
    with pytest.raises(TypeError):
        paged._code(torch.float32)
    with pytest.raises(ValueError):
        paged.PagedKVCache(n_layers=1, n_kv_heads=1, gqa_ratio=1, d_head=128, n_blocks=1, block_tokens=32, n_requests=1,
                           max_blocks=1, max_new=1, fmt="int4")
    with pytest.raises(kvq.KVQError):
        paged.PagedKVCache(n_layers=1, n_kv_heads=1, gqa_ratio=1, d_head=64, n_blocks=1, block_tokens=32, n_requests=1,
                           max_blocks=1, max_new=1)


def test_reference_quantizer():
    """The tests' own statement: half a step of error, exact codes on the grid, e4m3 against torch's cast."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((32, 128)).astype(np.float16).astype(np.float64)
    for fmt, rel in (("int8", 0.0), ("e4m3", 2.0 ** -4)):
        got = block_values(x, fmt)
        scale = np.abs(x).max() / (127 if fmt == "int8" else 448)
        # int8: half a step of the scale; e4m3: 2^-4 of the value, or half of its smallest step, 2^-10
        bound = scale / 2 if fmt == "int8" else np.maximum(rel * np.abs(x), scale * 2.0 ** -10)
        assert (np.abs(got - x) <= bound * (1 + 2.0 ** -20)).all()
    assert (block_values(np.zeros((32, 128)), "int8") == 0).all()
    assert np.isnan(block_values(np.where(x == x.max(), np.inf, x), "e4m3")).all()
    y = np.concatenate([rng.uniform(-448, 448, 20000), rng.uniform(-0.1, 0.1, 20000)]).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(e4m3(y.astype(np.float64)), want)


def test_reference_tables():
    t = Tables(4, 32, 2)
    q_start, pos, slots = t.step([40, 3])
    assert q_start == [0, 40, 43] and pos == list(range(40)) + [0, 1, 2]
    assert slots[:32] == list(range(32)) and slots[32:] == [-1 - i for i in range(8)] + [-1 - 32 - i for i in range(3)]
    assert t.step([-1, 0])[0] == [0, 0, 0] and t.lens == [0, 3] and t.free == [3, 2, 1, 0]
