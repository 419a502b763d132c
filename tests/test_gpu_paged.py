"""The paged 8-bit cache on the GPU against its plain statement (paged_reference): step tables, append, read
back, decode attention, and a serving loop of them with the prompt attention."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from bit_kv_cache_09_gb300 import build as kvq_build  # noqa: E402
from bit_kv_cache_09_gb300 import kvq  # noqa: E402
from bit_kv_cache_09_gb300.paged import PagedKVCache  # noqa: E402
from bit_kv_cache_09_gb300.prompt import PromptAttention  # noqa: E402
from paged_reference import Tables, attention, cached_values, tolerance  # noqa: E402

kvq_build.build()
SCALE = 1.0 / math.sqrt(128)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(**kw):
    base = dict(n_layers=1, n_kv_heads=2, gqa_ratio=4, d_head=128, n_blocks=64, block_tokens=32, n_requests=4,
                max_blocks=40, max_new=2000, fmt="int8", dtype=torch.float16)
    base.update(kw)
    return PagedKVCache(**base)


def rows(rng, n, heads, dtype, gain=1.0):
    x = rng.standard_normal((n, heads, 128)) * gain
    x[:, :, 5] *= 20.0  # a large channel
    return torch.from_numpy(x).to(dtype).cuda()


# ---- step tables -----------------------------------------------------------------------------------------------

def check_step(cache, ref, new, commit=True):
    lens = list(ref.lens)
    got = cache.step(ints(new), commit=commit)
    q_start, positions, slots = ref.step(new)
    n = q_start[-1]
    assert got.q_start.tolist() == q_start
    assert got.positions[:n].tolist() == positions
    assert got.slots[:n].tolist() == slots
    assert got.lens.tolist() == ref.lens
    assert got.free_count.item() == len(ref.free)
    assert cache.lens.tolist() == (ref.lens if commit else lens)
    if commit:
        assert cache.free_count.item() == len(ref.free)
        assert cache.free_list[:len(ref.free)].tolist() == ref.free
        for i, blocks in enumerate(ref.rows):
            assert cache.block_table[i, :len(blocks)].tolist() == blocks


@pytest.mark.parametrize("n_requests,bt,steps", [(1, 32, 12), (3, 64, 30), (67, 32, 25), (300, 128, 12), (1031, 32, 4)])
def test_tables_follow_a_serving_history(n_requests, bt, steps):
    rng = np.random.default_rng(n_requests)
    n_blocks = 40 * n_requests + 7
    cache = make(n_requests=n_requests, block_tokens=bt, n_blocks=n_blocks, max_blocks=300, max_new=400 * n_requests,
                 n_kv_heads=1, gqa_ratio=1)
    ref = Tables(n_blocks, bt, n_requests)
    for _ in range(steps):
        new = []
        for i in range(n_requests):
            x = rng.random()
            new.append(-1 if x < 0.15 else 0 if x < 0.25 else 1 if x < 0.7 else int(rng.integers(2, 400)))
        need = sum((ref.lens[i] + n) // bt - ref.lens[i] // bt for i, n in enumerate(new) if n > 0)
        if need > len(ref.free) + sum(len(ref.rows[i]) for i, n in enumerate(new) if n < 0):
            new = [-1] * n_requests
        check_step(cache, ref, new)
    cache.check_errors()


def test_tables_without_commit_can_be_built_again():
    cache, ref = make(), Tables(64, 32, 4)
    check_step(cache, ref, [100, 0, 33, 64])
    saved = ([list(r) for r in ref.rows], list(ref.free), list(ref.lens))
    for _ in range(3):
        ref.rows, ref.free, ref.lens = [list(r) for r in saved[0]], list(saved[1]), list(saved[2])
        check_step(cache, ref, [-1, 70, 1, 1], commit=False)
    ref.rows, ref.free, ref.lens = [list(r) for r in saved[0]], list(saved[1]), list(saved[2])
    check_step(cache, ref, [-1, 70, 1, 1])


def test_tables_largest_request_count():
    n = 8192
    cache = make(n_requests=n, n_blocks=n + 5, max_blocks=2, max_new=40 * n, n_kv_heads=1, gqa_ratio=1)
    ref = Tables(n + 5, 32, n)
    check_step(cache, ref, [(i * 7) % 34 for i in range(n)])
    check_step(cache, ref, [-1 if i % 3 == 0 else 1 for i in range(n)])


def test_tables_fill_a_request_to_the_brim():
    cache, ref = make(max_blocks=3, n_requests=2), Tables(64, 32, 2)
    check_step(cache, ref, [3 * 32 + 31, 5])
    cache.step(ints([1, 1]))  # one more does not fit: the whole step is refused
    with pytest.raises(kvq.KVQStepError) as e:
        cache.check_errors()
    assert e.value.bits == kvq.PAGED_ERR_LENGTH
    assert cache.lens.tolist() == [127, 5]


@pytest.mark.parametrize("new,bits", [
    ([-2, 1, 1, 1], kvq.PAGED_ERR_NEW), ([2001, 0, 0, 0], kvq.PAGED_ERR_NEW),
    ([1500, 600, 0, 0], kvq.PAGED_ERR_LENGTH),  # 100 + 1500 tokens are 50 blocks, the table has 41
    ([1200, 1200, 0, 0], kvq.PAGED_ERR_NEW | kvq.PAGED_ERR_BLOCKS),  # 2400 tokens of 2000, 74 blocks of 56
    ([2 ** 31 - 1] * 4, kvq.PAGED_ERR_NEW), ([1400, 0, 0, 0], kvq.PAGED_ERR_LENGTH),
    ([640, 640, 640, 0], kvq.PAGED_ERR_BLOCKS),
])
def test_tables_refuse_a_step_as_a_whole(new, bits):
    cache, ref = make(n_blocks=62, max_blocks=41), Tables(62, 32, 4)
    check_step(cache, ref, [100, 0, 33, 64])
    before = (cache.lens.clone(), cache.free_count.clone(), cache.free_list.clone(), cache.block_table.clone())
    step = cache.step(ints(new))
    with pytest.raises(kvq.KVQStepError) as e:
        cache.check_errors()
    assert e.value.bits == bits
    for a, b in zip(before, (cache.lens, cache.free_count, cache.free_list, cache.block_table)):
        assert torch.equal(a, b)
    assert step.q_start.tolist() == [0] * 5 and step.lens.tolist() == ref.lens and step.status[1].item() == 0
    cache.check_errors()  # reported once
    check_step(cache, ref, [1, 2, 3, 4])  # and the next step goes on


def test_tables_refuse_a_broken_state():
    for spoil in (lambda c: c.lens.fill_(-1), lambda c: c.free_count.fill_(65), lambda c: c.free_count.fill_(-1),
                  lambda c: c.lens.fill_(1280), lambda c: c.lens.fill_(2 ** 31 - 1)):
        cache = make()
        spoil(cache)
        cache.step(ints([1, 1, 1, 1]))
        with pytest.raises(kvq.KVQStepError) as e:
            cache.check_errors()
        assert e.value.bits & kvq.PAGED_ERR_STATE


# ---- append and read back --------------------------------------------------------------------------------------

def all_slots(ref):
    return ints([ref.slot(i, p, n) for i, n in enumerate(ref.lens) for p in range(n)])


@pytest.mark.parametrize("bt", [32, 64, 128])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_append_holds_the_same_however_it_is_split(bt, fmt, dtype):
    rng = np.random.default_rng(bt)
    lens, H, L = [1, bt - 1, bt, 3 * bt + 17], 3, 2
    k = [rows(rng, n, H, dtype) for n in lens]
    v = [rows(rng, n, H, dtype, 0.5) for n in lens]
    want = [np.concatenate([cached_values(x.double().cpu().numpy(), bt, fmt) for x in side]) for side in (k, v)]
    for split in ("whole", "ragged", "ones"):
        cache = make(block_tokens=bt, fmt=fmt, dtype=dtype, n_kv_heads=H, n_layers=L, max_new=8 * bt)
        ref, done = Tables(64, bt, 4), [0] * 4
        while done != lens:
            left = [n - d for n, d in zip(lens, done)]
            new = left if split == "whole" else [min(x, 1 if split == "ones" else int(rng.integers(0, bt + 9))) for x in left]
            step = cache.step(ints(new))
            ref.step(new)
            kn = torch.cat([x[d:d + n] for x, d, n in zip(k, done, new)])
            vn = torch.cat([x[d:d + n] for x, d, n in zip(v, done, new)])
            cache.append(1, kn, vn)
            done = [d + n for d, n in zip(done, new)]
            assert step.lens.tolist() == done
        cache.check_errors()
        got = cache.dequantize(1, all_slots(ref))
        for a, b in zip(got, want):
            assert np.array_equal(a.cpu().numpy(), b)
        assert not cache.buffers[0][:cache.buffers[0].numel() // 2].any()  # layer 0 was not touched


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_append_of_unusual_blocks(fmt, dtype):
    """All zeros, the type's smallest and largest values, one large entry, ties, infinities and NaN."""
    bt = 32
    tiny = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}[dtype]
    big = float(torch.finfo(dtype).max)
    x = torch.zeros(10 * bt, 2, 128, dtype=torch.float64)
    ramp = torch.arange(bt * 128, dtype=torch.float64).view(bt, 128)
    x[bt:2 * bt, 0] = tiny * (ramp % 5 - 2)
    x[2 * bt:3 * bt, 0] = big * ((ramp % 7) / 3 - 1)
    x[3 * bt + 4, 0, 9] = -3.0
    x[4 * bt:5 * bt, 0] = (ramp % 255 - 127) / 2  # int8: scale 1/2, exact codes; then ties at every quarter
    x[5 * bt:6 * bt, 0] = (ramp % 509 - 254) / 4
    x[5 * bt, 0, 0] = 63.5
    x[6 * bt, 0, 0] = math.inf
    x[7 * bt + 3, 0, 100] = math.nan
    x[8 * bt, 0, 0], x[8 * bt + 1, 0, 1] = -math.inf, math.nan
    x[9 * bt:10 * bt, 0] = 1.0
    x[:, 1] = 1.0  # the other head is not affected
    k = x.to(dtype).cuda()
    cache, ref = make(fmt=fmt, dtype=dtype, n_requests=1), Tables(64, bt, 1)
    cache.step(ints([10 * bt]))
    ref.step([10 * bt])
    cache.append(0, k, k.flip(1))
    want = cached_values(k.double().cpu().numpy(), bt, fmt)
    a, b = cache.dequantize(0, all_slots(ref))
    assert np.array_equal(a.cpu().numpy(), want, equal_nan=True)
    assert np.array_equal(b.flip(1).cpu().numpy(), want, equal_nan=True)


def test_append_takes_views_and_leaves_rows_behind_the_step():
    rng = np.random.default_rng(3)
    qkv = rows(rng, 90, 8 + 2 + 2, torch.float16)  # one projection's output with rows of padding behind
    cache, ref = make(), Tables(64, 32, 4)
    new = [0, 33, 0, 40]
    cache.step(ints(new))
    ref.step(new)
    qkv[73:] = math.nan
    cache.append(0, qkv[:, 8:10], qkv[:, 10:])
    k, v = cache.dequantize(0, all_slots(ref))
    x = qkv[:73].double().cpu().numpy()
    for got, h in ((k, 8), (v, 10)):
        want = np.concatenate([cached_values(x[a:b, h:h + 2], 32, "int8") for a, b in ((0, 33), (33, 73))])
        assert np.array_equal(got.cpu().numpy(), want)
    one = qkv[:1, 8:10].expand(73, 2, 128)  # the same row for every token
    cache.append(0, one, one)
    k, _ = cache.dequantize(0, all_slots(ref)[:33])
    assert np.array_equal(k[0].cpu().numpy(), cached_values(one[:32].double().cpu().numpy(), 32, "int8")[0])
    cache.check_errors()


def test_append_reports_missing_rows_and_bad_blocks():
    rng = np.random.default_rng(4)
    x = rows(rng, 70, 2, torch.float16)
    for n in (0, 1, 69):
        cache = make()
        cache.step(ints([40, 30, 0, 0]))
        cache.append(0, x[:n], x[:n])
        with pytest.raises(kvq.KVQStepError) as e:
            cache.check_errors()
        assert e.value.bits == kvq.PAGED_ERR_ROWS
    for bad in (-1, 64, 2 ** 31 - 1):
        cache = make()
        cache.step(ints([40, 30, 0, 0]))
        cache.block_table[0, 0] = bad
        cache.append(0, x, x)
        assert not cache.buffers[0].any() and not cache.buffers[1].any()
        cache.attention(0, rows(rng, 4, 8, torch.float16), SCALE)
        with pytest.raises(kvq.KVQStepError) as e:
            cache.check_errors()
        assert e.value.bits == kvq.PAGED_ERR_TABLE


def test_dequantize_of_any_slots():
    rng = np.random.default_rng(5)
    cache, ref = make(block_tokens=64), Tables(64, 64, 4)
    x = rows(rng, 300, 2, torch.float16)
    cache.step(ints([150, 0, 100, 50]))
    ref.step([150, 0, 100, 50])
    cache.append(0, x, x)
    slots = all_slots(ref)
    k, v = cache.dequantize(0, slots)
    pick = torch.from_numpy(rng.integers(0, 300, 777)).cuda()  # any order, repeated
    k2, v2 = cache.dequantize(0, slots[pick].contiguous())
    assert torch.equal(k2, k[pick]) and torch.equal(v2, v[pick])
    bad = ints([64 * 64, -1 - 4 * 64, 2 ** 31 - 1, -2 ** 31])
    k3, v3 = cache.dequantize(0, bad)
    assert torch.isnan(k3).all() and torch.isnan(v3).all()
    assert cache.dequantize(0, ints([]))[0].shape == (0, 2, 128)


# ---- decode attention ------------------------------------------------------------------------------------------

def fill(cache, rng, lens, layer=0, vgain=0.5):
    """Brings `lens` tokens into a fresh cache in two steps; returns the values it holds, per request."""
    c = cache.cfg
    ref = Tables(c.n_blocks, c.block_tokens, c.n_requests)
    k = [rows(rng, n, c.n_kv_heads, cache.dtype) for n in lens]
    v = [rows(rng, n, c.n_kv_heads, cache.dtype, vgain) for n in lens]
    first = [max(n - int(rng.integers(1, 40)), 0) for n in lens]
    for new, cut in ((first, lambda x, f: x[:f]), ([n - f for n, f in zip(lens, first)], lambda x, f: x[f:])):
        cache.step(ints(new))
        ref.step(new)
        cache.append(layer, torch.cat([cut(x, f) for x, f in zip(k, first)]), torch.cat([cut(x, f) for x, f in zip(v, first)]))
    fmt = "int8" if c.format == 0 else "e4m3"
    held = [[cached_values(x.double().cpu().numpy(), c.block_tokens, fmt).astype(np.float64) for x in (a, b)]
            for a, b in zip(k, v)]
    return held, ref


def check_rows(out, q, held, r, scale, dtype, active=None):
    for i, (k, v) in enumerate(held):
        if k.shape[0] == 0 or (active is not None and not active[i]):
            continue
        for h in range(k.shape[1]):
            x = q[i, h * r:(h + 1) * r].double().cpu().numpy()
            want, _, mean_abs, worst = attention(x, k[:, h], v[:, h], scale)
            # softmax weights are rounded to binary16 for the value product
            tol = tolerance(want, mean_abs, worst, dtype, 2.0 ** -11)
            err = np.abs(out[i, h * r:(h + 1) * r].double().cpu().numpy() - want)
            assert (err <= tol).all(), (i, h, float((err / tol).max()))


@pytest.mark.parametrize("r", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("fmt,dtype", [("int8", torch.float16), ("e4m3", torch.bfloat16), ("int8", torch.bfloat16),
                                       ("e4m3", torch.float16)])
def test_decode_ragged_lengths(r, fmt, dtype):
    rng = np.random.default_rng(r)
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 47, 64, 100, 0, 257, 1000]
    cache = make(gqa_ratio=r, fmt=fmt, dtype=dtype, n_requests=len(lens), n_blocks=60)
    held, _ = fill(cache, rng, lens)
    q = rows(rng, len(lens), 2 * r, dtype, 0.3)
    out = cache.attention(0, q, SCALE)
    check_rows(out, q, held, r, SCALE, dtype)
    assert not out[11].any()  # an empty request: zeros in a new tensor
    cache.check_errors()


@pytest.mark.parametrize("bt", [32, 64, 128])
@pytest.mark.parametrize("n", [1, 31, 63, 64, 65, 127, 128, 129, 255, 4000])
def test_decode_block_sizes(bt, n):
    rng = np.random.default_rng(n)
    cache = make(block_tokens=bt, n_requests=2, n_kv_heads=1, n_blocks=260, max_blocks=200, max_new=9000)
    held, _ = fill(cache, rng, [n, max(n // 2, 1)])
    q = rows(rng, 2, 4, torch.float16, 0.3)
    check_rows(cache.attention(0, q, SCALE), q, held, 4, SCALE, torch.float16)
    cache.check_errors()


@pytest.mark.parametrize("requests,heads,n", [(1, 1, 20000), (1, 8, 5000), (40, 8, 90), (3, 5, 3001)])
def test_decode_shapes_of_the_work_split(requests, heads, n):
    """Few long requests (each split over many thread blocks) and many short ones (several per thread block)."""
    rng = np.random.default_rng(heads)
    lens = [n + int(rng.integers(-n // 9, n // 9 + 1)) for _ in range(requests)]
    cache = make(n_requests=requests, n_kv_heads=heads, n_blocks=sum(lens) // 64 + 1, block_tokens=64,
                 max_blocks=max(lens) // 64 + 1, max_new=sum(lens), dtype=torch.bfloat16, fmt="e4m3")
    held, _ = fill(cache, rng, lens)
    q = rows(rng, requests, heads * 4, torch.bfloat16, 0.2)
    out = cache.attention(0, q, SCALE)
    check_rows(out, q, held, 4, SCALE, torch.bfloat16)
    assert torch.equal(out, cache.attention(0, q, SCALE))  # the order of the sums does not change
    cache.check_errors()


@pytest.mark.parametrize("n_requests,step", [(33, 1), (900, 31), (3000, 97), (8192, 4001)])
def test_decode_many_rows_few_in_the_step(n_requests, step):
    """Rows without new tokens between those with some: the search for a tile's request, over windows and samples."""
    rng = np.random.default_rng(n_requests)
    at = list(range(step // 2, n_requests, step))
    lens = [int(rng.integers(1, 150)) for _ in at]
    cache = make(n_requests=n_requests, n_kv_heads=1, n_blocks=len(at) * 5, max_blocks=5, max_new=sum(lens))
    new = [0] * n_requests
    for i, n in zip(at, lens):
        new[i] = n
    cache.step(ints(new))
    k, v = rows(rng, sum(lens), 1, torch.float16), rows(rng, sum(lens), 1, torch.float16, 0.5)
    cache.append(0, k, v)
    q = rows(rng, n_requests, 4, torch.float16, 0.3)
    out = cache.attention(0, q, SCALE)
    cache.check_errors()
    first = np.cumsum([0] + lens)
    held = [[cached_values(x[a:b].double().cpu().numpy(), 32, "int8").astype(np.float64) for x in (k, v)]
            for a, b in zip(first, first[1:])]
    check_rows(out[at], q[at], held, 4, SCALE, torch.float16)
    rest = torch.ones(n_requests, dtype=torch.bool)
    rest[at] = False
    assert not out[rest.cuda()].any()


def test_offsets_beyond_32_bits():
    """A pool of 5 GB whose blocks are taken from its far end, as second layer."""
    rng = np.random.default_rng(18)
    n_blocks = 20000
    cache = make(n_requests=2, n_kv_heads=8, block_tokens=128, n_blocks=n_blocks, max_blocks=20, n_layers=2, max_new=5000)
    cache.free_list.copy_(torch.arange(n_blocks, dtype=torch.int32, device="cuda"))  # the last block on top
    held, ref = fill(cache, rng, [1000, 333], layer=1)
    assert int(cache.block_table[0, 0]) == n_blocks - 1
    q = rows(rng, 2, 32, torch.float16, 0.3)
    check_rows(cache.attention(1, q, SCALE), q, held, 4, SCALE, torch.float16)
    page = cache.block_table[0, :7].long()
    slots = (page[:, None] * 128 + torch.arange(128, device="cuda")).flatten().int()
    k, v = cache.dequantize(1, slots)
    for got, want in ((k, held[0][0]), (v, held[0][1])):
        assert np.array_equal(got.double().cpu().numpy(), want[:896])
    cache.check_errors()


def test_decode_leaves_other_rows_and_masks_stale_tokens():
    """Requests without new tokens keep their rows; what earlier requests left behind the end of a tail or in
    released blocks (here infinities and NaN) reaches nobody."""
    rng = np.random.default_rng(11)
    cache = make(n_requests=3, n_blocks=6, n_kv_heads=2)
    bad = torch.full((100, 2, 128), math.nan, dtype=torch.float16, device="cuda")
    bad[::2] = math.inf
    cache.step(ints([31, 31, 38]))
    cache.append(0, bad, bad)
    cache.step(ints([-1, -1, -1]))
    lens = [33, 2, 21]
    k, v = rows(rng, 56, 2, torch.float16), rows(rng, 56, 2, torch.float16)
    cache.step(ints(lens))
    cache.append(0, k, v)
    held = [[cached_values(x[a:a + n].double().cpu().numpy(), 32, "int8").astype(np.float64) for x in (k, v)]
            for a, n in zip((0, 33, 35), lens)]
    q = rows(rng, 3, 8, torch.float16, 0.3)
    check_rows(cache.attention(0, q, SCALE), q, held, 4, SCALE, torch.float16)
    cache.step(ints([0, 0, 0]))
    out = torch.full_like(q, 7.0)
    cache.attention(0, q, SCALE, out=out)
    assert (out == 7.0).all()  # nobody takes part
    one = rows(rng, 1, 2, torch.float16)
    cache.step(ints([0, 1, 0]))
    cache.append(0, one, one)
    cache.attention(0, q, SCALE, out=out)
    assert (out[0] == 7.0).all() and (out[2] == 7.0).all()
    held[1] = [np.concatenate([x, one.double().cpu().numpy()]) for x in held[1]]
    check_rows(out, q, held, 4, SCALE, torch.float16, active=[0, 1, 0])
    fresh = cache.attention(0, q, SCALE)
    assert not fresh[0].any() and not fresh[2].any() and torch.equal(fresh[1], out[1])
    cache.check_errors()


def test_decode_nan_stays_in_its_block_and_head():
    rng = np.random.default_rng(12)
    cache = make(n_requests=2, n_kv_heads=2)
    k, v = rows(rng, 140, 2, torch.float16), rows(rng, 140, 2, torch.float16)
    k[5, 0, 3] = math.nan
    cache.step(ints([70, 70]))
    cache.append(0, k, v)
    out = cache.attention(0, rows(rng, 2, 8, torch.float16), SCALE)
    assert torch.isnan(out[0, :4]).all() and torch.isfinite(out[0, 4:]).all() and torch.isfinite(out[1]).all()


@pytest.mark.parametrize("requests,heads", [(2, 1), (200, 8)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_decode_a_tail_tile_of_infinite_scores(requests, heads, dtype):
    """Scores of -inf weigh 0 also where a whole tile has no other (in a warp of its own, or in front of others)."""
    rng = np.random.default_rng(13)
    n = 21
    cache = make(n_requests=requests, n_kv_heads=heads, dtype=dtype, max_new=n * requests)
    k, v = rows(rng, n * requests, heads, dtype), rows(rng, n * requests, heads, dtype)
    for lo, hi in ((0, 16), (16, n)):  # the first tile of the tails, then the second
        low = k.clone().view(requests, n, heads, 128)
        low[:, lo:hi, :, 0] = -math.inf
        cache.step(ints([n] * requests))
        cache.append(0, low.view(-1, heads, 128), v)
        q = rows(rng, requests, heads * 4, dtype, 0.3)
        q[:, :, 0] = 1.0
        keep = np.arange(16, n) if lo == 0 else np.arange(16)
        held = [[x.double().cpu().numpy().reshape(requests, n, heads, 128)[i, keep] for x in (k, v)] for i in range(requests)]
        check_rows(cache.attention(0, q, SCALE), q, held, 4, SCALE, dtype)
        cache.step(ints([-1] * requests))
    cache.check_errors()


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_decode_scales(scale):
    rng = np.random.default_rng(13)
    cache = make(n_requests=1)
    held, _ = fill(cache, rng, [300])
    q = rows(rng, 1, 8, torch.float16, 0.3)
    check_rows(cache.attention(0, q, scale), q, held, 4, scale, torch.float16)


def test_decode_flat_and_peaked_rows():
    """A flat softmax over many tokens and one that a single token takes: no weight is lost."""
    n = 30000
    cache = make(n_requests=2, n_kv_heads=1, n_blocks=2000, max_blocks=1000, max_new=2 * n + 64, gqa_ratio=1)
    k = torch.zeros(2 * n, 1, 128, dtype=torch.float16, device="cuda")
    k[0, 0, 0], k[n, 0, 0] = 16.0, 16.0
    v = torch.ones(2 * n, 1, 128, dtype=torch.float16, device="cuda")
    v[0] = v[n] = -1.0
    cache.step(ints([n, n]))
    cache.append(0, k, v)
    q = torch.zeros(2, 1, 128, dtype=torch.float16, device="cuda")
    q[0, 0, 0], q[1, 0, 0] = 0.0, 1.0
    out = cache.attention(0, q, 1.0).double().cpu().numpy()
    for i, s in enumerate((0.0, 16.0)):
        e = math.exp(s)
        want = (n - 1 - e) / (n - 1 + e)
        assert np.abs(out[i] - want).max() <= (2.0 ** -11) * (1 + abs(want)) + 2.0 ** -18
    cache.check_errors()


def test_decode_queries_are_a_view_and_large_or_small():
    """Rows of a fused projection; bfloat16 queries beyond what binary16 holds, each with its own scale."""
    rng = np.random.default_rng(14)
    cache = make(n_requests=2, dtype=torch.bfloat16, fmt="e4m3")
    held, _ = fill(cache, rng, [100, 65])
    qkv = rows(rng, 2, 12, torch.bfloat16)
    q = qkv[:, :8]
    q[0, 0] *= 2.0 ** 100
    q[0, 1] *= 2.0 ** -100
    q[1, 2] = 0.0
    out = cache.attention(0, q, SCALE)
    tame = q.clone()
    tame[0, 0] = 0
    check = [x for x in range(8) if x != 0]
    for i, (k, v) in enumerate(held):
        for j in check if i == 0 else range(8):
            want, _, mean_abs, worst = attention(q[i, j:j + 1].double().cpu().numpy(), k[:, j // 4], v[:, j // 4], SCALE)
            tol = tolerance(want, mean_abs, worst, torch.bfloat16, 2.0 ** -11)
            assert (np.abs(out[i, j:j + 1].double().cpu().numpy() - want) <= tol).all()
    # a row scaled by 2^100 gives all weight to its best key
    k, v = held[0]
    best = (k[:, 0] @ q[0, 0].double().cpu().numpy()).argmax()
    got = out[0, 0].double().cpu().numpy()
    assert (np.abs(got - v[best, 0]) <= 2.0 ** -8 * np.abs(v[best, 0]) + 2.0 ** -24).all()


@pytest.mark.parametrize("lens", [[3000, 40, 1, 700], [20000, 1, 1, 1]])
def test_a_wait_that_runs_out_is_reported(lens):
    """Every wait gives up at once: the error word says so, and the next call is right."""
    rng = np.random.default_rng(20)
    cache = make(n_kv_heads=4, n_blocks=sum(lens) // 32 + 4, max_blocks=max(lens) // 32 + 1, max_new=sum(lens))
    held, _ = fill(cache, rng, lens)
    q = rows(rng, 4, 16, torch.float16, 0.3)
    cache.attention(0, q, SCALE, flags=kvq.PAGED_ZERO_WAIT_LIMIT)
    with pytest.raises(kvq.KVQDeviceError) as e:
        cache.check_errors()
    assert e.value.word == kvq.DECODE_ERR_WAIT_TIMEOUT
    check_rows(cache.attention(0, q, SCALE), q, held, 4, SCALE, torch.float16)
    cache.check_errors()


# ---- streams, graphs, together ---------------------------------------------------------------------------------

def test_two_caches_on_two_streams():
    rng = np.random.default_rng(15)
    caches = [make(n_requests=2, n_kv_heads=4, n_blocks=200, max_blocks=99, max_new=6000) for _ in range(2)]
    held = [fill(c, rng, [2500, 1111])[0] for c in caches]
    qs = [rows(rng, 2, 16, torch.float16, 0.3) for _ in caches]
    streams = [torch.cuda.Stream() for _ in caches]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(caches[i].attention(0, qs[i], SCALE))
    torch.cuda.synchronize()
    for i in range(2):
        check_rows(outs[i][0], qs[i], held[i], 4, SCALE, torch.float16)
        assert all(torch.equal(outs[i][0], x) for x in outs[i])
        caches[i].check_errors()


def test_a_captured_step_is_replayed():
    """One decode step (tables, append, attention) as a CUDA graph: lengths move on from replay to replay, through
    ends of blocks, against the same steps made call by call."""
    rng = np.random.default_rng(16)
    lens = [30, 5, 95]
    pair = [make(n_requests=3, n_layers=2) for _ in range(2)]
    for c in pair:
        fill(c, np.random.default_rng(1), lens)
    new = ints([1, 1, 1])
    q, k, v = (rows(rng, 3, h, torch.float16, 0.3) for h in (8, 2, 2))
    out = torch.zeros(2, 3, 8, 128, dtype=torch.float16, device="cuda")

    def step(c, out):
        c.step(new)
        for layer in range(2):
            c.append(layer, k, v)
            c.attention(layer, q, SCALE, out=out[layer])

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(pair[0], out)
    for _ in range(40):
        for x in (q, k, v):
            x.copy_(torch.from_numpy(rng.standard_normal(x.shape)))
        graph.replay()
        want = torch.zeros_like(out)
        step(pair[1], want)
        assert torch.equal(out, want)
    assert pair[0].lens.tolist() == [n + 40 for n in lens]
    for c in pair:
        c.check_errors()


def test_attention_right_after_a_step_and_on_another_stream():
    """Without an append in between (every request's newest token is cached already): the tables of the step just
    built, each time other ones; then from a stream that waits for the step."""
    rng = np.random.default_rng(19)
    lens = [700, 33, 260, 5]
    cache = make(n_kv_heads=8, n_blocks=100)
    held, _ = fill(cache, rng, lens)
    q = rows(rng, 4, 32, torch.float16, 0.3)
    want = cache.attention(0, q, SCALE)
    check_rows(want, q, held, 4, SCALE, torch.float16)
    other, out = torch.cuda.Stream(), torch.zeros_like(want)
    cache.lens.zero_()
    cache.step(ints([0, 0, 0, 0]))
    for i in range(12):
        some = [n if (i >> (j % 3)) & 1 else 0 for j, n in enumerate(lens)]
        new = ints(some)
        out.zero_()
        cache.step(new, commit=False)  # lengths `some` over the same blocks
        if i % 2:
            other.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(other):
                cache.attention(0, q, SCALE, out=out)
            torch.cuda.current_stream().wait_stream(other)
        else:
            cache.attention(0, q, SCALE, out=out)
        late = cache.attention(0, q, SCALE, out=torch.zeros_like(out), early=False)
        assert torch.equal(out, late)
        for j, n in enumerate(some):
            assert bool(out[j].any()) == (n > 0)  # unfinished blocks hold what `fill` left
    cache.check_errors()


@pytest.mark.parametrize("fmt,dtype", [("int8", torch.float16), ("e4m3", torch.bfloat16)])
def test_serving_loop(fmt, dtype):
    """Prompts come and go: tables, prompt attention and append for the new ones, append and decode attention for the
    running ones, two layers, blocks reused; every output against the plain statement."""
    rng = np.random.default_rng(17)
    R, H, r, L, bt = 5, 2, 3, 2, 32
    cache = make(n_requests=R, n_kv_heads=H, gqa_ratio=r, n_layers=L, fmt=fmt, dtype=dtype, n_blocks=25, block_tokens=bt,
                 max_blocks=10)
    prompt = PromptAttention(n_kv_heads=H, gqa_ratio=r, dtype=dtype)
    raw = [[[np.zeros((0, H, 128)), np.zeros((0, H, 128))] for _ in range(R)] for _ in range(L)]
    ref = Tables(25, bt, R)
    for step_no in range(14):
        new = []
        for i in range(R):
            if ref.lens[i] == 0:
                new.append(int(rng.integers(1, 150)) if rng.random() < 0.6 else 0)
            else:
                new.append(-1 if ref.lens[i] > 120 and rng.random() < 0.5 else 1)
        was = list(ref.lens)
        need = sum((was[i] + n) // bt - was[i] // bt for i, n in enumerate(new) if n > 0)
        if need > len(ref.free):
            new = [min(n, 1) if was[i] else 0 for i, n in enumerate(new)]
        q_start, _, _ = ref.step(new)
        step = cache.step(ints(new))
        n = q_start[-1]
        assert step.q_start.tolist() == q_start
        for layer in range(L):
            qkv = rows(rng, n, H * r + 2 * H, dtype, 0.4)
            q, k, v = qkv[:, :H * r], qkv[:, H * r:H * r + H], qkv[:, H * r + H:]
            cache.append(layer, k, v)
            if n and any(x > 1 for x in new):
                out = prompt(q, k, v, step.q_start, softmax_scale=SCALE)
            newest = torch.zeros(R, H * r, 128, dtype=dtype, device="cuda")
            for i, x in enumerate(new):
                if x > 0:
                    newest[i] = q[q_start[i + 1] - 1]
            dec = cache.attention(layer, newest, SCALE)
            held = []
            for i, x in enumerate(new):
                if x < 0:
                    raw[layer][i] = [np.zeros((0, H, 128)), np.zeros((0, H, 128))]
                a, b = q_start[i], q_start[i + 1]
                raw[layer][i] = [np.concatenate([o, t[a:b].double().cpu().numpy()]) for o, t in zip(raw[layer][i], (k, v))]
                held.append([cached_values(o, bt, fmt).astype(np.float64) for o in raw[layer][i]])
                if x > 1 and was[i] == 0:
                    for j in range(H * r):
                        want, _, mean_abs, worst = attention(q[a:b, j].double().cpu().numpy(), raw[layer][i][0][:, j // r],
                                                             raw[layer][i][1][:, j // r], SCALE, see=range(1, x + 1))
                        tol = tolerance(want, mean_abs, worst, dtype, 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8)
                        assert (np.abs(out[a:b, j].double().cpu().numpy() - want) <= tol).all()
            check_rows(dec, newest, held, r, SCALE, dtype, active=[x > 0 for x in new])
    cache.check_errors()
    prompt.check_errors()
