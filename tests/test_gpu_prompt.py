"""Prompt attention on the GPU against its plain statement in 64 bits (paged_reference.attention)."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from bit_kv_cache_09_gb300 import build as kvq_build  # noqa: E402
from bit_kv_cache_09_gb300 import kvq  # noqa: E402
from bit_kv_cache_09_gb300.prompt import PromptAttention  # noqa: E402
from paged_reference import attention, lse_tolerance, tolerance  # noqa: E402

kvq_build.build()
SCALE = 1.0 / math.sqrt(128)
# softmax weights are rounded to the 16-bit type for the value product
WEIGHT_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def starts(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def rows(rng, n, heads, dtype, gain=1.0):
    x = rng.standard_normal((n, heads, 128)) * gain
    x[:, :, 7] *= 10.0
    return torch.from_numpy(x).to(dtype).cuda()


def check(out, lse, q, k, v, q_lens, kv_lens, causal, scale, r, heads=None, some=None):
    dtype = q.dtype
    a = b = 0
    rng = np.random.default_rng(0)
    for n, m in zip(q_lens, kv_lens):
        pick = np.arange(n) if some is None or n <= some else np.sort(rng.choice(n, some, replace=False))
        for j in range(q.shape[1]) if heads is None else heads:
            x = q[a:a + n, j].double().cpu().numpy()[pick]
            see = [i + 1 + m - n for i in pick] if causal else None
            want, wl, mean_abs, worst = attention(x, k[b:b + m, j // r].double().cpu().numpy(),
                                                  v[b:b + m, j // r].double().cpu().numpy(), scale, see)
            got = out[a:a + n, j].double().cpu().numpy()[pick]
            tol = tolerance(want, mean_abs, worst, dtype, WEIGHT_STEP[dtype])
            err = np.abs(got - want)
            assert (err <= tol).all(), (n, m, j, float((err / tol).max()))
            if lse is not None:
                g = lse[a:a + n, j].double().cpu().numpy()[pick]
                assert np.array_equal(np.isfinite(g), np.isfinite(wl))
                fine = np.isfinite(wl)
                assert (np.abs(g[fine] - wl[fine]) <= lse_tolerance(wl, worst)[fine]).all()
        a, b = a + n, b + m


def run(q_lens, kv_lens=None, r=4, H=2, dtype=torch.float16, causal=True, scale=SCALE, seed=0, some=None, gain=1.0):
    rng = np.random.default_rng(seed)
    kv = q_lens if kv_lens is None else kv_lens
    q, k, v = rows(rng, sum(q_lens), H * r, dtype, gain), rows(rng, sum(kv), H, dtype), rows(rng, sum(kv), H, dtype, 0.5)
    att = PromptAttention(n_kv_heads=H, gqa_ratio=r, dtype=dtype)
    out, lse = att(q, k, v, starts(q_lens), kv_start=None if kv_lens is None else starts(kv), softmax_scale=scale,
                   causal=causal, return_lse=True)
    check(out, lse, q, k, v, q_lens, kv, causal, scale, r, some=some)
    att.check_errors()
    return att, q, k, v, out, lse


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 385, 640])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_one_prompt(n, dtype):
    run([n], dtype=dtype, seed=n, some=90)


@pytest.mark.parametrize("r", [1, 2, 3, 5, 6, 7, 8])
def test_group_sizes(r):
    run([70, 1, 200], r=r, seed=r)
    run([300], kv_lens=[411], r=r, H=1, seed=r, dtype=torch.bfloat16, some=60)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_packed_sequences(causal, dtype):
    lens = [5, 0, 128, 1, 77, 300, 0, 64, 33]
    run(lens, causal=causal, dtype=dtype, seed=1)
    run(lens, kv_lens=[9, 4, 128, 200, 80, 299, 0, 0, 513], causal=causal, dtype=dtype, seed=2)


def test_rows_without_keys():
    """More queries than keys: the first rows of a causal sequence see nothing, get zeros and -inf."""
    _, _, _, _, out, lse = run([100, 40, 300], kv_lens=[60, 0, 3], seed=3)
    assert not out[:40].any() and (lse[:40] == -math.inf).all() and torch.isfinite(lse[40:100]).all()
    assert not out[100:140].any() and (lse[100:140] == -math.inf).all()
    run([10, 20], kv_lens=[0, 5], causal=False, seed=4)


def test_many_short_sequences():
    rng = np.random.default_rng(5)
    run([int(x) for x in rng.integers(0, 6, 700)], H=1, r=2, seed=5)


@pytest.mark.parametrize("n", [33, 40, 255, 256, 257, 600])
def test_many_sequences_of_several_items(n):
    """Empty, short and long sequences in any place: which item a thread block takes."""
    rng = np.random.default_rng(n)
    lens = [0 if x < 0.3 else int(rng.integers(1, 20)) if x < 0.9 else int(rng.integers(60, 300)) for x in rng.random(n)]
    lens[-1] = 70
    run(lens, kv_lens=[x + int(rng.integers(0, 9)) if x else 0 for x in lens], H=1, r=8, seed=n, some=3)


@pytest.mark.parametrize("r,H,n,ctx", [(4, 8, 1500, 0), (8, 1, 700, 2900), (1, 3, 2049, 0)])
def test_longer_prompts(r, H, n, ctx):
    run([n, 65], kv_lens=[n + ctx, 65], r=r, H=H, seed=n, some=6)


@pytest.mark.parametrize("scale", [0.0, 1e-4, 2.0])
def test_scales(scale):
    run([150, 40], scale=scale, seed=6)


def test_growing_scores():
    """Scores that grow along the keys (every tile brings a larger maximum) and that fall."""
    rng = np.random.default_rng(7)
    n, att = 600, PromptAttention(n_kv_heads=1, gqa_ratio=2)
    for sign in (1.0, -1.0):
        q, k, v = rows(rng, n, 2, torch.float16, 0.1), rows(rng, n, 1, torch.float16, 0.1), rows(rng, n, 1, torch.float16)
        q[:, :, 0] = 8.0
        k[:, 0, 0] = sign * torch.arange(n, device="cuda") * 0.2
        out, lse = att(q, k, v, starts([n]), softmax_scale=1.0, return_lse=True)
        check(out, lse, q, k, v, [n], [n], True, 1.0, 2, some=80)


def test_fused_views_and_given_outputs():
    rng = np.random.default_rng(8)
    lens, H, r = [90, 130], 2, 4
    qkv = rows(rng, 240, H * r + 2 * H, torch.float16)  # 20 rows of no sequence at the end
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    att = PromptAttention(n_kv_heads=H, gqa_ratio=r)
    wide = torch.full((240, 10, 128), 7.0, dtype=torch.float16, device="cuda")
    out = att(q, k, v, starts(lens), softmax_scale=SCALE, out=wide[:, 1:9])
    assert out.data_ptr() == wide[:, 1:9].data_ptr()
    check(out, None, q, k, v, lens, lens, True, SCALE, r)
    assert (wide[:, 0] == 7).all() and (wide[:, 9] == 7).all() and (wide[220:] == 7).all()
    new, lse = att(q, k, v, starts(lens), softmax_scale=SCALE, return_lse=True)
    assert torch.equal(new[:220], out[:220]) and not new[220:].any() and (lse[220:] == -math.inf).all()
    late = starts(lens) + 20  # rows of no sequence in front
    out = att(q, k, v, late, softmax_scale=SCALE, out=torch.full_like(new, 3.0))
    assert (out[:20] == 3).all()
    check(out[20:], None, q[20:], k[20:], v[20:], lens, lens, True, SCALE, r)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_values_of_one_sequence_stay_in_it(dtype):
    """Infinities and NaN in the neighbours' keys, values and queries and in rows of no sequence."""
    rng = np.random.default_rng(9)
    lens, H, r = [50, 37, 201, 20], 2, 4
    n = sum(lens) + 30
    q, k, v = rows(rng, n, H * r, dtype), rows(rng, n, H, dtype), rows(rng, n, H, dtype)
    att = PromptAttention(n_kv_heads=H, gqa_ratio=r, dtype=dtype)
    want, wl = att(q, k, v, starts(lens), softmax_scale=SCALE, return_lse=True)
    for value in (math.inf, -math.inf, math.nan):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for x in (q2, k2, v2):
            x[50:87] = value
            x[288:] = value
        got, gl = att(q2, k2, v2, starts(lens), softmax_scale=SCALE, return_lse=True)
        for a, b in ((0, 50), (87, 288)):
            assert torch.equal(got[a:b], want[a:b]) and torch.equal(gl[a:b], wl[a:b])


@pytest.mark.parametrize("q_lens,kv_lens,r,H", [
    ([1], [5000], 4, 2), ([40], [2200], 4, 8), ([64, 1, 30], [4000, 100, 2111], 4, 2), ([300], [2100], 8, 1),
    ([900], [9000], 4, 8), ([2300], [2300], 4, 8), ([200, 100], [150, 6000], 2, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_few_rows_over_many_keys(q_lens, kv_lens, r, H, causal):
    """Work that is split along the keys and joined; twice, since the counters have to be left at zero."""
    att, q, k, v, out, lse = run(q_lens, kv_lens=kv_lens, r=r, H=H, seed=12, causal=causal, some=6)
    again, lse2 = att(q, k, v, starts(q_lens), kv_start=starts(kv_lens), softmax_scale=SCALE, causal=causal, return_lse=True)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert not att.ws[256:1024].any()


def test_split_work_keeps_nan_and_masked_rows():
    rng = np.random.default_rng(13)
    q, k, v = rows(rng, 70, 4, torch.float16), rows(rng, 4000, 1, torch.float16), rows(rng, 4000, 1, torch.float16)
    att = PromptAttention(n_kv_heads=1, gqa_ratio=4)
    args = dict(kv_start=starts([4000]), softmax_scale=SCALE, return_lse=True)
    want, _ = att(q, k, v, starts([70]), **args)
    k[17] = math.nan  # every row sees it
    out, lse = att(q, k, v, starts([70]), **args)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    k[17], v[3999] = 0.0, 0.0
    q[5, 2] = math.nan  # one row
    out, lse = att(q, k, v, starts([70]), **args)
    assert torch.isnan(out[5, 2]).all() and torch.isfinite(out[:5]).all() and torch.isfinite(out[6:]).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,m,r", [(70, 70, 4), (300, 300, 1), (513, 700, 8), (40, 4100, 4), (130, 100, 2)])
def test_values_behind_a_query_do_not_reach_it(n, m, r, dtype):
    """Causal: infinities and NaN among the keys and values that a query does not see yet."""
    rng = np.random.default_rng(15)
    q, k, v = rows(rng, n, 2 * r, dtype), rows(rng, m, 2, dtype), rows(rng, m, 2, dtype)
    att = PromptAttention(n_kv_heads=2, gqa_ratio=r, dtype=dtype)
    args = dict(kv_start=starts([m]), softmax_scale=SCALE, return_lse=True)
    want, wl = att(q, k, v, starts([n]), **args)
    for at in sorted({m - 1, m - 2, max(m - 17, 0), max(m - n // 2, 0), max(m - n + 1, 0)}):
        first = max(n - m + at, 0)  # the first query that sees key `at`
        for value in (math.nan, math.inf):
            v2 = v.clone()
            v2[at, 0, 5] = value
            got, gl = att(q, k, v2, starts([n]), **args)
            check(got[:first], gl[:first], q[:first], k[:at], v[:at], [first], [at], True, SCALE, r, some=12)
            assert not torch.isfinite(got[first:, :r, 5]).any()
            clean = torch.ones(128, dtype=torch.bool)
            clean[5] = False
            assert torch.isfinite(got[:, r:]).all() and torch.isfinite(got[:, :, clean.cuda()]).all()
            assert torch.equal(got[:, r:], want[:, r:]) and torch.equal(gl, wl)
        k2 = k.clone()
        k2[at, 1] = math.nan
        got, gl = att(q, k2, v, starts([n]), **args)
        assert torch.equal(got[:first], want[:first]) and torch.equal(gl[:first], wl[:first])
        assert torch.isnan(got[first:, r:]).all() and torch.equal(got[:, :r], want[:, :r])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_infinite_scores_next_to_spoiled_values(dtype):
    """Rows in front of a value that is not finite: a score of -inf has weight 0 there too, and with a
    scale of 0 infinite products count as 0."""
    rng = np.random.default_rng(15)
    n, r = 40, 4
    q, k, v = rows(rng, n, 2 * r, dtype), rows(rng, n, 2, dtype), rows(rng, n, 2, dtype)
    q[:, :, 0] = 1.0
    att = PromptAttention(n_kv_heads=2, gqa_ratio=r, dtype=dtype)
    low = k.clone()
    low[0, :, 0] = -math.inf
    spoiled = v.clone()
    spoiled[n - 1, :, 5] = math.inf
    for values in (v, spoiled):
        got, lse = att(q, low, values, starts([n]), softmax_scale=SCALE, return_lse=True)
        assert torch.isnan(got[0]).all()
        check(got[1:n - 1], lse[1:n - 1], q[1:n - 1], k[1:n - 1], v[1:n - 1], [n - 2], [n - 2], True, SCALE, r)
        got, lse = att(q, low, values, starts([n]), softmax_scale=0.0, return_lse=True)
        check(got[:n - 1], lse[:n - 1], q[:n - 1], k[:n - 1], v[:n - 1], [n - 1], [n - 1], True, 0.0, r)


def test_bad_starts_do_not_leave_the_rows():
    """Starts beyond the rows or decreasing are clamped: outputs are unspecified there, the other rows stand."""
    rng = np.random.default_rng(10)
    q, k, v = rows(rng, 100, 8, torch.float16), rows(rng, 100, 2, torch.float16), rows(rng, 100, 2, torch.float16)
    att = PromptAttention(n_kv_heads=2, gqa_ratio=4)
    good = att(q, k, v, starts([60, 40]), softmax_scale=SCALE)
    for bad in ([0, 60, 500], [0, 60, -5], [0, 60, 2 ** 31 - 1]):
        t = torch.tensor(bad, dtype=torch.int32, device="cuda")
        assert torch.equal(att(q, k, v, t, softmax_scale=SCALE)[:60], good[:60])
    att(q, k, v, torch.tensor([-2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), softmax_scale=SCALE)
    torch.cuda.synchronize()


def test_streams_and_graph():
    rng = np.random.default_rng(11)
    lens = [200, 333]
    q, k, v = rows(rng, 533, 8, torch.bfloat16), rows(rng, 533, 2, torch.bfloat16), rows(rng, 533, 2, torch.bfloat16)
    att, s = PromptAttention(n_kv_heads=2, gqa_ratio=4, dtype=torch.bfloat16), starts(lens)
    want = att(q, k, v, s, softmax_scale=SCALE)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    each = [PromptAttention(n_kv_heads=2, gqa_ratio=4, dtype=torch.bfloat16) for _ in streams]
    torch.cuda.synchronize()
    for x, a in list(zip(streams, each)) * 3:
        with torch.cuda.stream(x):
            outs.append(a(q, k, v, s, softmax_scale=SCALE))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in outs)
    out, graph = torch.zeros_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att(q, k, v, s, softmax_scale=SCALE, out=out)
    for cut in ([533, 0], [1, 532], lens):
        s.copy_(starts(cut))
        graph.replay()
        assert torch.equal(out, att(q, k, v, s, softmax_scale=SCALE))
    assert torch.equal(out, want)


@pytest.mark.parametrize("n,m", [(20, 20), (700, 700), (40, 9000)])
def test_a_wait_that_runs_out_is_reported(n, m):
    """Every wait gives up at once: the error word says so, and the next call is right."""
    rng = np.random.default_rng(14)
    q, k, v = rows(rng, n, 8, torch.float16), rows(rng, m, 2, torch.float16), rows(rng, m, 2, torch.float16)
    att = PromptAttention(n_kv_heads=2, gqa_ratio=4)
    args = dict(kv_start=starts([m]), softmax_scale=SCALE)
    att(q, k, v, starts([n]), flags=kvq.PROMPT_ZERO_WAIT_LIMIT, **args)
    with pytest.raises(kvq.KVQDeviceError) as e:
        att.check_errors()
    assert e.value.word == kvq.DECODE_ERR_WAIT_TIMEOUT
    out = att(q, k, v, starts([n]), **args)
    check(out, None, q, k, v, [n], [m], True, SCALE, 4, some=20)
    att.check_errors()


def test_refusals_of_the_caller():
    att = PromptAttention(n_kv_heads=2, gqa_ratio=4)
    z = lambda *s, dtype=torch.float16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    good = dict(q=z(9, 8, 128), k=z(9, 2, 128), v=z(9, 2, 128), q_start=starts([9]))
    call = lambda **kw: att(**{**good, **kw}, softmax_scale=SCALE)  # noqa: E731
    for kw in (dict(q=z(9, 4, 128)), dict(k=z(8, 2, 128)), dict(q=good["q"].cpu()), dict(q_start=starts([9]).long()),
               dict(q_start=starts([])), dict(kv_start=starts([4, 5])), dict(out=z(9, 2, 128)), dict(v=z(9, 2, 64))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(TypeError):
        call(q=good["q"].bfloat16())
    with pytest.raises(RuntimeError):
        att(**good, softmax_scale=-1.0)
