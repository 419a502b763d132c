"""The serving operators of the paged 8-bit KV cache as measured cases: step tables, append and read back,
decode attention, and prompt attention over packed sequences.

``run`` computes an operator either in its plain form (elementary torch operations, binary32) or, with ``own`` set,
through the framework's calls. ``exact`` gives the results in 64 bits from the definitions.
"""

import math
import random

import torch

own = False

D = 128  # head dimension of the cache
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
TOP = {"int8": 127.0, "e4m3": 448.0}  # largest code of each cache format


# ---- cases -----------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a full batch: every request gets a token, a few finish and hand their blocks back
        dict(name="tables-step-64", kind="tables", requests=64, block=64, low=1, high=8192, new="token", gone=0.05),
        # a scheduler's mixed step: a thousand requests, most decode one token, others bring whole prompts
        dict(name="tables-mixed-1000", kind="tables", requests=1000, block=32, low=1, high=4096, new="mixed", gone=0.1),
        # one token per request into short contexts, the read-back of a test or an inspection after it
        dict(name="append-token-32", kind="append", requests=32, heads=8, block=64, fmt="e4m3", dtype="bf16", low=1,
             high=192, new="token"),
        # prompts of a batch quantized into the cache, ragged, rows of one fused projection
        dict(name="append-prompts-24", kind="append", requests=24, heads=8, block=64, fmt="int8", dtype="f16", low=100,
             high=4096, new="prompt"),
        # a single chat at 4k tokens: latency counts
        dict(name="decode-1x4096", kind="decode", requests=1, heads=8, ratio=4, block=64, fmt="int8", dtype="f16",
             low=4096, high=4096),
        # many chats of very different lengths
        dict(name="decode-64-ragged", kind="decode", requests=64, heads=8, ratio=4, block=32, fmt="e4m3", dtype="bf16",
             low=1, high=4096),
        # a steady batch at 8k tokens
        dict(name="decode-16x8192", kind="decode", requests=16, heads=8, ratio=4, block=64, fmt="int8", dtype="f16",
             low=8100, high=8250),
        # two long documents, eight query heads on each kv head
        dict(name="decode-2x65536", kind="decode", requests=2, heads=8, ratio=8, block=128, fmt="e4m3", dtype="f16",
             low=65536, high=65600),
        # a short question
        dict(name="prompt-1x77", kind="prompt", seqs=1, heads=8, ratio=4, dtype="f16", low=77, high=77, context=0,
             causal=True, fused=True),
        # a batch of ragged prompts packed one behind the other
        dict(name="prompt-12-ragged", kind="prompt", seqs=12, heads=8, ratio=4, dtype="f16", low=17, high=2048,
             context=0, causal=True, fused=True),
        # one long prompt
        dict(name="prompt-1x8192", kind="prompt", seqs=1, heads=8, ratio=4, dtype="bf16", low=8192, high=8192,
             context=0, causal=True, fused=False),
        # the next chunks of long prompts: their keys hold the chunks before as well
        dict(name="prompt-chunk-2", kind="prompt", seqs=2, heads=8, ratio=8, dtype="bf16", low=900, high=1100,
             context=9000, causal=True, fused=False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["tables", "append", "decode", "decode", "prompt", "prompt"])
    if kind == "tables":
        return dict(kind=kind, requests=_log(rng, 1, 1000), block=rng.choice([32, 64, 128]), low=1,
                    high=_log(rng, 16, 4096), new=rng.choice(["token", "mixed"]), gone=rng.choice([0.0, 0.05, 0.2]))
    fmt, dtype, block = rng.choice(["int8", "e4m3"]), rng.choice(["f16", "bf16"]), rng.choice([32, 64, 128])
    if kind == "append":
        new = rng.choice(["token", "prompt"])
        requests = _log(rng, 1, 32)
        high = _log(rng, 1, 256 if new == "token" else 2048)
        return dict(kind=kind, requests=requests, heads=rng.randint(1, 8), block=block, fmt=fmt, dtype=dtype, low=1,
                    high=high, new=new)
    if kind == "decode":
        requests = _log(rng, 1, 96)
        high = _log(rng, 1, 131072 // requests)
        return dict(kind=kind, requests=requests, heads=rng.randint(1, 8), ratio=rng.randint(1, 8), block=block,
                    fmt=fmt, dtype=dtype, low=rng.choice([1, max(1, high // 2)]), high=high)
    seqs = _log(rng, 1, 12)
    high = _log(rng, 1, 6000 // seqs)
    return dict(kind=kind, seqs=seqs, heads=rng.randint(1, 8), ratio=rng.randint(1, 4), dtype=dtype,
                low=rng.choice([1, max(1, high // 2)]), high=high, context=rng.choice([0, 0, _log(rng, 1, 2000)]),
                causal=rng.random() < 0.8, fused=rng.random() < 0.5)


def _plain(case):
    return {k: v for k, v in case.items() if k != "name"}


def _rng(case, what):
    return random.Random(what + repr(sorted(_plain(case).items())))


def _lens(case, n, what="lens"):
    """n lengths of the case's range, spread over their logarithm; the same for every seed."""
    rng = _rng(case, what)
    return [_log(rng, case["low"], case["high"]) if case["high"] > 1 else 1 for _ in range(n)]


def _steps(case):
    """(tokens held, tokens to add) of each request; -1 stands for a request that is done and leaves."""
    rng = _rng(case, "steps")
    held, new = [], []
    for n in _lens(case, case["requests"]):
        if case["kind"] == "tables":
            if rng.random() < case["gone"]:
                held.append(n), new.append(-1)
            elif case["new"] == "mixed" and rng.random() < 0.2:
                held.append(0), new.append(n)
            else:
                held.append(n), new.append(1)
        else:  # n tokens after the append
            held.append(n - 1 if case["new"] == "token" else 0), new.append(1 if case["new"] == "token" else n)
    return held, new


def work(case):
    size = 2
    if case["kind"] == "tables":
        held, new = _steps(case)
        n, bt = len(held), case["block"]
        tokens = sum(x for x in new if x > 0)
        blocks = sum((h + x) // bt - h // bt for h, x in zip(held, new) if x > 0)
        gone = sum(h // bt for h, x in zip(held, new) if x < 0)
        return {"bytes": 4 * (3 * n + n + 1) + 8 * (blocks + gone) + 8 * tokens, "flops": 0}
    if case["kind"] == "append":
        held, new = _steps(case)
        h, bt = case["heads"], case["block"]
        tokens, total = sum(new), sum(held) + sum(new)
        codes = total * h * 2 * D  # every row is read back: codes (or 16-bit rows) in, binary32 out
        return {"bytes": tokens * h * 2 * D * (size + 1) + codes + total * h * 2 * D * 4 + total * h * 8 // bt + 4 * total,
                "flops": 4 * tokens * h * D + 2 * total * h * D}
    if case["kind"] == "decode":
        lens, bt, h, r = _lens(case, case["requests"]), case["block"], case["heads"], case["ratio"]
        full = sum(n // bt * bt for n in lens)
        tail = sum(n % bt for n in lens)
        return {"bytes": h * (full * 2 * D + tail * 2 * D * size + full // bt * 8) + len(lens) * h * r * D * 2 * size,
                "flops": 4 * D * h * r * (full + tail)}
    lens = _lens(case, case["seqs"])
    ctx = _contexts(case)
    h, r = case["heads"], case["ratio"]
    pairs = sum(q * (q + 1) // 2 + q * c if case["causal"] else q * (q + c) for q, c in zip(lens, ctx))
    return {"bytes": (sum(lens) * h * r * 2 + (sum(lens) + sum(ctx)) * h * 2) * D * size + sum(lens) * h * r * 4,
            "flops": 4 * D * h * r * pairs}


def _contexts(case):
    rng = _rng(case, "context")
    return [rng.randint(case["context"] // 2, case["context"]) for _ in range(case["seqs"])]


# ---- inputs ----------------------------------------------------------------------------------------------------

def _keys(shape, gen, dtype):
    """Normal keys with four large channels per head, as the projections of a trained model give them."""
    x = torch.randn(shape, generator=gen, device="cuda")
    gain = torch.ones(shape[-2:], device="cuda")
    pick = torch.rand(shape[-2:], generator=gen, device="cuda").argsort(-1)[:, :4]
    gain.scatter_(1, pick, 20.0)
    return (x * gain + 5.0 * (gain > 1)).to(dtype)


def _values(shape, gen, dtype):
    return (0.5 * torch.randn(shape, generator=gen, device="cuda")).to(dtype)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _rows(lens):
    """(request, position) of every token of packed requests."""
    n = torch.tensor(lens, device="cuda")
    row = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), n, output_size=sum(lens))
    return row, torch.arange(sum(lens), device="cuda") - (n.cumsum(0) - n)[row]


def _context_rows(case, seed):
    """Keys and values of every token of every request (packed), and the tokens held and added."""
    if case["kind"] == "append":
        held, new = _steps(case)
    else:
        held = _lens(case, case["requests"])
        new = [1] * len(held)
        held = [n - 1 for n in held]
    gen = _gen(seed)
    total = sum(held) + sum(new)
    dtype = TYPES[case["dtype"]]
    kv = torch.empty((total, 2 * case["heads"], D), dtype=dtype, device="cuda")  # rows of one fused projection
    kv[:, :case["heads"]] = _keys((total, case["heads"], D), gen, dtype)
    kv[:, case["heads"]:] = _values((total, case["heads"], D), gen, dtype)
    return held, new, kv, gen


def prepare(case, seed):
    if case["kind"] == "tables":
        return _prepare_tables(case, seed)
    if case["kind"] == "prompt":
        return _prepare_prompt(case, seed)
    held, new, kv, gen = _context_rows(case, seed)
    h = case["heads"]
    after = [a + b for a, b in zip(held, new)]
    row, pos = _rows(after)
    is_new = pos >= torch.tensor(held, device="cuda")[row]
    state = dict(case=case, fresh=kv[is_new], new=new, held=held, after=after, row=row, pos=pos, is_new=is_new)
    if case["kind"] == "decode":
        state["q"] = torch.randn((len(new), h * case["ratio"], D), generator=gen, device="cuda").to(kv.dtype)
    if own:
        state["cache"] = _own_cache(case, state, kv)
    else:
        state["held_rows"] = _plain_held(case, state, kv)
    return state


def _own_cache(case, state, kv):
    """The framework's cache with the held tokens in it and the step planned (decode: the new token appended too)."""
    from bit_kv_cache_09_gb300.paged import PagedKVCache

    h, bt, after = case["heads"], case["block"], state["after"]
    cache = PagedKVCache(n_layers=1, n_kv_heads=h, gqa_ratio=case.get("ratio", 1), d_head=D,
                         n_blocks=sum(n // bt for n in after) + 3, block_tokens=bt, n_requests=len(after),
                         max_blocks=max(after) // bt + 1, max_new=max(1, sum(after)), fmt=case["fmt"], dtype=kv.dtype)
    if sum(state["held"]):
        cache.step(_int(state["held"]))
        rows = kv[~state["is_new"]]
        cache.append(0, rows[:, :h], rows[:, h:])
    cache.step(_int(state["new"]), commit=False)
    if case["kind"] == "decode":
        cache.append(0, state["fresh"][:, :h], state["fresh"][:, h:])
    row, pos = state["row"], state["pos"]
    full = torch.tensor(after, device="cuda")[row] // bt
    page = cache.block_table[row, torch.clamp(pos // bt, max=cache.block_table.shape[1] - 1)].long()
    state["slots"] = torch.where(pos // bt < full, page * bt + pos % bt, -1 - (row * bt + pos % bt)).int()
    return cache


def _prepare_tables(case, seed):
    held, new = _steps(case)
    bt, n = case["block"], case["requests"]
    used = sum(x // bt for x in held)
    need = sum((a + b) // bt - a // bt for a, b in zip(held, new) if b > 0)
    n_blocks = used + need + 5
    ids = torch.randperm(n_blocks, generator=_gen(seed), device="cuda").int()
    width = max(a + max(b, 0) for a, b in zip(held, new)) // bt + 1
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    blocks = [x // bt for x in held]
    row, pos = _rows(blocks)
    table[row, pos] = ids[:used]
    free = torch.zeros(n_blocks, dtype=torch.int32, device="cuda")
    free[:n_blocks - used] = ids[used:]
    state = dict(case=case, table=table, free=free, count=_int([n_blocks - used]), held=_int(held), new=_int(new),
                 tokens=sum(x for x in new if x > 0), n_blocks=n_blocks, held_list=held, new_list=new)
    if own:
        from bit_kv_cache_09_gb300.paged import PagedKVCache

        cache = PagedKVCache(n_layers=1, n_kv_heads=1, gqa_ratio=1, d_head=D, n_blocks=n_blocks, block_tokens=bt,
                             n_requests=n, max_blocks=width, max_new=max(1, state["tokens"]), fmt="int8",
                             dtype=torch.float16)
        cache.block_table.copy_(table), cache.free_list.copy_(free), cache.free_count.copy_(state["count"])
        cache.lens.copy_(state["held"])
        state["cache"] = cache
    return state


def _prepare_prompt(case, seed):
    lens, ctx = _lens(case, case["seqs"]), _contexts(case)
    h, nq, dtype, gen = case["heads"], case["heads"] * case["ratio"], TYPES[case["dtype"]], _gen(seed)
    kv_lens = [a + b for a, b in zip(lens, ctx)]
    nt, nk = sum(lens), sum(kv_lens)
    q = torch.randn((nt, nq, D), generator=gen, device="cuda").to(dtype)
    k, v = _keys((nk, h, D), gen, dtype), _values((nk, h, D), gen, dtype)
    if case["fused"] and nt == nk:  # views of one projection's output, as a model has them
        qkv = torch.cat([q, k, v], dim=1)
        q, k, v = qkv[:, :nq], qkv[:, nq:nq + h], qkv[:, nq + h:]
    state = dict(case=case, q=q, k=k, v=v, lens=lens, kv_lens=kv_lens,
                 q_start=_int([sum(lens[:i]) for i in range(len(lens) + 1)]),
                 kv_start=_int([sum(kv_lens[:i]) for i in range(len(lens) + 1)]))
    if own:
        from bit_kv_cache_09_gb300.prompt import PromptAttention

        state["attention"] = PromptAttention(n_kv_heads=h, gqa_ratio=case["ratio"], d_head=D, dtype=dtype)
    return state


# ---- one pass --------------------------------------------------------------------------------------------------

def run(state):
    case = state["case"]
    kind = case["kind"]
    scale = 1.0 / math.sqrt(D)
    if own:
        if kind == "prompt":
            out, lse = state["attention"](state["q"], state["k"], state["v"], state["q_start"],
                                          kv_start=state["kv_start"], softmax_scale=scale, causal=case["causal"],
                                          return_lse=True)
            return {"out": out, "lse": lse}
        cache = state["cache"]
        if kind == "tables":
            step = cache.step(state["new"], commit=False)
            return {"block_table": cache.block_table, "free_list": cache.free_list, "free_count": step.free_count,
                    "lens": step.lens, "q_start": step.q_start, "positions": step.positions[:state["tokens"]],
                    "slots": step.slots[:state["tokens"]]}
        if kind == "append":
            cache.append(0, state["fresh"][:, :case["heads"]], state["fresh"][:, case["heads"]:])
            k, v = cache.dequantize(0, state["slots"])
            return {"k": k, "v": v}
        return {"out": cache.attention(0, state["q"], scale)}
    if kind == "tables":
        return _tables_plain(state)
    if kind == "append":
        return _append_plain(state)
    if kind == "decode":
        return _decode_plain(state, scale)
    return _prompt_plain(state, scale)


# ---- plain forms -----------------------------------------------------------------------------------------------

def _tables_plain(state):
    bt, n, tokens = state["case"]["block"], state["case"]["requests"], state["tokens"]
    held, new = state["held"].long(), state["new"].long()
    gone = new < 0
    add = torch.clamp(new, min=0)
    after = torch.where(gone, torch.zeros_like(held), held + add)
    had, has = held // bt, (held + add) // bt
    rows = torch.arange(n, device=held.device)
    # released blocks go onto the free stack in row order
    free = state["free"].clone()
    count = state["count"].long()
    back = torch.where(gone, had, torch.zeros_like(had))
    width = state["table"].shape[1]
    col = torch.arange(width, device=held.device)
    place = (back.cumsum(0) - back)[:, None] + col
    taken = col < back[:, None]
    stack = torch.cat([free.long(), torch.zeros(1, dtype=torch.long, device=held.device)])
    stack = stack.scatter(0, torch.where(taken, count + place, free.numel()).view(-1), state["table"].long().reshape(-1))
    top = count + back.sum()
    # new blocks come from its top in row order
    want = torch.where(gone, torch.zeros_like(had), has - had)
    nth = (want.cumsum(0) - want)[:, None] + (col - had[:, None])
    fresh = (col >= had[:, None]) & (col < (had + want)[:, None])
    table = torch.where(fresh, stack[torch.clamp(top - 1 - nth, min=0, max=free.numel() - 1)].int(), state["table"])
    left = top - want.sum()
    at = torch.arange(free.numel(), device=held.device)
    free = torch.where((at >= count) & (at < left), stack[:-1].int(), free)
    q_start = torch.cat([add.new_zeros(1), add.cumsum(0)])
    row = torch.repeat_interleave(rows, add, output_size=tokens)
    pos = held[row] + torch.arange(tokens, device=held.device) - q_start[row]
    page = table[row, torch.clamp(pos // bt, max=width - 1)].long()
    slots = torch.where(pos // bt < after[row] // bt, page * bt + pos % bt, -1 - (row * bt + pos % bt))
    return {"block_table": table, "free_list": free, "free_count": left.int(), "lens": after.int(),
            "q_start": q_start.int(), "positions": pos.int(), "slots": slots.int()}


def _quantized(x, fmt):
    """Codes (as binary32) and scales of [.., block, heads, D] rows: one scale for the block's rows of a head."""
    amax = x.abs().amax(dim=(-3, -1), keepdim=True)
    scale = torch.clamp((amax.double() / TOP[fmt]).float(), min=2.0 ** -126)
    scale = torch.where(amax == 0, torch.ones_like(scale), scale)
    y = (x.double() / scale.double()).float()
    if fmt == "int8":
        return torch.clamp(torch.round(y), -127, 127), scale
    return torch.clamp(y, -448, 448).to(torch.float8_e4m3fn).float(), scale


def _padded(packed, row, pos, requests, length):
    out = torch.zeros((requests, length) + packed.shape[1:], dtype=packed.dtype, device=packed.device)
    out[row, pos] = packed
    return out


def _plain_held(case, state, kv):
    """The held tokens as a plain cache has them: codes and scales of full blocks, 16-bit rows of the last one."""
    bt, held = case["block"], state["held"] if case["kind"] == "append" else state["after"]
    n, blocks = len(held), max(state["after"]) // bt + 1
    keep = state["pos"] < torch.tensor(held, device="cuda")[state["row"]]
    rows = _padded(kv[keep], state["row"][keep], state["pos"][keep], n, blocks * bt)
    codes, scale = _quantized(rows.float().view(n, blocks, bt, 2 * case["heads"], D), case["fmt"])
    codes = codes.to(torch.int8 if case["fmt"] == "int8" else torch.float8_e4m3fn)
    lens = torch.tensor(held, device="cuda")
    tail = torch.clamp((lens // bt * bt)[:, None] + torch.arange(bt, device="cuda"), max=blocks * bt - 1)
    return dict(codes=codes, scale=scale, tail=torch.gather(rows, 1, tail[:, :, None, None].expand(-1, -1, 2 * case["heads"], D)),
                lens=lens, blocks=blocks)


def _held_values(held, bt):
    """Rows of a plain cache in binary32, padded: code x scale of full blocks, then the 16-bit rows."""
    n, blocks = held["codes"].shape[:2]
    x = (held["codes"].float() * held["scale"]).view((n, blocks * bt) + held["codes"].shape[3:])
    at = torch.arange(blocks * bt, device=x.device)
    full = (held["lens"] // bt * bt)[:, None]
    tail = held["tail"].float().repeat(1, blocks, 1, 1)  # row p of an unfinished block sits at p mod bt
    return torch.where((at < full)[:, :, None, None], x, tail), full


def _append_plain(state):
    case, held = state["case"], state["held_rows"]
    bt, h = case["block"], case["heads"]
    rows, full = _held_values(held, bt)
    n, length = rows.shape[:2]
    row, pos = state["row"], state["pos"]
    rows[row[state["is_new"]], pos[state["is_new"]]] = state["fresh"].float()
    codes, scale = _quantized(rows.view(n, length // bt, bt, 2 * h, D), case["fmt"])
    after = torch.tensor(state["after"], device=rows.device)
    at = torch.arange(length, device=rows.device)
    done = (at >= full) & (at < (after // bt * bt)[:, None])
    rows = torch.where(done[:, :, None, None], (codes * scale).view(rows.shape), rows)
    out = rows[row, pos]
    return {"k": out[:, :h].contiguous(), "v": out[:, h:].contiguous()}


def _decode_plain(state, scale):
    case = state["case"]
    h, r = case["heads"], case["ratio"]
    rows, _ = _held_values(state["held_rows"], case["block"])
    n, length = rows.shape[:2]
    k, v = rows[:, :, :h].permute(0, 2, 1, 3), rows[:, :, h:].permute(0, 2, 1, 3)
    q = state["q"].float().view(n, h, r, D)
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    there = torch.arange(length, device=s.device) < state["held_rows"]["lens"][:, None]
    s = torch.where(there[:, None, None], s, torch.full_like(s, -math.inf))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    v = torch.where(there[:, None, :, None], v, torch.zeros_like(v))
    out = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return {"out": out.reshape(n, h * r, D).to(state["q"].dtype)}


def _prompt_plain(state, scale):
    case = state["case"]
    h, r, seqs = case["heads"], case["ratio"], case["seqs"]
    lens, kv_lens = state["lens"], state["kv_lens"]
    lq, lk = torch.tensor(lens, device="cuda"), torch.tensor(kv_lens, device="cuda")
    (qr, qp), (kr, kp) = _rows(lens), _rows(kv_lens)
    nq, nk = max(lens), max(kv_lens)
    q = _padded(state["q"].float().view(-1, h, r, D), qr, qp, seqs, nq).permute(0, 2, 3, 1, 4).reshape(seqs, h, r * nq, D)
    k = _padded(state["k"].float(), kr, kp, seqs, nk).permute(0, 2, 3, 1)
    v = _padded(state["v"].float(), kr, kp, seqs, nk).permute(0, 2, 1, 3)
    s = (torch.matmul(q, k) * scale).view(seqs, h, r, nq, nk)
    at = torch.arange(nk, device=s.device)
    there = (at < lk[:, None])[:, None, :].expand(-1, nq, -1)
    if case["causal"]:
        there = there & (at <= torch.arange(nq, device=s.device)[None, :, None] + (lk - lq)[:, None, None])
    s = s.masked_fill(~there[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(seqs, h, r * nq, nk), v).view(seqs, h, r, nq, D)
    out = out / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(seqs, nq, h * r)
    out = out.permute(0, 3, 1, 2, 4).reshape(seqs, nq, h * r, D)
    return {"out": out[qr, qp].to(state["q"].dtype), "lse": lse[qr, qp]}


# ---- the definitions in 64 bits --------------------------------------------------------------------------------

def _exact_block(x, fmt):
    """The values one block of one head stands for after quantization. x: [tokens, D] float64."""
    amax = float(x.abs().max())
    scale = 1.0 if amax == 0.0 else max(float(torch.tensor(amax / TOP[fmt], dtype=torch.float64).float()), 2.0 ** -126)
    y = (x / scale).float().double()  # the operator's quotient is binary32
    if fmt == "int8":
        return y.round() * scale
    m, _ = torch.frexp(y)
    step = torch.clamp(y / torch.where(m == 0, torch.ones_like(m), m) / 16, min=2.0 ** -9)  # exact powers of two
    return (y / step).round() * step * scale


def _exact_rows(x, n, bt, fmt):
    """Held values of one request: x [n, heads, D] float64, full blocks quantized."""
    out = x.clone()
    for b in range(n // bt):
        for j in range(x.shape[1]):
            out[b * bt:(b + 1) * bt, j] = _exact_block(x[b * bt:(b + 1) * bt, j], fmt)
    return out


def exact(case, seed):
    if case["kind"] == "tables":
        return _exact_tables(case, seed)
    scale = 1.0 / math.sqrt(D)
    if case["kind"] == "prompt":
        return _exact_prompt(case, seed, scale)
    state = dict(zip(("held", "new", "kv", "gen"), _context_rows(case, seed)))
    h, bt = case["heads"], case["block"]
    after = [a + b for a, b in zip(state["held"], state["new"])]
    if sum(n // bt for n in after) * 2 * h > 60000:  # a block and head at a time would take too long
        return None
    first, rows = 0, []
    for n in after:
        rows.append(_exact_rows(state["kv"][first:first + n].double(), n, bt, case["fmt"]))
        first += n
    if case["kind"] == "append":
        rows = torch.cat(rows)
        return {"k": rows[:, :h], "v": rows[:, h:]}
    q = torch.randn((len(after), h * case["ratio"], D), generator=state["gen"], device="cuda").to(state["kv"].dtype)
    outs = []
    for i, x in enumerate(rows):
        for j in range(h):
            s = q[i, j * case["ratio"]:(j + 1) * case["ratio"]].double() @ x[:, j].T * scale
            outs.append(torch.softmax(s, -1) @ x[:, h + j])
    return {"out": torch.stack(outs).reshape(len(after), h * case["ratio"], D)}


def _exact_prompt(case, seed, scale):
    state = _prepare_prompt(case, seed)
    r = case["ratio"]
    outs, lses, q0, k0 = [], [], 0, 0
    for n, m in zip(state["lens"], state["kv_lens"]):
        heads, tops = [], []
        hide = None
        if case["causal"]:
            hide = torch.ones((n, m), dtype=torch.bool, device="cuda").triu(m - n + 1)
        for j in range(case["heads"] * r):
            s = state["q"][q0:q0 + n, j].double() @ state["k"][k0:k0 + m, j // r].double().T * scale
            if hide is not None:
                s.masked_fill_(hide, -math.inf)
            lse = torch.logsumexp(s, -1)
            heads.append(torch.exp(s - lse[:, None]) @ state["v"][k0:k0 + m, j // r].double())
            tops.append(lse)
        outs.append(torch.stack(heads, 1)), lses.append(torch.stack(tops, 1))
        q0, k0 = q0 + n, k0 + m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_tables(case, seed):
    state = _prepare_tables(case, seed)
    bt = case["block"]
    table, free = state["table"].tolist(), state["free"].tolist()
    held, new, count = state["held_list"], state["new_list"], int(state["count"])
    stack = free[:count]
    for i, x in enumerate(new):
        if x < 0:
            stack += table[i][:held[i] // bt]
    lens, q_start, positions, slots = [], [0], [], []
    for i, x in enumerate(new):
        after = 0 if x < 0 else held[i] + x
        if x > 0:
            for b in range(held[i] // bt, after // bt):
                table[i][b] = stack.pop()
            for p in range(held[i], after):
                positions.append(p)
                slots.append(table[i][p // bt] * bt + p % bt if p // bt < after // bt else -1 - (i * bt + p % bt))
        lens.append(after)
        q_start.append(q_start[-1] + max(x, 0))
    kept = list(free)
    for i in range(count, len(stack)):
        kept[i] = stack[i]
    return {"block_table": _int(table), "free_list": _int(kept), "free_count": _int([len(stack)]), "lens": _int(lens),
            "q_start": _int(q_start), "positions": _int(positions), "slots": _int(slots)}
