"""Workloads of the operators around the paged K/V cache: rotary positions, alone and with the
write into the pool, and attention over the pool whose scores are capped by a tanh, biased by
distance, or masked by a sliding window or a prefix.

A case is one pass of one operator ("op"): `run` computes it either in plain torch operations
or, with `own` set, through the framework's entry points.

Rotary positions ("rope", "write"): pair i of a row's first `rotary` dims turns by the angle
position * inv_freq[i]; a pair is dims (i, i + rotary/2) ("halves") or (2i, 2i + 1) ("pairs"):
    x' = amplitude * (x cos - y sin),   y' = amplitude * (x sin + y cos)
the other dims stay.  Attention ("decode", "prefill"): a query at position p attends to the
positions t of its sequence with max(0, p - window + 1) <= t <= max(p, prefix - 1):
    s = scale * <q, k_t>;  s = cap * tanh(s / cap);  s = s - slope_h * |p - t|;  out = softmax(s) V
each step only where the case has it.  Pools: k [blocks, kv heads, D/x, block size, x] with
x = 16 / element size, v [blocks, kv heads, D, block size].
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
ELEM = {"f32": 4, "f16": 2, "bf16": 2, "fp8": 1}
K_SCALE, V_SCALE = 0.0173, 0.0214          # of the FP8 pools; not powers of two


# --- the cases ------------------------------------------------------------------------------------

def _rope(op, tokens, heads, kv_heads, head_size, rotary, layout, dtype, longest, amplitude=1.0, fused=True,
          block_size=16, cache="", padded=False, name=None):
    """fused: q, k and v are views of one projection's rows [tokens, (heads + 2 kv heads) * head size]."""
    c = dict(op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, head_size=head_size, rotary=rotary, layout=layout,
             dtype=dtype, longest=longest, amplitude=amplitude, fused=fused)
    if op == "write":
        c.update(block_size=block_size, cache=cache or dtype, padded=padded)
    return dict(c, name=name) if name else c


def _decode(seqs, heads, kv_heads, head_size, block_size, shortest, longest, dtype, cap=0.0, alibi=False, window=0,
            cache="", name=None):
    c = dict(op="decode", seqs=seqs, heads=heads, kv_heads=kv_heads, head_size=head_size, block_size=block_size,
             shortest=shortest, longest=longest, dtype=dtype, cache=cache or dtype, cap=cap, alibi=alibi, window=window)
    return dict(c, name=name) if name else c


def _prefill(seqs, chunk, context, heads, kv_heads, head_size, block_size, dtype, cap=0.0, alibi=False, window=0,
             prefix=0, name=None):
    """Sequences with up to `context` cached tokens and up to `chunk` new ones; prefix: the longest prefix."""
    c = dict(op="prefill", seqs=seqs, chunk=chunk, context=context, heads=heads, kv_heads=kv_heads,
             head_size=head_size, block_size=block_size, dtype=dtype, cap=cap, alibi=alibi, window=window,
             prefix=prefix)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a generation step's rows, 28 query heads over 4 kv heads, for a cache that is written by a call of its own
        _rope("rope", 64, 28, 4, 128, 128, "halves", "f16", 4096, name="rope-step"),
        # many prompts' rows with half of each head rotated, at positions of long contexts
        _rope("rope", 16381, 32, 8, 128, 64, "pairs", "bf16", 1000000, amplitude=1.1386, name="rope-long-partial"),
        # the one new token of one request in a small layer: nothing but latency
        _rope("write", 1, 8, 2, 64, 64, "halves", "f16", 100, name="write-one-token"),
        # the chunks of 16 prompts, 512 tokens each, out of a fused projection
        _rope("write", 8192, 28, 4, 128, 128, "halves", "f16", 4096, name="write-prompts"),
        # an odd number of tokens into 8-bit pools, padding among them, a quarter of each head rotated in pairs
        _rope("write", 1537, 32, 8, 128, 32, "pairs", "bf16", 131072, block_size=32, cache="fp8", padded=True,
              name="write-fp8-padded"),
        # one short request in a small layer, capped scores: nothing but latency
        _decode(1, 8, 2, 64, 16, 100, 100, "f16", cap=50.0, name="decode-one-short"),
        # a full batch of ragged requests in a layer that looks back 1024 tokens, capped scores
        _decode(64, 28, 4, 128, 16, 512, 4096, "f16", cap=50.0, window=1024, name="decode-capped-window"),
        # a few very long contexts with capped scores
        _decode(4, 32, 8, 128, 16, 32768, 131072, "bf16", cap=30.0, name="decode-capped-long"),
        # one query head per kv head over an 8-bit cache, each head with its own bias by distance
        _decode(16, 32, 32, 128, 16, 1701, 2048, "f16", alibi=True, cache="fp8", name="decode-biased-fp8"),
        # a handful of new tokens each behind short contexts, biased by distance
        _prefill(3, 23, 300, 8, 2, 64, 16, "f16", alibi=True, name="prefill-few-tokens"),
        # 512-token chunks of 16 prompts in a layer that looks back 1024 tokens, capped scores
        _prefill(16, 512, 3584, 28, 4, 128, 16, "f16", cap=50.0, window=1024, name="prefill-capped-window"),
        # whole prompts whose first part every token sees, capped scores
        _prefill(4, 4096, 0, 32, 8, 128, 32, "bf16", cap=30.0, prefix=1111, name="prefill-prefix"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["rope", "write", "write", "decode", "decode", "decode", "prefill", "prefill"])
    d, bs = rng.choice([64, 128, 128]), rng.choice([16, 32])
    hkv, group = rng.choice([1, 2, 3, 4, 8, 8, 32]), rng.choice([1, 2, 4, 5, 7, 8, 10, 16])
    group = min(group, 64 // hkv)
    cap = rng.choice([0.0, 15.0, 30.0, 50.0])
    alibi = rng.random() < 0.35
    if op in ("rope", "write"):
        dtype = rng.choice(["f32", "f16", "f16", "bf16"])
        cache = "fp8" if op == "write" and rng.random() < 0.3 else dtype
        most = min(16384, 16381 * 40 * 128 * 2 // ((group + 2) * hkv * d * ELEM[dtype]))   # the listed ones' bytes
        tokens = _log(rng, 1, most)
        return _rope(op, tokens, hkv * group, hkv, d, rng.choice([r for r in (16, 32, 48, 64, 96, 128, d, d) if r <= d]),
                     rng.choice(["halves", "pairs"]), dtype, _log(rng, 100, 1000000), rng.choice([1.0, 1.0, 1.2079]),
                     rng.random() < 0.6, bs, cache, tokens >= 32 and rng.random() < 0.5)
    if op == "decode":
        dtype = rng.choice(["f32", "f16", "f16", "bf16", "bf16"])
        cache = "fp8" if dtype != "f32" and rng.random() < 0.3 else dtype
        s = _log(rng, 1, 256)
        most = min(131072, 300000 * 8 * 128 * 2 // (s * hkv * d * ELEM[dtype]))            # the largest listed case
        longest = _log(rng, 1, max(1, most))
        shortest = longest if rng.random() < 0.25 else max(1, int(longest * rng.uniform(0.0, 0.9)))
        window = _log(rng, 1, 2 * longest) if rng.random() < 0.5 else 0
        return _decode(s, hkv * group, hkv, d, bs, shortest, longest, dtype, cap, alibi, window, cache)
    dtype = rng.choice(["f16", "bf16"])
    s = _log(rng, 1, 32)
    # scores of the plain form (chunk x positions) and operations within the largest listed case's
    chunk = _log(rng, 1, min(4096, max(1, int(math.sqrt(4 * 4096 * 4096 * 32 / (s * hkv * group))))))
    context = _log(rng, 1, min(65536, max(1, 4 * 4096 * 4096 * 32 // (2 * s * hkv * group * chunk)),
                               max(1, 300000 * 8 * 128 // (s * hkv * d) - chunk)))
    context = 0 if rng.random() < 0.25 else context
    window = _log(rng, 1, 2 * (chunk + context)) if rng.random() < 0.5 else 0
    prefix = _log(rng, 1, chunk + context) if rng.random() < 0.35 else 0
    return _prefill(s, chunk, context, hkv * group, hkv, d, bs, dtype, cap, alibi, window, prefix)


def _spread(n, lo, hi, step=0.6180339887498949):
    """n whole numbers over [lo, hi], spread by the golden ratio from hi."""
    return [hi - int(round((hi - lo) * ((i * step) % 1.0))) for i in range(n)]


def _lens(c):
    """Per sequence: (tokens in the cache, new tokens, prefix)."""
    if c["op"] == "decode":
        return [(n, 1, 0) for n in _spread(c["seqs"], c["shortest"], c["longest"])]
    news = _spread(c["seqs"], (3 * c["chunk"] + 3) // 4, c["chunk"])
    cached = _spread(c["seqs"], c["context"] // 2, c["context"], 0.4142135623730951)
    pre = _spread(c["seqs"], c["prefix"] // 3, c["prefix"], 0.7320508075688772)
    return [(a + n, n, min(x, a + n)) for a, n, x in zip(cached, news, pre)]


def _seen(c, total, new, prefix):
    """(query, position) pairs that a sequence's new tokens see, and the first position any sees."""
    w = c["window"] or total
    pairs = 0
    first = total - new
    lo0, hi0 = max(0, first - w + 1), max(first, prefix - 1)
    # rows in runs on which both ends move in one way
    cuts = sorted({first, total} | {x for x in (w - 1, prefix - 1) if first < x < total})
    for a, b in zip(cuts, cuts[1:]):
        for end, sign in ((lambda p: max(p, prefix - 1), 1), (lambda p: max(0, p - w + 1), -1)):
            pairs += sign * (end(a) + end(b - 1)) * (b - a) // 2
        pairs += b - a
    return pairs, lo0, max(total - 1, hi0)


def work(case):
    d, hkv, h = case["head_size"], case["kv_heads"], case["heads"]
    if case["op"] in ("rope", "write"):
        t, e = case["tokens"], ELEM[case["dtype"]]
        rows = t * (2 * h + 2 * hkv) * d * e + 8 * t
        if case["op"] == "write":
            rows += t * hkv * d * 2 * ELEM[case["cache"]] + 8 * t
        return {"bytes": rows, "flops": 3 * t * (h + hkv) * case["rotary"]}
    e, kv = ELEM[case["dtype"]], ELEM[case.get("cache", case["dtype"])]
    nbytes = flops = 0
    for total, new, prefix in _lens(case):
        pairs, lo, hi = _seen(case, total, new, prefix)
        nbytes += (hi - lo + 1) * hkv * d * 2 * kv + 2 * new * h * d * e + 4
        nbytes += 4 * (hi // case["block_size"] - lo // case["block_size"] + 1)
        flops += 4 * pairs * h * d
    return {"bytes": nbytes, "flops": flops}


# --- what a program has in hand -----------------------------------------------------------------------

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _pools(gen, c, nb, st):
    """Pools of nb blocks: normal rows, key channels of different sizes; rows of a step past NaN come later."""
    d, bs, hkv, dt = c["head_size"], c["block_size"], c["kv_heads"], DTYPES[c["cache"] if "cache" in c else c["dtype"]]
    x = 16 // ELEM[c.get("cache", c["dtype"])]
    fp8 = dt == torch.float8_e4m3fn
    st["k_scale"], st["v_scale"] = (K_SCALE, V_SCALE) if fp8 else (1.0, 1.0)
    st["k_cache"] = torch.empty(nb, hkv, d // x, bs, x, dtype=dt, device="cuda")
    st["v_cache"] = torch.empty(nb, hkv, d, bs, dtype=dt, device="cuda")
    channel = torch.exp(0.3 * _randn(gen, hkv, d // x, 1, x))
    step = max(1, (1 << 26) // (hkv * bs * d))
    for a in range(0, nb, step):
        b = min(nb, a + step)
        st["k_cache"][a:b] = (_randn(gen, b - a, hkv, d // x, bs, x) * channel / st["k_scale"]).to(dt)
        st["v_cache"][a:b] = (_randn(gen, b - a, hkv, d, bs) / st["v_scale"]).to(dt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    d, hkv, h = case["head_size"], case["kv_heads"], case["heads"]
    dt = DTYPES[case["dtype"]]
    st = dict(case, dt=dt)
    if case["op"] in ("rope", "write"):
        t, r = case["tokens"], case["rotary"]
        channel = torch.exp(0.5 * _randn(gen, h + 2 * hkv, d))
        rows = (_randn(gen, t, h + 2 * hkv, d) * channel).to(dt)
        q, k, v = rows[:, :h], rows[:, h:h + hkv], rows[:, h + hkv:]
        if not case["fused"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        st["q"], st["key"], st["value"] = q, k, v
        # runs of consecutive positions, as prompts and chunks have them; a step's tokens lie anywhere
        run = 1 if t <= 256 else 512
        start = torch.randint(0, max(1, case["longest"] - run), (-(-t // run),), generator=gen, device="cuda")
        st["positions"] = (start.unsqueeze(1) + torch.arange(run, device="cuda")).flatten()[:t].contiguous()
        i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
        st["inv_freq"] = 10000.0 ** (-2.0 * i / r)
        st["q_out"] = torch.empty(t, h, d, dtype=dt, device="cuda")
        if case["op"] == "rope":
            st["k_out"] = torch.empty(t, hkv, d, dtype=dt, device="cuda")
            return st
        bs = case["block_size"]
        nb = -(-t // bs) + t // (4 * bs) + 2
        if t <= 256:
            slots = torch.randperm(nb * bs, generator=gen, device="cuda")[:t]
        else:
            perm = torch.randperm(nb, generator=gen, device="cuda")
            n = torch.arange(t, device="cuda")
            slots = perm[n // bs] * bs + n % bs
        if case["padded"]:
            slots = torch.where(torch.rand(t, generator=gen, device="cuda") < 0.1, torch.full_like(slots, -1), slots)
        st["slots"] = slots
        cdt, x = DTYPES[case["cache"]], 16 // ELEM[case["cache"]]
        fp8 = case["cache"] == "fp8"
        st["k_scale"], st["v_scale"] = (K_SCALE, V_SCALE) if fp8 else (1.0, 1.0)
        st["k_cache"] = torch.zeros(nb, hkv, d // x, bs, x, dtype=cdt, device="cuda")
        st["v_cache"] = torch.zeros(nb, hkv, d, bs, dtype=cdt, device="cuda")
        return st
    bs, lens = case["block_size"], _lens(case)
    n = [-(-total // bs) for total, _, _ in lens]
    nb = sum(n) + sum(n) // 8 + 1
    perm = torch.randperm(nb, generator=gen, device="cuda").int()
    table = torch.full((len(lens), max(n)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(n):
        table[i, :m] = perm[at:at + m]
        at += m
    _pools(gen, case, nb, st)
    st["block_tables"] = table
    st["seq_lens"] = torch.tensor([x[0] for x in lens], dtype=torch.int32, device="cuda")
    st["max_seq_len"] = max(x[0] for x in lens)
    # slots past a sequence's end hold anything, NaN among it
    last = table.gather(1, torch.tensor(n, device="cuda").unsqueeze(1) - 1).squeeze(1).long()
    past = torch.arange(bs, device="cuda") >= ((st["seq_lens"] - 1) % bs + 1).unsqueeze(1)
    seq, tok = past.nonzero(as_tuple=True)
    raw = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[st["k_cache"].element_size()]
    nan = {"fp8": 0x7F, "f16": 0x7E00, "bf16": 0x7FC0, "f32": 0x7FC00000}[case.get("cache", case["dtype"])]
    st["k_cache"].view(raw)[last[seq], :, :, tok] = nan
    st["v_cache"].view(raw)[last[seq], :, :, tok] = nan
    rows = sum(x[1] for x in lens)
    # scores of a size that the caps act on
    st["q"] = (2.5 * _randn(gen, rows, h, d)).to(dt)
    st["out"] = torch.empty_like(st["q"])
    st["softmax_scale"] = 1.0 / math.sqrt(d)
    slopes = [2.0 ** (-8.0 * (i + 1) / h) for i in range(h)]
    st["slopes"] = torch.tensor(slopes, dtype=torch.float32, device="cuda") if case["alibi"] else None
    if case["op"] == "prefill":
        ends = [0]
        for _, new, _ in lens:
            ends.append(ends[-1] + new)
        st["query_start_loc"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        prefixes = torch.tensor([x[2] for x in lens], dtype=torch.int32, device="cuda")
        st["prefix_lens"] = prefixes if case["prefix"] else None
    return st


# --- one pass -----------------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "write": _plain_write, "decode": _plain_decode, "prefill": _plain_prefill}[
        state["op"]](state)


def _run_own(st):
    import paged_kv_cache_306_gb300 as pa
    if st["op"] in ("rope", "write"):
        layout = pa.ROPE_HALVES if st["layout"] == "halves" else pa.ROPE_PAIRS
        if st["op"] == "rope":
            pa.pa_rope(st["q_out"], st["k_out"], st["q"], st["key"], st["positions"], st["inv_freq"], layout,
                       st["amplitude"])
            return st["q_out"], st["k_out"]
        pa.pa_rope_and_cache(st["q_out"], st["q"], st["key"], st["value"], st["k_cache"], st["v_cache"],
                             st["positions"], st["slots"], st["inv_freq"], layout, st["amplitude"], st["k_scale"],
                             st["v_scale"])
        return _written(st)
    if st["op"] == "decode":
        st["workspace"] = pa.pa_decode_masked(st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_tables"],
                                              st["seq_lens"], st["softmax_scale"], st["max_seq_len"], st["cap"],
                                              st["slopes"], st["window"], st["k_scale"], st["v_scale"],
                                              st.get("workspace"))
        return st["out"]
    pa.pa_prefill_masked(st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_tables"], st["seq_lens"],
                         st["query_start_loc"], st["softmax_scale"], st["max_seq_len"], st["cap"], st["slopes"],
                         st["window"], st["prefix_lens"])
    return st["out"]


def _written(st):
    """The rotated queries and the pools; what 8 bits hold comes back as the values, in the rows' type."""
    if st["cache"] != "fp8":
        return st["q_out"], st["k_cache"], st["v_cache"]
    return st["q_out"], st["k_cache"].to(st["dt"]) * st["k_scale"], st["v_cache"].to(st["dt"]) * st["v_scale"]


def _turn(x, st):
    """fp32 rows x [T, heads, D] with the rotary dims turned; the angles in 64 bits, since positions are far."""
    r = st["rotary"]
    angle = st["positions"].double().unsqueeze(1) * st["inv_freq"]
    cos = (torch.cos(angle) * st["amplitude"]).float().unsqueeze(1)
    sin = (torch.sin(angle) * st["amplitude"]).float().unsqueeze(1)
    x = x.float()
    y = x.clone()
    a, b = (x[..., :r // 2], x[..., r // 2:r]) if st["layout"] == "halves" else (x[..., 0:r:2], x[..., 1:r:2])
    if st["layout"] == "halves":
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, a * sin + b * cos
    else:
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_rope(st):
    return _turn(st["q"], st).to(st["dt"]), _turn(st["key"], st).to(st["dt"])


def _plain_write(st):
    q = _turn(st["q"], st).to(st["dt"])
    k, v = _turn(st["key"], st), st["value"].float()
    bs, cdt = st["block_size"], st["k_cache"].dtype
    if st["cache"] == "fp8":
        # the quotient in fp32, rounded once to the nearest code, at most 448 in size
        k = torch.clamp(k / torch.full_like(k, st["k_scale"]), -448.0, 448.0)
        v = torch.clamp(v / torch.full_like(v, st["v_scale"]), -448.0, 448.0)
    keep = (st["slots"] >= 0).nonzero().squeeze(1)
    at = st["slots"][keep]
    x = st["k_cache"].shape[4]
    raw = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[st["k_cache"].element_size()]
    st["k_cache"].view(raw)[at // bs, :, :, at % bs] = k[keep].to(cdt).view(raw).unflatten(-1, (-1, x))
    st["v_cache"].view(raw)[at // bs, :, :, at % bs] = v[keep].to(cdt).view(raw)
    st["q_out"] = q
    return _written(st)


def _gather(st):
    """fp32 K and V [S, Hkv, positions, D] of every block-table entry."""
    table = st["block_tables"].clamp(min=0).long()
    s, n = table.shape
    d, bs, hkv = st["head_size"], st["block_size"], st["kv_heads"]
    k = st["k_cache"][table].float().permute(0, 2, 1, 4, 3, 5).reshape(s, hkv, n * bs, d)
    v = st["v_cache"][table].float().permute(0, 2, 1, 4, 3).reshape(s, hkv, n * bs, d)
    return k * st["k_scale"], v * st["v_scale"]


def _attend(st, q, pos, prefix):
    """Attention of q [S, n, H, D] at positions pos [S, n] (those below zero have no row); fp32 [S, n, H, D]."""
    s, n, h, d = q.shape
    hkv = st["kv_heads"]
    k, v = _gather(st)
    t = torch.arange(k.shape[2], device="cuda")
    p = pos.unsqueeze(-1)
    see = t <= torch.maximum(p, prefix.view(-1, 1, 1) - 1)                                   # [S, n, L]
    if st["window"]:
        see = see & (t > p - st["window"])
    q = q.view(s, n, hkv, -1, d).permute(0, 2, 3, 1, 4).reshape(s, hkv, -1, d)               # rows: head, then token
    score = torch.matmul(q, k.transpose(2, 3)).view(s, h, n, -1) * st["softmax_scale"]
    if st["cap"]:
        score = st["cap"] * torch.tanh(score / st["cap"])
    if st["slopes"] is not None:
        score = score - st["slopes"].view(1, -1, 1, 1) * (t - p).abs().float().unsqueeze(1)
    score = score.masked_fill(~see.unsqueeze(1), -math.inf)
    w = torch.exp(score - score.amax(-1, keepdim=True))
    v = v.masked_fill((t >= st["seq_lens"].unsqueeze(1)).view(s, 1, -1, 1), 0.0)             # never 0 * NaN
    out = torch.matmul(w.view(s, hkv, -1, w.shape[-1]), v) / w.view(s, hkv, -1, w.shape[-1]).sum(-1, keepdim=True)
    return out.view(s, h, n, d).transpose(1, 2)


def _plain_decode(st):
    pos = (st["seq_lens"] - 1).unsqueeze(1)
    out = _attend(st, st["q"].float().unsqueeze(1), pos, torch.zeros_like(st["seq_lens"]))
    return out.squeeze(1).to(st["dt"])


def _plain_prefill(st):
    start, lens = st["query_start_loc"][:-1], st["seq_lens"]
    new = st["query_start_loc"][1:] - start
    i = torch.arange(st["chunk"], device="cuda")
    real = i < new.unsqueeze(1)
    row = torch.where(real, start.unsqueeze(1) + i, torch.zeros_like(i)).long()
    pos = (lens - new).unsqueeze(1) + torch.where(real, i, torch.zeros_like(i))
    prefix = st["prefix_lens"] if st["prefix_lens"] is not None else torch.zeros_like(lens)
    return _attend(st, st["q"].float()[row], pos, prefix)[real].to(st["dt"])


# --- the definition in 64 bits ------------------------------------------------------------------------

def _turned(x, st):
    """float64 rows of x turned pair by pair, each pair as a complex number."""
    r, out = st["rotary"], x.double().clone()
    a = st["positions"].double()
    for i in range(r // 2):
        at = (i, i + r // 2) if st["layout"] == "halves" else (2 * i, 2 * i + 1)
        turn = torch.polar(torch.full_like(a, st["amplitude"]), a * st["inv_freq"][i]).unsqueeze(1)
        z = torch.complex(x[..., at[0]].double(), x[..., at[1]].double()) * turn
        out[..., at[0]], out[..., at[1]] = z.real, z.imag
    return out


def _nearest_e4m3(x):
    """The nearest E4M3 value (ties to the even code) of float64 x, at most 448 in size."""
    grid = torch.tensor([m / 512.0 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127],
                        dtype=torch.float64, device=x.device)
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(grid, a).clamp(1, 126)
    lo = hi - 1
    up = (grid[hi] - a < a - grid[lo]) | ((grid[hi] - a == a - grid[lo]) & (hi % 2 == 0))
    return torch.copysign(grid[torch.where(up, hi, lo)], x)


def exact(case, seed):
    st = prepare(case, seed)
    d, hkv, h = case["head_size"], case["kv_heads"], case["heads"]
    if case["op"] == "rope":
        return _turned(st["q"], st), _turned(st["key"], st)
    if case["op"] == "write":
        q, k, v = _turned(st["q"], st), _turned(st["key"], st), st["value"].double()
        if case["cache"] == "fp8":
            ks, vs = (float(torch.tensor(x, dtype=torch.float32)) for x in (K_SCALE, V_SCALE))
            k, v = _nearest_e4m3(k / ks) * ks, _nearest_e4m3(v / vs) * vs
        nb, bs, x = st["v_cache"].shape[0], case["block_size"], st["k_cache"].shape[4]
        # a pool laid out by slot, then brought into the pools' order
        k_rows = torch.zeros(nb * bs, hkv, d, dtype=torch.float64, device="cuda")
        v_rows = torch.zeros_like(k_rows)
        keep = st["slots"] >= 0
        k_rows[st["slots"][keep]], v_rows[st["slots"][keep]] = k[keep], v[keep]
        return (q, k_rows.view(nb, bs, hkv, d // x, x).permute(0, 2, 3, 1, 4).contiguous(),
                v_rows.view(nb, bs, hkv, d).permute(0, 2, 3, 1).contiguous())
    lens, bs = _lens(case), case["block_size"]
    if sum(_seen(case, *x)[0] for x in lens) * h * d * 4 > 4e12 or sum(x[0] * x[1] for x in lens) * h * d > 2e12:
        return None
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for i, (total, new, prefix) in enumerate(lens):
        blocks = st["block_tables"][i, :-(-total // bs)].long()
        k = st["k_cache"][blocks].double().permute(1, 0, 3, 2, 4).reshape(hkv, -1, d)[:, :total] * _f32(st["k_scale"])
        v = st["v_cache"][blocks].double().permute(1, 0, 3, 2).reshape(hkv, -1, d)[:, :total] * _f32(st["v_scale"])
        for a in range(0, new, 512):
            b = min(new, a + 512)
            p = torch.arange(total - new + a, total - new + b, device="cuda")
            t = torch.arange(total, device="cuda")
            q = st["q"][row + a:row + b].double().view(b - a, hkv, -1, d)
            s = torch.einsum("nhgd,htd->hgnt", q, k) * st["softmax_scale"]
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            far = (p.unsqueeze(1) - t).double()
            if case["alibi"]:
                s -= st["slopes"].double().view(hkv, -1, 1, 1) * far.abs()
            hidden = (far < 0) & (t >= prefix)
            if case["window"]:
                hidden |= far >= case["window"]
            w = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
            out[row + a:row + b] = torch.einsum("hgnt,htd->nhgd", w, v).reshape(b - a, h, d)
        row += new
    return out


def _f32(x):
    return float(torch.tensor(x, dtype=torch.float32))
