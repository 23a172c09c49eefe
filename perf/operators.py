"""Workloads of the FP4 cache operators: the quantising write and the reads back of a
paged K/V cache held in 4 bits, and decode attention over it.

A case is one pass of one operator ("op"): `run` computes it either in plain torch
operations or, with `own` set, through the framework's entry points.

The FP4 pools (uint8 [num_blocks, num_kv_heads, tile_bytes], K and V alike): a token's
row of D dims in one kv head is D/16 groups of 16 dims.  A group holds 16 E2M1 codes
and one E4M3 scale sf, and stands for code * sf * s with the tensor's fp32 scale s:
    u  = fl32(max|x| / s),  sf = E4M3(min(fl32(u / 6), 448)),  F = fl32(sf * s),
    code = E2M1(fl32(x / F)), nearest, ties to even, at most 6 (0 where F is 0);
    a group with a NaN reads back as NaN.
A (block, head) tile is the block's codes, D/2 bytes a token (low nibble first), then
one scale byte per token and group; `_places` says where each byte of them is.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
K_SCALE, V_SCALE = 0.0173, 0.0214          # not powers of two; group scales land mid-range
ELEM = {"f32": 4, "f16": 2, "bf16": 2}


# --- the cases ------------------------------------------------------------------------------------

def _decode(seqs, heads, kv_heads, head_size, block_size, shortest, longest, dtype, name=None):
    c = dict(op="decode", seqs=seqs, heads=heads, kv_heads=kv_heads, head_size=head_size, block_size=block_size,
             shortest=shortest, longest=longest, dtype=dtype)
    return dict(c, name=name) if name else c


def _rows(op, tokens, kv_heads, head_size, block_size, dtype, padded, name=None):
    c = dict(op=op, tokens=tokens, kv_heads=kv_heads, head_size=head_size, block_size=block_size, dtype=dtype,
             padded=padded)
    return dict(c, name=name) if name else c


def _blocks(blocks, kv_heads, head_size, block_size, dtype, name=None):
    c = dict(op="expand", blocks=blocks, kv_heads=kv_heads, head_size=head_size, block_size=block_size, dtype=dtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one short request, a small layer: nothing but latency
        _decode(1, 8, 2, 64, 16, 100, 100, "f16", "decode-one-short"),
        # a full batch of ragged requests, seven query heads per kv head
        _decode(64, 28, 4, 128, 16, 512, 4096, "f16", "decode-ragged-batch"),
        # one query head per kv head: the cache's bytes weigh most
        _decode(16, 32, 32, 128, 16, 2048, 2048, "f16", "decode-one-head-each"),
        # a few very long contexts
        _decode(4, 32, 8, 128, 16, 32768, 131072, "bf16", "decode-long-contexts"),
        # odd lengths from one token on, ten query heads per kv head, the other head and block size
        _decode(37, 40, 4, 64, 32, 1, 3001, "bf16", "decode-wide-groups"),
        # a generation step's new tokens, written and read back
        _rows("write", 64, 4, 128, 16, "f16", False, "write-step"),
        # the chunks of 16 prompts, 512 tokens each
        _rows("write", 8192, 4, 128, 16, "f16", False, "write-prompts"),
        # fp32 rows, an odd number of heads and tokens, padding among them
        _rows("write", 1537, 3, 64, 32, "f32", True, "write-fp32-padded"),
        # part of one sequence's rows, for inspection or another cache
        _rows("read", 513, 8, 64, 16, "bf16", True, "read-some-rows"),
        # a long context's rows
        _rows("read", 65521, 8, 128, 32, "f16", False, "read-long-context"),
        # the cached context of 16 prompts into a 16-bit pool, before their next chunk attends to it
        _blocks(1793, 4, 128, 16, "f16", "expand-prompts"),
        # a whole long context
        _blocks(8192, 8, 128, 16, "bf16", "expand-long-context"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "write", "write", "read", "expand"])
    d, bs = rng.choice([64, 128, 128]), rng.choice([16, 32])
    if op == "decode":
        hkv, group = rng.choice([1, 2, 3, 4, 8, 8, 32]), rng.choice([1, 2, 4, 5, 7, 8, 10, 16, 20])
        s = _log(rng, 1, 256)
        most = min(131072, 327680 * 8 * 128 // (s * hkv * d))   # the cost of the largest listed case
        longest = _log(rng, 1, max(1, most))
        shortest = longest if rng.random() < 0.25 else max(1, int(longest * rng.uniform(0.0, 0.9)))
        return _decode(s, hkv * group, hkv, d, bs, shortest, longest, rng.choice(["f16", "bf16"]))
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    if op == "expand":
        return _blocks(_log(rng, 1, 8192 * 16 // bs), hkv, d, bs, rng.choice(["f16", "bf16"]))
    dtype = rng.choice(["f32", "f16", "bf16"])
    most = min(65536, (600 << 20) // ((4 if op == "write" else 2) * hkv * d * ELEM[dtype]))
    tokens = _log(rng, 1, most)
    return _rows(op, tokens, hkv, d, bs, dtype, tokens >= 32 and rng.random() < 0.5)


def _lens(c):
    """The sequences' lengths, spread over [shortest, longest] by the golden ratio."""
    span = c["longest"] - c["shortest"]
    return [c["longest"] - int(round(span * ((i * 0.6180339887498949) % 1.0))) for i in range(c["seqs"])]


def work(case):
    d, hkv = case["head_size"], case["kv_heads"]
    row = 2 * hkv * (d // 2 + d // 16)                        # a token's K and V in the FP4 pools
    if case["op"] == "decode":
        lens, h = _lens(case), case["heads"]
        blocks = sum(-(-n // case["block_size"]) for n in lens)
        return {"bytes": sum(lens) * row + 4 * case["seqs"] * h * d + 4 * blocks + 4 * len(lens),
                "flops": 4 * sum(lens) * h * d}
    if case["op"] == "expand":
        n = case["blocks"] * case["block_size"]
        return {"bytes": n * (row + 4 * hkv * d) + 16 * case["blocks"], "flops": 4 * n * hkv * d}
    t, e = case["tokens"], ELEM[case["dtype"]]
    plain = 2 * t * hkv * d * e
    return {"bytes": t * row + 8 * t + (2 if case["op"] == "write" else 1) * plain, "flops": 4 * t * hkv * d}


# --- the pools' bytes ------------------------------------------------------------------------------

def _places(d, bs, of, device):
    """Byte offsets in a tile: the codes' [bs, d/2] and the scales' [bs, d/16]."""
    t = torch.arange(bs, device=device).unsqueeze(1)
    tt, sub = t % 16, t // 16
    row = 16 * sub + ((tt // 4) ^ (3 * (tt % 2))) + 4 * (tt % 4)
    j = torch.arange(d // 2, device=device).unsqueeze(0)
    codes = row * (d // 2) + ((j ^ (32 * ((row // 2) % 2))) if d == 128 else j)
    groups = d // 16
    g = torch.arange(groups, device=device).unsqueeze(0)
    if of == "k":
        lane = groups // 4                                     # groups a lane of four holds
        in_sub = (2 * (tt // 4) + tt % 2) * 2 * groups + (g // lane) * 2 * lane + ((tt // 2) % 2) * lane + g % lane
    else:
        in_sub = g * 16 + tt
    return codes, bs * (d // 2) + sub * 16 * groups + in_sub


def _quantise(x, s):
    """Codes (0..15, uint8) and E4M3 scale bytes [..., d/16] of x [..., d] with the tensor scale s."""
    x = x.float().unflatten(-1, (-1, 16))
    s = torch.full((1,), s, dtype=torch.float32, device=x.device)
    six = torch.full((1,), 6.0, dtype=torch.float32, device=x.device)
    sf = torch.clamp(x.abs().amax(-1) / s / six, max=448.0).to(torch.float8_e4m3fn)
    f = (sf.float() * s).unsqueeze(-1)
    a = torch.where(f > 0, x.abs() / f, torch.zeros_like(x))
    mag = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
           + (a >= 3.5).byte() + (a > 5.0).byte())
    return (mag + 8 * torch.signbit(x).byte()).flatten(-2), sf.view(torch.uint8)


def _values(code, sf, s):
    """fp32 values of codes [..., d] with scale bytes [..., d/16]."""
    e2m1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    v = e2m1[(code & 7).int()]
    v = torch.where(code > 7, -v, v).unflatten(-1, (-1, 16)) * sf.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return (v * torch.full((1,), s, dtype=torch.float32, device=code.device)).flatten(-2)


def _unpack(tiles, d, bs, of, s):
    """fp32 [..., bs, d] of tiles [..., tile_bytes]."""
    codes, scales = _places(d, bs, of, tiles.device)
    two = tiles[..., codes]
    return _values(torch.stack((two & 15, two >> 4), -1).flatten(-2), tiles[..., scales], s)


def _pool(gen, n, hkv, d, bs, of, s):
    """n blocks of normal rows whose channels differ in size, quantised into tiles."""
    codes, scales = _places(d, bs, of, "cuda")
    tiles = torch.empty(n, hkv, bs * (d // 2 + d // 16), dtype=torch.uint8, device="cuda")
    channel = torch.exp(0.7 * torch.randn(hkv, 1, d, generator=gen, device="cuda"))
    step = max(1, (1 << 25) // (hkv * bs * d))
    for a in range(0, n, step):
        b = min(n, a + step)
        x = torch.randn(b - a, hkv, bs, d, generator=gen, device="cuda") * channel
        code, sf = _quantise(x, s)
        tiles[a:b, :, codes] = code[..., 0::2] | (code[..., 1::2] << 4)
        tiles[a:b, :, scales] = sf
    return tiles


# --- what a program has in hand -----------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    d, bs, hkv = case["head_size"], case["block_size"], case["kv_heads"]
    st = dict(case, dtype=DTYPES[case["dtype"]], k_scale=K_SCALE, v_scale=V_SCALE)
    if case["op"] == "decode":
        lens = _lens(case)
        n = [-(-x // bs) for x in lens]
        nb = sum(n) + sum(n) // 8 + 1
        perm = torch.randperm(nb, generator=gen, device="cuda").int()
        table = torch.full((len(lens), max(n)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, m in enumerate(n):
            table[i, :m] = perm[at:at + m]
            at += m
        st["block_tables"] = table
        st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["max_seq_len"] = max(lens)
        st["k_cache"] = _pool(gen, nb, hkv, d, bs, "k", K_SCALE)
        st["v_cache"] = _pool(gen, nb, hkv, d, bs, "v", V_SCALE)
        # slots past a sequence's end hold anything: NaN scales and the largest codes here
        last = table.gather(1, torch.tensor(n, device="cuda").unsqueeze(1) - 1).squeeze(1).long()
        past = torch.arange(bs, device="cuda") >= ((st["seq_lens"] - 1) % bs + 1).unsqueeze(1)
        seq, tok = past.nonzero(as_tuple=True)
        for of in ("k", "v"):
            codes, scales = _places(d, bs, of, "cuda")
            pool = st[of + "_cache"].transpose(1, 2)                 # [blocks, bytes, heads]
            pool[last[seq].unsqueeze(1), scales[tok]] = 0x7F
            pool[last[seq].unsqueeze(1), codes[tok]] = 0x77
        st["q"] = torch.randn(len(lens), case["heads"], d, generator=gen, device="cuda").to(st["dtype"])
        st["out"] = torch.empty_like(st["q"])
        st["softmax_scale"] = 1.0 / math.sqrt(d)
        return st
    if case["op"] == "expand":
        m = case["blocks"]
        nb, out_nb = m + m // 4 + 1, m + m // 8 + 2
        st["k_cache"] = _pool(gen, nb, hkv, d, bs, "k", K_SCALE)
        st["v_cache"] = _pool(gen, nb, hkv, d, bs, "v", V_SCALE)
        st["src_dst"] = torch.stack((torch.randperm(nb, generator=gen, device="cuda")[:m],
                                     torch.randperm(out_nb, generator=gen, device="cuda")[:m]), 1).contiguous()
        st["k_out"] = torch.zeros(out_nb, hkv, d // 8, bs, 8, dtype=st["dtype"], device="cuda")
        st["v_out"] = torch.zeros(out_nb, hkv, d, bs, dtype=st["dtype"], device="cuda")
        return st
    t = case["tokens"]
    nb = -(-t // bs) + t // (4 * bs) + 2
    # tokens fill blocks in order, the blocks lie anywhere; a decode step's tokens lie anywhere
    if t <= 256:
        slots = torch.randperm(nb * bs, generator=gen, device="cuda")[:t]
    else:
        perm = torch.randperm(nb, generator=gen, device="cuda")
        i = torch.arange(t, device="cuda")
        slots = perm[i // bs] * bs + i % bs
    if case["padded"]:
        slots = torch.where(torch.rand(t, generator=gen, device="cuda") < 0.1, torch.full_like(slots, -1), slots)
    st["slots"] = slots
    st["k_rows"] = torch.zeros(t, hkv, d, dtype=st["dtype"], device="cuda")
    st["v_rows"] = torch.zeros_like(st["k_rows"])
    if case["op"] == "read":
        st["k_cache"] = _pool(gen, nb, hkv, d, bs, "k", K_SCALE)
        st["v_cache"] = _pool(gen, nb, hkv, d, bs, "v", V_SCALE)
        return st
    channel = torch.exp(0.7 * torch.randn(hkv, d, generator=gen, device="cuda"))
    st["key"] = (torch.randn(t, hkv, d, generator=gen, device="cuda") * channel).to(st["dtype"])
    st["value"] = torch.randn(t, hkv, d, generator=gen, device="cuda").to(st["dtype"])
    tile = bs * (d // 2 + d // 16)
    st["k_cache"] = torch.zeros(nb, hkv, tile, dtype=torch.uint8, device="cuda")
    st["v_cache"] = torch.zeros(nb, hkv, tile, dtype=torch.uint8, device="cuda")
    return st


# --- one pass -----------------------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else {"decode": _plain_decode, "expand": _plain_expand, "write": _plain_write,
                                        "read": _plain_read}[state["op"]](state)


def _run_own(st):
    import paged_kv_cache_306_gb300 as pa
    if st["op"] == "decode":
        st["workspace"] = pa.pa_decode_fp4(st["out"], st["q"], st["k_cache"], st["v_cache"], st["block_tables"],
                                           st["seq_lens"], st["softmax_scale"], st["max_seq_len"], st["k_scale"],
                                           st["v_scale"], st.get("workspace"))
        return st["out"]
    if st["op"] == "expand":
        pa.pa_expand_blocks_fp4(st["k_out"], st["v_out"], st["k_cache"], st["v_cache"], st["src_dst"],
                                st["k_scale"], st["v_scale"])
        return st["k_out"], st["v_out"]
    if st["op"] == "write":   # what 4 bits hold comes back as the values: the write, then the rows read back
        pa.pa_reshape_and_cache_fp4(st["key"], st["value"], st["k_cache"], st["v_cache"], st["slots"],
                                    st["k_scale"], st["v_scale"])
    pa.pa_gather_cache_fp4(st["k_rows"], st["v_rows"], st["k_cache"], st["v_cache"], st["slots"],
                           st["k_scale"], st["v_scale"])
    return st["k_rows"], st["v_rows"]


def _plain_decode(st):
    d, bs, hkv = st["head_size"], st["block_size"], st["kv_heads"]
    table, lens, q = st["block_tables"], st["seq_lens"], st["q"].float()
    s, n = table.shape
    here = (torch.arange(n * bs, device="cuda") < lens.unsqueeze(1)).unsqueeze(1)          # [S, 1, L]

    def rows(of):
        x = _unpack(st[of + "_cache"][table.clamp(min=0).long()], d, bs, of, st[of + "_scale"])
        return x.transpose(1, 2).reshape(s, hkv, n * bs, d)

    q = q.view(s, hkv, -1, d)
    score = torch.matmul(q, rows("k").transpose(2, 3)) * st["softmax_scale"]                # [S, Hkv, g, L]
    score = score.masked_fill(~here.unsqueeze(2), -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    v = rows("v").masked_fill(~here.unsqueeze(-1), 0.0)
    out = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return out.view(s, -1, d).to(st["dtype"])


def _plain_expand(st):
    d, bs = st["head_size"], st["block_size"]
    src, dst = st["src_dst"][:, 0], st["src_dst"][:, 1]
    k = _unpack(st["k_cache"][src], d, bs, "k", st["k_scale"]).to(st["dtype"])              # [n, Hkv, bs, d]
    v = _unpack(st["v_cache"][src], d, bs, "v", st["v_scale"]).to(st["dtype"])
    st["k_out"][dst] = k.unflatten(-1, (d // 8, 8)).transpose(2, 3)
    st["v_out"][dst] = v.transpose(2, 3)
    return st["k_out"], st["v_out"]


def _plain_write(st):
    keep = (st["slots"] >= 0).view(-1, 1, 1)
    out = []
    for of, x in (("k", st["key"]), ("v", st["value"])):
        x = _values(*_quantise(x, st[of + "_scale"]), st[of + "_scale"])
        out.append(torch.where(keep, x, torch.zeros_like(x)).to(st["dtype"]))
    return tuple(out)


def _plain_read(st):
    d, bs, slots = st["head_size"], st["block_size"], st["slots"]
    keep, at = (slots >= 0).view(-1, 1, 1), slots.clamp(min=0)
    out = []
    for of in ("k", "v"):
        codes, scales = _places(d, bs, of, "cuda")
        flat = st[of + "_cache"].transpose(1, 2)                                            # [blocks, bytes, heads]
        block, tok = (at // bs).unsqueeze(1), at % bs
        two = flat[block, codes[tok]].transpose(1, 2)                                       # [t, Hkv, d/2]
        sf = flat[block, scales[tok]].transpose(1, 2).contiguous()
        x = _values(torch.stack((two & 15, two >> 4), -1).flatten(-2), sf, st[of + "_scale"])
        out.append(torch.where(keep, x, torch.zeros_like(x)).to(st["dtype"]))
    return tuple(out)


# --- the definition in 64 bits ------------------------------------------------------------------------

def _exact_rows(pool, blocks, d, bs, of, s):
    """float64 [blocks, Hkv, bs, d]: every byte of the tiles taken to its value one token at a time."""
    s = float(torch.tensor(s, dtype=torch.float32))
    tiles = pool[blocks]
    out = torch.empty(len(blocks), pool.shape[1], bs, d, dtype=torch.float64, device=pool.device)
    for t in range(bs):
        sub, r = divmod(t, 16)
        row = 16 * sub + ((r >> 2) ^ (3 if r & 1 else 0)) + 4 * (r & 3)
        two = tiles[..., row * (d // 2):(row + 1) * (d // 2)].int()
        if d == 128 and (row >> 1) & 1:
            two = torch.cat((two[..., 32:], two[..., :32]), -1)      # the halves of the row change places
        for odd in (0, 1):
            nib = (two >> 4) if odd else (two & 15)
            e, m = (nib >> 1) & 3, nib & 1
            mag = torch.where(e > 0, (1 + 0.5 * m.double()) * torch.exp2(e.double() - 1), 0.5 * m.double())
            out[:, :, t, odd::2] = torch.where(nib > 7, -mag, mag)
        for g in range(d // 16):
            if of == "v":
                at = g * 16 + r
            else:
                lane = d // 64
                at = (2 * (r >> 2) + (r & 1)) * (d // 8) + (g // lane) * 2 * lane + ((r >> 1) & 1) * lane + g % lane
            byte = tiles[..., bs * (d // 2) + sub * d + at].int()
            e, m = (byte >> 3) & 15, byte & 7
            sf = torch.where(e > 0, (1 + m.double() / 8) * torch.exp2(e.double() - 7), m.double() / 512)
            sf = torch.where((byte & 127) == 127, torch.full_like(sf, math.nan), sf)
            out[:, :, t, 16 * g:16 * g + 16] *= (sf * s).unsqueeze(-1)
    return out


def _nearest(x, grid):
    """The nearest of the sorted grid's values, ties to the one with the even index."""
    hi = torch.searchsorted(grid, x).clamp(1, len(grid) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return grid[torch.where(up, hi, lo)]


def exact(case, seed):
    st = prepare(case, seed)
    d, bs, hkv = case["head_size"], case["block_size"], case["kv_heads"]
    if case["op"] == "decode":
        out = torch.empty(case["seqs"], case["heads"], d, dtype=torch.float64, device="cuda")
        for i, n in enumerate(_lens(case)):
            blocks = st["block_tables"][i, :-(-n // bs)].long()
            k, v = (_exact_rows(st[of + "_cache"], blocks, d, bs, of, st[of + "_scale"]).transpose(0, 1)
                    .reshape(hkv, -1, d)[:, :n] for of in ("k", "v"))
            q = st["q"][i].double().view(hkv, -1, d)
            w = torch.softmax(torch.einsum("hgd,hld->hgl", q, k) * st["softmax_scale"], -1)
            out[i] = torch.einsum("hgl,hld->hgd", w, v).reshape(-1, d)
        return out
    if case["op"] == "expand":
        k, v = st["k_out"].double(), st["v_out"].double()
        for a in range(0, case["blocks"], 1024):
            pair = st["src_dst"][a:a + 1024]
            x = _exact_rows(st["k_cache"], pair[:, 0], d, bs, "k", st["k_scale"])
            k[pair[:, 1]] = x.view(len(pair), hkv, bs, d // 8, 8).permute(0, 1, 3, 2, 4)
            v[pair[:, 1]] = _exact_rows(st["v_cache"], pair[:, 0], d, bs, "v", st["v_scale"]).permute(0, 1, 3, 2)
        return k, v
    out = []
    if case["op"] == "write":
        e4m3 = torch.arange(127, device="cuda")
        e4m3 = torch.where(e4m3 > 7, (1 + (e4m3 % 8) / 8.0) * torch.exp2((e4m3 // 8).double() - 7),
                           e4m3.double() / 512)
        e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        for of, x in (("k", st["key"]), ("v", st["value"])):
            s = float(torch.tensor(st[of + "_scale"], dtype=torch.float32))
            y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            for a in range(0, len(x), 8192):
                g = x[a:a + 8192].double().unflatten(-1, (-1, 16))
                sf = _nearest((((g.abs().amax(-1) / s).float().double()) / 6).float().double(), e4m3)
                f = (sf * s).float().double().unsqueeze(-1)
                mag = _nearest((g.abs() / f.clamp(min=1e-300)).float().double() * (f > 0), e2m1)
                y[a:a + 8192] = (torch.copysign(mag, g) * sf.unsqueeze(-1) * s).flatten(-2)
            y[st["slots"] < 0] = 0
            out.append(y)
        return tuple(out)
    for of in ("k", "v"):
        y = torch.zeros(case["tokens"], hkv, d, dtype=torch.float64, device="cuda")
        for a in range(0, case["tokens"], 16384):
            at = st["slots"][a:a + 16384]
            blocks, back = torch.unique(at.clamp(min=0) // bs, return_inverse=True)
            x = _exact_rows(st[of + "_cache"], blocks, d, bs, of, st[of + "_scale"])
            x = x[back, :, at.clamp(min=0) % bs]
            x[at < 0] = 0
            y[a:a + 16384] = x
        out.append(y)
    return tuple(out)
