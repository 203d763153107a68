"""The serving operators of one MLA layer over a paged cache, as they are measured.

rope    rotary positions of the 64 (or more) position dims of query heads
append  new tokens' keys rotated and written to their pages, bf16 or MXFP8
unpack  MXFP8 pages read back into bf16 pages
chunk   causal attention of a chunk of new tokens over the paged cache

``run`` computes each in its plain form (elementary torch operations, 32 bits, angles in
64) or, where ``own`` is true, with the library's entry points.
"""
import functools
import math
import random

import torch

own = False

DEV = "cuda"
LATENT, ROPE_DIMS, KEY = 512, 64, 576       # latent, position dims, key width of the cache
GROUP = 32                                  # dims that share one scale in an MXFP8 row
PACKED = LATENT + LATENT // GROUP + 2 * ROPE_DIMS   # bytes of an MXFP8 row: 656
SCALE = 1.0 / math.sqrt(192.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
YARN = dict(base=10000.0, scaling="yarn", factor=40.0, orig_ctx=4096.0, amplitude=1.3688879454113936)
PLAIN = dict(base=10000.0, scaling="none", factor=1.0, orig_ctx=4096.0, amplitude=1.0)
LINEAR = dict(base=500000.0, scaling="linear", factor=8.0, orig_ctx=8192.0, amplitude=1.0)
ROPES = {"yarn": YARN, "none": PLAIN, "linear": LINEAR}


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one token's 16 query heads of a head shard, between two projections of a decode step
        dict(name="rope one token", op="rope", tokens=1, heads=16, dims=64, width=192, out_width=576,
             interleaved=True, rope="yarn", dtype="bf16", max_pos=131072),
        # a decode batch of 256 requests, all 128 heads, contexts up to 131,072
        dict(name="rope decode batch", op="rope", tokens=256, heads=128, dims=64, width=192,
             out_width=576, interleaved=True, rope="yarn", dtype="bf16", max_pos=131072),
        # a prompt's queries whose whole 128-dim head is rotated, half layout
        dict(name="rope prompt", op="rope", tokens=8191, heads=64, dims=128, width=128, out_width=128,
             interleaved=False, rope="linear", dtype="f16", max_pos=1048576),
        # one decode step's new token of each of 256 requests, written to a bf16 cache
        dict(name="append decode step", op="append", reqs=256, q_lo=1, q_hi=1, past_lo=16,
             past_hi=2048, lens=21, page=64, fmt="bf16", interleaved=True, rope="yarn"),
        # ragged prompts written to an MXFP8 cache
        dict(name="append prompts mxfp8", op="append", reqs=16, q_lo=301, q_hi=4096, past_lo=0,
             past_hi=0, lens=22, page=64, fmt="mxfp8", interleaved=True, rope="yarn"),
        # one short request's pages brought back for a decode
        dict(name="unpack one request", op="unpack", pages=8, page=64, pool=64),
        # the pages of a batch that resumes after a handoff
        dict(name="unpack batch", op="unpack", pages=8192, page=64, pool=9011),
        # the smallest decode configuration with a few new tokens: latency
        dict(name="chunk tiny", op="chunk", reqs=2, q_lo=1, q_hi=4, past_lo=60, past_hi=97, lens=31,
             heads=8, head_lo=0, head_hi=8, page=16),
        # four drafted tokens verified per request on one shard of 16 heads
        dict(name="chunk verify shard", op="chunk", reqs=64, q_lo=4, q_hi=4, past_lo=512,
             past_hi=4096, lens=32, heads=128, head_lo=16, head_hi=32, page=64),
        # a mixed step: single tokens and prompt chunks over pasts of all lengths
        dict(name="chunk mixed batch", op="chunk", reqs=16, q_lo=1, q_hi=256, past_lo=1,
             past_hi=3840, lens=33, heads=128, head_lo=0, head_hi=128, page=64),
        # whole prompts, causal from their first token
        dict(name="chunk whole prompts", op="chunk", reqs=4, q_lo=257, q_hi=1024, past_lo=0,
             past_hi=0, lens=34, heads=128, head_lo=0, head_hi=128, page=64),
        # the last 1,024-token chunk of a long prompt
        dict(name="chunk long prompt", op="chunk", reqs=1, q_lo=1024, q_hi=1024, past_lo=15360,
             past_hi=15360, lens=35, heads=128, head_lo=0, head_hi=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append", "unpack", "chunk", "chunk", "chunk"))
    if op == "rope":
        heads = rng.choice((1, 5, 8, 16, 40, 64, 128))
        dims = rng.choice((32, 64, 64, 128))
        width = dims + rng.choice((0, 32, 128))
        most = max(2, 67_000_000 // (heads * dims))
        return dict(op=op, tokens=_log(rng, 1, min(8192, most)), heads=heads, dims=dims, width=width,
                    out_width=rng.choice((dims, dims + 64, 512 + dims)), interleaved=rng.random() < 0.5,
                    rope=rng.choice(("yarn", "none", "linear")), dtype=rng.choice(("bf16", "bf16", "f16", "f32")),
                    max_pos=_log(rng, 64, 1048576))
    page = rng.choice((16, 32, 64, 64, 128))
    if op == "append":
        reqs = _log(rng, 1, 256)
        q_hi = _log(rng, 1, max(2, min(4096, 32768 // reqs)))
        past_hi = rng.choice((0, _log(rng, 1, 2048)))
        return dict(op=op, reqs=reqs, q_lo=rng.randint(1, q_hi), q_hi=q_hi, past_lo=past_hi // 3,
                    past_hi=past_hi, lens=rng.randrange(1 << 20), page=page,
                    fmt=rng.choice(("bf16", "mxfp8", "mxfp8")), interleaved=rng.random() < 0.5,
                    rope=rng.choice(("yarn", "none", "linear")))
    if op == "unpack":
        pages = _log(rng, 1, 524288 // page)
        return dict(op=op, pages=pages, page=page, pool=pages + _log(rng, 1, pages + 8))
    heads = rng.choice((8, 16, 16, 40, 64, 128, 128, 128))
    shard = heads if heads < 64 or rng.random() < 0.6 else heads // 4
    head_lo = rng.randrange(heads // shard) * shard
    reqs = _log(rng, 1, 64)
    most = 2_000_000_000 // (reqs * shard)                  # query tokens x keys of a request
    q_hi = _log(rng, 1, min(1024, max(2, most // 512)))
    past_hi = _log(rng, 1, max(2, min(32768, most // q_hi - q_hi)))
    past_lo = past_hi // 2
    if rng.random() < 0.25:
        past_lo = past_hi = 0
    return dict(op=op, reqs=reqs, q_lo=max(1, q_hi // 3), q_hi=q_hi, past_lo=past_lo, past_hi=past_hi,
                lens=rng.randrange(1 << 20), heads=heads, head_lo=head_lo, head_hi=head_lo + shard,
                page=page)


def _lengths(case):
    """(new tokens, whole context) of each request: whole numbers that the case alone fixes."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["reqs"])]
    return q, [n + r.randint(case["past_lo"], case["past_hi"]) for n in q]


def _visible(case):
    """Pairs of a new token and a token that it sees, over all requests."""
    return sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(*_lengths(case)))


def work(case):
    if case["op"] == "rope":
        size = torch.empty(0, dtype=DTYPES[case["dtype"]]).element_size()
        n = case["tokens"] * case["heads"] * case["dims"]
        return {"bytes": 2 * n * size + 4 * case["tokens"], "flops": 3 * n}
    if case["op"] == "append":
        q, _ = _lengths(case)
        n, row = sum(q), 2 * KEY if case["fmt"] == "bf16" else PACKED
        pages = sum(-(-x // case["page"]) for x in q)
        return {"bytes": n * (2 * KEY + row) + 8 * len(q) + 4 * pages, "flops": n * (3 * ROPE_DIMS + 3 * LATENT)}
    if case["op"] == "unpack":
        n = case["pages"] * case["page"]
        return {"bytes": n * (PACKED + 2 * KEY) + 8 * case["pages"], "flops": n * LATENT}
    q, ctx = _lengths(case)
    hs = case["head_hi"] - case["head_lo"]
    return {"bytes": sum(q) * hs * (2 * KEY + 2 * LATENT + 4) + sum(ctx) * 2 * KEY
            + 4 * sum(-(-c // case["page"]) for c in ctx) + 8 * len(q),
            "flops": 2 * (KEY + LATENT) * hs * _visible(case)}


# ---------------------------------------------------------------------------- inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _tables(case, gen):
    """Lengths, offsets and a shuffled block table over just the pages that the batch needs."""
    q, ctx = _lengths(case)
    pages = [-(-c // case["page"]) for c in ctx]
    total = sum(pages)
    ids = torch.randperm(total + 1, generator=gen, device=DEV)[:total].to(torch.int32)
    width = max(pages)
    table = torch.full((len(q), width), -1, dtype=torch.int32, device=DEV)
    col = torch.arange(width, device=DEV)
    table[col[None, :] < _ints(pages)[:, None]] = ids
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.tensor(q).cumsum(0)]).to(torch.int32).to(DEV)
    return dict(cu_q=cu, ctx_lens=_ints(ctx), table=table, q_max=max(q), tokens=sum(q), num_pages=total + 1)


def _latents(shape, gen):
    """Latents as a normalised projection leaves them: groups of dims of unlike size, a few far out."""
    x = torch.randn(shape, generator=gen, device=DEV)
    size = torch.exp(0.7 * torch.randn(shape[-1], generator=gen, device=DEV))
    far = 1.0 + 20.0 * (torch.rand(shape, generator=gen, device=DEV) < 0.001)
    return (x * size * far).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "rope":
        T, H, d = case["tokens"], case["heads"], case["dims"]
        dtype = DTYPES[case["dtype"]]
        s["x"] = _normal((T, H, case["width"]), gen, dtype)[..., case["width"] - d:]
        s["out"] = torch.zeros(T, H, case["out_width"], dtype=dtype, device=DEV)[..., case["out_width"] - d:]
        s["positions"] = torch.randint(0, case["max_pos"], (T,), generator=gen, device=DEV, dtype=torch.int32)
    elif case["op"] == "append":
        s.update(_tables(case, gen))
        s["latent"] = _latents((s["tokens"], LATENT), gen)
        s["k_rope"] = _normal((s["tokens"], ROPE_DIMS), gen)
        if case["fmt"] == "bf16":
            s["pool"] = _normal((s["num_pages"], case["page"], KEY), gen)
        else:
            s["pool"] = torch.zeros(s["num_pages"], case["page"], PACKED, dtype=torch.uint8, device=DEV)
    elif case["op"] == "unpack":
        n, P = case["pages"], case["page"]
        rows = case["pool"] * P
        src = torch.empty(rows, PACKED, dtype=torch.uint8, device=DEV)
        codes = (torch.randn(rows, LATENT, generator=gen, device=DEV) * 100.0).clamp_(-448, 448)
        src[:, :LATENT] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
        del codes
        src[:, LATENT:LATENT + LATENT // GROUP] = torch.randint(
            115, 125, (rows, LATENT // GROUP), generator=gen, device=DEV, dtype=torch.uint8)
        src[:, PACKED - 2 * ROPE_DIMS:] = _normal((rows, ROPE_DIMS), gen).view(torch.uint8)
        s["src"] = src.view(case["pool"], P, PACKED)
        s["dst"] = torch.zeros(n + 1, P, KEY, dtype=torch.bfloat16, device=DEV)
        s["src_ids"] = torch.randperm(case["pool"], generator=gen, device=DEV)[:n].to(torch.int32)
        s["dst_ids"] = torch.randperm(n + 1, generator=gen, device=DEV)[:n].to(torch.int32)
    else:
        s.update(_tables(case, gen))
        H, lo, hi = case["heads"], case["head_lo"], case["head_hi"]
        s["pool"] = _normal((s["num_pages"], case["page"], KEY), gen)
        s["q"] = _normal((s["tokens"], H, KEY), gen)
        s["out"] = torch.zeros(s["tokens"], H, LATENT, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros(s["tokens"], H, device=DEV)
    return s


# ---------------------------------------------------------------------------- plain forms

def _frequencies(dims, rope):
    """Radians per position of each pair, in 64 bits."""
    i = torch.arange(dims // 2, dtype=torch.float64, device=DEV)
    f = rope["base"] ** (-2.0 * i / dims)
    if rope["scaling"] == "linear":
        return f / rope["factor"]
    if rope["scaling"] == "yarn":
        def pair_of(turns):     # the pair that makes so many turns over the trained length
            return dims * math.log(rope["orig_ctx"] / (2 * math.pi * turns)) / (2 * math.log(rope["base"]))
        lo = max(math.floor(pair_of(32.0)), 0)
        hi = min(math.ceil(pair_of(1.0)), dims - 1)
        slow = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * ((1 - slow) + slow / rope["factor"])
    return f


def _rotated(x, positions, rope, interleaved):
    """x [T][...][d] rotated, in 32 bits (the angles in 64)."""
    d = x.shape[-1]
    angle = positions.double()[:, None] * _frequencies(d, rope)
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (d // 2,)
    c = (angle.cos() * rope["amplitude"]).float().view(shape)
    s = (angle.sin() * rope["amplitude"]).float().view(shape)
    x = x.float()
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * s, a * s + b * c), dim=-1).flatten(-2)
    a, b = x[..., :d // 2], x[..., d // 2:]
    return torch.cat((a * c - b * s, a * s + b * c), dim=-1)


def _where_new(s, page):
    """(position, row of the pool) of every new token."""
    t = torch.arange(s["tokens"], device=DEV)
    r = torch.searchsorted(s["cu_q"][1:], t, right=True)
    pos = s["ctx_lens"][r].long() - s["cu_q"][r + 1].long() + t
    return pos, s["table"][r, pos // page].long() * page + pos % page


def _scale_exponents(latent):
    """Exponent e of each group of 32 dims: the least with max |x| <= 448 * 2^e."""
    top = latent.float().view(latent.shape[0], -1, GROUP).abs().amax(-1)
    m, e = torch.frexp(top)                                 # top = m * 2^e, 1/2 <= m < 1
    e = e - 9 + (m > 448.0 / 512.0).to(e.dtype)
    return torch.where(top > 0, e, torch.full_like(e, -127)).clamp(-127, 127)


def _power_of_two(byte):
    """2^(byte - 127), exact: the byte is a float's exponent field (0 stands for 2^-127)."""
    return ((byte << 23) | ((byte == 0).to(byte.dtype) << 22)).to(torch.int32).view(torch.float32)


def _plain_append(s):
    case = s["case"]
    pos, row = _where_new(s, case["page"])
    k = _rotated(s["k_rope"], pos, ROPES[case["rope"]], case["interleaved"]).to(torch.bfloat16)
    flat = s["pool"].view(-1, s["pool"].shape[-1])
    if case["fmt"] == "bf16":
        flat[row] = torch.cat((s["latent"], k), dim=1)
        return s["pool"]
    e = _scale_exponents(s["latent"])
    x = s["latent"].float().view(-1, LATENT // GROUP, GROUP) * _power_of_two(127 - e)[..., None]
    x = x.view(-1, LATENT)
    codes = x.to(torch.float8_e4m3fn).view(torch.uint8)
    flat[row] = torch.cat((codes, (e + 127).to(torch.uint8), k.view(torch.uint8)), dim=1)
    return _values(s["pool"])


def _values(pool):
    """An MXFP8 pool as the values that it holds: codes, scale bytes, position dims."""
    g = LATENT + LATENT // GROUP
    return [pool[..., :LATENT].view(torch.float8_e4m3fn), pool[..., LATENT:g], pool[..., g:].view(torch.bfloat16)]


def _plain_unpack(s):
    rows = s["src"][s["src_ids"].long()]
    codes, scales, k = _values(rows)
    x = codes.float().view(*rows.shape[:2], LATENT // GROUP, GROUP)
    x = (x * _power_of_two(scales.to(torch.int32))[..., None]).flatten(-2)
    s["dst"][s["dst_ids"].long()] = torch.cat((x.to(torch.bfloat16), k), dim=-1)
    return s["dst"]


def _plain_chunk(s):
    case, table, cu, ctx = s["case"], s["table"].long().clamp(min=0), s["cu_q"].long(), s["ctx_lens"].long()
    lo, hi = case["head_lo"], case["head_hi"]
    B, hs, n = case["reqs"], hi - lo, cu[1:] - cu[:-1]
    keys = s["pool"][table].float().view(B, -1, KEY)                           # [B][L][576], padded
    i = torch.arange(s["q_max"], device=DEV)
    mine = i[None, :] < n[:, None]
    at = torch.where(mine, cu[:-1, None] + i, torch.full_like(mine, s["tokens"], dtype=torch.int64))
    q = s["q"][at.clamp(max=s["tokens"] - 1), lo:hi].float()                   # [B][Q][hs][576], padded
    x = torch.matmul(q.view(B, -1, KEY), keys.transpose(1, 2)).view(B, s["q_max"], hs, -1)
    x *= SCALE
    seen = torch.arange(x.shape[-1], device=DEV) <= (ctx - n)[:, None, None] + i[None, :, None]
    x.masked_fill_(~seen[:, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, -1, x.shape[-1]), keys[..., :LATENT]).view(B, s["q_max"], hs, LATENT)
    o = torch.where(l > 0, o / l, torch.zeros_like(o)).to(torch.bfloat16)
    out = torch.cat((s["out"], s["out"][:1]))                                  # one row more, for the padding
    out[at.flatten(), lo:hi] = o.flatten(0, 1)
    lse = torch.cat((s["lse"], s["lse"][:1]))
    lse[at.flatten(), lo:hi] = (m + l.log()).squeeze(-1).flatten(0, 1)
    return [out[:-1], lse[:-1]]


@functools.lru_cache(maxsize=None)
def _handle(dims, interleaved, rope):
    """The library's description of a model's rotary positions, which a program makes once."""
    from layout_agnostic_paged_gb300 import splash as S
    return S.make_rope_desc(dims, interleaved=interleaved, **ROPES[rope])


def _own(s):
    from layout_agnostic_paged_gb300 import splash as S
    case = s["case"]
    if case["op"] == "rope":
        S.splash_rope(s["x"], s["positions"], s["out"], _handle(case["dims"], case["interleaved"], case["rope"]))
        return s["out"]
    if case["op"] == "append":
        S.splash_kv_append(s["latent"], s["k_rope"], s["cu_q"], s["table"], s["ctx_lens"], s["pool"],
                           _handle(ROPE_DIMS, case["interleaved"], case["rope"]))
        return s["pool"] if case["fmt"] == "bf16" else _values(s["pool"])
    if case["op"] == "unpack":
        S.splash_kv_unpack(s["src"], s["dst"], s["src_ids"], s["dst_ids"])
        return s["dst"]
    lo, hi = case["head_lo"], case["head_hi"]
    if "ws" not in s:                       # scratch that a program allocates once
        s["ws"] = S.chunk_workspace(s["q"], s["pool"], s["table"], SCALE, lo, hi)
    S.splash_chunk_attn(s["q"], s["pool"], s["cu_q"], s["table"], s["ctx_lens"], lo, hi, 0, -1,
                        s["out"], s["lse"], s["ws"], SCALE)
    return [s["out"], s["lse"]]


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "rope":
        state["out"].copy_(_rotated(state["x"], state["positions"], ROPES[case["rope"]], case["interleaved"]))
        return state["out"]
    return {"append": _plain_append, "unpack": _plain_unpack, "chunk": _plain_chunk}[case["op"]](state)


# ---------------------------------------------------------------------------- 64 bits

def _turned(x, positions, rope, interleaved):
    """The rotation as a product of complex numbers."""
    d = x.shape[-1]
    pair = x.double().unflatten(-1, (d // 2, 2)) if interleaved else x.double().unflatten(-1, (2, d // 2)).transpose(-1, -2)
    f = [rope["base"] ** (-2.0 * i / d) for i in range(d // 2)]
    if rope["scaling"] == "linear":
        f = [v / rope["factor"] for v in f]
    if rope["scaling"] == "yarn":
        near = [d / 2 * math.log(rope["orig_ctx"] / (t * 2 * math.pi), rope["base"]) for t in (32, 1)]
        lo, hi = max(0, math.floor(near[0])), min(d - 1, math.ceil(near[1]))
        part = [min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001))) for i in range(d // 2)]
        f = [v * (p / rope["factor"] + 1.0 - p) for v, p in zip(f, part)]
    angle = torch.outer(positions.double(), torch.tensor(f, dtype=torch.float64, device=DEV))
    turn = torch.polar(torch.full_like(angle, rope["amplitude"]), angle)
    z = torch.view_as_complex(pair.contiguous()) * turn.view(turn.shape[0], *(1,) * (x.dim() - 2), d // 2)
    z = torch.view_as_real(z)
    return z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)


def _exp2(k):
    """2^k in 64 bits for whole numbers k, exact."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _nearest_e4m3(x):
    """x rounded to the nearest e4m3 value, ties to even: 4 significant bits, steps of 2^-9 at least."""
    step = _exp2((torch.frexp(x)[1] - 4).clamp(min=-9))
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned(s["x"], s["positions"], ROPES[case["rope"]], case["interleaved"])
    if case["op"] == "unpack":
        codes, scales, k = _values(s["src"][s["src_ids"].long()])
        x = codes.double() * _exp2(scales.long() - 127).repeat_interleave(GROUP, dim=-1)
        dst = s["dst"].double()
        dst[s["dst_ids"].long()] = torch.cat((x, k.double()), dim=-1)
        return dst
    q, ctx = _lengths(case)
    P = case["page"]
    table = s["table"].cpu()
    if case["op"] == "append":
        pos = torch.cat([torch.arange(c - n, c) for n, c in zip(q, ctx)])
        page = torch.cat([table[r, torch.arange(c - n, c) // P] for r, (n, c) in enumerate(zip(q, ctx))])
        pos, page = pos.to(DEV), page.long().to(DEV)
        k = _turned(s["k_rope"], pos, ROPES[case["rope"]], case["interleaved"])
        if case["fmt"] == "bf16":
            pool = s["pool"].double()
            pool[page, pos % P] = torch.cat((s["latent"].double(), k), dim=1)
            return pool
        codes, scales, rope = [v.double() for v in _values(s["pool"])]
        x = s["latent"].double().unflatten(-1, (-1, GROUP))
        top = x.abs().amax(-1, keepdim=True)
        e = torch.frexp(top / 448.0)[1]
        e = torch.where(top <= 448.0 * _exp2(e - 1), e - 1, e).clamp(-127, 127)
        codes[page, pos % P] = _nearest_e4m3(x / _exp2(e)).flatten(-2)
        scales[page, pos % P] = (e.squeeze(-1) + 127).double()
        rope[page, pos % P] = k
        return [codes, scales.to(torch.uint8), rope]
    lo, hi = case["head_lo"], case["head_hi"]
    if 2.0 * (KEY + LATENT) * (hi - lo) * sum(n * c for n, c in zip(q, ctx)) > 6e12:
        return None
    out, lse, first = s["out"].double(), s["lse"].double(), 0
    for r, (n, c) in enumerate(zip(q, ctx)):
        keys = s["pool"][table[r, :-(-c // P)].long().to(DEV)].flatten(0, 1)[:c].double()
        for a in range(0, n, 64):
            b = min(n, a + 64)
            x = s["q"][first + a:first + b, lo:hi].double() @ keys.T * SCALE
            hidden = torch.arange(c, device=DEV) > torch.arange(c - n + a, c - n + b, device=DEV)[:, None]
            x.masked_fill_(hidden[:, None, :], -math.inf)
            lse[first + a:first + b, lo:hi] = torch.logsumexp(x, -1)
            out[first + a:first + b, lo:hi] = torch.softmax(x, -1) @ keys[:, :LATENT]
        first += n
    return [out, lse]
