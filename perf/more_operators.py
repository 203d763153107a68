"""More operators of a serving step over the paged MLA cache, as they are measured.

tables  a batch's offsets, lengths, positions, slots and block table from its request lengths, with
        pages from a free list (and back to it)
norm    RMS norm of query and key heads with their rotary positions in the same pass
window  causal attention of new tokens that see a sliding window and a few first tokens
prefix  causal attention of new tokens whose requests share the pages of a long prefix

``run`` computes each in its plain form (elementary torch operations, 32 bits, angles in
64) or, where ``own`` is true, with the library's entry points.
"""
import functools
import math
import random

import torch

own = False

DEV = "cuda"
LATENT, KEY = 512, 576                      # value width and key width of the cache
SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
YARN = dict(base=10000.0, scaling="yarn", factor=40.0, orig_ctx=4096.0, amplitude=1.3688879454113936)
PLAIN = dict(base=10000.0, scaling="none", factor=1.0, orig_ctx=4096.0, amplitude=1.0)
LINEAR = dict(base=500000.0, scaling="linear", factor=8.0, orig_ctx=8192.0, amplitude=1.0)
ROPES = {"yarn": YARN, "none": PLAIN, "linear": LINEAR}


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 256 requests: a token each, a new page for one in 64
        dict(name="tables decode step", op="tables", reqs=256, q_lo=1, q_hi=1, past_lo=16, past_hi=8192, lens=11,
             page=64, short=False, back=False),
        # a mixed step that begins prompts, with some requests paused (no new token)
        dict(name="tables prompts", op="tables", reqs=61, q_lo=0, q_hi=1024, past_lo=0, past_hi=4096, lens=12,
             page=64, short=False, back=False),
        # four drafted tokens of each request, all of them rejected: pages taken and given back
        dict(name="tables drafts undone", op="tables", reqs=128, q_lo=4, q_hi=4, past_lo=64, past_hi=4096, lens=13,
             page=16, short=False, back=True),
        # prompts that are only scored: pages taken for the step and given back after it
        dict(name="tables scoring batch", op="tables", reqs=333, q_lo=16, q_hi=180, past_lo=0, past_hi=0, lens=14,
             page=16, short=False, back=True),
        # a decode step's query and key heads of one layer, 256 requests
        dict(name="norm decode batch", op="norm", tokens=256, heads=16, keys=2, width=128, norm=128, rope_lo=0,
             dims=128, interleaved=False, rope="none", dtype="bf16", max_pos=131072),
        # a prompt's query and key heads, of which half of the dims are rotated
        dict(name="norm prompt", op="norm", tokens=8191, heads=64, keys=8, width=128, norm=128, rope_lo=0,
             dims=64, interleaved=False, rope="linear", dtype="bf16", max_pos=1048576),
        # single tokens of a 16-head shard over a window with four first tokens
        dict(name="window decode shard", op="window", reqs=64, q_lo=1, q_hi=1, past_lo=512, past_hi=16384, lens=31,
             heads=128, head_lo=16, head_hi=32, page=64, window=1024, sinks=4),
        # whole prompts that are longer than the window, all heads
        dict(name="window prompts", op="window", reqs=3, q_lo=700, q_hi=2600, past_lo=0, past_hi=0, lens=32,
             heads=128, head_lo=0, head_hi=128, page=64, window=512, sinks=4),
        # a chunk of a long prompt over a wide window
        dict(name="window long chunk", op="window", reqs=1, q_lo=1024, q_hi=1024, past_lo=15360, past_hi=15360,
             lens=33, heads=128, head_lo=0, head_hi=128, page=64, window=4096, sinks=64),
        # single tokens of a 16-head shard behind one shared system prompt
        dict(name="prefix decode shard", op="prefix", groups=1, reqs_lo=64, reqs_hi=64, q_lo=1, q_hi=1,
             prefix_lo=8192, prefix_hi=8192, past_lo=16, past_hi=1024, lens=41, heads=128, head_lo=16, head_hi=32,
             page=64),
        # a few drafted tokens of many samples of three prompts
        dict(name="prefix drafted samples", op="prefix", groups=3, reqs_lo=9, reqs_hi=40, q_lo=2, q_hi=4,
             prefix_lo=1024, prefix_hi=5000, past_lo=1, past_hi=300, lens=42, heads=40, head_lo=0, head_hi=40,
             page=64),
        # a large batch behind a document of 32,768 tokens
        dict(name="prefix long document", op="prefix", groups=1, reqs_lo=256, reqs_hi=256, q_lo=1, q_hi=1,
             prefix_lo=32768, prefix_hi=32768, past_lo=1, past_hi=2048, lens=43, heads=128, head_lo=0, head_hi=16,
             page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tables", "norm", "window", "window", "prefix", "prefix"))
    if op == "tables":
        reqs = _log(rng, 1, 2048)
        q_hi = _log(rng, 1, max(2, 65536 // reqs))
        past_hi = rng.choice((0, _log(rng, 1, 16384)))
        return dict(op=op, reqs=reqs, q_lo=rng.randint(0, q_hi), q_hi=q_hi, past_lo=past_hi // 5, past_hi=past_hi,
                    lens=rng.randrange(1 << 20), page=rng.choice((16, 32, 64, 64, 128)), short=rng.random() < 0.2,
                    back=rng.random() < 0.5)
    if op == "norm":
        width = rng.choice((64, 96, 128, 128, 192, 256, 576))
        norm = 512 if width == 576 else width
        dims = 64 if width == 576 else rng.choice((32, 64, width))
        heads = 1 if width == 576 else rng.choice((1, 5, 16, 40, 64))
        keys = 0 if width == 576 else rng.choice((0, 1, 2, 8))
        most = max(2, 75_000_000 // (width * (heads + keys)))
        return dict(op=op, tokens=_log(rng, 1, min(32768, most)), heads=heads, keys=keys, width=width, norm=norm,
                    rope_lo=rng.choice((0, width - dims)) if width != 576 else 512, dims=dims,
                    interleaved=rng.random() < 0.5, rope=rng.choice(("yarn", "none", "linear")),
                    dtype=rng.choice(("bf16", "bf16", "f16", "f32")), max_pos=_log(rng, 64, 1048576))
    page = rng.choice((16, 32, 64, 64, 128))
    heads = rng.choice((8, 16, 16, 40, 64, 128, 128))
    shard = heads if heads < 64 or rng.random() < 0.5 else heads // 4
    head_lo = rng.randrange(heads // shard) * shard
    lens = rng.randrange(1 << 20)
    if op == "window":
        reqs = _log(rng, 1, 64)
        q_hi = _log(rng, 1, min(2048, max(2, 3_000_000 // (reqs * shard))))
        most = max(64, min(2_000_000 // reqs, 500_000_000 // (reqs * shard * q_hi)) - q_hi)
        past_hi = rng.choice((0, _log(rng, 1, min(32768, most))))
        return dict(op=op, reqs=reqs, q_lo=max(1, q_hi // 3), q_hi=q_hi, past_lo=past_hi // 2, past_hi=past_hi,
                    lens=lens, heads=heads, head_lo=head_lo, head_hi=head_lo + shard, page=page,
                    window=_log(rng, 1, 8192), sinks=rng.choice((0, 1, 4, 4, 64, 200)))
    groups = rng.choice((1, 1, 2, 5))
    reqs_hi = _log(rng, 1, 256 // groups)
    q_hi = rng.choice((1, 1, 4, 9))
    rows = groups * reqs_hi * q_hi * shard
    prefix_hi = _log(rng, 32, max(64, min(32768, 130_000_000 // rows)))
    return dict(op=op, groups=groups, reqs_lo=max(1, reqs_hi // 2), reqs_hi=reqs_hi, q_lo=1, q_hi=q_hi,
                prefix_lo=prefix_hi // 2, prefix_hi=prefix_hi, past_lo=0,
                past_hi=_log(rng, 1, max(2, min(2048, 60_000_000 // rows))), lens=lens, heads=heads,
                head_lo=head_lo, head_hi=head_lo + shard, page=page)


def _lengths(case):
    """(new tokens, whole context) of each request: whole numbers that the case alone fixes."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["reqs"])]
    return q, [n + r.randint(case["past_lo"], case["past_hi"]) for n in q]


def _grouped(case):
    """(requests, prefix) of each group, and (new tokens, whole context) of each request.  A prefix is a whole
    number of pages: what a cache of pages shares."""
    r, P = random.Random(case["lens"]), case["page"]
    groups, q, ctx = [], [], []
    for _ in range(case["groups"]):
        m = r.randint(case["reqs_lo"], case["reqs_hi"])
        prefix = max(1, r.randint(case["prefix_lo"], case["prefix_hi"]) // P) * P
        groups.append((m, prefix))
        for _ in range(m):
            q.append(r.randint(case["q_lo"], case["q_hi"]))
            ctx.append(prefix + r.randint(case["past_lo"], case["past_hi"]) + q[-1])
    return groups, q, ctx


def _pages(n, page):
    return -(-n // page)


def _served(case):
    """Free pages, requests served and pages taken of a tables case."""
    q, ctx = _lengths(case)
    need = [_pages(c, case["page"]) - _pages(c - n, case["page"]) for n, c in zip(q, ctx)]
    free = sum(need) * 2 // 3 if case["short"] else sum(need) + 5
    served = used = 0
    for n in need:
        if used + n > free:
            break
        used, served = used + n, served + 1
    return free, served, used


def work(case):
    if case["op"] == "tables":
        q, _ = _lengths(case)
        _, served, used = _served(case)
        n = sum(q[:served])
        back = 4 * len(q) + 12 * used if case["back"] else 0
        return {"bytes": 8 * len(q) + 8 * used + 8 * len(q) + 8 * n + back, "flops": 4 * n + 8 * len(q)}
    if case["op"] == "norm":
        size = torch.empty(0, dtype=DTYPES[case["dtype"]]).element_size()
        rows = case["tokens"] * (case["heads"] + case["keys"])
        return {"bytes": 2 * rows * case["width"] * size + 4 * case["tokens"],
                "flops": rows * (4 * case["norm"] + 3 * case["dims"])}
    hs, P = case["head_hi"] - case["head_lo"], case["page"]
    if case["op"] == "window":
        q, ctx = _lengths(case)
        w, s = case["window"], case["sinks"]
        pairs = keys = 0
        for n, c in zip(q, ctx):
            # the window of the token at position p begins at p + 1 - w; the first tokens before it are seen too
            pairs += sum(min(p + 1, w) + min(s, max(0, p + 1 - w)) for p in range(c - n, c))
            first = max(0, c - n + 1 - w) if n else c
            keys += c - first + min(s, first)
        pages = _pages(keys, P) + len(q)
    else:
        groups, q, ctx = _grouped(case)
        pairs = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(q, ctx))
        keys, r = 0, 0
        for m, prefix in groups:
            keys += prefix + sum(c - prefix for c in ctx[r:r + m])
            r += m
        pages = _pages(keys, P) + len(q)
    return {"bytes": sum(q) * hs * (2 * KEY + 2 * LATENT + 4) + keys * 2 * KEY + 4 * pages + 8 * len(q),
            "flops": 2 * (KEY + LATENT) * hs * pairs}


# ---------------------------------------------------------------------------- inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _offsets(counts):
    return _ints([0] + list(torch.tensor(counts).cumsum(0).tolist()))


def _shuffled(n, gen):
    return torch.randperm(n, generator=gen, device=DEV).to(torch.int32)


def _prepare_tables(s, gen):
    case = s["case"]
    q, ctx = _lengths(case)
    P, B = case["page"], case["reqs"]
    past = [c - n for n, c in zip(q, ctx)]
    free, _, _ = _served(case)
    have = [_pages(p, P) for p in past]
    width = max(1, max(_pages(c, P) for c in ctx))
    ids = _shuffled(sum(have) + free, gen)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(width, device=DEV)[None, :] < _ints(have)[:, None]
    table[held] = ids[:sum(have)]
    # the free list of a pool: as long as the pool has pages, its first `free` entries in use
    stack = torch.full((sum(have) + free,), -1, dtype=torch.int32, device=DEV)
    stack[:free] = ids[sum(have):]
    N = max(1, sum(q))
    s.update(past=_ints(past), new=_ints(q), table=table, stack=stack, free=_ints([free]),
             cu=torch.zeros(B + 1, dtype=torch.int32, device=DEV), ctx=torch.zeros(B, dtype=torch.int32, device=DEV),
             positions=torch.zeros(N, dtype=torch.int32, device=DEV),
             slots=torch.zeros(N, dtype=torch.int32, device=DEV), left=torch.zeros(2, dtype=torch.int32, device=DEV))


def _prepare_norm(s, gen):
    case = s["case"]
    T, D, dtype = case["tokens"], case["width"], DTYPES[case["dtype"]]
    rows = case["heads"] + case["keys"]
    # the heads of a projection's output, side by side: queries, then keys; sizes differ from dim to dim
    size = torch.exp(0.5 * torch.randn(rows, D, generator=gen, device=DEV))
    x = (torch.randn(T, rows, D, generator=gen, device=DEV) * size).to(dtype)
    s["q"], s["k"] = x[:, :case["heads"]], x[:, case["heads"]:] if case["keys"] else None
    s["q_out"] = torch.zeros(T, case["heads"], D, dtype=dtype, device=DEV)
    s["k_out"] = torch.zeros(T, case["keys"], D, dtype=dtype, device=DEV) if case["keys"] else None
    s["q_weight"] = (1 + 0.2 * torch.randn(case["norm"], generator=gen, device=DEV)).to(dtype)
    s["k_weight"] = (1 + 0.2 * torch.randn(case["norm"], generator=gen, device=DEV)).to(dtype) if case["keys"] else None
    s["positions"] = torch.randint(0, case["max_pos"], (T,), generator=gen, device=DEV, dtype=torch.int32)


def _prepare_attention(s, gen):
    case = s["case"]
    P = case["page"]
    shared = []                                             # (first request, requests, pages that they share)
    if case["op"] == "window":
        q, ctx = _lengths(case)
    else:
        groups, q, ctx = _grouped(case)
        r = 0
        for m, prefix in groups:
            shared.append((r, m, prefix // P))
            r += m
        s["cu_groups"] = _offsets([m for m, _ in groups])
        s["prefix_lens"] = _ints([p for _, p in groups])
    pages = [_pages(c, P) for c in ctx]
    total = sum(pages) - sum((m - 1) * k for _, m, k in shared)
    ids = torch.randperm(total + 1, generator=gen, device=DEV)[:total].to(torch.int32)
    table = torch.full((len(q), max(pages)), -1, dtype=torch.int32, device=DEV)
    fresh = torch.arange(max(pages), device=DEV)[None, :] < _ints(pages)[:, None]
    for first, m, k in shared:
        fresh[first + 1:first + m, :k] = False
    table[fresh] = ids
    for first, m, k in shared:
        table[first:first + m, :k] = table[first, :k].clone()
    N, H = sum(q), case["heads"]
    s.update(cu_q=_offsets(q), ctx_lens=_ints(ctx), table=table, q_max=max(q), tokens=N,
             pool=_normal((total + 1, P, KEY), gen), q=_normal((N, H, KEY), gen),
             out=torch.zeros(N, H, LATENT, dtype=torch.bfloat16, device=DEV), lse=torch.zeros(N, H, device=DEV))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": case}
    {"tables": _prepare_tables, "norm": _prepare_norm}.get(case["op"], _prepare_attention)(s, gen)
    return s


# ---------------------------------------------------------------------------- plain forms

def _plain_tables(s):
    case, P = s["case"], s["case"]["page"]
    past, new, free = s["past"].long(), s["new"].long(), s["free"].long()
    have, want = (past + P - 1) // P, (past + new + P - 1) // P
    taken = (want - have).cumsum(0)
    rows = s["positions"].numel()
    ok = (taken <= free) & (new.cumsum(0) <= rows)
    new, want = torch.where(ok, new, 0), torch.where(ok, want, have)
    need = want - have
    base = need.cumsum(0) - need
    s["cu"][1:] = new.cumsum(0)
    s["ctx"].copy_(past + new)
    s["left"].copy_(torch.cat((free - need.sum(), ok.sum()[None])))
    col = torch.arange(s["table"].shape[1], device=DEV)
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = (free - 1 - base[:, None] - (col - have[:, None])).clamp(0, max(0, s["stack"].numel() - 1))
    if s["stack"].numel():
        s["table"].copy_(torch.where(fresh, s["stack"][at], s["table"]))
    t = torch.arange(rows, device=DEV)
    cu = s["cu"].long()
    r = torch.searchsorted(cu[1:], t, right=True).clamp(max=case["reqs"] - 1)
    pos = past[r] + t - cu[r]
    live = t < cu[-1]
    pos = torch.where(live, pos, 0)
    slot = s["table"][r, pos // P].long() * P + pos % P
    s["positions"].copy_(torch.where(live, pos, s["positions"].long()))
    s["slots"].copy_(torch.where(live, slot, s["slots"].long()))
    if case["back"]:
        keep = torch.minimum(past, s["ctx"].long())
        gone = (col >= ((keep + P - 1) // P)[:, None]) & (col < ((s["ctx"].long() + P - 1) // P)[:, None])
        gone &= (s["table"] >= 0) & (s["table"] < s["stack"].numel())
        rank = gone.flatten().cumsum(0).view(gone.shape)
        n, count = rank[-1, -1], s["left"][0].long()
        to = torch.where(gone, count + n - rank, s["stack"].numel())
        stack = torch.cat((s["stack"], s["stack"].new_zeros(1)))
        stack[to.flatten()] = s["table"].flatten()
        s["stack"].copy_(stack[:-1])
        s["table"].masked_fill_(gone, -1)
        s["ctx"].copy_(keep)
        s["left"][0] += n
    return _table_outputs(s)


def _table_outputs(s):
    return [s["cu"], s["ctx"], s["positions"], s["slots"], s["table"], s["stack"], s["left"]]


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


def _plain_norm(s):
    case = s["case"]
    n, lo, d, rope = case["norm"], case["rope_lo"], case["dims"], ROPES[case["rope"]]
    angle = s["positions"].double()[:, None] * _frequencies(d, rope)
    c = (angle.cos() * rope["amplitude"]).float()[:, None]
    si = (angle.sin() * rope["amplitude"]).float()[:, None]
    for x, w, y in ((s["q"], s["q_weight"], s["q_out"]), (s["k"], s["k_weight"], s["k_out"])):
        if x is None:
            continue
        x = x.float()
        head = x[..., :n]
        x = torch.cat((head / torch.sqrt((head * head).mean(-1, keepdim=True) + EPS) * w.float(), x[..., n:]), dim=-1)
        z = x[..., lo:lo + d]
        if case["interleaved"]:
            a, b = z[..., 0::2], z[..., 1::2]
            z = torch.stack((a * c - b * si, a * si + b * c), dim=-1).flatten(-2)
        else:
            a, b = z[..., :d // 2], z[..., d // 2:]
            z = torch.cat((a * c - b * si, a * si + b * c), dim=-1)
        y.copy_(torch.cat((x[..., :lo], z, x[..., lo + d:]), dim=-1))
    return [y for y in (s["q_out"], s["k_out"]) if y is not None]


def _padded_queries(s):
    """Each request's query rows of the call's heads [B][Q][hs][576], and the rows of q that they are (a row past
    the last one for the padding)."""
    case, cu = s["case"], s["cu_q"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(s["q_max"], device=DEV)
    mine = i[None, :] < n[:, None]
    at = torch.where(mine, cu[:-1, None] + i, torch.full_like(mine, s["tokens"], dtype=torch.int64))
    return s["q"][at.clamp(max=s["tokens"] - 1), case["head_lo"]:case["head_hi"]].float(), at, n, i


def _results(s, at, o, lse):
    """o [B][Q][hs][512] and lse [B][Q][hs] to the rows of out and lse."""
    lo, hi = s["case"]["head_lo"], s["case"]["head_hi"]
    out = torch.cat((s["out"], s["out"][:1]))                                  # one row more, for the padding
    out[at.flatten(), lo:hi] = o.to(torch.bfloat16).flatten(0, 1)
    all_lse = torch.cat((s["lse"], s["lse"][:1]))
    all_lse[at.flatten(), lo:hi] = lse.flatten(0, 1)
    return [out[:-1], all_lse[:-1]]


def _plain_window(s):
    case, B = s["case"], s["case"]["reqs"]
    keys = s["pool"][s["table"].long().clamp(min=0)].float().view(B, -1, KEY)  # [B][L][576], padded
    q, at, n, i = _padded_queries(s)
    hs = q.shape[2]
    x = torch.matmul(q.view(B, -1, KEY), keys.transpose(1, 2)).view(B, s["q_max"], hs, -1)
    x *= SCALE
    t = torch.arange(x.shape[-1], device=DEV)
    p = ((s["ctx_lens"].long() - n)[:, None] + i)[:, :, None]                  # the rows' positions
    seen = (t <= p) & ((t > p - case["window"]) | (t < case["sinks"]))
    x.masked_fill_(~seen[:, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, -1, x.shape[-1]), keys[..., :LATENT]).view(B, s["q_max"], hs, LATENT) / l
    return _results(s, at, o, (m + l.log()).squeeze(-1))


def _plain_prefix(s):
    case, P = s["case"], s["case"]["page"]
    groups, new, ctx = _grouped(case)
    lo, hi = case["head_lo"], case["head_hi"]
    hs, B = hi - lo, len(new)
    # the prefix: all rows of a group over its keys
    tops, sums, accs, r, row = [], [], [], 0, 0
    for m, prefix in groups:
        rows = sum(new[r:r + m])
        keys = s["pool"][s["table"][r, :prefix // P].long()].float().view(-1, KEY)
        x = torch.matmul(s["q"][row:row + rows, lo:hi].float().reshape(-1, KEY), keys.T)
        x *= SCALE
        top = x.amax(-1, keepdim=True)
        x = x.sub_(top).exp_()
        tops.append(top)
        sums.append(x.sum(-1, keepdim=True))
        accs.append(torch.matmul(x, keys[:, :LATENT]))
        r, row = r + m, row + rows
    m1, l1, o1 = (torch.cat(v).view(s["tokens"], hs, -1) for v in (tops, sums, accs))
    # the rest of each request's keys, padded
    prefixes = [p for m, p in groups for _ in range(m)]
    rest = [c - p for c, p in zip(ctx, prefixes)]
    col = torch.arange(_pages(max(rest), P), device=DEV)
    page = (_ints(prefixes).long()[:, None] // P + col).clamp(max=s["table"].shape[1] - 1)
    keys = s["pool"][s["table"].long().gather(1, page).clamp(min=0)].float().view(B, -1, KEY)
    q, at, n, i = _padded_queries(s)
    x = torch.matmul(q.view(B, -1, KEY), keys.transpose(1, 2)).view(B, s["q_max"], hs, -1)
    x *= SCALE
    seen = torch.arange(x.shape[-1], device=DEV) <= (_ints(rest).long() - n)[:, None, None] + i[None, :, None]
    x.masked_fill_(~seen[:, :, None, :], -math.inf)
    back = at.clamp(max=s["tokens"] - 1)
    m1, l1, o1 = m1[back], l1[back], o1[back]
    m2 = torch.maximum(m1, x.amax(-1, keepdim=True))
    x = x.sub_(m2).exp_()
    old = (m1 - m2).exp()
    l = l1 * old + x.sum(-1, keepdim=True)
    o = o1 * old + torch.matmul(x.view(B, -1, x.shape[-1]), keys[..., :LATENT]).view(B, s["q_max"], hs, LATENT)
    return _results(s, at, o / l, (m2 + l.log()).squeeze(-1))


@functools.lru_cache(maxsize=None)
def _handle(dims, interleaved, rope):
    """The library's description of a model's rotary positions, which a program makes once."""
    from layout_agnostic_paged_gb300 import splash as S
    return S.make_rope_desc(dims, interleaved=interleaved, **ROPES[rope])


def _own(s):
    from layout_agnostic_paged_gb300 import splash as S
    case = s["case"]
    if case["op"] == "tables":
        S.splash_batch_tables(s["past"], s["new"], s["table"], case["page"], s["stack"], s["free"], s["cu"], s["ctx"],
                              s["positions"], s["slots"], s["left"])
        if case["back"]:
            S.splash_batch_release(s["ctx"], s["past"], s["table"], case["page"], s["stack"], s["left"])
        return _table_outputs(s)
    if case["op"] == "norm":
        S.splash_norm_rope(s["q"], s["q_weight"], s["q_out"], s["k"], s["k_weight"], s["k_out"], s["positions"],
                           _handle(case["dims"], case["interleaved"], case["rope"]), EPS, norm_dims=case["norm"],
                           rope_lo=case["rope_lo"])
        return [y for y in (s["q_out"], s["k_out"]) if y is not None]
    lo, hi = case["head_lo"], case["head_hi"]
    if "ws" not in s:                       # scratch that a program allocates once
        s["ws"] = S.chunk_workspace(s["q"], s["pool"], s["table"], SCALE, lo, hi, num_groups=case.get("groups", 0))
    if case["op"] == "window":
        S.splash_chunk_attn_ex(s["q"], s["pool"], s["cu_q"], s["table"], s["ctx_lens"], lo, hi, 0, -1, s["out"],
                               s["lse"], s["ws"], SCALE, window=case["window"], sinks=case["sinks"])
    else:
        S.splash_chunk_attn_ex(s["q"], s["pool"], s["cu_q"], s["table"], s["ctx_lens"], lo, hi, 0, -1, s["out"],
                               s["lse"], s["ws"], SCALE, cu_groups=s["cu_groups"], prefix_lens=s["prefix_lens"])
    return [s["out"], s["lse"]]


def run(state):
    if own:
        return _own(state)
    return {"tables": _plain_tables, "norm": _plain_norm, "window": _plain_window,
            "prefix": _plain_prefix}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- 64 bits

def _exact_tables(s):
    """The batch request by request, in Python's whole numbers."""
    case, P = s["case"], s["case"]["page"]
    table, stack = s["table"].tolist(), s["stack"].tolist()
    positions, slots = s["positions"].tolist(), s["slots"].tolist()
    past, new, free = s["past"].tolist(), s["new"].tolist(), s["free"].item()
    cu, ctx, served, stopped = [0], [], 0, False
    top = free
    for r, (p, n) in enumerate(zip(past, new)):
        need = _pages(p + n, P) - _pages(p, P)
        stopped = stopped or need > top or cu[-1] + n > len(positions)
        if not stopped:
            served += 1
            for k in range(need):
                table[r][_pages(p, P) + k] = stack[top - 1 - k]
            top -= need
            for i in range(n):
                positions[cu[-1] + i] = p + i
                slots[cu[-1] + i] = table[r][(p + i) // P] * P + (p + i) % P
        cu.append(cu[-1] + (0 if stopped else n))
        ctx.append(p + (0 if stopped else n))
    if case["back"]:
        for r in reversed(range(len(past))):
            for k in reversed(range(_pages(past[r], P), _pages(ctx[r], P))):
                stack[top], table[r][k] = table[r][k], -1
                top += 1
        ctx = past
    return [_ints(v) for v in (cu, ctx, positions, slots, table, stack, [top, served])]


def _exact_norm(s):
    case, rope = s["case"], ROPES[s["case"]["rope"]]
    n, lo, d = case["norm"], case["rope_lo"], case["dims"]
    f = [rope["base"] ** (-2.0 * i / d) for i in range(d // 2)]
    if rope["scaling"] == "linear":
        f = [v / rope["factor"] for v in f]
    if rope["scaling"] == "yarn":
        near = [d / 2 * math.log(rope["orig_ctx"] / (t * 2 * math.pi), rope["base"]) for t in (32, 1)]
        a, b = max(0, math.floor(near[0])), min(d - 1, math.ceil(near[1]))
        part = [min(1.0, max(0.0, (i - a) / (b - a if b > a else 0.001))) for i in range(d // 2)]
        f = [v * (p / rope["factor"] + 1.0 - p) for v, p in zip(f, part)]
    angle = torch.outer(s["positions"].double(), torch.tensor(f, dtype=torch.float64, device=DEV))
    turn = torch.polar(torch.full_like(angle, rope["amplitude"]), angle)[:, None]
    results = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        if x is None:
            continue
        y = x.double()
        power = torch.linalg.vector_norm(y[..., :n], dim=-1, keepdim=True) ** 2 / n
        y[..., :n] *= w.double() * (power + EPS) ** -0.5
        z = y[..., lo:lo + d]
        pair = z.unflatten(-1, (d // 2, 2)) if case["interleaved"] else z.unflatten(-1, (2, d // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        y[..., lo:lo + d] = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        results.append(y)
    return results


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(s)
    if case["op"] == "norm":
        return _exact_norm(s)
    P, lo, hi = case["page"], case["head_lo"], case["head_hi"]
    q, ctx = _lengths(case) if case["op"] == "window" else _grouped(case)[1:]
    window, sinks = (case["window"], case["sinks"]) if case["op"] == "window" else (max(ctx), 0)
    if 2.0 * (KEY + LATENT) * (hi - lo) * sum(n * min(c, window + sinks + 64) for n, c in zip(q, ctx)) > 6e12:
        return None
    table = s["table"].cpu()
    out, lse, first = s["out"].double(), s["lse"].double(), 0
    for r, (n, c) in enumerate(zip(q, ctx)):
        for a in range(0, n, 64):
            b = min(n, a + 64)
            # the keys that any of these rows sees, in order
            start = max(0, c - n + a + 1 - window)
            t = torch.cat((torch.arange(min(sinks, start)), torch.arange(start, c - n + b)))
            keys = s["pool"][table[r, t // P].long().to(DEV), (t % P).to(DEV)].double()
            t, p = t.to(DEV), torch.arange(c - n + a, c - n + b, device=DEV)[:, None]
            x = s["q"][first + a:first + b, lo:hi].double() @ keys.T * SCALE
            hidden = (t > p) | ((t >= sinks) & (p - t >= window))
            x.masked_fill_(hidden[:, None, :], -math.inf)
            lse[first + a:first + b, lo:hi] = torch.logsumexp(x, -1)
            out[first + a:first + b, lo:hi] = torch.softmax(x, -1) @ keys[:, :LATENT]
        first += n
    return [out, lse]
