"""Plain 64-bit forms of the serving operators (rotary positions, MXFP8 rows, causal chunk
attention) and the error bounds their tests use.  Shares no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch


# ------------------------------------------------------------------ rotary positions

def frequencies(dims, base=10000.0, scaling="none", factor=1.0, orig_ctx=4096.0, beta_fast=32.0,
                beta_slow=1.0, **_):
    i = np.arange(dims // 2, dtype=np.float64)
    f = base ** (-2.0 * i / dims)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        def pair(b):
            return dims * math.log(orig_ctx / (2 * math.pi * b)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), dims - 1)
        g = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        f = f * ((1 - g) + g / factor)
    return f


def rotate(x, positions, interleaved=True, amplitude=1.0, **rope):
    """x [T][...][d] (any float type) rotated, float64 on the CPU."""
    x = x.detach().cpu().double().numpy()
    d = x.shape[-1]
    w = np.asarray(positions.cpu(), dtype=np.float64)[:, None] * frequencies(d, **rope)
    w = w.reshape((x.shape[0],) + (1,) * (x.ndim - 2) + (d // 2,))
    c, s = np.cos(w) * amplitude, np.sin(w) * amplitude
    y = np.empty_like(x)
    ia = slice(0, d, 2) if interleaved else slice(0, d // 2)
    ib = slice(1, d, 2) if interleaved else slice(d // 2, d)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def rotate_bound(x, dtype, interleaved=True, amplitude=1.0, positions=None, **_):
    """Per element: half a step of the type of the result (added by the caller, relative to it) is the
    output rounding; this is the rest.  fp32: the angle (at most pi / 4) is rounded to 2^-24 relative and
    the 64-bit frequency itself is off by 2^-53 relative (times the angle unreduced), sincospi is within
    1 ulp, the amplitude and the two products and their sum round once each: under 6 * 2^-24 of |a| + |b|."""
    x = np.abs(x.detach().cpu().double().numpy())
    d = x.shape[-1]
    ia = slice(0, d, 2) if interleaved else slice(0, d // 2)
    ib = slice(1, d, 2) if interleaved else slice(d // 2, d)
    s = x[..., ia] + x[..., ib]
    out = np.empty_like(x)
    far = float(np.abs(np.asarray(positions.cpu(), dtype=np.float64)).max()) if positions is not None and len(positions) else 0.0
    out[..., ia] = out[..., ib] = s * abs(amplitude) * (6 * 2.0 ** -24 + far * 2.0 ** -50)
    if dtype == torch.float16:
        out += 2.0 ** -25                     # half of fp16's least step
    return out


# ------------------------------------------------------------------ MXFP8 rows

E4M3 = np.array(sorted({(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                        for e in range(16) for m in range(8) if not (e == 15 and m == 7)}))


def _code(v):
    """Nearest e4m3 code of |v| <= 448, ties to the even code (codes ascend with the value)."""
    i = np.clip(np.searchsorted(E4M3, v), 1, len(E4M3) - 1)
    lo, hi = E4M3[i - 1], E4M3[i]
    up = (v - lo > hi - v) | ((v - lo == hi - v) & (i % 2 == 0))
    return np.where(up, i, i - 1).astype(np.uint8)


def pack_rows(latent):
    """latent [N][512] -> (codes uint8 [N][512], scale bytes uint8 [N][16])."""
    x = latent.detach().cpu().double().numpy().reshape(len(latent), 16, 32)
    fin = np.where(np.isfinite(x), np.abs(x), 0.0)
    top = fin.max(-1)
    e = np.full(top.shape, -127)
    for k in range(-126, 121):                # the least e with top <= 448 * 2^e, by trying them all
        e = np.where(top > 448.0 * 2.0 ** (k - 1), k, e)
    s = 2.0 ** e[..., None].astype(np.float64)
    mag = np.where(np.isinf(x), 448.0, np.abs(np.where(np.isnan(x), 0, x)) / s)
    codes = _code(mag) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    codes = np.where(np.isnan(x), 0x7F, codes).astype(np.uint8)
    return codes.reshape(len(latent), 512), (e + 127).astype(np.uint8)


def unpack_rows(rows):
    """uint8 [...][656] -> float64 [...][576] (the rope dims as they are)."""
    r = rows.detach().cpu().contiguous()
    c = r[..., :512].numpy()
    mag = np.append(E4M3, np.nan)[c & 0x7F]
    b = r[..., 512:528].numpy().astype(np.int64)
    scale = np.where(b == 255, np.nan, 2.0 ** (b - 127.0))
    v = np.where(c >> 7, -mag, mag) * np.repeat(scale, 32, axis=-1)
    k = r[..., 528:].contiguous().view(torch.bfloat16).double().numpy()
    return np.concatenate([v, k], axis=-1)


# ------------------------------------------------------------------ ragged batches

class Batch:
    """A ragged batch of new tokens over a shuffled paged cache whose unused slots are NaN."""

    def __init__(self, q_lens, ctx_lens, heads, page, seed, device, pad_rows=0, spare=3, scale=1 / math.sqrt(192.0)):
        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.ctx, self.heads, self.page, self.scale = list(q_lens), list(ctx_lens), heads, page, scale
        B = len(q_lens)
        n_pages = [-(-c // page) for c in ctx_lens]
        total = sum(n_pages)
        ids = torch.randperm(total + spare, generator=g)[:total]
        table = torch.full((B, max(n_pages + [1])), -1, dtype=torch.int32)
        self.keys = []
        pool = torch.full((total + spare, page, 576), float("nan"), dtype=torch.bfloat16)
        o = 0
        for r in range(B):
            table[r, :n_pages[r]] = ids[o:o + n_pages[r]].to(torch.int32)
            k = torch.randn(ctx_lens[r], 576, generator=g).to(torch.bfloat16)
            self.keys.append(k)
            flat = torch.full((n_pages[r] * page, 576), float("nan"), dtype=torch.bfloat16)
            flat[:ctx_lens[r]] = k
            if n_pages[r]:
                pool[ids[o:o + n_pages[r]]] = flat.view(n_pages[r], page, 576)
            o += n_pages[r]
        cu = np.concatenate([[0], np.cumsum(q_lens)])
        self.rows = int(cu[-1]) + pad_rows
        self.q = torch.randn(self.rows, heads, 576, generator=g).to(torch.bfloat16).to(device)
        self.pool, self.table = pool.to(device), table.to(device)
        self.cu = torch.tensor(cu, dtype=torch.int32, device=device)
        self.ctx_t = torch.tensor(ctx_lens, dtype=torch.int32, device=device)
        self.device = device


def chunk_reference(b, head_lo, head_hi, tok_lo=0, tok_hi=-1, missing=None):
    """(out, lse, bound, lse_bound) float64 for the rows that requests own (NaN elsewhere).

    bound, per element: P is rounded to bf16 (half a step, 2^-8, of each weight), so the weighted sum is
    off by at most 2^-8 of A = sum p |v|.  A score is a sum of 576 exact products in fp32: 36 MMA steps, each
    off by at most 2^-22 of the sum of magnitudes (16 products and the accumulator, truncated), which moves p
    by that relative amount and the normaliser as much: 2 * delta * A.  ex2 and the sums add under 2^-12 A."""
    H, dev = b.heads, b.device
    out = torch.full((b.rows, H, 512), float("nan"), dtype=torch.float64, device=dev)
    lse = torch.full((b.rows, H), float("nan"), dtype=torch.float64, device=dev)
    bound, lb = torch.zeros_like(out), torch.zeros_like(lse)
    row = 0
    for r, (n, c) in enumerate(zip(b.q_lens, b.ctx)):
        k = b.keys[r].to(dev).double()
        for a in range(0, n, 32):
            m = min(32, n - a)
            q = b.q[row + a:row + a + m, head_lo:head_hi].double()
            s = (q.reshape(-1, 576) @ k.T * b.scale).view(m, head_hi - head_lo, c)
            mag = (q.reshape(-1, 576).abs() @ k.abs().T * abs(b.scale)).view(m, head_hi - head_lo, c)
            t = torch.arange(c, device=dev)
            end = torch.arange(a, a + m, device=dev) + (c - n) + 1
            see = (t < end[:, None]) & (t >= tok_lo)
            if tok_hi >= 0:
                see &= t < tok_hi
            if missing is not None:
                see &= ~missing[r].to(dev)[t]
            s = s.masked_fill(~see[:, None, :], -math.inf)
            l = torch.logsumexp(s, -1) if c else torch.full(s.shape[:2], -math.inf, device=dev, dtype=torch.float64)
            p = torch.exp(s - torch.where(l == -math.inf, 0.0, l)[..., None])
            delta = 36 * 2.0 ** -22 * (mag.masked_fill(~see[:, None, :], 0).amax(-1) if c else torch.zeros_like(l))
            o = p @ k[:, :512]
            A = p @ k[:, :512].abs()
            sl = slice(row + a, row + a + m)
            out[sl, head_lo:head_hi] = o
            lse[sl, head_lo:head_hi] = l
            bound[sl, head_lo:head_hi] = A * (2.0 ** -8 + 2.0 ** -12 + 2 * delta[..., None])
            lb[sl, head_lo:head_hi] = delta + 2.0 ** -20 * (1 + l.abs().nan_to_num(posinf=0))
        row += n
    return out, lse, bound, lb


def assert_chunk(b, out, lse, ref, head_lo, head_hi, what=""):
    ro, rl, bound, lb = ref
    own = int(b.cu[-1])
    o, l = out[:own, head_lo:head_hi].double(), lse[:own, head_lo:head_hi].double()
    ro, rl, bound, lb = (x[:own, head_lo:head_hi] for x in (ro, rl, bound, lb))
    assert torch.isfinite(o).all(), f"{what}: non-finite output"
    if out.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (ro.abs() + bound)
    over = (o - ro).abs() - bound
    assert (over <= 1e-30).all(), f"{what}: {int((over > 0).sum())} outputs past the bound, worst by {float(over.max()):.3e}"
    none = rl == -math.inf
    assert torch.equal(l == -math.inf, none), f"{what}: empty rows differ"
    assert (o[none] == 0).all(), f"{what}: an empty row is not zero"
    d = (l - rl).abs()[~none] - lb[~none]
    assert d.numel() == 0 or float(d.max()) <= 0, f"{what}: lse past the bound by {float(d.max()):.3e}"
