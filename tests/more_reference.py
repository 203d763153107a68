"""The 64-bit form of causal attention over chosen keys, for windows, first tokens and shared prefixes."""
from __future__ import annotations

import math

import torch


def attention_reference(b, head_lo, head_hi, window=0, sinks=0, tok_lo=0, tok_hi=-1, missing=None):
    """(out, lse, bound, lse_bound) like serving_reference.chunk_reference, whose bounds hold as they are: they count
    one product's and one exponential's errors per visible key.  window 0: every key up to a token's own."""
    H, dev = b.heads, b.device
    out = torch.full((b.rows, H, 512), float("nan"), dtype=torch.float64, device=dev)
    lse = torch.full((b.rows, H), float("nan"), dtype=torch.float64, device=dev)
    bound, lb = torch.zeros_like(out), torch.zeros_like(lse)
    row = 0
    for r, (n, c) in enumerate(zip(b.q_lens, b.ctx)):
        k = b.keys[r].to(dev).double()
        t = torch.arange(c, device=dev)
        for a in range(0, n, 32):
            m = min(32, n - a)
            p = torch.arange(a, a + m, device=dev)[:, None] + (c - n)      # positions
            see = (t <= p) & (t >= tok_lo)
            if window > 0:
                see &= (p - t < window) | (t < sinks)
            if tok_hi >= 0:
                see &= t < tok_hi
            if missing is not None:
                see &= ~missing[r].to(dev)[t]
            q = b.q[row + a:row + a + m, head_lo:head_hi].double()
            s = (q.reshape(-1, 576) @ k.T * b.scale).view(m, head_hi - head_lo, c)
            mag = (q.reshape(-1, 576).abs() @ k.abs().T * abs(b.scale)).view(m, head_hi - head_lo, c)
            s = s.masked_fill(~see[:, None, :], -math.inf)
            l = torch.logsumexp(s, -1) if c else torch.full(s.shape[:2], -math.inf, device=dev, dtype=torch.float64)
            pr = torch.exp(s - torch.where(l == -math.inf, 0.0, l)[..., None])
            delta = 36 * 2.0 ** -22 * (mag.masked_fill(~see[:, None, :], 0).amax(-1) if c else torch.zeros_like(l))
            A = pr @ k[:, :512].abs()
            sl = slice(row + a, row + a + m)
            out[sl, head_lo:head_hi] = pr @ k[:, :512]
            lse[sl, head_lo:head_hi] = l
            bound[sl, head_lo:head_hi] = A * (2.0 ** -8 + 2.0 ** -12 + 2 * delta[..., None])
            lb[sl, head_lo:head_hi] = delta + 2.0 ** -20 * (1 + l.abs().nan_to_num(posinf=0))
        row += n
    return out, lse, bound, lb
