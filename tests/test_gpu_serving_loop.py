"""Steps of a serving loop from request lengths to attention (marked gpu): tables from a free list, norm and rotation
of queries and keys, the cache, attention over a window or behind a shared prefix, and pages given back."""
import math
import os
import subprocess
import sys
import types

import numpy as np
import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S
from tests.more_reference import attention_reference
from tests.serving_reference import assert_chunk
from tests.test_gpu_norm_rope import reference as norm_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
P, H, EPS, SCALE = 16, 16, 1e-6, 1 / math.sqrt(192.0)
ROPE_KW = dict(scaling="yarn", factor=40.0)
ROPE = S.make_rope_desc(64, **ROPE_KW)


class Loop:
    """A layer's state between steps, and the host's record of every request's keys."""

    def __init__(self, B, num_pages, width, rows, seed, window=0, sinks=0, groups=0):
        self.g = torch.Generator().manual_seed(seed)
        i = lambda *n, v=-1: torch.full(n, v, dtype=torch.int32, device=DEV)
        self.B, self.rows, self.window, self.sinks = B, rows, window, sinks
        self.stack = torch.randperm(num_pages, generator=self.g).to(torch.int32).to(DEV)
        self.left = torch.tensor([num_pages, 0], dtype=torch.int32, device=DEV)
        self.table, self.lens, self.new = i(B, width), i(B, v=0), i(B, v=0)
        self.cu, self.pos, self.slots = i(B + 1, v=0), i(rows, v=0), i(rows, v=0)
        self.pool = torch.full((num_pages, P, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
        # a projection's output: the query heads, then the key
        self.x = torch.zeros(rows, H + 1, 576, dtype=torch.bfloat16, device=DEV)
        self.y = torch.zeros_like(self.x)
        self.qw, self.kw = (torch.rand(512, generator=self.g).add(0.5).to(torch.bfloat16).to(DEV) for _ in range(2))
        self.out = torch.zeros(rows, H, 512, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.zeros(rows, H, device=DEV)
        self.q = torch.zeros(rows, H, 576, dtype=torch.bfloat16, device=DEV)
        self.ws = S.chunk_workspace(self.q, self.pool, self.table, SCALE, num_groups=groups)
        self.keys = [torch.zeros(0, 576, dtype=torch.bfloat16) for _ in range(B)]
        self.groups = {}

    def feed(self, new):
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.x.copy_(torch.randn(self.x.shape, generator=self.g).to(torch.bfloat16))

    def launch(self):
        """One step, as a program enqueues it: nothing comes back to the host."""
        S.splash_batch_tables(self.lens, self.new, self.table, P, self.stack, self.left[:1], self.cu, self.lens, self.pos,
                              self.slots, self.left)
        S.splash_norm_rope(self.x[:, :H], self.qw, self.q, self.x[:, H:], self.kw, self.y[:, H:], self.pos, ROPE, EPS,
                           norm_dims=512, rope_lo=512)
        S.splash_kv_append(self.y[:, H, :512], self.y[:, H, 512:], self.cu, self.table, self.lens, self.pool)
        S.splash_chunk_attn_ex(self.q, self.pool, self.cu, self.table, self.lens, 0, H, 0, -1, self.out, self.lse, self.ws,
                               SCALE, window=self.window, sinks=self.sinks, **self.groups)
        if self.window:
            S.splash_batch_release(self.lens, None, self.table, P, self.stack, self.left, self.window, self.sinks)

    def verify(self, new, what):
        """The step's results against 64-bit forms, fed with the keys and queries as they were rounded."""
        N = sum(new)
        past = [len(k) for k in self.keys]
        assert self.left[1].item() == self.B and self.cu.tolist() == [0] + list(np.cumsum(new)), what
        assert self.lens.tolist() == [p + n for p, n in zip(past, new)], what
        pos = torch.tensor([p + i for p, n in zip(past, new) for i in range(n)], dtype=torch.int32)
        assert self.pos[:N].tolist() == pos.tolist(), what
        for x, y, w in ((self.x[:N, :H], self.q[:N], self.qw), (self.x[:N, H:], self.y[:N, H:], self.kw)):
            want, bound = norm_reference(x, w, pos, ROPE_KW, 64, EPS, 512, 512)
            err = np.abs(y.cpu().double().numpy() - want)
            assert (err <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all(), what
        assert torch.equal(self.pool.view(-1, 576)[self.slots[:N].long()], self.y[:N, H]), what
        k = self.y[:N, H].cpu()
        for r, n in enumerate(new):
            self.keys[r], k = torch.cat((self.keys[r], k[:n])), k[n:]
        b = types.SimpleNamespace(q_lens=new, ctx=[len(k) for k in self.keys], heads=H, scale=SCALE, keys=self.keys, q=self.q,
                                  rows=self.rows, cu=self.cu, device=DEV)
        assert S.splash_workspace_status(self.ws) == 0, what
        assert_chunk(b, self.out, self.lse, attention_reference(b, 0, H, self.window, self.sinks), 0, H, what)

    def step(self, new, what):
        self.feed(new)
        self.launch()
        self.verify(new, what)

    def owned(self):
        return sum((0 <= v) for v in self.table.flatten().tolist())


def test_a_window_lets_a_small_pool_serve_long_requests():
    # 5 requests of up to 150 tokens over 24 pages: what a window of 40 and 4 first tokens leaves is given back
    loop = Loop(5, 24, 12, 140, seed=1, window=40, sinks=4)
    loop.step([37, 5, 0, 70, 16], "prompts")
    for t in range(80):
        loop.step([1, t % 2, 1, int(t % 7 == 0), 3 if t < 20 else 1], f"step {t}")
        assert loop.left[0].item() + loop.owned() == 24
    free = sorted(loop.stack[:loop.left[0]].tolist() + [v for v in loop.table.flatten().tolist() if v >= 0])
    assert free == list(range(24))
    S.splash_batch_release(loop.lens, torch.zeros_like(loop.lens), loop.table, P, loop.stack, loop.left)
    assert sorted(loop.stack.tolist()) == list(range(24)) and loop.left[0].item() == 24 and (loop.table == -1).all()


def test_samples_of_one_prompt_share_its_pages():
    B, prefix = 40, 30 * P
    loop = Loop(B, 300, 40, 600, seed=2, groups=1)
    loop.step([prefix] + [0] * (B - 1), "the prompt")
    loop.table[1:, :prefix // P] = loop.table[0, :prefix // P]
    loop.lens.fill_(prefix)
    loop.keys = [loop.keys[0].clone() for _ in range(B)]
    loop.groups = dict(cu_groups=torch.tensor([0, B], dtype=torch.int32, device=DEV),
                       prefix_lens=torch.tensor([prefix], dtype=torch.int32, device=DEV))
    for t in range(6):
        loop.step([1 + (r * t) % 4 for r in range(B)], f"step {t}")
    # drafted tokens of every other request are rejected, then a step more, then the samples end but for the prompt
    keep = [len(k) - (2 if r % 2 else 0) for r, k in enumerate(loop.keys)]
    S.splash_batch_release(loop.lens, torch.tensor(keep, dtype=torch.int32, device=DEV), loop.table, P, loop.stack, loop.left)
    loop.keys = [k[:n] for k, n in zip(loop.keys, keep)]
    loop.step([2] * B, "after the rejection")
    S.splash_batch_release(loop.lens, torch.full_like(loop.lens, prefix), loop.table, P, loop.stack, loop.left)
    assert loop.left[0].item() == 300 - prefix // P
    last = torch.full_like(loop.lens, prefix)
    last[0] = 0
    S.splash_batch_release(loop.lens, last, loop.table, P, loop.stack, loop.left)
    assert sorted(loop.stack.tolist()) == list(range(300)) and loop.left[0].item() == 300


@pytest.mark.parametrize("window,sinks", [(0, 0), (33, 4)])
def test_a_captured_step_is_replayed_with_new_inputs(window, sinks):
    loop = Loop(9, 200, 12, 64, seed=3, window=window, sinks=sinks)
    loop.step([5, 17, 1, 9, 3, 2, 11, 4, 6], "prompts")
    g = torch.cuda.CUDAGraph()
    loop.feed([0] * 9)
    with torch.cuda.graph(g):                      # (an empty step's capture: capturing runs nothing)
        loop.launch()
    for t in range(25):
        new = [1 + (t + r) % 3 for r in range(9)]
        loop.feed(new)
        g.replay()
        loop.verify(new, f"replay {t}")


def test_two_layers_side_by_side():
    loops = [Loop(4, 60, 12, 60, seed=s, window=40, sinks=4) for s in (4, 5)]
    streams = [torch.cuda.Stream() for _ in loops]
    for t in range(12):
        new = [20, 3, 0, 7] if t == 0 else [1, 2, 1, 1]
        for loop in loops:
            loop.feed(new)
        torch.cuda.synchronize()
        for loop, s in zip(loops, streams):
            with torch.cuda.stream(s):
                loop.launch()
        torch.cuda.synchronize()
        for loop in loops:
            loop.verify(new, f"step {t}")


FIRST_CALLS = """
import torch
from layout_agnostic_paged_gb300 import splash as S
D = "cuda"
ints = lambda *n: torch.zeros(*n, dtype=torch.int32, device=D)
q, k = torch.randn(40, 16, 576, device=D).bfloat16(), torch.randn(40, 1, 576, device=D).bfloat16()
w, pos, rope = torch.ones(512, dtype=torch.bfloat16, device=D), ints(40), S.make_rope_desc(64)
pool, table, lens, new = torch.zeros(200, 64, 576, dtype=torch.bfloat16, device=D), ints(40, 4), ints(40), ints(40) + 1
stack, left, cu, slots = torch.arange(200, dtype=torch.int32, device=D), ints(2) + 200, ints(41), ints(40)
out, lse = torch.empty(40, 16, 512, dtype=torch.bfloat16, device=D), torch.empty(40, 16, device=D)
groups, prefix = torch.tensor([0, 40], dtype=torch.int32, device=D), ints(1)
ws, wg = S.chunk_workspace(q, pool, table, .1), S.chunk_workspace(q, pool, table, .1, num_groups=1)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    S.splash_batch_tables(lens, new, table, 64, stack, left[:1], cu, lens, pos, slots, left)
    S.splash_norm_rope(q, w, q, k, w, k, pos, rope, 1e-6, norm_dims=512, rope_lo=512)
    S.splash_kv_append(k[:, 0, :512], k[:, 0, 512:], cu, table, lens, pool)
    S.splash_chunk_attn_ex(q, pool, cu, table, lens, 0, 16, 0, -1, out, lse, ws, .1, window=100, sinks=4)
    S.splash_chunk_attn_ex(q, pool, cu, table, lens, 0, 16, 0, -1, out, lse, wg, .1, cu_groups=groups, prefix_lens=prefix)
    S.splash_batch_release(lens, None, table, 64, stack, left, window=100, sinks=4)
for _ in range(3):
    g.replay()
torch.cuda.synchronize()
assert lens.tolist() == [3] * 40 and left.tolist() == [160, 40] and torch.isfinite(out.float()).all()
assert S.splash_workspace_status(ws) == 0 and S.splash_workspace_status(wg) == 0
print("replayed")
"""


def test_a_process_may_begin_with_a_captured_step():
    # nothing has been launched before: kernels are loaded and their limits asked for during the capture
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "replayed" in r.stdout, r.stderr[-2000:]
