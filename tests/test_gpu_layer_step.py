"""One layer's step as the documentation gives it (marked gpu): the latent key is normed and rotated, the queries, which come out of
their up-projection, are only rotated; tables, cache, attention over a window and pages given back around them."""
import types

import numpy as np
import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S
from tests import serving_reference as R
from tests.more_reference import attention_reference
from tests.serving_reference import assert_chunk
from tests.test_gpu_norm_rope import reference as norm_reference
from tests.test_gpu_serving_loop import DEV, EPS, H, P, ROPE, ROPE_KW, SCALE, Loop

pytestmark = pytest.mark.gpu


class Layer(Loop):
    def launch(self):
        self.q.copy_(self.x[:, :H])
        self.y.copy_(self.x)
        q, k = self.q, self.y[:, H:]
        S.splash_batch_tables(self.lens, self.new, self.table, P, self.stack, self.left, self.cu, self.lens, self.pos, self.slots,
                              self.left)
        S.splash_rope(q[..., 512:], self.pos, q[..., 512:], ROPE)
        S.splash_norm_rope(k, self.kw, k, None, None, None, self.pos, ROPE, EPS, norm_dims=512, rope_lo=512)
        S.splash_kv_append(k[:, 0, :512], k[:, 0, 512:], self.cu, self.table, self.lens, self.pool)
        S.splash_chunk_attn_ex(q, self.pool, self.cu, self.table, self.lens, 0, H, 0, -1, self.out, self.lse, self.ws, SCALE,
                               window=self.window, sinks=self.sinks)
        S.splash_batch_release(self.lens, None, self.table, P, self.stack, self.left, window=self.window, sinks=self.sinks)

    def verify(self, new, what):
        N = sum(new)
        pos = torch.tensor([len(k) + i for k, n in zip(self.keys, new) for i in range(n)], dtype=torch.int32)
        q, want = self.q[:N].cpu().double().numpy(), self.x[:N, :H].cpu().double().numpy()
        part = self.x[:N, :H, 512:]
        bound = np.zeros_like(want)
        want[..., 512:] = R.rotate(part, pos, True, **ROPE_KW)
        bound[..., 512:] = R.rotate_bound(part, torch.bfloat16, True, positions=pos, **ROPE_KW)
        assert (q[..., :512] == want[..., :512]).all(), what
        assert (np.abs(q - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all(), what
        want, bound = norm_reference(self.x[:N, H:], self.kw, pos, ROPE_KW, 64, EPS, 512, 512)
        err = np.abs(self.y[:N, H:].cpu().double().numpy() - want)
        assert (err <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all(), what
        k = self.y[:N, H].cpu()
        for r, n in enumerate(new):
            self.keys[r], k = torch.cat((self.keys[r], k[:n])), k[n:]
        assert self.lens.tolist() == [len(k) for k in self.keys], what
        b = types.SimpleNamespace(q_lens=new, ctx=[len(k) for k in self.keys], heads=H, scale=SCALE, keys=self.keys, q=self.q,
                                  rows=self.rows, cu=self.cu, device=DEV)
        assert S.splash_workspace_status(self.ws) == 0, what
        assert_chunk(b, self.out, self.lse, attention_reference(b, 0, H, self.window, self.sinks), 0, H, what)


def test_a_captured_layer_is_replayed_step_by_step():
    layer = Layer(7, 60, 12, 130, seed=6, window=40, sinks=4)
    layer.step([37, 5, 0, 60, 16, 1, 9], "prompts")
    g = torch.cuda.CUDAGraph()
    layer.feed([0] * 7)
    with torch.cuda.graph(g):
        layer.launch()
    for t in range(40):
        new = [1 + (t + r) % 2 for r in range(7)]
        layer.feed(new)
        g.replay()
        layer.verify(new, f"replay {t}")
        assert layer.left[0].item() + layer.owned() == 60
