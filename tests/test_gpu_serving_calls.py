"""Calls of the serving operators that their documentation allows and that have no place in the tests of
each operator's values: padding before the first request, offsets that change between replays, ranges past
32 bits, broadcast inputs, graphs replayed at once, captured calls without work (marked gpu)."""
import numpy as np
import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S
from tests import serving_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = dict(dtype=torch.int32, device=DEV)


def led(b, lead):
    """Batch b with `lead` rows of padding in front."""
    g = torch.Generator().manual_seed(7)
    b.q = torch.cat((torch.randn(lead, b.heads, 576, generator=g).to(torch.bfloat16).to(DEV), b.q))
    b.cu = b.cu + lead
    b.rows += lead
    return b


def chunk(b, lo, hi, out, lse, ws=None, tok_lo=0, tok_hi=-1, stream=None):
    ws = S.chunk_workspace(b.q, b.pool, b.table, b.scale, lo, hi) if ws is None else ws
    S.splash_chunk_attn(b.q, b.pool, b.cu, b.table, b.ctx_t, lo, hi, tok_lo, tok_hi, out, lse, ws, b.scale, stream=stream)
    return ws


def buffers(b, dtype=torch.float32):
    return torch.full((b.rows, b.heads, 512), 7.0, dtype=dtype, device=DEV), torch.full((b.rows, b.heads), 7.0, device=DEV)


def assert_rows(b, out, lse, ref, lo, hi, first, what):
    """assert_chunk on the rows from `first` on, `ref` being that of the batch without padding in front."""
    inner = R.Batch.__new__(R.Batch)
    inner.cu = b.cu - first
    R.assert_chunk(inner, out[first:], lse[first:], ref, lo, hi, what)


@pytest.mark.parametrize("lo,hi", [(0, 24), (5, 12), (0, 1)])
@pytest.mark.parametrize("lead", [1, 5, 130])
def test_padding_before_the_first_request(lead, lo, hi):
    b = R.Batch([3, 0, 40, 1], [200, 10, 300, 77], 24, 32, 90, DEV, pad_rows=2)
    ref = R.chunk_reference(b, lo, hi)
    b = led(b, lead)
    out, lse = buffers(b)
    ws = chunk(b, lo, hi, out, lse)
    assert S.splash_workspace_status(ws) == 0
    assert (out[:lead] == 7).all() and (lse[:lead] == 7).all() and (out[-2:] == 7).all()
    assert_rows(b, out, lse, ref, lo, hi, lead, "led")


def test_append_skips_padding_before_the_first_request():
    b = R.Batch([3, 0, 40, 1], [200, 10, 300, 77], 1, 32, 91, DEV, pad_rows=2)
    lead, g = 9, torch.Generator().manual_seed(1)
    lat = torch.randn(b.rows + lead, 512, generator=g).to(torch.bfloat16).to(DEV)
    kr = torch.randn(b.rows + lead, 64, generator=g).to(torch.bfloat16).to(DEV)
    with_lead, without = b.pool.clone(), b.pool.clone()
    S.splash_kv_append(lat, kr, b.cu + lead, b.table, b.ctx_t, with_lead)
    S.splash_kv_append(lat[lead:], kr[lead:], b.cu, b.table, b.ctx_t, without)
    assert torch.equal(with_lead.view(torch.int16), without.view(torch.int16))
    assert not torch.equal(without.view(torch.int16), b.pool.view(torch.int16))


def test_append_of_one_broadcast_row():
    b = R.Batch([4, 2], [4, 30], 1, 16, 92, DEV)
    g = torch.Generator().manual_seed(2)
    lat, kr = (torch.randn(1, d, generator=g).to(torch.bfloat16).to(DEV) for d in (512, 64))
    one, many = b.pool.clone(), b.pool.clone()
    S.splash_kv_append(lat.expand(b.rows, 512), kr.expand(b.rows, 64), b.cu, b.table, b.ctx_t, one)
    S.splash_kv_append(lat.repeat(b.rows, 1), kr.repeat(b.rows, 1), b.cu, b.table, b.ctx_t, many)
    assert torch.equal(one.view(torch.int16), many.view(torch.int16))


def test_rope_of_a_broadcast_head_into_many():
    x = torch.randn(50, 1, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    pos = torch.arange(50, **I32) * 997
    desc = S.make_rope_desc(64)
    a, c = torch.empty(50, 8, 64, dtype=torch.bfloat16, device=DEV), torch.empty(50, 8, 64, dtype=torch.bfloat16, device=DEV)
    S.splash_rope(x.expand(50, 8, 64), pos, a, desc)
    S.splash_rope(x.repeat(1, 8, 1), pos, c, desc)
    assert torch.equal(a.view(torch.int16), c.view(torch.int16))


def test_token_ranges_past_32_bits():
    b = R.Batch([2, 9], [150, 300], 16, 64, 93, DEV)
    for lo, hi, ref in ((0, 1 << 40, R.chunk_reference(b, 0, 16)), (1 << 40, -1, R.chunk_reference(b, 0, 16, 1 << 31)),
                        (100, (1 << 31) - 1, R.chunk_reference(b, 0, 16, 100))):
        out, lse = buffers(b)
        ws = chunk(b, 0, 16, out, lse, None, lo, hi)
        assert S.splash_workspace_status(ws) == 0
        R.assert_chunk(b, out, lse, ref, 0, 16, f"[{lo}, {hi})")


def test_replayed_on_other_offsets():
    # one graph for every mix of up to 64 rows over three requests, as a serving program keeps it
    b = R.Batch([30, 4, 30], [500, 444, 70], 32, 64, 94, DEV)
    out, lse = buffers(b)
    ws = chunk(b, 0, 32, out, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chunk(b, 0, 32, out, lse, ws)
    for q in ([30, 4, 30], [1, 0, 1], [0, 0, 0], [0, 63, 1], [64, 0, 0]):
        b.q_lens = q
        b.cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(q)]), dtype=torch.int32))
        out.fill_(7)
        lse.fill_(7)
        graph.replay()
        assert S.splash_workspace_status(ws) == 0
        R.assert_chunk(b, out, lse, R.chunk_reference(b, 0, 32), 0, 32, f"{q}")
        assert (out[sum(q):] == 7).all() and (lse[sum(q):] == 7).all()


def test_two_graphs_at_once():
    bs = [R.Batch([20, 1, 1], [300, 6000 + 500 * i, 90], 128, 64, 95 + i, DEV) for i in range(2)]
    refs, outs, graphs = [R.chunk_reference(b, 0, 128) for b in bs], [buffers(b) for b in bs], []
    spaces = [chunk(b, 0, 128, *o) for b, o in zip(bs, outs)]
    torch.cuda.synchronize()
    for b, o, ws in zip(bs, outs, spaces):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(4):
                chunk(b, 0, 128, *o, ws)
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for b, o, ws, ref in zip(bs, outs, spaces, refs):
        assert S.splash_workspace_status(ws) == 0
        R.assert_chunk(b, *o, ref, 0, 128, "at once")


def test_a_captured_call_without_work():
    b = R.Batch([1, 2], [70, 90], 16, 64, 97, DEV)
    ws = S.chunk_workspace(b.q, b.pool, b.table, b.scale)
    out, lse = torch.empty(0, 16, 512, device=DEV), torch.empty(0, 16, device=DEV)
    cu = torch.zeros(3, **I32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.splash_chunk_attn(b.q[:0], b.pool, cu, b.table, b.ctx_t, 0, 16, 0, -1, out, lse, ws, b.scale)
    ws.fill_(0xFF)
    graph.replay()
    assert S.splash_workspace_status(ws) == 0


def test_one_token_of_one_head_everywhere():
    b = R.Batch([1], [1], 1, 16, 98, DEV)
    out, lse = buffers(b)
    ws = chunk(b, 0, 1, out, lse)
    assert S.splash_workspace_status(ws) == 0
    assert torch.equal(out[0, 0], b.keys[0][0, :512].to(DEV).float())
    R.assert_chunk(b, out, lse, R.chunk_reference(b, 0, 1), 0, 1, "one of everything")
