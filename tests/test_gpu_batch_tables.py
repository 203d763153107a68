"""Index arrays of a batch built on the device, and pages given back (marked gpu), against the same
steps in Python's whole numbers."""
import random

import pytest
import torch

from layout_agnostic_paged_gb300 import splash as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def pages(n, P):
    return -(-n // P)


class Cache:
    """A pool's free list and a batch's lengths and table; the same on the device and in lists."""

    def __init__(self, past, new, P, free, rows=None, width=None, seed=0, pool=None):
        rng = random.Random(seed)
        self.P, self.past, self.new = P, list(past), list(new)
        have = [pages(max(p, 0), P) for p in past]
        self.num_pages = pool or sum(have) + free + 3
        ids = rng.sample(range(self.num_pages), sum(have) + free)
        self.width = width or max([1] + [pages(p + n, P) for p, n in zip(past, new)])
        self.table = [[-1] * self.width for _ in past]
        o = 0
        for r, h in enumerate(have):
            for k in range(min(h, self.width)):
                self.table[r][k] = ids[o + k]
            o += h
        self.stack = ids[o:] + [-7] * (self.num_pages - free)
        self.free = free
        self.rows = sum(n for n in new if n > 0) if rows is None else rows
        self.pos, self.slots = [-5] * self.rows, [-5] * self.rows

    def device(self, lead=0):
        i = lambda v, n=None: torch.tensor(v, dtype=torch.int32, device=DEV).reshape(n if n is not None else (len(v),))
        odd = lambda n: torch.full((n + lead,), -5, dtype=torch.int32, device=DEV)[lead:]
        B = len(self.past)
        self.d = dict(past=i(self.past), new=i(self.new), table=i(self.table, (B, self.width)), stack=i(self.stack),
                      left=i([self.free, -5]), cu=odd(B + 1), ctx=odd(B), pos=odd(self.rows), slots=odd(self.rows))
        return self.d

    def build(self):
        """The expected (cu, ctx, positions, slots, table, left)."""
        pos, slots = self.pos, self.slots          # (rows behind the last token stay as they were)
        cu, ctx, top, served, go = [0], [], self.free, 0, True
        for r, (p, n) in enumerate(zip(self.past, self.new)):
            go = go and p >= 0 and n >= 0 and p + n <= self.width * self.P
            need = pages(p + n, self.P) - pages(p, self.P) if go else 0
            go = go and need <= top and cu[-1] + n <= self.rows
            if go:
                for k in range(need):
                    self.table[r][pages(p, self.P) + k] = self.stack[top - 1 - k]
                top -= need
                for i in range(n):
                    id = self.table[r][(p + i) // self.P]
                    pos[cu[-1] + i] = p + i
                    slots[cu[-1] + i] = id * self.P + (p + i) % self.P if 0 <= id < self.num_pages else -1
            served += go
            cu.append(cu[-1] + (n if go else 0))
            ctx.append(p + (n if go else 0))
        self.free = top
        return cu, ctx, pos, slots, self.table, [top, served]

    def release(self, ctx, keep, window=0, sinks=0):
        gone, out = [], []
        for r, c in enumerate(ctx):
            k = min(max(keep[r], 0), c)
            drop = set(range(pages(k, self.P), pages(c, self.P)))
            if window:
                drop |= {j for j in range(pages(c, self.P)) if j * self.P >= sinks and (j + 1) * self.P <= k + 1 - window}
            for j in sorted(drop):
                if 0 <= self.table[r][j] < self.num_pages:
                    gone.append(self.table[r][j])
                self.table[r][j] = -1
            out.append(k)
        for id in reversed(gone):
            if self.free < self.num_pages:
                self.stack[self.free] = id
                self.free += 1
        return out


def run_build(c, in_place=False):
    d = c.d
    ctx = d["past"] if in_place else d["ctx"]
    S.splash_batch_tables(d["past"], d["new"], d["table"], c.P, d["stack"], d["left"][:1], d["cu"], ctx, d["pos"],
                          d["slots"], d["left"])
    return ctx


def check_build(c, lead=0, in_place=False):
    stack = list(c.stack)
    c.device(lead)
    ctx = run_build(c, in_place)
    cu, want_ctx, pos, slots, table, left = c.build()
    d = c.d
    assert d["cu"].tolist() == cu and ctx.tolist() == want_ctx
    assert d["pos"].tolist() == pos and d["slots"].tolist() == slots
    assert d["table"].tolist() == table and d["left"].tolist() == left and d["stack"].tolist() == stack
    return ctx


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("B", [1, 2, 31, 256, 1023, 1024, 1025, 2500])
def test_single_tokens(B, P):
    rng = random.Random(B + P)
    past = [rng.randint(0, 5 * P) for _ in range(B)]
    need = sum(p % P == 0 for p in past)
    check_build(Cache(past, [1] * B, P, need, seed=B), in_place=B % 2 == 0)


@pytest.mark.parametrize("lead", [0, 1, 3])
@pytest.mark.parametrize("B,most", [(1, 5000), (3, 4000), (17, 700), (64, 300), (1100, 9)])
def test_ragged_prompts(B, most, lead):
    rng = random.Random(B)
    new = [rng.choice((0, rng.randint(0, most))) for _ in range(B)]
    past = [rng.choice((0, rng.randint(0, 900))) for _ in range(B)]
    check_build(Cache(past, new, 16, sum(new) // 16 + 2 * B, seed=B + 1), lead, in_place=lead == 1)


def test_lengths_around_page_borders():
    P, at = 16, [0, 1, 15, 16, 17, 31, 32, 33]
    both = [(p, n) for p in at for n in at]
    check_build(Cache([p for p, _ in both], [n for _, n in both], P, 500))


@pytest.mark.parametrize("rows", [2047, 2048, 2049, 4095, 4096, 4097, 4100])
def test_rows_at_the_border_of_the_two_forms(rows):
    check_build(Cache([5, 0, 77], [rows - 901, 900, 1], 64, 200))


def test_spare_rows_are_left_as_they_were():
    check_build(Cache([3, 20], [4, 5], 16, 9, rows=40))
    check_build(Cache([3, 20], [4, 5], 16, 9, rows=5000))


@pytest.mark.parametrize("free", [0, 1, 2, 5, 6, 7])
def test_a_batch_that_does_not_fit_is_cut(free):
    # needs 1, 0, 2, 0, 3, 0, 1 pages
    check_build(Cache([0, 3, 16, 5, 0, 1, 32], [5, 2, 17, 0, 48, 1, 1], 16, free))


@pytest.mark.parametrize("rows", [0, 1, 5, 6, 7, 8, 26, 27])
def test_a_batch_with_too_few_rows_is_cut(rows):
    check_build(Cache([0, 3, 16, 5], [5, 2, 19, 1], 16, 20, rows=rows))


@pytest.mark.parametrize("past,new", [([4, -1, 4], [1, 1, 1]), ([4, 4, 4], [1, -2, 1]), ([4, 40, 4], [1, 9, 1]),
                                      ([-2 ** 31, 4], [5, 1]), ([2 ** 31 - 1, 4], [2 ** 31 - 1, 1]), ([4, 48], [1, 1])])
def test_bad_lengths_end_the_batch(past, new):
    check_build(Cache([min(p, 48) for p in past], [1] * len(past), 16, 20, width=3))   # (the good one, for the table)
    c = Cache([p if 0 <= p <= 48 else 0 for p in past], [1] * len(past), 16, 20, rows=50, width=3)
    c.past, c.new = past, new
    check_build(c)


def test_a_stop_in_a_later_pass():
    n = 2100
    c = Cache([0] * n, [1] * n, 16, 1500)
    check_build(c)
    assert c.d["left"].tolist() == [0, 1500]


def test_nothing():
    check_build(Cache([], [], 16, 4, rows=3, width=2))
    check_build(Cache([5, 6], [0, 0], 16, 4, rows=0))
    check_build(Cache([0, 0], [0, 0], 16, 0, rows=4, width=1))


def test_the_count_may_be_left_itself():
    c, other = Cache([0, 20, 64], [5, 1, 30], 16, 9), Cache([0, 20, 64], [5, 1, 30], 16, 9)
    check_build(c)
    d = other.device()
    S.splash_batch_tables(d["past"], d["new"], d["table"], 16, d["stack"], d["left"], d["cu"], d["ctx"], d["pos"], d["slots"],
                          d["left"])
    for name in ("table", "cu", "ctx", "pos", "slots", "left"):
        assert torch.equal(d[name], c.d[name]), name


def test_a_table_without_pages():
    i = lambda *n: torch.zeros(*n, dtype=torch.int32, device=DEV)
    past, new, table, left = i(3), torch.tensor([0, 0, 1], dtype=torch.int32, device=DEV), i(3, 0), i(2)
    cu, ctx, pos, slots = i(4), i(3), i(5), i(5)
    S.splash_batch_tables(past, new, table, 16, i(0), left[:1], cu, ctx, pos, slots, left)
    assert left.tolist() == [0, 2] and cu.tolist() == [0] * 4 and ctx.tolist() == [0] * 3
    S.splash_batch_release(ctx, None, table, 16, i(0), left)
    assert ctx.tolist() == [0] * 3 and left[0].item() == 0


def test_counts_out_of_range_are_clamped():
    c = Cache([0, 0], [9, 9], 16, 2)
    c.device()
    c.d["left"][0] = -4
    run_build(c)
    assert c.d["left"].tolist() == [0, 0] and c.d["cu"].tolist() == [0, 0, 0] and c.d["ctx"].tolist() == [0, 0]
    c = Cache([0], [9], 16, 5, pool=5)
    c.device()
    c.d["left"][0] = 10 ** 9
    run_build(c)
    assert c.d["left"].tolist() == [4, 1] and c.d["table"][0, 0].item() == c.stack[4]


def test_bad_ids_have_no_slots():
    c = Cache([5, 0], [3, 3], 16, 4)
    c.table[0][0] = c.num_pages
    c.stack[3] = -2
    check_build(c)


# ------------------------------------------------------------------ pages given back

def check_release(c, ctx, keep, window=0, sinks=0):
    d = c.d
    k = torch.tensor(keep, dtype=torch.int32, device=DEV) if keep is not None else None
    S.splash_batch_release(ctx, k, d["table"], c.P, d["stack"], d["left"], window, sinks)
    want = c.release(ctx_list := c.ctx_before, keep if keep is not None else ctx_list, window, sinks)
    assert ctx.tolist() == want and d["table"].tolist() == c.table
    assert d["stack"].tolist() == c.stack and d["left"][0].item() == c.free


def built(past, new, P, free, **kw):
    c = Cache(past, new, P, free, **kw)
    ctx = check_build(c)
    c.ctx_before = ctx.tolist()
    return c, ctx


@pytest.mark.parametrize("B", [1, 7, 256, 257, 1000, 9000])
def test_dropping_the_step_restores_the_stack(B):
    rng = random.Random(B)
    past = [rng.randint(0, 70) for _ in range(B)]
    new = [rng.randint(0, 40) for _ in range(B)]
    c, ctx = built(past, new, 16, 4 * B)
    top, stack = 4 * B, list(c.stack)
    check_release(c, ctx, past)
    assert c.free == top and c.stack == stack


@pytest.mark.parametrize("P", [16, 128])
def test_keeping_some_tokens(P):
    rng = random.Random(P)
    past = [rng.randint(0, 9 * P) for _ in range(300)]
    new = [rng.randint(0, 3 * P) for _ in range(300)]
    c, ctx = built(past, new, P, 1200)
    keep = [rng.choice((0, p, p + n, p + n + 5, -3, rng.randint(0, p + n))) for p, n in zip(past, new)]
    check_release(c, ctx, keep)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 0), (33, 16), (100, 17), (64, 1000), (10 ** 9, 0),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
def test_pages_that_a_window_leaves(window, sinks):
    past, new = [0, 1, 15, 16, 17, 40, 100, 333, 700], [1, 0, 1, 1, 17, 3, 0, 9, 1]
    c, ctx = built(past, new, 16, 30)
    check_release(c, ctx, None, window, sinks)
    c.ctx_before = ctx.tolist()
    check_release(c, ctx, None, window, sinks)     # (nothing is given back twice)
    c.ctx_before = ctx.tolist()
    check_release(c, ctx, [0, 0, 20, 5, 34, 0, 99, 100, 650], window, sinks)


def test_long_requests():
    c, ctx = built([40000, 3, 50000], [9, 9, 9], 16, 9)
    check_release(c, ctx, [17, 12, 0])


def check_sparse(B, most, P, ctx_lo, keep_lo, window, sinks, holes, seed):
    """Tables with entries that went back before (a share `holes` of them) and that never were pages, against a mask."""
    g = torch.Generator().manual_seed(seed)
    ints = lambda lo, hi, *n: torch.randint(lo, hi, n, generator=g, dtype=torch.int32)
    pages = 1 << 20
    table = ints(-5, pages + 40, B, most)
    table[torch.rand(B, most, generator=g) < holes] = -1
    ctx = ints(ctx_lo, most * P + 1, B)
    keep = torch.minimum(ints(keep_lo, most * P + 1, B), ctx) if keep_lo is not None else ctx.clone()
    page = torch.arange(most)
    kept = -(-keep // P)
    gone = (page >= kept[:, None]) & (page < -(-ctx[:, None] // P))
    if window:
        gone |= (page * P >= sinks) & ((page + 1) * P <= keep[:, None] + 1 - window)
    ids = table[gone & (table >= 0) & (table < pages)]
    top = 11
    want = torch.full((pages,), -7, dtype=torch.int32)
    n = min(len(ids), pages - top)
    assert n == len(ids)
    want[top:top + n] = ids.flip(0)
    t, c, stack = table.to(DEV), ctx.to(DEV), torch.full((pages,), -7, dtype=torch.int32, device=DEV)
    left = torch.tensor([top, 5], dtype=torch.int32, device=DEV)
    S.splash_batch_release(c, keep.to(DEV) if keep_lo is not None else None, t, P, stack, left, window, sinks)
    assert torch.equal(stack.cpu(), want) and left.tolist() == [top + n, 5] and torch.equal(c.cpu(), keep)
    assert torch.equal(t.cpu(), torch.where(gone, -1, table))


# runs of a warp within one request and over many; several passes over the requests; more groups than there are marks
@pytest.mark.parametrize("B,most,P,ctx_lo,keep_lo,window,sinks,holes", [
    (1, 3000, 64, 180000, None, 4096, 4, .5), (1, 9000, 16, 140000, 0, 0, 0, .0), (64, 2048, 64, 100000, None, 4096, 100, .999),
    (5, 2100, 128, 0, 0, 1000, 300, .3), (1024, 40, 16, 0, 0, 100, 17, .2), (1025, 40, 16, 0, 0, 100, 17, .2),
    (3000, 70, 32, 0, None, 64, 0, .9), (4100, 3, 16, 0, 0, 0, 0, .5), (2500, 900, 16, 10000, None, 500, 1, .8),
    (3, 750000, 16, 11000000, None, 2048, 1, .95), (2049, 1200, 16, 19000, 19000, 333, 0, .97),
])
def test_pages_that_went_back_before(B, most, P, ctx_lo, keep_lo, window, sinks, holes):
    check_sparse(B, most, P, ctx_lo, keep_lo, window, sinks, holes, B + most)


def test_a_full_stack_and_bad_counts():
    c, ctx = built([16, 16, 16], [1, 1, 1], 16, 5)
    c.free = c.num_pages - 2                       # a count that does not fit the pages that are out
    c.d["left"][0] = c.free
    stack = list(c.stack)
    S.splash_batch_release(ctx, None, c.d["table"], 16, c.d["stack"], c.d["left"])      # (nothing)
    assert c.d["stack"].tolist() == stack
    k = torch.zeros(3, dtype=torch.int32, device=DEV)
    S.splash_batch_release(ctx, k, c.d["table"], 16, c.d["stack"], c.d["left"])
    assert c.d["left"][0].item() == c.num_pages and (c.d["table"] == -1).all() and (ctx == 0).all()


def test_lengths_past_the_table_are_clamped():
    c, ctx = built([16, 5], [1, 1], 16, 5, width=2)
    ctx.copy_(torch.tensor([10 ** 6, -4]))
    c.ctx_before = [32, 0]
    check_release(c, ctx, [3, 3])


# ------------------------------------------------------------------ calls around them

def test_a_captured_step_replays():
    c = Cache([15, 3, 60], [1, 1, 1], 16, 20)
    d = c.device()
    past0, table0, left0 = d["past"].clone(), d["table"].clone(), d["left"].clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run_build(c, in_place=True)                # (loads the kernels)
    s.synchronize()
    d["past"].copy_(past0), d["table"].copy_(table0), d["left"].copy_(left0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run_build(c, in_place=True)
    for _ in range(40):                            # a token more each time
        g.replay()
    torch.cuda.synchronize()
    for i in range(40):
        cu, ctx, pos, slots, table, left = c.build()
        c.past = ctx
    assert d["past"].tolist() == ctx and d["table"].tolist() == table and d["left"].tolist() == left
    assert d["pos"].tolist() == pos and d["slots"].tolist() == slots


def test_two_batches_on_two_streams():
    rng = random.Random(4)
    a, b = (Cache([rng.randint(0, 99) for _ in range(400)], [rng.randint(0, 30) for _ in range(400)], 16, 2000, seed=i)
            for i in range(2))
    for c in (a, b):
        c.device()
        c.stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for c in (a, b):
            d = c.d
            S.splash_batch_tables(d["past"], d["new"], d["table"], c.P, d["stack"], d["left"][:1], d["cu"], d["ctx"],
                                  d["pos"], d["slots"], d["left"], stream=c.stream)
            S.splash_batch_release(d["ctx"], d["past"], d["table"], c.P, d["stack"], d["left"], stream=c.stream)
    torch.cuda.synchronize()
    for c in (a, b):
        stack, free = list(c.stack), c.free
        cu, ctx, pos, slots, _, left = c.build()
        assert c.d["pos"].tolist() == pos and c.d["slots"].tolist() == slots and c.d["cu"].tolist() == cu
        assert c.d["stack"].tolist() == stack and c.d["left"].tolist() == [free, left[1]]


def test_refusals_of_the_binding():
    c = Cache([5, 6], [1, 1], 16, 4)
    d = c.device()
    with pytest.raises(ValueError, match="new_lens"):
        S.splash_batch_tables(d["past"], d["new"].long(), d["table"], 16, d["stack"], d["left"][:1], d["cu"], d["ctx"],
                              d["pos"], d["slots"], d["left"])
    with pytest.raises(ValueError, match="cu_q"):
        S.splash_batch_tables(d["past"], d["new"], d["table"], 16, d["stack"], d["left"][:1], d["cu"][:2], d["ctx"],
                              d["pos"], d["slots"], d["left"])
    with pytest.raises(S.SplashError):
        S.splash_batch_tables(d["past"], d["new"], d["table"], 24, d["stack"], d["left"][:1], d["cu"], d["ctx"],
                              d["pos"], d["slots"], d["left"])
    with pytest.raises(S.SplashError):
        S.splash_batch_release(d["ctx"], None, d["table"], 16, d["stack"], d["left"], window=-1)
    with pytest.raises(ValueError, match="keep_lens"):
        S.splash_batch_release(d["ctx"], d["cu"], d["table"], 16, d["stack"], d["left"])
