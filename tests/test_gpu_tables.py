"""pa_build_tables against a plain sequential model (and the host block
manager): tables, lengths, query starts, slots and the free count are whole
numbers and must be equal, for every block size, from no sequence to several
planning rounds, with and without groups, at both fill paths; in place, in a
captured step, short of blocks, and with bad lengths, groups and ids."""
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_158_gb300 as pa
from paged_kv_cache_158_gb300.pool import BlockManager

pytestmark = pytest.mark.gpu
DEV = "cuda"
UNTOUCHED = -7


@pytest.fixture(autouse=True)
def _clean():
    pa.pa_check_errors()
    yield
    torch.cuda.synchronize()


def model(tables, cached, new, free, num_free, starts, prefix, B, num_blocks, num_slots):
    """The definition, one sequence at a time."""
    S, W = tables.shape
    tables = tables.copy()
    bits = 0
    cached, new = [int(x) for x in cached], [int(x) for x in new]
    for s in range(S):
        if cached[s] < 0 or cached[s] > W * B or new[s] < 0 or cached[s] + new[s] > W * B:
            bits |= pa.PA_ERRBIT_CONTEXT
            cached[s], new[s] = min(max(cached[s], 0), W * B), 0
    leader, want = list(range(S)), [0] * S
    for g, p in enumerate(prefix):
        if 0 <= starts[g] < starts[g + 1] <= S:
            for s in range(starts[g] + 1, starts[g + 1]):
                leader[s], want[s] = starts[g], p

    def plan(new):
        pre, held, need = [0] * S, [0] * S, [0] * S
        clipped = False
        for s in range(S):
            if leader[s] != s:
                has = -(-(cached[leader[s]] + new[leader[s]]) // B)
                pre[s] = min(max(want[s], 0), has)
                clipped |= pre[s] != want[s]
            held[s] = max(-(-cached[s] // B), pre[s])
            need[s] = max(0, -(-(cached[s] + new[s]) // B) - held[s])
        return pre, held, need, clipped

    pre, held, need, clipped = plan(new)
    if clipped:
        bits |= pa.PA_ERRBIT_CONTEXT
    have = num_free if 0 <= num_free <= len(free) else 0
    if have != num_free or sum(need) > have:
        bits |= pa.PA_ERRBIT_POOL
    if sum(need) > have:
        new = [0] * S
        pre, held, need, _ = plan(new)
    top = num_free
    for s in range(S):
        for k in range(need[s]):
            top -= 1
            tables[s, held[s] + k] = free[top]
    for s in range(S):
        tables[s, :pre[s]] = tables[leader[s], :pre[s]]
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    slots = np.full(num_slots, -1, dtype=np.int64)
    if qs[-1] > num_slots:
        bits |= pa.PA_ERRBIT_TOKEN
    for s in range(S):
        for i in range(new[s]):
            p = cached[s] + i
            if qs[s] + i < num_slots and p // B >= pre[s]:
                b = int(tables[s, p // B])
                if 0 <= b < num_blocks:
                    slots[qs[s] + i] = b * B + p % B
                else:
                    bits |= pa.PA_ERRBIT_TOKEN
    ctx = np.array([c + n for c, n in zip(cached, new)], dtype=np.int32)
    return tables, ctx, qs, slots, top, bits


def i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int32).reshape(-1), device=DEV)


class Case:
    def __init__(self, rng, S, B, groups=0, hi=200, new_hi=70, pad=0, short=0, zero_new=False, spare=2):
        self.B = B
        cuts = sorted(rng.sample(range(S + 1), groups + 1)) if groups else []
        self.starts, self.prefix = cuts, [rng.randint(0, 5) for _ in range(groups)]
        self.cached = [rng.choice([0, 1, B - 1, B, B + 1, rng.randint(0, hi)]) for _ in range(S)]
        self.new = [0 if zero_new else rng.choice([0, 1, 1, B, rng.randint(0, new_hi)]) for _ in range(S)]
        for g, p in enumerate(self.prefix):
            for s in range(cuts[g], cuts[g + 1]):
                self.cached[s] += p * B
            if g % 2:
                self.new[cuts[g]] += self.cached[cuts[g]]
                self.cached[cuts[g]] = 0
        width = max([-(-(c + n) // B) for c, n in zip(self.cached, self.new)] + [1]) + spare
        held = [-(-c // B) for c in self.cached]
        need = sum(-(-(c + n) // B) for c, n in zip(self.cached, self.new)) + 3
        self.num_blocks = sum(held) + need
        ids = list(range(self.num_blocks))
        rng.shuffle(ids)
        self.tables = np.full((S, width), UNTOUCHED, dtype=np.int32)
        at = 0
        for s, n in enumerate(held):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        self.free = np.array(ids[at:] + [UNTOUCHED] * 3, dtype=np.int32)
        self.num_free = len(ids) - at - short
        self.num_slots = sum(self.new) + pad

    def run(self, in_place=False, stream=None, num_slots=None):
        S = len(self.cached)
        n = self.num_slots if num_slots is None else num_slots
        t = torch.tensor(self.tables, device=DEV)
        cached, new, nf = i32(self.cached), i32(self.new), i32([self.num_free])
        ctx = cached if in_place else torch.full((S,), -9, dtype=torch.int32, device=DEV)
        left = nf if in_place else torch.full((1,), -9, dtype=torch.int32, device=DEV)
        qs = torch.full((S + 1,), -9, dtype=torch.int32, device=DEV)
        slots = torch.full((n,), -9, dtype=torch.int64, device=DEV)
        gs, pb = (i32(self.starts), i32(self.prefix)) if self.prefix else (None, None)
        pa.pa_build_tables(t, ctx, qs, slots, left, i32(self.free), nf, cached, new, self.B,
                           self.num_blocks, pa.build_tables_workspace(S), gs, pb, stream=stream)
        got = (t.cpu().numpy(), ctx.cpu().numpy(), qs.cpu().numpy(), slots.cpu().numpy(), int(left[0]))
        return got + (pa.pa_check_errors()[1],)

    def check(self, **kw):
        got = self.run(**kw)
        n = kw.get("num_slots")
        ref = model(self.tables, self.cached, self.new, self.free, self.num_free, self.starts,
                    self.prefix, self.B, self.num_blocks, self.num_slots if n is None else n)
        for g, r, what in zip(got, ref, ("tables", "context", "query_start", "slots", "free", "bits")):
            assert np.array_equal(g, r), what
        return got


@pytest.mark.parametrize("B", [4, 8, 16, 32])
@pytest.mark.parametrize("S,groups", [(1, 0), (3, 1), (33, 4), (257, 9)])
def test_small_steps(S, groups, B):
    rng = random.Random(1000 * S + B)
    Case(rng, S, B, groups).check()
    Case(rng, S, B, groups, pad=37).check(in_place=True)


@pytest.mark.parametrize("S,groups", [(1000, 30), (1024, 0), (1025, 7), (2500, 1100)])
def test_both_fill_paths_and_several_planning_rounds(S, groups):
    """More than 4096 slots, more than 1024 sequences, more than 1024 groups."""
    rng = random.Random(S)
    Case(rng, S, 16, groups, hi=500, new_hi=300, pad=5000).check()
    Case(rng, S, 8, groups, hi=500, new_hi=30).check(in_place=True)


def test_one_long_prompt_and_the_border_of_the_fill_rule():
    for n in (4095, 4096, 4097, 100_001):
        c = Case(random.Random(n), 2, 16)
        c.cached, c.new = [0, 5], [n - 1, 1]
        c.tables = np.full((2, n // 16 + 2), UNTOUCHED, dtype=np.int32)
        c.tables[1, 0] = 0
        c.num_blocks = n // 16 + 20
        c.free = np.arange(1, c.num_blocks, dtype=np.int32)
        c.num_free, c.num_slots = len(c.free), n
        c.check()


def test_nothing_to_do():
    c = Case(random.Random(3), 40, 16, 3, zero_new=True)
    c.new = [0] * 40
    c.check()
    # no sequences: an all-padding slot map
    e = Case(random.Random(4), 1, 16)
    e.tables, e.cached, e.new = np.zeros((0, 4), np.int32), [], []
    e.num_slots = 9
    got = e.run()
    assert (got[3] == -1).all() and got[2].tolist() == [0] and got[4] == e.num_free and got[5] == 0


@pytest.mark.parametrize("S", [40, 1500])
def test_too_few_blocks_take_none(S):
    c = Case(random.Random(S), S, 16, 5, hi=300, new_hi=200, short=0)
    c.num_free = 3
    got = c.check()
    assert got[5] & pa.PA_ERRBIT_POOL and got[4] == 3
    c.num_free = len(c.free) + 1                 # a count past the list
    assert c.check()[5] & pa.PA_ERRBIT_POOL
    c.num_free = -1
    assert c.check()[5] & pa.PA_ERRBIT_POOL


def test_exactly_enough_blocks():
    c = Case(random.Random(8), 60, 16, 4)
    need = c.num_free - c.run()[4]
    c.free, c.num_free = c.free[:need], need
    got = c.check()
    assert got[4] == 0 and got[5] == 0


def test_bad_lengths_groups_and_ids_are_reported():
    c = Case(random.Random(5), 30, 16, 0)
    c.cached[3], c.new[4], c.new[7] = -5, -1, 10 ** 6
    assert c.check()[5] & pa.PA_ERRBIT_CONTEXT
    c = Case(random.Random(6), 30, 16, 3)
    c.prefix[1] = 50                              # more than its first sequence has
    assert c.check()[5] & pa.PA_ERRBIT_CONTEXT
    c = Case(random.Random(7), 30, 16, 0)
    c.starts, c.prefix = [20, 35], [2]            # past the batch: shares nothing
    c.check()
    c = Case(random.Random(9), 30, 16, 0)
    c.new = [20] * 30
    c.tables = np.full((30, 40), UNTOUCHED, dtype=np.int32)
    c.cached = [0] * 30
    c.num_blocks = 64
    c.free = np.arange(80, dtype=np.int32)        # ids past the pool
    c.num_free, c.num_slots = 80, 600
    assert c.check()[5] & pa.PA_ERRBIT_TOKEN
    c = Case(random.Random(10), 30, 16, 2, pad=0)
    assert c.check(num_slots=max(0, c.num_slots - 5))[5] & pa.PA_ERRBIT_TOKEN


def test_agrees_with_the_host_block_manager():
    """Prompts, then single tokens: the same tables and slots as append_tokens."""
    S, B, NB, W = 6, 16, 128, 20
    rng = random.Random(11)
    order = np.array(rng.sample(range(NB), NB), dtype=np.int32)
    bm = BlockManager(NB, B, S, W, free_order=order)
    for s in range(S):
        bm.add_sequence(s)
    t = torch.full((S, W), -1, dtype=torch.int32, device=DEV)
    ctx, nf = torch.zeros(S, dtype=torch.int32, device=DEV), i32([NB])
    free, ws = i32(order), pa.build_tables_workspace(S)
    for step in range(40):
        new = [rng.randint(0, 60) for _ in range(S)] if step == 0 else [rng.choice([0, 1, 1, 3]) for _ in range(S)]
        slots = torch.empty(sum(new), dtype=torch.int64, device=DEV)
        qs = torch.empty(S + 1, dtype=torch.int32, device=DEV)
        pa.pa_build_tables(t, ctx, qs, slots, nf, free, nf, ctx, i32(new), B, NB, ws)
        ref = []
        for s in range(S):
            pos = bm.append_tokens(s, new[s])
            ref += [int(bm.tables[s, p // B]) * B + int(p) % B for p in pos]
        assert slots.tolist() == ref
        assert np.array_equal(t.cpu().numpy(), bm.tables)
        assert ctx.tolist() == bm.lengths.tolist() and int(nf[0]) == bm.num_free()
    assert pa.pa_check_errors()[1] == 0


def test_captured_steps_advance_in_place():
    """A captured build replayed: lengths, tables and the free count advance on the GPU."""
    S, B, NB, W = 5, 8, 64, 12
    t = torch.full((S, W), -1, dtype=torch.int32, device=DEV)
    ctx, nf, new = torch.zeros(S, dtype=torch.int32, device=DEV), i32([NB]), i32([1, 1, 0, 1, 1])
    free, ws = i32(np.arange(NB)), pa.build_tables_workspace(S)
    slots = torch.empty(8, dtype=torch.int64, device=DEV)
    qs = torch.empty(S + 1, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pa.pa_build_tables(t, ctx, qs, slots, nf, free, nf, ctx, new, B, NB, ws)
    tables, lens, left = np.full((S, W), -1, dtype=np.int32), [0] * S, NB
    for _ in range(3 * B + 1):
        g.replay()
        tables, c, q, sl, left, bits = model(tables, lens, [1, 1, 0, 1, 1], np.arange(NB), left, [], [], B, NB, 8)
        lens = c.tolist()
        assert ctx.tolist() == lens and slots.tolist() == sl.tolist() and int(nf[0]) == left
        assert np.array_equal(t.cpu().numpy(), tables) and bits == 0
    assert pa.pa_check_errors()[1] == 0


def test_on_another_stream_and_two_at_once():
    a, b = Case(random.Random(20), 700, 16, 9, pad=4000), Case(random.Random(21), 30, 16, 2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        a.check(stream=s1)
    with torch.cuda.stream(s2):
        b.check()


def test_binding_refuses_what_the_shapes_do_not_allow():
    c = Case(random.Random(22), 4, 16)
    z = torch.zeros(4, dtype=torch.int32, device=DEV)
    t, qs = torch.zeros(4, 6, dtype=torch.int32, device=DEV), torch.zeros(5, dtype=torch.int32, device=DEV)
    sl, nf, ws = torch.zeros(4, dtype=torch.int64, device=DEV), i32([3]), pa.build_tables_workspace(4)
    ok = dict(block_size=16, num_blocks=8, workspace=ws)
    with pytest.raises(ValueError):
        pa.pa_build_tables(t, z[:3], qs, sl, nf, z, nf, z, z, **ok)
    with pytest.raises(ValueError):
        pa.pa_build_tables(t, z, qs, sl, nf, z, nf, z, z, group_start=qs, **ok)
    with pytest.raises(TypeError):
        pa.pa_build_tables(t, z, qs, sl.int(), nf, z, nf, z, z, **ok)
    with pytest.raises(pa.PAError):                      # the new lengths would be overwritten
        pa.pa_build_tables(t, z, qs, sl, nf, i32([1]), nf, z.clone(), z, **ok)
    with pytest.raises(pa.PAError):
        pa.pa_build_tables(t, z, qs, sl, nf, i32([1]), nf, z, z.clone(), 12, 8, ws)
    with pytest.raises(pa.PAError):
        pa.pa_build_tables(t, z, qs, sl, nf, i32([1]), nf, z, z.clone(), 16, 8, ws[:16])
    assert c.check()[5] == 0
