"""pa_decode_shared and its FP8 form against the attention formula in 64 bits,
every output, with dead slots poisoned, and against pa_decode: every head size
and block size, ragged groups (one member, more than one query tile, none),
prefixes that end inside a tile, members shorter than the prefix, empty rows,
prefixes longer than the bound; errors; graphs and streams; the step from
pa_build_tables to the attention.

Tolerance, from the arithmetic, for out = sum w_i v_i with softmax weights w:
each weight is rounded at most once to fp16 (2^-11 of its value, twice to first
order since the denominator moves too); its exponent carries the error e of the
fp32 logit, at most D + 2 additions and roundings each off by 2^-23 of the sum
of magnitudes (the tensor cores' additions are not rounded to nearest), and the
exponential's 2^-22; sums of c weights and products in fp32 add c 2^-23; the
output is rounded once (2^-11).  With A = sum w_i |v_i|:
|err| <= 2 (2^-11 + e + c 2^-23 + 2^-21) A + 2^-11 |out| + 2^-24."""
import math
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_158_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
KS, VS = 0.0137, 0.0119


@pytest.fixture(autouse=True)
def _clean():
    pa.pa_decode_set_partition_tokens(0)
    pa.pa_decode_shared_set_min_values(0)      # these batches are small: share all the same
    pa.pa_check_errors()
    yield
    pa.pa_decode_set_partition_tokens(0)
    pa.pa_decode_shared_set_min_values(-1)
    torch.cuda.synchronize()


class Batch:
    """sizes[g] sequences share pre[g] blocks; own[s] tokens follow; `lone` more
    sequences belong to no group."""

    def __init__(self, seed, sizes, pre, own, H, D, B, fp8=False, lone=0, ctx=None, sigma=1.0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        S = sum(sizes) + lone
        self.S, self.H, self.D, self.B, self.fp8 = S, H, D, B, fp8
        of = [p for n, p in zip(sizes, pre) for _ in range(n)] + [0] * lone
        gid = [k for k, n in enumerate(sizes) for _ in range(n)] + [-1] * lone
        own = [own[i % len(own)] for i in range(S)]
        self.ctx = [p * B + x for p, x in zip(of, own)] if ctx is None else list(ctx)
        need = [max(0, -(-c // B) - p) for c, p in zip(self.ctx, of)]
        self.NB = sum(pre) + sum(need) + 3
        ids = torch.randperm(self.NB, generator=g, device=DEV).cpu().numpy().astype(np.int32)
        at = np.concatenate([[0], np.cumsum(pre)]).astype(int)
        k = int(at[-1])
        self.bt = np.full((S, max([p + n for p, n in zip(of, need)] + [1]) + 1), 2 ** 30, dtype=np.int32)
        for s in range(S):
            if gid[s] >= 0:
                self.bt[s, :of[s]] = ids[at[gid[s]]:at[gid[s] + 1]]
            self.bt[s, of[s]:of[s] + need[s]] = ids[k:k + need[s]]
            k += need[s]
        self.starts = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        self.pre = list(pre)
        self.q = torch.randn(S, H, D, generator=g, device=DEV, dtype=torch.float16)
        live = torch.zeros(self.NB, B, dtype=torch.bool)
        for s, c in enumerate(self.ctx):
            i = np.arange(c)
            live[self.bt[s, i // B], i % B] = True
        dead = ~live.to(DEV)
        self.k, self.v = (torch.randn(self.NB, H, B, D, generator=g, device=DEV, dtype=torch.float16) * sigma
                          for _ in range(2))
        if fp8:
            self.k = (self.k.float() / KS).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            self.v = (self.v.float() / VS).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        for t in (self.k, self.v):
            t.permute(0, 2, 1, 3)[dead] = 0x7F if fp8 else float("nan")
        self.scale = 1 / math.sqrt(D)
        self.max_len, self.max_prefix = max(self.ctx + [0]), max(pre + [0]) * B

    def tensors(self):
        return (torch.tensor(self.bt, device=DEV), torch.tensor(self.ctx, dtype=torch.int32, device=DEV),
                torch.tensor(self.starts, device=DEV),
                torch.tensor(np.array(self.pre, dtype=np.int32).reshape(-1), device=DEV))

    def workspace(self):
        return pa.decode_shared_workspace(self.S, len(self.pre), self.H, self.D, self.max_len,
                                          self.max_prefix).fill_(0xFF)

    def call(self, out, ws, t):
        args = (out, self.q, self.k, self.v, *t, self.scale)
        if self.fp8:
            pa.pa_decode_shared_fp8(*args, KS, VS, self.max_len, self.max_prefix, ws)
        else:
            pa.pa_decode_shared(*args, self.max_len, self.max_prefix, ws)

    def run(self, ws=None, t=None):
        out = torch.full((self.S, self.H, self.D), float("nan"), dtype=torch.float16, device=DEV)
        self.call(out, self.workspace() if ws is None else ws, self.tensors() if t is None else t)
        return out

    def check(self, out, seqs=None):
        for s in range(self.S) if seqs is None else seqs:
            c = self.ctx[s]
            if c == 0:
                assert bool((out[s] == 0).all()), s
                continue
            i = torch.arange(c, device=DEV)
            bt = torch.tensor(self.bt[s], device=DEV).long()
            k, v = (x[bt[i // self.B], :, i % self.B] for x in (self.k, self.v))   # [c, H, D]
            if self.fp8:
                k, v = k.view(torch.float8_e4m3fn).double() * KS, v.view(torch.float8_e4m3fn).double() * VS
            k, v, q = k.double().permute(1, 0, 2), v.double().permute(1, 0, 2), self.q[s].double()[..., None]
            w = torch.softmax(self.scale * (k @ q)[..., 0], -1)[:, None]
            ref, mag = (w @ v)[:, 0], (w @ v.abs())[:, 0]
            e = abs(self.scale) * (k.abs() @ q.abs())[..., 0].amax(-1, keepdim=True) * ((self.D + 2) * 2.0 ** -23)
            tol = 2 * (2.0 ** -11 + e + c * 2.0 ** -23 + 2.0 ** -21) * mag + 2.0 ** -11 * ref.abs() + 2.0 ** -24
            err = (out[s].double() - ref).abs()
            assert bool(torch.isfinite(out[s]).all()), s
            assert bool((err <= tol).all()), (s, c, float((err / tol).max()))


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
@pytest.mark.parametrize("B", [4, 8, 16, 32])
@pytest.mark.parametrize("D", [64, 128])
def test_ragged_groups(D, B, fp8):
    """Groups of 1, 2, 5 and 33 members, prefixes from one block to several
    tiles, own parts from nothing to several partitions, two lone sequences."""
    pre = [3, 1, 128 // B + 1, 600 // B]
    b = Batch(D + B, [1, 2, 5, 33], pre, [0, 1, B - 1, B, B + 1, 70, 300, 0, 17], 3, D, B, fp8, lone=2)
    out = b.run()
    assert pa.pa_check_errors()[1] == 0
    b.check(out)
    assert torch.equal(out.view(torch.int16), b.run().view(torch.int16))   # the same call, the same bits


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
@pytest.mark.parametrize("S", [127, 128, 129, 300])
def test_more_members_than_one_query_tile(S, fp8):
    b = Batch(S, [S], [12], [0, 5, 16, 40], 2, 128, 16, fp8)
    b.check(b.run())


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_long_prefix_over_all_workers(fp8):
    b = Batch(7, [9], [20000 // 32], [1, 33], 4, 128, 32, fp8)
    b.check(b.run())
    b = Batch(8, [3, 40, 2], [100, 250, 7], [1, 33, 200], 40, 64, 32, fp8)
    b.check(b.run(), seqs=range(0, 45, 4))


def test_members_shorter_than_the_prefix_and_empty_rows():
    """A member that has not all of the prefix, the first one among them, is
    computed by itself; an empty one gets zeros."""
    B, p = 16, 20
    for ctx in ([p * B + 5, 100, 0, p * B, p * B + 40, 319], [10, 0, p * B, p * B + 1, p * B + 2, 5],
                [0] * 6, [5, 6, 7, 8, 9, p * B]):
        b = Batch(sum(ctx), [6], [p], [0], 4, 128, B, ctx=ctx)
        out = b.run()
        assert pa.pa_check_errors()[1] == 0
        b.check(out)


def test_prefix_bound_and_no_groups():
    b = Batch(21, [8, 8], [40, 9], [10, 100], 4, 128, 16)
    ref = b.run()
    b.check(ref)
    for bound in (0, 15, 16, 200, 10 ** 6):
        b.max_prefix = bound
        b.check(b.run())
    b.starts, b.pre = np.zeros(1, dtype=np.int32), []
    b.check(b.run())
    # no member has a group: the plain decode of the same batch
    out = torch.empty_like(ref)
    bt, ctx, _, _ = b.tensors()
    pa.pa_decode(out, b.q, b.k, b.v, bt, ctx, b.scale, b.max_len, pa.decode_workspace(b.S, b.H, b.D, b.max_len))
    assert float((out.float() - ref.float()).abs().max()) <= 2e-3


def test_groups_in_the_middle_of_the_batch():
    b = Batch(22, [4, 6], [10, 20], [7, 50], 4, 64, 16, lone=5)
    b.starts, b.pre = b.starts[1:], b.pre[1:]               # the first group is not named
    b.check(b.run())


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_more_sequences_than_one_launch(fp8):
    b = Batch(23, [1000, 150], [4, 9], [0, 3, 20], 2, 64, 16, fp8)
    b.check(b.run(), seqs=list(range(0, 1150, 37)) + [999, 1000, 1023, 1024, 1149])


def test_forced_partition_sizes():
    b = Batch(24, [5, 12], [30, 10], [700, 1, 333], 4, 128, 16)
    for p in (32, 96, 1024):
        pa.pa_decode_set_partition_tokens(p)
        b.check(b.run())


def test_growing_logits_move_the_reference():
    b = Batch(25, [20], [64], [40], 2, 128, 16, sigma=1.0)
    ramp = torch.linspace(0, 4, 64 * 16, device=DEV).view(64, 1, 16, 1)
    ids = torch.tensor(b.bt[0, :64], device=DEV).long()
    b.k[ids] = (b.k[ids].float() + ramp * b.q[3].float()[None, :, None]).half()
    b.check(b.run())
    b.scale = -b.scale
    b.check(b.run())


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_a_scale_of_zero_averages_the_values(fp8):
    b = Batch(31, [3, 40], [5, 9], [0, 3, 30], 3, 128, 16, fp8, lone=1)
    b.scale = 0.0
    b.check(b.run())


def test_infinite_logits_of_one_member_stay_in_its_row():
    b = Batch(26, [10], [30], [20], 2, 128, 16)
    b.q[4, 1] = float("inf")
    out = b.run()
    b.q[4, 1] = 0
    ref = b.run()
    keep = torch.ones(10, 2, dtype=torch.bool, device=DEV)
    keep[4, 1] = False
    assert torch.equal(out[keep], ref[keep])


def test_bad_groups_lengths_and_blocks_are_reported():
    b = Batch(27, [6, 6], [10, 20], [7, 50], 2, 64, 16)
    for starts in ([0, 7, 5], [-1, 6, 12], [0, 6, 13]):
        b.starts = np.array(starts, dtype=np.int32)
        out = b.run()
        assert pa.pa_check_errors()[1] == pa.PA_ERRBIT_CONTEXT
        b.check(out)                                         # nothing is shared; still the attention
    b.starts, b.pre = np.array([0, 6, 12], dtype=np.int32), [10, -1]
    b.check(b.run())
    assert pa.pa_check_errors()[1] == pa.PA_ERRBIT_CONTEXT
    b.pre = [10, 20]
    t = b.tensors()
    t[0][:6, 3] = b.NB
    out = b.run(t=t)
    assert pa.pa_check_errors()[1] == pa.PA_ERRBIT_BLOCK_ID
    b.check(out, seqs=range(6, 12))
    t = b.tensors()
    t[1][2] = -3
    out = b.run(t=t)
    assert pa.pa_check_errors()[1] == pa.PA_ERRBIT_CONTEXT
    b.ctx[2] = 0
    b.check(out)


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_small_batches_are_decoded_plainly(fp8):
    """Below 3 * 2^24 spared K and V values the bits are the plain decode's; from there on the prefix
    has its own pass, and the groups are read."""
    b = Batch(29, [9], [16], [30, 5], 4, 64, 16, fp8)
    spared = 2 * 8 * 4 * 64 * 256
    t = b.tensors()
    ref = torch.empty_like(b.run(t=t))
    if fp8:
        pa.pa_decode_fp8(ref, b.q, b.k, b.v, t[0], t[1], b.scale, KS, VS, b.max_len,
                         pa.decode_workspace(b.S, b.H, b.D, b.max_len))
    else:
        pa.pa_decode(ref, b.q, b.k, b.v, t[0], t[1], b.scale, b.max_len,
                     pa.decode_workspace(b.S, b.H, b.D, b.max_len))
    bad = (t[0], t[1], torch.tensor([4, 2], dtype=torch.int32, device=DEV), t[3])
    for values, plain in ((-1, True), (spared + 1, True), (spared, False), (0, False)):
        pa.pa_decode_shared_set_min_values(values)
        out = b.run(t=t)
        b.check(out)
        assert not plain or torch.equal(out.view(torch.int16), ref.view(torch.int16))
        b.check(b.run(t=bad))
        assert pa.pa_check_errors()[1] == (0 if plain else pa.PA_ERRBIT_CONTEXT)


@pytest.mark.parametrize("B,bound", [(4, 10 ** 6), (16, 15)])
def test_groups_are_not_read_where_nothing_can_be_shared(B, bound):
    b = Batch(28, [6, 6], [10, 20], [7, 50], 2, 64, B)
    b.starts, b.max_prefix = np.array([5, -7, 99], dtype=np.int32), bound
    b.check(b.run())
    assert pa.pa_check_errors()[1] == 0


def test_captured_and_replayed_with_new_lengths_and_groups():
    b = Batch(28, [4, 8], [20, 10], [60, 100], 4, 128, 16)
    t, ws = b.tensors(), b.workspace()
    out = torch.empty(b.S, b.H, b.D, dtype=torch.float16, device=DEV)
    b.call(out, ws, t)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.call(out, ws, t)
    full = list(b.ctx)
    for lens, pre in ((full, [20, 10]), ([c - 40 for c in full], [20, 10]), ([5, 0] + full[2:], [20, 3]),
                      (full, [0, 0])):
        b.ctx = lens
        t[1].copy_(torch.tensor(lens, dtype=torch.int32))
        t[3].copy_(torch.tensor(pre, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        b.check(out)
    assert pa.pa_check_errors()[1] == 0


def test_two_streams_with_a_workspace_each():
    a, b = Batch(29, [64], [64], [100], 8, 128, 16), Batch(30, [7, 7], [100, 5], [9], 8, 128, 16, True)
    ra, rb = a.run(), b.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            oa = a.run()
        with torch.cuda.stream(s2):
            ob = b.run()
        torch.cuda.synchronize()
        assert torch.equal(oa.view(torch.int16), ra.view(torch.int16))
        assert torch.equal(ob.view(torch.int16), rb.view(torch.int16))


@pytest.mark.parametrize("fp8", [False, True], ids=["fp16", "fp8"])
def test_shared_prompt_step_by_step(fp8):
    """The first sequence of a group brings the prompt, the others attach to its
    blocks; then all generate: tables and slots by pa_build_tables, the cache
    write, the attention."""
    S, H, D, B, W, P = 5, 2, 64, 16, 16, 9            # P shared blocks
    NB = 64
    rng = random.Random(31)
    g = torch.Generator(device=DEV)
    g.manual_seed(31)
    kc = torch.zeros(NB, H, B, D, dtype=torch.uint8 if fp8 else torch.float16, device=DEV)
    vc = torch.zeros_like(kc)
    tables = torch.full((S, W), -1, dtype=torch.int32, device=DEV)
    ctx = torch.zeros(S, dtype=torch.int32, device=DEV)
    free = torch.tensor(rng.sample(range(NB), NB), dtype=torch.int32, device=DEV)
    nf = torch.tensor([NB], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, S], dtype=torch.int32, device=DEV)
    pre = torch.tensor([P], dtype=torch.int32, device=DEV)
    ws = pa.build_tables_workspace(S)
    ws2 = pa.decode_shared_workspace(S, 1, H, D, W * B, P * B)
    hist = [torch.zeros(0, 2, H, D, device=DEV, dtype=torch.float64) for _ in range(S)]
    for step in range(20):
        if step == 0:
            new = [P * B + 3] + [P * B] * (S - 1)     # the others' tokens are the first one's
        else:
            new = [rng.choice([0, 1, 1, 2]) for _ in range(S)]
        T = sum(new)
        slots, qs = torch.empty(T + 4, dtype=torch.int64, device=DEV), torch.empty(S + 1, dtype=torch.int32, device=DEV)
        pa.pa_build_tables(tables, ctx, qs, slots, nf, free, nf, ctx, torch.tensor(new, dtype=torch.int32, device=DEV),
                           B, NB, ws, starts, pre)
        kv = torch.randn(T + 4, 2, H, D, generator=g, device=DEV, dtype=torch.float16)
        at = [sum(new[:s]) for s in range(S)]
        if step == 0:
            for s in range(1, S):
                kv[at[s]:at[s] + P * B] = kv[:P * B]
        k, v = kv[:, 0].contiguous(), kv[:, 1].contiguous()
        q = torch.randn(S, H, D, generator=g, device=DEV, dtype=torch.float16)
        out = torch.empty(S, H, D, dtype=torch.float16, device=DEV)
        if fp8:
            pa.pa_reshape_and_cache_fp8(k, v, kc, vc, slots, KS, VS)
            pa.pa_decode_shared_fp8(out, q, kc, vc, tables, ctx, starts, pre, 0.125, KS, VS, W * B, P * B, ws2)
        else:
            pa.pa_reshape_and_cache(k, v, kc, vc, slots)
            pa.pa_decode_shared(out, q, kc, vc, tables, ctx, starts, pre, 0.125, W * B, P * B, ws2)
        for s in range(S):
            x = kv[at[s]:at[s] + new[s]].double()
            if fp8:
                for j, sc in enumerate((KS, VS)):
                    f = torch.tensor(sc, dtype=torch.float32, device=DEV)
                    x[:, j] = (kv[at[s]:at[s] + new[s], j].float() / f).clamp(-448, 448).to(torch.float8_e4m3fn).double() * sc
            hist[s] = torch.cat([hist[s], x])
            kk, vv = hist[s][:, 0].permute(1, 0, 2), hist[s][:, 1].permute(1, 0, 2)
            w = torch.softmax(0.125 * (kk @ q[s].double()[..., None])[..., 0], -1)[:, None]
            ref, mag = (w @ vv)[:, 0], (w @ vv.abs())[:, 0]
            # logits: |q||k| / 8 below 64, 66 operations of 2^-23
            tol = 2 * (2.0 ** -11 + 64 * 66 * 2.0 ** -23 + 2.0 ** -15) * mag + 2.0 ** -11 * ref.abs() + 2.0 ** -24
            assert bool(((out[s].double() - ref).abs() <= tol).all()), (step, s)
    assert pa.pa_check_errors()[1] == 0


def test_binding_refuses_wrong_shapes():
    b = Batch(32, [2], [2], [5], 2, 64, 16)
    bt, ctx, st, pre = b.tensors()
    out, ws = torch.empty_like(b.q), b.workspace()
    with pytest.raises(ValueError):
        pa.pa_decode_shared(out, b.q, b.k, b.v, bt, ctx, st[:1], pre, 0.1, 100, 32, ws)
    with pytest.raises(TypeError):
        pa.pa_decode_shared(out, b.q, b.k, b.v, bt, ctx, st.long(), pre, 0.1, 100, 32, ws)
    with pytest.raises(pa.PAError):
        pa.pa_decode_shared(out, b.q, b.k, b.v, bt, ctx, st, pre, 0.1, 100, 32, ws[:64])
    with pytest.raises(pa.PAError):
        pa.pa_decode_shared(out, b.q, b.k, b.v, bt, ctx, st, pre, 0.1, -1, 32, ws)
