"""The latent cache: pa_latent_write bit for bit against numpy indexing, and
pa_latent_decode against the definition in 64 bits, every output, with dead
slots poisoned.

Tolerance of the decode, from its arithmetic, for out = sum w_i v_i with
softmax weights w: each weight is rounded once to fp16 (at most 2^-11 of its
value, twice to first order since the denominator moves too); its exponent
carries the error e of the fp32 logit, at most 576 additions each off by
2^-23 of the sum of magnitudes (the tensor cores' additions are not rounded to
nearest) plus two roundings and the exponential's 2^-22; sums of c weights and
products in fp32 add c 2^-23 more; the output is rounded once (2^-11).  With
A = sum w_i |v_i|:  |err| <= 2 (2^-11 + e + c 2^-23 + 2^-21) A + 2^-11 |out| + 2^-24."""
import math
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_158_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
LAT, ROW = 512, 576


@pytest.fixture(autouse=True)
def _clean():
    pa.pa_check_errors()
    yield
    torch.cuda.synchronize()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, sigma=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float16) * sigma


class Batch:
    def __init__(self, seed, ctx, H, B, sigma=0.7, width=2, order=None):
        g = gen(seed)
        self.S, self.H, self.B, self.ctx = len(ctx), H, B, list(ctx)
        need = [-(-c // B) for c in ctx]
        self.NB = sum(need) + 3
        ids = torch.randperm(self.NB, generator=g, device=DEV).cpu().numpy() if order is None else order(self.NB)
        self.bt = np.full((self.S, max(need + [0]) + width), 2 ** 30, dtype=np.int32)  # never read
        at = 0
        for s, n in enumerate(need):
            self.bt[s, :n] = ids[at:at + n]
            at += n
        self.q = normal(g, self.S, H, ROW)
        self.cache = normal(g, self.NB, B, ROW, sigma=sigma)
        live = torch.zeros(self.NB, B, dtype=torch.bool)
        for s, c in enumerate(ctx):
            i = np.arange(c)
            live[self.bt[s, i // B], i % B] = True
        self.cache[~live.to(DEV)] = float("nan")       # dead slots
        self.scale = 1 / math.sqrt(192)
        self.max_len = max(self.ctx + [0])

    def tensors(self):
        return torch.tensor(self.bt, device=DEV), torch.tensor(self.ctx, dtype=torch.int32, device=DEV)

    def run(self, ws=None, out=None, stream=None):
        bt, ctx = self.tensors()
        out = torch.full((self.S, self.H, LAT), float("nan"), dtype=torch.float16, device=DEV) if out is None else out
        ws = pa.latent_decode_workspace(self.S, self.H).fill_(0xFF) if ws is None else ws
        pa.pa_latent_decode(out, self.q, self.cache, bt, ctx, self.scale, self.max_len, ws, stream=stream)
        return out

    def check(self, out, seqs=None):
        for s in range(self.S) if seqs is None else seqs:
            c = self.ctx[s]
            if c == 0:
                assert (out[s] == 0).all()
                continue
            i = torch.arange(c, device=DEV)
            bt = torch.tensor(self.bt[s], device=DEV).long()
            k = self.cache[bt[i // self.B], i % self.B].double()
            q = self.q[s].double()
            w = torch.softmax(self.scale * (q @ k.T), -1)
            ref = w @ k[:, :LAT]
            e = abs(self.scale) * (q.abs() @ k.abs().T).amax(-1, keepdim=True) * (576 * 2.0 ** -23)
            tol = 2 * (2.0 ** -11 + e + c * 2.0 ** -23 + 2.0 ** -21) * (w @ k[:, :LAT].abs()) \
                + 2.0 ** -11 * ref.abs() + 2.0 ** -24
            err = (out[s].double() - ref).abs()
            assert bool(torch.isfinite(out[s]).all()), s
            assert bool((err <= tol).all()), (s, c, float((err / tol).max()))


@pytest.mark.parametrize("T", [1, 2, 63, 1000])
@pytest.mark.parametrize("B", [4, 8, 16, 32])
def test_write_is_bit_exact(T, B):
    g = gen(T * 100 + B)
    NB = 2 * T // B + 2
    wide = normal(g, T, ROW + 24)
    cache = normal(g, NB, B, ROW)
    slots = torch.randperm(NB * B, generator=g, device=DEV)[:T].contiguous()
    slots[::5] = -1
    latent, rope = wide[:, 8:8 + LAT], wide[:, LAT + 16:LAT + 16 + 64]   # slices of one projection
    ref = cache.clone()
    flat = ref.view(-1, ROW)
    keep = (slots >= 0).nonzero()[:, 0]
    flat[slots[keep]] = torch.cat([latent, rope], 1)[keep]
    pa.pa_latent_write(latent, rope, cache, slots)
    assert torch.equal(cache.view(torch.int16), ref.view(torch.int16))
    assert pa.pa_check_errors()[1] == 0
    pa.pa_latent_write(latent.contiguous(), rope.contiguous(), cache, slots)
    assert torch.equal(cache.view(torch.int16), ref.view(torch.int16))


def test_write_reports_slots_past_the_pool():
    g = gen(5)
    cache = normal(g, 3, 16, ROW)
    ref = cache.clone()
    slots = torch.tensor([48, 2, -3, 2 ** 40], device=DEV)
    lat, rope = normal(g, 4, LAT), normal(g, 4, 64)
    pa.pa_latent_write(lat, rope, cache, slots)
    assert pa.pa_check_errors()[1] == pa.PA_ERRBIT_SLOT
    ref.view(-1, ROW)[2] = torch.cat([lat, rope], 1)[1]
    assert torch.equal(cache, ref)
    pa.pa_latent_write(lat[:0], rope[:0], cache, slots[:0])


@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("H", [1, 16, 20, 64, 65, 128])
def test_ragged_batches(H, B):
    ctx = [0, 1, 2, B - 1, B, B + 1, 63, 64, 65, 127, 128, 129, 300, 0]
    b = Batch(H * 64 + B, ctx, H, B)
    out = b.run()
    b.check(out)
    assert pa.pa_check_errors()[1] == 0
    assert torch.equal(out.view(torch.int16), b.run().view(torch.int16))  # the same call, the same bits


@pytest.mark.parametrize("H,ctx", [(16, [1]), (16, [20001]), (128, [9000, 17]), (64, [64 * 152]),
                                   (40, [64 * 153 + 1, 5, 0, 4000]), (128, [700] * 90), (200, [500, 1000])])
def test_split_contexts(H, ctx):
    b = Batch(sum(ctx) + H, ctx, H, 32)
    b.check(b.run())
    assert pa.pa_check_errors()[1] == 0


def test_more_sequences_than_one_launch():
    rng = random.Random(2)
    b = Batch(3, [rng.randint(0, 90) for _ in range(1300)], 16, 16)
    b.check(b.run())


def test_large_logits_and_moving_maxima():
    """Logits that grow along the context move the reference again and again."""
    b = Batch(9, [1000, 777], 32, 16, sigma=1.0)
    for s in range(2):
        i = torch.arange(b.ctx[s], device=DEV)
        bt = torch.tensor(b.bt[s], device=DEV).long()
        rows = b.cache[bt[i // 16], i % 16].float()
        ramp = torch.linspace(0, 3, b.ctx[s], device=DEV)[:, None]
        b.cache[bt[i // 16], i % 16] = (rows + ramp * b.q[s, 0].float()[None]).half()
    b.check(b.run())
    b.scale = -b.scale                                # any multiplier
    b.check(b.run())


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-42])
def test_a_scale_of_zero_averages_the_rows(scale):
    b = Batch(16, [1, 31, 33, 100, 4000], 20, 16)
    b.scale = scale
    b.check(b.run())


def test_a_workspace_on_any_16_bytes():
    b = Batch(17, [3000, 40, 2000], 48, 16)
    n = pa.pa_latent_decode_workspace_size(b.S, b.H)
    for at in (16, 32, 48):
        buf = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device=DEV)
        b.check(b.run(ws=buf[at:at + n]))
        assert bool((buf[:at] == 0xA5).all()) and bool((buf[at + n:] == 0xA5).all())


def test_a_row_of_infinite_logits_stays_in_its_row():
    b = Batch(4, [100, 100], 16, 16)
    b.q[0, 3] = float("inf")
    out = b.run()
    clean = b.q.clone()
    clean[0, 3] = 0
    b.q = clean
    ref = b.run()
    keep = torch.ones(2, 16, dtype=torch.bool, device=DEV)
    keep[0, 3] = False
    assert torch.equal(out[keep], ref[keep])


@pytest.mark.parametrize("H", [1, 16, 40, 130])
def test_queries_of_the_next_sequence_stay_in_it(H):
    """A tile of 32 heads holds the rows that follow a sequence's last head: the next one's."""
    b = Batch(H, [70, 300, 33], H, 16)
    ref = b.run()
    b.check(ref)
    for bad in (float("nan"), float("inf"), -60000.0):
        q = b.q.clone()
        b.q[1] = bad
        out = b.run()
        assert torch.equal(out[0].view(torch.int16), ref[0].view(torch.int16))
        assert torch.equal(out[2].view(torch.int16), ref[2].view(torch.int16))
        b.q = q


def test_clipped_lengths_and_bad_blocks_are_reported():
    b = Batch(6, [200, 100, 50], 16, 16, width=0)
    bt, ctx = b.tensors()
    ws = pa.latent_decode_workspace(3, 16)
    out = torch.empty(3, 16, LAT, dtype=torch.float16, device=DEV)
    ctx[0], ctx[2] = 10 ** 6, -4
    b.bt[0, 12] = bt[0, 12] = b.bt[0, 0]               # its stale tail would be read: point it at live rows
    pa.pa_latent_decode(out, b.q, b.cache, bt, ctx, b.scale, 208, ws)
    assert pa.pa_check_errors()[1] == pa.PA_ERRBIT_CONTEXT
    b.ctx = [208, 100, 0]
    b.check(out)
    ctx[0], ctx[2] = 200, 50
    bt[1, 2] = b.NB                                    # a block id past the pool
    pa.pa_latent_decode(out, b.q, b.cache, bt, ctx, b.scale, 208, ws)
    assert pa.pa_check_errors()[1] == pa.PA_ERRBIT_BLOCK_ID
    b.ctx = [200, 100, 50]
    b.check(out, seqs=[0, 2])


def test_captured_and_replayed_with_new_lengths():
    b = Batch(12, [300, 41, 700], 64, 16)
    bt, ctx = b.tensors()
    ws, out = pa.latent_decode_workspace(3, 64), torch.empty(3, 64, LAT, dtype=torch.float16, device=DEV)
    g = torch.cuda.CUDAGraph()
    pa.pa_latent_decode(out, b.q, b.cache, bt, ctx, b.scale, 1000, ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pa.pa_latent_decode(out, b.q, b.cache, bt, ctx, b.scale, 1000, ws)
    for lens in ([300, 41, 700], [0, 40, 699], [5, 0, 0], [299, 41, 64]):
        b.ctx = lens
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        b.check(out)


def test_two_streams_with_a_workspace_each():
    a, b = Batch(13, [5000, 100], 128, 32), Batch(14, [333] * 20, 16, 16)
    ra, rb = a.run().clone(), b.run().clone()
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


def test_build_write_decode_step_in_one_graph():
    """A decode loop on the GPU: tables and slots from the lengths, the write of
    the new rows, the attention; each replay is one token of every sequence."""
    S, H, B, W = 5, 32, 16, 8
    NB = S * W
    g = gen(15)
    cache = torch.full((NB, B, ROW), float("nan"), dtype=torch.float16, device=DEV)
    tables = torch.full((S, W), -1, dtype=torch.int32, device=DEV)
    ctx = torch.zeros(S, dtype=torch.int32, device=DEV)
    nf = torch.tensor([NB], dtype=torch.int32, device=DEV)
    free = torch.randperm(NB, generator=g, device=DEV).int()
    new = torch.ones(S, dtype=torch.int32, device=DEV)
    qs, slots = torch.empty(S + 1, dtype=torch.int32, device=DEV), torch.empty(S, dtype=torch.int64, device=DEV)
    lat, rope, q = normal(g, S, LAT), normal(g, S, 64), normal(g, S, H, ROW)
    out = torch.empty(S, H, LAT, dtype=torch.float16, device=DEV)
    w1, w2 = pa.build_tables_workspace(S), pa.latent_decode_workspace(S, H)

    def step():
        pa.pa_build_tables(tables, ctx, qs, slots, nf, free, nf, ctx, new, B, NB, w1)
        pa.pa_latent_write(lat, rope, cache, slots)
        pa.pa_latent_decode(out, q, cache, tables, ctx, 0.07, W * B, w2)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    rows = []
    for n in range(1, 2 * B + 4):
        lat.copy_(normal(g, S, LAT))
        rope.copy_(normal(g, S, 64))
        rows.append(torch.cat([lat, rope], 1).double())
        graph.replay()
        torch.cuda.synchronize()
        k = torch.stack(rows, 1)                       # [S, n, ROW]
        w = torch.softmax(0.07 * (q.double() @ k.transpose(1, 2)), -1)
        ref = w @ k[:, :, :LAT]
        # 2^-11 twice for the weights, once for the output; fp32 logits of about 24 * 2^-23 * 576
        tol = 2 * (2.0 ** -11 + 0.07 * 600 * 576 * 2.0 ** -23 + 2.0 ** -20) * (w @ k[:, :, :LAT].abs()) + 2.0 ** -11 * ref.abs()
        assert ctx.tolist() == [n] * S
        assert ((out.double() - ref).abs() <= tol + 2.0 ** -24).all()
    assert pa.pa_check_errors()[1] == 0
