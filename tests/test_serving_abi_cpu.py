"""Refusals of the table build, the shared-prefix decode and the latent cache's calls, on the host,
before any CUDA call."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "paged_kv_cache_158_gb300", "_lib", "libpa.so")
OK, INVALID, UNSUPPORTED = 0, 1, 2
vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
P = [0x10000 * (k + 1) for k in range(16)]   # distinct, aligned, never read


@pytest.fixture(scope="module")
def lib():
    x = ctypes.CDLL(LIB)
    x.pa_build_tables_workspace_size.restype = sz
    x.pa_latent_decode_workspace_size.restype = sz
    x.pa_build_tables.argtypes = [vp, i32, vp, vp, vp, i32, vp, vp, i32, vp, vp, vp, vp, vp, i32, i32,
                                  i32, i32, vp, sz, vp]
    x.pa_decode_shared_workspace_size.restype = sz
    x.pa_decode_shared.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, vp] + [i32] * 6 + [f32, i32, i32, vp, sz, vp]
    x.pa_decode_shared_fp8.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, vp] + [i32] * 6 + [f32, f32, f32, i32,
                                                                                      i32, vp, sz, vp]
    x.pa_latent_write.argtypes = [vp, i64, vp, i64, vp, vp, i32, i32, i32, i32, i32, vp]
    x.pa_latent_decode.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, f32, i32, vp,
                                   sz, vp]
    return x


TABLES = dict(block_tables=P[0], max_blocks=8, context=P[1], query_start=P[2], slots=P[3], num_slots=10,
              free_out=P[4], free_list=P[5], free_len=20, num_free=P[6], cached=P[7], new=P[8],
              group_start=P[9], prefix=P[10], groups=2, seqs=4, block_size=16, num_blocks=64, ws=P[11],
              ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(block_size=12), UNSUPPORTED), (dict(max_blocks=0), INVALID), (dict(num_slots=-1), INVALID),
    (dict(free_len=-1), INVALID), (dict(groups=-1), INVALID), (dict(seqs=-1), INVALID),
    (dict(num_blocks=0), INVALID), (dict(block_tables=None), INVALID), (dict(context=None), INVALID),
    (dict(query_start=None), INVALID), (dict(slots=None), INVALID), (dict(slots=P[3] + 4), INVALID),
    (dict(free_out=None), INVALID), (dict(free_list=None), INVALID), (dict(num_free=P[6] + 2), INVALID),
    (dict(cached=None), INVALID), (dict(new=P[8] + 1), INVALID), (dict(group_start=None), INVALID),
    (dict(prefix=None), INVALID), (dict(ws=None), INVALID), (dict(ws=P[11] + 8), INVALID),
    (dict(ws_bytes=64), INVALID), (dict(context=P[8]), INVALID), (dict(query_start=P[7]), INVALID),
    (dict(free_out=P[5]), INVALID), (dict(block_tables=P[5]), INVALID), (dict(context=P[2]), INVALID),
    (dict(slots=P[0]), INVALID), (dict(slots=P[8]), INVALID), (dict(free_out=P[1]), INVALID), (dict(seqs=1 << 20, max_blocks=1 << 12,
                                                                              ws_bytes=1 << 30), UNSUPPORTED),
])
def test_build_tables_refusals(lib, change, status):
    assert lib.pa_build_tables(*dict(TABLES, **change).values()) == status


DECODE = dict(out=P[0], q=P[1], cache=P[2], bt=P[3], max_blocks=4, ctx=P[4], seqs=2, heads=16, lat=512,
              rope=64, block_size=16, num_blocks=8, scale=0.1, max_len=64, ws=P[5], ws_bytes=1 << 30,
              stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(lat=256), UNSUPPORTED), (dict(rope=32), UNSUPPORTED), (dict(block_size=4), UNSUPPORTED),
    (dict(block_size=64), UNSUPPORTED), (dict(heads=0), INVALID), (dict(heads=1025), UNSUPPORTED),
    (dict(seqs=-1), INVALID), (dict(num_blocks=0), INVALID), (dict(max_blocks=0), INVALID),
    (dict(max_len=-1), INVALID), (dict(out=None), INVALID), (dict(q=P[1] + 8), INVALID),
    (dict(cache=P[2] + 2), INVALID), (dict(bt=P[3] + 2), INVALID), (dict(ws=None), INVALID),
    (dict(ws_bytes=1000), INVALID), (dict(num_blocks=1 << 28), UNSUPPORTED),
    (dict(seqs=1024, max_blocks=1 << 27, max_len=2 ** 31 - 1), UNSUPPORTED), (dict(seqs=0, out=None), OK),
])
def test_latent_decode_refusals(lib, change, status):
    assert lib.pa_latent_decode(*dict(DECODE, **change).values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(lat=448), UNSUPPORTED), (dict(rope=72), UNSUPPORTED), (dict(block_size=24), UNSUPPORTED),
    (dict(tokens=-1), INVALID), (dict(num_blocks=0), INVALID), (dict(latent=None), INVALID),
    (dict(rope_p=P[1] + 8), INVALID), (dict(slots=P[3] + 4), INVALID), (dict(ls=504), INVALID),
    (dict(ls=513), INVALID), (dict(rs=60), INVALID), (dict(tokens=0, latent=None), OK),
])
def test_latent_write_refusals(lib, change, status):
    a = dict(latent=P[0], ls=512, rope_p=P[1], rs=64, cache=P[2], slots=P[3], tokens=3, lat=512, rope=64,
             block_size=16, num_blocks=8, stream=None)
    assert lib.pa_latent_write(*dict(a, **change).values()) == status


SHARED = dict(out=P[0], q=P[1], k=P[2], v=P[3], bt=P[4], max_blocks=8, ctx=P[5], starts=P[6], pre=P[7],
              groups=2, seqs=4, heads=8, D=128, block_size=16, num_blocks=64, scale=0.1)
SHARED_TAIL = dict(max_len=100, max_prefix=32, ws=P[8], ws_bytes=1 << 34, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(D=96), UNSUPPORTED), (dict(block_size=64), UNSUPPORTED), (dict(groups=-1), INVALID),
    (dict(groups=5), INVALID), (dict(seqs=-1), INVALID), (dict(heads=0), INVALID), (dict(num_blocks=0), INVALID),
    (dict(max_blocks=0), INVALID), (dict(max_len=-1), INVALID), (dict(max_prefix=-1), INVALID),
    (dict(out=None), INVALID), (dict(q=P[1] + 8), INVALID), (dict(k=None), INVALID), (dict(v=P[3] + 2), INVALID),
    (dict(bt=P[4] + 1), INVALID), (dict(ctx=None), INVALID), (dict(starts=None), INVALID),
    (dict(pre=P[7] + 2), INVALID), (dict(ws=None), INVALID), (dict(ws=P[8] + 8), INVALID),
    (dict(ws_bytes=1 << 10), INVALID), (dict(num_blocks=1 << 24), UNSUPPORTED),
    (dict(max_prefix=2 ** 31 - 1, heads=128), UNSUPPORTED),
    (dict(max_prefix=600_000_000, heads=128), UNSUPPORTED),   # 2^31 tiles of 64 tokens (dict(seqs=0, out=None), OK),
])
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_shared_refusals(lib, fp8, change, status):
    a = {k: change.get(k, v) for k, v in SHARED.items()}
    b = {k: change.get(k, v) for k, v in SHARED_TAIL.items()}
    if fp8:
        assert lib.pa_decode_shared_fp8(*a.values(), 0.5, 0.25, *b.values()) == status
        if status == OK:
            for ks, vs in ((0.0, 1.0), (1.0, -1.0), (float("inf"), 1.0), (1.0, float("nan"))):
                assert lib.pa_decode_shared_fp8(*a.values(), ks, vs, *b.values()) == INVALID
    else:
        assert lib.pa_decode_shared(*a.values(), *b.values()) == status


def test_workspace_sizes(lib):
    size = lib.pa_decode_shared_workspace_size
    assert size(4, 1, 8, 128, 100, 32) > 0 == size(4, 1, 8, 96, 100, 32)
    assert size(-1, 1, 8, 128, 100, 32) == size(4, 1, 0, 128, 100, 32) == size(4, 1, 8, 128, -1, 32) == 0
    # the prefix's partial rows: one for each (sequence, head), 128 more for each SM
    assert size(64, 1, 32, 128, 2048, 512) >= (64 * 32 + 152 * 128) * 128 * 4
    assert lib.pa_build_tables_workspace_size(-1) == 0 and lib.pa_build_tables_workspace_size(0) > 0
    assert lib.pa_build_tables_workspace_size(100) >= 100 * 20
    assert lib.pa_latent_decode_workspace_size(-1, 16) == 0 == lib.pa_latent_decode_workspace_size(4, 0)
    assert lib.pa_latent_decode_workspace_size(4, 128) >= (4 + 70) * 128 * 512 * 4
