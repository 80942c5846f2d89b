"""CPU checks of the window-and-sinks, paged-chunk and quantised-cache entry points: refusals before
any launch, workspace sizes, and the fp64 oracle they are tested against.  No compute call is made."""
import ctypes

import numpy as np
import pytest

import oracle
import synthetic as syn
from oracle import chunk


@pytest.fixture(scope="module")
def attn():
    import __graft_entry__

    __graft_entry__._cuda_build_module().build()
    import exact_io_aware_09_gb300 as m

    return m


def _no_cuda():
    import torch

    return not torch.cuda.is_available()


FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: the calls below fail their checks
ODD = ctypes.c_void_p((1 << 20) + 8)
NUL = ctypes.c_void_p(0)


def test_window_sinks_refusals(attn):
    L = attn.lib

    def fwd(hq=4, hkv=2, d=64, w=10, s=4, scale=0.125, q=FAKE, dt=1, B=1):
        return L.attn_fwd_window_sinks(q, FAKE, FAKE, FAKE, FAKE, B, hq, hkv, 8, 8, d, w, s, scale,
                                       NUL, dt)

    def bwd(hq=4, hkv=2, d=64, w=10, s=4, ws=FAKE, n=1 << 30, q=FAKE, lse=FAKE):
        return L.attn_bwd_window_sinks(q, FAKE, FAKE, FAKE, FAKE, lse, FAKE, FAKE, FAKE, 1, hq, hkv,
                                       8, 8, d, w, s, 0.125, 1, ws, n, NUL)

    for f in (fwd, bwd):
        assert f(w=-1) == -1 and f(s=-1) == -1 and f(hq=3) == -1 and f(d=96) == -2
        assert f(q=NUL) == -1 and f(q=ODD) == -3
        if _no_cuda():
            assert f() == -7 and f(s=0) == -7
    assert fwd(scale=float("inf")) == -1 and fwd(dt=2) == -1 and fwd(B=0) == 0
    assert bwd(ws=NUL) in (-4, -7) and bwd(lse=ctypes.c_void_p((1 << 20) + 2)) == -3


def test_paged_refusals(attn):
    L = attn.lib

    def f(hq=16, hkv=2, d=128, page=16, pages=64, width=64, total=40, mq=20, mk=1024, w=-1, s=0,
          q=FAKE, table=FAKE, ws=FAKE, n=1 << 40, B=3, scale=0.1, dt=0):
        return L.attn_fwd_paged(q, FAKE, FAKE, table, FAKE, FAKE, pages, page, width, total, mq, mk,
                                FAKE, FAKE, B, hq, hkv, d, w, s, scale, dt, ws, n, NUL)

    assert f(hq=15) == -1 and f(w=-2) == -1 and f(s=-1) == -1 and f(scale=0.0) == -1
    assert f(mq=2000) == -1                       # chunk longer than the cache
    assert f(mk=1025) == -1                       # past the table's reach
    assert f(page=24) == -2 and f(page=8) == -2 and f(page=1 << 17, width=1) == -2
    assert f(pages=1 << 28) == -2                 # more than 2^31 - 1 rows
    assert f(d=80) == -2 and f(hq=129, hkv=1) == -2
    assert f(q=NUL) == -1 and f(pages=0) == -1 and f(q=ODD) == -3
    assert f(table=ctypes.c_void_p((1 << 20) + 2)) == -3
    assert f(dt=3) == -1
    assert f(B=0) == 0 and f(total=0) == 0 and f(mq=0) == 0
    long = dict(page=64, width=512, mk=32768)     # a few query tiles over many key tiles: split
    need = attn.attn_fwd_paged_workspace_bytes(40, 3, 16, 2, 20, 32768, 128)
    assert need > 0 and f(n=need - 1, **long) == -4 and f(ws=NUL, **long) == -4
    if _no_cuda():
        assert f(ws=NUL, n=0, mk=64) == -7 and f(n=need, **long) == -7  # (one step of keys: no split)


def test_paged_workspace(attn):
    ws = attn.attn_fwd_paged_workspace_bytes
    # whole prompts: enough query tiles, nothing to split
    assert ws(16 * 8192, 16, 64, 8, 8192, 8192, 128) == 0
    assert ws(1, 1, 64, 8, 1, 100, 128) == 0      # one key tile
    one = ws(1, 1, 64, 8, 1, 32768, 128)
    assert one > 0 and one % ((128 * 4 + 8) * 64) == 0
    # a window bounds the key tiles, whatever the cache's length
    assert ws(1, 1, 64, 8, 1, 1 << 20, 128, window=1000, sinks=4) <= one
    for bad in ((0, 1, 64, 8, 1, 100, 128), (1, 0, 64, 8, 1, 100, 128), (1, 1, 3, 2, 1, 9999, 128)):
        assert ws(*bad) == 0


def test_cache_refusals(attn):
    L = attn.lib

    def write(k=FAKE, codes=FAKE, page=16, pages=8, width=4, total=9, B=2, hkv=2, d=64, dt=1, cu=FAKE):
        return L.attn_cache_write_fp8(k, FAKE, codes, FAKE, FAKE, FAKE, FAKE, cu, FAKE, pages, page,
                                      width, total, B, hkv, d, dt, NUL)

    def read(k=FAKE, codes=FAKE, page=16, pages=8, width=4, total=9, B=2, hkv=2, d=64, dt=1, cu=FAKE):
        return L.attn_cache_read_fp8(codes, FAKE, FAKE, FAKE, FAKE, cu, pages, page, width, k, FAKE,
                                     total, B, hkv, d, dt, NUL)

    for f in (write, read):
        assert f(total=-1) == -1 and f(B=-1) == -1 and f(hkv=0) == -1 and f(dt=2) == -1
        assert f(page=20) == -2 and f(d=32) == -2 and f(pages=1 << 28) == -2
        assert f(k=NUL) == -1 and f(codes=NUL) == -1 and f(pages=0) == -1 and f(width=0) == -1
        assert f(k=ODD) == -3 and f(codes=ODD) == -3 and f(cu=ctypes.c_void_p((1 << 20) + 1)) == -3
        assert f(total=0) == 0 and f(B=0) == 0
        if _no_cuda():
            assert f() == -7

    def dec(hq=8, hkv=2, d=64, split=512, mk=64, B=2, ws=FAKE, n=1 << 30, codes=FAKE, page=16, width=4):
        return L.attn_decode_paged_fp8(FAKE, codes, FAKE, FAKE, FAKE, FAKE, FAKE, 8, page, width, mk,
                                       FAKE, FAKE, B, hq, hkv, d, split, 0.1, 1, ws, n, NUL)

    assert dec(hq=9) == -1 and dec(mk=65) == -1 and dec(d=96) == -2 and dec(split=100) == -2
    assert dec(hq=34) == -2 and dec(B=65536) == -2 and dec(page=48) == -2
    # nine splits go through the workspace, eight do not
    assert dec(ws=NUL, mk=513, split=64, width=64) == -4 and dec(n=8, mk=513, split=64, width=64) == -4
    assert attn.attn_decode_paged_fp8_workspace_bytes(2, 8, 2, 512, 64, 64) == 0
    assert attn.attn_decode_paged_fp8_workspace_bytes(2, 8, 2, 513, 64, 64) > 0
    assert dec(codes=NUL) == -1 and dec(codes=ODD) == -3
    assert dec(B=0) == 0
    if _no_cuda():
        assert dec() == -7


def test_tensors_off_the_gpu_are_refused(attn):
    import torch

    q = torch.zeros((1, 1, 8, 64), dtype=torch.bfloat16)
    lse = torch.zeros((1, 1, 8))
    with pytest.raises(attn.AttnError):
        attn.attn_fwd_window_sinks(q, q, q, 4, 1)
    with pytest.raises(attn.AttnError):
        attn.attn_bwd_window_sinks(q, q, q, q, q, lse, 4, 1)
    pool = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)
    with pytest.raises(attn.AttnError):
        attn.attn_fwd_paged(q[0, 0, :, None], pool, pool, i32(0)[None], i32(0, 8), i32(8), 8, 8)
    codes, sc = torch.zeros((2, 16, 1, 64), dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones((2, 1, 16))
    cache = (codes, codes, sc, sc)
    with pytest.raises(attn.AttnError):
        attn.attn_cache_write_fp8(q[0].transpose(0, 1), q[0].transpose(0, 1), *cache, i32(0)[None],
                                  i32(0, 8), i32(8))
    with pytest.raises(attn.AttnError):
        attn.attn_cache_read_fp8(*cache, i32(0)[None], i32(0, 8), 8)
    with pytest.raises(attn.AttnError):
        attn.attn_decode_paged_fp8(q[0].transpose(0, 1)[:1], *cache, i32(0)[None], i32(8), 8)


# ---------------------------------------------------------------------------- the oracle itself
@pytest.mark.parametrize("N_q,N_kv,W", [(50, 50, 7), (20, 90, 0), (60, 30, 12), (40, 40, -1)])
def test_chunk_oracle_is_the_windowed_definition(N_q, N_kv, W):
    """Without sinks: the materialising oracle's rows under the same window."""
    d, dt = 64, "f16"
    cfg = syn.PrefillConfig("c", 1, 1, 1, N_q, N_kv, d, dt, True, 3)
    q, k, v = cfg.host_inputs()
    o, lse = oracle.attention_rows(q, k, v, dt, 1, 1, 1, N_q, N_kv, d, True, cfg.scale,
                                   window=None if W < 0 else W)
    x = [oracle.bits_to_double(b, dt)[0, 0] for b in (q, k, v)]
    r = chunk.attend(*x, np.arange(N_q) + N_kv - N_q, cfg.scale, W)
    assert np.allclose(r.o, o, rtol=0, atol=1e-12)
    assert np.array_equal(np.isneginf(r.lse), np.isneginf(lse))
    live = np.isfinite(lse)
    assert np.allclose(r.lse[live], lse[live], rtol=0, atol=1e-12)


def test_chunk_oracle_sinks_by_hand():
    """Four keys, window 0, one sink: the last row sees keys 0 and 3."""
    q, k = np.zeros((1, 2)), np.zeros((4, 2))
    v = np.array([[1.0, 0], [100, 0], [100, 0], [5, 2]])
    r = chunk.attend(q, k, v, [3], 1.0, 0, 1)
    assert np.allclose(r.o, [[3.0, 1.0]]) and np.allclose(r.lse, np.log(2.0))
    # sinks count from the sequence's start and never lie ahead of the row
    assert chunk.visible([1], 4, 0, 9).tolist() == [[True, True, False, False]]


def test_quantise_oracle_against_torch():
    """The nearest-even E4M3 value by table search equals torch's conversion, the scale brings the
    largest magnitude into (224, 448]."""
    import torch

    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)) * np.exp2(rng.integers(-30, 30, (200, 1)))
    x = torch.from_numpy(x).bfloat16().double().numpy()
    s, c = chunk.quantise(x)
    assert np.array_equal(np.exp2(np.round(np.log2(s))), s)
    top = np.abs(x).max(axis=1) / s
    assert np.all(top <= 448) and np.all(top > 224)
    want = torch.from_numpy(x / s[:, None]).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(c, want)


def test_backward_oracle_with_sinks_against_differences():
    """The fp64 gradients under the window with sinks, by central differences of the definition."""
    from oracle.backward import attention_backward

    N, d, W, s, scale = 24, 64, 5, 3, 0.2
    cfg = syn.PrefillConfig("c", 1, 1, 1, N, N, d, "f16", True, 8)
    bits = cfg.host_inputs()
    do = syn.host_normal_bits((1, 1, N, d), 9, "f16")
    g = attention_backward(*bits, do, "f16", 1, 1, 1, N, N, d, True, scale, window=W, sinks=s,
                           exact_o=True)
    x = [oracle.bits_to_double(b, "f16")[0, 0] for b in bits]
    dod = oracle.bits_to_double(do, "f16")[0, 0]
    loss = lambda a: float((dod * chunk.attend(*a, np.arange(N), scale, W, s).o).sum())
    rng = np.random.default_rng(1)
    for i in range(3):
        u = rng.standard_normal((N, d))
        h = 1e-5
        up, dn = list(x), list(x)
        up[i], dn[i] = x[i] + h * u, x[i] - h * u
        assert abs((loss(up) - loss(dn)) / (2 * h) - float((g[i][0, 0] * u).sum())) < 1e-5
