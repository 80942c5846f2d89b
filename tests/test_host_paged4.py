"""CPU checks of the page lists and of the 4-bit cache: refusals before any launch, workspace sizes, and the
oracle that the GPU tests use.  No compute call is made."""
import ctypes
import itertools

import numpy as np
import pytest

from oracle import paged4


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
ODD2 = ctypes.c_void_p((1 << 20) + 2)
NUL = ctypes.c_void_p(0)


def test_pages_refusals(attn):
    L = attn.lib

    def extend(table=FAKE, lens=FAKE, cu=FAKE, free=FAKE, n=FAKE, slots=FAKE, pages=8, page=16, width=4,
               total=9, B=2):
        return L.attn_pages_extend(table, lens, cu, free, n, slots, pages, page, width, total, B, NUL)

    def trim(table=FAKE, lens=FAKE, cu=FAKE, free=FAKE, n=FAKE, pages=8, page=16, width=4, B=2):
        return L.attn_pages_trim(table, lens, cu, free, n, pages, page, width, B, NUL)

    for f in (extend, trim):
        assert f(B=-1) == -1 and f(pages=-1) == -1 and f(pages=0) == -1 and f(width=0) == -1
        assert f(page=24) == -2 and f(page=8) == -2 and f(page=1 << 17) == -2 and f(pages=1 << 28) == -2
        assert f(width=(1 << 26) + 1) == -2            # a table that reaches past 2^30 tokens
        for name in ("table", "lens", "cu", "free", "n"):
            assert f(**{name: NUL}) == -1 and f(**{name: ODD2}) == -3
        if _no_cuda():
            assert f() == -7
    assert extend(total=-1) == -1 and extend(slots=NUL) == -1 and extend(slots=ODD) == -3
    assert extend(B=0, total=0) == 0 and trim(B=0) == 0
    if _no_cuda():
        assert extend(total=0, slots=NUL) == -7 and extend(B=0, table=NUL) == -7


def test_cache_refusals(attn):
    L = attn.lib

    def write(k=FAKE, codes=FAKE, scales=FAKE, slots=FAKE, page=16, pages=8, total=9, hkv=2, d=64, dt=1):
        return L.attn_cache_write_fp4(k, FAKE, codes, FAKE, scales, FAKE, slots, pages, page, total, hkv, d,
                                      dt, NUL)

    def read(k=FAKE, codes=FAKE, scales=FAKE, slots=FAKE, page=16, pages=8, total=9, hkv=2, d=64, dt=1,
             width=4, B=2, starts=FAKE):
        return L.attn_cache_read_fp4(codes, FAKE, scales, FAKE, slots, FAKE, starts, pages, page, width, k,
                                     FAKE, total, B, hkv, d, dt, NUL)

    for f in (write, read):
        assert f(total=-1) == -1 and f(hkv=0) == -1 and f(dt=2) == -1 and f(dt=-1) == -1
        assert f(page=20) == -2 and f(d=32) == -2 and f(d=96) == -2 and f(pages=1 << 28) == -2
        assert f(k=NUL) == -1 and f(codes=NUL) == -1 and f(scales=NUL) == -1 and f(slots=NUL) == -1
        assert f(pages=0) == -1
        assert f(k=ODD) == -3 and f(codes=ODD) == -3 and f(scales=ODD) == -3 and f(slots=ODD2) == -3
        assert f(total=0) == 0
        if _no_cuda():
            assert f() == -7
    assert read(B=-1) == -1 and read(B=0) == 0 and read(width=0) == -1 and read(starts=ODD2) == -3
    if _no_cuda():
        assert read(starts=NUL) == -7


def test_attention_refusals(attn):
    L = attn.lib

    def fwd(hq=16, hkv=2, d=128, page=16, pages=64, width=64, total=40, mq=20, mk=1024, w=-1, s=0, q=FAKE,
            codes=FAKE, scales=FAKE, table=FAKE, cu=FAKE, ws=FAKE, n=1 << 40, B=3, scale=0.1, dt=0, lse=FAKE):
        return L.attn_fwd_paged_fp4(q, codes, FAKE, scales, FAKE, table, cu, FAKE, pages, page, width, total,
                                    mq, mk, FAKE, lse, B, hq, hkv, d, w, s, scale, dt, ws, n, NUL)

    def dec(hq=16, hkv=2, d=128, page=16, pages=64, width=64, mk=1024, q=FAKE, codes=FAKE, scales=FAKE,
            table=FAKE, ws=FAKE, n=1 << 40, B=3, scale=0.1, dt=0, lse=FAKE):
        return L.attn_decode_paged_fp4(q, codes, FAKE, scales, FAKE, table, FAKE, pages, page, width, mk,
                                       FAKE, lse, B, hq, hkv, d, scale, dt, ws, n, NUL)

    for f in (fwd, dec):
        assert f(hq=15) == -1 and f(hkv=0) == -1 and f(B=-1) == -1 and f(mk=-1) == -1
        assert f(scale=0.0) == -1 and f(scale=float("inf")) == -1 and f(scale=float("nan")) == -1
        assert f(dt=3) == -1 and f(mk=1025) == -1          # past the table's reach
        assert f(page=24) == -2 and f(page=8) == -2 and f(pages=1 << 28) == -2
        assert f(d=80) == -2 and f(B=65536) == -2 and f(hq=65536, hkv=65536) == -2
        assert f(q=NUL) == -1 and f(codes=NUL) == -1 and f(scales=NUL) == -1 and f(table=NUL) == -1
        assert f(pages=0) == -1
        assert f(q=ODD) == -3 and f(codes=ODD) == -3 and f(scales=ODD) == -3 and f(ws=ODD) == -3
        assert f(table=ODD2) == -3 and f(lse=ODD2) == -3
        assert f(B=0) == 0
        if _no_cuda():
            assert f() == -7
    assert fwd(w=-2) == -1 and fwd(s=-1) == -1 and fwd(mq=2000) == -1 and fwd(cu=NUL) == -1
    assert fwd(hq=129, hkv=1) == -2 and dec(hq=17, hkv=1) == -2
    assert fwd(total=0) == 0 and fwd(mq=0) == 0
    long = dict(page=64, width=512, mk=32768, pages=1024)
    for f, need in ((fwd, attn.attn_fwd_paged_fp4_workspace_bytes(40, 3, 16, 2, 20, 32768, 128)),
                    (dec, attn.attn_decode_paged_fp4_workspace_bytes(3, 16, 2, 32768, 128))):
        assert need > 0 and f(n=need - 1, **long) == -4 and f(ws=NUL, **long) == -4
        if _no_cuda():
            assert f(n=need, **long) == -7 and f(ws=NUL, n=0, mk=64, **({"mq": 8} if f is fwd else {})) == -7


def test_workspaces(attn):
    fwd, dec = attn.attn_fwd_paged_fp4_workspace_bytes, attn.attn_decode_paged_fp4_workspace_bytes
    assert dec(1, 64, 8, 100, 128) == 0                        # one split
    assert dec(2, 16, 2, 1024, 64) == 0 < dec(2, 16, 2, 1025, 64)   # eight merge in a cluster
    assert dec(1, 64, 8, 32768, 128) == fwd(1, 1, 64, 8, 1, 32768, 128)
    # chunks of eight query tiles on copy the cache: K and V in 16 bits, to whole steps of 64 keys
    copy = 2 * 8192 * 8 * 128 * 2 * 2
    assert fwd(2 * 128, 2, 64, 8, 112, 8190, 128) < copy <= fwd(2 * 128, 2, 64, 8, 113, 8190, 128)
    # ... but not one of more than a gigabyte
    assert fwd(64 * 256, 64, 64, 8, 256, 32768, 128) < 1 << 30
    # a window bounds the keys of few rows, whatever the cache's length
    assert fwd(1, 1, 64, 8, 1, 1 << 20, 128, window=1000, sinks=4) <= dec(1, 64, 8, 32768, 128)
    for bad in ((0, 1, 64, 8, 1, 100, 128), (1, 0, 64, 8, 1, 100, 128), (1, 1, 3, 2, 1, 9999, 128),
                (1, 1, 129, 1, 1, 9999, 128)):
        assert fwd(*bad) == 0
    assert dec(0, 64, 8, 9999, 128) == 0 and dec(1, 9, 2, 9999, 128) == 0


def test_python_refusals(attn):
    """Shapes and types that the binding itself refuses, on CPU tensors (a call that passes these checks
    is refused for not being on a GPU)."""
    import torch

    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    u = lambda *s: torch.zeros(s, dtype=torch.uint8)
    h = lambda *s: torch.zeros(s, dtype=torch.float16)
    cache = lambda d=64, P=16: (u(3, 2, P, d // 2), u(3, 2, P, d // 2), u(3, 2, P, d // 16), u(3, 2, P, d // 16))
    c = cache()
    calls = {
        "extend": (attn.attn_pages_extend, [i(2, 4), i(2), i(3), i(8), i(1), 16, 5]),
        "trim": (attn.attn_pages_trim, [i(2, 4), i(2), i(2), i(8), i(1), 16]),
        "write": (attn.attn_cache_write_fp4, [h(5, 2, 64), h(5, 2, 64), *c, i(5)]),
        "read": (attn.attn_cache_read_fp4, [*c, i(2, 4), i(3), 5]),
        "decode": (attn.attn_decode_paged_fp4, [h(2, 4, 64), *c, i(2, 4), i(2), 40]),
        "chunk": (attn.attn_fwd_paged_fp4, [h(5, 4, 64), *c, i(2, 4), i(3), i(2), 4, 40]),
    }
    wrong = {
        "extend": {0: i(2, 4).long(), 1: i(3), 2: i(2), 3: i(8, 1), 4: i(2), 6: -1},
        "trim": {0: i(8), 1: i(3), 2: i(3), 3: i(8).long(), 4: i(0)},
        "write": {0: h(5, 3, 64), 1: h(4, 2, 64), 2: u(3, 2, 16, 64), 3: h(3, 2, 16, 32), 4: u(3, 2, 16, 8),
                  6: i(6)},
        "read": {0: u(3, 2, 32), 3: u(3, 2, 16, 4).int(), 4: i(3, 4), 5: i(3).long()},
        "decode": {0: h(2, 4, 128), 1: cache(128)[0], 5: i(3, 4), 6: i(2).long()},
        "chunk": {0: h(5, 4, 128), 4: cache(128)[3], 5: i(2), 6: i(4), 7: i(3)},
    }
    for name, (f, args) in calls.items():
        for at, bad in itertools.chain([(None, None)], wrong[name].items()):
            a = list(args)
            if at is not None:
                a[at] = bad
            with pytest.raises(attn.AttnError):
                f(*a)
    out = [h(2, 4, 64).bfloat16(), h(2, 4, 64)]
    for kw in (dict(o=out[0]), dict(lse=torch.zeros(2, 5)), dict(lse=torch.zeros(2, 4).double())):
        with pytest.raises(attn.AttnError):
            attn.attn_decode_paged_fp4(*calls["decode"][1], **kw)
    with pytest.raises(attn.AttnError):
        attn.attn_pages_extend(*calls["extend"][1], slots=i(4))
    with pytest.raises(attn.AttnError):
        attn.attn_cache_read_fp4(*calls["read"][1], starts=i(3))


def test_scale_type():
    """The scale bytes are fp16's bits shifted right by seven, in ascending order; the largest is 10240."""
    bits = (np.arange(len(paged4.E5M3), dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(bits, paged4.E5M3) and np.all(np.diff(paged4.E5M3) > 0)
    assert paged4.E5M3[paged4.MAX_SCALE] == 10240.0 and 6 * 10240.0 <= 65504 < 6 * paged4.E5M3[paged4.MAX_SCALE + 1]
    # every product of a code and a scale is exact in fp16 and in bf16
    import torch

    v = torch.from_numpy(np.outer(paged4.E5M3[:paged4.MAX_SCALE + 1], paged4.E2M1))
    assert torch.equal(v.half().double(), v) and torch.equal(v.bfloat16().double(), v)


@pytest.mark.parametrize("scale", [1.0, 1e-4, 3e-6, 2e4, 1e6])
def test_quantise(scale):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 64)).astype(np.float16 if scale < 1e4 else np.float32).astype(np.float64) * scale
    x[3] = 0.0
    x[4, 16:32] = 0.0
    codes, scales, val = paged4.quantise(x)
    assert codes.shape == (50, 32) and scales.shape == (50, 4)
    assert np.array_equal(paged4.values(codes, scales), val)
    f = np.repeat(paged4.E5M3[scales], 16, axis=1)
    inside = np.abs(x) <= 6 * f
    # within half the gap between codes (1 at 3 and below, 2 above; 1/2 in the lowest), in scales
    gap = np.where(np.abs(x) <= 2 * f, 0.5, np.where(np.abs(x) <= 4 * f, 1.0, 2.0)) * f
    assert np.all(np.abs(x - val)[inside] <= gap[inside] / 2)
    assert np.all((np.abs(val) == 6 * f)[~inside])
    # no other scale byte is nearer to a sixth of the largest magnitude
    a = np.abs(x).reshape(50, 4, 16).max(-1) / 6
    err = np.abs(paged4.E5M3[None, None, 1:paged4.MAX_SCALE + 1] - a[..., None]).min(-1)
    assert np.all(np.abs(paged4.E5M3[scales] - a)[a > 0] <= err[a > 0])
    assert np.all(scales[a == 0] == 0) and np.all(scales[a > 0] > 0)


def test_quantise_what_is_not_finite():
    x = np.ones((3, 32))
    x[0, 5], x[1, 20], x[2, 31] = np.nan, np.inf, -np.inf
    codes, scales, val = paged4.quantise(x)
    assert (scales == paged4.NAN_SCALE).sum() == 3 and np.isnan(val).sum() == 48
    assert np.array_equal(np.isnan(paged4.values(codes, scales)), np.isnan(val))


def test_lists():
    a = paged4.Lists(2, [5, 3, 9, 1], 16)
    assert a.extend([17, 0]) == [1 * 16 + i for i in range(16)] + [9 * 16]
    assert a.free == [5, 3] and a.extend([15, 16]) == [9 * 16 + i for i in range(1, 16)] + [3 * 16 + i for i in range(16)]
    assert a.extend([1, 17]) is None and a.len == [32, 16]
    a.trim([17, 0])
    assert a.free == [5, 3] and a.len == [17, 0]
    a.trim([16, 0])
    assert a.free == [5, 3, 9]


def test_plain_forms_agree_with_the_oracle():
    """The quantiser and the pages of the measured cases' plain forms, on the CPU."""
    import torch

    import perf.more_operators as m

    x = np.random.default_rng(1).standard_normal((40, 3, 128)) * 2.0 ** np.arange(-20, 20)[:, None, None]
    x = torch.from_numpy(x).bfloat16()
    codes, scales = m._split4(x)
    want = paged4.quantise(x.double().numpy())
    assert np.array_equal(codes.numpy(), want[0]) and np.array_equal(scales.numpy(), want[1])
    assert np.array_equal(m._join4(codes, scales).double().numpy(), want[2])
    assert torch.equal(m._rounded64(x), torch.from_numpy(want[2]))


def test_rows_without_a_bound_hide_no_other():
    """A row of huge scores, whose bound is infinite, leaves the other rows checked, and a bound that is not a
    number is refused."""
    from oracle import chunk

    rng = np.random.default_rng(5)
    q, k, v = (rng.standard_normal((n, 16)) for n in (4, 50, 50))
    q[2] *= 2.0 ** 80
    rows = chunk.attend(q, k, v, np.arange(46, 50), 0.25)
    tol = chunk.row_tolerance(rows, 2.0 ** -10, 2.0 ** -7, 2.0 ** -31)
    assert not np.isnan(tol[0]).any() and np.isinf(tol[0][2]).all() and np.isfinite(np.delete(tol[0], 2, 0)).all()
    chunk.check(rows.o, rows.lse, rows, tol)
    for row in (0, 1, 3):
        wrong = rows.o.copy()
        wrong[row, 3] += 0.1
        with pytest.raises(AssertionError, match="times the tolerance"):
            chunk.check(wrong, rows.lse, rows, tol)
    bad = tol[0].copy()
    bad[1, 1] = np.nan
    with pytest.raises(AssertionError, match="not a number"):
        chunk.check(rows.o, rows.lse, rows, (bad, tol[1]))


def test_an_infinite_bound_of_no_weight():
    """Infinity times a sum that is zero is no bound: it stays infinite."""
    from oracle import chunk

    rows = chunk.Rows(np.zeros((1, 2)), np.zeros(1), np.array([[0.0, 1.0]]), np.ones((1, 2)),
                      np.array([1e30]), np.ones(1))
    assert np.isposinf(chunk.row_tolerance(rows, 2.0 ** -10, 2.0 ** -7, 2.0 ** -31)[0]).all()


def test_pages_of_too_many_sequences(attn):
    """Sequences are numbered by 32 bits with room for a pass of the kernel behind the last."""
    for B in ((1 << 30) + 1, (1 << 31) - 1):
        assert attn.lib.attn_pages_extend(*[FAKE] * 6, 8, 16, 4, 9, B, NUL) == -2
        assert attn.lib.attn_pages_trim(*[FAKE] * 5, 8, 16, 4, B, NUL) == -2


@pytest.mark.parametrize("B,Hkv,max_k", [(43940, 31337, 52331392), (56806, 32749, 38733568), (36513, 20011, 98619648),
                                         (32768, 2048, 1 << 30)])
def test_no_copy_whose_size_passes_64_bits(attn, B, Hkv, max_k):
    """A chunk of eight query tiles whose f16 copy would be more bytes than 2^64, and little more: it goes by
    the codes, with the workspace of the 16-bit cache's call (none)."""
    rows = -(-max_k // 64) * 64
    assert B * Hkv * rows * 64 * 4 >= 1 << 64 and B * Hkv * rows * 64 * 4 % (1 << 64) <= 1 << 30
    args = (1024, B, Hkv, Hkv, 1024, max_k, 64)
    assert attn.attn_fwd_paged_workspace_bytes(*args) == 0
    assert attn.attn_fwd_paged_fp4_workspace_bytes(*args) == 0
