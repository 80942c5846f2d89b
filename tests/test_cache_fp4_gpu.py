"""GPU parity of writing and reading the 4-bit paged cache: codes, scale bytes and values exactly as
the fp64 definition gives them (every rounding of the format is to the nearest of a grid)."""
import numpy as np
import pytest

import synthetic as syn
from oracle import bits_to_double, paged4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    import exact_io_aware_09_gb300 as m

    return m


def empty_cache(n_pages, Hkv, page, d):
    """Codes and scales of bytes that no test's values give: (k codes, v codes, k scales, v scales)."""
    import torch

    full = lambda last: torch.full((n_pages, Hkv, page, last), 0xA5, dtype=torch.uint8, device="cuda")
    return full(d // 2), full(d // 2), full(d // 16), full(d // 16)


def dev(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def place(cache_part, slots, page):
    """[tokens, Hkv, bytes] of the pool rows at slots."""
    x = cache_part.cpu().numpy()
    return x[slots // page, :, slots % page]


def bits_of(x, dt):
    """The 16-bit numbers nearest to float64 x (as uint16)."""
    import torch

    t = torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.float16 if dt == "f16" else torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16)


def check_written(attn, bits_k, bits_v, dt, page, n_pages, slots, Hkv, d):
    """Writes the rows and compares the whole pools; returns the cache."""
    cache = empty_cache(n_pages, Hkv, page, d)
    attn.attn_cache_write_fp4(syn.bits_to_tensor(bits_k, dt, "cuda"), syn.bits_to_tensor(bits_v, dt, "cuda"),
                              *cache, dev(slots.astype(np.int32)))
    assert attn.attn_poll_status() == 0
    kept = slots >= 0
    for i, bits in enumerate((bits_k, bits_v)):
        codes, scales, _ = paged4.quantise(bits_to_double(bits[kept], dt))
        for got, want in ((cache[i], codes), (cache[2 + i], scales)):
            full = np.full(got.shape, 0xA5, dtype=np.uint8)
            full[slots[kept] // page, :, slots[kept] % page] = want
            assert np.array_equal(got.cpu().numpy(), full)
    return cache


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d,Hkv,page,total", [(64, 1, 16, 1), (128, 1, 16, 2), (128, 3, 16, 77), (64, 8, 64, 130),
                                              (128, 8, 256, 3000), (64, 5, 32, 1217 * 2 + 5)])
def test_write(attn, dt, d, Hkv, page, total):
    n_pages = -(-total // page) + 3
    slots = np.random.default_rng(total).permutation(n_pages * page)[:total]
    slots[total // 2:: 7] = -1                    # tokens that are not kept
    k = syn.host_normal_bits((total, Hkv, d), 5, dt)
    v = syn.host_normal_bits((total, Hkv, d), 6, dt)
    check_written(attn, k, v, dt, page, n_pages, slots, Hkv, d)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_every_magnitude_and_every_half(attn, dt):
    """Blocks of every size the type has, and values half way between two codes or two scales."""
    rng = np.random.default_rng(8)
    rows = []
    lo, hi = (-24, 15) if dt == "f16" else (-130, 127)
    for e in range(lo, hi + 1):
        rows.append(rng.normal(size=64) * 2.0 ** e)
        rows.append(rng.integers(-7, 8, size=64) * 2.0 ** e)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    for by in list(range(1, 40, 3)) + [90, 101, 119, 120, 127, 200, paged4.MAX_SCALE - 1, paged4.MAX_SCALE]:
        f = paged4.E5M3[by]
        for sign in (1.0, -1.0):
            x = np.zeros(64)
            for b in range(4):                    # the largest value 6 f keeps the scale at f
                x[16 * b:16 * b + 7] = sign * mids * f
                x[16 * b + 7:16 * b + 14] = sign * mids * f * (1 + 2.0 ** -7)
                x[16 * b + 15] = 6 * f
            rows.append(x)
        half = 3 * (f + paged4.E5M3[min(by + 1, len(paged4.E5M3) - 1)])  # amax / 6 between two scales
        rows.append(np.where(np.arange(64) % 16 == 3, half, 0.1 * half))
    rows += [np.zeros(64), -np.zeros(64), np.where(np.arange(64) == 40, -1.0, 0.0)]
    x = np.array(rows)
    x = np.where(np.abs(x) > (65504 if dt == "f16" else 3e38), 0.0, x)
    bits = bits_of(x, dt)[:, None, :]
    total = len(bits)
    check_written(attn, bits, np.roll(bits, 1, axis=0), dt, 16, -(-total // 16), np.arange(total), 1, 64)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_values_that_are_not_finite(attn, dt):
    x = np.random.default_rng(2).normal(size=(6, 2, 128))
    x[0, 0, 3], x[1, 1, 127], x[2, 0, 16] = np.nan, np.inf, -np.inf
    x[3, 0, :] = np.nan
    bits = bits_of(x, dt)
    cache = check_written(attn, bits, bits[::-1].copy(), dt, 16, 1, np.arange(6), 2, 128)
    got = read(attn, cache, [[0]], [6], dt)
    want = paged4.quantise(bits_to_double(bits, dt))[2]
    assert np.isnan(want).sum() == (3 + 8) * 16
    assert np.array_equal(got[0], want, equal_nan=True)
    assert np.array_equal(got[1], want[::-1], equal_nan=True)


def read(attn, cache, table, lengths, dt, starts=None, **kw):
    import torch

    cu = syn.cu_seqlens(lengths)
    k, v = attn.attn_cache_read_fp4(*cache, dev(np.asarray(table, dtype=np.int32)), dev(cu), int(cu[-1]),
                                    starts=None if starts is None else dev(np.asarray(starts, dtype=np.int32)),
                                    dtype=torch.float16 if dt == "f16" else torch.bfloat16, **kw)
    assert attn.attn_poll_status() == 0
    return k.double().cpu().numpy(), v.double().cpu().numpy()


def random_cache(n_pages, Hkv, page, d, seed):
    """Any codes, any scale bytes that a writer gives."""
    g = np.random.default_rng(seed)
    codes = [g.integers(0, 256, size=(n_pages, Hkv, page, d // 2), dtype=np.uint8) for _ in range(2)]
    scales = [g.integers(0, paged4.MAX_SCALE + 1, size=(n_pages, Hkv, page, d // 16)).astype(np.uint8)
              for _ in range(2)]
    return codes + scales


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d,Hkv,page,lengths", [(64, 2, 16, (1,)), (128, 8, 16, (1001, 0, 16, 17)),
                                                (64, 3, 64, (63, 64, 65, 640)),
                                                (128, 1, 128, (2000, 300, 1)), (128, 8, 32, (3001, 999))])
@pytest.mark.parametrize("from_start", [True, False])
def test_read(attn, dt, d, Hkv, page, lengths, from_start):
    table, n_pages, pg, sl = syn.paged_layout(list(lengths), page, seed=3)
    host = random_cache(n_pages, Hkv, page, d, seed=d + page)
    starts = None if from_start else [n // 3 for n in lengths]
    want_n = [n - (0 if from_start else n // 3) for n in lengths]
    got = read(attn, [dev(x) for x in host], table, want_n, dt, starts)
    cu = syn.cu_seqlens(lengths)
    keep = np.concatenate([np.arange(cu[b + 1] - w, cu[b + 1]) for b, w in enumerate(want_n)]).astype(np.int64)
    for i in range(2):
        want = paged4.values(host[i][pg, :, sl], host[2 + i][pg, :, sl])[keep]
        assert np.array_equal(got[i], want)


def test_every_code_and_scale(attn):
    """All 256 code bytes under every scale byte a writer gives, in both types."""
    n = paged4.MAX_SCALE + 1
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(1, 4, 1, 64), (n, 1, 16, 1))
    scales = np.broadcast_to(np.arange(n, dtype=np.uint8)[:, None, None, None], (n, 4, 16, 8)).copy()
    cache = [dev(x) for x in (codes, codes, scales, scales)]
    want = paged4.values(codes[:, :, 0], scales[:, :, 0])
    for dt in ("bf16", "f16"):
        k, v = read(attn, cache, np.arange(n)[:, None], [1] * n, dt)
        assert np.array_equal(k, want) and np.array_equal(v, want)


def test_rows_outside_the_sequences_stay(attn):
    import torch

    host = random_cache(4, 2, 16, 64, seed=1)
    cache = [dev(x) for x in host]
    out = [torch.full((30, 2, 64), 7.5, dtype=torch.float16, device="cuda") for _ in range(2)]
    cu = dev(np.array([4, 10, 25], dtype=np.int32))
    attn.attn_cache_read_fp4(*cache, dev(np.array([[2], [1]], dtype=np.int32)), cu, 30, k=out[0], v=out[1])
    assert attn.attn_poll_status() == 0
    for i, x in enumerate(out):
        x = x.double().cpu().numpy()
        assert (x[:4] == 7.5).all() and (x[25:] == 7.5).all()
        assert np.array_equal(x[4:10], paged4.values(host[i][2, :, :6], host[2 + i][2, :, :6]).swapaxes(0, 1))
        assert np.array_equal(x[10:25], paged4.values(host[i][1, :, :15], host[2 + i][1, :, :15]).swapaxes(0, 1))


def test_bad_slots_and_pages(attn):
    import torch

    k = syn.bits_to_tensor(syn.host_normal_bits((5, 2, 64), 1, "f16"), "f16", "cuda")
    cache = empty_cache(4, 2, 16, 64)
    attn.attn_cache_write_fp4(k, k, *cache, dev(np.array([64, -2, 2147483647, -2147483648, 3], dtype=np.int32)))
    assert attn.attn_poll_status() == -8
    touched = (cache[0] != 0xA5).any(-1).any(1).nonzero().tolist()
    assert touched == [[0, 3]]
    out = torch.full((40, 2, 64), 7.5, dtype=torch.float16, device="cuda")
    cu = dev(np.array([0, 10, 20, 30, 40], dtype=np.int32))
    table = dev(np.array([[0], [4], [-1], [1]], dtype=np.int32))
    attn.attn_cache_read_fp4(*cache, table, cu, 40, starts=dev(np.array([0, 0, 0, 10], dtype=np.int32)), k=out,
                             v=out.clone())
    assert attn.attn_poll_status() == -8
    same = (out == 7.5).all(-1).all(-1).cpu().numpy()
    assert not same[:10].any() and same[10:30].all() and not same[30:36].any() and same[36:].all()
    attn.attn_cache_read_fp4(*cache, table, cu, 40, starts=dev(np.array([-1, 0, 0, 0x7fffffff], dtype=np.int32)))
    assert attn.attn_poll_status() == -8


def test_a_pool_past_32_bit_offsets(attn):
    """Pools whose byte offsets and row numbers pass 2^32: the last page is written and read."""
    import torch

    Hkv, page, d = 8, 256, 128
    n_pages = (1 << 32) // (Hkv * page * (d // 2)) + 3
    cache = [torch.empty((n_pages, Hkv, page, w), dtype=torch.uint8, device="cuda")
             for w in (d // 2, d // 2, d // 16, d // 16)]
    assert cache[0].numel() > 1 << 32
    bits = [syn.host_normal_bits((20, Hkv, d), s, "bf16") for s in (1, 2)]
    slots = (n_pages - 1) * page + 200 + np.arange(20)
    attn.attn_cache_write_fp4(*(syn.bits_to_tensor(b, "bf16", "cuda") for b in bits), *cache,
                              dev(slots.astype(np.int32)))
    k, v = read(attn, cache, [[n_pages - 1]], [20], "bf16", starts=[200])
    for got, b in ((k, bits[0]), (v, bits[1])):
        assert np.array_equal(got, paged4.quantise(bits_to_double(b, "bf16"))[2])
