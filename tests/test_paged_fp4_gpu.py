"""GPU parity of attention over the 4-bit paged cache: the decode step and chunks of new tokens, against
the fp64 oracle over the values that the cache holds.

Tolerance (oracle/chunk.py derives the bound): keys and values are exact in fp16; the weights are rounded
to fp16 (spacing 2^-10 at 1; the largest is at least 2^7, so that a subnormal step of 2^-24 is 2^-31 of
it), o to its type, a bf16 query to fp16 after a power of two brings its largest element into [1, 2): an
element below fp16's normal numbers is off by at most 2^-25, of the largest element at least, which a
score sums over |k_c|."""
import numpy as np
import pytest

import synthetic as syn
from oracle import bits_to_double, chunk, paged4

pytestmark = pytest.mark.gpu

EPS = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10}


@pytest.fixture(scope="module")
def attn():
    import exact_io_aware_09_gb300 as m

    return m


def i32(x):
    import torch

    return torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")


class Cache:
    """A quantised cache of random rows; places that hold no token have NaN scales and random codes."""

    def __init__(self, lengths, Hkv, d, page, seed, k_scale=1.0, v_scale=1.0):
        import torch

        rng = np.random.default_rng(seed)
        T = int(np.sum(lengths))
        self.lengths = list(lengths)
        table, n_pages, self.pg, self.sl = syn.paged_layout(self.lengths, page, seed=seed)
        cu = syn.cu_seqlens(self.lengths)
        self.host, self.seqs = [], []
        for f in (k_scale, v_scale):
            x = rng.standard_normal((T, Hkv, d)) * f
            x[..., ::37] *= 4.0
            codes, scales, val = paged4.quantise(x)
            full = (rng.integers(0, 256, size=(n_pages, Hkv, page, d // 2), dtype=np.uint8),
                    np.full((n_pages, Hkv, page, d // 16), paged4.NAN_SCALE, dtype=np.uint8))
            full[0][self.pg, :, self.sl] = codes
            full[1][self.pg, :, self.sl] = scales
            self.host.append(full)
            self.seqs.append([val[cu[b]:cu[b + 1]] for b in range(len(self.lengths))])
        (kc, ks), (vc, vs) = self.host
        self.dev = [torch.from_numpy(x).cuda() for x in (kc, vc, ks, vs)]
        self.table = torch.from_numpy(table).cuda()
        self.seqlens = i32(self.lengths)


def oracle_rows(qd, cu, cache, scale, window, sinks):
    rows = chunk.attend_paged(qd, cu, cache.seqs[0], cache.seqs[1], scale, window, sinks)
    extra = np.zeros(rows.lse.shape)
    G = qd.shape[1] // cache.seqs[0][0].shape[1]
    for b in range(len(cache.lengths)):
        r = slice(int(cu[b]), int(cu[b + 1]))
        if r.stop == r.start or not cache.lengths[b]:
            continue
        k = np.abs(cache.seqs[0][b]).sum(-1).max(0)      # [Hkv]
        extra[r] = scale * np.abs(qd[r]).max(-1) * np.repeat(k, G)[None]
    return rows, extra


def compare(o, lse, rows, extra, dtype, what):
    live = ~np.isnan(rows.lse)
    tol = chunk.row_tolerance(rows, 2.0 ** -10, EPS[dtype], 2.0 ** -31,
                              2.0 ** -25 * extra if dtype == "bf16" else 0.0)
    pick = lambda x: x[live]
    chunk.check(pick(o.double().cpu().numpy()), pick(lse.double().cpu().numpy()),
                chunk.Rows(*(pick(x) for x in rows)), [pick(t) for t in tol], what)


HEADS = [(128, "bf16", 16, 2), (64, "f16", 16, 4), (64, "bf16", 3, 3), (128, "f16", 16, 1),
         (64, "bf16", 11, 1), (128, "bf16", 5, 1)]
DEC_LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 511, 512, 513, 1000, 3000]


def decode(attn, cache, Hq, Hkv, d, dtype, seed=5, q_scale=1.0, max_k=None, **kw):
    B = len(cache.lengths)
    q = syn.host_normal_bits((B, Hq, d), seed, dtype)
    if q_scale != 1.0:
        q = syn.round_bits((bits_to_double(q, dtype) * q_scale).astype(np.float32), dtype)
    scale = 1.0 / np.sqrt(d)
    o, lse = attn.attn_decode_paged_fp4(syn.bits_to_tensor(q, dtype, "cuda"), *cache.dev, cache.table,
                                        cache.seqlens, max(cache.lengths) if max_k is None else max_k,
                                        scale=scale, **kw)
    return o, lse, oracle_rows(bits_to_double(q, dtype), np.arange(B + 1), cache, scale, -1, 0)


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("d,dtype,Hq,Hkv", HEADS)
def test_decode(attn, page, d, dtype, Hq, Hkv):
    cache = Cache(DEC_LENGTHS, Hkv, d, page, page + d)
    o, lse, (rows, extra) = decode(attn, cache, Hq, Hkv, d, dtype)
    assert attn.attn_poll_status() == 0
    compare(o, lse, rows, extra, dtype, f"decode {d} {dtype} {Hq}/{Hkv} {page}")


@pytest.mark.parametrize("lengths", [(1,), (1001,), (1024, 1024), (9000,), (0, 0, 0)])
@pytest.mark.parametrize("d,dtype", [(64, "f16"), (128, "bf16")])
def test_decode_splits(attn, lengths, d, dtype):
    """One block, clusters of up to eight, and the workspace; a bound far above the lengths."""
    cache = Cache(lengths, 2, d, 16, 77)
    need = attn.attn_decode_paged_fp4_workspace_bytes(len(lengths), 16, 2, max(lengths), d)
    assert (need > 0) == (max(lengths) > 1024)
    for max_k in {max(lengths), cache.table.shape[1] * 16}:
        o, lse, (rows, extra) = decode(attn, cache, 16, 2, d, dtype, max_k=max_k)
        assert attn.attn_poll_status() == 0
        compare(o, lse, rows, extra, dtype, f"decode {lengths}")


def test_decode_many_sequences(attn):
    rng = np.random.default_rng(0)
    lengths = rng.integers(0, 300, size=700).tolist()
    cache = Cache(lengths, 2, 64, 32, 12)
    o, lse, (rows, extra) = decode(attn, cache, 4, 2, 64, "bf16")
    assert attn.attn_poll_status() == 0
    compare(o, lse, rows, extra, "bf16", "700 sequences")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_scale,k_scale,v_scale", [(40.0, 30.0, 1.0), (1.0, 1.0, 3000.0), (1.0, 1.0, 1e-4),
                                                     (1e-3, 1e-3, 1.0), (0.0, 1.0, 1.0)])
def test_decode_magnitudes(attn, dtype, q_scale, k_scale, v_scale):
    """One key takes nearly all the weight; large and small values; scores of zero."""
    cache = Cache([700, 33, 1500], 2, 128, 16, 4, k_scale, v_scale)
    o, lse, (rows, extra) = decode(attn, cache, 8, 2, 128, dtype, q_scale=q_scale)
    assert attn.attn_poll_status() == 0
    # (values of 1e-4 give o on both sides of fp16's smallest normal number: row_tolerance has both half
    # steps, 2^-11 |o| and 2^-25)
    compare(o, lse, rows, extra, dtype, f"magnitudes {q_scale} {k_scale} {v_scale}")


def test_decode_rising_scores(attn):
    """Every sixteen keys raise the maximum by more than the 2^8 that the state takes without moving it,
    or stay below it by less."""
    import torch

    d, n = 64, 640
    cache = Cache([n, n], 1, d, 16, 3)
    q = np.zeros((2, 2, d))
    q[:, :, 0] = 64.0
    for b, step in ((0, 3.0), (1, 0.05)):
        x = cache.seqs[0][b]
        x[:] = 0.0
        x[:, 0, 0] = np.arange(n) // 16 * step
        codes, scales, val = paged4.quantise(x)
        at = slice(b * n, (b + 1) * n)
        cache.dev[0][cache.pg[at], :, cache.sl[at]] = torch.from_numpy(codes).cuda()
        cache.dev[2][cache.pg[at], :, cache.sl[at]] = torch.from_numpy(scales).cuda()
        cache.seqs[0][b] = val
    o, lse = attn.attn_decode_paged_fp4(torch.from_numpy(q).half().cuda(), *cache.dev, cache.table,
                                        cache.seqlens, n, scale=1.0 / 8)
    assert attn.attn_poll_status() == 0
    rows, extra = oracle_rows(q, np.arange(3), cache, 1.0 / 8, -1, 0)
    compare(o, lse, rows, extra, "f16", "rising scores")


# (cached tokens, new ones among them)
FEW = [(1, 1), (16, 4), (17, 3), (300, 2), (64, 4), (65, 1), (1200, 4), (5, 0), (0, 0), (4, 4)]
MANY = [(1, 1), (200, 200), (130, 65), (700, 33), (64, 64), (900, 0), (1500, 129), (0, 0), (257, 256)]


def attend(attn, cache, news, Hq, Hkv, d, dtype, window=-1, sinks=0, before=0, behind=0, seed=6, q=None, **kw):
    import torch

    cu = before + syn.cu_seqlens(news)
    total = int(cu[-1]) + behind
    if q is None:
        q = syn.host_normal_bits((total, Hq, d), seed, dtype)
    scale = 1.0 / np.sqrt(d)
    qt = syn.bits_to_tensor(q, dtype, "cuda")
    o = torch.full_like(qt, 5.0)
    lse = torch.full((total, Hq), 5.0, device="cuda")
    attn.attn_fwd_paged_fp4(qt, *cache.dev, cache.table, i32(cu), cache.seqlens, max(news),
                            max(cache.lengths), window=window, sinks=sinks, o=o, lse=lse, scale=scale, **kw)
    rows = oracle_rows(bits_to_double(q, dtype), cu, cache, scale, window, sinks)
    outside = torch.ones(total, dtype=torch.bool)
    outside[int(cu[0]):int(cu[-1])] = False
    torch.cuda.synchronize()
    assert (o[outside] == 5.0).all() and (lse[outside] == 5.0).all(), "rows of no sequence"
    return o, lse, rows


MASKS = [(-1, 0), (0, 0), (3, 1), (100, 4), (100, 70), (5000, 3)]


@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("d,dtype,Hq,Hkv,page", [(128, "bf16", 4, 2, 16), (64, "f16", 4, 1, 64),
                                                 (64, "bf16", 6, 2, 32), (128, "f16", 2, 2, 128)])
def test_few_new_tokens(attn, window, sinks, d, dtype, Hq, Hkv, page):
    cache = Cache([a for a, _ in FEW], Hkv, d, page, page + 3)
    o, lse, (rows, extra) = attend(attn, cache, [b for _, b in FEW], Hq, Hkv, d, dtype, window, sinks,
                                   before=2, behind=3)
    assert attn.attn_poll_status() == 0
    compare(o, lse, rows, extra, dtype, f"few {d} {dtype} {window} {sinks}")


@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("d,dtype,Hq,Hkv,page", [(128, "bf16", 8, 2, 16), (64, "f16", 6, 2, 64),
                                                 (64, "bf16", 5, 1, 32), (128, "f16", 3, 3, 256)])
def test_chunks(attn, window, sinks, d, dtype, Hq, Hkv, page):
    cache = Cache([a for a, _ in MANY], Hkv, d, page, page + 5)
    o, lse, (rows, extra) = attend(attn, cache, [b for _, b in MANY], Hq, Hkv, d, dtype, window, sinks,
                                   before=1, behind=130)
    assert attn.attn_poll_status() == 0
    compare(o, lse, rows, extra, dtype, f"chunks {d} {dtype} {window} {sinks}")


@pytest.mark.parametrize("d,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("Hq,n", [(17, 1), (128, 1), (100, 3), (48, 2)])
def test_large_groups(attn, d, dtype, Hq, n):
    """Groups that do not divide the 128 rows of a tile, and the largest."""
    cache = Cache([600, 40], 1, d, 16, 8)
    o, lse, (rows, extra) = attend(attn, cache, [n, n], Hq, 1, d, dtype)
    assert attn.attn_poll_status() == 0
    compare(o, lse, rows, extra, dtype, f"group {Hq}")


@pytest.mark.parametrize("d,dtype,Hq,Hkv,n", [(128, "bf16", 16, 2, 5), (64, "f16", 8, 1, 1), (128, "f16", 8, 1, 2),
                                              (128, "bf16", 8, 1, 40)])
def test_long_caches_are_split(attn, d, dtype, Hq, Hkv, n):
    lengths = [9000, 20, 4097]
    cache = Cache(lengths, Hkv, d, 64, 9)
    news = [n, min(n, 20), n]
    need = attn.attn_fwd_paged_fp4_workspace_bytes(sum(news), 3, Hq, Hkv, n, 9000, d)
    assert need > 0
    o, lse, (rows, extra) = attend(attn, cache, news, Hq, Hkv, d, dtype)
    assert attn.attn_poll_status() == 0
    compare(o, lse, rows, extra, dtype, f"split {n}")


@pytest.mark.parametrize("d,dtype,n", [(64, "bf16", 3), (64, "f16", 8), (64, "f16", 5), (128, "bf16", 4)])
def test_part_of_a_tile_over_many_steps(attn, d, dtype, n):
    """24 to 64 rows of 128: the warps without rows pass the barriers on over hundreds of steps, in many
    blocks at a time; two calls give the same bits."""
    import torch

    lengths = [6000, 5111] * 12
    cache = Cache(lengths, 2, d, 32, 13)
    news = [n] * len(lengths)
    a = attend(attn, cache, news, 16, 2, d, dtype)
    b = attend(attn, cache, news, 16, 2, d, dtype)
    assert attn.attn_poll_status() == 0
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])
    compare(a[0], a[1], *a[2], dtype, f"part of a tile {d} {n}")


@pytest.mark.parametrize("q_scale,k_scale,v_scale", [(30.0, 30.0, 1.0), (1.0, 1.0, 3000.0), (1e-3, 1e-3, 1.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_chunk_magnitudes(attn, dtype, q_scale, k_scale, v_scale):
    lengths, news = [500, 200], [100, 200]
    cache = Cache(lengths, 2, 128, 16, 4, k_scale, v_scale)
    q = syn.host_normal_bits((300, 8, 128), 3, dtype)
    q = syn.round_bits((bits_to_double(q, dtype) * q_scale).astype(np.float32), dtype)
    o, lse, (rows, extra) = attend(attn, cache, news, 8, 2, 128, dtype, q=q)
    assert attn.attn_poll_status() == 0
    compare(o, lse, rows, extra, dtype, f"chunk magnitudes {q_scale} {k_scale} {v_scale}")


def test_far_apart_query_elements(attn):
    """bf16 queries whose elements span more than fp16's range, rows of zeros, rows of huge numbers."""
    rng = np.random.default_rng(1)
    for news, Hq in (([3, 1], 4), ([60, 31], 4)):
        total = sum(news)
        q = rng.standard_normal((total, Hq, 64)) * 2.0 ** rng.integers(-60, 4, size=(total, Hq, 64))
        q[0, 0] = 0.0
        q[1, 1] *= 2.0 ** 80
        q = syn.round_bits(q.astype(np.float32), "bf16")
        cache = Cache([90, 300], 1, 64, 16, 2, k_scale=2.0 ** -3)
        o, lse, (rows, extra) = attend(attn, cache, news, Hq, 1, 64, "bf16", q=q)
        assert attn.attn_poll_status() == 0
        compare(o, lse, rows, extra, "bf16", "far apart")


# few rows, codes converted by the kernel, and an f16 copy (eight query tiles and more)
@pytest.mark.parametrize("Hq,news", [(2, [4, 1]), (8, [40, 1]), (32, [41, 7])])
def test_nan_in_unseen_places(attn, Hq, news):
    """Places behind a sequence's end are NaN in every test here; keys before every window too."""
    import torch

    cache = Cache([400, 260], 1, 64, 16, 6)
    args = dict(window=30, sinks=5)
    ref, lse, (rows, extra) = attend(attn, cache, news, Hq, 1, 64, "f16", **args)
    compare(ref, lse, rows, extra, "f16", "before")
    for b, n in enumerate(news):
        at = np.arange(5, cache.lengths[b] - n - 30) + (0 if b == 0 else 400)
        for i in (2, 3):
            cache.dev[i][cache.pg[at], :, cache.sl[at]] = paged4.NAN_SCALE
    got, lse2, _ = attend(attn, cache, news, Hq, 1, 64, "f16", **args)
    assert attn.attn_poll_status() == 0
    assert torch.equal(got.view(torch.int16), ref.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("Hq,n", [(2, 2), (4, 30)])
def test_nan_that_is_seen(attn, Hq, n):
    cache = Cache([100, 100], 1, 64, 16, 6)
    cache.dev[3][cache.pg[10], 0, cache.sl[10], 1] = paged4.NAN_SCALE   # a value of the first sequence
    o, lse, _ = attend(attn, cache, [n, n], Hq, 1, 64, "f16")
    assert attn.attn_poll_status() == 0
    assert o[:n, :, 16:32].isnan().all() and o[:n, :, :16].isfinite().all() and o[:n, :, 32:].isfinite().all()
    assert o[n:].isfinite().all() and lse.isfinite().all()
    cache.dev[2][cache.pg[10], 0, cache.sl[10], 0] = paged4.NAN_SCALE   # and a key
    o, lse, _ = attend(attn, cache, [n, n], Hq, 1, 64, "f16")
    assert o[:n].isnan().all() and lse[:n].isnan().all() and o[n:].isfinite().all()


@pytest.mark.parametrize("Hq,n", [(2, 2), (4, 30)])
def test_bad_lengths_and_pages(attn, Hq, n):
    cache = Cache([100, 100, 100], 1, 64, 16, 6)
    o, lse, (rows, extra) = attend(attn, cache, [n] * 3, Hq, 1, 64, "f16")
    assert attn.attn_poll_status() == 0

    def others(bad):
        o, lse, _ = attend(attn, cache, [n] * 3, Hq, 1, 64, "f16")
        assert attn.attn_poll_status() == -8
        keep = np.ones(3 * n, dtype=bool)
        keep[bad * n:(bad + 1) * n] = False
        live = chunk.Rows(*(x[keep] for x in rows))
        compare(o[keep], lse[keep], live, extra[keep], "f16", "the other sequences")

    for wrong in (101, n - 1, -3, 2147483647):
        cache.seqlens[1] = wrong
        others(1)
    cache.seqlens[1] = 100
    for wrong in (-1, cache.dev[0].shape[0], 2147483647):
        was = int(cache.table[2, 3])
        cache.table[2, 3] = wrong
        others(2)
        cache.table[2, 3] = was
    o2, lse2, _ = attend(attn, cache, [n] * 3, Hq, 1, 64, "f16")
    assert attn.attn_poll_status() == 0
    compare(o2, lse2, rows, extra, "f16", "afterwards")
    if n * Hq > 16:
        return
    cache.seqlens[0] = 113
    B = 3
    q = syn.bits_to_tensor(syn.host_normal_bits((B, Hq, 64), 1, "f16"), "f16", "cuda")
    attn.attn_decode_paged_fp4(q, *cache.dev, cache.table, cache.seqlens, 112)
    assert attn.attn_poll_status() == -8


def test_a_serving_loop(attn):
    """Pages, writes and attention as a server runs them: prompts in chunks, decode steps, drafted tokens
    of which some go, sequences that end and new ones in their place; each step against the oracle."""
    import torch

    rng = np.random.default_rng(7)
    B, Hq, Hkv, d, page, n_pages, width = 6, 8, 2, 64, 16, 120, 20
    lists = paged4.Lists(B, rng.permutation(n_pages).tolist(), page)
    table, seqlens = i32(np.full((B, width), -1)), i32(np.zeros(B))
    free, n_free = i32(lists.free), i32([n_pages])
    cache = [torch.full((n_pages, Hkv, page, w), 0xFF, dtype=torch.uint8, device="cuda")
             for w in (d // 2, d // 2, d // 16, d // 16)]
    seqs = [[np.zeros((0, Hkv, d))] * B for _ in range(2)]
    scale = 1.0 / np.sqrt(d)
    plan = [[40, 3, 0, 70, 16, 1], [1] * 6, [33, 1, 90, 1, 1, 1], [4] * 6, [1, 0, 1, 1, 1, 0], [2, 5, 1, 7, 1, 3],
            [1] * 6]
    for step, news in enumerate(plan):
        cu = syn.cu_seqlens(news)
        total = int(cu[-1])
        bits = [syn.host_normal_bits((total, Hkv, d), 100 * step + i, "bf16") for i in range(2)]
        q = syn.host_normal_bits((total, Hq, d), 100 * step + 9, "bf16")
        qt = syn.bits_to_tensor(q, "bf16", "cuda")
        slots = attn.attn_pages_extend(table, seqlens, i32(cu), free, n_free, page, total)
        attn.attn_cache_write_fp4(*(syn.bits_to_tensor(x, "bf16", "cuda") for x in bits), *cache, slots)
        if news == [1] * 6:
            o, lse = attn.attn_decode_paged_fp4(qt, *cache, table, seqlens, width * page, scale=scale)
        else:
            o, lse = attn.attn_fwd_paged_fp4(qt, *cache, table, i32(cu), seqlens, max(news), width * page,
                                             scale=scale)
        back = attn.attn_cache_read_fp4(*cache, table, i32(cu), total, starts=seqlens - i32(news))
        assert attn.attn_poll_status() == 0
        assert slots.cpu().tolist() == lists.extend(news)
        for i in range(2):
            val = paged4.quantise(bits_to_double(bits[i], "bf16"))[2]
            assert np.array_equal(back[i].double().cpu().numpy(), val)
            seqs[i] = [np.concatenate([seqs[i][b], val[cu[b]:cu[b + 1]]]) for b in range(B)]
        state = Cache.__new__(Cache)
        state.lengths, state.seqs = [len(x) for x in seqs[0]], seqs
        rows, extra = oracle_rows(bits_to_double(q, "bf16"), cu, state, scale, -1, 0)
        compare(o, lse, rows, extra, "bf16", f"step {step}")
        keep = np.array([len(x) for x in seqs[0]])
        if step == 3:                       # three of four drafted tokens are not accepted
            keep -= 3
        elif step == 4:                     # two sequences end
            keep[[0, 3]] = 0
        attn.attn_pages_trim(table, seqlens, i32(keep), free, n_free, page)
        lists.trim(keep.tolist())
        seqs = [[x[:keep[b]] for b, x in enumerate(s)] for s in seqs]
        assert seqlens.cpu().tolist() == keep.tolist() and int(n_free) == len(lists.free)
    assert attn.attn_poll_status() == 0


@pytest.mark.parametrize("news", [1, 30])
def test_captured_step(attn, news):
    """A whole step (pages, write, attention) captured once and replayed; two graphs with workspaces of
    their own one after the other."""
    import torch

    B, Hq, Hkv, d, page, width = 3, 8, 1, 64, 16, 120
    start = [200, 7, 1300]
    cache = Cache(start, Hkv, d, page, 21)
    n_pages = cache.dev[0].shape[0]
    more = 40
    pools = [torch.cat([x, torch.full((more,) + x.shape[1:], 0xFF, dtype=torch.uint8, device="cuda")])
             for x in cache.dev]
    stack = list(range(n_pages, n_pages + more)) + list(range(n_pages))  # (an entry for every page)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[:, :cache.table.shape[1]] = cache.table
    free, n_free, seqlens = i32(stack), i32([more]), i32(start)
    cu = syn.cu_seqlens([news] * B)
    total = int(cu[-1])
    kv = [torch.empty((total, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q = torch.empty((total, Hq, d), dtype=torch.bfloat16, device="cuda")
    cut, lim = i32(cu), width * page
    graphs, outs = [], []
    for _ in range(2):
        def step():
            slots = attn.attn_pages_extend(table, seqlens, cut, free, n_free, page, total)
            attn.attn_cache_write_fp4(*kv, *pools, slots)
            return attn.attn_fwd_paged_fp4(q, *pools, table, cut, seqlens, news, lim)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    seqs = [list(s) for s in cache.seqs]
    for i in range(4):
        bits = [syn.host_normal_bits((total, Hkv, d), 50 * i + s, "bf16") for s in (1, 2)]
        qb = syn.host_normal_bits((total, Hq, d), 50 * i + 3, "bf16")
        for dst, b in zip(kv + [q], bits + [qb]):
            dst.copy_(syn.bits_to_tensor(b, "bf16", "cuda"))
        graphs[i % 2].replay()
        assert attn.attn_poll_status() == 0
        for s in range(2):
            val = paged4.quantise(bits_to_double(bits[s], "bf16"))[2]
            seqs[s] = [np.concatenate([x, val[cu[b]:cu[b + 1]]]) for b, x in enumerate(seqs[s])]
        state = Cache.__new__(Cache)
        state.lengths, state.seqs = [len(x) for x in seqs[0]], seqs
        rows, extra = oracle_rows(bits_to_double(qb, "bf16"), cu, state, 0.125, -1, 0)
        compare(*outs[i % 2], rows, extra, "bf16", f"replay {i}")


def test_another_stream(attn):
    """Calls on a stream of their own while the default one is busy; results belong to that stream."""
    import torch

    cache = Cache([900, 40, 5000], 2, 128, 16, 31)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kind in range(2):
        torch.cuda._sleep(50_000_000)
        if kind == 0:
            o, lse, (rows, extra) = decode(attn, cache, 4, 2, 128, "bf16", stream=side)
            side.synchronize()
            compare(o, lse, rows, extra, "bf16", "decode on another stream")
        else:
            q = syn.host_normal_bits((90, 8, 128), 6, "bf16")
            with torch.cuda.stream(side):
                qt = syn.bits_to_tensor(q, "bf16", "cuda")
                cu = i32([0, 40, 60, 90])
            o, lse = attn.attn_fwd_paged_fp4(qt, *cache.dev, cache.table, cu, cache.seqlens, 40, 5000,
                                             stream=side)
            side.synchronize()
            rows, extra = oracle_rows(bits_to_double(q, "bf16"), np.array([0, 40, 60, 90]), cache,
                                      1 / np.sqrt(128), -1, 0)
            compare(o, lse, rows, extra, "bf16", "chunk on another stream")
    assert attn.attn_poll_status(side) == 0


def test_a_pool_past_32_bit_offsets(attn):
    """Sequences in the last pages of pools whose byte offsets pass 2^32."""
    import torch

    lengths, Hkv, page, d = [300, 90], 8, 256, 128
    small = Cache(lengths, Hkv, d, page, 2)
    n = small.dev[0].shape[0]
    n_pages = (1 << 32) // (Hkv * page * (d // 2)) + n + 1
    big = [torch.empty((n_pages,) + x.shape[1:], dtype=torch.uint8, device="cuda") for x in small.dev]
    for x, y in zip(big, small.dev):
        x[-n:] = y
    small.dev = big
    small.table = torch.where(small.table >= 0, small.table + (n_pages - n), small.table)
    o, lse, (rows, extra) = decode(attn, small, 16, Hkv, d, "bf16")
    assert attn.attn_poll_status() == 0
    compare(o, lse, rows, extra, "bf16", "far pages")
    o, lse, (rows, extra) = attend(attn, small, [70, 30], 16, Hkv, d, "bf16")
    assert attn.attn_poll_status() == 0
    compare(o, lse, rows, extra, "bf16", "far pages, chunk")


# products of whole numbers in log2 units, far from zero: `lo` above base at tokens 0 .. 63, `hi` at tokens 64 and
# 128, base elsewhere.  The references lie 8 (or fp32's step there) below `hi`
FAR_SCORES = [(2.0 ** 24, 16, 24), (2.0 ** 24, 16, 26), (2.0 ** 25, 8, 16), (2.0 ** 27, 16, 32), (-2.0 ** 24, 4, 12),
              (2.0 ** 23, 3, 11), (-2.0 ** 25, 16, 24)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("B,Hq,n", [(640, 1, 1), (640, 8, 2), (1, 8, 40), (1, 32, 41)])
@pytest.mark.parametrize("base,lo,hi", FAR_SCORES)
def test_scores_far_from_zero(attn, base, lo, hi, B, Hq, n, dtype):
    """Scores of 10^7 and more whose differences are small: a reference of the weights that fp32 rounds must
    not carry a weight past fp16.  (B: as many sequences, all of the same pages, as leave a sequence in one
    split.)  Scores are exact, weights powers of two; o is rounded once, its weights half a step at most."""
    import torch

    L, d, page = 300, 64, 64
    x = np.zeros(L)
    x[:64], x[[64, 128]] = lo, hi
    n_pages = -(-L // page)
    kc = np.zeros((n_pages, 1, page, d // 2), dtype=np.uint8)
    ks = np.zeros((n_pages, 1, page, d // 16), dtype=np.uint8)
    at = lambda s: np.searchsorted(paged4.E5M3, s)
    pg, sl = np.arange(L) // page, np.arange(L) % page
    kc[pg, 0, sl, 0] = 6 + 8 * (base < 0)                       # channel 0: 4 times its scale
    ks[pg, 0, sl, 0] = at(abs(base) / 131072)                   # (and 32768 in the query)
    kc[pg, 0, sl, 8] = np.where(x > 0, 6, 0)                    # channel 16
    ks[pg, 0, sl, 1] = at(x / 4)
    v = np.random.default_rng(3).standard_normal((L, 1, d))
    codes, scales, val = paged4.quantise(v)
    vc, vs = kc.copy(), ks.copy()
    vc[pg, :, sl], vs[pg, :, sl] = codes, scales
    q = torch.zeros((B * n, Hq, d), dtype=syn.torch_dtype(dtype), device="cuda")
    q[..., 0], q[..., 16] = 32768.0, 1.0
    cache = [torch.from_numpy(a).cuda() for a in (kc, vc, ks, vs)]
    table = i32(np.tile(np.arange(n_pages), (B, 1)))
    scale = float(np.float32(np.log(2.0)))                      # (times log2 e in fp32: 1)
    assert np.float32(scale) * np.float32(1.4426950408889634) == 1.0
    if n == 1:
        o, lse = attn.attn_decode_paged_fp4(q, *cache, table, i32([L] * B), L, scale=scale)
    else:
        o, lse = attn.attn_fwd_paged_fp4(q, *cache, table, i32(np.arange(B + 1) * n), i32([L] * B), n, L,
                                         scale=scale)
    assert attn.attn_poll_status() == 0
    w = np.exp2(x - hi)[None] * (np.arange(L)[None] <= np.arange(L - n, L)[:, None])
    l = w.sum(1, keepdims=True)
    want, size = (w @ val[:, 0]) / l, (w @ np.abs(val[:, 0])) / l
    lim = (2.0 ** -11 + 2.0 ** -17) * size + 2.0 ** -32 * np.abs(val[:, 0]).sum(0)
    lim = (lim + EPS[dtype] / 2 * (np.abs(want) + lim) + 2.0 ** -25)[None, :, None]
    got = o.double().cpu().numpy().reshape(B, n, Hq, d)
    assert np.isfinite(got).all()
    assert (np.abs(got - want[None, :, None]) <= lim).all()
    ref = (base + hi + np.log2(l[:, 0])) * np.log(2.0)
    got = lse.double().cpu().numpy().reshape(B, n, Hq)
    assert (np.abs(got - ref[None, :, None]) <= 2.0 ** -22 * np.abs(ref)[None, :, None]).all()


@pytest.mark.parametrize("d,dtype", [(64, "f16"), (128, "bf16")])
def test_bad_pages_of_a_long_chunk(attn, d, dtype):
    """Over the f16 copy of the cache: a table entry outside the pool is reported, its tokens count as zeros
    whatever the workspace held, and the other sequences' rows are right.  Entries of pages before the tiles
    that a window reaches are not looked at."""
    import torch

    Hq, n, lengths = 32, 41, [400, 300, 500]
    cache = Cache(lengths, 1, d, 16, 6)
    need = attn.attn_fwd_paged_fp4_workspace_bytes(3 * n, 3, Hq, 1, n, max(lengths), d)
    assert need >= 3 * 448 * d * 4, "the call takes a copy"
    run = lambda **kw: attend(attn, cache, [n] * 3, Hq, 1, d, dtype, workspace=torch.full(
        (attn.attn_fwd_paged_fp4_workspace_bytes(3 * n, 3, Hq, 1, n, max(lengths), d, **kw),), 0xFF,
        dtype=torch.uint8, device="cuda"), **kw)
    o, lse, (rows, extra) = run()
    assert attn.attn_poll_status() == 0
    compare(o, lse, rows, extra, dtype, "all pages good")
    for bad, at in ((2, 3), (0, 24), (1, 18)):
        was = int(cache.table[bad, at])
        keep = np.ones(3 * n, dtype=bool)
        keep[bad * n:(bad + 1) * n] = False
        for wrong in (-1, cache.dev[0].shape[0], 2147483647, -2147483648):
            cache.table[bad, at] = wrong
            o, lse, _ = run()
            assert attn.attn_poll_status() == -8
            compare(o[keep], lse[keep], chunk.Rows(*(x[keep] for x in rows)), extra[keep], dtype, "the others")
            assert o.isfinite().all() and lse.isfinite().all()
        cache.table[bad, at] = was
    # a window of 30 keys with 5 sinks reads the tiles of 128 keys that hold either
    o, lse, (rows, extra) = run(window=30, sinks=5)
    assert attn.attn_poll_status() == 0
    for b, L in enumerate(lengths):
        first = (L - n - 30) // 128 * 128 // 16
        cache.table[b, 128 // 16:first] = -1
    o2, lse2, _ = run(window=30, sinks=5)
    assert attn.attn_poll_status() == 0
    compare(o2, lse2, rows, extra, dtype, "entries before the window")
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)


def test_far_apart_query_rows(attn):
    """bf16 queries whose elements span more than fp16's range and rows of zeros, by a tolerance that is a
    number everywhere; rows of huge numbers, whose scores are so far apart that one value is the answer."""
    rng = np.random.default_rng(11)
    for news, Hq in (([3, 1], 4), ([60, 31], 4), ([33, 7], 32)):
        total = sum(news)
        q = rng.standard_normal((total, Hq, 64)) * 2.0 ** rng.integers(-60, 4, size=(total, Hq, 64))
        q[0, 0] = 0.0
        huge = [(t, h) for t, h in ((1, 1), (total - 1, 2), (2, Hq - 1))]
        for t, h in huge:
            q[t, h] *= 2.0 ** 80
        q = syn.round_bits(q.astype(np.float32), "bf16")
        lengths = [90, 300]
        cache = Cache(lengths, 1, 64, 16, 2, k_scale=2.0 ** -3)
        o, lse, (rows, extra) = attend(attn, cache, news, Hq, 1, 64, "bf16", q=q)
        assert attn.attn_poll_status() == 0
        qd, cu = bits_to_double(q, "bf16"), syn.cu_seqlens(news)
        ordinary = np.ones((total, Hq), dtype=bool)
        for t, h in huge:
            ordinary[t, h] = False
            b = int(np.searchsorted(cu, t, side="right")) - 1
            seen = lengths[b] - news[b] + (t - cu[b]) + 1
            s = 0.125 * (cache.seqs[0][b][:seen, 0] @ qd[t, h])
            top, second = np.sort(s)[::-1][:2]
            off = 2.0 ** -20 * rows.score[t, h] + 2.0 ** -25 * extra[t, h]
            assert top - second > 2 * off + 100.0, "the largest score is not certain"
            assert np.array_equal(o[t, h].double().cpu().numpy(), cache.seqs[1][b][int(np.argmax(s)), 0])
            assert abs(float(lse[t, h]) - top) <= off + 2.0 ** -22 * abs(top)
        pick = chunk.Rows(*(x[ordinary] for x in rows))
        tol = chunk.row_tolerance(pick, 2.0 ** -10, EPS["bf16"], 2.0 ** -31, 2.0 ** -25 * extra[ordinary])
        assert all(np.isfinite(t).all() for t in tol)
        for got, want, lim in ((o, pick.o, tol[0]), (lse, pick.lse, tol[1])):
            got = got.double().cpu().numpy()[ordinary]
            assert (np.abs(got - want) <= lim).all()
