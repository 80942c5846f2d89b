"""GPU parity of attn_fwd_paged (chunks of new tokens over a paged cache) against the fp64 oracle.

Tolerances are derived in oracle/chunk.py (row_tolerance).  Every pool is shuffled, and rows that
hold no token of a sequence are NaN: pages end inside a tile, so any use of such a row shows.
Chunks of one token to several query tiles, caches of one token to many tiles (split and merged
when there are few query tiles), page sizes from 16 to 1024, group sizes that do and do not divide
128, with and without a window and sinks.
"""
import numpy as np
import pytest

import synthetic as syn
from oracle import bits_to_double, chunk

pytestmark = pytest.mark.gpu

EPS = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24}


@pytest.fixture(scope="module")
def attn():
    import exact_io_aware_09_gb300 as m

    return m


def build(lengths, chunks, Hq, Hkv, d, dtype, page, seed, tail=0):
    """Device tensors of a call and the oracle's view of it; `tail` packed rows follow the last
    sequence."""
    import torch

    cu_k = syn.cu_seqlens(lengths)
    k = syn.host_normal_bits((int(cu_k[-1]), Hkv, d), seed, dtype)
    v = syn.host_normal_bits((int(cu_k[-1]), Hkv, d), seed + 1, dtype)
    cu_q = syn.cu_seqlens(chunks)
    q = syn.host_normal_bits((int(cu_q[-1]) + tail, Hq, d), seed + 2, dtype)
    table, n_pages, pg, sl = syn.paged_layout(lengths, page, seed=seed)
    dev = lambda x: syn.bits_to_tensor(x, dtype, "cuda")
    kp = syn.scatter_to_pages(dev(k), n_pages, page, pg, sl)
    vp = syn.scatter_to_pages(dev(v), n_pages, page, pg, sl)
    args = (dev(q), kp, vp, torch.from_numpy(table).cuda(), torch.from_numpy(cu_q).cuda(),
            torch.tensor(lengths, dtype=torch.int32, device="cuda"), max(chunks), max(lengths))
    kd, vd = bits_to_double(k, dtype), bits_to_double(v, dtype)
    seqs = lambda x: [x[cu_k[b]:cu_k[b + 1]] for b in range(len(lengths))]
    return args, (bits_to_double(q, dtype), cu_q, seqs(kd), seqs(vd))


def run_and_check(attn, lengths, chunks, Hq, Hkv, d, dtype, page, window=-1, sinks=0, seed=1):
    import torch

    args, orc = build(lengths, chunks, Hq, Hkv, d, dtype, page, seed, tail=3)
    scale = 1.0 / np.sqrt(d)
    q = args[0]
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    attn.attn_fwd_paged(*args, window=window, sinks=sinks, o=o, lse=lse, scale=scale)
    assert attn.attn_poll_status() == 0
    rows = chunk.attend_paged(*orc, scale, window, sinks)
    n = int(orc[1][-1])
    # rows behind the last sequence are left as they were
    assert torch.all(o[n:] == 7.0) and torch.all(lse[n:] == 7.0)
    rows = chunk.Rows(*(x[:n] for x in rows))
    tol = chunk.row_tolerance(rows, EPS[dtype], EPS[dtype], TINY[dtype])
    chunk.check(o[:n].float().cpu().numpy(), lse[:n].cpu().numpy(), rows, tol,
                f"page {page} {Hq}/{Hkv} d={d} W={window} sinks={sinks}")
    return args, o, lse


LENGTHS = [1, 15, 16, 17, 127, 128, 129, 300, 1000, 2049]
CHUNKS = [1, 15, 1, 17, 100, 128, 2, 0, 333, 40]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("d,dtype,Hq,Hkv", [(128, "bf16", 16, 2), (64, "f16", 6, 2)])
def test_chunks(attn, page, d, dtype, Hq, Hkv):
    run_and_check(attn, LENGTHS, CHUNKS, Hq, Hkv, d, dtype, page, seed=page)


@pytest.mark.parametrize("W,s", [(0, 0), (0, 1), (100, 4), (127, 128), (300, 130), (2000, 5),
                                 (5000, 0)])
@pytest.mark.parametrize("d,dtype,Hq,Hkv", [(128, "f16", 8, 2), (64, "bf16", 5, 1)])
def test_window_and_sinks(attn, d, dtype, Hq, Hkv, W, s):
    run_and_check(attn, LENGTHS, CHUNKS, Hq, Hkv, d, dtype, 32, W, s, seed=7 + W + s)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (7, 1), (16, 1), (20, 1), (128, 1), (24, 8)])
def test_group_sizes(attn, Hq, Hkv):
    run_and_check(attn, [700, 130, 64], [70, 130, 3], Hq, Hkv, 128, "bf16", 64, seed=Hq)
    run_and_check(attn, [700, 130, 64], [1, 1, 1], Hq, Hkv, 64, "f16", 16, seed=Hq + 1)


# at most 16 (token, head) rows per key/value head: chunks of 16 / G tokens and fewer
FEW = [(16, 2, [1, 2, 1, 2, 2, 0, 1, 2, 2, 1]), (6, 2, [1, 5, 4, 3, 5, 0, 2, 5, 5, 1]),
       (16, 1, [1] * 10), (4, 4, [1, 15, 16, 8, 16, 0, 9, 16, 2, 16]), (8, 1, [1] * 10)]


@pytest.mark.parametrize("W,s", [(-1, 0), (0, 2), (63, 65), (200, 4), (1500, 300)])
@pytest.mark.parametrize("Hq,Hkv,chunks", FEW, ids=lambda x: str(x)[:8])
def test_few_rows(attn, Hq, Hkv, chunks, W, s):
    for d, dtype, page in ((128, "bf16", 16), (64, "f16", 64), (128, "f16", 256), (64, "bf16", 32)):
        run_and_check(attn, LENGTHS, chunks, Hq, Hkv, d, dtype, page, W, s, seed=W + 3 * Hq + d)


def test_few_rows_in_a_cluster_and_through_the_workspace(attn):
    """Eight splits and nine of 128 keys; a long cache, whose splits are longer."""
    for n in (1, 128, 1024, 1025, 9000, 40000):
        run_and_check(attn, [n, 3], [1, 1], 8, 1, 128, "bf16", 64, seed=n)
        run_and_check(attn, [n, 3], [1, 1], 2, 2, 64, "f16", 16, seed=n)


@pytest.mark.parametrize("lengths,chunks", [([1], [1]), ([5000], [1]), ([9000, 3], [2, 1]),
                                            ([4097], [9])])
@pytest.mark.parametrize("W,s", [(-1, 0), (1000, 4)])
def test_few_rows_are_split_and_merged(attn, lengths, chunks, W, s):
    run_and_check(attn, lengths, chunks, 8, 2, 128, "bf16", 16, W, s, seed=sum(lengths))
    run_and_check(attn, lengths, chunks, 4, 4, 64, "f16", 128, W, s, seed=sum(lengths) + 1)


def test_many_items(attn):
    """More work items than SMs, unsplit: blocks take over items of blocks not yet launched."""
    run_and_check(attn, [300] * 24 + [1500], [290] * 24 + [1500], 32, 8, 128, "bf16", 16, seed=3)
    run_and_check(attn, [300] * 24 + [1500], [290] * 24 + [1500], 16, 8, 64, "f16", 64, 200, 4,
                  seed=4)


def test_one_token_is_the_decode_step(attn):
    """One new token per sequence: attn_decode_paged's result within both kernels' rounding of O
    (half a step each and the weights' half step each: 4 half steps of the row's largest value)."""
    import torch

    lengths = [1, 64, 777, 3000]
    args, _ = build(lengths, [1] * 4, 16, 2, 128, "bf16", 32, 9)
    o, lse = attn.attn_fwd_paged(*args)
    q, kp, vp, table, _, seq, _, max_k = args
    o2, lse2 = attn.attn_decode_paged(q, kp, vp, table, seq, max_k)
    assert attn.attn_poll_status() == 0
    big = o2.float().abs().amax(-1, keepdim=True)
    assert torch.all((o.float() - o2.float()).abs() <= 4 * 2.0 ** -8 * big + 1e-2)
    assert torch.all((lse - lse2).abs() <= 1e-4)


def test_chunks_add_up_to_the_prefill(attn):
    """A prompt taken in chunks gives the rows of the prefill kernel on the whole of it."""
    import torch

    N, Hq, Hkv, d, page = 900, 8, 2, 128, 64
    args, _ = build([N], [N], Hq, Hkv, d, "bf16", page, 11)
    q, kp, vp, table = args[:4]
    whole, _ = attn.attn_fwd_paged(*args)
    parts = []
    for a, b in ((0, 1), (1, 130), (130, 514), (514, 900)):
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        seq = torch.tensor([b], dtype=torch.int32, device="cuda")
        parts.append(attn.attn_fwd_paged(q[a:b].contiguous(), kp, vp, table, cu, seq, b - a, b)[0])
    flat = lambda x: x[table[0, :-(-N // page)].long()].reshape(-1, Hkv, d)[:N].transpose(0, 1)[None]
    dense, _ = attn.attn_fwd(q.transpose(0, 1)[None].contiguous(), flat(kp).contiguous(),
                             flat(vp).contiguous(), causal=True)
    assert attn.attn_poll_status() == 0
    dense = dense[0].transpose(0, 1)
    big = dense.float().abs().amax(-1, keepdim=True)
    for got in (whole, torch.cat(parts)):
        assert torch.all((got.float() - dense.float()).abs() <= 4 * 2.0 ** -8 * big + 1e-2)


def test_bad_lengths_and_pages_are_reported(attn):
    """Lengths past their bounds and entries outside the pool are reported; the other sequences'
    rows are right and nothing outside the packed rows is written."""
    import torch

    lengths, chunks = [100, 300, 40], [10, 20, 5]
    args, orc = build(lengths, chunks, 8, 2, 128, "bf16", 16, 13)
    want, _ = attn.attn_fwd_paged(*args)
    assert attn.attn_poll_status() == 0
    for what in ("entry", "negative entry", "too long", "short"):
        a = list(args)
        a[3], a[5] = args[3].clone(), args[5].clone()
        if what == "entry":
            a[3][1, 3] = args[1].shape[0]
        elif what == "negative entry":
            a[3][1, 3] = -5
        elif what == "too long":
            a[5][1] = 301
        else:
            a[5][1] = 19  # fewer cached tokens than new ones
        o, _ = attn.attn_fwd_paged(*a)
        assert attn.attn_poll_status() == -8, what
        assert torch.equal(o[:10], want[:10]) and torch.equal(o[30:], want[30:]), what
    o, _ = attn.attn_fwd_paged(*args)
    assert attn.attn_poll_status() == 0 and torch.equal(o, want)


def test_pool_past_2_31_elements(attn):
    """A pool of 2.2e9 elements whose tokens lie in its last pages: the same bits as a small pool."""
    import torch

    lengths, chunks, page, Hkv, d = [3000, 500], [100, 1], 16, 8, 128
    args, _ = build(lengths, chunks, 16, Hkv, d, "bf16", page, 17)
    few = build(lengths, [2, 1], 16, Hkv, d, "bf16", page, 17)[0]  # the same cache, 4 rows a head
    want = attn.attn_fwd_paged(*args)
    want_few = attn.attn_fwd_paged(*few)
    n = args[1].shape[0]
    big_pages = 2 ** 31 // (page * Hkv * d) + 2 * n
    a = list(args)
    for i in (1, 2):
        pool = torch.zeros((big_pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
        pool[-n:] = args[i]
        a[i] = pool
    a[3] = torch.where(args[3] >= 0, args[3] + (big_pages - n), args[3])
    got = attn.attn_fwd_paged(*a)
    assert attn.attn_poll_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = attn.attn_fwd_paged(few[0], a[1], a[2], a[3], *few[4:])
    assert attn.attn_poll_status() == 0
    assert torch.equal(got[0], want_few[0]) and torch.equal(got[1], want_few[1])
    del a, pool
    torch.cuda.empty_cache()


def test_side_stream_and_graph_with_new_lengths(attn):
    """Captured once and replayed with other lengths, tables and queries in the same buffers."""
    import torch

    args, _ = build([600, 900], [4, 7], 16, 2, 128, "bf16", 32, 19)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = attn.attn_fwd_paged(*args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = attn.attn_fwd_paged(*args)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])
    args[5].copy_(torch.tensor([500, 333], dtype=torch.int32))
    args[4].copy_(torch.tensor([0, 6, 11], dtype=torch.int32))
    args[0].copy_(torch.randn_like(args[0]))
    graph.replay()
    want = attn.attn_fwd_paged(*args)
    assert attn.attn_poll_status() == 0
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_largest_window_and_sinks(attn):
    import torch

    args, _ = build([300, 900], [40, 200], 8, 2, 128, "bf16", 16, 27)
    few, _ = build([300, 900], [1, 2], 8, 2, 128, "bf16", 16, 28)
    for a in (args, few):
        want = attn.attn_fwd_paged(*a)
        for W, s in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (0, 2 ** 31 - 1), (-1, 2 ** 31 - 1)):
            got = attn.attn_fwd_paged(*a, window=W, sinks=s)
            assert attn.attn_poll_status() == 0
            big = want[0].float().abs().amax(-1, keepdim=True)
            assert torch.all((got[0].float() - want[0].float()).abs() <= 4 * 2.0 ** -8 * (big + 5.0))
            assert torch.all((got[1] - want[1]).abs() <= 1e-4)


def test_packed_rows_that_start_later(attn):
    """cu_seqlens_q[0] > 0: rows before the first sequence are left as they were, too."""
    import torch

    for chunks in ([2, 1], [60, 9]):
        args, _ = build([3000, 700], chunks, 16, 2, 128, "bf16", 32, 33)
        want = attn.attn_fwd_paged(*args)
        q = torch.cat([torch.randn_like(args[0][:3]), args[0]])
        o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        attn.attn_fwd_paged(q, *args[1:4], args[4] + 3, *args[5:], o=o, lse=lse)
        assert attn.attn_poll_status() == 0
        assert torch.all(o[:3] == 7.0) and torch.all(lse[:3] == 7.0)
        assert torch.equal(o[3:], want[0]) and torch.equal(lse[3:], want[1])


def test_two_streams_at_once(attn):
    """Calls of both kernels on two streams, each with its own workspace."""
    import torch

    a, _ = build([5000, 800], [3, 1], 16, 4, 128, "bf16", 16, 23)
    b, _ = build([9000], [1], 8, 8, 64, "f16", 16, 24)
    want = [attn.attn_fwd_paged(*x) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for st, x in zip(streams, (a, b)):
            with torch.cuda.stream(st):
                got.append(attn.attn_fwd_paged(*x))
    torch.cuda.synchronize()
    assert attn.attn_poll_status() == 0
    for i, g in enumerate(got):
        assert torch.equal(g[0], want[i % 2][0]) and torch.equal(g[1], want[i % 2][1])


def test_repeated_calls_are_bit_identical(attn):
    import torch

    args, _ = build([5000, 800, 2222], [3, 1, 200], 16, 4, 128, "bf16", 16, 23)
    a = attn.attn_fwd_paged(*args)
    for _ in range(5):
        b = attn.attn_fwd_paged(*args)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert attn.attn_poll_status() == 0


def test_nothing_to_do_and_refusals(attn):
    import torch

    args, _ = build([100, 50], [10, 1], 8, 2, 64, "f16", 16, 29)
    q, kp, vp, table, cu, seq, mq, mk = args
    o, lse = attn.attn_fwd_paged(q[:0], kp, vp, table, torch.zeros_like(cu), seq, 0, mk)
    assert o.shape[0] == 0 and attn.attn_poll_status() == 0
    bad = [
        dict(window=-2), dict(sinks=-1), dict(scale=0.0), dict(scale=float("nan")),
        dict(o=torch.empty_like(q, dtype=torch.bfloat16)), dict(lse=torch.empty(3, device="cuda")),
    ]
    for kw in bad:
        with pytest.raises(attn.AttnError):
            attn.attn_fwd_paged(*args, **kw)
    split, _ = build([5000], [1], 8, 2, 64, "f16", 16, 30)
    with pytest.raises(attn.AttnError):
        attn.attn_fwd_paged(*split, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    for a in ((q, kp, vp, table, cu, seq, mq, 10 ** 6),          # past the table's reach
              (q, kp, vp, table, cu, seq, mk + 1, mk),           # chunk longer than the cache
              (q, kp, vp, table.long(), cu, seq, mq, mk), (q, kp, vp, table, cu[:2], seq, mq, mk),
              (q, kp, vp.bfloat16(), table, cu, seq, mq, mk), (q, kp, vp, table, cu, seq.long(), mq, mk),
              (q[:, :7].contiguous(), kp, vp, table, cu, seq, mq, mk),  # 7 query heads for 2
              (q, kp[:, :24 - 16].contiguous(), vp[:, :8].contiguous(), table, cu, seq, mq, 8)):
        with pytest.raises(attn.AttnError):
            attn.attn_fwd_paged(*a)


@pytest.mark.parametrize("chunks,G", [((1, 1), 4), ((5, 1), 2), ((200, 33), 4), ((1, 130), 1)])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("sinks", [0, 20])
def test_pages_behind_the_window_need_no_entry(attn, chunks, G, page, sinks):
    """Table entries of pages outside the 128-key tiles of the sinks and the window: any number."""
    import torch

    window, lengths = 300, [4000, 2100]
    args, _ = build(lengths, list(chunks), 2 * G, 2, 128, "bf16", page, seed=5)
    o, lse = attn.attn_fwd_paged(*args, window=window, sinks=sinks)
    table = args[3].clone()
    freed = 0
    for b, n in enumerate(chunks):
        first = (-(-sinks // 128) * 128 + page - 1) // page
        last = (lengths[b] - n - window) // 128 * 128 // page
        for i in range(first, last):
            table[b, i] = (-1, 1 << 30)[i % 2]
            freed += 1
    assert freed > 0
    o2, lse2 = attn.attn_fwd_paged(*args[:3], table, *args[4:], window=window, sinks=sinks)
    assert attn.attn_poll_status() == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("as_int", [False, True])
def test_workspace_belongs_to_the_calls_stream(attn, as_int):
    """A call handed a busy stream, its workspace allocated inside: what the current stream
    allocates and fills while the call waits leaves its result alone."""
    import torch

    args, _ = build([3000, 5000], [4, 4], 16, 2, 128, "bf16", 64, seed=6)
    need = attn.attn_fwd_paged_workspace_bytes(8, 2, 16, 2, 4, 5000, 128)
    assert need > 0
    want, want_l = attn.attn_fwd_paged(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    o, lse = attn.attn_fwd_paged(*args, stream=side.cuda_stream if as_int else side)
    filled = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
              for n in (need, o.nbytes, lse.nbytes) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_l)
    del filled


@pytest.mark.parametrize("W,s", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (0, 2 ** 31 - 1),
                                 (-1, 2 ** 31 - 1)])
@pytest.mark.parametrize("chunks", [[40, 200], [1, 2]], ids=str)  # query tiles, few rows
def test_largest_window_and_sinks_by_the_definition(attn, chunks, W, s):
    run_and_check(attn, [300, 900], chunks, 8, 2, 128, "bf16", 16, W, s, seed=27)
    run_and_check(attn, [300, 900], chunks, 4, 2, 64, "f16", 64, W, s, seed=28)
