"""GPU parity of the quantised paged cache: writing, reading back and the decode step over it.

The codes and scales are compared with the fp64 definition exactly (the scale is a power of two,
so the only rounding is E4M3's nearest even), values read back with the rounding of their type, the
decode step with the tolerance derived in oracle/chunk.py.
"""
import numpy as np
import pytest

import synthetic as syn
from oracle import bits_to_double, chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    import exact_io_aware_09_gb300 as m

    return m


def pool(n_pages, page, Hkv, d):
    """An empty quantised cache whose every code is NaN and every scale 3."""
    import torch

    codes = lambda: torch.full((n_pages, page, Hkv, d), 0x7F, dtype=torch.uint8,
                               device="cuda").view(torch.float8_e4m3fn)
    scales = lambda: torch.full((n_pages, Hkv, page), 3.0, device="cuda")
    return codes(), codes(), scales(), scales()


def rows_bits(shape, dtype, seed):
    """N(0,1) rows with magnitudes spread over the type's range, zero rows, rows of one value, values
    at ties and at the format's ends."""
    bits = syn.host_normal_bits(shape, seed, dtype)
    x = syn.bits_to_float32(bits, dtype).copy()
    rng = np.random.default_rng(seed)
    top = 12 if dtype == "f16" else 60
    x *= np.exp2(rng.integers(-top, top, size=shape[:-1] + (1,))).astype(np.float32)
    flat = x.reshape(-1, shape[-1])
    flat[0] = 0.0
    if len(flat) > 4:
        flat[1] = 448.0
        flat[2, :8] = [448, 432, 416, 440, 17, 19, -17, -19]   # ties between neighbouring codes
        flat[2, 8:] = 2.0 ** -9 * 1.5
        flat[3] = 1e-30 if dtype == "bf16" else 2.0 ** -24
        flat[4] = 449.0 if dtype == "f16" else 452.0
    return syn.round_bits(x, dtype)


SEQ = [(1, 1), (5, 5), (17, 3), (64, 64), (300, 1), (513, 200), (70, 0)]  # (cached, new)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("d,dtype,Hkv", [(128, "bf16", 8), (64, "f16", 3), (128, "f16", 1),
                                         (64, "bf16", 2)])
def test_write_and_read(attn, page, d, dtype, Hkv):
    import torch

    lengths, news = [a for a, _ in SEQ], [b for _, b in SEQ]
    cu = syn.cu_seqlens(news)
    k, v = (rows_bits((int(cu[-1]) + 2, Hkv, d), dtype, page + i) for i in (1, 2))
    table, n_pages, pg, sl = syn.paged_layout(lengths, page, seed=page)
    cache = pool(n_pages, page, Hkv, d)
    dev = lambda x: syn.bits_to_tensor(x, dtype, "cuda")
    tab = torch.from_numpy(table).cuda()
    seq = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    attn.attn_cache_write_fp8(dev(k), dev(v), *cache, tab, torch.from_numpy(cu).cuda(), seq)
    assert attn.attn_poll_status() == 0
    # where each new token went
    cu_all = syn.cu_seqlens(lengths)
    at = np.concatenate([np.arange(cu_all[b + 1] - news[b], cu_all[b + 1]) for b in range(len(SEQ))])
    page_at, slot_at = pg[at], sl[at]
    for bits, codes, scales in ((k, cache[0], cache[2]), (v, cache[1], cache[3])):
        want_s, want_c = chunk.quantise(bits_to_double(bits[:cu[-1]], dtype))
        got_c, got_s = codes.float().cpu().numpy(), scales.cpu().numpy()
        assert np.array_equal(got_c[page_at, slot_at], want_c)
        assert np.array_equal(got_s[page_at, :, slot_at], want_s)
        got_c[page_at, slot_at] = np.nan  # and nothing else was touched
        got_s[page_at, :, slot_at] = 3.0
        assert np.isnan(got_c).all() and (got_s == 3.0).all()
    # read the new tokens back through a table that starts at each sequence's first new page
    whole = [b for b in range(len(SEQ)) if lengths[b] == news[b]]
    cu_r = syn.cu_seqlens([news[b] for b in whole])
    total = int(cu_r[-1]) + 3
    kr = torch.full((total, Hkv, d), 9.0, dtype=dev(k).dtype, device="cuda")
    vr = kr.clone()
    attn.attn_cache_read_fp8(*cache, tab[whole].contiguous(), torch.from_numpy(cu_r).cuda(), total,
                             k=kr, v=vr)
    assert attn.attn_poll_status() == 0
    src = np.concatenate([np.arange(cu[b], cu[b + 1]) for b in whole])
    for bits, got in ((k, kr), (v, vr)):
        s, c = chunk.quantise(bits_to_double(bits[src], dtype))
        want = syn.round_bits((s[..., None] * c).astype(np.float32), dtype)
        assert np.array_equal(syn.tensor_to_bits(got[:len(src)]), want)
        assert torch.all(got[len(src):] == 9.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_values_at_the_ends(attn, dtype):
    """Infinities and NaN become NaN codes and leave the row's other values alone; the largest
    finite values come back finite."""
    import torch

    dt = syn.torch_dtype(dtype)
    big = torch.finfo(dt).max
    d = 64
    x = torch.ones((4, 1, d), dtype=dt, device="cuda")
    x[0, 0, 3], x[0, 0, 4], x[0, 0, 5] = float("inf"), float("-inf"), float("nan")
    x[1] = big
    x[1, 0, 0] = -big
    x[2] = float("nan")
    x[3] = 2.0 ** (-133 if dtype == "bf16" else -24)  # the smallest subnormal
    cache = pool(1, 16, 1, d)
    tab = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    attn.attn_cache_write_fp8(x, x, *cache, tab, cu, cu[1:].contiguous())
    k, v = attn.attn_cache_read_fp8(*cache, tab, cu, 4, dtype=dt)
    assert attn.attn_poll_status() == 0
    s, c = chunk.quantise(x.double().cpu().numpy())
    assert np.array_equal(cache[0][0, :4].float().cpu().numpy(), c, equal_nan=True)
    assert np.array_equal(cache[2][0, :, :4].t().cpu().numpy(), s)
    assert torch.isnan(k[0, 0, 3:6]).all() and torch.all(k[0, 0, 6:] == 1.0)
    assert torch.isnan(k[2]).all() and torch.isfinite(k[1]).all()
    assert k[1, 0, 1] == big and k[1, 0, 0] == -big
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))


DEC_LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 511, 512, 513, 1000, 3000]


def make_cache(lengths, Hkv, d, page, seed, spread=3):
    """A quantised cache of random codes (NaN where no token is) with scales 2^-spread..2^spread
    around 2^-6, its table, and each sequence's (codes, scale) of K and V as float64."""
    import torch

    rng = np.random.default_rng(seed)
    T = int(np.sum(lengths))
    table, n_pages, pg, sl = syn.paged_layout(lengths, page, seed=seed)
    cache = pool(n_pages, page, Hkv, d)
    cu = syn.cu_seqlens(lengths)
    seqs = []
    for codes, scales in ((cache[0], cache[2]), (cache[1], cache[3])):
        x = rng.standard_normal((T, Hkv, d)) * 100.0
        c = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn)
        s = np.exp2(rng.integers(-6 - spread, -6 + spread + 1, size=(T, Hkv)).astype(np.float64))
        at = torch.from_numpy(pg).cuda(), torch.from_numpy(sl).cuda()
        codes.view(torch.uint8)[at] = c.view(torch.uint8).cuda()
        scales[at[0], :, at[1]] = torch.from_numpy(s).float().cuda()
        cd = c.double().numpy()
        seqs.append([(cd[cu[b]:cu[b + 1]], s[cu[b]:cu[b + 1]]) for b in range(len(lengths))])
    return cache, torch.from_numpy(table).cuda(), seqs


def decode_oracle(qd, seqs, scale, Hq, Hkv):
    """Rows of the decode step and, for its weights' rounding to fp16, the largest product of weight
    and value scale times the sum of the codes' magnitudes."""
    B, d = len(qd), qd.shape[-1]
    G = Hq // Hkv
    parts, extra, qk = [], np.zeros((B, Hq, d)), np.zeros((B, Hq))
    for b in range(B):
        (kc, ks), (vc, vs) = seqs[0][b], seqs[1][b]
        for h in range(Hq):
            hk = h // G
            k, v = kc[:, hk] * ks[:, hk, None], vc[:, hk] * vs[:, hk, None]
            pos = np.array([len(k) - 1])
            parts.append(chunk.attend(qd[b, h][None], k, v, pos, scale))
            if len(k):
                s = scale * (k @ qd[b, h])
                p = np.exp(s - s.max())
                p /= p.sum()
                extra[b, h] = (p * vs[:, hk]).max() * np.abs(vc[:, hk]).sum(axis=0)
                qk[b, h] = scale * np.abs(qd[b, h]).max() * np.abs(k).sum(axis=1).max()
    rows = chunk.Rows(*(np.concatenate(x) for x in zip(*parts)))
    return rows, extra.reshape(-1, d), qk.reshape(-1)


@pytest.mark.parametrize("split", [0, 64, 512])   # clusters of 1 to 8 blocks, and the workspace
@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("d,dtype,Hq,Hkv", [(128, "bf16", 16, 2), (64, "f16", 16, 4),
                                            (64, "bf16", 3, 3), (128, "f16", 16, 1),
                                            (64, "bf16", 11, 1), (128, "bf16", 5, 1)])
def test_decode(attn, page, d, dtype, Hq, Hkv, split):
    import torch

    B = len(DEC_LENGTHS)
    cache, table, seqs = make_cache(DEC_LENGTHS, Hkv, d, page, page + d)
    q = syn.host_normal_bits((B, Hq, d), 5, dtype)
    qt = syn.bits_to_tensor(q, dtype, "cuda")
    qd = bits_to_double(q, dtype)
    scale = 1.0 / np.sqrt(d)
    seq = torch.tensor(DEC_LENGTHS, dtype=torch.int32, device="cuda")
    o = torch.full_like(qt, float("nan"))
    lse = torch.full((B, Hq), float("nan"), device="cuda")
    attn.attn_decode_paged_fp8(qt, *cache, table, seq, max(DEC_LENGTHS), o=o, lse=lse, scale=scale,
                               split_size=split)
    assert attn.attn_poll_status() == 0
    rows, extra, qk = decode_oracle(qd, seqs, scale, Hq, Hkv)
    # weights and codes in fp16, o in the type of q; a bf16 query's conversion to fp16 is off by at
    # most 2^-25 of the row's largest element
    eps_o = 2.0 ** (-7 if dtype == "bf16" else -10)
    el, ls = chunk.row_tolerance(rows, 2.0 ** -10, eps_o, 0.0,
                                 2.0 ** -24 * qk if dtype == "bf16" else 0.0)
    el = el + 0.5 * 2.0 ** -24 * extra
    chunk.check(o.float().cpu().numpy().reshape(-1, d), lse.cpu().numpy().reshape(-1), rows,
                (el, ls), f"page {page} d={d}")


def test_decode_with_scales_far_apart(attn):
    """Value scales from 2^-60 to 2^40 and key scales to match: nothing leaves its range."""
    import torch

    lengths, Hq, Hkv, d = [700, 65], 8, 2, 128
    cache, table, seqs = make_cache(lengths, Hkv, d, 64, 3)
    rng = np.random.default_rng(4)  # several splits, of scales that differ by head
    f = np.exp2(rng.integers(-60, 41, size=(2, Hkv))).astype(np.float64)  # per sequence and head
    pages = [table[b][: -(-lengths[b] // 64)].long() for b in range(2)]
    for b in range(2):
        for h in range(Hkv):
            cache[3][pages[b], h] *= float(f[b, h])
        vc, vs = seqs[1][b]
        seqs[1][b] = (vc, vs * f[b])
    q = syn.host_normal_bits((2, Hq, d), 5, "bf16", 4)
    qt = syn.bits_to_tensor(q, "bf16", "cuda")
    scale = 1.0 / np.sqrt(d) / 16.0
    seq = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o, lse = attn.attn_decode_paged_fp8(qt, *cache, table, seq, 700, scale=scale)
    assert attn.attn_poll_status() == 0
    rows, extra, qk = decode_oracle(bits_to_double(q, "bf16"), seqs, scale, Hq, Hkv)
    el, ls = chunk.row_tolerance(rows, 2.0 ** -10, 2.0 ** -7, 0.0, 2.0 ** -24 * qk)
    el = (el - 2.0 ** -25) + 0.5 * 2.0 ** -24 * extra  # no fp16 subnormals in a bf16 output
    chunk.check(o.double().cpu().numpy().reshape(-1, d), lse.cpu().numpy().reshape(-1), rows,
                (el, ls), "far scales")


def test_write_then_decode_equals_reading_back(attn):
    """A cache filled by writes (a prompt, then token by token), read back and decoded by the 16-bit
    kernel: the quantised decode gives the same rows within both kernels' rounding."""
    import torch

    lengths, Hq, Hkv, d, page = [200, 77], 16, 2, 128, 32
    dt = torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(3)
    ks = [torch.randn((n, Hkv, d), generator=g, device="cuda").to(dt) for n in lengths]
    vs = [torch.randn((n, Hkv, d), generator=g, device="cuda").to(dt) for n in lengths]
    q = torch.randn((2, Hq, d), generator=g, device="cuda").to(dt)
    table, n_pages, _, _ = syn.paged_layout(lengths, page, seed=1)
    tab = torch.from_numpy(table).cuda()
    cache = pool(n_pages, page, Hkv, d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    first = [150, 30]
    attn.attn_cache_write_fp8(torch.cat([x[:n] for x, n in zip(ks, first)]),
                              torch.cat([x[:n] for x, n in zip(vs, first)]), *cache, tab,
                              i32([0, 150, 180]), i32(first))
    n = list(first)
    while n != lengths:
        add = [int(a < b) for a, b in zip(n, lengths)]
        tok = lambda xs: torch.cat([x[m:m + a] for x, m, a in zip(xs, n, add)])
        kn, vn = tok(ks), tok(vs)
        n = [a + b for a, b in zip(n, add)]
        attn.attn_cache_write_fp8(kn, vn, *cache, tab, i32([0, add[0], add[0] + add[1]]), i32(n))
    cu = i32([0, lengths[0], sum(lengths)])
    k, v = attn.attn_cache_read_fp8(*cache, tab, cu, sum(lengths))
    o, lse = attn.attn_decode_paged_fp8(q, *cache, tab, i32(lengths), max(lengths))
    o2, lse2 = attn.attn_decode_splitkv(q, k, v, cu, max(lengths))
    assert attn.attn_poll_status() == 0
    big = o2.float().abs().amax(-1, keepdim=True)
    assert torch.all((o.float() - o2.float()).abs() <= 4 * 2.0 ** -8 * big + 1e-2)
    assert torch.all((lse - lse2).abs() <= 1e-4)
    # what was read back is what was written, within half an E4M3 step of it
    x = torch.cat(ks).float()
    assert torch.all((k.float() - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * x.abs().amax(-1, keepdim=True))


def test_cache_past_2_31_codes(attn):
    """Codes past byte 2^31 of the pool: written, read back and attended to as in a small pool."""
    import torch

    lengths, Hq, Hkv, d, page = [100, 333], 16, 8, 128, 64
    table, n_pages, _, _ = syn.paged_layout(lengths, page, seed=2)
    far = 2 ** 31 // (page * Hkv * d) + n_pages
    dt = torch.bfloat16
    k, v = (torch.randn((433, Hkv, d), device="cuda").to(dt) for _ in range(2))
    q = torch.randn((2, Hq, d), device="cuda").to(dt)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu, seq = i32([0, 100, 433]), i32(lengths)
    out = []
    for shift in (0, far - n_pages):
        cache = pool(n_pages + shift, page, Hkv, d)
        tab = torch.from_numpy(table).cuda()
        tab = torch.where(tab >= 0, tab + shift, tab)
        attn.attn_cache_write_fp8(k, v, *cache, tab, cu, seq)
        out.append([*attn.attn_cache_read_fp8(*cache, tab, cu, 433),
                    *attn.attn_decode_paged_fp8(q, *cache, tab, seq, 333)])
        assert attn.attn_poll_status() == 0
        del cache
    assert all(torch.equal(x, y) for x, y in zip(*out))
    torch.cuda.empty_cache()


def test_nothing_to_do(attn):
    import torch

    Hkv, d, page = 2, 64, 16
    cache = pool(2, page, Hkv, d)
    before = [x.clone() for x in cache]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    x = torch.ones((0, Hkv, d), dtype=torch.float16, device="cuda")
    attn.attn_cache_write_fp8(x, x, *cache, i32([[0], [1]]), i32([0, 0, 0]), i32([5, 0]))
    k, v = attn.attn_cache_read_fp8(*cache, i32([[0], [1]]), i32([0, 0, 0]), 0)
    assert k.shape == (0, Hkv, d) and attn.attn_poll_status() == 0
    for a, b in zip(cache, before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # every sequence empty
    q = torch.ones((2, 4, d), dtype=torch.float16, device="cuda")
    for most in (0, 16):
        o, lse = attn.attn_decode_paged_fp8(q, *cache, i32([[0], [1]]), i32([0, 0]), most)
        assert attn.attn_poll_status() == 0
        assert not o.any() and torch.isneginf(lse).all()


def test_bad_tables_are_reported(attn):
    import torch

    Hkv, d, page = 2, 64, 16
    cache = pool(4, page, Hkv, d)
    before = [x.clone() for x in cache]
    x = torch.ones((8, Hkv, d), dtype=torch.float16, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    cu = i32([0, 8])
    for tab, seq in ((i32([[4]]), 8), (i32([[-1]]), 8), (i32([[0]]), 24), (i32([[0]]), 7)):
        attn.attn_cache_write_fp8(x, x, *cache, tab, cu, i32([seq]))
        assert attn.attn_poll_status() == -8
        if seq != 7:
            for a, b in zip(cache, before):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    out = torch.full_like(x, 5.0)
    attn.attn_cache_read_fp8(*cache, i32([[9]]), cu, 8, k=out, v=out.clone())
    assert attn.attn_poll_status() == -8 and torch.all(out == 5.0)
    q = torch.ones((1, 4, d), dtype=torch.float16, device="cuda")
    attn.attn_decode_paged_fp8(q, *cache, i32([[9]]), i32([8]), 8)
    assert attn.attn_poll_status() == -8
    attn.attn_decode_paged_fp8(q, *cache, i32([[0]]), i32([9]), 8)
    assert attn.attn_poll_status() == -8


def test_graph_of_a_step(attn):
    """Write and decode captured together and replayed with other tokens and lengths."""
    import torch

    Hq, Hkv, d, page = 8, 2, 128, 16
    cache = pool(20, page, Hkv, d)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    tab = torch.randperm(20, device="cuda").to(torch.int32).view(2, 10).contiguous()
    x = torch.randn((2, Hkv, d), device="cuda").bfloat16()
    prompt = torch.randn((200, Hkv, d), device="cuda").bfloat16()
    attn.attn_cache_write_fp8(prompt, prompt, *cache, tab, i32([0, 100, 200]), i32([100, 100]))
    q = torch.randn((2, Hq, d), device="cuda").bfloat16()
    seq, cu = i32([101, 60]), i32([0, 1, 2])

    def step():
        attn.attn_cache_write_fp8(x, x, *cache, tab, cu, seq)
        return attn.attn_decode_paged_fp8(q, *cache, tab, seq, 160)

    eager = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(eager[0], out[0]) and torch.equal(eager[1], out[1])
    x.copy_(torch.randn_like(x))
    seq.copy_(i32([102, 61]))
    graph.replay()
    want = step()
    assert attn.attn_poll_status() == 0
    assert torch.equal(want[0], out[0]) and torch.equal(want[1], out[1])


def test_refusals(attn):
    import torch

    Hkv, d, page = 2, 64, 16
    cache = pool(4, page, Hkv, d)
    x = torch.ones((8, Hkv, d), dtype=torch.float16, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    tab, cu, seq = i32([[0]]), i32([0, 8]), i32([8])
    q = torch.ones((1, 4, d), dtype=torch.float16, device="cuda")
    E = attn.AttnError
    with pytest.raises(E):
        attn.attn_cache_write_fp8(x, x.bfloat16(), *cache, tab, cu, seq)
    with pytest.raises(E):
        attn.attn_cache_write_fp8(x.float(), x.float(), *cache, tab, cu, seq)
    with pytest.raises(E):
        attn.attn_cache_write_fp8(x, x, cache[0].view(torch.uint8), *cache[1:], tab, cu, seq)
    with pytest.raises(E):
        attn.attn_cache_write_fp8(x, x, *cache[:2], cache[2].transpose(1, 2), cache[3], tab, cu, seq)
    with pytest.raises(E):
        attn.attn_cache_write_fp8(x[:, :1], x[:, :1], *cache, tab, cu, seq)
    with pytest.raises(E):
        attn.attn_cache_write_fp8(x, x, *cache, tab, cu.long(), seq)
    with pytest.raises(E):
        attn.attn_cache_read_fp8(*cache, tab, cu, 8, dtype=torch.float32)
    with pytest.raises(E):
        attn.attn_decode_paged_fp8(q.bfloat16()[..., :32], *cache, tab, seq, 8)
    with pytest.raises(E):
        attn.attn_decode_paged_fp8(q, *cache, tab, seq, 17)      # past the table's reach
    with pytest.raises(E):
        attn.attn_decode_paged_fp8(q, *cache, tab, seq, 8, split_size=100)
    with pytest.raises(E):
        attn.attn_decode_paged_fp8(q, *cache, i32([[0] * 40]), seq, 640, split_size=64,
                                   workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------- value rows far apart within a head
def written(attn, ks, vs, page, dtype):
    """A cache that attn_cache_write_fp8 filled with the sequences ks, vs (float64 [L, Hkv, d], rounded
    to dtype), its table, the lengths, and each sequence's (codes, scale) of K and V as float64."""
    import torch

    lengths = [len(x) for x in ks]
    Hkv, d = ks[0].shape[1:]
    table, n_pages, _, _ = syn.paged_layout(lengths, page, seed=page)
    cache = pool(n_pages, page, Hkv, d)
    tab = torch.from_numpy(table).cuda()
    cu = syn.cu_seqlens(lengths)
    seq = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    bits = [syn.round_bits(np.concatenate(x).astype(np.float32), dtype) for x in (ks, vs)]
    attn.attn_cache_write_fp8(*(syn.bits_to_tensor(x, dtype, "cuda") for x in bits), *cache, tab,
                              torch.from_numpy(cu).cuda(), seq)
    seqs = []
    for x in bits:
        s, c = chunk.quantise(bits_to_double(x, dtype))
        seqs.append([(c[cu[b]:cu[b + 1]], s[cu[b]:cu[b + 1]]) for b in range(len(lengths))])
    return cache, tab, seq, seqs


def check_decode(attn, q, cache, tab, seq, seqs, Hkv, dtype, what, **kw):
    """The decode step against the definition over the dequantised cache.

    Tolerance: that of chunk.row_tolerance for weights of 11 bits, o's subnormals those of its own type
    (values may be as small as 2^-120).  A weight is held as 2^7 times its share of
    a reference that lies at most 2^8 below the largest p_j 2^(b_j) among the keys whose value row is not
    zero (a row of zeros has no part in O, whatever its scale) and never above it, so that what fp16's
    subnormals lose, 2^-25 at most, is 2^-32 of that largest one.  The value scale's exponent is added to
    the score and taken out again: numbers of up to 2^7, rounded by 2^-18 each."""
    B, Hq, d = q.shape
    G, scale = Hq // Hkv, 1.0 / np.sqrt(d)
    qt = syn.bits_to_tensor(q, dtype, "cuda")
    o, lse = attn.attn_decode_paged_fp8(qt, *cache, tab, seq, int(seq.max()), scale=scale, **kw)
    assert attn.attn_poll_status() == 0
    qd = bits_to_double(q, dtype)
    parts, sub = [], np.zeros((B * Hq, d))
    for b in range(B):
        (kc, ks), (vc, vs) = seqs[0][b], seqs[1][b]
        for h in range(Hq):
            k, v = (c[:, h // G] * s[:, h // G, None] for c, s in ((kc, ks), (vc, vs)))
            parts.append(chunk.attend(qd[b, h][None], k, v, np.array([len(k) - 1]), scale))
            x = scale * (k @ qd[b, h])
            p = np.exp(x - x.max())
            w = p / p.sum() * vs[:, h // G] * np.any(vc[:, h // G] != 0, axis=1)
            sub[b * Hq + h] = 2.0 ** -32 * w.max(initial=0.0) * np.abs(vc[:, h // G]).sum(axis=0)
    rows = chunk.Rows(*(np.concatenate(x) for x in zip(*parts)))
    qk = np.abs(qd).reshape(B * Hq, d).max(axis=1) * np.array(
        [scale * np.abs(seqs[0][b][0][:, h // G] * seqs[0][b][1][:, h // G, None]).sum(axis=1).max()
         for b in range(B) for h in range(Hq)])
    bf16 = dtype == "bf16"
    t = 2.0 ** -20 * rows.score + 2.0 ** -17 + (2.0 ** -24 * qk if bf16 else 0.0)
    el = (np.expm1(2.0 * t)[:, None] + 2.0 ** -11 + 2.0 ** -17) * rows.pv + sub
    el += 2.0 ** (-8 if bf16 else -11) * (np.abs(rows.o) + el) + 2.0 ** (-134 if bf16 else -25)
    ls = 2.0 * t + 2.0 ** -18 + 2.0 ** -21 * np.abs(rows.lse)
    chunk.check(o.double().cpu().numpy().reshape(-1, d), lse.cpu().numpy().reshape(-1), rows, (el, ls),
                what)


# one block, a cluster of them, the workspace (33 splits); two column tiles
@pytest.mark.parametrize("split", [0, 64, 2048])
@pytest.mark.parametrize("Hq,Hkv,d,dtype,std", [(8, 2, 128, "bf16", 0.02), (8, 2, 128, "bf16", 1e-4),
                                                (6, 1, 64, "bf16", 1e-6), (16, 1, 64, "f16", 0.02),
                                                (8, 2, 128, "f16", 1e-2)])
def test_decode_over_zero_value_rows(attn, Hq, Hkv, d, dtype, std, split):
    """Tokens whose value rows are zero (padding, null tokens) and score highest: they take most of the
    softmax and nothing of O, which the small values of the others make."""
    rng = np.random.default_rng(7)
    lengths = [2048, 333, 40, 1]
    q = syn.host_normal_bits((len(lengths), Hq, d), 5, dtype)
    qd = bits_to_double(q, dtype)
    ks, vs = [], []
    for b, n in enumerate(lengths):
        k, v = rng.standard_normal((n, Hkv, d)), std * rng.standard_normal((n, Hkv, d))
        zero = np.arange(min(16, n)) if b < 2 else np.arange(n)  # of b = 2, 3: every row
        zero = np.concatenate([zero, rng.integers(0, n, n // 100)])
        v[zero] = 0.0
        k[zero] = 0.7 * qd[b, ::Hq // Hkv][None]  # a score of about 0.7 sqrt(d) for one query head a group
        ks.append(k)
        vs.append(v)
    cache, tab, seq, seqs = written(attn, ks, vs, 64, dtype)
    check_decode(attn, q, cache, tab, seq, seqs, Hkv, dtype, f"zero rows, std {std}", split_size=split)


@pytest.mark.parametrize("split", [0, 64])
@pytest.mark.parametrize("Hq,Hkv,d,dtype,spread", [(8, 2, 128, "bf16", 15), (3, 3, 64, "f16", 7),
                                                   (16, 1, 128, "bf16", 60), (11, 1, 64, "bf16", 15)])
def test_decode_with_value_scales_per_token(attn, Hq, Hkv, d, dtype, spread, split):
    """Value rows whose magnitudes differ from token to token by up to 2^(2 spread)."""
    rng = np.random.default_rng(8)
    lengths = [1500, 90, 700]
    q = syn.host_normal_bits((len(lengths), Hq, d), 6, dtype)
    row = lambda n: np.exp2(rng.integers(-spread, spread + 1, size=(n, Hkv, 1)).astype(np.float64))
    ks = [rng.standard_normal((n, Hkv, d)) for n in lengths]
    vs = [rng.standard_normal((n, Hkv, d)) * row(n) for n in lengths]
    cache, tab, seq, seqs = written(attn, ks, vs, 16, dtype)
    check_decode(attn, q, cache, tab, seq, seqs, Hkv, dtype, f"2^+-{spread}", split_size=split)


@pytest.mark.parametrize("split", [0, 64])
@pytest.mark.parametrize("exponent", [-110, 87, 100, 112])
def test_decode_of_the_largest_and_smallest_values(attn, exponent, split):
    """bf16 values about 2^exponent, whose scales lie 7 below: any the writer makes is read."""
    rng = np.random.default_rng(9)
    q = syn.host_normal_bits((2, 8, 128), 7, "bf16")
    ks = [rng.standard_normal((n, 2, 128)) for n in (900, 20)]
    vs = [rng.standard_normal((n, 2, 128)) * 2.0 ** exponent for n in (900, 20)]
    cache, tab, seq, seqs = written(attn, ks, vs, 32, "bf16")
    check_decode(attn, q, cache, tab, seq, seqs, 2, "bf16", f"2^{exponent}", split_size=split)


@pytest.mark.parametrize("split", [0, 64])
def test_decode_keeps_what_is_not_finite(attn, split):
    """A value that is not finite (a NaN code) shows in its channel and no other; a key's in every channel
    of its sequence; what lies behind a sequence's end in none."""
    import torch

    rng = np.random.default_rng(11)
    n, Hq, Hkv, d = 700, 8, 2, 128
    ks, vs = ([rng.standard_normal((n, Hkv, d)) for _ in range(3)] for _ in range(2))
    vs[0][333, 1, 17] = np.inf
    ks[1][5, 0, 3] = np.nan
    cache, tab, seq, seqs = written(attn, ks, vs, 64, "bf16")
    q = syn.bits_to_tensor(syn.host_normal_bits((3, Hq, d), 3, "bf16"), "bf16", "cuda")
    o, lse = attn.attn_decode_paged_fp8(q, *cache, tab, seq, n, split_size=split)
    assert attn.attn_poll_status() == 0
    bad = torch.zeros_like(o, dtype=torch.bool)
    bad[0, 4:, 17] = True
    bad[1, :4] = True
    assert torch.equal(torch.isnan(o), bad)
    assert torch.equal(torch.isnan(lse), bad.all(-1))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Hq", [1, 16])
@pytest.mark.parametrize("base,lo,hi", [(2.0 ** 24, 16, 24), (2.0 ** 24, 16, 26), (2.0 ** 25, 8, 16), (2.0 ** 27, 16, 32),
                                        (-2.0 ** 24, 4, 12), (2.0 ** 23, 3, 11), (-2.0 ** 25, 16, 24)])
def test_decode_of_scores_far_from_zero(attn, base, lo, hi, Hq, dtype):
    """Scores of 10^7 and more whose differences are small, in whole log2 units and exact: base + lo at tokens
    0 .. 15, base + hi at token 64, which the same warp takes a stage later, base elsewhere.  A reference of
    the weights that fp32 rounds must not carry a weight past fp16.  Weights are powers of two: o is off by
    its rounding and half a step of each weight at most."""
    import torch

    B, L, d, page = 700, 200, 64, 64     # (as many sequences as leave each in one split; all of the same pages)
    x = np.zeros(L)
    x[:16], x[64] = lo, hi
    k = np.zeros((L, 1, d), dtype=np.float32)
    k[:, 0, 0], k[:, 0, 1] = base / 32768, x
    v = np.random.default_rng(3).standard_normal((L, 1, d)).astype(np.float32)
    v[..., 5] = 300.0                                           # a value scale of 1: no exponent to add to a score
    bits = [syn.round_bits(a, "f16") for a in (k, v)]
    ks, kv = chunk.quantise(k.astype(np.float64))
    assert np.array_equal(ks[..., None] * kv, k.astype(np.float64)), "the keys have to be exact"
    vs, vv = chunk.quantise(bits_to_double(bits[1], "f16"))
    assert (vs == 1.0).all()
    val = vv[:, 0]
    n_pages = -(-L // page)
    cache = pool(n_pages, page, 1, d)
    i32 = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32), device="cuda")
    row = np.arange(n_pages)[None]
    attn.attn_cache_write_fp8(*(syn.bits_to_tensor(b, "f16", "cuda") for b in bits), *cache, i32(row), i32([0, L]),
                              i32([L]))
    q = torch.zeros((B, Hq, d), dtype=syn.torch_dtype(dtype), device="cuda")
    q[..., 0], q[..., 1] = 32768.0, 1.0
    scale = float(np.float32(np.log(2.0)))                      # (times log2 e in fp32: 1)
    o, lse = attn.attn_decode_paged_fp8(q, *cache, i32(np.tile(row, (B, 1))), i32([L] * B), L, scale=scale)
    assert attn.attn_poll_status() == 0
    w = np.exp2(x - hi)
    want, size = (w @ val) / w.sum(), (w @ np.abs(val)) / w.sum()
    # (half a step of a weight below fp16's normal numbers is 2^-32 of the largest)
    lim = (2.0 ** -11 + 2.0 ** -17) * size + 2.0 ** -32 * np.abs(val).sum(0)
    eps = 2.0 ** -11 if dtype == "f16" else 2.0 ** -8
    lim = lim + eps * (np.abs(want) + lim) + 2.0 ** -25
    got = o.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= lim).all()
    ref = (base + hi + np.log2(w.sum())) * np.log(2.0)
    assert (np.abs(lse.double().cpu().numpy() - ref) <= 2.0 ** -22 * abs(ref)).all()
