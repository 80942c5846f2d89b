"""GPU parity of the sliding window with sinks, forward and backward, against fp64 definitions.

attn_fwd_window_sinks: key j visible to row i, p = i + N_kv - N_q, iff j <= p and (p - j <= W or
j < s).  The forward tolerance is derived in oracle/chunk.py (row_tolerance), the gradients' in
oracle/backward.py (error_scales); the gradients are also tested against differences of the
forward definition.  Shapes cover sinks inside one key tile, across tiles, reaching into the window
and past the sequence, rows without keys, one row, ragged ends, grouped heads and more work items
than SMs.
"""
import numpy as np
import pytest

import synthetic as syn
from oracle import bits_to_double, chunk
from oracle.backward import attention_backward
from parity import check_grad

pytestmark = pytest.mark.gpu

EPS = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24}


@pytest.fixture(scope="module")
def attn():
    import exact_io_aware_09_gb300 as m

    return m


CASES = [
    # (B, Hq, Hkv, N_q, N_kv, d, dtype), W, sinks
    ((1, 2, 1, 1, 1, 64, "f16"), 0, 1),
    ((1, 2, 2, 300, 300, 64, "bf16"), 0, 4),
    ((1, 2, 1, 700, 700, 128, "f16"), 100, 1),
    ((2, 4, 2, 200, 933, 64, "bf16"), 100, 128),    # a whole sink tile, N_kv > N_q
    ((1, 2, 2, 900, 900, 128, "bf16"), 128, 130),   # sinks across two tiles
    ((1, 3, 1, 1017, 1017, 128, "f16"), 300, 500),  # sinks reach into the window of early rows
    ((1, 2, 2, 400, 100, 64, "f16"), 50, 7),        # N_kv < N_q: top rows see no key
    ((1, 2, 1, 1, 777, 128, "bf16"), 200, 4),       # one row
    ((1, 2, 2, 600, 600, 128, "bf16"), 5000, 9),    # wider than the sequence: causal
    ((1, 2, 2, 500, 500, 64, "bf16"), 30, 9999),    # every key a sink: causal
    ((2, 96, 8, 520, 520, 128, "bf16"), 127, 4),    # more items than SMs
    ((2, 30, 6, 777, 777, 64, "f16"), 200, 64),
    # few query tiles that see many keys, and many that do: the prefill kernel's variant
    ((1, 2, 1, 1300, 1300, 64, "bf16"), 1000, 5),
    ((1, 2, 1, 300, 2300, 128, "f16"), 1500, 129),
    ((1, 16, 2, 1500, 4500, 128, "bf16"), 4000, 4),
]
ids = lambda x: str(x)


def _inputs(shape, seed):
    B, Hq, Hkv, Nq, Nkv, d, dt = shape
    cfg = syn.PrefillConfig("sinks", B, Hq, Hkv, Nq, Nkv, d, dt, True, seed)
    return cfg, cfg.host_inputs()


def _oracle(cfg, q, k, v, W, s):
    q, k, v = (bits_to_double(x, cfg.dtype) for x in (q, k, v))
    pos = np.arange(cfg.N_q) + cfg.N_kv - cfg.N_q
    G = cfg.Hq // cfg.Hkv
    heads = [chunk.attend(q[b, h], k[b, h // G], v[b, h // G], pos, cfg.scale, W, s)
             for b in range(cfg.B) for h in range(cfg.Hq)]
    return chunk.Rows(*(np.stack(x) for x in zip(*heads)))


def _check(cfg, o, lse, rows, what):
    e = EPS[cfg.dtype]
    tol = chunk.row_tolerance(rows, e, e, TINY[cfg.dtype])
    chunk.check(o.float().cpu().numpy().reshape(rows.o.shape),
                lse.cpu().numpy().reshape(rows.lse.shape), rows, tol, what)


@pytest.mark.parametrize("shape,W,s", CASES, ids=ids)
def test_forward(attn, shape, W, s):
    import torch

    cfg, (q, k, v) = _inputs(shape, 900 + W + s + sum(shape[:6]))
    qt, kt, vt = (syn.bits_to_tensor(x, cfg.dtype, "cuda") for x in (q, k, v))
    o = torch.full_like(qt, float("nan"))
    lse = torch.full(qt.shape[:3], float("nan"), device="cuda")
    attn.attn_fwd_window_sinks(qt, kt, vt, W, s, o=o, lse=lse, scale=cfg.scale)
    assert attn.attn_poll_status() == 0
    _check(cfg, o, lse, _oracle(cfg, q, k, v, W, s), f"{shape} W={W} sinks={s}")


@pytest.mark.parametrize("shape,W,s", CASES, ids=ids)
def test_backward(attn, shape, W, s):
    import torch

    cfg, (q, k, v) = _inputs(shape, 1300 + W + s + sum(shape[:6]))
    do = syn.host_normal_bits(q.shape, 77 + s, cfg.dtype)
    qt, kt, vt, dot = (syn.bits_to_tensor(x, cfg.dtype, "cuda") for x in (q, k, v, do))
    o, lse = attn.attn_fwd_window_sinks(qt, kt, vt, W, s, scale=cfg.scale)
    nan = lambda t: torch.full_like(t, float("nan"))
    got = attn.attn_bwd_window_sinks(qt, kt, vt, o, dot, lse, W, s, scale=cfg.scale, dq=nan(qt),
                                     dk=nan(kt), dv=nan(vt))
    assert attn.attn_poll_status() == 0
    r = attention_backward(q, k, v, do, cfg.dtype, cfg.B, cfg.Hq, cfg.Hkv, cfg.N_q, cfg.N_kv, cfg.d,
                           True, cfg.scale, window=W, sinks=s, error_scales=True)
    for i, name in enumerate(("dq", "dk", "dv")):
        check_grad(name, got[i].float().cpu().numpy(), r[i], r[5].row[i], r[5].elem[i], cfg.dtype,
                   f"{shape} W={W} sinks={s}")
    again = attn.attn_bwd_window_sinks(qt, kt, vt, o, dot, lse, W, s, scale=cfg.scale)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


MANY = [
    # d = 64 with enough tiles for the gradient kernels of two blocks an SM
    ((8, 96, 96, 33, 33, 64, "f16"), 10, 3),
    ((8, 96, 96, 1, 130, 64, "bf16"), 64, 64),      # one row
    ((4, 64, 64, 200, 333, 64, "bf16"), 100, 0),    # N_kv > N_q
    ((4, 128, 64, 333, 300, 64, "bf16"), 90, 7),    # top rows see no key, grouped heads
    ((2, 130, 130, 300, 300, 64, "f16"), 5000, 9),  # causal
    ((2, 40, 10, 700, 700, 64, "bf16"), 200, 150),  # dQ alone
]


@pytest.mark.parametrize("shape,W,s", MANY, ids=ids)
def test_backward_with_many_tiles(attn, shape, W, s):
    test_backward(attn, shape, W, s)


def test_sink_tiles_cut_in_parts_with_many_tiles(attn):
    """The first key tile's query steps in several blocks, next to 800 short ones: four heads."""
    import torch

    shape, W, s = (1, 48, 48, 2100, 2100, 64, "bf16"), 100, 4
    cfg, (q, k, v) = _inputs(shape, 4501)
    do = syn.host_normal_bits(q.shape, 4502, cfg.dtype)
    t = [syn.bits_to_tensor(x, cfg.dtype, "cuda") for x in (q, k, v, do)]
    need = attn.attn_bwd_window_sinks_workspace_bytes(*shape[:6], W, s)
    assert need > attn.attn_bwd_window_sinks_workspace_bytes(*shape[:6], W, 0)  # partial sums
    o, lse = attn.attn_fwd_window_sinks(*t[:3], W, s, scale=cfg.scale)
    got = attn.attn_bwd_window_sinks(*t[:3], o, t[3], lse, W, s, scale=cfg.scale)
    assert attn.attn_poll_status() == 0
    hs = [0, 17, 31, 47]
    part = [np.ascontiguousarray(x[:, hs]) for x in (q, k, v, do)]
    r = attention_backward(*part, cfg.dtype, 1, 4, 4, 2100, 2100, 64, True, cfg.scale, window=W,
                           sinks=s, error_scales=True)
    for i, (name, g) in enumerate(zip(("dq", "dk", "dv"), got)):
        check_grad(name, g[:, hs].float().cpu().numpy(), r[i], r[5].row[i], r[5].elem[i], cfg.dtype,
                   "parts")
    assert all(bool(torch.isfinite(g).all()) for g in got)


def test_gradient_against_differences(attn):
    """The directional derivative of sum(do * o) along random directions, by central differences of
    the fp64 definition, against the GPU gradients: each gradient g lies within the row scales'
    norms of the exact one, so <g, u> lies within their product with |u|."""
    W, s = 40, 3
    cfg, (q, k, v) = _inputs((1, 2, 1, 150, 150, 64, "f16"), 5)
    do = syn.host_normal_bits(q.shape, 6, cfg.dtype)
    t = [syn.bits_to_tensor(x, cfg.dtype, "cuda") for x in (q, k, v, do)]
    o, lse = attn.attn_fwd_window_sinks(*t[:3], W, s, scale=cfg.scale)
    grads = attn.attn_bwd_window_sinks(*t[:3], o, t[3], lse, W, s, scale=cfg.scale)
    assert attn.attn_poll_status() == 0
    r = attention_backward(q, k, v, do, cfg.dtype, 1, 2, 1, 150, 150, 64, True, cfg.scale, window=W,
                           sinks=s, error_scales=True)
    x = [bits_to_double(b, cfg.dtype) for b in (q, k, v)]
    dod = bits_to_double(do, cfg.dtype)
    pos = np.arange(150)

    def loss(q_, k_, v_):
        return sum(float((dod[0, h] * chunk.attend(q_[0, h], k_[0, 0], v_[0, 0], pos, cfg.scale, W,
                                                   s).o).sum()) for h in range(2))

    rng = np.random.default_rng(3)
    for i in range(3):
        u = rng.standard_normal(x[i].shape)
        step = 2.0 ** -14
        args = lambda sign: [x[n] + sign * step * u if n == i else x[n] for n in range(3)]
        slope = (loss(*args(1.0)) - loss(*args(-1.0))) / (2.0 * step)
        g = grads[i].double().cpu().numpy()
        err = 2.0 * r[5].row[i] + 1e-2 * np.linalg.norm(r[i], axis=-1) + 1e-6
        # the differences' own error: step^2 times the third derivative, below 1e-3 here
        assert abs(float((g * u).sum()) - slope) <= float((err * np.linalg.norm(u, axis=-1)).sum()) + 1e-3


@pytest.mark.parametrize("d", [64, 128])
def test_no_sinks_is_the_window(attn, d):
    import torch

    cfg, (q, k, v) = _inputs((1, 4, 2, 600, 600, d, "bf16"), 21)
    t = [syn.bits_to_tensor(x, cfg.dtype, "cuda") for x in (q, k, v)]
    a = attn.attn_fwd_window(*t, 200, scale=cfg.scale)
    o, lse = attn.attn_fwd_window_sinks(*t, 200, 0, scale=cfg.scale)
    assert attn.attn_poll_status() == 0
    # both within half a step of O and their weights' half steps of it: 4 half steps of the row's
    # largest value and of its largest weighted |v| (at most about 5 here)
    big = a[0].float().abs().amax(-1, keepdim=True)
    assert torch.all((o.float() - a[0].float()).abs() <= 4 * 2.0 ** -8 * (big + 5.0))
    assert torch.all((lse - a[1]).abs() <= 1e-4)
    _check(cfg, o, lse, _oracle(cfg, q, k, v, 200, 0), "no sinks")


@pytest.mark.parametrize("d", [64, 128])
def test_wide_window_backward_is_the_causal_one(attn, d):
    import torch

    cfg, (q, k, v) = _inputs((1, 4, 2, 600, 600, d, "bf16"), 22)
    t = [syn.bits_to_tensor(x, cfg.dtype, "cuda") for x in (q, k, v)]
    do = torch.randn_like(t[0])
    o, lse = attn.attn_fwd(*t, causal=True, scale=cfg.scale)
    a = attn.attn_bwd(*t, o, do, lse, causal=True, scale=cfg.scale)
    b = attn.attn_bwd_window_sinks(*t, o, do, lse, 2 ** 31 - 1, 0, scale=cfg.scale)
    assert attn.attn_poll_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("nq,nkv", [(600, 600), (900, 300)])
def test_largest_window_and_sinks_are_all_keys(attn, nq, nkv):
    """2^31 - 1 of either: the causal result and gradients, rows without keys among them."""
    import torch

    cfg, (q, k, v) = _inputs((1, 4, 2, nq, nkv, 128, "bf16"), 23)
    t = [syn.bits_to_tensor(x, cfg.dtype, "cuda") for x in (q, k, v)]
    do = torch.randn_like(t[0])
    o, lse = attn.attn_fwd(*t, causal=True, scale=cfg.scale)
    g = attn.attn_bwd(*t, o, do, lse, causal=True, scale=cfg.scale)
    rows = _oracle(cfg, q, k, v, -1, 0)
    big = 2 ** 31 - 1
    for W, s in ((big, 0), (big, big), (0, big)):
        a, l = attn.attn_fwd_window_sinks(*t, W, s, scale=cfg.scale)
        assert attn.attn_poll_status() == 0
        _check(cfg, a, l, rows, f"W={W} sinks={s}")
        h = attn.attn_bwd_window_sinks(*t, o, do, lse, W, s, scale=cfg.scale)
        assert attn.attn_poll_status() == 0
        # the same products in other groups of tiles: sums of them in fp32, rounded once
        for x, y in zip(g, h):
            lim = 2.0 ** -7 * x.float().abs() + 2.0 ** -12 * x.float().abs().amax()
            assert torch.all((x.float() - y.float()).abs() <= lim)


def test_past_2_31_elements_sampled(attn):
    """Q, O, dO and dQ of 2.29e9 elements under a narrow window: sampled rows against a one-row
    problem over the keys the row sees."""
    import torch

    W, s = 200, 5
    cfg = syn.PrefillConfig("big", 1, 128, 8, 140000, 140000, 128, "bf16", True, 6201)
    q, k, v = cfg.device_inputs("cuda")
    do = syn.device_normal(q.shape, cfg.seed + 7, cfg.dtype, "cuda")
    o, lse = attn.attn_fwd_window_sinks(q, k, v, W, s, scale=cfg.scale)
    dq, dk, dv = attn.attn_bwd_window_sinks(q, k, v, o, do, lse, W, s, scale=cfg.scale)
    assert attn.attn_poll_status() == 0
    bits = lambda t: syn.tensor_to_bits(t.contiguous())
    for h in (0, 61, cfg.Hq - 1):
        for i in (0, 3, 127, 128, 204, 100001, cfg.N_q - 1):
            keys = sorted(set(range(max(0, i - W), i + 1)) | set(range(min(s, i + 1))))
            kr, vr = bits(k[0, h // 16][keys]), bits(v[0, h // 16][keys])
            qr, dor = bits(q[0, h, i:i + 1]), bits(do[0, h, i:i + 1])
            rq, _, _, _, _, sc = attention_backward(qr, kr, vr, dor, cfg.dtype, 1, 1, 1, 1, len(keys),
                                                    cfg.d, False, cfg.scale, error_scales=True)
            got = dq[0, h, i].float().cpu().numpy().reshape(1, 1, 1, cfg.d)
            check_grad("dq", got, rq, sc.row[0], sc.elem[0], cfg.dtype, f"head {h} row {i}")
            x = [bits_to_double(b, cfg.dtype) for b in (qr, kr, vr)]
            rows = chunk.attend(x[0], x[1], x[2], [len(keys) - 1], cfg.scale)
            _check(cfg, o[0, h, i], lse[0, h, i], rows, f"head {h} row {i}")
    del q, k, v, do, o, lse, dq, dk, dv
    torch.cuda.empty_cache()


@pytest.mark.parametrize("nq,nkv", [(0, 300), (300, 0)], ids=["no_queries", "no_keys"])
def test_empty_side(attn, nq, nkv):
    import torch

    q = torch.randn((2, 4, nq, 64), device="cuda").half()
    k = torch.randn((2, 2, nkv, 64), device="cuda").half()
    o, lse = attn.attn_fwd_window_sinks(q, k, k, 10, 4)
    grads = attn.attn_bwd_window_sinks(q, k, k, o, q, lse, 10, 4)
    assert attn.attn_poll_status() == 0
    assert not o.any() and torch.isneginf(lse).all() and not any(g.any() for g in grads)


@pytest.mark.parametrize("d", [64, 128])
def test_masked_scores_that_are_not_finite(attn, d):
    """Keys outside every row's mask share tiles with visible ones and give infinite and NaN scores:
    the rows are those of finite keys in their place.  Their values stay finite."""
    import torch

    W, s = 70, 5
    cfg, (q, k, v) = _inputs((1, 2, 1, 100, 900, d, "bf16"), 31)
    t = [syn.bits_to_tensor(x, cfg.dtype, "cuda") for x in (q, k, v)]
    a = attn.attn_fwd_window_sinks(*t, W, s, scale=cfg.scale)
    pos0 = 800  # row 0 sees keys 0-4 and 730-800
    t[1][:, :, s:pos0 - W] = float("nan")
    t[1][:, :, s + 1:pos0 - W:3] = float("inf")
    b = attn.attn_fwd_window_sinks(*t, W, s, scale=cfg.scale)
    assert attn.attn_poll_status() == 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("shape,W,s", [((1, 64, 8, 8192, 8192, 128, "bf16"), 1024, 4)], ids=ids)
def test_full_size(attn, shape, W, s):
    """The long grouped-query prefill under the 1024-key window, and its gradients: the eight query
    heads of one key/value head."""
    cfg, (q, k, v) = _inputs(shape, 4001)
    do = syn.host_normal_bits(q.shape, 4002, cfg.dtype)
    t = [syn.bits_to_tensor(x, cfg.dtype, "cuda") for x in (q, k, v, do)]
    o, lse = attn.attn_fwd_window_sinks(*t[:3], W, s, scale=cfg.scale)
    got = attn.attn_bwd_window_sinks(*t[:3], o, t[3], lse, W, s, scale=cfg.scale)
    assert attn.attn_poll_status() == 0
    hk = 5
    qs = slice(hk * 8, hk * 8 + 8)
    part = [np.ascontiguousarray(x) for x in (q[:, qs], k[:, hk:hk + 1], v[:, hk:hk + 1], do[:, qs])]
    r = attention_backward(*part, cfg.dtype, 1, 8, 1, 8192, 8192, 128, True, cfg.scale, window=W,
                           sinks=s, error_scales=True)
    for i, (name, g) in enumerate(zip(("dq", "dk", "dv"), got)):
        g = g[:, qs] if i == 0 else g[:, hk:hk + 1]
        check_grad(name, g.float().cpu().numpy(), r[i], r[5].row[i], r[5].elem[i], cfg.dtype, "8192")
    sub = syn.PrefillConfig("one", 1, 2, 1, 8192, 8192, 128, "bf16", True, 0)
    rows = _oracle(sub, part[0][:, :2], part[1], part[2], W, s)
    _check(cfg, o[:, qs][:, :2], lse[:, qs][:, :2], rows, "8192")


def test_two_streams_and_a_graph(attn):
    """Calls on a side stream, captured and replayed on new inputs: the same bits as eager calls."""
    import torch

    cfg, (q, k, v) = _inputs((1, 4, 2, 500, 500, 128, "bf16"), 41)
    t = [syn.bits_to_tensor(x, cfg.dtype, "cuda") for x in (q, k, v)]
    do = torch.randn_like(t[0])

    def step():
        o, lse = attn.attn_fwd_window_sinks(*t, 100, 4)
        return (o, lse, *attn.attn_bwd_window_sinks(*t, o, do, lse, 100, 4))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, out))
    t[0].copy_(torch.randn_like(t[0]))
    graph.replay()
    want = step()
    assert attn.attn_poll_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(want, out))


def test_refusals(attn):
    import torch

    q = torch.zeros((1, 2, 128, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((1, 2, 128), device="cuda")
    for W, s in ((-1, 4), (10, -1)):
        with pytest.raises(attn.AttnError):
            attn.attn_fwd_window_sinks(q, q, q, W, s)
        with pytest.raises(attn.AttnError):
            attn.attn_bwd_window_sinks(q, q, q, q, q, lse, W, s)
    with pytest.raises(attn.AttnError):
        attn.attn_fwd_window_sinks(q, q, q, 10, 4, o=q.half())
    with pytest.raises(attn.AttnError):
        attn.attn_fwd_window_sinks(q, q, q, 10, 4, lse=lse[:, :, :9])
    with pytest.raises(attn.AttnError):
        attn.attn_bwd_window_sinks(q, q, q, q, q.half(), lse, 10, 4)
    with pytest.raises(attn.AttnError):
        attn.attn_bwd_window_sinks(q, q, q, q, q, lse[:, :, :5], 10, 4)
    with pytest.raises(attn.AttnError):
        attn.attn_bwd_window_sinks(q, q, q, q, q, lse, 10, 4,
                                   workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


def test_many_shapes_hold_no_host_memory(attn):
    """What the backward launcher keeps of a shape (the order of its blocks) is bounded: 3,000 masks of
    160 heads, 4 KB each, leave less than half of that behind."""
    import os

    import torch

    q, k, v, do = (torch.randn((1, 160, 64, 64), device="cuda").bfloat16() for _ in range(4))
    grads = [torch.empty_like(x) for x in (q, k, v)]
    ws = torch.empty(attn.attn_bwd_window_sinks_workspace_bytes(1, 160, 160, 64, 64, 64, 0, 64) * 4,
                     device="cuda", dtype=torch.uint8)
    o, lse = attn.attn_fwd_window_sinks(q, k, v, 3, 2)

    def step(w, s):
        attn.attn_bwd_window_sinks(q, k, v, o, do, lse, w, s, dq=grads[0], dk=grads[1], dv=grads[2],
                                   workspace=ws)

    def resident():
        with open("/proc/self/statm") as f:
            return int(f.read().split()[1]) * os.sysconf("SC_PAGE_SIZE")

    step(3, 2)
    first = [x.clone() for x in grads]
    torch.cuda.synchronize()
    before = resident()
    for w in range(4, 54):
        for s in range(60):
            step(w, s)
    torch.cuda.synchronize()
    assert resident() - before < 6 << 20
    step(3, 2)  # forgotten meanwhile: the same bits
    assert attn.attn_poll_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(first, grads))
