"""Gradients whose incoming gradient, values or weights are far from 1 (attn_bwd and
attn_bwd_window_sinks, fp16): the products' 16-bit operands must not fall into fp16's subnormals, nor
past its largest number, where the gradients themselves are ordinary numbers.

Tolerance, per gradient and over all its elements: P and dS are rounded once for their products, O once
as the forward stores it (the reference takes D from that O), and the gradient once, each by at most
half a step, 2^-11 of the value.  The roundings are independent, so over the 10^5 and more terms here
their squares add up: sqrt(2) 2^-11 of the gradient's norm where its terms' signs are as random as these
inputs make them.  2^-10 is allowed, and half a subnormal step, 2^-25, for each element of the result.
"""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    import exact_io_aware_09_gb300 as m

    return m


def visible(nq, nkv, causal, window, sinks):
    import torch

    p = torch.arange(nq, device="cuda")[:, None] + (nkv - nq)
    j = torch.arange(nkv, device="cuda")[None, :]
    if window is not None:
        return (j <= p) & ((p - j <= window) | (j < sinks))
    return (j <= p) if causal else torch.ones_like(j <= p)


def reference(q, k, v, o, do, vis, scale):
    """(dq, dk, dv) in 64 bits, D from o as stored."""
    import torch

    B, Hq = q.shape[:2]
    G = Hq // k.shape[1]
    dq, dk, dv = (torch.zeros_like(t, dtype=torch.float64) for t in (q, k, v))
    for b in range(B):
        for h in range(Hq):
            qh, kh, vh, oh, gh = (t.double() for t in (q[b, h], k[b, h // G], v[b, h // G], o[b, h], do[b, h]))
            s = (scale * (qh @ kh.T)).masked_fill(~vis, -math.inf)
            m = s.amax(1, keepdim=True)
            e = torch.exp(s - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
            p = e / e.sum(1, keepdim=True).clamp_min(1e-300)
            ds = p * (gh @ vh.T - (gh * oh).sum(1, keepdim=True))
            dq[b, h] = scale * (ds @ kh)
            dk[b, h // G] += scale * (ds.T @ qh)
            dv[b, h // G] += p.T @ gh
    return dq, dk, dv


def inputs(B, Hq, Hkv, nq, nkv, d, seed, do_exp=0, v_exp=0, dtype="float16"):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    dt = getattr(torch, dtype)
    return (rnd(B, Hq, nq, d).to(dt), rnd(B, Hkv, nkv, d).to(dt),
            (rnd(B, Hkv, nkv, d) * 2.0 ** v_exp).to(dt), (rnd(B, Hq, nq, d) * 2.0 ** do_exp).to(dt))


def gradients(attn, q, k, v, do, causal=True, window=None, sinks=0):
    if window is None:
        o, lse = attn.attn_fwd(q, k, v, causal=causal)
        got = attn.attn_bwd(q, k, v, o, do, lse, causal=causal)
    else:
        o, lse = attn.attn_fwd_window_sinks(q, k, v, window, sinks)
        got = attn.attn_bwd_window_sinks(q, k, v, o, do, lse, window, sinks)
    assert attn.attn_poll_status() == 0
    vis = visible(q.shape[2], k.shape[2], causal, window, sinks)
    return got, reference(q, k, v, o, do, vis, 1.0 / math.sqrt(q.shape[3]))


def check(name, got, ref, what):
    import torch

    assert torch.isfinite(got).all(), f"{what}: non-finite {name}"
    err = float((got.double() - ref).norm())
    lim = 2.0 ** -10 * float(ref.norm()) + math.sqrt(ref.numel()) * 2.0 ** -25
    assert err <= lim, f"{what}: {name} off by {err / float(ref.norm()):.2e} of its norm, {err / lim:.2f} times the tolerance"


SHAPES = [
    # (B, Hq, Hkv, N_q, N_kv, d), causal, window, sinks
    ((1, 4, 2, 2048, 2048, 128), True, 1024, 4),    # key tiles with sinks cut in parts
    ((1, 8, 8, 1024, 1024, 64), True, 256, 4),
    ((8, 12, 12, 1024, 1024, 64), True, 256, 4),    # two blocks on an SM
    ((1, 4, 4, 500, 333, 64), True, 100, 0),        # top rows see no key
    ((1, 4, 2, 1024, 1024, 128), True, None, 0),
    ((1, 4, 4, 777, 900, 64), False, None, 0),
]
ids = lambda x: str(x)


@pytest.mark.parametrize("do_exp,v_exp", [(0, 0), (-10, 0), (-10, 4), (8, 6)])
@pytest.mark.parametrize("shape,causal,window,sinks", SHAPES, ids=ids)
def test_scaled_incoming_gradient(attn, shape, causal, window, sinks, do_exp, v_exp):
    x = inputs(*shape, 3, do_exp, v_exp)
    got, ref = gradients(attn, *x, causal, window, sinks)
    for name, a, b in zip(("dq", "dk", "dv"), got, ref):
        check(name, a, b, f"{shape} W={window} dO 2^{do_exp} V 2^{v_exp}")


@pytest.mark.parametrize("shape,causal,window,sinks", [SHAPES[0], SHAPES[2], SHAPES[4]], ids=ids)
def test_rows_and_sequences_of_different_size(attn, shape, causal, window, sinks):
    """A sequence whose incoming gradient is 2^-10 of the other's; in the other, later rows of 2^-8."""
    import torch

    shape = (2,) + shape[1:]
    q, k, v, do = inputs(*shape, 4)
    half = shape[3] // 2
    do[1] *= 2.0 ** -10
    do[0, :, half:] *= 2.0 ** -8
    got, ref = gradients(attn, q, k, v, do, causal, window, sinks)
    for b in range(2):
        for name, a, r in zip(("dq", "dk", "dv"), got, ref):
            check(name, a[b], r[b], f"sequence {b}")
    check("dq", got[0][0, :, half:], ref[0][0, :, half:], "later rows")
    again = attn.attn_bwd(q, k, v, q, torch.zeros_like(do), torch.zeros(q.shape[:3], device="cuda"))
    assert not any(t.any() for t in again)  # a zero gradient gives zeros


def test_weights_of_a_long_row(attn):
    """131,072 keys a row: weights about 2^-17."""
    x = inputs(1, 2, 1, 64, 131072, 64, 5)
    got, ref = gradients(attn, *x, False)
    for name, a, b in zip(("dq", "dk", "dv"), got, ref):
        check(name, a, b, "long rows")


@pytest.mark.parametrize("window", [None, 300])
def test_replayed_with_a_smaller_gradient(attn, window):
    """A captured backward pass takes the ranges of what it is replayed on: a large dO first, then one of
    2^-10 in the same buffers, the same bits as eager calls."""
    import torch

    q, k, v, do = inputs(1, 4, 2, 600, 600, 128, 6, 6)
    if window is None:
        o, lse = attn.attn_fwd(q, k, v, causal=True)
        step = lambda: attn.attn_bwd(q, k, v, o, do, lse, causal=True)
    else:
        o, lse = attn.attn_fwd_window_sinks(q, k, v, window, 4)
        step = lambda: attn.attn_bwd_window_sinks(q, k, v, o, do, lse, window, 4)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        do.mul_(2.0 ** -16)
    assert attn.attn_poll_status() == 0
