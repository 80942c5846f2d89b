"""A call handed a busy stream, everything it needs allocated inside: what the current stream allocates
and fills while the call waits leaves its results alone."""

import pytest

import synthetic as syn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    import exact_io_aware_09_gb300 as m

    return m


def cases(attn):
    """name -> (a call that returns tensors, the bytes of its workspace)."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s, dt=torch.bfloat16: torch.randn(s, generator=g, device="cuda").to(dt)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q, do, k, v = rnd(1, 8, 700, 128), rnd(1, 8, 700, 128), rnd(1, 2, 700, 128), rnd(1, 2, 700, 128)
    o, lse = attn.attn_fwd(q, k, v, causal=True)
    ow, lw = attn.attn_fwd_window_sinks(q, k, v, 200, 4)
    lengths = [3000, 5000]
    table, n_pages, _, _ = syn.paged_layout(lengths, 64, seed=2)
    tab, seq = torch.from_numpy(table).cuda(), i32(lengths)
    kp, vp = rnd(n_pages, 64, 2, 128), rnd(n_pages, 64, 2, 128)
    tok = rnd(2, 16, 128)
    cu = i32([0, 3000, 8000])
    kc, vc = rnd(8000, 2, 128), rnd(8000, 2, 128)
    codes = [torch.zeros((n_pages, 64, 2, 128), device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    cache = (*codes, *(torch.ones((n_pages, 2, 64), device="cuda") for _ in range(2)))
    attn.attn_cache_write_fp8(kc, vc, *cache, tab, cu, seq)
    ws = attn.attn_decode_workspace_bytes(2, 16, 5000, 512, 128)
    return {
        "attn_fwd": (lambda **kw: attn.attn_fwd(q, k, v, causal=True, **kw), 0),
        "attn_fwd_window": (lambda **kw: attn.attn_fwd_window(q, k, v, 200, **kw), 0),
        "attn_fwd_fp8": (lambda **kw: attn.attn_fwd_fp8(q, k, v, causal=True, **kw),
                         attn.attn_fwd_fp8_workspace_bytes(1, 8, 2, 700, 700, 128)),
        "attn_bwd": (lambda **kw: attn.attn_bwd(q, k, v, o, do, lse, causal=True, **kw),
                     attn.attn_bwd_workspace_bytes(1, 8, 700)),
        "attn_bwd_window_sinks": (
            lambda **kw: attn.attn_bwd_window_sinks(q, k, v, ow, do, lw, 200, 4, **kw),
            attn.attn_bwd_window_sinks_workspace_bytes(1, 8, 2, 700, 700, 128, 200, 4)),
        "attn_decode_paged": (lambda **kw: attn.attn_decode_paged(tok, kp, vp, tab, seq, 5000, **kw), ws),
        "attn_decode_splitkv": (lambda **kw: attn.attn_decode_splitkv(tok, kc, vc, cu, 5000, **kw), ws),
        "attn_decode_paged_fp8": (
            lambda **kw: attn.attn_decode_paged_fp8(tok, *cache, tab, seq, 5000, split_size=64, **kw),
            attn.attn_decode_paged_fp8_workspace_bytes(2, 16, 2, 5000, 128, 64)),
        "attn_cache_read_fp8": (lambda **kw: attn.attn_cache_read_fp8(*cache, tab, cu, 8000, **kw), 0),
    }


NAMES = ["attn_fwd", "attn_fwd_window", "attn_fwd_fp8", "attn_bwd", "attn_bwd_window_sinks",
         "attn_decode_paged", "attn_decode_splitkv", "attn_decode_paged_fp8", "attn_cache_read_fp8"]


@pytest.mark.parametrize("as_int", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_a_busy_stream_keeps_what_the_call_allocated(attn, name, as_int):
    import torch

    call, need = cases(attn)[name]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = call(stream=side.cuda_stream if as_int else side)
    filled = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
              for n in (max(need, 1), *(t.nbytes for t in got)) for _ in range(4)]
    torch.cuda.synchronize()
    assert attn.attn_poll_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    del filled


def test_the_default_stream_by_its_handle(attn):
    """The same with the busy stream the legacy default one, handed over as its handle, 0."""
    import torch

    call, need = cases(attn)["attn_decode_splitkv"]
    want = call()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    with torch.cuda.stream(torch.cuda.Stream()):
        got = call(stream=0)
        filled = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                  for n in (need, *(t.nbytes for t in got)) for _ in range(4)]
    torch.cuda.synchronize()
    assert attn.attn_poll_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del filled
