"""CPU checks of who owns what a call allocates: results and workspace belong to the stream the call
runs on, so that memory given back when the call returns is reused behind its kernels.  The library is
replaced by a stand-in; no compute call is made."""
import contextlib

import pytest


@pytest.fixture(scope="module")
def attn():
    import __graft_entry__

    __graft_entry__._cuda_build_module().build()
    import exact_io_aware_09_gb300 as m

    return m


def calls(attn):
    """Every entry point that takes a stream and allocates, on small tensors."""
    import torch

    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros((1, 4, 8, 128), dtype=bf), torch.zeros((1, 2, 8, 128), dtype=bf)
    lse = torch.zeros((1, 4, 8))
    tok, pool = torch.zeros((2, 4, 128), dtype=bf), torch.zeros((4, 16, 2, 128), dtype=bf)
    tab, seq, cu = torch.zeros((2, 1), dtype=i32), torch.ones(2, dtype=i32), torch.zeros(3, dtype=i32)
    flat = pool.view(64, 2, 128)
    codes = torch.zeros((4, 16, 2, 128), dtype=torch.uint8).view(torch.float8_e4m3fn)
    sc = torch.ones((4, 2, 16))
    cache = (codes, codes, sc, sc)
    mask = torch.ones((1, 1), dtype=torch.uint8)
    wide = torch.zeros((2, 400), dtype=i32)
    return {
        "attn_fwd": lambda **kw: attn.attn_fwd(q, k, k, **kw),
        "attn_fwd_fp8": lambda **kw: attn.attn_fwd_fp8(q, k, k, **kw),
        "attn_fwd_window": lambda **kw: attn.attn_fwd_window(q, k, k, 4, **kw),
        "attn_fwd_window_sinks": lambda **kw: attn.attn_fwd_window_sinks(q, k, k, 4, 1, **kw),
        "attn_fwd_block_sparse": lambda **kw: attn.attn_fwd_block_sparse(q, k, k, mask, **kw),
        "attn_bwd": lambda **kw: attn.attn_bwd(q, k, k, q, q, lse, **kw),
        "attn_bwd_window_sinks": lambda **kw: attn.attn_bwd_window_sinks(q, k, k, q, q, lse, 4, 1, **kw),
        "attn_decode_paged": lambda **kw: attn.attn_decode_paged(tok, pool, pool, tab, seq, 16, **kw),
        "attn_decode_splitkv": lambda **kw: attn.attn_decode_splitkv(tok, flat, flat, cu, 16, **kw),
        "attn_decode_splitkv_static": lambda **kw: attn.attn_decode_splitkv_static(tok, flat, flat, cu, 16,
                                                                                   **kw),
        "attn_fwd_paged": lambda **kw: attn.attn_fwd_paged(tok, pool, pool, wide, cu, seq, 1, 6400, **kw),
        "attn_cache_read_fp8": lambda **kw: attn.attn_cache_read_fp8(*cache, tab, cu, 2, **kw),
        "attn_decode_paged_fp8": lambda **kw: attn.attn_decode_paged_fp8(tok, *cache, wide, seq, 6400,
                                                                         split_size=64, **kw),
    }


NAMES = ["attn_fwd", "attn_fwd_fp8", "attn_fwd_window", "attn_fwd_window_sinks", "attn_fwd_block_sparse",
         "attn_bwd", "attn_bwd_window_sinks", "attn_decode_paged", "attn_decode_splitkv",
         "attn_decode_splitkv_static", "attn_fwd_paged", "attn_cache_read_fp8", "attn_decode_paged_fp8"]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_calls_stream(attn, monkeypatch, name):
    import torch

    owner, made = [None], []

    @contextlib.contextmanager
    def allocating(stream, device):
        assert device == torch.device("cpu")
        owner.append(stream)
        yield
        owner.pop()

    class Lib:
        def __getattr__(self, n):
            return getattr(real, n) if n.endswith("_bytes") else lambda *a: 0

    real = attn.lib
    call = calls(attn)[name]
    monkeypatch.setattr(attn, "lib", Lib())
    monkeypatch.setattr(attn, "_allocating", allocating)
    monkeypatch.setattr(attn, "_on_device", lambda *a: contextlib.nullcontext())
    monkeypatch.setattr(attn, "_device", lambda i: contextlib.nullcontext())
    monkeypatch.setattr(attn, "_dev_ptr", lambda t, n: 0)
    monkeypatch.setattr(attn, "_pointers", lambda w, n, t: (0, [0] * len(t)))
    monkeypatch.setattr(attn, "_stream_handle", lambda *a: 0)
    for f in ("empty", "empty_like"):
        real_f = getattr(torch, f)
        monkeypatch.setattr(torch, f,
                            lambda *a, real_f=real_f, **kw: (made.append(owner[-1]), real_f(*a, **kw))[1])
    call(stream="the call's")
    assert made and all(o == "the call's" for o in made), made


def test_handle_zero_is_the_default_stream(attn, monkeypatch):
    """The legacy default stream's handle is 0, which no external stream object stands for (torch makes a
    stream of its pool of it): the allocations are the device's default stream's."""
    import torch

    dev = torch.device("cuda", 1)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: ("external", handle, device))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    assert attn._allocating(0, dev) == ("default", dev)
    assert attn._allocating(1 << 20, dev) == ("external", 1 << 20, dev)
