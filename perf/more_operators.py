"""Cases of the page-list and 4-bit-cache operators: inputs, one pass of each in plain torch or
through the package, and the same from the definitions in 64 bits.

  extend  pages of a free list given to sequences that grow, and the slots of their new tokens
  trim    pages of sequences that are cut short, or end, back on the free list
  store   new keys and values quantised to 4 bits into a paged cache, and read back as it holds them
  read    a 4-bit paged cache read back as the packed 16-bit cache
  decode4 one decode step over a 4-bit paged cache
  paged4  a chunk of new tokens of each sequence over a 4-bit paged cache, causal, with or without
          a window and sinks

The cache: a row (the d values of a token and key/value head) in blocks of 16 values, each a scale
byte (five exponent and three mantissa bits: the bits of an fp16 number without its sign and its last
seven) and 16 codes of 4 bits (E2M1: 0, 1/2, 1, 3/2, 2, 3, 4, 6 and a sign), two to a byte.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------
def listed():
    return [
        # the bookkeeping of a decode step: one more token for each sequence of a serving batch
        dict(name="extend_step_b64", kind="extend", B=64, page=64, k_lo=1024, k_hi=32768, q_lo=1,
             q_hi=1, len_seed=41),
        # many whole prompts admitted at once
        dict(name="extend_prompts_b256", kind="extend", B=256, page=16, k_lo=0, k_hi=0, q_lo=1025,
             q_hi=8192, len_seed=42),
        # drafted tokens that were not accepted
        dict(name="trim_drafts_b64", kind="trim", B=64, page=16, k_lo=1024, k_hi=32768, q_lo=0,
             q_hi=7, len_seed=43),
        # sequences that end, their whole caches given back
        dict(name="trim_release_b512", kind="trim", B=512, page=16, k_lo=1024, k_hi=8192, q_lo=1024,
             q_hi=8192, len_seed=44),
        # a decode step's new tokens going into the cache, and what it holds of them
        dict(name="store_step_b64", kind="store", B=64, Hkv=8, d=128, dtype="bf16", page=64, q_lo=1,
             q_hi=1, k_lo=1, k_hi=2000, len_seed=45),
        # whole prompts going into the cache
        dict(name="store_prompts", kind="store", B=16, Hkv=8, d=128, dtype="bf16", page=16,
             q_lo=1025, q_hi=8192, k_lo=1025, k_hi=8192, len_seed=24),
        # one short sequence of a small model read back
        dict(name="read_one_user", kind="read", B=1, Hkv=4, d=64, dtype="f16", page=16, k_lo=1001,
             k_hi=1001, len_seed=26),
        # the packed 16-bit copy of a batch's cache
        dict(name="read_b32", kind="read", B=32, Hkv=8, d=128, dtype="bf16", page=32, k_lo=1024,
             k_hi=32768, len_seed=25),
        # one user's step on a small model
        dict(name="decode4_one_user", kind="decode4", B=1, Hq=16, Hkv=4, d=64, dtype="f16", page=16,
             k_lo=1001, k_hi=1001, len_seed=26),
        # the decode workload over a 4-bit cache
        dict(name="decode4_b64", kind="decode4", B=64, Hq=64, Hkv=8, d=128, dtype="bf16", page=64,
             k_lo=1024, k_hi=32768, len_seed=5000),
        # a serving batch verifying a few drafted tokens per sequence
        dict(name="paged4_verify_b64", kind="paged4", B=64, Hq=64, Hkv=8, d=128, dtype="bf16",
             page=64, q_lo=3, q_hi=8, k_lo=1024, k_hi=32768, window=-1, sinks=0, len_seed=5000),
        # two long prompts taken in 2048-token chunks, the last chunk over a 16-token-page cache
        dict(name="paged4_chunk_2048", kind="paged4", B=2, Hq=64, Hkv=8, d=128, dtype="bf16",
             page=16, q_lo=2048, q_hi=2048, k_lo=12001, k_hi=16384, window=-1, sinks=0, len_seed=21),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(math.floor(lo), int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most):
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    while hkv * g > most:
        g = max(1, g // 2)
    return hkv * g, hkv


def draw(rng):
    kind = rng.choice(["extend", "trim", "store", "read", "decode4", "decode4", "paged4", "paged4"])
    c = dict(kind=kind, page=rng.choice([16, 32, 64, 128, 256]), len_seed=rng.randrange(1 << 20))
    if kind in ("extend", "trim"):
        c["B"] = _log_int(rng, 1, 2048)
        room = 512 * 8192 // c["B"]  # tokens of a sequence
        c["k_hi"] = _log_int(rng, 1, max(1, min(32768, room)))
        c["k_lo"] = c["k_hi"] // rng.choice([1, 2, 16])
        most = min(8192, 256 * 8192 // c["B"]) if kind == "extend" else c["k_hi"]
        c["q_hi"] = 1 if rng.random() < 0.3 else _log_int(rng, 1, max(1, most))
        c["q_lo"] = c["q_hi"] // rng.choice([1, 2, 5])
        return c
    c["d"], c["dtype"] = rng.choice([64, 128]), rng.choice(["bf16", "f16"])
    hq, c["Hkv"] = _heads(rng, 64)
    if kind in ("decode4", "paged4"):
        c["Hq"] = hq
    c["k_hi"] = _log_int(rng, 16, 32768)
    c["k_lo"] = max(1, c["k_hi"] // rng.choice([1, 2, 16]))
    c["B"] = _log_int(rng, 1, max(1, min(64, 64 * 32768 * 8 // (c["Hkv"] * c["k_hi"]))))
    if kind == "paged4":
        c["q_hi"] = min(c["k_hi"], 1 if rng.random() < 0.25 else _log_int(rng, 1, 2048))
        c["q_lo"] = max(1, c["q_hi"] // rng.choice([1, 2, 5]))
        c["B"] = max(1, min(c["B"], 2 * 64 * 2048 * 12001 // (hq * c["q_hi"] * c["k_hi"])))
        far = rng.random() < 0.4
        c["window"] = _log_int(rng, 1, 8192) if far else -1
        c["sinks"] = rng.choice([0, 1, 4, 64, 130]) if far else 0
    elif kind == "store":
        c["k_hi"] = min(c["k_hi"], 8192)
        c["k_lo"] = min(c["k_lo"], c["k_hi"])
        c["q_hi"] = 1 if rng.random() < 0.3 else _log_int(rng, 1, c["k_hi"])
        c["q_lo"] = max(1, c["q_hi"] // 2)
        c["B"] = min(c["B"], 16)
    elif kind == "read":
        c["B"] = min(c["B"], 32)
    return c


def _lengths(c):
    """(new tokens, tokens in the cache) of every sequence of a case: for `extend` those before the
    new tokens, else those with them (for `trim` the new tokens are the ones that go)."""
    g = np.random.Generator(np.random.PCG64(c["len_seed"]))
    k = g.integers(c["k_lo"], c["k_hi"], size=c["B"], endpoint=True)
    if "q_hi" not in c:
        return np.ones_like(k) if c["kind"] == "decode4" else k, k
    q = g.integers(c["q_lo"], c["q_hi"], size=c["B"], endpoint=True)
    if c["kind"] == "trim":
        return np.minimum(q, k), k
    return q, k if c["kind"] == "extend" else np.maximum(k, q)


def _visible(c):
    """Query-key pairs that a case's mask keeps, per query head."""
    n = 0
    for q, k in zip(*_lengths(c)):
        pos = np.arange(q, dtype=np.int64) + k - q
        if c.get("window", -1) < 0:
            n += int((pos + 1).sum())
        else:
            near = np.minimum(pos + 1, c["window"] + 1)
            n += int((near + np.minimum(pos + 1 - near, c["sinks"])).sum())
    return n


def _keys_needed(c):
    """Cache tokens that some new token of its sequence sees."""
    q, k = _lengths(c)
    if c.get("window", -1) < 0:
        return int(k.sum())
    first = np.maximum(k - q - c["window"], 0)
    return int((k - first + np.minimum(first, c["sinks"])).sum())


def work(c):
    q, k = _lengths(c)
    P = c["page"]
    if c["kind"] == "extend":  # lengths and offsets; the new pages' entries; a slot per token
        new = int((-(-(k + q) // P) - -(-k // P)).sum())
        return {"bytes": 4 * (3 * c["B"] + 2 + 2 * new + int(q.sum())), "flops": 0}
    if c["kind"] == "trim":  # lengths; a page's entry read, put on the list and cleared
        gone = int((-(-k // P) - -(-(k - q) // P)).sum())
        return {"bytes": 4 * (3 * c["B"] + 2 + 3 * gone), "flops": 0}
    d = c["d"]
    row4, row16 = d // 2 + d // 16, 2 * d  # bytes of a row in 4 and in 16 bits
    if c["kind"] == "store":  # taken in 16 bits, kept in 4; those read, given out in 16
        return {"bytes": int(q.sum()) * (c["Hkv"] * 2 * (2 * row16 + 2 * row4) + 4), "flops": 0}
    if c["kind"] == "read":
        return {"bytes": int(k.sum()) * c["Hkv"] * 2 * (row16 + row4), "flops": 0}
    return {"bytes": int(q.sum()) * c["Hq"] * (2 * row16 + 4) + _keys_needed(c) * c["Hkv"] * 2 * row4,
            "flops": 4.0 * c["Hq"] * _visible(c) * d}


# --------------------------------------------------------------------------------------------
# the 4-bit format, in 32 bits
# --------------------------------------------------------------------------------------------
def _split4(x):
    """Codes [..., d/2] and scale bytes [..., d/16] (uint8) of finite rows x [..., d]."""
    x = x.float()
    blocks = x.unflatten(-1, (-1, 16))
    t = blocks.abs().amax(-1) / 6.0
    _, e = torch.frexp(t)  # t = m 2^e, m in [1/2, 1): the scale's last place is 2^(e - 4)
    step = torch.ldexp(torch.ones_like(t), (e - 4).clamp_min(-17))
    s = (torch.round(t / step) * step).clamp_max(10240.0)  # (round: halves to even)
    s = torch.where(t > 0, s.clamp_min(2.0 ** -17), s)
    y = blocks.abs() / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    # halves between two values go to the even code
    code = ((y > 0.25).byte() + (y >= 0.75).byte() + (y > 1.25).byte() + (y >= 1.75).byte()
            + (y > 2.5).byte() + (y >= 3.5).byte() + (y > 5.0).byte())
    code = (code + 8 * torch.signbit(blocks).byte()).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (s.half().view(torch.int16) >> 7).byte()


def _join4(codes, scales):
    """Rows [..., d] in float32 of codes and scale bytes."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    grid = torch.cat([grid, -grid])
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], -1).flatten(-2)
    s = (scales.short() << 7).view(torch.float16).float()
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _normal(shape, g, dtype, outliers=False):
    x = torch.randn(shape, generator=g, device="cuda")
    if outliers:  # a few channels carry large values, as keys of trained models do
        x[..., ::37] *= 8.0
    return x.to(dtype)


def _gpu(x):
    return torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()


def _offsets(n):
    return _gpu(np.concatenate([[0], np.cumsum(n)]))


def _tables(lengths, width, pool, page, g):
    """Block table [B, width] (-1 past a sequence's pages) in shuffled pages, and the shuffled pool."""
    pages = -(-lengths // page)
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    at = _gpu(np.cumsum(pages) - pages)[:, None] + col[None, :]
    held = col[None, :] < _gpu(pages)[:, None]
    return torch.where(held, perm[at.clamp_max(pool - 1)], torch.full_like(at, -1).int()), perm


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6151 + 29)
    nq, nk = _lengths(c)
    page, B = c["page"], c["B"]
    s = dict(case=dict(c), cu_q=_offsets(nq), total_q=int(nq.sum()), max_q=int(nq.max()))
    if c["kind"] in ("extend", "trim"):
        most = int((nk + nq).max()) if c["kind"] == "extend" else int(nk.max())
        width = max(1, -(-most // page))
        used = int((-(-nk // page)).sum())
        final = int((-(-(nk + nq) // page)).sum()) if c["kind"] == "extend" else used
        pool = final + 7  # a few pages are left
        table, perm = _tables(nk, width, pool, page, g)
        # the free list is a stack: its first n_free entries, the rest as earlier steps left them
        stack = torch.cat([perm[used:], perm[:used]])
        # one buffer, so that a pass starts from the same state with a single copy
        whole = torch.cat([table.flatten(), stack, _gpu(nk), _gpu([pool - used])])
        s["start"], s["now"] = whole, whole.clone()
        cut = [B * width, pool, B, 1]
        s["table"], s["free"], s["seqlens"], s["n_free"] = s["now"].split(cut)
        s["table"] = s["table"].view(B, width)
        s["keep"] = _gpu(nk - nq)
        return s
    d, Hkv, dt = c["d"], c["Hkv"], _DT[c["dtype"]]
    s["scale"] = 1.0 / math.sqrt(d)
    pool = int((-(-nk // page)).sum()) + 3
    s["table"], _ = _tables(nk, int((-(-nk // page)).max()), pool, page, g)
    s["seqlens"], s["first"], s["cu_k"] = _gpu(nk), _gpu(nk - nq), _offsets(nk)
    s["max_k"], s["total_k"] = int(nk.max()), int(nk.sum())
    shape = (pool, Hkv, page, d)
    for name in ("k", "v"):
        if c["kind"] == "store":  # the cache as earlier tokens left it
            s[name] = _normal((s["total_q"], Hkv, d), g, dt, outliers=name == "k")
            codes = torch.randint(0, 256, shape[:-1] + (d // 2,), generator=g, device="cuda",
                                  dtype=torch.uint8)
            scales = torch.full(shape[:-1] + (d // 16,), 0x70, device="cuda", dtype=torch.uint8)
        else:
            parts = [_split4(_normal((min(4096, pool - at),) + shape[1:], g, torch.float32,
                                     outliers=name == "k")) for at in range(0, pool, 4096)]
            codes, scales = (torch.cat(x) for x in zip(*parts))
        s[name + "_codes"], s[name + "_scales"] = codes, scales
    if c["kind"] == "store":
        b = np.repeat(np.arange(B), nq)
        t = np.arange(s["total_q"]) - np.repeat(np.cumsum(nq) - nq, nq) + np.repeat(nk - nq, nq)
        b, t = torch.from_numpy(b).cuda(), torch.from_numpy(t).cuda()
        s["slots"] = (s["table"][b, t // page] * page + t % page).int()
    elif c["kind"] != "read":
        s["q"] = _normal((s["total_q"], c["Hq"], d), g, dt)
    return s


# --------------------------------------------------------------------------------------------
# plain forms (32 bits, rounded once)
# --------------------------------------------------------------------------------------------
def _tokens_of(cu, B, total):
    """The sequence of each packed token, and the token's number in it."""
    n = (cu[1:] - cu[:-1]).long()
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), n, output_size=total)
    return b, torch.arange(total, device="cuda") - cu.long()[b]


def _plain_extend(s):
    c, P = s["case"], s["case"]["page"]
    L = s["seqlens"].long()
    n = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    have = (L + P - 1) // P
    need = (L + n + P - 1) // P - have
    off = torch.cumsum(need, 0) - need
    b, i = _tokens_of(s["cu_q"], c["B"], s["total_q"])
    t = L[b] + i
    j = t // P
    k = s["n_free"].long() - 1 - (off[b] + j - have[b])
    page = torch.where(j < have[b], s["table"][b, j], s["free"][k.clamp(0, len(s["free"]) - 1)])
    s["table"][b, j] = page
    s["seqlens"] += n.int()
    s["n_free"] -= need.sum().int()
    return [s["table"], s["seqlens"], s["free"], s["n_free"], (page * P + t % P).int()]


def _plain_trim(s):
    P = s["case"]["page"]
    have, left = (s["seqlens"].long() + P - 1) // P, (s["keep"].long() + P - 1) // P
    n = have - left
    off = torch.cumsum(n, 0) - n
    j = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    gone = (j >= left[:, None]) & (j < have[:, None])
    k = s["n_free"].long() + n.sum() - 1 - (off[:, None] + j - left[:, None])
    room = torch.cat([s["free"], s["free"][:1]])  # the last place takes what does not go
    room[torch.where(gone, k, torch.full_like(k, len(s["free"])))] = s["table"]
    s["free"].copy_(room[:-1])
    s["table"].masked_fill_(gone, -1)
    s["seqlens"].copy_(s["keep"])
    s["n_free"] += n.sum().int()
    return [s["table"], s["seqlens"], s["free"], s["n_free"]]


def _dequantised(s, name, page, slot):
    """Rows [..., Hkv, d] at pages and slots of the same shape."""
    return _join4(s[name + "_codes"][page, :, slot], s[name + "_scales"][page, :, slot])


def _plain_store(s):
    c, P = s["case"], s["case"]["page"]
    page, slot = s["slots"].long() // P, s["slots"].long() % P
    for name in ("k", "v"):
        s[name + "_codes"][page, :, slot], s[name + "_scales"][page, :, slot] = _split4(s[name])
    b, i = _tokens_of(s["cu_q"], c["B"], s["total_q"])
    t = s["first"].long()[b] + i
    page, slot = s["table"][b, t // P].long(), t % P
    return [_dequantised(s, name, page, slot).to(_DT[c["dtype"]]) for name in ("k", "v")]


def _plain_read(s):
    c, P = s["case"], s["case"]["page"]
    b, t = _tokens_of(s["cu_k"], c["B"], s["total_k"])
    page, slot = s["table"][b, t // P].long(), t % P
    return [_dequantised(s, name, page, slot).to(_DT[c["dtype"]]) for name in ("k", "v")]


def _plain_paged4(s):
    c = s["case"]
    B, Hq, Hkv, d, P = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    nq, L, G = s["max_q"], s["max_k"], c["Hq"] // c["Hkv"]
    j = torch.arange(L, device="cuda")
    at = s["table"][:, j // P].long().clamp_min(0), (j % P)[None, :].expand(B, L)
    n = s["cu_q"][1:] - s["cu_q"][:-1]
    i = torch.arange(nq, device="cuda")
    there = i[None, :] < n[:, None]
    row = (s["cu_q"][:-1, None] + i[None, :]).clamp_max(s["total_q"] - 1).long()
    q = s["q"][row].float().view(B, nq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nq, d)
    x = (q @ _dequantised(s, "k", *at).permute(0, 2, 3, 1)).mul_(s["scale"])
    pos = ((s["seqlens"] - n)[:, None] + i[None, :])[:, :, None]
    seen = j <= pos
    if c.get("window", -1) >= 0:
        seen = seen & ((pos - j <= c["window"]) | (j < c["sinks"]))
    x.view(B, Hkv, G, nq, L).masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)  # (rows past a chunk's end see a key too: the first)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(x.sub_(m))
    l = p.sum(-1, keepdim=True)
    o = (p @ _dequantised(s, "v", *at).transpose(1, 2)) / l
    o = o.view(B, Hkv, G, nq, d).permute(0, 3, 1, 2, 4)
    lse = (m + torch.log(l)).view(B, Hkv, G, nq).permute(0, 3, 1, 2)
    if nq == 1:  # every sequence has its one token
        return [o.reshape(B, Hq, d).to(s["q"].dtype), lse.reshape(B, Hq)]
    return [o[there].reshape(-1, Hq, d).to(s["q"].dtype), lse[there].reshape(-1, Hq)]


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------
def _own(s):
    import exact_io_aware_09_gb300 as attn

    c = s["case"]
    if c["kind"] == "extend":
        slots = attn.attn_pages_extend(s["table"], s["seqlens"], s["cu_q"], s["free"], s["n_free"],
                                       c["page"], s["total_q"])
        return [s["table"], s["seqlens"], s["free"], s["n_free"], slots]
    if c["kind"] == "trim":
        attn.attn_pages_trim(s["table"], s["seqlens"], s["keep"], s["free"], s["n_free"], c["page"])
        return [s["table"], s["seqlens"], s["free"], s["n_free"]]
    cache = s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"]
    if c["kind"] == "store":
        attn.attn_cache_write_fp4(s["k"], s["v"], *cache, s["slots"])
        return list(attn.attn_cache_read_fp4(*cache, s["table"], s["cu_q"], s["total_q"],
                                             starts=s["first"], dtype=_DT[c["dtype"]]))
    if c["kind"] == "read":
        return list(attn.attn_cache_read_fp4(*cache, s["table"], s["cu_k"], s["total_k"],
                                             dtype=_DT[c["dtype"]]))
    if c["kind"] == "decode4":
        return list(attn.attn_decode_paged_fp4(s["q"], *cache, s["table"], s["seqlens"], s["max_k"],
                                               scale=s["scale"]))
    return list(attn.attn_fwd_paged_fp4(s["q"], *cache, s["table"], s["cu_q"], s["seqlens"],
                                        s["max_q"], s["max_k"], window=c["window"],
                                        sinks=c["sinks"], scale=s["scale"]))


_PLAIN = {"extend": _plain_extend, "trim": _plain_trim, "store": _plain_store, "read": _plain_read,
          "decode4": _plain_paged4, "paged4": _plain_paged4}


def run(s):
    if "start" in s:  # what the last pass changed
        s["now"].copy_(s["start"])
    return _own(s) if own else _PLAIN[s["case"]["kind"]](s)


# --------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_E5M3 = [m * 2.0 ** -17 for m in range(8)] + [(8 + m) * 2.0 ** (e - 18) for e in range(1, 32)
                                              for m in range(8)]


def _nearest(x, grid):
    """Places in the ascending grid of the values nearest to x >= 0, the even one of two as near."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    up, down = grid[hi] - x, x - grid[hi - 1]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def _rounded64(x):
    """What the cache holds of rows x, float64."""
    out = []
    for part in x.split(8192):
        y = part.double().unflatten(-1, (-1, 16))
        top = y.abs().amax(-1)
        at = _nearest(top / 6.0, _E5M3).clamp_max(_E5M3.index(10240.0))
        at = torch.where(top > 0, at.clamp_min(1), at)
        f = torch.tensor(_E5M3, dtype=torch.float64, device=x.device)[at][..., None]
        at = _nearest(y.abs() / torch.where(f > 0, f, torch.ones_like(f)), _E2M1)
        v = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)[at]
        out.append((torch.sign(y) * v * f).flatten(-2))
    return torch.cat(out)


def _pages_of(s, b, n):
    """Page and slot of sequence b's first n tokens."""
    P = s["case"]["page"]
    t = torch.arange(int(n), device="cuda")
    return s["table"][b, : -(-int(n) // P)].long()[t // P], t % P


def _held64(s, name, page, slot):
    codes, by = s[name + "_codes"][page, :, slot], s[name + "_scales"][page, :, slot]
    both = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device=codes.device)
    v = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64, device=codes.device)
    v[..., 0::2], v[..., 1::2] = both[codes.long() % 16], both[codes.long() // 16]
    f = torch.tensor(_E5M3, dtype=torch.float64, device=codes.device)[by.long().clamp_max(len(_E5M3) - 1)]
    return v * f.repeat_interleave(16, -1)


def _attend64(q, k, v, seen, scale):
    logits = torch.einsum("id,jd->ij", q, k) * scale
    logits = torch.where(seen, logits, logits.new_full((), -math.inf))
    lse = torch.logsumexp(logits, 1)
    return torch.einsum("ij,jd->id", torch.exp(logits - lse[:, None]), v), lse


def exact(c, seed):
    nq, nk = _lengths(c)
    s = prepare(c, seed)
    P = c["page"]
    if c["kind"] in ("extend", "trim"):
        table, free = s["table"].tolist(), s["free"].tolist()
        left, slots = int(s["n_free"]), []
        if c["kind"] == "extend":
            for row, q, k in zip(table, nq.tolist(), nk.tolist()):
                for t in range(k, k + q):
                    if t % P == 0:
                        left -= 1
                        row[t // P] = free[left]
                    slots.append(row[t // P] * P + t % P)
            out = [nk + nq, free, [left], slots]
        else:
            for row, q, k in reversed(list(zip(table, nq.tolist(), nk.tolist()))):
                for j in reversed(range(-(-(k - q) // P), -(-k // P))):
                    free[left], row[j] = row[j], -1
                    left += 1
            out = [nk - nq, free, [left]]
        return [_gpu(table)] + [_gpu(x) for x in out]
    if c["kind"] == "store":
        return [_rounded64(s["k"]), _rounded64(s["v"])]
    if c["kind"] == "read":
        at = [torch.cat(x) for x in zip(*(_pages_of(s, b, n) for b, n in enumerate(nk)))]
        return [torch.cat([_held64(s, name, *(a[i:i + 65536] for a in at))
                           for i in range(0, len(at[0]), 65536)]) for name in ("k", "v")]
    if 4.0 * c["Hq"] * float((nq * nk).sum()) * c["d"] > 8e12:
        return None
    G, at_q = c["Hq"] // c["Hkv"], np.concatenate([[0], np.cumsum(nq)])
    o = torch.zeros_like(s["q"], dtype=torch.float64)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        at = _pages_of(s, b, nk[b])
        k, v = _held64(s, "k", *at), _held64(s, "v", *at)
        seen = np.tril(np.ones((nq[b], nk[b]), dtype=bool), nk[b] - nq[b])
        if c.get("window", -1) >= 0:
            near = np.triu(np.ones_like(seen), nk[b] - nq[b] - c["window"])
            near[:, :c["sinks"]] = True
            seen &= near
        seen = torch.from_numpy(seen).cuda().repeat(G, 1)  # the heads of a group one after another
        r = slice(int(at_q[b]), int(at_q[b + 1]))
        for h in range(c["Hkv"]):
            q = s["q"][r, h * G:(h + 1) * G].double().transpose(0, 1).reshape(-1, c["d"])
            x, y = _attend64(q, k[:, h], v[:, h], seen, s["scale"])
            o[r, h * G:(h + 1) * G] = x.view(G, -1, c["d"]).transpose(0, 1)
            lse[r, h * G:(h + 1) * G] = y.view(G, -1).t()
    return [o, lse]
