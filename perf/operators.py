"""Cases of the window-and-sinks, paged-chunk and quantised-cache operators: inputs, one pass of
each in plain torch or through the package, and the same from the definitions in 64 bits.

  window  attention over the last W keys and the first few (sinks), forward, or forward and
          gradients as a training step runs them
  paged   a chunk of new tokens of each sequence over a paged 16-bit cache (one token each: the
          decode step), causal, with or without the window and the sinks
  write   new keys and values quantised to 8 bits as they go into a paged cache
  read    a quantised paged cache read back as the packed 16-bit cache
  decode8 one decode step over a quantised paged cache
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
        # a short prompt of a small model: one call's latency
        dict(name="window_short_prompt", kind="window", backward=False, B=1, Hq=4, Hkv=2, Nq=333,
             Nkv=333, d=64, dtype="f16", window=100, sinks=4),
        # the long grouped-query prefill under the 1024-key window
        dict(name="window_gqa_8192", kind="window", backward=False, B=1, Hq=64, Hkv=8, Nq=8192,
             Nkv=8192, d=128, dtype="bf16", window=1024, sinks=4),
        # a training step of the GPT-2 shape with local attention
        dict(name="window_train_gpt2", kind="window", backward=True, B=8, Hq=12, Hkv=12, Nq=1024,
             Nkv=1024, d=64, dtype="bf16", window=256, sinks=4),
        # a training step of the long grouped-query shape
        dict(name="window_train_gqa_8192", kind="window", backward=True, B=1, Hq=64, Hkv=8,
             Nq=8192, Nkv=8192, d=128, dtype="bf16", window=1024, sinks=64),
        # two long prompts taken in 2048-token chunks, the last chunk over a 16-token-page cache
        dict(name="paged_chunk_2048", kind="paged", B=2, Hq=64, Hkv=8, d=128, dtype="bf16",
             page=16, q_lo=2048, q_hi=2048, k_lo=12001, k_hi=16384, window=-1, sinks=0,
             len_seed=21),
        # a serving batch verifying a few drafted tokens per sequence
        dict(name="paged_verify_b64", kind="paged", B=64, Hq=64, Hkv=8, d=128, dtype="bf16",
             page=64, q_lo=3, q_hi=8, k_lo=1024, k_hi=32768, window=-1, sinks=0, len_seed=5000),
        # single tokens of long streams that keep a window and four sinks
        dict(name="paged_token_window", kind="paged", B=16, Hq=32, Hkv=8, d=64, dtype="f16",
             page=16, q_lo=1, q_hi=1, k_lo=5000, k_hi=60001, window=4095, sinks=4, len_seed=22),
        # a decode step's new tokens going into the cache
        dict(name="write_step_b64", kind="write", B=64, Hkv=8, d=128, dtype="bf16", page=64,
             q_lo=1, q_hi=1, k_lo=1, k_hi=2000, len_seed=23),
        # whole prompts going into the cache
        dict(name="write_prompts", kind="write", B=16, Hkv=8, d=128, dtype="bf16", page=16,
             q_lo=1025, q_hi=8192, k_lo=1025, k_hi=8192, len_seed=24),
        # the packed 16-bit copy of a quantised cache
        dict(name="read_b32", kind="read", B=32, Hkv=8, d=128, dtype="bf16", page=32, k_lo=1024,
             k_hi=32768, len_seed=25),
        # the decode workload over a quantised cache
        dict(name="decode8_b64", kind="decode8", B=64, Hq=64, Hkv=8, d=128, dtype="bf16", page=64,
             k_lo=1024, k_hi=32768, len_seed=5000),
        # one user's step on a small model
        dict(name="decode8_one_user", kind="decode8", B=1, Hq=16, Hkv=4, d=64, dtype="f16",
             page=16, k_lo=1001, k_hi=1001, len_seed=26),
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
    kind = rng.choice(["window", "window", "paged", "paged", "write", "read", "decode8"])
    d = rng.choice([64, 128])
    c = dict(kind=kind, d=d, dtype=rng.choice(["bf16", "f16"]))
    if kind == "window":
        c["Hq"], c["Hkv"] = _heads(rng, 64)
        c["backward"] = rng.random() < 0.5
        # a training step runs over whole sequences; a forward pass may add rows to older keys
        c["Nq"] = _log_int(rng, 64 if c["backward"] else 1, 8192)
        same = c["backward"] or rng.random() < 0.6
        c["Nkv"] = c["Nq"] if same else _log_int(rng, 1, 8192)
        # scores of the plain form: at most those of the largest listed case
        c["B"] = _log_int(rng, 1, max(1, min(8, 8192 * 8192 * 64 // (c["Hq"] * c["Nq"] * c["Nkv"]))))
        c["window"] = _log_int(rng, 16 if c["backward"] else 0.6, 4096)
        c["sinks"] = rng.choice([0, 1, 4, 64, 128, 200])
        return c
    c["page"] = rng.choice([16, 32, 64, 128, 256])
    c["len_seed"] = rng.randrange(1 << 20)
    hq, hkv = _heads(rng, 64)
    c["Hkv"] = hkv
    if kind in ("paged", "decode8"):
        c["Hq"] = hq
    c["k_hi"] = _log_int(rng, 16, 32768)
    c["k_lo"] = max(1, c["k_hi"] // rng.choice([1, 2, 16]))
    tokens = 64 * 32768 * 8 // (hkv * c["k_hi"])
    c["B"] = _log_int(rng, 1, max(1, min(64, tokens)))
    if kind == "paged":
        c["q_hi"] = min(c["k_hi"], 1 if rng.random() < 0.25 else _log_int(rng, 1, 2048))
        c["q_lo"] = max(1, c["q_hi"] // rng.choice([1, 2, 5]))
        c["B"] = max(1, min(c["B"], 2 * 64 * 2048 * 12001 // (hq * c["q_hi"] * c["k_hi"])))
        far = rng.random() < 0.4
        c["window"] = _log_int(rng, 1, 8192) if far else -1
        c["sinks"] = rng.choice([0, 1, 4, 64, 130]) if far else 0
    elif kind == "write":
        c["k_hi"] = min(c["k_hi"], 8192)
        c["k_lo"] = min(c["k_lo"], c["k_hi"])
        c["q_hi"] = 1 if rng.random() < 0.3 else _log_int(rng, 1, c["k_hi"])
        c["q_lo"] = max(1, c["q_hi"] // 2)
        c["B"] = min(c["B"], 16)
    elif kind == "read":
        c["B"] = min(c["B"], 32)
    return c


def _lengths(c):
    """(new tokens, tokens in the cache) of every sequence of a case."""
    g = np.random.Generator(np.random.PCG64(c["len_seed"]))
    k = g.integers(c["k_lo"], c["k_hi"], size=c["B"], endpoint=True)
    if "q_hi" not in c:
        return np.zeros_like(k), k
    q = g.integers(c["q_lo"], c["q_hi"], size=c["B"], endpoint=True)
    return q, np.maximum(k, q)


def _visible(c):
    """Query-key pairs a case's mask keeps, per head (and per batch entry for `window`)."""
    if c["kind"] == "window":
        pos = np.arange(c["Nq"], dtype=np.int64) + c["Nkv"] - c["Nq"]
        pos = pos[pos >= 0]
        seqs = [pos]
    else:
        nq, nk = _lengths(c)
        seqs = [np.arange(n, dtype=np.int64) + L - n for n, L in zip(nq, nk)]
    n = 0
    for pos in seqs:
        if c["window"] < 0:
            n += int((pos + 1).sum())
        else:
            near = np.minimum(pos + 1, c["window"] + 1)
            n += int((near + np.minimum(pos + 1 - near, c["sinks"])).sum())
    return n


def _keys_needed(c):
    """Cache tokens that some new token of its sequence sees."""
    nq, nk = _lengths(c)
    if c["window"] < 0:
        return int(nk.sum())
    first = np.maximum(nk - nq - c["window"], 0)
    return int((nk - first + np.minimum(first, c["sinks"])).sum())


def work(c):
    d = c["d"]
    if c["kind"] == "window":
        q, kv = c["B"] * c["Hq"] * c["Nq"] * d * 2, c["B"] * c["Hkv"] * c["Nkv"] * d * 2
        lse = c["B"] * c["Hq"] * c["Nq"] * 4
        pairs = c["B"] * c["Hq"] * _visible(c)
        if c["backward"]:  # S, P V; S, dP, dV, dQ, dK: o and lse come out too
            return {"bytes": 4 * q + 4 * kv + lse, "flops": 14.0 * pairs * d}
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 4.0 * pairs * d}
    nq, nk = _lengths(c)
    if c["kind"] == "paged":
        t = int(nq.sum())
        return {"bytes": t * c["Hq"] * (4 * d + 4) + _keys_needed(c) * c["Hkv"] * 4 * d,
                "flops": 4.0 * c["Hq"] * _visible(c) * d}
    if c["kind"] == "write":
        return {"bytes": int(nq.sum()) * c["Hkv"] * 2 * (2 * d + d + 4), "flops": 0}
    if c["kind"] == "read":
        return {"bytes": int(nk.sum()) * c["Hkv"] * 2 * (2 * d + d + 4), "flops": 0}
    return {"bytes": int(nk.sum()) * c["Hkv"] * 2 * (d + 4) + c["B"] * c["Hq"] * (4 * d + 4),
            "flops": 4.0 * c["Hq"] * int(nk.sum()) * d}


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------
def _normal(shape, g, dtype, outliers=False):
    x = torch.randn(shape, generator=g, device="cuda")
    if outliers:  # a few channels carry large values, as keys and values of trained models do
        x[..., :: 37] *= 8.0
    return x.to(dtype)


def _split(x):
    """Power-of-two scale of each row of x (its largest magnitude at most 448 times it), and the
    row's 8-bit values."""
    a = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(a)  # a = m 2^e, m in [1/2, 1)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp_min(-126)
    e = torch.where(a > 0, e, torch.zeros_like(e))
    return torch.ldexp(torch.ones_like(a), e), torch.ldexp(x, -e).to(torch.float8_e4m3fn)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    dt, d = _DT[c["dtype"]], c["d"]
    s = dict(case=dict(c), scale=1.0 / math.sqrt(d))
    if c["kind"] == "window":
        s["q"] = _normal((c["B"], c["Hq"], c["Nq"], d), g, dt)
        s["k"] = _normal((c["B"], c["Hkv"], c["Nkv"], d), g, dt)
        s["v"] = _normal((c["B"], c["Hkv"], c["Nkv"], d), g, dt)
        if c["backward"]:
            s["do"] = _normal((c["B"], c["Hq"], c["Nq"], d), g, dt)
        return s
    nq, nk = _lengths(c)
    page, B, Hkv = c["page"], c["B"], c["Hkv"]
    n_pages = -(-nk // page)
    pool = int(n_pages.sum()) + 3  # a few free pages
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    at = np.concatenate([[0], np.cumsum(n_pages)])
    width = int(n_pages.max())
    col = torch.arange(width, device="cuda")
    first = torch.from_numpy(at[:-1]).cuda()[:, None]
    held = col[None, :] < torch.from_numpy(n_pages).cuda()[:, None]
    s["table"] = torch.where(held, perm[(first + col[None, :]).clamp_max(pool - 1)],
                             torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()
    s["seqlens"] = torch.from_numpy(nk.astype(np.int32)).cuda()
    s["max_k"] = int(nk.max())
    s["cu_q"] = torch.from_numpy(np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)).cuda()
    s["cu_k"] = torch.from_numpy(np.concatenate([[0], np.cumsum(nk)]).astype(np.int32)).cuda()
    s["max_q"], s["total_q"], s["total_k"] = int(nq.max()), int(nq.sum()), int(nk.sum())
    shape = (pool, page, Hkv, d)
    if c["kind"] == "paged":
        s["q"] = _normal((s["total_q"], c["Hq"], d), g, dt)
        s["k_pages"], s["v_pages"] = _normal(shape, g, dt), _normal(shape, g, dt)
        return s
    if c["kind"] == "decode8":
        s["q"] = _normal((B, c["Hq"], d), g, dt)
    if c["kind"] == "write":
        s["k"] = _normal((s["total_q"], Hkv, d), g, dt, outliers=True)
        s["v"] = _normal((s["total_q"], Hkv, d), g, dt)
    for name in ("k", "v"):
        if c["kind"] == "write":  # the cache as earlier tokens left it
            codes = torch.randint(0, 127, shape, generator=g, device="cuda", dtype=torch.uint8)
            s[name + "_pages"] = codes.view(torch.float8_e4m3fn)
            s[name + "_scales"] = torch.full((pool, Hkv, page), 0.25, device="cuda")
        else:
            sc, codes = _split(_normal(shape, g, dt, outliers=name == "k").float())
            s[name + "_pages"] = codes
            s[name + "_scales"] = sc[..., 0].transpose(1, 2).contiguous()
    return s


# --------------------------------------------------------------------------------------------
# plain forms (32 bits, rounded once)
# --------------------------------------------------------------------------------------------
def _softmax_parts(s):
    """Weights and log-sum-exp of masked scores (-inf where masked; a row may have none)."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    e = torch.exp(s - m)
    l = e.sum(-1, keepdim=True)
    lse = (m + torch.log(l))[..., 0]
    return e / torch.where(l > 0, l, torch.ones_like(l)), lse


def _keep(pos, keys, window, sinks):
    """Whether the query at position pos sees the key."""
    seen = keys <= pos
    if window >= 0:
        seen = seen & ((pos - keys <= window) | (keys < sinks))
    return seen


def _plain_window(s):
    c = s["case"]
    B, Hq, Hkv, Nq, Nkv, d = (c[n] for n in ("B", "Hq", "Hkv", "Nq", "Nkv", "d"))
    dt = s["q"].dtype
    # the query heads of one key/value head side by side: [B, Hkv, G * Nq, d]
    q = s["q"].float().view(B, Hkv, -1, d)
    k, v = s["k"].float(), s["v"].float()
    pos = torch.arange(Nq, device="cuda")[:, None] + (Nkv - Nq)
    seen = _keep(pos, torch.arange(Nkv, device="cuda")[None, :], c["window"], c["sinks"])
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"])
    x = x.view(B, Hkv, -1, Nq, Nkv).masked_fill_(~seen, -math.inf).view(B, Hkv, -1, Nkv)
    p, lse = _softmax_parts(x)
    del x
    o = p @ v
    out = [o.view(B, Hq, Nq, d).to(dt), lse.view(B, Hq, Nq)]
    if c["backward"]:
        do = s["do"].float().view(B, Hkv, -1, d)
        dp = do @ v.transpose(-1, -2)
        dv = p.transpose(-1, -2) @ do
        ds = p * dp.sub_((do * o).sum(-1, keepdim=True))
        del p, dp
        dq = (ds @ k) * s["scale"]
        dk = (ds.transpose(-1, -2) @ q) * s["scale"]
        out += [dq.view(B, Hq, Nq, d).to(dt), dk.to(dt), dv.to(dt)]
    return out


def _gather(s, pages, length):
    """[B, length, Hkv, d] rows of a paged tensor (page, slot first), zeros past each sequence."""
    page = s["case"]["page"]
    t = torch.arange(length, device="cuda")
    at = s["table"][:, t // page].long().clamp_min(0) * page + t % page
    rows = pages.reshape((-1,) + pages.shape[2:])[at]
    return rows, t[None, :] < s["seqlens"][:, None]


def _plain_paged(s):
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    nq_max, L, G = s["max_q"], s["max_k"], Hq // Hkv
    k, held = _gather(s, s["k_pages"], L)
    v, _ = _gather(s, s["v_pages"], L)
    k = torch.where(held[..., None, None], k, torch.zeros_like(k)).float()
    v = torch.where(held[..., None, None], v, torch.zeros_like(v)).float()
    n = s["cu_q"][1:] - s["cu_q"][:-1]
    i = torch.arange(nq_max, device="cuda")
    there = i[None, :] < n[:, None]
    row = (s["cu_q"][:-1, None] + i[None, :]).clamp_max(s["total_q"] - 1).long()
    q = s["q"][row].float()  # [B, nq, Hq, d]
    q = q.view(B, nq_max, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nq_max, d)
    x = (q @ k.permute(0, 2, 3, 1)).mul_(s["scale"])
    pos = (s["seqlens"] - n)[:, None] + i[None, :]
    seen = _keep(pos[:, :, None], torch.arange(L, device="cuda"), c["window"], c["sinks"])
    x.view(B, Hkv, G, nq_max, L).masked_fill_(~seen[:, None, None], -math.inf)
    p, lse = _softmax_parts(x)
    del x
    o = (p @ v.transpose(1, 2)).view(B, Hkv, G, nq_max, d).permute(0, 3, 1, 2, 4)
    lse = lse.view(B, Hkv, G, nq_max).permute(0, 3, 1, 2)
    return [o[there].reshape(-1, Hq, d).to(s["q"].dtype), lse[there].reshape(-1, Hq)]


def _plain_write(s):
    c = s["case"]
    page = c["page"]
    n = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    b = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), n, output_size=s["total_q"])
    i = torch.arange(s["total_q"], device="cuda")
    t = i - s["cu_q"].long()[b] + (s["seqlens"].long() - n)[b]
    at, slot = s["table"][b, t // page].long(), t % page
    for name in ("k", "v"):
        scale, codes = _split(s[name].float())
        s[name + "_pages"].view(torch.uint8)[at, slot] = codes.view(torch.uint8)
        s[name + "_scales"][at, :, slot] = scale[..., 0]
    return [s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]]


def _dequantised(s, name, at):
    codes = s[name + "_pages"].view((-1,) + s[name + "_pages"].shape[2:])
    scale = s[name + "_scales"].transpose(1, 2).reshape(-1, s["case"]["Hkv"])
    return codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scale[at][..., None]


def _plain_read(s):
    c = s["case"]
    page = c["page"]
    b = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), s["seqlens"].long(),
                                output_size=s["total_k"])
    t = torch.arange(s["total_k"], device="cuda") - s["cu_k"].long()[b]
    at = s["table"][b, t // page].long() * page + t % page
    return [_dequantised(s, name, at).to(_DT[c["dtype"]]) for name in ("k", "v")]


def _plain_decode8(s):
    c = s["case"]
    B, Hq, Hkv, d, L, page = c["B"], c["Hq"], c["Hkv"], c["d"], s["max_k"], c["page"]
    t = torch.arange(L, device="cuda")
    at = s["table"][:, t // page].long().clamp_min(0) * page + t % page
    held = t[None, :] < s["seqlens"][:, None]
    q = s["q"].float().view(B, Hkv, -1, d)
    x = (q @ _dequantised(s, "k", at).permute(0, 2, 3, 1)).mul_(s["scale"])
    p, lse = _softmax_parts(x.masked_fill_(~held[:, None, None], -math.inf))
    o = p @ _dequantised(s, "v", at).transpose(1, 2)
    return [o.view(B, Hq, d).to(s["q"].dtype), lse.view(B, Hq)]


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------
def _own(s):
    import exact_io_aware_09_gb300 as attn

    c = s["case"]
    if c["kind"] == "window":
        o, lse = attn.attn_fwd_window_sinks(s["q"], s["k"], s["v"], c["window"], c["sinks"],
                                            scale=s["scale"])
        if not c["backward"]:
            return [o, lse]
        return [o, lse, *attn.attn_bwd_window_sinks(s["q"], s["k"], s["v"], o, s["do"], lse,
                                                    c["window"], c["sinks"], scale=s["scale"])]
    if c["kind"] == "paged":
        return list(attn.attn_fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu_q"],
                                        s["seqlens"], s["max_q"], s["max_k"], window=c["window"],
                                        sinks=c["sinks"], scale=s["scale"]))
    cache = (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
    if c["kind"] == "write":
        attn.attn_cache_write_fp8(s["k"], s["v"], *cache, s["table"], s["cu_q"], s["seqlens"])
        return list(cache)
    if c["kind"] == "read":
        return list(attn.attn_cache_read_fp8(*cache, s["table"], s["cu_k"], s["total_k"],
                                             dtype=_DT[c["dtype"]]))
    return list(attn.attn_decode_paged_fp8(s["q"], *cache, s["table"], s["seqlens"], s["max_k"],
                                           scale=s["scale"]))


_PLAIN = {"window": _plain_window, "paged": _plain_paged, "write": _plain_write,
          "read": _plain_read, "decode8": _plain_decode8}


def run(s):
    return _own(s) if own else _PLAIN[s["case"]["kind"]](s)


# --------------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------------
def _attend64(q, k, v, mask, scale, do=None):
    """One head: o, lse (and dq, dk, dv), float64; mask [rows, keys] of what each row sees."""
    logits = torch.einsum("id,jd->ij", q, k) * scale
    logits = torch.where(mask, logits, logits.new_full((), -math.inf))
    lse = torch.logsumexp(logits, 1)
    w = torch.where(mask, torch.exp(logits - lse[:, None]), logits.new_zeros(()))
    o = torch.einsum("ij,jd->id", w, v)
    if do is None:
        return o, lse
    g = torch.einsum("id,jd->ij", do, v)
    g = w * (g - torch.einsum("ij,ij->i", w, g)[:, None])
    return (o, lse, torch.einsum("ij,jd->id", g, k) * scale,
            torch.einsum("ij,id->jd", g, q) * scale, torch.einsum("ij,id->jd", w, do))


def _mask64(nq, nk, window, sinks):
    m = np.tril(np.ones((nq, nk), dtype=bool), nk - nq)
    if window >= 0:
        near = np.triu(np.ones((nq, nk), dtype=bool), nk - nq - window)
        near[:, :sinks] = True
        m &= near
    return torch.from_numpy(m).cuda()


def _tokens(s, b, n):
    """Flat pool rows of sequence b's first n tokens."""
    page = s["case"]["page"]
    return np.concatenate([np.arange(page) + int(p) * page
                           for p in s["table"][b, : -(-n // page)].tolist()] or [[]])[:n].astype(np.int64)


def _rows64(s, name, at):
    x = s[name + "_pages"]
    rows = x.reshape(-1, *x.shape[2:])
    if x.element_size() == 2:
        return rows[at].double()
    f = s[name + "_scales"].double().permute(0, 2, 1).reshape(-1, s["case"]["Hkv"], 1)
    return rows.view(torch.uint8)[at].view(torch.float8_e4m3fn).double() * f[at]


def _quantise64(x):
    """Scale and E4M3 value of each row of x, float64: the nearest of the format's values, the
    one of even mantissa where two are as near."""
    x = x.double()
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 448.0)) / 448.0))
    for step in (1.0, -1.0):  # put right what the logarithm's rounding left
        f = torch.exp2(e + (step if step < 0 else 0.0))
        e = torch.where((top > 448.0 * f) if step > 0 else ((top <= 448.0 * f) & (top > 0)), e + step, e)
    e = e.clamp_min(-126)
    grid = [m * 2.0 ** -9 for m in range(8)]
    grid += [(8 + m) * 2.0 ** (x - 10) for x in range(1, 16) for m in range(8)][:-1]
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    y = x.abs() / torch.exp2(e)[..., None]
    hi = torch.searchsorted(grid, y).clamp(1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - y, y - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.exp2(e), torch.sign(x) * grid[pick]


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "window":
        if c["B"] * c["Hq"] * c["Nq"] * c["Nkv"] * c["d"] * (6 if c["backward"] else 2) > 4e12:
            return None
        m = _mask64(c["Nq"], c["Nkv"], c["window"], c["sinks"])
        G = c["Hq"] // c["Hkv"]
        out = [torch.zeros_like(s["q"], dtype=torch.float64),
               torch.zeros(s["q"].shape[:3], dtype=torch.float64, device="cuda")]
        if c["backward"]:
            out += [torch.zeros_like(s[n], dtype=torch.float64) for n in ("q", "k", "v")]
        for b in range(c["B"]):
            for h in range(c["Hq"]):
                k, v = s["k"][b, h // G].double(), s["v"][b, h // G].double()
                do = s["do"][b, h].double() if c["backward"] else None
                r = _attend64(s["q"][b, h].double(), k, v, m, s["scale"], do)
                out[0][b, h], out[1][b, h] = r[0], r[1]
                if c["backward"]:
                    out[2][b, h] = r[2]
                    out[3][b, h // G] += r[3]
                    out[4][b, h // G] += r[4]
        return out
    nq, nk = _lengths(c)
    if c["kind"] in ("paged", "decode8"):
        if c["kind"] == "decode8":
            nq = np.ones_like(nk)
        if 4.0 * c["Hq"] * float((nq * nk).sum()) * c["d"] > 8e12:
            return None
        G, at_q = c["Hq"] // c["Hkv"], np.concatenate([[0], np.cumsum(nq)])
        o = torch.zeros_like(s["q"], dtype=torch.float64)
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            at = torch.from_numpy(_tokens(s, b, int(nk[b]))).cuda()
            k, v = _rows64(s, "k", at), _rows64(s, "v", at)
            m = _mask64(int(nq[b]), int(nk[b]), c.get("window", -1), c.get("sinks", 0))
            m = m.repeat(G, 1)  # the query heads of a key/value head one after another
            r = slice(int(at_q[b]), int(at_q[b + 1]))
            for h in range(c["Hkv"]):
                q = s["q"][r, h * G:(h + 1) * G].double().transpose(0, 1).reshape(-1, c["d"])
                x, y = _attend64(q, k[:, h], v[:, h], m, s["scale"])
                o[r, h * G:(h + 1) * G] = x.view(G, -1, c["d"]).transpose(0, 1)
                lse[r, h * G:(h + 1) * G] = y.view(G, -1).t()
        return [o, lse]
    if c["kind"] == "read":
        at = torch.from_numpy(np.concatenate([_tokens(s, b, int(n)) for b, n in enumerate(nk)])).cuda()
        return [_rows64(s, "k", at), _rows64(s, "v", at)]
    out = [s["k_pages"].double(), s["v_pages"].double(), s["k_scales"].double(), s["v_scales"].double()]
    new = np.concatenate([_tokens(s, b, int(nk[b]))[nk[b] - nq[b]:] for b in range(c["B"])])
    page, slot = torch.from_numpy(new // c["page"]).cuda(), torch.from_numpy(new % c["page"]).cuda()
    for i, name in enumerate(("k", "v")):
        f, y = _quantise64(s[name])
        out[i][page, slot] = y
        out[i + 2][page, :, slot] = f
    return out
