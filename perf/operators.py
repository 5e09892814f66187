"""Cases of the history cache: block tables and slot maps from request lengths, the append of new
keys and values to 8-bit blocks, and attention over those blocks.

A request's history is held in blocks of `bs` tokens: int8 codes [blocks][kv heads][bs][dim] with one
fp32 scale for each block and head.  512 values of an item vector are 8 heads of 64 or 4 of 128.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def _tables(name, B, cached, new, bs):
    return {"name": name, "op": "tables", "B": B, "cached_lo": cached[0], "cached_hi": cached[1],
            "new_lo": new[0], "new_hi": new[1], "bs": bs}


def _append(name, B, cached, new, Hkv, D, bs, dtype):
    return dict(_tables(name, B, cached, new, bs), op="append", Hkv=Hkv, D=D, dtype=dtype)


def _attend(name, B, cached, new, Hq, Hkv, D, bs, dtype, causal=True, window=0, lse=False):
    return dict(_append(name, B, cached, new, Hkv, D, bs, dtype), op="attend", Hq=Hq, causal=causal,
                window=window, lse=lse)


def listed():
    return [
        # one decode step of a middling batch: the call whose latency a token waits for
        _tables("tables_step_256", 256, (1, 4096), (1, 1), 16),
        # 4,096 requests arrive with their histories
        _tables("tables_admit_4096", 4096, (0, 0), (1, 1024), 16),
        # the new token of every request goes into its last, partly filled block
        _append("append_step_256", 256, (1, 4096), (1, 1), 8, 64, 16, "bf16"),
        # histories of fp32 item vectors (512 = 4 x 128), continued in the middle of blocks
        _append("append_admit_fp32", 64, (0, 100), (1, 4096), 4, 128, 64, "fp32"),
        # a large admission: about 160 thousand tokens
        _append("append_admit_large", 160, (0, 0), (256, 2048), 8, 128, 32, "bf16"),
        # the smallest decode step
        _attend("attend_step_small", 4, (17, 300), (1, 1), 8, 8, 64, 16, "bf16"),
        # an ordinary decode step, ragged histories, grouped heads
        _attend("attend_step_256", 256, (64, 4096), (1, 1), 32, 8, 128, 16, "bf16"),
        # two requests with very long histories: the keys have to be split
        _attend("attend_step_long", 2, (65535, 131071), (1, 1), 16, 4, 128, 64, "fp16", lse=True),
        # 4,096 requests, short fp32 histories of 512-value tokens
        _attend("attend_step_4096_fp32", 4096, (0, 1000), (1, 1), 4, 4, 128, 32, "fp32"),
        # several drafted tokens per request, a window over the history
        _attend("attend_drafts_window", 64, (1, 8192), (1, 7), 16, 2, 64, 16, "bf16", window=1024,
                lse=True),
        # 1,024 candidates of each request look at its history, not at each other
        _attend("attend_candidates", 32, (100, 4096), (1024, 1024), 8, 8, 64, 16, "fp16",
                causal=False),
        # chunks of new history behind what is cached
        _attend("attend_chunks", 6, (0, 8000), (500, 4096), 16, 4, 128, 64, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Another case of the listed ranges, no dearer than the largest listed ones."""
    while True:
        op = rng.choice(["tables", "append", "attend", "attend", "attend"])
        bs = rng.choice([16, 32, 64, 128])
        if op == "tables":
            step = rng.random() < 0.5
            c = _tables("", _log_int(rng, 1, 4096), (0, rng.choice([0, _log_int(rng, 1, 8192)])),
                        (1, 1) if step else (0, _log_int(rng, 1, 1500)), bs)
        else:
            D = rng.choice([32, 64, 128])
            Hkv = rng.choice([1, 2, 3, 4, 8])
            dtype = rng.choice(["bf16", "fp16", "fp32"])
            if op == "append":
                step = rng.random() < 0.5
                c = _append("", _log_int(rng, 1, 1024), (0, _log_int(rng, 1, 4096)),
                            (1, 1) if step else (0, _log_int(rng, 1, 4096)), Hkv, D, bs, dtype)
            else:
                kind = rng.choice(["step", "step", "drafts", "chunk", "candidates"])
                top = {"step": 100000, "drafts": 8192, "chunk": 8000, "candidates": 4096}[kind]
                most = {"step": 1, "drafts": 9, "chunk": 4096, "candidates": 1100}[kind]
                cached = _log_int(rng, 1, top)
                new = _log_int(rng, 1, most)
                c = _attend("", _log_int(rng, 1, 4096 if most < 10 else 40), (cached // 50, cached),
                            (max(1, new // 3), new), Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv, D, bs,
                            dtype, causal=kind != "candidates",
                            window=rng.choice([0, 0, 0, 1000]) if kind != "candidates" else 0,
                            lse=rng.random() < 0.3)
        del c["name"]
        w = work(c)
        if w["bytes"] > 8.4e8 or w["flops"] > 1.3e11 or not _lengths(c)[1].any():
            continue
        if c["op"] == "attend":  # the plain form's padded tensors
            L = c["cached_hi"] + c["new_hi"] + c["bs"]
            if c["B"] * c["Hkv"] * L * c["D"] > 2.2e9 or c["B"] * c["Hq"] * c["new_hi"] * L > 2.3e9:
                continue
        if c["op"] == "tables" and c["B"] * (c["cached_hi"] + c["new_hi"]) > 4e7:
            continue
        return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, even in their logarithm (of x + 1)."""
    if lo == hi:
        return np.full(n, lo, np.int64)
    u = (np.arange(n) + 0.5) / n
    x = np.exp(np.log(lo + 1) + u * (np.log(hi + 1) - np.log(lo + 1))) - 1
    return np.clip(np.rint(x), lo, hi).astype(np.int64)


def _lengths(c):
    """(cached, new) of the case's requests before they are shuffled; the same for every seed."""
    n = c["B"]
    cached = _spread(c["cached_lo"], c["cached_hi"], n)
    new = _spread(c["new_lo"], c["new_hi"], n)
    step = next(s for s in range(max(1, int(n * 0.618)), 2 * n + 2) if math.gcd(s, n) == 1)
    return cached, new[(np.arange(n) * step) % n]


def work(c):
    cached, new = _lengths(c)
    bs, total = c["bs"], int(new.sum())
    if c["op"] == "tables":
        need = int((-(-(cached + new) // bs) - -(-cached // bs)).sum())
        return {"bytes": 16 * c["B"] + 8 * total + 8 * need, "flops": 0}
    Hkv, D, e = c["Hkv"], c["D"], BYTES[c["dtype"]]
    if c["op"] == "append":
        touched = int((-(-(cached + new) // bs) - cached // bs)[new > 0].sum())
        return {"bytes": 2 * total * Hkv * D * (e + 1) + 8 * total + 8 * touched * Hkv, "flops": 0}
    length = cached + new if c["causal"] else cached
    keys, pairs = 0, 0
    for n, L in zip(new.tolist(), length.tolist()):
        if not c["causal"]:
            keys, pairs = keys + L, pairs + n * L
            continue
        last = L - n + np.arange(n) + 1  # keys up to each query's own
        seen = np.minimum(last, c["window"]) if c["window"] else last
        keys += int(L - (last[0] - seen[0])) if n else 0
        pairs += int(seen.sum())
    return {"bytes": 2 * total * c["Hq"] * D * e + 2 * keys * Hkv * (D + 4 / bs) + 4 * keys / bs,
            "flops": 4 * D * c["Hq"] * pairs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    rng = np.random.default_rng(seed)
    g = torch.Generator(DEV).manual_seed(seed)
    B, bs = c["B"], c["bs"]
    cached, new = _lengths(c)
    order = rng.permutation(B)
    cached, new = cached[order], new[order]
    old, every = -(-cached // bs), -(-(cached + new) // bs)
    max_blocks = int(every.max()) + 1
    n_blocks = int(every.sum()) + B // 8 + 2
    total = int(new.sum())
    blocks = torch.randperm(n_blocks, generator=g, device=DEV).int()
    table = torch.full((B, max_blocks), -1, dtype=torch.int32)
    held = old if c["op"] == "tables" else every
    col = np.arange(max_blocks)
    mine = torch.from_numpy(col[None, :] < held[:, None])
    table = table.to(DEV)
    table[mine.to(DEV)] = blocks[: int(held.sum())]
    s = {"op": c["op"], "bs": bs, "table": table, "total": total,
         "cached": torch.from_numpy(cached.astype(np.int32)).to(DEV),
         "new": torch.from_numpy(new.astype(np.int32)).to(DEV)}
    if c["op"] == "tables":
        s["free"] = blocks[int(held.sum()):].contiguous()
        s["free_count"] = torch.full((1,), s["free"].numel(), dtype=torch.int64, device=DEV)
        s["padded"] = total + 3  # a batch padded behind the last request
        return s
    Hkv, D, t = c["Hkv"], c["D"], TYPES[c["dtype"]]

    def codes():
        out = torch.empty((n_blocks, Hkv, bs, D), dtype=torch.int8, device=DEV)
        piece = max(1, (1 << 27) // (Hkv * bs * D))
        for i in range(0, n_blocks, piece):
            x = torch.randn(out[i:i + piece].shape, generator=g, device=DEV)
            out[i:i + piece] = (x * 36).round_().clamp_(-127, 127).to(torch.int8)
        return out

    def scales():
        x = torch.randn((n_blocks, Hkv), generator=g, device=DEV)
        return 0.0275 * torch.exp(0.3 * x)

    s |= {"k_cache": codes(), "v_cache": codes(), "k_scale": scales(), "v_scale": scales()}
    cu = np.zeros(B + 1, np.int64)
    np.cumsum(new, out=cu[1:])
    if c["op"] == "append":
        req = np.repeat(np.arange(B), new)
        pos = torch.from_numpy(cached[req] + np.arange(total) - cu[req]).to(DEV)
        blk = table[torch.from_numpy(req).to(DEV), pos // bs].long()
        s["slots"] = blk * bs + pos % bs
        s["k"] = torch.randn((total, Hkv, D), generator=g, device=DEV).to(t)
        s["v"] = torch.randn((total, Hkv, D), generator=g, device=DEV).to(t)
        return s
    s["q"] = torch.randn((total, c["Hq"], D), generator=g, device=DEV).to(t)
    s["cu_new"] = torch.from_numpy(cu.astype(np.int32)).to(DEV)
    s["seq_len"] = s["cached"] + s["new"] if c["causal"] else s["cached"].clone()
    s |= {"max_new": int(new.max()), "causal": c["causal"], "window": c["window"], "lse": c["lse"]}
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)


def _own(s):
    from hashed_sparse_table_b200 import binding as b
    if s["op"] == "tables":
        B = s["cached"].numel()
        cu = torch.empty(B + 1, dtype=torch.int32, device=DEV)
        seq = torch.empty(B, dtype=torch.int32, device=DEV)
        slots = torch.empty(s["padded"], dtype=torch.int64, device=DEV)
        left = torch.empty(1, dtype=torch.int64, device=DEV)
        b.mpzch_kv_tables(s["cached"], s["new"], s["bs"], s["free"], s["free_count"], s["table"], cu,
                          seq, slots, left)
        return [s["table"], cu, seq, slots, left]
    if s["op"] == "append":
        b.mpzch_kv_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"],
                          s["v_scale"])
        return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], device=DEV) if s["lse"] else None
    b.mpzch_kv_attend(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                      s["cu_new"], s["seq_len"], s["max_new"], out, causal=s["causal"],
                      window=s["window"], lse=lse)
    return [out, lse] if s["lse"] else [out]


def _plain_tables(s):
    bs, table = s["bs"], s["table"]
    B, width = table.shape
    cached, new = s["cached"].long(), s["new"].long()
    end = torch.cumsum(new, 0)
    start = end - new
    old, every = (cached + bs - 1) // bs, (cached + new + bs - 1) // bs
    bad = (cached < 0) | (new < 0) | (every > width) | (end > s["padded"])
    need = torch.where(bad, 0, every - old)
    upto = torch.cumsum(need, 0)
    count = s["free_count"]
    ok = ~bad & ((need == 0) | (upto <= count))
    col = torch.arange(width, device=DEV)
    fresh = ok[:, None] & (col >= old[:, None]) & (col < every[:, None])
    at = count - 1 - ((upto - need)[:, None] + col - old[:, None])
    table.copy_(torch.where(fresh, s["free"][at.clamp(0, s["free"].numel() - 1)], table))
    row = torch.arange(s["padded"], device=DEV)
    req = torch.searchsorted(end, row, right=True).clamp(max=B - 1)
    pos = cached[req] + row - start[req]
    blk = table[req, (pos // bs).clamp(0, width - 1)].long()
    slots = torch.where((row < end[-1]) & ok[req], blk * bs + pos % bs, -1)
    cu = torch.cat([torch.zeros_like(end[:1]), end]).int()
    left = count - torch.where(ok, upto, 0).max()
    return [table, cu, torch.where(ok, cached + new, cached).int(), slots, left]


def _plain_append(s):
    slots, bs = s["slots"], s["k_cache"].shape[2]
    blk, off = slots // bs, slots % bs
    first = torch.ones_like(slots, dtype=torch.bool)
    first[1:] = (slots[1:] != slots[:-1] + 1) | (off[1:] == 0)
    run_of = torch.cumsum(first, 0) - 1
    n = slots.numel()
    # one entry per batch row, of which the first ones are runs: no count is brought to the host
    most = min(n, n // bs + 2 * s["cached"].numel())
    run_blk = torch.zeros_like(slots).index_put_((run_of,), blk)
    held = torch.full_like(slots, bs).scatter_reduce_(0, run_of, off, "amin")
    real = torch.arange(n, device=DEV) <= run_of[-1]
    step = torch.arange(bs, device=DEV)
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x.float()
        a = torch.zeros((n, x.shape[1]), device=DEV).index_reduce_(0, run_of, x.abs().amax(2), "amax")
        before = torch.where(held[:, None] > 0, scale[run_blk], 0.0)
        after = torch.maximum(before, a / torch.tensor(127.0, device=DEV))
        kept = cache[run_blk[:most]]
        f, g = before[:most, :, None, None], after[:most, :, None, None]
        old = (step < held[:most, None])[:, None, :, None] & (f != g)
        fresh = torch.where(old, _codes(kept.float() * f, g), kept)
        # rows that are no run repeat the first one
        fresh = torch.where(real[:most, None, None, None], fresh, fresh[:1])
        cache.index_copy_(0, torch.where(real[:most], run_blk[:most], run_blk[0]), fresh)
        cache[blk, :, off] = _codes(x, after[run_of][:, :, None])
        scale.index_copy_(0, torch.where(real, run_blk, run_blk[0]),
                          torch.where(real[:, None], after, after[:1]))
    return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _codes(x, scale):
    q = torch.where(scale > 0, x / scale, 0.0)
    return q.round().clamp(-127, 127).to(torch.int8)


def _plain_attend(s):
    q, table, bs = s["q"], s["table"], s["bs"]
    B, width = table.shape
    N, Hq, D = q.shape
    Hkv = s["k_cache"].shape[1]
    G, T = Hq // Hkv, s["max_new"]
    cu, seq = s["cu_new"].long(), s["seq_len"].long()
    new = cu[1:] - cu[:-1]
    t = torch.arange(T, device=DEV)
    key = torch.arange(width * bs, device=DEV)
    pos = (seq - new)[:, None] + t  # [B, T]
    sees = (key < seq[:, None, None]).expand(B, T, width * bs)
    if s["causal"]:
        sees = sees & (key <= pos[:, :, None])
    if s["window"]:
        sees = sees & (key > pos[:, :, None] - s["window"])
    tab = table.clamp(min=0).long()

    def held(cache, scale):
        x = cache[tab].float() * scale[tab][..., None, None]  # [B, width, Hkv, bs, D]
        return x.transpose(1, 2).reshape(B, Hkv, width * bs, D)

    rows = q[(cu[:-1, None] + t).clamp(max=N - 1)].float()  # [B, T, Hq, D]
    rows = rows.view(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    w = rows @ held(s["k_cache"], s["k_scale"]).transpose(2, 3)
    w = (w * (1 / math.sqrt(D))).view(B, Hkv, G, T, -1)
    w.masked_fill_(~sees[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = w.sum(-1, keepdim=True)
    o = (w.view(B, Hkv, G * T, -1) @ held(s["v_cache"], s["v_scale"])).view(B, Hkv, G, T, D)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D)
    row = torch.arange(N, device=DEV)
    req = torch.searchsorted(cu[1:], row, right=True)
    out = o[req, row - cu[req]].to(q.dtype)
    if not s["lse"]:
        return [out]
    lse = (top + total.log()).permute(0, 3, 1, 2, 4).reshape(B, T, Hq)
    return [out, lse[req, row - cu[req]]]


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None  # whole numbers only
    if case["op"] == "append":
        return _exact_scales(s)
    N, Hq, D = s["q"].shape
    Hkv, bs = s["k_cache"].shape[1], s["bs"]
    out = torch.zeros((N, Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((N, Hq), -math.inf, dtype=torch.float64, device=DEV)
    cu, seq = s["cu_new"].tolist(), s["seq_len"].tolist()
    for b, L in enumerate(seq):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo or L == 0:
            continue
        ids = s["table"][b, : -(-L // bs)].long()
        k = s["k_cache"][ids].double() * s["k_scale"][ids].double()[:, :, None, None]
        v = s["v_cache"][ids].double() * s["v_scale"][ids].double()[:, :, None, None]
        k = torch.einsum("nhtd->hntd", k).reshape(Hkv, -1, D)[:, :L]
        v = torch.einsum("nhtd->hntd", v).reshape(Hkv, -1, D)[:, :L]
        at = torch.arange(lo, hi, device=DEV) - hi + L
        far = at[:, None] - torch.arange(L, device=DEV)[None]
        hide = torch.zeros_like(far, dtype=torch.bool)
        if s["causal"]:
            hide |= far < 0
        if s["window"]:
            hide |= far >= s["window"]
        rows = s["q"][lo:hi].double().unflatten(1, (Hkv, Hq // Hkv))
        z = torch.einsum("nhgd,hld->nhgl", rows, k) / D ** 0.5
        z = z.masked_fill(hide[:, None, None], -math.inf)
        n = torch.logsumexp(z, 3)
        lse[lo:hi] = n.flatten(1)
        p = torch.exp(z - n[..., None])  # a row that sees nothing: NaN, and then 0
        out[lo:hi] = torch.einsum("nhgl,hld->nhgd", p.nan_to_num(nan=0.0), v).flatten(1, 2)
    return [out, lse] if case["lse"] else [out]


def _exact_scales(s):
    """The blocks' scales after the append; the codes are whole numbers."""
    bs = s["k_cache"].shape[2]
    blk, off = s["slots"] // bs, s["slots"] % bs
    new = [None, None]
    for x, name in ((s["k"], "k_scale"), (s["v"], "v_scale")):
        scale = s[name].double().clone()
        # a block that gets its first token forgets the scale that it had
        scale[blk[off == 0]] = 0.0
        a = x.double().abs().amax(2) / 127
        at = blk[:, None].expand(a.shape)
        new.append(scale.scatter_reduce(0, at, a, "amax"))
    return new
