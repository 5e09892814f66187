"""History cache on the GPU at the ends of its number ranges: value scales near the smallest and
the largest numbers of binary32, held codes under negative scales, and weights that lie in blocks
far smaller than their neighbours."""
import numpy as np
import pytest
import torch

import kv_ref as ref
from test_gpu_kv import dev, history, kv, make_cache, run_append  # noqa: F401 (kv: fixture)

pytestmark = pytest.mark.gpu


def attend(kv, c, causal=False, window=0, scale=0.125):
    """(out, want, size) for the case, rows of no request not expected."""
    q = c["q"].cuda()
    out = torch.full_like(q, 7.0)
    kv.mpzch_kv_attend(q, *(dev(c[x]) for x in ("kc", "vc", "ks", "vs", "table", "cu", "seq")),
                       int(np.diff(c["cu"]).max()), out, softmax_scale=scale, causal=causal,
                       window=window)
    want, _, size = ref.attend(c["q"].double().numpy(), c["kc"], c["vc"], c["ks"], c["vs"],
                               c["table"], c["cu"], c["seq"], scale, causal, window)
    return out.double().cpu().numpy(), want, size


def bound(want, size, keys, D, kind, low=None):
    """ref.attend_bound without its absolute allowance: `low` (the same as size[2], for the weights
    that are subnormal in fp16) if given, what the smallest reference of the weights, 2^-119,
    leaves (2^-25 2^-7 2^-118 for each code), and half a step of the smallest numbers of the type
    and of binary32 (two roundings there)."""
    spread, reach, codes = size
    half = {"bf16": 2.0**-8, "fp16": 2.0**-11, "fp32": 2.0**-24}[kind]
    tiny = {"bf16": 2.0**-134, "fp16": 2.0**-25, "fp32": 0.0}[kind] + 2.0**-149
    full = ref.attend_bound(want, (spread, reach, codes if low is None else low), keys, D, kind)
    full -= 1e-37 + (2.0**-25 if kind == "fp16" else 0.0)
    return full + tiny + keys * 127 * 2.0**-150 * (1 + half)


# ------------------------------------------------------------------ attention: smallest scales
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("size", [2.0**-121, 2.0**-122, 1e-40, 1e-44])
@pytest.mark.parametrize("length", [100, 3000])
def test_attend_smallest_value_scales(kv, kind, rows, size, length):
    """Every block of one request next to nothing; of the next one the first blocks alone, in
    front of ordinary ones; of the third every other."""
    c = history(50, [length] * 3, [rows] * 3, 2, 2, 64, 16, kind)
    n = -(-length // 16)
    small = np.float32(size) * (1 + np.arange(n) % 3).astype(np.float32)[:, None]
    c["vs"][c["table"][0, :n]] = small
    c["vs"][c["table"][1, :3]] = small[:3]
    c["vs"][c["table"][2, :n:2]] = small[::2]
    got, want, s = attend(kv, c)
    assert np.isfinite(got).all()
    for b in range(3):
        at = slice(b * rows, b * rows + rows)
        mine = tuple(x[at] for x in s)
        assert (np.abs(got - want)[at] <= bound(want[at], mine, length, 64, kind)).all(), b
    assert kind == "fp16" or size < 1e-40 or (got[:rows] != 0).any()


# ------------------------------------------------------------------ append: held codes
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,bs", [(32, 16), (128, 128)])
def test_append_behind_negative_scales_and_lowest_codes(kv, kind, D, bs):
    """Held codes whose quotient passes 127: the old scale is negative and larger than the new one
    (by little, by much, beyond the range of the packed quotient), or the code is -128."""
    rng = np.random.default_rng(51)
    H, blocks = 2, 24
    kc, ks = make_cache(rng, blocks, H, bs, D)
    vc, vs = make_cache(rng, blocks, H, bs, D)
    for cache in (kc, vc):
        cache[:, :, ::3] = -128
        cache[:, :, 1::5, 3] = 100
    size = np.float32(10.0) ** rng.uniform(-3, 8, (blocks, H)).astype(np.float32)
    ks[:12], vs[4:16] = -size[:12], -size[4:16]
    ks[20], vs[20] = -1e-30, 1e-30
    ks[21], vs[21] = -3e38, -1e-40
    slots = np.concatenate([b * bs + np.arange(9, 12) for b in range(blocks)])
    k, v = (rng.standard_normal((len(slots), H, D)).astype(np.float32) for _ in range(2))
    at = slice(20 * 3, 22 * 3)
    if kind != "fp16":
        k[at] *= np.float32(1e-31)
        v[at] *= np.float32(1e-31)
    k[3 * 3:4 * 3], v[5 * 3:6 * 3] = 0, 0  # the new scale is 0
    run_append(kv, k, v, slots, kc, vc, ks, vs, kind)


# ------------------------------------------------------------------ attention: largest values
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("length", [100, 20000])
def test_attend_largest_values(kv, kind, rows, length):
    """Values whose sum passes the range of binary32 and whose mean does not."""
    c = history(52, [length, 60], [rows] * 2, 2, 1, 64, 16, kind)
    c["vs"][:] = np.float32(2.0**120)
    c["vc"] = (np.abs(c["vc"].astype(np.int16)) // 2 + 60).astype(np.int8)
    got, want, s = attend(kv, c)
    assert np.abs(want).max() > 2.0**126
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= bound(want, s, length, 64, kind)).all()


# ------------------------------------------------------------------ attention: uneven scales
def products(c, scale, causal=False):
    """The largest of (softmax weight times value scale) over the keys of each row and head, times
    the sum of |code| over the keys: what bounds the bits that weights lose below fp16's normal
    numbers when their reference is the row's own largest product."""
    q = c["q"].double().numpy()
    n, Hq, D = q.shape
    H, bs = c["kc"].shape[1:3]
    low = np.zeros(q.shape)
    for b, L in enumerate(c["seq"]):
        s, e = int(c["cu"][b]), int(c["cu"][b + 1])
        ids = c["table"][b, :-(-int(L) // bs)]
        pos = int(L) - (e - s) + np.arange(e - s)[:, None]
        for hq in range(Hq):
            h = hq // (Hq // H)
            k = (c["kc"][ids, h].astype(float) * c["ks"][ids, h].astype(float)[:, None, None])
            z = scale * q[s:e, hq] @ k.reshape(-1, D)[:L].T
            if causal:
                z = np.where(np.arange(L)[None] <= pos, z, -np.inf)
            p = np.exp(z - z.max(1, keepdims=True))
            sees = np.isfinite(z)
            p /= p.sum(1, keepdims=True)
            each = np.repeat(np.abs(c["vs"][ids, h].astype(float)), bs)[:L]
            codes = np.abs(c["vc"][ids, h].astype(float)).reshape(-1, D)[:L]
            low[s:e, hq] = (p * each).max(1)[:, None] * (sees @ codes)
    return low


def leaning(seed, lens, rows, kind, gap, Hq=2, H=2, order=1):
    """A history in which the first or the second half of a request's blocks holds the keys that a
    row attends to: even rows look at small blocks, odd ones at large ones, whose value scales are
    2^gap apart, and a score of about 40 (in log2 units) lies between the two kinds of keys."""
    c = history(seed, lens, [rows] * len(lens), Hq, H, 64, 16, kind)
    sign = 1 - 2 * (np.arange(len(c["q"])) % 2)
    q = c["q"].float() * 0.1
    q[:, :, 0] = torch.from_numpy(4.0 * sign).float()[:, None]
    c["q"] = q.to(c["q"].dtype)
    for b, L in enumerate(lens):
        n = -(-L // 16)
        ids = c["table"][b, :n]
        small = np.arange(n) % 2 == 0 if order == 0 else (np.arange(n) < n // 2) == (order > 0)
        c["kc"][ids[small], :, :, 0] = 127
        c["kc"][ids[~small], :, :, 0] = -127
        c["ks"][ids] = 0.2
        c["vs"][ids] = (np.where(small, 2.0**-gap, 1.0)[:, None]
                        * (1 + 0.3 * np.arange(n) / n)[:, None]).astype(np.float32)
    return c


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows", [1, 2, 40, 150])
@pytest.mark.parametrize("gap", [13, 24, 36])
@pytest.mark.parametrize("order", [1, -1, 0])
def test_attend_weights_in_blocks_of_small_scale(kv, kind, rows, gap, order):
    """Nearly all weight lies on keys whose values are 2^gap below those of their neighbours, in
    front of them, behind them and in turn: the output keeps the small values' bits, and rows of
    the same tile that look at the large ones keep theirs."""
    c = leaning(53, [300, 2000, 33], rows, kind, gap, order=order)
    got, want, s = attend(kv, c, scale=0.15)
    low = products(c, 0.15)
    # weights in fp16 parts end at 2^-32 of the row's largest product
    off = bound(want, s, 2000, 64, kind, low)
    assert (np.abs(got - want) <= off).all(), np.max(np.abs(got - want) / off)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [1, 40])
def test_attend_large_values_that_later_scores_outweigh(kv, kind, rows):
    """Scores that rise from block to block by hundreds while the value scales fall: what came
    first is large but has no weight in the end."""
    for scale in (0.05, 1.0, 20.0):
        c = history(54, [900, 60], [rows] * 2, 2, 2, 64, 16, kind)
        c["q"] = (torch.ones_like(c["q"]) + 0.01 * c["q"].float()).to(c["q"].dtype)
        for b, n in enumerate((57, 4)):
            ids = c["table"][b, :n]
            c["kc"][ids] = (np.linspace(-100, 100, n)[:, None, None, None]
                            + np.random.default_rng(55).integers(-20, 20, c["kc"][ids].shape)).astype(np.int8)
            c["ks"][ids] = 0.02
            c["vs"][ids] = np.float32(2.0) ** np.linspace(20, -20, n)[:, None]
        got, want, s = attend(kv, c, scale=scale)
        low = products(c, scale)
        off = bound(want, s, 900, 64, kind, low)
        assert (np.abs(got - want) <= off).all(), (scale, np.max(np.abs(got - want) / off))
