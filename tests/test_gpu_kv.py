"""History cache on the GPU: block tables and slots, the int8 append (both bit for bit) and
attention (against 64 bits, bounds from the kernels' roundings: tests/kv_ref.py)."""
import numpy as np
import pytest
import torch

import kv_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def kv():
    from hashed_sparse_table_b200 import binding
    torch.cuda.set_device(0)
    return binding


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def host(t):
    return t.detach().cpu().numpy()


# ------------------------------------------------------------------ block tables
def run_tables(kv, cached, new, bs, free, count, table, n_slots, shift=0):
    B = len(cached)
    cu = torch.full((B + 1,), -7, dtype=torch.int32, device="cuda")
    seq = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((n_slots + shift,), -7, dtype=torch.int64, device="cuda")[shift:]
    left = torch.full((1,), -7, dtype=torch.int64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tab = dev(table)
    before = kv.mpzch_launch_count()
    kv.mpzch_kv_tables(dev(cached), dev(new), bs, dev(free), dev(np.array([count], np.int64)), tab,
                       cu, seq, slots, left, status)
    assert kv.mpzch_launch_count() == before + 1
    got = host(tab), host(cu), host(seq), host(slots), int(left), int(status)
    want = ref.tables(cached, new, bs, free, count, table, n_slots)
    for name, g, w in zip(("table", "cu_new", "seq_len", "slots", "left", "status"), got, want):
        assert np.array_equal(g, w), name
    return got


def tables_case(seed, B, bs, most_cached, most_new, spare=5, width=None):
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, most_cached + 1, B).astype(np.int32)
    new = rng.integers(0, most_new + 1, B).astype(np.int32)
    width = width or (most_cached + most_new) // bs + 2
    old = -(-cached.astype(np.int64) // bs)
    need = int((-(-(cached.astype(np.int64) + new) // bs) - old).sum())
    ids = rng.permutation(int(old.sum()) + need + spare).astype(np.int32)
    table = np.full((B, width), -3, np.int32)
    table[np.arange(width)[None, :] < old[:, None]] = ids[:int(old.sum())]
    return cached, new, ids[int(old.sum()):], table, int(new.sum())


@pytest.mark.parametrize("B,bs,most_cached,most_new", [
    (1, 16, 0, 1), (1, 16, 40, 0), (3, 32, 100, 1), (7, 64, 0, 300), (256, 16, 500, 1),
    (255, 128, 500, 40), (1023, 16, 64, 3), (1024, 16, 64, 9), (1025, 16, 64, 9),
    (4096, 16, 30, 20), (4097, 32, 30, 20), (16384, 16, 20, 2)])
def test_tables_match_the_definition(kv, B, bs, most_cached, most_new):
    cached, new, free, table, total = tables_case(B, B, bs, most_cached, most_new)
    got = run_tables(kv, cached, new, bs, free, len(free), table, total)
    assert got[5] == 0
    # room behind the last request is filled with -1, whatever the slots' alignment
    run_tables(kv, cached, new, bs, free, len(free), table, total + 9, shift=1)


def test_tables_without_requests_rows_or_blocks(kv):
    e = np.zeros(0, np.int32)
    run_tables(kv, e, e, 16, e, 0, np.zeros((0, 4), np.int32), 5)
    run_tables(kv, e, e, 16, e, 0, np.zeros((0, 0), np.int32), 0)
    z = np.zeros(3, np.int32)
    got = run_tables(kv, z, z, 16, e, 0, np.zeros((3, 0), np.int32), 0)
    assert got[5] == 0
    run_tables(kv, z, z + 1, 16, e, 0, np.zeros((3, 0), np.int32), 3)  # no room for a block


def test_tables_one_long_request(kv):
    cached, new = np.array([5, 1, 17], np.int32), np.array([0, 300001, 2], np.int32)
    width = 300100 // 16
    free = np.random.default_rng(1).permutation(20000).astype(np.int32)
    table = np.full((3, width), -1, np.int32)
    table[:, 0], table[2, 1] = [20001, 20002, 20003], 20004
    run_tables(kv, cached, new, 16, free, len(free), table, 300003)


@pytest.mark.parametrize("count", [0, 1, 37, 150, 10**6, -5])
def test_tables_short_list_serves_requests_in_order(kv, count):
    cached, new, free, table, total = tables_case(11, 200, 16, 60, 40)
    got = run_tables(kv, cached, new, 16, free, count, table, total)
    assert (got[5] & ref.NOBLOCK != 0) == (count < len(free) - 5)


def test_tables_refuse_single_requests(kv):
    cached, new, free, table, total = tables_case(12, 300, 16, 60, 40)
    cached[5], cached[6], new[9] = -1, -(2**31), -4
    cached[20], new[21] = 2**31 - 1, 2**31 - 1
    new[30] = table.shape[1] * 16 + 1 - cached[30]
    got = run_tables(kv, cached, new, 16, free, len(free), table, total)
    assert got[5] & ref.BADLEN
    # rows past the room for slots
    cached, new, free, table, total = tables_case(13, 300, 16, 60, 40)
    run_tables(kv, cached, new, 16, free, len(free), table, total - 700)
    run_tables(kv, cached, new, 16, free, len(free), table, 0)
    # the sum of the lengths passes 31 bits
    new[:] = 2**30
    run_tables(kv, cached, new, 16, free, len(free), table, 100)


# ------------------------------------------------------------------ append
def make_cache(rng, blocks, H, bs, D):
    q = rng.integers(-127, 128, (blocks, H, bs, D)).astype(np.int8)
    s = (0.02 * np.exp(rng.standard_normal((blocks, H)))).astype(np.float32)
    return q, s


def as_type(x, kind):
    """(torch tensor of the type, its values as float32)"""
    t = torch.from_numpy(x).to(TYPES[kind])
    return t.cuda(), t.float().numpy()


def run_append(kv, k, v, slots, kc, vc, ks, vs, kind, fused=False):
    kt, kx = as_type(k, kind)
    vt, vx = as_type(v, kind)
    if fused:  # slices of one projection's output
        both = torch.cat([kt, vt], 1)
        kt, vt = both[:, :k.shape[1]], both[:, k.shape[1]:]
    c = [dev(x) for x in (kc, vc, ks, vs)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.mpzch_kv_append(kt, vt, dev(slots), *c, status)
    kc, vc, ks, vs = kc.copy(), vc.copy(), ks.copy(), vs.copy()
    bits = ref.append(kx, slots, kc, ks) | ref.append(vx, slots, vc, vs)
    for name, g, w in zip(("k_scale", "v_scale"), c[2:], (ks, vs)):
        assert np.array_equal(host(g), w, equal_nan=True), name
    for name, g, w in zip(("k_cache", "v_cache"), c[:2], (kc, vc)):
        assert np.array_equal(host(g), w), name
    assert int(status) == bits
    return kc, vc, ks, vs


def slots_of(rng, cached, new, bs, blocks):
    """Slots of requests whose blocks are drawn without repetition."""
    ids, out = iter(rng.permutation(blocks)), []
    for c, w in zip(cached, new):
        mine = [next(ids) for _ in range(c // bs, -(-(c + w) // bs))]
        pos = c + np.arange(w)
        out.append(np.array(mine, np.int64)[pos // bs - c // bs] * bs + pos % bs if w else
                   np.zeros(0, np.int64))
    return np.concatenate(out)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,bs,H", [(32, 16, 3), (64, 32, 2), (128, 16, 1), (128, 64, 4),
                                    (64, 128, 2), (32, 128, 1), (128, 128, 2)])
def test_append_matches_the_definition_bit_for_bit(kv, kind, D, bs, H):
    rng = np.random.default_rng(D * bs + H)
    cached = [0, 5, bs - 1, bs, 3 * bs + 2, 0, 7, 1, 2 * bs - 1]
    new = [1, 1, 1, 1, 4 * bs + 3, bs, 0, bs - 1, 2]
    slots = slots_of(rng, cached, new, bs, 40)
    kc, ks = make_cache(rng, 40, H, bs, D)
    vc, vs = make_cache(rng, 40, H, bs, D)
    # sizes below and above the held tokens', so that some scales grow and some stay
    k, v = (rng.standard_normal((len(slots), H, D)).astype(np.float32)
            * np.exp(1.5 * rng.standard_normal((len(slots), 1, 1))).astype(np.float32)
            for _ in range(2))
    done = run_append(kv, k, v, slots, kc, vc, ks, vs, kind, fused=True)
    run_append(kv, k, v, slots, *done, kind)  # the same again: nothing is requantised


@pytest.mark.parametrize("n", [1, 31, 300, 5000])
def test_append_of_single_tokens(kv, n):
    """One token of each of n requests, as in a decode step, some padded."""
    rng = np.random.default_rng(n)
    H, D, bs = 2, 64, 16
    cached = rng.integers(0, 200, n)
    slots = slots_of(rng, cached, [1] * n, bs, n)
    slots[rng.random(n) < 0.1] = -1
    kc, ks = make_cache(rng, n, H, bs, D)
    vc, vs = make_cache(rng, n, H, bs, D)
    k, v = (rng.standard_normal((n, H, D)).astype(np.float32) for _ in range(2))
    run_append(kv, k, v, slots, kc, vc, ks, vs, "bf16")


def test_append_of_a_long_batch(kv):
    rng = np.random.default_rng(3)
    H, D, bs = 4, 64, 32
    new = rng.integers(0, 900, 40)
    cached = rng.integers(0, 100, 40)
    slots = slots_of(rng, cached, new, bs, 1000)
    kc, ks = make_cache(rng, 1000, H, bs, D)
    vc, vs = make_cache(rng, 1000, H, bs, D)
    k, v = (rng.standard_normal((len(slots), H, D)).astype(np.float32) for _ in range(2))
    run_append(kv, k, v, slots, kc, vc, ks, vs, "fp16")


def test_append_zeros_nan_infinities_and_subnormals(kv):
    rng = np.random.default_rng(4)
    H, D, bs = 2, 32, 16
    kc, ks = make_cache(rng, 12, H, bs, D)
    vc, vs = make_cache(rng, 12, H, bs, D)
    ks[1, 0], ks[2, 1], vs[3, 0] = np.nan, np.inf, 0.0
    slots = np.concatenate([b * bs + np.arange(4, 9) for b in range(6)] +
                           [b * bs + np.arange(0, 3) for b in range(6, 12)])
    k, v = (rng.standard_normal((len(slots), H, D)).astype(np.float32) for _ in range(2))
    k[6, 0, 3], k[11, 1, 4], v[16, 1, 0], v[21, 0, 31] = np.nan, np.inf, -np.inf, np.nan
    k[30:33], v[33:36] = 0.0, -0.0          # a fresh block of zeros: scale 0
    k[36:39] *= np.float32(1e-40)           # subnormal scale
    v[36:39] *= np.float32(1e-44)
    k[39:42] *= np.float32(1e38)
    run_append(kv, k, v, slots, kc, vc, ks, vs, "fp32")


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_append_halves_between_two_codes(kv, kind):
    """Values whose quotient by the scale lies on a half or a rounding away from one, for block
    maxima over the whole exponent range of the type."""
    rng = np.random.default_rng(6)
    H, D, bs, blocks = 1, 128, 16, 300
    low, high = {"bf16": (-126, 120), "fp16": (-14, 15), "fp32": (-126, 120)}[kind]
    top = np.ldexp(1 + rng.random(blocks), rng.integers(low, high, blocks)).astype(np.float32)
    top = torch.from_numpy(top).to(TYPES[kind]).float().numpy()
    x = np.zeros((blocks, bs, H, D), np.float32)
    scale = top / np.float32(127)
    half = (rng.integers(-127, 127, x.shape) + 0.5).astype(np.float32)
    with np.errstate(over="ignore", under="ignore"):
        x = half * scale[:, None, None, None]
        off = rng.integers(-2, 3, x.shape)
        x = (x.view(np.int32) + np.where(x != 0, off, 0).astype(np.int32)).view(np.float32)
    x = np.clip(x, -top[:, None, None, None], top[:, None, None, None])
    x[:, 0, 0, 0] = top
    # and halves by construction: powers of two below the maximum
    x[:, 1, 0] = top[:, None] * np.ldexp(1.0, -rng.integers(0, 9, D)).astype(np.float32)
    x = x.reshape(blocks * bs, H, D)
    kc, ks = make_cache(rng, blocks, H, bs, D)
    slots = np.arange(blocks * bs, dtype=np.int64)
    run_append(kv, x, -x[::-1].copy(), slots, kc, kc.copy(), ks, ks.copy(), kind)


def test_append_skips_bad_slots(kv):
    rng = np.random.default_rng(5)
    H, D, bs = 1, 128, 16
    kc, ks = make_cache(rng, 6, H, bs, D)
    vc, vs = make_cache(rng, 6, H, bs, D)
    slots = np.array([-1, 0, 1, -1, 2 * bs + 15, 3 * bs, 6 * bs, 2**62, -2**63, 5 * bs + 4, 5 * bs + 5,
                      6 * bs - 1, 6 * bs], np.int64)
    k, v = (rng.standard_normal((len(slots), H, D)).astype(np.float32) for _ in range(2))
    slots[11] = -1
    run_append(kv, k, v, slots, kc, vc, ks, vs, "fp32")
    run_append(kv, k[:0], v[:0], slots[:0], kc, vc, ks, vs, "fp32")


# ------------------------------------------------------------------ attention
def history(seed, lens, new, Hq, H, D, bs, kind, spare=3):
    rng = np.random.default_rng(seed)
    B = len(lens)
    used = [-(-L // bs) for L in lens]
    blocks = sum(used) + spare
    ids = rng.permutation(blocks)
    width = max(used, default=0) + 2
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at:at + u]
        at += u
    kc, ks = make_cache(rng, blocks, H, bs, D)
    vc, vs = make_cache(rng, blocks, H, bs, D)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((int(cu[-1]), Hq, D)).astype(np.float32))
    return dict(q=q.to(TYPES[kind]), kc=kc, vc=vc, ks=ks, vs=vs, table=table, cu=cu,
                seq=np.array(lens, np.int32), kind=kind)


def run_attend(kv, c, causal=True, window=0, scale=None, lse=True, out=None, q=None, status=0,
               **options):
    D = c["q"].shape[2]
    scale = D ** -0.5 if scale is None else scale
    q = c["q"].cuda() if q is None else q
    out = torch.full_like(q, 7.0) if out is None else out
    got_lse = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    bits = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = np.diff(c["cu"]).max(initial=0)
    kv.mpzch_kv_attend(q, dev(c["kc"]), dev(c["vc"]), dev(c["ks"]), dev(c["vs"]), dev(c["table"]),
                       dev(c["cu"]), dev(c["seq"]), int(w), out, softmax_scale=scale,
                       causal=causal, window=window, lse=got_lse, status=bits, **options)
    assert int(bits) == status
    check_attend(c, out, got_lse, scale, causal, window)
    return out, got_lse


def check_attend(c, out, got_lse, scale, causal, window):
    want, lse, size = ref.attend(c["q"].double().numpy(), c["kc"], c["vc"], c["ks"],
                                          c["vs"], c["table"], c["cu"], c["seq"], scale, causal,
                                          window)
    rows = np.zeros(len(want), bool)
    for s, e in zip(c["cu"][:-1], c["cu"][1:]):
        rows[max(int(s), 0):max(int(e), 0)] = True
    got = out.double().cpu().numpy()
    assert (got[~rows] == 7.0).all(), "a row of no request was written"
    keys = int(max(c["seq"].max(initial=0), 1))
    D, kind = got.shape[2], c["kind"]
    nan = np.isnan(want[rows])
    assert np.array_equal(np.isnan(got[rows]), nan)
    bound = ref.attend_bound(want, size, keys, D, kind)[rows]
    if kind == "fp16":  # results past the type's range (65,520 and up round to infinity)
        over = np.abs(want[rows]) - bound >= 65520
        assert (got[rows][over] == np.copysign(np.inf, want[rows][over])).all()
        edge = over | (np.abs(want[rows]) + bound >= 65504)
        got, want = got.copy(), want.copy()
        got[rows] = np.where(edge, 0, got[rows])
        want[rows] = np.where(edge, 0, want[rows])
    off = np.abs(got - want)[rows]
    worst = np.nanmax(off / bound, initial=0.0)
    assert worst <= 1.0, worst
    if got_lse is not None:
        g = host(got_lse).astype(np.float64)
        assert (g[~rows] == 7.0).all()
        empty = np.isneginf(lse[rows])
        assert np.array_equal(np.isneginf(g[rows]), empty)
        fine = np.isfinite(lse) & rows[:, None]
        assert (np.abs(g[fine] - lse[fine]) <= ref.lse_bound(size, keys, D, kind)[fine]).all()


ODD_LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("Hq,H,D,bs", [(1, 1, 32, 16), (4, 2, 64, 16), (3, 3, 128, 64),
                                       (8, 1, 128, 16), (5, 1, 64, 128), (32, 2, 32, 32),
                                       (17, 1, 128, 32)])
def test_attend_single_tokens(kv, kind, Hq, H, D, bs):
    c = history(Hq * D + bs, ODD_LENGTHS, [1] * len(ODD_LENGTHS), Hq, H, D, bs, kind)
    run_attend(kv, c)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("Hq,H,D,bs", [(2, 2, 32, 16), (4, 2, 64, 32), (8, 2, 128, 16),
                                       (3, 1, 64, 128), (10, 2, 128, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 100)])
def test_attend_ragged_rows(kv, kind, Hq, H, D, bs, causal, window):
    lens = [0, 5, 64, 130, 257, 400, 33, 700, 129, 1]
    new = [3, 9, 64, 2, 130, 0, 33, 1, 200, 1]  # more rows than keys in some: rows that see none
    c = history(Hq * D + bs + window, lens, new, Hq, H, D, bs, kind)
    run_attend(kv, c, causal, window)


@pytest.mark.parametrize("kind,H,D,bs", [("bf16", 2, 128, 16), ("fp16", 1, 64, 64),
                                         ("fp32", 1, 32, 128)])
def test_attend_long_history(kv, kind, H, D, bs):
    """Few items over many blocks of threads: the parts are joined."""
    c = history(77, [20011, 3], [1, 1], 4 * H, H, D, bs, kind)
    run_attend(kv, c)
    run_attend(kv, c, window=7000)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_attend_many_requests(kv, kind):
    rng = np.random.default_rng(8)
    n = 1500
    c = history(8, rng.integers(0, 90, n), rng.integers(0, 3, n), 2, 2, 64, 16, kind)
    run_attend(kv, c)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,H,D,bs", [(2, 2, 64, 16), (5, 1, 128, 32), (4, 2, 128, 128)])
def test_attend_tiles_cut_over_blocks(kv, kind, Hq, H, D, bs):
    """Many rows over long histories: items of several row tiles whose steps are shared out over
    blocks of threads, more and fewer steps than blocks; tiles that end inside their halves."""
    c = history(31, [6000, 700, 2], [300, 129, 2], Hq, H, D, bs, kind)
    run_attend(kv, c)
    run_attend(kv, c, window=900)
    c = history(32, [30000], [20], Hq, H, D, bs, kind)
    run_attend(kv, c, causal=False)
    run_attend(kv, c)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_attend_tiles_of_many_requests(kv, kind):
    """More requests than threads of a block, most of them short, some without rows or keys."""
    rng = np.random.default_rng(33)
    n = 1500
    new = rng.integers(0, 4, n)
    new[::97] = rng.integers(20, 150, len(new[::97]))  # more rows than the row kernel takes
    lens = rng.integers(0, 60, n)
    lens[::50] += 300
    c = history(33, lens, new, 4, 2, 64, 16, kind)
    run_attend(kv, c)
    run_attend(kv, c, causal=False)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("n,new,D", [(63, 4, 128), (64, 4, 128), (64, 5, 128), (64, 8, 64), (64, 9, 64),
                                     (300, 3, 64)])
def test_attend_between_the_row_and_the_tile_kernel(kv, kind, n, new, D):
    """8 query heads a kv head: 24 to 72 rows, fewer and more requests."""
    rng = np.random.default_rng(37)
    w = rng.integers(0, new + 1, n)
    w[3] = new
    c = history(37, rng.integers(0, 400, n) + w, w, 8, 1, D, 16, kind)
    run_attend(kv, c)
    run_attend(kv, c, window=100)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,D", [(1, 64), (9, 32), (150, 64), (150, 128)])
def test_attend_negative_and_zero_scales(kv, kind, rows, D):
    c = history(34, [300, 260], [rows] * 2, 2, 1, D, 16, kind)
    c["ks"][::3] *= -1
    c["vs"][1::4] *= -1
    c["ks"][::5] = 0
    c["vs"][2::5] = 0
    run_attend(kv, c)
    run_attend(kv, c, scale=-0.2, causal=False)
    c["vs"][:] = 0
    out, _ = run_attend(kv, c)
    assert (out == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_attend_tiles_scores_far_apart(kv, kind):
    """Scores of thousands: nearly all weight on one key, weights far below the largest, rows
    whose maximum rises step by step (the accumulators are rescaled)."""
    c = history(35, [900], [150], 2, 2, 64, 16, kind)
    run_attend(kv, c, scale=20.0, causal=False)
    ids = c["table"][0, :57]
    c["ks"][ids] = np.float32(0.002) * np.float32(1.12) ** np.arange(57)[:, None]
    c["vs"][ids] = np.float32(0.01) * np.float32(1.3) ** np.arange(57)[:, None]
    run_attend(kv, c, scale=0.5)
    c["vs"][ids] = c["vs"][ids[::-1]]
    run_attend(kv, c, scale=0.5, causal=False)
    # scores past 2^20: finite, and a weighted mean of the values
    q = c["q"].cuda()
    out = torch.empty_like(q)
    kv.mpzch_kv_attend(q, dev(c["kc"]), dev(c["vc"]), dev(c["ks"]), dev(c["vs"]), dev(c["table"]),
                       dev(c["cu"]), dev(c["seq"]), 150, out, softmax_scale=1e9, causal=False)
    got = out.float()
    assert got.isfinite().all() and got.abs().max() <= 128 * float(c["vs"].max())


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("length", [112, 128, 129, 144, 496, 512, 513, 528])
@pytest.mark.parametrize("more", [0, 124, 125])
def test_attend_around_the_longest_whole_history(kv, kind, length, more):
    """Tables that hold up to 128 or 512 keys and more, of up to 256 items and more: items go
    whole to a warp, or are cut."""
    c = history(36, [length, 40, 0, length - 7] + [9] * more, [1, 2, 1, 1] + [1] * more, 4, 2, 64, 16,
                kind)
    for width in (length // 16 + 1, length // 16 + 40):
        t = np.full((4 + more, width), -1, np.int32)
        t[:, :min(width, c["table"].shape[1])] = c["table"][:, :width]
        run_attend(kv, {**c, "table": t})


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_attend_strides_untouched_rows_and_scales(kv, kind):
    """q inside a fused projection, out inside a wider tensor, rows behind the last request, a
    negative softmax scale."""
    c = history(9, [40, 333, 150], [1, 4, 70], 4, 2, 64, 16, kind)
    n = c["q"].shape[0]
    pad = 5
    wide = torch.full((n + pad, 8, 64), 3.0, dtype=TYPES[kind], device="cuda")
    wide[:n, 2:6] = c["q"].cuda()
    c["q"] = torch.cat([c["q"], torch.full((pad, 4, 64), 3.0, dtype=TYPES[kind])])
    out = torch.full((n + pad, 10, 64), 7.0, dtype=TYPES[kind], device="cuda")
    run_attend(kv, c, q=wide[:, 2:6], out=out[:, 3:7], scale=-0.3)
    keep = torch.ones(10, dtype=torch.bool)
    keep[3:7] = False
    assert (out[:, keep] == 7.0).all()
    run_attend(kv, c, q=wide[:, 2:6], out=out[:, 3:7].fill_(7.0), scale=0.0, causal=False)


@pytest.mark.parametrize("rows,Hq", [(1, 2), (3, 1), (1, 1), (25, 1)])
def test_attend_dimensions_of_one_with_any_stride(kv, rows, Hq):
    """One row, one head: torch gives such a dimension whatever stride the view came with."""
    c = history(38, [90], [rows], Hq, 1, 64, 16, "bf16")
    shape, full = (rows, Hq, 64), c["q"].stride()
    stride = (full[0] if rows > 1 else 77, full[1] if Hq > 1 else 33, 1)
    q = torch.as_strided(c["q"].cuda(), shape, stride)
    out = torch.as_strided(torch.full((rows * Hq * 64,), 7.0, dtype=torch.bfloat16, device="cuda"),
                           shape, stride)
    run_attend(kv, c, q=q, out=out)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows", [1, 40])
def test_attend_value_scales_far_apart(kv, kind, rows):
    """Blocks whose value scales span 24 powers of two, in both orders, and blocks of scale 0; the
    keys with the largest weights lie in the small ones."""
    for order in (1, -1):
        c = history(10, [512] * 2, [rows] * 2, 2, 2, 64, 16, kind)
        for b in range(2):
            ids = c["table"][b, :32]
            c["vs"][ids] = np.float32(2.0) ** np.linspace(-12, 12, 32)[::order, None]
            c["vs"][ids[7]] = 0.0
            c["ks"][ids] = 0.004
        run_attend(kv, c, causal=False)


@pytest.mark.parametrize("rows", [1, 40])
def test_attend_hides_bad_blocks(kv, rows):
    c = history(11, [300, 200, 90], [rows] * 3, 4, 2, 64, 16, "bf16")
    c["table"][0, 3], c["table"][1, 0], c["table"][1, 7] = -1, 10**6, -2**31
    c["table"][2, :] = 2**31 - 1  # nothing left to see
    run_attend(kv, c, status=ref.BADBLOCK)


@pytest.mark.parametrize("rows", [1, 40])
def test_attend_cuts_bad_lengths(kv, rows):
    c = history(12, [100, 60, 70, 80], [rows] * 4, 2, 1, 64, 16, "fp16")
    c["seq"][0], c["seq"][1] = -4, 2**31 - 1
    c["table"][1] = c["table"][2]
    c["table"][1, 5:] = c["table"][0, :c["table"].shape[1] - 5]
    bad = (c["table"][1] < 0).any()
    run_attend(kv, c, causal=False, status=ref.BADLEN | (ref.BADBLOCK if bad else 0))
    c = history(13, [100, 60, 70, 80], [rows] * 4, 2, 1, 64, 16, "fp16")
    c["cu"][4] += 100  # past the batch
    run_attend(kv, c, status=ref.BADLEN)
    c["cu"][:] = [5, 0, rows, rows, rows + 2]  # steps back
    run_attend(kv, c, status=ref.BADLEN)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows", [2, 40])
def test_attend_nan_and_infinities_stay_where_they_are_seen(kv, kind, rows):
    """Scales that are NaN or infinite in blocks that a row does not see, and in keys behind the
    last one, do not reach it; a query row with a NaN gives NaN in that row alone."""
    c = history(14, [16 * 6, 16 * 6 + 5, 40], [rows] * 3, 2, 2, 64, 16, kind)
    # the last block of request 0 is seen by its last rows only; a window hides the first one
    for b, col, x in ((0, 5, np.nan), (1, 0, np.inf)):
        c["vs"][c["table"][b, col]] = x
        c["ks"][c["table"][b, col]] = x
    c["q"][rows * 2, 0, 3] = float("nan")
    c["q"][rows * 2 + 1, 1, 0] = float("inf")
    q = c["q"].cuda()
    out = torch.full_like(q, 7.0)
    kv.mpzch_kv_attend(q, dev(c["kc"]), dev(c["vc"]), dev(c["ks"]), dev(c["vs"]), dev(c["table"]),
                       dev(c["cu"]), dev(c["seq"]), rows, out, window=48)
    sees_bad = np.zeros((len(q), 2), bool)
    for t in range(rows):
        sees_bad[t] = 96 - rows + t >= 80
        sees_bad[rows + t] = 101 - rows + t - 48 < 15
    sees_bad[rows * 2, 0] = sees_bad[rows * 2 + 1, 1] = True
    # rows of request 2 before its first key see nothing: no NaN there
    if rows > 40:
        sees_bad[rows * 2:rows * 2 + 2] = False
    got = np.isnan(out.float().cpu().numpy())
    assert np.array_equal(got.all(2), sees_bad) and np.array_equal(got.any(2), sees_bad)
    clean = {**c, "ks": np.nan_to_num(c["ks"], nan=1.0, posinf=1.0),
             "vs": np.nan_to_num(c["vs"], nan=1.0, posinf=1.0),
             "q": torch.nan_to_num(c["q"], nan=1.0, posinf=1.0)}
    want, _, size = ref.attend(clean["q"].double().numpy(), c["kc"], c["vc"], clean["ks"],
                                        clean["vs"], c["table"], c["cu"], c["seq"], 0.125, True, 48)
    fine = ~sees_bad
    off = np.abs(out.double().cpu().numpy() - want)[fine]
    assert (off <= ref.attend_bound(want, size, 101, 64, kind)[fine]).all()


def test_attend_large_and_tiny_queries(kv):
    """Rows of very different size: the row's scaling keeps each exact; a row whose scores are far
    apart picks one key."""
    for kind, sizes in (("fp32", [1e30, 1e-30, 3e3, 1e-3, 0.0]), ("fp16", [6e4, 1e-7, 300, 1, 0.0]),
                        ("bf16", [1e30, 1e-38, 3e3, 1, 0.0])):
        c = history(15, [700], [5], 1, 1, 64, 16, kind)
        x = c["q"].float() / c["q"].float().abs().max() * torch.tensor(sizes)[:, None, None]
        c["q"] = x.to(TYPES[kind])
        for scale in (0.125, 1e-6):
            want, _, size = ref.attend(
                c["q"].double().numpy(), c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["cu"],
                c["seq"], scale, False, 0)
            out = torch.empty_like(c["q"].cuda())
            kv.mpzch_kv_attend(c["q"].cuda(), dev(c["kc"]), dev(c["vc"]), dev(c["ks"]),
                               dev(c["vs"]), dev(c["table"]), dev(c["cu"]), dev(c["seq"]), 5, out,
                               softmax_scale=scale, causal=False)
            got = out.double().cpu().numpy()
            assert np.isfinite(got).all()
            # where the scores' own rounding decides (reach beyond 1e4), only the range is held
            calm = (size[1] < 1e4)[..., None] & np.ones_like(got, bool)
            bound = ref.attend_bound(want, size, 700, 64, kind)
            assert (np.abs(got - want) <= bound)[calm].all()
            assert (np.abs(got) <= 130 * c["vs"].max()).all()


def test_attend_offsets_past_31_bits(kv):
    """Blocks whose codes lie beyond 2^31 and 2^32 bytes of the cache."""
    H, D, bs = 8, 128, 128
    blocks = (2**32 // (H * D * bs)) + 40
    kc = torch.zeros((blocks, H, bs, D), dtype=torch.int8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = (torch.zeros((blocks, H), device="cuda") for _ in range(2))
    ids = [blocks - 1, 5, blocks // 2 + 3, blocks - 30]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    n = 3 * bs + 50
    rng = np.random.default_rng(16)
    k, v = (torch.from_numpy(rng.standard_normal((n, H, D)).astype(np.float32)).cuda()
            for _ in range(2))
    slots = np.concatenate([np.int64(i) * bs + np.arange(bs) for i in ids])[:n]
    kv.mpzch_kv_append(k, v, dev(slots), kc, vc, ks, vs)
    small = dict(kind="bf16", table=np.arange(4, dtype=np.int32)[None],
                 seq=np.array([n], np.int32))
    for name, t in (("kc", kc), ("vc", vc), ("ks", ks), ("vs", vs)):
        small[name] = host(t[torch.tensor(ids).cuda()])
    want_k = np.zeros((4, H, bs, D), np.int8)
    ref.append(host(k), np.arange(n, dtype=np.int64), want_k, np.zeros((4, H), np.float32))
    assert np.array_equal(small["kc"], want_k)
    for rows in (1, 50):
        small["q"] = torch.from_numpy(rng.standard_normal((rows, H, D)).astype(np.float32)).bfloat16()
        small["cu"] = np.array([0, rows], np.int32)
        q = small["q"].cuda()
        out = torch.empty_like(q)
        kv.mpzch_kv_attend(q, kc, vc, ks, vs, table, dev(small["cu"]), dev(small["seq"]), rows, out)
        check_attend(small, out, None, D ** -0.5, True, 0)


def test_attend_results_repeat(kv):
    c = history(17, [3000, 5, 800, 64], [1, 1, 60, 8], 8, 2, 128, 16, "bf16")
    first = run_attend(kv, c)
    for _ in range(3):
        again = run_attend(kv, c)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ------------------------------------------------------------------ together
def step_reference(model, kc, vc, ks, vs, table, cached, new, free, count, x, bs):
    """One step of the pipeline below, on the host: float32 projections are given."""
    q, k, v = x
    table, cu, seq, slots, left, bits = ref.tables(cached, new, bs, free, count, table, len(k))
    bits |= ref.append(k, slots, kc, ks) | ref.append(v, slots, vc, vs)
    return table, cu, seq, slots, left, bits


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_items_to_history_to_attention(kv, kind):
    """Item rows from the int8 serving snapshot -> projections -> block tables -> append ->
    attention, over an admission and several single-token steps."""
    rng = np.random.default_rng(20)
    bs, H, G, D, B, dim = 16, 2, 4, 64, 9, 128
    # a snapshot with 3000 of 4096 rows live
    tbl = kv.MpzchTable(4096, dim, 8)
    keys = rng.choice(10**9, 3000, replace=False).astype(np.int64)
    tbl.writeback(dev(keys), dev(rng.standard_normal((3000, dim)).astype(np.float32)), 0)
    all_rows = torch.arange(4096, dtype=torch.int32, device="cuda")
    snap_q, snap_s, snap_k = tbl.export_int8(all_rows)
    h = kv.MpzchHistory(200, bs, H, D, B, 20)
    w = [torch.randn(dim, heads * D, generator=torch.Generator().manual_seed(i)).cuda() / dim**0.5
         for i, heads in enumerate((H * G, H, H))]
    state = dict(kc=np.zeros((200, H, bs, D), np.int8), vc=np.zeros((200, H, bs, D), np.int8),
                 ks=np.zeros((200, H), np.float32), vs=np.zeros((200, H), np.float32),
                 table=np.full((B, 20), -1, np.int32), seq=np.zeros(B, np.int32), count=200)
    free = np.arange(200, dtype=np.int32)
    for step, new in enumerate([rng.integers(0, 70, B)] + [np.ones(B, np.int64)] * 3 +
                               [rng.integers(0, 6, B)]):
        new = new.astype(np.int32)
        n = int(new.sum())
        ids = dev(rng.choice(np.concatenate([keys, [10**10]]), n))
        rows = torch.empty(n, dtype=torch.int32, device="cuda")
        hit = torch.empty(n, dtype=torch.uint8, device="cuda")
        items = torch.empty((n, dim), device="cuda")
        kv.mpzch_serve_gather(snap_k, 8, snap_q, snap_s, ids, rows, hit, items)
        q, k, v = (torch.mm(items, m).to(TYPES[kind]) for m in w)
        q, k, v = q.view(n, H * G, D), k.view(n, H, D), v.view(n, H, D)
        cu, slots = h.extend(dev(new), n)
        h.append(k, v, slots)
        out = h.attend(q, cu, int(new.max()))
        assert int(h.status) == 0
        state["table"], want_cu, state["seq"], want_slots, state["count"], _ = ref.tables(
            state["seq"], new, bs, free, state["count"], state["table"], n)
        ref.append(host(k.float()), want_slots, state["kc"], state["ks"])
        ref.append(host(v.float()), want_slots, state["vc"], state["vs"])
        assert np.array_equal(host(slots), want_slots) and np.array_equal(host(cu), want_cu)
        assert np.array_equal(host(h.block_table), state["table"])
        assert int(h.free_count) == state["count"]
        for name, t in (("kc", h.k_cache), ("vc", h.v_cache), ("ks", h.k_scale), ("vs", h.v_scale)):
            assert np.array_equal(host(t), state[name]), (step, name)
        check_attend({**state, "q": q.cpu(), "cu": want_cu, "kind": kind}, out, None, D ** -0.5,
                     True, 0)
    tbl.close()


def test_step_captured_and_replayed_on_its_own_stream(kv):
    """tables -> append -> attend captured twice (two graphs, each with its workspace), replayed
    with other lengths and values than those of the capture."""
    rng = np.random.default_rng(21)
    bs, H, G, D, B = 16, 2, 2, 64, 6
    h = kv.MpzchHistory(300, bs, H, D, B, 40)
    n = 64  # padded batch
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros((n, x, D), dtype=torch.bfloat16, device="cuda") for x in (H * G, H, H))
    seq, count = h.seq_len.clone(), h.free_count.clone()
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    seq2, left = torch.zeros_like(seq), torch.zeros_like(count)
    slots = torch.zeros(n, dtype=torch.int64, device="cuda")
    outs = [torch.full_like(q, 7.0) for _ in range(2)]

    def step(out):
        kv.mpzch_kv_tables(seq, new, bs, h.free_blocks, count, h.block_table, cu, seq2, slots, left,
                           h.status)
        kv.mpzch_kv_append(k, v, slots, *h.cache(), h.status)
        kv.mpzch_kv_attend(q, *h.cache(), h.block_table, cu, seq2, n, out, status=h.status)

    graphs = []
    for out in outs:
        step(out)  # loads the kernels
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(out)
        graphs.append(g)
    assert int(h.status) == 0
    state = dict(kc=np.zeros((300, H, bs, D), np.int8), vc=np.zeros((300, H, bs, D), np.int8),
                 ks=np.zeros((300, H), np.float32), vs=np.zeros((300, H), np.float32),
                 table=host(h.block_table), seq=np.zeros(B, np.int32), count=300)
    side = torch.cuda.Stream()
    for i in range(5):
        w = (rng.integers(0, 11, B) if i % 2 == 0 else np.ones(B)).astype(np.int32)
        new.copy_(dev(w))
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(i)).bfloat16())
        out = outs[i % 2].fill_(7.0)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graphs[i % 2].replay()
        torch.cuda.current_stream().wait_stream(side)
        state["table"], want_cu, state["seq"], want_slots, state["count"], _ = ref.tables(
            state["seq"], w, bs, np.arange(300, dtype=np.int32), state["count"], state["table"], n)
        ref.append(host(k.float()), want_slots, state["kc"], state["ks"])
        ref.append(host(v.float()), want_slots, state["vc"], state["vs"])
        assert np.array_equal(host(slots), want_slots)
        assert np.array_equal(host(h.k_cache), state["kc"])
        assert np.array_equal(host(h.v_scale), state["vs"])
        check_attend({**state, "q": q.cpu(), "cu": want_cu, "kind": "bf16"}, out, None, D ** -0.5,
                     True, 0)
        seq.copy_(seq2)
        count.copy_(left)
    assert int(h.status) == 0


CAPTURE_FIRST = """
import sys
sys.path[:0] = [%r, %r]
import numpy as np, torch
import kv_ref as ref, test_gpu_kv as t
from hashed_sparse_table_b200 import binding as kv
for rows, kind in ((1, "bf16"), (30, "fp16")):
    c = t.history(40, [700, 90], [rows] * 2, 4, 2, 64, 16, kind)
    a = [c["q"].cuda()] + [t.dev(c[x]) for x in ("kc", "vc", "ks", "vs", "table", "cu", "seq")]
    out = torch.full_like(a[0], 7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.mpzch_kv_attend(*a, rows, out)
    assert (out == 7.0).all()
    g.replay()
    torch.cuda.synchronize()
    t.check_attend(c, out, None, 0.125, True, 0)
print("captured")
"""


def test_first_calls_of_a_process_can_be_captured():
    """No call before the capture has loaded the kernels."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    done = subprocess.run([sys.executable, "-c", CAPTURE_FIRST % (os.path.dirname(here), here)],
                          capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "captured" in done.stdout, done.stderr[-2000:]


def test_calls_on_two_streams_at_once(kv):
    """Two attention calls in flight together, each with a workspace, one on a raw stream."""
    a = history(22, [5000, 10], [1, 1], 8, 2, 64, 16, "bf16")
    b = history(23, [4000, 700], [1, 30], 4, 4, 128, 32, "fp16")
    side = torch.cuda.Stream()
    jobs = []
    for c in (a, b):
        jobs.append([c["q"].cuda()] + [dev(c[x]) for x in ("kc", "vc", "ks", "vs", "table", "cu",
                                                            "seq")])
    outs = [torch.empty_like(j[0]) for j in jobs]
    spaces = [torch.empty(kv.mpzch_kv_attend_workspace(j[0].shape[1], j[1].shape[1], j[0].shape[2]),
                          dtype=torch.uint8, device="cuda") for j in jobs]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, j in enumerate(jobs):
            kv.mpzch_kv_attend(*j, 30, outs[i], workspace=spaces[i], stream=side if i else None)
    torch.cuda.synchronize()
    for c, out in zip((a, b), outs):
        check_attend(c, out, None, c["q"].shape[2] ** -0.5, True, 0)


def test_refusals_on_the_device(kv):
    c = history(24, [40], [1], 4, 2, 64, 16, "bf16")
    q = c["q"].cuda()
    cache = [dev(c[x]) for x in ("kc", "vc", "ks", "vs")]
    rest = [dev(c[x]) for x in ("table", "cu", "seq")]
    out = torch.empty_like(q)
    for change in (dict(out=out.half()), dict(out=out[:, :2]), dict(window=5, causal=False),
                   dict(window=-1), dict(softmax_scale=float("nan")), dict(lse=out[..., 0]),
                   dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
                   dict(stream=torch.cuda.Stream()), dict(status=torch.zeros(1, device="cuda")),
                   dict(q=q.transpose(1, 2)), dict(q=q.double()), dict(q=q[:, :3], out=out[:, :3]),
                   dict(q=q.cpu()), dict(max_new=-1)):
        args = {"q": q, "max_new": 1, "out": out, **change}
        with pytest.raises((ValueError, kv.MpzchError)):
            kv.mpzch_kv_attend(args.pop("q"), *cache, *rest, args.pop("max_new"), args.pop("out"),
                               **args)
    odd = torch.zeros(2 * 64 * 4 + 1, dtype=torch.bfloat16, device="cuda")[1:257].view(1, 4, 64)
    with pytest.raises(kv.MpzchError):  # not on a 16-byte boundary
        kv.mpzch_kv_attend(odd, *cache, *rest, 1, out)
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    for bad in ((k, k.half(), slots), (k, k, slots.int()), (k[:, :1], k, slots),
                (k.expand(2, 2, 64), k, slots), (odd[:, :2], k, slots)):
        with pytest.raises((ValueError, kv.MpzchError)):
            kv.mpzch_kv_append(*bad, *cache)
