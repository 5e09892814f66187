"""History cache without a GPU: the C entries refuse bad arguments before any CUDA call, the
binding refuses tensors that are not on the current device, and the restatement used by the GPU
tests agrees with brute force on small cases."""
import ctypes as C

import numpy as np
import pytest

import kv_ref as ref

EINVAL = -1


@pytest.fixture(scope="module")
def lib():
    from hashed_sparse_table_b200 import build
    build.build()
    from hashed_sparse_table_b200 import binding
    return binding.lib()


FAKE = 0x1000


def tables(lib, **change):
    a = dict(cached=FAKE, new=FAKE + 256, n=4, bs=16, free=FAKE, n_free=9, count=FAKE, table=FAKE,
             max_blocks=3, cu=FAKE + 512, seq=FAKE + 1024, slots=FAKE, n_slots=5, left=FAKE + 64,
             status=None, stream=None)
    a.update(change)
    return lib.mpzch_kv_tables(*a.values())


@pytest.mark.parametrize("change", [
    dict(n=-1), dict(n=16385), dict(bs=0), dict(bs=15), dict(bs=256), dict(n_free=-1),
    dict(n_free=2**31 - 1), dict(max_blocks=-1), dict(n_slots=-1), dict(n_slots=2**31 - 1),
    dict(count=None), dict(left=None), dict(left=FAKE), dict(cu=None), dict(free=None),
    dict(slots=None), dict(cached=None), dict(new=None), dict(seq=None), dict(table=None),
    dict(seq=FAKE), dict(seq=FAKE + 256), dict(cu=FAKE), dict(cu=FAKE + 256)])
def test_tables_refusals(lib, change):
    assert tables(lib, **change) == EINVAL


def append(lib, **change):
    a = dict(k=FAKE, ksn=128, ksh=64, v=FAKE, vsn=128, vsh=64, n=3, dtype=2, slots=FAKE, kc=FAKE,
             vc=FAKE + 4096, ks=FAKE, vs=FAKE + 4096, blocks=9, bs=16, H=2, D=64, status=None,
             stream=None)
    a.update(change)
    return lib.mpzch_kv_append(*a.values())


@pytest.mark.parametrize("change", [
    dict(n=-1), dict(n=2**31), dict(dtype=3), dict(dtype=-1), dict(bs=8), dict(D=48), dict(D=256),
    dict(H=0), dict(H=5000), dict(blocks=-1), dict(blocks=2**31), dict(k=None), dict(v=None),
    dict(slots=None), dict(kc=None), dict(vc=None), dict(ks=None), dict(vs=None), dict(vc=FAKE),
    dict(vs=FAKE), dict(k=FAKE + 2), dict(ksn=129), dict(vsh=63), dict(ksn=-128), dict(kc=FAKE + 8),
    dict(dtype=0, ksn=130, ksh=64)])
def test_append_refusals(lib, change):
    assert append(lib, **change) == EINVAL


def attend(lib, **change):
    a = dict(q=FAKE, qsn=256, qsh=64, n=3, dtype=2, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, blocks=9,
             bs=16, Hq=4, H=2, D=64, table=FAKE, max_blocks=5, cu=FAKE, seq=FAKE, B=2, max_new=2,
             scale=0.125, causal=1, window=0, out=FAKE, osn=256, osh=64, lse=None, ws=FAKE,
             ws_bytes=1 << 40, status=None, stream=None)
    a.update(change)
    return lib.mpzch_kv_attend(*a.values())


@pytest.mark.parametrize("change", [
    dict(n=-1), dict(n=2**31), dict(dtype=5), dict(bs=17), dict(Hq=5), dict(Hq=0), dict(H=0),
    dict(Hq=8192), dict(D=16), dict(blocks=-1), dict(max_blocks=-1), dict(max_blocks=2**27),
    dict(B=-1), dict(B=16385), dict(max_new=-1), dict(scale=float("inf")),
    dict(scale=float("nan")), dict(scale=3e38), dict(n=2**31 // 4), dict(window=-1), dict(window=4, causal=0), dict(q=None),
    dict(out=None), dict(cu=None), dict(seq=None), dict(table=None), dict(kc=None), dict(vc=None),
    dict(ks=None), dict(vs=None), dict(ws=None), dict(ws_bytes=100), dict(ws=FAKE + 16),
    dict(q=FAKE + 4), dict(out=FAKE + 8), dict(osn=0), dict(osh=0), dict(osh=32), dict(osn=56), dict(qsn=250), dict(osh=-64), dict(kc=FAKE + 1)])
def test_attend_refusals(lib, change):
    assert attend(lib, **change) == EINVAL


def test_empty_calls_touch_nothing(lib):
    assert append(lib, n=0, k=None, v=None, slots=None) == 0
    assert attend(lib, n=0, q=None, out=None) == 0
    assert attend(lib, B=0, cu=None, seq=None) == 0


def test_workspace_sizes(lib):
    f = lib.mpzch_kv_attend_workspace
    for bad in ((0, 1, 64), (4, 0, 64), (5, 2, 64), (4, 2, 60), (8192, 1, 64)):
        assert f(*bad) == -1
    assert 0 < f(8, 8, 32) < f(8, 8, 64) < f(8, 8, 128) < 1 << 28


def test_binding_refuses_tensors_elsewhere(lib, monkeypatch):
    import torch
    from hashed_sparse_table_b200 import binding
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    i32 = torch.zeros(4, dtype=torch.int32)
    i64 = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="cached_len"):
        binding.mpzch_kv_tables(i32, i32, 16, i32, i64, i32, i32, i32, i64, i64)
    c = torch.zeros((3, 2, 16, 64), dtype=torch.int8)
    s = torch.zeros((3, 2))
    with pytest.raises(ValueError, match="k_cache"):
        binding.mpzch_kv_append(s, s, i64, c, c, s, s)
    with pytest.raises(ValueError, match="k_cache"):
        binding.mpzch_kv_attend(s, c, c, s, s, i32, i32, i32, 1, s)


# ------------------------------------------------------------------ the restatement itself
def test_reference_tables_by_simulation():
    """Token by token: a request opens a block whenever it fills one."""
    rng = np.random.default_rng(0)
    for _ in range(30):
        B, bs = int(rng.integers(1, 8)), 16
        cached, new = rng.integers(0, 50, B), rng.integers(0, 40, B)
        ids = rng.permutation(200)
        table, at = np.full((B, 8), -1, np.int32), 0
        for b in range(B):
            for j in range(-(-int(cached[b]) // bs)):
                table[b, j], at = ids[at], at + 1
        free = list(ids[at:])
        got = ref.tables(cached, new, bs, np.array(free), len(free), table, int(new.sum()))
        slots = []
        for b in range(B):
            for t in range(int(cached[b]), int(cached[b] + new[b])):
                if t % bs == 0:
                    table[b, t // bs] = free.pop()
                slots.append(table[b, t // bs] * bs + t % bs)
        assert np.array_equal(got[0], table) and got[3].tolist() == slots
        assert got[4] == len(free) and got[5] == 0
        assert np.array_equal(got[2], cached + new)


def test_reference_append_stays_within_half_a_step():
    """After any sequence of appends a token is within half a step of its value for its own
    rounding and half a step more for each later growth of the scale."""
    rng = np.random.default_rng(1)
    cache, scale = np.zeros((1, 1, 16, 32), np.int8), np.zeros((1, 1), np.float32)
    x = rng.standard_normal((16, 1, 32)).astype(np.float32) * np.exp(rng.standard_normal((16, 1, 1)))
    x = x.astype(np.float32)
    steps, room = [], np.zeros(16)
    at = 0
    for w in (1, 2, 1, 5, 7):
        old = scale[0, 0]
        assert ref.append(x[at:at + w], np.arange(at, at + w), cache, scale) == 0
        s = float(scale[0, 0])
        if s != old:
            room[:at] += s / 2
        room[at:at + w] = s / 2
        at += w
        assert abs(s - np.abs(x[:at]).max() / 127) <= s * 2.0**-23
    off = np.abs(cache[0, 0].astype(np.float64) * float(scale[0, 0]) - x[:, 0])
    assert (off <= room[:, None] * (1 + 1e-5)).all()


def test_reference_attention_by_hand():
    """Two keys, one of them hidden from the first row; the value is exact by hand."""
    kc, vc = np.zeros((1, 1, 16, 32), np.int8), np.zeros((1, 1, 16, 32), np.int8)
    kc[0, 0, 1, 0], vc[0, 0, 0, 0], vc[0, 0, 1, 0] = 2, 10, 30
    one = np.ones((1, 1), np.float32)
    q = np.zeros((2, 1, 32))
    q[:, 0, 0] = 1.0
    out, lse, _ = ref.attend(q, kc, vc, one, one, np.zeros((1, 1), np.int32), [0, 2], [2], 0.5,
                                True, 0)
    assert out[0, 0, 0] == 10 and lse[0, 0] == 0
    e = np.e
    assert abs(out[1, 0, 0] - (10 + 30 * e) / (1 + e)) < 1e-12 and abs(lse[1, 0] - np.log(1 + e)) < 1e-12
    out, lse, _ = ref.attend(q, kc, vc, one, one, np.zeros((1, 1), np.int32), [0, 2], [2], 0.5,
                                True, 1)
    assert out[1, 0, 0] == 30
    out, lse, _ = ref.attend(q, kc, vc, one, one, np.zeros((1, 1), np.int32), [0, 2], [1], 0.5,
                                True, 0)
    assert (out[0] == 0).all() and np.isneginf(lse[0, 0])


def test_bound_catches_a_shifted_mask():
    """A mask that is one key off passes the bound by far somewhere."""
    rng = np.random.default_rng(2)
    kc, vc = (rng.integers(-127, 128, (4, 1, 16, 64)).astype(np.int8) for _ in range(2))
    s = np.full((4, 1), 0.02, np.float32)
    q = rng.standard_normal((3, 1, 64))
    table = np.arange(4, dtype=np.int32)[None]
    args = (kc, vc, s, s, table, [0, 3])
    out, _, size = ref.attend(q, *args, [60], 0.125, True, 0)
    other = ref.attend(q, *args, [59], 0.125, True, 0)[0]
    for kind in ("bf16", "fp16", "fp32"):
        bound = ref.attend_bound(out, size, 60, 64, kind)
        assert (np.abs(out - other) / bound).max() > 3
