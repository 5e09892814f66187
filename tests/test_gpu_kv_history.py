"""MpzchHistory on the GPU: its lengths and its count of free blocks stand still in memory, so that
a captured step goes on from where the last replay, or an eager step between two, has left it."""
import numpy as np
import pytest
import torch

import kv_ref as ref
from test_gpu_kv import check_attend, dev, host, kv  # noqa: F401 (kv: fixture)

pytestmark = pytest.mark.gpu


def test_captured_history_step_goes_on_at_every_replay(kv):
    rng = np.random.default_rng(60)
    bs, H, G, D, B, blocks, n = 16, 2, 2, 64, 5, 120, 48
    h = kv.MpzchHistory(blocks, bs, H, D, B, 20)
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros((n, x, D), dtype=torch.bfloat16, device="cuda") for x in (H * G, H, H))
    out = torch.full_like(q, 7.0)
    lengths, left = h.seq_len, h.free_count

    def step():
        cu, slots = h.extend(new, n)
        h.append(k, v, slots)
        h.attend(q, cu, n, out=out)
        return cu, slots

    step()  # nothing new: loads the kernels
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cu, slots = step()
    state = dict(kc=np.zeros((blocks, H, bs, D), np.int8), ks=np.zeros((blocks, H), np.float32),
                 table=np.full((B, 20), -1, np.int32), seq=np.zeros(B, np.int32), count=blocks)
    state["vc"], state["vs"] = state["kc"].copy(), state["ks"].copy()
    for i in range(6):
        w = rng.integers(0, 9, B).astype(np.int32)
        new.copy_(dev(w))
        for t in (q, k, v):
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)).bfloat16())
        out.fill_(7.0)
        if i == 3:
            got_cu, got_slots = step()  # an eager one between two replays
        else:
            g.replay()
            got_cu, got_slots = cu, slots
        state["table"], want_cu, state["seq"], want_slots, state["count"], _ = ref.tables(
            state["seq"], w, bs, np.arange(blocks, dtype=np.int32), state["count"], state["table"], n)
        ref.append(host(k.float()), want_slots, state["kc"], state["ks"])
        ref.append(host(v.float()), want_slots, state["vc"], state["vs"])
        assert np.array_equal(host(h.seq_len), state["seq"]), i
        assert int(h.free_count) == state["count"]
        assert np.array_equal(host(got_slots), want_slots) and np.array_equal(host(got_cu), want_cu)
        assert np.array_equal(host(h.block_table), state["table"])
        assert np.array_equal(host(h.k_cache), state["kc"])
        check_attend({**state, "q": q.cpu(), "cu": want_cu, "kind": "bf16"}, out, None, D ** -0.5,
                     True, 0)
    assert h.seq_len is lengths and h.free_count is left
    assert int(h.status) == 0
