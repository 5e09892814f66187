"""Attention on the GPU into outputs of unusual strides."""
import numpy as np
import pytest
import torch

from test_gpu_kv import history, kv, run_attend  # noqa: F401 (kv: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("Hq,stride", [
    (2, (64, 200 * 64)),     # heads in front of rows
    (2, (128, 64)),          # the ordinary order
    (2, (3 * 64, 40 * 64)),  # neither stride passes all of the other, and no head meets another
    (3, (3 * 64, 2 * 64 * 20 + 64))])
def test_outputs_whose_heads_lie_apart_are_taken(kv, rows, Hq, stride):
    c = history(70, [90, 300], [rows] * 2, Hq, 1, 64, 16, "bf16")
    n = 2 * rows
    at = sorted(i * stride[0] + j * stride[1] for i in range(n) for j in range(Hq))
    assert min(b - a for a, b in zip(at, at[1:])) >= 64
    flat = torch.full((at[-1] + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = torch.as_strided(flat, (n, Hq, 64), (*stride, 1))
    run_attend(kv, c, out=out)
    rest = np.ones(len(flat), bool)
    for x in at:
        rest[x:x + 64] = False
    assert (flat.float().cpu().numpy()[rest] == 7.0).all()
