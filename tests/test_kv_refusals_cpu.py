"""Calls of the history cache that are refused before anything is launched: what the C entries and
the binding check without a GPU."""
import itertools

import numpy as np
import pytest

from test_kv_cpu import EINVAL, attend, lib, tables  # noqa: F401 (lib: fixture)


def overlapping(n, sn, h, sh, dim):
    seen = np.zeros((n - 1) * sn + (h - 1) * sh + dim, int)
    for i, j in itertools.product(range(n), range(h)):
        seen[i * sn + j * sh:i * sn + j * sh + dim] += 1
    return seen.max() > 1


@pytest.mark.parametrize("n,H", [(2, 2), (3, 4), (4, 4), (5, 2), (7, 6), (9, 3)])
def test_outputs_whose_heads_overlap_are_refused(lib, n, H):
    """Every pair of strides that puts a head on another one, found by counting; 32 elements a
    head, 8 to a 16-byte boundary."""
    pairs = [x for x in itertools.product(range(0, 32 * 12 + 1, 8), repeat=2)
             if overlapping(n, x[0], H, x[1], 32)]
    for sn, sh in pairs:
        assert attend(lib, n=n, Hq=H, H=1, D=32, osn=sn, osh=sh) == EINVAL, (sn, sh)
    # not a matter of each stride alone
    assert (32, 32) in pairs and (40, 40) in pairs


def test_history_attend_on_a_stream_of_its_own_needs_an_output():
    """An output from torch's allocator belongs to the current stream."""
    import torch
    from hashed_sparse_table_b200 import binding
    h = object.__new__(binding.MpzchHistory)
    q = torch.zeros((1, 2, 64))
    with pytest.raises(ValueError, match="output"):
        h.attend(q, None, 1, stream=object(), workspace=q)


def test_whole_numbers_past_32_bits_are_refused(monkeypatch):
    """ctypes drops the upper bits, so a window of 2^32 + 5 was one of 5.  (CPU tensors on a
    current device of -1; what is refused never reaches the library.)"""
    import torch
    from hashed_sparse_table_b200 import binding
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: calls.append(args) or 0
    monkeypatch.setattr(binding, "_lib", Lib())
    i32, i64 = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    cu, table = torch.zeros(3, dtype=torch.int32), torch.zeros((2, 4), dtype=torch.int32)
    cache, scale = torch.zeros((3, 2, 16, 64), dtype=torch.int8), torch.zeros((3, 2))
    q, ws = torch.zeros((2, 2, 64)), torch.zeros(256, dtype=torch.uint8)

    def attend(max_new=1, window=0):
        binding.mpzch_kv_attend(q, cache, cache, scale, scale, table, cu, i32, max_new, q.clone(),
                                window=window, workspace=ws, stream=0)

    def tables(block_size):
        binding.mpzch_kv_tables(i32, i32, block_size, i32, i64, table, cu, i32, i64, i64, stream=0)

    attend(window=2**31 - 1)
    tables(16)
    assert len(calls) == 2
    for call in (lambda x: attend(window=x), lambda x: attend(max_new=x), tables):
        for x in (2**31, 2**32 + 16, -2**32 + 16, 2**70):
            with pytest.raises(ValueError, match="32 bits"):
                call(x)
    assert len(calls) == 2


@pytest.mark.parametrize("bs,most", [(16, 2**27 - 64), (32, 2**26 - 32), (128, 2**24 - 8)])
def test_tables_whose_lengths_would_pass_31_bits_are_refused(lib, bs, most):
    """The same limit as attention's: max_blocks * block_size below 2^31 - 1024 (lengths are
    int32: with more blocks c + w could come back negative)."""
    assert most * bs == 2**31 - 1024
    for blocks in (most, most + 1, 2**27, 2**31 - 1):
        assert tables(lib, bs=bs, max_blocks=blocks) == EINVAL, blocks
        assert attend(lib, bs=bs, max_blocks=blocks) == EINVAL, blocks


def test_overlap_of_outputs_with_huge_strides_is_seen(lib):
    """Rows times stride pass 63 bits."""
    far = 2**39
    for n in (2, 2**25, 2**29):
        assert attend(lib, n=n, Hq=2, H=1, osn=far, osh=far) == EINVAL
