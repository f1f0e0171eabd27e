"""Seeds and offsets of the dropout calls: whole numbers of 64 bits, or a
refusal (CPU: the arguments are checked before the device is)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from newton_schulz_05_amd import MuonError
from newton_schulz_05_amd import operators as O


@pytest.mark.parametrize("v", [0, 7, (1 << 64) - 1, True, 3.0, np.int64(5), np.uint64((1 << 64) - 1), torch.tensor(9)])
def test_whole_numbers(v):
    assert O._u64(v, "seed") == int(v)


@pytest.mark.parametrize("v", [-1, 1 << 64, 1.5, 2.0 ** 64, float("nan"), float("inf"), "7", None, torch.tensor(0.5)])
def test_refused(v):
    with pytest.raises(MuonError) as e:
        O._u64(v, "seed")
    assert e.value.status == 1 and "seed" in str(e.value)
