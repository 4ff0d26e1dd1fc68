"""The types that key limits may have (CPU only: what the binding hands on)."""
import pytest
import torch

import deterministic_attn_backward_gb300 as dab

CPU = torch.device("cpu")


@pytest.mark.parametrize("S", [4, 300, 40_000])
@pytest.mark.parametrize("dtype", [torch.int8, torch.uint8, torch.int16, torch.int32, torch.int64])
def test_limits_of_every_whole_type_keep_their_values(dtype, S):
    """Also where the number of rows does not fit the type."""
    limit = torch.zeros(S, dtype=dtype)
    limit[:4] = torch.tensor([100, 3, 0, 2], dtype=dtype)
    got = dab._limit(limit, "causal", S, CPU)
    assert got.dtype is torch.int32 and got.shape == (S,)
    # a limit above S counts as S
    assert [min(x, S) for x in got[:4].tolist()] == [min(100, S), 3, 0, 2] and torch.count_nonzero(got[4:]) == 0


def test_negative_and_huge_limits():
    assert dab._limit(torch.tensor([-5, 2], dtype=torch.int8), "causal", 2, CPU).tolist() == [-5, 2]
    assert dab._limit(torch.tensor([-2 ** 40, 2 ** 40]), "causal", 2, CPU).tolist() == [0, 2]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bool, torch.complex64, torch.uint16, torch.uint32, torch.uint64])
def test_other_types_are_refused(dtype):
    with pytest.raises(TypeError):
        dab._limit(torch.zeros(4, dtype=dtype), "causal", 4, CPU)
