"""An activation that is no name, or no hashable value at all, is a ValueError that says so."""
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from group_wise_affine_qlinear_b200 import build as qb


@pytest.fixture(scope="module", autouse=True)
def _built():
    qb.build()


@pytest.mark.parametrize("activation", ["relu", "", 1, False, ["silu"], {"silu": 1}, torch.nn.functional.silu, torch.zeros(3)])
def test_unknown_activations(activation):
    x, c = torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros((8, 8), dtype=torch.int32)
    s = torch.zeros((8, 1), dtype=torch.float16)
    with pytest.raises(ValueError, match="activation must be one of"):
        ql.forward_epilogue(x, c, s, s, activation=activation)
