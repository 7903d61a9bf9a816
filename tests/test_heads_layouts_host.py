"""Which layouts of queries and keys in one buffer the C entry takes: what it answers, against every element's place."""
import ctypes

import numpy as np
import pytest
import torch

import group_wise_affine_qlinear_b200 as ql
from group_wise_affine_qlinear_b200 import build as qb

INVALID, CUDA = 1, 5
BASE, D, SIZE = 1 << 40, 16, 2


class Heads(ctypes.Structure):
    """ql_heads of include/qlinear.h."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("in_token", ctypes.c_int64),
                ("in_head", ctypes.c_int64), ("out_token", ctypes.c_int64), ("out_head", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("heads", ctypes.c_int32)]


@pytest.fixture(scope="module")
def L():
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up: without a GPU a call that passes its checks ends at the device")
    qb.build()
    return ql.lib()


def _in_place(L, M, q, k):
    """Queries and keys (offset, token stride, head stride, heads), in place."""
    sets = [Heads(BASE + SIZE * at, BASE + SIZE * at, t, h, t, h, None, n) for at, t, h, n in (q, k)]
    return L.qlinear_qk_norm_rotary(ctypes.byref(sets[0]), ctypes.byref(sets[1]), 1, 1, 1e-6, None, 0, 0, None, None, 0, 0,
                                    None, M, D, None)


def _places(M, s):
    at, t, h, n = s
    return (at + t * np.arange(M)[:, None, None] + h * np.arange(n)[None, :, None] + np.arange(D)).ravel()


@pytest.mark.parametrize("M,q,k", [
    (5, (0, 96, 16, 4), (64, 96, 16, 2)),                  # rows [q | k]
    (5, (0, 96, 32, 3), (16, 96, 32, 3)),                  # [M][H][q, k]
    (5, (0, 144, 48, 3), (16, 144, 48, 3)),                # [M][H][q, k, v]
    (5, (0, 128, 64, 2), (48, 128, 64, 2)),
    (5, (0, 16, 160, 3), (80, 16, 160, 3)),                # [H][q, k][M]
    (5, (0, 32, 160, 3), (16, 32, 160, 3)),                # [H][M][q, k]
    (5, (0, 16, 80, 4), (320, 16, 80, 2)),                 # [q | k][M]
    (5, (0, 96, 32, 3), (16, 96, 999 * 16, 1)),            # one key head between the query heads
    (1, (0, 7 * 16, 32, 3), (16, 5 * 16, 32, 3)),          # one token
    (5, (0, 96, 16, 4), (0, 96, 16, 4)),                   # the same
    (5, (0, 96, 16, 4), (48, 96, 16, 2)),                  # the last query head is the first key head
    (5, (0, 96, 32, 3), (8, 96, 32, 3)),                   # half a head off
    (5, (0, 96, 32, 3), (24, 96, 32, 3)),
    (5, (0, 96, 32, 3), (32, 96, 32, 3)),                  # a head on
    (5, (0, 96, 16, 4), (64, 112, 16, 2)),                 # rows of different lengths
    (5, (0, 16, 80, 4), (240, 16, 80, 2)),
])
def test_queries_and_keys_in_one_buffer(L, M, q, k):
    shared = np.intersect1d(_places(M, q), _places(M, k)).size > 0
    assert _in_place(L, M, q, k) == (INVALID if shared else CUDA)


def test_no_layout_that_shares_an_element_passes(L):
    """Random strides: a refusal of what shares none is allowed there, the reverse never."""
    rng = np.random.default_rng(0)
    passed = 0
    for _ in range(3000):
        M, u = int(rng.integers(1, 6)), 8
        sets = []
        for _ in range(2):
            n = int(rng.integers(1, 5))
            sets.append((u * int(rng.integers(0, 40)), u * int(rng.integers(0, 25)), u * int(rng.integers(0, 25)), n))
        if rng.random() < 0.6:
            sets[1] = (sets[1][0], sets[0][1], sets[0][2], sets[1][3])
        r = _in_place(L, M, *sets)
        assert r in (INVALID, CUDA)
        if r == CUDA:
            passed += 1
            a, b = _places(M, sets[0]), _places(M, sets[1])
            assert np.unique(a).size == a.size and np.unique(b).size == b.size and np.intersect1d(a, b).size == 0, (M, sets)
    assert passed > 50
