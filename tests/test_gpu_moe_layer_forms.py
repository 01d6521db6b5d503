"""The forms of ar_moe_layer that sizes choose: tiles of 32 output rows, passes over an
expert's weights with fewer columns than binary16 tiles have, and columns that do not fit in
shared memory at all.  Against the definition in binary64, with test_gpu_moe_layer.py's bound
(and its finer one for h, where it is two numbers)."""
import pytest

from test_gpu_moe_layer import _check
from test_gpu_moe_layer_hidden import Layer
from test_gpu_moe_layer_hidden import _check as _check_hidden

import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,K,E,H,F", [
    (16, 4, 4, 8192, 48), (16, 4, 4, 4872, 48), (33, 2, 2, 4888, 40), (32, 2, 3, 5120, 130),
    (9, 1, 1, 4879, 129)])
def test_tiles_of_32_rows(dtype, T, K, E, H, F):
    """Several tokens, more pairs of an expert than columns fit, a last tile that is not whole;
    33 tokens have tiles of 16 rows."""
    _check(T, K, E, H, F, dtype, seed=T + H)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H", [3000, 7000, 10000, 14000, 17000, 20000, 30000])
def test_every_number_of_columns(dtype, H):
    """More pairs of an expert than columns beside the rings, for 16 columns down to a few:
    what is fetched ahead has the order in which it is used."""
    _check(20, 2, 3, H, 33, dtype, seed=H)
    _check(24, 1, 1, H, 16, dtype, ids=[[0]] * 24, seed=H)


@pytest.mark.parametrize("dtype,H", [("fp32", 36480), ("fp32", 36496), ("bf16", 72576),
                                     ("bf16", 72592)])
def test_rows_of_x_beyond_shared_memory(dtype, H):
    """Room for one column, and for none: the first launch then reads x and its weights on the
    way, the second has its rings."""
    _check(10, 1, 2, H, 16, dtype, seed=3)
    _check(3, 2, 2, H, 48, dtype, seed=4)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_h_in_tiles_of_32_rows(dtype):
    for T, K, F in ((16, 4, 48), (20, 2, 200), (9, 1, 129)):
        _check_hidden(Layer(4, 4872, F, F), T, K, dtype, seed=F)
    ids = torch.zeros(20, 1, dtype=torch.int32, device="cuda")
    _check_hidden(Layer(1, 5000, 64, 1), 20, 1, dtype, ids=ids)
