"""What a call over the FP4 entry cache means does not depend on the kernel that its size picks: the tile kernel, the
read-back path of calls with many rows, or the CUDA-core kernel of other shapes."""
import numpy as np
import pytest
import torch

from oracle import lcsa_oracle as O
from workloads import gen

pytestmark = pytest.mark.gpu

DEV = "cuda"
# A rounding to BF16 is off by at most 2^-8 of the value.  Weights and rotated keys are rounded once each and averaged
# over the keys, so an output moves by a fraction of 2 * 2^-8 times the size of its keys (about 1 here, 5 where an
# output is a mean of few keys).
ATT_MAX = 1e-2


@pytest.fixture(scope="module")
def lcsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    return build_library()


def np64(t):
    return t.detach().double().cpu().numpy()


def expand(cache):
    return O.dequantize_entries_fp4(*(t.cpu().numpy() if t.dtype == torch.uint8 else np64(t) for t in cache))


def inputs(lcsa, B, Tq, Nc, Tkv, seed, H=64, D=512, R=64, dtype="bf16"):
    x = gen.make_attn_inputs(B, Tq, H, D, Nc, Tkv, dtype, seed=seed, device=DEV, unit_scale=True)
    return x, lcsa.quantize_entries_fp4(x["ckv"], R)


def poison(cache, b, rows):
    cache[1][b, rows] = 255                            # scale NaN
    cache[2][b, rows] = float("inf")


# ------------------------------------------------------------------ sequences stay apart
@pytest.mark.parametrize("B,Nc", [(2, 1475), (3, 1500), (2, 2000), (2, 1472), (1, 1475), (2, 1400), (1, 1400)])
def test_large_dense_calls_keep_sequences_apart(lcsa, B, Nc):
    """The last tile of a sequence's entries is not whole; what the next sequence's first entries hold does not matter.
    (1400: fewer entries than the last rows' positions would show.)"""
    Tq, q_pos0, m, W = 900, 5000, 4, 128
    x, cache = inputs(lcsa, B, Tq, Nc, W + Tq - 1, 61)
    args = (x["kv"], x["sink"], q_pos0, q_pos0 - W + 1, m, W)
    clean, lse = lcsa.hca_dense_attn_fp4(x["q"], cache, *args, return_lse=True)
    ref, ref_lse = lcsa.hca_dense_attn(x["q"], lcsa.dequantize_entries_fp4(cache), *args, return_lse=True)
    assert (clean - ref).abs().max() <= 2 * ATT_MAX and (lse - ref_lse).abs().max() <= 4e-3
    for b in range(1, B):
        poison(cache, b, slice(0, 64))
    out, lse2 = lcsa.hca_dense_attn_fp4(x["q"], cache, *args, return_lse=True)
    assert torch.equal(out[0], clean[0]) and torch.equal(lse2[0], lse[0])
    assert not torch.isfinite(out[1:]).any()           # those sequences see their NaN
    assert lcsa.get_device_status() == 0
