"""The FP4 entry cache (MXFP4 body, BF16 rotary dims) on the GPU: writing and
reading back bit for bit against the oracle, and the core attention over the
cache against the oracle's attention over the entries read back."""
import numpy as np
import pytest
import torch

from oracle import lcsa_oracle as O
from workloads import gen

pytestmark = pytest.mark.gpu

DEV = "cuda"
# Attention in BF16 with FP32 sums: weights and rotated keys are rounded by at most 2^-9 of their value each, so an
# output, a mean of keys of unit size, moves by about 2^-8 times its own size at most and far less on average.
ATT_MAX, ATT_MEAN, LSE_TOL = 1e-2, 1e-3, 2e-3


@pytest.fixture(scope="module")
def lcsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    return build_library()


def np64(t):
    return t.detach().double().cpu().numpy()


def parts(cache):
    return tuple(t.cpu().numpy() if t.dtype == torch.uint8 else np64(t) for t in cache)


def expand(cache):
    return O.dequantize_entries_fp4(*parts(cache))


# ------------------------------------------------------------------ writing
def _entries(dtype, D, R, seed):
    """Rows [40, D] with the edge cases of the scale and code rules."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(40, D, generator=g) * torch.exp2(torch.randint(-20, 20, (40, 1), generator=g).float())
    x[0, :32] = 0.0                                     # all-zero block
    x[1, :32] = -0.0                                    # negative zeros code +0
    x[2, :32] = torch.randn(32, generator=g) * 2.0 ** -130     # a block of subnormals
    x[3, :32] = 1.0
    x[3, 0] = 4.0                                       # scale 1, then every midpoint: ties go to the even code
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 6.0, 7.5])
    x[3, 1:17] = mids
    x[4, :32] = x[4, :32] * 1e-3
    x[4, 5], x[4, 6], x[4, 7] = 1.0, -2.0 ** -140, 2.0 ** -140  # values that round to zero keep their sign
    x[5, 0] = 3.0e38                                    # the largest scales
    x[6, :32] = 2.0 ** -126
    x[7, 3] = float("inf")                              # blocks without a scale
    x[8, 4] = float("nan")
    x[9, 0] = -float("inf")
    return x.to(torch.float32 if dtype == "fp32" else torch.bfloat16)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D,R", [(512, 64), (64, 32), (72, 8), (32, 0), (640, 64), (288, 96)])
def test_quantize_entries_fp4_bit_exact(lcsa, dtype, D, R):
    x = _entries(dtype, D, R, 81)
    cache = lcsa.quantize_entries_fp4(x.to(DEV), R)
    for got, ref in zip(parts(cache), O.quantize_entries_fp4(x.double().numpy(), R)):
        np.testing.assert_array_equal(got, ref)
    assert lcsa.get_device_status() == 0


@pytest.mark.parametrize("B,n,rows,row0", [(3, 1, 9, 4), (2, 131, 200, 69), (1, 5, 5, 0), (5, 2, 300, 0)])
def test_quantize_entries_fp4_appends(lcsa, B, n, rows, row0):
    """Rows row0 .. row0+n-1 of every sequence are written, the others stay as they were."""
    g = torch.Generator().manual_seed(82)
    x = torch.randn(B, n, 512, generator=g).to(torch.bfloat16)
    cache = lcsa.empty_fp4_cache(B, rows)
    cache[0].random_(0, 256)
    cache[1].random_(0, 256)
    cache[2].normal_()
    before = [t.clone() for t in cache]
    lcsa.quantize_entries_fp4(x.to(DEV), 64, cache=cache, row0=row0)
    for got, old, ref in zip(cache, before, O.quantize_entries_fp4(x.double().numpy(), 64)):
        want = old.clone()
        want[:, row0:row0 + n] = torch.as_tensor(ref).to(want.dtype)
        assert torch.equal(got, want)
    with pytest.raises(lcsa.LcsaError):
        lcsa.quantize_entries_fp4(x.to(DEV), 64, cache=cache, row0=rows - n + 1)


# ------------------------------------------------------------------ reading back
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,R", [(512, 64), (64, 32), (72, 8), (32, 0), (640, 64)])
def test_dequantize_entries_fp4_bit_exact(lcsa, out, D, R):
    g = torch.Generator().manual_seed(83)
    cache = lcsa.empty_fp4_cache(2, 300, D, R)
    cache[0].copy_(torch.randint(0, 256, cache[0].shape, generator=g, dtype=torch.uint8))     # every code
    nblk = (D - R) // 32
    cache[1][..., :nblk] = torch.randint(0, 253, (2, 300, nblk), generator=g, dtype=torch.uint8).to(DEV)
    cache[1][0, 5, 0] = 255                             # a block without a scale reads back as NaN
    cache[2].copy_(torch.randn(cache[2].shape, generator=g))
    ref = expand(cache)
    got = lcsa.dequantize_entries_fp4(cache, out_dtype=out)
    assert got.dtype == out
    np.testing.assert_array_equal(np64(got), ref)
    idx = torch.randint(0, 300, (2, 77), generator=g, dtype=torch.int32)
    idx[0, 3] = idx[1, 70] = -1
    idx[1, 4] = idx[1, 5]
    got = np64(lcsa.dequantize_entries_fp4(cache, idx=idx.to(DEV), out_dtype=out))
    want = np.stack([ref[b][idx[b].clamp(min=0).numpy()] for b in range(2)])
    want[idx.numpy() < 0] = 0.0
    np.testing.assert_array_equal(got, want)
    assert lcsa.get_device_status() == 0


def test_dequantize_bad_index_gives_a_zero_row_and_is_flagged(lcsa):
    cache = lcsa.quantize_entries_fp4(torch.ones(1, 10, 512, device=DEV), 64)
    got = lcsa.dequantize_entries_fp4(cache, idx=torch.tensor([[3, 10, -2, 2147483647, 9]], dtype=torch.int32, device=DEV))
    assert lcsa.get_device_status() == 2
    assert lcsa.get_device_status() == 0
    assert got[0, :, 0].tolist() == [1, 0, 0, 0, 1]


# ------------------------------------------------------------------ attention
def check_attn(lcsa, x, cache, idx, q_pos0, kv_pos0, m, W, R, rows=None, sink=True, **kw):
    B, Tq = x["q"].shape[:2]
    sk = x["sink"] if sink else None
    args = (q_pos0, kv_pos0, m, W, R)
    if idx is not None:
        out, lse = lcsa.csa_sparse_attn_fp4(x["q"], cache, idx, x["kv"], sk, *args, return_lse=True, **kw)
    else:
        out, lse = lcsa.hca_dense_attn_fp4(x["q"], cache, x["kv"], sk, *args, return_lse=True, **kw)
    assert lcsa.get_device_status() == 0
    d = expand(cache)
    ref_sink = np64(sk) if sink else None
    rows = rows or [(b, i) for b in range(B) for i in range(Tq)]
    okw = dict(rows=rows)
    if "softmax_scale" in kw:
        okw["scale"] = kw["softmax_scale"]
    if "rope_base" in kw:
        okw["base"] = kw["rope_base"]
    if idx is not None:
        ref, ref_lse = O.csa_sparse_attn(np64(x["q"]), d, idx.cpu().numpy(), np64(x["kv"]), q_pos0, kv_pos0, m, W,
                                         ref_sink, R, **okw)
    else:
        ref, ref_lse = O.hca_dense_attn(np64(x["q"]), d, np64(x["kv"]), q_pos0, kv_pos0, m, W, ref_sink, R, **okw)
    got = np64(out)[[r[0] for r in rows], [r[1] for r in rows]]
    got_lse = np64(lse)[[r[0] for r in rows], [r[1] for r in rows]]
    err = np.abs(got - ref)
    assert err.max() <= ATT_MAX, f"max abs err {err.max():.3e}"
    assert err.mean() <= ATT_MEAN, f"mean abs err {err.mean():.3e}"
    np.testing.assert_allclose(got_lse, ref_lse, atol=LSE_TOL)
    return out


def made(lcsa, B, Tq, Nc, q_pos0, Tkv, seed, unit=True, H=64, D=512, R=64, dtype="bf16"):
    x = gen.make_attn_inputs(B, Tq, H, D, Nc, Tkv, dtype, seed=seed, device=DEV, unit_scale=unit)
    return x, lcsa.quantize_entries_fp4(x["ckv"], R)


def selection(B, Tq, k, q_pos0, m, Nc, seed):
    nv = [O.n_visible(q_pos0 + i, m, Nc) for i in range(Tq)]
    return gen.make_topk_idx(B, Tq, k, nv, seed=seed, device=DEV)


@pytest.mark.parametrize("B,k,Tq,Nc,q_pos0,unit", [
    (2, 256, 40, 700, 2700, True),       # several tiles
    (2, 256, 40, 700, 2700, False),      # spec scale
    (2, 2048, 9, 2500, 9000, True),      # full k
    (2, 100, 20, 900, 3000, True),       # odd k: ragged last tile
    (1, 3001, 4, 5000, 19000, True),     # k > 2048, odd
    (3, 61, 37, 9, 0, True),             # first rows: empty and short selections
    (1, 2048, 1, 20000, 80003, True),    # one decode query
    (7, 1, 1, 5, 21, True),              # one selected entry
    (1, 127, 170, 300, 1200, True),      # more rows than SMs
    (1, 129, 3, 300, 1200, False),
])
def test_csa_sparse_attn_fp4_parity(lcsa, B, k, Tq, Nc, q_pos0, unit):
    x, cache = made(lcsa, B, Tq, Nc, q_pos0, q_pos0 + Tq, 91, unit)
    check_attn(lcsa, x, cache, selection(B, Tq, k, q_pos0, 4, Nc, 92), q_pos0, 0, 4, 128, 64)


@pytest.mark.parametrize("B,m,Tq,Nc,q_pos0,W,sink", [
    (2, 128, 130, 40, 2000, 128, True),  # crosses a 128-block boundary
    (2, 16, 20, 400, 5000, 128, False),  # many entries, no sink
    (1, 128, 70, 40, 0, 128, True),      # t < m: window only
    (2, 128, 3, 40, 0, 0, False),        # no key at all: zero rows
    (1, 128, 3, 40, 126, 0, True),       # W = 0, the first entry becomes visible
    (2, 4, 5, 1000, 3999, 300, True),    # a window of several tiles
    (1, 4, 1, 130, 5000, 1, True),       # every entry visible, a window of one row
    (3, 128, 1, 1, 128, 128, False),
])
def test_hca_dense_attn_fp4_parity(lcsa, B, m, Tq, Nc, q_pos0, W, sink):
    x, cache = made(lcsa, B, Tq, Nc, q_pos0, q_pos0 + Tq, 93)
    check_attn(lcsa, x, cache, None, q_pos0, 0, m, W, 64, sink=sink)


@pytest.mark.parametrize("Nc,splits_of", [(1040, "few tiles"), (8192, "many tiles")])
def test_hca_fp4_long_context_decode(lcsa, Nc, splits_of):
    B, q_pos0, W = 2, Nc * 128 + 5, 128
    kv_pos0 = q_pos0 - W + 1
    x, cache = made(lcsa, B, 1, Nc, q_pos0, W, 94)
    check_attn(lcsa, x, cache, None, q_pos0, kv_pos0, 128, W, 64)


def test_attn_fp4_window_ring_and_options(lcsa):
    """A decode ring (kv_pos0 > 0), a ring that lost its oldest rows, another softmax scale and rotary base."""
    B, Tq, Nc, q_pos0, W = 2, 3, 500, 2100, 128
    x, cache = made(lcsa, B, Tq, Nc, q_pos0, 90 + Tq, 95)
    idx = selection(B, Tq, 300, q_pos0, 4, Nc, 96)
    check_attn(lcsa, x, cache, idx, q_pos0, q_pos0 - 90, 4, W, 64)
    check_attn(lcsa, x, cache, idx, q_pos0, q_pos0 - 90, 4, W, 64, softmax_scale=0.01)
    check_attn(lcsa, x, cache, None, q_pos0, q_pos0 - 90, 4, W, 64, rope_base=500.0)
    check_attn(lcsa, x, cache, None, q_pos0, q_pos0 - 90, 4, W, 64, sink=False)


@pytest.mark.parametrize("dtype,H,D,R", [("fp32", 4, 64, 32), ("bf16", 4, 64, 32), ("bf16", 8, 576, 64),
                                         ("fp32", 64, 512, 64), ("bf16", 16, 512, 64)])
def test_attn_fp4_other_shapes(lcsa, dtype, H, D, R):
    """Shapes of the CUDA-core kernels."""
    B, Tq, Nc, q_pos0, W = 2, 5, 60, 230, 64
    x, cache = made(lcsa, B, Tq, Nc, q_pos0, q_pos0 + Tq, 97, H=H, D=D, R=R, dtype=dtype)
    check_attn(lcsa, x, cache, selection(B, Tq, 20, q_pos0, 4, Nc, 98), q_pos0, 0, 4, W, R)
    check_attn(lcsa, x, cache, None, q_pos0, 0, 4, W, R)


def test_attn_fp4_bf16_output_and_caller_buffers(lcsa):
    B, Tq, Nc, q_pos0 = 2, 3, 400, 1700
    x, cache = made(lcsa, B, Tq, Nc, q_pos0, q_pos0 + Tq, 99)
    idx = selection(B, Tq, 200, q_pos0, 4, Nc, 100)
    ref = lcsa.csa_sparse_attn_fp4(x["q"], cache, idx, x["kv"], x["sink"], q_pos0, 0)
    out = torch.full((B, Tq, 64, 512), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(lcsa.attn_fp4_workspace_bytes(x["q"], cache, idx, x["kv"], 4, 128, q_pos0=q_pos0) + 256,
                     dtype=torch.uint8, device=DEV)
    got = lcsa.csa_sparse_attn_fp4(x["q"], cache, idx, x["kv"], x["sink"], q_pos0, 0, out=out, workspace=ws)
    assert got is out
    assert torch.equal(out, ref.to(torch.bfloat16))       # the same sums, rounded once


def test_attn_fp4_bad_index_is_skipped_and_flagged(lcsa):
    B, Tq, m, W, k, Nc, q_pos0 = 1, 3, 4, 128, 64, 500, 2400
    x, cache = made(lcsa, B, Tq, Nc, q_pos0, q_pos0 + Tq, 101)
    idx = selection(B, Tq, k, q_pos0, m, Nc, 102)
    bad = idx.clone()
    bad[0, 1, k - 1] = Nc + 7                            # past the cache
    bad[0, 2, :] = Nc                                    # every slot of row 2
    out = lcsa.csa_sparse_attn_fp4(x["q"], cache, bad, x["kv"], x["sink"], q_pos0, 0, m, W, 64)
    assert lcsa.get_device_status() == 2
    assert lcsa.get_device_status() == 0                 # read and cleared
    sel = bad.cpu().numpy().copy()
    sel[sel >= Nc] = -1                                  # the skipped slots are no keys at all
    ref, _ = O.csa_sparse_attn(np64(x["q"]), expand(cache), sel, np64(x["kv"]), q_pos0, 0, m, W, np64(x["sink"]), 64)
    err = np.abs(np64(out).reshape(ref.shape) - ref)
    assert err.max() <= ATT_MAX and err.mean() <= ATT_MEAN
