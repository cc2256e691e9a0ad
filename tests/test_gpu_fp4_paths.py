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


# ------------------------------------------------------------------ holes in a selection
def holed(B, Tq, k, q_pos0, m, Nc, seed):
    """A selection with holes, and the same entries without them (padded at the end)."""
    idx = gen.make_topk_idx(B, Tq, k, [O.n_visible(q_pos0 + i, m, Nc) for i in range(Tq)], seed=seed, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(seed)
    hole = torch.rand(idx.shape, generator=g, device=DEV) < 0.1
    hole[..., k // 2] = True
    hole[0, 0] = True                                  # nothing left
    hole[0, 1, :-1] = True                             # only the last slot
    hole[-1, 2, 0] = True
    idx[hole] = -1
    idx[0, 3, k // 3] = -5                             # any negative number is no key
    tight = torch.full_like(idx, -1)
    live = idx >= 0
    place = live.cumsum(-1) - 1
    b, i, s = live.nonzero(as_tuple=True)
    tight[b, i, place[b, i, s]] = idx[b, i, s]
    return idx, tight


def check_holes(lcsa, x, cache, idx, tight, q_pos0, kv_pos0, m, W, R, rows, exact):
    args = (x["kv"], x["sink"], q_pos0, kv_pos0, m, W, R)
    out, lse = lcsa.csa_sparse_attn_fp4(x["q"], cache, idx, *args, return_lse=True)
    assert lcsa.get_device_status() == 0
    same, same_lse = lcsa.csa_sparse_attn_fp4(x["q"], cache, tight, *args, return_lse=True)
    if exact:                                          # the same keys in the same order
        assert torch.equal(out, same) and torch.equal(lse, same_lse)
    else:                                              # each within ATT_MAX of the exact value, keys up to 5
        assert (out - same).abs().max() <= 2 * 5 * ATT_MAX and (lse - same_lse).abs().max() <= 4e-3
    d, q, kv, s = expand(cache), np64(x["q"]), np64(x["kv"]), np64(x["sink"])
    for b, i in rows:
        sel = idx[b, i].cpu().numpy()
        ref, _ = O.attend_one(q[b, i], q_pos0 + i, sel[sel >= 0], d[b], m, kv[b], kv_pos0, W, s, R)
        # (5: windows that are not whole leave means of few keys)
        assert np.abs(np64(out[b, i]) - ref).max() <= (1 if exact else 5) * ATT_MAX


@pytest.mark.parametrize("k", [600, 61])
def test_holes_in_the_selections_of_a_large_call(lcsa, k):
    B, Tq, q_pos0, m, W, Nc = 2, 1500 if k == 600 else 3000, 5000, 4, 128, 1475
    x, cache = inputs(lcsa, B, Tq, Nc, W + Tq - 1, 62)
    idx, tight = holed(B, Tq, k, q_pos0, m, Nc, 63)
    rows = [(0, 0), (0, 1), (0, 2), (0, 3), (1, 2), (1, Tq - 1)]
    assert lcsa.attn_fp4_workspace_bytes(x["q"], cache, idx, x["kv"], m, W, q_pos0=q_pos0, kv_pos0=q_pos0 - W + 1) > 0
    check_holes(lcsa, x, cache, idx, tight, q_pos0, q_pos0 - W + 1, m, W, 64, rows, True)


def test_holes_where_windows_are_not_whole(lcsa):
    """A call whose first rows go to another kernel than the rest."""
    B, Tq, q_pos0, m, W, Nc, k = 2, 1500, 40, 4, 128, 400, 300
    x, cache = inputs(lcsa, B, Tq, Nc, q_pos0 + Tq, 64)
    idx, tight = holed(B, Tq, k, q_pos0, m, Nc, 65)
    check_holes(lcsa, x, cache, idx, tight, q_pos0, 0, m, W, 64, [(0, 0), (1, 50), (1, 86), (1, 87), (0, 1400)], False)


@pytest.mark.parametrize("dtype,H,D,R", [("fp32", 4, 64, 32), ("bf16", 16, 512, 64), ("fp32", 64, 512, 64)])
def test_holes_in_selections_of_other_shapes(lcsa, dtype, H, D, R):
    B, Tq, Nc, q_pos0, m, W, k = 2, 5, 60, 230, 4, 64, 20
    x, cache = inputs(lcsa, B, Tq, Nc, q_pos0 + Tq, 66, H=H, D=D, R=R, dtype=dtype)
    idx, tight = holed(B, Tq, k, q_pos0, m, Nc, 67)
    check_holes(lcsa, x, cache, idx, tight, q_pos0, 0, m, W, R, [(b, i) for b in range(B) for i in range(Tq)], True)


# ------------------------------------------------------------------ NaN in one part of a long key list
@pytest.mark.parametrize("B", [1, 140])
@pytest.mark.parametrize("bad", [slice(40, 41), slice(0, 256)])
@pytest.mark.parametrize("large", ["key", "sink"])
def test_nan_reaches_the_output_beside_far_larger_logits(lcsa, B, bad, large):
    """One key list over many CTAs (B = 1) or in one (B = 140): a NaN among keys whose weights vanish beside another
    key's, or the sink's, is a NaN of the output."""
    Nc, m, q_pos0, W = 3000, 4, 12005, 128
    x, _ = inputs(lcsa, B, 1, Nc, W, 68)
    base = torch.randn(512, generator=torch.Generator().manual_seed(3)).to(DEV)
    base[448:] = 0                                     # rotation leaves the logits alone
    x["q"] = (x["q"].float() * 0.1 + 4 * base).bfloat16()
    x["ckv"] = (x["ckv"].float() * 0.1).bfloat16()
    sink = x["sink"].clone()
    if large == "key":
        x["ckv"][:, 2900] = (4 * base).bfloat16()      # a logit of some 300
    else:
        sink += 300.0
    cache = lcsa.quantize_entries_fp4(x["ckv"], 64)
    call = lambda: lcsa.hca_dense_attn_fp4(x["q"], cache, x["kv"], sink, q_pos0, q_pos0 - W + 1, m, W, return_lse=True)
    out, lse = call()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    cache[1][:, bad] = 255
    out, lse = call()
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    assert lcsa.get_device_status() == 0


# ------------------------------------------------------------------ workspaces
@pytest.mark.parametrize("sparse", [True, False])
def test_a_workspace_too_small_for_reading_back_is_left_alone(lcsa, sparse):
    """Calls of the tile kernel's shape run without the room to read the cache back; nothing is allocated then."""
    B, Tq, q_pos0, m, W, Nc, k = 2, 900, 5000, 4, 128, 1475, 600
    x, cache = inputs(lcsa, B, Tq, Nc, W + Tq - 1, 69)
    idx = gen.make_topk_idx(B, Tq, k, [O.n_visible(q_pos0 + i, m, Nc) for i in range(Tq)], seed=70, device=DEV) if sparse else None
    kv_pos0 = q_pos0 - W + 1
    need = lcsa.attn_fp4_workspace_bytes(x["q"], cache, idx, x["kv"], m, W, q_pos0=q_pos0, kv_pos0=kv_pos0)
    assert need > 0
    out = torch.zeros(B, Tq, 64, 512, device=DEV)

    def call(**kw):
        if sparse:
            return lcsa.csa_sparse_attn_fp4(x["q"], cache, idx, x["kv"], x["sink"], q_pos0, kv_pos0, m, W, **kw)
        return lcsa.hca_dense_attn_fp4(x["q"], cache, x["kv"], x["sink"], q_pos0, kv_pos0, m, W, **kw)

    want = call()
    for size in (need - 256, 0):
        ws = torch.full((size,), 0x5A, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        held = torch.cuda.memory_allocated()
        assert call(out=out.zero_(), workspace=ws) is out
        assert torch.cuda.max_memory_allocated() == held
        assert (ws == 0x5A).all()
        assert (out - want).abs().max() <= 2 * ATT_MAX
    assert lcsa.get_device_status() == 0


def test_a_workspace_too_small_for_other_shapes_is_refused(lcsa):
    B, Tq, Nc, q_pos0, m, W = 2, 5, 60, 230, 4, 64
    x, cache = inputs(lcsa, B, Tq, Nc, q_pos0 + Tq, 71, H=4, D=64, R=32, dtype="fp32")
    need = lcsa.attn_fp4_workspace_bytes(x["q"], cache, None, x["kv"], m, W, R=32, q_pos0=q_pos0)
    assert need > 0
    args = (x["q"], cache, x["kv"], x["sink"], q_pos0, 0, m, W, 32)
    want = lcsa.hca_dense_attn_fp4(*args)
    assert torch.equal(lcsa.hca_dense_attn_fp4(*args, workspace=torch.empty(need, dtype=torch.uint8, device=DEV)), want)
    with pytest.raises(lcsa.LcsaError):
        lcsa.hca_dense_attn_fp4(*args, workspace=torch.empty(need - 256, dtype=torch.uint8, device=DEV))


# ------------------------------------------------------------------ rows whose window is not whole
@pytest.mark.parametrize("sparse", [True, False])
@pytest.mark.parametrize("B,Tq,back", [(1, 200, 60), (3, 500, 0), (1, 700, 126)])
def test_rows_whose_window_is_not_whole(lcsa, sparse, B, Tq, back):
    """Their kernel's results, whatever the other rows' kernel (its keys split where the rows are few) finds in the
    workspace."""
    Nc, m, W, k = 8192 if Tq == 200 else 2048, 4, 128, 1024
    q_pos0 = 4 * Nc - Tq
    x, cache = inputs(lcsa, B, Tq, Nc, back + Tq, 79)
    idx = gen.make_topk_idx(B, Tq, k, [O.n_visible(q_pos0 + i, m, Nc) for i in range(Tq)], seed=80, device=DEV) if sparse else None
    kv_pos0 = q_pos0 - back
    need = lcsa.attn_fp4_workspace_bytes(x["q"], cache, idx, x["kv"], m, W, q_pos0=q_pos0, kv_pos0=kv_pos0)
    assert need > 0 or sparse and Tq == 200

    def call(ws):
        args = (x["kv"], x["sink"], q_pos0, kv_pos0, m, W)
        kw = dict(return_lse=True, workspace=ws)
        return lcsa.csa_sparse_attn_fp4(x["q"], cache, idx, *args, **kw) if sparse else lcsa.hca_dense_attn_fp4(x["q"], cache, *args, **kw)

    want, want_lse = call(torch.empty(0, dtype=torch.uint8, device=DEV))
    first = None
    for fill in (0xFF, 0x3C):
        out, lse = call(torch.full((need,), fill, dtype=torch.uint8, device=DEV))
        assert (out - want).abs().max() <= 2 * ATT_MAX and (lse - want_lse).abs().max() <= 4e-3
        first = first or (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    rows = [(0, 0), (B - 1, 126 - back), (B - 1, 127 - back), (0, Tq - 1)]
    sel = (idx.cpu().numpy(),) if sparse else ()
    want, _ = (O.csa_sparse_attn if sparse else O.hca_dense_attn)(np64(x["q"]), expand(cache), *sel, np64(x["kv"]), q_pos0, kv_pos0,
                                                                  m, W, np64(x["sink"]), 64, rows=rows)
    assert np.abs(np64(out)[[r[0] for r in rows], [r[1] for r in rows]] - want).max() <= ATT_MAX
    assert lcsa.get_device_status() == 0


# ------------------------------------------------------------------ arguments
def test_positions_of_any_integer_type(lcsa):
    """As in the calls over BF16 entries: numpy integers and tensors of one element are positions."""
    B, Nc, q_pos0, m, W = 2, 100, 420, 4, 128
    x, cache = inputs(lcsa, B, 1, Nc, W, 72)
    want = lcsa.hca_dense_attn_fp4(x["q"], cache, x["kv"], x["sink"], q_pos0, q_pos0 - W + 1, m, W)
    for t in (np.int64, np.int32, torch.tensor):
        got = lcsa.hca_dense_attn_fp4(x["q"], cache, x["kv"], x["sink"], t(q_pos0), t(q_pos0 - W + 1), m, W)
        assert torch.equal(got, want)


# ------------------------------------------------------------------ capacity
@pytest.mark.parametrize("sparse", [True, False])
def test_a_cache_larger_than_its_entries(lcsa, sparse):
    """The rows of a cache that is allocated for a longer context hold anything; many rows at its start."""
    B, Tq, q_pos0, m, W, k = 2, 2048, 0, 4, 128, 512
    n = (q_pos0 + Tq) // m
    x, cache = inputs(lcsa, B, Tq, n, q_pos0 + Tq, 73)
    idx = gen.make_topk_idx(B, Tq, k, [O.n_visible(q_pos0 + i, m, n) for i in range(Tq)], seed=74, device=DEV) if sparse else None
    big = lcsa.empty_fp4_cache(B, 120000)
    big[0].fill_(0x77)
    big[1].fill_(255)
    big[2].fill_(float("nan"))
    for t, c in zip(big, cache):
        t[:, :n] = c

    def call(c):
        if sparse:
            return lcsa.csa_sparse_attn_fp4(x["q"], c, idx, x["kv"], x["sink"], q_pos0, 0, m, W)
        return lcsa.hca_dense_attn_fp4(x["q"], c, x["kv"], x["sink"], q_pos0, 0, m, W)

    want, got = call(cache), call(big)
    if sparse:
        assert (got - want).abs().max() <= 2 * 5 * ATT_MAX          # by another kernel
    else:
        assert torch.equal(got, want)
    assert lcsa.get_device_status() == 0


# ------------------------------------------------------------------ long selections
def test_many_rows_of_more_selected_entries_than_2048(lcsa):
    """Calls that take no workspace whatever their rows."""
    B, Tq, q_pos0, m, W, Nc, k = 1, 600, 16000, 4, 128, 4150, 2501
    x, cache = inputs(lcsa, B, Tq, Nc, W + Tq - 1, 75)
    idx = gen.make_topk_idx(B, Tq, k, [O.n_visible(q_pos0 + i, m, Nc) for i in range(Tq)], seed=76, device=DEV)
    kv_pos0 = q_pos0 - W + 1
    assert lcsa.attn_fp4_workspace_bytes(x["q"], cache, idx, x["kv"], m, W, q_pos0=q_pos0, kv_pos0=kv_pos0) == 0
    out = lcsa.csa_sparse_attn_fp4(x["q"], cache, idx, x["kv"], x["sink"], q_pos0, kv_pos0, m, W)
    rows = [(0, 0), (0, 311), (0, 599)]
    want, _ = O.csa_sparse_attn(np64(x["q"]), expand(cache), idx.cpu().numpy(), np64(x["kv"]), q_pos0, kv_pos0, m, W,
                                np64(x["sink"]), 64, rows=rows)
    assert np.abs(np64(out)[[r[0] for r in rows], [r[1] for r in rows]] - want).max() <= ATT_MAX
    assert lcsa.get_device_status() == 0


# ------------------------------------------------------------------ offsets
def test_offsets_past_two_gigabytes(lcsa):
    """Rows of a cache behind 2^31 bytes of codes and of rotary dims: written, read back and attended to as in a cache
    of their own."""
    B, Nc, m, W, k, D = 2, 9_000_000, 4, 128, 300, 512
    q_pos0 = 4 * Nc + 2
    g = torch.Generator(device=DEV).manual_seed(77)
    new = torch.randn(B, 400, D, generator=g, device=DEV).bfloat16()
    cache = lcsa.empty_fp4_cache(B, Nc)
    lcsa.quantize_entries_fp4(new, 64, cache=cache, row0=Nc - 400)
    own = lcsa.quantize_entries_fp4(new, 64)
    for t, o in zip(cache, own):
        assert torch.equal(t[:, Nc - 400:], o)
        assert not t[1, :Nc - 400].any()
    idx = torch.arange(Nc - 400, Nc, dtype=torch.int32, device=DEV).expand(B, -1).contiguous()
    assert torch.equal(lcsa.dequantize_entries_fp4(cache, idx=idx), lcsa.dequantize_entries_fp4(own))
    x = gen.make_attn_inputs(B, 1, 64, D, 1, W, "bf16", seed=78, device=DEV, unit_scale=True)
    sel = idx[:, 400 - k:].reshape(B, 1, k).contiguous()
    args = (x["sink"], q_pos0, q_pos0 - W + 1, m, W)
    out = lcsa.csa_sparse_attn_fp4(x["q"], cache, sel, x["kv"], *args)
    # positions count by their differences alone: the selected rows as entries 0 .. k-1 of a shorter sequence
    e, t = expand(tuple(c[:, 400 - k:].contiguous() for c in own)), q_pos0 - (Nc - k) * m
    for b in range(B):
        want, _ = O.attend_one(np64(x["q"])[b, 0], t, np.arange(k), e[b], m, np64(x["kv"])[b], t - W + 1, W, np64(x["sink"]), 64)
        assert np.abs(np64(out)[b, 0] - want).max() <= ATT_MAX
    assert lcsa.get_device_status() == 0


# ------------------------------------------------------------------ precision
@pytest.mark.parametrize("B,Nc", [(1, 3000), (140, 40), (2, 1)])
def test_weights_sum_to_one(lcsa, B, Nc):
    """Dims in which all keys agree come back as they are, whatever the weights' rounding: FP32 sums of the rounded
    weights, off by 2^-24 a step."""
    m, W = 4, 128
    q_pos0 = 4 * Nc + 3
    x, _ = inputs(lcsa, B, 1, Nc, W, 81)
    x["q"][..., 64:] = 0                               # logits from the first 64 dims, which differ
    x["ckv"][..., 64:] = 1.5
    x["kv"][..., 64:] = 1.5
    x["ckv"][..., 448:] = x["kv"][..., 448:] = 0       # (dims that turn)
    cache = lcsa.quantize_entries_fp4(x["ckv"], 64)
    x["q"] = (x["q"].float() * 4).bfloat16()           # logits of standard deviation sqrt(64) * 4 / 22.6 = 1.4
    out = lcsa.hca_dense_attn_fp4(x["q"], cache, x["kv"], None, q_pos0, q_pos0 - W + 1, m, W)
    # sums of up to 64 products a tile and 49 tiles, two roundings each, in the numerator and the sum
    assert (out[..., 64:448] - 1.5).abs().max() <= 1.5 * 2 * 113 * 2.0 ** -24 * 4
    assert (out[..., 448:] == 0).all()


@pytest.mark.parametrize("t", [3, 1000, 1048575])
def test_queries_are_not_rounded(lcsa, t):
    """A key at the query's own position: its logit is the product of the two as given, at any position."""
    B, W = 3, 1
    x, cache = inputs(lcsa, B, 1, 1, 1, 82)
    out, lse = lcsa.hca_dense_attn_fp4(x["q"], tuple(c[:, :0].contiguous() for c in cache), x["kv"], None, t, t, 128, W,
                                       return_lse=True)
    q, k = np64(x["q"])[:, 0], np64(x["kv"])[:, 0]
    terms = np.abs(q * k[:, None]).sum(-1) * 512 ** -0.5
    # 512 products summed in FP32 (2^-24 a step at most), the scale and the logarithm: a few roundings of the sum
    assert (np.abs(np64(lse)[:, 0] - np.einsum("bhd,bd->bh", q, k) * 512 ** -0.5) <= terms * 520 * 2.0 ** -24).all()
    assert torch.equal(out[:, 0], x["kv"].float().expand(-1, 64, -1))
