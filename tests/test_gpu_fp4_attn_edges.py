"""Attention over the FP4 entry cache where it can go wrong: extreme scales and logits, masked rows that hold Inf or
NaN, holes in a selection, the read-back path of large calls, alignment, streams, captured graphs, and a decode step
through the calls a server makes."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import lcsa_oracle as O
from workloads import gen

pytestmark = pytest.mark.gpu

DEV = "cuda"
# BF16 keys and weights, FP32 sums: a rounding is off by at most 2^-9 of its value.  An output is a mean of keys, so
# with keys up to `size` it moves by at most 2 * 2^-9 * size, plus the logits' error: the queries' and keys' rotary
# dims are rounded (64 of 512 products, 2^-8 each in the worst case), which for unit inputs is far below 0.1 in a logit
# of standard deviation 1 and averages out; 1e-2 covers both for unit keys.
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


def inputs(lcsa, B, Tq, Nc, Tkv, seed, unit=True):
    x = gen.make_attn_inputs(B, Tq, 64, 512, Nc, Tkv, "bf16", seed=seed, device=DEV, unit_scale=unit)
    return x, lcsa.quantize_entries_fp4(x["ckv"], 64)


def selection(B, Tq, k, q_pos0, m, Nc, seed):
    return gen.make_topk_idx(B, Tq, k, [O.n_visible(q_pos0 + i, m, Nc) for i in range(Tq)], seed=seed, device=DEV)


def oracle(x, cache, idx, q_pos0, kv_pos0, m, W, sink=True, rows=None):
    s = np64(x["sink"]) if sink else None
    if idx is not None:
        return O.csa_sparse_attn(np64(x["q"]), expand(cache), idx.cpu().numpy(), np64(x["kv"]), q_pos0, kv_pos0, m, W, s, 64,
                                 rows=rows)
    return O.hca_dense_attn(np64(x["q"]), expand(cache), np64(x["kv"]), q_pos0, kv_pos0, m, W, s, 64, rows=rows)


def run(lcsa, x, cache, idx, q_pos0, kv_pos0, m, W, sink=True, **kw):
    s = x["sink"] if sink else None
    if idx is not None:
        return lcsa.csa_sparse_attn_fp4(x["q"], cache, idx, x["kv"], s, q_pos0, kv_pos0, m, W, **kw)
    return lcsa.hca_dense_attn_fp4(x["q"], cache, x["kv"], s, q_pos0, kv_pos0, m, W, **kw)


# ------------------------------------------------------------------ values
@pytest.mark.parametrize("power", [-100, -20, 12, 60])
def test_entry_scales(lcsa, power):
    """Entries of any size (the scale's second factor, subnormal products): q shrinks as the keys grow, so the logits
    stay; the outputs are compared in units of the keys."""
    B, Nc, q_pos0, m = 2, 300, 1300, 4
    x, _ = inputs(lcsa, B, 1, Nc, q_pos0 + 1, 11)
    f = 2.0 ** power
    x["ckv"] = (x["ckv"].float() * f).bfloat16()
    x["kv"] = (x["kv"].float() * f).bfloat16()
    x["q"] = (x["q"].float() / f).bfloat16()
    cache = lcsa.quantize_entries_fp4(x["ckv"], 64)
    out = np64(run(lcsa, x, cache, None, q_pos0, 0, m, 128))
    ref, _ = oracle(x, cache, None, q_pos0, 0, m, 128)
    assert np.abs(out.reshape(ref.shape) - ref).max() <= ATT_MAX * f
    assert lcsa.get_device_status() == 0


@pytest.mark.parametrize("Nc", [5, 70, 1000])
def test_very_negative_logits(lcsa, Nc):
    """Every logit far below zero (weights against zero would all vanish), the last tile partly filled."""
    B, m = 2, 4
    q_pos0 = 4 * Nc + 43
    x, _ = inputs(lcsa, B, 1, Nc, 40, 12)
    base = torch.randn(512, generator=torch.Generator().manual_seed(3)).to(DEV)
    base[448:] = 0                                     # rotation leaves the logits alone
    x["ckv"] = (x["ckv"].float() * 0.1 + 4 * base).bfloat16()
    x["kv"] = (x["kv"].float() * 0.1 + 4 * base).bfloat16()
    x["q"] = (x["q"].float() * 0.1 - 4 * base).bfloat16()
    cache = lcsa.quantize_entries_fp4(x["ckv"], 64)
    for sink in (False, True):
        out = np64(run(lcsa, x, cache, None, q_pos0, q_pos0 - 39, m, 40, sink))
        ref, _ = oracle(x, cache, None, q_pos0, q_pos0 - 39, m, 40, sink)
        assert np.isfinite(out).all()
        # logits near -360: a BF16 rounding of a product of that size is averaged over 512 dims; keys reach 16
        assert np.abs(out.reshape(ref.shape) - ref).max() <= 0.25
    assert lcsa.get_device_status() == 0


def test_growing_logits(lcsa):
    """Later tiles have ever larger logits: the reference of the exponent moves in every tile."""
    B, m, Nc = 2, 4, 1500
    q_pos0 = 4 * Nc + 1
    x, _ = inputs(lcsa, B, 1, Nc, 64, 13)
    u = torch.randn(64, 512, generator=torch.Generator().manual_seed(4)).to(DEV)
    u[:, 448:] = 0
    x["q"] = u.view(1, 1, 64, 512).expand(B, 1, -1, -1).bfloat16().contiguous()
    ramp = torch.linspace(0, 2, Nc, device=DEV)[None, :, None]
    x["ckv"] = (x["ckv"].float() * 0.5 + ramp * u.mean(0) * 64).bfloat16()
    cache = lcsa.quantize_entries_fp4(x["ckv"], 64)
    out, lse = run(lcsa, x, cache, None, q_pos0, q_pos0 - 63, m, 64, return_lse=True)
    ref, ref_lse = oracle(x, cache, None, q_pos0, q_pos0 - 63, m, 64)
    size = max(1.0, float(np.abs(expand(cache)).max()))
    assert np.abs(np64(out).reshape(ref.shape) - ref).max() <= ATT_MAX * size
    np.testing.assert_allclose(np64(lse).reshape(ref_lse.shape), ref_lse, atol=2e-2)


# ------------------------------------------------------------------ what masked rows hold
def poison(cache, b, rows):
    cache[1][b, rows] = 255                            # scale NaN
    cache[2][b, rows] = float("inf")


@pytest.mark.parametrize("Tq", [1, 3, 130])
def test_masked_rows_do_not_reach_outputs(lcsa, Tq):
    """Entries that are not selected or not visible yet, and raw rows outside of the windows, may hold anything."""
    B, Nc, q_pos0, m, W, k = 2, 500, 1600, 4, 128, 150
    x, cache = inputs(lcsa, B, Tq, Nc, W + Tq + 30, 14)
    kv_pos0 = q_pos0 - W + 1 - 7
    idx = selection(B, Tq, k, q_pos0, m, Nc, 15)
    clean_csa = run(lcsa, x, cache, idx, q_pos0, kv_pos0, m, W)
    clean_hca = run(lcsa, x, cache, None, q_pos0, kv_pos0, m, W)
    seen = torch.zeros(B, Nc, dtype=torch.bool, device=DEV)
    for b in range(B):
        seen[b, idx[b][idx[b] >= 0].long()] = True
    first_hidden = (q_pos0 + Tq - 1) // m
    dirty = [t.clone() for t in cache]
    for b in range(B):
        poison(dirty, b, ~seen[b])
    kv = x["kv"].clone()
    kv[:, :7] = float("nan")
    kv[:, W + Tq + 6:] = float("inf")
    x["kv"] = kv
    assert torch.equal(run(lcsa, x, tuple(dirty), idx, q_pos0, kv_pos0, m, W), clean_csa)
    dirty = [t.clone() for t in cache]
    for b in range(B):
        poison(dirty, b, torch.arange(Nc, device=DEV) >= first_hidden)
    assert torch.equal(run(lcsa, x, tuple(dirty), None, q_pos0, kv_pos0, m, W), clean_hca)
    assert lcsa.get_device_status() == 0


def test_nan_that_is_seen_reaches_the_output(lcsa):
    B, Nc, q_pos0, m = 2, 100, 420, 4
    x, cache = inputs(lcsa, B, 1, Nc, 128, 16)
    clean = run(lcsa, x, cache, None, q_pos0, q_pos0 - 127, m, 128)
    poison(cache, 1, torch.tensor([40], device=DEV))
    out = run(lcsa, x, cache, None, q_pos0, q_pos0 - 127, m, 128)
    assert torch.equal(out[0], clean[0])               # another sequence
    assert torch.isnan(out[1]).all()


def test_holes_in_a_selection(lcsa):
    """-1 anywhere in a row of the selection is no key; a row of nothing but -1 leaves the window and the sink."""
    B, Tq, Nc, q_pos0, m, k = 2, 3, 400, 1650, 4, 130
    x, cache = inputs(lcsa, B, Tq, Nc, 128 + Tq, 17)
    idx = selection(B, Tq, k, q_pos0, m, Nc, 18)
    idx[0, 0, ::3] = -1
    idx[1, 2] = -1
    idx[0, 1, 5] = idx[0, 1, 6]                        # the same entry twice counts twice
    kv_pos0 = q_pos0 - 127
    out = np64(run(lcsa, x, cache, idx, q_pos0, kv_pos0, m, 128))
    d, q, kv, s = expand(cache), np64(x["q"]), np64(x["kv"]), np64(x["sink"])
    for b in range(B):
        for i in range(Tq):
            sel = idx[b, i].cpu().numpy()
            ref, _ = O.attend_one(q[b, i], q_pos0 + i, sel[sel >= 0], d[b], m, kv[b], kv_pos0, 128, s, 64)
            assert np.abs(out[b, i] - ref).max() <= ATT_MAX


# ------------------------------------------------------------------ large calls
@pytest.mark.parametrize("sparse", [True, False])
@pytest.mark.parametrize("q_pos0", [0, 60, 5000])
def test_read_back_path_equals_attention_over_the_entries_read_back(lcsa, sparse, q_pos0):
    """Calls of many rows attend over the cache read back: bit for bit the BF16 call's results, except for rows whose
    window is not whole (their own kernel), which agree with it to rounding."""
    B, Tq, m, W, k = 2, 900, 4, 128, 600
    Nc = (q_pos0 + Tq) // m
    x, cache = inputs(lcsa, B, Tq, Nc, q_pos0 + Tq, 19)
    idx = selection(B, Tq, k, q_pos0, m, Nc, 20) if sparse else None
    assert lcsa.attn_fp4_workspace_bytes(x["q"], cache, idx, x["kv"], m, W, q_pos0=q_pos0) > 0
    out, lse = run(lcsa, x, cache, idx, q_pos0, 0, m, W, return_lse=True)
    entries = lcsa.dequantize_entries_fp4(cache)
    args = (q_pos0, 0, m, W)
    if sparse:
        ref, ref_lse = lcsa.csa_sparse_attn(x["q"], entries, idx, x["kv"], x["sink"], *args, return_lse=True)
    else:
        ref, ref_lse = lcsa.hca_dense_attn(x["q"], entries, x["kv"], x["sink"], *args, return_lse=True)
    part = max(0, W - 1 - q_pos0)
    assert torch.equal(out[:, part:], ref[:, part:]) and torch.equal(lse[:, part:], ref_lse[:, part:])
    # both are within ATT_MAX of the exact value; keys reach about 5 here (the first rows are means of few keys)
    assert (out[:, :part] - ref[:, :part]).abs().max() <= 2 * 5 * ATT_MAX if part else True
    rows = [(0, 0), (1, 3), (0, 127), (1, 899)]
    want, _ = oracle(x, cache, idx, q_pos0, 0, m, W, rows=rows)
    got = np64(out)[[r[0] for r in rows], [r[1] for r in rows]]
    assert np.abs(got - want).max() <= 5 * ATT_MAX


@pytest.mark.parametrize("W", [128, 100])
def test_large_calls_mask_what_a_cache_holds_beyond_its_entries(lcsa, W):
    """Rows of the cache and of the raw buffer past the call's last position hold NaN, from position 0 on."""
    B, Tq, m, Nc = 3, 700, 4, 400
    x, cache = inputs(lcsa, B, Tq, Nc, Tq + 90, 21)
    clean = run(lcsa, x, cache, None, 0, 0, m, W)
    cache[1][:, Tq // m:] = 255
    x["kv"] = x["kv"].clone()
    x["kv"][:, Tq:] = float("nan")
    out = run(lcsa, x, cache, None, 0, 0, m, W)
    assert torch.equal(out, clean)


# ------------------------------------------------------------------ how it is called
def test_tensors_at_16_byte_alignment(lcsa):
    B, Tq, Nc, q_pos0, m = 2, 2, 200, 900, 4
    x, cache = inputs(lcsa, B, Tq, Nc, 128 + Tq, 22)
    want = run(lcsa, x, cache, None, q_pos0, q_pos0 - 127, m, 128)

    def shifted(t):
        step = 16 // t.element_size()
        buf = torch.empty(t.numel() + step, dtype=t.dtype, device=DEV)
        s = buf[step:].view(t.shape)
        s.copy_(t)
        assert s.data_ptr() % 32 == 16
        return s

    y = {n: shifted(t) if n != "sink" else t for n, t in x.items()}
    c2 = tuple(shifted(t) for t in cache)
    out = shifted(torch.zeros_like(want))
    assert run(lcsa, y, c2, None, q_pos0, q_pos0 - 127, m, 128, out=out) is out
    assert torch.equal(out, want)
    c3 = tuple(shifted(torch.zeros_like(t)) for t in cache)
    lcsa.quantize_entries_fp4(shifted(x["ckv"]), 64, cache=c3)
    assert all(torch.equal(a, b) for a, b in zip(c3, cache))
    back = shifted(torch.zeros(B, Nc, 512, dtype=torch.bfloat16, device=DEV))
    assert torch.equal(lcsa.dequantize_entries_fp4(c3, out=back), lcsa.dequantize_entries_fp4(cache))


def test_streams_and_repeated_calls(lcsa):
    """Two streams at once, and the same call again: the same bits."""
    B, Tq, Nc, q_pos0, m = 4, 1, 3000, 12005, 4
    x, cache = inputs(lcsa, B, Tq, Nc, 128, 23)
    idx = selection(B, Tq, 1000, q_pos0, m, Nc, 24)
    a = run(lcsa, x, cache, idx, q_pos0, q_pos0 - 127, m, 128)
    h = run(lcsa, x, cache, None, q_pos0, q_pos0 - 127, m, 128)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for rep in range(6):
        for s, sel in zip(streams, (idx, None)):
            with torch.cuda.stream(s):
                got.append((sel is not None, run(lcsa, x, cache, sel, q_pos0, q_pos0 - 127, m, 128)))
    torch.cuda.synchronize()
    for is_csa, out in got:
        assert torch.equal(out, a if is_csa else h)
    assert lcsa.get_device_status() == 0


def test_captured_graphs_replay_on_new_inputs(lcsa):
    """A decode step captured twice (append, then attend), replayed in turn with other contents."""
    B, Nc, m, W = 3, 600, 4, 128
    q_pos0 = 4 * Nc
    x, cache = inputs(lcsa, B, 1, Nc, W, 25)
    big, bcache = inputs(lcsa, B, 700, Nc, 3200, 26)
    new = x["ckv"][:, :1].contiguous()
    graphs, outs = [], []
    for y, c, p0, k0 in ((x, cache, q_pos0, q_pos0 - W + 1), (big, bcache, 2400, 0)):
        run(lcsa, y, c, None, p0, k0, m, W)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            lcsa.quantize_entries_fp4(new, 64, cache=c, row0=Nc - 1)
            outs.append(run(lcsa, y, c, None, p0, k0, m, W))
        graphs.append(g)
    for seed in (31, 32):
        fresh = torch.randn(x["q"].shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).bfloat16()
        x["q"].copy_(fresh)
        new.copy_(torch.randn(new.shape, generator=torch.Generator(device=DEV).manual_seed(seed + 50), device=DEV))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], run(lcsa, x, cache, None, q_pos0, q_pos0 - W + 1, m, W))
        assert torch.equal(outs[1], run(lcsa, big, bcache, None, 2400, 0, m, W))
    del graphs


def test_sizes_of_nothing_and_one(lcsa):
    B, m = 2, 128
    x, cache = inputs(lcsa, B, 1, 1, 1, 27)
    # no entry visible, a window of the row itself, no sink: the row comes back (rotated there and back)
    out = np64(run(lcsa, x, cache, None, 0, 0, m, 1, sink=False))
    assert np.abs(out - np64(x["kv"])[:, :, None]).max() <= 2.0 ** -7 * float(x["kv"].abs().max())
    empty = tuple(t[:, :0].contiguous() for t in cache)
    assert torch.equal(run(lcsa, x, empty, None, 0, 0, m, 1, sink=False),
                       run(lcsa, x, cache, None, 0, 0, m, 1, sink=False))
    none = {**x, "kv": x["kv"][:, :0].contiguous()}
    assert (run(lcsa, none, empty, None, 5, 0, m, 0, sink=False) == 0).all()
    q0 = {**x, "q": x["q"][:, :0].contiguous()}
    assert run(lcsa, q0, cache, None, 5, 0, m, 1).shape == (B, 0, 64, 512)
    assert lcsa.get_device_status() == 0


FIRST_CALL = """
import sys, torch
import long_context_compressed_softmax_b200 as lcsa
g = torch.Generator(device="cuda").manual_seed(5)
B, Nc, m, W, p0 = int(sys.argv[1]), 3000, 4, 128, 12005
t = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
q, kv = t(B, 1, 64, 512), t(B, W, 512)
cache = lcsa.quantize_entries_fp4(t(B, Nc, 512), 64)
idx = torch.arange(1024, dtype=torch.int32, device="cuda").expand(B, 1, -1).contiguous()
call = lambda: lcsa.csa_sparse_attn_fp4(q, cache, idx, kv, None, p0, p0 - W + 1, m, W)
if sys.argv[2] == "captured":
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = call()
    graph.replay()
else:
    out = call()
torch.cuda.synchronize()
ref = lcsa.csa_sparse_attn(q, lcsa.dequantize_entries_fp4(cache), idx, kv, None, p0, p0 - W + 1, m, W)
err = (out.float() - ref.float()).abs().max().item()
assert err <= 2 * %r, err
assert lcsa.get_device_status() == 0
print("done")
"""


@pytest.mark.parametrize("how", ["eager", "captured"])
def test_split_call_as_the_first_of_a_process(lcsa, how):
    """A split call sets the kernel up by itself, in a capture too."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL % ATT_MAX, "1", how], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["done"]


@pytest.mark.parametrize("sink", [False, True])
def test_split_call_with_empty_splits(lcsa, sink):
    """A selection whose keys all lie in one split, or of holes alone: parts without keys count for nothing."""
    B, Nc, q_pos0, m, k = 1, 3000, 12005, 4, 1024
    x, cache = inputs(lcsa, B, 1, Nc, 1, 47)
    for live in (0, 1, 3):
        idx = torch.full((B, 1, k), -1, dtype=torch.int32, device=DEV)
        idx[..., k - live:] = torch.arange(live, dtype=torch.int32, device=DEV) * 7
        out, lse = run(lcsa, x, cache, idx, q_pos0, q_pos0, m, 0, sink, return_lse=True)
        ref, _ = oracle(x, cache, idx, q_pos0, q_pos0, m, 0, sink)
        assert np.abs(np64(out).reshape(ref.shape) - ref).max() <= 3e-2     # of one key up to 5: 2 * 2^-9 * 5
        if live == 0 and not sink:
            assert (out == 0).all() and (lse == float("-inf")).all()
        elif live == 0:
            assert torch.allclose(lse[0, 0], x["sink"], rtol=1e-5, atol=1e-5)
    assert lcsa.get_device_status() == 0


# ------------------------------------------------------------------ together
def test_decode_step_through_the_calls_of_a_server(lcsa):
    """Raw rows -> entries -> FP4 cache (prefill, then one appended in decode) -> top-k -> attention, against the same
    step over BF16 entries read back and over the oracle."""
    B, T, m, W, k, D = 2, 1027, 4, 128, 64, 512
    inp = gen.make_compress_inputs(B, T + 1, D, "bf16", seed=41, device=DEV, kv_scale=1.0)
    raw, gate = inp["kv"], inp["gate"]
    cache = lcsa.empty_fp4_cache(B, 300)
    entries = lcsa.csa_compress(raw[:, :T].contiguous(), gate[:, :T].contiguous(), m)       # 256 entries
    n = entries.shape[1]
    lcsa.quantize_entries_fp4(entries, 64, cache=cache)
    last = lcsa.csa_compress(raw, gate, m)[:, n:].contiguous()                             # the entry that T + 1 completes
    assert last.shape[1] == 1
    lcsa.quantize_entries_fp4(last, 64, cache=cache, row0=n)
    t = T                                                                                   # position of the new token
    iq = gen.make_indexer_inputs(B, 1, n + 1, dtype="bf16", seed=42, device=DEV)
    idx = lcsa.indexer_topk(iq["q_idx"], iq["w"], iq["k_idx"], t, m, k)
    x = gen.make_attn_inputs(B, 1, 64, D, 1, 1, "bf16", seed=43, device=DEV, unit_scale=True)
    kv = raw[:, t - W + 1:].contiguous()
    out = lcsa.csa_sparse_attn_fp4(x["q"], cache, idx, kv, x["sink"], t, t - W + 1, m, W)
    ref = lcsa.csa_sparse_attn(x["q"], lcsa.dequantize_entries_fp4(cache), idx, kv, x["sink"], t, t - W + 1, m, W)
    assert (out - ref).abs().max() <= 2 * ATT_MAX
    want, _ = O.csa_sparse_attn(np64(x["q"]), expand(cache), idx.cpu().numpy(), np64(kv), t, t - W + 1, m, W,
                                np64(x["sink"]), 64)
    assert np.abs(np64(out).reshape(want.shape) - want).max() <= ATT_MAX
    assert lcsa.get_device_status() == 0
