"""FP4 entry cache without a GPU: pins of the oracle's format and the argument
checks of the calls (all before any device work)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import lcsa_oracle as O


@pytest.fixture(scope="module")
def lcsa():
    from conftest import build_library
    return build_library()


# ------------------------------------------------------------------ format pins
def test_fp4_entry_format():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((7, 512)) * np.exp2(rng.integers(-20, 20, (7, 1)))
    x[0, :32] = 0.0
    x[1, 32:64] = np.nan
    codes, scales, rope = O.quantize_entries_fp4(x, 64)
    assert codes.shape == (7, 224) and scales.shape == (7, 16) and rope.shape == (7, 64)
    assert (scales[:, 14:] == 0).all()                       # padding
    assert scales[0, 0] == 0 and scales[1, 1] == 255
    d = O.dequantize_entries_fp4(codes, scales, rope)
    np.testing.assert_array_equal(rope, torch.tensor(x[:, 448:]).to(torch.bfloat16).double().numpy())
    assert np.isnan(d[1, 32:64]).all()
    ok = np.isfinite(d)
    # nearest E2M1 number: off by at most half the widest spacing (between 4 and 6) of the block's scale,
    # and by up to 2 (6 to 8) where a value above 6 saturates
    step = np.exp2(np.repeat(scales[:, :14].astype(float) - 127, 32, axis=1))
    assert (np.abs(d[:, :448] - x[:, :448]) <= 2.0 * step)[ok[:, :448]].all()
    # every value the cache stands for is a BF16 number
    b = torch.tensor(d[ok]).to(torch.bfloat16).double().numpy()
    np.testing.assert_array_equal(b, d[ok])


def test_fp4_entry_roundtrip_of_representable_entries():
    rng = np.random.default_rng(6)
    codes = rng.integers(0, 256, (5, 224)).astype(np.uint8)
    codes[:, ::16] |= 0x07                                   # a magnitude 6 in every block keeps its scale
    codes = np.where((codes & 0x0F) == 0x08, codes & 0xF0, codes)        # no -0 codes
    codes = np.where((codes & 0xF0) == 0x80, codes & 0x0F, codes).astype(np.uint8)
    scales = np.zeros((5, 16), dtype=np.uint8)
    scales[:, :14] = rng.integers(0, 250, (5, 14))           # 2^-127 .. 2^122
    rope = torch.randn(5, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).double().numpy()
    d = O.dequantize_entries_fp4(codes, scales, rope)
    c2, s2, r2 = O.quantize_entries_fp4(d, 64)
    np.testing.assert_array_equal(c2, codes)
    np.testing.assert_array_equal(s2, scales)
    np.testing.assert_array_equal(r2, rope)
    np.testing.assert_array_equal(torch.tensor(d).to(torch.bfloat16).double().numpy(), d)


# ------------------------------------------------------------------ arguments
def test_fp4_scale_bytes(lcsa):
    assert lcsa.fp4_scale_bytes(512, 64) == 16
    assert lcsa.fp4_scale_bytes(64, 32) == 16
    assert lcsa.fp4_scale_bytes(640, 64) == 32               # 18 blocks
    assert lcsa.fp4_scale_bytes(512, 0) == 16
    for D, R in ((512, 60), (512, 512), (100, 64), (500, 64), (0, 0), (512, -8), (64, 36)):
        assert lcsa.fp4_scale_bytes(D, R) == 0


def test_fp4_struct_layout(lcsa):
    assert ctypes.sizeof(lcsa.Fp4Entries) == 3 * ctypes.sizeof(ctypes.c_void_p)
    assert [lcsa.Fp4Entries.codes.offset, lcsa.Fp4Entries.scales.offset, lcsa.Fp4Entries.rope.offset] == [0, 8, 16]


def test_quantize_entries_fp4_checks_arguments(lcsa):
    L, bf = lcsa.lib, lcsa.LCSA_BF16
    E = lambda **kw: ctypes.byref(lcsa.Fp4Entries(**{"codes": 0x1000, "scales": 0x2000, "rope": 0x3000, **kw}))
    call = lambda x=0x4000, B=1, n=4, D=512, R=64, dt=bf, e=None, rows=8, row0=0: L.lcsa_quantize_entries_fp4(
        ctypes.c_void_p(x), B, n, D, R, dt, e or E(), rows, row0, None)
    assert call(D=500) == 1 and call(R=60) == 1 and call(D=64) == 1 and call(dt=7) == 1
    assert call(row0=-1) == 1 and call(row0=5) == 1 and call(n=9) == 1 and call(n=-1) == 1 and call(B=-1) == 1
    assert call(row0=9, n=0) == 1 and call(row0=2 ** 62, n=2 ** 62, rows=2 ** 62) == 1
    assert call(x=0) == 1 and call(x=0x4002) == 1
    assert call(e=E(codes=0)) == 1 and call(e=E(scales=0x2008)) == 1 and call(e=E(rope=0)) == 1
    assert L.lcsa_quantize_entries_fp4(ctypes.c_void_p(0x4000), 1, 4, 512, 64, bf, None, 8, 0, None) == 1
    assert call(n=0) == 0 and call(B=0, x=0) == 0
    if not torch.cuda.is_available():
        assert call() == 4 and call(R=0, D=64, e=E(rope=0)) == 4          # valid, but no device: no CPU path


def test_dequantize_entries_fp4_checks_arguments(lcsa):
    L, bf = lcsa.lib, lcsa.LCSA_BF16
    E = lambda **kw: ctypes.byref(lcsa.Fp4Entries(**{"codes": 0x1000, "scales": 0x2000, "rope": 0x3000, **kw}))
    call = lambda e=None, B=1, rows=8, D=512, R=64, idx=None, n=8, out=0x4000, dt=bf: L.lcsa_dequantize_entries_fp4(
        e or E(), B, rows, D, R, ctypes.c_void_p(idx), n, ctypes.c_void_p(out), dt, None)
    assert call(R=4) == 1 and call(D=65) == 1 and call(dt=3) == 1 and call(n=-1) == 1 and call(rows=-1) == 1
    assert call(n=9) == 1                                    # all rows: no more than there are
    assert call(out=0) == 1 and call(out=0x4008) == 1 and call(idx=0x5002) == 1
    assert call(e=E(codes=0x1004)) == 1 and call(e=E(scales=0)) == 1
    assert call(n=0, out=0) == 0
    if not torch.cuda.is_available():
        assert call() == 4 and call(idx=0x5004, n=100) == 4


def test_entries_beyond_64_bits_are_refused(lcsa):
    L, bf, e = lcsa.lib, lcsa.LCSA_BF16, lcsa.Fp4Entries(0x1000, 0x2000, 0x3000)
    huge = 2 ** 62
    assert L.lcsa_quantize_entries_fp4(ctypes.c_void_p(0x4000), 4, huge, 512, 64, bf, ctypes.byref(e), huge, 0, None) == 1
    assert L.lcsa_dequantize_entries_fp4(ctypes.byref(e), 4, huge, 512, 64, None, huge, ctypes.c_void_p(0x4000), bf, None) == 1
    assert L.lcsa_dequantize_entries_fp4(ctypes.byref(e), 4, 8, 512, 64, ctypes.c_void_p(0x5000), huge, ctypes.c_void_p(0x4000), bf,
                                         None) == 1


def test_attn_fp4_checks_arguments(lcsa):
    L = lcsa.lib
    A = lambda **kw: lcsa.AttnArgs(**{**dict(q=0x10000, out=0x20000, kv=0x30000, idx=0x40000, B=1, Tq=1, H=64, D=512,
                                             R=64, Nc=8, k=8, Tkv=8, m=4, W=8, dtype=lcsa.LCSA_BF16,
                                             out_dtype=lcsa.LCSA_BF16), **kw})
    E = lambda **kw: lcsa.Fp4Entries(**{"codes": 0x50000, "scales": 0x60000, "rope": 0x70000, **kw})
    ws = ctypes.c_void_p(0x100000)

    def both(a, e):
        r = [f(ctypes.byref(a), ctypes.byref(e) if e is not None else None, ws, 1 << 40, None)
             for f in (L.lcsa_csa_sparse_attn_fp4, L.lcsa_hca_dense_attn_fp4)]
        assert r[0] == r[1]
        return r[0]

    assert both(A(), None) == 1                              # no cache
    for bad in (dict(codes=0x50008), dict(scales=0x60004), dict(rope=0), dict(codes=0)):
        assert both(A(), E(**bad)) == 1, bad
    for bad in (dict(R=60), dict(D=500), dict(q=0), dict(out=0x20008), dict(kv=0), dict(m=0), dict(W=-1),
                dict(q_pos0=-1), dict(lse=0x80004), dict(sink=0x80002), dict(dtype=9)):
        assert both(A(**bad), E()) == 1, bad
    assert L.lcsa_csa_sparse_attn_fp4(ctypes.byref(A(k=0)), ctypes.byref(E()), ws, 1 << 40, None) == 1
    assert both(A(B=0), E()) == 0 and both(A(Tq=0), None) == 0
    # a shape of the CUDA-core kernels needs room for the entries read back
    small = A(H=4, D=64, R=32, Nc=16)
    assert L.lcsa_attn_fp4_workspace(ctypes.byref(small), 0) >= 16 * 64 * 2
    if not torch.cuda.is_available():
        assert both(A(), E()) == 4 and both(small, E()) == 4              # valid, but no device: no CPU path


def test_fp4_binding_refuses_what_does_not_fit(lcsa):
    c = torch.zeros(2, 8, 224, dtype=torch.uint8)
    s = torch.zeros(2, 8, 16, dtype=torch.uint8)
    r = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    q = torch.zeros(2, 1, 64, 512, dtype=torch.bfloat16)
    kv = torch.zeros(2, 4, 512, dtype=torch.bfloat16)
    for bad in ((c, s[:, :4], r), (c, s[..., :14].contiguous(), r), (c, s, r[..., :32].contiguous()), (c[0], s[0], r[0])):
        with pytest.raises(ValueError):
            lcsa.dequantize_entries_fp4(bad)
    with pytest.raises(TypeError):
        lcsa.dequantize_entries_fp4((c, s, r.float()))
    with pytest.raises(ValueError):                          # on the CPU
        lcsa.dequantize_entries_fp4((c, s, r))
    with pytest.raises(ValueError):                          # another number of sequences
        lcsa.hca_dense_attn_fp4(q[:1], (c, s, r), kv[:1], None, 0, 0)
    with pytest.raises(ValueError):                          # another entry shape
        lcsa.hca_dense_attn_fp4(q, (c, s, r), kv, None, 0, 0, R=32)
    with pytest.raises(ValueError):
        lcsa.empty_fp4_cache(1, 4, 500, 64, "cpu")
    with pytest.raises(ValueError):                          # non-contiguous rows
        lcsa.quantize_entries_fp4(torch.zeros(4, 8, 512).transpose(0, 1))
