"""Which way a call over the FP4 entry cache goes (seen by the workspace that it asks for) and what it refuses, without
a GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lcsa():
    from conftest import build_library
    return build_library()


def args(lcsa, **kw):
    return lcsa.AttnArgs(**{**dict(q=0x10000, out=0x20000, kv=0x30000, idx=0x40000, B=1, Tq=2048, H=64, D=512, R=64, Nc=8192,
                                   k=2048, Tkv=2048 + 127, m=4, W=128, q_pos0=30720, kv_pos0=30720 - 127,
                                   dtype=lcsa.LCSA_BF16, out_dtype=lcsa.LCSA_BF16), **kw})


def workspace(lcsa, sparse, **kw):
    return lcsa.lib.lcsa_attn_fp4_workspace(ctypes.byref(args(lcsa, **kw)), sparse)


def test_more_selected_entries_than_the_read_back_kernel_stages(lcsa):
    """Beyond 2048 selected entries that kernel splits every row and writes 128 KB of partial outputs a split: a call of
    the tile kernel needs no memory."""
    assert workspace(lcsa, 1) > 0
    for k in (2049, 4096, 8192):
        assert workspace(lcsa, 1, k=k) == 0
    assert workspace(lcsa, 0, m=128, Nc=1024, q_pos0=129024, kv_pos0=129024 - 127, k=0) > 0


def test_the_read_back_counts_what_is_visible(lcsa):
    """The first rows of a prefill into a cache allocated for a long context."""
    first = dict(q_pos0=0, kv_pos0=0, Tkv=2048)
    assert workspace(lcsa, 1, **first, Nc=512) > 0
    assert workspace(lcsa, 1, **first, Nc=262144) == 0         # 262,144 entries for 511 that can be selected
    # dense calls read back no more than the last tile that a row sees
    small, large = workspace(lcsa, 0, **first, Nc=512), workspace(lcsa, 0, **first, Nc=262144)
    assert 512 * 1024 <= small == large


def test_the_read_back_counts_the_rows_that_it_serves(lcsa):
    """Rows whose window begins before the raw rows do are the tile kernel's in any case."""
    short = dict(B=32, Nc=50, k=512, q_pos0=0, kv_pos0=0)
    assert workspace(lcsa, 1, **short, Tq=150, Tkv=150) == 0               # 32 prompts of 150 tokens: 23 rows of each are left
    assert workspace(lcsa, 0, **short, Tq=150, Tkv=150) == 0
    assert workspace(lcsa, 1, **{**short, "Nc": 1000}, Tq=1000, Tkv=1000) > 0
    # the same rows with their windows in kv
    whole = dict(B=32, Nc=1050, k=512, q_pos0=4000, kv_pos0=4000 - 127, Tq=150, Tkv=150 + 127)
    assert workspace(lcsa, 1, **whole) > 0
    assert workspace(lcsa, 1, **{**whole, "kv_pos0": 4200, "Tkv": 100}) == 0    # no row's window is whole


def test_attention_over_entries_beyond_64_bits_is_refused(lcsa):
    L, big = lcsa.lib, 2 ** 31 - 1
    e = lcsa.Fp4Entries(0x50000, 0x60000, 0x70000)
    for a in (args(lcsa, B=big, Nc=big, D=1504, R=64, Tq=1, H=1, Tkv=0, k=1),
              args(lcsa, B=big, Tq=big, H=big, D=64, R=32, Nc=1, Tkv=0, k=1),
              args(lcsa, B=big, Tq=1, H=1, D=1504, R=64, Nc=1, Tkv=big, k=1),
              args(lcsa, B=big, Tq=big, H=1, D=64, R=32, Nc=1, Tkv=0, k=big)):
        for f in (L.lcsa_csa_sparse_attn_fp4, L.lcsa_hca_dense_attn_fp4):
            if f is L.lcsa_hca_dense_attn_fp4 and a.k == big:
                continue
            assert f(ctypes.byref(a), ctypes.byref(e), ctypes.c_void_p(0x100000), 1 << 62, None) == 1


def test_a_strided_workspace_is_refused(lcsa):
    """Its size in elements is not the bytes behind its first one."""
    c = (torch.zeros(1, 8, 224, dtype=torch.uint8), torch.zeros(1, 8, 16, dtype=torch.uint8),
         torch.zeros(1, 8, 64, dtype=torch.bfloat16))
    q, kv = torch.zeros(1, 1, 64, 512, dtype=torch.bfloat16), torch.zeros(1, 4, 512, dtype=torch.bfloat16)
    for ws in (torch.zeros(64, dtype=torch.uint8)[::2], torch.zeros(1, dtype=torch.uint8).expand(4096)):
        with pytest.raises(ValueError, match="contiguous"):
            lcsa.hca_dense_attn_fp4(q, c, kv, None, 0, 0, workspace=ws)
        with pytest.raises(ValueError, match="contiguous"):
            lcsa.csa_sparse_attn_fp4(q, c, torch.zeros(1, 1, 1, dtype=torch.int32), kv, None, 0, 0, workspace=ws)
