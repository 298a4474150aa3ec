"""Sizes that the C calls' 32-bit counts cannot hold are refused by the wrappers:
ctypes would cut them (2**32 rows would be none, and the call do nothing)."""
import pytest
import torch

import huffman_decode_amd as hd
from huffman_decode_amd import step

BF16, I32 = torch.bfloat16, torch.int32
MANY = 1 << 32


class NoLibrary:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was called")


class NoCache:
    """What the wrappers read of a cache."""
    device, dim, kv_heads, _ref = -1, 64, 1, None


@pytest.fixture
def cpu(monkeypatch):
    """CPU tensors pass for the GPU's, and nothing is called."""
    monkeypatch.setattr(step, "_device", lambda name, t: t.get_device())
    monkeypatch.setattr(step, "_lib", NoLibrary)


def _rows(*shape, dtype=torch.float32):
    """`shape` over one row's memory."""
    return torch.zeros(1, *shape[1:], dtype=dtype).expand(*shape)


def _refused(fn, *args, **kw):
    with pytest.raises(ValueError, match=r"below 2\*\*3[12]"):
        fn(*args, **kw)


@pytest.mark.parametrize("rows", [MANY, MANY + 3])
def test_rows(cpu, rows):
    x, out = _rows(rows, 8), _rows(rows, 8, dtype=BF16)
    _refused(step.df11_add_rms_norm, x, torch.ones(8), out, 1e-5)
    _refused(step.df11_silu_mul, x, x, out)
    _refused(step.df11_logits, x, x)


def test_tokens_heads_and_positions(cpu):
    i = torch.zeros(1, dtype=I32)
    q, o, t = torch.zeros(1, 2, 64), torch.zeros(1, 2, 64, dtype=BF16), torch.zeros(1, 32)
    kv = torch.zeros(1, 1, 64)
    many, many_out = _rows(MANY, 2, 64), _rows(MANY, 2, 64, dtype=BF16)
    wide, wide_out = (torch.zeros(1, 1, 64, dtype=d).expand(1, MANY, 64) for d in (torch.float32, BF16))
    _refused(step.df11_rope_append, NoCache, many, kv, kv, t, t, i, i, many_out)
    _refused(step.df11_rope_append, NoCache, wide, kv, kv, t, t, i, i, wide_out)
    _refused(step.df11_rope_append, NoCache, q, kv, kv, _rows(MANY, 32), _rows(MANY, 32), i, i, o)
    _refused(step.df11_attention, NoCache, many_out, i, i, i[None], many_out, 1, 1)
    _refused(step.df11_attention, NoCache, wide_out, i, i, i[None], wide_out, 1, 1)


def test_plain_numbers(cpu):
    for n in (MANY + 1, -1):
        for at in range(5):
            sizes = [1, 2, 1, 1, 5000]
            sizes[at] = n
            _refused(step.df11_attention_workspace_bytes, NoCache, *sizes)


def test_block_bytes():
    assert hd.kv_block_bytes(MANY + 16, 64) == 0 and hd.kv_block_bytes(16, MANY + 64) == 0
    assert hd.kv_block_bytes(-(MANY - 16), 64) == 0
    assert hd.kv_block_bytes(16, 64) == 1088


def test_attention_launches_that_64_bits_cannot_count():
    """Sequences x key heads x row blocks past 2^64: refused, not taken for the
    few that are left of the product."""
    import ctypes
    kv_heads, block = 1 << 15, 1088
    cache = step.KvCacheDesc(0x10000, kv_heads * block, kv_heads * block, block, 1, kv_heads, 64, 16, None)
    ref = ctypes.byref(cache)
    lib = step._lib()
    # 2^31 sequences, 2^15 key heads, 2^18 blocks of 128 rows
    assert lib.df11_attention_workspace_bytes(ref, 4, kv_heads, 1 << 31, 1 << 25, 5000) == 0
    a = 0x10000
    args = (ref, a, kv_heads * 64, 64, 4, kv_heads, a, a, 1 << 31, a, 313, 313, 1 << 25, 5000, 0.1, 1, 0, a,
            kv_heads * 64, 64, None, a, 1 << 60, None)
    assert lib.df11_attention(*args) == -1


def test_outputs_that_repeat_a_row_are_refused():
    """Two tokens' results in one place: whichever came last would be left."""
    import ctypes
    cache = step.KvCacheDesc(0x10000, 4 * 2 * 1088, 2 * 1088, 1088, 4, 2, 64, 16, None)
    ref, lib, a = ctypes.byref(cache), step._lib(), 0x10000
    for out_stride in (0, 56):
        assert lib.df11_attention(ref, a, 256, 64, 5, 4, a, a, 2, a, 3, 3, 4, 48, 0.1, 1, 0, a, out_stride, 64,
                                  None, None, 0, None) == -1
    for k_stride, v_stride in ((0, 128), (128, 0), (63, 128)):
        assert lib.df11_kv_read(ref, a, a, k_stride, 64, a, v_stride, 64, 3, None) == -1


def test_updates_in_place_keep_the_rows_where_they_are():
    """One array as input and output, under two strides or types: rows would be
    read after others were written over them."""
    lib, a = step._lib(), 0x10000

    def norm(rows, residual, residual_out, stride, out_stride):
        return lib.df11_add_rms_norm(a, 1, 64, residual, residual_out, 0, stride, out_stride, a, 0, 1e-5, a, 0,
                                     64, None, rows, 64, None)

    def logits(rows, kind, stride, out_stride):
        none = [None, 0, 0] + [None] * 7 + [0, 0, None, 0]
        return lib.df11_logits(a, kind, stride, a, out_stride, *none, rows, 100, None)
    assert norm(3, a, a, 64, 72) == -1
    assert logits(3, 1, 100, 104) == -1 and logits(3, 0, 100, 100) == -1 and logits(1, 0, 100, 100) == -1


@pytest.mark.parametrize("dim,whole", [(64, 1792), (128, 1536), (256, 1280)])
@pytest.mark.parametrize("batch", [1, 8])
def test_a_sequence_is_cut_where_that_was_measured_faster(dim, whole, batch):
    """Single tokens over up to `whole` tokens: one chunk and no workspace."""
    import ctypes
    block = step.kv_block_bytes(64, dim)
    cache = step.KvCacheDesc(0x10000, 64 * 8 * block, 8 * block, block, 64, 8, dim, 64, None)
    lib, ref = step._lib(), ctypes.byref(cache)
    for kv in (1, 1031, 1281, whole - 1, whole):
        if kv <= whole:
            assert lib.df11_attention_workspace_bytes(ref, batch, 32, batch, 1, kv) == 0, kv
    assert lib.df11_attention_workspace_bytes(ref, batch, 32, batch, 1, whole + 1) == 2 * batch * 32 * (dim + 2) * 4
