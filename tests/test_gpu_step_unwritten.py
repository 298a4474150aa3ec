"""GPU tests of df11_attention over a cache whose unused slots hold any bytes:
pages are handed out as memory gave them, and what no query sees does not
matter.  Scale bytes above 252 make infinities or NaN of 4-bit codes; the
zero weight of a hidden token does not hide those by itself."""
import numpy as np
import pytest
import torch

import step_reference as ref
from test_gpu_step_attention import Case, _go

pytestmark = pytest.mark.gpu

REAL = ref.Pages


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Random(REAL):
    """Pages of random bytes, a third of the scales among 250 .. 255."""

    def __init__(self, n_pages, kv_heads, page_tokens, dim, fill=0):
        super().__init__(n_pages, kv_heads, page_tokens, dim)
        rng = np.random.default_rng(5)
        self.blocks[...] = rng.integers(0, 256, self.blocks.shape)
        scales = self.blocks[..., page_tokens * dim:]
        high = rng.integers(250, 256, scales.shape).astype(np.uint8)
        scales[...] = np.where(rng.random(scales.shape) < 0.3, high, scales)


def _filled(byte):
    return lambda n_pages, kv_heads, page, dim, fill=0: REAL(n_pages, kv_heads, page, dim, byte)


@pytest.mark.parametrize("queries", [1, 40])   # few rows to a key head, and many
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("held", [0xFC, 0xFD, 0xFE, 0x7F, "random"])
def test_unused_slots_may_hold_anything(held, dim, page, queries, monkeypatch):
    monkeypatch.setattr(ref, "Pages", Random if held == "random" else _filled(held))
    c = Case([70, 41, 100, 129], [queries] * 4, 4, 2, dim, page, seed=31)
    out, lse = _go(c)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    _go(c, window=30)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("byte", [253, 254])
@pytest.mark.parametrize("queries", [6, 60])
def test_tokens_that_some_queries_see(queries, byte, dim):
    """A value scale that append never writes, at a token in the queries' midst:
    those before it are as they would be without it."""
    c = Case([200], [queries], 4, 2, dim, 16, seed=32)
    out, lse = _go(c)
    at = 200 - queries // 2     # queries from queries / 2 on see it
    slot, n, m = c.seq[0][at], 16 * dim // 2, 16 * dim // 32
    c.host.blocks[slot // 16, :, 2 * n + m + slot % 16] = byte
    c.host.blocks[slot // 16, :, n + slot % 16] = 0x77          # two codes of 6
    got, got_lse = c.run()
    first = queries - queries // 2
    assert torch.isfinite(got[:first].float()).all()
    assert torch.equal(got[:first], out[:first]) and torch.equal(got_lse, lse)
