"""GPU tests of df11_attention with more than 64 rows to a key head (prompts),
at pages that hold a whole tile of 64 tokens and at smaller ones: windows, ragged
lengths, hidden tokens that hold NaN, pages out of range, infinite queries.

The cases, the 64-bit form and the bounds are those of
test_gpu_step_attention.py."""
import numpy as np
import pytest
import torch

import huffman_decode_amd as hd

import step_reference as ref
from test_gpu_step_attention import Case, _go

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 40, 100000])
@pytest.mark.parametrize("page", [64, 128, 256])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_pages_of_a_tile_and_more(dim, page, window, causal):
    """Whole prompts, later chunks, more queries than tokens, none at all, and
    sequences that end inside a page."""
    _go(Case([70, 130, 5, 0, 33, 300], [70, 20, 9, 3, 0, 100], 4, 2, dim, page, seed=21), causal=causal,
        window=window)


@pytest.mark.parametrize("heads,kv_heads,q", [(4, 4, 150), (8, 1, 40), (6, 2, 300), (48, 1, 7), (5, 1, 70)])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_over_several_workgroups(dim, page, heads, kv_heads, q):
    _go(Case([q + 37, q], [q, q - 3], heads, kv_heads, dim, page, seed=22))


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_split_prompts(dim, page):
    """Few prompts over many tokens: chunks of tokens over workgroups, joined."""
    c = Case([1100, 700, 3], [40, 36, 3], 4, 2, dim, page, seed=23)
    need = hd.df11_attention_workspace_bytes(hd.KvCache(torch.from_numpy(c.host.blocks).cuda(), dim, page),
                                             len(c.q), 4, 3, 40, 1100)
    assert need > 0
    a, b = _go(c), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), "two runs differ"
    _go(c, window=300)
    _go(c, causal=False)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_hidden_tokens_do_not_count_whatever_they_hold(dim, page):
    """A NaN key or value of a token reaches exactly the queries that see it."""
    c = Case([140, 90], [140, 1], 2, 1, dim, page, seed=24)
    n, m = page * dim // 2, page * dim // 32
    s, last = c.seq[0], dim // 32 - 1

    def nan_at(slot, group, value):
        c.host.blocks[slot // page, 0, 2 * n + (m if value else 0) + group * page + slot % page] = 255
    nan_at(s[70], last, True)    # the last 32 channels of queries from 70 on are NaN
    nan_at(s[120], 0, False)     # queries from 120 on are NaN throughout
    out, lse = c.run()
    c.check(out, lse)
    got = out.float().cpu()
    assert torch.isfinite(got[:70]).all() and torch.isfinite(got[70:120, :, :dim - 32]).all()
    assert torch.isnan(got[70:120, :, dim - 32:]).all() and torch.isnan(got[120:140]).all()
    assert torch.isfinite(got[140]).all()
    out, lse = c.run(window=10)
    c.check(out, lse, window=10)
    got = out.float().cpu()
    assert torch.isnan(got[70:80, :, dim - 32:]).all() and torch.isfinite(got[80:120]).all()
    assert torch.isfinite(got[130:140]).all()


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_pages_out_of_range_are_hidden(dim, page):
    c = Case([150, 200], [40, 40], 4, 2, dim, page, seed=25)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.table[0, 70 // page], c.table[1, 0] = 1 << 20, -7
    out, lse = c.run(status=status)
    assert int(status.item()) > 0
    got = out.double().cpu().numpy()
    for b, at, page_at in ((0, 0, 70 // page), (1, 40, 0)):
        k, v = c.host.load(c.seq[b])
        t = np.arange(len(k))
        keep = t[t // page != page_at]
        for i in range(40):
            see = keep[keep <= len(k) - 40 + i]
            o, _, mass, reach = ref.attention(c.q[at + i:at + i + 1].double().numpy(), k[see], v[see], dim ** -0.5,
                                              False, 0)
            delta = (dim + 8) * 2.0 ** -23 * reach[..., None]
            bound = (2.0 ** -8 + 2 * delta + 2.0 ** -18) * mass + 2.0 ** -8 * np.abs(o)
            assert (np.abs(got[at + i] - o[0]) <= bound[0] * (1 + 1e-6)).all(), (b, i)


@pytest.mark.parametrize("queries", [3, 60])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_infinite_queries_stay_in_their_rows(value, page, queries):
    """Scores of both infinities and NaN: no softmax, so NaN, in that row only
    (few rows and many)."""
    c = Case([150], [queries], 4, 2, 128, page, seed=26)
    c.q[1, 1, 5] = value
    out, lse = c.run()
    with np.errstate(invalid="ignore"):
        c.check(out, lse)
    got = out.float().cpu()
    assert torch.isnan(got[1, 1]).all() and torch.isnan(lse[1, 1])
    got[1, 1] = 0
    assert torch.isfinite(got).all()
