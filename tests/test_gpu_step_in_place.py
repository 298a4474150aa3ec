"""GPU test of df11_logits in place where rows start between 16-byte boundaries:
a group of 4 ids then begins in the row before, which another workgroup updates
at the same time."""
import pytest
import torch

import step_reference as ref
from test_gpu_step_rows import _close, _history, U

import huffman_decode_amd as hd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("rows,vocab,pad", [(7, 4097, 0), (5, 4098, 0), (6, 5001, 0), (300, 8193, 0), (9, 4100, 3),
                                            (8, 12287, 2), (64, 9, 0)])
def test_logits_in_place(rows, vocab, pad):
    g = torch.Generator().manual_seed(vocab + rows)
    whole = (4 * torch.randn(rows, vocab + pad, generator=g)).cuda()
    z = whole[:, :vocab]
    t, lens, prompts = _history(rows, 90, vocab, 3)
    n = min(9, vocab)
    kw = {"tokens": t, "lens": lens, "prompt_lens": prompts,
          "repetition": 0.5 + torch.rand(rows, generator=g), "frequency": torch.rand(rows, generator=g) - 0.3,
          "presence": torch.rand(rows, generator=g) - 0.3,
          "bias_ids": torch.randint(-2, vocab + 2, (rows, n), generator=g).to(torch.int32),
          "bias_values": torch.randn(rows, n, generator=g),
          "mask": torch.randint(-2**31, 2**31, (rows, -(-vocab // 32)), generator=g).to(torch.int32)}
    want, size = ref.logits(z.cpu(), **kw)
    rest = whole[:, vocab:].clone()
    print("[gpu] logits in place", rows, vocab, pad, flush=True)
    hd.df11_logits(z, z, **{k: v.cuda() for k, v in kw.items()})
    _close(z, want, size * 6 * U, "in place")
    assert torch.equal(whole[:, vocab:], rest)
