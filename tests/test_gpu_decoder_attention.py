"""The decoder's attention against softmax in 64 bits, inside the decoder and
through it.

Inside: every df11_attention call that the decoder makes is compared with
softmax attention in 64 bits over what the decoder's own cache then holds, within
the bounds of test_gpu_step_attention.py.

Through it: logits of a plain model that rounds to BF16 and to 4 bits where the
decoder does and takes its attention in 64 bits.  The decoder's attention rounds
its weights to BF16, so from the first layer on the two differ by about a
rounding to BF16 at every stage: what one rounds up the other may round down.
Bound, before any run: a stage (norm, rotated queries, stored keys and values,
attention, residual, norm, activation, residual: 8 of a layer, and the final
norm) adds an error of at most 2^-8 of its values (root mean square: less than
the largest error of a rounding to BF16), independent of the others; 17 stages add to sqrt(17) * 2^-8;
twice that for stored keys and values, whose few other roundings to 4 bits are
larger.  Logits are then within 2^-5 of their spread (root mean square), and the
largest of 1056 within 4 times that."""
import numpy as np
import pytest
import torch

import step_reference as ref
from huffman_decode_amd import decoder
from huffman_decode_amd.decoder import StepInputs, from_weights
from test_gpu_decoder import BF16, CFG, Plain, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _setup(seed, page, lens):
    words, norms = _weights(seed)
    cols = 256 // page
    dec = from_weights(CFG, words, norms, n_pages=2 * cols, page_tokens=page, max_tokens=128, n_positions=256)
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(2 * cols, generator=g).to(torch.int32).view(2, cols)
    embed = torch.randn(CFG.vocab, CFG.hidden, generator=g).to(BF16)
    ids = [torch.randint(0, CFG.vocab, (n,), generator=g) for n in lens]
    return words, norms, dec, table, embed, ids


def _step(table, page, new, first):
    """Inputs of a step with new[b] tokens of sequence b, its first at first[b]."""
    pos = [torch.arange(f, f + n) for n, f in zip(new, first)]
    slots = [table[b, p // page] * page + p % page for b, p in enumerate(pos)]
    kv = [f + n for n, f in zip(new, first)]
    return pos, StepInputs(torch.cat(pos).to(torch.int32).cuda(), torch.cat(slots).to(torch.int32).cuda(),
                           torch.tensor([0, new[0], sum(new)], dtype=torch.int32).cuda(),
                           torch.tensor(kv, dtype=torch.int32).cuda(), table.cuda(), max(new), max(kv))


class Exact(Plain):
    """The plain model with attention in 64 bits."""

    def attend(self, q, k, v):
        held = [ref.values(*ref.quantise(x)) for x in (k, v)]
        o = ref.attention(q.double().numpy(), *held, CFG.head_dim ** -0.5, True, 0)[0]
        return torch.from_numpy(o).float().to(BF16).double()


@pytest.mark.parametrize("page", [16, 64])
def test_every_call_of_the_decoder(page, monkeypatch):
    lens = [70, 9]
    words, norms, dec, table, embed, ids = _setup(5, page, lens)
    calls = []

    def checked(cache, q, q_start, kv_lens, page_table, out, *args, **kw):
        decoder_attention(cache, q, q_start, kv_lens, page_table, out, *args, **kw)
        host = ref.Pages(cache.n_pages, cache.kv_heads, cache.page_tokens, cache.dim)
        host.blocks = cache.pages.cpu().numpy()
        starts, got = q_start.tolist(), out.double().cpu().numpy()
        for b, n in enumerate(kv_lens.tolist()):
            t = np.arange(n)
            slots = page_table[b].cpu().numpy().astype(np.int64)[t // page] * page + t % page
            k, v = host.load(slots)
            at = slice(starts[b], starts[b + 1])
            o, _, mass, reach = ref.attention(q[at].double().cpu().numpy(), k, v, cache.dim ** -0.5, True, 0)
            delta = (cache.dim + 8) * 2.0 ** -23 * reach[..., None]
            bound = (2.0 ** -8 + 2 * delta + 2.0 ** -18) * mass + 2.0 ** -8 * np.abs(o)
            assert (np.abs(got[at] - o) <= bound * (1 + 1e-6)).all(), (len(calls), b)
        calls.append(len(got))
    decoder_attention = decoder.df11_attention
    monkeypatch.setattr(decoder, "df11_attention", checked)
    _, step = _step(table, page, lens, [0, 0])
    dec.forward(embed[torch.cat(ids)].cuda(), step)
    for i in range(2):
        _, step = _step(table, page, [1, 1], [n + i for n in lens])
        dec.forward(embed[[3 + i, 8 + i]].cuda(), step)
    assert calls == [79, 79, 2, 2, 2, 2]


def test_logits_with_attention_in_64_bits(monkeypatch):
    page, lens = 64, [70, 9]
    words, norms, dec, table, embed, ids = _setup(6, page, lens)
    plain = [Exact(words, norms, dec.cos.cpu(), dec.sin.cpu()) for _ in lens]
    monkeypatch.setattr("test_gpu_decoder._attention", plain[0].attend)
    new, first = ids, [0, 0]
    for i in range(3):
        pos, step = _step(table, page, [len(n) for n in new], first)
        last = torch.tensor([len(new[0]) - 1, len(new[0]) + len(new[1]) - 1]).cuda()
        got = dec.forward(embed[torch.cat(new)].cuda(), step, last).double().cpu()
        want = torch.stack([p.step(embed[n], x)[-1] for p, n, x in zip(plain, new, pos)])
        off = (got - want) / want.std()
        rms, most = float(off.square().mean().sqrt()), float(off.abs().max())
        print(f"[gpu] step {i}: logits off by {most:.4f} of their spread, rms {rms:.4f}", flush=True)
        assert rms <= 2.0 ** -5 and most <= 2.0 ** -3
        first = [f + len(n) for f, n in zip(first, new)]
        new = [got.argmax(1)[:1], got.argmax(1)[1:]]
    assert int(dec.status.item()) == 0
