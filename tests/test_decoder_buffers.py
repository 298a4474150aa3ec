"""The buffers that huffman_decode_amd/decoder.py keeps between steps: what a
captured step has the address of stays allocated as long as the decoder."""
import weakref

import numpy as np
import pytest
import torch

from huffman_decode_amd import decoder
from huffman_decode_amd import workloads as wl
from huffman_decode_amd.decoder import Decoder, DecoderConfig, DecoderLayer, StepInputs, from_weights

CFG = DecoderConfig(hidden=64, mlp=96, heads=4, kv_heads=2, head_dim=64, vocab=80, layers=1)
BF16 = torch.bfloat16


class NoMatrix:
    def workspace_bytes(self, tokens):
        return 0


class NoCache:
    @classmethod
    def empty(cls, *args):
        return cls()


def test_no_workspace_of_attention_is_freed_before_the_decoder(monkeypatch):
    """A graph captured at any step holds the address of the workspace of that
    step, so a later step that needs more must leave it allocated."""
    handed = []
    monkeypatch.setattr(decoder, "KvCache", NoCache)
    monkeypatch.setattr(decoder, "df11_attention_workspace_bytes",
                        lambda cache, tokens, heads, batch, max_queries, max_kv: max_kv)
    monkeypatch.setattr(decoder, "df11_attention",
                        lambda *a, workspace=None, **k: handed.append((weakref.ref(workspace),
                                                                       workspace.data_ptr(), workspace.numel())))
    one = NoMatrix()
    norm = torch.ones(CFG.hidden)
    dec = Decoder(CFG, [DecoderLayer(one, one, one, one, norm, norm)], norm, one, n_pages=1, device="cpu")
    sizes = [4096, 1 << 20, 4096, 3 << 20, 1 << 20]
    i = torch.zeros(2, dtype=torch.int32)
    for n in sizes:
        dec._attend(None, 1, StepInputs(i, i, i, i[:1], i[None], 1, n))
    for (ref, address, held), n in zip(handed, sizes):
        assert held >= n
        assert ref() is not None and ref().data_ptr() == address, f"the workspace of {held} bytes was freed"
    # what is kept stays in proportion to the largest
    assert sum(s for _, s in {(a, s) for _, a, s in handed}) <= 3 * handed[-1][2]


def _words(seed):
    rng = np.random.default_rng(seed)
    words, norms = {}, {}
    for i in range(CFG.layers):
        for name, (r, c) in CFG.shapes().items():
            words[i, name] = wl.to_bf16((rng.standard_normal(r * c) / np.sqrt(c)).astype(np.float32))
        norms[i, "attn"] = norms[i, "mlp"] = torch.ones(CFG.hidden, dtype=BF16)
    words["head"] = wl.to_bf16((rng.standard_normal(CFG.vocab * CFG.hidden) / 8).astype(np.float32))
    norms["final"] = torch.ones(CFG.hidden, dtype=BF16)
    return words, norms


@pytest.mark.gpu
def test_a_captured_step_after_a_step_that_needs_a_larger_workspace():
    """A single-token step whose tokens are split over workgroups is captured;
    an eager prompt then needs more workspace, other tensors are allocated, and
    replays must neither change those tensors nor differ from the eager step."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    page, cols = 64, 64                                   # up to 4096 tokens a sequence
    words, norms = _words(1)
    dec = from_weights(CFG, words, norms, n_pages=2 * cols, page_tokens=page, max_tokens=128, n_positions=4096)
    table = torch.arange(2 * cols, dtype=torch.int32).view(2, cols).cuda()
    x = torch.randn(128, CFG.hidden, generator=torch.Generator().manual_seed(2)).to(BF16).cuda()

    def i32(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def prompt(max_kv):
        at = torch.arange(128, dtype=torch.int32, device="cuda")
        return dec.forward(x, StepInputs(at, table[0, (at // page).long()] * page + at % page, i32(0, 128),
                                         i32(128), table[:1], 128, max_kv))
    prompt(128)
    step = StepInputs(i32(128, 0), i32(128, cols * page), i32(0, 1, 2), i32(129, 1), table, 1, cols * page)
    need = decoder.df11_attention_workspace_bytes(dec.caches[0], 2, CFG.heads, 2, 1, cols * page)
    more = decoder.df11_attention_workspace_bytes(dec.caches[0], 128, CFG.heads, 1, 128, cols * page)
    assert 0 < need < more
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = dec.forward(x[:2], step)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dec.forward(x[:2], step)
    print("[gpu] captured with", need, "bytes; a prompt with", more, flush=True)
    prompt(cols * page)
    others = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in [need] * 64 + [more] * 4]
    for r in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {r}"
        assert all(bool((t == 0x5A).all()) for t in others), f"replay {r} wrote into other tensors"
        assert torch.equal(dec.forward(x[:2], step), want)
    assert int(dec.status.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 20, 40])
@pytest.mark.parametrize("wrong", ["position", "negative position", "slot", "kv_len", "queries"])
def test_what_an_index_out_of_range_leaves_out_is_nan(wrong, tokens):
    """A token past the rotary table or the cache, a sequence past the stated
    limits: its logits are NaN, not numbers made of an earlier step's queries or
    attention rows; those of the other sequence are as ever, bit by bit."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    page, n_pos = 16, 128
    words, norms = _words(3)
    dec = from_weights(CFG, words, norms, n_pages=12, page_tokens=page, max_tokens=2 * tokens, n_positions=n_pos)
    table = torch.arange(12, dtype=torch.int32).view(2, 6).cuda()
    g = torch.Generator().manual_seed(4)

    def i32(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def run(x, first, positions=None, slots=None, kv=None, max_queries=tokens):
        at = torch.arange(tokens, device="cuda")
        pos = torch.cat([at + first, at + first]).to(torch.int32)
        seq = torch.arange(2, device="cuda").repeat_interleave(tokens)
        own = table[seq, (pos // page).long()] * page + pos % page
        return dec.forward(x, StepInputs(pos if positions is None else positions(pos),
                                         own if slots is None else slots(own), i32(0, tokens, 2 * tokens),
                                         i32(first + tokens, first + tokens) if kv is None else kv, table,
                                         max_queries, 80))

    def last(t, value):  # the last token's entry
        t = t.clone()
        t[-1] = value
        return t
    x = [torch.randn(2 * tokens, CFG.hidden, generator=g).to(BF16).cuda() for _ in range(2)]
    run(x[0], 0)
    want = run(x[1], tokens).clone()
    assert torch.isfinite(want).all() and int(dec.status.item()) == 0
    run(x[0], 0)
    bad = torch.zeros(2 * tokens, dtype=torch.bool)
    bad[-1] = True
    if wrong == "position":
        got = run(x[1], tokens, positions=lambda p: last(p, n_pos))
    elif wrong == "negative position":
        got = run(x[1], tokens, positions=lambda p: last(p, -1))
    elif wrong == "slot":
        got = run(x[1], tokens, slots=lambda s: last(s, 12 * page))
    elif wrong == "kv_len":
        got, bad[tokens:] = run(x[1], tokens, kv=i32(2 * tokens, 81)), True
    else:
        got, bad[:] = run(x[1], tokens, max_queries=tokens - 1), True
        if tokens == 1:  # no queries at all: nothing is launched, and nothing counted
            dec.status.fill_(1)
    print("[gpu]", wrong, tokens, "status", int(dec.status.item()), flush=True)
    assert int(dec.status.item()) > 0
    nan = torch.isnan(got).cpu()
    assert bool(nan[bad].all()) and not bool(nan[~bad].any())
    assert torch.equal(got.cpu()[~bad], want.cpu()[~bad])
