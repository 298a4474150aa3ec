"""A transformer decoder over DF11 weights: the matrix products straight from
the compressed streams, the operators of :mod:`huffman_decode_amd.step`
between them, keys and values in the paged 4-bit cache.

The DF11 pages describe inference that decompresses a block's weights just
before its products (page "DFloat11: lossless BFloat16 compression", section
"Architecture").  Here a step of up to 64 tokens never writes them out: its
products decode operand tiles and multiply them on the matrix cores
(``df11_decode_gemm_tiled``).  A longer prompt decodes each matrix once
(``df11_decode_tiled``) and multiplies it with torch.

The weights are lossless; the cache is not: keys and values are rounded to 4
bits and a power of two per 32 channels, so logits differ from those of the
same BF16 weights over a BF16 cache.

The layer is the common pre-norm one: root-mean-square norms, grouped query
heads with rotary positions, silu(gate) * up.  Weights are row-major [out, in]
BF16 words; q, k and v are stacked by rows, as are gate and up.  Pages are the
caller's to hand out.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (TILED_MAX_BATCH, TiledDevice, df11_decode_gemm_tiled, df11_decode_tiled,
               df11_tiled_workspace_bytes, encode_tiled, tiled_to_device)
from .step import (KvCache, df11_add_rms_norm, df11_attention, df11_attention_workspace_bytes,
                   df11_logits, df11_rope_append, df11_silu_mul)


@dataclass
class DecoderConfig:
    hidden: int
    mlp: int
    heads: int
    kv_heads: int
    head_dim: int
    vocab: int
    layers: int
    eps: float = 1e-5
    rope_base: float = 10000.0

    @property
    def qkv_rows(self) -> int:
        return (self.heads + 2 * self.kv_heads) * self.head_dim

    def shapes(self) -> dict[str, tuple[int, int]]:
        """[rows, cols] of a layer's matrices (rows multiples of 16, cols of 32)."""
        return {"qkv": (self.qkv_rows, self.hidden), "o": (self.hidden, self.heads * self.head_dim),
                "gate_up": (2 * self.mlp, self.hidden), "down": (self.hidden, self.mlp)}


class Linear:
    """One [rows, cols] matrix as a DF11 stream in operand-tile order."""

    def __init__(self, weights, rows: int, cols: int, device="cuda"):
        """weights: rows * cols BF16 words (numpy uint16), row-major."""
        self.rows, self.cols = rows, cols
        self.td: TiledDevice = tiled_to_device(encode_tiled(weights, [(rows, cols)]), device)

    def workspace_bytes(self, tokens: int) -> int:
        if tokens > TILED_MAX_BATCH:
            return 2 * self.rows * self.cols
        return df11_tiled_workspace_bytes(self.td.mats, tokens)

    def __call__(self, x, out, workspace) -> None:
        """out [tokens, rows] float32 = x [tokens, cols] bfloat16 times the matrix."""
        tokens = x.shape[0]
        if tokens <= TILED_MAX_BATCH:
            df11_decode_gemm_tiled(self.td, x, out, workspace)
            return
        w = workspace[: 2 * self.rows * self.cols].view(torch.bfloat16)
        df11_decode_tiled(self.td, w)
        # fp32 results, as the tiled product's: what follows rounds once
        torch.mm(x, w.view(self.rows, self.cols).t(), out_dtype=torch.float32, out=out)


@dataclass
class DecoderLayer:
    qkv: Linear
    o: Linear
    gate_up: Linear
    down: Linear
    attn_norm: torch.Tensor   # [hidden]
    mlp_norm: torch.Tensor


@dataclass
class StepInputs:
    """What a step works on.  Sequence b has the new tokens q_start[b] ..
    q_start[b + 1] - 1 and kv_lens[b] tokens in the cache, the new ones
    included; all on the GPU, int32."""
    positions: torch.Tensor    # [tokens]
    slots: torch.Tensor        # [tokens], negative: not stored
    q_start: torch.Tensor      # [sequences + 1]
    kv_lens: torch.Tensor      # [sequences]
    page_table: torch.Tensor   # [sequences, pages]
    max_queries: int
    max_kv: int


class Decoder:
    """Layers, final norm and head over one cache per layer, with every buffer a
    step of up to ``max_tokens`` tokens needs.  A step allocates its logits (and
    the rows picked for them), and attention's workspace when it needs a larger
    one than the steps before.  Whatever a step has used stays allocated as long
    as the decoder, so a captured step can be replayed after any other.

    ``status`` (an int32 tensor of one element that the caller reads, and may
    clear) counts what the layers left out because an index was out of range: a
    token whose position is not in the rotary table (``n_positions``) or whose
    slot is not in the cache, a sequence past ``max_queries`` or ``max_kv``.
    Their logits are NaN.  A token left out has stored no key: what its slot
    held before is what later tokens of its sequence read."""

    def __init__(self, config: DecoderConfig, layers: list[DecoderLayer], final_norm, head: Linear,
                 n_pages: int, page_tokens: int = 64, max_tokens: int = 64, n_positions: int = 4096,
                 device="cuda"):
        if len(layers) != config.layers:
            raise ValueError(f"{len(layers)} layers, {config.layers} configured")
        c = self.config = config
        self.layers, self.final_norm, self.head = layers, final_norm, head
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.caches = [KvCache.empty(n_pages, c.kv_heads, c.head_dim, page_tokens, device, self.status)
                       for _ in layers]
        half = c.head_dim // 2
        angle = torch.arange(n_positions, dtype=torch.float64)[:, None] * c.rope_base ** (
            -torch.arange(half, dtype=torch.float64) / half)
        self.cos, self.sin = (t.float().to(device) for t in (torch.cos(angle), torch.sin(angle)))

        def new(*shape, dtype):
            return torch.empty(max_tokens, *shape, dtype=dtype, device=device)
        bf16, f32 = torch.bfloat16, torch.float32
        self.residual, self.normed = new(c.hidden, dtype=bf16), new(c.hidden, dtype=bf16)
        self.qkv_out, self.hidden_out = new(c.qkv_rows, dtype=f32), new(c.hidden, dtype=f32)
        self.gate_up_out, self.act = new(2 * c.mlp, dtype=f32), new(c.mlp, dtype=bf16)
        self._left_out = torch.empty(2, max_tokens, c.heads, c.head_dim, dtype=bf16, device=device)
        self.q, self.attended = self._left_out
        linears = [head] + [m for l in layers for m in (l.qkv, l.o, l.gate_up, l.down)]
        need = max(m.workspace_bytes(n) for m in linears
                   for n in {min(max_tokens, TILED_MAX_BATCH), max_tokens})
        self.workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
        self.attention_workspace = torch.empty(0, dtype=torch.uint8, device=device)
        self._outgrown: list[torch.Tensor] = []

    def _attend(self, cache: KvCache, tokens: int, step: StepInputs) -> None:
        c = self.config
        need = df11_attention_workspace_bytes(cache, tokens, c.heads, step.kv_lens.shape[0],
                                              step.max_queries, step.max_kv)
        held = self.attention_workspace.numel()
        if need > held:
            # The one before is kept: a graph captured with it still writes there, and
            # so may a step on another stream.  At least doubled, so that all of them
            # together are at most twice the last.
            self._outgrown.append(self.attention_workspace)
            self.attention_workspace = torch.empty(max(need, 2 * held), dtype=torch.uint8,
                                                   device=self.q.device)
        df11_attention(cache, self.q[:tokens], step.q_start, step.kv_lens, step.page_table,
                       self.attended[:tokens], step.max_queries, step.max_kv,
                       workspace=self.attention_workspace if need else None)

    def forward(self, embedded, step: StepInputs, rows=None):
        """Hidden states of embedded [tokens, hidden] (bfloat16) through the
        layers, which append the tokens to the caches.  Returns fp32 logits
        [rows, vocab] of the given rows (an int64 index tensor; None: all)."""
        c, tokens = self.config, embedded.shape[0]
        if tokens > self.residual.shape[0]:
            raise ValueError(f"{tokens} tokens, buffers for {self.residual.shape[0]}")
        x, residual = embedded, None
        h, normed = self.residual[:tokens], self.normed[:tokens]
        # The operators leave out the rows of an index that is out of range, the same
        # ones in every layer: such a row stays NaN instead of an earlier step's.
        self._left_out[:, :tokens].fill_(float("nan"))
        for layer, cache in zip(self.layers, self.caches):
            if residual is None:
                h.copy_(embedded)
                df11_add_rms_norm(x, layer.attn_norm, normed, c.eps)
                residual = h
            else:
                df11_add_rms_norm(x, layer.attn_norm, normed, c.eps, residual=h)
            qkv = self.qkv_out[:tokens]
            layer.qkv(normed, qkv, self.workspace)
            q, k, v = qkv.unflatten(1, (c.heads + 2 * c.kv_heads, c.head_dim)).split(
                (c.heads, c.kv_heads, c.kv_heads), 1)
            df11_rope_append(cache, q, k, v, self.cos, self.sin, step.positions, step.slots,
                             self.q[:tokens])
            self._attend(cache, tokens, step)
            out = self.hidden_out[:tokens]
            layer.o(self.attended[:tokens].flatten(1), out, self.workspace)
            df11_add_rms_norm(out, layer.mlp_norm, normed, c.eps, residual=h)
            both, act = self.gate_up_out[:tokens], self.act[:tokens]
            layer.gate_up(normed, both, self.workspace)
            df11_silu_mul(both[:, :c.mlp], both[:, c.mlp:], act)
            layer.down(act, out, self.workspace)
            x = out
        df11_add_rms_norm(x, self.final_norm, normed, c.eps, residual=h)
        last = normed if rows is None else normed[rows]
        logits = torch.empty(last.shape[0], c.vocab, dtype=torch.float32, device=last.device)
        self.head(last, logits, self.workspace)
        return logits

    def next_tokens(self, logits, **penalties):
        """The most likely id of each row after df11_logits (its keyword
        arguments: tokens, lens, repetition, bias_ids, mask, ...), in place."""
        df11_logits(logits, logits, **penalties)
        return logits.argmax(1)


def from_weights(config: DecoderConfig, words: dict, norms: dict, device="cuda", **options) -> Decoder:
    """A decoder from BF16 words (numpy uint16, row-major): words[layer, name]
    for the names of ``config.shapes()`` and words["head"]; norms[layer,
    "attn" | "mlp"] and norms["final"]: [hidden] tensors."""
    shapes = config.shapes()
    layers = [DecoderLayer(*(Linear(words[i, name], *shapes[name], device) for name in shapes),
                           norms[i, "attn"].to(device), norms[i, "mlp"].to(device))
              for i in range(config.layers)]
    head = Linear(words["head"], config.vocab, config.hidden, device)
    return Decoder(config, layers, norms["final"].to(device), head, device=device, **options)
