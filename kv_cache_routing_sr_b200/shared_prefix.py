"""A batch that shares a long prefix: one decode token of every sequence over the
prefix once for all, and over each sequence's own suffix.

The prefix (a system prompt, a document that many questions are asked about, the
samples of one prompt) is stored once, bf16 [Hkv, max_prefix_len, 128]. Every
sequence has its own cache for what follows it, bf16 or 8-bit [B, Hkv,
max_suffix_len, 128], whose slot 0 holds position prefix_len, and at least one
position in it (the token being decoded). One step:

1. routing of every (sequence, KV head) unit, as without a prefix: k0 / v0 are the
   prefix's position-0 rows, [B, Hkv, 128];
2. ``sr_decode_attention_partial`` (or the 8-bit form) over the suffixes;
3. ``sr_prefix_attention``: the active query heads of all sequences over the prefix,
   joined with the suffixes' partials by the log-sum-exp rule of the SinkRouter
   README's split-K reduction (decode-time procedure list).

Sink units skip both caches and get v0.
"""
from __future__ import annotations

import torch

from . import native


class SharedPrefixDecoder:
    """Owns the route buffers, partials and workspaces of one layer shape's steps."""

    def __init__(self, batch, n_q_heads, n_kv_heads, max_prefix_len, max_suffix_len, max_splits: int = 0,
                 device="cuda"):
        # before the workspaces, behind whose initialisation any stream may use them
        self.q = torch.empty(batch, n_q_heads, native.HEAD_DIM, dtype=torch.bfloat16, device=device)
        self.o_suffix = torch.empty(batch, n_q_heads, native.HEAD_DIM, dtype=torch.float32, device=device)
        self.lse_suffix = torch.empty(batch, n_q_heads, dtype=torch.float32, device=device)
        self.suffix = native.Decoder(batch, n_q_heads, n_kv_heads, max_suffix_len, max_splits, device=device)
        self.workspace = native.PrefixWorkspace(batch, n_q_heads, n_kv_heads, max_prefix_len, device=device)

    @property
    def out(self):
        return self.suffix.out

    @property
    def route_mask(self):
        return self.suffix.route_mask

    @property
    def active_list(self):
        return self.suffix.active_list

    def _check(self, q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, k0, v0, seq_lens, kv_scales, n_splits):
        """Everything that a launch of the step would refuse or read past, before the
        first one: an appended token is not taken back."""
        s = self.suffix
        native._loaded().step_fits(s.out, s.shape[2], q, k0, v0, k_prefix, v_prefix, prefix_len, k_cache, v_cache,
                                   kv_scales, seq_lens)
        if n_splits != 0:
            native._expect_splits(s.shape, n_splits, native.SPLITS_BY_UNIT, s.workspace)

    def _attend(self, q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, v0, seq_lens, kv_scales, n_splits, stream):
        s = self.suffix
        if kv_scales is None:
            native.decode_attention_partial(q, k_cache, v_cache, None, v0, seq_lens, s.active_list, self.o_suffix,
                                            self.lse_suffix, n_splits or native.SPLITS_BY_UNIT, s.workspace, stream)
        else:
            # 0 cuts an 8-bit cache by unit
            native.decode_attention_quant_partial(q, k_cache, v_cache, kv_scales, v0, seq_lens, s.active_list,
                                                  self.o_suffix, self.lse_suffix, max(n_splits, 0), s.workspace, stream)
        return native.prefix_attention(q, k_prefix, v_prefix, prefix_len, v0, s.route_mask, s.out, None, self.o_suffix,
                                       self.lse_suffix, self.workspace, stream)

    def step(self, q, k_prefix, v_prefix, prefix_len: int, k_cache, v_cache, k0, v0, seq_lens, tau, kv_scales=None,
             n_splits: int = 0, stream=None):
        """One step on rotated queries; seq_lens [B] are the suffixes' lengths (>= 1).
        kv_scales: the scales of an 8-bit suffix cache, None for bf16. Returns out
        bf16 [B, Hq, 128]."""
        self._check(q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, k0, v0, seq_lens, kv_scales, n_splits)
        native.route(q, k0, tau, self.route_mask, self.active_list, stream)
        return self._attend(q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, v0, seq_lens, kv_scales, n_splits,
                            stream)

    def append_step(self, q_in, k_new, v_new, rope_cos, rope_sin, k_prefix, v_prefix, prefix_len: int, k_cache,
                    v_cache, k0, v0, seq_lens, tau, kv_scales=None, n_splits: int = 0, device_error=None,
                    stream=None):
        """A whole step from the un-rotated projections: the new token joins its
        sequence's suffix at position prefix_len + seq_lens[b], then the attention.
        The suffix caches and seq_lens are updated in place; the rotated query is
        kept in self.q."""
        self._check(q_in, k_prefix, v_prefix, prefix_len, k_cache, v_cache, k0, v0, seq_lens, kv_scales, n_splits)
        native.rope_append_route_kv(q_in, k_new, v_new, rope_cos, rope_sin, seq_lens, k_cache, v_cache, kv_scales, k0,
                                    v0, tau, pos_offset=prefix_len, q_out=self.q, route_mask=self.route_mask,
                                    active_list=self.active_list, device_error=device_error, stream=stream)
        return self._attend(self.q, k_prefix, v_prefix, prefix_len, k_cache, v_cache, v0, seq_lens, kv_scales,
                            n_splits, stream)
