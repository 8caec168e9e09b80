"""One speculative step of a hybrid model's attention layer over the 4-bit cache.

Requests of different lengths share a pool of pages.  In every step each of them
brings draft tokens; their pages and places, positions, keys and values, and the
attention over all that came before are

    gdn_page_slots -> gdn_rotary -> gdn_kv_append -> gdn_kv_attention -> projection
    -> gdn_gated_norm -> logits -> gdn_sample -> accepted = matches with the draft

and the rejected tokens go by shortening the sequences (their pages stay held and
are written over).  `rollback_error` compares the next step with one whose cache
never saw the rejected tokens.

    python examples/speculative_attention.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_recurrence_step_gb300 as gdn  # noqa: E402


class AttentionLayer:
    """Random bf16 weights; a pool of pages, and the requests that share it."""

    def __init__(self, dev, *, B=4, d_model=256, vocab=512, Hq=8, H=2, D=64, R=32, page=16, pages=200, width=40, seed=0):
        self.dev, self.gen = dev, torch.Generator(device=dev).manual_seed(seed)
        self.Hq, self.H, self.D, self.page = Hq, H, D, page
        w = lambda *s: (torch.randn(*s, generator=self.gen, device=dev) / s[-1] ** 0.5).bfloat16()  # noqa: E731
        self.embed, self.head = w(vocab, d_model), w(vocab, d_model)
        self.qkv, self.out = w((Hq + 2 * H) * D, d_model), w(d_model, Hq * D)
        self.norm = torch.ones(d_model, device=dev, dtype=torch.bfloat16)
        self.inv_freq, self.rope_scale = gdn.rotary_frequencies(R, scaling="parts_scaled", factor=4.0, trained=4096,
                                                                device=dev)
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
        self.cache = gdn.gdn_kv_cache(pages, H, page, D, device=dev)
        self.lengths, self.held, self.table = z(B), z(B), z(B, width)
        self.ring, self.ring_state = torch.arange(pages, dtype=torch.int32, device=dev), z(2)
        self.ring_state[1] = pages

    def forward(self, tokens, add=None):
        """Logits [B,T,V] of the tokens, of which sequence b has add[b] (None: all; -1
        ends it), and how many tokens each got."""
        T, D = tokens.shape[1], self.D
        s = gdn.gdn_page_slots(self.lengths, add, self.held, self.ring_state, self.table, self.ring, T=T, page=self.page,
                               lengths_out=self.lengths, held_out=self.held, ring_state_out=self.ring_state)
        x = self.embed[tokens]
        h = gdn.gdn_gated_norm(x, self.norm).y
        q, k, v = (h @ self.qkv.T).split([self.Hq * D, self.H * D, self.H * D], -1)
        heads = lambda t: t.unflatten(-1, (-1, D))  # noqa: E731
        r = gdn.gdn_rotary(heads(q), s.positions, self.inv_freq, k=heads(k), scale=self.rope_scale)
        gdn.gdn_kv_append(r.k, heads(v), s.slots, self.cache)
        y = torch.zeros_like(r.q)  # (rows that are not there stay zero)
        gdn.gdn_kv_attention(r.q, self.cache, self.table, self.lengths, new=s.granted, y=y)
        out = gdn.gdn_gated_norm(y.flatten(2) @ self.out.T, self.norm, residual=x, residual_scale=0.5)
        return out.y @ self.head.T, s.granted

    def shorten(self, rejected):
        """Rolls every sequence back by `rejected` tokens."""
        self.lengths -= rejected


def speculative_step(layer, draft, noise, **settings):
    """The T tokens of `draft` ([B,T]; the first is certain) and how many of each
    sequence stay (1 to T); the rest is rolled back."""
    logits, granted = layer.forward(draft)
    out = gdn.gdn_sample(logits, noise, **settings)
    match = (out.token[:, :-1] == draft[:, 1:]).int()
    accepted = (1 + match.cumprod(1).sum(1)).int()
    layer.shorten(granted - accepted)
    return out.token, accepted


def rollback_error(layer, other, nxt):
    """Largest difference of the next token's logits between a layer that was rolled
    back and one that never saw the rejected tokens."""
    return float((layer.forward(nxt)[0].float() - other.forward(nxt)[0].float()).abs().max())


def main():
    dev = torch.device("cuda:0")
    layer, plain = AttentionLayer(dev), AttentionLayer(dev)
    B, T, V = 4, 6, 512
    prompt = torch.randint(0, V, (B, 300), generator=layer.gen, device=dev)
    lengths = torch.tensor([300, 17, 120, 1], dtype=torch.int32, device=dev)
    for m in (layer, plain):
        m.forward(prompt, lengths)
    for step in range(4):
        draft = torch.randint(0, V, (B, T), generator=layer.gen, device=dev)
        noise = torch.empty(B, T, V, device=dev).exponential_(generator=layer.gen)
        token, accepted = speculative_step(layer, draft, noise, temperature=0.7, top_k=50)
        plain.forward(draft, accepted)
        nxt = token.gather(1, (accepted - 1).long()[:, None]).long()
        print(f"step {step}: kept {accepted.tolist()} of {T}, lengths {layer.lengths.tolist()}, "
              f"off by {rollback_error(layer, plain, nxt):.1e}")


if __name__ == "__main__":
    main()
