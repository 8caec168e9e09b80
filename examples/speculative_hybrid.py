"""One speculative step of a small hybrid model, with its rollback.

Two recurrent layers (a gated delta rule layer and a selective state space
layer) and a sampling head work on T draft tokens of every sequence:

    projection -> gdn_causal_conv -> gdn_step_record     -> gdn_gated_norm -> projection -> + residual
    projection -> gdn_causal_conv -> gdn_selective_scan  -> gdn_gated_norm -> projection -> + residual
    norm -> logits -> gdn_sample -> accepted = matches with the draft, from the first on

The rejected suffix of every sequence is then rolled back: the delta rule
state from the tape (gdn_state_replay), the other states by repeating their
calls from the snapshot with lengths = accepted.  `rollback_error` compares
what comes out with a run over the accepted tokens alone.

    python examples/speculative_hybrid.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_recurrence_step_gb300 as gdn  # noqa: E402


class HybridModel:
    """Random weights of the right distributions; bf16, f32 states."""

    def __init__(self, dev, *, d_model=512, vocab=4096, Hk=4, Hv=8, Dk=64, Dv=64, H=8, P=64, G=2, N=64, seed=0):
        self.dev, self.gen = dev, torch.Generator(device=dev).manual_seed(seed)
        self.Hk, self.Hv, self.Dk, self.Dv = Hk, Hv, Dk, Dv
        self.H, self.P, self.G, self.N = H, P, G, N
        w = lambda *s: (torch.randn(*s, generator=self.gen, device=dev) / s[-1] ** 0.5).bfloat16()  # noqa: E731
        self.embed, self.head = w(vocab, d_model), w(vocab, d_model)
        self.norms = [torch.ones(d_model, device=dev, dtype=torch.bfloat16) for _ in range(3)]
        self.gdn_channels = 2 * Hk * Dk + Hv * Dv
        self.gdn_in = w(self.gdn_channels + Hv * Dv + 2 * Hv, d_model)      # q, k, v | gate | beta, decay
        self.gdn_conv, self.gdn_out = w(self.gdn_channels, 4), w(d_model, Hv * Dv)
        self.gdn_norm = torch.ones(Dv, device=dev, dtype=torch.bfloat16)
        self.ssm_channels = H * P + 2 * G * N
        self.ssm_in = w(self.ssm_channels + H * P + H, d_model)             # x, B, C | gate | step
        self.ssm_conv, self.ssm_out = w(self.ssm_channels, 4), w(d_model, H * P)
        self.ssm_norm = torch.ones(H, P, device=dev, dtype=torch.bfloat16)  # a row per head
        self.A = -torch.rand(H, generator=self.gen, device=dev) - 0.5
        self.skip = torch.ones(H, device=dev)
        self.dt_bias = torch.full((H,), -2.0, device=dev)

    def new_state(self, B):
        z = lambda *s, dtype=torch.float32: torch.zeros(*s, device=self.dev, dtype=dtype)  # noqa: E731
        return {"gdn": z(B, self.Hv, self.Dv, self.Dk), "gdn_conv": z(B, 3, self.gdn_channels, dtype=torch.bfloat16),
                "ssm": z(B, self.H, self.P, self.N), "ssm_conv": z(B, 3, self.ssm_channels, dtype=torch.bfloat16)}

    def gdn_inputs(self, h):
        B, T, _ = h.shape
        proj = h @ self.gdn_in.T
        qkv, gate, mix = proj.split([self.gdn_channels, self.Hv * self.Dv, 2 * self.Hv], -1)
        beta, decay = torch.sigmoid(mix.float()).bfloat16().split([self.Hv, self.Hv], -1)
        return qkv, gate.unflatten(-1, (self.Hv, self.Dv)), beta.contiguous(), (0.9 + 0.1 * decay).contiguous()

    def forward(self, tokens, state, *, lengths=None):
        """Logits [B,T,V], the state after the tokens, and what the rollback needs."""
        Hk, Hv, Dk, Dv = self.Hk, self.Hv, self.Dk, self.Dv
        keep, new = {}, {}
        res = self.embed[tokens]
        h = gdn.gdn_gated_norm(res, self.norms[0]).y
        # the gated delta rule layer
        qkv, gate, beta, decay = self.gdn_inputs(h)
        conv = gdn.gdn_causal_conv(qkv, self.gdn_conv, state["gdn_conv"], lengths=lengths)
        q, k, v = conv.y.split([Hk * Dk, Hk * Dk, Hv * Dv], -1)
        unit = lambda t: torch.nn.functional.normalize(t.unflatten(-1, (Hk, Dk)).float(), dim=-1).bfloat16()  # noqa: E731
        mask = None
        if lengths is not None:
            mask = (torch.arange(tokens.shape[1], device=self.dev) < lengths[:, None]).int()
        rec = gdn.gdn_step_record(unit(q), unit(k), v.unflatten(-1, (Hv, Dv)).contiguous(), decay, beta, state["gdn"],
                                  mask, capture_tape=True)
        new["gdn"], new["gdn_conv"] = rec.state_out, conv.state_out
        keep.update(qkv=qkv, rec=rec)
        mixed = gdn.gdn_gated_norm(rec.y, self.gdn_norm, gate=gate).y.flatten(2) @ self.gdn_out.T
        out = gdn.gdn_gated_norm(mixed, self.norms[1], residual=res, residual_scale=0.5)
        res = out.residual_out
        # the selective state space layer
        xbc, gate, step = (out.y @ self.ssm_in.T).split([self.ssm_channels, self.H * self.P, self.H], -1)
        conv = gdn.gdn_causal_conv(xbc, self.ssm_conv, state["ssm_conv"], lengths=lengths)
        x, Bm, Cm = conv.y.split([self.H * self.P, self.G * self.N, self.G * self.N], -1)
        x, Bm, Cm = x.unflatten(-1, (self.H, self.P)), Bm.unflatten(-1, (self.G, self.N)), Cm.unflatten(-1, (self.G, self.N))
        scan = gdn.gdn_selective_scan(x, step, self.A, Bm, Cm, state["ssm"], D=self.skip, dt_bias=self.dt_bias,
                                      lengths=lengths)
        new["ssm"], new["ssm_conv"] = scan.state_out, conv.state_out
        keep.update(xbc=xbc, scan=(x, step, Bm, Cm))
        mixed = gdn.gdn_gated_norm(scan.y, self.ssm_norm, gate=gate.unflatten(-1, (self.H, self.P)),
                                   gate_first=True).y.flatten(2) @ self.ssm_out.T
        out = gdn.gdn_gated_norm(mixed, self.norms[2], residual=res, residual_scale=0.5)
        return out.y @ self.head.T, new, keep

    def roll_back(self, state, keep, accepted):
        """The state after the accepted tokens, from the snapshot."""
        rec, (x, step, Bm, Cm) = keep["rec"], keep["scan"]
        only = dict(lengths=accepted, write_y=False)
        return {"gdn": gdn.gdn_state_replay(rec.delta_log, rec.k_log, rec.g_log, state["gdn"], accepted=accepted),
                "gdn_conv": gdn.gdn_causal_conv(keep["qkv"], self.gdn_conv, state["gdn_conv"], **only).state_out,
                "ssm": gdn.gdn_selective_scan(x, step, self.A, Bm, Cm, state["ssm"], D=self.skip, dt_bias=self.dt_bias,
                                              **only).state_out,
                "ssm_conv": gdn.gdn_causal_conv(keep["xbc"], self.ssm_conv, state["ssm_conv"], **only).state_out}


def speculative_step(model, draft, state, noise, **settings):
    """Runs the T tokens of `draft` ([B,T]; the first is certain, each further
    one a guess for what follows the one before it) and keeps as many as match
    what the model samples.  Returns the sampled tokens, the number of tokens
    that stay (1 to T), and the state after those."""
    logits, _, keep = model.forward(draft, state)
    out = gdn.gdn_sample(logits, noise, **settings)
    match = (out.token[:, :-1] == draft[:, 1:]).int()
    accepted = (1 + match.cumprod(1).sum(1)).int()
    return out.token, accepted, model.roll_back(state, keep, accepted)


def rollback_error(model, draft, accepted, state, rolled):
    """Largest difference, of every state, from a run that never saw the rejected
    tokens."""
    _, want, _ = model.forward(draft, state, lengths=accepted)
    return {n: float((rolled[n].float() - want[n].float()).abs().max()) for n in want}


def main():
    dev = torch.device("cuda:0")
    model = HybridModel(dev)
    B, T = 4, 6
    state = model.new_state(B)
    prompt = torch.randint(0, 4096, (B, 200), generator=model.gen, device=dev)
    logits, state, _ = model.forward(prompt, state)
    nxt = logits[:, -1].float().argmax(-1, keepdim=True)
    for step in range(4):
        # a draft that is right now and then: the model's own greedy guess with some tokens changed
        draft = torch.cat([nxt, torch.randint(0, 4096, (B, T - 1), generator=model.gen, device=dev)], 1)
        for t in range(1, T):
            guess = model.forward(draft[:, :t], state)[0][:, -1].float().argmax(-1)
            right = torch.rand(B, generator=model.gen, device=dev) < 0.8
            draft[:, t] = torch.where(right, guess, draft[:, t])
        noise = torch.empty(B, T, 4096, device=dev).exponential_(generator=model.gen)
        token, accepted, rolled = speculative_step(model, draft, state, noise, temperature=0.05, top_k=50, top_p=0.95)
        err = rollback_error(model, draft, accepted, state, rolled)
        print(f"step {step}: kept {accepted.tolist()} of {T} tokens; rollback off by "
              + ", ".join(f"{n} {e:.1e}" for n, e in err.items()))
        nxt = token.gather(1, (accepted - 1).long()[:, None]).long()
        state = rolled


if __name__ == "__main__":
    main()
