"""A small stack of recurrent blocks on the library's operators.

Each block is  residual add + RMS norm -> projection -> short convolution -> state update ->
projection, the state update being either the selective state-space scan or KDA.  The stack
trains (autograd through every operator), reads a prompt and goes on token by token from
the states that the prompt left.

    python examples/recurrent_block.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_cumsum_gb300 as kda  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class Block(torch.nn.Module):
    """`mixer` is "ssm" (heads of head_dim columns, one group of state_dim) or "kda" (heads of
    head_dim keys and values)."""

    def __init__(self, dim, mixer, heads=4, head_dim=64, state_dim=64, taps=4):
        super().__init__()
        self.mixer, self.H, self.P, self.N = mixer, heads, head_dim, state_dim
        wide = heads * head_dim
        self.conv_cols = wide + 2 * state_dim if mixer == "ssm" else 3 * wide
        extra = heads if mixer == "ssm" else heads + wide  # dt, or beta and the gate
        p = torch.nn.Parameter
        self.norm = p(torch.ones(dim))
        self.w_in = p((torch.randn(dim, self.conv_cols + extra) * dim ** -0.5).to(BF16))
        self.w_out = p((torch.randn(wide, dim) * wide ** -0.5).to(BF16))
        self.conv_w = p(torch.randn(self.conv_cols, taps) * taps ** -0.5)
        self.conv_b = p(torch.zeros(self.conv_cols))
        self.A_log = p(torch.log(torch.rand(heads) * 15 + 1))
        self.dt_bias = p(torch.full((heads,) if mixer == "ssm" else (heads, head_dim), -3.0))
        self.D = p(torch.ones(heads))

    def split(self, u):
        """The projection's columns: the convolution's, and the rest."""
        return u[..., :self.conv_cols], u[..., self.conv_cols:]

    def heads(self, c, rest):
        """The state update's inputs, as column ranges of the convolved projection."""
        H, P, N = self.H, self.P, self.N
        if self.mixer == "ssm":
            x, Bm, Cm = c.split([H * P, N, N], -1)
            return x.unflatten(-1, (H, P)), rest, Bm.unsqueeze(-2), Cm.unsqueeze(-2)
        q, k, v = (t.unflatten(-1, (H, P)) for t in c.split(H * P, -1))
        return q, k, v, rest[..., H:].unflatten(-1, (H, P)).float(), rest[..., :H]

    def kda_options(self):
        return dict(A_log=self.A_log, dt_bias=self.dt_bias, beta_sigmoid_scale=1.0,
                    use_qk_l2norm_in_kernel=True, g_scale=1.4426950408889634)

    # ---------------------------------------------------------------- training
    def train_step(self, x, res):
        y, res = kda.add_rms_norm_autograd(x, self.norm, residual=res)
        c, rest = self.split(y @ self.w_in)
        c, _ = kda.short_conv_autograd(c, self.conv_w, self.conv_b)
        ins = self.heads(c, rest)
        if self.mixer == "ssm":
            o, _ = kda.ssm_scan_autograd(ins[0], ins[1], self.A_log, *ins[2:], D=self.D, dt_bias=self.dt_bias)
        else:
            o, _ = kda.kda_autograd(*ins, **self.kda_options())
        return o.flatten(-2) @ self.w_out, res

    # ----------------------------------------------------------------- serving
    def _project(self, x, res):
        """The 8-bit entry: the norm's output leaves in 8 bits with a scale per 128 columns.  (An
        8-bit matrix product would take q and scale; here they are multiplied out.)"""
        q, scale, res = kda.add_rms_norm_quant(x, self.norm, residual=res, out_dtype="e4m3", group=128)
        wide = scale.repeat_interleave(128, -1)[..., :q.shape[-1]]
        return (q.float() * wide).to(BF16) @ self.w_in, res

    def new_cache(self, slots, device):
        """Convolution rows and states of `slots` sequences."""
        N = self.N if self.mixer == "ssm" else self.P
        return dict(conv=torch.zeros(slots, self.conv_w.shape[1] - 1, self.conv_cols, dtype=BF16, device=device),
                    state=torch.zeros(slots, self.H, N, self.P, device=device))

    @torch.no_grad()
    def prompt(self, x, res, cache, slots, cu):
        """Packed prompts x [1, T, dim] of sequences cu; their states go to cache[slots]."""
        u, res = self._project(x, res)
        c, rest = self.split(u)
        c, cache["conv"][slots] = kda.short_conv(c, self.conv_w, self.conv_b,
                                                 output_final_state=True, cu_seqlens=cu)
        ins = self.heads(c, rest)
        if self.mixer == "ssm":
            o, ht = kda.ssm_scan(ins[0], ins[1], self.A_log, *ins[2:], D=self.D,
                                 dt_bias=self.dt_bias, output_final_state=True, cu_seqlens=cu)
        else:
            o, ht = kda.chunk_kda(*ins, output_final_state=True, cu_seqlens=cu, **self.kda_options())
        cache["state"][slots] = ht
        return o.flatten(-2) @ self.w_out, res

    @torch.no_grad()
    def token(self, x, res, cache, slots):
        """One token x [n, dim] of the sequences in `slots` (int32)."""
        u, res = self._project(x, res)
        c, rest = self.split(u)
        c = kda.short_conv_step(c, cache["conv"], self.conv_w, self.conv_b, state_indices=slots)
        ins = self.heads(c, rest)
        if self.mixer == "ssm":
            o = kda.ssm_step(ins[0], ins[1], self.A_log, *ins[2:], cache["state"], D=self.D,
                             dt_bias=self.dt_bias, state_indices=slots)
        else:
            one = [t.unsqueeze(1) for t in ins]
            o, ht = kda.recurrent_kda(*one, cache["state"][slots.long()], output_final_state=True,
                                      **self.kda_options())
            cache["state"][slots.long()] = ht
            o = o.squeeze(1)
        return o.flatten(-2) @ self.w_out, res


class Stack(torch.nn.Module):
    def __init__(self, vocab=256, dim=256, mixers=("ssm", "kda", "ssm")):
        super().__init__()
        self.embed = torch.nn.Parameter((torch.randn(vocab, dim) * 0.5).to(BF16))
        self.blocks = torch.nn.ModuleList(Block(dim, m) for m in mixers)
        self.norm = torch.nn.Parameter(torch.ones(dim))

    def logits(self, ids):
        """[B, T] -> [B, T, vocab], with gradients."""
        x, res = self.embed[ids], None
        for b in self.blocks:
            x, res = b.train_step(x, res)
        return kda.add_rms_norm_autograd(x, self.norm, residual=res)[0] @ self.embed.t()

    def new_cache(self, slots):
        return [b.new_cache(slots, self.embed.device) for b in self.blocks]

    @torch.no_grad()
    def _head(self, x, res):
        return kda.add_rms_norm(x, self.norm, residual=res)[0] @ self.embed.t()

    @torch.no_grad()
    def prompt(self, prompts, cache, slots):
        """Reads the prompts (lists of token ids); the logits after each one's last token."""
        dev = self.embed.device
        lens = torch.tensor([len(p) for p in prompts])
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32).to(dev)
        x, res = self.embed[torch.tensor(sum(prompts, []), device=dev)][None], None
        for b, c in zip(self.blocks, cache):
            x, res = b.prompt(x, res, c, slots.long(), cu)
        last = (lens.cumsum(0) - 1).to(dev)
        return self._head(x[0, last], res[0, last])

    @torch.no_grad()
    def token(self, ids, cache, slots):
        """One more token for each of the sequences in `slots`; the logits after it."""
        x, res = self.embed[ids], None
        for b, c in zip(self.blocks, cache):
            x, res = b.token(x, res, c, slots)
        return self._head(x, res)


def main():
    torch.manual_seed(0)
    stack = Stack().cuda()
    data = torch.arange(0, 4 * 96, device="cuda").reshape(4, 96) * 7 % 256  # a sequence to learn
    opt = torch.optim.AdamW(stack.parameters(), lr=2e-3)
    for step in range(30):
        loss = torch.nn.functional.cross_entropy(stack.logits(data[:, :-1]).float().flatten(0, 1),
                                                 data[:, 1:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        if step % 10 == 0 or step == 29:
            print(f"step {step}: loss {loss.item():.3f}")
    cache, slots = stack.new_cache(8), torch.tensor([5, 2], dtype=torch.int32, device="cuda")
    out = stack.prompt([data[0, :40].tolist(), data[1, :17].tolist()], cache, slots)
    for _ in range(8):
        ids = out.argmax(-1)
        print("next tokens", ids.tolist())
        out = stack.token(ids, cache, slots)


if __name__ == "__main__":
    main()
