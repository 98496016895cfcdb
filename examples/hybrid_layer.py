"""A hybrid layer served end to end: an SSD mixer followed by an attention block, as Zamba-like models
interleave them, with random weights.

  python examples/hybrid_layer.py            # a batch of ragged prompts, in chunks, then single tokens

The layer keeps what its requests need between calls: the SSD mixer's conv and SSM states, and the
attention block's paged int8 key/value cache.  A prompt goes through in chunks of any length (the
attention of a later chunk reads the earlier ones back from the cache), then token by token.
"""
from __future__ import annotations

import sys
from pathlib import Path

import torch

if str(Path(__file__).resolve().parents[1]) not in sys.path:
    sys.path.insert(0, str(Path(__file__).resolve().parents[1]))

from selective_state_space_prefill_gb300 import binding as ssm          # noqa: E402
from selective_state_space_prefill_gb300.rope import rope_frequencies   # noqa: E402


class HybridLayer:
    """x -> x + mixer(x) -> x + attention(x) for up to ``batch`` requests of up to ``max_len`` tokens."""

    def __init__(self, batch=2, d_model=512, ssd_heads=16, q_heads=8, kv_heads=2, head_dim=64, max_len=1024, page=64,
                 cache=torch.int8, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device=device) / k ** 0.5).to(torch.bfloat16)

        self.B, self.H, self.G = batch, ssd_heads, 1
        self.q_heads, self.kv_heads, self.dim, self.page, self.max_len = q_heads, kv_heads, head_dim, page, max_len
        hp, cx = 64 * ssd_heads, 64 * ssd_heads + 128
        self.w_in = weight(hp + cx + ssd_heads, d_model)            # [z | x B C | dt]
        self.w_out = weight(d_model, hp)
        self.conv_w = (torch.rand(cx, 4, generator=g, device=device) - 0.5).contiguous()
        self.conv_b = torch.zeros(cx, device=device)
        self.A = -(1.0 + 15.0 * torch.rand(ssd_heads, generator=g, device=device))
        self.D = torch.ones(ssd_heads, device=device)
        self.dt_bias = torch.full((ssd_heads,), -4.0, device=device)
        self.conv_state = torch.zeros(batch, 3, cx, device=device)
        self.ssm_state = torch.zeros(batch, ssd_heads, 64, 64, device=device)

        self.w_qkv = weight((q_heads + 2 * kv_heads) * head_dim, d_model)
        self.w_o = weight(d_model, q_heads * head_dim)
        self.cos, self.sin = ssm.attn_rope_table(rope_frequencies(head_dim)[0], max_len, device=device)
        pages = -(-max_len // page)
        shape = (batch * pages, kv_heads, page, head_dim)
        # the pool's pages dealt to the requests in turn, as an allocator would hand them out
        self.table = torch.arange(batch * pages, dtype=torch.int32, device=device).view(pages, batch).t().contiguous()
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=cache, device=device) for _ in range(2))
        i8 = cache == torch.int8
        self.k_scale, self.v_scale = ((torch.zeros(shape[:3], device=device) for _ in range(2)) if i8 else (None, None))
        self.workspace = torch.empty(max(1, ssm.attn_decode_workspace_bytes(batch, q_heads, kv_heads, head_dim, max_len)),
                                     dtype=torch.uint8, device=device)
        self.lens = [0] * batch

    def _slots(self, rows, pos):
        return (self.table[rows, pos // self.page] * self.page + pos % self.page).to(torch.int32)

    def _mixer(self, x, states):
        """The SSD mixer over x [1 or B, L, d_model]; states (conv, ssm) in and out."""
        hp, cx = 64 * self.H, 64 * self.H + 128 * self.G
        h = x @ self.w_in.T
        args = (self.conv_w, self.conv_b, self.A, self.D, self.dt_bias, self.H, self.G)
        z, xbc, dt = h[..., :hp], h[..., hp:hp + cx], h[..., hp + cx:]
        if x.shape[1] == 1:
            y = ssm.ssd_decode_step(xbc[:, 0].contiguous(), z[:, 0].contiguous(), dt[:, 0].contiguous(), *args, *states,
                                    out_dtype=torch.bfloat16)[:, None]
        else:
            y, c, s = ssm.ssd_prefill(xbc, z, dt, *args, conv_state_in=states[0], ssm_state_in=states[1],
                                      out_dtype=torch.bfloat16)
            states[0].copy_(c)
            states[1].copy_(s)
        y = y.reshape(-1, hp)
        return x + ssm.out_proj_partial(y, self.w_out, block_amax=False)[0].view(x.shape)

    def _append(self, x, rows, pos):
        """Rotate and cache the projections of x [T, d_model]; returns the rotated queries."""
        qkv = (x @ self.w_qkv.T).view(x.shape[0], -1, self.dim)
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)
        return ssm.attn_append(q, k, v, pos.to(torch.int32), self.cos, self.sin, self.k_cache, self.v_cache,
                               self._slots(rows, pos), self.k_scale, self.v_scale)[0]

    def _attention_out(self, x, o):
        return x + ssm.out_proj_partial(o.reshape(x.shape[0], -1), self.w_o, block_amax=False)[0]

    def prefill(self, chunks):
        """The next chunk of each request's prompt: a list of [L_b, d_model], empty for a request that has
        none.  Returns their outputs."""
        dev = self.table.device
        new = [c.shape[0] for c in chunks]
        mixed = []
        for b, c in enumerate(chunks):
            states = (self.conv_state[b:b + 1], self.ssm_state[b:b + 1])
            mixed.append(self._mixer(c[None], states)[0] if c.shape[0] else c)
        x = torch.cat(mixed)
        rows = torch.cat([torch.full((n,), b, device=dev) for b, n in enumerate(new)])
        pos = torch.cat([torch.arange(n, device=dev) + s for n, s in zip(new, self.lens)])
        q = self._append(x, rows, pos)
        self.lens = [s + n for s, n in zip(self.lens, new)]
        # a request without a chunk takes no part: no keys either
        keys = [s if n else 0 for s, n in zip(self.lens, new)]
        cu_q, cu_k = (torch.tensor([0] + v, device=dev).cumsum(0).to(torch.int32) for v in (new, keys))
        k, v = ssm.attn_cache_read(self.k_cache, self.v_cache, self.table, cu_k, sum(keys), self.k_scale, self.v_scale)
        o, _ = ssm.attn_prefill(q, k, v, cu_q, cu_k, max(new))
        return list(self._attention_out(x, o).split(new))

    def decode(self, x):
        """One token of every request: x [B, d_model].  Returns the layer's output [B, d_model]."""
        dev = self.table.device
        x = self._mixer(x[:, None], (self.conv_state, self.ssm_state))[:, 0]
        pos = torch.tensor(self.lens, device=dev)
        q = self._append(x, torch.arange(self.B, device=dev), pos)
        self.lens = [n + 1 for n in self.lens]
        lens = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        o, _ = ssm.attn_decode_step(q, self.k_cache, self.v_cache, self.table, lens, self.max_len, self.k_scale, self.v_scale,
                                    workspace=self.workspace)
        return self._attention_out(x, o)


def main():
    torch.manual_seed(0)
    layer = HybridLayer(batch=3)
    prompts = [torch.randn(n, 512, device="cuda").to(torch.bfloat16) for n in (700, 129, 5)]
    layer.prefill([p[:256] for p in prompts])
    layer.prefill([p[256:] for p in prompts])                   # two of the three are done after the first chunk
    x = torch.randn(3, 512, device="cuda").to(torch.bfloat16)
    for _ in range(8):
        x = layer.decode(x)
        x = ssm.norm_rms(x)[0]
    torch.cuda.synchronize()
    status = ssm.device_status()
    print(f"cached tokens {layer.lens}, last output RMS {float(x.float().square().mean().sqrt()):.3f}, status {status}")


if __name__ == "__main__":
    main()
