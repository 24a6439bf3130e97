"""One decoder block as a serving program runs it: latent attention over the
paged cache, then the routed MoE layer, for a prompt, for agents that branch
off it, and for their next tokens.

    python examples/latent_moe_block.py

What happens, all on one GPU through the C ABI:
 1. a prompt's tokens get pages (moe_kv_reserve), their latent rows are stored
    (moe_kv_append), the block runs on them (moe_latent_prefill, moe_layer_forward);
 2. three agents branch off the prompt (moe_kv_fork): its full pages are shared,
    the last one is copied;
 3. each of the four sequences gets a token of its own and takes one decode step,
    the shared pages read once for all of them (moe_latent_decode with
    shared_tokens);
 4. two agents leave (moe_kv_free) and the pages in use move together
    (moe_kv_compact).
The projections around the attention are plain matrix products of the caller.
The step's attention is checked against the expanded form on the same cache.
Random weights, seeded: the block has no trained model behind it.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import edge_moe_serving_gb300 as moe  # noqa: E402
from moe_inputs import CONFIGS  # noqa: E402
from moe_inputs.device import DeviceCache, DeviceLayer  # noqa: E402

HEADS, DN, DV, RANK, ROPE, PAGE = 4, 64, 64, 128, 32, 16
MAX_SEQS, MAX_BLOCKS, N_PAGES = 4, 16, 48


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Block:
    """Weights, cache and workspaces of one decoder block."""

    def __init__(self, seed=0):
        self.cfg = CONFIGS["tiny"]
        H = self.cfg.H
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") / shape[-1] ** 0.5).to(torch.bfloat16)

        self.w_q = w(HEADS * (DN + ROPE), H)
        self.w_latent = w(RANK + ROPE, H)
        self.w_kv = w(HEADS, DN + DV, RANK)
        self.w_o = w(H, HEADS * DV)
        self.scale = (DN + ROPE) ** -0.5
        self.experts, self.layer = DeviceCache(self.cfg, "cuda:0"), DeviceLayer(self.cfg, 0, "cuda:0")
        self.pages = torch.empty(1, N_PAGES, PAGE, RANK + ROPE, dtype=torch.bfloat16, device="cuda")
        self.table = torch.full((MAX_SEQS, MAX_BLOCKS), -1, dtype=torch.int32, device="cuda")
        self.lens, self.refs = _i32([0] * MAX_SEQS), _i32([0] * N_PAGES)
        self.status = _i32([0])
        self.cache = moe.moe_kv_cache(self.pages.data_ptr(), self.table.data_ptr(), self.lens.data_ptr(),
                                      self.refs.data_ptr(), 1, N_PAGES, PAGE, RANK, ROPE, MAX_SEQS, MAX_BLOCKS, 0)

    def _ws(self, nbytes):
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")

    def _norm(self, x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def store(self, x, seqs, n_new, lens):
        """Pages for n_new tokens of each sequence (lens: what they hold), and their latent rows in them."""
        ws = self._ws(moe.moe_kv_workspace_size(self.cache, len(seqs)))
        moe.moe_kv_reserve(self.cache, _i32(seqs), _i32(n_new), len(seqs), ws, ws.numel(), self.status)
        rows = self._norm(x) @ self.w_latent.T
        rows = torch.cat([self._norm(rows[:, :RANK]), rows[:, RANK:]], 1).contiguous()
        tok_seq = _i32([s for s, n in zip(seqs, n_new) for _ in range(n)])
        tok_pos = _i32([p for n, at in zip(n_new, lens) for p in range(at, at + n)])
        moe.moe_kv_append(self.cache, 0, rows, tok_seq, tok_pos, len(x), self.status)

    def queries(self, x):
        return (self._norm(x) @ self.w_q.T).view(len(x), HEADS, DN + ROPE).contiguous()

    def attend_expanded(self, q, seqs, offsets, kv_tokens):
        B, T = len(seqs), len(q)
        ws = self._ws(moe.moe_latent_prefill_workspace_size(self.cache, B, T, HEADS, DN, DV, kv_tokens))
        out = torch.empty(T, HEADS, DV, dtype=torch.bfloat16, device="cuda")
        moe.moe_latent_prefill(self.cache, 0, q, _i32(seqs), _i32(offsets), B, T, HEADS, DN, DV, self.w_kv, self.scale,
                               kv_tokens, out, ws, ws.numel(), self.status)
        return out

    def attend_absorbed(self, q, seqs, shared):
        """One token a sequence: the key projection folded into the query, the value projection applied afterwards."""
        B = len(seqs)
        w_k, w_v = self.w_kv[:, :DN].float(), self.w_kv[:, DN:].float()
        lat = torch.einsum("bhd,hdr->bhr", q[..., :DN].float(), w_k).to(torch.bfloat16)
        qa = torch.cat([lat, q[..., DN:]], -1).contiguous()
        ws = self._ws(moe.moe_latent_decode_workspace_size(self.cache, B, 1, HEADS, shared))
        out = torch.empty(B, HEADS, RANK, dtype=torch.bfloat16, device="cuda")
        moe.moe_latent_decode(self.cache, 0, qa, _i32(seqs), B, 1, HEADS, self.scale, shared, out, None, ws, ws.numel(),
                              self.status)
        return torch.einsum("bhr,hdr->bhd", out.float(), w_v).to(torch.bfloat16)

    def finish(self, x, attn):
        """Output projection, residual, routed experts, residual."""
        T = len(x)
        h = x + attn.reshape(T, -1) @ self.w_o.T
        n = moe.moe_layer_workspace_size(self.layer.struct, self.experts.struct, T, moe.MOE_FFN_AUTO)
        ws, out = self._ws(n), torch.empty_like(h)
        moe.moe_layer_forward(self.layer.struct, self.experts.struct, self._norm(h).contiguous(), T, out, 0, 1, 0, 0,
                              moe.MOE_FFN_AUTO, None, ws, n, self.status, None)
        return h + out


def main(prompt_tokens=100, seed=0):
    """Runs the four steps; returns the step's attention in both forms, the block's outputs and the pages in use."""
    b = Block(seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(prompt_tokens, b.cfg.H, generator=g, device="cuda").to(torch.bfloat16)
    b.store(x, [0], [prompt_tokens], [0])
    y = b.finish(x, b.attend_expanded(b.queries(x), [0], [0, prompt_tokens], prompt_tokens))

    ws = b._ws(moe.moe_kv_workspace_size(b.cache, 3))
    moe.moe_kv_fork(b.cache, _i32([0, 0, 0]), _i32([1, 2, 3]), 3, ws, ws.numel(), b.status)

    seqs = [0, 1, 2, 3]
    x1 = torch.randn(4, b.cfg.H, generator=g, device="cuda").to(torch.bfloat16)
    b.store(x1, seqs, [1] * 4, [prompt_tokens] * 4)
    q1 = b.queries(x1)
    absorbed = b.attend_absorbed(q1, seqs, prompt_tokens // PAGE * PAGE)
    expanded = b.attend_expanded(q1, seqs, [0, 1, 2, 3, 4], 4 * (prompt_tokens + 1))
    y1 = b.finish(x1, absorbed)

    moe.moe_kv_free(b.cache, _i32([1, 2]), 2, b.status)
    n_live = _i32([0])
    moe.moe_kv_compact(b.cache, n_live, ws, ws.numel(), b.status)
    assert int(b.status.item()) == 0, f"device status {int(b.status.item())}"
    return absorbed, expanded, y, y1, int(n_live.item()), b


if __name__ == "__main__":
    absorbed, expanded, y, y1, n_live, block = main()
    rel = float((absorbed.float() - expanded.float()).norm() / expanded.float().norm())
    print(f"prompt block {tuple(y.shape)}, step {tuple(y1.shape)}, absorbed against expanded form: rel {rel:.1e}, "
          f"{n_live} pages in use")
