"""A block of a hybrid model run from prompt to generated tokens: one KDA layer, then one
latent-attention layer, random weights.

    python examples/hybrid_block.py            # bf16; needs the GPU and the built library

The prompts of several sequences are packed.  The KDA layer keeps a state per sequence
(kda.prefill, kda.decode_step).  The latent layer keeps one row of 576 channels per token in a paged
cache: kda.latent_append normalises, rotates and stores the rows and rotates the queries;
kda.latent_prefill attends over the prompt with keys and values expanded per head; kda.latent_decode
attends over the cache with the up-projections absorbed into the query and the output.  The script
then prefills the prompts with the generated tokens' inputs appended and compares: the last rows of
the expanded form must be what the absorbed steps gave.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from kda_gated_delta_04_gb300 import kda  # noqa: E402

R, P, N = kda.KDA_LATENT_DIM, kda.KDA_LATENT_PE_DIM, kda.KDA_LATENT_HEAD_DIM


def rms(x, eps=1e-6):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + eps)).to(x.dtype)


class KdaLayer:
    """q, k, v, the decay and beta from the block's input; the state is the library's."""

    def __init__(self, dim, heads, g, dt):
        self.heads, d = heads, 128
        self.w = [(torch.randn(dim, heads * d, generator=g, device="cuda") * dim ** -0.5).to(dt) for _ in range(4)]
        self.w_beta = (torch.randn(dim, heads, generator=g, device="cuda") * dim ** -0.5).to(dt)
        self.out = (torch.randn(heads * d, dim, generator=g, device="cuda") * (heads * d) ** -0.5).to(dt)

    def inputs(self, x):
        q, k, v, a = ((x @ w).view(-1, self.heads, 128) for w in self.w)
        return q, k, v, -0.1 * torch.sigmoid(a.float()), torch.sigmoid((x @ self.w_beta).float())

    def prefill(self, x, cu):
        o, self.state = kda.prefill(*self.inputs(x), cu, qk_l2norm=True)
        return o.flatten(1) @ self.out

    def step(self, x):
        return kda.decode_step(*self.inputs(x), self.state, qk_l2norm=True).flatten(1) @ self.out


class LatentLayer:
    """Queries, the joint latent projection, the up-projections of keys and values, and a paged cache."""

    def __init__(self, dim, heads, g, dt, pages, page, positions=4096):
        def normal(*shape, fan):
            return (torch.randn(*shape, generator=g, device="cuda") * fan ** -0.5).to(dt)
        self.heads, self.page, self.scale = heads, page, (N + P) ** -0.5
        self.w_q, self.w_kv = normal(dim, heads * (N + P), fan=dim), normal(dim, R + P, fan=dim)
        self.w_k, self.w_v = normal(heads, N, R, fan=R), normal(heads, R, N, fan=R)  # key, value up-projections
        self.norm = torch.ones(R, dtype=dt, device="cuda")
        self.out = normal(heads * N, dim, fan=heads * N)
        angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, P, 2, device="cuda", dtype=torch.float64) / P))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.cache = torch.zeros(pages, page, R + P, dtype=dt, device="cuda")
        self.workspace = kda.latent_decode_workspace_for(heads, kda._dtype_code(self.norm), "cuda")
        self.errors = torch.zeros(1, dtype=torch.int32, device="cuda")

    def prefill(self, x, cu, positions, slots):
        q = (x @ self.w_q).view(-1, self.heads, N + P)
        kv = x @ self.w_kv
        latent, k_pe = torch.empty_like(kv[:, :R]), torch.empty_like(kv[:, R:])
        kda.latent_append(kv[:, :R], kv[:, R:], self.cache, slots, norm_weight=self.norm, cos_sin=self.cos_sin,
                          positions=positions, q_pe=q[..., N:], latent_out=latent, k_pe_out=k_pe, errors=self.errors)
        k = (latent @ self.w_k.flatten(0, 1).T).view(-1, self.heads, N)
        v = (latent @ self.w_v.permute(1, 0, 2).flatten(1)).view(-1, self.heads, N)
        o, _ = kda.latent_prefill(q, k, k_pe, v, self.scale, cu, errors=self.errors)
        return o.flatten(1) @ self.out

    def step(self, x, positions, slots, table, lens):
        q = (x @ self.w_q).view(-1, self.heads, N + P)
        kv = x @ self.w_kv
        absorbed = torch.empty(x.shape[0], self.heads, R + P, dtype=x.dtype, device="cuda")
        absorbed[..., :R] = torch.bmm(q[..., :N].transpose(0, 1), self.w_k).transpose(0, 1)
        kda.latent_append(kv[:, :R], kv[:, R:], self.cache, slots, norm_weight=self.norm, cos_sin=self.cos_sin,
                          positions=positions, q_pe=q[..., N:], q_pe_out=absorbed[..., R:], errors=self.errors)
        o, _ = kda.latent_decode(absorbed, self.cache, table, lens, self.scale, workspace=self.workspace,
                                 errors=self.errors)
        return torch.bmm(o.transpose(0, 1), self.w_v).transpose(0, 1).flatten(1) @ self.out


def run(lens=(300, 77, 5), steps=4, dim=512, heads=4, dtype=torch.bfloat16, page=64, seed=0):
    """Prefills the prompts, generates `steps` tokens each (their inputs are random vectors), and returns the
    largest difference of the latent layer's step outputs from a prefill of everything, relative to the
    latter's largest value."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = len(lens)
    per_seq = -(-(max(lens) + steps) // page)
    first, second = KdaLayer(dim, heads, g, dtype), LatentLayer(dim, heads, g, dtype, n * per_seq, page)
    table = torch.randperm(n * per_seq, generator=g, device="cuda").int().view(n, per_seq)
    prompts = [torch.randn(l, dim, generator=g, device="cuda").to(dtype) for l in lens]
    tokens = torch.randn(steps, n, dim, generator=g, device="cuda").to(dtype)

    def slots_of(seq, pos):
        return table[seq, pos // page] * page + (pos % page).int()

    def packed(lengths):
        seq = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(lengths, device="cuda"))
        pos = torch.cat([torch.arange(l, device="cuda") for l in lengths])
        cu = torch.tensor([sum(lengths[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
        return cu, pos.int(), slots_of(seq, pos).int()

    cu, pos, slots = packed(lens)
    x = torch.cat(prompts)
    h = rms(x + first.prefill(x, cu))
    second.prefill(h, cu, pos, slots)
    inputs, outputs = [h], []  # the latent layer's
    held = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for t in range(steps):
        h = rms(tokens[t] + first.step(tokens[t]))
        y = second.step(h, held, slots_of(torch.arange(n, device="cuda"), held.long()).int(), table, held + 1)
        held += 1
        inputs.append(h)
        outputs.append(y)
    # the same inputs as one prefill
    ends = [sum(lens[:i + 1]) for i in range(n)]
    everything = torch.cat([torch.cat([inputs[0][e - l:e]] + [s[i:i + 1] for s in inputs[1:]])
                            for i, (l, e) in enumerate(zip(lens, ends))])
    longer = [l + steps for l in lens]
    cu2, pos2, slots2 = packed(longer)
    want = second.prefill(everything, cu2, pos2, slots2)
    rows = torch.tensor([[int(cu2[i + 1]) - steps + t for i in range(n)] for t in range(steps)], device="cuda")
    assert second.errors.item() == 0
    far = (torch.stack(outputs).float() - want[rows].float()).abs().max() / want[rows].float().abs().max()
    return far.item()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--prompts", type=int, nargs="+", default=[1500, 300, 77, 5])
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    far = run(tuple(a.prompts), a.steps, dim=2048, heads=a.heads)
    print(f"{len(a.prompts)} prompts, {a.steps} steps: the absorbed steps are within {far:.1e} of the expanded prefill")
