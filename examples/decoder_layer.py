"""One decoder layer served with the library: prefill, then decode steps.

The attention half (rotary positions, the paged 8-bit cache, attention over
it) and the routed MoE with a LoRA adapter for each sequence, as a server
would call them.  Weights are random; the projections around attention are
plain matrix products.  The same tokens once as one prompt and once as a
shorter prompt plus decode steps have to give the same layer output up to
rounding, which main() checks.

    python examples/decoder_layer.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import moe_lora_expert_gb300 as m  # noqa: E402


class DecoderLayer:
    """Hidden size H, Hq query heads on Hkv key heads of D, E experts."""

    def __init__(self, H=1024, Hq=16, Hkv=4, D=64, E=16, I=256, top_k=4, adapters=2, rank=8, max_positions=4096,
                 num_pages=64, page_size=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape, std=0.02):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.w_qkv, self.w_out, self.w_router = w(H, (Hq + 2 * Hkv) * D, std=0.05), w(Hq * D, H), w(H, E)
        self.moe = m.MoeLoraLayer(w(E, 2 * I, H), w(E, H, I), top_k, w(adapters, E, rank, H), w(adapters, E, 2 * I, rank),
                                  w(adapters, E, rank, I), w(adapters, E, H, rank), scaling=2.0)
        # a context stretched four times past the trained 1024 positions
        self.cos_sin = m.rope_table(max_positions, D, scaling={"kind": "yarn", "factor": 4.0, "original": 1024}, device="cuda")
        self.cache = m.PagedKVCache.create(num_pages, Hkv, page_size, D)

    def forward(self, x, adapter, block_table, seq_lens, cu_q=None, max_q_len=None):
        """x [N, H]: the new tokens, sequence after sequence; adapter [N]."""
        N = x.shape[0]
        qkv = (x @ self.w_qkv).view(N, self.Hq + 2 * self.Hkv, self.D)
        q, k, v = qkv.split([self.Hq, self.Hkv, self.Hkv], dim=1)             # strided views, taken as they are
        q = self.cache.append(k, v, block_table, seq_lens, cu_q=cu_q, max_q_len=max_q_len, q=q, cos_sin=self.cos_sin)
        a = self.cache.attend(q, block_table, seq_lens, cu_q=cu_q, max_q_len=max_q_len)
        x = x + a.view(N, -1) @ self.w_out
        return x + self.moe.forward(x, (x @ self.w_router).float(), adapter)


def main(prompts=(37, 150), steps=5):
    layer = DecoderLayer()
    B, P = len(prompts), layer.cache.page_size
    longest = max(prompts) + steps
    width = -(-longest // P)
    pages = torch.randperm(2 * B * width)[:2 * B * width].to(torch.int32).cuda()
    assert pages.numel() <= layer.cache.num_pages
    whole_table, step_table = pages.view(2, B, width)[0].contiguous(), pages.view(2, B, width)[1].contiguous()
    g = torch.Generator(device="cuda").manual_seed(1)
    H = layer.w_qkv.shape[0]
    tokens = [torch.randn((n + steps, H), generator=g, device="cuda").to(torch.bfloat16) for n in prompts]
    adapter = [torch.full((n + steps,), b - 1, dtype=torch.int32, device="cuda") for b, n in enumerate(prompts)]   # -1: none

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def run(lens, table):
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        return layer.forward(torch.cat([t[:n] for t, n in zip(tokens, lens)]), torch.cat([a[:n] for a, n in zip(adapter, lens)]),
                             table, ints(lens), cu_q=ints(cu), max_q_len=max(lens)), cu

    whole, cu = run([n + steps for n in prompts], whole_table)
    run(list(prompts), step_table)
    worst = 0.0
    for i in range(steps):
        x = torch.stack([t[n + i] for t, n in zip(tokens, prompts)])
        out = layer.forward(x, ints([b - 1 for b in range(B)]), step_table, ints([n + i + 1 for n in prompts]))
        want = torch.stack([whole[cu[b] + n + i] for b, n in enumerate(prompts)])
        worst = max(worst, float((out.float() - want.float()).norm() / want.float().norm()))
    status = [layer.cache.device_status(), layer.moe.device_status()]
    print(f"{B} prompts {tuple(prompts)}, {steps} decode steps: relative difference to one prefill {worst:.2e}, status {status}")
    return worst, status


if __name__ == "__main__":
    worst, status = main()
    sys.exit(0 if worst < 2e-2 and status == [0, 0] else 1)
