"""One attention layer of a target model around the verify step.

A batch of prompts enters (rope and append, prompt attention), then each
speculative step runs

    dspark_score_compact    budget and ragged packing of the drafts
    dspark_rope_append      the packed rows' keys and values into the paged cache
    dspark_step_attention   the packed rows over the cache
    dspark_verify           accept, resample, commit

on one stream without a host round trip.  The model is a toy (random embedding,
one attention layer, tied output); the shapes and calls are a real one's.

    python examples/target_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from confidence_driven_speculative_gb300 import binding  # noqa: E402


class Model:
    def __init__(self, V, d, Hq, Hkv, D, device, gen):
        n = lambda *s, std=1.0: (std * torch.randn(s, generator=gen, device=device)).to(torch.bfloat16)
        self.V, self.d, self.Hq, self.Hkv, self.D = V, d, Hq, Hkv, D
        self.embed = n(V, d)
        self.qkv = n(d, (Hq + 2 * Hkv) * D, std=d ** -0.5)
        self.out = n(Hq * D, d, std=(Hq * D) ** -0.5)
        self.freq = binding.rope_freq(D, 1.0e4, device=device)

    def project(self, ids):
        """q, k, v [rows, heads, D] of token ids: views of one product."""
        x = self.embed[ids.clamp(min=0).long()] @ self.qkv
        q, k, v = x.split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], dim=1)
        return q.unflatten(1, (-1, self.D)), k.unflatten(1, (-1, self.D)), v.unflatten(1, (-1, self.D))

    def logits(self, attended):
        return (attended.flatten(1) @ self.out) @ self.embed.T


def run(B=4, gamma=8, V=1024, d=256, Hq=8, Hkv=2, D=128, page=16, steps=3, prompt=(70, 3, 129, 40),
        device="cuda", seed=0):
    """Returns what the last step left: the attention call's inputs and output, and the lengths
    committed after each step."""
    gen = torch.Generator(device=device).manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=device)
    model = Model(V, d, Hq, Hkv, D, device, gen)
    lens = list(prompt[:B])
    max_pages = -(-(max(lens) + (steps + 1) * (gamma + 1)) // page)
    num_pages = B * max_pages
    cache = torch.zeros((2, num_pages, page, Hkv, D), dtype=torch.bfloat16, device=device)
    table = torch.randperm(num_pages, generator=gen, device=device).to(torch.int32).view(B, max_pages)
    common = dict(Hq=Hq, Hkv=Hkv, D=D, page_size=page, num_pages=num_pages, max_pages=max_pages, rot_dim=D)
    paged = dict(k_cache=cache[0], v_cache=cache[1], block_table=table, rope_freq=model.freq)

    # ---- the prompts enter -------------------------------------------------
    off = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), **i32)
    total = sum(lens)
    req = torch.repeat_interleave(torch.arange(B, device=device), torch.tensor(lens, device=device)).int()
    pos = torch.cat([torch.arange(n, device=device) for n in lens]).int()
    ids = torch.randint(0, V, (total,), generator=gen, **i32)
    h = binding.AttnBuffers(B=B, rows=total, q_max=max(lens), k_rot=True, **common)
    q, k, v = model.project(ids)
    h.bind(q=q, k=k, v=v, row_off=off, row_req=req, packed_pos=pos, **paged)
    binding.dspark_rope_append(h.attn)
    binding.dspark_prompt_attention(h.attn)
    last = model.logits(h.out[off[1:].long() - 1]).argmax(-1).int()  # each prompt's next token
    seq_lens = torch.tensor(lens, **i32)                            # tokens in the cache

    # ---- speculative steps ---------------------------------------------------
    rows = B * (gamma + 1)
    bufs = binding.StepBuffers(B, gamma, V, d, device=device)
    att = binding.AttnBuffers(B=B, rows=rows, q_max=gamma + 1, **common)
    lengths = [seq_lens.clone()]
    for step in range(steps):
        draft_logits = 2.0 * torch.randn((B, gamma, V), generator=gen, device=device)
        start = seq_lens.clone()  # verify commits into seq_lens
        bufs.bind({
            "draft_logits": draft_logits.to(torch.bfloat16), "hidden": torch.randn(
                (B, gamma, d), generator=gen, device=device).to(torch.bfloat16),
            "draft_tokens": draft_logits.argmax(-1).int(), "last_tokens": last, "seq_lens": start,
            "head_w": torch.randn(d, generator=gen, device=device) * d ** -0.5,
            "head_bias": torch.full((B,), 1.5, device=device),
            "sts_tau": torch.ones(gamma, device=device), "cost_c": 0.2, "cap_T": B * gamma // 2,
            "temperature": 1.0, "seed": step}, seq_lens_commit=seq_lens)
        binding.dspark_score_compact(bufs.step)
        q, k, v = model.project(bufs.packed_ids)
        att.bind(q=q, k=k, v=v, row_off=bufs.row_off, row_req=bufs.row_req,
                 packed_pos=bufs.packed_pos, seq_lens=start, **paged)
        binding.dspark_rope_append(att.attn)
        binding.dspark_step_attention(att.attn)
        bufs.bind_target(model.logits(att.out).contiguous())
        binding.dspark_verify(bufs.step)
        last = bufs.out_tokens.gather(1, bufs.accept_len[:, None].long())[:, 0].contiguous()
        lengths.append(seq_lens.clone())
    torch.cuda.synchronize()
    if bufs.device_status() or att.device_status() or h.device_status():
        raise RuntimeError("a kernel gave up on a wait")
    return {"q_rot": att.q_rot, "out": att.out, "cache": cache, "table": table, "start": start,
            "row_off": bufs.row_off, "lengths": lengths, "emitted": bufs.num_emitted, "scale": D ** -0.5}


if __name__ == "__main__":
    r = run()
    print("cached tokens after the prompts and each step:")
    for x in r["lengths"]:
        print("  ", x.tolist())
