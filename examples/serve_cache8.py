"""Serving with the live 8-bit cache, and offloading what it holds.

A batch of sequences goes through one attention layer the way an engine runs
it: the prompts' K and V are written into 8-bit pages and their queries attend;
then tokens are generated one at a time, the step (write + attend) captured once
as a CUDA graph and replayed while lengths grow; finished sequences are read back
into 16-bit pages of the page codec's layout, which encodes and seals them for
offload.  Keys, values and queries are random stand-ins for a model's
projections.

    python examples/serve_cache8.py [--seqs 8] [--prompt 700] [--steps 64]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from kv_cache_page_gb300 import cache8, codec  # noqa: E402


def serve(seqs=8, prompt=700, steps=64, *, kv_heads=8, q_heads=32, head_dim=128, block_tokens=16, seed=0):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt, T = torch.bfloat16, block_tokens

    def draw(n, heads):
        return torch.randn(n, heads, head_dim, generator=g, device=dev).to(dt)

    # the engine's side: pages handed out as sequences grow, prompts of uneven length
    prompts = [max(1, prompt - 37 * s) for s in range(seqs)]
    width = -(-(max(prompts) + steps) // T)
    cache = cache8.Cache8(dtype="bf16", head_dim=head_dim, num_kv_heads=kv_heads, num_q_heads=q_heads,
                          block_tokens=T, num_blocks=seqs * width)
    layer = cache.new_layer(dev)
    tables = torch.randperm(seqs * width, generator=g, device=dev).to(torch.int32).view(seqs, width)
    lens = torch.tensor(prompts, dtype=torch.int32, device=dev)
    errors = torch.zeros(seqs, dtype=torch.int32, device=dev)

    # the prompts, all at once
    rows = sum(prompts)
    cu = torch.zeros(seqs + 1, dtype=torch.int32, device=dev)
    cu[1:] = lens.cumsum(0)
    batch = cache8.Batch(tables, lens, cu, n_new=rows, max_new=max(prompts), max_len=max(prompts), errors=errors)
    k, v, q = draw(rows, kv_heads), draw(rows, kv_heads), draw(rows, q_heads)
    out = torch.empty_like(q)
    workspace = torch.zeros(max(1, cache.attend_workspace(batch)), dtype=torch.uint8, device=dev)
    cache.write(layer, batch, k, v)
    cache.attend(layer, batch, q, out, workspace=workspace)

    # generation: one captured step, replayed
    step = cache8.Batch(tables, lens, max_new=1, max_len=max(prompts) + steps, errors=errors)
    k1, v1, q1 = (torch.empty(seqs, h, head_dim, dtype=dt, device=dev) for h in (kv_heads, kv_heads, q_heads))
    out1, lse1 = torch.empty_like(q1), torch.empty(seqs, q_heads, device=dev)
    work1 = torch.zeros(max(1, cache.attend_workspace(step)), dtype=torch.uint8, device=dev)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cache.write(layer, step, k1, v1)
        cache.attend(layer, step, q1, out1, lse=lse1, workspace=work1)
    for _ in range(steps):
        lens += 1
        k1.copy_(draw(seqs, kv_heads))
        v1.copy_(draw(seqs, kv_heads))
        q1.copy_(draw(seqs, q_heads))
        graph.replay()

    # offload of sequence 0: its tokens back in 16 bits, in whole pages of the codec's layout (an E4M3 value of
    # a page scale is exact in bf16; the codec's scale per token and head is another one, so its codes round these
    # values once more)
    n = prompts[0] + steps
    blocks = -(-n // T)
    pages = torch.zeros(2, blocks, T, kv_heads, head_dim, dtype=dt, device=dev)
    whole = cache8.Batch(tables[:1], lens[:1], torch.tensor([0, n], dtype=torch.int32, device=dev), n_new=n)
    cache.read(layer, whole, pages[0].view(-1, kv_heads, head_dim)[:n], pages[1].view(-1, kv_heads, head_dim)[:n])
    store = codec.Codec(dtype="bf16", layout="separate", head_dim=head_dim, num_kv_heads=kv_heads, block_tokens=T,
                        num_layers=1, num_blocks=blocks, strides=(T * kv_heads * head_dim, kv_heads * head_dim, head_dim),
                        k_codec="fp8_dynamic", v_codec="fp8_dynamic")
    slot = store.segment_bytes(0)[0]
    segs = [(0, b, r, (2 * b + r) * slot) for b in range(blocks) for r in range(2)]
    descs = codec.descriptors(segs, dev)
    slots = torch.empty(len(segs) * slot, dtype=torch.uint8, device=dev)
    status = torch.empty(len(segs), dtype=torch.uint8, device=dev)
    headers = torch.empty(32 * len(segs), dtype=torch.uint8, device=dev)
    store.encode_sealed([pages[0], pages[1]], descs, len(segs), slots, slots.numel(), status, headers)
    torch.cuda.synchronize()
    return {"out": out, "step_out": out1, "step_lse": lse1, "errors": errors, "pages": pages, "tokens": n,
            "encoded": int((status == codec.SEG_ENCODED).sum()), "segments": len(segs), "slot_bytes": slots.numel(),
            "cache_bytes_per_token": 2 * kv_heads * (head_dim + 4 / T)}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("seqs", 8), ("prompt", 700), ("steps", 64)):
        ap.add_argument("--" + name, type=int, default=value)
    r = serve(**vars(ap.parse_args()))
    assert not r["errors"].any()
    print("prompt rows %d, last step's lse %.3f .. %.3f, sequence 0: %d tokens read back, %d of %d segments encoded "
          "(%d slot bytes); the cache holds %.0f bytes a token"
          % (r["out"].shape[0], r["step_lse"].min(), r["step_lse"].max(), r["tokens"], r["encoded"], r["segments"],
             r["slot_bytes"], r["cache_bytes_per_token"]))
