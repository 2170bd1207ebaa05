"""Serving from the engine's own 16-bit pages, and offloading them through the codec.

A batch of sequences goes through one attention layer the way an engine runs it, on
vLLM's packed pages [block, head, token, 2 x head_dim]: the prompts are appended, their
keys and queries turned by their positions on the way, and attend; tokens are generated
one at a time, the step (append + attend) captured once as a CUDA graph and replayed
while lengths grow; drafted tokens are checked together and the rejected ones forgotten;
the first sequence's pages are encoded and sealed where they lie, restored into other
pages, and generation goes on over those.  Keys, values and queries are random
stand-ins for a model's projections.

    python examples/serve_cache16.py [--seqs 8] [--prompt 300] [--steps 64]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from kv_cache_page_gb300 import cache8, cache16, codec  # noqa: E402


def serve(seqs=8, prompt=300, steps=64, *, drafts=4, kv_heads=8, q_heads=32, head_dim=128, block_tokens=16, seed=0):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt, T = torch.bfloat16, block_tokens

    def projections(n):
        """Queries, keys and values of n tokens side by side, as one projection leaves them."""
        x = torch.randn(n, q_heads + 2 * kv_heads, head_dim, generator=g, device=dev).to(dt)
        return x[:, :q_heads], x[:, q_heads:q_heads + kv_heads], x[:, q_heads + kv_heads:]

    prompts = [max(1, prompt - 17 * s) for s in range(seqs)]
    width = -(-(max(prompts) + steps + drafts + 1) // T)
    blocks = (seqs + 1) * width  # the last `width` pages are where the restored sequence goes
    strides = (2 * kv_heads * T * head_dim, 2 * head_dim, 2 * T * head_dim)
    pages = torch.zeros(blocks, kv_heads, T, 2 * head_dim, dtype=dt, device=dev)
    cache = cache16.Cache16(dtype="bf16", head_dim=head_dim, num_kv_heads=kv_heads, num_q_heads=q_heads, block_tokens=T,
                            num_blocks=blocks, strides=strides)
    layer = cache16.Layer(pages[..., :head_dim], pages[..., head_dim:])
    rotation = cache8.Rotation.of(head_dim, width * T, device=dev)
    tables = torch.randperm(seqs * width, generator=g, device=dev).to(torch.int32).view(seqs, width)
    lens = torch.tensor(prompts, dtype=torch.int32, device=dev)
    errors = torch.zeros(seqs, dtype=torch.int32, device=dev)

    # the prompts, all at once
    rows = sum(prompts)
    cu = torch.zeros(seqs + 1, dtype=torch.int32, device=dev)
    cu[1:] = lens.cumsum(0)
    batch = cache8.Batch(tables, lens, cu, n_new=rows, max_new=max(prompts), max_len=max(prompts), errors=errors)
    workspace = torch.zeros(cache.attend_workspace(batch), dtype=torch.uint8, device=dev)  # for every batch of this cache
    q, k, v = projections(rows)
    turned, out = torch.empty(rows, q_heads, head_dim, dtype=dt, device=dev), torch.empty(rows, q_heads, head_dim, dtype=dt, device=dev)
    cache.append(layer, batch, k, v, rotation=rotation, q=q, q_out=turned)
    cache.attend(layer, batch, turned, out, workspace=workspace)

    # generation: one captured step, replayed
    step = cache8.Batch(tables, lens, max_new=1, max_len=width * T, errors=errors)
    q1, k1, v1 = projections(seqs)
    out1, lse1 = torch.empty(seqs, q_heads, head_dim, dtype=dt, device=dev), torch.empty(seqs, q_heads, device=dev)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cache.append(layer, step, k1, v1, rotation=rotation, q=q1, q_out=q1)
        cache.attend(layer, step, q1, out1, lse=lse1, workspace=workspace)

    def generate():
        lens.add_(1)
        for x, y in zip((q1, k1, v1), projections(seqs)):
            x.copy_(y)
        graph.replay()

    for _ in range(steps):
        generate()

    # drafted tokens, checked together; all but the first of each sequence are rejected: its length says so
    lens.add_(drafts)
    cu.copy_(drafts * torch.arange(seqs + 1, device=dev))
    check = cache8.Batch(tables, lens, cu, n_new=seqs * drafts, max_new=drafts, max_len=width * T, errors=errors)
    qd, kd, vd = projections(seqs * drafts)
    outd = torch.empty(seqs * drafts, q_heads, head_dim, dtype=dt, device=dev)
    cache.append(layer, check, kd, vd, rotation=rotation, q=qd, q_out=qd)
    cache.attend(layer, check, qd, outd, workspace=workspace)
    lens.sub_(drafts - 1)

    # offload of sequence 0 from the live pages, restored into others
    held = prompts[0] + steps + 1
    used = -(-held // T)
    store = codec.Codec(dtype="bf16", layout="packed", head_dim=head_dim, num_kv_heads=kv_heads, block_tokens=T,
                        num_layers=1, num_blocks=blocks, strides=strides, k_codec="fp8_dynamic", v_codec="fp8_dynamic")
    slot = store.segment_bytes(0)[0]
    here = tables[0, :used].tolist()
    there = [seqs * width + i for i in range(used)]
    descs = [codec.descriptors([(0, b, r, (2 * i + r) * slot) for i, b in enumerate(of) for r in range(2)], dev) for of in (here, there)]
    n = 2 * used
    slots = torch.empty(n * slot, dtype=torch.uint8, device=dev)
    status, result = torch.empty(n, dtype=torch.uint8, device=dev), torch.empty(n, dtype=torch.uint8, device=dev)
    headers = torch.empty(32 * n, dtype=torch.uint8, device=dev)
    store.encode_sealed([pages], descs[0], n, slots, slots.numel(), status, headers)
    store.decode_verified([pages], descs[1], n, slots, slots.numel(), headers, result)
    tables[0] = torch.arange(seqs * width, blocks, dtype=torch.int32, device=dev)
    generate()
    torch.cuda.synchronize()
    return {"out": out, "draft_out": outd, "draft_q": qd, "step_out": out1, "step_lse": lse1, "step_q": q1, "errors": errors,
            "pages": pages, "tables": tables, "lens": lens, "restored": int((result == codec.SEG_ENCODED).sum()), "segments": n,
            "rotation": rotation, "prompt_q": q, "prompt_turned": turned}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("seqs", 8), ("prompt", 300), ("steps", 64)):
        ap.add_argument("--" + name, type=int, default=value)
    r = serve(**vars(ap.parse_args()))
    assert not r["errors"].any()
    print("prompt rows %d, last step's lse %.3f .. %.3f, sequence 0: %d of %d segments restored"
          % (r["out"].shape[0], r["step_lse"].min(), r["step_lse"].max(), r["restored"], r["segments"]))
