"""Serve from a prefix that arrives compressed.

A context's K and V are compressed into range-coded streams (what a store would keep or a link
would carry), restored, written into the 4-bit paged cache of all layers, and then
tokens are decoded against it: each step writes the new token's K and V and attends, layer
by layer, in a captured graph. Queries, K and V of the new tokens are random here, in
place of a model's.

    python examples/serve_from_prefix.py [--layers 32] [--tokens 4096] [--steps 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from kv_cache_compression_cg_gb300 import cache4, codec, synth  # noqa: E402


def serve(layers=32, tokens=4096, steps=16, heads=32, kv_heads=8, dim=128, page=64, say=print):
    """-> largest error of the last token's attention against plain attention over the
    values the cache holds, relative to the weighted mean of |v|."""
    torch.manual_seed(0)
    C = kv_heads * dim
    work = synth.WORKLOADS["ctx4096"]
    k_host, v_host = synth.generate(synth.Workload("prefix", layers, tokens, C, work.chunk_tokens, work.bins_k[:layers], work.bins_v[:layers],
                                                   work.kind, work.seed, rho=work.rho, outlier_frac=work.outlier_frac, outlier_scale=work.outlier_scale))
    k, v = torch.from_numpy(k_host).cuda(), torch.from_numpy(v_host).cuda()

    # the prefix, through the codec
    cd = codec.Codec(layers, tokens, C, list(work.bins_k[:layers]), list(work.bins_v[:layers]), fmt=3)
    out = cd.compress(k, v)
    restored = torch.empty(layers, 2, tokens, C, dtype=torch.float16, device="cuda")
    cd.decompress_into(restored[:, 0], restored[:, 1])

    # into the cache: one sequence, room for its steps
    pages = -(-(tokens + steps) // page)
    cache = cache4.Cache4(layers, pages, page, kv_heads, dim, group=64)
    table = torch.randperm(pages, device="cuda").to(torch.int32).reshape(1, pages)
    kv_len = torch.tensor([tokens], dtype=torch.int32, device="cuda")
    prefix = cache4.Batch4(table, kv_len, torch.tensor([0, tokens], dtype=torch.int32, device="cuda"), rows=tokens)
    cache.write_layers(restored[:, 0], restored[:, 1], prefix)

    # a step of all layers, captured once: the batch's lengths are read on the device by each replay
    step = cache4.Batch4(table, kv_len)
    q = torch.randn(layers, 1, heads, dim, dtype=torch.float16, device="cuda")
    new = torch.randn(2, layers, 1, C, dtype=torch.float16, device="cuda")
    attended = torch.empty_like(q)

    def run():
        kv_len.add_(1)
        for layer in range(layers):
            cache.write(new[0, layer], new[1, layer], step, layer)
            cache.attend(q[layer], step, layer, out=attended[layer])

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    kept = []
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps):
        q.normal_()
        new.normal_()
        graph.replay()
        kept.append(new.clone())
    end.record()
    torch.cuda.synchronize()
    if int(cd.out.status.item()) or int(cd.dstatus.item()) or int(cache.status.item()):
        raise RuntimeError("a call raised a status flag")
    say(f"{layers} layers, {tokens} tokens: streams {out.total_bytes() / 1e6:.1f} MB, binary16 {restored.numel() * 2 / 1e6:.1f} MB, "
        f"4-bit pool {cache.nbytes / 1e6:.1f} MB; {start.elapsed_time(end) / steps * 1e3:.0f} us a token")

    # the last step against plain attention: over what the cache holds, and over the same tokens in binary16
    whole = cache4.Batch4(table, kv_len, torch.tensor([0, tokens + steps], dtype=torch.int32, device="cuda"), rows=tokens + steps)
    full = torch.cat([restored] + [n.transpose(0, 1) for n in kept], 2).float()

    def plain(k, v):
        kk, vv = (x.unflatten(-1, (kv_heads, dim)).repeat_interleave(heads // kv_heads, 2) for x in (k, v))
        p = torch.softmax(torch.einsum("lhd,lthd->lht", q[:, 0].float(), kk) * dim ** -0.5, -1)
        return torch.einsum("lht,lthd->lhd", p, vv), torch.einsum("lht,lthd->lhd", p, vv.abs())

    got = attended[:, 0].float()
    want, size = plain(*cache.read_layers(whole, dtype=torch.float32))
    off = float(((got - want).abs() / size).max())
    say(f"largest difference from plain attention over the cache's values: {off:.1e} of the weighted mean of |v|")
    fine, _ = plain(full[:, 0], full[:, 1])
    say(f"difference from attention over the same tokens in binary16: {float((got - fine).norm() / fine.norm()):.3f} in the 2-norm")
    return off


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=32)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    serve(a.layers, a.tokens, a.steps)
