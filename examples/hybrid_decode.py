"""Decode steps of a hybrid stack: recurrent layers (Gated DeltaNet) with an attention layer after
every third, one grouped-query and one over a latent cache in turn.

One step is one CUDA graph: kv_plan hands out the pages and slots of the step's tokens for all
attention layers, each of those appends its keys and values (or latent rows) and attends over its
pages, and the recurrent layers advance their states. Lengths, page counts and the free list stay
on the GPU and are updated in place, so the same graph is replayed step after step.

    python examples/hybrid_decode.py [--batch 64] [--prompt 1000] [--steps 200] [--layers 8]

Weights are random and projections are plain torch products: the point is how the calls go together.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import linear_attention_decode_gdn_gb300 as gdn  # noqa: E402

HEAD, LATENT, TAIL = 128, 512, 64


class HybridDecoder:
    def __init__(self, batch, heads=16, heads_kv=4, layers=8, page_size=64, max_len=4096, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.batch, self.heads, self.heads_kv, self.page_size = batch, heads, heads_kv, page_size
        width = heads * HEAD
        weight = lambda rows, cols: torch.randn(rows, cols, generator=g, device=device).mul_(rows ** -0.5).bfloat16()  # noqa: E731
        ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
        empty = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=device)  # noqa: E731
        self.kinds = [("attn" if i % 8 == 3 else "latent") if i % 4 == 3 else "gdn" for i in range(layers)]

        # the cache's bookkeeping, one for all attention layers
        max_pages = -(-max_len // page_size)
        pages = batch * max_pages
        self.length, self.held, self.table = ints(batch), ints(batch), ints(batch, max_pages)
        self.free_list, self.free_count = torch.arange(pages, dtype=torch.int32, device=device), ints(1) + pages
        self.cu_new = ints(batch + 1)
        self.slots = empty(batch, dtype=torch.int64)
        self.status = ints(1)
        self.num_pages = pages

        self.x, self.y = empty(batch, width), empty(batch, width)  # a step's input and output
        self.x.normal_(generator=g)
        self.dims = gdn.make_dims(batch, heads, HEAD, flags=gdn.QKV_BF16 | gdn.GATE_RAW, q_scale=HEAD ** -0.5)
        self.row = torch.arange(batch, dtype=torch.int32, device=device)
        self.layers = []
        for kind in self.kinds:
            layer = {"kind": kind}
            if kind == "gdn":
                layer["in"] = weight(width, 3 * width + 2 * heads)
                layer["out"] = weight(width, width)
                layer["state"] = gdn.Pools.allocate(self.dims).state
                layer["o"] = empty(batch, heads, HEAD, dtype=torch.float32)
            elif kind == "attn":
                layer["in"] = weight(width, (heads + 2 * heads_kv) * HEAD)
                layer["out"] = weight(width, width)
                layer["k"], layer["v"] = (torch.zeros(pages, page_size, heads_kv, HEAD, dtype=torch.bfloat16, device=device)
                                          for _ in range(2))
                layer["kv"] = gdn.make_paged_kv(layer["k"], layer["v"])
                layer["o"] = empty(batch, 1, heads, HEAD)
            else:  # absorbed queries straight from the input, values stay latent
                layer["in"] = weight(width, heads * (LATENT + TAIL) + LATENT + TAIL)
                layer["out"] = weight(heads * LATENT, width)
                layer["k"] = torch.zeros(pages, page_size, 1, LATENT + TAIL, dtype=torch.bfloat16, device=device)
                layer["kv"] = gdn.make_paged_kv(layer["k"], dv=LATENT)
                layer["o"] = empty(batch, 1, heads, LATENT)
            self.layers.append(layer)
        size = max([gdn.attn_workspace_bytes(x["kv"], batch, 1, heads) for x in self.layers if "kv" in x] + [16])
        self.workspace = empty(size, dtype=torch.uint8)
        self.graph = None

    def admit(self, lengths):
        """Stands in for prompts: the requests' lengths and their pages (whose rows stay zero)."""
        new = torch.tensor(lengths, dtype=torch.int32, device=self.length.device)
        slots = torch.empty(int(new.sum()), dtype=torch.int64, device=new.device)
        self._plan(new, slots)

    def _plan(self, new, slots):
        gdn.kv_plan(self.length, new, self.held, self.table, self.free_list, self.free_count, kv_len=self.length,
                    cu_new=self.cu_new, slot_map=slots, held_out=self.held, free_count_out=self.free_count,
                    page_size=self.page_size, num_pages=self.num_pages, status=self.status)

    def _recurrent(self, layer, x):
        B, H = self.batch, self.heads
        qkv, gates = (x @ layer["in"]).split([3 * H * HEAD, 2 * H], dim=1)
        q, k, v = qkv.contiguous().view(B, 3, H, HEAD).unbind(1)
        gates = gates.float()
        inputs = gdn.make_inputs(q=q.contiguous(), k=k.contiguous(), v=v.contiguous(), log_decay=(gates[:, :H] + 3).contiguous(),
                                 beta=gates[:, H:].contiguous(), slot=self.row)
        gdn.decode_dense(self.dims, inputs, layer["state"], layer["o"], self.status)
        return layer["o"].flatten(1).bfloat16()

    def _attention(self, layer, x):
        B, H, KV = self.batch, self.heads, self.heads_kv
        mixed = (x @ layer["in"]).view(B, H + 2 * KV, HEAD)
        layer["q"] = mixed[:, None, :H]
        gdn.kv_append(layer["kv"], mixed[:, H:H + KV], mixed[:, H + KV:], self.slots, status=self.status)
        gdn.attn_decode(layer["kv"], layer["q"], self.table, self.length, layer["o"], self.workspace, status=self.status)
        return layer["o"].view(B, H * HEAD)

    def _latent(self, layer, x):
        B, H, row = self.batch, self.heads, LATENT + TAIL
        mixed = x @ layer["in"]
        layer["q"] = mixed[:, :H * row].view(B, 1, H, row)
        new = mixed[:, None, H * row:]
        gdn.kv_append(layer["kv"], new[..., :LATENT], new[..., LATENT:], self.slots, status=self.status)
        gdn.latent_decode(layer["kv"], layer["q"], self.table, self.length, layer["o"], self.workspace, status=self.status)
        return layer["o"].view(B, H * LATENT)

    def eager(self):
        """One step: x -> y, every cache and state one token further."""
        run = {"gdn": self._recurrent, "attn": self._attention, "latent": self._latent}
        self._plan(None, self.slots)
        x = self.x
        for layer in self.layers:
            normed = (x.float() * torch.rsqrt(x.float().square().mean(1, keepdim=True) + 1e-6)).bfloat16()
            x = x + run[layer["kind"]](layer, normed) @ layer["out"]
        self.y.copy_(x)

    def capture(self):
        """Captures eager() (which has to have run once) for step()."""
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.eager()

    def step(self):
        if self.graph is None:
            self.eager()
        else:
            self.graph.replay()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--layers", type=int, default=8)
    a = ap.parse_args(argv)
    model = HybridDecoder(a.batch, layers=a.layers, max_len=a.prompt + a.steps + 8)
    model.admit([max(1, a.prompt - 7 * i) for i in range(a.batch)])
    model.eager()
    model.capture()
    model.step()
    torch.cuda.synchronize()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps):
        model.step()
    end.record()
    torch.cuda.synchronize()
    if model.status.item() != 0:
        raise SystemExit(f"device status {model.status.item():#x}")
    ms = begin.elapsed_time(end) / a.steps
    print(f"{a.batch} requests, {a.layers} layers ({', '.join(model.kinds)}): {ms * 1e3:.1f} us a step, "
          f"{a.batch / ms * 1e3:.0f} tokens/s, {int(model.length.max())} positions, {model.free_count.item()} pages free")


if __name__ == "__main__":
    main()
