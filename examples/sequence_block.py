"""A sequence block on top of a dynamic table: candidates read a user's history.

    python examples/sequence_block.py [--steps 20] [--batch 256] [--history 1000]

Per step, on one GPU:
  1. the history's item ids are looked up in a dynamic table (gathered rows,
     packed by sample) and the embeddings of its actions -- a small fixed
     vocabulary, a plain [actions, dim] table -- are added;
  2. both the history and the candidates' category embeddings go through a
     layer norm;
  3. every candidate attends to its sample's history (ragged, from no item to
     `history`), 4 heads of 32;
  4. the loss (squared distance to a fixed target) goes back through all of it:
     the attention's gradients, layer norm's, the two vocabularies' by sorted
     tokens, and the dynamic table's own update.
`serve` answers one candidate a user from the trained parts.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dynamic_embedding_tables_amd import recis, sequence  # noqa: E402

DIM, HEADS = 128, 4
ACTIONS, CATEGORIES = 50, 2000


class Block:
    def __init__(self, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def table(rows):
            return torch.randn(rows, DIM, device="cuda", generator=gen) / math.sqrt(DIM)

        self.items = recis.Table(DIM, "bf16", "adagrad")
        # master weights in float32; the operators read them in bfloat16
        self.dense = {"actions": table(ACTIONS), "categories": table(CATEGORIES),
                      "hist_w": torch.ones(DIM, device="cuda"), "hist_b": torch.zeros(DIM, device="cuda"),
                      "cand_w": torch.ones(DIM, device="cuda"), "cand_b": torch.zeros(DIM, device="cuda")}
        self.error = torch.zeros(1, dtype=torch.int32, device="cuda")

    def forward(self, batch, flags):
        b, d = batch, self.dense
        feature = recis.DeviceFeature(b["items"], b["offsets"], slot=1, ops=recis.RECIS_OP_HASH | recis.RECIS_OP_MOD,
                                      mod=10**8)
        n, samples = b["items"].numel(), b["candidates"].shape[0]
        res = recis.LookupResult(n, samples)
        self.items.insert_find([feature], samples, res, flags=flags)
        rows = torch.empty(n, DIM, dtype=torch.bfloat16, device="cuda")
        self.items.forward(res, "none", rows)
        scale = math.sqrt(DIM)
        history = rows + sequence.embed(b["actions"], d["actions"].bfloat16(), scale=scale, error=self.error)
        wanted = sequence.embed(b["candidates"], d["categories"].bfloat16(), scale=scale, error=self.error)
        hist, hm, hr = sequence.layer_norm(history, d["hist_w"], d["hist_b"])
        cand, cm, cr = sequence.layer_norm(wanted, d["cand_w"], d["cand_b"])
        q = cand.view(samples, -1, HEADS, DIM // HEADS)
        kv = hist.view(n, HEADS, DIM // HEADS)
        packed = {"kv_offsets": b["offsets"], "max_kv_len": b["longest"], "error": self.error}
        out, lse = sequence.cross_attention(q, kv, kv, return_lse=True, **packed)
        return out, (res, history, hm, hr, wanted, cm, cr, q, kv, packed, lse, scale)

    def step(self, batch, lr):
        out, (res, history, hm, hr, wanted, cm, cr, q, kv, packed, lse, scale) = self.forward(
            batch, recis.RECIS_GROUP_BY_OCCURRENCE)
        off = out.float() - batch["target"]
        loss = 0.5 * (off * off).sum() / off.shape[0]
        dq, dk, dv = sequence.cross_attention_backward((off / off.shape[0]).bfloat16(), q, kv, kv, out, lse, **packed)
        d = self.dense
        dhist, dhw, dhb = sequence.layer_norm_backward((dk + dv).view(history.shape), history, hm, hr, d["hist_w"])
        dcand, dcw, dcb = sequence.layer_norm_backward(dq.view(wanted.shape), wanted, cm, cr, d["cand_w"])
        grads = {"hist_w": dhw, "hist_b": dhb, "cand_w": dcw, "cand_b": dcb,
                 "actions": sequence.embed_backward(batch["actions"], dhist, ACTIONS, scale=scale, dtype=torch.float32),
                 "categories": sequence.embed_backward(batch["candidates"], dcand, CATEGORIES, scale=scale,
                                                       dtype=torch.float32)}
        self.items.backward_update(res, "none", dhist, "bf16", lr=lr)
        for name, g in grads.items():
            d[name] -= lr * g
        return loss

    def serve(self, batch):
        """One candidate a user against the table as it is (no insert)."""
        one = dict(batch, candidates=batch["candidates"][:, :1].contiguous())
        return self.forward(one, recis.RECIS_FIND_ONLY)[0]


def make_batch(samples, history, candidates, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens = torch.randint(0, history + 1, (samples,), device="cuda", generator=gen)
    offsets = torch.zeros(samples + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = lens.cumsum(0)
    n = int(offsets[-1])

    def ids(size, most):   # few of them often
        return (torch.rand(size, device="cuda", generator=gen) ** 4 * most).long()

    return {"items": ids((n,), 10**7), "actions": ids((n,), ACTIONS), "offsets": offsets, "longest": history,
            "candidates": ids((samples, candidates), CATEGORIES),
            "target": torch.randn(samples, candidates, HEADS, DIM // HEADS, device="cuda", generator=gen) * 0.1}


def main(steps=20, samples=256, history=1000, candidates=20, lr=0.01):
    block, batch = Block(), make_batch(samples, history, candidates, 1)
    losses = []
    for i in range(steps):
        losses.append(float(block.step(batch, lr)))
        if i % 5 == 0 or i == steps - 1:
            print(f"step {i}: loss {losses[-1]:.4f}", flush=True)
    answer = block.serve(batch)
    sequence.check(block.error)
    block.items.check()
    print("served", tuple(answer.shape), "from", int(block.items.stats().keys), "items", flush=True)
    return losses, answer


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--batch", type=int, default=256)
    p.add_argument("--history", type=int, default=1000)
    a = p.parse_args()
    main(a.steps, a.batch, a.history)
