"""The sequence operators together with a dynamic table, as the example runs them."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_the_block_trains_and_serves():
    import sequence_block as ex
    losses, answer = ex.main(steps=8, samples=32, history=60, candidates=5)
    assert losses == sorted(losses, reverse=True) and losses[-1] < 0.98 * losses[0]
    assert answer.shape == (32, 1, ex.HEADS, ex.DIM // ex.HEADS) and bool(torch.isfinite(answer.float()).all())


def test_the_block_gradient_is_its_loss_difference():
    """The action vocabulary's gradient, through layer norm and attention, against the loss itself."""
    import sequence_block as ex
    block, batch = ex.Block(seed=3), ex.make_batch(16, 40, 4, 5)
    before = {k: v.clone() for k, v in block.dense.items()}

    def loss():
        out, _ = block.forward(batch, ex.recis.RECIS_GROUP_BY_OCCURRENCE)
        off = out.float() - batch["target"]
        return float(0.5 * (off * off).sum() / off.shape[0])

    loss()                                    # the items enter the table
    block.step(batch, lr=0.0)                 # nothing moves
    assert all(torch.equal(before[k], v) for k, v in block.dense.items())
    # with a step of 1 the weights move by the gradient (the table's own rows do not: lr 0 left them)
    block.dense = {k: v.clone() for k, v in before.items()}
    block.items.backward_update = lambda *a, **k: None
    block.step(batch, lr=1.0)
    grad = {k: before[k] - v for k, v in block.dense.items()}
    for name in ("hist_w", "hist_b", "cand_w", "cand_b"):
        way = grad[name] / grad[name].norm()
        h = 0.5   # bfloat16 activations: a step far above their rounding
        moved = []
        for sign in (1, -1):
            block.dense = {k: v.clone() for k, v in before.items()}
            block.dense[name] += sign * h * way
            moved.append(loss())
        slope = (moved[0] - moved[1]) / (2 * h)
        assert slope == pytest.approx(float(grad[name].norm()), rel=0.15), name


@pytest.mark.parametrize("name", ["actions", "categories"])
def test_the_vocabulary_gradients_are_the_loss_difference(name):
    """The two vocabularies' gradients, through layer norm and attention, along themselves against the difference
    quotient of the same loss in 64 bits.  The block rounds some 12 times to bfloat16 on the way there and back (2^-8
    each at most): 1/16 of the gradient's norm is more than they can move it together."""
    import sequence_block as ex
    block, batch = ex.Block(seed=4), ex.make_batch(16, 40, 4, 6)
    block.forward(batch, 0)                   # the items enter the table
    n, samples = batch["items"].numel(), 16
    res = ex.recis.LookupResult(n, samples)
    feature = ex.recis.DeviceFeature(batch["items"], batch["offsets"], slot=1,
                                     ops=ex.recis.RECIS_OP_HASH | ex.recis.RECIS_OP_MOD, mod=10**8)
    block.items.insert_find([feature], samples, res, flags=ex.recis.RECIS_FIND_ONLY)
    rows = torch.empty(n, ex.DIM, dtype=torch.bfloat16, device="cuda")
    block.items.forward(res, "none", rows)
    assert bool(rows.any())
    dense = {k: (v.bfloat16() if k in ("actions", "categories") else v).cpu().double() for k, v in block.dense.items()}
    rows, host = rows.cpu().double(), {k: v.cpu() if isinstance(v, torch.Tensor) else v for k, v in batch.items()}

    def loss(d):
        def norm(x, w, b):
            x = x - x.mean(-1, keepdim=True)
            return x / (x.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt() * d[w] + d[b]

        hist = norm(rows + ex.DIM**0.5 * d["actions"][host["actions"]], "hist_w", "hist_b")
        cand = norm(ex.DIM**0.5 * d["categories"][host["candidates"]], "cand_w", "cand_b")
        total = 0.0
        for b in range(samples):
            kv = hist[host["offsets"][b]:host["offsets"][b + 1]].view(-1, ex.HEADS, ex.DIM // ex.HEADS).transpose(0, 1)
            q = cand[b].view(-1, ex.HEADS, ex.DIM // ex.HEADS).transpose(0, 1)
            s = q @ kv.transpose(1, 2) * kv.shape[-1] ** -0.5
            out = (torch.softmax(s, -1) @ kv).transpose(0, 1) if kv.shape[1] else torch.zeros_like(q).transpose(0, 1)
            total += 0.5 * (out - host["target"][b].double()).pow(2).sum() / samples
        return float(total)

    before = block.dense[name].clone()
    block.items.backward_update = lambda *a, **k: None
    block.step(batch, lr=1.0)                 # the weights move by the gradient
    grad = (before - block.dense[name]).cpu().double()
    way, h = grad / grad.norm(), 2.0**-8
    slope = (loss({**dense, name: dense[name] + h * way}) - loss({**dense, name: dense[name] - h * way})) / (2 * h)
    assert slope == pytest.approx(float(grad.norm()), rel=1 / 16)
