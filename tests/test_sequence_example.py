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
