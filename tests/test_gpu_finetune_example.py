"""The fine-tuning example end to end: block norms, QLoRA linears with 8-bit
checkpoints, token log probabilities and 8-bit AdamW in one training loop."""
import importlib.util
import os

import pytest
import torch

from tests._gpu import needs_gpu, say

pytestmark = [pytest.mark.gpu, needs_gpu]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location(
        "finetune_block", os.path.join(ROOT, "examples", "finetune_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_learns_and_answers(ex):
    say("[example] act8")
    model, losses, table = ex.train(vocab=1024, dim=256, ffn=704, batch=1024, steps=80)
    assert torch.isfinite(losses).all()
    assert float(losses[0]) > 6.0 and float(losses[-5:].mean()) < 0.6 * float(losses[0])
    ids, logp, entropy = ex.answer(model, torch.arange(200, device="cuda"), k=3)
    assert float((ids[:, 0].long() == table[:200]).float().mean()) > 0.5
    assert (logp[:, 0] >= logp[:, 1]).all() and (entropy > 0).all()


def test_checkpoints_in_8_bits_train_like_whole_activations(ex):
    """The same steps with x kept in bf16: the adapters' gradients differ by the
    checkpoint's rounding alone, so the losses stay close."""
    say("[example] act8 against bf16")
    a = ex.train(vocab=512, dim=256, ffn=704, batch=512, steps=15, act8=True)[1]
    b = ex.train(vocab=512, dim=256, ffn=704, batch=512, steps=15, act8=False)[1]
    assert float(a[0]) == float(b[0])
    assert float((a - b).abs().max()) < 0.05 * float(b[0])
