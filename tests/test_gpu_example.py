"""What the example's block learns with."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_example_steps_only_what_it_has_the_gradient_of():
    """The gate's gradient is whole; the norm's weight also acts through the
    experts, of whose gradient the block has nothing, so it stays."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    blocks = []

    class Block(mod.Block):
        def __init__(self, *args, **kw):
            super().__init__(*args, **kw)
            blocks.append((self, self.gate.clone(), self.norm.clone()))
    mod.Block = Block
    losses = mod.main(steps=10)
    (block, gate, norm), = blocks
    assert not torch.equal(block.gate, gate) and torch.equal(block.norm, norm)
    assert losses[-1] < losses[0]
