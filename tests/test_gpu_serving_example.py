"""The serving example (examples/serve_looped_block.py): quantized linears,
cache and attention together.  A row's state after many single-token steps,
forks and evictions is that of one pass over the same tokens."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 4)])
def test_steps_and_one_pass_agree(lq, window, sinks):
    spec = importlib.util.spec_from_file_location("serve_looped_block", os.path.join(ROOT, "examples", "serve_looped_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    step, whole, used = example.run(window, sinks)
    # 8-bit activation codes: a code that falls the other way by the order of fp32
    # sums moves a group's product by 1/127 of its largest element; over four
    # blocks of residual width one such flip stays under a hundredth of the state
    assert float((step - whole).norm() / whole.norm()) < 1e-2
    assert all(after <= before for before, after in used)
    if window:
        assert used[-1][1] <= 5 * 5  # sinks' page, and the window's 24 tokens and the new one in at most 3; 5 rows
