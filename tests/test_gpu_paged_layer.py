"""The paged-attention calls together, as examples/paged_layer.py uses them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_steps_of_any_size_give_what_one_step_gives():
    """The same tokens as whole prompts, chunks and single tokens.  Every value passes
    through four bf16 roundings (the q/k/v projection, the rotation, the attention's
    weights, its output), each up to 2^-8 of it, and the two runs may round each the
    other way; the output projection averages over the heads' columns, where a
    difference of 8 * 2^-8 = 0.03 of the rms in every one at once is the worst there
    can be.  A token at the wrong place or page shows as a difference near 1."""
    spec = importlib.util.spec_from_file_location("paged_layer", os.path.join(ROOT, "examples", "paged_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # columns are not all at their rms: the largest of 500 x 1024 values of unit rms is near 5
    assert m.run() <= 5 * 8 * 2.0 ** -8
