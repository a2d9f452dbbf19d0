"""The example that runs scored routing and the adapters together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "adapted_layer.py")


def test_adapted_layer_example():
    spec = importlib.util.spec_from_file_location("adapted_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, loads, error = example.main()
    assert all(b < a for a, b in zip(losses[:5], losses[1:5])), losses
    assert losses[-1] < 0.7 * losses[0], losses
    # the served tokens (one in eight without an adapter, exact from the start)
    # are as near the target as the trained batch
    assert error < losses[0]
