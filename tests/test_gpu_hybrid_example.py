"""The hybrid serving example, Linear layers over a pool of states and a Full layer over 8-bit pages in the same steps,
against the dense paths (both sides within 1e-2 of the formulas, so 2e-2 of each other)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_serving.py")


@pytest.mark.parametrize("sizes", [{}, {"prompts": (1, 1, 5), "decode": 4, "linear_layers": 1},
                                   {"prompts": (40, 300, 17), "d_h": 64, "chunk": 64, "page_size": 16},
                                   {"prompts": (1300, 2, 129), "d_h": 48, "heads": 2, "chunk": 2000, "decode": 3}])
def test_example(sizes):
    spec = importlib.util.spec_from_file_location("hybrid_serving", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert max(module.main(**sizes)) <= 2e-2
