"""The paged serving example against the dense path (both within 1e-2 max |I| of the formula, so 2e-2 of each other)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_serving.py")


@pytest.mark.parametrize("sizes", [{}, {"prompts": (1, 1, 5), "decode": 0}, {"prompts": (40, 300), "d_h": 60,
                                                                          "chunk": 64, "page_size": 16},
                                   {"prompts": (513, 2, 129), "d_h": 128, "heads": 2, "decode": 3}])
def test_example(sizes):
    spec = importlib.util.spec_from_file_location("paged_serving", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module.main(**sizes) <= 2e-2
