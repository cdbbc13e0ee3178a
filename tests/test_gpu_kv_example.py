"""The serving example: all cache calls and the descriptor path together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_serving_example():
    spec = importlib.util.spec_from_file_location("kv_serving",
                                                  os.path.join(ROOT, "examples", "kv_serving.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    out = ex.main(steps=8)
    # Prompts of 45, 7 and 130 tokens, the last one branched; 8 steps, request 1
    # ends before the fifth, request 0 at the end.
    assert out["lens"] == [0, 0, 138, 138, 0, 0, 0, 0]
    # 138 tokens are five pages of 32: four full ones shared, the fifth of each its own.
    assert out["live"] == 6 and out["last"] == 5
    assert out["spilled"] == 2 and out["entries"] == 2      # 45 + 8 tokens
    assert out["finite"]
