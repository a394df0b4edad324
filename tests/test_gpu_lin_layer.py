"""The example that runs linear attention and the norms around it together (it checks its own results)."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_attention_layer_example(dtype):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "linear_attention_layer.py")
    spec = importlib.util.spec_from_file_location("linear_attention_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    errors = mod.main(["--dtype", dtype, "--steps", "8"])
    parts = {"norm", "attention", "head norm", "sum", "next norm", "state"}
    assert set(errors) == {f"{of} {part}" for of in ("prompts", "tokens") for part in parts} | {"train s", "train y", "train state"} | {
        f"d {w}" for w in ("x", "states", "first", "w_in", "head", "w_out", "post", "pre")}
