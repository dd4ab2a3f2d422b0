"""The example runs the router, the experts, the shared projection and its adapters together."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapted_layer.py")
_spec = importlib.util.spec_from_file_location("adapted_layer", _PATH)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


@pytest.mark.parametrize("tokens", [384, 1536])
def test_finetuning_reduces_the_error(tokens):
    errors = [e for e, _ in example.finetune(tokens=tokens, steps=25)]
    assert errors[-1] < 0.8 * errors[0]


def test_decode_step_replays():
    eager, replayed = example.serve()
    assert all(torch.equal(a, b) for a, b in zip(eager, replayed))
    assert all(torch.isfinite(a).all() and a.abs().max() > 0 for a in eager)
