"""The example that trains two tenants' adapters beside a packed projection by
distillation and serves them: the loss falls, and a request without an adapter
gets the projection's own result (asserted in the example)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_adapter_distillation_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapter_distillation.py")
    spec = importlib.util.spec_from_file_location("adapter_distillation", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    first, last = mod.main(steps=40, tokens=256, verbose=False)
    assert last < 0.7 * first, (first, last)
