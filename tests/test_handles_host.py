"""CPU: what the binding takes for a handle (no GPU)."""
import ctypes as C
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pa():
    subprocess.run([sys.executable, os.path.join(ROOT, "windowed_prefill_attention_gb300", "build.py")], check=True,
                   capture_output=True)
    import windowed_prefill_attention_gb300 as mod
    return mod


@pytest.mark.parametrize("h", (None, 0, C.c_void_p()), ids=("None", "0", "null"))
def test_destroying_no_handle_does_nothing(pa, h):
    pa.pa_destroy(h)


@pytest.mark.parametrize("form", (C.c_void_p, int), ids=("c_void_p", "int"))
def test_a_handle_is_a_pointer_or_its_address(pa, monkeypatch, form):
    class Library:
        destroyed = []

        def pa_destroy(self, h):
            self.destroyed.append(h)
    monkeypatch.setattr(pa, "_lib", Library())
    monkeypatch.setitem(pa._geometry, 4096, (8, 2, 10, 10))
    h = form(4096)
    assert pa._geometry_of(h)[:4] == (8, 2, 10, 10)
    pa.pa_destroy(h)
    assert Library.destroyed == [h] and 4096 not in pa._geometry
    for gone in (h, None, 0, C.c_void_p(), "handle", []):
        with pytest.raises(ValueError):
            pa._geometry_of(gone)
