"""Host side of the operators' Python entries (CPU): the first call from several
threads."""
import sys
import threading

import pytest
import torch

from mixture_experts_layer_sigmoid_gb300 import _build, operators


@pytest.fixture
def fresh(monkeypatch):
    """The module as before its first call."""
    _build.build()
    for name in ("_torch", "_lib", "_stream"):
        monkeypatch.setattr(operators, name, None)
    monkeypatch.setattr(operators, "_dtypes", {})


def test_a_second_thread_never_sees_half_of_the_first_call(fresh):
    """Stops before every line of the first call and looks as another thread would:
    where the library is set, all that a call uses besides it is set too."""
    seen = []

    def trace(frame, event, arg):
        if frame.f_code is operators._load.__code__:
            seen.append((operators._lib is None, operators._stream is None or operators._torch is None or not operators._dtypes))
            return trace
        return None

    def run():
        sys.settrace(trace)
        try:
            operators._load()
        finally:
            sys.settrace(None)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert len(seen) > 3 and operators._lib is not None and operators._stream is not None
    assert not any(missing and not before for before, missing in seen)
