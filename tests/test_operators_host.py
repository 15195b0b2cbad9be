"""Host side of the operators' Python entries (CPU): the first call from several
threads, and the index that the movers accept."""
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


def index(E=5, offsets=None, counts=True, rows=12):
    i32 = dict(dtype=torch.int32)
    d = dict(row_of=torch.zeros((4, 2), **i32), slot_of=torch.zeros(rows, **i32),
             offsets=torch.zeros(E + 1 if offsets is None else offsets, **i32))
    if counts:
        d["counts"] = torch.zeros(E, **i32)
    return d


def check(ix, rows=12):
    operators._load()
    return operators._sorted(ix, 64, torch.float32, torch.zeros(1), rows)


def test_the_rows_in_use_are_read_after_the_last_expert():
    _build.build()
    ix = index()
    assert check(ix).in_use == ix["offsets"].data_ptr() + 4 * 5
    ix = index(counts=False)
    assert check(ix).in_use == ix["offsets"].data_ptr() + 4 * 5
    ix = index(E=1)
    assert check(ix).in_use == ix["offsets"].data_ptr() + 4


@pytest.mark.parametrize("bad", [dict(offsets=9), dict(offsets=5), dict(offsets=1), dict(offsets=0), dict(offsets=0, counts=False),
                                 dict(offsets=1, counts=False)])
def test_offsets_of_another_length_are_refused(bad):
    """One entry after each expert's is where the rows in use stand."""
    with pytest.raises(ValueError):
        check(index(**bad))


def test_missing_offsets_are_refused():
    ix = index()
    del ix["offsets"]
    with pytest.raises(ValueError):
        check(ix)
