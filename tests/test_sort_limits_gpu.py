"""The token sort next to its limits: T k and rows just below 2^31, where a sum of
a few more no longer fits 32 bits. One value wide, so that it fits the device;
compared exactly, a stretch at a time."""
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu

PART = 1 << 27


def need(gb):
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB")


def parts(n):
    for lo in range(0, n, PART):
        yield lo, min(n, lo + PART), torch.arange(lo, min(n, lo + PART), device="cuda")


def filled(n, dtype, value):
    """n values, a stretch at a time: value(positions)."""
    t = torch.empty(n, dtype=dtype, device="cuda")
    for lo, hi, at in parts(n):
        t[lo:hi] = value(at).to(dtype)
    return t


def same(t, value):
    return all(bool((t[lo:hi] == value(at).to(t.dtype)).all()) for lo, hi, at in parts(t.numel()))


@pytest.mark.parametrize("T,k", [((1 << 31) - 3, 1), ((1 << 31) // 4 - 1, 4), ((1 << 31) - 32, 1), ((1 << 31) - 31, 1)])
def test_index_of_most_slots(T, k):
    need(60)
    n, E = T * k, 3
    topk = filled(n, torch.int32, lambda i: i % E).view(T, k)
    ix = moe.sort_index(topk, E)
    counts = [n // E + (e < n % E) for e in range(E)]
    starts = torch.tensor([0, counts[0], counts[0] + counts[1]], device="cuda")
    assert ix["counts"].tolist() == counts and ix["offsets"].tolist() == [0, *torch.tensor(counts).cumsum(0).tolist()]
    assert same(ix["row_of"].view(-1), lambda i: starts[i % E] + i // E)
    # rows of one expert are its slots in order
    expert = lambda r: (r >= starts[1]).long() + (r >= starts[2]).long()  # noqa: E731
    assert same(ix["slot_of"], lambda r: (r - starts[expert(r)]) * E + expert(r))


@pytest.mark.parametrize("n,E", [((1 << 31) - 7, 1), ((1 << 31) - 52, 16)])
def test_padding_up_to_the_last_row(n, E):
    """The last segment's padding ends four rows below 2^31; the others hold one slot."""
    need(60)
    topk = filled(n, torch.int32, lambda i: i.clamp_max(E - 1)).view(n, 1)
    ix = moe.sort_index(topk, E, 4)
    rows, last = (1 << 31) - 4, 4 * (E - 1)
    assert ix["slot_of"].numel() == rows and ix["counts"].tolist() == [1] * (E - 1) + [n - E + 1]
    assert ix["offsets"].tolist() == [*range(0, last + 1, 4), rows]
    assert same(ix["row_of"].view(-1), lambda i: torch.where(i < E - 1, 4 * i, last + i - (E - 1)))
    slot = lambda r: torch.where(r < last, torch.where(r % 4 == 0, r // 4, -1), r - last + (E - 1))  # noqa: E731
    assert same(ix["slot_of"], lambda r: torch.where(slot(r) < n, slot(r), -1))


@pytest.fixture(scope="module")
def moved():
    """T tokens of one value, every seventh slot dropped, its row padding."""
    need(90)
    T = (1 << 31) - 3
    live = lambda i: i % 7 != 0  # noqa: E731
    minus = lambda i: torch.where(live(i), i, torch.full_like(i, -1))  # noqa: E731
    index = dict(row_of=filled(T, torch.int32, minus).view(T, 1), slot_of=filled(T, torch.int32, minus),
                 offsets=torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                 counts=torch.tensor([T], dtype=torch.int32, device="cuda"))
    x = filled(T, torch.bfloat16, lambda i: 1 + i % 251).view(T, 1)
    kept = lambda i: torch.where(live(i), 1 + i % 251, torch.zeros_like(i))  # noqa: E731
    yield T, index, x, kept
    index.clear()
    del x
    torch.cuda.empty_cache()


def test_most_tokens_out_and_back(moved):
    T, index, x, kept = moved
    Xp = moe.sort_rows(x, index, out=torch.full_like(x, 7.0))
    assert same(Xp.view(-1), kept)
    assert same(moe.unsort_rows(Xp, index).view(-1), kept)


def test_gradient_of_most_tokens(moved):
    T, index, x, kept = moved
    rows, dg = moe.unsort_rows_backward(x, x, index)
    assert same(rows.view(-1), kept)
    assert same(dg.view(-1), lambda i: kept(i) ** 2)


def test_gradient_of_most_tokens_without_the_gates(moved):
    T, index, x, kept = moved
    rows, none = moe.unsort_rows_backward(x, x, index, want_dgates=False)
    assert none is None and same(rows.view(-1), kept)
