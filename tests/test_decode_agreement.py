"""What the program that compares drafted trees with the same tokens one by one takes for agreement."""
import pytest

torch = pytest.importorskip("torch")


def logits(*top):
    """Rows of 50 logits with the given largest ones; and the greedy tokens."""
    g = torch.Generator().manual_seed(1)
    rows = [torch.rand(50, generator=g) for _ in top]
    for row, t in zip(rows, top):
        row[t] = 3.0
    return list(top), rows


def agree(*a):
    from weight_quantized_decode_gb300.decode_block import agree as f
    return f(*a)


def test_the_same():
    t, rows = logits(4, 9, 2)
    assert agree(t, rows, t, rows)
    assert agree(t, rows, t, [r * (1 + 1e-3) for r in rows])
    assert agree(t, rows, t[:2], rows[:2])


@pytest.mark.parametrize("at", [0, 1, 2])
def test_another_token(at):
    t, rows = logits(4, 9, 2)
    said = list(t)
    said[at] = 20
    assert not agree(t, rows, said, [r * (1 + 1e-3) for r in rows])


@pytest.mark.parametrize("at", [0, 1, 2])
def test_rows_too_far_apart(at):
    t, rows = logits(4, 9, 2)
    seen = list(rows)
    seen[at] = rows[at] + 0.1 * torch.arange(50)
    assert not agree(t, rows, t, seen)
    seen[at] = rows[at].clone()
    seen[at][7] = float("nan")
    assert not agree(t, rows, t, seen)


def test_two_tokens_that_change_places():
    t, rows = logits(4, 9, 2)
    rows[1][30] = 2.999
    seen = [r.clone() for r in rows]
    seen[1][30] = 3.001
    said = [4, 30, 17]                       # behind them nothing is compared
    assert agree(t, rows, said, [seen[0], seen[1], 100 * seen[2]])
    rows[1][30] = 2.99                       # further apart than the rows are
    seen[1][30] = 2.99
    seen[1][0] += 0.001
    assert not agree(t, rows, said, seen)
