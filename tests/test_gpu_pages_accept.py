"""Accepted rows in states where sequences share their last page: what adds nothing is no fault."""
import random

import pytest

from test_gpu_pages import BF, FP, Both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("tokens", [5, 16, 128, 130])
def test_a_fork_that_adds_nothing(lib, page, tokens):
    """Two sequences on the same pages, the last one partly filled or full: a step without a row for either of them, then for
    one of them.  The other's reserve is left out, as nothing is to be written."""
    x = Both(1, 20, page, 2, 2, 10)
    x.reserve([tokens, 0])
    x.append([tokens, 0])
    x.accept([tokens, 0])
    x.select([0, 0])
    x.accept([0, 0])
    x.accept([0, 0], [[3], [0]])
    x.reserve([0, 2])
    x.append([0, 2])
    x.accept([0, 2])
    x.accept([0, 0])


def test_rows_of_shared_pages_still_count_as_a_fault(lib):
    """Sequences that hold the page too: one that would add a row, one that adds none."""
    x = Both(1, 20, 16, 1, 3, 4)
    x.reserve([21, 0, 0])
    x.accept([21, 0, 0])
    x.select([0, 0, 0])
    x.accept([0, 1, 0])
    x.accept([0, 0, 0])
    x.accept([-1, 0, 0])


# lives whose calls all differ: one seed a life
LIVES = [(16, 2, BF, "apart"), (16, 1, FP, "fused"), (32, 1, BF, "heads"), (64, 3, FP, "tokens"), (128, 1, BF, "apart")]


@pytest.mark.parametrize("seed", range(20))
def test_lives_of_forks(lib, seed):
    """Random steps of sequences that fork, stay, go on and end; those that would break a rule are part of them."""
    page, h, dtype, form = LIVES[seed % len(LIVES)]
    x = Both(2, 41, page, h, 5, 9, dtype, form, seed=1000 + seed)
    r = random.Random(1000 + seed)
    for step in range(40):
        some = [r.choice([0, 0, 1, r.randint(0, 2 * page)]) for _ in range(5)]
        op = r.choice(["step", "step", "accept", "path", "select", "select", "trim", "compact"])
        if op == "step":
            x.reserve(some)
            x.append(some, layer=r.choice([None, 0, 1]))
            x.accept([n if r.random() < 0.8 else r.randint(0, n) for n in some])
        elif op == "accept":
            x.accept(some)
        elif op == "path":
            x.accept([r.choice([0, r.randint(0, 6)]) for _ in range(5)], [sorted(r.sample(range(30), 6)) for _ in range(5)])
        elif op == "select":
            x.select([r.choice([b, b, r.randrange(5), r.randrange(5), -1 if r.random() < 0.3 else b]) for b in range(5)])
        elif op == "trim":
            x.trim([r.choice([-1, -1, -1, 0, r.randint(0, 4 * page)]) for _ in range(5)])
        else:
            x.compact()
