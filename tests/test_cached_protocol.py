"""The barriers of the attention over a paged cache under random timings (CPU): tasks of few rows, of one tile and of
pairs in any order, with warps that have no step in some of them, must never pass a phase that is not theirs, meet a
tile or a state of another, or stop.  Each of the two waits that keep the tasks of few rows apart, and the even number
of stages, is shown to be needed."""
import random

import pytest

from cached_protocol_model import FEW, PAIR, SINGLE, ProtocolError, random_tasks, simulate


@pytest.mark.parametrize("part", range(6))
def test_random_tasks(part):
    for seed in range(part, 900, 6):
        simulate(random_tasks(random.Random(seed)), seed)


@pytest.mark.parametrize("tasks", [[(SINGLE, 1)] * 20 + [(FEW, 3)] * 3, [(FEW, 1), (SINGLE, 1), (FEW, 5)] * 6,
                                   [(FEW, 9)] * 20, [(SINGLE, 2), (SINGLE, 1)] * 10 + [(PAIR, 3)], [(FEW, 1)] * 40])
def test_tasks_that_leave_warps_without_a_step(tasks):
    for seed in range(60):
        simulate(tasks, seed)


@pytest.mark.parametrize("broken", [dict(passed=False), dict(fews_over=False), dict(stages=3)])
def test_the_model_catches_what_the_kernel_must_not_do(broken):
    caught = 0
    for seed in range(400):
        try:
            simulate(random_tasks(random.Random(seed)), seed, **broken)
        except ProtocolError:
            caught += 1
    assert caught > 0
