"""The attention kernel's hand-overs between warps, copies and products, on a CPU model with
random interleavings: calls that run through, calls in which a wait runs out at any point, and
the mistakes that the kernel must not make, which the model has to find."""

from __future__ import annotations

from tests.attend_protocol import Fault, trial


def faults(seeds, **kw):
    found = set()
    for seed in seeds:
        try:
            trial(seed, **kw)
        except Fault as e:
            found.add(str(e))
    return found


def test_calls_run_through():
    assert not any(trial(seed, give_up=0.0) for seed in range(150))


def test_a_wait_that_runs_out_anywhere_ends_the_call_with_nothing_in_flight():
    gave_up = sum(trial(seed) for seed in range(1000))
    assert 500 < gave_up < 1000


def test_copies_and_products_are_waited_for_also_when_another_role_gives_up_later():
    found = faults(range(300), mistakes=("drain",))
    assert {"exit with copies in flight", "exit with products or commits in flight"} <= found


def test_a_stage_whose_products_are_not_issued_is_not_given_back():
    seeds = range(1530, 1960)
    assert not faults(seeds, deep=True)
    assert faults(seeds, deep=True, mistakes=("hand back",)) == {"copy into a stage that is being filled"}
