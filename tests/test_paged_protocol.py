"""CPU tests of the order that the barriers of the attention kernel of many rows give (paged_protocol.py): whatever the warps'
speeds, no wait lasts, and every buffer holds what its reader asks for."""
import random

import pytest

import paged_protocol as pp


def draw(seed):
    r = random.Random(seed)
    items = [(r.random() < .5, r.choice((1, 1, 1, 2, 3, 5, r.randint(1, 12))), r.random() < .6) for _ in range(r.randint(1, 10))]
    return r.randint(2, 8), items, r.choice([None] + pp.NAMES)


@pytest.mark.parametrize("block", range(8))
def test_any_row_tiles_at_any_speeds(block):
    for seed in range(40 * block, 40 * block + 40):
        stages, items, slow = draw(seed)
        warps, flying = pp.run(seed, stages, items, pp.source_rules(), slow)
        assert flying is not None and all(w.ok for w in warps), (seed, items, slow)


def short_row_tiles(rules):
    """Narrow row tiles of one token tile one after the other, of which the second chain has nothing, with its issuing warp slow:
    the seeds of 60 at which some wait gave up."""
    late = []
    for seed in range(60):
        warps, flying = pp.run(seed, 6, [(False, 1, True)] * 6, rules, "issue 1")
        if flying is None or not all(w.ok for w in warps):
            late.append(seed)
    return late


def test_row_tiles_of_one_token_tile():
    assert short_row_tiles(pp.source_rules()) == []


def test_the_model_sees_a_wait_that_nothing_orders():
    """With a wait for queries that the chain does not use, their barrier goes on by two phases unseen."""
    assert short_row_tiles(dict(pp.source_rules(), queries_by_need=False))


def late_ends(rules, seeds):
    """A warp that stops, or a copy that lands, later than any wait lasts: the draws after which some warp never ended, or ended
    with a copy or a product of the block still on its way."""
    bad = []
    for seed in seeds:
        stages, items, _ = draw(seed)
        r = random.Random(seed)
        late = {"late_copy": r.randint(1, 40)} if r.random() < .3 else {"pause": (r.choice(pp.NAMES), r.randint(1, 60))}
        _, flying = pp.run(seed, stages, items, rules, **late)
        if flying != 0:
            bad.append((seed, late, flying))
    return bad


@pytest.mark.parametrize("block", range(6))
def test_all_warps_end_after_waits_that_gave_up(block):
    assert late_ends(pp.source_rules(), range(1000 * block, 1000 * block + 60)) == []


@pytest.mark.parametrize("rule", ["stand_in", "end_together"])
def test_the_model_sees_warps_that_never_meet_and_what_is_left_on_its_way(rule):
    assert late_ends(dict(pp.source_rules(), **{rule: False}), range(600))
