"""The prefix kernel's barriers with a ring of two tiles (keys and values as two parts of 128 columns),
explored on the CPU: two row tiles, both streams look at every tile, K always in the first stage
and V in the second."""
import pytest

import test_prefix_barriers_host as model


def test_the_ring_of_two_is_the_source_s():
    text = model.source()
    assert "SPLIT && D == 128 ? 2 : kRing" in text
    assert "const bool pair = SPLIT || " in text
    assert "const bool late = kRing == 4 && n >= 8;" in text
    assert "go_block = late ? 1 : 0, go_part = late ? 0 : 3" in text


@pytest.mark.parametrize("n", [1, 2, 3, 4, 7])
def test_no_order_of_events_is_stuck_or_early(monkeypatch, n):
    monkeypatch.setattr(model, "RING", 2)
    assert model.explore(True, n, model.start_waits(model.source(), n)) is None


def test_a_later_start_is_found_stuck_and_one_tile_early(monkeypatch):
    """Why the second stream does not start with the first one's second block, and why a single tile does not
    take turns: the exploration sees both."""
    monkeypatch.setattr(model, "RING", 2)
    start = model.start_waits(model.source(), 8)
    assert "stuck" in model.explore(True, 8, start)
    assert model.explore(False, 4, start) is not None
