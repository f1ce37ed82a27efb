"""paged_tables refuses outputs that lie over its inputs or over each other (no GPU needed: the
addresses are compared on the host and never followed)."""
import itertools

import pytest

import shape_driven_tile_gb300 as sdt
from shape_driven_tile_gb300 import paged

ARG = -10
BATCH, PAGES, FREE, SLOTS = 4, 10, 5, 6
SIZES = dict(lens=4 * BATCH, new_tokens=4 * BATCH, free_pages=4 * FREE, table=4 * BATCH * PAGES, kv_lens=4 * BATCH,
             starts=4 * BATCH + 4, used=4, slots=8 * SLOTS)
INPUTS = ("lens", "new_tokens", "free_pages")


def place():
    """Every buffer right behind the last one, at 8 bytes."""
    at, where = 0x10000, {}
    for name, size in SIZES.items():
        where[name] = at
        at += -(-size // 8) * 8
    return where


def call(where, stride=PAGES, batch=BATCH):
    rc = sdt.lib().paged_tables(paged._STEP.pack(*(where[n] for n in SIZES), batch, 16, PAGES, stride, FREE, SLOTS), None)
    return rc, sdt.lib().sdt_last_error().decode()


PAIRS = [(a, b) for a, b in itertools.combinations(SIZES, 2) if not {a, b} <= set(INPUTS)]


@pytest.mark.parametrize("a,b", PAIRS)
def test_overlaps_are_refused(a, b):
    step = 8 if "slots" in (a, b) else 4
    for x, y in ((a, b), (b, a)):
        for shift in {0, (SIZES[y] - 1) // step * step}:  # x at y's first and at y's last element
            where = place()
            where[x] = where[y] + shift
            rc, why = call(where)
            assert rc == ARG and "overlap" in why, (x, y, shift)


def test_lengths_in_place_are_refused():
    where = place()
    where["kv_lens"] = where["lens"]
    rc, why = call(where)
    assert rc == ARG and "lens and kv_lens overlap" in why


def test_overlap_with_a_wide_table_counts_its_rows_only():
    where = place()
    where["table"] = 0x80000
    wide = 4 * (PAGES + BATCH)  # bytes between rows: BATCH entries are free behind each
    for row in range(BATCH - 1):
        gap = 0x80000 + row * wide + 4 * PAGES
        for off, over in ((-4, True), (4, True)):
            rc, why = call({**where, "lens": gap + off}, stride=PAGES + BATCH)
            assert (rc == ARG and "overlap" in why) is over


TAKEN_AT = 0x40000


def call_taken(where, taken):
    rc = sdt.lib().paged_tables_taken(paged._STEP.pack(*(where[n] for n in SIZES), BATCH, 16, PAGES, PAGES, FREE, SLOTS), taken, None)
    return rc, sdt.lib().sdt_last_error().decode()


def test_the_place_overlaps_nothing():
    for name, size in SIZES.items():
        for shift in (0, size - 4, -4):
            rc, why = call_taken(place(), place()[name] + shift)
            assert rc == ARG and "overlap" in why
    assert call_taken(place(), None)[0] == -1 and call_taken(place(), TAKEN_AT + 2)[0] == -2


def test_lengths_in_place_with_a_place_in_the_list_are_exactly_the_same_buffer():
    where = place()
    where["kv_lens"] = where["lens"] + 4
    rc, why = call_taken(where, TAKEN_AT)
    assert rc == ARG and "overlap" in why
    where["kv_lens"] = where["lens"]
    where["starts"] = where["lens"]  # the other outputs still may not
    rc, why = call_taken(where, TAKEN_AT)
    assert rc == ARG and "overlap" in why
