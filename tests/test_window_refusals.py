"""Host-side refusals of the attention side of a window (no GPU): the codes come
back before anything is enqueued."""

import ctypes
import random

from test_abi import FAKE, lib  # noqa: F401 (a fixture)
from test_window_abi import _attend, _cache


def _overlap(a, ld_a, b, ld_b, rows, width):
    """Whether two sets of rows share an element, by listing them."""
    mine = {a + i * ld_a + x for i in range(rows) for x in range(width)}
    return any(b + i * ld_b + x in mine for i in range(rows) for x in range(width))


def test_output_over_the_queries(lib):  # noqa: F811
    """Row sets that share an element with the queries are refused, at any strides."""
    width = 256  # 4 heads of 64
    rng = random.Random(5)
    refused = 0
    at = FAKE.value
    cases = [(256, 0, 256, 5), (256, 255, 256, 1), (512, 300, 512, 3), (256, 4 * 256, 256, 5),
             (600, 256, 300, 4), (1000, -255, 1000, 2)]
    cases += [(rng.randrange(256, 1200), rng.randrange(-2500, 2500), rng.randrange(256, 1200),
               rng.randrange(1, 9)) for _ in range(300)]
    for ld_q, off, ld_out, rows in cases:
        if not _overlap(0, ld_q, off, ld_out, rows, width):
            continue  # (would be enqueued)
        refused += 1
        out = ctypes.c_void_p(at + 2 * off)
        assert _attend(lib, _cache(), ld_q=ld_q, out=out, ld_out=ld_out, rows=rows) == -1, \
            (ld_q, off, ld_out, rows)
    assert refused > 100
    assert _attend(lib, _cache(), out=FAKE, rows=0) == 0  # no rows, nothing shared
