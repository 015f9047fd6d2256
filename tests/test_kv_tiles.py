"""The calls of test_gpu_attend_tiles.py are launched with pairs of tiles (32 rows), by the
rule that the library uses (csrc/qmm_attend_shape.h). CPU only."""

import pytest

import test_gpu_attend_tiles as tiles
from test_kv_bounds_sanitized import driver, run  # noqa: F401  (driver: a fixture)

# the calls of the file (arguments of Pairs, hints), but for sizes that leave the launch as it is
CALLS = [(shape, {}) for shape in tiles.SHAPES]
CALLS += [(shape, {"window": w}) for shape in tiles.SHAPES for w in (5, 200, 40)]
for _dim in tiles.DIMS:
    CALLS += [(([9000, 200, 1], [20, 1, 1], 1, 1, _dim, 64), {"max_q": 20, "max_len": n})
              for n in (9000, tiles.LONG)]
    CALLS += [(([300, 1000], [50, 50], 2, 4, _dim, 16), {}),
              (([700], [150], 2, 4, _dim, 32), {}),
              (([330, 45], [20, 20], 2, 4, _dim, 64), {"window": 100}),
              (([400], [100], 2, 2, _dim, 32), {})]
    CALLS += [(([3000, 300], [100, 60], 2, 4, _dim, 32), {"max_q": n, "max_len": 3000})
              for n in (17, 33, 100)]
CALLS += [(([300], [20], 2, 2, 64, 64), {}), (([300], [20], 1, 4, 128, 16), {}),
          (([200], [40], 2, 4, 128, 32), {}), (([70], [70], 1, 2, 96, 16), {}),
          (([300, 200], [130, 130], 2, 1, 128, 16), {}),
          (([3000, 700], [60, 33], 2, 4, 128, 64), {"max_q": 60, "max_len": 3000})]


def launch(driver, args, **hints):
    s = tiles.Pairs(*args)
    return dict(zip(("tiles", "splits", "min_part", "rows", "waves", "few"),
                    map(int, run(driver, *tiles.sizes(s, **hints)).split())))


@pytest.mark.parametrize("call", range(len(CALLS)))
def test_pairs_of_tiles(driver, call):  # noqa: F811
    args, hints = CALLS[call]
    assert launch(driver, args, **hints)["rows"] == 32, (args, hints)


def test_numbers_of_parts(driver):  # noqa: F811
    """... among them one part, a few, and more than the few that a row's own threads join."""
    s = ([9000, 200, 1], [20, 1, 1], 1, 1, 128, 64)
    assert launch(driver, s, max_q=20, max_len=9000)["splits"] == 5
    assert launch(driver, s, max_q=20, max_len=tiles.LONG)["splits"] == 17
    assert launch(driver, tiles.SHAPES[0])["splits"] == 1
