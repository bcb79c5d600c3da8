"""The choice of tiles and runs of the int8 products and gradients (csrc/i8_plan.h) on the CPU,
compiled by itself (tests/sanitize/i8_plan_driver.cpp)."""
import os
import random
import shutil
import tempfile

import pytest

from tests.test_host_sanitizers import ROOT, SAN, _run

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")

RUNS = (1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16)
MEASURED = { # (parts, M, K, N): {tile: us with each of RUNS, weights from HBM; 0: not measured}
    (1, 4096, 4096, 16): {
        0: (89.2, 49.7, 37, 30, 26.2, 23.8, 22.7, 20.8, 19.8, 18.8, 19.1, 18.8),
        1: (67.2, 38.8, 29.3, 24, 21.4, 19.8, 19.1, 17.7, 16.9, 16.4, 16.9, 17.2),
        2: (56, 33, 25.3, 21, 18.8, 17.6, 17.1, 16.1, 17.5, 17, 17.2, 17.1)},
    (1, 4096, 4096, 64): {
        0: (89.9, 51.3, 38.6, 32.5, 29.1, 27.1, 26.3, 25.6, 24.8, 25, 25.5, 27.6),
        1: (67.8, 40.3, 30.9, 26.6, 24.1, 23, 22.8, 22.5, 22.3, 22.7, 23.7, 25.9),
        2: (56.3, 34.1, 26.4, 23.3, 21.4, 20.4, 20.6, 20.6, 22.6, 23.2, 23.9, 24.8)},
    (1, 4096, 4096, 130): {
        0: (90.4, 54, 42.3, 37, 34.1, 30.9, 30.8, 32.1, 29.2, 29.5, 29.6, 30.6),
        1: (68.8, 43.3, 34, 30.8, 28, 26.7, 26.2, 28.8, 29.7, 31.8, 33.4, 35.9),
        2: (56.2, 35, 34.2, 30.5, 27.6, 26.4, 26.2, 27.9, 31.1, 32.4, 33.3, 34.5)},
    (1, 4096, 4096, 256): {
        0: (94.7, 60, 49.4, 43.9, 40.5, 38.1, 38.1, 37.2, 37.3, 38.4, 40.5, 42.5),
        1: (70.5, 44.9, 36.4, 35, 31.4, 30.7, 31.1, 31.5, 41.3, 43.9, 46, 47.3),
        2: (56.2, 37.6, 36.5, 33.9, 31.5, 31.4, 37.7, 38, 41.4, 42.2, 48.5, 51.3)},
    (1, 4096, 4096, 512): {
        0: (95.3, 63.2, 52.4, 47.5, 45.9, 45.9, 47.8, 48.9, 66.3, 70.8, 75.1, 78.3),
        1: (68.7, 48.1, 42, 39.7, 54.4, 53.3, 54.2, 56.3, 67.5, 73.6, 0, 0),
        2: (56.8, 48.5, 43.3, 49.4, 54.6, 53, 60.1, 62.1, 68.9, 0, 0, 0)},
    (1, 4096, 4096, 1024): {
        0: (94.7, 69.1, 62.1, 63.5, 86.8, 85.9, 89, 91.9, 110.6, 121.5, 0, 0),
        1: (68.1, 58.1, 75.4, 71.8, 86.2, 88.3, 100.6, 0, 0, 0, 0, 0),
        2: (73.4, 79.5, 76.9, 85.6, 89.1, 0, 0, 0, 0, 0, 0, 0)},
    (1, 4096, 4096, 4096): {
        0: (121.6, 176.7, 208.1, 250.1, 0, 0, 0, 0, 0, 0, 0, 0),
        1: (151.1, 208.3, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0),
        2: (230.4, 251.5, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)},
    (1, 4096, 14336, 130): {
        0: (91.3, 61.3, 50.8, 46.6, 67.8, 64.4, 63.9, 62.1, 76.6, 79.1, 92.6, 0),
        1: (69.6, 49.7, 64.1, 57, 63.3, 63.5, 67.5, 0, 0, 0, 0, 0),
        2: (73, 51.8, 58.1, 57.7, 62.2, 64.7, 68, 0, 0, 0, 0, 0)},
    (1, 14336, 4096, 130): {
        0: (303.5, 160.2, 112.6, 88.6, 74.9, 65.7, 60.1, 55.3, 49.4, 46.9, 45.8, 45.5),
        1: (225.4, 122.3, 86.4, 68.8, 59, 52.7, 49, 45.7, 59.9, 58.2, 56.1, 54.7),
        2: (185.1, 100.9, 89.5, 71.1, 59.7, 55.8, 50.2, 47.2, 57.3, 59.1, 56.8, 55.5)},
    (1, 14336, 4096, 2048): {
        0: (312.4, 231.8, 279.8, 259.5, 300.6, 300.3, 329.8, 0, 0, 0, 0, 0),
        1: (255.4, 283.9, 297.1, 314, 0, 0, 0, 0, 0, 0, 0, 0),
        2: (455.6, 413.8, 396.8, 0, 0, 0, 0, 0, 0, 0, 0, 0)},
}


@pytest.fixture(scope="module")
def ask():
    """Queries to the driver's answers, pairs of numbers."""
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "i8_plan_driver")
        _run(["g++", "-std=c++17", *SAN, "-I" + os.path.join(ROOT, "quantized_unpack_q4_amd", "csrc"), "-o",
              exe, os.path.join(ROOT, "tests", "sanitize", "i8_plan_driver.cpp")], d)

        def asked(queries):
            path = os.path.join(d, "queries")
            with open(path, "w") as f:
                f.write("".join(" ".join(map(str, q)) + "\n" for q in queries))
            out = _run(["/bin/sh", "-c", "%s < %s" % (exe, path)], d).split("\n")
            assert "all checks passed" in out
            return [tuple(map(int, l.split())) for l in out[:len(queries)]]

        yield asked


def test_the_plan_is_near_the_best_measured(ask):
    """No choice is more than 8% from the best of its size: the rule once took 128 x 64 tiles for 512
    rows, the slowest of the three."""
    for size, plan in zip(MEASURED, ask([("grad", *s) for s in MEASURED])):
        us = {(t, r): v for t, row in MEASURED[size].items() for r, v in zip(RUNS, row) if v}
        assert us[plan] <= 1.08 * min(us.values()), (size, plan, us[plan], min(us.values()))


def test_runs_are_of_whole_stages(ask):
    """Every run has a stage."""
    rng = random.Random(5)
    sizes = [(rng.choice((1, 2)), *(int(2 ** rng.uniform(0, b)) for b in (21, 17, 21))) for _ in range(3000)]
    sizes = [(p, m, min(k, 131071), min(n, (1 << 37) // k)) for p, m, k, n in sizes]
    for (parts, M, K, N), (tile, runs) in zip(sizes, ask([("grad", *s) for s in sizes])):
        assert tile in range(3) and 1 <= runs <= min(16, parts * -(-M // 64)), (parts, M, K, N, tile, runs)


def test_product_tiles_at_their_measured_sizes(ask):
    """The sizes the rule's comment names, and the tile that was the fastest."""
    named = {(4096, 14336, 130, 0): 64, (4096, 14336, 1024, 0): 128, (4096, 14336, 4096, 0): 256,
             (1003, 2048, 77, 0): 64, (4096, 512, 1024, 0): 128, (28672, 4096, 64, 1): 64,
             (28672, 4096, 130, 1): 256}
    got = [t for t, _ in ask([("tile", *s, 256) for s in named])]
    assert got == list(named.values())


def test_every_form_of_the_tiles_is_tested(ask):
    """The sizes of tests/test_gpu_i8_tiles.py take the tiles they name, and leave none out."""
    from tests import test_gpu_i8_tiles as sizes

    def lie(rows, N): # of 256-row tiles on 256 CUs
        tiles = -(-rows // 256) * -(-N // 256)
        rest = tiles % 256
        cut = rest if rest and 2 * rest <= 256 else 0
        return "whole" if not cut else "halves" if cut == tiles else "both"

    for cases, rows in ((sizes.PRODUCTS, 1), (sizes.GATED, 2)):
        got = ask([("tile", rows * M, K, N, rows - 1, 256) for M, K, N in cases])
        for (M, K, N), (tile, _) in zip(cases, got):
            assert N > 16 and cases[M, K, N] == (tile, K % 128 == 0, lie(rows * M, N) if tile == 256 else None)
        forms = set(cases.values())
        assert forms == {(t, e, None) for t in (64, 128) for e in (False, True)} | {
            (256, e, l) for e in (False, True) for l in ("whole", "halves", "both")}
    for cases, parts in ((sizes.GRADIENTS, 1), (sizes.GATED_GRADIENTS, 2)):
        got = ask([("grad", parts, *s) for s in cases])
        for (M, K, N), (tile, runs) in zip(cases, got):
            assert cases[M, K, N] == (tile, M % 64 == 0, runs > 1), (M, K, N, tile, runs)
        assert set(cases.values()) == {(t, e, r) for t in range(3) for e in (False, True) for r in (False, True)}
