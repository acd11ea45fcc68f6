"""Host test of the order in which the weighing kernel's product warps go through their
rings of key and query tiles (csrc/paged_rings.h, the code that the kernel runs):
barriers, copies, conversion and the tensor cores' queues are modelled, and roles
take turns at random, some of them slow.  No schedule may multiply a tile that is
not (all) there, or come to a standstill, whatever units of one and of two key
tiles follow one another."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kv_cache_quantization_turboquantrvq_gb300", "csrc")


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("rings") / "rings_harness")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-I", CSRC, os.path.join(ROOT, "tests", "rings_harness.cpp"), "-o", exe])
    return exe


# (key tiles, query tiles) of the units that a block takes one after another
PATTERNS = {
    "one then two": [(1, 1), (1, 1), (2, 1)],
    "short prompts": [(1, 1), (1, 1), (1, 1), (2, 1), (1, 1), (2, 1), (1, 1), (2, 2), (2, 1), (1, 1), (2, 1), (2, 1)],
    "two tiles": [(2, 1), (2, 3), (2, 2), (2, 1), (2, 5)],
    "one tile": [(1, 1), (1, 2), (1, 1), (1, 4), (1, 1), (1, 1)],
    "nothing between": [(1, 1), (2, 0), (1, 0), (2, 1), (1, 0), (1, 2), (2, 1), (1, 1), (2, 2)],
    "long": [(2, 9), (1, 1), (2, 1), (1, 7), (2, 2), (1, 1), (1, 1), (2, 1)],
}
PATTERNS.update({"random %d" % i: (lambda r: [(r.choice([1, 2]), r.choice([0, 1, 1, 1, 2, 3, 6])) for _ in range(20)])(random.Random(i))
                 for i in range(4)})


def _run(exe, cache, walk, units, runs):
    r = subprocess.run([exe, cache, walk, str(runs), "1"] + [str(x) for u in units for x in u], capture_output=True, text=True,
                       check=True)
    return [int(x) for x in r.stdout.split()]


@pytest.mark.parametrize("cache", ["16", "e4m3"])
@pytest.mark.parametrize("pattern", list(PATTERNS))
def test_every_tile_is_there_when_it_is_multiplied(harness, cache, pattern):
    units = PATTERNS[pattern]
    wrong, stuck, products = _run(harness, cache, "kernel", units, 500)
    assert (wrong, stuck) == (0, 0)
    assert products == sum(k * q for k, q in units)


@pytest.mark.parametrize("cache", ["16", "e4m3"])
def test_the_model_shows_wrong_orders(harness, cache):
    """A warp that steps over the other's tiles, and one that waits for them but is not waited for."""
    wrong, _, _ = _run(harness, cache, "skip", PATTERNS["short prompts"], 500)
    assert wrong > 0
    _, stuck, _ = _run(harness, cache, "wait", PATTERNS["short prompts"], 500)
    assert stuck > 0
