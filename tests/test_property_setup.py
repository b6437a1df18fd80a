"""The property tests draw fresh examples in every run, whatever the seed, and the suite needs no plugin to start."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(*args):
    return subprocess.run([sys.executable, "-m", "pytest", "-q", *args], cwd=ROOT, capture_output=True, text=True)


@pytest.mark.parametrize("seed", [2, 3, 5])
def test_the_2_4_round_trip_draws_enough_cases(seed):
    """With these seeds it failed a health check: too many of its draws were of other patterns."""
    got = run("tests/test_oracle_pins.py", "-k", "code6_round_trip_on_random", "--hypothesis-seed=%d" % seed)
    assert got.returncode == 0, got.stdout


def test_collection_without_the_hypothesis_plugin():
    got = run("-p", "no:hypothesispytest", "--collect-only", "tests/test_quant_scheme.py")
    assert got.returncode == 0, got.stdout + got.stderr
