"""The seeds of generated inputs are the same in every process (no GPU needed)."""

import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
KEYS = [(3, 40, 1, "layer", 0), (1, 2, 3), ("rms",)]


def _gen(*key):
    return hash(key) % (1 << 31)


@pytest.mark.parametrize("salt", ["1", "2"])
def test_seeds_do_not_depend_on_the_process(salt):
    here = [_gen(*k) for k in KEYS]
    code = f"import conftest; print([conftest.repeatable_hash(k) % (1 << 31) for k in {KEYS!r}])"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, PYTHONHASHSEED=salt, PYTHONPATH=HERE))
    assert r.stdout.strip() == str(here), r.stderr[-500:]
    assert here[1] == hash(KEYS[1]) % (1 << 31)
