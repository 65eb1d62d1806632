import os
import sys
import zlib

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: takes more than a few seconds on the CPU")


def repeatable_hash(key):
    """hash(key), but for keys with strings, whose hash differs from process to process."""
    return zlib.crc32(repr(key).encode()) if "'" in repr(key) else hash(key)


@pytest.fixture(autouse=True)
def _inputs_of_every_run_alike(request, monkeypatch):
    """Modules whose generators are seeded by hash() make the same inputs in each run."""
    if hasattr(getattr(request, "module", None), "_gen"):
        monkeypatch.setattr(request.module, "hash", repeatable_hash, raising=False)
