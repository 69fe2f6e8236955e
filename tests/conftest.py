import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a B200 (sm_100a) GPU and the built libsfa.so")


@pytest.fixture(scope="session", autouse=True)
def built():
    """Both the library and the extension module over it, whichever of them is missing."""
    from frame_sparse_attention_b200 import build
    if not (os.path.exists(build.LIB) and os.path.exists(build.BIND)):
        build.build()
