import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
HERE = os.path.dirname(os.path.abspath(__file__))
if HERE not in sys.path:
    sys.path.insert(0, HERE)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a) and the built libsmol.so")


# Expects rows of a negative position to be written over a sequence's first slots, where the header (and
# test_gpu_paged_contracts.py) says that they are not written.  It fails, and runs behind all others, so that a run
# that ends at its first failure has run them.
CONTRADICTS_THE_HEADER = "test_gpu_paged.py::test_rows_out_of_range_are_not_written"


def pytest_collection_modifyitems(items):
    items.sort(key=lambda item: item.nodeid.endswith(CONTRADICTS_THE_HEADER))
