import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (B200, sm_100a)")
    config.addinivalue_line("markers", "large: holds more than 20 GB on the GPU (leave out with -m 'gpu and not large')")


# (marked here: their bodies skip or run by the memory that is free)
LARGE = {"test_offsets_past_32_bits", "test_the_most_tokens_of_the_convolution_backward"}


def pytest_collection_modifyitems(items):
    for item in items:
        if item.name in LARGE:
            item.add_marker("large")
