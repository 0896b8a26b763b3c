"""What the kernels' sources must not hold."""
import os

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "compressed_sparse_attention_05_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(os.listdir(CSRC)))
def test_no_multicast(name):
    """The library also runs as one replica per GPU of a machine: no copy or commit goes to several CTAs at once."""
    with open(os.path.join(CSRC, name)) as f:
        assert ".multicast" not in f.read()
