"""CPU check of the kernels that may be launched while the one before them still
writes (programmatic launch): what they read of the cache and of the workspace goes
through coherent loads, since the read-only path is for data that nothing writes
during a kernel's whole lifetime."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "long_context_flashattention_gb300", "csrc")


def code_of(name):
    """The file's text without comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", ["dfa_paged.cu", "dfa_serve.cuh"])
def test_no_read_only_loads_in_early_launched_kernels(name):
    """(dfa_serve.cuh holds the loads of lengths and table entries.)"""
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", code_of(name))


def test_only_the_decode_is_launched_early():
    """A kernel elsewhere that gets the attribute has to come under the check above."""
    for name in sorted(os.listdir(CSRC)):
        if name != "dfa_paged.cu":
            assert "StreamSerialization" not in code_of(name), name
