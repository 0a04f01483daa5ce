"""A kernel that gives up on a wait ends behind its own copies and products: each source
that issues some waits for the last of them, with a limit that no call sets (read from
the sources; no GPU).  The testing aid for it is checked on the host."""
import os
import re

import pytest
import torch

from paged_kv_decode_06_gb300 import binding
from paged_kv_decode_06_gb300 import build as builder
from tests import test_abi, test_walk_abi

KERNELS = ["pa_split.cuh", "pa_split_tc.cuh", "pa_mla.cu", "pa_mla_tc.cu",
           "pa_shared.cu"]


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(builder.CSRC, name)).read())


@pytest.mark.parametrize("name", KERNELS)
def test_the_last_copies_and_products_are_waited_for(name):
    code = _code(name)
    assert re.search(r"(bulk_load|tma_load_\dd)\(", code)
    assert re.search(r"wait\([^;]*kDrainNs\)|\bDrain \w+;", code)
    assert not re.search(r"drain\w*(\(\w+\))?, 0u, p\.wait_ns", code)


@pytest.fixture(scope="module")
def lib():
    builder.build()
    return binding.load()


def test_give_up_option(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for k, want in ((-1, binding.PA_ERR_INVALID_ARG), (3, binding.PA_ERR_CUDA)):      # (past the checks: no device here)
        o = binding.make_options(test_give_up_cta=k)
        assert test_abi._opt_call(lib, o) == want
        for call in test_walk_abi.CALLS:
            assert call(lib, dict(test_walk_abi._args(), opts=o)) == want


def test_give_up_option_of_mla(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for k, want in ((-1, binding.PA_ERR_INVALID_ARG), (2, binding.PA_ERR_CUDA)):
        assert test_abi._mla_call(lib, dict(test_abi._mla_args(), opts=binding.make_options(test_give_up_cta=k))) == want
