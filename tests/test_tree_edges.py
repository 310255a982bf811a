"""Refusals of the tree-draft operators at the edges of their use, without a GPU."""
import pytest
import torch

import mtp_speculative_decoding_row_gb300 as mtp
from mtp_speculative_decoding_row_gb300 import build as mtp_build
from mtp_speculative_decoding_row_gb300 import tree

i32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    mtp_build.build()
    return mtp.load_library()


# the places of mtp_tree_commit_args' pointers, each 1 MB from the next
INPUTS = dict(tokens=0, target_tokens=1, parents=2, n_nodes=3, page_table=4, cache_len=5)
OUTPUTS = dict(out_tokens=10, accept_len=11, path=12, new_len=13, row_flags=14)


@pytest.mark.parametrize("into", INPUTS)
@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("ahead", [0, 4, -4])
def test_commit_refuses_outputs_over_inputs(lib, out, into, ahead):
    """B = 2, T = 3, two pages a sequence: ranges of 6, 4 or 2 integers that
    meet in whole or in part."""
    p = [(1 + i) << 20 for i in range(15)]
    p[OUTPUTS[out]] = p[INPUTS[into]] + ahead
    assert lib.mtp_tree_commit(tree._COMMIT.pack(*p, *([64] * 16), 1, 1, 2, 3, 2, 64, 5, 16, 2), None) == 1


def verify_args(**new):
    a = dict(tokens=torch.zeros(2, 4, dtype=i32), target_tokens=torch.zeros(2, 4, dtype=i32))
    a.update(new)
    return a


@pytest.mark.parametrize("new, error, text", [
    ({}, ValueError, "CUDA"),                                   # complete but for the device
    (dict(cache_len=torch.zeros(2, dtype=i32)), ValueError, "CUDA"),
    (dict(cache_len=torch.zeros(3, dtype=i32)), ValueError, "cache_len"),
    (dict(page_table=torch.zeros(2, 2, dtype=i32)), ValueError, "page_table is of no use"),
    (dict(v_new=torch.zeros(1, 2, 4, 2, 8)), ValueError, "k_new is required"),
    (dict(k_new=torch.zeros(1, 2, 4, 2, 8)), ValueError, "v_new is required"),
    (dict(k_new=torch.zeros(1, 2, 4, 2, 8), v_new=torch.zeros(1, 2, 4, 2, 8), k_cache=torch.zeros(1, 5, 16, 2, 8),
          v_cache=torch.zeros(1, 5, 16, 2, 8)), ValueError, "page_table is required"),
    (dict(k_new=torch.zeros(1, 2, 4, 2, 8), v_new=torch.zeros(1, 2, 4, 2, 8), k_cache=torch.zeros(1, 5, 16, 2, 8),
          v_cache=torch.zeros(1, 5, 16, 2, 8), page_table=torch.zeros(2, 2, dtype=i32)), ValueError, "cache_len is required"),
])
def test_commit_without_caches(new, error, text):
    with pytest.raises(error, match=text):
        mtp.mtp_tree_commit(**verify_args(**new))


def test_host_validation_of_the_verification_alone(lib):
    def call(layers=0, **at):
        p = [(1 + i) << 20 for i in range(15)]
        for k, v in at.items():
            p[{**INPUTS, **OUTPUTS, "k_new": 6}[k]] = v
        return lib.mtp_tree_commit(tree._COMMIT.pack(*p, *([64] * 16), 0, layers, at.get("B", 2), 3, 0, 0, 0, 0, 0), None)

    assert call() == 1                                   # a table of no pages
    assert call(page_table=0, tokens=0) == 1 and call(page_table=0, new_len=0) == 1
    assert call(page_table=0, out_tokens=1 << 20) == 1   # over tokens
