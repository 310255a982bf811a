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
