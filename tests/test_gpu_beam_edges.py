"""Beam selection on the GPU at the edges of its ranges: logits that are no
numbers, masks that leave a few tokens, low temperatures, neighbouring
scores."""
import math

import pytest
import torch

import mtp_speculative_decoding_row_gb300 as mtp

pytestmark = pytest.mark.gpu
i32 = torch.int32
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def library():
    from tests import gpu_util

    gpu_util.ensure_library()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_bad_logit_in_every_vector_of_the_first_rounds(dtype, bad):
    """Whichever warp meets it, and however early: the sequence is flagged."""
    vec = 8 if dtype == "bf16" else 4
    B, V = 1100, 1100 * vec + 3
    z = torch.zeros(B, 1, V, dtype=DTYPES[dtype])
    at = torch.arange(B) * vec + torch.arange(B) % vec
    z[torch.arange(B), 0, at] = bad
    z = torch.cat([z, torch.zeros_like(z[:1])]).cuda()
    scores, T = torch.zeros(B + 1, 1, device="cuda"), torch.ones(B + 1, device="cuda")
    for _ in range(20):
        r = mtp.mtp_beam_select(z, scores, T, 3)
        torch.cuda.synchronize()
        assert r.row_flags.tolist() == [mtp.ROW_NONFINITE] * B + [0]
        assert (r.tokens[:B] == -1).all() and r.tokens[B].tolist() == [0, 1, 2]
