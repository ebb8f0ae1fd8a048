"""Further edges of the attention half on the GPU, against the same formulas in 64 bits."""
import math

import pytest
import torch

from test_gpu_attention_half import Batch, M, attend64, check_attention, gen, normal  # noqa: F401

pytestmark = pytest.mark.gpu


# Few row tiles under a table that is long enough for clusters (of 8, 4 and 2 CTAs by these counts), and sequences of so
# few key tiles that most CTAs of a cluster have none and come to its join at once.
@pytest.mark.parametrize("D,seqs,tiles", [(64, 7, 16), (128, 7, 40), (64, 10, 9), (128, 18, 8), (64, 20, 5), (128, 36, 4)])
def test_short_sequences_under_tables_that_make_clusters(M, D, seqs, tiles):  # noqa: F811
    g = gen(41 + D + seqs)
    new = 20
    total = [(1, 0, 20, 128, 129, 300, 384)[i % 7] for i in range(seqs)]
    B = Batch(M, g, 4, 2, D, 16, [new] * seqs, total, fill=math.nan)
    assert B.q_start is None
    wide = torch.full((seqs, tiles * 8), 0x7fffffff, dtype=torch.int32, device="cuda")
    wide[:, :B.table.shape[1]] = B.table
    B.table = wide
    q = normal(g, B.T, 4, D).bfloat16()
    for _ in range(10):
        check_attention(M, B, q)
