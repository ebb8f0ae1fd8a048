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


# ---- activations far from zero -------------------------------------------------------------------------------------
def activated(M, z, act, wide):
    """act of each z (bf16) by itself: one product of z and 1, the others zeros; fp32 with a residual of zeros."""
    x = torch.zeros((z.numel(), 8), dtype=torch.bfloat16, device="cuda")
    x[:, 3] = z
    w = torch.zeros((5, 8), dtype=torch.bfloat16, device="cuda")
    w[:, 3] = 1
    shape = (z.numel(), 5)
    resid = torch.zeros(shape, device="cuda") if wide else None
    out = torch.empty(shape, device="cuda", dtype=torch.float32 if wide else torch.bfloat16)
    ws = torch.zeros(M.moe_linear_workspace_bytes(*x.shape, 5), dtype=torch.uint8, device="cuda")
    M.moe_linear(x, w, out, ws, act=act, resid=resid)
    M.moe_check_status(ws)
    same = (out == out[:, :1]) | out.isnan() & out[:, :1].isnan()
    assert same.all()
    return out[:, 0].double()


@pytest.mark.parametrize("wide", [False, True])
def test_gelu_keeps_its_relative_accuracy(M, wide):  # noqa: F811
    """z/2 (1 + erf(z / sqrt 2)) is z/2 erfc(u), u = -z / sqrt 2: no cancellation for negative z.  The kernel's form has
    e^(-u^2), whose argument is rounded twice (2 u^2 of 2^-24 at the most, and as much for its constant), a polynomial that
    is fitted to 1.3 units of the last place (2^-23) and takes 2 more by its own roundings, a reciprocal (1, and 1 for its
    argument), a power of two (2) and four products and sums (2)."""
    z = torch.linspace(-12, 12, 3001, device="cuda").bfloat16()
    u = -z.double() / math.sqrt(2)
    ref = 0.5 * z.double() * torch.special.erfc(u)
    tol = (2 * u * u + 10) * 2.0 ** -23 + (0 if wide else 2.0 ** -8)
    err = (activated(M, z, "gelu", wide) - ref).abs()
    assert (err <= tol * ref.abs()).all(), f"worst {(err / (tol * ref.abs())).nan_to_num(0).max().item():.3g}"


@pytest.mark.parametrize("wide", [False, True])
def test_silu_keeps_its_relative_accuracy(M, wide):  # noqa: F811
    """z / (1 + e^-z) down to where it leaves fp32's normal numbers (-91).  The power of two is within 2 units of the last
    place (2^-23), its argument is rounded twice (|z| of 2^-24 each); a sum (1/2), a quotient (2), two products (1)."""
    z = torch.linspace(-91, 91, 4001, device="cuda").bfloat16()
    ref = z.double() / (1 + torch.exp(-z.double()))
    tol = (z.double().abs() + 6) * 2.0 ** -23 + (0 if wide else 2.0 ** -8)
    err = (activated(M, z, "silu", wide) - ref).abs()
    assert (err <= tol * ref.abs()).all(), f"worst {(err / (tol * ref.abs())).nan_to_num(0).max().item():.3g}"


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("wide", [False, True])
def test_activations_of_what_is_not_ordinary(M, act, wide):  # noqa: F811
    """Infinities and NaN as the formulas have them (0 times an infinity is NaN), signed zeros, the largest values."""
    big = torch.finfo(torch.bfloat16).max
    z = torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, big, -big, 300.0, -300.0], device="cuda").bfloat16()
    out = activated(M, z, act, wide).tolist()
    assert out[0] == math.inf and math.isnan(out[1]) and math.isnan(out[2])
    assert out[3:] == [0.0, 0.0, big, 0.0, 0.0 + 300.0, 0.0]
