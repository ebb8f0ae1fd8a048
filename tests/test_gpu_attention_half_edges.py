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


# ---- starts and lengths that are wrong -----------------------------------------------------------------------------
class Part:
    """One sequence of a batch, as attend64 wants it."""

    def __init__(self, B, b, m, n):
        self.H, self.V, self.D, self.new, self.total, self.T = B.H, B.V, B.D, [m], [n], m
        self.keys = lambda _: tuple(x[:, :n] for x in B.keys(b))


def sequences(starts, T):
    """(sequence, first row, rows) of the pairs that lie in the rows."""
    return [(b, s, e - s) for b, (s, e) in enumerate(zip(starts, starts[1:])) if 0 <= s <= e <= T]


STARTS = [([0, 30, 20, 42], 42), ([0, 10, 43, 42], 42), ([-1, 10, 30, 42], 42), ([42, 42, 42, 43], 42), ([20, 42, 0, 20], 42),
          ([0, 42, 0, 42], 42), ([0x7fffffff, -0x80000000, 5, 42], 42), ([0, 1000, 10, 1000], 1000), ([3, 9, 30, 42], 42)]


@pytest.mark.parametrize("starts,T", STARTS)
def test_attention_of_starts_that_are_wrong(M, starts, T):  # noqa: F811
    """A pair that decreases or leaves the rows is reported; what is written then is right for a sequence that has the row;
    where the starts do not decrease, all others are right; nothing beside the rows is written."""
    g = gen(51 + T)
    B = Batch(M, g, 4, 2, 64, 16, [T] * 3, [T + 20, T, T + 3])
    q = normal(g, T, 4, 64).bfloat16()
    room = torch.full((T + 40, 4, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    out = room[20:20 + T]
    M.moe_attn_forward(B.dims, q, out, B.k, B.v, B.kv_len, B.table, B.ws,
                       q_start=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    status(M, B.ws, 6 if len(sequences(starts, T)) < 3 else 0)
    assert (room[:20] == 3.0).all() and (room[20 + T:] == 3.0).all()
    fine = out == 3.0
    untouched = fine.flatten(1).all(1)
    for b, s, m in sequences(starts, T):
        ref, tol = attend64(Part(B, b, m, B.total[b]), q[s:s + m], 0, 0)
        right = (out[s:s + m].double() - ref).abs() <= tol
        fine[s:s + m] |= right
        if sorted(starts) == starts:
            assert right.all()
    assert fine.all()
    held = torch.zeros(T, dtype=torch.bool, device="cuda")
    for _, s, m in sequences(starts, T):
        held[s:s + m] = True
    assert untouched[~held].all()


def status(M, ws, code):  # noqa: F811
    if code == 0:
        return M.moe_check_status(ws)
    with pytest.raises(M.MoeError) as e:
        M.moe_check_status(ws)
    assert e.value.code == code


def normed_rows(M, B, T, starts, lens, g):  # noqa: F811
    """What moe_qk_norm_rope leaves, and which row of which sequence may have written each cached row."""
    qkv = normal(g, T, (B.H + 2 * B.V) * B.D).bfloat16()
    room = torch.full((T + 40, B.H, B.D), 3.0, device="cuda", dtype=torch.bfloat16)
    k, v = B.k.clone(), B.v.clone()
    M.moe_qk_norm_rope(B.dims, qkv, room[20:20 + T], k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), B.table,
                       B.ws, q_start=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    assert (room[:20] == 3.0).all() and (room[20 + T:] == 3.0).all()
    cap, table, may, zero = B.table.shape[1] * B.ps, B.table.tolist(), {}, torch.zeros(T, dtype=torch.bool)
    for b, s, m in sequences(starts, T):
        n = lens[b] if 0 <= lens[b] <= cap else 0
        for i in range(m):
            p = n - m + i
            if p >= 0:
                may.setdefault((table[b][p // B.ps], p % B.ps), []).append(s + i)
            else:
                zero[s + i] = True
    return qkv.view(T, -1, B.D), room[20:20 + T], k, v, may, zero.cuda()


def check_normed(B, qkv, q, k, v, may, zero, all_written):
    heads = qkv.double()
    ref = heads / torch.sqrt((heads * heads).mean(-1, keepdim=True) + 1e-6)
    tol = 2.0 ** -8 * ref.abs() + 24 * 2.0 ** -23 * ref.abs() + 1e-30
    is_right = ((q.double() - ref[:, :B.H]).abs() <= tol[:, :B.H]).flatten(1).all(1)
    is_zero, is_old = (q == 0).flatten(1).all(1), (q == 3.0).flatten(1).all(1)
    held = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for rows in may.values():
        held[rows] = True
    assert (is_old | is_right & held | is_zero & zero).all()
    if all_written:
        assert not is_old[held | zero].any()
    changed = ((k != B.k) | (v != B.v)).any(3).any(1).nonzero().tolist()
    assert {tuple(x) for x in changed} <= set(may)  # no cached row outside the sequences' own
    for page, row in changed:
        assert any(torch.equal(v[page, :, row], qkv[t, B.H + B.V:])
                   and ((k[page, :, row].double() - ref[t, B.H:B.H + B.V]).abs() <= tol[t, B.H:B.H + B.V]).all()
                   for t in may[page, row])
    if all_written:
        assert {tuple(x) for x in changed} == set(may)


@pytest.mark.parametrize("starts,T", STARTS)
def test_norm_of_starts_that_are_wrong(M, starts, T):  # noqa: F811
    g = gen(61 + T)
    B = Batch(M, g, 4, 2, 64, 16, [T] * 3, [T + 20, T, T + 3])
    made = normed_rows(M, B, T, starts, B.total, g)
    status(M, B.ws, 6 if len(sequences(starts, T)) < 3 else 0)
    check_normed(B, *made, all_written=sorted(starts) == starts)


@pytest.mark.parametrize("length", [-1, 81, 0x7fffffff, -0x80000000])
def test_norm_of_lengths_that_are_wrong(M, length):  # noqa: F811
    """Such a length counts as 0: the sequence's queries are zeros and none of its keys is written."""
    g = gen(71)
    B = Batch(M, g, 4, 2, 64, 16, [10, 20, 12], [70, 50, 60])
    assert B.table.shape[1] == 5
    made = normed_rows(M, B, 42, [0, 10, 30, 42], [70, length, 60], g)
    status(M, B.ws, 6)
    check_normed(B, *made, all_written=True)
    assert (made[1][10:30] == 0).all()
