"""The attention half on the GPU: each operator against its formula in 64 bits, and the states in which it can go
wrong (empty rows, foreign bits behind masks, bad pages, padding, graphs, streams, far offsets).

Tolerances.  A rounding to bf16 is off by at most half a step, 2^-8 of the value; to fp32 by 2^-24.  An fp32 sum of n
terms is off by at most n 2^-24 of the sum of their magnitudes; the tensor core truncates, which doubles that, and adds
16 products at a time, which divides n by 16.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

H16, H32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def M():
    import __graft_entry__

    __graft_entry__.build()
    assert torch.cuda.is_available()
    import bit_block_quantized_moe_b200 as m

    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


# ---- moe_linear ----------------------------------------------------------------------------------------------------
def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    return z


def check_linear(out, x, w, bias, act, resid):
    x, w = x.double(), w.double()
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    ref = act64(z, act)
    # sums: K / 16 steps of the tensor core, up to 32 fp32 sums of slices or parts, the bias; |act'| <= 1.13; the
    # activation's own functions are good to 2^-20 of z
    tol = 1.13 * (x.shape[1] / 16 + 34) * 2 * H32 * mag + 2.0 ** -20 * z.abs() + 1e-30
    if resid is not None:
        ref = ref + resid.double()
        tol = tol + H32 * ref.abs()
    else:
        tol = tol * (1 + H16) + H16 * ref.abs()
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), f"largest error over tolerance: {(err / tol).max().item():.3g}"


LINEAR = [(1, 8, 1, "none", False, False), (1, 2048, 2560, "none", True, False), (3, 2048, 2560, "none", True, False),
          (8, 2048, 2048, "none", False, True), (16, 64, 130, "gelu", True, False), (17, 72, 129, "none", False, False),
          (65, 136, 1001, "silu", True, False), (300, 2048, 257, "none", True, True),
          (129, 1160, 384, "gelu", False, True), (777, 1160, 1001, "silu", True, False),
          (1024, 2048, 2048, "none", False, True), (2500, 520, 640, "gelu", True, False),
          (5000, 256, 72, "silu", False, True), (4, 65536, 40, "none", False, False),
          (4000, 200, 1100, "silu", True, False), (4000, 1096, 1100, "none", True, True),
          (40000, 64, 100, "none", True, False), (20000, 1160, 100, "gelu", False, True),
          (16, 136, 20000, "none", True, False), (9, 2048, 300, "gelu", True, True)]


@pytest.mark.parametrize("T,K,N,act,has_bias,has_resid", LINEAR)
def test_linear(M, T, K, N, act, has_bias, has_resid):
    g = gen(T + K + N)
    x = normal(g, T, K).bfloat16()
    w = (normal(g, N, K) * K ** -0.5).bfloat16()
    bias = normal(g, N) if has_bias else None
    resid = 2 * normal(g, T, N) if has_resid else None
    ws = torch.zeros(M.moe_linear_workspace_bytes(T, K, N), dtype=torch.uint8, device="cuda")
    out = torch.full((T, N), math.nan, device="cuda", dtype=torch.float32 if has_resid else torch.bfloat16)
    M.moe_linear(x, w, out, ws, bias=bias, act=act, resid=resid)
    M.moe_check_status(ws)
    check_linear(out, x, w, bias, act, resid)
    again = torch.empty_like(out)
    M.moe_linear(x, w, again, ws, bias=bias, act=act, resid=resid)
    assert torch.equal(out, again)  # every sum in a fixed order


def test_linear_strided_rows_in_place_and_nothing_else_written(M):
    g = gen(1)
    T, K, N = 37, 128, 131
    wide = normal(g, T, 320).bfloat16()
    x = wide[:, 64:64 + K]
    w = normal(g, N, K).bfloat16()
    ws = torch.zeros(M.moe_linear_workspace_bytes(T, K, N), dtype=torch.uint8, device="cuda")
    room = torch.full((T * N + 64,), 7.0, device="cuda")
    room[:T * N] = normal(g, T * N)
    before = room.clone()
    out = room[:T * N].view(T, N)
    M.moe_linear(x, w, out, ws, resid=out)
    check_linear(out, x, w, None, "none", before[:T * N].view(T, N))
    assert torch.equal(room[T * N:], before[T * N:])


def test_linear_infinities_stay_in_their_rows(M):
    g = gen(2)
    T, K, N = 40, 256, 200
    x, w = normal(g, T, K).bfloat16(), normal(g, N, K).bfloat16()
    x[11, 3], x[29, 200], w[150, 17] = math.inf, math.nan, math.inf
    ws = torch.zeros(M.moe_linear_workspace_bytes(T, K, N), dtype=torch.uint8, device="cuda")
    out = torch.empty((T, N), device="cuda", dtype=torch.bfloat16)
    M.moe_linear(x, w, out, ws)
    bad = torch.zeros((T, N), dtype=torch.bool, device="cuda")
    bad[11], bad[29], bad[:, 150] = True, True, True
    assert torch.equal(~torch.isfinite(out), bad)


# ---- a paged batch -------------------------------------------------------------------------------------------------
class Batch:
    """Sequences of new[b] tokens at the end of total[b], pages in random order, foreign bits in every unused row."""

    def __init__(self, M, g, H, V, D, ps, new, total, extra_rows=0, ragged=None, fill=None):
        self.H, self.V, self.D, self.ps, self.new, self.total = H, V, D, ps, new, total
        self.dims = M.moe_attn_dims(H, V, D, ps)
        self.T = sum(new) + extra_rows
        pages = [-(-n // ps) for n in total]
        order = torch.randperm(sum(pages) + 3, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(new), max(max(pages), 1)), 0x7fffffff, dtype=torch.int32, device="cuda")
        at = 0
        for b, p in enumerate(pages):
            self.table[b, :p] = order[at:at + p]
            at += p
        shape = (sum(pages) + 3, V, ps, D)
        self.k, self.v = normal(g, *shape).bfloat16(), normal(g, *shape).bfloat16()
        if fill is not None:  # rows of no token
            used = torch.zeros(shape[0], ps, dtype=torch.bool, device="cuda")
            for b, n in enumerate(total):
                for p in range(pages[b]):
                    used[self.table[b, p], :min(ps, n - p * ps)] = True
            free = ~used[:, None, :, None].expand(shape)
            self.k[free], self.v[free] = fill, fill
        self.kv_len = torch.tensor(total, dtype=torch.int32, device="cuda")
        ragged = len(set(new)) > 1 or extra_rows > 0 if ragged is None else ragged
        starts = torch.tensor([0] + new).cumsum(0)
        self.q_start = starts.to(torch.int32).cuda() if ragged else None
        self.ws = torch.zeros(M.moe_attn_workspace_bytes(self.dims, len(new), self.T), dtype=torch.uint8,
                              device="cuda")

    def keys(self, b):
        """Keys and values of sequence b, [V, n, D] in 64 bits."""
        n = self.total[b]
        pages = self.table[b, :-(-n // self.ps)].long()
        return tuple(x[pages].transpose(0, 1).reshape(self.V, -1, self.D)[:, :n].double() for x in (self.k, self.v))


def attend64(B, q, window, sinks, scale=None):
    """(out, tolerance) by the formula, [T, H, D] in 64 bits; a row that sees nothing is zero."""
    D, G = B.D, B.H // B.V
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros((B.T, B.H, D), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    row = 0
    for b, (m, n) in enumerate(zip(B.new, B.total)):
        if n:
            k, v = B.keys(b)
            i = (n - m + torch.arange(m, device="cuda"))[:, None]
            j = torch.arange(n, device="cuda")[None]
            seen = (j <= i) & ((i - j < window) | (j < sinks) if window else torch.ones_like(j <= i))
            some = seen.any(1)
            for h in range(B.H):
                qh = q[row:row + m, h].double()
                s = scale * (qh @ k[h // G].T)
                mag = abs(scale) * (qh.abs() @ k[h // G].abs().T)
                s = s.masked_fill(~seen, -math.inf)
                w = torch.softmax(s, -1).masked_fill(~some[:, None], 0.0)
                # a score is off by its sum (D / 16 steps) and by four roundings (scale, log2 e, their product, the
                # difference to the maximum), a weight by twice the largest of these, by exp2 (2^-22) and by its
                # rounding to bf16
                ds = torch.where(seen, (D / 16 + 2) * 2 * H32 * mag + 4 * H32 * (s.abs() + 1), 0.0).nan_to_num(0.0)
                big = torch.where(seen, s.abs(), 0.0).amax(-1, keepdim=True)
                rel = 2 * ds.amax(-1, keepdim=True) + 4 * H32 * big + 2.0 ** -20 + H16
                out[row:row + m, h] = w @ v[h // G].nan_to_num(0, 0, 0)
                tol[row:row + m, h] = rel * (w @ v[h // G].abs().nan_to_num(0, 0, 0))
        row += m
    return out, tol * (1 + H16) + H16 * out.abs() + 1e-30


def check_attention(M, B, q, window=0, sinks=0, scale=None, rows=None):
    out = torch.full((B.T, B.H, B.D), 3.0, device="cuda", dtype=torch.bfloat16)
    M.moe_attn_forward(B.dims, q, out, B.k, B.v, B.kv_len, B.table, B.ws, q_start=B.q_start, window=window,
                       n_sinks=sinks, scale=scale)
    M.moe_check_status(B.ws)
    ref, tol = attend64(B, q, window, sinks, scale)
    n = sum(B.new)
    err = (out[:n].double() - ref[:n]).abs()
    ok = err <= tol[:n]
    assert ok.all(), f"{(~ok).sum().item()} of {ok.numel()} off, first at {(~ok).nonzero()[0].tolist()}, " \
                     f"worst {(err / tol[:n]).nan_to_num(math.inf).max().item():.3g}"
    assert (out[n:] == 3.0).all()  # rows of no sequence
    again = torch.empty_like(out)
    M.moe_attn_forward(B.dims, q, again, B.k, B.v, B.kv_len, B.table, B.ws, q_start=B.q_start, window=window,
                       n_sinks=sinks, scale=scale)
    assert torch.equal(out[:n], again[:n])  # joined in a fixed order
    return out


WINDOWS = [  # H, V, D, page, new, totals, window, sinks
    (16, 2, 128, 64, 1, [1], 0, 0),
    (16, 2, 128, 64, 1, [500], 0, 0),
    (16, 2, 128, 64, 3, [65, 3, 64, 63, 1000, 4], 0, 0),
    (8, 8, 64, 16, 1, [17, 16, 15, 1, 2000], 0, 0),
    (5, 1, 128, 32, 8, [300, 8, 9, 33], 0, 0),
    (12, 4, 64, 128, 5, [127, 128, 129, 5, 700], 0, 0),
    (32, 4, 64, 16, 3, [5000, 300, 40, 3], 128, 4),
    (16, 2, 128, 64, 8, [3000, 64, 200], 1, 0),
    (16, 2, 128, 64, 4, [3000, 64, 200], 7, 70),
    (64, 1, 64, 64, 8, [900, 77], 200, 3),
    (128, 1, 128, 16, 2, [400, 1500], 0, 0),
    (6, 2, 128, 64, 1, [20000, 1, 3], 0, 0),
    (4, 2, 64, 32, 2, [64 + 31] * 70, 50, 1),
    (32, 8, 128, 64, 1, [9000], 4096, 4),
    (16, 2, 128, 64, 8, [1000, 8, 70, 9, 2000, 300], 0, 0),   # more rows than a window's tiles: the chunk kernel
    (40, 4, 64, 16, 7, [500, 7, 1200], 100, 2),
    (16, 2, 128, 64, 3, [70000], 0, 0),                       # many parts of few groups
    (80, 2, 128, 64, 5, [6000], 0, 0),
    (4, 2, 64, 16, 1, [1 + 7 * i % 90 for i in range(900)], 0, 0),
    (8, 1, 128, 64, 3, [37 * i % 700 for i in range(40)], 0, 0),   # 17 to 32 rows of many groups
    (20, 4, 64, 16, 4, [2900, 4, 0, 3, 100, 64, 65, 800, 15], 90, 5),
    (32, 8, 64, 128, 6, [500, 129, 6, 3000], 0, 0),
    (17, 1, 128, 32, 1, [5 * i for i in range(31)], 0, 0),
    (16, 1, 128, 16, 2, [900 - 30 * i for i in range(30)], 333, 1),
]


@pytest.mark.parametrize("H,V,D,ps,new,total,window,sinks", WINDOWS)
def test_attention_of_a_window(M, H, V, D, ps, new, total, window, sinks):
    g = gen(H * V + D + ps + new + len(total))
    B = Batch(M, g, H, V, D, ps, [new] * len(total), total, fill=math.nan)
    check_attention(M, B, (1.5 * normal(g, B.T, H, D)).bfloat16(), window, sinks)


CHUNKS = [  # H, V, D, page, new, totals, window, sinks
    (16, 2, 128, 64, [9], [9], 0, 0),
    (16, 2, 128, 64, [64], [64], 0, 0),
    (16, 2, 128, 64, [257], [257], 0, 0),
    (4, 4, 64, 16, [130], [400], 0, 0),
    (4, 4, 128, 128, [129, 1, 300], [129, 700, 301], 0, 0),
    (12, 4, 64, 16, [33, 700, 1, 0, 128, 17], [900, 701, 1, 40, 1000, 17], 333, 5),
    (5, 1, 128, 32, [100, 37], [100, 300], 16, 0),
    (7, 1, 64, 64, [200, 50], [1000, 50], 64, 130),
    (128, 1, 64, 64, [20, 3], [40, 200], 0, 0),
    (72, 1, 128, 16, [40], [170], 30, 2),
    (2, 1, 128, 64, [1000], [1500], 1, 0),
    (8, 2, 128, 64, [1024], [1024], 0, 0),
    (3, 3, 128, 64, [600, 600], [600, 2000], 1000, 1),
    (16, 2, 128, 64, [16], [9000], 0, 0),
    (8, 2, 64, 16, [200], [5000], 0, 0),
    (20, 1, 128, 32, [11, 40], [4000, 60], 0, 0),
    (8, 1, 128, 64, [16], [40000], 0, 0),                     # few rows over long caches: parts joined by a second launch
    (6, 2, 64, 32, [30, 1], [9000, 3], 0, 0),
    (7, 1, 128, 16, [20, 0, 13], [13, 0, 17000], 6000, 3),
    (128, 1, 64, 64, [3], [30000], 0, 0),
    (4, 4, 64, 16, [40], [5000], 5000, 0),
    (6, 1, 64, 128, [12, 9, 30], [12, 3000, 900], 700, 9),
    (4, 1, 64, 16, [i % 11 for i in range(700)], [i % 11 + i % 70 for i in range(700)], 0, 0),
]


@pytest.mark.parametrize("H,V,D,ps,new,total,window,sinks", CHUNKS)
def test_attention_of_prompt_chunks(M, H, V, D, ps, new, total, window, sinks):
    g = gen(H * V + D + ps + sum(new))
    B = Batch(M, g, H, V, D, ps, new, total, fill=math.nan, ragged=True)
    check_attention(M, B, (1.5 * normal(g, B.T, H, D)).bfloat16(), window, sinks)


def test_attention_uniform_chunks_need_no_starts(M):
    g = gen(4)
    B = Batch(M, g, 8, 2, 64, 32, [40] * 3, [40, 100, 41])
    assert B.q_start is None
    check_attention(M, B, normal(g, B.T, 8, 64).bfloat16())


@pytest.mark.parametrize("new", [1, 30])
def test_attention_strided_queries_and_scale(M, new):
    g = gen(5)
    B = Batch(M, g, 8, 2, 128, 64, [new] * 2, [100, 200])
    qkv = normal(g, B.T, 12 * 128).bfloat16()
    q = qkv[:, :8 * 128].view(B.T, 8, 128)
    for scale in (0.03, 1.0, -0.1, 0.0):
        check_attention(M, B, q, scale=scale)


@pytest.mark.parametrize("new", [4, 20])
def test_attention_large_scores(M, new):
    """Scores of thousands: one key takes all the weight, and no exponential overflows."""
    g = gen(6)
    B = Batch(M, g, 4, 2, 64, 16, [new] * 2, [100, 333])
    check_attention(M, B, (300 * normal(g, B.T, 4, 64)).bfloat16())


@pytest.mark.parametrize("new", [1, 3, 40])
def test_attention_padding_and_short_sequences(M, new):
    """kv_len 0 is padding: its rows are zeros; a length below the new tokens leaves the first rows empty."""
    g = gen(7)
    B = Batch(M, g, 4, 2, 64, 16, [new] * 4, [0, 50, max(new - 1, 0), 0], fill=math.nan)
    out = check_attention(M, B, normal(g, B.T, 4, 64).bfloat16())
    assert (out[:new] == 0).all() and (out[3 * new:] == 0).all() and (out[2 * new] == 0).all()


def test_attention_rows_behind_the_last_sequence(M):
    g = gen(8)
    B = Batch(M, g, 4, 2, 64, 16, [10, 0, 21], [30, 0, 21], extra_rows=13)
    check_attention(M, B, normal(g, B.T, 4, 64).bfloat16())


@pytest.mark.parametrize("new", [4, 8, 50, 300])
def test_attention_foreign_bits_behind_masks(M, new):
    """NaN and infinities in later tokens and before the window reach no row that does not see them."""
    g = gen(9)
    B = Batch(M, g, 4, 2, 128, 64, [new], [new + 400])
    q = normal(g, B.T, 4, 128).bfloat16()
    window, sinks = 100, 3
    first = new + 400 - new
    page = lambda p: (int(B.table[0, p // 64]), p % 64)  # noqa: E731
    # before every window and behind the sinks: seen by nobody
    for p in (3, 40, first - window - 30):
        pg, r = page(p)
        B.k[pg, :, r], B.v[pg, :, r] = math.nan, math.inf
    check_attention(M, B, q, window, sinks)
    # the last token: seen by the last query alone
    pg, r = page(first + new - 1)
    B.v[pg, 0, r] = math.inf
    B.v[pg, 1, r] = math.nan
    out = torch.empty((B.T, 4, 128), device="cuda", dtype=torch.bfloat16)
    M.moe_attn_forward(B.dims, q, out, B.k, B.v, B.kv_len, B.table, B.ws, window=window, n_sinks=sinks)
    ref, tol = attend64(B, q, window, sinks)
    assert ((out[:-1].double() - ref[:-1]).abs() <= tol[:-1]).all()
    assert not torch.isfinite(out[-1]).any()


@pytest.mark.parametrize("new", [2, 40])
def test_attention_pages_outside_the_cache(M, new):
    """The bad page is reported and its tokens are seen by nobody; the others stay right."""
    g = gen(10)
    B = Batch(M, g, 4, 2, 64, 16, [new] * 2, [100, 200])
    q = normal(g, B.T, 4, 64).bfloat16()
    good = B.table.clone()
    for value in (-1, B.k.shape[0], 0x7fffffff):
        B.table = good.clone()
        B.table[1, 2] = value  # tokens 32 .. 47 of sequence 1
        out = torch.full((B.T, 4, 64), 3.0, device="cuda", dtype=torch.bfloat16)
        M.moe_attn_forward(B.dims, q, out, B.k, B.v, B.kv_len, B.table, B.ws)
        with pytest.raises(M.MoeError) as e:
            M.moe_check_status(B.ws)
        assert e.value.code == 6
        M.moe_check_status(B.ws)  # cleared
        B.table = good
        ref, tol = attend64(B, q, 0, 0)
        assert ((out[:new].double() - ref[:new]).abs() <= tol[:new]).all()
        # sequence 1 without those keys
        k, v = B.keys(1)
        keep = torch.ones(200, dtype=torch.bool, device="cuda")
        keep[32:48] = False
        i, j = (200 - new + torch.arange(new, device="cuda"))[:, None], torch.arange(200, device="cuda")
        for h in range(4):
            s = q[new:, h].double() @ k[h // 2].T / 8
            w = torch.softmax(s.masked_fill(~(keep & (j <= i)), -math.inf), -1)
            d = (out[new:, h].double() - w @ v[h // 2]).abs()
            assert (d <= 3 * H16 * (w @ v[h // 2].abs()) + 1e-6).all()


PATHS = [  # H, V, D, page, new, totals
    (4, 2, 64, 16, 20, [6000]),                              # some parts an item
    (4, 1, 128, 64, 12, [20000]),                            # many
    (8, 2, 64, 16, 6, [50 + 40 * i for i in range(16)]),     # a window of 24 rows, 32 groups
    (16, 2, 128, 64, 3, [700] * 16),
    (16, 2, 128, 32, 2, [9000]),                             # a window of 16 rows, many parts
]


@pytest.mark.parametrize("H,V,D,ps,new,total", PATHS)
def test_attention_odd_inputs_on_every_path(M, H, V, D, ps, new, total):
    """Scales of either sign and none, scores of thousands, values that are not finite, a bad page, padding."""
    g = gen(31 + H + D)
    n = len(total)
    B = Batch(M, g, H, V, D, ps, [new] * n, total, fill=math.nan)
    q = normal(g, B.T, H, D).bfloat16()
    for scale in (1.0, -0.1, 0.0):
        check_attention(M, B, q, scale=scale)
    check_attention(M, B, (300 * q.float()).bfloat16())
    # the last token of the last sequence: only its last query sees it
    p = total[-1] - 1
    pg, r = int(B.table[n - 1, p // ps]), p % ps
    kept = B.v[pg, 0, r].clone()
    out = torch.empty((B.T, H, D), device="cuda", dtype=torch.bfloat16)
    run = lambda: M.moe_attn_forward(B.dims, q, out, B.k, B.v, B.kv_len, B.table, B.ws, q_start=B.q_start)  # noqa: E731
    run()
    want = out.clone()
    for bad in (math.inf, math.nan):
        B.v[pg, 0, r] = bad
        run()
        M.moe_check_status(B.ws)
        assert torch.equal(out[:-1], want[:-1]) and torch.equal(out[-1, H // V:], want[-1, H // V:])
        assert not torch.isfinite(out[-1, :H // V]).any()
    B.v[pg, 0, r] = kept
    # a page outside the cache: its tokens are seen by nobody, and the next call is right again
    at = (total[-1] - new - 1) // ps
    page = int(B.table[n - 1, at])
    B.table[n - 1, at] = -7
    run()
    with pytest.raises(M.MoeError) as e:
        M.moe_check_status(B.ws)
    assert e.value.code == 6
    assert torch.equal(out[:-new], want[:-new]) and torch.isfinite(out).all()
    B.table[n - 1, at] = page
    # a sequence that is padding now
    B.kv_len[0] = 0
    run()
    M.moe_check_status(B.ws)
    assert (out[:new] == 0).all()
    B.kv_len[0] = total[0]
    run()
    assert torch.equal(out, want)


def test_attention_bad_sequences(M):
    g = gen(11)
    B = Batch(M, g, 4, 2, 64, 16, [10, 20, 12], [10, 50, 60])
    q = normal(g, B.T, 4, 64).bfloat16()
    ref, tol = attend64(B, q, 0, 0)
    # sequence 1 ends before it starts (and then sequence 2 starts where it should not), or ends behind the rows
    for starts in ([0, 30, 20, 42], [0, 10, 43, 42], [-1, 10, 30, 42]):
        out = torch.full((B.T, 4, 64), 3.0, device="cuda", dtype=torch.bfloat16)
        M.moe_attn_forward(B.dims, q, out, B.k, B.v, B.kv_len, B.table, B.ws,
                           q_start=torch.tensor(starts, dtype=torch.int32, device="cuda"))
        with pytest.raises(M.MoeError):
            M.moe_check_status(B.ws)
        if starts[0] < 0:
            assert (out[:10] == 3.0).all()
            assert ((out[10:].double() - ref[10:]).abs() <= tol[10:]).all()
    # lengths outside the table count as nothing seen
    for n in (-1, B.table.shape[1] * 16 + 1, 0x7fffffff):
        B.kv_len[1] = n
        out = torch.full((B.T, 4, 64), 3.0, device="cuda", dtype=torch.bfloat16)
        M.moe_attn_forward(B.dims, q, out, B.k, B.v, B.kv_len, B.table, B.ws, q_start=B.q_start)
        with pytest.raises(M.MoeError):
            M.moe_check_status(B.ws)
        assert (out[10:30] == 0).all()
        assert ((out[30:].double() - ref[30:]).abs() <= tol[30:]).all()


@pytest.mark.parametrize("new", [1, 16])
def test_attention_offsets_beyond_32_bits(M, new):
    """A cache of 2.3e9 elements a side, the sequence in its last pages."""
    g = gen(12)
    V, ps, D = 8, 128, 128
    n_pages = 2300000000 // (V * ps * D)
    dims = M.moe_attn_dims(16, V, D, ps)
    k = torch.empty((n_pages, V, ps, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    small = Batch(M, g, 16, V, D, ps, [new], [500])
    last = torch.arange(n_pages - small.k.shape[0], n_pages, device="cuda")
    k[last], v[last] = small.k, small.v
    q = normal(g, new, 16, D).bfloat16()
    out = torch.empty_like(q)
    M.moe_attn_forward(dims, q, out, k, v, small.kv_len, small.table + int(last[0]), small.ws)
    M.moe_check_status(small.ws)
    ref, tol = attend64(small, q, 0, 0)
    assert ((out.double() - ref).abs() <= tol).all()
    # and the rows that the norm writes there
    qkv = normal(g, new, 32 * D).bfloat16()
    M.moe_qk_norm_rope(dims, qkv, out, k, v, small.kv_len, small.table + int(last[0]), small.ws)
    M.moe_qk_norm_rope(dims, qkv, torch.empty_like(out), small.k, small.v, small.kv_len, small.table, small.ws)
    assert torch.equal(k[last], small.k) and torch.equal(v[last], small.v)


@pytest.mark.parametrize("new", [2, 24])
def test_attention_in_a_graph_with_growing_lengths(M, new):
    """One capture, replayed while the sequences grow: lengths and tables are read on the device."""
    g = gen(13)
    B = Batch(M, g, 8, 2, 64, 16, [new] * 3, [400, 600, 500])
    q = normal(g, B.T, 8, 64).bfloat16()
    out = torch.empty((B.T, 8, 64), device="cuda", dtype=torch.bfloat16)

    def call():
        M.moe_attn_forward(B.dims, q, out, B.k, B.v, B.kv_len, B.table, B.ws, window=300, n_sinks=2)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([400, 600, 500], [new, 0, 77], [399, 1 + new, 500]):
        B.total = lens
        B.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        ref, tol = attend64(B, q, 300, 2)
        assert ((out.double() - ref).abs() <= tol).all()
    M.moe_check_status(B.ws)


def test_two_streams_with_their_own_workspaces(M):
    g = gen(14)
    jobs = []
    for i in range(4):
        new = (1, 40, 3, 70)[i]
        B = Batch(M, g, 8, 2, 128, 64, [new] * 2, [3000 + i, 900])
        jobs.append((B, normal(g, B.T, 8, 128).bfloat16(), torch.empty((B.T, 8, 128), device="cuda",
                                                                     dtype=torch.bfloat16), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for B, q, out, s in jobs:
            M.moe_attn_forward(B.dims, q, out, B.k, B.v, B.kv_len, B.table, B.ws, stream=s)
    torch.cuda.synchronize()
    for B, q, out, s in jobs:
        ref, tol = attend64(B, q, 0, 0)
        assert ((out.double() - ref).abs() <= tol).all()


# ---- moe_qk_norm_rope ----------------------------------------------------------------------------------------------
def norm64(h, gain, eps, pos, theta, r):
    """(rows, tolerance): norm, gain and rotation of h [T, heads, D] in 64 bits."""
    h = h.double()
    n = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    if gain is not None:
        n = n * gain.double()
    # the mean (D / 32 + 5 sums), root, quotient, two products, the rotation's two products and sum, sine and cosine
    # (4 steps of fp32 with their argument)
    mag = n.abs()
    if r:
        a = pos.double()[:, None, None] * theta ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
        x, y = n[..., :r // 2].clone(), n[..., r // 2:r].clone()
        n[..., :r // 2] = x * a.cos() - y * a.sin()
        n[..., r // 2:r] = y * a.cos() + x * a.sin()
        pair = x.abs() + y.abs()
        mag = torch.cat([pair, pair, mag[..., r:]], -1)
    return n, 24 * 2.0 ** -23 * mag + H16 * n.abs() + 1e-30


NORMS = [  # H, V, D, page, new, totals, rot, gain
    (16, 2, 128, 64, [3], [262147], 128, True),
    (16, 2, 128, 64, [1], [1], 128, False),
    (4, 4, 64, 16, [33, 700, 1, 0, 128, 17], [900, 701, 1, 40, 1000, 17], 64, True),
    (5, 1, 128, 32, [100, 37], [100, 300], 32, True),
    (7, 1, 64, 128, [2, 2, 2], [2, 129, 500000], 16, True),
    (12, 3, 128, 128, [513], [513], 96, False),
    (1, 1, 64, 16, [16], [1000000], 48, True),
    (8, 2, 64, 64, [65] * 40, [65 + 7 * i for i in range(40)], 0, True),
]


@pytest.mark.parametrize("H,V,D,ps,new,total,rot,gain", NORMS)
def test_norm_and_rotation(M, H, V, D, ps, new, total, rot, gain):
    g = gen(H + V + D + ps + sum(new))
    T, theta, eps = sum(new), 1e6, 1e-6
    # pages of the new tokens alone; a table row as long as the sequence
    first = [(n - m) // ps for m, n in zip(new, total)]
    count = [-(-n // ps) - f for n, f in zip(total, first)]
    order = torch.randperm(sum(count) + 2, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(new), max(-(-n // ps) for n in total)), -7, dtype=torch.int32, device="cuda")
    at, place, pos = 0, [], []
    for b, (m, n) in enumerate(zip(new, total)):
        table[b, first[b]:first[b] + count[b]] = order[at:at + count[b]]
        for p in range(n - m, n):
            place.append((int(order[at + p // ps - first[b]]), p % ps))
            pos.append(p)
        at += count[b]
    k, v = (normal(g, sum(count) + 2, V, ps, D).bfloat16() for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    qkv = (1.3 * normal(g, T, H + 2 * V, D)).bfloat16()
    qkv[0, 0] = 0  # an empty head
    gq, gk = ((1 + 0.3 * normal(g, D)), (1 + 0.3 * normal(g, D))) if gain else (None, None)
    dims = M.moe_attn_dims(H, V, D, ps)
    ws = torch.zeros(M.moe_attn_workspace_bytes(dims, len(new), T), dtype=torch.uint8, device="cuda")
    q = torch.full((T, H, D), math.nan, dtype=torch.bfloat16, device="cuda")
    starts = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda() if len(set(new)) > 1 else None
    M.moe_qk_norm_rope(dims, qkv.view(T, -1), q, k, v, torch.tensor(total, dtype=torch.int32, device="cuda"), table, ws,
                       rope=M.moe_rope_init(theta, rot) if rot else None, q_start=starts, q_gain=gq, k_gain=gk, eps=eps)
    M.moe_check_status(ws)
    pos = torch.tensor(pos, device="cuda")
    ref, tol = norm64(qkv[:, :H], gq, eps, pos, theta, rot)
    assert ((q.double() - ref).abs() <= tol).all()
    ref, tol = norm64(qkv[:, H:H + V], gk, eps, pos, theta, rot)
    pg, r = torch.tensor([p for p, _ in place], device="cuda"), torch.tensor([x for _, x in place], device="cuda")
    assert ((k[pg, :, r].double() - ref).abs() <= tol).all()
    assert torch.equal(v[pg, :, r], qkv[:, H + V:])
    k[pg, :, r], v[pg, :, r] = k0[pg, :, r], v0[pg, :, r]
    assert torch.equal(k, k0) and torch.equal(v, v0)  # nothing else written


def test_norm_padding_bad_pages_and_foreign_rows(M):
    g = gen(20)
    H, V, D, ps = 4, 2, 64, 16
    dims = M.moe_attn_dims(H, V, D, ps)
    table = torch.tensor([[0, 1], [2, 9], [3, 4], [5, 6]], dtype=torch.int32, device="cuda")  # page 9 is none
    kv_len = torch.tensor([0, 20, 3, 17], dtype=torch.int32, device="cuda")
    starts = torch.tensor([2, 4, 8, 12, 13], dtype=torch.int32, device="cuda")
    T = 15
    k, v = (normal(g, 7, V, ps, D).bfloat16() for _ in range(2))
    k0 = k.clone()
    qkv = normal(g, T, (H + 2 * V) * D).bfloat16()
    q = torch.full((T, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(M.moe_attn_workspace_bytes(dims, 4, T), dtype=torch.uint8, device="cuda")
    M.moe_qk_norm_rope(dims, qkv, q, k, v, kv_len, table, ws, q_start=starts)
    with pytest.raises(M.MoeError) as e:
        M.moe_check_status(ws)
    assert e.value.code == 6
    assert (q[:2] == 3.0).all() and (q[13:] == 3.0).all()   # rows of no sequence
    assert (q[2:4] == 0).all() and (q[8] == 0).all()        # negative positions
    written = {(3, 0), (3, 1), (3, 2), (6, 0)}              # sequence 1 stands in the page that is none
    for p in range(7):
        for r in range(ps):
            assert torch.equal(k[p, :, r], k0[p, :, r]) != ((p, r) in written)
    ref, tol = norm64(qkv.view(T, -1, D)[:, :H], None, 1e-6, None, 1.0, 0)
    for rows in (slice(4, 8), slice(9, 13)):
        assert ((q[rows].double() - ref[rows]).abs() <= tol[rows]).all()


def test_refusals_of_the_binding(M):
    d = M.moe_attn_dims(4, 2, 64, 16)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(M.moe_linear_workspace_bytes(4, 64, 8), dtype=torch.uint8, device="cuda")
    w, out = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((4, 8), dtype=torch.bfloat16,
                                                                                  device="cuda")
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(w=w[:, :32]), dict(out=out.float()), dict(out=out[:3]),
                dict(act="relu"), dict(resid=out), dict(bias=torch.zeros(7, device="cuda")), dict(w=w.t().contiguous().t())):
        a = dict(x=x, w=w, out=out, workspace=ws) | bad
        with pytest.raises(ValueError):
            M.moe_linear(**a)
    k = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    lens, table = torch.ones(2, dtype=torch.int32, device="cuda"), torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    base = dict(q=q, out=torch.empty_like(q), k_cache=k, v_cache=k.clone(), kv_len=lens, page_table=table,
                workspace=torch.zeros(M.moe_attn_workspace_bytes(d, 2, 2), dtype=torch.uint8, device="cuda"))
    M.moe_attn_forward(d, **base)
    for bad in (dict(q=q.float()), dict(q=q[:, :2]), dict(k_cache=k.transpose(1, 2)), dict(kv_len=lens.long()),
                dict(page_table=table[:1]), dict(q_start=lens), dict(out=q[:1]), dict(v_cache=k[:2]),
                dict(kv_len=lens.cpu())):
        with pytest.raises(ValueError):
            M.moe_attn_forward(d, **(base | bad))
