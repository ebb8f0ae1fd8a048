"""Q2DecoderLayer on the GPU: the operators of the attention half run together with the MoE half, as a serving loop
runs them (a prompt chunk, then windows; eager and as a captured graph)."""
import pytest
import torch

from gen import CONFIGS, make_layer
from test_gpu_attention_half import H16, attend64, check_linear, norm64

pytestmark = pytest.mark.gpu

HEADS, KV, D, PS, EPS, THETA = 4, 2, 64, 16, 1e-6, 1e6


@pytest.fixture(scope="module")
def M():
    import __graft_entry__

    __graft_entry__.build()
    import bit_block_quantized_moe_b200 as m

    return m


def build(M, seed=0, window=0, n_sinks=0, pages=40):
    cfg = CONFIGS["tiny"]
    w = make_layer(cfg, seed=seed)
    moe = M.Q2MoeLayer(cfg.hidden, cfg.inter, cfg.n_experts, cfg.top_k, w["router_w"], w["router_b"], w["experts"],
                       w["shared"], device="cuda")
    cache = M.PagedKvCache(pages, HEADS, KV, D, PS)
    g = torch.Generator().manual_seed(seed + 1)
    draw = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    width = (HEADS + 2 * KV) * D
    return M.Q2DecoderLayer(moe, cache, draw(width, cfg.hidden) * cfg.hidden ** -0.5,
                            draw(cfg.hidden, HEADS * D) * (HEADS * D) ** -0.5, b_qkv=0.1 * draw(width),
                            q_gain=1 + 0.2 * draw(D), k_gain=1 + 0.2 * draw(D), rope_theta=THETA, window=window,
                            n_sinks=n_sinks)


def normed(M, resid):
    x = torch.empty(resid.shape, dtype=torch.bfloat16, device="cuda")
    M.moe_rmsnorm_residual(resid, None, x, resid.shape[0], resid.shape[1], EPS)
    return x


class Step:
    """What attend64 wants to know of a batch."""

    def __init__(self, layer, new, total, table):
        c = layer.cache
        self.H, self.V, self.D, self.ps, self.new, self.total = HEADS, KV, D, PS, new, total
        self.T, self.table, self.k, self.v = sum(new), table, c.k, c.v

    def keys(self, b):
        n = self.total[b]
        pages = self.table[b, :-(-n // PS)].long()
        return tuple(x[pages].transpose(0, 1).reshape(KV, -1, D)[:, :n].double() for x in (self.k, self.v))


def check_step(M, layer, resid, new, total, table, q_start):
    """One call of the layer, every stage against its formula on the stage's own inputs."""
    T, hidden = resid.shape
    x = normed(M, resid)
    before = resid.clone()
    kv_len = torch.tensor(total, dtype=torch.int32, device="cuda")
    x_next = torch.empty_like(x)
    layer.forward(x, resid, x_next, kv_len, table, q_start=q_start)
    layer.check_status()
    qkv, q, o, mid = layer._qkv[:T], layer._q[:T], layer._o[:T], layer._mid[:T]
    check_linear(qkv, x, layer.w_qkv, layer.b_qkv, "none", None)
    pos = torch.cat([torch.arange(n - m, n, device="cuda") for m, n in zip(new, total)])
    heads = qkv.view(T, HEADS + 2 * KV, D)
    ref, tol = norm64(heads[:, :HEADS], layer.q_gain, EPS, pos, THETA, D)
    assert ((q.view(T, HEADS, D).double() - ref).abs() <= tol).all()
    ref, tol = norm64(heads[:, HEADS:HEADS + KV], layer.k_gain, EPS, pos, THETA, D)
    step, row = Step(layer, new, total, table), 0
    for b, (m, n) in enumerate(zip(new, total)):
        k, v = step.keys(b)
        kr = slice(row, row + m)
        assert ((k[:, n - m:].transpose(0, 1) - ref[kr]).abs() <= tol[kr]).all()
        assert torch.equal(v[:, n - m:].transpose(0, 1).to(torch.bfloat16), heads[kr, HEADS + KV:])
        row += m
    ref, tol = attend64(step, q.view(T, HEADS, D), layer.window, layer.n_sinks)
    assert ((o.view(T, HEADS, D).double() - ref).abs() <= tol).all()
    # the residual between the halves, its norm, and the MoE half as the layer alone gives it
    between = torch.empty_like(resid)
    ws = torch.zeros(M.moe_linear_workspace_bytes(T, HEADS * D, hidden), dtype=torch.uint8, device="cuda")
    M.moe_linear(o, layer.w_out, between, ws, resid=before)
    check_linear(between, o, layer.w_out, None, "none", before)
    assert torch.equal(normed(M, between), mid)
    x_alone = torch.empty_like(x)
    layer.moe.forward_residual(mid, between, x_alone, EPS)
    assert torch.equal(between, resid) and torch.equal(x_alone, x_next)
    return o.clone()


@pytest.mark.parametrize("window,n_sinks", [(0, 0), (20, 2)])
def test_prompt_then_windows(M, window, n_sinks):
    layer = build(M, window=window, n_sinks=n_sinks)
    g = torch.Generator(device="cuda").manual_seed(3)
    hidden = layer.moe.dims.hidden
    draw = lambda t: torch.randn((t, hidden), generator=g, device="cuda")  # noqa: E731
    lens, new = [37, 5, 18], [37, 5, 18]
    prompts = draw(sum(new))
    for s, n in enumerate(lens):
        layer.cache.grow(s, n)
    starts = torch.tensor([0, 37, 42, 60], dtype=torch.int32, device="cuda")
    check_step(M, layer, prompts.clone(), new, lens, layer.cache.table(range(3)), starts)
    tokens = [[prompts[a:b]] for a, b in ((0, 37), (37, 42), (42, 60))]
    for m in (1, 3, 8):
        lens = [n + m for n in lens]
        for s, n in enumerate(lens):
            layer.cache.grow(s, n)
        rows = draw(3 * m)
        last = check_step(M, layer, rows.clone(), [m] * 3, lens, layer.cache.table(range(3)), None)
        for s in range(3):
            tokens[s].append(rows[s * m:(s + 1) * m])
    # all tokens of a sequence as one chunk into a fresh cache: the same last rows, as each is within its tolerance
    fresh = build(M, window=window, n_sinks=n_sinks)
    for s in range(3):
        fresh.cache.release(0)
        fresh.cache.grow(0, lens[s])
        table = fresh.cache.table([0])
        o = check_step(M, fresh, torch.cat(tokens[s]), [lens[s]], [lens[s]], table, None)
        a, b = o[-8:].double(), last[8 * s:8 * s + 8].double()
        step = Step(fresh, [8], [lens[s]], table)
        _, tol = attend64(step, fresh._q[:lens[s]][-8:].view(8, HEADS, D), window, n_sinks)
        # twice the tolerance of one side, and keys and queries that may round the other way (one step of bf16 each)
        assert ((a - b).abs() <= (2 * tol + 16 * H16 * tol.amax()).view(8, -1)).all()


def test_windows_replayed_from_a_graph(M):
    """Decode steps of one token from one captured graph: lengths, tables and activations change in place."""
    layer = build(M)
    g = torch.Generator(device="cuda").manual_seed(5)
    hidden, lens = layer.moe.dims.hidden, [20, 33]
    for s in range(2):
        layer.cache.grow(s, 64)
    table = layer.cache.table(range(2))
    layer.cache.k.normal_(generator=g)
    layer.cache.v.normal_(generator=g)
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    resid = torch.zeros((2, hidden), device="cuda")
    x, x_next = (torch.zeros((2, hidden), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step():
        M.moe_rmsnorm_residual(resid, None, x, 2, hidden, EPS)
        layer.forward(x, resid, x_next, kv_len, table)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rows = torch.randn((4, 2, hidden), generator=g, device="cuda")
    got = []
    for run in (graph.replay, step):
        k, v = layer.cache.k.clone(), layer.cache.v.clone()
        out = []
        for i in range(4):
            kv_len.copy_(torch.tensor([n + i + 1 for n in lens], dtype=torch.int32))
            resid.copy_(rows[i])
            run()
            out.append((resid.clone(), x_next.clone()))
        got.append(out)
        layer.cache.k.copy_(k)
        layer.cache.v.copy_(v)
    for (a, b), (c, d) in zip(*got):
        assert torch.equal(a, c) and torch.equal(b, d)
    layer.check_status()


def test_a_graph_outlives_the_buffers_of_its_call(M, monkeypatch):
    """A larger eager call makes larger buffers; the graph captured before it still owns its own."""
    layer = build(M)
    g = torch.Generator(device="cuda").manual_seed(11)
    hidden = layer.moe.dims.hidden
    layer.cache.grow(0, 30)
    layer.cache.grow(1, 500)
    layer.cache.k.normal_(generator=g)
    layer.cache.v.normal_(generator=g)
    one, long = layer.cache.table([0]), layer.cache.table([1])
    start = torch.randn((1, hidden), generator=g, device="cuda")
    resid, x_next = start.clone(), torch.empty((1, hidden), dtype=torch.bfloat16, device="cuda")
    x = torch.empty_like(x_next)
    kv_len = torch.tensor([30], dtype=torch.int32, device="cuda")

    def step():
        M.moe_rmsnorm_residual(resid, None, x, 1, hidden, EPS)
        layer.forward(x, resid, x_next, kv_len, one)

    step()
    want = resid.clone(), x_next.clone()
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        with pytest.raises(RuntimeError, match="reserve"):
            layer.reserve(9, 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    many = torch.randn((400, hidden), generator=g, device="cuda")
    x_many = torch.empty((400, hidden), dtype=torch.bfloat16, device="cuda")
    M.moe_rmsnorm_residual(many, None, x_many, 400, hidden, EPS)
    layer.forward(x_many, many, torch.empty_like(x_many), torch.tensor([500], dtype=torch.int32, device="cuda"), long)
    held = [torch.full((400, hidden), 7.0, device="cuda") for _ in range(64)]  # takes what the allocator has free
    resid.copy_(start)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(resid, want[0]) and torch.equal(x_next, want[1])
    assert all((h == 7.0).all() for h in held)
    layer.check_status()


def test_padding_rows_keep_their_residual_until_the_moe_half(M):
    layer = build(M)
    g = torch.Generator(device="cuda").manual_seed(7)
    hidden = layer.moe.dims.hidden
    layer.cache.grow(0, 10)
    table = torch.cat([layer.cache.table([0]), torch.full((1, 1), -1, dtype=torch.int32, device="cuda")])
    resid = torch.randn((4, hidden), generator=g, device="cuda")
    x, x_next = normed(M, resid), torch.empty((4, hidden), dtype=torch.bfloat16, device="cuda")
    layer.forward(x, resid, x_next, torch.tensor([10, 0], dtype=torch.int32, device="cuda"), table)
    layer.check_status()
    assert (layer._o[2:4] == 0).all()
    assert torch.equal(layer._mid[2:4], x[2:4])


def test_refused_shapes(M):
    layer = build(M)
    with pytest.raises(ValueError):
        M.Q2DecoderLayer(layer.moe, layer.cache, layer.w_qkv[:-1], layer.w_out)
    with pytest.raises(ValueError):
        M.Q2DecoderLayer(layer.moe, layer.cache, layer.w_qkv, layer.w_out[:, 1:])
    with pytest.raises(M.MoeError):
        M.Q2DecoderLayer(layer.moe, layer.cache, layer.w_qkv, layer.w_out, rotary_dim=24)


def test_large_layer_shapes(M):
    """The shapes of the full-size layer's attention half, a window and a chunk, stage by stage on sampled rows."""
    g = torch.Generator(device="cuda").manual_seed(9)
    hidden, heads, kv, dim, ps = 2048, 16, 2, 128, 64
    dims = M.moe_attn_dims(heads, kv, dim, ps)
    w = (torch.randn(((heads + 2 * kv) * dim, hidden), generator=g, device="cuda") * hidden ** -0.5).bfloat16()
    rope = M.moe_rope_init(THETA, dim)
    for T, n in ((3, 3003), (700, 900)):
        x = torch.randn((T, hidden), generator=g, device="cuda").bfloat16()
        pages = -(-n // ps)
        k = torch.randn((pages + 1, kv, ps, dim), generator=g, device="cuda").bfloat16()
        v = torch.randn_like(k)
        table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None].contiguous()
        kv_len = torch.tensor([n], dtype=torch.int32, device="cuda")
        ws = torch.zeros(max(M.moe_attn_workspace_bytes(dims, 1, T), M.moe_linear_workspace_bytes(T, hidden, w.shape[0])),
                         dtype=torch.uint8, device="cuda")
        qkv = torch.empty((T, w.shape[0]), dtype=torch.bfloat16, device="cuda")
        q, o = (torch.empty((T, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        M.moe_linear(x, w, qkv, ws)
        M.moe_qk_norm_rope(dims, qkv, q, k, v, kv_len, table, ws, rope=rope)
        M.moe_attn_forward(dims, q, o, k, v, kv_len, table, ws)
        M.moe_check_status(ws)
        check_linear(qkv, x, w, None, "none", None)
        ref, tol = norm64(qkv.view(T, -1, dim)[:, :heads], None, EPS, torch.arange(n - T, n, device="cuda"), THETA, dim)
        assert ((q.double() - ref).abs() <= tol).all()

        class S:
            H, V, D, ps_, new, total = heads, kv, dim, ps, [T], [n]

            @staticmethod
            def keys(b):
                at = table[0].long()
                return tuple(z[at].transpose(0, 1).reshape(kv, -1, dim)[:, :n].double() for z in (k, v))

        S.T = T
        ref, tol = attend64(S, q, 0, 0)
        assert ((o.double() - ref).abs() <= tol).all()
