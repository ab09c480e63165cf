"""The experts' calls as they are used together: route -> dispatch -> experts ->
combine and back, on other streams, captured into graphs, through MoeBuffers,
with rows past 2^32 bytes, and what the binding refuses on a GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import combine_topk_route_amd as moe
    from expertshelp import (BF, DEV, HALF, act64, assert_bits, gen, ints, normal,
                             offsets_of)


def step(logits, x, w1, w2, k, act="silu"):
    """One layer forward: what a training program keeps for the way back."""
    E = w1.shape[0]
    idx, w, send, buf = moe.moe_route_dispatch(logits, x, k)
    off = send.expert_offsets
    h, gate_up = moe.moe_expert_gated(buf, off, w1, act, save_gate_up=True)
    y, _ = moe.moe_expert_matmul(h, off, w2)
    out = moe.moe_combine(y, send.pair_row, w)
    return dict(E=E, idx=idx, w=w, send=send, buf=buf, h=h, gate_up=gate_up, y=y, out=out)


def back(s, dout, w1, w2, act="silu"):
    off = s["send"].expert_offsets
    dy, dwr = moe.moe_combine_backward(dout, s["y"], s["send"].pair_row, s["w"])
    down = moe.moe_expert_matmul_backward(dy, s["h"], off, w2)
    up = moe.moe_expert_gated_backward(down.dx, s["gate_up"], s["buf"], off, w1, act)
    dx = moe.moe_combine(up.dx, s["send"].pair_row, torch.ones_like(s["w"]))
    return dict(dx=dx, dw1=up.dw, dw2=down.dw, dwr=dwr, dy=dy, dh=down.dx, dgate_up=up.dgate_up,
                dbuf=up.dx)


def layer64(x, idx, w, w1, w2, act):
    """The layer in 64 bits from the routing given, differentiable."""
    out = torch.zeros((x.shape[0], w2.shape[1]), dtype=torch.float64)
    I = w2.shape[2]
    for e in range(w1.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            z = x[t] @ w1[e].t()
            y = (act64(z[:, :I], act) * z[:, I:]) @ w2[e].t()
            out = out.index_add(0, t, w[t, j][:, None] * y)
    return out


@pytest.mark.parametrize("T,k,E,H,I,act", [(5, 2, 4, 64, 72, "silu"), (33, 3, 7, 136, 64, "gelu"),
                                           (70, 8, 16, 72, 40, "silu")])
def test_layer_gradients(T, k, E, H, I, act):
    """Every gradient of the chain against autograd of the layer in 64 bits, and
    against differences of it.

    Each of the chain's tensors is rounded to bf16 once, half a step of 2^-8 of
    its value: forward gate/up (kept), h and y; backward dy, dh, dgate_up, dbuf
    and the outputs.  To first order the relative error of a gradient in the
    2-norm is at most the number of roundings on its way times 2^-8, times the
    ratio by which the products can enlarge a relative error; for these random
    matrices that ratio is near 1, and 4 is allowed.  At most 6 roundings lie
    on one way (gate, up, dy, dh, dgate_up, dx), so 24 * 2^-8 bounds it."""
    g = gen(20)
    logits = torch.randn((T, E), generator=g, device=DEV)
    x = normal(g, T, H)
    w1, w2 = normal(g, E, 2 * I, H, scale=H**-0.5), normal(g, E, H, I, scale=I**-0.5)
    dout = normal(g, T, H)
    s = step(logits, x, w1, w2, k, act)
    r = back(s, dout, w1, w2, act)
    idx = s["idx"].cpu()
    leaf = [t.double().cpu().requires_grad_() for t in (x, s["w"], w1, w2)]
    ref = layer64(leaf[0], idx, leaf[1], leaf[2], leaf[3], act)
    bound = 24 * HALF

    def near(got, want, what):
        rel = float((got.double().cpu() - want).norm() / want.norm())
        assert rel <= bound, f"{what}: {rel:.3g} of {bound:.3g}"

    near(s["out"], ref.detach(), "out")
    d64 = dout.double().cpu()
    grads = torch.autograd.grad(ref, leaf, d64)
    for name, want in zip(("dx", "dwr", "dw1", "dw2"), grads):
        near(r[name], want, name)
    # along a random direction of all four: central differences of the layer in 64 bits
    h = 1e-5
    gc = torch.Generator().manual_seed(21)
    dirs = [torch.randn(t.shape, generator=gc, dtype=torch.float64) for t in leaf]
    with torch.no_grad():
        at = [[a + sign * h * v for a, v in zip(leaf, dirs)] for sign in (1, -1)]
        up, dn = (layer64(p[0], idx, p[1], p[2], p[3], act) for p in at)
        diff = float(((up - dn) * d64).sum() / (2 * h))
        got = sum(float((r[n].double().cpu() * v).sum()) for n, v in zip(("dx", "dwr", "dw1", "dw2"), dirs))
        size = sum(float(w.norm()) * float(v.norm()) for w, v in zip(grads, dirs))
    # |<got - want, v>| <= |got - want| |v|; differences in 64 bits add h^2 times a third derivative
    assert abs(got - diff) <= bound * size + 1e-6 * size


def test_whole_numbers_through_the_chain():
    """With relu, small whole numbers and weights of 1 everything up to combine is exact."""
    T, k, E, H, I = 40, 2, 6, 64, 72
    g = gen(22)
    logits = torch.randn((T, E), generator=g, device=DEV)
    x = ints(g, -1, 1, T, H)
    # one input feature for each inner one, so that h stays below 257
    w1 = torch.zeros((E, 2 * I, H), dtype=BF, device=DEV)
    w1[:, torch.arange(2 * I), torch.arange(2 * I) % H] = ints(g, -3, 3, E, 2 * I)
    w2 = ints(g, -1, 1, E, H, I)
    s = step(logits, x, w1, w2, k, "relu")
    z = torch.einsum("th,enh->ten", x.double(), w1.double())
    h = z[..., :I].clamp(min=0) * z[..., I:]
    y = torch.einsum("tei,ehi->teh", h, w2.double())
    want = torch.gather(y, 1, s["idx"].long()[:, :, None].expand(-1, -1, H)).reshape(T * k, H)
    got = s["y"][s["send"].pair_row.reshape(-1).long()]
    assert_bits(got, want, "y")


def test_on_another_stream():
    g = gen(23)
    T, k, E, H, I = 64, 2, 8, 136, 72
    logits, x = torch.randn((T, E), generator=g, device=DEV), normal(g, T, H)
    w1, w2 = normal(g, E, 2 * I, H, scale=H**-0.5), normal(g, E, H, I, scale=I**-0.5)
    idx, w, send, buf = moe.moe_route_dispatch(logits, x, k)
    off = send.expert_offsets
    want, wgu = moe.moe_expert_gated(buf, off, w1, save_gate_up=True)
    wy, _ = moe.moe_expert_matmul(want, off, w2, act="gelu", save_pre=True)
    wb = moe.moe_expert_gated_backward(want, wgu, buf, off, w1)
    wm = moe.moe_expert_matmul_backward(wy, want, off, w2, act="gelu", pre=wy, need_dbias=True)
    wc = moe.moe_combine_backward(x, wy, send.pair_row, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        h, gu = moe.moe_expert_gated(buf, off, w1, save_gate_up=True, stream=handle)
        y, _ = moe.moe_expert_matmul(h, off, w2, act="gelu", save_pre=True, stream=handle)
        b = moe.moe_expert_gated_backward(h, gu, buf, off, w1, stream=handle)
        m = moe.moe_expert_matmul_backward(y, h, off, w2, act="gelu", pre=y, need_dbias=True,
                                           stream=handle)
        c = moe.moe_combine_backward(x, y, send.pair_row, w, stream=handle)
        s.synchronize()
        for a, z in zip((h, gu, y, *b, *m, *c), (want, wgu, wy, *wb, *wm, *wc)):
            assert torch.equal(a.view(torch.uint8), z.view(torch.uint8))


def test_two_calls_at_once():
    """Two streams with work of their own under way together share nothing."""
    g = gen(24)
    E, H, I = 8, 520, 264
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    off = offsets_of([30, 0, 500, 3, 64, 65, 200, 1])
    P = int(off[-1])
    data = [(normal(g, P, H), normal(g, E, 2 * I, H, scale=H**-0.5), normal(g, P, I)) for _ in streams]
    want = []
    for x, w, dh in data:
        h, gu = moe.moe_expert_gated(x, off, w, save_gate_up=True)
        want.append((h, gu, *moe.moe_expert_gated_backward(dh, gu, x, off, w)))
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, (x, w, dh) in zip(streams, data):
            h, gu = moe.moe_expert_gated(x, off, w, save_gate_up=True, stream=s)
            got.append((h, gu, *moe.moe_expert_gated_backward(dh, gu, x, off, w, stream=s)))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(u.view(torch.int16), v.view(torch.int16)) for u, v in zip(a, b))


@pytest.mark.parametrize("T,k,E,H,I", [(16, 2, 8, 136, 72), (600, 4, 4, 136, 264)])
def test_captured_and_replayed(T, k, E, H, I):
    """A whole training step in one graph: every replay equals the eager step, with eager work
    between the replays, and on new inputs with another routing."""
    g = gen(25)
    w1, w2 = normal(g, E, 2 * I, H, scale=H**-0.5), normal(g, E, H, I, scale=I**-0.5)
    inputs = [(torch.randn((T, E), generator=g, device=DEV) * sc, normal(g, T, H), normal(g, T, H))
              for sc in (1.0, 1.0, 5.0)]
    ws = torch.zeros(max(1, moe.moe_route_dispatch_workspace_bytes(T, E, k)), dtype=torch.uint8,
                     device=DEV)

    def whole(logits, x, dout):
        idx, w, send, buf = moe.moe_route_dispatch(logits, x, k, workspace=ws)
        off = send.expert_offsets
        h, gu = moe.moe_expert_gated(buf, off, w1, save_gate_up=True)
        y, pre = moe.moe_expert_matmul(h, off, w2, act="gelu", save_pre=True)
        out = moe.moe_combine(y, send.pair_row, w)
        dy, dwr = moe.moe_combine_backward(dout, y, send.pair_row, w)
        m = moe.moe_expert_matmul_backward(dy, h, off, w2, act="gelu", pre=pre, need_dbias=True)
        b = moe.moe_expert_gated_backward(m.dx, gu, buf, off, w1, dw_dtype=torch.float32)
        return (out, dwr, m.dw, m.dbias, b.dw, moe.moe_combine(b.dx, send.pair_row, torch.ones_like(w)))

    ins = [t.clone() for t in inputs[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            whole(*ins)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = whole(*ins)
    for n in (0, 0, 1, 2, 0):
        for a, b in zip(ins, inputs[n]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = whole(*inputs[n])  # eager work between the replays
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"output {i}, inputs {n}"


def test_buffers_run_the_experts():
    T, k, E, H, I = 24, 2, 8, 136, 72
    g = gen(26)
    bufs = moe.MoeBuffers(32, H, E, k, intermediate=I)
    w1, w2 = normal(g, E, 2 * I, H, scale=H**-0.5), normal(g, E, H, I, scale=I**-0.5)
    for n in (T, 32, 1):
        logits, x = torch.randn((n, E), generator=g, device=DEV), normal(g, n, H)
        idx, w, send, buf = bufs.route_dispatch(logits, x)
        before = torch.cuda.memory_allocated()
        y = bufs.experts(buf, w1, w2)
        out = bufs.combine(y, send.pair_row, w)
        assert torch.cuda.memory_allocated() == before, "a step allocated memory"
        s = step(logits, x, w1, w2, k)
        assert torch.equal(out, s["out"]) and torch.equal(y, s["y"])
    with pytest.raises(ValueError, match="intermediate"):
        moe.MoeBuffers(4, H, E, k).experts(buf, w1, w2)
    with pytest.raises(ValueError, match="at most"):
        bufs.experts(torch.empty((65, H), dtype=BF, device=DEV), w1, w2)


def test_rows_past_32_bit_offsets():
    """Row offsets past 2^32 bytes on both sides of a product and in its gradients."""
    rows, K, N = 1_100_000, 2048, 64  # 4.5 GB of rows
    g = gen(27)
    x = torch.zeros((rows, K), dtype=BF, device=DEV)
    counts = [rows - 300, 37, 0, 263]
    off = offsets_of(counts)
    x[-300:] = ints(g, -2, 2, 300, K)
    w = ints(g, -2, 2, 4, N, K)
    y, _ = moe.moe_expert_matmul(x, off, w)
    for e, a, b in [(1, rows - 300, rows - 263), (3, rows - 263, rows)]:
        assert_bits(y[a:b], x[a:b].double() @ w[e].double().t(), f"y of expert {e}")
    assert bool((y[: rows - 300] == 0).all())
    dy = torch.zeros((rows, N), dtype=BF, device=DEV)
    dy[-300:] = ints(g, -2, 2, 300, N)
    r = moe.moe_expert_matmul_backward(dy, x, off, w, dw_dtype=torch.float32, need_dbias=True)
    for e, a, b in [(1, rows - 300, rows - 263), (3, rows - 263, rows)]:
        assert_bits(r.dx[a:b], dy[a:b].double() @ w[e].double(), f"dx of expert {e}")
        assert_bits(r.dw[e], dy[a:b].double().t() @ x[a:b].double(), f"dw of expert {e}")
        assert_bits(r.dbias[e], dy[a:b].double().sum(0), f"dbias of expert {e}")
    assert bool((r.dw[0] == 0).all()) and bool((r.dx[: rows - 300] == 0).all())


def test_weights_past_32_bit_offsets():
    """An expert whose weights start past 2^32 bytes, and whose up half lies 2^31 behind its gate."""
    E, H, I = 2, 16384, 65536  # 4.3 GB an expert, 2.1 GB from gate to up
    g = gen(28)
    w = torch.zeros((E, 2 * I, H), dtype=BF, device=DEV)
    cols = torch.arange(I - 300, I, device=DEV)
    w[1, cols] = ints(g, -1, 1, 300, H)
    w[1, I + cols] = ints(g, -1, 1, 300, H)
    x = torch.zeros((5, H), dtype=BF, device=DEV)
    x[:, ::97] = ints(g, -1, 1, 5, len(range(0, H, 97)))
    h, gu = moe.moe_expert_gated(x, offsets_of([2, 3]), w, act="relu", save_gate_up=True)
    z = x[2:].double() @ torch.cat([w[1, cols], w[1, I + cols]]).double().t()
    assert_bits(gu[2:, I - 300:I], z[:, :300], "gate")
    assert_bits(gu[2:, 2 * I - 300:], z[:, 300:], "up")
    assert_bits(h[2:, I - 300:], z[:, :300].clamp(min=0) * z[:, 300:], "h")
    assert bool((h[:2] == 0).all()) and bool((h[2:, : I - 300] == 0).all())


def test_refusals():
    g = gen(29)
    E, H, I, P = 4, 64, 72, 20
    off = offsets_of([5, 5, 5, 5])
    x, w1, w2 = normal(g, P, H), normal(g, E, 2 * I, H), normal(g, E, H, I)
    h, gu = moe.moe_expert_gated(x, off, w1, save_gate_up=True)
    y, _ = moe.moe_expert_matmul(h, off, w2)
    torch.cuda.synchronize()
    bad = [
        (ValueError, "w_gate_up must be", lambda: moe.moe_expert_gated(x, off, w2)),
        (ValueError, "w_gate_up must be", lambda: moe.moe_expert_gated(x, off, w1[:, 1:].contiguous())),
        (ValueError, "contiguous", lambda: moe.moe_expert_gated(x.t(), off, w1)),
        (ValueError, "contiguous", lambda: moe.moe_expert_gated(x, off, w1.transpose(1, 2))),
        (ValueError, "expert_offsets must be", lambda: moe.moe_expert_gated(x, off[:-1], w1)),
        (TypeError, "int32", lambda: moe.moe_expert_gated(x, off.long(), w1)),
        (TypeError, "bfloat16", lambda: moe.moe_expert_gated(x.half(), off, w1)),
        (ValueError, "act must be", lambda: moe.moe_expert_gated(x, off, w1, "tanh")),
        (ValueError, "h must be", lambda: moe.moe_expert_gated(x, off, w1, h=y)),
        (ValueError, "device", lambda: moe.moe_expert_gated(x, off.cpu(), w1)),
        (moe.MoeError, "invalid", lambda: moe.moe_expert_gated(x, off, w1, "none")),
        (moe.MoeError, "alignment", lambda: moe.moe_expert_matmul(normal(g, P, 12), off, normal(g, E, 8, 12))),
        (ValueError, "w must be", lambda: moe.moe_expert_matmul(x, off, w2)),
        (ValueError, "bias must have", lambda: moe.moe_expert_matmul(h, off, w2, bias=normal(g, H))),
        (ValueError, "residual must be", lambda: moe.moe_expert_matmul(h, off, w2, residual=h)),
        (ValueError, "pre", lambda: moe.moe_expert_matmul_backward(y, h, off, w2, act="silu")),
        (ValueError, "dpre is written", lambda: moe.moe_expert_matmul_backward(y, h, off, w2, dpre=y)),
        (ValueError, "dy must be", lambda: moe.moe_expert_matmul_backward(h, h, off, w2)),
        (TypeError, "dw must be", lambda: moe.moe_expert_matmul_backward(y, h, off, w2,
                                                                         dw_dtype=torch.float16)),
        (ValueError, "dw must be", lambda: moe.moe_expert_matmul_backward(y, h, off, w2, dw=w1)),
        (ValueError, "dh must be", lambda: moe.moe_expert_gated_backward(y, gu, x, off, w1)),
        (ValueError, "gate_up must be", lambda: moe.moe_expert_gated_backward(h, h, x, off, w1)),
        (ValueError, "dout must be", lambda: moe.moe_combine_backward(
            h, y, torch.zeros((10, 2), dtype=torch.int32, device=DEV), torch.ones((10, 2), device=DEV))),
        (ValueError, "capacity", lambda: moe.moe_combine_backward(
            y[:10], y, torch.zeros((10, 2), dtype=torch.int32, device=DEV),
            torch.ones((10, 2), device=DEV), capacity=21)),
        (moe.MoeError, "capacity", lambda: moe.moe_combine_backward(
            y[:10], y, torch.zeros((10, 2), dtype=torch.int32, device=DEV),
            torch.ones((10, 2), device=DEV), capacity=19)),
    ]
    for i, (kind, text, call) in enumerate(bad):
        with pytest.raises(kind, match=text):
            call()
            pytest.fail(f"call {i} was accepted")
    # a refused call has left no error behind for the next one
    h2, _ = moe.moe_expert_gated(x, off, w1)
    assert torch.equal(h2, h)


def test_views_at_any_aligned_offset():
    """Contiguous views into larger tensors at 16-byte steps, and none at others."""
    g = gen(30)
    E, H, I, P = 3, 72, 40, 11
    flat = normal(g, P * H + 64)
    w = normal(g, E, 2 * I, H, scale=H**-0.5)
    off = offsets_of([4, 0, 7])
    for shift in (8, 24, 40):
        x = flat[shift:shift + P * H].view(P, H)
        h, _ = moe.moe_expert_gated(x, off, w)
        ref, _ = moe.moe_expert_gated(x.clone(), off, w)
        assert torch.equal(h, ref)
    with pytest.raises(moe.MoeError, match="alignment"):
        moe.moe_expert_gated(flat[1:1 + P * H].view(P, H), off, w)
