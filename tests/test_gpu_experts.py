"""The experts' products, their gradients and combine's gradient on the GPU
against their definitions in 64 bits (bounds in expertshelp)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import combine_topk_route_amd as moe
    from expertshelp import (BF, DEV, HALF, act64, assert_bits, assert_within, gen, ints, normal,
                             offsets_of, product64, slope64, spans, weight64)

# Rows of each expert: none, one, and both sides of every tile height.
COUNTS = {
    "one_row": [1],
    "empty_between": [0, 3, 0, 0, 17, 1, 0],
    "heights": [15, 16, 17, 31, 32, 33, 63, 64, 65],
    "tall": [127, 128, 129, 255, 256, 257],
    "hot": [2, 700, 0, 5, 40],
    "many": [(7 * e) % 5 for e in range(300)],
    "none": [0, 0, 0],
}
# Inner and outer features: the smallest, both sides of the tiles, odd multiples of 8.
SIZES = [(8, 8), (64, 64), (72, 136), (120, 264), (520, 248), (1000, 72), (256, 520)]
SMALL = ["one_row", "empty_between", "hot"]
CASES = [(c, 72, 136) for c in COUNTS] + [(c, a, b) for c in SMALL for a, b in SIZES] \
    + [("tall", 256, 520), ("tall", 520, 248), ("many", 8, 8)]
CASES = sorted(set(CASES))
PAD = 5  # rows in front of the first expert and behind the last one


def rows_of(counts):
    return sum(counts) + 2 * PAD


def fill(t, sp, value):
    """`value` in the rows that belong to no expert."""
    inside = torch.zeros(t.shape[0], dtype=torch.bool, device=t.device)
    for _, a, b in sp:
        inside[a:b] = True
    t[~inside] = value
    return inside


@pytest.mark.parametrize("name,K,N", CASES)
def test_matmul_exact(name, K, N):
    counts = COUNTS[name]
    g = gen(1)
    P, E, sp = rows_of(counts), len(counts), spans(counts, PAD)
    x, w = ints(g, -2, 2, P, K), ints(g, -2, 2, E, N, K)
    inside = fill(x, sp, float("nan"))
    y = torch.full((P, N), 77.0, dtype=BF, device=DEV)
    moe.moe_expert_matmul(x, offsets_of(counts, PAD), w, y=y)
    want, _ = product64(torch.where(inside[:, None], x, 0), w, sp)
    assert_bits(y[inside], want[inside], "y")
    assert bool((y[~inside] == 77).all()), "rows outside the experts were written"


@pytest.mark.parametrize("name,K,N", [("hot", 72, 136), ("heights", 520, 248), ("one_row", 8, 8),
                                      ("tall", 120, 264), ("empty_between", 256, 520)])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
def test_matmul_epilogue(name, K, N, act):
    counts = COUNTS[name]
    g = gen(2)
    P, E, sp = rows_of(counts), len(counts), spans(counts, PAD)
    x, w = normal(g, P, K), normal(g, E, N, K, scale=2 * K**-0.5)
    bias, res = normal(g, E, N), normal(g, P, N)
    off = offsets_of(counts, PAD)
    y, pre = moe.moe_expert_matmul(x, off, w, bias=bias, act=act, residual=res, save_pre=True)
    z, mag = product64(x, w, sp)
    inside = torch.zeros(P, dtype=torch.bool, device=DEV)
    for e, a, b in sp:
        z[a:b] += bias[e].double()
        inside[a:b] = True
    zerr = (K + 1) * 2.0**-23 * (mag + bias.double().abs().max())
    assert_within(pre[inside], z[inside], (HALF * z.abs() + zerr)[inside], "pre")
    want = act64(z, act) + res.double()
    # |act'| <= 1.2; the activation's own fp32 arithmetic is within 2^-18 of |z| + 1
    tol = HALF * want.abs() + 1.2 * zerr * 1.01 + 2.0**-18 * (z.abs() + 1)
    assert_within(y[inside], want[inside], tol[inside], "y")
    # the parts alone, and the residual overwritten in place
    plain, none = moe.moe_expert_matmul(x, off, w, act=act)
    assert none is None
    z0, _ = product64(x, w, sp)
    assert_within(plain[inside], act64(z0, act)[inside],
                  (HALF * z0.abs() + 1.3 * zerr + 2.0**-18 * (z0.abs() + 1))[inside], "act alone")
    over = res.clone()
    moe.moe_expert_matmul(x, off, w, bias=bias, act=act, residual=over, y=over)
    assert torch.equal(over[inside], y[inside]) and torch.equal(over[~inside], res[~inside])


@pytest.mark.parametrize("name,H,I", CASES)
def test_gated_exact(name, H, I):
    counts = COUNTS[name]
    g = gen(3)
    P, E, sp = rows_of(counts), len(counts), spans(counts, PAD)
    # |gate|, |up| <= 2 H: their product stays below 2^24
    x, w = ints(g, -1, 1, P, H), ints(g, -2, 2, E, 2 * I, H)
    inside = fill(x, sp, float("inf"))
    h = torch.full((P, I), 77.0, dtype=BF, device=DEV)
    gu = torch.full((P, 2 * I), 77.0, dtype=BF, device=DEV)
    off = offsets_of(counts, PAD)
    moe.moe_expert_gated(x, off, w, act="relu", h=h, gate_up=gu)
    z, _ = product64(torch.where(inside[:, None], x, 0), w, sp)
    assert_bits(gu[inside], z[inside], "gate_up")
    assert_bits(h[inside], (z[:, :I].clamp(min=0) * z[:, I:])[inside], "h")
    assert bool((h[~inside] == 77).all()) and bool((gu[~inside] == 77).all())
    h2, none = moe.moe_expert_gated(x, off, w, act="relu")
    assert none is None and torch.equal(h2[inside], h[inside])


@pytest.mark.parametrize("name,H,I", [("hot", 72, 136), ("heights", 520, 248), ("one_row", 8, 8),
                                      ("tall", 256, 520), ("many", 64, 64)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_activations(name, H, I, act):
    counts = COUNTS[name]
    g = gen(4)
    P, E, sp = rows_of(counts), len(counts), spans(counts, PAD)
    x, w = normal(g, P, H), normal(g, E, 2 * I, H, scale=3 * H**-0.5)
    h, _ = moe.moe_expert_gated(x, offsets_of(counts, PAD), w, act=act)
    z, mag = product64(x, w, sp)
    inside = torch.zeros(P, dtype=torch.bool, device=DEV)
    for _, a, b in sp:
        inside[a:b] = True
    gate, up = z[:, :I], z[:, I:]
    err = H * 2.0**-23 * mag
    ge, ue = err[:, :I], err[:, I:]
    want = act64(gate, act) * up
    tol = HALF * want.abs() + (1.2 * ge + 2.0**-18 * (gate.abs() + 1)) * (up.abs() + ue) \
        + gate.abs() * ue
    assert_within(h[inside], want[inside], tol[inside], "h")


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_far_arguments_stay_finite(act):
    """Factors of some thousands either way: the activations reach 0 or the
    identity, and their slopes 0 or 1, without an infinity or a NaN."""
    H = I = 64
    x = torch.zeros((4, H), dtype=BF, device=DEV)
    x[:, 0] = torch.tensor([-8192.0, -100.0, 100.0, 8192.0])
    w = torch.zeros((1, 2 * I, H), dtype=BF, device=DEV)
    w[0, :, 0] = 1
    off = offsets_of([4])
    h, gu = moe.moe_expert_gated(x, off, w, act=act, save_gate_up=True)
    want = torch.tensor([0.0, 0.0, 1e4, 2.0**26], device=DEV)
    assert_bits(h, want[:, None].expand(4, I).double(), "h")
    dh = torch.ones((4, I), dtype=BF, device=DEV)
    r = moe.moe_expert_gated_backward(dh, gu, x, off, w, act=act)
    assert_bits(r.dgate_up[:, 0], torch.tensor([0.0, 0.0, 100.0, 8192.0], device=DEV).double(), "dg")
    assert_bits(r.dgate_up[:, I], torch.tensor([0.0, 0.0, 100.0, 8192.0], device=DEV).double(), "du")
    assert bool(torch.isfinite(r.dx.float()).all() and torch.isfinite(r.dw.float()).all())


@pytest.mark.parametrize("name,K,N", CASES)
def test_matmul_backward_exact(name, K, N):
    counts = COUNTS[name]
    g = gen(5)
    P, E, sp = rows_of(counts), len(counts), spans(counts, PAD)
    x, w, dy = ints(g, -2, 2, P, K), ints(g, -2, 2, E, N, K), ints(g, -2, 2, P, N)
    inside = fill(x, sp, float("nan"))
    fill(dy, sp, float("inf"))
    off = offsets_of(counts, PAD)
    dx = torch.full((P, K), 77.0, dtype=BF, device=DEV)
    r = moe.moe_expert_matmul_backward(dy, x, off, w, dx=dx, need_dbias=True)
    assert r.dpre is None
    x0, d0 = torch.where(inside[:, None], x, 0), torch.where(inside[:, None], dy, 0)
    want, _ = product64(d0, w.transpose(1, 2), sp)
    assert_bits(dx[inside], want[inside], "dx")
    assert bool((dx[~inside] == 77).all()), "rows outside the experts were written"
    ww, _ = weight64(d0, x0, sp, E)
    assert_bits(r.dw, ww, "dw")
    db = torch.stack([d0[a:b].double().sum(0) for _, a, b in sp])
    assert_bits(r.dbias, db, "dbias")
    r32 = moe.moe_expert_matmul_backward(dy, x, off, w, need_dx=False, dw_dtype=torch.float32)
    assert r32.dx is None and r32.dw.dtype == torch.float32
    assert_bits(r32.dw, ww, "dw in fp32")


@pytest.mark.parametrize("name,K,N", [("hot", 72, 136), ("heights", 520, 248), ("one_row", 8, 8),
                                      ("tall", 256, 520), ("empty_between", 64, 64)])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_matmul_backward_activations(name, K, N, act):
    counts = COUNTS[name]
    g = gen(6)
    P, E, sp = rows_of(counts), len(counts), spans(counts, PAD)
    x, w = normal(g, P, K), normal(g, E, N, K, scale=K**-0.5)
    dy, pre = normal(g, P, N), normal(g, P, N, scale=2.0)
    inside = fill(dy, sp, float("nan"))
    off = offsets_of(counts, PAD)
    r = moe.moe_expert_matmul_backward(dy, x, off, w, act=act, pre=pre, need_dbias=True)
    z = pre.double()
    d = torch.where(inside[:, None], dy.double() * slope64(z, act), 0)
    derr = 2.0**-18 * torch.where(inside[:, None], dy.double().abs(), 0) * (z.abs() + 1)
    assert_within(r.dpre[inside], d[inside], (HALF * d.abs() + derr)[inside], "dpre")
    db = torch.stack([d[a:b].sum(0) for _, a, b in sp])
    dbt = torch.stack([(derr[a:b] + (b - a) * 2.0**-23 * d[a:b].abs()).sum(0) for _, a, b in sp])
    assert_within(r.dbias, db, dbt * 1.01, "dbias")
    # dx and dw from dpre as it is stored
    dp = torch.where(inside[:, None], r.dpre, 0)
    want, mag = product64(dp, w.transpose(1, 2), sp)
    assert_within(r.dx[inside], want[inside],
                  (HALF * want.abs() + N * 2.0**-23 * mag)[inside], "dx")
    ww, wmag = weight64(dp, x, sp, E)
    assert_within(r.dw, ww, HALF * ww.abs() + max(counts) * 2.0**-23 * wmag, "dw")


@pytest.mark.parametrize("name,H,I", CASES)
def test_gated_backward_exact(name, H, I):
    counts = COUNTS[name]
    g = gen(7)
    P, E, sp = rows_of(counts), len(counts), spans(counts, PAD)
    x, w = ints(g, -2, 2, P, H), ints(g, -2, 2, E, 2 * I, H)
    gu, dh = ints(g, -8, 8, P, 2 * I), ints(g, -2, 2, P, I)
    inside = fill(x, sp, float("nan"))
    fill(dh, sp, float("inf"))
    off = offsets_of(counts, PAD)
    dx = torch.full((P, H), 77.0, dtype=BF, device=DEV)
    dgu = torch.full((P, 2 * I), 77.0, dtype=BF, device=DEV)
    r = moe.moe_expert_gated_backward(dh, gu, x, off, w, act="relu", dx=dx, dgate_up=dgu)
    gate, up = gu[:, :I].double(), gu[:, I:].double()
    d = torch.cat([dh.double() * up * (gate > 0), dh.double() * gate.clamp(min=0)], 1)
    d = torch.where(inside[:, None], d, 0)
    assert_bits(dgu[inside], d[inside], "dgate_up")
    want, _ = product64(d, w.transpose(1, 2), sp)
    assert_bits(dx[inside], want[inside], "dx")
    assert bool((dx[~inside] == 77).all()), "rows outside the experts were written"
    assert bool((dgu[~inside] == 77).all())
    ww, _ = weight64(d, torch.where(inside[:, None], x, 0), sp, E)
    assert_bits(r.dw, ww, "dw")
    r32 = moe.moe_expert_gated_backward(dh, gu, x, off, w, act="relu", need_dx=False,
                                        dw_dtype=torch.float32)
    assert r32.dx is None
    assert_bits(r32.dw, ww, "dw in fp32")


@pytest.mark.parametrize("name,H,I", [("hot", 72, 136), ("heights", 520, 248), ("one_row", 8, 8)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_backward_activations(name, H, I, act):
    counts = COUNTS[name]
    g = gen(8)
    P, E, sp = rows_of(counts), len(counts), spans(counts, PAD)
    x, w = normal(g, P, H), normal(g, E, 2 * I, H, scale=H**-0.5)
    gu, dh = normal(g, P, 2 * I, scale=2.0), normal(g, P, I)
    inside = fill(dh, sp, float("nan"))
    off = offsets_of(counts, PAD)
    r = moe.moe_expert_gated_backward(dh, gu, x, off, w, act=act)
    gate, up = gu[:, :I].double(), gu[:, I:].double()
    dh64 = torch.where(inside[:, None], dh.double(), 0)
    d = torch.cat([dh64 * up * slope64(gate, act), dh64 * act64(gate, act)], 1)
    size = dh64.abs() * (gate.abs() + 1)
    derr = 2.0**-18 * torch.cat([size * up.abs(), size], 1)
    assert_within(r.dgate_up[inside], d[inside], (HALF * d.abs() + derr)[inside], "dgate_up")
    dp = torch.where(inside[:, None], r.dgate_up, 0)
    want, mag = product64(dp, w.transpose(1, 2), sp)
    assert_within(r.dx[inside], want[inside],
                  (HALF * want.abs() + 2 * I * 2.0**-23 * mag)[inside], "dx")
    ww, wmag = weight64(dp, x, sp, E)
    assert_within(r.dw, ww, HALF * ww.abs() + max(counts) * 2.0**-23 * wmag, "dw")


def test_no_rows():
    off = offsets_of([0, 0])
    w = torch.ones((2, 16, 8), dtype=BF, device=DEV)
    x = torch.empty((0, 8), dtype=BF, device=DEV)
    h, gu = moe.moe_expert_gated(x, off, w, save_gate_up=True)
    assert h.shape == (0, 8) and gu.shape == (0, 16)
    y, _ = moe.moe_expert_matmul(x, off, w)
    assert y.shape == (0, 16)
    r = moe.moe_expert_gated_backward(h, gu, x, off, w)
    assert r.dx.shape == (0, 8) and bool((r.dw == 0).all())
    r = moe.moe_expert_matmul_backward(y, x, off, w, need_dbias=True)
    assert bool((r.dw == 0).all()) and bool((r.dbias == 0).all())
    r = moe.moe_expert_matmul_backward(y, x, off, w, act="silu", pre=y, need_dbias=True)
    assert bool((r.dw == 0).all()) and bool((r.dbias == 0).all())


def test_offsets_outside_the_buffer_are_held_to_it():
    """Offsets past the buffer, below zero or out of order: the rows they name
    inside the buffer are computed, nothing else is read or written."""
    g = gen(9)
    x, w = ints(g, -2, 2, 40, 64), ints(g, -2, 2, 4, 72, 64)
    off = torch.tensor([-7, 10, 4, 30, 1000], dtype=torch.int32, device=DEV)
    y = torch.full((40, 72), 77.0, dtype=BF, device=DEV)
    moe.moe_expert_matmul(x, off, w, y=y)
    # expert 0: [0, 10), expert 1: none, expert 2: [4, 30), expert 3: [30, 40)
    for e, a, b in [(0, 0, 4), (2, 10, 30), (3, 30, 40)]:
        assert_bits(y[a:b], x[a:b].double() @ w[e].double().t(), f"expert {e}")
    r = moe.moe_expert_matmul_backward(y.clamp(-2, 2), x, off, w)
    assert bool((r.dw[1] == 0).all()) and bool(torch.isfinite(r.dw.float()).all())


@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (3, 2, 64), (131, 6, 2056), (16, 8, 520), (5, 32, 72),
                                   (40, 3, 7168)])
def test_combine_backward(T, k, H):
    g = gen(10)
    cap = T * k + 3
    row = torch.randperm(cap, generator=g, device=DEV)[:T * k].to(torch.int32).view(T, k)
    row[0, 0] = -1 if T > 1 else row[0, 0]
    if T > 2:
        row[2, 1] = cap  # past the buffer: skipped as combine skips it
    dout, y = normal(g, T, H), normal(g, cap, H)
    w = torch.rand((T, k), generator=g, device=DEV)
    dy = torch.full((cap, H), 77.0, dtype=BF, device=DEV)
    _, dw = moe.moe_combine_backward(dout, y, row, w, dy=dy)
    want = torch.full((cap, H), 77.0, dtype=BF, device=DEV)
    for t in range(T):
        for j in range(k):
            r = int(row[t, j])
            if not 0 <= r < cap:
                assert float(dw[t, j]) == 0
                continue
            want[r] = (w[t, j] * dout[t].float()).to(BF)  # one fp32 product, one rounding
            terms = dout[t].double() * y[r].double()
            assert abs(float(dw[t, j]) - float(terms.sum())) <= H * 2.0**-23 * float(terms.abs().sum())
    assert torch.equal(dy, want)


def test_repeated_calls_give_the_same_bits():
    counts = COUNTS["hot"]
    g = gen(11)
    P, E = sum(counts), len(counts)
    x, w, dh = normal(g, P, 520), normal(g, E, 496, 520), normal(g, P, 248)
    off = offsets_of(counts)
    first = None
    for _ in range(3):
        h, gu = moe.moe_expert_gated(x, off, w, save_gate_up=True)
        r = moe.moe_expert_gated_backward(dh, gu, x, off, w)
        got = [t.view(torch.int16) for t in (h, gu, r.dx, r.dw, r.dgate_up)]
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        first = got


# Rows for tall tiles: every height, both sides of 256 and 288, spread over two and three tiles.
TALL = [257, 288, 289, 255, 600, 1, 0, 700, 33, 64, 96, 161]


def assert_rows_written(t, sp, mark):
    inside = fill(t.clone(), sp, 0)
    assert bool((t[~inside] == mark).all()), "rows outside the experts were written"


@pytest.mark.parametrize("K", [72, 64, 520])
def test_tall_tiles_exact(K):
    """Enough rows and outputs for the tall tiles, forward and data gradient."""
    g = gen(12)
    N = 4112
    P, E, sp = rows_of(TALL), len(TALL), spans(TALL, PAD)
    off = offsets_of(TALL, PAD)
    x, w, dy = ints(g, -2, 2, P, K), ints(g, -2, 2, E, N, K), ints(g, -2, 2, P, K)
    inside = fill(x, sp, float("nan"))
    y = torch.full((P, N), 77.0, dtype=BF, device=DEV)
    moe.moe_expert_matmul(x, off, w, y=y)
    x0 = torch.where(inside[:, None], x, 0)
    want, _ = product64(x0, w, sp)
    assert_bits(y[inside], want[inside], "y")
    assert_rows_written(y, sp, 77)
    # the data gradient of a product with K outputs and N inputs
    wt = w.transpose(1, 2).contiguous()
    dx = torch.full((P, N), 77.0, dtype=BF, device=DEV)
    fill(dy, sp, float("inf"))
    moe.moe_expert_matmul_backward(dy, torch.zeros((P, N), dtype=BF, device=DEV), off, wt, dx=dx,
                                   need_dw=False)
    want, _ = product64(torch.where(inside[:, None], dy, 0), w, sp)
    assert_bits(dx[inside], want[inside], "dx")
    assert_rows_written(dx, sp, 77)
    # the gated block: N = 2 I, |gate| and |up| at most 2 K, their product below 2^24
    z, _ = product64(torch.clamp(x0, -1, 1), w, sp)
    h, gu = moe.moe_expert_gated(x.clamp(-1, 1), off, w, act="relu", save_gate_up=True)
    assert_bits(gu[inside], z[inside], "gate_up")
    assert_bits(h[inside], (z[:, :N // 2].clamp(min=0) * z[:, N // 2:])[inside], "h")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_tall_tiles_epilogue(act):
    g = gen(13)
    K, N = 136, 4112
    P, E, sp = rows_of(TALL), len(TALL), spans(TALL, PAD)
    off = offsets_of(TALL, PAD)
    x, w = normal(g, P, K), normal(g, E, N, K, scale=K**-0.5)
    bias, res = normal(g, E, N), normal(g, P, N)
    y, pre = moe.moe_expert_matmul(x, off, w, bias=bias, act=act, residual=res, save_pre=True)
    z, mag = product64(x, w, sp)
    inside = fill(x.clone(), sp, 0)
    for e, a, b in sp:
        z[a:b] += bias[e].double()
    zerr = (K + 1) * 2.0**-23 * (mag + bias.double().abs().max())
    assert_within(pre[inside], z[inside], (HALF * z.abs() + zerr)[inside], "pre")
    want = act64(z, act) + res.double()
    tol = HALF * want.abs() + 1.22 * zerr + 2.0**-18 * (z.abs() + 1)
    assert_within(y[inside], want[inside], tol[inside], "y")
    over = res.clone()
    moe.moe_expert_matmul(x, off, w, bias=bias, act=act, residual=over, y=over)
    assert torch.equal(over[inside], y[inside]) and torch.equal(over[~inside], res[~inside])


# One sequence of tiles a CU: lengths from no stage to several, tiles of the same expert apart.
SEQUENCE = [0, 1, 63, 64, 65, 0, 0, 128, 129, 700, 5, 0, 191, 192, 193, 2, 300, 31, 32, 0, 77, 256, 1, 0]


@pytest.mark.parametrize("N,K", [(1032, 776), (1288, 1160)])
@pytest.mark.parametrize("counts", [SEQUENCE, [0] * 23 + [9], [0] * 24], ids=["mixed", "one", "none"])
def test_weight_gradient_sequences(N, K, counts):
    g = gen(14)
    P, E, sp = rows_of(counts), len(counts), spans(counts, PAD)
    off = offsets_of(counts, PAD)
    x, d, w = ints(g, -2, 2, P, K), ints(g, -2, 2, P, N), torch.zeros((E, N, K), dtype=BF, device=DEV)
    inside = fill(x, sp, float("nan"))
    fill(d, sp, float("inf"))
    want, _ = weight64(torch.where(inside[:, None], d, 0), torch.where(inside[:, None], x, 0), sp, E)
    for dtype in (BF, torch.float32):
        dw = torch.full((E, N, K), 77.0, dtype=dtype, device=DEV)
        moe.moe_expert_matmul_backward(d, x, off, w, dw=dw, need_dx=False)
        assert_bits(dw, want, f"dw as {dtype}")


@pytest.mark.parametrize("per", [5, 200])
def test_weights_beyond_the_cache(per):
    """Weights over 256 MiB, which go past the caches: few rows an expert and about a tall tile's."""
    g = gen(15)
    E, N, K = 64, 2048, 1088
    counts = [(per + 37 * e) % (2 * per + 1) for e in range(E)]
    P, sp = rows_of(counts), spans(counts, PAD)
    off = offsets_of(counts, PAD)
    x, w, d = ints(g, -1, 1, P, K), ints(g, -2, 2, E, N, K), ints(g, -2, 2, P, N)
    inside = fill(x, sp, float("nan"))
    x0 = torch.where(inside[:, None], x, 0)
    z, _ = product64(x0, w, sp)
    y, _ = moe.moe_expert_matmul(x, off, w)
    assert_bits(y[inside], z[inside], "y")
    _, gu = moe.moe_expert_gated(x, off, w, save_gate_up=True)
    assert_bits(gu[inside], z[inside], "gate_up")
    r = moe.moe_expert_matmul_backward(d, x, off, w, need_dw=False)
    want, _ = product64(torch.where(inside[:, None], d, 0), w.transpose(1, 2), sp)
    assert_bits(r.dx[inside], want[inside], "dx")


# Few rows and few outputs, where a block's waves share the inner axis: runs around a tile's 32 rows,
# all rows at one expert of many, one row each.
FEW = {
    "heights": [31, 0, 32, 33, 1, 15, 16, 17, 2],
    "one_of_many": [0] * 20 + [600] + [0] * 11,
    "each_one": [1] * 40,
}


@pytest.mark.parametrize("name", FEW)
@pytest.mark.parametrize("K,N", [(8, 48), (24, 16), (256, 80), (1016, 48), (1032, 112), (2312, 48),
                                 (264, 1008)])
def test_few_rows_exact(name, K, N):
    counts = FEW[name]
    g = gen(16)
    P, E, sp, I = rows_of(counts), len(counts), spans(counts, PAD), N // 2
    off = offsets_of(counts, PAD)
    # |gate|, |up| <= K: their product stays below 2^24
    x, w = ints(g, -1, 1, P, K), ints(g, -1, 1, E, N, K)
    inside = fill(x, sp, float("nan"))
    y = torch.full((P, N), 77.0, dtype=BF, device=DEV)
    moe.moe_expert_matmul(x, off, w, y=y)
    z, _ = product64(torch.where(inside[:, None], x, 0), w, sp)
    assert_bits(y[inside], z[inside], "y")
    assert_rows_written(y, sp, 77.0)
    h = torch.full((P, I), 77.0, dtype=BF, device=DEV)
    gu = torch.full((P, N), 77.0, dtype=BF, device=DEV)
    moe.moe_expert_gated(x, off, w, act="relu", h=h, gate_up=gu)
    assert_bits(gu[inside], z[inside], "gate_up")
    assert_bits(h[inside], (z[:, :I].clamp(min=0) * z[:, I:])[inside], "h")
    assert_rows_written(h, sp, 77.0)
    assert_rows_written(gu, sp, 77.0)
    alone, none = moe.moe_expert_gated(x, off, w, act="relu")
    assert none is None and torch.equal(alone[inside], h[inside])


@pytest.mark.parametrize("name", FEW)
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
def test_few_rows_epilogue(name, act):
    counts = FEW[name]
    g = gen(17)
    K, N = 1288, 104
    P, E, sp = rows_of(counts), len(counts), spans(counts, PAD)
    off = offsets_of(counts, PAD)
    x, w = normal(g, P, K), normal(g, E, N, K, scale=K**-0.5)
    bias, res = normal(g, E, N), normal(g, P, N)
    y, pre = moe.moe_expert_matmul(x, off, w, bias=bias, act=act, residual=res, save_pre=True)
    z, mag = product64(x, w, sp)
    inside = fill(x.clone(), sp, 0)
    for e, a, b in sp:
        z[a:b] += bias[e].double()
    zerr = (K + 1) * 2.0**-23 * (mag + bias.double().abs().max())
    assert_within(pre[inside], z[inside], (HALF * z.abs() + zerr)[inside], "pre")
    want = act64(z, act) + res.double()
    tol = HALF * want.abs() + 1.22 * zerr + 2.0**-18 * (z.abs() + 1)
    assert_within(y[inside], want[inside], tol[inside], "y")
    over = res.clone()
    moe.moe_expert_matmul(x, off, w, bias=bias, act=act, residual=over, y=over)
    assert torch.equal(over[inside], y[inside]) and torch.equal(over[~inside], res[~inside])


@pytest.mark.parametrize("name", ["empty_between", "heights", "tall", "hot", "many"])
@pytest.mark.parametrize("K,N", [(8, 2064), (64, 4096), (72, 2064), (120, 2064), (520, 4112), (1000, 2064)])
def test_wide_products_exact(name, K, N):
    """Few rows against many outputs: the tiles of 128 rows at every height."""
    counts = COUNTS[name]
    g = gen(18)
    P, E, sp, I = rows_of(counts), len(counts), spans(counts, PAD), N // 2
    off = offsets_of(counts, PAD)
    x, w = ints(g, -1, 1, P, K), ints(g, -1, 1, E, N, K)
    inside = fill(x, sp, float("nan"))
    y = torch.full((P, N), 77.0, dtype=BF, device=DEV)
    moe.moe_expert_matmul(x, off, w, y=y)
    z, _ = product64(torch.where(inside[:, None], x, 0), w, sp)
    assert_bits(y[inside], z[inside], "y")
    assert_rows_written(y, sp, 77.0)
    h = torch.full((P, I), 77.0, dtype=BF, device=DEV)
    gu = torch.full((P, N), 77.0, dtype=BF, device=DEV)
    moe.moe_expert_gated(x, off, w, act="relu", h=h, gate_up=gu)
    assert_bits(gu[inside], z[inside], "gate_up")
    assert_bits(h[inside], (z[:, :I].clamp(min=0) * z[:, I:])[inside], "h")
    assert_rows_written(h, sp, 77.0)
    assert_rows_written(gu, sp, 77.0)


@pytest.mark.parametrize("name", ["heights", "hot"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
def test_wide_products_epilogue(name, act):
    counts = COUNTS[name]
    g = gen(19)
    K, N = 136, 2056
    P, E, sp = rows_of(counts), len(counts), spans(counts, PAD)
    off = offsets_of(counts, PAD)
    x, w = normal(g, P, K), normal(g, E, N, K, scale=K**-0.5)
    bias, res = normal(g, E, N), normal(g, P, N)
    y, pre = moe.moe_expert_matmul(x, off, w, bias=bias, act=act, residual=res, save_pre=True)
    z, mag = product64(x, w, sp)
    inside = fill(x.clone(), sp, 0)
    for e, a, b in sp:
        z[a:b] += bias[e].double()
    zerr = (K + 1) * 2.0**-23 * (mag + bias.double().abs().max())
    assert_within(pre[inside], z[inside], (HALF * z.abs() + zerr)[inside], "pre")
    want = act64(z, act) + res.double()
    tol = HALF * want.abs() + 1.22 * zerr + 2.0**-18 * (z.abs() + 1)
    assert_within(y[inside], want[inside], tol[inside], "y")
    over = res.clone()
    moe.moe_expert_matmul(x, off, w, bias=bias, act=act, residual=over, y=over)
    assert torch.equal(over[inside], y[inside]) and torch.equal(over[~inside], res[~inside])


# dbias's strips: 16 columns a block, 64 columns by 1024 threads, 64 columns by 256.
@pytest.mark.parametrize("counts,N", [
    ([700], 8), ([3, 0, 515], 72), ([2100, 31, 0, 1], 24), ([127, 128, 129, 5], 1032), ([600, 1], 4104),
    ([(5 * e) % 9 for e in range(130)], 264),
], ids=["one", "few", "long", "middle", "two", "many"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
def test_bias_gradient(counts, N, act):
    g = gen(20)
    P, E, sp, K = rows_of(counts), len(counts), spans(counts, PAD), 8
    off = offsets_of(counts, PAD)
    x, w = normal(g, P, K), normal(g, E, N, K)
    dy, pre = normal(g, P, N), normal(g, P, N, scale=2.0)
    inside = fill(dy, sp, float("nan"))
    fill(pre, sp, float("inf"))
    dpre = None if act == "none" else torch.full((P, N), 77.0, dtype=BF, device=DEV)
    dbias = torch.full((E, N), 77.0, device=DEV)
    kw = dict(act=act, pre=None if act == "none" else pre, need_dx=False, need_dw=False)
    moe.moe_expert_matmul_backward(dy, x, off, w, dpre=dpre, dbias=dbias, **kw)
    d = dy.double() * slope64(pre.double(), act)
    # the slope's own fp32 arithmetic is within 2^-18 of 1 + |pre|; a sum of n terms within n 2^-23
    derr = 2.0**-18 * (1 + pre.double().abs()) * dy.double().abs() + 2.0**-23 * d.abs()
    if act == "none":
        derr = torch.zeros_like(d)
    for e, a, b in sp:
        want = d[a:b].sum(0)
        tol = derr[a:b].sum(0) + (b - a) * 2.0**-23 * d[a:b].abs().sum(0)
        assert_within(dbias[e], want, tol, f"dbias of expert {e}")
    if act != "none":
        assert_within(dpre[inside], d[inside], (HALF * d.abs() + derr * 1.01)[inside], "dpre")
        assert_rows_written(dpre, sp, 77.0)
        alone = torch.full((P, N), 77.0, dtype=BF, device=DEV)
        moe.moe_expert_matmul_backward(dy, x, off, w, dpre=alone, **kw)
        assert torch.equal(alone, dpre)
    again = torch.empty_like(dbias)
    moe.moe_expert_matmul_backward(dy, x, off, w, dbias=again, **kw)
    assert torch.equal(again, dbias)
