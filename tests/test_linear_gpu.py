"""The matrix product with an epilogue on the GPU (linear_fwd, linear_bwd) against 64-bit products."""
import numpy as np
import pytest
import torch

import gated_convolution_sequence_amd as hc
import layer_ref as ref
from gpu_util import DEV, log
from layer_ref import check, to_np

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ACTS = ("none", "relu", "gelu", "silu", "sigmoid")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.layer_lib()
    yield
    torch.cuda.synchronize()


def inputs(M, N, K, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda *s, scale=1.0: (scale * torch.randn(*s, generator=gen)).to(dtype).to(DEV)
    return dict(x=mk(M, K), w=mk(N, K, scale=max(K, 1) ** -0.5), b=mk(N), r=mk(M, N), dy=mk(M, N))


def check_fwd(t, act, bias, residual, what):
    b, r = (t["b"] if bias else None), (t["r"] if residual else None)
    y, z = hc.linear_fwd(t["x"], t["w"], bias=b, residual=r, act=act, save_preact=True)
    plain, none = hc.linear_fwd(t["x"], t["w"], bias=b, residual=r, act=act)
    assert none is None and torch.equal(plain, y)
    n = lambda v: None if v is None else to_np(v)
    wy, ey, wz, ez = ref.linear_fwd(n(t["x"]), n(t["w"]), n(b), n(r), act)
    check(z, wz, ez, z.dtype, what + " z")
    check(y, wy, ey, y.dtype, what + " y")
    return z


def check_bwd(t, z, act, what, **need):
    got = hc.linear_bwd(t["x"], t["w"], t["dy"], preact=z if act != "none" else None, act=act, **need)
    want = ref.linear_bwd(*(to_np(v) for v in (t["x"], t["w"], z, t["dy"])), act, t["x"].dtype == BF16)
    for name, g, (w, e) in zip(("dx", "dw", "db"), got, want):
        if g is not None:
            check(g, w, e, g.dtype, "%s %s" % (what, name))
    return got


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 4096, 512), (2, 17, 33), (3, 100, 8), (5, 129, 70), (8, 256, 1024), (9, 24, 2048),
          (15, 48, 40), (16, 64, 96), (17, 80, 72), (33, 130, 264), (48, 512, 520), (64, 64, 64), (65, 72, 136),
          (100, 200, 300), (127, 129, 131), (128, 128, 128), (200, 264, 1032), (256, 256, 64), (257, 520, 200),
          (300, 1, 50), (1000, 72, 24), (513, 385, 96), (4, 72, 2056), (16, 100, 4100), (8, 4100, 2056),
          (24, 64, 1032), (31, 8200, 40), (32, 128, 1024), (2100, 1900, 1801)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_sizes(shape, dtype):
    M, N, K = shape
    log("linear %s %s" % (shape, dtype))
    t = inputs(M, N, K, dtype, M + N + K)
    act = ACTS[(M + N + K) % 5]
    z = check_fwd(t, act, True, True, "fwd")
    check_bwd(t, z, act, "bwd")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M", [3, 200])
def test_epilogues(act, bias, residual, M):
    t = inputs(M, 136, 72, BF16, 7)
    z = check_fwd(t, act, bias, residual, "fwd")
    check_bwd(t, z, act, "bwd")


@pytest.mark.parametrize("N,K", [(451, 463), (451, 464), (456, 463)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act,db", [("none", False), ("none", True), ("gelu", False)])
def test_odd_rows(N, K, dtype, act, db):
    """Rows of no whole 16 bytes, inside wider buffers of NaN; workspaces of NaN."""
    M = 500 if act != "none" or db else 5000  # (copies pay off later where they are a launch of their own)
    t = inputs(M, N, K, dtype, 9)

    def wide(v):
        big = torch.full((v.shape[0], v.shape[1] + 13), float("nan"), dtype=dtype, device=DEV)
        big[:, 5:5 + v.shape[1]] = v
        return big[:, 5:5 + v.shape[1]]

    z = check_fwd(t, act, True, False, "fwd")
    ws = torch.full((hc.linear_workspace_bytes(M, N, K, act, 0 if dtype == BF16 else 1, True),), 255,
                    dtype=torch.uint8, device=DEV)
    want = check_bwd(t, z, act, "bwd", need_db=db, workspace=ws)
    for need in ((1, 0), (0, 1)):
        check_bwd(t, z, act, "bwd", need_dx=bool(need[0]), need_dw=bool(need[1]), need_db=db, workspace=ws.fill_(255))
    t["x"], t["dy"] = wide(t["x"]), wide(t["dy"])
    check_fwd(t, act, False, True, "fwd strided")
    check_bwd(t, z, act, "bwd strided", need_db=db, workspace=ws.fill_(255))
    for v in want[:2]:
        assert torch.isfinite(v).all()


@pytest.mark.parametrize("need", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1), (0, 0, 0)])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_parts_of_the_backward(need, act):
    t = inputs(150, 80, 72, BF16, 8)
    _, z = hc.linear_fwd(t["x"], t["w"], act=act, save_preact=True)
    whole = hc.linear_bwd(t["x"], t["w"], t["dy"], preact=z, act=act)
    got = hc.linear_bwd(t["x"], t["w"], t["dy"], preact=z, act=act, need_dx=bool(need[0]), need_dw=bool(need[1]),
                        need_db=bool(need[2]))
    for n, g, w in zip(need, got, whole):
        assert (g is not None) == bool(n)
        if n:
            assert torch.equal(g, w)


@pytest.mark.parametrize("M,N,K", [(1, 200, 96), (7, 96, 200), (40, 320, 128), (130, 257, 72), (300, 512, 256),
                                   (640, 768, 512)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_whole_numbers_are_exact(M, N, K, dtype):
    """Sparse units and small integers: every sum is exact in any order, so every bit is."""
    gen = torch.Generator().manual_seed(M)
    mk = lambda *s: (torch.randint(-1, 2, s, generator=gen) * (torch.rand(s, generator=gen) < 0.2)).float()
    x, w, b, r, dy = mk(M, K), mk(N, K), mk(N), mk(M, N), mk(M, N)
    c = lambda v: v.to(dtype).to(DEV)
    y, _ = hc.linear_fwd(c(x), c(w), bias=c(b), residual=c(r), act="relu")
    assert torch.equal(y.cpu().float(), torch.relu(x @ w.t() + b) + r)
    dx, dw, db = hc.linear_bwd(c(x), c(w), c(dy))
    assert torch.equal(dx.cpu().float(), dy @ w)
    assert torch.equal(dw.cpu().float(), dy.t() @ x)
    assert torch.equal(db.cpu().float(), dy.sum(0))


@pytest.mark.parametrize("dtype,off,pad", [(BF16, 0, 8), (BF16, 8, 24), (BF16, 1, 3), (F32, 4, 4), (F32, 1, 1)])
@pytest.mark.parametrize("M", [4, 100, 300])
def test_strides_and_offsets(dtype, off, pad, M):
    """Rows wider than their features, off any alignment; nothing beside the outputs' columns is written."""
    N, K = 136, 72
    t = inputs(M, N, K, dtype, 11)

    def view(v):
        big = torch.full((off + M * (v.shape[1] + pad),), float("nan"), dtype=dtype, device=DEV)
        out = big[off:].view(M, v.shape[1] + pad)[:, :v.shape[1]]
        out.copy_(v)
        return out

    t.update(x=view(t["x"]), r=view(t["r"]), dy=view(t["dy"]))
    act = "gelu"
    z = check_fwd(t, act, True, True, "fwd")
    check_bwd(t, z, act, "bwd")
    bigs = {n: torch.full((off + M * (c + pad),), 7.0, dtype=dtype, device=DEV) for n, c in (("y", N), ("dx", K))}
    y = bigs["y"][off:].view(M, N + pad)[:, :N]
    dx = bigs["dx"][off:].view(M, K + pad)[:, :K]
    want = hc.linear_fwd(t["x"], t["w"], bias=t["b"], residual=t["r"], act=act)[0]
    hc.linear_fwd(t["x"], t["w"], bias=t["b"], residual=t["r"], act=act, out=y)
    hc.linear_bwd(t["x"], t["w"], t["dy"], preact=z, act=act, dx=dx)
    check(y, to_np(want), 0.0, dtype, "y")
    check(dx, *ref.linear_bwd(*(to_np(v) for v in (t["x"], t["w"], z, t["dy"])), act, dtype == BF16)[0], dtype, "dx")
    for n, c in (("y", N), ("dx", K)):
        assert torch.all(bigs[n][:off] == 7.0) and torch.all(bigs[n][off:].view(M, c + pad)[:, c:] == 7.0)


def test_residual_in_place():
    for M in (3, 300):
        t = inputs(M, 128, 64, BF16, 13)
        want = hc.linear_fwd(t["x"], t["w"], residual=t["r"], act="silu")[0]
        r = t["r"].clone()
        got = hc.linear_fwd(t["x"], t["w"], residual=r, act="silu", out=r)[0]
        assert got is r and torch.equal(r, want)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("M", [3, 130])
def test_non_finite_values_stay_in_their_rows(bad, M):
    """A row of x that is not finite spoils its own outputs only (tiles read past their rows and columns)."""
    t = inputs(M, 100, 72, BF16, 14)
    want, _ = hc.linear_fwd(t["x"], t["w"])
    x = t["x"].clone()
    x[M - 1, 5] = bad
    got, _ = hc.linear_fwd(x, t["w"])
    assert torch.equal(got[:-1], want[:-1]) and not torch.isfinite(got[-1]).any()


def test_empty_sizes():
    e = lambda *s: torch.empty(*s, dtype=BF16, device=DEV)
    b = torch.randn(6, device=DEV).to(BF16)
    for M in (4, 200):
        y, _ = hc.linear_fwd(e(M, 0), e(6, 0), bias=b)
        assert torch.equal(y, b.expand(M, 6))
    y, _ = hc.linear_fwd(e(0, 8), e(6, 8), bias=b)
    assert y.shape == (0, 6)
    dx, dw, db = hc.linear_bwd(e(0, 8), e(6, 8), e(0, 6))
    assert dx.shape == (0, 8) and torch.all(dw == 0) and torch.all(db == 0)
    dx, dw, db = hc.linear_bwd(e(4, 8), e(0, 8), e(4, 0))
    assert torch.all(dx == 0) and dw.shape == (0, 8) and db.shape == (0,)


def test_leading_dimensions():
    t = inputs(60, 40, 24, BF16, 15)
    y, z = hc.linear_fwd(t["x"].view(3, 20, 24), t["w"], residual=t["r"].view(3, 20, 40), act="silu", save_preact=True)
    want, wz = hc.linear_fwd(t["x"], t["w"], residual=t["r"], act="silu", save_preact=True)
    assert y.shape == (3, 20, 40) and torch.equal(y.view(60, 40), want) and torch.equal(z.view(60, 40), wz)
    dx, _, _ = hc.linear_bwd(t["x"].view(3, 20, 24), t["w"], t["dy"].view(3, 20, 40), preact=z, act="silu")
    assert dx.shape == (3, 20, 24)


def test_operand_past_4_gib():
    """x of 4.5 GB: rows at offsets past 2^32 bytes, forward and in dw's contraction."""
    M, N, K, ldx = 70000, 72, 64, 1 << 15
    log("linear past 4 GiB")
    t = inputs(M, N, K, BF16, 16)
    big = torch.empty(M * ldx, dtype=BF16, device=DEV).view(M, ldx)
    x = big[:, 100 * 8:100 * 8 + K]
    x.copy_(t["x"])
    assert torch.equal(hc.linear_fwd(x, t["w"])[0], hc.linear_fwd(t["x"], t["w"])[0])
    got, want = hc.linear_bwd(x, t["w"], t["dy"]), hc.linear_bwd(t["x"], t["w"], t["dy"])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M", [8, 1100])
def test_runs_streams_and_graphs_give_the_same_bits(M):
    N, K = 264, 1032
    n = [hc.linear_workspace_bytes(M, N, K, "silu", 0, bw) for bw in (False, True)]
    ws = [torch.empty(max(16, v), dtype=torch.uint8, device=DEV) for v in n]
    static = inputs(M, N, K, BF16, 20)

    def both(t):
        y, z = hc.linear_fwd(t["x"], t["w"], bias=t["b"], residual=t["r"], act="silu", save_preact=True,
                             workspace=ws[0])
        return (y, z, *hc.linear_bwd(t["x"], t["w"], t["dy"], preact=z, act="silu", workspace=ws[1]))

    want = both(static)
    for _ in range(3):
        for a, b in zip(both(static), want):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, z = hc.linear_fwd(static["x"], static["w"], bias=static["b"], residual=static["r"], act="silu",
                         save_preact=True, stream=side)
    g = hc.linear_bwd(static["x"], static["w"], static["dy"], preact=z, act="silu", stream=side)
    side.synchronize()
    for a, b in zip((y, z, *g), want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both(static)
    for r in range(3):
        for name, v in inputs(M, N, K, BF16, 30 + r).items():
            static[name].copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = [v.clone() for v in outs]
        for a, b in zip(kept, both(static)):
            assert torch.equal(a, b), "replay %d" % r


@pytest.mark.parametrize("act", ACTS)
def test_autograd_against_differences(act):
    """Central differences of the forward in fp32.  Rounding: 2^-23 of a loss of order 1 over a step of 2^-6
    (2^-16); the third derivative over 6 times h^2: 2^-13.  relu: inputs a step away from its corner.
    Bound: 2^-8 of the largest gradient."""
    M, N, K = 3, 5, 4
    t = inputs(M, N, K, F32, 40)
    h = 2.0 ** -6
    if act == "relu":
        z = t["x"] @ t["w"].t() + t["b"]
        assert z.abs().min() > 4 * h * max(1.0, float(t["x"].abs().max()), float(t["w"].abs().max()))
    args = [t[n].clone().requires_grad_(True) for n in ("x", "w", "b", "r")]
    wy = t["dy"] / M

    def loss(*a):
        return (hc.LinearAct.apply(*a, act) * wy).double().sum()

    loss(*args).backward()
    for i, a in enumerate(args):
        num = torch.empty_like(a)
        for j in range(a.numel()):
            vals = []
            for sign in (1, -1):
                moved = a.detach().clone()
                moved.view(-1)[j] += sign * h
                with torch.no_grad():
                    vals.append(loss(*[moved if m == i else o.detach() for m, o in enumerate(args)]))
            num.view(-1)[j] = (vals[0] - vals[1]) / (2 * h)
        assert (num - a.grad).abs().max() <= 2.0 ** -8 * a.grad.abs().max(), i


def test_memory_of_another_stream_is_not_reused_early():
    """A call queued behind long work on a side stream: what it allocated stays its own meanwhile."""
    t = inputs(300, 256, 2048, F32, 60)
    dz = torch.randn(300, 256, device=DEV)
    want = hc.linear_bwd(t["x"], t["w"], t["dy"], preact=dz, act="gelu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some milliseconds
    got = hc.linear_bwd(t["x"], t["w"], t["dy"], preact=dz, act="gelu", stream=side)
    n = hc.linear_workspace_bytes(300, 256, 2048, "gelu", 1, backward=True)
    filled = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all(bool((f == 255).all()) for f in filled)


def test_refusals():
    t = inputs(4, 8, 16, BF16, 50)
    with pytest.raises(ValueError):
        hc.linear_fwd(t["x"], t["w"], act="tanh")
    with pytest.raises(ValueError):
        hc.linear_fwd(t["x"][:, :8], t["w"])
    with pytest.raises(ValueError):
        hc.linear_fwd(t["x"], t["w"].float())
    with pytest.raises(ValueError):
        hc.linear_fwd(t["x"], t["w"], bias=t["b"][:4])
    with pytest.raises(ValueError):
        hc.linear_fwd(t["x"], t["w"], residual=t["x"])
    with pytest.raises(ValueError):
        hc.linear_fwd(torch.zeros(16, 4, dtype=BF16, device=DEV).t(), t["w"])
    with pytest.raises(ValueError):
        hc.linear_bwd(t["x"], t["w"], t["dy"], act="silu")
    sq = torch.zeros(8, 8, dtype=BF16, device=DEV)
    with pytest.raises(hc.LayerError) as e:  # y on top of x
        hc.linear_fwd(sq, torch.zeros(8, 8, dtype=BF16, device=DEV), out=sq)
    assert e.value.status == -6
    with pytest.raises(TypeError):
        hc.linear_fwd(t["x"].half(), t["w"].half())
