"""Layer and root-mean-square norm, forward and backward, against 64 bits."""
import pytest
import torch

import gated_convolution_sequence_amd as hc
import model_ref as ref
from gpu_util import DEV, log
from model_ref import check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.model_lib()
    yield
    torch.cuda.synchronize()


def randn(*shape, seed, dtype=F32, scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(*shape, generator=gen, device=DEV)).to(dtype)


def inputs(M, D, dtype, seed, kind="layer"):
    x = randn(M, D, seed=seed) * (1 + randn(D, seed=seed + 1).abs()) + 0.5 * randn(D, seed=seed + 2)
    return dict(x=x.to(dtype), w=(1 + 0.3 * randn(D, seed=seed + 3)).to(dtype),
                b=randn(D, seed=seed + 4, dtype=dtype) if kind == "layer" else None, dy=randn(M, D, seed=seed + 5, dtype=dtype))


def check_all(x, w, b, dy, kind, eps=1e-5, what="", **kw):
    """Both directions of rows x [M, D]; returns (y, dx, dw, db)."""
    y, mean, rstd = hc.norm_fwd(x, w, b, kind=kind, eps=eps, save_stats=True)
    want = ref.norm_fwd(x, w, b, kind, eps)
    check(y, *want[0], what + " y")
    if kind == "layer":
        check(mean, *want[1], what + " mean")
    check(rstd, *want[2], what + " rstd")
    got = hc.norm_bwd(x, w, dy, mean, rstd, kind=kind, **kw)
    for name, g, r in zip(("dx", "dw", "db"), got, ref.norm_bwd(x, w, dy, mean, rstd, kind)):
        if g is not None:
            check(g, *r, what + " " + name)
    return (y, *got)


# every row form: a wave (1, 2, 4, 8 chunks), 256 and 1024 lanes, longer than registers hold, in both directions
DS = [1, 2, 7, 8, 64, 100, 512, 513, 1000, 1024, 1025, 2048, 4096, 4100, 8192, 8200, 16384, 16392, 33001, 70000]


@pytest.mark.parametrize("D", DS)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_row_lengths(D, dtype, kind):
    log("norm D=%d %s %s" % (D, dtype, kind))
    check_all(**inputs(37, D, dtype, D, kind), kind=kind, what="D=%d" % D)


@pytest.mark.parametrize("M", [1, 2, 3, 5, 511, 2049, 5000])
@pytest.mark.parametrize("D", [96, 1001, 4096])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_row_counts(M, D, dtype):
    log("norm M=%d D=%d %s" % (M, D, dtype))
    check_all(**inputs(M, D, dtype, M + D), kind="layer", what="M=%d" % M)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("w,b", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_without_weight_or_bias(dtype, w, b, kind):
    t = inputs(70, 200, dtype, 3)
    t["w"], t["b"] = t["w"] if w else None, t["b"] if b else None
    _, _, dw, db = check_all(**t, kind=kind, what="w %s b %s" % (w, b))
    assert (dw is not None) == w and db is not None


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,off", [(64, 8), (64, 3), (1001, 5), (4096, 1), (20000, 7)])
def test_rows_inside_wider_buffers_of_nan(dtype, D, off):
    """Strides and starts of any alignment; nothing around the rows is read or written."""
    M, t = 41, inputs(41, D, dtype, 5)

    def wide(v):
        big = torch.full((M, D + 13), float("nan"), dtype=dtype, device=DEV)
        big[:, off:off + D] = v
        return big[:, off:off + D]

    y, dx, dw, db = check_all(**t, kind="layer")
    x, dy, out, dout = wide(t["x"]), wide(t["dy"]), wide(t["x"]), wide(t["x"])
    got, mean, rstd = hc.norm_fwd(x, t["w"], t["b"], save_stats=True, out=out)
    n = hc.norm_workspace_bytes(M, D, 0 if dtype == BF16 else 1)
    grads = hc.norm_bwd(x, t["w"], dy, mean, rstd, dx=dout, workspace=torch.full((n,), 255, dtype=torch.uint8, device=DEV))
    assert got.data_ptr() == out.data_ptr() and grads[0].data_ptr() == dout.data_ptr()
    for a, b in zip((got, *grads), (y, dx, dw, db)):
        assert torch.equal(a, b)
    for big in (out, dout):
        base = big._base
        assert torch.isnan(base[:, :off]).all() and torch.isnan(base[:, off + D:]).all()


def test_leading_dimensions():
    t = inputs(60, 72, BF16, 6)
    want = check_all(**t, kind="layer")
    x, dy = t["x"].view(3, 4, 5, 72), t["dy"].view(3, 4, 5, 72)
    y, mean, rstd = hc.norm_fwd(x, t["w"], t["b"], save_stats=True)
    assert y.shape == x.shape and mean.shape == rstd.shape == (3, 4, 5)
    dx, dw, db = hc.norm_bwd(x, t["w"], dy, mean, rstd)
    for a, b in zip((y, dx), want[:2]):
        assert torch.equal(a.view(60, 72), b)
    assert torch.equal(dw, want[2]) and torch.equal(db, want[3])
    one = hc.norm_fwd(t["x"][0], t["w"], t["b"])[0]
    assert one.shape == (72,) and torch.equal(one, want[0][0])


@pytest.mark.parametrize("D", [64, 4096, 9000])
def test_means_far_from_zero(D):
    """A mean of 1000 deviations: deviations are formed from the mean, not from sums of squares."""
    t = inputs(33, D, F32, 8)
    t["x"] = t["x"] * 0.01 + 10.0
    check_all(**t, kind="layer", what="far")


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_equal_values_and_zeros(kind):
    t = inputs(8, 130, F32, 9)
    t["x"][0], t["x"][1] = 2.0, 0.0
    check_all(**t, kind=kind, what="equal")
    assert torch.equal(hc.norm_fwd(t["x"], None, None, kind=kind)[0][1], torch.zeros(130, device=DEV))


def test_a_bad_row_is_alone():
    t = inputs(9, 300, BF16, 10)
    good = hc.norm_fwd(t["x"], t["w"], t["b"])[0]
    t["x"][4, 17], t["x"][6, 2] = float("nan"), float("inf")
    y = hc.norm_fwd(t["x"], t["w"], t["b"])[0]
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y[keep], good[keep]) and torch.isnan(y[4]).all() and torch.isnan(y[6]).any()


@pytest.mark.parametrize("need", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1), (0, 0, 0)])
@pytest.mark.parametrize("D", [100, 3000, 40000])
def test_parts_of_the_backward(need, D):
    t = inputs(50, D, BF16, 11)
    _, mean, rstd = hc.norm_fwd(t["x"], t["w"], t["b"], save_stats=True)
    whole = hc.norm_bwd(t["x"], t["w"], t["dy"], mean, rstd)
    got = hc.norm_bwd(t["x"], t["w"], t["dy"], mean, rstd, need_dx=bool(need[0]), need_dw=bool(need[1]), need_db=bool(need[2]))
    for n, g, w in zip(need, got, whole):
        assert (g is not None) == bool(n) and (not n or torch.equal(g, w))


def test_no_rows_and_no_channels():
    x, w = torch.zeros(0, 16, device=DEV), torch.ones(16, device=DEV)
    y, mean, rstd = hc.norm_fwd(x, w, w, save_stats=True)
    dx, dw, db = hc.norm_bwd(x, w, x, mean, rstd)
    assert y.shape == dx.shape == (0, 16) and not dw.any() and not db.any()
    x = torch.zeros(5, 0, device=DEV)
    assert hc.norm_fwd(x)[0].shape == (5, 0)


def test_offsets_past_32_bits():
    """Rows 70 000 apart by 65 536 elements: 9 GB."""
    M, D = 70000, 24
    x = torch.empty(M, 65536, dtype=BF16, device=DEV)[:, :D]
    x.copy_(randn(M, D, seed=12, dtype=BF16))
    t = inputs(M, D, BF16, 13)
    t["x"] = x
    check_all(**t, kind="layer", what="far rows")


def test_refusals():
    x, w = torch.zeros(4, 16, device=DEV), torch.ones(16, device=DEV)
    stat = torch.ones(4, device=DEV)
    for bad in (lambda: hc.norm_fwd(x.cpu()), lambda: hc.norm_fwd(x, w[:8]), lambda: hc.norm_fwd(x, kind="batch"),
                lambda: hc.norm_fwd(x.t()), lambda: hc.norm_fwd(x, w.bfloat16()), lambda: hc.norm_fwd(x, out=x[:2]),
                lambda: hc.norm_bwd(x, w, x[:2], stat, stat), lambda: hc.norm_bwd(x, w, x, None, stat),
                lambda: hc.norm_bwd(x, w, x, stat, stat, kind="rms"), lambda: hc.norm_bwd(x, w, x, stat, stat.double()),
                lambda: hc.norm_bwd(x, w, x, stat, stat, workspace=torch.zeros(4, dtype=torch.uint8, device=DEV)),
                lambda: hc.norm_fwd(torch.tensor(1.0, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: hc.norm_fwd(x, w, out=x), lambda: hc.norm_fwd(x, w, eps=-1.0)):
        with pytest.raises(hc.ModelError):
            bad()
    with pytest.raises(TypeError):
        hc.norm_fwd(x.half())


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradients_against_differences(kind):
    """Autograd in fp32 against central differences in 64 bits of the definition."""
    M, D, eps, h = 3, 10, 1e-3, 1e-5
    t = inputs(M, D, F32, 14)
    leaves = [t[n].clone().requires_grad_(True) for n in ("x", "w", "b")]
    (hc.Norm.apply(*leaves, kind, eps) * t["dy"]).sum().backward()

    def value(vs):
        return float((ref.norm_fwd(*vs, kind, eps)[0][0] * t["dy"].double()).sum())

    plain = [v.detach().double() for v in leaves]
    for i, leaf in enumerate(leaves):
        for at in range(0, leaf.numel(), 4):
            up, down = [[v.clone() for v in plain] for _ in range(2)]
            up[i].view(-1)[at] += h
            down[i].view(-1)[at] -= h
            slope = (value(up) - value(down)) / (2 * h)
            # differences: h^2 times third derivatives (1e-10 times some tens), 1e-16 / h; the kernel some U
            assert abs(float(leaf.grad.view(-1)[at]) - slope) <= 2e-5 * (1 + abs(slope)), (i, at)


def test_autograd_hands_out_what_is_wanted():
    t = inputs(20, 40, F32, 15)
    x = t["x"].clone().requires_grad_(True)
    hc.Norm.apply(x, t["w"]).sum().backward()
    assert x.grad is not None
    w = t["w"].clone().requires_grad_(True)
    hc.Norm.apply(t["x"], w, t["b"], "rms").sum().backward()
    assert w.grad is not None
    (g,) = torch.autograd.grad(hc.Norm.apply(x, w, t["b"]).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
