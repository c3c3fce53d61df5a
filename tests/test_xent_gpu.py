"""Softmax cross entropy of a readout and its gradients, against 64 bits."""
import math

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


def inputs(M, K, V, dtype, seed, bias=True, masked=0.25):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=gen, device=DEV)).to(dtype)

    target = torch.randint(0, V, (M,), generator=gen, device=DEV)
    off = torch.rand(M, generator=gen, device=DEV) < masked
    target[off] = torch.where(torch.arange(M, device=DEV) % 2 == 0, -100, V)[off]
    return dict(x=randn(M, K), w=randn(V, K, scale=2 * max(K, 1) ** -0.5), target=target,
                bias=randn(V, scale=0.5) if bias else None,
                dloss=torch.rand(M, generator=gen, device=DEV) / max(1, M))


def check_all(x, w, target, bias, dloss, what="", **kw):
    loss, lse = hc.xent_fwd(x, w, target, bias=bias)
    want = ref.xent_fwd(x, w, target, bias)
    check(loss, *want[0], what + " loss")
    check(lse, *want[1], what + " lse")
    got = hc.xent_bwd(x, w, target, lse, dloss, bias=bias, **kw)
    for name, g, r in zip(("dx", "dw", "db"), got, ref.xent_bwd(x, w, target, lse, dloss, bias, x.dtype == BF16)):
        if g is not None:
            check(g, *r, what + " " + name)
    return (loss, lse, *got)


# few rows; 64-, 128- and 256-wide tiles; ragged everywhere; one entry; no channels
SIZES = [(1, 8, 3), (1, 64, 1), (5, 100, 7), (16, 64, 300), (16, 4096, 1000), (17, 64, 1000), (33, 72, 500), (64, 8, 4),
         (130, 200, 257), (300, 129, 1000), (1021, 77, 503), (2048, 64, 2048), (2304, 40, 2304), (4096, 64, 4096),
         (4000, 72, 4097), (7, 1, 9), (40, 1, 9), (4, 0, 6), (40, 0, 70), (700, 1500, 33)]


@pytest.mark.parametrize("shape", SIZES, ids=lambda s: "%dx%dx%d" % s)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_sizes(shape, dtype):
    log("xent %s %s" % (shape, dtype))
    check_all(**inputs(*shape, dtype, sum(shape), bias=sum(shape) % 2 == 0), what=str(shape))


@pytest.mark.parametrize("M", [1, 16, 17, 200, 5000])
@pytest.mark.parametrize("masked", [0.0, 1.0, 0.97])
def test_masks(M, masked):
    """Rows without a target cost nothing; none may have one."""
    t = inputs(M, 96, 310, BF16, M, masked=masked)
    loss, lse, dx, dw, db = check_all(**t, what="masked %.2f" % masked)
    off = (t["target"] < 0) | (t["target"] >= 310)
    assert not loss[off].any() and not lse[off].any() and not dx[off].any()
    if masked == 1.0:
        assert not dw.any() and not db.any()


@pytest.mark.parametrize("M", [16, 150, 3000])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_what_masked_rows_hold_is_not_read(M, dtype):
    t = inputs(M, 80, 200, dtype, 3, masked=0.4)
    want = check_all(**t)
    off = (t["target"] < 0) | (t["target"] >= 200)
    t["x"][off] = float("nan")
    t["dloss"][off] = float("inf")
    for a, b in zip(check_all(**t), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("value", [2 ** 40, 1 << 32, -(1 << 63), (1 << 63) - 1, -1, 50])
def test_targets_outside_the_vocabulary(value):
    for M in (10, 100):
        t = inputs(M, 40, 50, F32, 4, masked=0.0)
        t["target"][3] = value
        loss, lse, dx, _, _ = check_all(**t)
        assert loss[3] == 0 and lse[3] == 0 and not dx[3].any()


@pytest.mark.parametrize("M", [12, 90])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_entries_that_cannot_occur(M, dtype):
    """A bias of -inf, or of the type's lowest value, takes entries out; all of a tile, and all of a wave's columns."""
    t = inputs(M, 64, 700, dtype, 5, masked=0.2)
    t["bias"][100:420] = -math.inf
    t["bias"][500] = torch.finfo(dtype).min
    t["target"][t["target"] >= 0] %= 100
    _, _, _, dw, db = check_all(**t)
    assert not dw[100:420].any() and not db[100:420].any() and not dw[500].any()


@pytest.mark.parametrize("M", [5, 50])
def test_target_that_cannot_occur(M):
    t = inputs(M, 32, 60, F32, 6, masked=0.0)
    t["bias"][7] = -math.inf
    t["target"][:] = 9
    t["target"][2] = 7
    loss, lse = hc.xent_fwd(t["x"], t["w"], t["target"], bias=t["bias"])
    assert loss[2] == math.inf and torch.isfinite(lse).all() and torch.isfinite(loss[[0, 1, 3, 4]]).all()
    t["bias"][:] = -math.inf  # nothing can occur
    loss, lse = hc.xent_fwd(t["x"], t["w"], t["target"], bias=t["bias"])
    assert (lse == -math.inf).all() and torch.isnan(loss).all()


@pytest.mark.parametrize("M", [6, 70])
def test_large_logits(M):
    """Logits of some thousands: nothing overflows, the largest decides."""
    t = inputs(M, 64, 300, F32, 7)
    t["w"] *= 600
    check_all(**t, what="large")


@pytest.mark.parametrize("M", [6, 70])
def test_bad_rows_are_alone(M):
    t = inputs(M, 64, 300, F32, 8, masked=0.0)
    loss, lse = hc.xent_fwd(t["x"], t["w"], t["target"], bias=t["bias"])
    t["x"][3, 5], t["x"][1, 2] = math.nan, math.inf
    bad, _ = hc.xent_fwd(t["x"], t["w"], t["target"], bias=t["bias"])
    keep = [i for i in range(M) if i not in (1, 3)]
    assert torch.equal(bad[keep], loss[keep]) and torch.isnan(bad[3]) and not torch.isfinite(bad[1])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,K,V", [(9, 64, 130), (9, 63, 130), (150, 64, 300), (150, 77, 301), (3000, 101, 2100)])
def test_rows_inside_wider_buffers_of_nan(dtype, M, K, V):
    t = inputs(M, K, V, dtype, 9)
    want = check_all(**t)

    def wide(v):
        big = torch.full((M, K + 13), float("nan"), dtype=dtype, device=DEV)
        big[:, 5:5 + K] = v
        return big[:, 5:5 + K]

    code = 0 if dtype == BF16 else 1
    x, out = wide(t["x"]), wide(t["x"])
    ws = [torch.full((hc.xent_workspace_bytes(M, K, V, code, b),), 255, dtype=torch.uint8, device=DEV) for b in (False, True)]
    loss, lse = hc.xent_fwd(x, t["w"], t["target"], bias=t["bias"], workspace=ws[0])
    got = hc.xent_bwd(x, t["w"], t["target"], lse, t["dloss"], bias=t["bias"], dx=out, workspace=ws[1])
    assert got[0].data_ptr() == out.data_ptr()
    for a, b in zip((loss, lse, *got), want):
        assert torch.equal(a, b)
    base = out._base
    assert torch.isnan(base[:, :5]).all() and torch.isnan(base[:, 5 + K:]).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,K,V", [(9, 64, 130), (150, 64, 300), (150, 63, 300), (2304, 64, 2304), (4096, 64, 4096)])
def test_weights_at_any_element(dtype, M, K, V):
    """Workspaces of the reported size hold what a call needs at any alignment (bytes behind them stay)."""
    t = inputs(M, K, V, dtype, 10)
    code = 0 if dtype == BF16 else 1
    flat = torch.empty(V * K + 3, dtype=dtype, device=DEV)
    w = flat[3:].view(V, K)
    w.copy_(t["w"])
    t["w"] = w
    check_all(**t)
    sizes = [hc.xent_workspace_bytes(M, K, V, code, b) for b in (False, True)]
    big = [torch.full((n + 4096,), 171, dtype=torch.uint8, device=DEV) for n in sizes]
    ws = [x[:n] for x, n in zip(big, sizes)]
    _, lse = hc.xent_fwd(t["x"], w, t["target"], bias=t["bias"], workspace=ws[0])
    hc.xent_bwd(t["x"], w, t["target"], lse, t["dloss"], bias=t["bias"], workspace=ws[1])
    for x, n in zip(big, sizes):
        assert bool((x[n:] == 171).all())


@pytest.mark.parametrize("need", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1), (0, 0, 0)])
@pytest.mark.parametrize("M,K,V", [(100, 72, 300), (4096, 64, 4096)])
def test_parts_of_the_backward(need, M, K, V):
    t = inputs(M, K, V, BF16, 11)
    got = check_all(**t, need_dx=bool(need[0]), need_dw=bool(need[1]), need_db=bool(need[2]))[2:]
    for n, g in zip(need, got):
        assert (g is not None) == bool(n)


@pytest.mark.parametrize("M", [8191, 8192, 8193, 16384, 70001])
@pytest.mark.parametrize("K,V", [(8, 3), (100, 4), (264, 1), (1, 130)])
@pytest.mark.parametrize("masked", [0.0, 0.5, 0.999])
def test_many_rows_of_few_entries(M, K, V, masked):
    """Rows numbered by several workgroups, short rows packed several a wave, narrow bias gradients."""
    t = inputs(M, K, V, BF16 if K != 100 else F32, M + V, masked=masked)
    t["target"][M // 2:M // 2 + 3000] = -1  # a stretch without
    loss, _, dx, _, _ = check_all(**t, what="%d rows" % M)
    off = (t["target"] < 0) | (t["target"] >= V)
    assert not loss[off].any() and not dx[off].any()


def test_pieces_of_the_vocabulary():
    """Rows so many that a piece holds 2048 entries: three pieces, dx added up over them."""
    M, K, V = 66000, 24, 5000
    t = inputs(M, K, V, BF16, 12, masked=0.1)
    assert hc.xent_workspace_bytes(M, K, V, 0, True) < M * V * 2
    check_all(**t, what="pieces")
    t = inputs(33000, 20, 4500, F32, 13, masked=0.1)
    check_all(**t, what="pieces f32")


def test_offsets_past_32_bits():
    """Rows 66 000 apart by 65 537 elements (8.6 GB), and logits past 2^32 of them together."""
    M, K, V = 66000, 16, 66000
    t = inputs(M, K, 64, BF16, 14)
    x = torch.empty(M, 65537, dtype=BF16, device=DEV)[:, :K]
    x.copy_(t["x"])
    t["x"] = x
    check_all(**t, what="far rows")
    t = inputs(M, K, V, BF16, 15, bias=False)
    loss, lse = hc.xent_fwd(t["x"], t["w"], t["target"])
    pick = torch.tensor([0, 1, 32767, 65535, 65536, 65999], device=DEV)
    want = ref.xent_fwd(t["x"][pick], t["w"], t["target"][pick], None)
    check(loss[pick], *want[0], "loss")
    check(lse[pick], *want[1], "lse")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_upstream_gradients(dtype):
    """Of either sign, of very unlike sizes, 0, and alike: where p is small those leave one rounding, the output's."""
    t = inputs(200, 64, 5000, dtype, 21, masked=0.1)
    t["dloss"] = torch.randn(200, device=DEV) * torch.exp2(torch.randint(-30, 30, (200,), device=DEV).float())
    check_all(**t, what="unlike")
    t["dloss"].zero_()
    _, _, dx, dw, db = check_all(**t, what="zero")
    assert not dx.any() and not dw.any() and not db.any()
    t["dloss"].fill_(1.0 / 173)
    t["w"] *= 0.01  # p about 1 / 5000
    t["bias"].zero_()
    loss, lse, dx, dw, _ = check_all(**t, what="alike")
    want = ref.xent_bwd(t["x"], t["w"], t["target"], lse, t["dloss"], t["bias"], False)
    if dtype == BF16:  # rows of targets: rounded once, and p (a part in 5000, in both) once more
        hit = torch.bincount(t["target"][(t["target"] >= 0) & (t["target"] < 5000)], minlength=5000) == 1
        err = (dw.double() - want[1][0])[hit].norm() / want[1][0][hit].norm()
        assert err < 2.0 ** -9 * 1.1, err


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("masked", [0.0, 0.5, 0.99, 0.998, 1.0])
def test_rows_far_apart(dtype, masked):
    """8.6 GB of rows: fetched where they are, or, where a tile's lie past 32-bit offsets, packed first."""
    M, K, V = 66000, 16, 300
    t = inputs(M, K, V, dtype, 22, masked=masked)
    x = torch.empty(M, 65536 * 2 // t["x"].element_size(), dtype=dtype, device=DEV)[:, :K]
    x.copy_(t["x"])
    near = check_all(**t)
    t["x"] = x
    for a, b in zip(check_all(**t, what="masked %.3f" % masked), near):
        assert torch.equal(a, b)
    for need in ((1, 0), (0, 1)):
        check_all(**t, need_dx=bool(need[0]), need_dw=bool(need[1]))
    t = {**inputs(M, K, 7, dtype, 24, masked=masked), "x": x}  # no more entries than columns
    x.copy_(inputs(M, K, 7, dtype, 24)["x"])
    check_all(**t, what="few entries")


@pytest.mark.parametrize("M,K,V", [(300, 64, 31), (300, 64, 500), (20000, 72, 9), (5000, 1024, 512)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("masked", [0.0, 0.3])
def test_dloss_alike_or_not(M, K, V, dtype, masked):
    """dw from e or from e dloss, with x in place or packed: dloss alike, of one sign, of both, all negative, NaN, 0."""
    t = inputs(M, K, V, dtype, 23, masked=masked)
    own = t["dloss"].clone()
    for what, d in (("own", own), ("alike", torch.full_like(own, 0.3)), ("negative", torch.full_like(own, -0.3)),
                    ("signs", torch.where(own > own.mean(), 0.3, -0.3)), ("zero", torch.zeros_like(own))):
        check_all(**{**t, "dloss": d}, what=what)
    rows = torch.nonzero((t["target"] >= 0) & (t["target"] < V))[:, 0]
    d = torch.full_like(own, 0.3)
    d[rows[len(rows) // 2]] = math.nan
    loss, lse = hc.xent_fwd(t["x"], t["w"], t["target"], bias=t["bias"])
    dx, dw, db = hc.xent_bwd(t["x"], t["w"], t["target"], lse, d, bias=t["bias"])
    assert torch.isnan(dw).all() and torch.isnan(db).all() and torch.isnan(dx[rows[len(rows) // 2]]).all()
    assert torch.isfinite(dx[rows[:len(rows) // 2]]).all()


@pytest.mark.parametrize("M", [8, 200])
def test_the_same_bits_again(M):
    t = inputs(M, 520, 1000, BF16, 16)
    first = check_all(**t)
    for _ in range(3):
        for a, b in zip(check_all(**t), first):
            assert torch.equal(a, b)


def test_leading_dimensions_and_no_rows():
    t = inputs(60, 40, 90, F32, 17)
    want = check_all(**t)
    x, target = t["x"].view(3, 20, 40), t["target"].view(3, 20)
    loss, lse = hc.xent_fwd(x, t["w"], target, bias=t["bias"])
    assert loss.shape == lse.shape == (3, 20) and torch.equal(loss.view(-1), want[0])
    dx, dw, db = hc.xent_bwd(x, t["w"], target, lse, t["dloss"].view(3, 20), bias=t["bias"])
    assert torch.equal(dx.view(60, 40), want[2]) and torch.equal(dw, want[3]) and torch.equal(db, want[4])
    x, target = t["x"][:0], t["target"][:0]
    loss, lse = hc.xent_fwd(x, t["w"], target, bias=t["bias"])
    dx, dw, db = hc.xent_bwd(x, t["w"], target, lse, loss, bias=t["bias"])
    assert loss.shape == (0,) and dx.shape == (0, 40) and not dw.any() and not db.any()


def test_refusals():
    t = inputs(20, 32, 50, F32, 18)
    x, w, target, bias, dloss = (t[n] for n in ("x", "w", "target", "bias", "dloss"))
    for bad in (lambda: hc.xent_fwd(x.cpu(), w, target), lambda: hc.xent_fwd(x, w[:, :8], target),
                lambda: hc.xent_fwd(x, w, target.int()), lambda: hc.xent_fwd(x, w, target[:3]),
                lambda: hc.xent_fwd(x, w.t().contiguous().t(), target), lambda: hc.xent_fwd(x, w, target, bias=bias[:3]),
                lambda: hc.xent_fwd(x, w.bfloat16(), target), lambda: hc.xent_bwd(x, w, target, dloss.double(), dloss),
                lambda: hc.xent_bwd(x, w, target, dloss, dloss[:2]),
                lambda: hc.xent_bwd(x, w, target, dloss, dloss, dx=x[:3]),
                lambda: hc.xent_fwd(x, w, target, workspace=torch.zeros(4, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(hc.ModelError):
        hc.xent_fwd(x, w[:0], target)
    with pytest.raises(hc.ModelError):
        hc.xent_bwd(x, w, target, dloss, dloss, dx=x)
    with pytest.raises(TypeError):
        hc.xent_fwd(x.half(), w, target)


def test_gradients_against_differences():
    """Autograd in fp32 against central differences in 64 bits of the definition."""
    h = 1e-5
    t = inputs(20, 6, 9, F32, 19)
    leaves = [t[n].clone().requires_grad_(True) for n in ("x", "w", "bias")]
    weight = torch.rand(20, device=DEV)
    (hc.LinearXent.apply(leaves[0], leaves[1], t["target"], leaves[2]) * weight).sum().backward()

    def value(vs):
        return float((ref.xent_fwd(vs[0], vs[1], t["target"], vs[2])[0][0] * weight.double()).sum())

    plain = [v.detach().double() for v in leaves]
    for i, leaf in enumerate(leaves):
        for at in range(0, leaf.numel(), 5):
            up, down = [[v.clone() for v in plain] for _ in range(2)]
            up[i].view(-1)[at] += h
            down[i].view(-1)[at] -= h
            slope = (value(up) - value(down)) / (2 * h)
            assert abs(float(leaf.grad.view(-1)[at]) - slope) <= 2e-5 * (1 + abs(slope)), (i, at)


def test_autograd_hands_out_what_is_wanted():
    t = inputs(30, 16, 40, F32, 20)
    x = t["x"].clone().requires_grad_(True)
    hc.LinearXent.apply(x, t["w"], t["target"]).mean().backward()  # an expanded scalar comes back
    assert x.grad is not None
    bias = t["bias"].clone().requires_grad_(True)
    hc.LinearXent.apply(t["x"], t["w"], t["target"], bias).sum().backward()
    assert bias.grad is not None
    (g,) = torch.autograd.grad(hc.LinearXent.apply(x, t["w"], t["target"]).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
