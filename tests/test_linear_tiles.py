"""Every tile shape and operand path of the matrix product, against 64-bit products.

The library picks them by size.  ``fwd_variant`` and ``bwd_variants`` state
which one a call takes (the rule of plan_of, few_rows and pad_rows in
hyena_linear.hip), and a test without a GPU checks that the cases below reach
all of them; a change of a threshold there has to be made here too."""
import pytest
import torch

import gated_convolution_sequence_amd as hc
import layer_ref as ref
from gpu_util import DEV, log
from layer_ref import check, to_np
from test_linear_gpu import check_bwd, check_fwd, inputs

BF16, F32 = torch.bfloat16, torch.float32


def cdiv(a, b):
    return -(-a // b)


def plan(sizes, f32, direct):
    """(tiles, splits of each product) for sizes (M, N, C) of the products that run in one launch."""
    bk, n = (32 if f32 else 64), len(sizes)
    t128 = sum(cdiv(M, 128) * cdiv(N, 128) for M, N, _ in sizes)
    t256 = sum(cdiv(M, 256) * cdiv(N, 256) for M, N, _ in sizes)
    large = not f32 and direct and t256 >= 128 and 4 * cdiv(t256, 256) <= cdiv(t128, 256) * 5 // 4
    fine = not large and t128 < 192
    edge = 256 if large else 64 if fine else 128
    tiles = [cdiv(M, edge) * cdiv(N, edge) for M, N, _ in sizes]
    work = sum(t * (cdiv(C, bk) + 4) for t, (_, _, C) in zip(tiles, sizes))
    share = max(4, cdiv(work, 256 if large else 1024 if f32 and fine and n == 2 else 256 * n))
    splits = []
    for _, _, C in sizes:
        steps = cdiv(C, bk)
        cut = cdiv(steps, share) if steps * 2 > share * 3 and steps >= 12 else 1
        splits.append(cdiv(steps, cdiv(steps, cut)))
    blocks = sum(t * s for t, s in zip(tiles, splits))
    deep = direct and (not f32 and n == 1 if fine else not large and blocks <= 256)
    name = "large" if large else "fine" if fine else "small"
    return name + (" deep" if deep else "" if direct else " registers"), splits


def pads(M, N, K, f32, least):
    return K * (4 if f32 else 2) % 16 != 0 and M * N * K >= least


def whole_16(n, f32):
    return n * (4 if f32 else 2) % 16 == 0


def fwd_variant(M, N, K, f32):
    """For contiguous, aligned operands."""
    if M <= 16 and (K <= 2048 or N >= 4096):
        return "rows 16"
    if M <= 32 and K <= 1024 and N <= 8192:
        return "rows 32"
    return plan([(M, N, K)], f32, whole_16(K, f32) or pads(M, N, K, f32, 2e9 if f32 else 7e9))[0]


def bwd_variants(M, N, K, f32, act, dx, dw, db):
    """The products' tiles, and their splits: [(product, variant, splits)]."""
    least = 0 if act != "none" or db else 1e9
    ok = whole_16(K, f32) or pads(M, N, K, f32, least)
    make = act != "none" or (ok and pads(M, K, N, f32, least))
    sizes = ([(N, K, M)] if dw else []) + ([(M, K, N)] if dx else [])
    name, splits = plan(sizes, f32, ok and (make or whole_16(N, f32)))
    return [(p, name, s) for p, s in zip((["dw"] if dw else []) + (["dx"] if dx else []), splits)]


# M, N, K; ragged against every tile and step
FORWARD = [
    ("large", BF16, (3684, 4000, 200)),
    ("large", BF16, (3684, 4001, 501)),            # padded rows
    ("large", BF16, (4096, 4096, 72)),             # whole tiles, a step and a bit
    ("small deep", BF16, (2100, 1900, 264)), ("small deep", F32, (1604, 1900, 200)),
    ("small", BF16, (2010, 2500, 200)), ("small", F32, (2010, 2500, 200)),
    ("small", F32, (2010, 2501, 403)),             # padded rows
    ("small registers", BF16, (2010, 2500, 201)), ("small registers", F32, (2010, 2500, 201)),
    ("fine", F32, (300, 520, 204)),
    ("fine deep", BF16, (300, 520, 200)),
    ("fine registers", BF16, (300, 520, 201)), ("fine registers", F32, (300, 520, 201)),
    ("rows 16", BF16, (13, 136, 200)), ("rows 16", F32, (13, 136, 200)),
    ("rows 32", BF16, (29, 136, 200)), ("rows 32", F32, (29, 136, 200)),
]

# and act, (dx, dw, db)
BACKWARD = [
    ("large", BF16, (3300, 200, 3904), "silu", (1, 1, 1)),   # dw cut along its rows
    ("large", BF16, (2500, 2504, 2600), "none", (1, 1, 0)),
    ("large", BF16, (3300, 200, 3904), "none", (1, 0, 1)),
    ("large", BF16, (200, 3304, 3904), "gelu", (0, 1, 0)),
    ("large", BF16, (3301, 201, 3901), "gelu", (1, 1, 1)),   # padded rows
    ("small deep", BF16, (700, 696, 2104), "silu", (1, 1, 1)), ("small deep", F32, (350, 348, 4096), "silu", (1, 1, 1)),
    ("small", BF16, (2100, 1904, 1800), "none", (1, 1, 1)), ("small", F32, (1300, 1292, 1804), "gelu", (1, 1, 1)),
    ("small", F32, (1300, 1291, 1801), "gelu", (1, 1, 1)),
    ("small registers", BF16, (200, 201, 6201), "none", (1, 1, 0)),
    ("small registers", F32, (200, 201, 6201), "none", (1, 1, 0)),
    ("fine", BF16, (500, 264, 264), "silu", (1, 1, 1)), ("fine", F32, (500, 264, 264), "silu", (1, 1, 1)),
    ("fine deep", BF16, (500, 264, 264), "silu", (1, 0, 0)), ("fine deep", BF16, (500, 264, 264), "silu", (0, 1, 1)),
    ("fine registers", BF16, (500, 201, 203), "none", (1, 1, 0)),
    ("fine registers", F32, (500, 201, 203), "none", (1, 1, 0)),
]


def test_the_cases_reach_every_variant():
    for want, dtype, (M, N, K) in FORWARD:
        assert fwd_variant(M, N, K, dtype == F32) == want, (want, M, N, K)
    got = {(v, d) for v, d, _ in FORWARD}
    both = ("small deep", "small", "small registers", "fine registers", "rows 16", "rows 32")
    assert got == {(v, d) for v in both for d in (BF16, F32)} | {("large", BF16), ("fine deep", BF16), ("fine", F32)}
    cut = set()
    for want, dtype, (M, N, K), act, need in BACKWARD:
        for product, name, splits in bwd_variants(M, N, K, dtype == F32, act, *need):
            assert name == want, (want, name, M, N, K, act, need)
            cut.add((product, name, splits > 1))
    got = {(v, d) for v, d, *_ in BACKWARD}
    both = ("small deep", "small", "small registers", "fine", "fine registers")
    assert got == {(v, d) for v in both for d in (BF16, F32)} | {("large", BF16), ("fine deep", BF16)}
    assert {("dw", "large", True), ("dw", "large", False), ("dx", "large", False), ("dw", "fine", True)} <= cut


@pytest.mark.gpu
@pytest.mark.parametrize("variant,dtype,size", FORWARD, ids=str)
def test_forward(variant, dtype, size):
    log("linear forward %s %s %s" % (variant, dtype, size))
    t = inputs(*size, dtype, sum(size))
    check_fwd(t, "silu", True, True, variant)


@pytest.mark.gpu
@pytest.mark.parametrize("variant,dtype,size,act,need", BACKWARD, ids=str)
def test_backward(variant, dtype, size, act, need):
    log("linear backward %s %s %s %s %s" % (variant, dtype, size, act, need))
    t = inputs(*size, dtype, sum(size))
    _, z = hc.linear_fwd(t["x"], t["w"], bias=t["b"], act=act, save_preact=act != "none")
    z = torch.zeros_like(t["dy"]) if z is None else z
    got = check_bwd(t, z, act, variant, need_dx=bool(need[0]), need_dw=bool(need[1]), need_db=bool(need[2]))
    assert [g is not None for g in got] == [bool(n) for n in need]


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(3684, 4000, 200), (2010, 2500, 200)], ids=str)
def test_rows_of_wider_buffers_at_the_large_tiles(size):
    """Column slices in, a column slice out: NaN beside the operands, nothing written beside the output."""
    M, N, K = size
    t = inputs(M, N, K, BF16, 3)
    wide = torch.full((M, K + 24), float("nan"), dtype=BF16, device=DEV)
    wide[:, 8:8 + K] = t["x"]
    out = torch.full((M, N + 16), 7.0, dtype=BF16, device=DEV)
    y, _ = hc.linear_fwd(wide[:, 8:8 + K], t["w"], bias=t["b"], residual=t["r"], act="gelu", out=out[:, 8:8 + N])
    wy, ey, _, _ = ref.linear_fwd(*(to_np(t[n]) for n in ("x", "w", "b", "r")), "gelu")
    check(y, wy, ey, BF16, "y")
    assert torch.all(out[:, :8] == 7.0) and torch.all(out[:, 8 + N:] == 7.0)


@pytest.mark.gpu
def test_values_past_4_gib():
    """x of 4.5 GB: its rows at offsets past 2^32 bytes, against 64 bits."""
    M, N, K, ldx = 70000, 72, 64, 1 << 15
    t = inputs(M, N, K, BF16, 16)
    big = torch.empty(M * ldx, dtype=BF16, device=DEV).view(M, ldx)
    t["x"] = big[:, 800:800 + K].copy_(t["x"])
    z = check_fwd(t, "silu", True, True, "fwd")
    check_bwd(t, z, "silu", "bwd")


@pytest.mark.gpu
def test_runs_at_the_large_tiles_give_the_same_bits():
    t = inputs(3300, 200, 3904, BF16, 4)
    first = hc.linear_bwd(t["x"], t["w"], t["dy"], act="none")
    for _ in range(3):
        for a, b in zip(hc.linear_bwd(t["x"], t["w"], t["dy"], act="none"), first):
            assert torch.equal(a, b)
    t = inputs(3684, 4000, 200, BF16, 5)
    first = hc.linear_fwd(t["x"], t["w"], residual=t["r"])[0]
    for _ in range(3):
        assert torch.equal(hc.linear_fwd(t["x"], t["w"], residual=t["r"])[0], first)
    r = t["r"].clone()  # the residual updated in place
    assert torch.equal(hc.linear_fwd(t["x"], t["w"], residual=r, out=r)[0], first)
