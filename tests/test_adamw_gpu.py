"""AdamW over lists of tensors and the norm of all gradients, against 64 bits."""
import math

import pytest
import torch

import gated_convolution_sequence_amd as hc
import model_ref as ref
from gpu_util import DEV, log
from model_ref import check

pytestmark = pytest.mark.gpu
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
# none, one, around a scale's and a workgroup's span, odd ones; more than a launch takes
SIZES = [5, 0, 1, 7, 8, 9, 255, 256, 257, 1000, 8191, 8192, 8193, 20001, 0, 70000]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.model_lib()
    yield
    torch.cuda.synchronize()


def lists(sizes, dtype, seed, master=False, bits=32, off=0):
    """Tensors at ``off`` elements past an aligned address."""
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def new(scale, dt):
        out = []
        for n in sizes:
            out.append(torch.empty(n + off, dtype=dt, device=DEV)[off:])
            out[-1].copy_(scale * torch.randn(n, generator=gen, device=DEV))
        return out

    t = dict(params=new(0.5, dtype), grads=new(1e-2, dtype), exp_avgs=new(3e-3, F32), exp_avg_sqs=new(1e-2, F32))
    for v in t["exp_avg_sqs"]:
        v.square_()
    if master:
        t["masters"] = new(0.5, F32)
    if bits == 8:
        for name in ("exp_avgs", "exp_avg_sqs"):
            codes, scales = [], []
            for x in t[name]:
                x = x.sqrt() if name == "exp_avg_sqs" else x
                pad = torch.nn.functional.pad(x, (0, -x.numel() % 256)).view(-1, 256)
                s = pad.abs().amax(1) / 448
                c = torch.empty(x.numel() + off, dtype=torch.uint8, device=DEV)[off:].view(F8)
                c.copy_((pad / s.clamp(min=1e-30)[:, None]).view(-1)[:x.numel()].to(F8))
                codes.append(c)
                scales.append(s)
            t[name], t[name[:-1] + "_scales"] = codes, scales
    return t


def copies(t):
    return {k: [x.clone() for x in v] for k, v in t.items()}


def check_step(t, step, hyper=HYPER, scale=1.0, seed=0, what="", **kw):
    """One step in place on t against 64 bits on its state before."""
    old = copies(t)
    eight = "exp_avg_scales" in t
    hc.adamw_step(**t, step=kw.pop("step_arg", step), seed=kw.pop("seed_arg", seed), **{**hyper, **kw})
    for i, g in enumerate(old["grads"]):
        at = "%s tensor %d" % (what, i)
        m, v = old["exp_avgs"][i], old["exp_avg_sqs"][i]
        if eight:
            m = ref.decode(m, old["exp_avg_scales"][i])
            v = ref.decode(v, old["exp_avg_sq_scales"][i]) ** 2
        p = (old.get("masters") or old["params"])[i]
        new, mn, vn = ref.adamw(p, g, m, v, step, hyper["lr"], hyper["betas"], hyper["eps"], hyper["weight_decay"], scale)
        if "masters" in t:
            check(t["masters"][i], *new, at + " master")
            assert torch.equal(t["params"][i], t["masters"][i].to(t["params"][i].dtype)), at
        else:
            check(t["params"][i], *new, at + " param")
        if not eight:
            check(t["exp_avgs"][i], *mn, at + " m")
            check(t["exp_avg_sqs"][i], *vn, at + " v")
            continue
        bm, bv = ref.random_bits(g.numel(), seed, i, g.device)
        # decoding rounds each product once more (twice squared)
        ref.check_codes(t["exp_avgs"][i], t["exp_avg_scales"][i], mn[0], mn[1] + 2 * ref.U * mn[0].abs(), bm, at + " m")
        root = vn[0].sqrt()
        ref.check_codes(t["exp_avg_sqs"][i], t["exp_avg_sq_scales"][i], root, 6 * ref.U * root, bv, at + " r")
        assert torch.equal(t["grads"][i], old["grads"][i])


@pytest.mark.parametrize("dtype,master", [(BF16, True), (BF16, False), (F32, False), (F32, True)])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("off", [0, 3])
def test_steps(dtype, master, bits, off):
    log("adamw %s master %s bits %d" % (dtype, master, bits))
    t = lists(SIZES, dtype, 1, master, bits, off)
    for step in (1, 2, 1000):
        check_step(t, step, seed=77 + step, what="step %d" % step)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """Three launches' worth; in 8 bits the place in the list takes part in the rounding."""
    gen = torch.Generator().manual_seed(2)
    t = lists([int(n) for n in torch.randint(0, 600, (130,), generator=gen)], BF16, 3, True, bits)
    check_step(t, 5, seed=(1 << 32) - 3)


def test_a_tensor_past_32_bits():
    """An eighth more than 2^32 elements in 8 bits: the index's high half takes part in the rounding (29 GB)."""
    n = (1 << 32) + (1 << 29) + 77
    t = dict(params=[torch.zeros(n, dtype=BF16, device=DEV)], grads=[torch.full((n,), 0.5, dtype=BF16, device=DEV)],
             exp_avgs=[torch.zeros(n, dtype=torch.uint8, device=DEV).view(F8)],
             exp_avg_sqs=[torch.zeros(n, dtype=torch.uint8, device=DEV).view(F8)],
             exp_avg_scales=[torch.zeros(-(-n // 256), device=DEV)], exp_avg_sq_scales=[torch.zeros(-(-n // 256), device=DEV)])
    t["grads"][0][-1000:] = torch.linspace(-1, 1, 1000, device=DEV).to(BF16)
    hc.adamw_step(**t, step=1, seed=5, **HYPER)
    g = t["grads"][0][-1000:].double()
    new, mn, vn = ref.adamw(torch.zeros_like(g), g, 0 * g, 0 * g, 1, HYPER["lr"], HYPER["betas"], 1e-8, 0.1)
    check(t["params"][0][-1000:], *new, "param")
    i = torch.arange(n - 1000, n, device=DEV)
    h = ref.mix((i & 0xFFFFFFFF) ^ ref.mix((5 + (i >> 32)) & 0xFFFFFFFF))
    # whole blocks of 256 only: the first of these elements that starts one
    skip = int(-(n - 1000) % 256)
    ref.check_codes(t["exp_avgs"][0][-1000 + skip:], t["exp_avg_scales"][0][(n - 1000 + skip) // 256:], mn[0][skip:],
                    mn[1][skip:] + 2 * ref.U * mn[0][skip:].abs(), (h & 0xFFFF)[skip:], "m")
    assert float(t["params"][0][0]) == float(t["params"][0][1 << 32])


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_and_moments(bits):
    """A first step without gradient: nothing but the decay moves, and 0 / (0 + eps) is 0."""
    t = lists([700], F32, 4, bits=bits)
    for k in ("grads", "exp_avgs", "exp_avg_sqs", *(["exp_avg_scales", "exp_avg_sq_scales"] if bits == 8 else [])):
        for x in t[k]:
            x.view(torch.uint8 if x.dtype == F8 else x.dtype).zero_()
    before = t["params"][0].clone()
    check_step(t, 1, what="zeros")
    assert (t["params"][0] - before * (1 - 3e-4)).abs().max() <= 2 * ref.U * before.abs().max()
    assert not t["exp_avgs"][0].float().any()


def test_moments_in_8_bits_keep_moving():
    """beta2 = 0.999 moves v by less than half a code a step: over many steps the mean still follows."""
    n, steps = 1 << 16, 300
    t = dict(params=[torch.zeros(n, device=DEV)], grads=[torch.full((n,), 2.0, device=DEV)],
             exp_avgs=[torch.zeros(n, dtype=torch.uint8, device=DEV).view(F8)],
             exp_avg_sqs=[torch.zeros(n, dtype=torch.uint8, device=DEV).view(F8)],
             exp_avg_scales=[torch.zeros(n // 256, device=DEV)], exp_avg_sq_scales=[torch.zeros(n // 256, device=DEV)])
    for step in range(1, steps + 1):
        hc.adamw_step(**t, step=step, lr=0.0, betas=(0.9, 0.999), seed=step)
    v = ref.decode(t["exp_avg_sqs"][0], t["exp_avg_sq_scales"][0]) ** 2
    want = 4.0 * (1 - 0.999 ** steps)
    # a block's values are one code apart from its largest; random rounding spreads r by at most a code (1/8) and
    # the mean over 65536 of them by far less; squaring lifts the mean by the spread's square (under 1 %)
    assert abs(float(v.mean()) / want - 1) < 0.03


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [0.0, 0.25, math.nan, math.inf, -math.inf])
def test_gradient_scale(bits, value):
    t = lists(SIZES, BF16, 5, True, bits)
    scale = torch.tensor([value], device=DEV)
    if math.isfinite(value):
        return check_step(t, 3, scale=value, grad_scale=scale)
    old = copies(t)
    hc.adamw_step(**t, step=3, grad_scale=scale, **HYPER)
    for k in t:
        for a, b in zip(t[k], old[k]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) if a.dtype == F8 else torch.equal(a, b), k


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_takes_its_numbers_from_the_device(bits):
    """Replays with other gradients, rates, steps and seeds, each against an eager step, with eager work between."""
    t = lists([4000, 300, 9], BF16, 6, True, bits)
    lr = torch.zeros(1, device=DEV)
    step, seed = (torch.zeros(1, dtype=torch.int64, device=DEV) for _ in range(2))
    scale = torch.ones(1, device=DEV)
    start = copies(t)

    def call():
        hc.adamw_step(**t, step=step, lr=lr, seed=seed, betas=HYPER["betas"], eps=1e-8, weight_decay=0.1, grad_scale=scale)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in t:
        for a, b in zip(t[k], start[k]):
            a.copy_(b)
    eager = copies(t)
    for r in range(1, 5):
        for a, b in zip(t["grads"], eager["grads"]):
            a.copy_(torch.randn(a.shape, device=DEV) * 1e-2)
            b.copy_(a)
        lr.fill_(1e-3 * r), step.fill_(r), seed.fill_(100 + r), scale.fill_(0.5 + 0.1 * r)
        torch.cuda.synchronize()
        graph.replay()
        hc.adamw_step(**eager, step=r, lr=float(lr), seed=100 + r, betas=HYPER["betas"], eps=1e-8, weight_decay=0.1,
                      grad_scale=scale)
        torch.cuda.synchronize()
        for k in t:
            for a, b in zip(t[k], eager[k]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) if a.dtype == F8 else torch.equal(a, b), (r, k)


@pytest.mark.parametrize("bits", [32, 8])
def test_neighbours_in_one_buffer(bits):
    """Tensors that touch, and a gradient that two parameters share: accepted; the same tensor twice is not."""
    flat = [torch.randn(2000, device=DEV) for _ in range(3)]
    flat[2].square_()
    if bits == 8:
        flat[1:] = [torch.zeros(2000, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2)]
    t = dict(zip(("params", "exp_avgs", "exp_avg_sqs"), ([f[:999], f[999:]] for f in flat)))
    if bits == 8:
        s = torch.zeros(2, 8, device=DEV)
        t["exp_avg_scales"], t["exp_avg_sq_scales"] = ([x[:4], x[4:]] for x in s)
    g = torch.randn(1001, device=DEV)
    t["grads"] = [g[:999], g]
    check_step(t, 2, seed=9)
    t["params"] = [t["params"][0], flat[0][:1001]]
    with pytest.raises(hc.ModelError):
        hc.adamw_step(**t, step=3, **HYPER)


def test_a_step_below_one_on_the_device_counts_as_one():
    t = lists([100], F32, 7)
    check_step(t, 1, step_arg=torch.zeros(1, dtype=torch.int64, device=DEV))


# ---- norm of all gradients ------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("off", [0, 1])
def test_norm(dtype, off):
    """Squares in 64 bits: one rounding to fp32 (and one of the scale)."""
    g = lists(SIZES + [40000, 100000], dtype, 8, off=off)["grads"]
    want = math.sqrt(sum(float(x.double().square().sum()) for x in g))
    for most in (want / 3, want * 3, 0.0):
        norm, scale = hc.grad_norm(g, max_norm=most)
        assert norm.shape == scale.shape == () and norm.dtype is scale.dtype is F32
        assert abs(float(norm) / want - 1) <= 2.0 ** -24 * 1.01
        assert abs(float(scale) - min(1.0, most / want)) <= 2.0 ** -24 * 1.01
    norm, none = hc.grad_norm(g)
    assert none is None and abs(float(norm) / want - 1) <= 2.0 ** -24 * 1.01


def test_norm_of_many_large_and_zero():
    g = [torch.full((3,), 1e30, device=DEV) for _ in range(100)]
    norm, scale = hc.grad_norm(g, max_norm=1.0)
    assert abs(float(norm) / (1e30 * math.sqrt(300)) - 1) < 1e-6 and float(scale) > 0
    norm, scale = hc.grad_norm([torch.zeros(70, device=DEV)], max_norm=1.0)
    assert float(norm) == 0 and float(scale) == 1
    norm, scale = hc.grad_norm([torch.zeros(0, device=DEV)], max_norm=1.0)
    assert float(norm) == 0 and float(scale) == 1


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_norm_of_what_is_not_finite_skips_the_step(value):
    t = lists([500, 60000], BF16, 9, True)
    t["grads"][1][33333] = value
    norm, scale = hc.grad_norm(t["grads"], max_norm=1.0)
    assert not math.isfinite(float(norm)) and math.isnan(float(scale))
    old = copies(t)
    hc.adamw_step(**t, step=1, grad_scale=scale, **HYPER)
    for k in ("params", "masters", "exp_avgs", "exp_avg_sqs"):
        for a, b in zip(t[k], old[k]):
            assert torch.equal(a, b)
    # a norm that 64 bits hold and fp32 does not
    norm, scale = hc.grad_norm([torch.full((1000,), 3e38, device=DEV)], max_norm=1.0)
    assert float(norm) == math.inf and math.isnan(float(scale))


def test_clipped_step():
    t = lists(SIZES, BF16, 10, True)
    norm, scale = hc.grad_norm(t["grads"], max_norm=0.5)
    check_step(t, 4, scale=float(scale), grad_scale=scale)


def test_refusals():
    t = lists([10, 20], F32, 11)
    bad = [dict(params=[]), dict(grads=t["grads"][:1]), dict(grads=[t["grads"][1], t["grads"][0]]),
           dict(exp_avgs=[x.double() for x in t["exp_avgs"]]), dict(exp_avg_sqs=[x.cpu() for x in t["exp_avg_sqs"]]),
           dict(masters=t["params"][:1]), dict(grad_scale=torch.ones(2, device=DEV)),
           dict(grad_scale=torch.ones(1, device=DEV, dtype=torch.float64)), dict(exp_avg_scales=t["params"]),
           dict(params=[torch.zeros(20, device=DEV)[::2], t["params"][1]]), dict(step=torch.ones(1, device=DEV))]
    for b in bad:
        with pytest.raises(ValueError):
            hc.adamw_step(**{**t, "step": 1, **HYPER, **b})
    e = lists([10, 20], F32, 12, bits=8)
    for b in (dict(exp_avg_scales=None), dict(exp_avg_sq_scales=[e["exp_avg_sq_scales"][0]] * 3),
              dict(exp_avg_scales=[torch.zeros(2, device=DEV)] * 2), dict(exp_avg_sqs=t["exp_avg_sqs"])):
        with pytest.raises(ValueError):
            hc.adamw_step(**{**e, "step": 1, **HYPER, **b})
    for b in (dict(step=0), dict(betas=(1.0, 0.9)), dict(eps=-1.0), dict(lr=math.nan), dict(exp_avgs=t["params"])):
        with pytest.raises(hc.ModelError):
            hc.adamw_step(**{**t, "step": 1, **HYPER, **b})
    with pytest.raises(TypeError):
        hc.adamw_step(**{**t, "params": [x.half() for x in t["params"]]}, step=1, **HYPER)
    with pytest.raises(ValueError):
        hc.grad_norm([])
    with pytest.raises(hc.ModelError):
        hc.grad_norm(t["grads"], max_norm=-1.0)
