"""The model operators together: a training step of a small model against 64 bits, captured steps, streams, one token."""
import threading

import pytest
import torch

import gated_convolution_sequence_amd as hc
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HYPER = dict(lr=2e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    hc.layer_lib(), hc.model_lib()
    yield
    torch.cuda.synchronize()


def weights(D, V, dtype, seed=0):
    """Embedding, and per block a norm and a square projection; a last norm and the readout with its bias."""
    gen = torch.Generator().manual_seed(seed)

    def new(*shape, scale, shift=0.0):
        return (shift + scale * torch.randn(*shape, generator=gen)).to(DEV, dtype)

    w = [new(V, D, scale=1.0)]
    for _ in range(2):
        w += [new(D, scale=0.1, shift=1.0), new(D, scale=0.1), new(D, D, scale=D ** -0.5)]
    return w + [new(D, scale=0.1, shift=1.0), new(V, D, scale=D ** -0.5), new(V, scale=0.1)]


def loss_of(w, tokens, target):
    x = w[0][tokens]
    for i in range(2):
        g, b, p = w[1 + 3 * i:4 + 3 * i]
        x = hc.LinearAct.apply(hc.Norm.apply(x, g, b), p, None, x, "silu")
    x = hc.Norm.apply(x, w[7], None, "rms")
    return hc.LinearXent.apply(x, w[8], target, w[9])


def plain_loss(w, tokens, target):
    x = w[0][tokens]
    for i in range(2):
        g, b, p = w[1 + 3 * i:4 + 3 * i]
        z = torch.nn.functional.layer_norm(x, x.shape[-1:], g, b, 1e-5) @ p.t()
        x = z * torch.sigmoid(z) + x
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * w[7]
    z = (x @ w[8].t() + w[9]).flatten(0, 1)
    return torch.nn.functional.cross_entropy(z, target.flatten(), ignore_index=-100, reduction="none").view(target.shape)


def data(B, L, V, seed):
    gen = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, V, (B, L), generator=gen)
    target = torch.randint(0, V, (B, L), generator=gen)
    target[torch.rand(B, L, generator=gen) < 0.3] = -100
    return tokens.to(DEV), target.to(DEV)


def grads_of(w, tokens, target):
    leaves = [x.detach().requires_grad_(True) for x in w]
    loss = loss_of(leaves, tokens, target)
    (loss.sum() / (target >= 0).sum()).backward()
    return loss.detach(), [x.grad for x in leaves]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,V", [(64, 300), (129, 1001)])
def test_a_training_step(dtype, D, V):
    """Loss, every gradient, and the weights after a clipped step.

    A gradient passes some ten operators, each within a few units of its type's rounding (bf16 2^-8, in sums of
    independent ones): 2^-4 of its largest element in bf16, 2^-14 in fp32.  The step is held to the gradients that
    the operators gave: a first step's corrected moments are g and g^2."""
    log("training step %s D=%d" % (dtype, D))
    tokens, target = data(3, 50, V, 1)
    w = weights(D, V, dtype)
    loss, grads = grads_of(w, tokens, target)
    exact = [x.double().requires_grad_(True) for x in w]
    want = plain_loss(exact, tokens, target)
    (want.sum() / (target >= 0).sum()).backward()
    tol = 2.0 ** -4 if dtype == BF16 else 2.0 ** -14
    assert (loss.double() - want).abs().max() <= tol * want.abs().max()
    assert not loss[target < 0].any()
    for i, (g, x) in enumerate(zip(grads, exact)):
        assert (g.double() - x.grad).abs().max() <= tol * x.grad.abs().max(), i
    # the step itself, from these gradients
    norm, scale = hc.grad_norm(grads, max_norm=0.5)
    true = torch.sqrt(sum(g.double().square().sum() for g in grads))
    assert abs(float(norm) / float(true) - 1) < 1e-6 and abs(float(scale) - min(1, 0.5 / float(true))) < 1e-6
    masters = [x.float().clone() for x in w]
    m, v = ([torch.zeros_like(x) for x in masters] for _ in range(2))
    hc.adamw_step(w, grads, m, v, step=1, masters=masters, grad_scale=scale, **HYPER)
    for p, old, q, g in zip(w, exact, masters, grads):
        gs = g.double() * float(scale)
        new = old.detach() * (1 - 2e-3 * 0.1) - 2e-3 * gs / (gs.abs() + 1e-8)
        # eight units of the sum's largest part
        assert (q.double() - new).abs().max() <= 8 * 2.0 ** -24 * (old.abs().max() + 2e-3)
        assert torch.equal(p, q.to(dtype))


def test_training_by_captured_steps():
    """Forward, backward and step in one graph; replays on new data, masks, rates and steps give the eager bits."""
    D, V = 96, 500
    tokens, target = data(2, 40, V, 2)
    lr, step = torch.zeros(1, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)

    def make():
        w = weights(D, V, BF16, 3)
        masters = [x.float() for x in w]
        return dict(w=w, masters=masters, m=[torch.zeros_like(x) for x in masters], v=[torch.zeros_like(x) for x in masters])

    def train(s, lr, step, tokens, target):
        w = s["w"]
        # without autograd, so that no graph of the leaves outlives the call
        x0 = w[0][tokens]
        y0, mean, rstd = hc.norm_fwd(x0, w[1], w[2], save_stats=True)
        x1, z = hc.linear_fwd(y0, w[3], residual=x0, act="silu", save_preact=True)
        y1, _, r1 = hc.norm_fwd(x1, w[7], kind="rms", save_stats=True)
        loss, lse = hc.xent_fwd(y1, w[8], target, bias=w[9])
        count = (target >= 0).sum().clamp(min=1)
        dloss = torch.ones_like(loss) / count
        dy1, dw8, dw9 = hc.xent_bwd(y1, w[8], target, lse, dloss, bias=w[9])
        dx1, dw7, _ = hc.norm_bwd(x1, w[7], dy1, None, r1, kind="rms", need_db=False)
        dy0, dw3, _ = hc.linear_bwd(y0, w[3], dx1, preact=z, act="silu", need_db=False)
        dx0, dw1, dw2 = hc.norm_bwd(x0, w[1], dy0, mean, rstd)
        idx = [1, 2, 3, 7, 8, 9]
        grads = [dw1, dw2, dw3, dw7, dw8, dw9]
        _, scale = hc.grad_norm(grads, max_norm=1.0)
        hc.adamw_step([w[i] for i in idx], grads, [s["m"][i] for i in idx], [s["v"][i] for i in idx], step=step, lr=lr,
                      betas=HYPER["betas"], weight_decay=0.1, masters=[s["masters"][i] for i in idx], grad_scale=scale)
        return loss, dx0

    static, eager, start = make(), make(), make()
    train(static, lr, step, tokens, target)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = train(static, lr, step, tokens, target)
    for k in static:
        for a, b in zip(static[k], start[k]):
            a.copy_(b)
    for r in range(1, 6):
        t, g = data(2, 40, V, 10 + r)
        if r == 3:
            g.fill_(-100)  # no target at all
        if r == 4:
            g.random_(0, V)  # all
        tokens.copy_(t), target.copy_(g)
        lr.fill_(1e-3 / r), step.fill_(r)
        torch.cuda.synchronize()
        graph.replay()
        want = train(eager, torch.full((1,), 1e-3 / r, device=DEV), torch.tensor([r], device=DEV), t, g)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), r
        for k in static:
            for i, (a, b) in enumerate(zip(static[k], eager[k])):
                assert torch.equal(a, b), (r, k, i)


def test_calls_on_streams_of_several_threads():
    """Each entry point on a stream of its own while the others run: the bits of the call alone."""
    gen = torch.Generator(device=DEV).manual_seed(5)

    def randn(*shape, dtype=BF16):
        return torch.randn(*shape, generator=gen, device=DEV).to(dtype)

    x, w, b, dy = randn(3000, 512), randn(512), randn(512), randn(3000, 512)
    y, mean, rstd = hc.norm_fwd(x, w, b, save_stats=True)
    readout = randn(2000, 512) * 0.05
    target = torch.randint(-500, 2000, (3000,), generator=gen, device=DEV)
    loss, lse = hc.xent_fwd(x, readout, target)
    dloss = torch.rand(3000, generator=gen, device=DEV)
    grads = [randn(n) for n in (7, 40000, 333)]

    def adam(stream):
        p, m, v = [g.clone() for g in grads], *([torch.zeros(g.shape, device=DEV) for g in grads] for _ in range(2))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        norm, scale = hc.grad_norm(grads, max_norm=1.0, stream=stream)
        hc.adamw_step(p, grads, m, v, step=2, lr=1e-2, grad_scale=scale, stream=stream)
        return (norm, *p, *m, *v)

    jobs = [lambda s: hc.norm_fwd(x, w, b, save_stats=True, stream=s), lambda s: hc.norm_bwd(x, w, dy, mean, rstd, stream=s),
            lambda s: hc.xent_fwd(x, readout, target, stream=s), lambda s: hc.xent_fwd(x[:9], readout, target[:9], stream=s),
            lambda s: hc.xent_bwd(x, readout, target, lse, dloss, stream=s), adam]
    alone = [job(None) for job in jobs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        for _ in range(20):
            got = jobs[i](stream)
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, alone[i]) if a is not None):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_one_token_after_a_batch():
    """A norm and the loss of single rows equal the batch's rows: the same sums, whatever else runs beside them."""
    gen = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(700, 1000, generator=gen, device=DEV).to(BF16)
    w = torch.randn(1000, generator=gen, device=DEV).to(BF16)
    y = hc.norm_fwd(x, w)[0]
    for i in (0, 350, 699):
        assert torch.equal(hc.norm_fwd(x[i], w)[0], y[i])


@pytest.mark.parametrize("shift", [16, 48, 240])
def test_workspaces_at_any_16_bytes(shift):
    """A workspace of the reported size, 16 bytes aligned: bytes around it stay, results do too."""
    gen = torch.Generator(device=DEV).manual_seed(7)
    M, K, V = 300, 200, 1500
    x = torch.randn(M, K, generator=gen, device=DEV).to(BF16)
    w = (torch.randn(V, K, generator=gen, device=DEV) * 0.1).to(BF16)
    target = torch.randint(-300, V, (M,), generator=gen, device=DEV)
    bias = torch.zeros(V, dtype=BF16, device=DEV)
    loss, lse = hc.xent_fwd(x, w, target, bias=bias)
    want = hc.xent_bwd(x, w, target, lse, loss, bias=bias)

    def space(n):
        big = torch.full((n + 4096,), 90, dtype=torch.uint8, device=DEV)
        return big, big[shift:shift + n]

    big, ws = space(hc.xent_workspace_bytes(M, K, V))
    a, b = hc.xent_fwd(x, w, target, bias=bias, workspace=ws)
    assert torch.equal(a, loss) and torch.equal(b, lse)
    assert bool((big[:shift] == 90).all()) and bool((big[shift + ws.numel():] == 90).all())
    big, ws = space(hc.xent_workspace_bytes(M, K, V, 0, True))
    for a, b in zip(hc.xent_bwd(x, w, target, lse, loss, bias=bias, workspace=ws), want):
        assert torch.equal(a, b)
    assert bool((big[:shift] == 90).all()) and bool((big[shift + ws.numel():] == 90).all())
