"""The gated projection on the GPU against its 64-bit definition: forward, input
and parameter gradients, both types, few rows and tiles, odd sizes and strides."""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _inputs(dtype, M, K, F, bias, seed=0):
    g = torch.Generator().manual_seed(1000 + seed)
    x = torch.randn(M, K, generator=g).to(DT[dtype])
    w = (torch.randn(2 * F, K, generator=g) * max(K, 1) ** -0.5).to(DT[dtype])
    b = (torch.randn(2 * F, generator=g) * 0.2).to(DT[dtype]) if bias else None
    dh = torch.randn(M, F, generator=g).to(DT[dtype])
    return x, w, b, dh


def _cuda(t):
    return None if t is None else t.cuda()


def _run(x, w, b, dh, gate, plan=None):
    """H without gradients, then H and the gradients through autograd."""
    from fp32_emulated_gemm_amd.gated import gated_linear
    xs, ws, bs = _cuda(x), _cuda(w), _cuda(b)
    h0 = gated_linear(xs, ws, bs, gate=gate, plan=plan)
    leaves = [t.requires_grad_(True) for t in (xs, ws, bs) if t is not None]
    h = gated_linear(xs, ws, bs, gate=gate)
    grads = torch.autograd.grad(h, leaves, dh.cuda())
    return {"h0": h0, "h": h.detach(), "dx": grads[0], "dw": grads[1], **({"db": grads[2]} if b is not None else {})}


SHAPES = [(1, 64, 32), (1, 1, 1), (2, 7, 3), (3, 100, 33), (16, 64, 16), (17, 129, 50), (64, 256, 128), (65, 64, 64),
          (130, 96, 40), (200, 72, 129), (257, 320, 136), (300, 1000, 70), (513, 136, 260), (640, 200, 257)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,F", SHAPES)
def test_forward_and_gradients(dtype, M, K, F):
    x, w, b, dh = _inputs(dtype, M, K, F, bias=(M + F) % 2 == 0)
    want = ref.gated(x, w, b, "silu", dh)
    got = _run(x, w, b, dh, "silu")
    ref.check(got["h0"], want["h"], "H")
    for name in ("h", "dx", "dw", "db"):
        if name in got:
            ref.check(got[name], want[name], name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["silu", "gelu", "gelu_tanh", "sigmoid", "relu"])
@pytest.mark.parametrize("M", [5, 150])
def test_gates(dtype, gate, M):
    x, w, b, dh = _inputs(dtype, M, 64, 48, True, seed=7)
    if gate == "relu":
        # integers: the sign of every gate value is exact on both sides
        g = torch.Generator().manual_seed(3)
        x = torch.randint(-3, 4, x.shape, generator=g).to(x.dtype)
        w = torch.randint(-2, 3, w.shape, generator=g).to(w.dtype)
        b = torch.full(b.shape, 0.5).to(b.dtype)
    want = ref.gated(x, w, b, gate, dh)
    got = _run(x, w, b, dh, gate)
    ref.check(got["h0"], want["h"], "H")
    for name in ("h", "dx", "dw", "db"):
        ref.check(got[name], want[name], name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,F", [(700, 768, 520), (2100, 264, 300), (1500, 512, 1100)])
def test_larger_tiles_and_k_slices(dtype, M, K, F):
    x, w, b, dh = _inputs(dtype, M, K, F, True, seed=9)
    want = ref.gated(x, w, b, "gelu", dh)
    got = _run(x, w, b, dh, "gelu")
    for name in ("h0", "h", "dx", "dw", "db"):
        ref.check(got[name], want[name.rstrip("0")], name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("K", [64, 65])
def test_strides(dtype, M, K):
    """Rows of wider buffers, unaligned starts, transposed and expanded operands."""
    from fp32_emulated_gemm_amd.gated import gated_linear, plan_weight
    F = 40
    x, w, b, _ = _inputs(dtype, M, K, F, True, seed=11)
    want = ref.gated(x, w, b, "silu")["h"]
    for pad, off in ((8, 0), (5, 3), (16, 8)):
        xs = torch.full((M, K + pad), float("nan"), dtype=x.dtype, device="cuda")[:, off:off + K]
        ws = torch.full((2 * F, K + pad), float("nan"), dtype=x.dtype, device="cuda")[:, off:off + K]
        xs.copy_(x)
        ws.copy_(w)
        ref.check(gated_linear(xs, ws, b.cuda()), want, f"padded by {pad} from {off}")
        ref.check(gated_linear(xs, ws, b.cuda(), plan=plan_weight(ws)), want, "with a plan")
    xt = x.t().contiguous().cuda().t()
    wt = w.t().contiguous().cuda().t()
    ref.check(gated_linear(xt, wt, b.cuda()), want, "transposed")
    one = x[:1].cuda().expand(M, K)
    want1 = ref.gated(x[:1].expand(M, K), w, b, "silu")["h"]
    ref.check(gated_linear(one, w.cuda(), b.cuda()), want1, "expanded")
    lead = gated_linear(x.cuda().reshape(1, M, 1, K), w.cuda(), b.cuda())
    assert lead.shape == (1, M, 1, F)
    ref.check(lead.reshape(M, F), want, "leading dimensions")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,F", [(0, 64, 32), (5, 0, 32), (100, 0, 32), (5, 64, 0), (100, 64, 0), (0, 0, 0)])
def test_empty(dtype, M, K, F):
    x, w, b, dh = _inputs(dtype, M, K, F, True, seed=13)
    want = ref.gated(x, w, b, "silu", dh)
    got = _run(x, w, b, dh, "silu")
    for name in ("h0", "h", "dx", "dw", "db"):
        ref.check(got[name], want[name.rstrip("0")], name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_partial_gradients_and_expanded_grad(dtype):
    """Only what requires a gradient is computed; dH may be an expanded scalar."""
    from fp32_emulated_gemm_amd.gated import gated_linear
    x, w, b, _ = _inputs(dtype, 90, 72, 40, True, seed=15)
    want = ref.gated(x, w, b, "silu", torch.ones(90, 40, dtype=x.dtype))
    for names in (("x",), ("w",), ("b",), ("x", "b"), ("w", "b")):
        t = {"x": x.cuda(), "w": w.cuda(), "b": b.cuda()}
        for name in names:
            t[name].requires_grad_(True)
        gated_linear(t["x"], t["w"], t["b"]).sum().backward()
        for name in ("x", "w", "b"):
            assert (t[name].grad is not None) == (name in names)
            if name in names:
                ref.check(t[name].grad, want["d" + name], f"d{name} of {names}")


@pytest.mark.parametrize("gate", ["silu", "gelu", "gelu_tanh", "sigmoid"])
def test_gradient_against_differences(gate):
    """<gradient, d> against the central difference of the kernel's own forward along d; the
    tolerance adds the difference's own error (its value on the 64-bit definition), the forward
    bounds over the step, and the gradient's bound."""
    from fp32_emulated_gemm_amd.gated import gated_linear
    x, w, b, dh = _inputs("f32", 24, 20, 12, True, seed=17)
    want = ref.gated(x, w, b, gate, dh)
    got = _run(x, w, b, dh, gate)
    g = torch.Generator().manual_seed(5)
    eps = 2.0 ** -6
    for name, base in (("x", x), ("w", w), ("b", b)):
        d = (torch.randint(0, 2, base.shape, generator=g) * 2 - 1).float()

        def at(sign, forward):
            t = {"x": x, "w": w, "b": b}
            t[name] = base + sign * eps * d
            return forward(t["x"], t["w"], t["b"])

        def kernel(*a):
            return (gated_linear(*(v.cuda() for v in a), gate=gate).double().cpu() * dh.double()).sum().item()

        def exact(*a):
            return (ref.gated(*a, gate)["h"][0] * dh.double()).sum().item()

        def noise(*a):
            return (ref.gated(*a, gate)["h"][1] * dh.double().abs()).sum().item()

        slope = (got["d" + name].double().cpu() * d.double()).sum().item()
        true = (want["d" + name][0] * d.double()).sum().item()
        diff = (at(1, kernel) - at(-1, kernel)) / (2 * eps)
        own = abs((at(1, exact) - at(-1, exact)) / (2 * eps) - true)
        tol = own + (at(1, noise) + at(-1, noise)) / (2 * eps) + want["d" + name][1].sum().item()
        assert abs(diff - slope) <= tol, (name, diff, slope, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_and_special_values(dtype):
    """Saturated gates stay finite; an Inf or NaN reaches its own row only."""
    from fp32_emulated_gemm_amd.gated import gated_linear
    for M in (4, 100):
        x, w, b, _ = _inputs(dtype, M, 64, 32, False, seed=19)
        x = (x.float() * 60).to(x.dtype)
        want = ref.gated(x, w, None, "silu")["h"]
        clean = gated_linear(x.cuda(), w.cuda())
        ref.check(clean, want, "saturated")
        for bad in (float("nan"), float("inf")):
            y = x.clone()
            y[2, 5] = bad
            h = gated_linear(y.cuda(), w.cuda()).cpu()
            assert not torch.isfinite(h[2]).all()
            keep = [i for i in range(M) if i != 2]
            assert torch.equal(h[keep], clean.cpu()[keep])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_deterministic_and_another_stream(dtype):
    x, w, b, dh = _inputs(dtype, 777, 264, 200, True, seed=21)
    one, two = _run(x, w, b, dh, "silu"), _run(x, w, b, dh, "silu")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        three = _run(x, w, b, dh, "silu")
    side.synchronize()
    for name in one:
        assert torch.equal(one[name], two[name]) and torch.equal(one[name], three[name]), name


def test_graph_capture_bf16_and_few_rows():
    """Captured calls replay the eager result, with eager work between the replays."""
    from fp32_emulated_gemm_amd.gated import gated_linear, plan_weight
    for dtype, M in (("bf16", 300), ("bf16", 9), ("f32", 9)):
        x, w, b, _ = _inputs(dtype, M, 136, 72, True, seed=23)
        xs, ws, bs = x.cuda(), w.cuda(), b.cuda()
        plan = plan_weight(ws)
        want = gated_linear(xs, ws, bs, plan=plan)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out = gated_linear(xs, ws, bs, plan=plan)
        for k in range(3):
            xs.copy_((x.float() * (k + 1)).to(x.dtype))
            eager = gated_linear(xs, ws, bs, plan=plan)
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager), (dtype, M, k)
            assert k > 0 or torch.equal(out, want)


def test_modules():
    from fp32_emulated_gemm_amd.gated import GatedFeedForward, GatedLinear
    torch.manual_seed(1)
    gate, up, down = (torch.nn.Linear(48, 80), torch.nn.Linear(48, 80), torch.nn.Linear(80, 48))
    x = torch.randn(70, 48)
    w, b = torch.cat((gate.weight, up.weight)).detach(), torch.cat((gate.bias, up.bias)).detach()
    want = ref.gated(x, w, b, "gelu")["h"]
    m = GatedLinear.from_linears(gate, up, "gelu").cuda()
    ref.check(m(x.cuda()).detach(), want, "GatedLinear")
    m.fix_weights()
    assert not any(p.requires_grad for p in m.parameters())
    ref.check(m(x.cuda()), want, "GatedLinear, fixed weights")
    with torch.no_grad():
        m.weight.mul_(2)
    with pytest.raises(RuntimeError):
        m(x.cuda())
    block = GatedFeedForward.from_linears(gate, up, down, "gelu").cuda()
    xs = x.cuda().requires_grad_(True)
    y = block(xs)
    full = down.double()(want[0])
    assert (y.detach().double().cpu() - full).abs().max() < 1e-4 * full.abs().max()
    y.sum().backward()
    assert xs.grad is not None and block.up.weight.grad is not None and block.up.bias.grad is not None


def test_refusals():
    from fp32_emulated_gemm_amd.gated import GatedLinear, gated_linear, plan_weight
    x, w, b, _ = (_cuda(t) for t in _inputs("f32", 8, 16, 6, True))
    with pytest.raises(ValueError):
        gated_linear(x, w, b, gate="tanh")
    with pytest.raises(ValueError):
        GatedLinear(4, 4, gate="tanh")
    with pytest.raises(TypeError):
        gated_linear(x.half(), w.half())
    with pytest.raises(TypeError):
        gated_linear(x, w.bfloat16())
    with pytest.raises(TypeError):
        gated_linear(x, w, b.double())
    with pytest.raises(ValueError):
        gated_linear(x, w[:11])
    with pytest.raises(ValueError):
        gated_linear(x, w[:, :15].contiguous())
    with pytest.raises(ValueError):
        gated_linear(x, w, b[:5])
    with pytest.raises(ValueError):
        gated_linear(x.cpu(), w)
    with pytest.raises(ValueError):
        gated_linear(x, w.cpu())
    with pytest.raises(ValueError):
        gated_linear(x, w, b, plan=plan_weight(w[:10]))
