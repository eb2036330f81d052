"""Calls of the experts' operators and 4-bit weights as programs make them: modules,
graphs, streams, layouts of the tensors, refusals, operands past 32-bit offsets."""
import pytest
import torch

import experts_reference as xr
import ops_reference as ref

pytestmark = pytest.mark.gpu


def _layer(dtype, features=96, hidden=72, experts=5, bias=True, gate="silu", seed=0):
    from fp32_emulated_gemm_amd.experts import ExpertFeedForward
    torch.manual_seed(seed)
    m = ExpertFeedForward(features, hidden, experts, bias=bias, gate=gate, device="cuda", dtype=xr.DT[dtype])
    with torch.no_grad():
        for p in (m.up_bias, m.down_bias):
            if p is not None:
                p.normal_(std=0.1)
    return m


def _inputs(dtype, T, k, m, seed=1, padded=True):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(m.experts, generator=g)[:k] for _ in range(T)]).int()
    if padded:
        ids[::7] = -1
    x = torch.randn(T, m.features, generator=g).to(xr.DT[dtype])
    weights = torch.softmax(torch.randn(T, k, generator=g), 1)
    dy = torch.randn(T, m.features, generator=g).to(x.dtype)
    return x, ids, weights, dy


def _reference(m, x, ids, weights, up=None, down=None):
    """The layer in float64 with autograd, token by token."""
    P = {n: p.detach().double().cpu().requires_grad_(True) for n, p in m.named_parameters()} if up is None else None
    if up is None:
        up, down, ub, db = P["up"], P["down"], P.get("up_bias"), P.get("down_bias")
    else:
        ub, db = (None if b is None else b.detach().double().cpu() for b in (m.up_bias, m.down_bias))
    x, weights = x.double().requires_grad_(True), weights.double().requires_grad_(True)
    ys = []
    for t in range(x.shape[0]):
        y = x.new_zeros(x.shape[1])
        for j, e in enumerate(ids[t].tolist()):
            if e < 0:
                continue
            z = up[e] @ x[t] + (0 if ub is None else ub[e])
            F = z.shape[0] // 2
            act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[m.gate]
            y = y + weights[t, j] * (down[e] @ (act(z[:F]) * z[F:]) + (0 if db is None else db[e]))
        ys.append(y)
    return torch.stack(ys), x, weights, P


def _near(got, want, rel, label):
    """Relative to the tensor's largest value: sums of products of several rounded steps."""
    err = (got.detach().double().cpu() - want.detach()).abs().max().item()
    assert err <= rel * want.abs().max().item() + 1e-30, f"{label}: {err:.3g} of {want.abs().max().item():.3g}"


# a chain of four products of at most 96 terms: float32 2 * 96 roundings each; bfloat16 has four
# rounded tensors on the way (xs, h, ys, dZ), 2^-8 each, and its output
REL = {"f32": 4 * 2 * 96 * 2.0 ** -24, "bf16": 5 * 2.0 ** -8}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,gate,bias", [(1, 2, "silu", False), (9, 3, "gelu", True), (150, 2, "silu", True)])
def test_layer_of_experts(dtype, T, k, gate, bias):
    m = _layer(dtype, bias=bias, gate=gate)
    x, ids, weights, dy = _inputs(dtype, T, k, m, padded=T > 1)
    want, x64, w64, P = _reference(m, x, ids, weights)
    want.backward(dy.double())
    xd, wd = x.cuda().requires_grad_(True), weights.cuda().requires_grad_(True)
    y = m(xd, ids.cuda(), wd)
    y.backward(dy.cuda())
    _near(y, want, REL[dtype], "y")
    _near(xd.grad, x64.grad, REL[dtype], "dx")
    _near(wd.grad, w64.grad, REL[dtype], "dweights")
    for name, p in m.named_parameters():
        _near(p.grad, P[name].grad, REL[dtype], name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 120])
def test_layer_of_experts_in_4_bits(dtype, T):
    from fp32_emulated_gemm_amd.quant4 import Quant4ExpertFeedForward
    m = _layer(dtype)
    q = Quant4ExpertFeedForward.from_experts(m, group=32)
    x, ids, weights, _ = _inputs(dtype, T, 2, m)
    up, down = (q._held(n).dequantize().double().cpu() for n in ("up", "down"))
    want = _reference(m, x, ids, weights, up, down)[0]
    _near(q(x.cuda(), ids.cuda(), weights.cuda()), want, REL[dtype], "y")
    copy = Quant4ExpertFeedForward.from_experts(m, group=32)
    copy.load_state_dict(q.state_dict())
    moved = copy.to("cpu").to("cuda")
    assert torch.equal(moved(x.cuda(), ids.cuda(), weights.cuda()), q(x.cuda(), ids.cuda(), weights.cuda()))


@pytest.mark.parametrize("kind", ["torch", "emulated", "gated"])
def test_layers_in_4_bits(kind):
    from fp32_emulated_gemm_amd.gated import GatedLinear
    from fp32_emulated_gemm_amd.linear import Linear
    from fp32_emulated_gemm_amd.quant4 import Quant4Linear
    torch.manual_seed(3)
    plain = torch.nn.Linear(130, 40, device="cuda")
    layer = {"torch": lambda: plain, "emulated": lambda: Linear.from_linear(plain),
             "gated": lambda: GatedLinear(130, 24, gate="gelu", device="cuda", dtype=torch.float32)}[kind]()
    q = Quant4Linear.from_linear(layer, group=64, symmetric=kind == "torch")
    x = torch.randn(2, 5, 130, device="cuda")
    z = x.double() @ q.weight.dequantize().double().T + layer.bias.double()
    want = z if kind != "gated" else torch.nn.functional.gelu(z[..., :24]) * z[..., 24:]
    with torch.no_grad():
        y = q(x)
    assert y.shape == want.shape
    assert (y - want).abs().max() <= 2.0 ** -17 * want.abs().max()     # 130 terms of 4-bit values, offset by 16
    assert "group=64" in repr(q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 200])
def test_captured_and_replayed(dtype, T):
    """The layer, its gradients and its 4-bit form in a graph: every replay, with other inputs and eager
    work between them, equals the eager result bit for bit."""
    from fp32_emulated_gemm_amd.quant4 import Quant4ExpertFeedForward
    m = _layer(dtype)
    q = Quant4ExpertFeedForward.from_experts(m)
    leaves = (m.up, m.down, m.up_bias, m.down_bias)
    x, ids, weights, dy = (t.cuda() for t in _inputs(dtype, T, 2, m))
    x.requires_grad_(True)

    def step():
        y = m(x, ids, weights)
        grads = torch.autograd.grad(y, (x, *leaves), dy)
        with torch.no_grad():
            return [y.detach(), *grads, q(x, ids, weights)]

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(3):
        new = _inputs(dtype, T, 2, m, seed=10 + seed)
        with torch.no_grad():
            for to, frm in zip((x, ids, weights, dy), new):
                to.copy_(frm)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(held, want)):
            assert torch.equal(a, b), (seed, k)


def test_on_another_stream():
    from fp32_emulated_gemm_amd.quant4 import Quant4ExpertFeedForward
    m = _layer("bf16")
    q = Quant4ExpertFeedForward.from_experts(m)
    x, ids, weights, _ = (t.cuda() for t in _inputs("bf16", 300, 2, m))
    with torch.no_grad():
        want = m(x, ids, weights), q(x, ids, weights)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        got = []
        for s in streams:
            with torch.cuda.stream(s):
                got.append((m(x, ids, weights), q(x, ids, weights)))
        torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [6, 300])
def test_layouts(dtype, T):
    """Transposed and strided rows, weights, biases and output gradients equal contiguous ones."""
    from fp32_emulated_gemm_amd.experts import expert_linear, sort_tokens
    from fp32_emulated_gemm_amd.quant4 import quant4_linear, quantize
    n, N, K, P = 4, 48, 56, 2 * T
    g = torch.Generator("cuda").manual_seed(T)
    ids = torch.randint(-1, n, (T, 2), generator=g, device="cuda", dtype=torch.int32)
    order = sort_tokens(ids, n)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(xr.DT[dtype])

    wide, across = normal(P, K + 11), normal(K, P)
    weight, bias = normal(n, K, N).transpose(1, 2), normal(N, n).t()
    dh = normal(N, P).t()
    w4 = quantize(weight, 32)
    one = quantize(weight[0], 32)
    for x in (wide[:, 3:3 + K], wide[:, 8:8 + K], across.t(), wide[:1, :K].expand(P, K)):
        leaf = x.detach().requires_grad_(True)
        a = expert_linear(leaf, weight, order, bias)
        da, = torch.autograd.grad(a, (leaf,), dh)
        flat = x.detach().contiguous().requires_grad_(True)
        b = expert_linear(flat, weight.contiguous(), order, bias.contiguous())
        db, = torch.autograd.grad(b, (flat,), dh.contiguous())
        with torch.no_grad():
            c, d = quant4_linear(x, w4, bias, order=order), quant4_linear(flat, w4, bias.contiguous(), order=order)
            e, f = quant4_linear(x, one), quant4_linear(flat, one)
        for got, want in ((a, b), (da, db), (c, d), (e, f)):
            # other kernels where rows do not lie: the same sums in another order
            assert (got.double() - want.double()).abs().max() <= (2.0 ** -7 if dtype == "bf16" else 2.0 ** -18) * want.abs().max()


@pytest.mark.parametrize("loss", [lambda y: y.sum(), lambda y: y.square().sum()])
def test_second_derivatives_are_refused(loss):
    """A recorded backward pass gives the gradients of one that is not, and no derivative of its own (torch
    refuses at the backward node, or has no node where the incoming gradient is a constant)."""
    from fp32_emulated_gemm_amd.experts import ExpertFeedForward
    torch.manual_seed(1)
    m = ExpertFeedForward(24, 16, 3, device="cuda")
    x = torch.randn(5, 24, device="cuda", requires_grad=True)
    ids = (torch.arange(10, device="cuda").view(5, 2) % 3).int()
    weights = torch.rand(5, 2, device="cuda", requires_grad=True)
    leaves = (x, weights, *m.parameters())
    plain = torch.autograd.grad(loss(m(x, ids, weights)), leaves)
    recorded = torch.autograd.grad(loss(m(x, ids, weights)), leaves, create_graph=True)
    for a, b in zip(plain, recorded):
        assert torch.equal(a, b)
        with pytest.raises(RuntimeError):
            b.sum().backward(retain_graph=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P,K,ld", [(1, 129, 130), (2, 129, 130), (5, 63, 66), (17, 1, 2), (40, 255, 258), (65, 33, 40)])
def test_odd_rows_at_even_strides(dtype, P, K, ld):
    """The last element of the last row, and nothing behind it (NaN there), in each product."""
    from fp32_emulated_gemm_amd.experts import expert_linear, sort_tokens
    from fp32_emulated_gemm_amd.quant4 import quant4_linear, quantize
    g = torch.Generator("cuda").manual_seed(P + K)
    wide = torch.full((P, ld), float("nan"), device="cuda", dtype=xr.DT[dtype])
    wide[:, :K] = torch.randn(P, K, generator=g, device="cuda").to(wide.dtype)
    wide[:, K - 1] = 8.0                         # a lost last column shows
    x = wide[:, :K]
    weight = torch.randn(1, 32, K, generator=g, device="cuda").to(wide.dtype)
    order = sort_tokens(torch.zeros(P, device="cuda", dtype=torch.int32), 1)
    w4 = quantize(weight, 32)
    one = quantize(weight[0], 32)
    for got, w in ((expert_linear(x, weight, order), weight[0]), (quant4_linear(x, w4, order=order), w4.dequantize()[0]),
                   (quant4_linear(x, one), one.dequantize())):
        want = x.double() @ w.double().t()
        # the sums' roundings, of terms up to 31 scales in 4 bits (a scale: at most 2/15 of the
        # largest weight); in bfloat16 also the result's, and an unpacked weight's
        w = w.double().abs()
        room = x.double().abs() @ (w + 62 / 15 * w.amax(1, keepdim=True)).t()
        tol = (K / 4 + 8) * 2.0 ** -24 * room
        if dtype == "bf16":
            tol = tol + 2.0 ** -8 * (want.abs() + x.double().abs() @ w.t())
        assert ((got.double() - want).abs() <= tol).all()


def test_refusals():
    from fp32_emulated_gemm_amd.experts import combine_tokens, expert_linear, gather_tokens, sort_tokens
    from fp32_emulated_gemm_amd.quant4 import quant4_linear, quantize
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    order = sort_tokens(ids, 3)
    x, ys, w = torch.zeros(4, 8, device="cuda"), torch.zeros(8, 8, device="cuda"), torch.zeros(3, 6, 8, device="cuda")
    w4, bank = quantize(w[0]), quantize(w)
    for bad in (lambda: sort_tokens(ids, 1025), lambda: sort_tokens(ids, -1), lambda: gather_tokens(ys, order),
                lambda: combine_tokens(x, order), lambda: combine_tokens(ys, order, torch.zeros(4, 3, device="cuda")),
                lambda: expert_linear(ys, w[:2], order), lambda: expert_linear(ys, w[:, :, :4], order),
                lambda: expert_linear(ys, w[:, :5], order, gate="silu"), lambda: expert_linear(ys, w, order, gate="tanh"),
                lambda: expert_linear(ys, w, order, torch.zeros(3, 5, device="cuda")),
                lambda: expert_linear(ys, w.cpu(), order), lambda: quant4_linear(x, bank), lambda: quant4_linear(ys, w4, order=order),
                lambda: quant4_linear(x[:, :4], w4), lambda: quant4_linear(x, w4, torch.zeros(5, device="cuda")),
                lambda: quant4_linear(x[0, 0], bank, order=order),
                lambda: quant4_linear(x, quantize(w[0, :5]), gate="silu")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gather_tokens(x.double(), order), lambda: expert_linear(ys, w.bfloat16(), order),
                lambda: combine_tokens(ys, order, torch.zeros(4, 2, device="cuda", dtype=torch.bfloat16)),
                lambda: quant4_linear(x.half(), w4), lambda: quant4_linear(x, w4, torch.zeros(6, device="cuda").bfloat16())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(RuntimeError):
        quant4_linear(x.clone().requires_grad_(True), w4)
    with torch.no_grad():
        quant4_linear(x.clone().requires_grad_(True), w4)


def test_tangents_are_refused():
    from torch.autograd import forward_ad
    from fp32_emulated_gemm_amd.experts import combine_tokens, expert_linear, gather_tokens, sort_tokens
    from fp32_emulated_gemm_amd.quant4 import quant4_linear, quantize
    order = sort_tokens(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 3)
    x, ys, w = torch.ones(4, 8, device="cuda"), torch.ones(8, 8, device="cuda"), torch.ones(3, 6, 8, device="cuda")
    w4 = quantize(w[0])
    with forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))   # noqa: E731
        for bad in (lambda: gather_tokens(dual(x), order), lambda: combine_tokens(dual(ys), order),
                    lambda: expert_linear(dual(ys), w, order), lambda: expert_linear(ys, dual(w), order),
                    lambda: quant4_linear(dual(x), w4)):
            with pytest.raises(NotImplementedError):
                bad()
        assert torch.equal(quant4_linear(x, w4), quant4_linear(x.clone(), w4))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_past_32_bit_offsets(dtype):
    """The last rows and the last expert of operands of more than 2^32 bytes."""
    from fp32_emulated_gemm_amd.experts import combine_tokens, expert_linear, gather_tokens, sort_tokens
    from fp32_emulated_gemm_amd.quant4 import quant4_linear, quantize_values, pack
    dt = xr.DT[dtype]
    T, K = 300_000, 8192
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ids[-1], ids[0] = -1, 1
    order = sort_tokens(ids, 2)
    x = torch.zeros(T, K, dtype=dt, device="cuda")
    x[-3:] = torch.randn(3, K, device="cuda").to(dt)
    xs = gather_tokens(x, order)
    assert torch.equal(xs[T - 4:T - 2], x[T - 3:T - 1]) and not xs[T - 2:].any()
    y = combine_tokens(xs, order)
    assert torch.equal(y[T - 3:T - 1], x[T - 3:T - 1]) and not y[-1].any()
    w = torch.randn(2, 64, K, device="cuda").to(dt) * K ** -0.5
    h = expert_linear(xs, w, order)
    want = x[T - 3:T - 1].double() @ w[0].double().T
    assert (h[T - 4:T - 2].double() - want).abs().max() <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -19) * want.abs().max()
    del x, xs, y, h
    n, N = 40, 8192
    bank = torch.zeros(n, N, K, dtype=dt, device="cuda")
    bank[-1, -16:] = torch.randn(16, K, device="cuda").to(dt)
    few = torch.randn(8, K, device="cuda").to(dt)
    order = sort_tokens(torch.full((8, 1), n - 1, dtype=torch.int32, device="cuda"), n)
    want = few.double() @ bank[-1].double().T
    tol = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -19) * want.abs().max()
    assert (expert_linear(few, bank, order).double() - want).abs().max() <= tol
    q, scale, zero = quantize_values(bank)
    del bank
    w4 = pack(q, scale, zero)
    del q
    want = few.double() @ (w4.dequantize(torch.bfloat16)[-1].double().T if dtype == "bf16" else w4.dequantize()[-1].double().T)
    assert (quant4_linear(few, w4, order=order).double() - want).abs().max() <= 2 * tol + 2.0 ** -8 * want.abs().max()
