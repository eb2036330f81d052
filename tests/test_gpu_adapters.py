"""The linear layer with low-rank adapters on the GPU against its 64-bit
definition: mixtures of adapters in any order, rows without one, odd ranks and
sizes, gradients, isolation of special values."""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _inputs(dtype, M, K, N, n, r, bias=True, scale=True, seed=0):
    g = torch.Generator().manual_seed(2000 + seed)
    dt = DT[dtype]
    return {"x": torch.randn(M, K, generator=g).to(dt),
            "w": (torch.randn(N, K, generator=g) * max(K, 1) ** -0.5).to(dt),
            "a": (torch.randn(n, r, K, generator=g) * max(K, 1) ** -0.5).to(dt),
            "b": (torch.randn(n, N, r, generator=g) * max(r, 1) ** -0.5).to(dt),
            "bias": (torch.randn(N, generator=g) * 0.2).to(dt) if bias else None,
            "scale": torch.rand(n, generator=g) + 0.5 if scale else None,
            "dy": torch.randn(M, N, generator=g).to(dt)}


def _ids(kind, M, n, seed=0):
    g = torch.Generator().manual_seed(77 + seed)
    if kind == "none":
        return torch.full((M,), -1, dtype=torch.int32)
    if kind == "one":
        return torch.full((M,), n - 1, dtype=torch.int32)
    if kind == "mixed":                      # any order, ids outside [0, n) on both sides
        return torch.randint(-2, n + 2, (M,), generator=g, dtype=torch.int32)
    spans = torch.randint(-1, n, (M // 37 + 1,), generator=g, dtype=torch.int32)   # requests of 37 rows
    return spans.repeat_interleave(37)[:M].contiguous()


def _cuda(t):
    return None if t is None else t.cuda()


def _run(t, ids, plan=False):
    from fp32_emulated_gemm_amd.adapters import adapter_linear, plan_weight
    c = {k: _cuda(v) for k, v in t.items()}
    p = plan_weight(c["w"], backward=True) if plan else None
    i = ids.cuda()
    y0 = adapter_linear(c["x"], c["w"], c["a"], c["b"], i, c["scale"], c["bias"], plan=p)
    leaves = [c[k].requires_grad_(True) for k in ("x", "a", "b")]
    y = adapter_linear(*leaves[:1], c["w"], *leaves[1:], i, c["scale"], c["bias"], plan=p)
    dx, da, db = torch.autograd.grad(y, leaves, c["dy"])
    return {"y0": y0, "y": y.detach(), "dx": dx, "da": da, "db": db}


def _check(t, ids, got, label=""):
    want = ref.adapter(t["x"], t["w"], t["a"], t["b"], ids, t["scale"], t["bias"], t["dy"])
    for name in ("y0", "y", "dx", "da", "db"):
        if name in got:
            ref.check(got[name], want[name.rstrip("0")], f"{label} {name}")


SHAPES = [(1, 64, 32, 1, 8), (1, 1, 1, 1, 1), (3, 17, 9, 2, 3), (16, 128, 64, 16, 8), (33, 100, 50, 5, 5),
          (64, 256, 96, 64, 16), (65, 64, 64, 3, 12), (130, 72, 200, 4, 17), (257, 320, 136, 7, 32),
          (300, 200, 70, 2, 64), (520, 136, 260, 9, 40), (700, 1000, 129, 6, 100)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N,n,r", SHAPES)
def test_forward_and_gradients(dtype, M, K, N, n, r):
    t = _inputs(dtype, M, K, N, n, r, bias=M % 2 == 0, scale=N % 2 == 0)
    for kind in ("spans", "mixed"):
        ids = _ids(kind, M, n)
        _check(t, ids, _run(t, ids, plan=kind == "mixed"), kind)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["none", "one"])
@pytest.mark.parametrize("M", [7, 150])
def test_all_or_no_rows(dtype, kind, M):
    t = _inputs(dtype, M, 96, 80, 3, 8, seed=3)
    ids = _ids(kind, M, 3)
    got = _run(t, ids)
    _check(t, ids, got, kind)
    if kind == "none":
        assert not got["da"].any() and not got["db"].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large(dtype):
    for M, K, N, n, r in ((2100, 264, 1030, 11, 16), (4100, 520, 512, 3, 8)):
        t = _inputs(dtype, M, K, N, n, r, seed=5)
        ids = _ids("spans", M, n)
        _check(t, ids, _run(t, ids, plan=True), f"{M} rows")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N,n,r", [(0, 64, 32, 2, 4), (5, 0, 32, 2, 4), (100, 0, 32, 2, 4), (5, 64, 0, 2, 4),
                                       (100, 64, 0, 2, 4), (5, 64, 32, 0, 4), (100, 64, 32, 0, 4), (100, 64, 32, 2, 0),
                                       (5, 64, 32, 2, 0)])
def test_empty(dtype, M, K, N, n, r):
    t = _inputs(dtype, M, K, N, n, r, seed=7)
    ids = _ids("mixed", M, max(n, 1))
    _check(t, ids, _run(t, ids))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [6, 150])
@pytest.mark.parametrize("K", [64, 67])
def test_strides(dtype, M, K):
    from fp32_emulated_gemm_amd.adapters import adapter_linear, plan_weight
    N, n, r = 50, 4, 12
    t = _inputs(dtype, M, K, N, n, r, seed=9)
    ids = _ids("mixed", M, n)
    c = {k: _cuda(v) for k, v in t.items()}
    want = ref.adapter(t["x"], t["w"], t["a"], t["b"], ids, t["scale"], t["bias"])["y"]
    rest = (c["a"], c["b"], ids.cuda(), c["scale"], c["bias"])
    for pad, off in ((8, 0), (5, 3)):
        xs = torch.full((M, K + pad), float("nan"), dtype=c["x"].dtype, device="cuda")[:, off:off + K]
        ws = torch.full((N, K + pad), float("nan"), dtype=c["x"].dtype, device="cuda")[:, off:off + K]
        xs.copy_(t["x"])
        ws.copy_(t["w"])
        ref.check(adapter_linear(xs, ws, *rest), want, f"padded by {pad} from {off}")
        ref.check(adapter_linear(xs, ws, *rest, plan=plan_weight(ws)), want, "with a plan")
    xt, wt = c["x"].t().contiguous().t(), c["w"].t().contiguous().t()
    at = c["a"].transpose(1, 2).contiguous().transpose(1, 2)
    bt = c["b"].transpose(1, 2).contiguous().transpose(1, 2)
    every = torch.stack((ids, ids + 1), 1).cuda()[:, 0]
    ref.check(adapter_linear(xt, wt, at, bt, every, c["scale"], c["bias"]), want, "transposed")
    lead = adapter_linear(c["x"].reshape(2, M // 2, K), c["w"], c["a"], c["b"], ids.cuda().reshape(2, M // 2),
                          c["scale"], c["bias"])
    assert lead.shape == (2, M // 2, N)
    ref.check(lead.reshape(M, N), want, "leading dimensions")
    # a bank that does not start on 16 bytes
    flat = torch.empty(c["b"].numel() + 1, dtype=c["b"].dtype, device="cuda")[1:].view(c["b"].shape)
    flat.copy_(c["b"])
    ref.check(adapter_linear(c["x"], c["w"], c["a"], flat, *rest[2:]), want, "unaligned bank")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [12, 200])
def test_special_values_stay_with_their_adapter(dtype, M):
    """Inf and NaN in one adapter, or in one row, leave the other rows' bits alone."""
    t = _inputs(dtype, M, 64, 48, 4, 8, seed=11)
    ids = _ids("mixed", M, 4)
    clean = _run(t, ids)
    rows = ids == 2
    assert rows.any() and not rows.all()
    for bad in (float("nan"), float("inf")):
        for which in ("a", "b"):
            s = dict(t)
            s[which] = t[which].clone()
            s[which][2, 1, 3] = bad
            got = _run(s, ids)
            for name in ("y0", "y", "dx"):
                assert torch.equal(got[name].cpu()[~rows], clean[name].cpu()[~rows]), (bad, which, name)
            for name in ("da", "db"):
                assert torch.equal(got[name].cpu()[[0, 1, 3]], clean[name].cpu()[[0, 1, 3]]), (bad, which, name)
            assert not torch.isfinite(got["y"].cpu()[rows]).all()
        s = dict(t)
        s["x"] = t["x"].clone()
        s["x"][1, 0] = bad
        got = _run(s, ids)
        keep = [i for i in range(M) if i != 1]
        for name in ("y0", "y"):
            assert torch.equal(got[name].cpu()[keep], clean[name].cpu()[keep]), (bad, name)


def test_gradient_against_differences():
    """<gradient, d> against the central difference of the kernel's own forward along d (Y is linear
    in each operand, so the difference has no error of its own beyond the forward's bounds)."""
    from fp32_emulated_gemm_amd.adapters import adapter_linear
    t = _inputs("f32", 90, 24, 20, 3, 5, seed=13)
    ids = _ids("mixed", 90, 3)
    want = ref.adapter(t["x"], t["w"], t["a"], t["b"], ids, t["scale"], t["bias"], t["dy"])
    got = _run(t, ids)
    g = torch.Generator().manual_seed(5)
    eps = 0.5
    for name in ("x", "a", "b"):
        d = (torch.randint(0, 2, t[name].shape, generator=g) * 2 - 1).float()
        val, noise = [], 0.0
        for sign in (1, -1):
            s = dict(t)
            s[name] = t[name] + sign * eps * d
            c = {k: _cuda(v) for k, v in s.items()}
            y = adapter_linear(c["x"], c["w"], c["a"], c["b"], ids.cuda(), c["scale"], c["bias"])
            val.append((y.double().cpu() * t["dy"].double()).sum().item())
            r = ref.adapter(s["x"], s["w"], s["a"], s["b"], ids, s["scale"], s["bias"])["y"]
            # the definition at the rounded operands, so that rounding t + eps d does not count
            noise += (r[1] * t["dy"].double().abs()).sum().item()
        slope = (got["d" + name].double().cpu() * d.double()).sum().item()
        diff = (val[0] - val[1]) / (2 * eps)
        step = {"x": t["x"], "a": t["a"], "b": t["b"]}[name]
        round_err = (2.0 ** -24 * (step.double().abs() + eps) * want["d" + name][0].abs()).sum().item() / eps
        tol = noise / (2 * eps) + want["d" + name][1].sum().item() + round_err
        assert abs(diff - slope) <= tol, (name, diff, slope, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_deterministic_and_another_stream(dtype):
    t = _inputs(dtype, 900, 264, 200, 5, 16, seed=15)
    ids = _ids("mixed", 900, 5)
    one, two = _run(t, ids), _run(t, ids, plan=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        three = _run(t, ids)
    side.synchronize()
    for name in one:
        assert torch.equal(one[name], two[name]) and torch.equal(one[name], three[name]), name


def test_graph_capture_bf16_and_few_rows():
    from fp32_emulated_gemm_amd.adapters import adapter_linear, plan_weight
    for dtype, M in (("bf16", 300), ("bf16", 9), ("f32", 9)):
        t = _inputs(dtype, M, 136, 72, 4, 8, seed=17)
        c = {k: _cuda(v) for k, v in t.items()}
        i = _ids("mixed", M, 4).cuda()
        plan = plan_weight(c["w"])

        def call():
            return adapter_linear(c["x"], c["w"], c["a"], c["b"], i, c["scale"], c["bias"], plan=plan)

        call()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out = call()
        for k in range(3):
            i.copy_(_ids("mixed", M, 4, seed=k))
            eager = call()
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager), (dtype, M, k)


def test_module():
    from fp32_emulated_gemm_amd.adapters import AdapterLinear
    torch.manual_seed(2)
    layer = torch.nn.Linear(48, 40).cuda()
    m = AdapterLinear.from_linear(layer, adapters=3, rank=4, alpha=8)
    x, ids = torch.randn(70, 48, device="cuda"), _ids("mixed", 70, 3).cuda()
    full = layer.double()(x.double())
    assert (m(x, ids).double() - full).abs().max() < 1e-4 * full.abs().max()      # up starts at zero
    with torch.no_grad():
        m.up.normal_()
    want = ref.adapter(x.cpu(), m.weight.detach().cpu(), m.down.detach().cpu(), m.up.detach().cpu(), ids.cpu(),
                       m.scale.cpu(), m.bias.detach().cpu())["y"]
    y = m(x, ids)
    ref.check(y.detach(), want, "AdapterLinear")
    y.sum().backward()
    assert m.down.grad is not None and m.up.grad is not None and m.weight.grad is None
    with torch.no_grad():
        m.weight.mul_(2)
    with pytest.raises(RuntimeError):
        m(x, ids)
    m.fix_weights()
    m(x, ids)


def test_refusals():
    from fp32_emulated_gemm_amd.adapters import adapter_linear, plan_weight
    t = _inputs("f32", 8, 16, 6, 2, 4)
    c = {k: _cuda(v) for k, v in t.items()}
    i = _ids("mixed", 8, 2).cuda()
    x, w, a, b = c["x"], c["w"], c["a"], c["b"]
    with pytest.raises(TypeError):
        adapter_linear(x, w, a, b, i.long())
    with pytest.raises(TypeError):
        adapter_linear(x, w, a.bfloat16(), b, i)
    with pytest.raises(TypeError):
        adapter_linear(x.half(), w.half(), a.half(), b.half(), i)
    with pytest.raises(TypeError):
        adapter_linear(x, w, a, b, i, scale=c["scale"].double())
    with pytest.raises(TypeError):
        adapter_linear(x, w, a, b, [0] * 8)
    with pytest.raises(ValueError):
        adapter_linear(x, w, a, b, i[:7])
    with pytest.raises(ValueError):
        adapter_linear(x, w, a[:1], b, i)
    with pytest.raises(ValueError):
        adapter_linear(x, w, a, b[:, :5].contiguous(), i)
    with pytest.raises(ValueError):
        adapter_linear(x, w, a, b, i, bias=c["bias"][:5])
    with pytest.raises(ValueError):
        adapter_linear(x, w, a, b, i, scale=c["scale"][:1])
    with pytest.raises(ValueError):
        adapter_linear(x, w, a, b, i.cpu())
    with pytest.raises(ValueError):
        adapter_linear(x, w, a, b, i, plan=plan_weight(a[0]))
    for name in ("w", "bias", "scale"):
        s = dict(c)
        s[name] = c[name].clone().requires_grad_(True)
        y = adapter_linear(s["x"], s["w"], s["a"], s["b"], i, s["scale"], s["bias"])
        with pytest.raises(RuntimeError):
            y.sum().backward()
