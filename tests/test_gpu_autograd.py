"""Gradients through autograd: the same bits as the gradient calls', for every
argument that has one."""
import pytest
import torch

from lossless_bf16_tensor_sign_amd import zc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def rand(*shape, dtype=torch.float32, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def some_slots(T, k, E=5, seed=3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    e = torch.randint(-1, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    return zc.expert_slots(e, E)[0]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(dtype, score, renorm):
    x = rand(70, 24, dtype=dtype)
    bias = 0.1 * rand(24)
    kw = dict(score=score, renorm=renorm, scale=2.5)
    e, w = zc.route(x, 4, bias=bias, groups=4, top_groups=2, **kw)
    assert not w.requires_grad
    leaf = x.clone().requires_grad_()
    e2, w2 = zc.route(leaf, 4, bias=bias, groups=4, top_groups=2, **kw)
    assert torch.equal(e, e2) and torch.equal(w, w2) and w2.requires_grad and not e2.requires_grad
    g = rand(70, 4)
    w2.backward(g)
    assert torch.equal(leaf.grad, zc.route_grad(x, e, g, **kw))
    # a gradient that is not contiguous, a row view of the logits, a token without experts
    leaf = rand(70, 30, dtype=dtype).requires_grad_()
    valid = torch.arange(70, device=DEV) != 3
    e3, w3 = zc.route(leaf[:, 3:27], 4, valid=valid, **kw)
    w3.sum().backward()
    want = zc.route_grad(leaf.detach()[:, 3:27].contiguous(), e3, torch.ones(70, 4, device=DEV), **kw)
    assert torch.equal(leaf.grad[:, 3:27], want) and not leaf.grad[:, :3].any() and not leaf.grad[3].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [1, 9, 128, 301])
def test_dispatch(dtype, H):
    T, k = 37, 3
    s = some_slots(T, k)
    x = rand(T, H, dtype=dtype).requires_grad_()
    rows = zc.dispatch(x, s)
    assert torch.equal(rows.detach(), zc.dispatch(x.detach(), s)) and rows.requires_grad
    g = rand(T * k, H, dtype=dtype)
    rows.backward(g)
    assert torch.equal(x.grad, zc.combine(g, s))
    x.grad = None
    zc.dispatch(x, s).t().sum(1).sum().backward()                 # strides (0, 0)
    assert torch.equal(x.grad, zc.combine(torch.ones_like(g), s))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [1, 9, 128, 301])
@pytest.mark.parametrize("needs", ["rows", "weights", "base", "rows weights", "rows base", "weights base",
                                   "rows weights base"])
def test_combine(dtype, H, needs):
    T, k = 37, 3
    s = some_slots(T, k)
    d = rand(T, H, dtype=dtype, seed=9)
    for weighted in (True, False):
        y, w, b = rand(T * k, H, dtype=dtype), rand(T, k, seed=1) if weighted else None, rand(T, H, dtype=dtype, seed=2)
        for t, name in ((y, "rows"), (w, "weights"), (b, "base")):
            if t is not None and name in needs:
                t.requires_grad_()
        if not any(t is not None and t.requires_grad for t in (y, w, b)):
            continue
        for up, back in ((d, lambda o: o.backward(d)),
                         (torch.full_like(d, 2.0), lambda o: (o * 2).sum().backward())):       # strides (0, 0)
            for t in (y, w, b):
                if t is not None:
                    t.grad = None
            out = zc.combine(y, s, weights=w, base=b)
            with torch.no_grad():
                again = zc.combine(y, s, weights=w, base=b)
                dy, dw = zc.combine_grad(up, y, s, w) if weighted else (zc.dispatch(up, s), None)
            assert out.requires_grad and not again.requires_grad and torch.equal(out.detach(), again)
            back(out)
            for t, name, want in ((y, "rows", dy), (w, "weights", dw), (b, "base", up)):
                if t is not None:
                    assert (t.grad is None) == (name not in needs)
                    assert t.grad is None or torch.equal(t.grad, want)


@pytest.mark.parametrize("stream", [False, True])
def test_layer(stream):
    # router, experts and shared path; by hand with the gradient calls and through autograd
    T, E, k, H = 200, 8, 2, 64
    x, router = rand(T, H), rand(H, E) * H ** -0.5
    scale = 1.0 + rand(E)
    d = rand(T, H, seed=5)
    side = torch.cuda.Stream() if stream else None
    kw = dict(score="sigmoid", scale=1.5)

    def expert(rows, counts, c):
        ends = counts.cumsum(0)[:-1]
        which = torch.bucketize(torch.arange(rows.shape[0], device=DEV), ends, right=True).clamp(max=E - 1)
        return rows * c[which][:, None]
    logits = x @ router
    e, w = zc.route(logits, k, **kw)
    s, n = zc.expert_slots(e, E)
    back = expert(zc.dispatch(x, s), n, scale)
    out = zc.combine(back, s, weights=w, base=x)
    d_back, d_w = zc.combine_grad(d, back, s, w)
    d_logits = zc.route_grad(logits, e, d_w, **kw)

    xs, rs, cs = (t.clone().requires_grad_() for t in (x, router, scale))
    lg = xs @ rs
    torch.cuda.synchronize()
    e2, w2 = zc.route(lg, k, stream=side, **kw)
    s2, n2 = zc.expert_slots(e2, E, stream=side)
    torch.cuda.synchronize()
    r2 = zc.dispatch(xs, s2, stream=side)
    torch.cuda.synchronize()
    back2 = expert(r2, n2, cs)
    torch.cuda.synchronize()
    out2 = zc.combine(back2, s2, weights=w2, base=xs, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, out2.detach())
    out2.backward(d)
    torch.cuda.synchronize()
    assert torch.equal(rs.grad, x.t() @ d_logits)
    # three paths join in x, in an order of autograd's own: two fp32 additions
    parts = [d, zc.combine(expert(d_back, n, scale), s), d_logits @ router.t()]
    mag = sum(p.abs() for p in parts)
    assert ((xs.grad - sum(parts)).abs() <= 4 * 2.0 ** -24 * mag + 1e-30).all()
    assert cs.grad is not None and cs.grad.shape == (E,)


def test_gradients_have_no_gradient():
    x = rand(5, 8).requires_grad_()
    e, w = zc.route(x, 2)
    (g,) = torch.autograd.grad(w[:, 0].sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
