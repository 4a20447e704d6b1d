"""Routing, slots and rows at the limits between their kernels' forms, and all
of them in a captured graph.  Tolerances as in test_gpu_moe.py."""
import numpy as np
import pytest
import torch

from lossless_bf16_tensor_sign_amd import zc
from tests import ref_ops as ref
from tests.test_gpu_moe import DEV, ROUND, TINY, TYPES, U, check_route, say, some_slots

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("E,groups,top,k", [(512, 2, 1, 8), (1024, 2, 1, 32), (512, 4, 1, 9), (256, 2, 1, 8),
                                            (128, 2, 1, 4), (16, 2, 1, 3), (1024, 8, 3, 12), (6, 2, 1, 3)])
def test_groups_of_many_lanes(group_score, E, groups, top, k):
    # one logit of a token is above the others, at any place of any group: a
    # group's score has to come from all of its lanes
    say("route, groups of", E // groups, group_score)
    rng = np.random.default_rng(E + groups)
    T = 16
    x = rng.integers(-3, 2, size=(T, E)).astype(np.float32)
    at = rng.integers(0, E, size=T)
    at[:4] = [0, E - 1, E // groups - 1, E // groups]
    x[np.arange(T), at] = 2.0
    x = torch.from_numpy(x)
    for score in ("sigmoid", "softmax"):
        e, _ = check_route(x, k, torch.float32, score, groups=groups, top_groups=top, group_score=group_score)
        # (two others may sum to more than it and its second)
        assert group_score == "top2" or np.array_equal(e[:, 0].cpu().numpy(), at)
        check_route(x, k, torch.bfloat16, score, groups=groups, top_groups=top, group_score=group_score, renorm=False)


@pytest.mark.parametrize("pairs", [2047, 2048, 2049, 2561, 4095, 4096, 4097, 4609])
@pytest.mark.parametrize("E", [1, 64, 1000, 1024])
def test_slots_about_one_workgroup(pairs, E):
    # one workgroup up to 4096 pairs, of which it holds 2048 in registers
    say("slots", pairs, E)
    rng = np.random.default_rng(pairs + E)
    e = rng.integers(-1, E + 1, size=pairs)
    s, c = zc.expert_slots(torch.from_numpy(e.astype(np.int32)).to(DEV), E, row_values=520)
    rs, rc = ref.slots(e, E, 520)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(c.cpu().numpy(), rc)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [9, 41, 129, 151, 301, 304, 513])
def test_combine_over_its_base_with_a_shared_last_word(dtype, H):
    # rows that follow one another in a wave, and whose last word begins in
    # its neighbour's: 129, 301 (bf16, f16), 41, 151 (fp32) and more
    T, k = 300, 2
    rng = np.random.default_rng(H)
    sd, _ = some_slots(rng, T, k, 0.1)
    y, base = (torch.randn(n, H, device=DEV).to(dtype) for n in (T * k, T))
    want = zc.combine(y, sd, base=base)
    code = {torch.bfloat16: zc.ZC_BF16, torch.float16: zc.ZC_F16, torch.float32: zc.ZC_F32}[dtype]
    st = zc.ops_lib().zc_combine(zc._ptr(y), code, T, H, zc._ptr(sd), k, None, zc._ptr(base), H, zc._ptr(base),
                                 zc._stream(None))
    assert st == zc.ZC_OK and torch.equal(base, want)


@pytest.mark.parametrize("T", [60, 3000])
def test_graph_replays_of_a_whole_layer(T):
    # 240 pairs (one launch of slots) and 12000 (two)
    E, k, H = 64, 4, 264
    x = torch.empty(T, E, device=DEV)
    h, d = (torch.empty(T, H, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    valid = torch.arange(T, device=DEV) % 11 != 5

    def layer():
        e, w = zc.route(x, k, score="sigmoid", groups=8, top_groups=4, valid=valid)
        s, c = zc.expert_slots(e, E, row_values=H)
        rows = zc.dispatch(h, s)
        out = zc.combine(rows, s, weights=w, base=h)
        d_rows, d_w = zc.combine_grad(d, rows, s, w)
        return (e, w, s, c, rows, out, d_rows, d_w, zc.combine(d_rows, s),
                zc.route_grad(x, e, d_w, score="sigmoid"), zc.route_grad(x, e, d_w, renorm=False))

    def fill(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        for t in (x, h, d):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = layer()
    for r in range(1, 5):
        fill(r)
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, layer())):
            assert torch.equal(a, b), (r, i)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,k,megabytes", [(8, 2, 60), (100, 8, 60), (200, 3, 60), (130, 2, 400), (520, 4, 60),
                                           (520, 1, 400), (1024, 6, 60), (2049, 4, 400), (2049, 2, 60)])
def test_rows_that_stream_past_the_caches(dtype, H, k, megabytes):
    # calls of more than 32 MB load and store past the caches; rows' gradients
    # from 256 MB on
    T = megabytes * 1000000 // (H * k * torch.finfo(dtype).bits // 8) + 3
    say("streamed rows", dtype, T, k, H)
    g = torch.Generator(device=DEV).manual_seed(H + k)
    e = torch.randint(-1, 40, (T, k), generator=g, device=DEV, dtype=torch.int32)
    s, _ = zc.expert_slots(e, 40)
    live = (s >= 0)[..., None]
    x, base, d = (torch.randn(T, H, generator=g, device=DEV).to(dtype) for _ in range(3))
    w = torch.randn(T, k, generator=g, device=DEV)
    rows = zc.dispatch(x, s)
    at = torch.where(s >= 0, s, ~s).long()
    for j in range(k):
        assert torch.equal(rows[at[:, j]], torch.where(live[:, j], x, torch.zeros_like(x)))
    y = torch.randn(T * k, H, generator=g, device=DEV).to(dtype)
    for wt, bs in ((w, base), (None, None)):
        want = torch.zeros(T, H, dtype=torch.float64, device=DEV) if bs is None else bs.double()
        mag = want.abs()
        for j in range(k):
            part = torch.where(live[:, j], y[at[:, j]].double() * (1.0 if wt is None else wt[:, j, None].double()), 0.0)
            want, mag = want + part, mag + part.abs()
        err = (zc.combine(y, s, weights=wt, base=bs).double() - want).abs()
        assert (err <= (k + 2) * U * mag + ROUND[dtype] * want.abs() + TINY[dtype]).all()
    dy, dw = zc.combine_grad(d, y, s, w)
    for j in range(k):
        one = torch.where(live[:, j], d.double() * w[:, j, None].double(), 0.0)
        assert ((dy[at[:, j]].double() - one).abs() <= (U + ROUND[dtype]) * one.abs() + TINY[dtype]).all()
        prod = torch.where(live[:, j], d.double() * y[at[:, j]].double(), 0.0)
        assert ((dw[:, j].double() - prod.sum(1)).abs() <= H * U * prod.abs().sum(1) + 1e-37).all()
