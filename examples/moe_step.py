"""Training steps of one MoE layer around the codec, on one GPU.

Two data-parallel ranks are played in turn.  On each, the router picks every
token's experts, the token rows go into per-expert chunks, the chunks are
compressed and decoded (the all-to-all would carry the streams), the experts
work on them, and their rows go back the same way and are joined.  The
backward pass runs the gradients of those calls.  The ranks' bf16 gradients
are then compressed, decoded and summed (the reduce-scatter's receiving
side), clipped by their norm and stepped by AdamW on fp32 masters, and the
new bf16 parameters go through the codec once more (the all-gather).

The layer learns the map of a fixed random layer of the same form; the loss
falls from step to step.

  python examples/moe_step.py [--steps N] [--tokens T] [--hidden H]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lossless_bf16_tensor_sign_amd import zc  # noqa: E402

DEV = "cuda:0"
ROUTER = dict(score="sigmoid", renorm=True, scale=1.0)


class Layer:
    """Router [H, E] and expert matrices [E, H, H] as views of one flat bf16
    buffer, the form in which parameters are gathered."""

    def __init__(self, hidden, experts, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.E, self.H = experts, hidden
        n = hidden * experts + experts * hidden * hidden
        self.flat = (torch.randn(n, generator=g, device=DEV) * hidden ** -0.5).to(torch.bfloat16)

    def views(self, flat):
        r = self.H * self.E
        return flat[:r].view(self.H, self.E), flat[r:].view(self.E, self.H, self.H)


def through_codec(rows, counts):
    """rows as they arrive after an all-to-all of compressed chunks."""
    buf, _, offsets = zc.compress_dev(rows.view(torch.int16).view(-1), counts)
    y, _ = zc.decompress_dev(buf, counts, rows.numel(), d_in_offsets=offsets)
    return y.view(torch.bfloat16).view_as(rows)


def per_expert(rows, mats, ends, transpose=False):
    """Each expert's matrix on its chunk of rows."""
    out = torch.zeros_like(rows)
    for e, m in enumerate(mats):
        a, b = ends[e], ends[e + 1]
        if b > a:
            out[a:b] = rows[a:b] @ (m.t() if transpose else m)
    return out


def forward(layer, x, k, valid, bias):
    router, mats = layer.views(layer.flat)
    logits = x @ router
    experts, weights = zc.route(logits, k, bias=bias, valid=valid, **ROUTER)
    slots, counts = zc.expert_slots(experts, layer.E, row_values=layer.H)
    ends = [0] + np.cumsum(counts.cpu().numpy()[:-1] // layer.H).tolist()    # for the experts' plain products
    sent = through_codec(zc.dispatch(x, slots), counts)
    back = through_codec(per_expert(sent, mats, ends), counts)
    out = zc.combine(back, slots, weights=weights, base=x)
    return out, dict(x=x, logits=logits, experts=experts, weights=weights, slots=slots, ends=ends, sent=sent, back=back)


def backward(layer, s, d_out):
    """Gradient of the flat parameters (bf16), for d_out."""
    _, mats = layer.views(layer.flat)
    flat = torch.empty_like(layer.flat)
    d_router, d_mats = layer.views(flat)
    d_back, d_weights = zc.combine_grad(d_out, s["back"], s["slots"], s["weights"])
    for e in range(layer.E):
        a, b = s["ends"][e], s["ends"][e + 1]
        d_mats[e] = s["sent"][a:b].t() @ d_back[a:b]
    d_logits = zc.route_grad(s["logits"], s["experts"], d_weights, **ROUTER)
    d_router.copy_(s["x"].t() @ d_logits)
    # what a layer below would get: the shared path, the dispatched rows' and the router's
    d_x = zc.combine(per_expert(d_back, mats, s["ends"], transpose=True), s["slots"], base=d_out)
    d_x += d_logits @ layer.views(layer.flat)[0].t()
    return flat, d_x


def train(steps=8, tokens=512, hidden=128, experts=8, k=2, ranks=2, eight_bit=True, say=print):
    """Losses of the steps."""
    teacher, layer = Layer(hidden, experts, seed=1), Layer(hidden, experts, seed=2)
    n = layer.flat.numel()
    master = layer.flat.float()
    grad = torch.empty(n, device=DEV)
    if eight_bit:
        state = [torch.zeros(n, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.zeros(-(-n // zc.ZC_STATE_BLOCK), device=DEV) for _ in range(2)]
        kw = dict(avg_scales=[scales[0]], sq_scales=[scales[1]])
    else:
        state, kw = [torch.zeros(n, device=DEV) for _ in range(2)], {}
    opt = zc.AdamWTensors([layer.flat], [grad], [state[0]], [state[1]], masters=[master], **kw)
    grads = zc.TensorList([grad])                # made once: every step's sum is decoded into grad
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    need = zc.zc_reduce_scratch_bytes(n, ranks)
    scratch = torch.empty(need, dtype=torch.uint8, device=DEV) if need else None
    bias = torch.zeros(experts, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    xs = [torch.randn(tokens, hidden, generator=g, device=DEV).to(torch.bfloat16) for _ in range(ranks)]
    valid = torch.arange(tokens, device=DEV) < tokens - tokens // 16          # the batch ends in padding
    targets = [forward(teacher, x, k, valid, bias)[0] for x in xs]
    losses = []
    for step in range(1, steps + 1):
        loss, parts, load = 0.0, [], torch.zeros(experts, device=DEV)
        for x, want in zip(xs, targets):
            out, saved = forward(layer, x, k, valid, bias)
            diff = out.float() - want.float()
            loss += float(diff.square().mean()) / ranks
            flat, _ = backward(layer, saved, (diff * (2.0 / diff.numel() / ranks)).to(torch.bfloat16))
            parts.append(flat)
            load += torch.bincount(saved["experts"][valid].flatten().long(), minlength=experts)
        # reduce-scatter: compressed per rank, decoded and summed
        buf, _ = zc.compress(torch.cat(parts).view(torch.int16), np.full(ranks, n, np.int64))
        assert zc.zc_decompress_reduce(buf, n, ranks, grad, status, scratch) == zc.ZC_OK
        clip = zc.grad_norm(grads, max_norm=1.0)
        zc.adamw(opt, step=step, lr=2e-3, betas=(0.9, 0.95), weight_decay=0.0, grad_scale=clip[1:])
        # all-gather: the parameters as the other ranks receive them
        stream, sizes = zc.compress(layer.flat.view(torch.int16), [n])
        got, _ = zc.decompress(stream, [n])
        assert torch.equal(got.view(torch.bfloat16), layer.flat) and not status.any()
        bias += 1e-3 * torch.sign(load.mean() - load)                         # balance
        losses.append(loss)
        say("step %d  loss %.5f  gradient norm %.4f  parameters %.2f bits per value"
            % (step, loss, float(clip[0]), 8.0 * int(sizes[0]) / n))
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=128)
    a = ap.parse_args()
    train(a.steps, a.tokens, a.hidden)
