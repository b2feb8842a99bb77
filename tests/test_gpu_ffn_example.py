"""The example's feed-forward layers: each stage against float64 on what the stage
before it gave, whole layers twice, and whole layers captured into graphs."""

import importlib.util
import os

import pytest
import torch

from gpu_util import say
from oracle import ffn

pytestmark = pytest.mark.gpu


def load_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def inputs(T, hidden):
    g = torch.Generator(device="cuda").manual_seed(T)
    return [torch.randn(T, hidden, generator=g, device="cuda").bfloat16() for _ in range(2)]


def real(codes, scale):
    """E4M3 codes and row scales as float64."""
    return codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]


def near(got, want, steps):
    """Within `steps` half steps of bf16 of the whole array's size, and 2^-12 for sums in fp32."""
    got, want = got.double(), want.double()
    assert torch.isfinite(got).all()
    assert (got - want).norm() <= (steps * 2.0 ** -8 + 2.0 ** -12) * want.norm()


@pytest.mark.parametrize("T", [1, 40, 700])
def test_dense_layer(gpu_lib, T):
    layer = load_example().FeedForward(hidden=512, inner=1376)
    x, residual = inputs(T, 512)
    say("dense", T)
    y = layer(x, residual)
    n = gpu_lib.add_rms_norm_quantize(x, layer.norm, residual)
    s = n.sum.double()
    near(s, x.double() + residual.double(), 1)
    z = real(n.q, n.scale) @ real(*layer.w_in).T
    gate, up = z.chunk(2, 1)
    h = gpu_lib.fp8_gemm_fused(T, 1376, 512, n.q, layer.w_in[0], n.scale, layer.w_in[1], act="silu", gated=True)
    near(h, torch.nn.functional.silu(gate) * up, 1)
    q, scale = gpu_lib.fp8_quantize_ex(h)
    near(y, real(q, scale) @ real(*layer.w_out).T + s, 1)
    assert torch.equal(y, layer(x, residual))


@pytest.mark.parametrize("T,groups", [(1, 1), (30, 1), (30, 4), (600, 4)])
def test_experts_layer(gpu_lib, T, groups):
    layer = load_example().Experts(hidden=512, inner=288, experts=16, top_k=3, groups=groups)
    x, residual = inputs(T, 512)
    say("experts", T, groups)
    y = layer(x, residual)
    n = gpu_lib.add_rms_norm_quantize(x, layer.norm, residual, return_norm=True)
    r = layer.route(n.norm)
    logits = (n.norm.float() @ layer.router.T).cpu().numpy()
    ids, weights, *_ = ffn.route(logits, 3, bias=layer.bias.cpu().numpy(), score="sigmoid", groups=groups,
                                     top_groups=max(1, groups // 2), group_top=2 if groups > 1 else 1)
    assert (r.ids.cpu().numpy() == ids).all()
    h, e = layer.experts_of(n, r)
    a, b, c = real(n.q, n.scale), real(*layer.w_in), real(*layer.w_out)
    q, scale = gpu_lib.fp8_quantize_ex(h)
    back = real(q, scale)
    want = n.sum.double()
    for j in range(3):
        id, slot = r.ids[:, j].long(), r.slots[:, j].long()
        assert (r.rows[slot].long() == torch.arange(T, device="cuda")).all()
        z = (b[id] @ a[:, :, None]).squeeze(2)
        gate, up = z.chunk(2, 1)
        near(h[slot], torch.nn.functional.silu(gate) * up, 1)
        near(e[slot], (c[id] @ back[slot][:, :, None]).squeeze(2), 1)
        want = want + r.weights[:, j, None].double() * e[slot].double()
    near(y, want, 1)
    assert torch.equal(y, layer(x, residual))


@pytest.mark.parametrize("T", [3, 90])
def test_captured_layers(gpu_lib, T):
    """Both layers in one graph beside a second graph of their own; every replay, on new
    rows, is the eager result, with eager work in between."""
    example = load_example()
    dense, experts = example.FeedForward(hidden=512, inner=1376), example.Experts(hidden=512, inner=288, experts=16, top_k=3, groups=4)

    def path(x, residual):
        y = dense(x, residual)
        return y, experts(y, x)

    x, residual = inputs(T, 512)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        path(x, residual)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(path(x, residual))
        graphs.append(g)
    for rep in range(4):
        a, b = inputs(T + 100 * rep, 512)
        x.copy_(a[:T]), residual.copy_(b[:T])
        say("replay", T, rep)
        eager = [t.clone() for t in path(x, residual)]
        torch.cuda.synchronize()
        for g, out in zip(graphs, outs):
            g.replay()
            torch.cuda.synchronize()
            for t, e in zip(out, eager):
                assert torch.equal(t, e), rep
