"""The operators next to the projection run together as a fine-tuning step
uses them: layer norm, the int8 projection, the adapters beside it, their
backward passes, the gradient through the frozen weight, and clipping; eager,
captured in a graph, and on two streams at once.

The reference is the same step in 64 bits (autograd), with the projection as
the product with its recovered weight, whose gradient is what the step asks
for. Every tensor that the step hands from one operator to the next is fp16
(half a step of 2^-11, relative): y, the projection's gradient, dX. A gradient
collects at most four of those, each spread over a sum of independent terms,
so its error stays below 4 * 2^-11 of its norm; 2^-8 leaves a factor of two.
"""
import math

import pytest
import torch

from mixed_precision_int8_b200 import binding as L, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    L.load_library()
    yield


class Layer:
    def __init__(self, s, h, o, n, r, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
        self.s, self.h, self.o, self.n, self.r = s, h, o, n, r
        self.x = rnd(s, h).half()
        self.gamma, self.beta = 1 + 0.1 * rnd(h), 0.1 * rnd(h)
        self.pw = L.llmint8_prepare_weight((rnd(h, o) * 0.02).half())
        self.A, self.B = (rnd(n, r, h) * h ** -0.5).half(), (rnd(n, r, o) * 0.05).half()
        self.scale = 0.5 + torch.rand(n, generator=g, device="cuda")
        self.ad = L.Adapters(self.A, self.B, self.scale)
        self.ids = (torch.arange(s, device="cuda") * (n + 1) // s - 1).to(torch.int32)
        self.dout = (rnd(s, o) * 0.1).half()
        self.mm = L.Workspace(s, h, o)
        self.ws = L.AdapterWorkspace(s, h, o, n, r)
        self.bw = L.BackwardWorkspace(s, h, o)
        self.lw = L.LayerNormWorkspace(s, h)
        self.v = torch.empty(s, r, device="cuda")
        self.grads = [torch.empty(t.shape, device="cuda")
                      for t in (self.A, self.B, self.gamma, self.beta)]
        self.list = L.GradList(self.grads)

    def step(self, max_norm):
        dA, dB, dgamma, dbeta = self.grads
        y, mean, rstd = L.llmint8_layernorm_forward(self.x, self.gamma, self.beta)
        out = L.llmint8_matmul(y, self.pw, 6.0, workspace=self.mm)
        L.llmint8_adapters_forward(y, self.ad, self.ids, base=out, out=out, v=self.v,
                                   workspace=self.ws)
        dy = L.llmint8_matmul_backward(self.dout, self.pw, workspace=self.bw)
        L.llmint8_adapters_backward(y, self.dout, self.ad, self.ids, v=self.v, base=dy, dX=dy,
                                    dA=dA, dB=dB, workspace=self.ws)
        dx, g, b = L.llmint8_layernorm_backward(dy, self.x, self.gamma, mean, rstd,
                                                workspace=self.lw)
        dgamma.copy_(g)
        dbeta.copy_(b)
        return out, dx, L.llmint8_clip_grads(self.list, max_norm)

    def reference(self):
        d = torch.float64
        x, gamma, beta, A, B = (t.to(d).requires_grad_() for t in
                                (self.x, self.gamma, self.beta, self.A, self.B))
        m = x.mean(1, keepdim=True)
        y = (x - m) / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + 1e-5) * gamma + beta
        WR = (self.pw.wq.to(d) * self.pw.aw.to(d)[:, None] / 127).T
        out = y @ WR
        for a in range(self.n):
            rows = (self.ids == a).to(d)[:, None]
            out = out + rows * float(self.scale[a]) * (y @ A[a].T @ B[a])
        out.backward(self.dout.to(d))
        return out.detach(), x.grad, [A.grad, B.grad, gamma.grad, beta.grad]


def near(got, ref, bound):
    assert float((got.double() - ref).norm() / ref.norm()) < bound


@pytest.mark.parametrize("s,h,o,n,r", [(9, 272, 528, 2, 8), (300, 1040, 784, 3, 16),
                                       (700, 528, 2064, 2, 64)])
def test_step(s, h, o, n, r):
    layer = Layer(s, h, o, n, r)
    ref_out, ref_dx, ref = layer.reference()
    out, dx, norm = layer.step(float("inf"))
    # the forward product is quantised: a step of 1/254 of a row's and of a
    # column's largest value per factor, of values a third of that
    near(out, ref_out, 2.0 ** -5)
    near(dx, ref_dx, 2.0 ** -8)
    for got, want in zip(layer.grads, ref):
        near(got, want, 2.0 ** -8)
    want = math.sqrt(sum(float((g.double() ** 2).sum()) for g in layer.grads))
    assert abs(float(norm) / want - 1) < 2.0 ** -22
    before = [g.clone() for g in layer.grads]
    _, _, norm = layer.step(want / 2)
    assert abs(float(norm) / want - 1) < 2.0 ** -22
    for got, g in zip(layer.grads, before):
        # the coefficient's rounding and the product's
        assert ((got - g / 2).abs() <= 2.0 ** -22 * g.abs()).all()
    for ws in (layer.mm, layer.ws, layer.bw, layer.lw):
        assert L.llmint8_read_device_status(ws) == 0


def test_step_in_a_graph_and_on_two_streams_at_once():
    layers = [Layer(300, 1040, 784, 3, 16, seed=1), Layer(200, 528, 2064, 2, 64, seed=2)]
    want = []
    for layer in layers:
        want.append([t.clone() for t in layer.step(1.0)] + [g.clone() for g in layer.grads])
    torch.cuda.synchronize()
    # two layers with workspaces of their own, on two streams, again and again
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(10):
        got = []
        for layer, stream in zip(layers, streams):
            with torch.cuda.stream(stream):
                got.append(layer.step(1.0))
        torch.cuda.synchronize()
        for layer, res, ref in zip(layers, got, want):
            for a, b in zip(list(res) + layer.grads, ref):
                assert torch.equal(a, b)
    # one layer captured twice: the graphs share its workspaces, one after
    # another, with eager steps between them
    layer, ref = layers[0], want[0]
    graphs, held = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(layer.step(1.0))
        graphs.append(graph)
    for k in (0, 1, 1, 0):
        graphs[k].replay()
        for a, b in zip(list(held[k]) + layer.grads, ref):
            assert torch.equal(a, b)
        for a, b in zip(list(layer.step(1.0)) + layer.grads, ref):
            assert torch.equal(a, b)
