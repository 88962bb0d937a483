"""4-bit operators and the layer's own kernels on one stream, each reading what the one before wrote or
rewriting what it has read. The 4-bit quantisers and few-row products let the next kernel of the stream start
while they still run; every kernel that is launched programmatically has to wait for its predecessor
before it touches memory. Eager, and replayed from a graph: the bytes of the same calls with a
synchronisation after each."""
import pytest
import torch

import tensor_transformer_layer_megatron_b200 as mgt
from mgt_inputs import LayerConfig, make_inputs, pack_params
from tensor_transformer_layer_megatron_b200.runner import LayerRun

pytestmark = pytest.mark.gpu


def quantised(fmt, w):
    q = mgt.Mx4(fmt, *w.shape)
    if fmt == "nvfp4":
        mgt.mx4_tensor_factor(w, q.factor)
    mgt.mx4_quantize(w, q)
    return q


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("hidden,seq,swiglu", [(256, 40, 0), (256, 160, 1), (2048, 40, 1), (2048, 160, 0)])
def test_layer_between_4bit_calls(fmt, hidden, seq, swiglu):
    cfg = LayerConfig("mx4-h%d" % hidden, hidden=hidden, heads=2 * hidden // 256, ffn=2 * hidden, seq=seq, micro_batch=2,
                      tp_size=2, dtype="bf16", seed=4503, swiglu=swiglu)
    t = make_inputs(cfg, nonzero_affine=True)
    rows, h = 2 * seq, hidden
    gen = torch.Generator("cuda").manual_seed(1)
    w = [quantised(fmt, torch.randn(h, h, device="cuda", generator=gen) * h ** -0.5) for _ in range(2)]
    wide = torch.randn(384, h, device="cuda", generator=gen, dtype=torch.float32).bfloat16()

    class State:
        def __init__(self):
            self.run = r = LayerRun(mgt.Layer.from_config(cfg), pack_params(cfg, t), t["x"], t["dy"])
            self.x, self.y, self.dx, self.dy = (v.view(rows, h) for v in (r.x, r.y, r.dx, r.dy))
            self.q, self.qd = mgt.Mx4(fmt, rows, h), mgt.Mx4(fmt, rows, h)
            self.qt = mgt.Mx4(fmt, h, rows, factor=self.q.factor)
            self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
            self.wg = torch.empty(rows, 384, device="cuda")
            self.codes = torch.empty(rows * h, dtype=torch.uint8, device="cuda")
            self.scales = torch.empty(2, device="cuda")

        def calls(self):
            s, r = self, self.run
            factor = (lambda v, q: [lambda: mgt.mx4_tensor_factor(v, q.factor)]) if fmt == "nvfp4" else lambda v, q: []
            return [
                r.fwd,
                *factor(s.y, s.q),
                lambda: mgt.mx4_quantize(s.y, s.q, s.qt),
                lambda: mgt.gemm_mx4(s.q, w[0], s.dy, s.st),  # the layer's backward reads it next
                r.bwd,
                *factor(s.dx, s.qd),
                lambda: mgt.mx4_quantize(s.dx, s.qd),
                lambda: mgt.gemm_bf16(s.dx, wide, s.wg, rows, 384, h, 0, 0, h, h, 384, s.st),
                lambda: mgt.mx4_quantize(s.wg, mgt.Mx4("mxfp4", rows, 384)),
                lambda: mgt.gemm_mx4(s.qd, w[1], s.x, s.st),  # the next forward reads it
                lambda: mgt.fp8_quantize(s.x, s.codes, s.scales),
            ]

        def result(self):
            torch.cuda.synchronize()
            self.run.check()
            assert int(self.st) == 0
            return [v.clone() for v in (self.x, self.y, self.dx, self.dy, self.wg, self.codes, self.q.codes, self.qt.codes,
                                        self.qd.codes, *self.run.grads.values())]

    turns = 3
    a = State()
    for _ in range(turns):
        for call in a.calls():
            call()
            torch.cuda.synchronize()
    want = a.result()
    assert all(torch.isfinite(v).all() for v in want if v.dtype.is_floating_point)

    def same(got):
        return all(torch.equal(g, v) for g, v in zip(got, want))

    for _ in range(3):
        b = State()
        torch.cuda.synchronize()
        for _ in range(turns):
            for call in b.calls():
                call()
        assert same(b.result())
    c = State()
    x0, dy0 = c.x.clone(), c.dy.clone()
    for call in c.calls():
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in c.calls():
            call()
    for _ in range(2):
        c.x.copy_(x0)
        c.dy.copy_(dy0)
        for _ in range(turns):
            graph.replay()
        assert same(c.result())
