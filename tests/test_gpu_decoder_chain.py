"""The decoder-side operators one after the other with nothing between them, each starting while the one before it ends:
the same bits as with the GPU waited for after every call, call after call on new contents of the same buffers, alone, in a
captured graph and on two streams at once."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from audio_encoder_aut_b200 import _lib as A  # noqa: E402

HQ, HK, HD, D = 4, 2, 64, 256


class Chain:
    """States -> 8-bit key/value projection (weights quantised on the way) -> key norm and rotation in place -> cross
    attention of 8-bit projected, normed, rotated queries."""

    def __init__(self, nq, nk, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.nq, self.nk = nq, nk
        self.x = {"q": torch.empty(nq, D, device="cuda"), "k": torch.empty(nk, D, device="cuda")}
        self.w = {"q": torch.empty(HQ * HD, D, device="cuda"), "k": torch.empty(2 * HK * HD, D, device="cuda")}
        self.codes, self.scales, self.wide = {}, {}, {}
        for side in "qk":
            for name, t in (("x", self.x[side]), ("w", self.w[side])):
                self.codes[name + side] = torch.empty(t.shape, dtype=torch.int8, device="cuda")
                self.scales[name + side] = torch.empty(t.shape[0], device="cuda")
            self.wide[side] = torch.empty(self.x[side].shape[0], self.w[side].shape[0], dtype=torch.bfloat16, device="cuda")
        self.pos = {"q": torch.arange(nq, dtype=torch.int32, device="cuda") + nk, "k": torch.arange(nk, dtype=torch.int32, device="cuda")}
        self.cu_q, self.cu_k = np.array([0, nq], np.int32), np.array([0, nk], np.int32)
        self.ws = torch.empty(A.aut_cross_attention_workspace_bytes(HQ, HK, HD, self.cu_q, self.cu_k), dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out = torch.empty(nq, HQ * HD, dtype=torch.bfloat16, device="cuda")
        self.new_inputs()

    def new_inputs(self):
        for t in (*self.x.values(), *self.w.values()):
            t.normal_(generator=self.g)

    def spoil(self):
        """Nothing of an earlier run is left to be taken for this one's."""
        for t in (*self.codes.values(), self.ws):
            t.fill_(77)
        for t in (*self.scales.values(), *self.wide.values(), self.out):
            t.fill_(float("nan"))

    def run(self, stream=None, wait=False):
        st = torch.cuda.current_stream().cuda_stream if stream is None else stream

        def done(status):
            assert status == A.AUT_OK
            if wait:
                torch.cuda.synchronize()

        for side in "kq":
            for name, t in (("w", self.w[side]), ("x", self.x[side])):
                done(A.aut_quantize_rows(t.data_ptr(), A.F32, D, t.shape[0], D, self.codes[name + side].data_ptr(),
                                         self.scales[name + side].data_ptr(), st))
            y = self.wide[side]
            done(A.aut_linear_i8(self.codes["x" + side].data_ptr(), self.scales["x" + side].data_ptr(), self.codes["w" + side].data_ptr(),
                                 self.scales["w" + side].data_ptr(), None, y.data_ptr(), y.shape[0], y.shape[1], D, A.EPI_BF16,
                                 self.status.data_ptr(), 0, 0, st))
        q, kv = self.wide["q"], self.wide["k"]
        wq, wk = HQ * HD, 2 * HK * HD
        done(A.aut_qk_norm_rope(A.aut_head_rows(q.data_ptr(), wq, q.data_ptr(), wq, None, self.pos["q"].data_ptr(), self.nq, HQ),
                                A.aut_head_rows(kv.data_ptr(), wk, kv.data_ptr(), wk, None, self.pos["k"].data_ptr(), self.nk, HK),
                                HD, A.BF16, A.BF16, HD, 1e4, False, 1e-6, st))
        done(A.aut_cross_attention(q.data_ptr(), wq, kv.data_ptr(), wk, kv.data_ptr() + wk, wk, self.out.data_ptr(), wq, A.BF16, HQ, HK, HD,
                                   self.cu_q, self.cu_k, None, 1 / math.sqrt(HD), self.ws.data_ptr(), self.ws.numel(),
                                   self.status.data_ptr(), 0, st))

    def results(self):
        return [t.clone() for t in (*self.codes.values(), *self.scales.values(), *self.wide.values(), self.out)]

    def wanted(self):
        self.spoil()
        self.run(wait=True)
        assert int(self.status.item()) == 0 and not torch.isnan(self.out).any()
        return self.results()

    def same(self, want):
        assert int(self.status.item()) == 0
        return all(torch.equal(a, b) for a, b in zip(self.results(), want))


SIZES = [(1, 20), (1, 700), (32, 33), (200, 900), (600, 5000)]  # both kernels of the 8-bit layer and of the attention, split keys


@pytest.mark.parametrize("nq,nk", SIZES)
def test_chain_without_waits(nq, nk):
    c = Chain(nq, nk, 1)
    for _ in range(20):
        c.new_inputs()
        want = c.wanted()
        c.spoil()
        c.run()
        assert c.same(want)


@pytest.mark.parametrize("nq,nk", SIZES)
def test_captured_chain_on_new_contents(nq, nk):
    c = Chain(nq, nk, 2)
    c.wanted()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.run()
    for _ in range(20):
        c.new_inputs()
        want = c.wanted()
        c.spoil()
        graph.replay()
        assert c.same(want)


def test_two_chains_at_once():
    """A workspace each, on two streams: every round starts from spoilt buffers."""
    pair = Chain(1, 700, 3), Chain(600, 5000, 4)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        want = []
        for c in pair:
            c.new_inputs()
            want.append(c.wanted())
            c.spoil()
        torch.cuda.synchronize()
        for _ in range(3):
            for c, s in zip(pair, streams):
                c.run(stream=s.cuda_stream)
        torch.cuda.synchronize()
        assert all(c.same(w) for c, w in zip(pair, want))
