"""The library's calls from several host threads at once, and after a call
whose launch was refused."""
import ctypes
import threading

import pytest
import torch

from helpers import need_gpu

pytestmark = pytest.mark.gpu


def in_threads(*works):
    """Runs the functions at once, one thread and one stream each (the
    stream's handle is their argument); what they raised comes back."""
    streams = [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()
    gate, raised = threading.Barrier(len(works)), []

    def one(work, stream):
        try:
            torch.cuda.set_device(0)
            gate.wait()
            work(stream.cuda_stream)
        except Exception as e:      # noqa: BLE001 - handed to the test's thread
            raised.append(e)

    threads = [threading.Thread(target=one, args=a) for a in zip(works, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return raised


def accepted(sdm, code):
    if code != sdm.SDM_OK:
        raise AssertionError(sdm.lib().sdm_last_error().decode())


class Forward:
    """A glr_scan call on buffers of its own."""

    def __init__(self, sdm, T, D, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.sdm, self.T, self.D = sdm, T, D
        self.h0, self.x, self.r, self.g = n(1, D), n(1, T, D), n(1, T, D), n(1, T, D)
        self.rate = torch.rand(D, generator=gen, device="cuda")
        self.y, self.hT = torch.empty_like(self.x), torch.empty_like(self.h0)
        self.want = sdm.glr_scan(self.h0, self.x, self.r, self.g, self.rate, state_out=torch.empty_like(self.h0))

    def call(self, stream):
        p = [t.data_ptr() for t in (self.h0, self.hT, self.x, self.r, self.g, self.rate, self.y)]
        return self.sdm.lib().glr_scan(p[0], p[1], p[2], self.D, p[3], self.D, p[4], self.D, self.sdm.SDM_DTYPE_F32, p[5],
                                       None, None, 1, self.T, self.D, p[6], None, stream)

    def right(self):
        return torch.equal(self.y, self.want)


class Backward(Forward):
    def __init__(self, sdm, T, D, seed):
        super().__init__(sdm, T, D, seed)
        _, self.carry = sdm.glr_scan_train(self.h0, self.x, self.r, self.g, self.rate, state_out=self.hT)
        self.dy = self.y.normal_()
        self.grads = [torch.empty_like(self.x) for _ in range(3)]
        self.drate = torch.empty_like(self.rate)
        self.want = sdm.glr_scan_backward(self.h0, self.x, self.r, self.g, self.rate, self.carry, self.dy,
                                          dstate_out=self.hT)

    def call(self, stream):
        D = self.D
        p = [t.data_ptr() for t in (self.h0, self.hT, self.x, self.r, self.g, self.rate, self.carry, self.dy, *self.grads,
                                    self.drate)]
        return self.sdm.lib().glr_scan_backward(p[0], p[1], p[2], D, p[3], D, p[4], D, None, None, self.sdm.SDM_DTYPE_F32,
                                                p[5], None, None, p[6], p[7], 1, self.T, D, p[8], p[9], p[10], D, p[11],
                                                None, 0, None, stream)

    def right(self):
        return all(torch.equal(a, b) for a, b in zip((*self.grads, self.drate), self.want))


@pytest.mark.parametrize("kind,lengths,n", [(Forward, (40, 513, 300), 4000), (Backward, (4099, 5000), 1500)],
                         ids=["forward", "backward"])
def test_threads_with_calls_of_other_lengths(kind, lengths, n):
    """fp32 sequences of one channel block: their lengths are split over clusters
    of different sizes, so the calls want different amounts of shared memory."""
    sdm = need_gpu()
    calls = [kind(sdm, T, 64, i) for i, T in enumerate(lengths)]

    def work(c):
        def run(stream):
            for _ in range(n):
                accepted(sdm, c.call(stream))
        return run

    assert not in_threads(*(work(c) for c in calls))
    assert all(c.right() for c in calls)


def test_a_refused_launch_is_not_the_next_call_s_error():
    """A launch into a stream whose capture was invalidated is refused by CUDA; the
    call says so, and the one after it is judged by its own launch."""
    sdm = need_gpu()
    c = Forward(sdm, 40, 64, 7)
    torch.cuda.synchronize()
    rt = ctypes.CDLL("libcudart.so.13")
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(stream), 1) == 0
    assert rt.cudaStreamBeginCapture(stream, 1) == 0        # thread-local mode
    assert rt.cudaStreamSynchronize(stream) != 0            # not allowed in a capture, which ends as invalid
    refused = c.call(stream)
    assert rt.cudaStreamEndCapture(stream, ctypes.byref(graph)) != 0
    assert rt.cudaStreamDestroy(stream) == 0
    rt.cudaGetLastError()                                   # this test's own errors
    assert refused == sdm.SDM_ERR_CUDA
    accepted(sdm, c.call(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert c.right()


class SparseScan:
    """An sdm_scan call on buffers of its own, B H sequences of two tokens."""

    def __init__(self, sdm, B, H, seed, N=64, T=2, W=4, dv=64):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.rand(s, generator=gen, device="cuda")  # noqa: E731
        idx = [n(B, T, H, N).argsort(-1)[..., :W].to(torch.int32).contiguous() for _ in range(2)]
        w = [n(B, T, H, W) / W for _ in range(2)]
        self.sdm, self.sizes = sdm, (B, T, H, N, dv)
        self.args = (n(B, T, H, dv), n(B, T, H), n(B, T, H), idx[0], w[0], idx[1], w[1])
        self.start = n(B, H, N, dv)
        self.state, self.want_state = self.start.clone(), self.start.clone()
        self.want = sdm.sdm_scan(self.want_state, *self.args)
        self.y = torch.empty_like(self.want)
        self.ws = torch.empty(sdm.sdm_scan_workspace_size(B, T, H, W, W), dtype=torch.uint8, device="cuda")

    def call(self, stream):
        v, al, be, iw, ww, ir, wr = (t.data_ptr() for t in self.args)
        W = self.args[3].shape[-1]
        return self.sdm.lib().sdm_scan(self.state.data_ptr(), v, self.sdm.SDM_DTYPE_F32, al, be, iw, ww, W, ir, wr, W,
                                       *self.sizes, self.sdm.SDM_RESID_SHARED, self.y.data_ptr(), self.ws.data_ptr(),
                                       self.ws.numel(), None, stream)

    def right(self):
        self.state.copy_(self.start)        # the loops went on with the state
        accepted(self.sdm, self.call(torch.cuda.current_stream().cuda_stream))
        return torch.equal(self.y, self.want) and torch.equal(self.state, self.want_state)


class SseScan(SparseScan):
    """An sse_scan call, token by token, N + 1 partitions in shared memory."""

    def __init__(self, sdm, N, seed, B=1, T=3, H=2, c=128, d=32, topk=2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.rand(s, generator=gen, device="cuda")  # noqa: E731
        self.sdm, self.sizes, self.topk = sdm, (B, T, H, N, c, d), topk
        self.args = (n(B, T, H, N), n(B, T, H, c), n(B, T, H, c).bfloat16(), n(B, T, H, d).bfloat16(), n(B, T, H, c))
        self.start = n(B, H, N + 1, c, d)
        self.state, self.want_state = self.start.clone(), self.start.clone()
        self.want = sdm.sse_scan(self.want_state, self.args[0], topk, *self.args[1:])
        self.y = torch.empty_like(self.want)
        self.ws = torch.empty(sdm.sse_scan_workspace_size(B, T, H, N, topk, c, d), dtype=torch.uint8, device="cuda")

    def call(self, stream):
        logits, k, q, v, al = (t.data_ptr() for t in self.args)
        return self.sdm.lib().sse_scan(self.state.data_ptr(), logits, self.topk, k, q, v, al, self.sdm.SSE_WRITE_ADDITIVE,
                                       *self.sizes, self.y.data_ptr(), None, self.ws.data_ptr(), self.ws.numel(), None,
                                       stream)


@pytest.mark.parametrize("kind,a,b", [(SparseScan, (8, 16), (10, 20)), (SseScan, (4,), (12,))], ids=["sdm", "sse"])
def test_threads_with_scans_of_other_sizes(kind, a, b):
    """sdm_scan with 128 and 200 (batch, head) pairs: 512 and 800 warps, which fit
    the GPU at once with four and with two of them a CTA.  sse_scan with
    tables of 5 and 13 partitions.  (Between setting a limit of the call's own
    and the launch there are few instructions: one call in 48,000 was refused.)"""
    sdm = need_gpu()
    calls = [kind(sdm, *(b if i % 2 else a), i) for i in range(6)]

    def work(c):
        def run(stream):
            for i in range(8000):
                if i % 200 == 0:        # no thread waits long for room in its stream's queue
                    torch.cuda.ExternalStream(stream).synchronize()
                accepted(sdm, c.call(stream))
        return run

    assert not in_threads(*(work(c) for c in calls))
    assert all(c.right() for c in calls)
