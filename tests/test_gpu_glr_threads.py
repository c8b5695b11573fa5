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
