"""Split contractions keep FP32 partials in a workspace between the kernel that
writes them and the one that adds them up.  No other call may get between the
two, whoever makes it: every result equals, bit for bit, the same call's alone."""
import sys
import threading

import pytest
import torch

import swiglu_mlp_gb300 as swg
import synth

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def empty(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="cuda")


class Calls:
    """One of each kind of call that splits its contraction, on its own data
    (``fixed``: gemm_splitk_noalloc too, whose array all streams share)."""

    def __init__(self, seed, fixed=False):
        g = synth.generator(seed)
        self.fixed = fixed
        self.off = torch.tensor([0, 2, 2, 5], dtype=torch.int32).cuda()
        self.A, self.B = synth.normal((5, 4096), g).cuda(), synth.normal((3, 4096, 264), g, 0.02).cuda()
        self.long = torch.tensor([0, 6000 + seed % 7], dtype=torch.int32).cuda()
        self.X, self.D = synth.normal((6016, 72), g).cuda(), synth.normal((6016, 136), g, 0.1).cuda()
        self.Q, self.S = swg.mx4_alloc(5, 8192, swg.MXFP4)
        self.W, self.SW = swg.mx4_alloc(264, 8192, swg.MXFP4)
        swg.mx4_quantize_into(self.Q, self.S, synth.normal((5, 8192), g).cuda(), swg.MXFP4)
        swg.mx4_quantize_into(self.W, self.SW, synth.normal((264, 8192), g, 0.02).cuda(), swg.MXFP4)
        self.outs = [empty(5, 264), empty(1, 72, 136, dtype=torch.float32)] + [empty(5, 264) for _ in range(2 + fixed)]
        torch.cuda.synchronize()

    def run(self, stream=None):
        o = self.outs
        swg.gemm_grouped_into(o[0], self.A, self.B, self.off, stream=stream)
        swg.gemm_grouped_wgrad_into(o[1], self.X, self.D, self.long, stream=stream)
        swg.gemm_mx4_into(o[2], self.Q, self.S, self.W, self.SW, 8192, swg.MXFP4, stream=stream)
        args = (0, 0, 5, 264, 4096, 1.0, self.A, 4096, self.B, 264, 0.0)
        swg.gemm_ex(*args, o[3], 264, swg.BF16, 9, stream=stream)
        if self.fixed:
            swg.gemm_splitk_noalloc(*args, o[4], 264, swg.BF16, 9, stream=stream)

    def launches(self):
        before = swg.launch_count()
        self.run()
        return swg.launch_count() - before

    def alone(self):
        self.run()
        torch.cuda.synchronize()
        self.want = [t.clone() for t in self.outs]
        self.bad = torch.zeros(len(self.outs), dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()

    def compare(self):
        """Counts differing results on the current stream, and spoils them."""
        for i, (t, w) in enumerate(zip(self.outs, self.want)):
            self.bad[i] += (t != w).sum()
            t.fill_(-1.0)


def in_threads(works):
    """Runs them at once, the interpreter changing threads as often as it can."""
    errors, old = [], sys.getswitchinterval()

    def guarded(f):
        try:
            f()
        except Exception as e:          # raised on the main thread below
            errors.append(repr(e))

    threads = [threading.Thread(target=guarded, args=(f,)) for f in works]
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join(timeout=120)
    finally:
        sys.setswitchinterval(old)
    assert not errors and not any(t.is_alive() for t in threads), errors


def test_every_call_here_splits():
    c = Calls(1, fixed=True)
    assert c.launches() == 10            # a product and a sum each


def test_threads_sharing_one_stream():
    calls = [Calls(10 + i, fixed=True) for i in range(4)]
    for c in calls:
        c.alone()
    s = torch.cuda.Stream()

    def work(c):
        def f():
            with torch.cuda.stream(s):
                for _ in range(60):
                    c.run()
                    c.compare()
        return f

    in_threads([work(c) for c in calls])
    torch.cuda.synchronize()
    assert swg.get_device_error() == 0
    assert [c.bad.tolist() for c in calls] == [[0] * 5] * 4


def test_default_stream_of_each_thread():
    """cudaStreamPerThread: one handle, in every thread another stream."""
    per_thread = 2
    calls = [Calls(20 + i) for i in range(4)]
    for c in calls:
        c.alone()
    first = threading.Barrier(len(calls))
    bad = [0] * len(calls)

    def work(i):
        def f():
            c = calls[i]
            c.run(per_thread)
            first.wait(60)
            for _ in range(40):
                for _ in range(5):
                    c.run(per_thread)
                assert swg.get_device_error(per_thread) == 0     # synchronises this thread's
                bad[i] += sum(not torch.equal(t, w) for t, w in zip(c.outs, c.want))
        return f

    in_threads([work(i) for i in range(len(calls))])
    assert bad == [0] * len(calls)


def captured(c, s):
    with torch.cuda.stream(s):
        c.run()                                  # the first run on a stream is not captured
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.run()
    return graph


def test_graphs_of_one_stream_run_at_once():
    """Two graphs captured on one stream, replayed on two others while that
    stream runs calls of its own."""
    calls = [Calls(30 + i) for i in range(3)]
    for c in calls:
        c.alone()
    s = torch.cuda.Stream()
    runs = [captured(c, s).replay for c in calls[:2]] + [calls[2].run]
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), s]
    torch.cuda.synchronize()
    for _ in range(100):
        for c, run, t in zip(calls, runs, streams):
            with torch.cuda.stream(t):
                run()
                c.compare()
    torch.cuda.synchronize()
    assert swg.get_device_error() == 0
    assert [c.bad.tolist() for c in calls] == [[0] * 4] * 3


def test_destroyed_graphs_leave_their_buffers_to_others():
    c = Calls(40)
    s = torch.cuda.Stream()
    captured(c, s).reset()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(400):
        graph = captured(c, s)
        graph.replay()
        s.synchronize()
        graph.reset()
    torch.cuda.synchronize()
    # 140 MB (0.35 MB of partials for each graph), if none were reused
    assert free - torch.cuda.mem_get_info()[0] < 16 << 20
    assert swg.get_device_error() == 0


def test_graphs_that_outlive_a_shutdown():
    """swg_shutdown frees what graphs held; destroying them later is harmless,
    and later captures get buffers of their own."""
    c = Calls(41)
    c.alone()
    s = torch.cuda.Stream()
    old = captured(c, s)
    torch.cuda.synchronize()
    swg.shutdown()
    new = captured(c, s)
    old.reset()
    for t in c.outs:
        t.zero_()
    torch.cuda.synchronize()
    new.replay()
    torch.cuda.synchronize()
    assert swg.get_device_error() == 0
    assert all(torch.equal(t, w) for t, w in zip(c.outs, c.want))
