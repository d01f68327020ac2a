"""Plans and 4-bit products by several threads, on several streams and in graphs."""
import threading

import numpy as np
import pytest
import torch

import routing_plain as plain
import swiglu_mlp_gb300 as swg
from experts_plain import f64
from test_routing_gpu import check_plan, close, gen, logits_of
from test_w4_gpu import product, weight

pytestmark = pytest.mark.gpu


def in_threads(*fs):
    errors = []

    def guarded(f):
        try:
            f()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    ts = [threading.Thread(target=guarded, args=(f,)) for f in fs]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("shared", [True, False])
def test_threads_with_plans(shared):
    """Calls of two threads, whose counts of chunks share a workspace on one stream."""
    one = torch.cuda.Stream()
    work = []
    for k, (T, E, top) in enumerate(((3000, 64, 4), (700, 100, 6))):
        l = logits_of(T, E, "f32", k)
        want = plain.route(f64(l), None, top)[0]
        outs = [(torch.empty((T, top), dtype=torch.int32, device="cuda"), torch.empty((T, top), device="cuda"),
                 swg.expert_plan_alloc(T, E, top), swg.expert_plan_alloc(T, E, top)) for _ in range(20)]
        work.append((l.cuda(), want, E, outs, one if shared else torch.cuda.Stream()))
    torch.cuda.synchronize()

    def calls(l, want, E, outs, stream):
        for e, w, p, again in outs:
            swg.expert_route_into(e, w, l, plan=p, stream=stream)
            swg.expert_sort_into(again, e, stream=stream)

    in_threads(*(lambda a=a: calls(*a) for a in work))
    torch.cuda.synchronize()
    for l, want, E, outs, stream in work:
        for e, w, p, again in outs:
            assert np.array_equal(e.cpu().numpy(), want)
            check_plan(p, want, E)
            check_plan(again, want, E)
        assert swg.get_device_error(stream) == 0


@pytest.mark.parametrize("M,N,K", [(5, 300, 704), (5, 200, 8200), (40, 200, 6200), (12, 300, 904), (16, 2100, 8704)])
def test_products_in_two_graphs_at_once(M, N, K):
    """Each form of the product captured, and replayed beside another with new rows."""
    W, w = weight(1, N, K, 64, True, "bf16", 3)
    off = np.array([0, M])
    sets = [(torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"), torch.empty((M, N), device="cuda")) for _ in range(2)]
    s = torch.cuda.Stream()
    graphs = []
    for A, C in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            swg.gemm_w4_into(C, A, *(t[0] for t in W), 64, stream=s)
        graphs.append(g)
    for seed in range(3):
        for k, (A, _) in enumerate(sets):
            A.copy_(torch.randn((M, K), generator=gen(10 * seed + k)))
        torch.cuda.synchronize()
        for g in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        assert swg.get_device_error(s) == 0
        for A, C in sets:
            want, tol = product(f64(A), w, off, 1.0, 0.0, np.zeros((M, N)), "f32")
            close(C, want, tol, f"{M} {N} {K}")
