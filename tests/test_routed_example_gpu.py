"""The expert-MLP example's router, its gradients and its decoding step, against
64 bits."""
import numpy as np
import pytest
import torch

import routing_plain as plain
from experts_plain import f64
from test_expert_mlp_example_gpu import example, rel  # noqa: F401

pytestmark = pytest.mark.gpu


def test_router_and_decoding_step(example, capsys):  # noqa: F811
    r = example.main(["--tokens", "90", "--experts", "6", "--top", "2", "--width", "136", "--hidden", "72", "--decode", "11"])
    assert "decode, 11" in capsys.readouterr().out
    router = r["router"]
    want, weights = plain.route(f64(router.logits), None, 2)
    assert np.array_equal(router.experts.cpu().numpy(), want)
    for got, ref in zip(router.plan, plain.plan(want, 6)):
        assert np.array_equal(got.cpu().numpy(), ref)
    assert torch.equal(r["rows"], r["x"][r["tokens"]])
    # gradients of the rows and logits, by autograd from the rows' results
    logits = router.logits.double().cpu().requires_grad_()
    out = r["out"].double().cpu().requires_grad_()
    p = logits.gather(1, torch.from_numpy(want).long()).softmax(-1)
    position = router.position.long().cpu()
    (out[position] * p[..., None]).sum(1).backward(r["d_result"].double().cpu())
    assert rel(r["d_out"], out.grad) < 2.0 ** -9         # one rounding to bfloat16, and what FP32 adds to it
    assert rel(r["d_logits"], logits.grad) < 1e-5        # FP32: sums of 136 products, differences of two of them
    # A code is within half a step of a 15th of its group's range; 64 normal values range
    # over some 4.8 of their deviations, so each is off by 0.32 / sqrt(12) = 0.09 of its own.
    # Three products and roundings to bfloat16 on the way: some 0.16 of the result, and not none.
    assert 0.02 < r["off_w4"] < 0.35
