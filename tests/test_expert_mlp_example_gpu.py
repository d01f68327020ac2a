"""The expert-MLP example at a small size against autograd in 64 bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_mlp", os.path.join(ROOT, "examples", "expert_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_example(example, fmt, capsys):
    r = example.main(["--tokens", "150", "--experts", "5", "--top", "2", "--width", "200", "--hidden", "136",
                      "--format", fmt])
    assert "backward" in capsys.readouterr().out
    mlp, off = r["mlp"], r["offsets"].tolist()
    assert off[0] == 0 and off[-1] == 300
    rows = r["rows"].double().cpu().requires_grad_()
    w, wd = (t.double().cpu().requires_grad_() for t in (mlp.w_fused, mlp.w_down))
    outs = []
    for e in range(5):
        h = rows[off[e]:off[e + 1]] @ w[e]
        outs.append((torch.nn.functional.silu(h[:, 0::2]) * h[:, 1::2]) @ wd[e])
    out = torch.cat(outs)
    out.backward(r["d_out"].double().cpu())
    want = torch.zeros(150, 200, dtype=torch.float64).index_add_(
        0, r["tokens"].cpu(), out.detach() * r["weights"].double().cpu()[:, None])
    # two bf16 roundings forward, three backward: 2^-9 of the norm each, and as
    # much again for their growth through the products
    assert rel(r["result"], want) < 4 * 2.0 ** -9
    for got, ref in zip(r["grads"], (rows.grad, w.grad, wd.grad)):
        assert rel(got, ref) < 6 * 2.0 ** -9
    # An E2M1 value is within 1/4 of itself (1/6 on the average of its steps) of
    # what it stands for, mostly much less: rows and weights of two products
    # keep the result well within half its norm, and it is not the 16-bit one.
    assert 0.01 < r["off"] < 0.5
