"""The serving operators have no backward pass: with autograd on, a tensor that requires grad is refused by name
instead of giving a result that is cut off from it (CPU, no GPU call: the refusal comes before the device check)."""
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_engram_amd as eg  # noqa: E402

BF = torch.bfloat16
LINEAR = (eg.engram_linear, eg.make_linear_layout(64, 40),
          dict(x=torch.zeros((3, 64), dtype=BF), w=torch.zeros((40, 64), dtype=BF), bias=torch.zeros(40),
               residual=torch.zeros((3, 40), dtype=BF), out=torch.zeros((3, 40), dtype=BF)))
NORM = (eg.engram_residual_norm, eg.make_norm_layout(2, 64, gate=eg.GATE_TOKEN),
        dict(x=torch.zeros((1, 3, 2, 64), dtype=BF), y=torch.zeros((1, 3, 2, 64), dtype=BF), gate=torch.zeros((1, 3, 2)),
             post_weight=torch.zeros((2, 64)), pre_weight=torch.zeros((2, 64)), out=torch.zeros((1, 3, 2, 64), dtype=BF),
             h=torch.zeros((1, 3, 2, 64), dtype=BF)))


@pytest.mark.parametrize("call,layout,args,name", [(*op, k) for op in (LINEAR, NORM) for k in op[2]])
def test_tensors_that_require_grad_are_refused(call, layout, args, name):
    args = args | {name: args[name].clone().requires_grad_()}
    with pytest.raises(ValueError, match=f"^{name} requires grad"):
        call(layout, **args)
    for off in (torch.no_grad, torch.inference_mode):  # without autograd it is an ordinary call
        with off(), pytest.raises(ValueError, match="must be on a GPU"):
            call(layout, **args)


def test_results_of_other_operations_are_refused_too():
    w = torch.zeros((40, 64), dtype=BF, requires_grad=True)
    with pytest.raises(ValueError, match="^w requires grad"):
        eg.engram_linear(LINEAR[1], LINEAR[2]["x"], w * 2)
    with pytest.raises(ValueError, match="must be on a GPU"):
        eg.engram_linear(LINEAR[1], LINEAR[2]["x"], (w * 2).detach())
