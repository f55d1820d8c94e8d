"""The operators of a training step together, as a user's loop runs them, against float64's automatic gradients."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

BF16 = torch.bfloat16
U = torch.finfo(BF16).eps / 2


@pytest.fixture(scope="module")
def example():
    import train_head

    return train_head


def step64(step):
    """Loss and gradients of the step's present weights by torch.autograd in float64.  The kernels round y and d_hidden to
    bf16 on the way, which is not done here."""
    x, r = step.x.double().requires_grad_(), step.stream.double()
    gamma, head = step.gamma.double().requires_grad_(), step.head.double().requires_grad_()
    z = x + r
    y = z / (z.square().mean(1, keepdim=True) + 1e-6).sqrt() * gamma
    seen = step.labels >= 0
    loss = torch.nn.functional.cross_entropy((y @ head.T)[seen], step.labels[seen].long(), reduction="none")
    total = (loss * step.weight.double()[seen]).sum()
    total.backward()
    return total.detach(), x.grad, gamma.grad, head.grad


@pytest.mark.parametrize("N,H,V", [(256, 512, 4096), (300, 264, 1001)])
def test_gradients_of_a_step(example, N, H, V):
    step = example.HeadTrainer(N, H, V, max_norm=1e9)
    total, dx, dgamma, dhead = step64(step)
    loss, norm = step()
    # y is rounded to bf16 (U of each, up or down as often): logits are off by about U / sqrt(H) of their terms' sum
    assert abs(float(loss) - float(total)) <= 1e-3 * float(total)
    for got, want in ((step.norm_grad.outputs["dx"], dx), (step.gradients["gamma"], dgamma), (step.gradients["head"], dhead)):
        # up to four roundings to bf16 in a row (y, dz, d_hidden, dx), each under U / 2 in the 2-norm
        assert (got.double() - want).norm() <= 2 * U * want.norm()
    assert abs(float(norm) ** 2 - float(dgamma.square().sum() + dhead.square().sum())) <= 4 * U * float(norm) ** 2


def test_a_step_captured_follows_its_buffers(example):
    step = example.HeadTrainer(200, 256, 2000, lr=0.0, max_norm=0.01)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            loss, norm = step()
    torch.cuda.synchronize()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        step.x.copy_(torch.randn(200, 256, device="cuda", generator=g))
        step.labels.copy_(torch.randint(-300, 2000, (200,), device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        kept = [loss.clone(), norm.clone()] + [t.clone() for t in step.gradients.values()]
        again = step()
        torch.cuda.synchronize()
        for a, b in zip(kept, [*again, *step.gradients.values()]):
            assert torch.equal(a, b)


def test_example_runs(example, capsys):
    example.main(["--rows", "64", "--steps", "2"])
    assert "step 1" in capsys.readouterr().out


def test_a_workspace_apart_from_what_is_bound():
    """Scratch that shares memory with a tensor of the call is refused; a part of a larger buffer beside the others is not."""
    from speculative_decoding_drafter_gb300 import training as tr

    N, C, V = 4, 64, 100
    n = max(tr.dflash2_residual_norm_grad_workspace_bytes(N, C), tr.dflash2_grad_clip_workspace_bytes(2)) + 256
    arena = torch.zeros(n + 4096, dtype=torch.uint8, device="cuda")
    ws, beside = arena[:n], arena[n + (-n) % 256:]
    z, gamma = torch.ones(N, C, dtype=BF16, device="cuda"), torch.ones(C, dtype=BF16, device="cuda")
    inside = arena[256:256 + 2 * N * C].view(BF16).view(N, C)
    for call in (lambda: tr.dflash2_residual_norm_grad(z, gamma, z, dx=inside, workspace=ws),
                 lambda: tr.dflash2_residual_norm_grad(inside, gamma, z, workspace=ws),
                 lambda: tr.dflash2_residual_norm_grad(z, gamma, z, dgamma=arena[512:512 + 4 * C].view(torch.float32), workspace=ws),
                 lambda: tr.dflash2_grad_clip([inside, z], workspace=ws),
                 lambda: tr.dflash2_grad_clip([z], max_norm=1.0, out=[inside], workspace=ws),
                 lambda: tr.dflash2_grad_clip([z], norm=arena[256:260].view(torch.float32), workspace=ws)):
        with pytest.raises(ValueError, match="overlap"):
            call()
    dgamma = beside[:4 * C].view(torch.float32)
    got = tr.dflash2_residual_norm_grad(z, gamma, z, dgamma=dgamma, workspace=ws)
    assert torch.equal(got["dgamma"], tr.dflash2_residual_norm_grad(z, gamma, z)["dgamma"])
    assert float(tr.dflash2_grad_clip([dgamma], workspace=ws)["norm"]) == float(tr.dflash2_grad_clip([dgamma])["norm"])

    ids, W = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.zeros(V, C, dtype=BF16, device="cuda")
    scratch = tr.LossWorkspace(N, C, V)
    rows = scratch.view[256:256 + 4 * N].view(torch.float32)
    x = torch.zeros(N, device="cuda")
    for call in (lambda: tr.dflash2_lm_head_loss(z, W, ids, loss=rows, workspace=scratch),
                 lambda: tr.dflash2_lm_head_loss(z, W, ids, lse=rows, workspace=scratch),
                 lambda: tr.dflash2_lm_head_loss_grad(z, W, ids, rows, x, workspace=scratch),
                 lambda: tr.dflash2_lm_head_loss_grad(z, W, ids, x, x, d_hidden=scratch.view[256:256 + 2 * N * C].view(BF16).view(N, C),
                                                      workspace=scratch)):
        with pytest.raises(ValueError, match="overlap"):
            call()
