"""The example block: the operators together, in training and token by token."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "recurrent_block.py")


@pytest.fixture(scope="module")
def block():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    spec = importlib.util.spec_from_file_location("recurrent_block", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _autograd(p, x, bounds):
    """The block in float64 torch operations, token by token."""
    import torch
    q = {n: t.double().requires_grad_() for n, t in p.items()}
    xd = x.double().requires_grad_()
    u = xd @ q["w_in"].t() + q["b_in"]
    H = u.shape[1]
    out = []
    for lo, hi in bounds:
        line = torch.cat([u.new_zeros(3, H), u[lo:hi]])
        h = u.new_zeros(H)
        for t in range(hi - lo):
            z = (line[t:t + 4] * q["w_conv"].t()).sum(0) + q["b_conv"]
            v = z * torch.sigmoid(z)
            r, i = (v @ q["w_gate"].t() + q["b_gate"]).chunk(2)
            log_a = -8.0 * torch.nn.functional.softplus(q["lam"]) * torch.sigmoid(r)
            h = torch.exp(log_a) * h + torch.sqrt(-torch.expm1(2 * log_a)) * torch.sigmoid(i) * v
            out.append(h)
    y = torch.stack(out) @ q["w_out"].t() + q["b_out"] + xd
    return y, q, xd


def test_gradients_of_the_block(block):
    """float32 block against autograd in float64.  Every product and scan is good
    to some 1e-6 of its terms' size; a chain of six stays within 1e-4."""
    import torch
    p = block.make_block(12, 20, dtype=torch.float32, seed=3)
    lengths = [5, 0, 1, 30]
    offsets = torch.tensor([0, 5, 5, 6, 36], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    x, dy = (torch.randn(sum(lengths), 12, generator=gen, device="cuda") for _ in range(2))
    y, kept = block.forward(p, x, offsets, train=True)
    grads, dx = block.backward(p, kept, dy)
    torch.cuda.synchronize()
    want, q, xd = _autograd({n: t.cpu() for n, t in p.items()}, x.cpu(),
                            [(0, 5), (5, 5), (5, 6), (6, 36)])
    want.backward(dy.double().cpu())

    def near(a, b):
        b = b.detach()
        return (a.double().cpu() - b).norm() <= 1e-4 * b.norm()

    assert near(y, want) and near(dx, xd.grad)
    for n, t in grads.items():
        assert near(t, q[n].grad), n


def test_training_and_generation(block):
    import torch
    p = block.make_block(64, 128)
    losses = block.train(p)
    # the target's part beyond x has a mean square of about 0.9; a block that does
    # not learn stays there
    assert losses[-1] < 0.5 * losses[0], losses
    x = torch.randn(3, 40, 64, device="cuda").to(torch.bfloat16)
    whole, _ = block.forward(p, x)
    _, state = block.forward(p, x[:, :33].contiguous())
    for t in range(33, 40):
        y = block.step(p, x[:, t].contiguous(), state)
        # the same values rounded to bfloat16 at the same places, from sums in
        # another order: a few of its steps (2^-8) apart, of values up to about 4
        assert (y.float() - whole[:, t].float()).abs().max() <= 8 * 4 * 2.0 ** -8
