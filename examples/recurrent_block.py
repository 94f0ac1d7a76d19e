"""A recurrent token-mixing block on the library's sequence operators: training
on a packed batch of ragged sequences, then generation token by token.

    python examples/recurrent_block.py

The block, for tokens of width C and H recurrent channels:

    u = x W_in^T + b_in                          linear
    v = silu(causal depthwise filter of u)       causal_conv, 4 taps
    r, i = halves of v W_gate^T + b_gate         linear
    h = gated recurrence of v under r and i      gated_scan
    y = h W_out^T + b_out + x                    linear with a residual

It is trained to add to each token a slow average of the tokens before it,
which takes the recurrence's long memory.  Needs a GPU.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import depthwise_convolution_amd as dw  # noqa: E402

TAPS = 4


def make_block(C, H, device="cuda", dtype=torch.bfloat16, seed=0):
    """Parameters of a block: matrices in `dtype`, the rest float32."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)

    def normal(*shape, std, kind=dtype):
        return (torch.randn(shape, generator=gen, device=device) * std).to(kind)

    # decays between 0.9 and 0.999 a token where the gate is fully open
    decay = torch.rand(H, generator=gen, device=device) * 0.099 + 0.9
    f32 = torch.float32
    return {"w_in": normal(H, C, std=C ** -0.5), "b_in": torch.zeros(H, device=device),
            "w_conv": normal(H, TAPS, std=TAPS ** -0.5, kind=f32),
            "b_conv": torch.zeros(H, device=device),
            "w_gate": normal(2 * H, H, std=H ** -0.5), "b_gate": torch.zeros(2 * H, device=device),
            "lam": torch.log(torch.expm1(-torch.log(decay) / 8.0)),
            "w_out": normal(C, H, std=0.1 * H ** -0.5), "b_out": torch.zeros(C, device=device)}


def forward(p, x, offsets=None, state=None, train=False):
    """(y, state): x is (sequences, tokens, C), or (tokens, C) with offsets.
    state: what a continuation passes on; with train, what backward needs."""
    rows, h0 = (None, None) if state is None else state
    u = dw.linear(x, p["w_in"], p["b_in"])
    v, rows = dw.causal_conv(u, p["w_conv"], p["b_conv"], act="silu", init=rows,
                             offsets=offsets)
    gates = dw.linear(v, p["w_gate"], p["b_gate"])
    r, i = gates.chunk(2, dim=-1)           # column ranges: read where they are
    scanned = dw.gated_scan(v, r, i, p["lam"], h0=h0, offsets=offsets, save_states=train)
    h, hT = scanned[:2]
    y = dw.linear(h, p["w_out"], p["b_out"], res=x)
    if train:
        return y, (x, u, v, r, i, h, scanned[2], offsets)
    return y, (rows, hT)


def backward(p, kept, dy):
    """Gradients of the parameters, and of x."""
    x, u, v, r, i, h, states, offsets = kept
    g = {}
    dh, g["w_out"], g["b_out"] = dw.linear_grad(dy, h, p["w_out"])
    # the recurrence writes both gates' gradients into one tensor, as the
    # product that made the gates wants them
    dgates = h.new_empty((*h.shape[:-1], 2 * h.shape[-1]))
    dr, di = dgates.chunk(2, dim=-1)
    dv, g["lam"] = torch.empty_like(h), torch.empty_like(p["lam"])
    packed = offsets is not None
    seqs, tokens = (len(offsets) - 1, h.shape[0]) if packed else h.shape[:2]
    space = torch.empty(dw.dwconv_scan_workspace_size(True, seqs, tokens, packed, h.shape[-1]),
                        dtype=torch.uint8, device=h.device)
    dw.dwconv_scan_grad(dh, v, r, i, p["lam"], states, dv, dr, di, g["lam"], workspace=space,
                        offsets=offsets)
    dv2, g["w_gate"], g["b_gate"] = dw.linear_grad(dgates, v, p["w_gate"])
    du, g["w_conv"], g["b_conv"], _ = dw.causal_conv_grad(dv + dv2, u, p["w_conv"], p["b_conv"],
                                                          act="silu", offsets=offsets)
    dx, g["w_in"], g["b_in"] = dw.linear_grad(du, x, p["w_in"])
    return g, dx + dy


def step(p, x, state):
    """One token of each sequence, (sequences, C); the state is updated in place."""
    rows, h = state
    u = dw.linear(x, p["w_in"], p["b_in"])
    v = dw.causal_conv_step(u, rows, p["w_conv"], p["b_conv"], act="silu")
    r, i = dw.linear(v, p["w_gate"], p["b_gate"]).chunk(2, dim=-1)
    y = dw.gated_scan_step(v, r, i, p["lam"], h)
    return dw.linear(y, p["w_out"], p["b_out"], res=x)


def slow_average(x, keep=0.95):
    """Along a sequence, avg = keep * avg + sqrt(1 - keep^2) * x."""
    age = torch.arange(len(x), device=x.device)
    age = age[:, None] - age
    weights = torch.where(age >= 0, keep ** age.clamp(min=0).float(), 0.0)
    return (1 - keep * keep) ** 0.5 * weights @ x.float()


def train(p, steps=150, lengths=(190, 1, 64, 0, 300, 77, 128), rate=1e-2, seed=1):
    """Losses of `steps` Adam steps on random sequences of those lengths; the
    target is the token plus the slow average up to it."""
    C, dev = p["w_in"].shape[1], p["lam"].device
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    bounds = torch.tensor([0, *lengths]).cumsum(0).to(torch.int32)
    offsets = bounds.to(dev)
    master = {n: t.float().clone() for n, t in p.items()}
    m = {n: torch.zeros_like(t) for n, t in master.items()}
    s = {n: torch.zeros_like(t) for n, t in master.items()}
    losses = []
    for k in range(1, steps + 1):
        x = torch.randn(sum(lengths), C, generator=gen, device=dev).to(p["w_in"].dtype)
        target = x.float() + torch.cat([slow_average(x[lo:hi]) for lo, hi in
                                        zip(bounds[:-1].tolist(), bounds[1:].tolist())])
        y, kept = forward(p, x, offsets, train=True)
        off = y.float() - target
        losses.append(off.square().mean())
        grads, _ = backward(p, kept, (off * (2.0 / off.numel()) * 1024).to(x.dtype))
        for n, t in grads.items():
            t = t.float() / 1024                # the loss was scaled for 16 bits
            m[n].lerp_(t, 0.1)
            s[n].lerp_(t * t, 0.02)
            master[n] -= rate * (m[n] / (1 - 0.9 ** k)) / \
                ((s[n] / (1 - 0.98 ** k)).sqrt() + 1e-8)
            p[n].copy_(master[n])
    return [float(v) for v in losses]


def main():
    p = make_block(64, 256)
    losses = train(p)
    print(f"loss {losses[0]:.3f} at the start, {losses[-1]:.3f} after {len(losses)} steps")
    x = torch.randn(3, 100, 64, device="cuda").to(torch.bfloat16)
    whole, _ = forward(p, x)
    prompt, state = forward(p, x[:, :90].contiguous())
    tokens = [step(p, x[:, t].contiguous(), state) for t in range(90, 100)]
    apart = (torch.stack(tokens, 1).float() - whole[:, 90:].float()).abs().max()
    print(f"ten tokens one by one against all at once: at most {float(apart):.3g} apart")


if __name__ == "__main__":
    main()
