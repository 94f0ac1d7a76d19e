"""The mixing operators together, as a token-mixing block uses them: 8-bit
projections, linear attention, a normalisation of each head, a projection back
onto the residual; prompts, single tokens, gradients, replays.  And each of them
where addresses pass 32 bits.
"""
import numpy as np
import pytest

import depthwise_convolution_amd as dw

from . import mixing_reference as ref
from .sequence_reference import bounds_of
from .test_gpu_mixing import (ATTENTION_CASES, DTYPES, _abs, _attention_inputs, _back, _draw,
                              _floor16, _gpu, _longest, _near, torch)  # noqa: F401

pytestmark = pytest.mark.gpu

D, H, KV, DK, DV = 96, 4, 2, 24, 32         # a block's widths
WIDE = H * DK + KV * DK + KV * DV


class Block:
    def __init__(self, torch, dtype, seed):
        rng = np.random.default_rng(seed)
        self.dtype = dtype
        self.wi, self.si = dw.quantize_rows(_draw(torch, rng, (WIDE, D), "float32", D ** -0.5)[0])
        self.wo, self.so = dw.quantize_rows(_draw(torch, rng, (D, H * DV), "float32", 0.1)[0])
        self.bi, self.g = (_draw(torch, rng, (n,), "float32", 0.1)[0] for n in (WIDE, H * DV))
        self.g += 1.0
        self.decay = torch.tensor([-0.01, -0.1, -1.0, 0.0], device="cuda")

    def project(self, x):
        p = dw.linear_i8(x, self.wi, self.si, self.bi)
        q, k, v = p.split([H * DK, KV * DK, KV * DV], -1)      # column ranges
        return q.unflatten(-1, (H, DK)), k.unflatten(-1, (KV, DK)), v.unflatten(-1, (KV, DV))

    def finish(self, y, x):
        n = dw.group_norm(y.reshape(-1, H * DV), H, self.g, act="silu")
        return n, dw.linear_i8(n.reshape(*x.shape[:-1], H * DV), self.wo, self.so, res=x)

    def prompt(self, x, offsets):
        q, k, v = self.project(x)
        y, h = dw.linear_attention(q, k, v, self.decay, offsets=offsets)
        return q, k, v, y, h, *self.finish(y, x)

    def step(self, x, h):
        q, k, v = self.project(x)
        y = dw.linear_attention_step(q, k, v, self.decay, h)
        return q, k, v, y, *self.finish(y, x)


LENGTHS = [130, 0, 1, 200, 64]


@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_of_a_block(torch, dtype):      # noqa: F811
    """Every stage against float64, from what the stage before it gave."""
    print(f"\n[case] block {dtype}", flush=True)
    net, rng = Block(torch, dtype, 1), np.random.default_rng(2)
    offsets = np.concatenate([[0], np.cumsum(LENGTHS)]).astype(np.int32)
    x, xr = _draw(torch, rng, (int(offsets[-1]), D), dtype)
    q, k, v, y, h, n, out = net.prompt(x, _gpu(torch, offsets, "int32"))
    torch.cuda.synchronize()

    def product(got, rows, w, s, b, res, what):
        number, scale = ref.quantize(rows)
        z0 = (number @ _back(w).T) * scale.astype(np.float64)[:, None] * _back(s)
        want = z0 + b + res
        tol = 4 * ref.EPS * np.abs(z0) + 2 * ref.EPS * (np.abs(z0 + b) + np.abs(want))
        _near(got, want, ref.store_tol(want, tol, dtype), what)

    p = torch.cat([t.flatten(-2) for t in (q, k, v)], -1)
    product(p, xr, net.wi, net.si, _back(net.bi), 0.0, "q, k, v")
    parts, bounds = [_back(t) for t in (q, k, v)], bounds_of(offsets)
    want, state = ref.attention(*parts, _back(net.decay), DK ** -0.5, bounds, None)
    qa, ka, va = (np.abs(t) for t in parts)
    big, big_state = ref.attention(qa, ka, va, _back(net.decay), DK ** -0.5, bounds, None)
    floor = _floor16(dtype, DK ** -0.5 * DK * qa.max() * ka.max(), va,
                     DK ** -0.5 * big_state.max(), qa)
    tol = ref.attention_tol(big, DK, max(LENGTHS), dtype, floor)
    _near(y, want, ref.store_tol(want, tol, dtype), "y")
    small = 2.0 ** -22 * 64 * ka.max() * va.max() if dtype == "float16" else 0.0
    _near(h, state, ref.attention_tol(big_state, 0, max(LENGTHS), dtype, small, True), "h")
    norm = ref.Norm(_back(y).reshape(len(xr), -1), H, _back(net.g), 0.0, 1e-5, "silu")
    want, tol = norm.forward()
    _near(n, want, ref.store_tol(want, tol, dtype), "n")
    product(out, _back(n), net.wo, net.so, 0.0, xr, "out")


@pytest.mark.parametrize("dtype", DTYPES)
def test_tokens_after_the_prompt(torch, dtype):     # noqa: F811
    """Five more tokens, one at a time, and the same tokens in a longer prompt: the
    projections are the same bits (their sums are of integers), the rest agrees to the
    tolerances of both."""
    net, rng = Block(torch, dtype, 3), np.random.default_rng(4)
    seqs, first, more = 3, 70, 5
    x, _ = _draw(torch, rng, (seqs, first + more, D), dtype)
    q, k, v, y, h, _, out = net.prompt(x, None)
    _, _, _, _, state, _, _ = net.prompt(x[:, :first].contiguous(), None)
    got = []
    for t in range(first, first + more):
        q1, k1, v1, y1, n1, out1 = net.step(x[:, t].contiguous(), state)
        for one, all_of in ((q1, q), (k1, k), (v1, v)):
            assert torch.equal(one, all_of[:, t])
        # the stages behind a token's result, from that result
        n2, out2 = net.finish(y1, x[:, t].contiguous())
        assert torch.equal(n1, n2) and torch.equal(out1, out2)
        got.append(y1)
    torch.cuda.synchronize()
    parts = [np.abs(_back(t)).reshape(-1, *t.shape[-2:]) for t in (q, k, v)]
    bounds = [(s * (first + more), (s + 1) * (first + more)) for s in range(seqs)]
    big, big_state = ref.attention(*parts, _back(net.decay), DK ** -0.5, bounds, None)
    floor = _floor16(dtype, DK ** -0.5 * DK * parts[0].max() * parts[1].max(), parts[2],
                     DK ** -0.5 * big_state.max(), parts[0])
    tol = ref.store_tol(big, ref.attention_tol(big, DK, first + more, dtype, floor), dtype)
    tol = tol.reshape(seqs, first + more, H, DV)[:, first:]
    _near(torch.stack(got, 1), _back(y)[:, first:], 2 * tol, "y")
    small = 2.0 ** -22 * 64 * parts[1].max() * parts[2].max() if dtype == "float16" else 0.0
    _near(state, _back(h), 2 * ref.attention_tol(big_state, 0, first + more, dtype, small, True),
          "h")


def test_gradient_through_attention_and_norm(torch):    # noqa: F811
    """The gradients of a float32 block's middle, attention and then the heads' norm,
    against float64's chain, whose last stage is given the first's result as the GPU
    computed it."""
    rng = np.random.default_rng(5)
    off = np.array([0, 90, 91, 260], np.int32)
    (q, qr), (k, kr), (v, vr) = (_draw(torch, rng, (260, n, w), "float32")
                                 for n, w in ((H, DK), (KV, DK), (KV, DV)))
    dn, dnr = _draw(torch, rng, (260, H * DV), "float32")
    w, wr = _draw(torch, rng, (H * DV,), "float32")
    decay = torch.tensor([-0.01, -0.1, -1.0, 0.0], device="cuda")
    go = _gpu(torch, off, "int32")
    y, _ = dw.linear_attention(q, k, v, decay, offsets=go)
    flat = y.reshape(260, H * DV)
    _, stats = dw.group_norm(flat, H, w, act="silu", save_stats=True)
    dy, dwt, _ = dw.group_norm_grad(dn, flat, stats, H, w, act="silu")
    dq, dk, dv, _ = dw.linear_attention_grad(dy.reshape(y.shape), q, k, v, decay, offsets=go)
    torch.cuda.synchronize()
    chain = ref.Norm(_back(flat), H, wr, 0.0, 1e-5, "silu").gradient(dnr)
    want, tol = chain["dx"]
    _near(dy, want, ref.store_tol(want, tol, "float32"), "dy")
    _near(dwt, *chain["dw"], "dw")
    args = (qr, kr, vr, _back(decay), DK ** -0.5, bounds_of(off), None, None)
    want = ref.attention_grad(_back(dy).reshape(260, H, DV), *args)
    big = ref.attention_grad(np.abs(_back(dy)).reshape(260, H, DV), np.abs(qr), np.abs(kr),
                             np.abs(vr), *args[3:])
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        tol = ref.attention_tol(big[name], max(DK, DV) + H // KV, 169, "float32")
        _near(got, want[name], ref.store_tol(want[name], tol, "float32"), name)


def test_block_in_a_graph(torch):      # noqa: F811
    """A decoding step captured once and replayed as the states go on, with eager steps
    between the replays that leave it alone."""
    net = Block(torch, "bfloat16", 6)
    x = torch.randn(5, D, device="cuda").bfloat16()
    state = torch.zeros(5, H, DK, DV, device="cuda")
    other = state.clone()
    net.step(x, other)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = net.step(x, state)[-1]
    state.zero_()
    other.zero_()
    for turn in range(4):
        x.copy_(torch.randn(5, D, device="cuda").bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = kept.clone()
        want = net.step(x, other)[-1]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(state, other), turn


def test_two_streams_at_once(torch):     # noqa: F811
    """Calls of different inputs on two streams, with workspaces of their own."""
    nets = [Block(torch, "bfloat16", s) for s in (7, 8)]
    off = _gpu(torch, np.array([0, 300, 900], np.int32), "int32")
    xs = [torch.randn(900, D, device="cuda").bfloat16() for _ in nets]
    want = [net.prompt(x, off) for net, x in zip(nets, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in nets]
    got = [None, None]
    for turn in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = nets[i].prompt(xs[i], off)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


# --------------------------------------------- the rounding of a result alone
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("case", range(len(ATTENTION_CASES)))
def test_16_bit_operands_are_two_numbers(torch, case, dtype):   # noqa: F811
    """Scores, and the state where it meets q, are held in two numbers of the type: cut
    to 8 bits and the rest rounded for bfloat16 (2^-7 times 2^-8), rounded twice for
    float16 (2^-11 times 2^-11).  What is left is the rounding of the result."""
    spec = ATTENTION_CASES[case]
    Dk, scale = spec[3], spec[3] ** -0.5
    print(f"\n[case] two numbers {spec} {dtype}", flush=True)
    g, r = _attention_inputs(torch, spec, dtype, case + 50)
    y, _ = dw.linear_attention(g["q"], g["k"], g["v"], g["log_decay"], h0=g["h0"],
                               offsets=g["off"])
    torch.cuda.synchronize()
    want, _ = ref.attention(r["q"], r["k"], r["v"], r["log_decay"], scale, r["bounds"], r["h0"])
    qa, ka, va, ha = _abs(r, "q", "k", "v", "h0")
    big, big_state = ref.attention(qa, ka, va, r["log_decay"], scale, r["bounds"], ha)
    tokens = _longest(r)
    floor = _floor16(dtype, scale * 64 * Dk, va, scale * np.max(big_state, initial=0.0), qa)
    left = 2.0 ** (-15 if dtype == "bfloat16" else -22)
    tol = ref.attention_tol(big, Dk, tokens, "float32") + left * big + floor
    _near(y, want, ref.store_tol(want, tol, dtype), "y")


# ------------------------------------------------ addresses beyond 32 bits
def _far(torch, t, ld):
    """The rows of t, `ld` elements apart."""
    store = torch.empty(t.shape[0] * ld, dtype=t.dtype, device="cuda")
    view = store.as_strided((t.shape[0], t.shape[1]), (ld, 1))
    view.copy_(t)
    return view


def test_rows_far_apart(torch):     # noqa: F811
    """Rows that lie over 2^32 bytes, each operator as on rows side by side."""
    rng = np.random.default_rng(9)
    rows, ld = 2500, (1 << 21) - 8          # 10 GB of bfloat16
    x = _draw(torch, rng, (rows, 128), "bfloat16")[0]
    far = _far(torch, x, ld)
    assert far.stride(0) * (rows - 1) * 2 > 1 << 33
    q = far.unflatten(-1, (2, 64))
    g = torch.tensor([-0.01, -0.2], device="cuda")
    off = _gpu(torch, np.array([0, 1000, 1003, rows], np.int32), "int32")
    near = x.unflatten(-1, (2, 64))
    for a, b in zip(dw.linear_attention(q, q, q, g, offsets=off),
                    dw.linear_attention(near, near, near, g, offsets=off)):
        assert torch.equal(a, b)
    for a, b in zip(dw.linear_attention_grad(q, q, q, q, g, offsets=off)[:3],
                    dw.linear_attention_grad(near, near, near, near, g, offsets=off)[:3]):
        assert torch.equal(a, b)
    out = _far(torch, torch.zeros_like(x), ld)
    dw.dwconv_norm_fwd(far, 4, None, None, out, act="silu")
    assert torch.equal(out, dw.group_norm(x, 4, act="silu"))
    number, scale = dw.quantize_rows(x)
    for got, want in zip(dw.quantize_rows(far), (number, scale)):
        assert torch.equal(got, want)
    w, ws = dw.quantize_rows(_draw(torch, rng, (72, 128), "float32")[0])
    assert torch.equal(dw.linear_i8(far, w, ws, res=far[:, :72]),
                       dw.linear_i8(x, w, ws, res=x[:, :72]))
    del far, out
    # positions of one image over as many bytes, and its gradient
    img = _draw(torch, rng, (rows, 48), "float32")[0]
    far = _far(torch, img, 1 << 20)
    def image(t):                           # (1, rows, 48)
        return t.as_strided((1, *t.shape), (t.stride(0) * rows, t.stride(0), 1))
    y, s = dw.group_norm(img[None], 6, act="silu", save_stats=True)
    z, s2 = dw.group_norm(image(far), 6, act="silu", save_stats=True)
    assert torch.equal(y, z) and torch.equal(s, s2)
    for a, b in zip(dw.group_norm_grad(y, img[None], s, 6, act="silu"),
                    dw.group_norm_grad(y, image(far), s, 6, act="silu")):
        assert torch.equal(a, b)


def test_states_beyond_32_bits(torch):      # noqa: F811
    """The last of more states than 2^31 elements hold, as among few."""
    rng = np.random.default_rng(10)
    seqs, last = 140000, 40
    q, k, v = (_draw(torch, rng, (seqs, 1, 128), "bfloat16")[0] for _ in range(3))
    g = torch.tensor([-0.1], device="cuda")
    h = torch.empty(seqs, 1, 128, 128, device="cuda")
    assert h.numel() > 1 << 31
    h.fill_(0.5)
    h[-last:] = torch.randn(last, 1, 128, 128, device="cuda")
    few = h[-last:].clone()
    y = dw.linear_attention_step(q, k, v, g, h)
    want = dw.linear_attention_step(q[-last:].contiguous(), k[-last:].contiguous(),
                                    v[-last:].contiguous(), g, few)
    assert torch.equal(y[-last:], want) and torch.equal(h[-last:], few)
    one = [t[:, None] for t in (q, k, v)]
    y, hT = dw.linear_attention(*one, g, h0=h)
    want, few = dw.linear_attention(*(t[-last:].contiguous() for t in one), g, h0=few)
    assert torch.equal(y[-last:], want) and torch.equal(hT[-last:], few)
