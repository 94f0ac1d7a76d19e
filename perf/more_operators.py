"""What three further operators are measured on: linear attention with a decay
for each head, group normalisation with an activation (channels last), and the
matrix product in 8-bit integers with a scale for each row and each column --
what a token-mixing block has around its projections, and, the last two, a
separable convolution net around its depthwise filters.

With ``own`` false ``run`` computes each operator in plain torch operations in
float32; with ``own`` true it calls the library.  ``exact`` computes the
definition in float64.

Linear attention keeps a matrix S for each head, S = exp(log_decay) * S + k v^T,
and answers scale * q S.  Queries are (..., heads, dk), keys (..., kv heads,
dk), values (..., kv heads, dv); a group of adjacent query heads shares a key
and value head.  Dense batches are (sequences, tokens, ...), packed ones
(tokens, ...) with the sequences' int32 offsets, sequences of no token and of
one token among them.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
CHUNK = 64          # tokens that the plain form takes together
EPS = 1e-5          # group normalisation


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one generated token for each of 64 running sequences: bound by their states
        {"name": "attention step", "op": "att_step", "dtype": "bf16", "seqs": 64, "heads": 16,
         "kv_heads": 16, "dk": 128, "dv": 128},
        # a training or prefill batch of equal lengths
        {"name": "attention forward", "op": "att_fwd", "dtype": "bf16", "seqs": 8,
         "tokens": 4096, "heads": 16, "kv_heads": 16, "dk": 128, "dv": 128, "packed": False,
         "carry": False},
        # a serving batch of ragged prompts that continue from carried states, four query
        # heads to a key head, widths that are no power of two
        {"name": "attention forward ragged", "op": "att_fwd", "dtype": "f16", "seqs": 37,
         "tokens": 20011, "heads": 12, "kv_heads": 3, "dk": 96, "dv": 80, "packed": True,
         "carry": True},
        # one very long document and few heads: split along its tokens
        {"name": "attention forward long", "op": "att_fwd", "dtype": "bf16", "seqs": 1,
         "tokens": 65537, "heads": 8, "kv_heads": 8, "dk": 128, "dv": 128, "packed": False,
         "carry": False},
        # the gradient of a training batch
        {"name": "attention gradient", "op": "att_grad", "dtype": "bf16", "seqs": 8,
         "tokens": 2048, "heads": 16, "kv_heads": 16, "dk": 128, "dv": 128, "packed": False,
         "carry": False},
        # the gradient over packed documents in float32, keys shared, states carried
        {"name": "attention gradient ragged", "op": "att_grad", "dtype": "f32", "seqs": 23,
         "tokens": 8209, "heads": 6, "kv_heads": 2, "dk": 64, "dv": 64, "packed": True,
         "carry": True},
        # eight 56x56x128 images
        {"name": "norm image", "op": "norm_fwd", "dtype": "f32", "seqs": 8, "height": 56,
         "width": 56, "channels": 128, "groups": 32, "act": "silu"},
        # one 512x512x256 image
        {"name": "norm image large", "op": "norm_fwd", "dtype": "f32", "seqs": 1,
         "height": 512, "width": 512, "channels": 256, "groups": 32, "act": "none"},
        # every head of every token of a batch by itself, as after linear attention
        {"name": "norm tokens", "op": "norm_fwd", "dtype": "bf16", "seqs": 16384, "height": 1,
         "width": 1, "channels": 2048, "groups": 16, "act": "silu"},
        # the gradient over a training batch of images
        {"name": "norm gradient", "op": "norm_grad", "dtype": "f16", "seqs": 16, "height": 64,
         "width": 64, "channels": 320, "groups": 32, "act": "silu"},
        # eight running sequences through a projection: bound by the weights
        {"name": "linear i8 decode", "op": "linear_i8", "dtype": "bf16", "rows": 8,
         "outs": 8192, "ins": 2048, "act": "silu", "bias": True, "res": False},
        # a block's widening projection over a prefill batch
        {"name": "linear i8 forward", "op": "linear_i8", "dtype": "bf16", "rows": 16384,
         "outs": 8192, "ins": 2048, "act": "silu", "bias": True, "res": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["att_step", "att_fwd", "att_fwd", "att_grad", "att_grad", "norm_fwd",
                     "norm_fwd", "norm_grad", "linear_i8", "linear_i8"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op.startswith("att"):
        kv = _log(rng, 1, 16)
        group = rng.choice([1, 1, 1, 2, 3, 4, 8])
        dims = [16, 32, 64, 64, 128, 128, 128, 256, rng.randint(1, 256)]
        case |= {"heads": kv * group, "kv_heads": kv, "dk": rng.choice(dims),
                 "dv": rng.choice(dims)}
        width = kv * group * max(case["dk"], case["dv"])
        state = kv * group * case["dk"] * case["dv"]
        if op == "att_step":
            return case | {"seqs": _log(rng, 1, max(1, min(256, (1 << 24) // state)))}
        most = (1 << 26 if op == "att_fwd" else 1 << 25) // width
        if case["dtype"] == "f32":
            most //= 4
        total = _log(rng, 1, max(1, min(65536, most)))
        seqs = _log(rng, 1, max(1, min(64, total, (1 << 24) // state)))
        packed = rng.random() < 0.5
        return case | {"seqs": seqs, "packed": packed, "carry": rng.random() < 0.5,
                       "tokens": total if packed else max(1, total // seqs)}
    if op.startswith("norm"):
        groups = _log(rng, 1, 64)
        tokens = rng.random() < 0.4     # one position: groups of 16 channels and more
        channels = groups * _log(rng, 16 if tokens else 1, min(256, 4096 // groups))
        if tokens:
            seqs, height, width = _log(rng, 1, 32768), 1, 1
        else:
            seqs, height, width = _log(rng, 1, 32), _log(rng, 4, 512), _log(rng, 4, 512)
        most = 1 << (26 if op == "norm_fwd" else 25)
        while seqs * height * width * channels > most:
            if seqs > 1:
                seqs = (seqs + 1) // 2
            else:
                height, width = (height + 1) // 2, (width + 1) // 2
        return case | {"seqs": seqs, "height": height, "width": width, "channels": channels,
                       "groups": groups, "act": rng.choice(["none", "silu", "silu"])}

    def wide():                         # widths as models have them, and odd ones
        unit = rng.choice([64, 64, 64, 8, 1])
        return max(unit, _log(rng, 48, 8192) // unit * unit)

    rows, outs, ins = _log(rng, 1, 16384), wide(), wide()
    e = BYTES[case["dtype"]]
    while rows * outs * ins > 2.7e11 or rows * (2 * outs + ins) * e > 6e8:
        rows = (rows + 1) // 2
    return case | {"rows": rows, "outs": outs, "ins": ins, "bias": rng.random() < 0.7,
                   "res": rng.random() < 0.5,
                   "act": rng.choice(["none", "silu", "relu", "relu6"])}


def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op.startswith("att"):
        h, kv, dk, dv, s = (case[n] for n in ("heads", "kv_heads", "dk", "dv", "seqs"))
        row = (h * dk + kv * (dk + dv) + h * dv) * e        # q, k, v, y of a token
        state = s * h * dk * dv * 4
        if op == "att_step":
            return {"bytes": s * row + 2 * state + 4 * h, "flops": 5.0 * s * h * dk * dv}
        rows = case["tokens"] * (1 if case["packed"] else s)
        small = 4 * h + (4 * (s + 1) if case["packed"] else 0)
        if op == "att_fwd":
            return {"bytes": rows * row + state * (2 if case["carry"] else 1) + small,
                    "flops": 4.0 * rows * h * dk * dv}
        grads = (h * dk + kv * (dk + dv)) * e
        return {"bytes": rows * (row + grads) + (3 * state if case["carry"] else 0) + small,
                "flops": 10.0 * rows * h * dk * dv}
    if op.startswith("norm"):
        c, n = case["channels"], case["seqs"] * case["height"] * case["width"]
        stats = 8 * case["seqs"] * case["groups"]
        if op == "norm_fwd":
            return {"bytes": 2 * n * c * e + 8 * c, "flops": 12.0 * n * c}
        return {"bytes": 3 * n * c * e + stats + 16 * c, "flops": 24.0 * n * c}
    m, n, k = case["rows"], case["outs"], case["ins"]
    io = m * k + m * n + (m * n if case["res"] else 0)
    return {"bytes": io * e + n * k + 4 * n + (n * 4 if case["bias"] else 0),
            "flops": 2.0 * m * n * k + 8.0 * m * n + 4.0 * m * k}


# ------------------------------------------------------------------ inputs
def _offsets(seqs, tokens, seed):
    """Sequence bounds of a packed batch: random cuts, some of them at one
    place (no token between them) or one token apart."""
    rng = np.random.RandomState(seed % (1 << 31))
    cuts = np.sort(rng.randint(0, tokens + 1, seqs - 1))
    if seqs >= 4:
        cuts[1] = cuts[0]
        cuts[-1] = min(tokens, cuts[-2] + 1)
    return np.concatenate([[0], cuts, [tokens]]).astype(np.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    op = case["op"]
    s = {"op": op, "act": case.get("act"), "groups": case.get("groups")}
    if op.startswith("att"):
        h, kv, dk, dv, seqs = (case[n] for n in ("heads", "kv_heads", "dk", "dv", "seqs"))
        s["scale"] = dk ** -0.5
        # memories of 4 to 8192 tokens, one for each head
        memory = torch.rand(h, generator=gen, device=dev) * math.log(2048.0) + math.log(4.0)
        s["log_decay"] = -torch.exp(-memory)
        lead = (seqs,)
        if op != "att_step":
            lead = (case["tokens"],) if case["packed"] else (seqs, case["tokens"])
            s["offsets"] = None
            if case["packed"]:
                s["offsets"] = torch.from_numpy(_offsets(seqs, case["tokens"], seed)).to(dev)
        s["q"], s["k"] = normal(*lead, h, dk), normal(*lead, kv, dk)
        s["v"] = normal(*lead, kv, dv)
        state = (seqs, h, dk, dv)
        if op == "att_step":
            s["h"] = normal(*state, dtype=torch.float32)
            return s
        carry = case["carry"]
        s["h0"] = normal(*state, dtype=torch.float32) if carry else None
        if op == "att_grad":
            s["dy"] = normal(*lead, h, dv)
            s["dhT"] = normal(*state, dtype=torch.float32) if carry else None
        return s
    if op.startswith("norm"):
        c = case["channels"]
        lead = (case["seqs"],)
        if case["height"] * case["width"] > 1:
            lead = (case["seqs"], case["height"], case["width"])
        spread, at = normal(c, std=0.3).float().exp(), normal(c).float()
        s["x"] = (normal(*lead, c, dtype=torch.float32) * spread + at).to(dt)
        s["w"], s["b"] = normal(c, std=0.2, dtype=torch.float32) + 1, normal(
            c, std=0.2, dtype=torch.float32)
        if op == "norm_grad":
            s["dy"] = normal(*lead, c)
            s["stats"] = _stats(s["x"], s["groups"])     # kept by the forward
        return s
    m, n, k = case["rows"], case["outs"], case["ins"]
    s["x"] = normal(m, k)
    # the weights as a program keeps them: numbers and a scale for each output
    w = normal(n, k, std=k ** -0.5, dtype=torch.float32)
    s["w_scale"] = w.abs().amax(1) / 127
    s["w"] = torch.round(w.double() / s["w_scale"].double()[:, None]).to(torch.int8)
    s["b"] = normal(n, std=0.1, dtype=torch.float32) if case["bias"] else None
    s["res"] = normal(m, n) if case["res"] else None
    return s


# ------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "relu6":
        return torch.clamp(z, 0, 6)
    return z


class _Chunks:
    """The rows of a batch in chunks of CHUNK tokens that begin with a sequence:
    the chunks of sequence s are numbered from start[s] // CHUNK + s on, so that
    their number does not depend on the lengths (some chunks have no row).
    Turned round, a sequence's last token comes first."""

    def __init__(self, x, offsets, back):
        if offsets is None:
            offsets = torch.arange(x.shape[0] + 1, device=x.device) * x.shape[1]
        self.n = x.numel() // (x.shape[-1] * x.shape[-2])
        offsets = offsets.long()
        start, end = offsets[:-1], offsets[1:]
        seqs = len(start)
        base = start // CHUNK + torch.arange(seqs, device=x.device)
        ids = torch.arange(self.n // CHUNK + seqs, device=x.device)
        self.seq = torch.searchsorted(base, ids, right=True) - 1
        place = ids - base[self.seq]
        at = place[:, None] * CHUNK + torch.arange(CHUNK, device=x.device)
        length = (end - start)[self.seq][:, None]
        self.valid = at < length
        row = start[self.seq][:, None] + (length - 1 - at if back else at)
        self.rows = torch.where(self.valid, row, self.n)      # row n: none
        self.count = self.valid.sum(1)
        self.first = place == 0
        self.last = base + torch.clamp((end - start - 1) // CHUNK, min=0)

    def gather(self, x, heads):
        """(chunks, heads, CHUNK, width) in float32, zero where there is no row."""
        x = x.reshape(self.n, x.shape[-2], x.shape[-1])
        x = torch.cat([x, torch.zeros_like(x[:1])]) if self.n else x.new_zeros(
            1, *x.shape[1:])
        x = x[self.rows].float().transpose(1, 2)
        return x.repeat_interleave(heads // x.shape[1], 1).contiguous()

    def scatter(self, y):
        """(rows, heads, width) of the chunks' rows."""
        out = y.new_zeros(self.n + 1, y.shape[1], y.shape[3])
        out[self.rows.reshape(-1)] = y.transpose(1, 2).reshape(-1, y.shape[1], y.shape[3])
        return out[:self.n]


def _walk(q, k, v, log_decay, scales, late, h0, chunks):
    """For each row i of a sequence

        y[i] = scales[0] * sum_{j <= i} a^(i - j) (q[i] . k[j]) v[j]
               + scales[1] * a^(i + 1 - late) q[i] h0

    and the state after it, the chunks' states in doubling steps."""
    heads = len(log_decay)
    q, k, v = (chunks.gather(t, heads) for t in (q, k, v))
    g = log_decay[:, None, None]
    i = torch.arange(CHUNK, device=g.device)
    gap = i[:, None] - i[None]
    fade = torch.where(gap >= 0, torch.exp(g * gap.clamp(min=0)), 0.0)
    y = torch.matmul(torch.matmul(q, k.transpose(2, 3).contiguous()) * fade * scales[0], v)
    count = chunks.count[:, None, None, None]
    left = (count - 1 + late - i[:, None]).clamp(min=0)
    b = torch.matmul((k * torch.exp(g * left)).transpose(2, 3).contiguous(), v) * scales[2]
    a = torch.exp(g * count)
    first = chunks.first[:, None, None, None]
    before = torch.zeros_like(b[:1]) if h0 is None else h0[chunks.seq]
    b = torch.where(first, b + a * before, b)
    a = torch.where(first, 0.0, a)
    step = 1
    while step < len(b):
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    into = torch.where(first, before, torch.cat([b[:1], b[:-1]]))
    y = y + scales[1] * torch.exp(g * (i[:, None] + 1 - late)) * torch.matmul(q, into)
    return chunks.scatter(y), b[chunks.last]


def _att_fwd(s):
    q, scale = s["q"], s["scale"]
    chunks = _Chunks(q, s["offsets"], False)
    y, last = _walk(q, s["k"], s["v"], s["log_decay"], (scale, scale, 1.0), 0, s["h0"], chunks)
    return y.to(q.dtype).reshape(*q.shape[:-1], -1), last


def _att_grad(s):
    q, k, v, dy, g, scale = (s[n] for n in ("q", "k", "v", "dy", "log_decay", "scale"))
    ahead, back = (_Chunks(q, s["offsets"], turned) for turned in (False, True))

    def flip(h):
        return None if h is None else h.transpose(2, 3).contiguous()

    def shared(t, like):                # the sum over the query heads of a key head
        t = t.reshape(len(t), like.shape[-2], -1, like.shape[-1]).sum(2)
        return t.to(like.dtype).reshape(like.shape)

    dq, _ = _walk(dy, v, k, g, (scale, scale, 1.0), 0, flip(s["h0"]), ahead)
    dk, dh0 = _walk(v, dy, q, g, (scale, 1.0, scale), 1, flip(s["dhT"]), back)
    dv, _ = _walk(k, q, dy, g, (scale, 1.0, scale), 1, s["dhT"], back)
    out = [dq.to(q.dtype).reshape(q.shape), shared(dk, k), shared(dv, v)]
    return out if s["h0"] is None else [*out, flip(dh0)]


def _att_step(s):
    q, k, v, h = s["q"].float(), s["k"].float(), s["v"].float(), s["h"]
    group = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    a = torch.exp(s["log_decay"])[:, None, None]
    h.copy_(a * h + k[..., None] * v[..., None, :])
    y = s["scale"] * (q[..., None] * h).sum(2)
    return y.to(s["q"].dtype), h


def _grouped(x, groups):
    """(instances, positions, groups, channels of a group) in float32."""
    c = x.shape[-1]
    return x.float().reshape(x.shape[0], -1, groups, c // groups)


def _stats(x, groups):
    """(instances, groups, 2): the mean, and the reciprocal of the deviation."""
    x = _grouped(x, groups)
    mean = x.mean((1, 3))
    var = (x - mean[:, None, :, None]).square().mean((1, 3))
    return torch.stack([mean, 1 / torch.sqrt(var + EPS)], 2)


def _normal(x, stats):
    return (x - stats[:, None, :, None, 0]) * stats[:, None, :, None, 1]


def _norm_fwd(s):
    x = s["x"]
    xhat = _normal(_grouped(x, s["groups"]), _stats(x, s["groups"]))
    z = xhat.reshape(x.shape) * s["w"] + s["b"]
    return _act(z, s["act"]).to(x.dtype)


def _norm_grad(s):
    x, w, stats = s["x"], s["w"], s["stats"]
    xhat = _normal(_grouped(x, s["groups"]), stats)
    dz = s["dy"].float()
    if s["act"] == "silu":
        z = xhat.reshape(x.shape) * w + s["b"]
        p = 1 / (1 + torch.exp(-z))
        dz = dz * p * (1 + z * (1 - p))
    over = tuple(range(x.dim() - 1))
    dw, db = (dz * xhat.reshape(x.shape)).sum(over), dz.sum(over)
    dx = _grouped(dz * w, s["groups"])
    dx = dx - dx.mean((1, 3), True) - xhat * (dx * xhat).mean((1, 3), True)
    return (dx * stats[:, None, :, None, 1]).to(x.dtype).reshape(x.shape), dw, db


def _linear_i8(s):
    x = s["x"].float()
    scale = torch.clamp(x.abs().amax(1) / 127, min=2.0 ** -126)
    # a quotient next to a half has to fall on its side of it: in 64 bits
    xq = torch.round(x.double() / scale.double()[:, None]).clamp(-127, 127).float()
    z = (xq @ s["w"].float().t()) * (scale[:, None] * s["w_scale"])
    if s["b"] is not None:
        z = z + s["b"]
    y = _act(z, s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(s["x"].dtype)


PLAIN = {"att_step": _att_step, "att_fwd": _att_fwd, "att_grad": _att_grad,
         "norm_fwd": _norm_fwd, "norm_grad": _norm_grad, "linear_i8": _linear_i8}


# ------------------------------------------------------------- the library
def _library(s):
    import depthwise_convolution_amd as dw
    op = s["op"]
    if op == "att_step":
        y = dw.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["h"],
                                     scale=s["scale"])
        return y, s["h"]
    if op == "att_fwd":
        return dw.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], h0=s["h0"],
                                   offsets=s["offsets"], scale=s["scale"])
    if op == "att_grad":
        grads = dw.linear_attention_grad(s["dy"], s["q"], s["k"], s["v"], s["log_decay"],
                                         h0=s["h0"], dhT=s["dhT"], offsets=s["offsets"],
                                         scale=s["scale"])
        return list(grads[:3] if s["h0"] is None else grads)
    if op == "norm_fwd":
        return dw.group_norm(s["x"], s["groups"], s["w"], s["b"], eps=EPS, act=s["act"])
    if op == "norm_grad":
        return dw.group_norm_grad(s["dy"], s["x"], s["stats"], s["groups"], s["w"], s["b"],
                                  act=s["act"])
    return dw.linear_i8(s["x"], s["w"], s["w_scale"], s["b"], act=s["act"], res=s["res"])


def run(state):
    return _library(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------- the definition, 64 bits
def _act64(z, act):
    return {"none": lambda v: v, "silu": lambda v: v * torch.sigmoid(v),
            "relu": lambda v: torch.maximum(v, torch.zeros_like(v)),
            "relu6": lambda v: torch.minimum(torch.maximum(v, torch.zeros_like(v)),
                                             torch.full_like(v, 6.0))}[act](z)


class _Tokens:
    """The tokens of a batch, one of every sequence at a time, the longest
    sequences first: for step t the rows of those that have a token t."""

    def __init__(self, s):
        q = s["q"]
        if s["offsets"] is None:
            bounds = [(n * q.shape[1], (n + 1) * q.shape[1]) for n in range(q.shape[0])]
        else:
            at = s["offsets"].tolist()
            bounds = list(zip(at[:-1], at[1:]))
        order = sorted(range(len(bounds)), key=lambda n: bounds[n][0] - bounds[n][1])
        self.order = torch.tensor(order, device=q.device)
        self.start = torch.tensor([bounds[n][0] for n in order], device=q.device)
        lengths = [bounds[n][1] - bounds[n][0] for n in order]
        self.running, self.steps = [], lengths[0]
        alive = len(order)
        for t in range(self.steps):
            while lengths[alive - 1] <= t:
                alive -= 1
            self.running.append(alive)


def _exact_att(s):
    """Token by token; gradients from the state that each token has seen and
    the cotangent of the state that it has left."""
    q, k, v = (s[n].double().flatten(0, -3) for n in ("q", "k", "v"))
    heads, kv = q.shape[1], k.shape[1]
    key_head = torch.arange(heads, device=q.device) // (heads // kv)
    tokens = _Tokens(s)
    a = torch.exp(s["log_decay"].double())[:, None, None]
    scale = s["scale"]
    shape = (len(tokens.order), heads, k.shape[2], v.shape[2])
    h = q.new_zeros(shape) if s["h0"] is None else s["h0"].double()[tokens.order]
    grad = s["op"] == "att_grad"
    y = torch.zeros_like(q) if grad else q.new_zeros(len(q), heads, v.shape[2])
    dy = s["dy"].double().flatten(0, -3) if grad else None
    for t in range(tokens.steps):
        n = tokens.running[t]
        rows = tokens.start[:n] + t
        new = h[:n]
        new *= a
        new += k[rows][:, key_head].unsqueeze(3) * v[rows][:, key_head].unsqueeze(2)
        if grad:        # dq
            y[rows] = scale * torch.matmul(new, dy[rows].unsqueeze(3)).squeeze(3)
        else:
            y[rows] = scale * torch.matmul(q[rows].unsqueeze(2), new).squeeze(2)
    back = torch.empty_like(tokens.order)
    back[tokens.order] = torch.arange(len(back), device=back.device)
    if not grad:
        return y.reshape(*s["q"].shape[:-1], -1), h[back]
    g = q.new_zeros(shape) if s["dhT"] is None else s["dhT"].double()[tokens.order]
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for t in reversed(range(tokens.steps)):
        n = tokens.running[t]
        rows = tokens.start[:n] + t
        now = g[:n]                     # of the state that token t leaves
        now += scale * q[rows].unsqueeze(3) * dy[rows].unsqueeze(2)
        vk, kk = v[rows][:, key_head].unsqueeze(3), k[rows][:, key_head].unsqueeze(2)
        dk[rows] = torch.matmul(now, vk).reshape(n, kv, -1, k.shape[2]).sum(2)
        dv[rows] = torch.matmul(kk, now).reshape(n, kv, -1, v.shape[2]).sum(2)
        now *= a
    out = [y.reshape(s["q"].shape), dk.reshape(s["k"].shape), dv.reshape(s["v"].shape)]
    return out if s["h0"] is None else [*out, g[back]]


def _exact_norm(s):
    x = s["x"].double().requires_grad_(s["op"] == "norm_grad")
    w, b = (s[n].double().requires_grad_(x.requires_grad) for n in ("w", "b"))
    rows = x.reshape(x.shape[0], -1, x.shape[-1])
    parts = rows.reshape(rows.shape[0], rows.shape[1], s["groups"], -1).transpose(1, 2)
    parts = parts.reshape(rows.shape[0], s["groups"], -1)
    var, mean = torch.var_mean(parts, 2, correction=0, keepdim=True)
    normed = (parts - mean) / torch.sqrt(var + EPS)
    normed = normed.reshape(rows.shape[0], s["groups"], rows.shape[1], -1).transpose(1, 2)
    y = _act64(normed.reshape(x.shape) * w + b, s["act"])
    if s["op"] == "norm_fwd":
        return y
    y.backward(s["dy"].double())
    return x.grad, w.grad, b.grad


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("att_fwd", "att_grad"):
        return _exact_att(s)
    if op == "att_step":
        group = s["q"].shape[1] // s["k"].shape[1]
        k, v = (s[n].double().repeat_interleave(group, 1) for n in ("k", "v"))
        h = torch.exp(s["log_decay"].double())[:, None, None] * s["h"].double()
        h = h + torch.matmul(k.unsqueeze(3), v.unsqueeze(2))
        return s["scale"] * torch.matmul(s["q"].double().unsqueeze(2), h).squeeze(2), h
    if op.startswith("norm"):
        return _exact_norm(s)
    x = s["x"].double()
    scale = (x.abs().amax(1, keepdim=True).float() / 127).clamp(min=2.0 ** -126).double()
    xq = torch.clamp(torch.round(x / scale), -127, 127)
    z = torch.matmul(xq * scale, (s["w"].double() * s["w_scale"].double()[:, None]).t())
    z = _act64(z if s["b"] is None else z + s["b"].double(), s["act"])
    return z if s["res"] is None else z + s["res"].double()
