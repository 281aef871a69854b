"""Measured cases of a training step's ends and joints: AdamW over many tensors with
states in 32 or 8 bits, log probabilities of tokens with their gradient, and the
norms, gate and residual between two blocks with their gradient.

Every case is one call (the 8-bit step: a call and the reading back of its states)
of a training or scoring program. ``run`` computes it either in plain torch
operations (32-bit arithmetic, one rounding at the end) or, with ``own`` set, through
the library's public entry points. Sizes are those of the GPT-2 760M set (width 1536,
MLP 6144, 50304 tokens) and of the 8B layer (4096, 6144, 14336).
"""
import math
import random
import struct

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, **kw):
    return dict(name=name, op=op, **kw)


def listed():
    return [
        # the vectors of one MLP block (biases, norm parameters), which stay on AdamW
        _case("adam_vectors", "adam", sizes="block_vectors", w="f32", g="f32", state="f32",
              packed=False, clip=False),
        # a whole GPT-2 760M set: 24 layers and the embedding, mixed precision
        _case("adam_model", "adam", sizes="gpt2_760m", w="bf16", g="bf16", state="f32",
              packed=False, clip=True),
        # one 8B layer with its states in 8 bits
        _case("adam_layer_8bit", "adam", sizes="layer_8b", w="bf16", g="bf16", state="8bit",
              packed=False, clip=True),
        # many odd tensors back to back in flat buffers (no alignment), 8 bits
        _case("adam_ragged_8bit", "adam", sizes="drawn", count=61, total=9_000_001, shape_seed=3,
              w="f32", g="f32", state="8bit", packed=True, clip=False),
        # the logits of one decoded token: its probability, five alternatives, entropy
        _case("score_token", "tokens", rows=1, vocab=50304, dtype="bf16", top=5, masked=47),
        # the same for a ragged prompt, twenty alternatives
        _case("score_prompt", "tokens", rows=77, vocab=50304, dtype="bf16", top=20, masked=47),
        # the loss of a training batch and the gradient of its logits
        _case("loss_train", "tokens_loss", rows=16384, vocab=50304, dtype="bf16", masked=47),
        # gradient of log probabilities and entropy (a policy's update), odd sizes, fp32
        _case("policy_gradient", "tokens_bwd", rows=2045, vocab=50301, dtype="f32", masked=0),
        # between two blocks, decoding one token
        _case("join_token", "join", rows=1, cols=1536, stream="bf16", block="bf16", post="rms",
              pre="rms", gate="none"),
        # between two blocks of a training batch, a learned gate per channel
        _case("join_train", "join", rows=16384, cols=1536, stream="bf16", block="bf16",
              post="layer", pre="layer", gate="vector"),
        # its backward pass
        _case("join_train_backward", "join_bwd", rows=16384, cols=1536, stream="bf16",
              block="bf16", post="layer", pre="layer", gate="vector"),
        # the 8B layer's width, fp32 residual stream, a gate per token and channel, odd rows
        _case("join_backward_8b", "join_bwd", rows=4093, cols=4096, stream="f32", block="bf16",
              post="rms", pre="rms", gate="matrix"),
    ]


def _size(rng, lo, hi):
    """Log-uniform; half of the draws on a multiple of 8, odd ones among the rest."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        v = v // 8 * 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["adam", "adam", "tokens", "tokens_loss", "tokens_bwd", "join", "join_bwd"])
    if op == "adam":
        count = _size(rng, 1, 200)
        return dict(op=op, sizes="drawn", count=count, total=max(count, _size(rng, 300, 150_000_000)),
                    shape_seed=rng.randrange(1 << 30), w=rng.choice(["bf16", "f32"]),
                    g=rng.choice(["bf16", "f32"]), state=rng.choice(["f32", "8bit"]),
                    packed=rng.random() < 0.3, clip=rng.random() < 0.5)
    if op in ("tokens", "tokens_loss", "tokens_bwd"):
        vocab = _size(rng, 200, 260_000)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 16384 * 50304 // (2 if dtype == "f32" else 1)
        c = dict(op=op, rows=_size(rng, 1, max(1, min(16384, most // vocab))), vocab=vocab,
                 dtype=dtype, masked=rng.choice([0, 1, vocab // 7]))
        if op == "tokens":
            # sorting every row, the plain form's way to its alternatives, has its price
            c["top"] = rng.choice([0, 1, 8, 20, 32])
            if c["top"]:
                c["rows"] = min(c["rows"], max(1, 100_000_000 // vocab))
        return c
    cols = _size(rng, 64, 16384)
    return dict(op=op, rows=_size(rng, 1, min(16384, 16384 * 4096 // cols)), cols=cols,
                stream=rng.choice(["bf16", "f32"]), block=rng.choice(["bf16", "f32"]),
                post=rng.choice(["none", "layer", "rms"]), pre=rng.choice(["layer", "rms"]),
                gate=rng.choice(["none", "vector", "matrix"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

BETA1, BETA2, LR, DECAY, EPS, STEP = 0.9, 0.95, 1e-3, 0.1, 1e-8, 37
X_SCALE, B_SCALE, NORM_EPS = 0.9, 1.25, 1e-5
SPAN = 256  # elements per scale of an 8-bit state


def _f32(x):
    """The fp32 number that a hyperparameter is passed as."""
    return struct.unpack("f", struct.pack("f", x))[0]


def _adam_sizes(case):
    kind = case["sizes"]
    if kind == "block_vectors":
        return [6144, 1536, 1536, 1536]
    if kind == "layer_8b":
        return [4096 * 6144, 4096 * 4096, 14336 * 4096, 14336 * 4096, 4096 * 14336]
    if kind == "gpt2_760m":
        layer = [1536 * 1536] * 4 + [6144 * 1536] * 2 + [6144] + [1536] * 9
        return layer * 24 + [50304 * 1536]
    r = random.Random(case["shape_seed"])
    parts = [math.exp(r.gauss(0.0, 2.0)) for _ in range(case["count"])]
    scale = (case["total"] - case["count"]) / sum(parts)
    return [1 + int(p * scale) for p in parts]


class _Gen:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=torch.float32)

    def whole(self, hi, *shape):
        return torch.randint(0, hi, shape, generator=self.g, device="cuda")

    def activation(self, rows, cols):
        """Hidden states: token scales that vary, a few outlier channels, and (past the
        first rows) some all-zero padding tokens."""
        x = self.normal(rows, cols)
        x *= torch.exp(0.3 * self.normal(rows, 1))
        x *= torch.where(self.normal(1, cols) > 2.6, 8.0, 1.0)
        x[5::97] = 0.0
        return x

    def gradient(self, rows, cols):
        return self.normal(rows, cols) * torch.exp(0.5 * self.normal(rows, 1)) * 2e-3


def _rows(t):
    """The values of ``t`` in rows padded to a multiple of 8 elements."""
    r, c = t.shape
    buf = torch.zeros((r, (c + 7) // 8 * 8), dtype=t.dtype, device=t.device)
    buf[:, :c] = t
    return buf[:, :c]


def _prepare_adam(case, g):
    """Flat buffers, as a program with gradient buckets keeps them, and the tensors in
    them: padded to 16 elements, or (packed) back to back."""
    sizes = _adam_sizes(case)
    step = 1 if case["packed"] else 16
    at, spans, total, blocks = [], [], 0, 0
    for n in sizes:
        at.append(total)
        spans.append(blocks)
        total += (n + step - 1) // step * step
        blocks += (n + SPAN - 1) // SPAN
    grad = 1e-3 * g.normal(total) * torch.exp(g.normal(total))
    w = (0.02 * g.normal(total)).to(TYPES[case["w"]])
    st = {"case": case, "w": w, "g": grad.to(TYPES[case["g"]])}
    if case["clip"]:
        st["clip"] = torch.full((), 0.7, device="cuda")
    cut = lambda t, first: [t[i:i + n] for i, n in zip(first, sizes)]  # noqa: E731
    parts = [cut(st["w"], at), cut(st["g"], at)]
    if case["state"] == "f32":
        st["m"] = 3e-4 * g.normal(total)
        st["v"] = (1e-3 * g.normal(total)).square()
        parts += [cut(st["m"], at), cut(st["v"], at)]
    else:
        # a first moment around zero; a second moment whose codes avoid the zero
        st["m"] = g.whole(256, total).to(torch.uint8)
        st["v"] = (1 + g.whole(255, total)).to(torch.uint8)
        st["ms"] = 3e-4 * (0.5 + g.normal(blocks).abs())
        st["vs"] = 1e-3 * (0.5 + g.normal(blocks).abs())
        spaces = [slice(i, i + (n + SPAN - 1) // SPAN) for i, n in zip(spans, sizes)]
        parts += [cut(st["m"], at), [st["ms"][s] for s in spaces],
                  cut(st["v"], at), [st["vs"][s] for s in spaces]]
        st["m_value"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
        st["v_value"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
        st["states"] = [p[2:] for p in zip(*parts)]
        st["values"] = list(zip(cut(st["m_value"], at), cut(st["v_value"], at)))
    st["items"] = list(zip(*parts))
    return st


def prepare(case, seed):
    g = _Gen(seed)
    op = case["op"]
    if op == "adam":
        return _prepare_adam(case, g)
    rows = case["rows"]
    st = {"case": case}
    if op.startswith("tokens"):
        vocab = case["vocab"]
        x = 2.0 * g.normal(rows, vocab) * torch.exp(0.2 * g.normal(rows, 1))
        x += 2.0 * g.normal(1, vocab)  # frequent and rare tokens
        if case["masked"]:  # padding of the vocabulary, or tokens a grammar excludes
            x[:, vocab - case["masked"]:] = -math.inf
        st["x"] = _rows(x.to(TYPES[case["dtype"]]))
        del x
        t = g.whole(vocab - case["masked"], rows)
        t[3::31] = -1  # prompt or padding positions, which have no target
        st["targets"] = t
        if op == "tokens_loss":
            st["weight"] = torch.full((rows,), 1.0 / rows, device="cuda") * (0.5 + g.normal(rows).abs())
        if op == "tokens_bwd":
            xf = st["x"].float()
            m = xf.amax(dim=1)
            e = torch.exp(xf - m[:, None])
            s = e.sum(dim=1)
            st["stats"] = torch.stack([m, torch.log(s)], dim=1)
            y = torch.clamp(xf - m[:, None], min=-1e4)
            st["entropy"] = torch.log(s) - (e * y).sum(dim=1) / s
            st["dlogprob"] = g.normal(rows) / rows
            st["dentropy"] = 0.01 * g.normal(rows) / rows
        return st
    cols = case["cols"]
    dt, bt = TYPES[case["stream"]], TYPES[case["block"]]
    b = _rows((0.5 * g.activation(rows, cols)).to(bt))
    st["b"] = b
    if case["post"] != "none":
        st["post_gamma"] = 1.0 + 0.2 * g.normal(cols)
    if case["post"] == "layer":
        st["post_beta"] = 0.1 * g.normal(cols)
    st["pre_gamma"] = 1.0 + 0.2 * g.normal(cols)
    if case["pre"] == "layer":
        st["pre_beta"] = 0.1 * g.normal(cols)
    if case["gate"] == "vector":
        st["gate"] = 0.3 + 0.2 * g.normal(cols)
    if case["gate"] == "matrix":
        st["gate"] = _rows(torch.sigmoid(g.normal(rows, cols)).to(bt))
    x = g.activation(rows, cols)
    if op == "join":
        st["x"] = _rows(x.to(dt))
        return st
    # the backward pass has the new stream (x stands for it), the block's output and statistics
    st["r"] = _rows(x.to(dt))
    st["stats"] = torch.cat([_moments(b.float(), case["post"]),
                             _moments(st["r"].float(), case["pre"])], dim=1)
    st["dh"] = _rows(g.gradient(rows, cols).to(bt))
    st["dr"] = _rows(g.gradient(rows, cols).to(dt))
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _moments(z, kind):
    """(mean, reciprocal deviation) of each row as two columns; (0, 1) without a norm."""
    mean = z.mean(dim=1, keepdim=True) if kind == "layer" else torch.zeros_like(z[:, :1])
    if kind == "none":
        return torch.cat([mean, mean + 1.0], dim=1)
    d = z - mean
    return torch.cat([mean, 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + NORM_EPS)], dim=1)


# An 8-bit state's value is scale * F(code). F is a float with an exponent of 4 bits (bias
# 15, subnormals for exponent 0) and a mantissa of 3 bits (first moment, whose top bit is
# the sign) or 4; the largest F is TOP.
MANTISSA = {"m": 3, "v": 4}
TOP = {"m": 1.875, "v": 1.9375}
TINY = 2.0 ** -100  # a span whose largest magnitude is below it counts as zeros
# dither of element i at step t: (i * first + t * second) mod 2^32, of which the top bits are added
DITHER = {"m": (0x9E3779B9, 0xC13FA9A9), "v": (0xC13FA9A9, 0x9E3779B9)}


def _decode(codes, scale, which):
    code = codes.int()
    mag = code & 127 if which == "m" else code
    k = MANTISSA[which]
    e = mag >> k
    f = ((mag & ((1 << k) - 1)) + torch.where(e > 0, 1 << k, 0)).float()
    f = f * torch.exp2((e.clamp(min=1) - (15 + k)).float())
    if which == "m":
        f = torch.where(code > 127, -f, f)
    return f * scale.repeat_interleave(SPAN)[:code.numel()]


def _encode(x, which, t):
    """Codes and scales of x (fp32; non-negative for the second moment)."""
    n = x.numel()
    spans = (n + SPAN - 1) // SPAN
    a = torch.zeros(spans * SPAN, device=x.device)
    a[:n] = x.abs()
    a = a.view(spans, SPAN)
    top = a.amax(dim=1, keepdim=True)
    live = top >= TINY
    y = a * torch.where(live, TOP[which] / top, torch.zeros_like(top))
    first, second = DITHER[which]
    i = torch.arange(spans * SPAN, device=x.device).view(spans, SPAN)
    drop = 23 - MANTISSA[which]
    d = ((i * first + t * second) & 0xFFFFFFFF) >> (32 - drop)
    # places of the code, then those that the dither rounds away
    normal = y.view(torch.int32).long() - (112 << 23)
    places = torch.where(y < 2.0 ** -14, (y * 2.0 ** 37).long(), normal)
    code = (places + d) >> drop
    low = 0 if which == "m" else 1
    code = torch.where((a > 0) & live, code.clamp(low, 127 if which == "m" else 255), 0)
    code = code.view(-1)[:n]
    if which == "m":
        code = torch.where((x < 0) & (code > 0), code + 128, code)
    scale = torch.where(live, top / TOP[which], torch.zeros_like(top))
    return code.to(torch.uint8), scale[:, 0]


def _adam_plain(st, w, g, *state):
    c = st["case"]
    b1, b2 = _f32(BETA1), _f32(BETA2)
    gf = g.float()
    if c["clip"]:
        gf = gf * st["clip"]
    if c["state"] == "f32":
        m, v = state
        mf, vf = m, v
    else:
        m, ms, v, vs = state
        mf, vf = _decode(m, ms, "m"), _decode(v, vs, "v").square()
    mf = b1 * mf + (1.0 - b1) * gf
    vf = b2 * vf + (1.0 - b2) * gf * gf
    u = (mf / (1.0 - b1 ** STEP)) / (torch.sqrt(vf / (1.0 - b2 ** STEP)) + EPS)
    wf = w.float()
    w.copy_(wf - LR * (DECAY * wf + u))
    if c["state"] == "f32":
        m.copy_(mf)
        v.copy_(vf)
        return
    m8, s8 = _encode(mf, "m", STEP)
    m.copy_(m8)
    ms.copy_(s8)
    v8, s8 = _encode(torch.sqrt(vf), "v", STEP)
    v.copy_(v8)
    vs.copy_(s8)


def _read_plain(state, value):
    m, ms, v, vs = state
    value[0].copy_(_decode(m, ms, "m"))
    value[1].copy_(_decode(v, vs, "v").square())


def _adam_outputs(st):
    if st["case"]["state"] == "f32":
        return [st["w"], st["m"], st["v"]]
    return [st["w"], st["m_value"], st["v_value"]]


def _softmax_plain(st):
    x = st["x"].float()
    top = x.amax(dim=1, keepdim=True)
    y = x - top
    e = torch.exp(y)
    s = e.sum(dim=1, keepdim=True)
    t = st["targets"]
    there = t >= 0
    yt = torch.gather(y, 1, t.clamp(min=0)[:, None])[:, 0]
    logprob = torch.where(there, yt - torch.log(s)[:, 0], torch.zeros_like(yt))
    return top, y, e, s, there, logprob


def _norm_gradient(dy, z, gamma, stats, kind):
    """(gradient of the norm's input, normalised input)"""
    if kind == "none":
        return dy, z
    xh = (z - stats[:, :1]) * stats[:, 1:]
    q = dy * gamma
    d = q - xh * (q * xh).mean(dim=1, keepdim=True)
    if kind == "layer":
        d = d - q.mean(dim=1, keepdim=True)
    return d * stats[:, 1:], xh


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op == "adam":
        [_adam_plain(st, *item) for item in st["items"]]
        if c["state"] == "8bit":
            [_read_plain(*pair) for pair in zip(st["states"], st["values"])]
        return _adam_outputs(st)
    if op == "tokens":
        top, y, e, s, there, logprob = _softmax_plain(st)
        log_s = torch.log(s)
        entropy = (log_s - (e * y.clamp(min=-1e4)).sum(dim=1, keepdim=True) / s)[:, 0]
        out = [logprob, entropy, torch.cat([top, log_s], dim=1)]
        if c["top"]:
            # equal logits: the lowest token first
            _, order = torch.sort(y, dim=1, descending=True, stable=True)
            ids = order[:, :c["top"]]
            out += [torch.gather(y, 1, ids) - log_s, ids]
        return out
    if op == "tokens_loss":
        _, _, e, s, there, logprob = _softmax_plain(st)
        w = torch.where(there, st["weight"], torch.zeros_like(st["weight"]))[:, None]
        d = e * (w / s)
        d.scatter_add_(1, st["targets"].clamp(min=0)[:, None], -w)
        return [logprob, d.to(TYPES[c["dtype"]])]
    if op == "tokens_bwd":
        x, t = st["x"].float(), st["targets"]
        there = t >= 0
        logp = x - st["stats"][:, :1] - st["stats"][:, 1:]
        p = torch.exp(logp)
        dl = torch.where(there, st["dlogprob"], torch.zeros_like(st["dlogprob"]))[:, None]
        d = -p * (dl + st["dentropy"][:, None] * (logp.clamp(min=-1e4) + st["entropy"][:, None]))
        d.scatter_add_(1, t.clamp(min=0)[:, None], dl)
        return [d.to(TYPES[c["dtype"]])]
    dt, bt = TYPES[c["stream"]], TYPES[c["block"]]
    b = st["b"].float()
    gate = st["gate"].float() if "gate" in st else 1.0
    if op == "join":
        s1 = _moments(b, c["post"])
        u = b
        if c["post"] != "none":
            u = (b - s1[:, :1]) * s1[:, 1:] * st["post_gamma"]
        if c["post"] == "layer":
            u = u + st["post_beta"]
        r = X_SCALE * st["x"].float() + B_SCALE * (gate * u)
        s2 = _moments(r, c["pre"])
        h = (r - s2[:, :1]) * s2[:, 1:] * st["pre_gamma"]
        if c["pre"] == "layer":
            h = h + st["pre_beta"]
        return [r.to(dt), h.to(bt), torch.cat([s1, s2], dim=1)]
    dh = st["dh"].float()
    dr, xh2 = _norm_gradient(dh, st["r"].float(), st["pre_gamma"], st["stats"][:, 2:], c["pre"])
    dr = dr + st["dr"].float()
    du = B_SCALE * (gate * dr)
    db, xh1 = _norm_gradient(du, b, st.get("post_gamma"), st["stats"][:, :2], c["post"])
    out = [(X_SCALE * dr).to(dt), db.to(bt), (dh * xh2).sum(dim=0)]
    if c["pre"] == "layer":
        out.append(dh.sum(dim=0))
    if c["post"] != "none":
        out.append((du * xh1).sum(dim=0))
    if c["post"] == "layer":
        out.append(du.sum(dim=0))
    if c["gate"] != "none":
        u = xh1 if c["post"] == "none" else xh1 * st["post_gamma"]
        if c["post"] == "layer":
            u = u + st["post_beta"]
        dgate = B_SCALE * (dr * u)
        out.append(dgate.sum(dim=0) if c["gate"] == "vector" else dgate.to(bt))
    return out


def _run_own(st):
    import matrix_aware_optimizers_amd as mao
    c = st["case"]
    op = c["op"]
    if op == "adam":
        mao.adamw_step_many(st["items"], STEP, lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS,
                            weight_decay=DECAY, grad_scale=st.get("clip"))
        if c["state"] == "8bit":
            mao.adamw8_read(st["states"], out=st["values"])
        return _adam_outputs(st)
    if op == "tokens":
        r = mao.token_logprobs(st["x"], st["targets"], top=c["top"])
        out = [r.logprob, r.entropy, r.stats]
        return out + [r.top_logprobs, r.top_ids] if c["top"] else out
    if op == "tokens_loss":
        return list(mao.token_loss(st["x"], st["targets"], st["weight"]))
    if op == "tokens_bwd":
        return [mao.token_logprobs_backward(st["x"], st["targets"], st["stats"],
                                            dlogprob=st["dlogprob"], dentropy=st["dentropy"],
                                            entropy=st["entropy"])]
    post, pre = c["post"], c["pre"]
    kw = dict(gate=st.get("gate"), x_scale=X_SCALE, b_scale=B_SCALE, post=post,
              post_gamma=st.get("post_gamma"), post_beta=st.get("post_beta"), pre=pre,
              pre_gamma=st["pre_gamma"])
    if op == "join":
        return list(mao.residual_norm(st["x"], st["b"], pre_beta=st.get("pre_beta"), eps=NORM_EPS,
                                      **kw))
    g = mao.residual_norm_backward(st["dh"], st["dr"], st["b"], st["r"], st["stats"], **kw)
    out = [g.dX, g.dB, g.dpre_gamma]
    out += [g.dpre_beta] if pre == "layer" else []
    out += [g.dpost_gamma] if post != "none" else []
    out += [g.dpost_beta] if post == "layer" else []
    return out + ([g.dgate] if c["gate"] != "none" else [])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# work and exact results
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "adam":
        n = sum(_adam_sizes(case))
        b = n * (2 * size[case["w"]] + size[case["g"]])
        if case["state"] == "f32":
            return {"bytes": b + 16 * n, "flops": 16 * n}
        # codes and scales in and out, and the values that are read back
        return {"bytes": b + 4 * n + 16 * n // SPAN + 4 * n, "flops": 40 * n}
    r = case["rows"]
    if op.startswith("tokens"):
        v, es = case["vocab"], size[case["dtype"]]
        if op == "tokens":
            return {"bytes": r * (es * v + 8 + 16 + 12 * case["top"]), "flops": 5 * r * v}
        return {"bytes": r * (2 * es * v + 24), "flops": (6 if op == "tokens_loss" else 8) * r * v}
    c, xs, bs = case["cols"], size[case["stream"]], size[case["block"]]
    gate = bs * r * c if case["gate"] == "matrix" else 0
    if op == "join":
        return {"bytes": 2 * (xs + bs) * r * c + gate + 16 * r, "flops": 16 * r * c}
    return {"bytes": 3 * (xs + bs) * r * c + 2 * gate + 16 * r, "flops": 36 * r * c}


def _exact_float(codes, mantissa):
    """F of codes in 64 bits, by its exponent and mantissa."""
    e = torch.div(codes, 1 << mantissa, rounding_mode="floor").double()
    f = (codes % (1 << mantissa)).double() / (1 << mantissa)
    return torch.where(e == 0, f * 2.0 ** -14, torch.exp2(e - 15.0) * (1.0 + f))


def _exact_store(x, which):
    """What a state that is to hold x (64 bits) holds, span by span, in 64 bits."""
    n, mant = x.numel(), MANTISSA[which]
    pad = torch.nn.functional.pad(x.abs(), (0, -n % SPAN)).view(-1, SPAN)
    largest = pad.amax(dim=1, keepdim=True)
    scale = largest / (2.0 - 0.5 ** mant)
    y = pad / scale
    # within its binade: the step below y, and y's place between two steps
    e = torch.floor(torch.log2(y)).clamp(min=-14.0)
    place = (y * torch.exp2(-e) - 1.0) * (1 << mant)
    first, second = DITHER[which]
    i = torch.arange(pad.numel(), device=x.device).view(-1, SPAN)
    low = 32 - 23 + mant  # bits of the dither that are cut off
    d = torch.div((i * first + STEP * second) % (1 << 32), 1 << low, rounding_mode="floor")
    code = (e + 15.0) * (1 << mant) + torch.floor(place + d.double() * 0.5 ** (23 - mant))
    code = code.clamp(0 if which == "m" else 1, (16 << mant) - 1)
    code = torch.where(pad > 0, code, torch.zeros_like(code)).long()
    v = (_exact_float(code, mant) * scale).view(-1)[:n]
    return v * torch.sign(x)


def _exact_adam(st, out, i, item):
    c = st["case"]
    b1, b2, lr, wd, eps = (_f32(x) for x in (BETA1, BETA2, LR, DECAY, EPS))
    w, g = item[0].double(), item[1].double()
    if c["clip"]:
        g = g * st["clip"].double()
    if c["state"] == "f32":
        m, v = item[2].double(), item[3].double()
    else:
        span = torch.arange(w.numel(), device=w.device) // SPAN
        k = item[2].long()
        m = _exact_float(k % 128, 3) * torch.where(k > 127, -1.0, 1.0) * item[3].double()[span]
        v = (_exact_float(item[4].long(), 4) * item[5].double()[span]).square()
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g.square()
    u = m / (1.0 - b1 ** STEP) / ((v / (1.0 - b2 ** STEP)).sqrt() + eps)
    if c["state"] == "8bit":
        m, v = _exact_store(m, "m"), _exact_store(v.sqrt(), "v").square()
    at = slice(i, i + w.numel())
    out[0][at], out[1][at], out[2][at] = w - lr * (wd * w + u), m, v


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "adam":
        # storage between the tensors keeps what it held
        first = [st["w"], st["m"], st["v"]] if case["state"] == "f32" else [st["w"], st["m_value"], st["v_value"]]
        out = [t.double() for t in first]
        for item in st["items"]:
            _exact_adam(st, out, item[0].storage_offset(), item)
        return out
    if op.startswith("tokens"):
        parts = []
        rows = max(1, (1 << 27) // case["vocab"])
        for a in range(0, case["rows"], rows):
            parts.append(_exact_tokens(st, slice(a, a + rows)))
        return [None if p[0] is None else torch.cat(p) for p in zip(*parts)]
    b, pre, post = st["b"].double(), case["pre"], case["post"]
    gate = st["gate"].double() if "gate" in st else torch.ones((), dtype=torch.float64, device="cuda")
    xs, bs = _f32(X_SCALE), _f32(B_SCALE)
    n = case["cols"]
    g1 = st["post_gamma"].double() if post != "none" else None
    g2 = st["pre_gamma"].double()

    def normed(z, kind):
        if kind == "none":
            return z, torch.zeros_like(z[:, 0]), torch.ones_like(z[:, 0])
        mean = z.sum(1) / n if kind == "layer" else torch.zeros_like(z[:, 0])
        d = z - mean[:, None]
        rstd = (d.square().sum(1) / n + _f32(NORM_EPS)).rsqrt()
        return d * rstd[:, None], mean, rstd

    if op == "join":
        u, m1, r1 = normed(b, post)
        if post != "none":
            u = u * g1
        if post == "layer":
            u = u + st["post_beta"].double()
        r = xs * st["x"].double() + bs * gate * u
        h, m2, r2 = normed(r, pre)
        h = h * g2
        if pre == "layer":
            h = h + st["pre_beta"].double()
        return [r, h, torch.stack([m1, r1, m2, r2], dim=1)]
    dh, s = st["dh"].double(), st["stats"].double()

    def back(dy, z, mean, rstd, kind):
        xh = (z - mean[:, None]) * rstd[:, None]
        d = dy - xh * ((dy * xh).sum(1, keepdim=True) / n)
        if kind == "layer":
            d = d - dy.sum(1, keepdim=True) / n
        return d * rstd[:, None], xh

    dr, xh2 = back(dh * g2, st["r"].double(), s[:, 2], s[:, 3], pre)
    dr = dr + st["dr"].double()
    du = bs * gate * dr
    if post == "none":
        db, xh1 = du, b
    else:
        db, xh1 = back(du * g1, b, s[:, 0], s[:, 1], post)
    out = [xs * dr, db, (dh * xh2).sum(0)]
    out += [dh.sum(0)] if pre == "layer" else []
    out += [(du * xh1).sum(0)] if post != "none" else []
    out += [du.sum(0)] if post == "layer" else []
    if "gate" in st:
        u = xh1 if post == "none" else xh1 * g1
        u = u + st["post_beta"].double() if post == "layer" else u
        out.append((bs * dr * u).sum(0) if case["gate"] == "vector" else bs * dr * u)
    return out


def _exact_tokens(st, at):
    c = st["case"]
    x, t = st["x"][at].double(), st["targets"][at]
    line = torch.arange(t.numel(), device="cuda")
    has = t >= 0
    hit = t.clamp(min=0)
    if c["op"] == "tokens_bwd":
        s = st["stats"][at].double()
        lp = (x - s[:, :1]) - s[:, 1:]
        p = lp.exp()
        dl = st["dlogprob"][at].double() * has
        # p log p has the limit 0
        plogp = torch.where(p > 0, p * lp, torch.zeros_like(p))
        de = st["dentropy"][at].double()[:, None]
        d = -p * dl[:, None] - de * (plogp + p * st["entropy"][at].double()[:, None])
        d[line, hit] += dl
        return [d]
    big = x.amax(1)
    e = (x - big[:, None]).exp()
    s = e.sum(1)
    logprob = torch.where(has, x[line, hit] - big - s.log(), torch.zeros_like(s))
    if c["op"] == "tokens_loss":
        w = st["weight"][at].double() * has
        d = e * (w / s)[:, None]
        d[line, hit] -= w
        return [logprob, d]
    p = e / s[:, None]
    entropy = -torch.where(p > 0, p * p.log(), torch.zeros_like(p)).sum(1)
    out = [logprob, entropy, torch.stack([big, s.log()], dim=1)]
    if c["top"]:
        # value and place in one order: larger values first, then lower places
        ids = torch.sort(-st["x"][at].double(), dim=1, stable=True).indices[:, :c["top"]]
        out += [torch.gather(x, 1, ids) - (big + s.log())[:, None], ids]
    return out
