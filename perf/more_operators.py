"""Cases of a recurrent frame model's operators and of its answers' logits.

Four operators, each in the forms a program calls:

* gated linear recurrence over time: `recur` (forward; also the form of single
  frames with a kept state) and `recur_train` (forward, then the gradients of
  all inputs and of the first state);
* root-mean-square norm with the residual's addition: `rms` (forward),
  `rms_train` (forward, then the gradients of the input and the weight) and
  `rms_8bit` (forward, e4m3 values with a scale per row);
* distillation from a teacher's top log probabilities: `distill` (the loss)
  and `distill_train` (the loss, then the logits' gradient);
* penalties for repeated tokens, biases and masks of allowed tokens on logits:
  `adjust`.

`run` computes them from elementary torch operations in 32 bits (`own` is
false) or calls this package (`own` is true).  `exact` is the definition in
64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ---- cases -------------------------------------------------------------------

def _recur(op, dtype, batch, time, channels, gate, state, ragged):
    return dict(op=op, dtype=dtype, batch=batch, time=time, channels=channels, gate=gate, state=state,
                ragged=ragged)


def _rms(op, dtype, rows, width, residual):
    return dict(op=op, dtype=dtype, rows=rows, width=width, residual=residual)


def _distill(op, dtype, rows, vocab, top, temperature, rest):
    return dict(op=op, dtype=dtype, rows=rows, vocab=vocab, top=top, temperature=temperature, rest=rest)


def _adjust(dtype, rows, vocab, history, biases, masked):
    return dict(op="adjust", dtype=dtype, rows=rows, vocab=vocab, history=history, biases=biases, masked=masked)


def listed():
    return [
        # one frame of 8 streams with their states
        dict(_recur("recur", "bf16", 8, 1, 1024, True, True, False), name="recur decode 8x1x1024 bf16"),
        # an encoder's forward pass over 8 utterances of up to 1501 positions
        dict(_recur("recur", "bf16", 8, 1501, 1024, True, False, True), name="recur encoder 8x1501x1024 bf16"),
        # one long recording that goes on from a kept state
        dict(_recur("recur", "f16", 1, 100003, 256, True, True, False), name="recur long 1x100003x256 f16"),
        # a short utterance trained in float32 at the example model's width
        dict(_recur("recur_train", "f32", 1, 101, 128, True, False, False), name="recur train 1x101x128 f32"),
        # a training batch of 16 utterances
        dict(_recur("recur_train", "bf16", 16, 1501, 2048, True, False, True), name="recur train 16x1501x2048 bf16"),
        # one decoding step of 8 streams: the norm in front of each layer, with the residual
        dict(_rms("rms", "bf16", 8, 1024, True), name="rms decode 8x1024 bf16"),
        # a training batch of 64 utterances, 1501 positions each
        dict(_rms("rms_train", "bf16", 96064, 1024, True), name="rms train 96064x1024 bf16"),
        # the same layer's input for 8-bit products, 8 x 3002 positions of a wide model
        dict(_rms("rms_8bit", "bf16", 24016, 4096, True), name="rms 8 bits 24016x4096 bf16"),
        # frame-wise character scores of 8 x 3001 mel frames from a teacher's best 8, trained in float32
        dict(_distill("distill_train", "f32", 24008, 129, 8, 2.0, False), name="distill train 24008x129 f32"),
        # a training batch of transcripts over a subword vocabulary, the teacher's best 20 and the rest's mass
        dict(_distill("distill_train", "bf16", 4096, 32000, 20, 1.0, True), name="distill train 4096x32000 bf16"),
        # one decoding step of 8 streams: 448 tokens so far, a few biases
        dict(_adjust("bf16", 8, 50001, 448, 16, False), name="adjust decode 8x50001 bf16"),
        # a decoding step of many requests with long histories, biases and a grammar's mask
        dict(_adjust("f16", 256, 131072, 4000, 300, True), name="adjust decode 256x131072 f16"),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case of the listed ranges: from one row or frame to a training batch,
    every type, odd and ragged sizes."""
    most = {}
    for c in listed():
        kind = c["op"].split("_")[0]
        most[kind] = max(most.get(kind, 0), work(c)["bytes"])
    while True:
        op = rng.choice(["recur", "recur_train", "recur_train", "rms", "rms_train", "rms_8bit", "distill",
                         "distill_train", "distill_train", "adjust", "adjust"])
        dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
        if op.startswith("recur"):
            time = 1 if op == "recur" and rng.random() < 0.3 else _spread(rng, 2, 100003)
            case = _recur(op, dtype, _spread(rng, 1, 64), time, _spread(rng, 24, 4096), rng.random() < 0.7,
                          rng.random() < 0.5, rng.random() < 0.5)
        elif op.startswith("rms"):
            case = _rms(op, dtype if op != "rms_8bit" else rng.choice(["bf16", "f16"]), _spread(rng, 1, 96064),
                        _spread(rng, 40, 8192), rng.random() < 0.6)
        elif op.startswith("distill"):
            vocab = _spread(rng, 29, 131072)
            rest = rng.random() < 0.5
            case = _distill(op, dtype, _spread(rng, 1, 24008), vocab, min(vocab // 2, rng.choice([1, 5, 8, 20, 64])),
                            1.0 if rest else rng.choice([1.0, 2.0, 4.0]), rest)
        else:
            case = _adjust(dtype, _spread(rng, 1, 512), _spread(rng, 29, 131072), _spread(rng, 1, 16384),
                           rng.choice([0, 16, 300]), rng.random() < 0.5)
        if work(case)["bytes"] <= most[op.split("_")[0]]:
            return case


def _lengths(case):
    """Valid frames of each entry: between half and all of them if ragged."""
    t, b = case["time"], case["batch"]
    return [max(1, t - (i * t) // (2 * b)) if case["ragged"] else t for i in range(b)]


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    train = op.endswith("_train")
    if op.startswith("recur"):
        valid, whole = sum(_lengths(case)) * case["channels"], case["batch"] * case["time"] * case["channels"]
        ins = 3 if case["gate"] else 2
        states = 4 * case["batch"] * case["channels"] * ((2 if case["state"] else 1) + (2 if train and case["state"] else 0))
        # x, forget, gate in, y out; in training dy in and the inputs' gradients out, of all frames
        n = ins * valid + whole + (valid + ins * whole if train else 0)
        return {"bytes": n * size + states, "flops": valid * (50 if train else 16)}
    if op.startswith("rms"):
        n, res = case["rows"] * case["width"], case["residual"]
        if op == "rms_8bit":
            return {"bytes": n * (size * (3 if res else 1) + 1) + case["rows"] * 4 + case["width"] * size,
                    "flops": n * 8}
        # x and the residual in, y and the sum out; in training dy and the sum's gradient in, dx out
        ends = (4 if res else 2) + ((3 if res else 2) if train else 0)
        return {"bytes": n * size * ends + case["width"] * size * (2 if train else 1),
                "flops": n * (14 if train else 5)}
    if op.startswith("distill"):
        n = case["rows"] * case["vocab"]
        return {"bytes": n * size * (2 if train else 1) + case["rows"] * (8 + 12 * case["top"]),
                "flops": n * (8 if train else 4)}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * size * 2 + (n // 8 if case["masked"] else 0) +
            case["rows"] * (8 * case["history"] + 12 * case["biases"] + 12), "flops": n * 5}


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).add_(mean).to(dtype)

    op = case["op"]
    s = dict(case=case)
    if op.startswith("recur"):
        b, t, c = case["batch"], case["time"], case["channels"]
        # one projection's output: x, forget (memories of a few to some hundred frames), gate
        parts = 3 if case["gate"] else 2
        p = normal(b, t, parts * c)
        p[..., c:2 * c].mul_(1.5).add_(3.0)
        s["x"], s["forget"] = p[..., :c], p[..., c:2 * c]
        s["gate"] = p[..., 2 * c:] if case["gate"] else None
        s["state"] = normal(b, c, dtype=torch.float32) if case["state"] else None
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        if op == "recur_train":
            s["dy"] = normal(b, t, c)
            s["dstate"] = normal(b, c, dtype=torch.float32) if case["state"] else None
        return s
    if op.startswith("rms"):
        n, w = case["rows"], case["width"]
        s["x"] = normal(n, w)
        s["residual"] = normal(n, w, std=3.0) if case["residual"] else None
        s["w"] = normal(w, std=0.2, mean=1.0)
        if op == "rms_train":
            s["dy"] = normal(n, w)
            s["dsum"] = normal(n, w, std=0.5) if case["residual"] else None
        return s
    n, v = case["rows"], case["vocab"]
    s["x"] = normal(n, v, std=2.5)
    if op.startswith("distill"):
        # the teacher: the same rows with some noise, its best entries kept as token_logprobs gives them
        ids, lps = [], []
        step = max(1, (1 << 27) // v)
        for i in range(0, n, step):
            x = s["x"][i:i + step].float()
            y = torch.log_softmax(x + torch.randn(x.shape, generator=g, device="cuda"), -1)
            top = y.topk(case["top"], -1)
            ids.append(top.indices)
            lps.append(top.values)
        s["ids"], s["lps"] = torch.cat(ids), torch.cat(lps)
        if op == "distill_train":
            s["dloss"] = torch.rand(n, generator=g, device="cuda").add_(0.5)
        return s
    # tokens so far, frequent ones again and again; rows of different lengths
    h = case["history"]
    s["history"] = torch.rand(n, h, generator=g, device="cuda").pow_(3).mul_(v).long().clamp_(max=v - 1)
    s["lengths"] = torch.randint(h // 2, h + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    s["repetition"] = torch.rand(n, generator=g, device="cuda").mul_(0.3).add_(1.0)
    s["frequency"] = torch.rand(n, generator=g, device="cuda").mul_(0.2)
    s["presence"] = torch.rand(n, generator=g, device="cuda").mul_(0.5)
    s["bias_ids"] = s["bias"] = s["allowed"] = None
    if case["biases"]:
        s["bias_ids"] = torch.randint(-1, v, (n, case["biases"]), generator=g, device="cuda")
        s["bias"] = normal(n, case["biases"], std=4.0, dtype=torch.float32)
    if case["masked"]:
        words = (v + 31) // 32
        s["allowed"] = torch.randint(-(1 << 31), 1 << 31, (n, words), generator=g, device="cuda").int()
    return s


# ---- one pass ----------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op.startswith("recur"):
        return (_recur_own if own else _recur_plain)(s, op == "recur_train")
    if op == "rms_8bit":
        return (_rms_8bit_own if own else _rms_8bit_plain)(s)
    if op.startswith("rms"):
        return (_rms_own if own else _rms_plain)(s, op == "rms_train")
    if op.startswith("distill"):
        return (_distill_own if own else _distill_plain)(s, op == "distill_train")
    return (_adjust_own if own else _adjust_plain)(s)


def _recur_own(s, train):
    from stft_mel_spectrogram_amd import (gated_recurrence, gated_recurrence_backward, gated_recurrence_forward)
    args = (s["x"], s["forget"], s["gate"], s["state"])
    if not train:
        return gated_recurrence(*args, lengths=s["lengths"])
    y, last, saved = gated_recurrence_forward(*args, lengths=s["lengths"])
    grads = gated_recurrence_backward(s["dy"], *args, saved, lengths=s["lengths"], grad_state=s["dstate"])
    return (y, last, *(d for d in grads if d is not None))


def _scan(a, u, first):
    """h[t] = a[t] h[t - 1] + u[t] along axis 1, h[-1] = first, by doubling:
    each step joins every position with the one `n` before it."""
    u[:, 0] += a[:, 0] * first
    n = 1
    while n < a.shape[1]:
        u = torch.cat((u[:, :n], u[:, n:] + a[:, n:] * u[:, :-n]), 1)
        a = torch.cat((a[:, :n], a[:, n:] * a[:, :-n]), 1)
        n *= 2
    return u


def _recur_plain(s, train):
    x, f = s["x"].float(), s["forget"].float()
    b, t, c = x.shape
    dt, dev = s["x"].dtype, s["x"].device
    first = s["state"] if s["state"] is not None else torch.zeros(b, c, device=dev)
    seen = None
    if s["lengths"] is not None:
        seen = (torch.arange(t, device=dev) < s["lengths"][:, None])[..., None]
    a = 1.0 / (1.0 + (-f).exp())
    rest = 1.0 / (1.0 + f.exp())
    u = rest * x
    if seen is not None:
        a, u = torch.where(seen, a, torch.ones_like(a)), torch.where(seen, u, torch.zeros_like(u))
    h = _scan(a, u.clone(), first)
    last = h[:, -1].clone()
    o = h
    if s["gate"] is not None:
        g = s["gate"].float()
        sg = 1.0 / (1.0 + (-g).exp())
        o = h * (g * sg)
    if seen is not None:
        o = torch.where(seen, o, torch.zeros_like(o))
    y = o.to(dt)
    if not train:
        return y, last
    dy = s["dy"].float()
    if seen is not None:
        dy = torch.where(seen, dy, torch.zeros_like(dy))
    e = dy * (g * sg) if s["gate"] is not None else dy.clone()
    end = s["dstate"] if s["dstate"] is not None else torch.zeros(b, c, device=dev)
    # d[t] = e[t] + a[t + 1] d[t + 1], from the end
    after = torch.cat((torch.ones_like(a[:, :1]), a[:, 1:].flip(1)), 1)
    d = _scan(after, e.flip(1), end).flip(1)
    before = torch.cat((first[:, None], h[:, :-1]), 1)
    dx, df = rest * d, d * (before - x) * (a * rest)
    if seen is not None:
        dx, df = torch.where(seen, dx, torch.zeros_like(dx)), torch.where(seen, df, torch.zeros_like(df))
    out = [y, last, dx.to(dt), df.to(dt)]
    if s["gate"] is not None:
        out.append((dy * h * (sg * (1.0 + g * (1.0 - sg)))).to(dt))
    if s["state"] is not None:
        out.append(a[:, 0] * d[:, 0])
    return tuple(out)


def _rms_own(s, train):
    from stft_mel_spectrogram_amd import rms_norm, rms_norm_backward, rms_norm_forward
    if not train:
        return rms_norm(s["x"], s["w"], s["residual"], EPS)
    y, total, rstd = rms_norm_forward(s["x"], s["w"], s["residual"], EPS)
    dx, dw = rms_norm_backward(s["dy"], total, s["w"], rstd, s["dsum"])
    return (y, total, dx, dw) if s["residual"] is not None else (y, dx, dw)


def _rms_plain(s, train):
    dt = s["x"].dtype
    total = s["x"]
    if s["residual"] is not None:
        total = (s["x"].float() + s["residual"].float()).to(dt)
    z, w = total.float(), s["w"].float()
    rstd = 1.0 / (z.square().mean(-1, keepdim=True) + EPS).sqrt()
    y = (z * rstd * w).to(dt)
    outs = (y, total) if s["residual"] is not None else (y,)
    if not train:
        return outs if len(outs) > 1 else y
    dy = s["dy"].float()
    u = z * rstd
    g = dy * w
    dx = rstd * (g - u * (g * u).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return (*outs, dx.to(dt), (dy * u).sum(0).to(dt))


def _rms_8bit_own(s):
    from stft_mel_spectrogram_amd import rms_norm_quantized
    return rms_norm_quantized(s["x"], s["w"], s["residual"], EPS)


def _rms_8bit_plain(s):
    dt = s["x"].dtype
    total = s["x"]
    if s["residual"] is not None:
        total = (s["x"].float() + s["residual"].float()).to(dt)
    z = total.float()
    y = z / (z.square().mean(-1, keepdim=True) + EPS).sqrt() * s["w"].float()
    most = y.abs().amax(-1, keepdim=True)
    scale = torch.where(most == 0, torch.ones_like(most), most / 448.0)
    q = (y / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return (q, scale.squeeze(-1), total) if s["residual"] is not None else (q, scale.squeeze(-1))


def _distill_own(s, train):
    from stft_mel_spectrogram_amd import (topk_distillation, topk_distillation_backward,
                                          topk_distillation_forward)
    c = s["case"]
    how = dict(temperature=c["temperature"], rest=c["rest"])
    if not train:
        return topk_distillation(s["x"], s["ids"], s["lps"], **how)
    loss, stats = topk_distillation_forward(s["x"], s["ids"], s["lps"], **how)
    return loss, topk_distillation_backward(s["dloss"], s["x"], s["ids"], s["lps"], stats, **how)


def _distill_plain(s, train):
    tau, ids = s["case"]["temperature"], s["ids"]
    x = s["x"].float() / tau
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    z = e.sum(-1, keepdim=True)
    lse = m + z.log()
    if s["case"]["rest"]:
        lq = s["lps"]
        q = lq.exp()
        # what the teacher leaves for all others: a difference near 0
        q_rest = (1.0 - s["lps"].double().exp().sum(-1, keepdim=True)).clamp(min=0).float()
        others = e.scatter(-1, ids, 0.0)
        z_rest = others.sum(-1, keepdim=True)
        loss_rest = torch.where(q_rest > 0, q_rest * (q_rest.log() - (z_rest / z).log()), torch.zeros_like(q_rest))
        loss = (q * (lq - (x.gather(-1, ids) - lse))).sum(-1) + loss_rest.squeeze(-1)
    else:
        t = s["lps"] / tau
        t = t - t.amax(-1, keepdim=True)
        lq = t - t.exp().sum(-1, keepdim=True).log()
        q = lq.exp()
        loss = (q * (lq - (x.gather(-1, ids) - lse))).sum(-1) * (tau * tau)
    if not train:
        return loss
    dx = e / z
    if s["case"]["rest"]:
        dx = dx * (q.sum(-1, keepdim=True) + q_rest) - others * (q_rest / z_rest)
    dx.scatter_add_(-1, ids, -q)
    dx *= s["dloss"][:, None] * tau
    return loss, dx.to(s["x"].dtype)


def _adjust_own(s):
    from stft_mel_spectrogram_amd import adjust_logits
    return adjust_logits(s["x"], s["history"], s["lengths"], repetition=s["repetition"], frequency=s["frequency"],
                         presence=s["presence"], bias_ids=s["bias_ids"], bias=s["bias"], allowed=s["allowed"])


def _adjust_plain(s):
    x = s["x"].float()
    n, v = x.shape
    dev = x.device
    ones = (torch.arange(s["history"].shape[1], device=dev) < s["lengths"][:, None]).float()
    count = torch.zeros_like(x).scatter_add_(-1, s["history"], ones)
    rep = s["repetition"][:, None]
    x = torch.where(count > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias_ids"] is not None:
        real = s["bias_ids"] >= 0
        x.scatter_add_(-1, s["bias_ids"].clamp(min=0), torch.where(real, s["bias"], torch.zeros_like(s["bias"])))
    if s["allowed"] is not None:
        bits = (s["allowed"][..., None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
        x = torch.where(bits.view(n, -1)[:, :v] != 0, x, torch.full_like(x, -math.inf))
    return x.to(s["x"].dtype)


# ---- the definition in 64 bits -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("recur"):
        return _recur_exact(s, op == "recur_train")
    if op.startswith("rms"):
        return _rms_exact(s, op)
    if op.startswith("distill"):
        return _distill_exact(s, op == "distill_train")
    return _adjust_exact(s)


def _recur_exact(s, train):
    """Frame by frame, forward and back."""
    c = s["case"]
    if c["time"] > 20011 or (train and c["batch"] * c["time"] * c["channels"] > 1 << 28):
        return None
    b, t, n = s["x"].shape
    f64 = dict(dtype=torch.float64, device=s["x"].device)
    lengths = torch.tensor(_lengths(c), device=s["x"].device)
    h = s["state"].double() if s["state"] is not None else torch.zeros(b, n, **f64)
    y = torch.zeros(b, t, n, **f64)
    hs = [h]
    for i in range(t):
        on = (i < lengths)[:, None]
        a = torch.sigmoid(s["forget"][:, i].double())
        h = torch.where(on, a * h + (1 - a) * s["x"][:, i].double(), h)
        o = h * torch.nn.functional.silu(s["gate"][:, i].double()) if c["gate"] else h
        y[:, i] = o * on
        if train:
            hs.append(h)
    if not train:
        return y, h
    last = h
    d = s["dstate"].double() if s["dstate"] is not None else torch.zeros(b, n, **f64)
    dx, df, dg = torch.zeros_like(y), torch.zeros_like(y), torch.zeros_like(y)
    for i in reversed(range(t)):
        on = (i < lengths)[:, None]
        a, x, dy = (torch.sigmoid(s["forget"][:, i].double()), s["x"][:, i].double(), s["dy"][:, i].double())
        if c["gate"]:
            g = s["gate"][:, i].double()
            sg = torch.sigmoid(g)
            dg[:, i] = dy * hs[i + 1] * (sg + g * sg * (1 - sg)) * on
            dy = dy * g * sg
        dh = d + dy * on
        dx[:, i] = (1 - a) * dh * on
        df[:, i] = dh * (hs[i] - x) * a * (1 - a) * on
        d = torch.where(on, a * dh, dh)
    return (y, last, dx, df, *((dg,) if c["gate"] else ()), *((d,) if c["state"] else ()))


def _rms_exact(s, op):
    ys, sums, dxs, scales = [], [], [], []
    w = s["w"].double()
    dw = torch.zeros_like(w)
    step = max(1, (1 << 25) // w.numel())
    for i in range(0, s["x"].shape[0], step):
        z = s["x"][i:i + step]
        if s["residual"] is not None:
            # the sum is kept in the rows' own type, and that is what is normed
            z = (z.double() + s["residual"][i:i + step].double()).to(z.dtype)
            sums.append(z)
        z = z.double()
        r = ((z * z).sum(1, keepdim=True) / w.numel() + EPS) ** -0.5
        y = z * r * w
        if op == "rms_8bit":
            scale = y.abs().max(1, keepdim=True).values / 448
            scales.append(scale[:, 0])
            y = y / scale
        ys.append(y)
        if op == "rms_train":
            dy = s["dy"][i:i + step].double()
            dw += (dy * z * r).sum(0)
            g = dy * w
            dx = r * g - z * r ** 3 * ((g * z).sum(1, keepdim=True) / w.numel())
            dxs.append(dx if s["dsum"] is None else dx + s["dsum"][i:i + step].double())
    out = [torch.cat(ys)]
    if scales:
        out.append(torch.cat(scales))
    if sums:
        out.append(torch.cat(sums).double())
    if dxs:
        out += [torch.cat(dxs), dw]
    return tuple(out) if len(out) > 1 else out[0]


def _distill_exact(s, train):
    tau, rest = s["case"]["temperature"], s["case"]["rest"]
    losses, dxs = [], []
    step = max(1, (1 << 24) // s["case"]["vocab"])
    for i in range(0, s["x"].shape[0], step):
        lp = torch.log_softmax(s["x"][i:i + step].double() / tau, 1)
        ids = s["ids"][i:i + step]
        t = s["lps"][i:i + step].double()
        lq = t if rest else torch.log_softmax(t / tau, 1)
        q = lq.exp()
        loss = (q * (lq - lp.gather(1, ids))).sum(1)
        target = torch.zeros_like(lp).scatter_add_(1, ids, q)
        if rest:
            left = (1 - q.sum(1, keepdim=True)).clamp(min=0)
            r = torch.log_softmax(lp.scatter(1, ids, -math.inf), 1)          # within the others
            lp_rest = torch.logsumexp(lp.scatter(1, ids, -math.inf), 1, keepdim=True)
            loss = loss + torch.where(left > 0, left * (left.log() - lp_rest), torch.zeros_like(left))[:, 0]
            target = target + left * r.exp()
        losses.append(tau ** 2 * loss)
        if train:
            whole = target.sum(1, keepdim=True)
            dxs.append(tau * s["dloss"][i:i + step].double()[:, None] * (lp.exp() * whole - target))
    return (torch.cat(losses), torch.cat(dxs)) if train else torch.cat(losses)


def _adjust_exact(s):
    n, v = s["x"].shape
    out = []
    for r in range(n):
        x = s["x"][r].double()
        seen = torch.bincount(s["history"][r, :int(s["lengths"][r])], minlength=v)
        rep = s["repetition"][r].double()
        x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
        x = x - s["frequency"][r].double() * seen - s["presence"][r].double() * (seen > 0)
        if s["bias_ids"] is not None:
            keep = s["bias_ids"][r] >= 0
            x = x.index_add(0, s["bias_ids"][r][keep], s["bias"][r][keep].double())
        if s["allowed"] is not None:
            words = s["allowed"][r].long() & 0xFFFFFFFF
            i = torch.arange(v, device=x.device)
            x = x.masked_fill((words[i // 32] >> (i % 32)) & 1 == 0, -math.inf)
        out.append(x)
    return torch.stack(out)
