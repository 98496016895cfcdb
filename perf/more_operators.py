"""The operators around the mixers of a served model's decode step: their cases, plain forms and calls.

Four operators, in the order in which a step with drafted tokens runs them:

  norm     residual addition and root-mean-square norm, over the row or over groups of its channels; bf16,
           fp32 or int8 out (one scale per row and group)
  linear   a projection with 4-bit weights, a scale (and a zero) per group of a row's weights; activations in
           bf16 or in int8 as the norm gives them
  probs    probabilities of logits, each row at its temperature (0: the first largest one)
  verify   drafted tokens against the target's probabilities from given random numbers: how many are kept,
           and the token after them

With ``own`` false ``run`` computes them from elementary torch operations (fp32; fp64 where a cumulative sum
meets a border); with ``own`` true it makes the calls a user makes of the package.  ``exact`` evaluates the
definitions in fp64.  int8 rows are returned as the values they stand for, in bf16.
"""
import math

import torch

own = False

DEV = "cuda"
_TYPES = dict(bf16=torch.bfloat16, f32=torch.float32, int8=torch.int8)
_SIZE = dict(bf16=2, f32=4, int8=1)


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one request's token between two blocks of a 1536-wide model: latency
        dict(name="norm_step_b1", op="norm", rows=1, width=1536, groups=1, x="bf16", residual="bf16", out="bf16"),
        # a decode batch before a projection with 8-bit activations
        dict(name="norm_step_b64_int8", op="norm", rows=64, width=7168, groups=1, x="bf16", residual="bf16", out="int8"),
        # the grouped norm after an SSD mixer of 80 heads of 64: fp32 rows of four prompts, no residual
        dict(name="norm_groups_b4_l2048", op="norm", rows=4 * 2048, width=5120, groups=8, x="f32", residual="", out="bf16"),
        # a 16384-token prompt of a 7168-wide model with its residual stream in fp32
        dict(name="norm_prompt_l16384", op="norm", rows=16384, width=7168, groups=1, x="bf16", residual="f32", out="bf16"),
        # one request's output projection of a small model: latency
        dict(name="linear_b1_small", op="linear", rows=1, inner=1536, outer=768, group=64, x="bf16", blocks=1, zeros=False,
             scales="bf16", out="bf16"),
        # one request's input projection of a 4096-wide model
        dict(name="linear_b1", op="linear", rows=1, inner=4096, outer=16384, group=128, x="bf16", blocks=1, zeros=False,
             scales="bf16", out="bf16"),
        # eight requests' output projection, 8-bit activations, small groups with zeros
        dict(name="linear_b8_int8", op="linear", rows=8, inner=8192, outer=4096, group=32, x="int8", blocks=1, zeros=True,
             scales="f32", out="f32"),
        # logits of a batch of blocks of drafted tokens over a vocabulary of an odd size
        dict(name="linear_b64_vocab", op="linear", rows=64, inner=2560, outer=50021, group=128, x="bf16", blocks=1, zeros=True,
             scales="bf16", out="f32"),
        # one request's block of four drafted tokens and the token after it
        dict(name="probs_b5", op="probs", rows=5, vocab=50021, x="bf16", temperature="one"),
        # a batch of 64 such blocks of eight, a temperature for each row, some greedy
        dict(name="probs_b512", op="probs", rows=512, vocab=131072, x="bf16", temperature="rows"),
        # one request's four drafted tokens
        dict(name="verify_b1", op="verify", batch=1, drafts=4, vocab=50021, draft_probs=True, ragged=False),
        # a batch with blocks of up to seven drafted tokens
        dict(name="verify_b64", op="verify", batch=64, drafts=7, vocab=131072, draft_probs=True, ragged=True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "probs", "verify"])
    if op == "norm":
        groups = rng.choice([1, 1, 1, 2, 4, 8, 16])
        width = 8 * groups * _logint(rng, max(1, 64 // (8 * groups)), 16384 // (8 * groups))
        return dict(op=op, rows=_logint(rng, 1, min(16384, 110_000_000 // width)), width=width, groups=groups,
                    x=rng.choice(["bf16", "bf16", "f32"]), residual=rng.choice(["", "bf16", "f32"]),
                    out=rng.choice(["bf16", "f32", "int8"]))
    if op == "linear":
        group, rows = rng.choice([32, 64, 128, 128]), _logint(rng, 1, 64)
        inner = group * _logint(rng, 1, 16384 // group)
        outer = _logint(rng, 64, min(50021, max(64, 120_000_000 // inner)))
        x, n = rng.choice(["bf16", "bf16", "int8"]), inner // group
        blocks = rng.choice([b for b in (1, 2, 4, 8) if n % b == 0]) if x == "int8" else 1
        return dict(op=op, rows=rows, inner=inner, outer=outer, group=group, x=x, blocks=blocks, zeros=rng.random() < 0.5,
                    scales=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
    vocab = rng.choice([_logint(rng, 1000, 200_000), 8 * _logint(rng, 125, 25_000)])
    if op == "probs":
        return dict(op=op, rows=_logint(rng, 1, min(512, 60_000_000 // vocab)), vocab=vocab, x=rng.choice(["bf16", "f32"]),
                    temperature=rng.choice(["one", "rows"]))
    drafts = rng.choice([0, 1, 2, 3, 4, 5, 7, 11])
    return dict(op=op, batch=_logint(rng, 1, min(128, 60_000_000 // (vocab * (drafts + 1)))), drafts=drafts, vocab=vocab,
                draft_probs=drafts > 0 and rng.random() < 0.7, ragged=rng.random() < 0.5)


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        per = _SIZE[case["x"]] + _SIZE[case["out"]] + (2 * _SIZE[case["residual"]] if case["residual"] else 0)
        return dict(bytes=n * per + 4 * case["width"] + (4 * case["rows"] * case["groups"] if case["out"] == "int8" else 0),
                    flops=6 * n)
    if case["op"] == "linear":
        m, k, n = case["rows"], case["inner"], case["outer"]
        per_group = _SIZE[case["scales"]] + (1 if case["zeros"] else 0)
        return dict(bytes=n * k // 2 + n * (k // case["group"]) * per_group + m * k * _SIZE[case["x"]] + m * n * _SIZE[case["out"]],
                    flops=2 * m * n * k)
    if case["op"] == "probs":
        n = case["rows"] * case["vocab"]
        return dict(bytes=n * (_SIZE[case["x"]] + 4), flops=5 * n)
    # the row that the token after the kept ones comes from: the target's, and the drafts' where one was refused
    n = case["batch"] * case["vocab"]
    return dict(bytes=n * (8 if case["draft_probs"] else 4), flops=3 * n)


# ------------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _activations(rows, width, dtype, g):
    """N(0, 1) with a gain per channel: some channels stand out, as in a residual stream."""
    x = torch.randn(rows, width, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(width, generator=g, device=DEV))
    return x.to(dtype)


def _rows_of(n, k, dtype, multiple):
    """Rows [n, k] whose stride is a multiple of 16 bytes."""
    return torch.zeros(n, -(-k // multiple) * multiple, dtype=dtype, device=DEV)[:, :k]


def _weights(case, g):
    """Weights of a projection quantised to 4 bits by groups: codes [outer, inner / 2] (even places in the low
    half), scales and zeros [outer, inner / group]."""
    n, k, group = case["outer"], case["inner"], case["group"]
    groups = k // group
    codes = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)
    scales = _rows_of(n, groups, _TYPES[case["scales"]], 8)
    zeros = _rows_of(n, groups, torch.uint8, 16) if case["zeros"] else None
    step = max(1, (1 << 26) // k)
    for a in range(0, n, step):
        w = torch.randn(min(step, n - a), groups, group, generator=g, device=DEV) / k ** 0.5
        if zeros is None:
            s = w.abs().amax(-1) / 7.0
            s = s.to(scales.dtype)
            c = torch.round(w / s.float()[..., None]).clamp_(-7, 7) + 8
        else:
            low, high = w.amin(-1), w.amax(-1)
            s = ((high - low) / 15.0).to(scales.dtype)
            z = torch.round(-low / s.float()).clamp_(0, 15)
            c = (torch.round(w / s.float()[..., None]) + z[..., None]).clamp_(0, 15)
            zeros[a:a + step] = z.to(torch.uint8)
        scales[a:a + step] = s
        c = c.to(torch.uint8).view(c.shape[0], k // 2, 2)
        codes[a:a + step] = c[..., 0] | (c[..., 1] << 4)
    return codes, scales, zeros


def _logits(rows, vocab, g, sharp=2.5):
    return sharp * torch.randn(rows, vocab, generator=g, device=DEV)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        s["x"] = _activations(case["rows"], case["width"], _TYPES[case["x"]], g)
        s["residual"] = 3 * _activations(case["rows"], case["width"], _TYPES[case["residual"]], g) if case["residual"] else None
        s["weight"] = 1.0 + 0.2 * torch.randn(case["width"], generator=g, device=DEV)
        s["eps"] = 1e-5
        return s
    if case["op"] == "linear":
        x = _activations(case["rows"], case["inner"], torch.float32, g)
        if case["x"] == "int8":
            x = x.view(case["rows"], case["blocks"], -1)
            s["x_scale"] = (x.abs().amax(-1) / 127.0).contiguous()
            x = torch.round(x / s["x_scale"][..., None]).clamp_(-127, 127).view(case["rows"], -1)
        else:
            s["x_scale"] = None
        s["x"] = x.to(_TYPES[case["x"]])
        s["codes"], s["scales"], s["zeros"] = _weights(case, g)
        return s
    if case["op"] == "probs":
        s["logits"] = _logits(case["rows"], case["vocab"], g).to(_TYPES[case["x"]])
        s["temperature"] = None
        if case["temperature"] == "rows":
            t = 0.3 + 1.2 * torch.rand(case["rows"], generator=g, device=DEV)
            s["temperature"] = torch.where(torch.rand(case["rows"], generator=g, device=DEV) < 0.2, 0.0, t)
        return s
    b, t, v = case["batch"], case["drafts"], case["vocab"]
    # a draft model that is near the target's, and tokens drawn from it
    target = _logits(b * (t + 1), v, g).view(b, t + 1, v)
    s["draft_probs"] = None
    if case["draft_probs"]:
        noise = _logits(b * t, v, g, 1.0).view(b, t, v)
        s["draft_probs"] = torch.softmax(target[:, :t] + noise, -1)
        draft = torch.multinomial(s["draft_probs"].view(b * t, v), 1, generator=g)
    else:
        draft = (target[:, :t] * 3).reshape(b * t, v).argmax(-1) if t else torch.zeros(0, device=DEV)
    s["target_probs"] = torch.softmax(target if case["draft_probs"] else 4 * target, -1)
    s["draft"] = draft.view(b, t).to(torch.int32)
    s["u"] = torch.rand(b, t + 1, generator=g, device=DEV)
    s["n_draft"] = torch.randint(0, t + 1, (b,), generator=g, device=DEV, dtype=torch.int32) if case["ragged"] else None
    return s


# ------------------------------------------------------------------------------ the plain forms
def _plain_norm(s):
    case = s["case"]
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    y = r.view(case["rows"], case["groups"], -1)
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"])
    y = y * s["weight"].view(1, case["groups"], -1)
    outs = []
    if case["out"] == "int8":
        amax = y.abs().amax(-1)
        inv = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
        scale = amax / 127.0
        codes = torch.round(y * inv[..., None]).clamp_(-127, 127).to(torch.int8)
        outs += [_values(codes, scale), scale]
    else:
        outs += [y.view(case["rows"], -1).to(_TYPES[case["out"]])]
    if s["residual"] is not None:
        outs += [r.to(s["residual"].dtype)]
    return tuple(outs)


def _values(codes, scale):
    """What int8 codes [rows, groups, channels] stand for, in bf16."""
    out = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
    return torch.mul(codes, scale[..., None], out=out).view(codes.shape[0], -1)


def _plain_linear(s):
    case = s["case"]
    n, k, group = case["outer"], case["inner"], case["group"]
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = (x.view(x.shape[0], case["blocks"], -1) * s["x_scale"][..., None]).view(x.shape[0], k)
    c = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).view(n, k // group, group).float()
    c = c - (8.0 if s["zeros"] is None else s["zeros"].float()[..., None])
    w = (c * s["scales"].float()[..., None]).view(n, k)
    return torch.matmul(x, w.t()).to(_TYPES[case["out"]])


def _first_largest(x):
    """One-hot rows: the lowest index of each row's maximum."""
    index = torch.arange(x.shape[1], device=x.device)
    first = torch.where(x == x.amax(-1, keepdim=True), index, x.shape[1]).amin(-1, keepdim=True)
    return (index == first).to(x.dtype)


def _plain_probs(s):
    x = s["logits"].float()
    d = x - x.amax(-1, keepdim=True)
    if s["temperature"] is None:
        e = torch.exp(d)
        return e / e.sum(-1, keepdim=True)
    t = s["temperature"][:, None]
    greedy = t <= 2.0 ** -100
    e = torch.exp(d / torch.where(greedy, 1.0, t))
    return torch.where(greedy, _first_largest(x), e / e.sum(-1, keepdim=True))


def _plain_verify(s):
    p, q, u = s["target_probs"], s["draft_probs"], s["u"]
    b, t = s["draft"].shape
    at = torch.arange(b, device=DEV)
    count = torch.full((b,), t, device=DEV) if s["n_draft"] is None else s["n_draft"].long()
    draft = s["draft"].long()
    kept = torch.zeros(b, dtype=torch.long, device=DEV)
    if t:
        pd = p[:, :t].gather(2, draft[..., None])[..., 0].double()
        qd = torch.ones_like(pd) if q is None else q.gather(2, draft[..., None])[..., 0].double()
        take = (u[:, :t].double() * qd < pd) & (torch.arange(t, device=DEV) < count[:, None])
        kept = take.to(torch.int32).cumprod(1).sum(1)
    row = p[at, kept].double()
    if t:
        refused = kept < count
        where = kept.clamp(max=t - 1)
        if q is None:
            off = torch.zeros_like(row).scatter_(1, draft[at, where][:, None], 1.0)
        else:
            off = q[at, where].double()
        left = (row - off).clamp_(min=0.0)
        row = torch.where((refused & (left.sum(1) > 0))[:, None], left, row)
    c = row.cumsum(1)
    token = (c <= u[:, t:].double() * c[:, -1:]).sum(1)
    place = torch.arange(t + 1, device=DEV)
    tokens = torch.where(place == kept[:, None], token[:, None], -1)
    if t:
        tokens[:, :t] = torch.where(place[:t] < kept[:, None], draft, tokens[:, :t])
    return tokens.to(torch.int32), kept.to(torch.int32)


# ------------------------------------------------------------------------------ the framework's calls
def _own(s):
    from selective_state_space_prefill_gb300 import binding as ssm
    case = s["case"]
    if case["op"] == "norm":
        out, residual, scale = ssm.norm_rms(s["x"], s["weight"], s["residual"], eps=s["eps"], n_groups=case["groups"],
                                            out_dtype=_TYPES[case["out"]])
        if scale is not None:
            out = (_values(out.view(case["rows"], case["groups"], -1), scale), scale)
        else:
            out = (out,)
        return out if residual is None else out + (residual,)
    if case["op"] == "linear":
        return ssm.w4_linear(s["x"], s["codes"], s["scales"], s["zeros"], x_scale=s["x_scale"], out_dtype=_TYPES[case["out"]])
    if case["op"] == "probs":
        return ssm.spec_probs(s["logits"], s["temperature"])
    return ssm.spec_verify(s["draft"], s["target_probs"], s["u"], s["draft_probs"], s["n_draft"])


def run(state):
    if own:
        return _own(state)
    return dict(norm=_plain_norm, linear=_plain_linear, probs=_plain_probs, verify=_plain_verify)[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        size = case["width"] // case["groups"]
        parts, scales, sums = [], [], []
        for a in range(0, case["rows"], 2048):
            r = s["x"][a:a + 2048].to(f64)
            if s["residual"] is not None:
                r = r + s["residual"][a:a + 2048].to(f64)
                sums.append(r)
            columns, steps = [], []
            for j in range(0, case["width"], size):
                part = r[:, j:j + size]
                power = torch.linalg.vector_norm(part, dim=1, keepdim=True) ** 2 / size
                y = part / torch.sqrt(power + s["eps"]) * s["weight"][j:j + size].to(f64)
                if case["out"] == "int8":
                    step = y.abs().max(1, keepdim=True).values / 127
                    y = torch.where(step > 0, torch.round(y / step) * step, 0.0)
                    steps.append(step)
                columns.append(y)
            parts.append(torch.cat(columns, 1))
            if steps:
                scales.append(torch.cat(steps, 1))
        return tuple(torch.cat(v) for v in (parts, scales, sums) if v)
    if case["op"] == "linear":
        m, k, n = case["rows"], case["inner"], case["outer"]
        place = torch.arange(k, device=DEV)
        x = s["x"].to(f64)
        if s["x_scale"] is not None:
            x = x * s["x_scale"].to(f64)[:, place // (k // case["blocks"])]
        out = torch.empty(m, n, dtype=f64, device=DEV)
        step = max(1, (1 << 25) // k)
        for a in range(0, n, step):
            byte = s["codes"][a:a + step].to(torch.int32)[:, place // 2]
            code = (byte // torch.where(place % 2 == 1, 16, 1)) % 16
            zero = 8 if s["zeros"] is None else s["zeros"][a:a + step].to(torch.int32)[:, place // case["group"]]
            w = (code - zero).to(f64) * s["scales"][a:a + step].to(f64)[:, place // case["group"]]
            out[:, a:a + step] = torch.einsum("mk,nk->mn", x, w)
        return out
    if case["op"] == "probs":
        out = torch.empty(s["logits"].shape, dtype=f64, device=DEV)
        for r in range(case["rows"]):
            x = s["logits"][r].to(f64)
            t = 1.0 if s["temperature"] is None else float(s["temperature"][r])
            if t <= 2.0 ** -100:
                out[r] = 0.0
                out[r, int((x == x.max()).nonzero()[0])] = 1.0
            else:
                out[r] = torch.exp(x / t - torch.logsumexp(x / t, 0))
        return out
    b, t = s["draft"].shape
    tokens = torch.full((b, t + 1), -1, dtype=torch.int32)
    counts = torch.zeros(b, dtype=torch.int32)
    for i in range(b):
        n = t if s["n_draft"] is None else int(s["n_draft"][i])
        kept = 0
        while kept < n:
            d = int(s["draft"][i, kept])
            q = 1.0 if s["draft_probs"] is None else float(s["draft_probs"][i, kept, d])
            if not float(s["u"][i, kept]) * q < float(s["target_probs"][i, kept, d]):
                break
            tokens[i, kept] = d
            kept += 1
        mass = s["target_probs"][i, kept].to(f64)
        if kept < n:
            if s["draft_probs"] is None:
                less = mass.clone()
                less[int(s["draft"][i, kept])] = 0.0
            else:
                less = torch.relu(mass - s["draft_probs"][i, kept].to(f64))
            mass = less if float(less.sum()) > 0 else mass
        total = torch.cumsum(mass, 0)
        border = float(s["u"][i, t]) * float(total[-1])
        tokens[i, kept] = int(torch.searchsorted(total, border, right=True))
        counts[i] = kept
    return tokens, counts
