"""The attention operators of a hybrid SSM/attention layer: their cases, their plain forms and their calls.

Four operators, as a serving program chains them around an attention block:

  append   rotary positions on q and k; k and v written into the paged cache (bf16, or int8 with one
           scale per token and head, quantised as written); an int8 cache is read back, so that the
           state comes out as the values it stands for
  read     pages back to packed rows (dequantised): the context of a prompt's next chunk
  prefill  causal attention over packed prompts of different lengths, grouped heads
  decode   one token per request over the paged cache

With ``own`` false ``run`` computes them from elementary torch operations in fp32; with ``own`` true it
makes the calls a user makes of the package.  ``exact`` evaluates the definitions in fp64.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # a single request's next token into a small int8 cache: the latency of one step
        dict(name="append_step_b1", op="append", batch=1, new=1, longest=201, ragged=0, q_heads=32, kv_heads=8,
             dim=128, rot=128, interleaved=False, factor=1.0, cache="int8", page=16),
        # a full decode batch, bf16 cache, half of each head rotated in interleaved pairs
        dict(name="append_step_b256", op="append", batch=256, new=1, longest=256, ragged=11, q_heads=64, kv_heads=8,
             dim=128, rot=64, interleaved=True, factor=1.0, cache="bf16", page=64),
        # a long prompt of a 7168-wide layer written to an int8 cache, positions interpolated 4x
        dict(name="append_prompt_l16384", op="append", batch=1, new=16384, longest=16384, ragged=0, q_heads=56,
             kv_heads=8, dim=128, rot=128, interleaved=False, factor=4.0, cache="int8", page=64),
        # the context of one short chat turn, before its next chunk
        dict(name="read_l777", op="read", batch=1, longest=777, ragged=0, kv_heads=8, dim=128, cache="int8",
             page=64, out="bf16"),
        # the contexts of a batch of long conversations
        dict(name="read_b16_ragged", op="read", batch=16, longest=16384, ragged=5, kv_heads=8, dim=128, cache="int8",
             page=64, out="bf16"),
        # one short prompt, 1536 wide, heads not shared: latency to the first token
        dict(name="prefill_l77", op="prefill", batch=1, longest=77, ragged=0, context=0, q_heads=24, kv_heads=24,
             dim=64, lse=False),
        # a packed batch of prompts of different lengths
        dict(name="prefill_b8_ragged", op="prefill", batch=8, longest=4096, ragged=3, context=0, q_heads=32,
             kv_heads=8, dim=128, lse=False),
        # two prompts' next chunk of 2048 tokens over long contexts read back from the cache
        dict(name="prefill_chunk_2048", op="prefill", batch=2, longest=2048, ragged=0, context=12289, q_heads=56,
             kv_heads=8, dim=128, lse=True),
        # one whole prompt of 16384 tokens, 7168 wide: the largest
        dict(name="prefill_l16384", op="prefill", batch=1, longest=16384, ragged=0, context=0, q_heads=56, kv_heads=8,
             dim=128, lse=False),
        # one chat request's next token: latency
        dict(name="decode_b1_l4096", op="decode", batch=1, longest=4096, ragged=0, q_heads=32, kv_heads=8, dim=128,
             cache="int8", page=16, lse=False),
        # a serving batch of ragged contexts over an int8 cache
        dict(name="decode_b64_ragged", op="decode", batch=64, longest=8192, ragged=7, q_heads=64, kv_heads=8, dim=128,
             cache="int8", page=64, lse=True),
        # few requests with very long contexts, bf16 cache: the split over the long axis
        dict(name="decode_b4_l65536", op="decode", batch=4, longest=65536, ragged=0, q_heads=56, kv_heads=8, dim=128,
             cache="bf16", page=64, lse=False),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    while True:
        case = _draw(rng)
        if case.get("q_heads", 0) * case["dim"] != 3072 and 3072 not in case.values():
            return case


def _draw(rng):
    op = rng.choice(["append", "read", "prefill", "decode"])
    dim = rng.choice([64, 64, 80, 96, 128, 128, 128])
    kv = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12])
    while kv * group > 64:
        group = rng.choice([1, 2, 3, 4])
    ragged = rng.choice([0, rng.randrange(1, 1 << 20)])
    cache = rng.choice(["int8", "bf16"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "append":
        batch = _logint(rng, 1, 256)
        new = 1 if rng.random() < 0.5 else _logint(rng, 1, max(1, 16384 // batch))
        longest = new + _logint(rng, 1, max(1, 32768 // batch))
        rot = rng.choice([dim, dim, dim // 2 // 8 * 8])
        return dict(op=op, batch=batch, new=new, longest=longest, ragged=ragged, q_heads=kv * group, kv_heads=kv,
                    dim=dim, rot=rot, interleaved=rng.random() < 0.5, factor=rng.choice([1.0, 2.0, 8.0]),
                    cache=cache, page=page)
    if op == "read":
        batch = _logint(rng, 1, 64)
        return dict(op=op, batch=batch, longest=_logint(rng, 1, 131072 // batch), ragged=ragged, kv_heads=min(kv, 8), dim=dim,
                    cache=cache, page=page, out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "prefill":
        batch = _logint(rng, 1, 16)
        longest = _logint(rng, 1, 16000 // batch)
        context = rng.choice([0, 0, _logint(rng, 1, 16384 // batch)])
        while context and longest * (longest / 2 + context) * batch > 1.3e8:
            context //= 2
        heads = kv * group if longest * (longest / 2 + context) * batch < 3e7 else kv * max(1, min(group, 32 // kv))
        return dict(op=op, batch=batch, longest=longest, ragged=ragged, context=context, q_heads=heads, kv_heads=kv,
                    dim=dim, lse=rng.random() < 0.5)
    batch = _logint(rng, 1, 256)
    return dict(op=op, batch=batch, longest=_logint(rng, 1, 262144 // batch), ragged=ragged, q_heads=min(kv, 8) * group,
                kv_heads=min(kv, 8), dim=dim, cache=cache, page=page, lse=rng.random() < 0.5)


def _lengths(case):
    """Tokens of each sequence (after this pass): all the longest, or spread log-uniformly below it."""
    n, hi = case["batch"], case["longest"]
    if not case["ragged"]:
        return [hi] * n
    r = random.Random(case["ragged"])
    lo = max(case.get("new", 1), hi // 16, 1)
    return [hi] + [_logint(r, lo, hi) for _ in range(n - 1)]


def _cache_bytes_per_token(case):
    return case["kv_heads"] * (2 * case["dim"] + 8 if case["cache"] == "int8" else 4 * case["dim"])


def work(case):
    lens = _lengths(case)
    if case["op"] == "append":
        t = case["batch"] * case["new"]
        d, hq, hk = case["dim"], case["q_heads"], case["kv_heads"]
        # q in and out, k in and (rotated) out, v in, cache rows, cos/sin rows
        b = t * (4 * d * hq + 4 * d * hk + 2 * d * hk + _cache_bytes_per_token(case) + 4 * case["rot"])
        f = t * (3 * case["rot"] * (hq + hk) + 4 * d * hk)
        if case["cache"] == "int8":       # read back: rows and scales in, bf16 rows out
            b += sum(lens) * (_cache_bytes_per_token(case) + 4 * d * hk)
            f += sum(lens) * 2 * d * hk
        return dict(bytes=b, flops=f)
    if case["op"] == "read":
        e = 4 if case["out"] == "f32" else 2
        return dict(bytes=sum(lens) * (_cache_bytes_per_token(case) + 2 * e * case["dim"] * case["kv_heads"]),
                    flops=sum(lens) * 2 * case["dim"] * case["kv_heads"])
    if case["op"] == "prefill":
        pairs = sum(n * (n + 1) // 2 + n * case["context"] for n in lens)
        tq, tk = sum(lens), sum(n + case["context"] for n in lens)
        return dict(bytes=2 * case["dim"] * (2 * tq * case["q_heads"] + 2 * tk * case["kv_heads"]),
                    flops=4 * case["dim"] * case["q_heads"] * pairs)
    return dict(bytes=sum(lens) * _cache_bytes_per_token(case) + 4 * case["batch"] * case["q_heads"] * case["dim"],
                flops=4 * case["dim"] * case["q_heads"] * sum(lens))


# ------------------------------------------------------------------------------ inputs
def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=DEV)


def _heads(t, heads, dim, g, spread):
    """[t, heads, dim] ~ N(0, 1) with a gain per channel (keys have channels that stand out)."""
    x = torch.randn(t, heads, dim, generator=g, device=DEV)
    if spread:
        x *= torch.exp(spread * torch.randn(heads, dim, generator=g, device=DEV))
    return x.to(torch.bfloat16)


def _pages(case, lens, g):
    """Page table [batch, most pages] (a shuffled pool, as after some serving) and the pool's size."""
    page = case["page"]
    most = max(-(-n // page) for n in lens)
    need = [-(-n // page) for n in lens]
    pool = sum(need)
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(lens), most, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool


def _quantise(x):
    """(codes, scales) of x [..., dim] fp32: one scale per row, absmax / 127, ties to even."""
    amax = x.abs().amax(-1)
    inv = torch.where(amax > 0, 127.0 / amax, torch.zeros_like(amax))
    return torch.round(x * inv[..., None]).clamp_(-127, 127).to(torch.int8), amax / 127.0


def _cache(case, pool, g, spread):
    """One cache [pool, kv_heads, page, dim] and, for int8, its scales [pool, kv_heads, page]."""
    shape = (pool, case["kv_heads"], case["page"], case["dim"])
    gain = torch.exp(spread * torch.randn(case["kv_heads"], 1, case["dim"], generator=g, device=DEV))
    rows = torch.empty(shape, device=DEV, dtype=torch.int8 if case["cache"] == "int8" else torch.bfloat16)
    scales = torch.empty(shape[:3], device=DEV) if case["cache"] == "int8" else None
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for p in range(0, pool, step):
        x = torch.randn((min(step, pool - p),) + shape[1:], generator=g, device=DEV) * gain
        if scales is None:
            rows[p:p + step] = x.to(torch.bfloat16)
        else:
            rows[p:p + step], scales[p:p + step] = _quantise(x)
    return rows, scales


def _rope_table(case, n_pos):
    """cos and sin [n_pos, rot / 2] in fp32, angles in fp64, positions interpolated by the factor."""
    half = case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half) / case["factor"]
    angle = torch.arange(n_pos, device=DEV, dtype=torch.float64)[:, None] * freq
    return torch.cos(angle).float().contiguous(), torch.sin(angle).float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    lens = _lengths(case)
    s = dict(case=case, lens=lens, scale=case["dim"] ** -0.5)
    if case["op"] == "append":
        b, new, d, hq, hk = case["batch"], case["new"], case["dim"], case["q_heads"], case["kv_heads"]
        qkv = _heads(b * new, hq + 2 * hk, d, g, 0.3)        # the rows of one fused projection
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["table"], pool = _pages(case, lens, g)
        s["k_cache"], s["k_scale"] = _cache(case, pool, g, 0.3)
        s["v_cache"], s["v_scale"] = _cache(case, pool, g, 0.0)
        pos = torch.cat([torch.arange(n - new, n, device=DEV) for n in lens])
        row = torch.arange(b, device=DEV).repeat_interleave(new)
        page = s["table"][row, pos // case["page"]].long()
        s["pos"] = pos.to(torch.int32)
        s["slots"] = (page * case["page"] + pos % case["page"]).to(torch.int32)
        s["cos"], s["sin"] = _rope_table(case, max(lens))
        s["cu"] = _cu(lens)
        s["total"] = sum(lens)
        return s
    if case["op"] == "prefill":
        hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
        klens = [n + case["context"] for n in lens]
        s["q"] = _heads(sum(lens), hq, d, g, 0.2)
        s["k"] = _heads(sum(klens), hk, d, g, 0.2)
        # without a context v is still in the rows of the fused projection, with one it was read back
        s["v"] = _heads(sum(klens), hk, d, g, 0.0) if case["context"] else _heads(sum(klens), 2 * hk, d, g, 0.0)[:, hk:]
        s["cu_q"], s["cu_k"] = _cu(lens), _cu(klens)
        s["klens"] = klens
        return s
    s["table"], pool = _pages(case, lens, g)
    s["k_cache"], s["k_scale"] = _cache(case, pool, g, 0.2)
    s["v_cache"], s["v_scale"] = _cache(case, pool, g, 0.0)
    s["cu"], s["total"] = _cu(lens), sum(lens)
    if case["op"] == "decode":
        s["q"] = _heads(case["batch"], case["q_heads"], case["dim"], g, 0.2)
        s["seq"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        if own:
            from selective_state_space_prefill_gb300 import binding as ssm
            n = ssm.attn_decode_workspace_bytes(case["batch"], case["q_heads"], case["kv_heads"], case["dim"], max(lens))
            s["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------ the plain forms
def _rotate(x, cos, sin, interleaved):
    """x [t, heads, dim] fp32, cos/sin [t, half]."""
    half = cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2] = a * c - b * s
        y[..., 1:2 * half:2] = b * c + a * s
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half] = a * c - b * s
        y[..., half:2 * half] = b * c + a * s
    return y


def _rows(s, name, b, n, out_dtype):
    """Tokens 0..n-1 of sequence b from cache `name`, [n, kv_heads, dim]."""
    page = s["case"]["page"]
    ids = s["table"][b, :-(-n // page)].long()
    x = s[name + "_cache"][ids].float()
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][ids][..., None]
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:n].to(out_dtype)


def _plain_read(s, out_dtype):
    k = torch.cat([_rows(s, "k", b, n, out_dtype) for b, n in enumerate(s["lens"])])
    v = torch.cat([_rows(s, "v", b, n, out_dtype) for b, n in enumerate(s["lens"])])
    return k, v


def _plain_append(s):
    case = s["case"]
    cos, sin = s["cos"][s["pos"].long()], s["sin"][s["pos"].long()]
    q = _rotate(s["q"].float(), cos, sin, case["interleaved"]).to(torch.bfloat16)
    k = _rotate(s["k"].float(), cos, sin, case["interleaved"])
    v = s["v"].float()
    slot = s["slots"].long()
    page, off = slot // case["page"], slot % case["page"]
    for name, x in (("k", k), ("v", v)):
        if case["cache"] == "int8":
            codes, scale = _quantise(x)
            s[name + "_cache"][page, :, off] = codes
            s[name + "_scale"][page, :, off] = scale
        else:
            s[name + "_cache"][page, :, off] = x.to(torch.bfloat16)
    return q, k.to(torch.bfloat16)


def _plain_prefill(s):
    case = s["case"]
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    group = hq // hk
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(s["q"].shape[:2], device=DEV)
    aq = ak = 0
    for n, nk in zip(s["lens"], s["klens"]):
        q = s["q"][aq:aq + n].float().view(n, hk, group, d).permute(1, 2, 0, 3)         # [hk, group, n, d]
        k, v = (x[ak:ak + nk].float().transpose(0, 1) for x in (s["k"], s["v"]))        # [hk, nk, d]
        rows = max(1, min(n, (1 << 28) // (nk * group)))                                # of a head at a time
        heads = max(1, min(hk, (1 << 28) // (nk * group * rows)))
        for h in range(0, hk, heads):
            for r in range(0, n, rows):
                e = min(n, r + rows)
                see = e + nk - n                             # keys that the last of these rows sees
                qh = q[h:h + heads, :, r:e].reshape(-1, group * (e - r), d)
                x = torch.matmul(qh, k[h:h + heads, :see].transpose(1, 2)) * s["scale"]
                i = torch.arange(r, e, device=DEV).repeat(group)[:, None]
                x = torch.where(torch.arange(see, device=DEV)[None, :] <= i + (nk - n), x, float("-inf"))
                m = x.amax(-1, keepdim=True)
                p = torch.exp(x - m)
                total = p.sum(-1, keepdim=True)
                o = torch.matmul(p, v[h:h + heads, :see]) / total
                own_heads = slice(h * group, (h * group) + o.shape[0] * group)
                out[aq + r:aq + e, own_heads] = o.view(-1, e - r, d).transpose(0, 1).to(torch.bfloat16)
                lse[aq + r:aq + e, own_heads] = (m + torch.log(total)).view(-1, e - r).transpose(0, 1)
        aq, ak = aq + n, ak + nk
    return (out, lse) if case["lse"] else (out,)


def _plain_decode(s):
    case = s["case"]
    hk = case["kv_heads"]
    group = case["q_heads"] // hk
    out = torch.empty(s["q"].shape, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(s["q"].shape[:2], device=DEV)
    for b, n in enumerate(s["lens"]):
        q = s["q"][b].float().view(hk, group, -1)
        k = _rows(s, "k", b, n, torch.float32).permute(1, 0, 2)
        v = _rows(s, "v", b, n, torch.float32).permute(1, 0, 2)
        x = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        total = p.sum(-1, keepdim=True)
        out[b] = (torch.matmul(p, v) / total).reshape(case["q_heads"], -1).to(torch.bfloat16)
        lse[b] = (m + torch.log(total)).reshape(-1)
    return (out, lse) if case["lse"] else (out,)


# ------------------------------------------------------------------------------ the framework's calls
def _own(s):
    from selective_state_space_prefill_gb300 import binding as ssm
    case = s["case"]
    if case["op"] == "append":
        q, k = ssm.attn_append(s["q"], s["k"], s["v"], s["pos"], s["cos"], s["sin"], s["k_cache"], s["v_cache"],
                               s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                               interleaved=case["interleaved"], k_out=True)
        if case["cache"] == "bf16":
            return q, k, s["k_cache"], s["v_cache"]
        kr, vr = ssm.attn_cache_read(s["k_cache"], s["v_cache"], s["table"], s["cu"], s["total"],
                                     k_scale=s["k_scale"], v_scale=s["v_scale"])
        return q, k, kr, vr
    if case["op"] == "read":
        return ssm.attn_cache_read(s["k_cache"], s["v_cache"], s["table"], s["cu"], s["total"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"],
                                   out_dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
    if case["op"] == "prefill":
        out, lse = ssm.attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], case["longest"], scale=s["scale"],
                                    lse=case["lse"])
    else:
        out, lse = ssm.attn_decode_step(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq"], case["longest"],
                                        k_scale=s["k_scale"], v_scale=s["v_scale"], scale=s["scale"],
                                        lse=case["lse"], workspace=s["workspace"])
    return (out, lse) if case["lse"] else (out,)


def run(state):
    if own:
        return _own(state)
    case = state["case"]
    if case["op"] == "append":
        q, k = _plain_append(state)
        if case["cache"] == "bf16":
            return q, k, state["k_cache"], state["v_cache"]
        return (q, k) + _plain_read(state, torch.bfloat16)
    if case["op"] == "read":
        return _plain_read(state, torch.float32 if case["out"] == "f32" else torch.bfloat16)
    return _plain_prefill(state) if case["op"] == "prefill" else _plain_decode(state)


# ------------------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    if work(case)["flops"] > 2e12 or work(case)["bytes"] > 6e9:
        return None
    s = prepare(case, seed)
    f64 = torch.float64

    def values(name, b, n):
        """Sequence b's first n rows of a cache, token by token through the page table."""
        t = torch.arange(n, device=DEV)
        pg, off = s["table"][b].long()[t // case["page"]], t % case["page"]
        x = s[name + "_cache"][pg, :, off].to(f64)
        return x if s[name + "_scale"] is None else x * s[name + "_scale"][pg, :, off].to(f64)[:, :, None]

    if case["op"] == "read":
        return (torch.cat([values("k", b, n) for b, n in enumerate(s["lens"])]),
                torch.cat([values("v", b, n) for b, n in enumerate(s["lens"])]))
    if case["op"] == "append":
        half = case["rot"] // 2
        i = torch.arange(case["dim"], device=DEV)
        turned = i < 2 * half
        partner = (i ^ 1) if case["interleaved"] else torch.where(i < half, i + half, i - half)
        partner = torch.where(turned, partner, i)
        pair = (i // 2) if case["interleaved"] else i % max(half, 1)
        sign = torch.where((i % 2 == 0) if case["interleaved"] else (i < half), -1.0, 1.0).to(f64)
        pair = torch.where(turned, pair, torch.zeros_like(pair))
        pos = s["pos"].long()
        c = torch.where(turned, s["cos"][pos][:, pair].to(f64), 1.0)[:, None]
        w = torch.where(turned, s["sin"][pos][:, pair].to(f64) * sign, 0.0)[:, None]
        q, k = (x.to(f64) * c + x.to(f64)[:, :, partner] * w for x in (s["q"], s["k"]))
        v = s["v"].to(f64)
        if case["cache"] == "bf16":
            caches = []
            for name, x in (("k", k), ("v", v)):
                full = s[name + "_cache"].to(f64)
                full[s["slots"].long() // case["page"], :, s["slots"].long() % case["page"]] = x
                caches.append(full)
            return (q, k, *caches)
        outs = []
        for name, x in (("k", k), ("v", v)):
            whole = [values(name, b, n) for b, n in enumerate(s["lens"])]
            step = x.abs().amax(-1, keepdim=True) / 127.0
            held = torch.where(step > 0, torch.round(x / step) * step, 0.0)
            for b, n in enumerate(s["lens"]):
                whole[b][n - case["new"]:] = held[b * case["new"]:(b + 1) * case["new"]]
            outs.append(torch.cat(whole))
        return (q, k, *outs)

    group = case["q_heads"] // case["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=f64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=f64, device=DEV)
    aq = ak = 0
    for b, n in enumerate(s["lens"]):
        if case["op"] == "decode":
            nq, nk = 1, n
            k, v = values("k", b, n), values("v", b, n)
        else:
            nq, nk = n, s["klens"][b]
            k, v = s["k"][ak:ak + nk].to(f64), s["v"][ak:ak + nk].to(f64)
            ak += nk
        for h in range(case["q_heads"]):
            kh, vh = k[:, h // group], v[:, h // group]
            for r in range(0, nq, 2048):
                e = min(nq, r + 2048)
                x = s["q"][aq + r:aq + e, h].to(f64) @ kh.T * s["scale"]
                future = torch.arange(nk, device=DEV)[None, :] > torch.arange(r, e, device=DEV)[:, None] + (nk - nq)
                x.masked_fill_(future, float("-inf"))
                l = torch.logsumexp(x, 1)
                out[aq + r:aq + e, h] = torch.exp(x - l[:, None]) @ vh
                lse[aq + r:aq + e, h] = l
        aq += nq
    return (out, lse) if case["lse"] else (out,)
