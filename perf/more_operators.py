"""Measured cases of attention over packed sequences and what stands beside it.

Three operators: ``rope`` turns queries and keys by their positions (and gradients back), ``packed`` is attention over
sequences of different lengths that lie one behind the other without padding, with its backward pass, ``prefix`` is the
same attention where all sequences also see one shared stretch of keys ahead of their own.

Packed tensors are [tokens, heads, d]; sequence b has the query rows cu_q[b] to cu_q[b + 1] and the key rows cu_k[b] to
cu_k[b + 1], of which the first used_k[b] count where that is given.  The logsumexp is [H, tokens].  Rows behind the
last sequence stay as they were.
"""

import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases

def _rope(name, form, B, N, H, Hkv, d, rot, interleaved, factor, inverse):
    return {"name": name, "op": "rope", "form": form, "B": B, "N": N, "H": H, "Hkv": Hkv, "d": d, "rot": rot,
            "interleaved": interleaved, "factor": factor, "inverse": inverse}


def _packed(name, form, B, T, H, Hkv, d, causal, grad, history=0):
    return {"name": name, "op": "packed", "form": form, "B": B, "T": T, "H": H, "Hkv": Hkv, "d": d, "causal": causal,
            "grad": grad, "history": history}


def _prefix(name, form, B, P, T, H, Hkv, d):
    return {"name": name, "op": "prefix", "form": form, "B": B, "P": P, "T": T, "H": H, "Hkv": Hkv, "d": d,
            "causal": "bottom_right"}


def listed():
    return [
        # A decoding step of 64 sequences, far into their contexts.
        _rope("rope_step", "dense", 64, 1, 32, 8, 128, 128, False, 1.0, False),
        # Packed prompts, queries and keys still inside the fused projection's output.
        _rope("rope_prompts", "packed", 16, 32768, 32, 8, 128, 128, False, 1.0, False),
        # The gradients of a model that turns 64 of 96 channels, neighbouring channels paired, positions stretched.
        _rope("rope_gradients_d96", "packed", 9, 8191, 12, 4, 96, 64, True, 4.0, True),
        # A few short prompts: nothing but latency.
        _packed("packed_short", "prompts", 4, 150, 16, 16, 64, "top_left", False),
        # Prompts of all lengths that arrive together, four query heads to a key/value head.
        _packed("packed_prompts", "prompts", 16, 16384, 32, 8, 128, "top_left", False),
        # A server's batch: most sequences add one token to a long history, some a piece of a prompt.
        _packed("packed_server", "mixed", 48, 2048, 32, 8, 128, "bottom_right", False, 8192),
        # Sentences for an encoder, every token sees its whole sentence.
        _packed("packed_encoder_d96", "prompts", 32, 8000, 12, 12, 96, "none", False),
        # A training step on packed documents, the benchmark's 16 heads.
        _packed("packed_training", "prompts", 24, 16384, 16, 16, 128, "top_left", True),
        # The same for a smaller model with shared heads, the last rows padding.
        _packed("packed_training_d64", "padded", 9, 8190, 32, 8, 64, "top_left", True),
        # Four answers to one short question.
        _prefix("prefix_short", "steps", 4, 1000, 200, 16, 16, 64),
        # A decoding step of 64 answers behind one long document.
        _prefix("prefix_step", "steps", 64, 8192, 32768, 32, 8, 128),
        # Prompts of their own behind one long instruction.
        _prefix("prefix_prompts", "prompts", 16, 6000, 4000, 32, 8, 128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "packed", "packed", "packed", "prefix", "prefix"])
    d = rng.choice([64, 96, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    H = Hkv * rng.randint(1, max(1, min(8, 32 // Hkv)))
    B = _log(rng, 1, 64)
    if op == "rope":
        rot = 2 * rng.randint(4, d // 2) // 16 * 16 if rng.random() < 0.5 else d
        most = 32768 * 40 * 128 // ((H + Hkv) * d)
        if rng.random() < 0.3:
            c = _rope("", "dense", B, _log(rng, 1, max(1, min(4096, most // B))), H, Hkv, d, max(16, rot),
                      rng.random() < 0.5, rng.choice([1.0, 4.0, 8.0]), rng.random() < 0.3)
        else:
            c = _rope("", "packed", B, _log(rng, B, max(B, min(65536, most))), H, Hkv, d, max(16, rot),
                      rng.random() < 0.5, rng.choice([1.0, 4.0, 8.0]), rng.random() < 0.3)
    elif op == "packed":
        grad = rng.random() < 0.5
        form = rng.choice(["prompts", "prompts", "padded"]) if grad else rng.choice(["prompts", "padded", "mixed"])
        T = _log(rng, 2 * B, max(2 * B, 16384 if form != "mixed" else 4096))
        causal = "bottom_right" if form == "mixed" else rng.choice(["none", "top_left", "top_left"])
        c = _packed("", form, B, T, H, Hkv, d, causal, grad, _log(rng, 16, 16384) if form == "mixed" else 0)
    else:
        form = rng.choice(["steps", "prompts"])
        c = _prefix("", form, B, _log(rng, 1, 16384), _log(rng, 2 * B, 32768 if form == "steps" else 4096), H, Hkv, d)
    del c["name"]
    # No dearer than the listed ones of its operator.
    limit = [max(work(x)[n] for x in listed() if x["op"] == op) for n in ("bytes", "flops")]
    while work(c)["bytes"] > limit[0] or work(c)["flops"] > limit[1]:
        long = max((n for n in ("N", "T", "P", "history") if n in c), key=lambda n: c[n])
        c[long] = max(1, c[long] * 3 // 4)
        c["B"] = max(1, min(c["B"], c.get("T", c["B"])))
    return c


def _lengths(case):
    """(query rows, key rows, key rows that count) of each sequence: part of the case, not of the seed.  The key rows
    of a server's cache have room for more than what counts."""
    B, form = case["B"], case["form"]
    total = case["N"] if case["op"] == "rope" else case["T"]
    r = random.Random(B * 1000003 + total)
    weights = [r.uniform(0.1, 1.0) ** 2 for _ in range(B)]
    if B > 4:
        weights[r.randrange(B)] = sum(weights) / 3  # one long sequence
    parts = [max(1, int(total * w / sum(weights))) for w in weights]
    if B > 8:
        parts[r.randrange(B)] = 0  # and one empty one
    if case["op"] == "prefix":
        if form == "steps":
            return [1] * B, parts, parts
        return parts, parts, parts
    if form == "mixed":
        q = [1] * B
        for i in range(0, B, 6):
            q[i] = max(1, total // (B // 6 + 1))
        used = [n + r.randint(0, case["history"]) for n in q]
        room = -(-max(used) // 64) * 64
        return q, [room] * B, used
    return parts, parts, parts


def _starts(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return out


def _visible(case):
    """Visible (query row, key) pairs of one query head."""
    lq, _, used = _lengths(case)
    n = 0
    for a, b in zip(lq, used):
        if case["causal"] == "none":
            n += a * b
        else:  # equal lengths, or the last row sees every key
            n += sum(max(0, b - a + 1 + i) for i in range(a))
    return n + (case["P"] * sum(lq) if case["op"] == "prefix" else 0)


def work(case):
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        tokens = case["B"] * case["N"] if case["form"] == "dense" else sum(_lengths(case)[0])
        # Three operations a channel.  Channels that are not turned are passed on.
        return {"bytes": tokens * ((H + Hkv) * d * 4 + 4), "flops": 3 * tokens * (H + Hkv) * case["rot"]}
    lq, _, used = _lengths(case)
    tq, tk = sum(lq), sum(used) + case.get("P", 0)
    moved = tq * H * (4 * d + 4) + tk * Hkv * 4 * d
    flops = 4 * d * H * _visible(case)
    if case.get("grad"):
        # dO in; dQ, dK, dV out.  Five products in place of two.
        moved += tq * H * 4 * d + tk * Hkv * 4 * d
        flops = flops * 7 // 2
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------ inputs

def _frequencies(rot, factor, base=10000.0):
    """Radians a position of each channel pair, in 64 bits; factor > 1 stretches the slow ones for long contexts: by
    the factor where a pair turns less than once over 4096 positions, not at all above 32 times, between these in
    proportion."""
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    out = []
    for x in f:
        turns = 4096.0 * x / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / 31.0))
        out.append(x * keep + x / factor * (1.0 - keep))
    return torch.tensor(out, dtype=torch.float64)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    H, Hkv, d = case["H"], case["Hkv"], case["d"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)

    def keys(*shape):
        """A few strong channels, as rotary keys have."""
        x = torch.randn(shape, generator=g, device=dev)
        return (x * (1.0 + 3.0 * (torch.rand(shape[-1], generator=g, device=dev) < 0.05))).to(torch.bfloat16)

    st = {"case": case}
    if case["op"] == "rope":
        freq = _frequencies(case["rot"], case["factor"])
        st["freq"] = freq.to(dev)
        st["mscale"] = 0.1 * math.log(case["factor"]) + 1.0
        if case["form"] == "dense":
            B, N = case["B"], case["N"]
            st["q"], st["k"] = normal(B, H, N, d), normal(B, Hkv, N, d)
            first = torch.randint(0, 131072, (B, 1), generator=g, device=dev)
            pos = first + torch.arange(N, device=dev)
        else:
            lens = _lengths(case)[0]
            T = sum(lens)
            fused = normal(T, H + 2 * Hkv, d)
            st["q"], st["k"] = fused[:, :H], fused[:, H:H + Hkv]
            pos = torch.cat([torch.arange(n, device=dev) for n in lens])
        st["pos"] = pos.to(torch.int32)
        st["q_out"] = torch.empty(st["q"].shape, dtype=torch.bfloat16, device=dev)
        st["k_out"] = torch.empty(st["k"].shape, dtype=torch.bfloat16, device=dev)
        if own:
            import exact_attention_92_gb300 as fa

            st["phases"] = fa.rope_phases(freq)
        return st
    lq, lk, used = _lengths(case)
    pad = 37 if case["form"] == "padded" else 0
    tq, tk = sum(lq) + pad, sum(lk) + pad
    i32 = dict(dtype=torch.int32, device=dev)
    st["cu_q"], st["cu_k"] = torch.tensor(_starts(lq), **i32), torch.tensor(_starts(lk), **i32)
    st["used_k"] = torch.tensor(used, **i32) if case["form"] == "mixed" else None
    st["q"], st["k"], st["v"] = normal(tq, H, d), keys(tk, Hkv, d), normal(tk, Hkv, d)
    st["o"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros((H, tq), dtype=torch.float32, device=dev)
    if case["op"] == "prefix":
        st["k_prefix"], st["v_prefix"] = keys(case["P"], Hkv, d), normal(case["P"], Hkv, d)
    elif case["grad"]:
        st["dout"] = normal(tq, H, d)
        st["dq"], st["dk"], st["dv"] = (torch.zeros_like(st[n]) for n in ("q", "k", "v"))
    return st


# ------------------------------------------------------------- the operators

def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import exact_attention_92_gb300 as fa

        if op == "rope":
            fa.fa_rope(st["q"], st["k"], st["q_out"], st["k_out"], st["phases"], positions=st["pos"],
                       interleaved=case["interleaved"], mscale=st["mscale"], inverse=case["inverse"])
            return {"q": st["q_out"], "k": st["k_out"]}
        if op == "prefix":
            fa.fa_prefix_fwd(st["q"], st["k_prefix"], st["v_prefix"], st["k"], st["v"], st["o"], st["lse"],
                             st["cu_q"], st["cu_k"], causal=case["causal"])
            return {"o": st["o"], "lse": st["lse"]}
        fa.fa_packed_fwd(st["q"], st["k"], st["v"], st["o"], st["lse"], st["cu_q"], st["cu_k"], used_k=st["used_k"],
                         causal=case["causal"])
        if not case["grad"]:
            return {"o": st["o"], "lse": st["lse"]}
        fa.fa_packed_bwd(st["q"], st["k"], st["v"], st["o"], st["lse"], st["dout"], st["dq"], st["dk"], st["dv"],
                         st["cu_q"], st["cu_k"], causal=case["causal"])
        return {n: st[n] for n in ("o", "lse", "dq", "dk", "dv")}
    if op == "rope":
        return _plain_rope(st)
    return _plain_attention(st)


def _plain_rope(st):
    case = st["case"]
    rot = case["rot"]
    angle = st["pos"].double()[..., None] * st["freq"]
    if case["inverse"]:
        angle = -angle
    cos, sin = (f(angle).float() * st["mscale"] for f in (torch.cos, torch.sin))
    # [tokens, heads, d] or [B, heads, N, d]: the heads' axis goes in.
    cos, sin = (x[:, None] for x in (cos, sin))
    out = {}
    for name in ("q", "k"):
        x = st[name].float()
        y = x.clone()
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        out[name] = y.to(torch.bfloat16)
    return out


def _plain_attention(st):
    case = st["case"]
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    G, scale = H // Hkv, 1.0 / math.sqrt(d)
    lq, lk, used = _lengths(case)
    sq, sk = _starts(lq), _starts(lk)
    names = ("o", "lse", "dq", "dk", "dv") if case.get("grad") else ("o", "lse")
    out = {n: torch.zeros_like(st[n]) for n in names}
    for b in range(case["B"]):
        nq, nk = lq[b], used[b]
        if nq == 0:
            continue
        rows, cols = slice(sq[b], sq[b] + nq), slice(sk[b], sk[b] + nk)
        ahead = 0  # keys of the prefix
        k, v = st["k"][cols], st["v"][cols]
        if case["op"] == "prefix":
            ahead = case["P"]
            k, v = torch.cat([st["k_prefix"], k]), torch.cat([st["v_prefix"], v])
        last = ahead + nk - 1
        if case["causal"] == "top_left":
            last = torch.arange(nq, device=k.device)
        elif case["causal"] == "bottom_right":
            last = torch.arange(nq, device=k.device) + ahead + nk - nq
        hidden = torch.arange(k.shape[0], device=k.device)[None] > torch.as_tensor(last, device=k.device).view(-1, 1)
        step = max(1, min(Hkv, (1 << 28) // (G * nq * max(1, k.shape[0]))))
        for h in range(0, Hkv, step):
            hk, hq = slice(h, min(Hkv, h + step)), slice(h * G, min(Hkv, h + step) * G)
            # [kv heads, G, rows, d] and [kv heads, 1, keys, d]
            q = st["q"][rows, hq].float().transpose(0, 1).reshape(-1, G, nq, d)
            kf, vf = (x[:, hk].float().transpose(0, 1)[:, None] for x in (k, v))
            s = (q @ kf.transpose(-1, -2)).mul_(scale).masked_fill_(hidden, -math.inf)
            m = s.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            p = s.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            p /= torch.where(l > 0, l, torch.ones_like(l))
            o = p @ vf
            out["o"][rows, hq] = o.flatten(0, 1).transpose(0, 1).to(torch.bfloat16)
            out["lse"][hq, rows] = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf)).flatten(0, 1)[..., 0]
            if not case.get("grad"):
                continue
            do = st["dout"][rows, hq].float().transpose(0, 1).reshape(-1, G, nq, d)
            ds = (do @ vf.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
            out["dq"][rows, hq] = (ds @ kf).flatten(0, 1).transpose(0, 1).to(torch.bfloat16)
            out["dk"][cols, hk] = (ds.transpose(-1, -2) @ q).sum(1).transpose(0, 1).to(torch.bfloat16)
            out["dv"][cols, hk] = (p.transpose(-1, -2) @ do).sum(1).transpose(0, 1).to(torch.bfloat16)
    return out


# ----------------------------------------------- the definition, in 64 bits

def _exact_rope(case, st):
    pairs = case["rot"] // 2
    # Angles reduced to one turn before the functions see them.
    turns = st["pos"].double().unsqueeze(-1) * (st["freq"] / (2 * math.pi))
    turns = (turns - torch.round(turns)) * (-1.0 if case["inverse"] else 1.0)
    unit = torch.polar(torch.full_like(turns, st["mscale"]), turns * (2 * math.pi)).unsqueeze(1)
    out = {}
    for name in ("q", "k"):
        x = st[name].double()
        turned, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
        if case["interleaved"]:
            z = torch.view_as_complex(turned.reshape(*turned.shape[:-1], pairs, 2).contiguous()) * unit
            turned = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(turned[..., :pairs].contiguous(), turned[..., pairs:].contiguous()) * unit
            turned = torch.cat([z.real, z.imag], -1)
        out[name] = torch.cat([turned, rest], -1)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, st)
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    lq, lk, used = _lengths(case)
    names = ("o", "lse", "dq", "dk", "dv") if case.get("grad") else ("o", "lse")
    out = {n: torch.zeros(st[n].shape, dtype=torch.float64, device="cuda") for n in names}
    q0 = k0 = 0
    for b in range(case["B"]):
        nq, nk = lq[b], used[b]
        for h in range(H if nq else 0):
            q = st["q"][q0:q0 + nq, h].double()
            k, v = (st[n][k0:k0 + nk, h * Hkv // H].double() for n in ("k", "v"))
            seen = torch.ones((nq, nk), dtype=torch.bool, device="cuda")
            if case["causal"] != "none":
                seen = seen.tril(nk - nq if case["causal"] == "bottom_right" else 0)
            if case["op"] == "prefix":
                kp, vp = (st[n][:, h * Hkv // H].double() for n in ("k_prefix", "v_prefix"))
                k, v = torch.cat([kp, k]), torch.cat([vp, v])
                seen = torch.cat([torch.ones((nq, case["P"]), dtype=torch.bool, device="cuda"), seen], 1)
            logits = torch.where(seen, (q @ k.T) * d ** -0.5, -math.inf)
            lse = torch.logsumexp(logits, 1)
            w = torch.exp(logits - torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))[:, None])
            o = w @ v
            out["o"][q0:q0 + nq, h], out["lse"][h, q0:q0 + nq] = o, lse
            if case.get("grad"):
                do = st["dout"][q0:q0 + nq, h].double()
                ds = w * (do @ v.T - (o * do).sum(1)[:, None])
                out["dq"][q0:q0 + nq, h] = (ds @ k) * d ** -0.5
                out["dk"][k0:k0 + nk, h * Hkv // H] += (ds.T @ q) * d ** -0.5
                out["dv"][k0:k0 + nk, h * Hkv // H] += w.T @ do
        q0, k0 = q0 + lq[b], k0 + lk[b]
    return out
