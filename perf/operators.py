"""What is measured of the operators around the dense output head: the final norm with the residual's
addition and its int8 output, the int8 matrix product with scales per token and channel and the dense head
on it, and the rules on logits (penalties, biases, grammar masks) with the choice of the token.

`run` computes an operator in its plain form, elementary torch operations in float32, or (`own`) through the
framework's entry points.  `exact` computes the same from the definitions in float64.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # -- the norm ahead of the head
        # one sequence's decode step: the smallest call, where latency counts
        {"name": "norm_decode", "op": "norm", "B": 1, "d": 2048, "dtype": "bf16", "residual": True, "offset": 0.0,
         "out": False, "q": True},
        # a decode batch in float32 with the (1 + w) weights of the 1152-wide head, hidden states for fh_forward
        {"name": "norm_batch_f32", "op": "norm", "B": 61, "d": 1152, "dtype": "f32", "residual": False, "offset": 1.0,
         "out": True, "q": False},
        # every position of long prompts, the residual stream written back and both outputs kept
        {"name": "norm_prefill", "op": "norm", "B": 16384, "d": 2560, "dtype": "bf16", "residual": True, "offset": 0.0,
         "out": True, "q": True},
        # -- the int8 product
        # logits of one token: the whole 128256 x 2048 table is read for one row
        {"name": "product_decode", "op": "product", "B": 1, "n": 128256, "k": 2048, "out": "f32"},
        # logits of a batch of sequences (or of a draft's positions)
        {"name": "product_batch", "op": "product", "B": 64, "n": 151936, "k": 2560, "out": "f32"},
        # a projection of odd width over a ragged batch
        {"name": "product_ragged", "op": "product", "B": 333, "n": 5003, "k": 1152, "out": "bf16"},
        # a projection over a prompt's positions: bound by the matrix cores
        {"name": "product_prefill", "op": "product", "B": 4096, "n": 10240, "k": 2560, "out": "bf16"},
        # -- the dense head on it
        # greedy token of one sequence from the 262144 x 1152 head
        {"name": "head_decode", "op": "head", "B": 1, "n": 262144, "k": 1152, "T": 0.0, "logits": False},
        # a large decode batch, tokens sampled, logits kept for what follows
        {"name": "head_batch", "op": "head", "B": 128, "n": 128256, "k": 2048, "T": 0.75, "logits": True},
        # -- the rules on logits
        # one sequence, greedy, its prompt and a few hundred generated tokens
        {"name": "rules_decode", "op": "rules", "B": 1, "v": 128256, "n": 0, "L": 1000, "bias": 16, "mask": 0.25,
         "T": 0.0},
        # a batch with long histories, half of it under a grammar, tokens sampled
        {"name": "rules_batch", "op": "rules", "B": 64, "v": 151936, "n": 0, "L": 8192, "bias": 64, "mask": 0.25,
         "T": 0.75},
        # the retrieved candidates of eight queries (512 probes of 16 tokens)
        {"name": "rules_candidates", "op": "rules", "B": 8, "v": 128256, "n": 8192, "L": 2000, "bias": 32, "mask": 0.25,
         "T": 0.75},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "product", "head", "rules"))
    if op == "norm":
        dt, d = rng.choice(("bf16", "bf16", "f32")), _log(rng, 64, 8192)
        if rng.random() < 0.6:
            d = (d + 63) // 64 * 64
        q = dt == "bf16" and rng.random() < 0.6
        top = min(16384, 16384 * 2560 // (d if dt == "bf16" else 2 * d))
        return {"op": op, "B": _log(rng, 1, top), "d": d, "dtype": dt, "residual": rng.random() < 0.6,
                "offset": rng.choice((0.0, 1.0)), "out": not q or rng.random() < 0.5, "q": q}
    if op in ("product", "head"):
        k = _log(rng, 64, 8192)
        if rng.random() < 0.8:
            k = (k + 31) // 32 * 32
        n = _log(rng, 1000, min(262144, 388_000_000 // k))
        if op == "head":
            return {"op": op, "B": _log(rng, 1, max(1, min(256, 16_000_000 // n))), "n": n, "k": k,
                    "T": rng.choice((0.0, 0.75, 1.25)), "logits": rng.random() < 0.5}
        top = min(4096, 41_000_000 // n, 4096 * 10240 * 2560 // (n * k))
        return {"op": op, "B": _log(rng, 1, max(1, top)), "n": n, "k": k, "out": rng.choice(("f32", "bf16"))}
    v = _log(rng, 1000, 262144)
    n = _log(rng, 64, min(v, 32768)) if rng.random() < 0.35 else 0
    B = _log(rng, 1, max(1, min(256, 64 * 151936 // v)))
    return {"op": op, "B": B, "v": v, "n": n, "L": rng.choice((0, _log(rng, 1, 32768), _log(rng, 64, 8192))),
            "bias": rng.choice((0, _log(rng, 1, 300))), "mask": rng.choice((0.0, 0.01, 0.25, 0.9)),
            "T": rng.choice((0.0, 0.75, 1.25))}


def _sampling(T):
    """(mode, temperature) of a call: greedy where T is 0, else tokens sampled at T."""
    return (2, T) if T else (0, 1.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    st = {"case": case, "seed": seed}
    if own:
        import lm_output_head_amd
        st["fh"] = lm_output_head_amd
    if case["op"] == "norm":
        B, d, dt = case["B"], case["d"], _DT[case["dtype"]]
        # a residual stream: most channels of order one, a few outlier channels
        chan = torch.ones(d, device=dev)
        chan[torch.randint(0, d, (max(1, d // 256),), generator=g, device=dev)] = 12.0
        st["x"] = (torch.randn(B, d, generator=g, device=dev) * chan).to(dt)
        st["r"] = (torch.randn(B, d, generator=g, device=dev) * chan * 2).to(dt) if case["residual"] else None
        st["w"] = (torch.randn(d, generator=g, device=dev) * 0.2 + (1.0 - case["offset"])).to(dt)
        return st
    if case["op"] in ("product", "head"):
        B, n, k = case["B"], case["n"], case["k"]
        # weights and activations as symmetric quantisation leaves them: normal values, the largest at 127
        w = torch.randn(n, k, generator=g, device=dev)
        top = w.abs().amax(1, keepdim=True)
        st["w"] = torch.round(w * (127.0 / top)).to(torch.int8)
        st["ws"] = (top[:, 0] / (127.0 * math.sqrt(k))).contiguous()
        a = torch.randn(B, k, generator=g, device=dev)
        top = a.abs().amax(1, keepdim=True)
        st["q"] = torch.round(a * (127.0 / top)).to(torch.int8)
        st["qs"] = (top[:, 0] * (3.0 / 127.0)).contiguous()
        if own:  # the weight's handle, laid out once as a program that serves from it does
            st["head"] = st["fh"].W8A8Head(codes=st["w"], scales=st["ws"])
        return st
    B, v, n, L, nb = case["B"], case["v"], case["n"], case["L"], case["bias"]
    width = n or v
    st["z"] = torch.randn(B, width, generator=g, device=dev) * 3.0
    st["ids"] = None
    if n:  # distinct tokens in no order, as clusters list them
        at = torch.rand(B, v, generator=g, device=dev).topk(n, dim=1).indices
        st["ids"] = at.to(torch.int32).contiguous()
    st["history"] = st["n_prompt"] = st["n_history"] = None
    if L:  # a text's tokens: frequent ones come many times
        u = torch.rand(B, L, generator=g, device=dev)
        st["history"] = (v * u ** 6).to(torch.int32).clamp_(max=v - 1)
        st["n_history"] = torch.randint((L + 1) // 2, L + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        st["n_prompt"] = (st["n_history"] * torch.rand(B, generator=g, device=dev)).to(torch.int32)
    st["rep"] = 1.0 + 0.25 * torch.rand(B, generator=g, device=dev)
    st["freq"] = 0.5 * torch.rand(B, generator=g, device=dev)
    st["pres"] = 0.5 * torch.rand(B, generator=g, device=dev)
    st["bias_ids"] = st["bias"] = None
    if nb:
        st["bias_ids"] = torch.randint(0, v, (B, nb), generator=g, device=dev, dtype=torch.int32)
        st["bias"] = torch.randn(B, nb, generator=g, device=dev) * 4.0
    st["mask"] = st["mask_row"] = None
    if case["mask"]:  # a bit per token, four grammars' states, every other sequence under one of them
        words = (v + 31) // 32
        bits = torch.rand(4, words * 32, generator=g, device=dev) < case["mask"]
        place = torch.ones(32, dtype=torch.int64, device=dev) << torch.arange(32, device=dev)
        word = (bits.view(4, words, 32) * place).sum(2)
        st["mask"] = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32).contiguous()
        row = torch.arange(B, device=dev)
        st["mask_row"] = torch.where(row % 2 == 0, row // 2 % 4, row * 0 - 1).to(torch.int32)
    if own:  # the rules' tensors as a program keeps them, updated in place from step to step
        st["rules"] = st["fh"].LogitRules(
            v, history=st["history"], n_prompt=st["n_prompt"], n_history=st["n_history"], repetition=st["rep"],
            frequency=st["freq"], presence=st["pres"], bias_ids=st["bias_ids"], bias=st["bias"], mask=st["mask"],
            mask_row=st["mask_row"])
    return st


# ------------------------------------------------------------------- plain forms

def _uniforms(seed, rows, ids):
    """Philox4x32-10 (Salmon et al. 2011) of counter (id / 4, row, 1, 0) under key `seed`: word id mod 4 as a
    uniform in (0, 1).  Products of 32-bit words wrap in int64, whose bits are the 64 that count."""
    low = 0xFFFFFFFF
    x0, x1 = ids // 4, rows.expand_as(ids)
    x2, x3 = torch.ones_like(ids), torch.zeros_like(ids)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        p, r = x0 * 0xD2511F53, x2 * 0xCD9E8D57
        x0, x1, x2, x3 = ((r >> 32) & low) ^ x1 ^ k0, r & low, ((p >> 32) & low) ^ x3 ^ k1, p & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    w = torch.stack((x0, x1, x2, x3)).gather(0, (ids % 4)[None])[0]
    return ((w >> 9).float() + 0.5) * 2.0 ** -23


def _choose(z, ids, T, seed):
    """Token, its logit and the log-sum-exp of rows of logits; -1 and -inf where a row has none left."""
    x = z / T if T else z
    key = x
    if T:
        rows = torch.arange(z.shape[0], device=z.device)[:, None]
        key = x - torch.log(-torch.log(_uniforms(seed, rows, ids)))
    best = key.amax(1, keepdim=True)
    live = best[:, 0] > -math.inf
    token = torch.where(key == best, ids, 1 << 40).amin(1)
    at = (ids == token[:, None]).to(torch.int8).argmax(1, keepdim=True)
    top = x.amax(1, keepdim=True)
    shift = torch.where(top > -math.inf, top, 0.0)
    return {"token": torch.where(live, token, -1).to(torch.int32),
            "token_logit": torch.where(live, z.gather(1, at)[:, 0], -math.inf),
            "lse": (x - shift).exp().sum(1).log() + shift[:, 0]}


def _plain_norm(st):
    case = st["case"]
    s = st["x"].float()
    got = {}
    if case["residual"]:
        s = s + st["r"].float()
        got["residual"] = s.to(st["x"].dtype)
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-6) * (case["offset"] + st["w"].float())
    if case["out"]:
        got["out"] = y.to(st["x"].dtype)
    if case["q"]:
        scale = y.abs().amax(1, keepdim=True) / 127.0
        q = torch.round(y / scale).clamp(-127.0, 127.0)
        got["values"], got["scale"] = (q * scale).to(torch.bfloat16), scale[:, 0]
    return got


def _plain_product(st):
    # in slices of the channels: a float32 copy of a whole table would be four times its size
    acc = [st["q"].float() @ w.float().T for w in st["w"].split(65536)]
    return torch.cat(acc, 1) * (st["qs"][:, None] * st["ws"][None, :])


def _plain_rules(st):
    z, v = st["z"], st["case"]["v"]
    B = z.shape[0]
    ids = torch.arange(v, device=z.device).expand(B, v) if st["ids"] is None else st["ids"].long()
    if st["history"] is not None:
        place = torch.arange(st["history"].shape[1], device=z.device)[None]
        valid = place < st["n_history"][:, None]
        made = valid & (place >= st["n_prompt"][:, None])
        h = st["history"].long()
        seen = torch.zeros(B, v, device=z.device).scatter_add_(1, h, valid.float()).gather(1, ids) > 0
        count = torch.zeros(B, v, device=z.device).scatter_add_(1, h, made.float()).gather(1, ids)
        rep = st["rep"][:, None]
        z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
        z = z - st["freq"][:, None] * count
        z = z - st["pres"][:, None] * (count > 0)
    if st["bias_ids"] is not None:
        add = torch.zeros(B, v, dtype=torch.float64, device=z.device)
        add.scatter_add_(1, st["bias_ids"].long(), st["bias"].double())
        z = z + add.float().gather(1, ids)
    if st["mask"] is not None:
        word = st["mask"][st["mask_row"].clamp(min=0).long()].long().gather(1, ids >> 5)
        open_ = ((word >> (ids & 31)) & 1).bool() | (st["mask_row"] < 0)[:, None]
        z = torch.where(open_, z, -math.inf)
    return {"logits": z, **_choose(z, ids, st["case"]["T"], st["seed"])}


def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        if op == "norm":
            return _plain_norm(st)
        if op == "rules":
            return _plain_rules(st)
        z = _plain_product(st)
        if op == "product":
            return z.to(_DT[case["out"]])
        ids = torch.arange(case["n"], device=z.device).expand(case["B"], case["n"])
        return {**_choose(z, ids, case["T"], st["seed"]), "logits": z if case["logits"] else None}
    if op == "norm":
        r = st["fh"].rmsnorm(st["x"], st["w"], residual=st["r"], eps=1e-6, weight_offset=case["offset"],
                             want_out=case["out"], want_q=case["q"])
        got = {name: r[name] for name in ("residual", "out") if name in r}
        if case["q"]:  # the codes as the values they stand for
            got["scale"] = r["q_scale"]
            got["values"] = torch.empty(r["q"].shape, dtype=torch.bfloat16, device=r["q"].device)
            torch.mul(r["q"], r["q_scale"][:, None], out=got["values"])
        return got
    if op == "product":
        return st["head"].matmul(st["q"], st["qs"], dtype=_DT[case["out"]])
    mode, T = _sampling(case["T"])
    if op == "head":
        r = st["head"].forward(st["q"], st["qs"], mode=mode, temperature=T, seed=st["seed"], want_logits=case["logits"])
    else:
        r = st["fh"].logits_apply(st["z"], st["rules"], ids=st["ids"], mode=mode, temperature=T, seed=st["seed"])
    return {name: r.get(name) for name in ("token", "token_logit", "lse", "logits")}


def work(case):
    op, B = case["op"], case["B"]
    if op == "norm":
        d, e = case["d"], 2 if case["dtype"] == "bf16" else 4
        per = e * (1 + 2 * case["residual"] + case["out"]) + case["q"]
        return {"bytes": B * d * per + d * e + 4 * B * case["q"], "flops": 8 * B * d}
    if op in ("product", "head"):
        n, k = case["n"], case["k"]
        written = B * n * (4 if case["out"] == "f32" else 2) if op == "product" else 12 * B + 4 * B * n * case["logits"]
        return {"bytes": n * k + B * k + 4 * (n + B) + written, "flops": 2 * B * n * k}
    v, n = case["v"], case["n"]
    masked = min(4, (B + 1) // 2) * ((v + 31) // 32) * 4 if case["mask"] else 0
    return {"bytes": B * ((n * 12) if n else v * 8) + 4 * B * case["L"] + 8 * B * case["bias"] + masked + 28 * B,
            "flops": B * (n or v) * (10 + 60 * bool(case["T"]))}


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definitions in float64; counts of tokens by sorting instead of tables, sums of biases by prefix sums."""
    st = prepare(case, seed)
    if case["op"] == "norm":
        s = st["x"].double() + (st["r"].double() if case["residual"] else 0.0)
        y = s / (s.pow(2).sum(1, keepdim=True) / case["d"] + 1e-6).sqrt() * (st["w"].double() + case["offset"])
        top = y.abs().max(1).values
        got = {"out": y if case["out"] else None, "residual": s if case["residual"] else None}
        if case["q"]:
            step = top / 127
            got["scale"] = step
            got["values"] = (y / step[:, None]).round() * step[:, None]
        return got
    if case["op"] in ("product", "head"):
        a = st["q"].double() * st["qs"].double()[:, None]
        parts = []
        for lo in range(0, case["n"], 16384):
            w = st["w"][lo:lo + 16384].double() * st["ws"][lo:lo + 16384].double()[:, None]
            parts.append(torch.mm(a, w.t().contiguous()))
        z = torch.cat(parts, 1)
        if case["op"] == "product":
            return z
        T = case["T"] or 1.0
        return {"token": None, "token_logit": None if case["T"] else z.max(1).values,
                "lse": torch.logsumexp(z / T, 1), "logits": z if case["logits"] else None}
    B, v = case["B"], case["v"]
    z = st["z"].double().clone()
    ids = st["ids"].long() if st["ids"] is not None else torch.arange(v, device=z.device)[None].repeat(B, 1)
    for b in range(B):
        if st["history"] is not None:
            text = st["history"][b, :int(st["n_history"][b])].long()
            prompt = int(st["n_prompt"][b])
            for tokens, made in ((text, False), (text[prompt:], True)):
                if not tokens.numel():
                    continue
                kinds, times = tokens.sort().values.unique_consecutive(return_counts=True)
                where = torch.searchsorted(kinds, ids[b]).clamp(max=kinds.numel() - 1)
                hit = kinds[where] == ids[b]
                if made:
                    drop = st["freq"][b].double() * times[where].double() + st["pres"][b].double()
                    z[b] -= drop * hit
                else:
                    rep = st["rep"][b].double()
                    z[b] = torch.where(hit & (z[b] > 0), z[b] / rep, torch.where(hit, z[b] * rep, z[b]))
        if st["bias_ids"] is not None:
            order = st["bias_ids"][b].long().argsort()
            kinds, times = st["bias_ids"][b].long()[order].unique_consecutive(return_counts=True)
            run_ = torch.cat((torch.zeros(1, dtype=torch.float64, device=z.device),
                              st["bias"][b].double()[order].cumsum(0)))
            end = times.cumsum(0)
            where = torch.searchsorted(kinds, ids[b]).clamp(max=kinds.numel() - 1)
            z[b] += torch.where(kinds[where] == ids[b], (run_[end] - run_[end - times])[where], 0.0)
        if st["mask"] is not None and int(st["mask_row"][b]) >= 0:
            words = st["mask"][int(st["mask_row"][b])].long()
            shut = torch.bitwise_right_shift(words[ids[b] // 32], ids[b] % 32) % 2 == 0
            z[b, shut] = -math.inf
    T = case["T"] or 1.0
    return {"logits": z, "token": None, "token_logit": None if case["T"] else z.max(1).values,
            "lse": torch.logsumexp(z / T, 1)}
