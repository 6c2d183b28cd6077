"""What is measured of the operators around an fp8 head and of decoding by beams: hidden states in 8-bit floating
point with a scale per 128 (after the final norm, or as they are), the product with a weight that has a scale per
block of 128 x 128 and the dense head on it, the choice of the best continuations over beams and vocabulary, and
the reordering of caches and histories that follows it.

`run` computes an operator in its plain form, elementary torch operations in float32 (the beams' totals in float64,
where neighbours decide), or (`own`) through the framework's entry points.  `exact` computes the same from the
definitions in float64.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_F8 = torch.float8_e4m3fn


def listed():
    return [
        # -- hidden states in fp8
        # one sequence's decode step: the smallest call, where latency counts
        {"name": "quant_decode", "op": "quant", "B": 1, "d": 2048, "dtype": "bf16", "norm": True, "residual": True,
         "out": False},
        # every position of long prompts ahead of a projection, the residual stream written back
        {"name": "quant_prefill", "op": "quant", "B": 16384, "d": 2560, "dtype": "bf16", "norm": True,
         "residual": True, "out": False},
        # -- the fp8 product
        # logits of a batch of sequences (or of a draft's positions)
        {"name": "product_batch", "op": "product", "B": 64, "n": 151936, "k": 2560, "out": "f32"},
        # a projection of odd width over a ragged batch
        {"name": "product_ragged", "op": "product", "B": 333, "n": 5003, "k": 1152, "out": "bf16"},
        # a projection over a prompt's positions: bound by the matrix cores
        {"name": "product_prefill", "op": "product", "B": 4096, "n": 10240, "k": 2560, "out": "bf16"},
        # -- the dense head on it
        # greedy token of one sequence from the 128256 x 2048 head: the whole table is read for one row
        {"name": "head_decode", "op": "head", "B": 1, "n": 128256, "k": 2048, "T": 0.0, "logits": False},
        # a large decode batch, tokens sampled, logits kept for what follows
        {"name": "head_batch", "op": "head", "B": 128, "n": 262144, "k": 1152, "T": 0.75, "logits": True},
        # -- the beams' choice
        # one sequence of four beams over all tokens
        {"name": "beams_decode", "op": "beams", "S": 1, "W": 4, "v": 128256, "n": 0, "keep": 4, "mask": 0.0,
         "finished": 0.0, "lse": False},
        # sixteen sequences of eight beams under grammars, some beams finished, twice the beams kept
        {"name": "beams_batch", "op": "beams", "S": 16, "W": 8, "v": 151936, "n": 0, "keep": 16, "mask": 0.25,
         "finished": 0.2, "lse": False},
        # the retrieved candidates of two sequences of four beams (512 probes of 16 tokens), their sums known
        {"name": "beams_candidates", "op": "beams", "S": 2, "W": 4, "v": 128256, "n": 8192, "keep": 8, "mask": 0.0,
         "finished": 0.0, "lse": True},
        # -- the reordering
        # the token histories of one sequence's beams
        {"name": "reorder_history", "op": "reorder", "S": 1, "W": 4, "count": 1, "H": 0, "L": 1000, "D": 0,
         "heads_first": False},
        # keys and values of eight layers, eight sequences of eight beams
        {"name": "reorder_cache", "op": "reorder", "S": 8, "W": 8, "count": 16, "H": 8, "L": 2000, "D": 64,
         "heads_first": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quant", "product", "product", "head", "beams", "beams", "reorder"))
    if op == "quant":
        dt, d = rng.choice(("bf16", "bf16", "f32")), _log(rng, 64, 8192)
        if rng.random() < 0.6:
            d = (d + 63) // 64 * 64
        norm = rng.random() < 0.7
        top = min(16384, 16384 * 2560 // (d if dt == "bf16" else 2 * d))
        return {"op": op, "B": _log(rng, 1, top), "d": d, "dtype": dt, "norm": norm,
                "residual": norm and rng.random() < 0.6, "out": norm and rng.random() < 0.3}
    if op in ("product", "head"):
        k = _log(rng, 64, 8192)
        if rng.random() < 0.8:
            k = (k + 127) // 128 * 128
        n = _log(rng, 1000, min(262144, 388_000_000 // k))
        if op == "head":
            return {"op": op, "B": _log(rng, 1, max(1, min(256, 33_000_000 // n))), "n": n, "k": k,
                    "T": rng.choice((0.0, 0.75, 1.25)), "logits": rng.random() < 0.5}
        top = min(4096, 41_000_000 // n, 4096 * 10240 * 2560 // (n * k))
        return {"op": op, "B": _log(rng, 1, max(1, top)), "n": n, "k": k, "out": rng.choice(("f32", "bf16"))}
    if op == "beams":
        v = _log(rng, 1000, 262144)
        n = _log(rng, 64, min(v, 32768)) if rng.random() < 0.3 else 0
        W = rng.choice((1, 2, 3, 4, 5, 8, 10, 16, 32))
        S = _log(rng, 1, max(1, min(64, 16 * 8 * 151936 // (v * W))))
        return {"op": op, "S": S, "W": W, "v": v, "n": n, "keep": rng.choice((W, 2 * W)),
                "mask": rng.choice((0.0, 0.01, 0.25, 0.9)), "finished": rng.choice((0.0, 0.2, 0.6)),
                "lse": rng.random() < 0.3}
    W = rng.choice((2, 3, 4, 5, 8, 10, 16, 32))
    if rng.random() < 0.3:
        return {"op": op, "S": _log(rng, 1, 64), "W": W, "count": 1, "H": 0, "L": _log(rng, 16, 32768), "D": 0,
                "heads_first": False}
    H, D, L = rng.choice((1, 2, 4, 8)), rng.choice((64, 80, 128, 130)), _log(rng, 16, 8192)
    S = _log(rng, 1, max(1, min(64, 2 ** 20 * 64 // (W * H * L * D // 16))))
    count = _log(rng, 1, max(1, min(48, 16 * 64 * 8 * 2000 * 64 // (S * W * H * L * D))))
    return {"op": op, "S": S, "W": W, "count": count, "H": H, "L": L, "D": D, "heads_first": rng.random() < 0.6}


def _sampling(T):
    """(mode, temperature) of a call: greedy where T is 0, else tokens sampled at T."""
    return (2, T) if T else (0, 1.0)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    st = {"case": case, "seed": seed}
    if own:
        import lm_output_head_amd
        st["fh"] = lm_output_head_amd
    if case["op"] == "quant":
        B, d, dt = case["B"], case["d"], _DT[case["dtype"]]
        # a residual stream: most channels of order one, a few outlier channels
        chan = torch.ones(d, device=dev)
        chan[torch.randint(0, d, (max(1, d // 256),), generator=g, device=dev)] = 12.0
        st["x"] = (_normal(g, B, d) * chan).to(dt)
        st["r"] = (_normal(g, B, d) * chan * 2).to(dt) if case["residual"] else None
        st["w"] = (_normal(g, d) * 0.2 + 1.0).to(dt) if case["norm"] else None
        return st
    if case["op"] in ("product", "head"):
        B, n, k = case["B"], case["n"], case["k"]
        G, N = (k + 127) // 128, (n + 127) // 128
        # a block's largest weight stands at 448, and so does the largest of 128 activations
        st["w"] = (_normal(g, n, k) * (448.0 / 4.2)).clamp_(-448.0, 448.0).to(_F8)
        st["ws"] = (torch.rand(N, G, generator=g, device=dev) * 0.5 + 0.75) * (4.2 / 448.0 / math.sqrt(k))
        st["q"] = (_normal(g, B, k) * (448.0 / 2.7)).clamp_(-448.0, 448.0).to(_F8)
        st["qs"] = (torch.rand(B, G, generator=g, device=dev) * 0.5 + 0.75) * (3.0 * 2.7 / 448.0)
        if own:  # the weight's handle, laid out once as a program that serves from it does
            st["head"] = st["fh"].FP8Head(codes=st["w"], scales=st["ws"])
        return st
    S, W = case["S"], case["W"]
    if case["op"] == "beams":
        v, n = case["v"], case["n"]
        R, width = S * W, n or v
        st["z"] = _normal(g, R, width) * 3.0
        if case["mask"]:  # what a grammar allows, every other sequence under one
            shut = torch.rand(R, width, generator=g, device=dev) >= case["mask"]
            shut &= (torch.arange(R, device=dev)[:, None] // W) % 2 == 0
            st["z"].masked_fill_(shut, -math.inf)
        st["ids"] = None
        if n:  # distinct tokens in no order, as clusters list them
            at = torch.rand(R, v, generator=g, device=dev).topk(n, dim=1).indices
            st["ids"] = at.to(torch.int32).contiguous()
        # totals of beams some tokens in: near each other, descending
        st["scores"] = (_normal(g, S, W) * 1.5 - 20.0).sort(dim=1, descending=True).values.contiguous()
        st["finished"] = None
        if case["finished"]:
            st["finished"] = (torch.rand(S, W, generator=g, device=dev) < case["finished"]).to(torch.int32)
        st["eos"] = int(v * 0.37)
        st["lse"] = torch.logsumexp(st["z"].double(), 1).float() if case["lse"] else None
        return st
    R, L = S * W, case["L"]
    if case["H"]:
        shape = (R, case["H"], L, case["D"]) if case["heads_first"] else (R, L, case["H"], case["D"])
        st["states"] = [_normal(g, *shape).to(torch.bfloat16) for _ in range(case["count"])]
    else:
        st["states"] = [torch.randint(0, 128256, (R, L), generator=g, device=dev, dtype=torch.int32)]
    st["dim"] = 2 if case["heads_first"] else 1
    # a sequence's beams are of one length; its next beams come from any of them
    st["lengths"] = torch.randint((L + 1) // 2, L + 1, (S, 1), generator=g, device=dev).to(torch.int32).repeat(1, W)
    st["lengths"] = st["lengths"].reshape(-1).contiguous()
    st["parent"] = torch.randint(0, W, (S, W), generator=g, device=dev, dtype=torch.int32)
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


def _choose(z, T, seed):
    """Token, its logit and the log-sum-exp of rows of logits of all tokens."""
    ids = torch.arange(z.shape[1], device=z.device).expand(z.shape)
    x = z / T if T else z
    key = x
    if T:
        rows = torch.arange(z.shape[0], device=z.device)[:, None]
        key = x - torch.log(-torch.log(_uniforms(seed, rows, ids)))
    best = key.amax(1, keepdim=True)
    token = torch.where(key == best, ids, 1 << 40).amin(1)
    top = x.amax(1, keepdim=True)
    return {"token": token.to(torch.int32), "token_logit": z.gather(1, token[:, None])[:, 0],
            "lse": (x - top).exp().sum(1).log() + top[:, 0]}


def _spread(scale, width):
    """[R x G] scales as [R x width], each for its 128 columns."""
    return scale.repeat_interleave(128, 1)[:, :width]


def _plain_quant(st):
    x, d = st["x"], st["case"]["d"]
    y, got = x.float(), {}
    if st["r"] is not None:
        y = y + st["r"].float()
        got["residual"] = y.to(x.dtype)
    if st["w"] is not None:
        y = y * torch.rsqrt((y * y).mean(1, keepdim=True) + 1e-6) * st["w"].float()
        if st["case"]["out"]:
            got["out"] = y.to(x.dtype)
    whole = torch.nn.functional.pad(y, (0, -d % 128)).view(x.shape[0], -1, 128)
    got["q_scale"] = whole.abs().amax(2) / 448.0
    got["q"] = (y / _spread(got["q_scale"], d)).clamp(-448.0, 448.0).to(_F8)
    return got


def _plain_product(st):
    # in slices of the channels: a float32 copy of a whole table would be four times its size
    a = st["q"].float() * _spread(st["qs"], st["case"]["k"])
    rows = 65536
    acc = [a @ (st["w"][lo:lo + rows].float() * _spread(st["ws"][lo // 128:(lo + rows) // 128], st["case"]["k"])
                .repeat_interleave(128, 0)[:st["w"].shape[0] - lo]).T for lo in range(0, st["w"].shape[0], rows)]
    return torch.cat(acc, 1)


def _plain_beams(st):
    case = st["case"]
    S, W, M = case["S"], case["W"], case["keep"]
    z = st["z"].double()
    if st["lse"] is None:
        top = z.amax(1, keepdim=True)
        shift = torch.where(top > -math.inf, top, 0.0)
        lse = (z - shift).exp().sum(1, keepdim=True).log() + shift
    else:
        lse = st["lse"].double()[:, None]
    score = st["scores"].double().view(-1, 1)
    total = torch.where(z > -math.inf, score + (z - lse), -math.inf)
    # a finished beam's one candidate is a last column
    done = torch.zeros_like(score, dtype=torch.bool) if st["finished"] is None else st["finished"].view(-1, 1) != 0
    total = torch.cat((torch.where(done, -math.inf, total), torch.where(done, score, -math.inf)), 1)
    n = total.shape[1]
    # equal totals stay in the order of beam and place
    value, at = total.view(S, W * n).sort(dim=1, descending=True, stable=True)
    value, at = value[:, :M], at[:, :M]
    live = value > -math.inf
    parent, place = at // n, at % n
    row = torch.arange(S, device=z.device)[:, None] * W + parent
    last = place == n - 1
    place = torch.where(last, 0, place)
    token = place if st["ids"] is None else st["ids"][row, place].long()
    token = torch.where(last, st["eos"], token)
    got = {"score": value.float(), "token": torch.where(live, token, -1).to(torch.int32),
           "parent": torch.where(live, parent, -1).to(torch.int32)}
    if st["finished"] is not None:
        got["finished"] = (live & (token == st["eos"])).to(torch.int32)
    return got


def _plain_reorder(st):
    S, W = st["case"]["S"], st["case"]["W"]
    rows = (torch.arange(S, device="cuda")[:, None] * W + st["parent"].long()).view(-1)
    for x in st["states"]:
        shape = [1] * x.dim()
        shape[0], at = x.shape[0], [1] * x.dim()
        at[st["dim"]] = x.shape[st["dim"]]
        here = torch.arange(x.shape[st["dim"]], device="cuda").view(at) < st["lengths"][rows].view(shape)
        x.copy_(torch.where(here, x[rows], x))
    return st["states"]


def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        if op == "quant":
            return _plain_quant(st)
        if op == "beams":
            return _plain_beams(st)
        if op == "reorder":
            return _plain_reorder(st)
        z = _plain_product(st)
        if op == "product":
            return z.to(_DT[case["out"]])
        return {**_choose(z, case["T"], st["seed"]), "logits": z if case["logits"] else None}
    if op == "quant":
        if not case["norm"]:
            return st["fh"].fp8_quant(st["x"])
        return st["fh"].rmsnorm_fp8(st["x"], st["w"], residual=st["r"], eps=1e-6, want_out=case["out"])
    if op == "product":
        return st["head"].matmul(st["q"], st["qs"], dtype=_DT[case["out"]])
    if op == "head":
        mode, T = _sampling(case["T"])
        r = st["head"].forward(st["q"], st["qs"], mode=mode, temperature=T, seed=st["seed"], want_logits=case["logits"])
        return {name: r.get(name) for name in ("token", "token_logit", "lse", "logits")}
    if op == "beams":
        return st["fh"].beam_select(st["z"], st["scores"], keep=case["keep"], ids=st["ids"], v=case["v"],
                                    lse=st["lse"], finished=st["finished"], eos=st["eos"])
    st["fh"].beam_reorder(st["states"], st["parent"], lengths=st["lengths"], length_dim=st["dim"])
    return st["states"]


def work(case):
    op = case["op"]
    if op == "quant":
        B, d, e = case["B"], case["d"], 2 if case["dtype"] == "bf16" else 4
        per = e * (1 + 2 * case["residual"] + case["out"]) + 1
        return {"bytes": B * d * per + d * e * case["norm"] + 4 * B * ((d + 127) // 128),
                "flops": B * d * (8 if case["norm"] else 3)}
    if op in ("product", "head"):
        B, n, k = case["B"], case["n"], case["k"]
        written = B * n * (4 if case["out"] == "f32" else 2) if op == "product" else 12 * B + 4 * B * n * case["logits"]
        scales = 4 * ((k + 127) // 128) * (B + (n + 127) // 128)
        return {"bytes": n * k + B * k + scales + written, "flops": 2 * B * n * k}
    S, W = case["S"], case["W"]
    if op == "beams":
        n = case["n"] or case["v"]
        read = S * W * (1.0 - case["finished"]) * n  # a finished beam's logits do not count
        return {"bytes": 4 * read + 8 * S * W + 16 * S * case["keep"], "flops": read * (1 if case["lse"] else 4)}
    # of beams with any parent, those with another than themselves are written, their distinct parents read;
    # three quarters of the positions count
    row = 0.75 * case["L"] * (2 * case["H"] * case["D"] if case["H"] else 4) * case["count"]
    moved, read = W - 1.0, W * (1.0 - (1.0 - (W - 1.0) / W ** 2) ** W)
    return {"bytes": S * (moved + read) * row + 8 * S * W, "flops": 0}


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definitions in float64; the codes as the quotients that they round."""
    st = prepare(case, seed)
    if case["op"] == "quant":
        s = st["x"].double() + (st["r"].double() if st["r"] is not None else 0.0)
        y = s
        if case["norm"]:
            y = s / (s.pow(2).sum(1, keepdim=True) / case["d"] + 1e-6).sqrt() * st["w"].double()
        got, scale = {"residual": s if case["residual"] else None, "out": y if case["out"] else None}, []
        q = torch.empty_like(y)
        for lo in range(0, case["d"], 128):
            part = y[:, lo:lo + 128]
            scale.append(part.abs().max(1).values / 448)
            q[:, lo:lo + 128] = part / scale[-1][:, None]
        got["q"], got["q_scale"] = q, torch.stack(scale, 1)
        return got
    if case["op"] in ("product", "head"):
        z = torch.zeros(case["B"], case["n"], dtype=torch.float64, device="cuda")
        # block row by block row of the weight, every 128 of k with its scales
        for j in range(0, case["n"], 16384):
            w = st["w"][j:j + 16384].double()
            for i in range(0, case["k"], 128):
                per = st["ws"][j // 128:j // 128 + 128, i // 128].double()
                w[:, i:i + 128] *= per[:, None].expand(-1, 128).reshape(-1)[:w.shape[0], None]
            a = st["q"].double()
            for i in range(0, case["k"], 128):
                a[:, i:i + 128] *= st["qs"][:, i // 128].double()[:, None]
            z[:, j:j + 16384] = torch.mm(a, w.t().contiguous())
        if case["op"] == "product":
            return z
        T = case["T"] or 1.0
        return {"token": None, "token_logit": None if case["T"] else z.max(1).values,
                "lse": torch.logsumexp(z / T, 1), "logits": z if case["logits"] else None}
    S, W = case["S"], case["W"]
    if case["op"] == "beams":
        M, score = case["keep"], torch.full((S, case["keep"]), -math.inf, dtype=torch.float64, device="cuda")
        for s in range(S):
            best = []
            for w in range(W):
                if st["finished"] is not None and int(st["finished"][s, w]):
                    best.append(st["scores"][s, w].double()[None])
                    continue
                z = st["z"][s * W + w].double()
                lse = torch.logsumexp(z, 0) if st["lse"] is None else st["lse"][s * W + w].double()
                z = z[z > -math.inf].topk(min(M, int((z > -math.inf).sum()))).values
                best.append(st["scores"][s, w].double() + z - lse)
            best = torch.cat(best).sort(descending=True).values[:M]
            score[s, :best.numel()] = best
        return {"score": score, "token": None, "parent": None, "finished": None}
    if not case["H"]:
        return None  # whole numbers
    got = []
    for x in st["states"]:
        new = x.clone()
        for s in range(S):
            length = int(st["lengths"][s * W])
            for m in range(W):
                new[s * W + m].narrow(st["dim"] - 1, 0, length).copy_(
                    x[s * W + int(st["parent"][s, m])].narrow(st["dim"] - 1, 0, length))
        got.append(new.double())
    return got
