"""The serving operators' cases: their inputs, plain forms, 64-bit values and work.

Four operators of a served mixture-of-experts model whose weights are FP8 / FP4 codes:

* ``route``: the router, logits [T, E] -> the k best experts of a token and their weights;
* ``group``: positions sorted by group (expert or adapter) with the groups' offsets;
* ``moe``: the whole mixture-of-experts layer for a few tokens, from router logits to output;
* ``lora``: the low-rank adapters of many requests added beside a shared projection's output.

``own`` chooses what ``run`` computes with: False, elementary torch operations in 32 bits;
True, the package's entry points.  Both get the same state.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases --------------------------------------------------------------------
def _route(name, T, E, k, dtype, scoring="softmax", renormalize=True, masked=False):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "dtype": dtype,
            "scoring": scoring, "renormalize": renormalize, "masked": masked}


def _group(name, n, G, skew, dropped):
    return {"name": name, "op": "group", "n": n, "G": G, "skew": skew, "dropped": dropped}


def _moe(name, T, H, I, E, k, fmt, mode, dtype, scoring="softmax", activation="silu"):
    return {"name": name, "op": "moe", "T": T, "H": H, "I": I, "E": E, "k": k, "fmt": fmt,
            "mode": mode, "dtype": dtype, "scoring": scoring, "activation": activation}


def _lora(name, M, K, N, r, G, dtype, runs, plan="kept", activation="none"):
    return {"name": name, "op": "lora", "M": M, "K": K, "N": N, "r": r, "G": G, "dtype": dtype,
            "runs": runs, "plan": plan, "activation": activation}


def listed():
    return [
        # one token's routing while it decodes, eight experts: nothing but latency
        _route("route_1", 1, 8, 2, "f32"),
        # a prompt's tokens over many small experts, sigmoid scores
        _route("route_prompt", 4096, 256, 8, "bf16", "sigmoid"),
        # a decode step's rows by the adapter that each request asked for (some have none)
        _group("group_step", 61, 32, 0.5, 0.2),
        # the (token, slot) pairs of 16384 tokens sorted for the grouped GEMM, eight experts
        _group("group_prompt", 32768, 8, 0.3, 0.0),
        # one user decoding: one token, two of eight large experts, per-row scales
        _moe("moe_1", 1, 4096, 14336, 8, 2, "e4m3", "rowwise", "bf16"),
        # a few users over many small experts of a ragged width, block scales
        _moe("moe_7_small_experts", 7, 2048, 1376, 64, 6, "e4m3", "mx32", "f16", "sigmoid"),
        # a medium batch with 4-bit experts
        _moe("moe_32_fp4", 32, 4096, 14336, 8, 2, "e2m1", "mx32", "bf16"),
        # the largest decode batch: every expert is read, 32 tokens each
        _moe("moe_128", 128, 4096, 14336, 8, 2, "e4m3", "rowwise", "bf16"),
        # one request with an adapter, square projection
        _lora("lora_1", 1, 4096, 4096, 16, 8, "bf16", 1),
        # a decode step: every row a request of its own, an up projection
        _lora("lora_64", 64, 4096, 14336, 32, 32, "bf16", 1),
        # odd everything, the rows sorted in the call, the activation fused
        _lora("lora_odd", 333, 2064, 1000, 24, 11, "f16", 9, "called", "silu"),
        # prompts: long runs of rows with the same adapter
        _lora("lora_prompt", 8192, 4096, 4096, 64, 8, "bf16", 700),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "group", "moe", "moe", "lora", "lora"])
    if op == "route":
        E = _log_int(rng, 4, 512)
        c = _route("", _log_int(rng, 1, 16384), E, rng.randint(1, min(8, E)),
                   rng.choice(["f32", "bf16", "f16"]), rng.choice(["softmax", "sigmoid"]),
                   rng.random() < 0.7, rng.random() < 0.3)
    elif op == "group":
        c = _group("", _log_int(rng, 1, 65536), _log_int(rng, 1, 256), round(rng.random(), 3),
                   rng.choice([0.0, 0.1, 0.5]))
    elif op == "moe":
        fmt, mode = rng.choice([("e4m3", "rowwise"), ("e4m3", "mx32"), ("e4m3", "tensor"),
                                ("e2m1", "mx32")])
        unit = 16 if mode != "mx32" else 32
        H = _log_int(rng, 512, 4096) // unit * unit
        inner = _log_int(rng, 256, 14336) // unit * unit
        E = min(_log_int(rng, 4, 128), 8 * 4096 * 14336 // (H * inner))
        c = _moe("", _log_int(rng, 1, 128), H, inner, E, rng.randint(1, min(8, E)), fmt, mode,
                 rng.choice(["bf16", "f16"]), rng.choice(["softmax", "sigmoid"]),
                 rng.choice(["silu", "silu", "gelu"]))
        # no more (token, slot) products than the largest listed case
        c["T"] = max(1, min(c["T"], 128 * 2 * 4096 * 14336 // (c["k"] * H * inner)))
    else:
        M = _log_int(rng, 1, 8192)
        c = _lora("", M, _log_int(rng, 512, 8192) // 8 * 8, _log_int(rng, 256, 14336),
                  8 * rng.randint(1, 16), _log_int(rng, 1, 64), rng.choice(["bf16", "f16"]),
                  _log_int(rng, 1, 1024), rng.choice(["kept", "called"]),
                  rng.choice(["none", "none", "silu"]))
        if M > 1024:                      # prompts: no more than the largest listed case
            c["r"] = min(c["r"], 64)
            c["G"] = min(c["G"], 8)
            c["N"] = min(c["N"], 4096)
            c["K"] = min(c["K"], 4096)
    del c["name"]
    return c


# ---- inputs -------------------------------------------------------------------
def _quantize(w, fmt, mode):
    """fp32 [R, K] -> codes uint8 [R, K or K/2] and scales, as a model's weights are stored."""
    if mode == "tensor":
        s = w.abs().amax() / 448.0
        return (w / s).to(torch.float8_e4m3fn).view(torch.uint8), s.view(1)
    if mode == "rowwise":
        s = w.abs().amax(1) / 448.0
        return (w / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), s
    b = w.view(w.shape[0], -1, 32)
    e = torch.frexp(b.abs().amax(2)).exponent - 1 - (8 if fmt == "e4m3" else 2)
    v = torch.ldexp(b, -e[:, :, None]).view(w.shape)
    scales = (e + 127).to(torch.uint8)
    if fmt == "e4m3":
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scales
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    c = torch.bucketize(v.abs(), edges).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    return c[:, 0::2] | (c[:, 1::2] << 4), scales


def _expert_weights(gen, E, N, K, fmt, mode):
    codes, scales = [], []
    for _ in range(E):
        w = torch.randn(N, K, generator=gen, device="cuda") * 0.02
        q, s = _quantize(w, fmt, mode)
        codes.append(q)
        scales.append(s)
    return torch.stack(codes), torch.cat(scales) if mode != "mx32" else torch.stack(scales)


def _logits(gen, T, E, dtype):
    """Router logits: some experts are preferred by every token."""
    return (1.5 * torch.randn(T, E, generator=gen, device="cuda")
            + 0.7 * torch.randn(1, E, generator=gen, device="cuda")).to(dtype)


def _activations(gen, M, K, dtype):
    """Normalised activations: unit variance, one channel in 128 ten times as large."""
    x = torch.randn(M, K, generator=gen, device="cuda")
    x[:, torch.rand(K, generator=gen, device="cuda") < 1 / 128] *= 10.0
    return x.to(dtype)


def _row_groups(gen, n, G, skew, dropped, runs):
    """Group of each position: runs of equal ones, low groups preferred by `skew`, -1 for none."""
    k = (n + runs - 1) // runs
    u = torch.rand(k, generator=gen, device="cuda") ** (1.0 + 2.0 * skew)
    g = (u * G).to(torch.int32).clamp(0, G - 1)
    g[torch.rand(k, generator=gen, device="cuda") < dropped] = -1
    return g.repeat_interleave(runs)[:n].contiguous()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    s = dict(c)
    if c["op"] == "route":
        s["logits"] = _logits(gen, c["T"], c["E"], _DT[c["dtype"]])
        if c["masked"]:          # experts that are switched off for a token; expert 0 never is
            off = torch.rand(c["T"], c["E"], generator=gen, device="cuda") < 0.3
            off[:, 0] = False
            s["logits"][off] = -math.inf
    elif c["op"] == "group":
        s["ids"] = _row_groups(gen, c["n"], c["G"], c["skew"], c["dropped"], 1)
    elif c["op"] == "moe":
        s["logits"] = _logits(gen, c["T"], c["E"], torch.float32)
        s["x"] = _activations(gen, c["T"], c["H"], _DT[c["dtype"]])
        s["qw13"], s["sw13"] = _expert_weights(gen, c["E"], 2 * c["I"], c["H"], c["fmt"], c["mode"])
        s["qw2"], s["sw2"] = _expert_weights(gen, c["E"], c["H"], c["I"], c["fmt"], c["mode"])
    else:
        dt = _DT[c["dtype"]]
        s["x"] = _activations(gen, c["M"], c["K"], dt)
        pitch = (c["N"] + 7) // 8 * 8
        s["base"] = torch.randn(c["M"], pitch, generator=gen, device="cuda").to(dt)[:, :c["N"]]
        s["a"] = (torch.randn(c["G"], c["r"], c["K"], generator=gen, device="cuda")
                  / math.sqrt(c["K"])).to(dt)
        s["b"] = (0.1 * torch.randn(c["G"], c["N"], c["r"], generator=gen, device="cuda")).to(dt)
        s["scales"] = 0.5 + torch.rand(c["G"], generator=gen, device="cuda")
        s["ids"] = _row_groups(gen, c["M"], c["G"], 0.3, 0.0 if c["M"] == 1 else 0.1, c["runs"])
        if c["plan"] == "kept":  # one sort serves every projection of a step
            s["order"], s["offsets"] = _plain_group(s["ids"], c["G"])
    return s


# ---- plain forms --------------------------------------------------------------
def _scores(logits, k, scoring, renormalize):
    """The k largest logits of a row (ties: lowest expert first) and their weights."""
    f = logits.float()
    top, ids = torch.sort(f, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k].to(torch.int32)
    if scoring == "sigmoid":
        w = 1.0 / (1.0 + torch.exp(-top))
    else:
        m = f.amax(1, keepdim=True)
        w = torch.exp(top - m) / torch.exp(f - m).sum(1, keepdim=True)
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    none = torch.isneginf(top)
    return ids.masked_fill(none, -1), w.masked_fill(none, 0.0)


def _plain_group(ids, G):
    key = torch.where((ids >= 0) & (ids < G), ids, G)
    order = torch.sort(key, stable=True).indices.to(torch.int32)
    per = torch.zeros(G + 1, dtype=torch.int32, device=ids.device)
    per.index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(G + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(per[:G], 0)
    return order, offsets


def _weights32(q, s, fmt, mode, pick):
    """Codes [E, N, K or K/2] and scales -> fp32 weights [P, N, K] of the experts `pick`."""
    E, N = q.shape[:2]
    if pick is not None:
        q = q[pick]
    if fmt == "e4m3":
        w = q.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=q.device)
        w = torch.stack((table[(q & 15).int()], table[(q >> 4).int()]), -1).flatten(2)
    if mode == "mx32":
        s = s if pick is None else s[pick]
        w = w.view(w.shape[0], N, -1, 32) * torch.exp2(s.float() - 127.0)[..., None]
        return w.flatten(2)
    s = s.view(E, -1, 1) if pick is None else s.view(E, -1, 1)[pick]
    return w * s


def _act(v, kind):
    if kind == "silu":
        return v / (1.0 + torch.exp(-v))
    if kind == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v / math.sqrt(2.0)))
    return v


def _plain_moe(s):
    ids, w = _scores(s["logits"], s["k"], s["scoring"], True)
    x = s["x"].float()
    pairs = s["T"] * s["k"]
    if pairs <= s["E"]:               # few pairs: each with its own expert's weights
        pick = ids.flatten().long()
        xs = x.repeat_interleave(s["k"], 0)[:, None, :]
    else:                             # every expert on every token, the others weighted zero
        pick = None
        xs = x.expand(s["E"], -1, -1)
    w13 = _weights32(s["qw13"], s["sw13"], s["fmt"], s["mode"], pick)
    gu = torch.matmul(xs, w13.transpose(1, 2))
    del w13
    h = _act(gu[..., :s["I"]], s["activation"]) * gu[..., s["I"]:]
    w2 = _weights32(s["qw2"], s["sw2"], s["fmt"], s["mode"], pick)
    y = torch.matmul(h, w2.transpose(1, 2))
    if pick is not None:
        y = (y.view(s["T"], s["k"], -1) * w[..., None]).sum(1)
    else:
        part = torch.zeros(s["T"], s["E"], device=x.device).scatter_add_(1, ids.long(), w)
        y = (y * part.t()[..., None]).sum(0)
    return {"out": y.to(s["x"].dtype), "ids": ids, "weights": w}


def _plain_lora(s):
    G, r = s["a"].shape[:2]           # every row through every adapter, the others zeroed
    v = torch.matmul(s["x"].float(), s["a"].float().view(G * r, -1).t()).view(-1, G, r)
    mine = s["ids"][:, None] == torch.arange(G, device=v.device)
    v = v * (mine * s["scales"])[..., None]
    d = torch.matmul(v.view(-1, G * r), s["b"].float().transpose(1, 2).reshape(G * r, -1))
    return _act(s["base"].float() + d, s["activation"]).to(s["x"].dtype)


def run(s):
    if own:
        import block_scaled_gemm_fp8gemm_amd as F
    if s["op"] == "route":
        if own:
            return F.moe_route(s["logits"], s["k"], s["scoring"], s["renormalize"])
        return _scores(s["logits"], s["k"], s["scoring"], s["renormalize"])
    if s["op"] == "group":
        return F.group_rows(s["ids"], s["G"]) if own else _plain_group(s["ids"], s["G"])
    if s["op"] == "moe":
        if not own:
            return _plain_moe(s)
        out, ids, weights = F.moe_layer(s["x"], s["logits"], s["qw13"], s["sw13"], s["qw2"],
                                        s["sw2"], s["k"], s["mode"], s["fmt"], s["scoring"],
                                        activation=s["activation"])
        return {"out": out, "ids": ids, "weights": weights}
    if not own:
        return _plain_lora(s)
    if s["plan"] == "called":
        order, offsets = F.group_rows(s["ids"], s["G"])
    else:
        order, offsets = s["order"], s["offsets"]
    return F.lora(s["x"], s["base"], s["a"], s["b"], order, offsets, s["scales"],
                  s["activation"])


# ---- work ---------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["T"] * c["E"] * size + c["T"] * c["k"] * 8,
                "flops": 3 * c["T"] * c["E"]}
    if c["op"] == "group":
        return {"bytes": 8 * c["n"] + 4 * (c["G"] + 1), "flops": c["n"]}
    if c["op"] == "moe":
        used = c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])    # experts read, expected
        per = 3 * c["H"] * c["I"]
        size = {"e4m3": 1.0, "e2m1": 0.5}[c["fmt"]] + (1 / 32 if c["mode"] == "mx32" else 0.0)
        return {"bytes": int(used * per * size) + 4 * c["T"] * c["H"] + 4 * c["T"] * c["E"],
                "flops": 2 * c["T"] * c["k"] * per}
    rows = max(1, round(0.9 * c["M"]))
    segments = max(1, -(-rows // c["runs"]))
    used = c["G"] * (1.0 - (1.0 - 1.0 / c["G"]) ** segments)
    return {"bytes": 2 * c["M"] * (c["K"] + 2 * c["N"]) + int(2 * used * c["r"] * (c["K"] + c["N"])),
            "flops": 2 * rows * c["r"] * (c["K"] + c["N"])}


# ---- values in 64 bits, written from the definitions -----------------------------
def _route64(logits, k, scoring, renormalize):
    l = logits.double().cpu()
    order = torch.argsort(l, dim=1, descending=True, stable=True)[:, :k]
    p = torch.sigmoid(l) if scoring == "sigmoid" else torch.softmax(l, 1)
    w = torch.gather(p, 1, order)
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    gone = torch.gather(l, 1, order) == -math.inf
    return order.masked_fill(gone, -1).to(torch.int32), w.masked_fill(gone, 0.0)


def _decode64(q, s, fmt, mode, e, N):
    """fp64 weights [N, K] of expert e."""
    c = q[e].int()
    if fmt == "e4m3":
        sign = 1.0 - 2.0 * (c >> 7).double()
        ex, man = (c >> 3) & 15, (c & 7).double()
        v = sign * torch.where(ex > 0, (1.0 + man / 8.0) * torch.exp2(ex.double() - 7.0),
                               man * 2.0 ** -9)
    else:
        c = torch.stack((c & 15, c >> 4), -1).flatten(1)
        ex, man = (c >> 1) & 3, (c & 1).double()
        v = torch.where(ex > 0, (1.0 + man / 2.0) * torch.exp2(ex.double() - 1.0), man / 2.0)
        v = v * (1.0 - 2.0 * (c >> 3).double())
    if mode == "mx32":
        return (v.view(N, -1, 32) * torch.exp2(s[e].double() - 127.0)[..., None]).view(N, -1)
    if mode == "rowwise":
        return v * s.view(-1, N)[e].double()[:, None]
    return v * s[e].double()


def _act64(v, kind):
    if kind == "silu":
        return v * torch.sigmoid(v)
    if kind == "gelu":
        return v * torch.special.ndtr(v)
    return v


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _route64(s["logits"], s["k"], s["scoring"], s["renormalize"])
    if case["op"] == "group":
        return None                       # whole numbers: compared as they are
    if case["op"] == "moe":
        ids, w = _route64(s["logits"], s["k"], s["scoring"], True)
        x = s["x"].double()
        y = torch.zeros(s["T"], s["H"], dtype=torch.float64, device=x.device)
        for e in range(s["E"]):
            rows, slots = torch.nonzero(ids == e, as_tuple=True)
            if not rows.numel():
                continue
            w13 = _decode64(s["qw13"], s["sw13"], s["fmt"], s["mode"], e, 2 * s["I"])
            xe = x[rows.to(x.device)]
            h = _act64(xe @ w13[:s["I"]].t(), s["activation"]) * (xe @ w13[s["I"]:].t())
            del w13
            w2 = _decode64(s["qw2"], s["sw2"], s["fmt"], s["mode"], e, s["H"])
            y.index_add_(0, rows.to(x.device), (h @ w2.t()) * w[rows, slots].to(x.device)[:, None])
        return {"out": y, "ids": None, "weights": w}
    x, out = s["x"].double(), s["base"].double().clone()
    for g in range(s["G"]):
        rows = torch.nonzero(s["ids"] == g).flatten()
        if rows.numel():
            v = x[rows] @ s["a"][g].double().t()
            out[rows] += s["scales"][g].double() * (v @ s["b"][g].double().t())
    return _act64(out, s["activation"])
