"""Cases of the whole-layer operators for serving: the Mixture-of-Experts layer for a few tokens in one kernel
(``MoELayer.decode``) and the layer with low-rank adapters of many requests beside its expert projections
(``MoELayer.decode`` and ``MoELayer.forward`` with adapters).

A case is a dict: ``op`` ("decode": up to 64 tokens, "forward": any number), the layer's sizes (S tokens, width d, E experts,
K per token, hidden width h, ``shared`` always-on expert), its router (softmax or sigmoid, group limit), the expert weights'
type ("bf16", or "e4m3" codes with a scale per output channel), the activation, and the adapters (``adapters`` = their
number, 0 for none, ``rank``).

The layer: y = sum_k g_k E_k(x), E(x) = (silu(x Wg') * (x Wu')) Wd' or gelu(x W1' + b1) W2' + b2, where a projection
W' of a token with adapter a and expert e is W[e] + scale[a] B[a][e] A[a][e].
"""
import math

import torch

own = False

ROUTER_BIAS_VAR = 0.5  # per-expert logit offsets: uneven expert loads, as a trained router has them


def _case(name, op, S, d, E, K, h, weights="bf16", act="swiglu", score="softmax", groups=1, topk_groups=1, shared=0,
          adapters=0, rank=0, spread="mixed"):
    c = dict(op=op, S=S, d=d, E=E, K=K, h=h, weights=weights, act=act, score=score, groups=groups,
             topk_groups=topk_groups, shared=shared, adapters=adapters, rank=rank, spread=spread)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one stream of a chat: a single token through a Mixtral-shaped layer, where latency is all
        _case("decode_mixtral_bf16_s1", "decode", 1, 4096, 8, 2, 14336),
        # a small batch of streams: every expert is touched by a token or two
        _case("decode_mixtral_bf16_s8", "decode", 8, 4096, 8, 2, 14336),
        # the same single token with the experts stored in 8 bits
        _case("decode_mixtral_e4m3_s1", "decode", 1, 4096, 8, 2, 14336, weights="e4m3"),
        # a server's ordinary decode batch over 8-bit experts, an odd number of streams
        _case("decode_mixtral_e4m3_s31", "decode", 31, 4096, 8, 2, 14336, weights="e4m3"),
        # two streams through a DeepSeek-shaped layer: many fine experts, sigmoid router with groups, a shared expert
        _case("decode_dsv3_bf16_s2", "decode", 2, 7168, 256, 8, 2048, score="sigmoid", groups=8, topk_groups=2, shared=1),
        # the smallest call: a narrow GeLU layer with odd widths, as in a draft model
        _case("decode_gelu_odd_s3", "decode", 3, 1000, 8, 2, 1352, act="gelu"),
        # a full batch of the widest kind that the decode call takes, over fine 8-bit experts
        _case("decode_fine_e4m3_s64", "decode", 64, 2048, 64, 8, 1408, weights="e4m3"),
        # a decode batch of 16 requests with adapters of their own
        _case("adapters_decode_mixtral_s16", "decode", 16, 4096, 8, 2, 14336, adapters=8, rank=16),
        # many customers' adapters of a higher rank over 8-bit experts, one token each
        _case("adapters_decode_fine_e4m3_s33", "decode", 33, 2048, 64, 8, 1408, weights="e4m3", adapters=32, rank=64),
        # prompts of several requests in one prefill batch, each run of tokens with its adapter
        _case("adapters_prefill_mixtral_s2048", "forward", 2048, 4096, 8, 2, 14336, adapters=4, rank=16, spread="runs"),
        # a ragged prefill batch over fine 8-bit experts with more adapters
        _case("adapters_prefill_fine_e4m3_s3001", "forward", 3001, 2048, 64, 8, 1408, weights="e4m3", adapters=12, rank=32,
              spread="runs"),
        # prompts' tails and single tokens in one batch: every token has another adapter than its neighbour
        _case("adapters_mixed_gelu_s333", "forward", 333, 1000, 8, 2, 1352, act="gelu", adapters=16, rank=8),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return min(hi, max(lo, int(v) // step * step))


def draw(rng):
    e4m3 = rng.random() < 0.5
    step = 16 if e4m3 else 8
    act = "swiglu" if e4m3 or rng.random() < 0.75 else "gelu"
    E = rng.choice([4, 8, 8, 16, 32, 60, 64, 128])
    K = rng.choice([k for k in (1, 2, 2, 4, 6, 8) if k <= E // 2])
    kind = rng.choice(["decode", "decode", "adapters", "adapters", "forward"])
    d = _log_int(rng, 512, 4096, step)
    h = max(512 // step * step, min(14336, _log_int(rng, 512, 14336, step), int(4.0e8 / (E * d)) // step * step))
    score = rng.choice(["softmax", "softmax", "sigmoid"])
    groups = 4 if score == "sigmoid" and E in (16, 32, 64, 128) else 1
    topk_groups = 2 if groups > 1 else 1
    if topk_groups * (E // groups) < K:
        groups = topk_groups = 1
    shared = rng.choice([0, 0, 1])
    most = int(1.4e12 / (6 * (K + shared) * d * h))
    S = _log_int(rng, 1, 64) if kind != "forward" else _log_int(rng, 65, max(65, min(3001, most)))
    n = 0 if kind == "decode" else rng.randint(1, 16 if E >= 60 else 32)
    r = 0 if n == 0 else rng.choice([8, 16, 16, 32, 64])
    return _case(None, "forward" if kind == "forward" else "decode", S, d, E, K, h, weights="e4m3" if e4m3 else "bf16",
                 act=act, score=score, groups=groups, topk_groups=topk_groups, shared=shared, adapters=n, rank=r,
                 spread=rng.choice(["mixed", "runs"]))


def _normal(gen, shape, var, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * math.sqrt(var)).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 17)
    S, d, E, h, ns = case["S"], case["d"], case["E"], case["h"], case["shared"]
    e4m3, bf16 = case["weights"] == "e4m3", torch.bfloat16

    def stack(n, k):
        """[E + ns][n][k] weights ~ N(0, 1/k): bf16, or E4M3 codes with a scale per output channel."""
        w = torch.empty((E + ns, n, k), dtype=torch.uint8 if e4m3 else bf16, device="cuda")
        s = torch.empty((E + ns, n), device="cuda") if e4m3 else None
        for i in range(E + ns):
            t = _normal(gen, (n, k), 1.0 / k)
            if e4m3:
                s[i] = t.abs().amax(1).clamp_min(1e-30) / 448
                w[i] = (t / s[i][:, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                w[i] = t
        return w, s

    st = dict(case=dict(case), x=_normal(gen, (S, d), 1.0, bf16))
    w = dict(w_router=_normal(gen, (E, d), 1.0 / d, bf16), router_bias=None, sel_bias=None)
    if case["score"] == "softmax":
        w["router_bias"] = _normal(gen, (E,), ROUTER_BIAS_VAR)
    else:
        w["sel_bias"] = _normal(gen, (E,), 0.01)
    if case["act"] == "gelu":
        w["w1"], _ = stack(h, d)
        w["w2"], _ = stack(d, h)
        w["b1"], w["b2"] = _normal(gen, (E + ns, h), 0.01), _normal(gen, (E + ns, d), 0.01)
    else:
        w["w_gate"], w["s_gate"] = stack(h, d)
        w["w_up"], w["s_up"] = stack(h, d)
        w["w_down"], w["s_down"] = stack(d, h)
    st["weights"] = w
    st["adapters"] = st["ids"] = None
    n, r = case["adapters"], case["rank"]
    if n:
        a = dict(scale=torch.rand((n,), generator=gen, device="cuda") + 0.5)  # alpha / rank
        for name, out, inp in (("gate", h, d), ("up", h, d), ("down", d, h)):
            if name == "gate" and case["act"] == "gelu":
                continue
            a["a_" + name] = torch.stack([_normal(gen, (E + ns, r, inp), 1.0 / inp, bf16) for _ in range(n)])
            a["b_" + name] = torch.stack([_normal(gen, (E + ns, out, r), 0.1 / r, bf16) for _ in range(n)])
        st["adapters"] = a
        if case["spread"] == "runs":  # prompts one after another: about 4 n runs, some without an adapter
            runs = torch.randint(-1, n, (4 * n,), generator=gen, device="cuda", dtype=torch.int32)
            at = torch.sort(torch.randint(0, 4 * n, (S,), generator=gen, device="cuda")).values
            st["ids"] = runs[at].contiguous()
        else:
            st["ids"] = torch.randint(-1, n, (S,), generator=gen, device="cuda", dtype=torch.int32)
    if own:
        from mixture_experts_layer_bias_b200 import synthetic as syn
        from mixture_experts_layer_bias_b200.layer import MoELayer

        cfg = syn.LayerConfig(
            "layer", S=S, d=d, E=E, K=case["K"], h=h, score_fn=syn.SOFTMAX if case["score"] == "softmax" else syn.SIGMOID,
            num_groups=case["groups"], topk_groups=case["topk_groups"], num_shared=ns,
            activation=syn.SWIGLU if case["act"] == "swiglu" else syn.GELU, weight_dtype=syn.E4M3 if e4m3 else syn.BF16)
        st["layer"] = MoELayer(cfg, w, S=S, adapters=st["adapters"])
    return st


def _route(case, w, x):
    """Experts [S, K] in descending order of their keys and gates; in 64 bits, so that no close pair of keys is swapped."""
    E, G = case["E"], case["groups"]
    logits = x.double() @ w["w_router"].double().T
    if w["router_bias"] is not None:
        logits = logits + w["router_bias"].double()
    score = logits if case["score"] == "softmax" else torch.sigmoid(logits)
    key = score if w["sel_bias"] is None else score + w["sel_bias"].double()
    if G > 1:
        by_group = key.view(-1, G, E // G).sum(2)
        rank = torch.sort(by_group, dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        kept = torch.zeros_like(by_group, dtype=torch.bool).scatter_(1, rank, True)
        key = key.masked_fill(~kept.repeat_interleave(E // G, dim=1), -math.inf)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :case["K"]]
    picked = score.gather(1, idx)
    gates = torch.softmax(picked, 1) if case["score"] == "softmax" else picked / picked.sum(1, keepdim=True)
    return idx, gates.float()


def _projection(w, scale, rows, idx, dense):
    """rows [S, K, in] of tokens with experts idx [S, K] times their experts' weights, [S, K, out], in 32 bits. dense: every
    expert's product with every token, one batched product; else the slots' weights are picked first."""
    w = w.view(torch.float8_e4m3fn) if w.dtype == torch.uint8 else w
    S, K, n = rows.shape
    if not dense:
        at = idx.reshape(-1)
        m = w.view(torch.uint8)[at].view(w.dtype).float()
        m = m if scale is None else m * scale[at][:, :, None]
        return torch.bmm(m, rows.reshape(S * K, n, 1)).view(S, K, -1)
    m = w.float()
    m = m if scale is None else m * scale[:, :, None]
    t = torch.arange(S, device=rows.device)[:, None].expand(S, K)
    every = rows.new_zeros((w.shape[0], S, n))
    every[idx, t] = rows
    return torch.bmm(every, m.transpose(1, 2))[idx, t]


def _adapted(st, name, rows, idx):
    """scale[a] B[a][e] A[a][e] row for the slots' experts idx and their tokens' adapters; zero where a token has none."""
    a, ids = st["adapters"], st["ids"].long()
    S, K = idx.shape
    at = ids.clamp_min(0)[:, None].expand(S, K)
    u = (a["a_" + name][at, idx].float() @ rows[..., None])
    out = (a["b_" + name][at, idx].float() @ u).squeeze(-1) * a["scale"][at][..., None]
    return torch.where((ids >= 0)[:, None, None], out, 0.0)


def _expert_rows(st, rows, idx, dense):
    w, case = st["weights"], st["case"]

    def project(name, weight, x):
        y = _projection(w[weight], w.get("s_" + name), x, idx, dense)
        return y if st["adapters"] is None else y + _adapted(st, name, x, idx)

    if case["act"] == "gelu":
        z = project("up", "w1", rows) + w["b1"][idx]
        hid = 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
        return project("down", "w2", hid) + w["b2"][idx]
    g = project("gate", "w_gate", rows)
    return project("down", "w_down", g * torch.sigmoid(g) * project("up", "w_up", rows))


def run(state):
    case, x = state["case"], state["x"]
    if own:
        layer = state["layer"]
        y = (layer.decode if case["op"] == "decode" else layer.forward)(x, adapter_ids=state["ids"])
        return dict(y=y, experts=layer.topk_idx, gates=layer.topk_w, counts=layer.counts)
    S, K, E = case["S"], case["K"], case["E"]
    idx, gates = _route(case, state["weights"], x)
    rows = x.float()[:, None, :]
    y = (_expert_rows(state, rows.expand(S, K, -1), idx, S * K >= E) * gates[:, :, None]).sum(1)
    if case["shared"]:
        y = y + _expert_rows(state, rows, torch.full((S, 1), E, device=x.device), S >= E + 1)[:, 0]
    counts = (idx.reshape(-1, 1) == torch.arange(E, device=x.device)).sum(0)
    return dict(y=y.to(torch.bfloat16), experts=idx.int(), gates=gates, counts=counts.int())


def _touched(n, share, times):
    """Expected number of distinct ones of n things, each met with this share, `times` times."""
    return n * (1.0 - (1.0 - share) ** times)


def work(case):
    S, d, E, K, h, ns, n, r = (case[k] for k in ("S", "d", "E", "K", "h", "shared", "adapters", "rank"))
    mats = 3 if case["act"] == "swiglu" else 2
    size = 1 if case["weights"] == "e4m3" else 2
    used = _touched(E, K / E, S) + ns
    rows = S * (K + ns)
    read = used * mats * h * d * size + E * d * 2 + S * d * 2 + (used * (2 * h + d) * 4 if size == 1 else 0)
    flops = 2.0 * rows * mats * h * d + 2.0 * S * E * d
    if n:
        with_adapter = n / (n + 1.0)
        pairs = _touched(n * E, with_adapter * K / (n * E), S) + ns * _touched(n, 1.0 / (n + 1), S)
        per = r * ((mats - 1) * (d + h) + (h + d))
        read += pairs * per * 2 + S * 4
        flops += 2.0 * rows * with_adapter * per
    return {"bytes": read + S * d * 2 + S * K * 8 + E * 4, "flops": flops}


def exact(case, seed):
    """The layer expert by expert in 64 bits."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    w, ad, f64 = st["weights"], st["adapters"], torch.float64
    x = st["x"].to(f64)
    S, K, E, r_ = case["S"], case["K"], case["E"], torch.arange(case["S"], device="cuda")
    z = torch.einsum("sd,ed->se", x, w["w_router"].to(f64))
    if w["router_bias"] is not None:
        z += w["router_bias"].to(f64)
    s = z if case["score"] == "softmax" else 1 / (1 + torch.exp(-z))
    key = s.clone() if w["sel_bias"] is None else s + w["sel_bias"].to(f64)
    if case["groups"] > 1:
        size = E // case["groups"]
        total = torch.stack([key[:, g * size:(g + 1) * size].sum(1) for g in range(case["groups"])], 1)
        best = torch.zeros_like(total)
        left = total.clone()
        for _ in range(case["topk_groups"]):
            at = left.argmax(1)
            best[r_, at] = 1
            left[r_, at] = -math.inf
        key[best.repeat_interleave(size, 1) == 0] = -math.inf
    picks = []
    for _ in range(K):
        at = key.argmax(1)
        picks.append(at)
        key[r_, at] = -math.inf
    experts = torch.stack(picks, 1)
    top = s.gather(1, experts)
    gates = torch.exp(top - top.max(1, keepdim=True).values) if case["score"] == "softmax" else top
    gates = gates / gates.sum(1, keepdim=True)

    def value(name, e):
        m = w[name][e]
        if m.dtype == torch.uint8:
            return m.view(torch.float8_e4m3fn).to(f64) * w["s_" + name[2:]][e].to(f64)[:, None]
        return m.to(f64)

    def adapters_of(y, which, rows, tokens, e):
        if ad is None:
            return y
        ids = st["ids"][tokens]
        for a in range(case["adapters"]):
            m = (ids == a).nonzero()[:, 0]
            if len(m):
                y[m] += (rows[m] @ ad["a_" + which][a, e].to(f64).T) @ ad["b_" + which][a, e].to(f64).T * float(ad["scale"][a])
        return y

    y = torch.zeros_like(x)
    for e in range(E + case["shared"]):
        tokens, slot = (experts == e).nonzero(as_tuple=True) if e < E else (r_, None)
        if not len(tokens):
            continue
        rows = x[tokens]
        if case["act"] == "gelu":
            a = adapters_of(rows @ value("w1", e).T, "up", rows, tokens, e) + w["b1"][e].to(f64)
            hid = a * 0.5 * torch.erfc(-a / math.sqrt(2))
            out = adapters_of(hid @ value("w2", e).T, "down", hid, tokens, e) + w["b2"][e].to(f64)
        else:
            g = adapters_of(rows @ value("w_gate", e).T, "gate", rows, tokens, e)
            hid = g / (1 + torch.exp(-g)) * adapters_of(rows @ value("w_up", e).T, "up", rows, tokens, e)
            out = adapters_of(hid @ value("w_down", e).T, "down", hid, tokens, e)
        y[tokens] += out if slot is None else out * gates[tokens, slot][:, None]
    return dict(y=y, experts=None, gates=gates, counts=None)
