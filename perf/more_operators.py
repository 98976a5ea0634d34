"""What is measured of the operators around a mixture-of-experts layer served in 8-bit
integers and trained with a router that balances itself.

Five operators of the package, each beside its plain form in torch:

* scored routing: router logits -> sigmoid or softmax scores, the experts chosen by score
  plus a balance bias inside the best groups of experts, their weights (the scores without
  the bias, renormalised, scaled), counts, balance loss and each pair's row;
* its gradient with respect to the logits;
* a layer's product in 8-bit integers: activations quantised to one scale a token, times
  weights with one scale an output channel;
* the same for every expert of a layer in one launch, in the contiguous and the masked
  layout;
* an AdamW step over a list of tensors, with the gradients' clipping in it and states in 32
  bits or in 8.

`own` false: the plain forms. `own` true: the package's calls.
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 128                                     # elements of an 8-bit state that share a scale
BETA1, BETA2, EPS = 0.9, 0.95, 1e-8


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one token of a decode step over many experts in groups: the latency
        dict(name="route_t1_e256_g8_k8_f32", op="route", T=1, E=256, groups=8, open=4, best=2, k=8, t="f32",
             score="sigmoid", bias=True, renorm=True, masked=0.0, closed=0, max_m=0),
        # a training batch over the same experts, padding tokens among it
        dict(name="route_t32768_e256_g8_k8_f32", op="route", T=32768, E=256, groups=8, open=4, best=2, k=8,
             t="f32", score="sigmoid", bias=True, renorm=True, masked=0.1, closed=0, max_m=0),
        # the gradient of a batch of softmax scores over few experts, and of an odd
        # one of sigmoid scores with closed experts
        dict(name="route_bwd_t4096_e64_k6_bf16", op="route_bwd", T=4096, E=64, groups=1, open=1, best=1, k=6,
             t="bf16", score="softmax", bias=False, renorm=False, masked=0.0, closed=0),
        dict(name="route_bwd_t20011_e160_g8_k6_f32", op="route_bwd", T=20011, E=160, groups=8, open=3, best=1,
             k=6, t="f32", score="sigmoid", bias=True, renorm=True, masked=0.2, closed=5),
        # a decode step's product; an odd prompt of a small layer; the dense product
        # of the library's benchmark
        dict(name="int8_16x4096x7168_bf16", op="int8", M=16, N=4096, K=7168, t="bf16"),
        dict(name="int8_777x2064x1040_f32", op="int8", M=777, N=2064, K=1040, t="f32"),
        dict(name="int8_4096x8192x8192_bf16", op="int8", M=4096, N=8192, K=8192, t="bf16"),
        # the experts of the library's benchmark: a prompt's tokens dealt unevenly
        # over 8, and decode slabs of 32
        dict(name="experts_t4096_g8_4096x7168_bf16", op="experts", layout="contiguous", T=4096, G=8, max_m=0,
             N=4096, K=7168, t="bf16", skew=1.2),
        dict(name="experts_g32_slab256_7168x2048_bf16", op="experts", layout="masked", T=0, G=32, max_m=256,
             N=7168, K=2048, t="bf16", skew=0.0),
        # a router's and a few norms' tensors; a model of many odd sizes with fp32
        # states; the experts of the benchmark with 8-bit states
        dict(name="adamw_12_small_f32", op="adamw", n=12, total=40_000, spread=2.0, p="f32", g="f32", copy=False,
             bits=32, clip=False),
        dict(name="adamw_300_bf16_copy", op="adamw", n=300, total=50_000_000, spread=6.0, p="f32", g="bf16",
             copy=True, bits=32, clip=True),
        dict(name="adamw8_8_experts_bf16_copy", op="adamw", n=8, total=8 * 4096 * 7168, spread=0.0, p="f32",
             g="bf16", copy=True, bits=8, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "int8", "int8", "experts", "experts", "adamw", "adamw"])
    t = rng.choice(["f32", "bf16", "f16"])
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 1, 2, 4, 8, 16, _log(rng, 2, 32)])
        size = _log(rng, 2 if groups == 1 else 1, max(2, 1024 // groups))
        E = groups * size
        T = _log(rng, 1, max(1, min(65536, 32768 * 256 // E)))
        opened = rng.randint(1, groups)
        c = dict(op=op, T=T, E=E, groups=groups, open=opened, best=rng.randint(1, min(2, size)),
                 k=rng.randint(1, min(opened * size, 16)), t=t, score=rng.choice(["sigmoid", "sigmoid", "softmax"]),
                 bias=rng.random() < 0.7, renorm=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.3]),
                 closed=rng.choice([0, 0, rng.randint(0, E // 2)]))
        if op == "route":
            c["max_m"] = rng.choice([0, 0, rng.randint(1, 2 * T)])
        return c
    if op == "int8":
        M = _log(rng, 1, 8192)
        N = 16 * _log(rng, 1, 512)
        return dict(op=op, M=M, N=N, K=16 * _log(rng, 1, max(1, min(512, 4096 * 8192 * 8192 // (M * N * 16)))), t=t)
    if op == "experts":
        layout = rng.choice(["contiguous", "masked"])
        G = _log(rng, 1, 64)
        N = 16 * _log(rng, 1, 512)
        K = 16 * _log(rng, 1, max(1, min(512, 32 * 7168 * 2048 // (G * N * 16))))
        if layout == "contiguous":
            return dict(op=op, layout=layout, T=_log(rng, 1, 4096), G=G, max_m=0, N=N, K=K, t=t,
                        skew=rng.choice([0.0, 1.2]))
        return dict(op=op, layout=layout, T=0, G=G, max_m=_log(rng, 1, max(1, min(512, 32 * 256 // G))), N=N, K=K,
                    t=t, skew=0.0)
    p = rng.choice(["f32", "f32", "bf16", "f16"])
    return dict(op=op, n=_log(rng, 1, 500), total=_log(rng, 2_000, 100_000_000), spread=rng.uniform(0, 6), p=p,
                g=rng.choice(["f32", "bf16"]), copy=p == "f32" and rng.random() < 0.5, bits=rng.choice([8, 32]),
                clip=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _new(shape, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _activations(rows, cols, kind, g):
    """Tokens as a layer gives them: some channels larger than the rest, tokens
    that differ in size."""
    x = torch.randn(rows, cols, device=DEV, generator=g)
    x *= torch.exp(0.5 * torch.randn(1, cols, device=DEV, generator=g))
    x *= torch.exp(0.5 * torch.randn(rows, 1, device=DEV, generator=g))
    return x.to(TYPES[kind])


def _weights(rows, cols, g):
    """8-bit weights and their channels' scales, as a checkpoint holds them."""
    w = torch.randint(-127, 128, (rows, cols), dtype=torch.int8, device=DEV, generator=g)
    # (normal rather than uniform: the sum of two uniform halves, near enough)
    w = (w // 2 + torch.randint(-63, 64, (rows, cols), dtype=torch.int8, device=DEV, generator=g)).to(torch.int8)
    return w, (0.5 + torch.rand(rows, device=DEV, generator=g)) * 1e-3


def _expert_counts(c):
    """How many tokens each expert takes: the same for all seeds, so that the layout is."""
    G, T = c["G"], c["T"]
    rng = random.Random("%(T)d %(G)d %(skew)r" % c)
    picks = rng.choices(range(G), weights=[(i + 1.0) ** -c["skew"] for i in range(G)], k=T)
    return [picks.count(i) for i in range(G)]


def _prepare_route(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    x = torch.randn(T, E, device=DEV, generator=g) * 1.2 + 0.7 * torch.randn(1, E, device=DEV, generator=g) - 1.0
    if c["closed"]:                             # experts that take no token
        x[:, torch.randperm(E, device=DEV, generator=g)[: c["closed"]]] = -math.inf
    s = dict(case=c, logits=x.to(TYPES[c["t"]]), coef=0.01, scale=2.5, bias=None)
    if c["bias"]:                               # (moved by a fixed rate each step: few different values)
        s["bias"] = torch.round(50 * torch.randn(E, device=DEV, generator=g)) * 1e-3
    mask = torch.rand(T, device=DEV, generator=g) >= c["masked"]
    s["mask"] = mask if c["masked"] else None
    if c["op"] == "route":
        i32, f32 = torch.int32, torch.float32
        s["out"] = dict(expert_ids=_new((T, k), i32), weights=_new((T, k), f32), counts=_new((E,), i32),
                        routed=_new((1,), i32), prob_sum=_new((E,), f32), loss=_new((1,), f32),
                        group_offsets=_new((E + 1,), i32), slots=_new((T, k), i32))
        # (one int32 and one float for each expert and 32 tokens: a bound on what
        # the call asks for, whatever it uses)
        s["workspace"] = _new(((1 << 20) + 16 * E * (T // 32 + 64),), torch.uint8)
        return s
    s["ids"] = _select(s)
    s["counts"] = torch.bincount(s["ids"][s["ids"] >= 0].long(), minlength=E).to(torch.int32)
    s["routed"] = (s["ids"][:, 0] >= 0).sum().to(torch.int32).reshape(1)
    s["d_weights"] = torch.randn(T, k, device=DEV, generator=g)
    s["d_loss"] = torch.ones(1, device=DEV)
    s["d_logits"] = _new((T, E), s["logits"].dtype)
    return s


def _prepare_int8(c, g):
    M, N, K = c["M"], c["N"], c["K"]
    w, sw = _weights(N, K, g)
    return dict(case=c, x=_activations(M, K, c["t"], g), w=w, sw=sw, q=_new((M, K), torch.int8),
                sa=_new((M,), torch.float32), d=_new((M, N), torch.bfloat16))


def _prepare_experts(c, g, rng):
    G, N, K = c["G"], c["N"], c["K"]
    w, sw = _weights(G * N, K, g)
    s = dict(case=c, w=w.view(G, N, K), sw=sw.view(G, N))
    if c["layout"] == "contiguous":             # each expert's rows padded with zeros to 128
        counts = _expert_counts(c)
        ends = [0]
        for n in counts:
            ends.append(ends[-1] + (n + 127) // 128 * 128)
        rows = torch.cat([torch.arange(n, device=DEV) + e for n, e in zip(counts, ends)])
        x = torch.zeros(ends[-1], K, dtype=TYPES[c["t"]], device=DEV)
        x[rows] = _activations(c["T"], K, c["t"], g)
        s["ends"], s["group"] = ends, torch.tensor(ends, dtype=torch.int32, device=DEV)
        s["x"], s["d"] = x, _new((ends[-1], N), torch.bfloat16)
    else:
        counts = [rng.randint(0, c["max_m"]) for _ in range(G)]
        s["group"] = torch.tensor(counts, dtype=torch.int32, device=DEV)
        s["x"] = _activations(G * c["max_m"], K, c["t"], g).view(G, c["max_m"], K)
        s["d"] = torch.zeros(G, c["max_m"], N, dtype=torch.bfloat16, device=DEV)
    s["q"] = _new(tuple(s["x"].shape), torch.int8)
    s["sa"] = _new(tuple(s["x"].shape[:-1]), torch.float32)
    return s


def _prepare_adamw(c, g):
    # one model's sizes for all seeds, log-uniform over 2^spread, odd ones among them;
    # a tensor starts at a multiple of 128 of one buffer for each kind of tensor
    rng = random.Random("%(n)d %(total)d %(spread)r" % c)
    w = [2.0 ** rng.uniform(0, c["spread"]) if c["spread"] else 1.0 for _ in range(c["n"])]
    sizes = [max(1, int(c["total"] * x / sum(w))) for x in w]
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + (n + BLOCK - 1) // BLOCK * BLOCK)
    size = starts[-1]

    def views(flat):
        return [flat[a:a + n] for a, n in zip(starts, sizes)]
    block = torch.arange(size // BLOCK, device=DEV)
    first = torch.tensor(starts[:-1], device=DEV) // BLOCK
    number = torch.searchsorted(first, block, right=True) - 1       # the tensor of each block
    place = torch.arange(size, device=DEV)
    live = place - torch.tensor(starts[:-1], device=DEV)[number].repeat_interleave(BLOCK) \
        < torch.tensor(sizes, device=DEV)[number].repeat_interleave(BLOCK)
    del place
    # tensors differ in the size of their gradients
    level = (10.0 ** (-4 + 3 * torch.rand(c["n"], device=DEV, generator=g)))[number].repeat_interleave(BLOCK) * live
    s = dict(case=c, step=100, lr=1e-3, decay=0.1, max_norm=1.0, seed=12345, number=number, within=block - first[number])
    del live
    p = torch.randn(size, device=DEV, generator=g) * 0.02 * (level > 0)
    grad = torch.randn(size, device=DEV, generator=g) * level
    s["p"], s["g"] = p.to(TYPES[c["p"]]), grad.to(TYPES[c["g"]])
    m = 0.3 * level * torch.randn(size, device=DEV, generator=g)
    r = level * torch.exp(0.5 * torch.randn(size, device=DEV, generator=g))
    if c["bits"] == 32:
        s["m"], s["v"] = m, r * r
    else:                                       # (the state that some earlier step left)
        s["m"], s["m_scale"] = _state_codes(m, torch.zeros((), dtype=torch.int64, device=DEV), False)
        s["v"], s["v_scale"] = _state_codes(r, torch.zeros((), dtype=torch.int64, device=DEV), True)
    s["copy"] = s["p"].to(torch.bfloat16) if c["copy"] else None
    s["sumsq"] = s["g"].double().square().sum().reshape(1)
    s["norm"] = _new((1,), torch.float32)
    s["p_list"], s["g_list"] = views(s["p"]), views(s["g"])
    s["m_list"], s["v_list"] = views(s["m"]), views(s["v"])
    s["copy_list"] = views(s["copy"]) if c["copy"] else None
    if c["bits"] == 8:
        spans = [(a // BLOCK, b // BLOCK) for a, b in zip(starts, starts[1:])]
        s["m_scale_list"] = [s["m_scale"][a:b] for a, b in spans]
        s["v_scale_list"] = [s["v_scale"][a:b] for a, b in spans]
    s["list"] = None                            # (what a user's program makes of its tensors once)
    return s


def prepare(case, seed):
    g, rng = _gen(seed), random.Random(seed)
    if case["op"] in ("route", "route_bwd"):
        return _prepare_route(case, g)
    if case["op"] == "int8":
        return _prepare_int8(case, g)
    if case["op"] == "experts":
        return _prepare_experts(case, g, rng)
    return _prepare_adamw(case, g)


# ---------------------------------------------------------------------------
# the package's calls

def _route_own(s):
    import moe_grouped_gemm_quantizer_amd as fp8g
    c, o = s["case"], s["out"]
    fp8g.moe_route_scored(s["logits"], c["k"], o["expert_ids"], o["weights"], o["counts"], o["routed"],
                          o["prob_sum"], o["loss"], o["group_offsets"], o["slots"], s["workspace"],
                          score=c["score"], bias=s["bias"], groups=c["groups"], open_groups=c["open"],
                          group_best=c["best"], token_mask=s["mask"], renormalise=c["renorm"], scale=s["scale"],
                          loss_coef=s["coef"], align=128, max_m=c["max_m"])
    return o


def _route_bwd_own(s):
    import moe_grouped_gemm_quantizer_amd as fp8g
    c = s["case"]
    fp8g.moe_route_scored_backward(s["logits"], s["ids"], s["d_weights"], s["d_loss"], s["counts"], s["routed"],
                                   s["d_logits"], score=c["score"], renormalise=c["renorm"], scale=s["scale"],
                                   loss_coef=s["coef"])
    return s["d_logits"]


def _int8_own(s):
    import moe_grouped_gemm_quantizer_amd as fp8g
    fp8g.int8_quantize(s["x"], s["q"], s["sa"])
    fp8g.gemm_int8(s["q"], s["sa"], s["w"], s["sw"], s["d"])
    return dict(d=s["d"], scales=s["sa"])


def _experts_own(s):
    import moe_grouped_gemm_quantizer_amd as fp8g
    x, q, sa = s["x"], s["q"], s["sa"]
    fp8g.int8_quantize(x.view(-1, x.shape[-1]), q.view(-1, x.shape[-1]), sa.view(-1))
    if s["case"]["layout"] == "contiguous":
        fp8g.grouped_gemm_int8_contiguous(q, sa, s["w"], s["sw"], s["d"], s["group"])
    else:
        fp8g.grouped_gemm_int8_masked(q, sa, s["w"], s["sw"], s["d"], s["group"])
    return dict(d=s["d"], scales=sa)


def _adamw_own(s):
    import moe_grouped_gemm_quantizer_amd as fp8g
    c = s["case"]
    if s["list"] is None:
        if c["bits"] == 32:
            s["list"] = fp8g.adamw_tensors(s["p_list"], s["g_list"], s["m_list"], s["v_list"], copies=s["copy_list"])
        else:
            s["list"] = fp8g.adamw_tensors(s["p_list"], s["g_list"], s["m_list"], s["v_list"],
                                           m_scales=s["m_scale_list"], v_scales=s["v_scale_list"],
                                           copies=s["copy_list"])
    s["step"] += 1
    clip = dict(sumsq=s["sumsq"], max_norm=s["max_norm"], norm=s["norm"]) if c["clip"] else {}
    fp8g.adamw_step(s["list"], s["step"], s["lr"], beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=s["decay"],
                    seed=s["seed"], **clip)
    return _adamw_outputs(s)


# ---------------------------------------------------------------------------
# the plain forms

def _scores(logits, score, dtype):
    x = logits.to(dtype)
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    z = p.sum(1, keepdim=True)
    return p / torch.where(z > 0, z, torch.ones_like(z))


def _select(s):
    """The chosen experts of each token: by score plus bias (without a bias by the
    logits, whose order is the same), ties to the lower expert, inside the groups
    whose best experts' sum is largest, ties to the lower group. -1: none. In 64
    bits, since neighbours may differ by less than 32 bits tell."""
    c, x = s["case"], s["logits"]
    T, E, k, groups = c["T"], c["E"], c["k"], c["groups"]
    may = x.float() > -math.inf
    if s["mask"] is not None:
        may = may & s["mask"][:, None]
    by = x.double()
    if s["bias"] is not None or c["open"] < groups:
        v = _scores(x, c["score"], torch.float64)
        if s["bias"] is not None:
            v = v + s["bias"].double()
            by = v
        if c["open"] < groups:
            inside = torch.where(may, v, -math.inf).view(T, groups, -1).topk(c["best"], 2).values
            value = torch.where(inside > -math.inf, inside, 0.0).sum(2)
            value = torch.where(inside[:, :, 0] > -math.inf, value, -math.inf)
            best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :c["open"]]
            opened = torch.zeros(T, groups, dtype=torch.bool, device=DEV).scatter_(1, best, True)
            may = may & opened.repeat_interleave(E // groups, 1)
    value, ids = torch.sort(torch.where(may, by, -math.inf), dim=1, descending=True, stable=True)
    return torch.where(value[:, :k] > -math.inf, ids[:, :k], -1).to(torch.int32)


def _route_plain(s):
    c, x = s["case"], s["logits"]
    T, E, k = c["T"], c["E"], c["k"]
    ids = _select(s)
    live = ids >= 0
    at = ids.clamp(min=0).long()
    p = _scores(x, c["score"], torch.float32)
    w = torch.where(live, p.gather(1, at), torch.zeros((), device=DEV))
    if c["renorm"]:
        z = w.sum(1, keepdim=True)
        w = w / torch.where(z > 0, z, torch.ones_like(z))
    w = w * s["scale"]
    if c["score"] == "sigmoid":                 # the loss goes by each expert's share of the row
        z = p.sum(1, keepdim=True)
        p = p / torch.where(z > 0, z, torch.ones_like(z))
    takes = torch.zeros(T, E, dtype=torch.int32, device=DEV).scatter_add_(1, at, live.int())
    counts = takes.sum(0, dtype=torch.int32)
    on = live[:, 0]
    routed = on.sum(dtype=torch.int32).reshape(1)
    prob_sum = torch.where(on[:, None], p, torch.zeros((), device=DEV)).sum(0)
    n = routed.float().clamp(min=1.0)
    loss = s["coef"] * (E * counts.float() / (k * n) * (prob_sum / n)).sum().reshape(1)
    if c["max_m"]:
        offsets = torch.arange(E + 1, dtype=torch.int32, device=DEV) * c["max_m"]
    else:
        offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        offsets[1:] = ((counts + 127) // 128 * 128).cumsum(0)
    rank = (takes.cumsum(0, dtype=torch.int32) - takes).gather(1, at)
    fits = live & (rank < c["max_m"]) if c["max_m"] else live
    slots = torch.where(fits, offsets[at] + rank, -1).to(torch.int32)
    return dict(expert_ids=ids, weights=w, counts=counts, routed=routed, prob_sum=prob_sum, loss=loss,
                group_offsets=offsets, slots=slots)


def _route_bwd_plain(s):
    c, ids = s["case"], s["ids"]
    E, k = c["E"], c["k"]
    live = ids >= 0
    at = ids.clamp(min=0).long()
    p = _scores(s["logits"], c["score"], torch.float32)
    zero = torch.zeros((), device=DEV)
    dw = torch.where(live, s["d_weights"] * s["scale"], zero)
    if c["renorm"]:                             # w = scale p / z over the chosen
        pc = torch.where(live, p.gather(1, at), zero)
        z = pc.sum(1, keepdim=True)
        z = torch.where(z > 0, z, torch.ones_like(z))
        dw = torch.where(live, (dw - (dw * (pc / z)).sum(1, keepdim=True)) / z, zero)
    n = s["routed"].float().clamp(min=1)
    f = (s["d_loss"] * s["coef"] * E * s["counts"].float() / (k * n * n)).expand(c["T"], E)
    if c["score"] == "sigmoid":
        z = p.sum(1, keepdim=True)
        z = torch.where(z > 0, z, torch.ones_like(z))
        dp = (f - (f * p / z).sum(1, keepdim=True)) / z
        dx = p * (1 - p) * dp.scatter_add(1, at, dw)
    else:
        dp = f.scatter_add(1, at, dw)
        dx = p * (dp - (p * dp).sum(1, keepdim=True))
    return torch.where(live[:, :1], dx, zero).to(s["logits"].dtype)


def _quantised(x):
    """Rows as codes -127 .. 127 (held as fp32) and one scale each; a row below 2^-120
    counts as zero."""
    x = x.float()
    top = x.abs().amax(-1, keepdim=True)
    some = top >= 2.0 ** -120
    inv = torch.where(some, 127.0 / torch.where(some, top, torch.ones_like(top)), torch.zeros_like(top))
    return torch.round(x * inv), torch.where(some, top / 127.0, torch.zeros_like(top))[..., 0]


def _int8_plain(s):
    q, sa = _quantised(s["x"])
    return dict(d=((q @ s["w"].float().t()) * sa[:, None] * s["sw"]).to(torch.bfloat16), scales=sa)


def _experts_plain(s):
    q, sa = _quantised(s["x"])
    if s["case"]["layout"] == "masked":
        d = (torch.bmm(q, s["w"].float().transpose(1, 2).contiguous()) * sa[..., None] * s["sw"][:, None])
        valid = torch.arange(s["case"]["max_m"], device=DEV) < s["group"][:, None]
        return dict(d=torch.where(valid[..., None], d, torch.zeros((), device=DEV)).to(torch.bfloat16), scales=sa)
    # one product for each expert: their rows differ
    parts = [(q[i:j] @ w.float().t()) * sa[i:j, None] * sw
             for i, j, w, sw in zip(s["ends"], s["ends"][1:], s["w"], s["sw"])]
    return dict(d=torch.cat(parts).to(torch.bfloat16), scales=sa)


def _mix(h):
    """A 32-bit hash: xor-shifts and odd multipliers, modulo 2^32 (held in 64 bits)."""
    h = ((h ^ (h >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    h = ((h ^ (h >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _random_bits(s):
    """32 bits for each element: of the seed, the step, the tensor's number, the block
    and the place in it."""
    key = _mix(torch.tensor((s["seed"] + _mix(s["step"])) & 0xFFFFFFFF, device=DEV))
    base = _mix((_mix((key + s["number"]) & 0xFFFFFFFF) + s["within"]) & 0xFFFFFFFF)
    j = torch.arange(BLOCK, device=DEV) * 0x9E3779B9
    return _mix((base[:, None] + j) & 0xFFFFFFFF).view(-1)


def _state_codes(x, bits, root):
    """x in blocks of 128 as e4m3 codes and the byte of their power-of-two scale, rounded
    up with the probability of the part that is cut off (`bits`: 16 random ones for each
    element); `root`: not negative, and no code 0 but for 0."""
    y = x.view(-1, BLOCK)
    m, e = torch.frexp(y.abs().amax(1, keepdim=True))
    # the smallest power of two that brings the largest value to 448 = 0.875 2^9 or below
    e = torch.where(m > 0, (e - 9 + (m > 0.875).int()).clamp(-126, 126), torch.zeros_like(e))
    z = (y.abs() * ((127 - e) << 23).view(torch.float32)).view(-1)
    small = z < 2.0 ** -6
    z = torch.where(small, z + 2.0 ** -6, z).view(torch.int32)
    code = ((z + (bits << 4).to(torch.int32)) >> 20) - torch.where(small, 968, 960).to(torch.int32)
    if root:
        code = torch.where(x > 0, code.clamp(min=1), code)
    else:
        code = code + 128 * torch.signbit(x).int()
    return code.to(torch.uint8), (e + 127).to(torch.uint8).view(-1)


def _state_values(codes, scale):
    return (codes.view(torch.float8_e4m3fn).float().view(-1, BLOCK) *
            (scale.int() << 23).view(torch.float32)[:, None]).view(-1)


def _adamw_outputs(s):
    out = dict(p=s["p"], m=s["m"], v=s["v"])
    if s["case"]["bits"] == 8:                  # the codes as the values they stand for, in units of their scale
        out.update(m=s["m"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn), m_scale=s["m_scale"],
                   v_scale=s["v_scale"])
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    if s["case"]["clip"]:
        out["norm"] = s["norm"]
    return out


def _adamw_plain(s):
    c = s["case"]
    s["step"] += 1
    p, g = s["p"].float(), s["g"].float()
    if c["clip"]:
        norm = s["sumsq"].sqrt()
        g = g * (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
        s["norm"].copy_(norm)
    eight = c["bits"] == 8
    m = _state_values(s["m"], s["m_scale"]) if eight else s["m"]
    v = _state_values(s["v"], s["v_scale"]).square() if eight else s["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g.square() * (1 - BETA2)
    r = v.double().sqrt().float()               # (rounded once, whatever the device's square root does)
    c1, c2 = 1 - BETA1 ** s["step"], math.sqrt(1 - BETA2 ** s["step"])
    p = p * (1 - s["lr"] * s["decay"]) - (s["lr"] / c1) * m / (r / c2 + EPS)
    s["p"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    if eight:
        bits = _random_bits(s)
        for name, x, cut in (("m", m, bits & 0xFFFF), ("v", r, bits >> 16)):
            code, scale = _state_codes(x, cut, name == "v")
            s[name].copy_(code)
            s[name + "_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_outputs(s)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _route_own, "route_bwd": _route_bwd_own, "int8": _int8_own, "experts": _experts_own,
                "adamw": _adamw_own}[op](state)
    return {"route": _route_plain, "route_bwd": _route_bwd_plain, "int8": _int8_plain, "experts": _experts_plain,
            "adamw": _adamw_plain}[op](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "route":
        return dict(bytes=c["T"] * (c["E"] * SIZE[c["t"]] + 12 * c["k"] + 1) + 16 * c["E"], flops=c["T"] * c["E"] * 6)
    if c["op"] == "route_bwd":
        return dict(bytes=c["T"] * (2 * c["E"] * SIZE[c["t"]] + 8 * c["k"]) + 4 * c["E"], flops=c["T"] * c["E"] * 10)
    if c["op"] == "int8":
        return dict(bytes=c["M"] * (c["K"] * SIZE[c["t"]] + 2 * c["N"] + 4) + c["N"] * (c["K"] + 4),
                    flops=2 * c["M"] * c["N"] * c["K"])
    if c["op"] == "experts":
        # (of a slab half the rows on average; their quantising takes all of them)
        rows = c["T"] if c["layout"] == "contiguous" else c["G"] * c["max_m"]
        used = c["T"] if c["layout"] == "contiguous" else rows // 2
        return dict(bytes=rows * (c["K"] * SIZE[c["t"]] + 4) + 2 * used * c["N"] + c["G"] * c["N"] * (c["K"] + 4),
                    flops=2 * used * c["N"] * c["K"])
    each = 2 * SIZE[c["p"]] + SIZE[c["g"]] + 2 * c["copy"] + (16 if c["bits"] == 32 else 4 + 4 / BLOCK)
    return dict(bytes=int(each * c["total"]), flops=(14 if c["bits"] == 32 else 40) * c["total"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_largest(v, n):
    """The n largest of each row, one after the other: their numbers, -1 for -inf."""
    v, ids = v.clone(), []
    number = torch.arange(v.shape[1], device=v.device)
    for _ in range(n):
        top = v.amax(1, keepdim=True)
        i = torch.where(v == top, number, v.shape[1]).amin(1, keepdim=True)
        ids.append(torch.where(top > -math.inf, i, -1))
        v.scatter_(1, i, -math.inf)
    return torch.cat(ids, 1)


def _exact_route(c, s):
    T, E, k = c["T"], c["E"], c["k"]
    x = s["logits"].double()
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    score = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, 1))
    value = score if s["bias"] is None else score + s["bias"]
    by = x if s["bias"] is None else value
    shut = x == -math.inf
    if s["mask"] is not None:
        shut |= ~s["mask"][:, None]
    if c["open"] < c["groups"]:
        size = E // c["groups"]
        inside = torch.where(shut, -math.inf, value).view(T, c["groups"], size).sort(2, descending=True).values
        total = inside[..., :c["best"]].nan_to_num(neginf=0.0).sum(2)
        total = torch.where(inside[..., 0] == -math.inf, -math.inf, total)
        chosen = _exact_largest(total, c["open"])
        group = torch.arange(E, device=DEV) // size
        shut |= ~(chosen[:, :, None] == group).any(1)
    ids = _exact_largest(torch.where(shut, -math.inf, by), k)
    use, at = ids >= 0, ids.clamp(min=0)
    w = torch.where(use, score.gather(1, at), zero)
    if c["renorm"]:
        w = torch.where(use, w / w.sum(1, keepdim=True), zero)
    on = use[:, 0]
    psum = (score[on] / score[on].sum(1, keepdim=True)).sum(0)
    n = max(int(on.sum()), 1)
    cnt = torch.bincount(at[use], minlength=E).double()
    loss = s["coef"] * E / k * (cnt * psum).sum().reshape(1) / n / n
    return dict(expert_ids=None, weights=w * s["scale"], counts=None, routed=None, prob_sum=psum, loss=loss,
                group_offsets=None, slots=None)


def _exact_route_bwd(c, s):
    # by reverse differentiation of the forward definition
    x, ids = s["logits"].double(), s["ids"].long()
    on = ids[:, 0] >= 0
    if not bool(on.any()):
        return torch.zeros_like(x)
    xr, ir = x[on].requires_grad_(True), ids[on]
    score = torch.sigmoid(xr) if c["score"] == "sigmoid" else torch.softmax(xr, 1)
    w = torch.where(ir >= 0, score.gather(1, ir.clamp(min=0)), torch.zeros((), dtype=x.dtype, device=DEV))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    share = score / score.sum(1, keepdim=True)
    n = float(s["routed"])
    f = c["E"] * s["counts"].double() / (c["k"] * n)
    y = (s["scale"] * w * s["d_weights"][on].double()).sum() \
        + float(s["d_loss"]) * s["coef"] * (f * share.sum(0) / n).sum()
    grad = torch.autograd.grad(y, xr)[0]
    return torch.zeros_like(x).index_copy(0, on.nonzero()[:, 0], grad)


def _exact_codes(x):
    x = x.double()
    top = x.abs().max(-1, keepdim=True).values
    zero = top < 2.0 ** -120
    scale = torch.where(zero, torch.ones_like(top), top / 127)
    return torch.where(zero, torch.zeros_like(x), torch.round(x / scale)), (scale * ~zero)[..., 0]


def _exact_values(codes, scale):
    b = codes.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    size = torch.where(e == 0, m * 2.0 ** -9, torch.ldexp(m + 8, e - 10))
    size = torch.where(b > 127, -size, size).view(-1, BLOCK)
    return torch.ldexp(size, scale.long()[:, None] - 127).view(-1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        return _exact_route(c, s)
    if c["op"] == "route_bwd":
        return _exact_route_bwd(c, s)
    if c["op"] == "int8":
        q, sa = _exact_codes(s["x"])
        return dict(d=torch.mm(q, s["w"].double().t()) * sa[:, None] * s["sw"].double(), scales=sa)
    if c["op"] == "experts":
        q, sa = _exact_codes(s["x"])
        d = torch.zeros(s["d"].shape, dtype=torch.float64, device=DEV)
        for g in range(c["G"]):
            w, sw = s["w"][g].double().t().contiguous(), s["sw"][g].double()
            if c["layout"] == "contiguous":
                i, j = s["ends"][g], s["ends"][g + 1]
                if j > i:
                    d[i:j] = torch.mm(q[i:j], w) * sa[i:j, None] * sw
            else:
                n = int(s["group"][g])
                if n:
                    d[g, :n] = torch.mm(q[g, :n], w) * sa[g, :n, None] * sw
        return dict(d=d, scales=sa)
    t = s["step"] + 1
    p, g = s["p"].double(), s["g"].double()
    out = {}
    if c["clip"]:
        norm = torch.sqrt(s["sumsq"])
        g = g * min(1.0, s["max_norm"] / (float(norm) + 1e-6))
        out["norm"] = norm
    if c["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        m, v = _exact_values(s["m"], s["m_scale"]), _exact_values(s["v"], s["v_scale"]) ** 2
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    p = p - s["lr"] * s["decay"] * p - s["lr"] * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    out.update(p=p, m=m, v=v) if c["bits"] == 32 else out.update(p=p, m=None, v=None, m_scale=None, v_scale=None)
    if c["copy"]:
        out["copy"] = p
    return out
