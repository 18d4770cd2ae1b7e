"""Measured cases of the expert-routing and optimizer operators.

Where ``own`` is true, ``run`` makes the calls that a user of the library
makes; where it is false it computes the same results in their plain form,
with elementary torch operations in 32 bits (64 for sums of squares).

Definitions (t: token, k: choice, e: expert; tensors bf16 unless said otherwise):

* plan: of ids [tokens, top_k], expert e keeps the pairs (t, k) that name it, in
  the order of t * top_k + k, the first `capacity` of them where that is not 0.
  They get the slots offsets[e], offsets[e] + 1, ...; a segment's length is its
  count rounded up to 16, or the capacity; pairs that no expert keeps have slot
  -1, slots that no pair has have source -1 (else t * top_k + k).
* gather: y[slot] = x[t], 0 where a segment has no pair; with the cast,
  y = bf16(w[t, k] * x[t]) goes to FP8 codes, each segment's codes transposed in
  a block of its own.
* combine: y[t] = base[t] + sum over k of w[t, k] * x[slot(t, k)].
* its backward: dx[slot] = bf16(w[t, k] * dy[t]), dw[t, k] = dy[t] . x[slot].
* norm: the 2-norm of all gradients, and factor = min(1, most / norm).
* AdamW, every step rounded to 32 bits, t steps taken with this one:
      g = grad * factor        m = b1 m + (1 - b1) g      v = b2 v + ((1 - b2) g) g
      p = p (1 - lr wd) - (lr / (1 - b1^t) m) / (sqrt(v) / sqrt(1 - b2^t) + eps)
  In 8 bits m and v are E4M3 codes times a power of two per 256 values, the
  least that keeps them within 448 (2^-126 or more).  A value x between two codes
  goes to the lower one plus floor(place + u / 65536) where u is a 16-bit random
  number; a v above 0 stays above 0.  A bf16 parameter is rounded that way too.
  Random words: Philox4x32-7, key seed, counter (group, 2 i + s, t) for tensor i:
  s = 0, four values a group, low half for m and high half for v; s = 1, eight
  parameters a group, low half first.
"""
import math

import numpy as np
import torch

own = False

E4M3, E5M2 = 0, 1
FP8_MAX = (448.0, 57344.0)
FP8_TYPE = (torch.float8_e4m3fn, torch.float8_e5m2)
MASK32 = 0xFFFFFFFF
BLOCK = 256
BETA1, BETA2, EPS, LR, DECAY, MOST = 0.9, 0.999, 1e-8, 1e-3, 0.01, 1.0

# The six linears of the toy block (weights, then the three biases).
TOY_BLOCK = "25165824,12582912,4194304,8388608,16777216,16777216,12288,8192,2048"


def listed():
    return [
        # One decode step of 64 requests: latency alone.
        dict(name="plan_decode", op="plan", tokens=64, top_k=8, experts=64, capacity=0, none=0.0),
        # A long training batch, or the prompts of many requests.
        dict(name="plan_batch", op="plan", tokens=65536, top_k=4, experts=128, capacity=0,
             none=0.0),
        # Prompts in a padded batch to bf16 experts; padding tokens go to none.
        dict(name="gather_prompts", op="gather", tokens=4096, cols=2048, top_k=8, experts=64,
             capacity=0, none=0.1),
        # The toy block's tokens into the experts' first FP8 linears.
        dict(name="gather_cast_train", op="gather_cast", tokens=8192, cols=2048, top_k=2,
             experts=8, capacity=0, none=0.0, weights=False, fmt=E4M3),
        # The output gradient of the experts' last linears: odd sizes, fixed capacity.
        dict(name="gather_cast_gradient_odd", op="gather_cast", tokens=5003, cols=1168, top_k=3,
             experts=13, capacity=1456, none=0.05, weights=True, fmt=E5M2),
        # One decode step of 16 requests: latency alone.
        dict(name="combine_decode", op="combine", tokens=16, cols=2048, top_k=2, experts=8,
             capacity=0, none=0.0, weights=True, base=False),
        # A long training batch back onto the residual stream, the largest of its kind.
        dict(name="combine_train", op="combine", tokens=16384, cols=4096, top_k=4, experts=64,
             capacity=0, none=0.0, weights=True, base=True),
        # Its backward for bf16 experts at the toy block's sizes.
        dict(name="combine_backward_train", op="combine_backward", tokens=8192, cols=2048,
             top_k=2, experts=8, capacity=0, none=0.0, dx=True),
        # The weights' gradient alone (the rows' goes through the cast), odd sizes.
        dict(name="combine_backward_odd", op="combine_backward", tokens=1037, cols=1160, top_k=6,
             experts=37, capacity=0, none=0.1, dx=False),
        # The smallest step: one linear's adapters, bf16, states in 8 bits.
        dict(name="adamw_adapters_8bit", op="adamw", sizes="262144,262144", param="bf16",
             grad="bf16", bits=8, copy=False, clip=False),
        # A toy block's fp32 master weights with clipping: the largest.
        dict(name="adamw_block_fp32", op="adamw", sizes=TOY_BLOCK, param="fp32", grad="fp32",
             bits=32, copy=False, clip=True),
        # Eight experts' linears and odd biases in one step, states in 8 bits, bf16 copies.
        dict(name="adamw_experts_8bit", op="adamw", sizes=",".join(["4194304", "4194304", "1037"] * 8),
             param="fp32", grad="bf16", bits=8, copy=True, clip=True),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return min(hi, max(lo, int(v) // step * step))


def draw(rng):
    op = rng.choice(["plan", "gather", "gather_cast", "combine", "combine_backward", "adamw",
                     "adamw"])
    if op == "adamw":
        count, left, sizes = _spread(rng, 1, 20), 1 << 26, []
        for _ in range(count):
            n = min(left, _spread(rng, 1, 1 << 24))
            sizes.append(n - n % 4 + rng.randrange(4) if n > 8 else n)
            left = max(1, left - n)
        return dict(op=op, sizes=",".join(map(str, sizes)), param=rng.choice(["fp32", "bf16"]),
                    grad=rng.choice(["fp32", "bf16"]), bits=rng.choice([8, 32]), copy=False,
                    clip=rng.random() < 0.5)
    most = 65536 if op == "plan" else 16384
    case = dict(op=op, tokens=_spread(rng, 1, most), top_k=rng.randint(1, 8),
                experts=_spread(rng, 8, 128), capacity=0, none=rng.choice([0.0, 0.05, 0.3]))
    pairs = case["tokens"] * case["top_k"]
    if rng.random() < 0.4:
        # 1.25 times an expert's even share.
        case["capacity"] = (int(1.25 * pairs / case["experts"]) // 16 + 1) * 16
    if op == "plan":
        return case
    case["cols"] = _spread(rng, 64, 8192, 16 if op == "gather_cast" else 8)
    while case["tokens"] * case["top_k"] * case["cols"] > 1 << 27:
        case["cols"] = case["cols"] // 32 * 16
    if op == "gather_cast":
        return dict(case, weights=rng.random() < 0.5, fmt=rng.choice([E4M3, E5M2]))
    if op == "combine":
        return dict(case, weights=rng.random() < 0.7, base=rng.random() < 0.5)
    return dict(case, dx=rng.random() < 0.5) if op == "combine_backward" else case


def _rows(case):
    """Rows of a buffer in expert order."""
    pairs, experts, capacity = case["tokens"] * case["top_k"], case["experts"], case["capacity"]
    return experts * capacity if capacity else (pairs + 15 * min(experts, pairs)) // 16 * 16


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = torch.bfloat16

    def normal(shape, std=1.0, dtype=bf):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case=case)
    if case["op"] == "adamw":
        _prepare_adamw(s, g, normal)
        return s
    tokens, top_k, experts = case["tokens"], case["top_k"], case["experts"]
    # A router's choice: experts of uneven popularity, those of a token distinct.
    score = torch.randn(tokens, experts, generator=g, device="cuda")
    score += torch.randn(experts, generator=g, device="cuda")
    best = score.topk(top_k, dim=1)
    off = torch.rand(tokens, generator=g, device="cuda") < case["none"]
    s["ids"] = best.indices.to(torch.int32).masked_fill(off[:, None], -1)
    s["w"] = best.values.softmax(1)
    if case["op"] == "plan":
        _own_experts(s)
        return s
    rows, cols = _rows(case), case["cols"]
    if case["op"] in ("gather", "gather_cast"):
        gradient = case.get("fmt") == E5M2
        s["x"] = normal((tokens, cols), 1e-3 if gradient else 1.0)
        if case["op"] == "gather_cast":
            # The delayed scale that an amax of about five standard deviations leaves.
            s["scale"] = torch.full((1,), FP8_MAX[case["fmt"]] / (5e-3 if gradient else 5.0),
                                    device="cuda")
    elif case["op"] == "combine":
        s["x"] = normal((rows, cols))
        s["base"] = normal((tokens, cols)) if case["base"] else None
    else:
        s["x"], s["dy"] = normal((rows, cols)), normal((tokens, cols), 1e-3)
    _own_experts(s)
    return s


def _own_experts(s):
    """The plan (built once for all calls of a layer) and the outputs."""
    c = s["case"]
    if not own:
        if c["op"] != "plan":
            s["plan"] = _plain_plan(s)
        return
    import delayed_scaling_linear_amd as dsl
    tokens, top_k = c["tokens"], c["top_k"]
    s["plan"] = plan = dsl.ExpertPlan.empty(tokens, top_k, c["experts"], c["capacity"])
    if c["op"] == "plan":
        return
    dsl.fp8_expert_plan(s["ids"], plan)
    like = dict(device="cuda", dtype=torch.bfloat16)
    if c["op"] == "gather":
        s["y"] = torch.zeros(plan.rows, c["cols"], **like)
    elif c["op"] == "gather_cast":
        s["out"] = dsl.Float8Tensor.empty(plan.rows, c["cols"], c["fmt"])
        s["out"].data.zero_()
        s["out"].data_t.zero_()
        s["amax"] = torch.zeros(1, device="cuda")
    elif c["op"] == "combine":
        s["y"] = torch.empty(tokens, c["cols"], **like)
    else:
        s["dw"] = torch.empty(tokens, top_k, device="cuda")
        s["dx"] = torch.zeros(plan.rows, c["cols"], **like) if c["dx"] else None


def _sizes(case):
    return [int(n) for n in case["sizes"].split(",")]


def _scales(x):
    """The power of two of each 256 values (the flat state is a whole number of them)."""
    top = x.view(-1, BLOCK).abs().amax(1)
    f, e = torch.frexp(top)
    e = e - 9 + (f > 0.875).int()
    return torch.ldexp(torch.ones_like(top), e.clamp(min=-126))


def _prepare_adamw(s, g, normal):
    """Tensors lie one after another, each from a multiple of 256 values on."""
    c = s["case"]
    sizes = _sizes(c)
    at, starts = 0, []
    for n in sizes:
        starts.append(at)
        at += (n + BLOCK - 1) // BLOCK * BLOCK
    inside = torch.zeros(at, device="cuda")
    for a, n in zip(starts, sizes):
        inside[a:a + n] = 1.0
    types = {"fp32": torch.float32, "bf16": torch.bfloat16}
    f32 = torch.float32
    s["p"] = (normal((at,), 0.02, f32) * inside).to(types[c["param"]])
    s["g"] = (normal((at,), 1e-3, f32) * inside).to(types[c["grad"]])
    m = normal((at,), 3e-4, f32) * inside
    v = (normal((at,), 1e-3, f32) ** 2 + 1e-8) * inside
    if c["bits"] == 8:
        s["m_scale"], s["v_scale"] = _scales(m), _scales(v)
        for name, x in (("m", m), ("v", v)):
            x = (x.view(-1, BLOCK) / s[name + "_scale"][:, None]).view(-1)
            s[name] = x.to(FP8_TYPE[E4M3]).view(torch.uint8)
    else:
        s["m"], s["v"] = m, v
    s["copy"] = torch.zeros(at, device="cuda", dtype=torch.bfloat16) if c["copy"] else None
    s["steps"] = torch.randint(50, 1000, (1,), generator=g, device="cuda")
    s["seed"] = int(torch.randint(0, 2 ** 62, (1,), generator=g, device="cuda"))
    s["lr"] = torch.full((1,), LR, device="cuda")
    s["starts"], s["sizes"] = starts, sizes
    if own:
        import delayed_scaling_linear_amd as dsl

        def part(name, i, block=1):
            t = s[name]
            return None if t is None else t[starts[i] // block:(starts[i] + sizes[i] + block - 1)
                                            // block]

        tensors = []
        for i in range(len(sizes)):
            scales = {}
            if c["bits"] == 8:
                scales = dict(m_scale=part("m_scale", i, BLOCK), v_scale=part("v_scale", i, BLOCK))
            tensors.append(dsl.AdamWTensor(part("p", i), part("g", i), part("m", i), part("v", i),
                                           copy=part("copy", i), weight_decay=DECAY, **scales))
        s["opt"] = dsl.AdamW(tensors, lr=s["lr"], betas=(BETA1, BETA2), eps=EPS, seed=s["seed"])
        s["opt"].steps.copy_(s["steps"])
        if c["clip"]:
            s["norm"], s["factor"] = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
            s["flag"] = torch.zeros(1, dtype=torch.int32, device="cuda")
            s["ws"] = torch.empty(dsl.fp8_grad_norm_workspace_bytes(), dtype=torch.uint8,
                                  device="cuda")


# ---- the plain form ----------------------------------------------------------

def _plain_plan(s):
    c = s["case"]
    experts, capacity, rows = c["experts"], c["capacity"], _rows(c)
    ids = s["ids"].reshape(-1).long()
    mine = torch.arange(experts, device="cuda")[:, None] == ids
    rank = mine.cumsum(1, dtype=torch.int32).gather(0, ids.clamp(min=0)[None])[0] - 1
    counts = mine.sum(1)
    if capacity:
        counts = counts.clamp(max=capacity)
        lengths = torch.full_like(counts, capacity)
    else:
        lengths = (counts + 15) // 16 * 16
    offsets = torch.cat([torch.zeros_like(lengths[:1]), lengths.cumsum(0)])
    keep = (ids >= 0) & (rank < counts[ids.clamp(min=0)])
    slots = torch.where(keep, offsets[ids.clamp(min=0)] + rank, -1)
    sources = torch.full((rows,), -1, device="cuda", dtype=torch.int64)
    sources[slots[keep]] = torch.nonzero(keep)[:, 0]
    i32 = torch.int32
    return {"offsets": offsets.to(i32), "counts": counts.to(i32),
            "slots": slots.view(c["tokens"], -1).to(i32), "sources": sources.to(i32)}


def _plain_rows(s, x, weights):
    """bf16(w * x[t]) in expert order, 0 where there is no pair."""
    source = s["plan"]["sources"].long()
    y = x[source.clamp(min=0) // s["case"]["top_k"]]
    if weights is not None:
        y = (weights.reshape(-1)[source.clamp(min=0)][:, None] * y.float()).to(torch.bfloat16)
    return torch.where((source >= 0)[:, None], y, torch.zeros_like(y))


def _plain_gather_cast(s):
    c = s["case"]
    rows, cols, top = _rows(c), c["cols"], FP8_MAX[c["fmt"]]
    y = _plain_rows(s, s["x"], s["w"] if c["weights"] else None).float()
    codes = (y * s["scale"]).clamp(-top, top).to(FP8_TYPE[c["fmt"]]).view(torch.uint8)
    # Where element (r, c) of each segment's transpose lies.
    offsets = s["plan"]["offsets"].long()
    r = torch.arange(rows, device="cuda")
    segment = torch.searchsorted(offsets[1:], r, right=True).clamp(max=c["experts"] - 1)
    first, last = offsets[segment], offsets[segment + 1]
    place = (first * cols + r - first)[:, None] + torch.arange(cols, device="cuda") * \
        (last - first)[:, None]
    used = r < offsets[-1]
    codes_t = torch.zeros(rows * cols, device="cuda", dtype=torch.uint8)
    codes_t[place[used].reshape(-1)] = codes[used].reshape(-1)
    t = FP8_TYPE[c["fmt"]]
    return {"codes": codes.view(t), "codes_t": codes_t.view(cols, rows).view(t),
            "amax": y.abs().max(), "scale_inv": 1.0 / s["scale"]}


def _plain_combine(s):
    c = s["case"]
    slots = s["plan"]["slots"].long()
    x = s["x"][slots.clamp(min=0)].float()
    if c["weights"]:
        x = x * s["w"][:, :, None]
    y = torch.where((slots >= 0)[:, :, None], x, 0.0).sum(1)
    if c["base"]:
        y = s["base"].float() + y
    return {"y": y.to(torch.bfloat16)}


def _plain_combine_backward(s):
    slots = s["plan"]["slots"].long()
    dot = (s["x"][slots.clamp(min=0)].float() * s["dy"].float()[:, None, :]).sum(2)
    out = {"dw": torch.where(slots >= 0, dot, 0.0)}
    if s["case"]["dx"]:
        out["dx"] = _plain_rows(s, s["dy"], s["w"])
    return out


def _philox(e, word1, t, seed):
    """Philox4x32-7 words [..., 4] for groups e (int64)."""
    c = [e, torch.full_like(e, word1), (t & MASK32).expand_as(e), (t >> 32).expand_as(e)]
    k = [seed & MASK32, (seed >> 32) & MASK32]
    for _ in range(7):
        lo, hi = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((hi >> 32) & MASK32) ^ c[1] ^ k[0], hi & MASK32,
             ((lo >> 32) & MASK32) ^ c[3] ^ k[1], lo & MASK32]
        k = [(k[0] + 0x9E3779B9) & MASK32, (k[1] + 0xBB67AE85) & MASK32]
    return torch.stack(c, -1)


def _to_codes(x, u, floor):
    """E4M3 codes of x (within 448), rounded by the 16-bit numbers u.  Below 2^-6
    the codes are a step of 2^-9 apart, as they are from 2^-6 on."""
    ax = x.abs()
    low = ax < 2.0 ** -6
    bits = torch.where(low, ax + 2.0 ** -6, ax).view(torch.int32)
    code = ((bits + (u << 4)) >> 20) - torch.where(low, 968, 960)
    if floor:
        code = torch.where((code == 0) & (x > 0), 1, code)
    code = code | ((x.view(torch.int32) >> 24) & 0x80)
    return torch.where(torch.isfinite(x), code, 0x7F).to(torch.uint8)


def _plain_state(codes, scale, n):
    x = codes.view(FP8_TYPE[E4M3]).float().view(-1, BLOCK) * scale[:, None]
    return x.view(-1)[:n]


def _plain_store(x, u, codes, scale, n, floor):
    """x to codes and scales of one tensor, in place."""
    full = torch.zeros(codes.numel(), device="cuda")
    full[:n] = x
    scale.copy_(_scales(torch.where(torch.isfinite(full), full, 0.0)))
    full = (full.view(-1, BLOCK) * (1.0 / scale)[:, None]).view(-1)
    codes[:n] = _to_codes(full[:n], u, floor)


def _plain_adamw(s):
    c = s["case"]
    out, factor = {}, None
    if c["clip"]:
        norm = (s["g"].double() ** 2).sum().sqrt()
        factor = torch.where(norm > MOST, MOST / norm, 1.0).float()
        out = {"norm": norm.float().view(1), "factor": factor.view(1)}
    s["steps"] += 1
    t = s["steps"]
    lr = s["lr"].double()
    step = (lr / (1.0 - BETA1 ** t.double())).float()
    root = (1.0 / (1.0 - BETA2 ** t.double()).sqrt()).float()
    decay = (1.0 - lr * DECAY).float()
    for i, (a, n) in enumerate(zip(s["starts"], s["sizes"])):
        full = (n + BLOCK - 1) // BLOCK * BLOCK
        p, g = s["p"][a:a + n], s["g"][a:a + n].float()
        m, v = s["m"][a:a + full], s["v"][a:a + full]
        if factor is not None:
            g = g * factor
        if c["bits"] == 8:
            ms, vs = (s[k][a // BLOCK:(a + full) // BLOCK] for k in ("m_scale", "v_scale"))
            m32, v32 = _plain_state(m, ms, n), _plain_state(v, vs, n)
        else:
            m32, v32 = m[:n], v[:n]
        m32 = m32 * BETA1 + g * (1.0 - BETA1)
        v32 = v32 * BETA2 + (g * (1.0 - BETA2)) * g
        new = p.float() * decay - (m32 * step) / (v32.sqrt() * root + EPS)
        if c["bits"] == 8:
            e = torch.arange((n + 3) // 4, device="cuda")
            w = _philox(e, 2 * i, t, s["seed"]).view(-1)[:n]
            _plain_store(m32, (w & 0xFFFF).int(), m, ms, n, False)
            _plain_store(v32, (w >> 16).int(), v, vs, n, True)
        else:
            m[:n], v[:n] = m32, v32
        if c["param"] == "bf16":
            e = torch.arange((n + 7) // 8, device="cuda")
            w = _philox(e, 2 * i + 1, t, s["seed"])
            u = torch.stack((w & 0xFFFF, w >> 16), -1).view(-1)[:n].int()
            new = ((new.view(torch.int32) + u) & -65536).view(torch.float32)
        p.copy_(new)
        if c["copy"]:
            s["copy"][a:a + n] = new
    return _adamw_out(s, out)


def _adamw_out(s, out):
    c = s["case"]
    out = dict(out, p=s["p"], steps=s["steps"])
    if c["copy"]:
        out["copy"] = s["copy"]
    if c["bits"] == 8:
        t = FP8_TYPE[E4M3]
        return dict(out, m=s["m"].view(t), v=s["v"].view(t), m_scale=s["m_scale"],
                    v_scale=s["v_scale"])
    return dict(out, m=s["m"], v=s["v"])


# ---- the library's calls -----------------------------------------------------

def _own_run(s):
    import delayed_scaling_linear_amd as dsl
    c = s["case"]
    if c["op"] == "adamw":
        out = {}
        if c["clip"]:
            dsl.fp8_grad_norm(s["opt"].grads, s["norm"], s["ws"], max_norm=MOST,
                              factor=s["factor"], noop_flag=s["flag"])
            out = {"norm": s["norm"], "factor": s["factor"]}
            dsl.fp8_adamw_step(s["opt"], grad_scale=s["factor"], noop_flag=s["flag"])
        else:
            dsl.fp8_adamw_step(s["opt"])
        s["steps"] = s["opt"].steps
        return _adamw_out(s, out)
    plan = s["plan"]
    if c["op"] == "plan":
        dsl.fp8_expert_plan(s["ids"], plan)
        return {"offsets": plan.offsets, "counts": plan.counts, "slots": plan.slots,
                "sources": plan.sources}
    if c["op"] == "gather":
        dsl.fp8_expert_gather(plan, s["x"], s["y"])
        return {"y": s["y"]}
    if c["op"] == "gather_cast":
        out = s["out"]
        dsl.fp8_expert_gather_cast_transpose_amax(plan, s["x"], s["scale"], out, s["amax"],
                                                  weights=s["w"] if c["weights"] else None)
        t = FP8_TYPE[c["fmt"]]
        return {"codes": out.data.view(t), "codes_t": out.data_t.view(t), "amax": s["amax"][0],
                "scale_inv": out.scale_inv}
    if c["op"] == "combine":
        dsl.fp8_expert_combine(plan, s["x"], s["y"], weights=s["w"] if c["weights"] else None,
                               base=s["base"])
        return {"y": s["y"]}
    dsl.fp8_expert_combine_backward(plan, s["dy"], s["x"], s["dw"],
                                    weights=s["w"] if c["dx"] else None, dx=s["dx"])
    return {"dw": s["dw"], "dx": s["dx"]} if c["dx"] else {"dw": s["dw"]}


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "adamw":
        return _plain_adamw(state)
    if op == "plan":
        return _plain_plan(state)
    if op == "gather":
        return {"y": _plain_rows(state, state["x"], None)}
    if op == "gather_cast":
        return _plain_gather_cast(state)
    return _plain_combine(state) if op == "combine" else _plain_combine_backward(state)


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        p, g = (2 if case[k] == "bf16" else 4 for k in ("param", "grad"))
        state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        # Clipping needs every gradient before the first update: a second read.
        moved = n * (2 * p + g * (2 if case["clip"] else 1) + state + (2 if case["copy"] else 0))
        return {"bytes": int(moved), "flops": (15 + (2 if case["clip"] else 0)) * n}
    tokens, top_k, experts = case["tokens"], case["top_k"], case["experts"]
    live = tokens * (1.0 - case["none"])
    pairs = live * top_k
    # Segments end 7.5 rows short of a multiple of 16 on average.
    rows = experts * case["capacity"] if case["capacity"] else pairs + 7.5 * min(experts, pairs)
    index = 4 * (tokens * top_k + rows)
    if case["op"] == "plan":
        return {"bytes": int(index + 4 * tokens * top_k + 8 * experts), "flops": tokens * top_k}
    cols = case["cols"]
    if case["op"] in ("gather", "gather_cast"):
        moved = 2 * live * cols + 2 * rows * cols + 4 * rows
        moved += 4 * pairs if case.get("weights") else 0
        return {"bytes": int(moved), "flops": int(rows * cols)}
    if case["op"] == "combine":
        moved = 2 * pairs * cols + 2 * tokens * cols * (2 if case["base"] else 1)
        moved += 4 * tokens * top_k * (2 if case["weights"] else 1)
        return {"bytes": int(moved), "flops": int(2 * pairs * cols)}
    moved = 2 * live * cols + 2 * pairs * cols + 8 * tokens * top_k
    moved += 2 * rows * cols + 4 * pairs if case["dx"] else 0
    return {"bytes": int(moved), "flops": int(2 * pairs * cols)}


# ---- 64-bit results from the definitions -------------------------------------
# Apart from the plain forms above: the plan by one walk over the sorted pairs, each
# expert's rows by themselves, the random words by numpy's unsigned integers.

def _exact_plan(case, ids):
    experts, capacity, rows = case["experts"], case["capacity"], _rows(case)
    flat = ids.cpu().numpy().reshape(-1)
    order = np.argsort(flat, kind="stable")
    order = order[np.searchsorted(flat[order], 0):]
    ends = np.searchsorted(flat[order], np.arange(experts + 1))
    offsets, counts = [0], []
    slots, sources = np.full(flat.size, -1, np.int32), np.full(rows, -1, np.int32)
    for e in range(experts):
        pairs = order[ends[e]:ends[e + 1]]
        if capacity:
            pairs = pairs[:capacity]
        at = offsets[-1] + np.arange(len(pairs))
        slots[pairs], sources[at] = at, pairs
        counts.append(len(pairs))
        offsets.append(offsets[-1] + (capacity or -(-len(pairs) // 16) * 16))
    i32 = np.int32
    return {"offsets": np.array(offsets, i32), "counts": np.array(counts, i32),
            "slots": slots.reshape(ids.shape), "sources": sources}


def _on_grid(v, fmt):
    """v rounded to the format's grid, ties to even (mantissa bits 3 and 2,
    least exponents -6 and -14)."""
    exponent = torch.frexp(v)[1] - 1
    step = torch.ldexp(torch.ones_like(v), exponent.clamp(min=(-6, -14)[fmt]) - (3, 2)[fmt])
    return torch.round(v / step) * step


def _exact_experts(case, s):
    plan = _exact_plan(case, s["ids"])
    if case["op"] == "plan":
        return plan
    top_k = case["top_k"]
    slots = torch.from_numpy(plan["slots"]).cuda().long()
    sources = torch.from_numpy(plan["sources"]).cuda().long()
    live = torch.nonzero(sources >= 0)[:, 0]
    token, w = sources[live] // top_k, s["w"].reshape(-1)[sources[live]]
    if case["op"] == "combine":
        y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        if s["base"] is not None:
            y += s["base"]
        rows = s["x"][live].double()
        y.index_add_(0, token, rows * w.double()[:, None] if case["weights"] else rows)
        return {"y": y}
    out = torch.zeros(_rows(case), case["cols"], dtype=torch.float64, device="cuda")
    if case["op"] == "combine_backward":
        dy = s["dy"].double()
        dw = torch.zeros(slots.numel(), dtype=torch.float64, device="cuda")
        for part in live.split(1 << 14):
            of = sources[part]
            dw[of] = (dy[of // top_k] * s["x"][part].double()).sum(1)
        if not case["dx"]:
            return {"dw": dw.view(slots.shape)}
        out[live] = dy[token] * w.double()[:, None]
        return {"dw": dw.view(slots.shape), "dx": out}
    out[live] = s["x"][token].double()
    if case["op"] == "gather":
        return {"y": out}
    if case["weights"]:
        # The codes are those of the rows as a bf16 tensor would hold them.
        out[live] = (out[live] * w.double()[:, None]).float().to(torch.bfloat16).double()
    top, scale = FP8_MAX[case["fmt"]], s["scale"].double()
    codes = _on_grid((out * scale).float().double().clamp(-top, top), case["fmt"])
    codes_t = torch.zeros_like(codes).view(-1)
    offsets = plan["offsets"].tolist()
    for a, b in zip(offsets, offsets[1:]):
        codes_t[a * case["cols"]:b * case["cols"]] = codes[a:b].t().reshape(-1)
    return {"codes": codes, "codes_t": codes_t.view(case["cols"], -1), "amax": out.abs().max(),
            "scale_inv": 1.0 / scale}


def _exact_words(groups, word1, t, seed):
    u64, m = np.uint64, np.uint64(MASK32)
    x0 = np.arange(groups, dtype=u64)
    x1, x2, x3 = (np.full_like(x0, v) for v in (word1, t & MASK32, t >> 32))
    key0, key1 = seed & MASK32, seed >> 32
    for _ in range(7):
        p0, p1 = x0 * u64(0xD2511F53), x2 * u64(0xCD9E8D57)
        x0, x1 = (p1 >> u64(32)) ^ x1 ^ u64(key0), p1 & m
        x2, x3 = (p0 >> u64(32)) ^ x3 ^ u64(key1), p0 & m
        key0, key1 = (key0 + 0x9E3779B9) & MASK32, (key1 + 0xBB67AE85) & MASK32
    halves = np.stack([x0, x1, x2, x3], 1).astype("<u4").view("<u2").reshape(-1)
    return torch.from_numpy(halves.astype(np.int32)).cuda().double()


def _exact_codes(x, u, floor):
    """(codes' values, powers of two) of the 256-value blocks of x."""
    blocks = torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)
    u = torch.nn.functional.pad(u, (0, -u.numel() % BLOCK)).view(-1, BLOCK)
    most = blocks.abs().amax(1)
    exponent = torch.ceil(torch.log2(most.clamp(min=1e-300) / 448.0)).clamp(min=-126)
    scale = torch.exp2(exponent)
    y = blocks.abs() / scale[:, None]
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
    value = torch.floor(y / step + u / 65536.0) * step
    if floor:
        value = torch.where((value == 0) & (y > 0), 2.0 ** -9, value)
    return (value * torch.sign(blocks)).view(-1), scale


def _exact_adamw(case, s):
    f32 = lambda x: x.float().double()      # noqa: E731
    t = int(s["steps"]) + 1
    out, gs = {}, 1.0
    g_all = s["g"].double()
    if case["clip"]:
        norm = torch.linalg.vector_norm(g_all)
        gs = min(1.0, MOST / float(norm))
        out = {"norm": norm.view(1), "factor": torch.tensor([gs], dtype=torch.float64)}
    lr = float(s["lr"].double())
    step, root = lr / (1.0 - BETA1 ** t), 1.0 / math.sqrt(1.0 - BETA2 ** t)
    names = ["p", "m", "v"] + (["copy"] if case["copy"] else [])
    new = {k: torch.zeros(s["p"].shape, dtype=torch.float64, device="cuda") for k in names}
    if case["bits"] == 8:
        # Blocks that no tensor has do not exist: sizes are rounded up to them.
        new["m_scale"], new["v_scale"] = s["m_scale"].double(), s["v_scale"].double()
    for i, (a, n) in enumerate(zip(s["starts"], s["sizes"])):
        at, full = slice(a, a + n), (n + BLOCK - 1) // BLOCK * BLOCK
        g = g_all[at] * gs
        blocks = slice(a // BLOCK, (a + full) // BLOCK)

        def state(k):
            if case["bits"] == 32:
                return s[k][at].double()
            x = s[k][a:a + full].view(FP8_TYPE[E4M3]).double().view(-1, BLOCK)
            return (x * s[k + "_scale"][blocks].double()[:, None]).view(-1)[:n]

        m, v = state("m"), state("v")
        m1, v1 = BETA1 * m + (1.0 - BETA1) * g, BETA2 * v + (1.0 - BETA2) * g * g
        p = s["p"][at].double() * (1.0 - lr * DECAY) - step * m1 / (root * v1.sqrt() + EPS)
        if case["bits"] == 8:
            # The codes are those of the 32-bit values that each step leaves.
            b1, c1, b2, c2 = (float(np.float32(x)) for x in (BETA1, 1 - BETA1, BETA2, 1 - BETA2))
            g32 = f32(g_all[at] * float(np.float32(gs)))
            m1 = f32(f32(m * b1) + f32(g32 * c1))
            v1 = f32(f32(v * b2) + f32(f32(g32 * c2) * g32))
            u = _exact_words((n + 3) // 4, 2 * i, t, s["seed"])
            for k, x, half, floor in (("m", m1, 0, False), ("v", v1, 1, True)):
                codes, scale = _exact_codes(x, u[half::2][:n], floor)
                new[k][at], new[k + "_scale"][blocks] = codes[:n], scale
        else:
            new["m"][at], new["v"][at] = m1, v1
        if case["param"] == "bf16":
            u = _exact_words((n + 7) // 8, 2 * i + 1, t, s["seed"])[:n]
            unit = torch.exp2(torch.floor(torch.log2(p.abs().clamp(min=2.0 ** -126))) - 7)
            p = torch.floor(p.abs() / unit + u / 65536.0) * unit * torch.sign(p)
        new["p"][at] = p
        if case["copy"]:
            new["copy"][at] = p
    return dict(out, steps=s["steps"] + 1, **new)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_adamw(case, s) if case["op"] == "adamw" else _exact_experts(case, s)
