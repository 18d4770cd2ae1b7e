"""Measured cases of the dropout and low-rank adapter operators.

Where ``own`` is true, ``run`` makes the calls that a user of the library
makes; where it is false it computes the same results in their plain form,
with elementary torch operations in 32 bits.

Definitions (r, c: row and column; every input bf16 unless said otherwise):

* dropout: with rng = (seed, offset), T = round(65536 p) and the group index
  e = (r * cols + c) // 8, the word w = Philox4x32-7(counter (e, offset), key
  seed)[(c % 8) // 2] gives element (r, c) its low (even c) or high (odd c)
  16 bits u; the element is kept where u >= T and then multiplied by
  f = fp32(65536 / (65536 - T)), else it is +0.  y = residual + dropout(x).
* adapters: row r belongs to adapter a = row_adapter[r] (-1: none), and
      h[r]  = alpha[a] * dropout(x[r]) A[a]^T          (fp32)
      y[r]  = base[r] + h[r] B[a]^T
  a row without an adapter has h = 0 and y = base.  With g = alpha[a] * dy B[a]:
      dx[r] = base[r] + f * keep * (g[r] A[a])
      dA[a] = sum over its rows of g[r]^T dropout(x[r])
      dB[a] = sum over its rows of dy[r]^T h[r]
"""
import math

import numpy as np
import torch

own = False

E4M3, E5M2 = 0, 1
FP8_MAX = (448.0, 57344.0)
FP8_TYPE = (torch.float8_e4m3fn, torch.float8_e5m2)
MASK32 = 0xFFFFFFFF


def listed():
    return [
        # Smallest fused dropout: one short sequence of the tiny linear, where a launch counts.
        dict(name="dropout_cast_tiny", op="dropout_cast", rows=128, cols=256, p=0.1, residual=True,
             fmt=E4M3, dbias=False),
        # The residual stream of the toy block (8 x 1024 tokens, hidden 2048) into the next linear.
        dict(name="dropout_cast_residual", op="dropout_cast", rows=8192, cols=2048, p=0.1,
             residual=True, fmt=E4M3, dbias=False),
        # Its backward at the widest output gradient: E5M2 codes, transpose and bias gradient.
        dict(name="dropout_cast_gradient", op="dropout_cast", rows=8192, cols=8192, p=0.1,
             residual=False, fmt=E5M2, dbias=True),
        # A packed batch of ragged length, fp32 activations, no cast.
        dict(name="dropout_fp32_ragged", op="dropout", rows=1037, cols=1160, p=0.25, residual=True,
             dtype="fp32"),
        # Dropout of bf16 activations that no linear reads next.
        dict(name="dropout_bf16", op="dropout", rows=8192, cols=2048, p=0.05, residual=False,
             dtype="bf16"),
        # One token of one request: latency alone.
        dict(name="adapter_decode_1", op="adapter_fwd", rows=1, k=2048, n=2048, rank=16,
             adapters=8, order="scatter", none=0.0, p=0.0, keep_h=False),
        # One decode step of 64 requests over 32 adapters, some on the base model alone.
        dict(name="adapter_decode_64", op="adapter_fwd", rows=64, k=2048, n=8192, rank=16,
             adapters=32, order="scatter", none=0.2, p=0.0, keep_h=False),
        # Prompts of nine requests in one batch, mixed lengths, the qkv projection.
        dict(name="adapter_prompts", op="adapter_fwd", rows=8192, k=2048, n=6144, rank=64,
             adapters=9, order="runs", none=0.1, p=0.0, keep_h=False),
        # Training forward of one adapter with dropout on its input; h is kept for the backward.
        dict(name="adapter_train_forward", op="adapter_fwd", rows=8192, k=2048, n=8192, rank=16,
             adapters=1, order="runs", none=0.0, p=0.1, keep_h=True),
        # Its backward.
        dict(name="adapter_train_backward", op="adapter_bwd", rows=8192, k=2048, n=8192, rank=16,
             adapters=1, order="runs", none=0.0, p=0.1, grads="fp32"),
        # Odd sizes: three adapters over interleaved rows, a rank between powers of two.
        dict(name="adapter_backward_odd", op="adapter_bwd", rows=1003, k=1048, n=776, rank=24,
             adapters=3, order="scatter", none=0.1, p=0.05, grads="bf16"),
        # The largest: several adapters trained together over long batches.
        dict(name="adapter_backward_large", op="adapter_bwd", rows=16384, k=8192, n=2048,
             rank=128, adapters=4, order="runs", none=0.0, p=0.0, grads="fp32"),
    ]


def _spread(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return min(hi, max(lo, int(v) // step * step))


def draw(rng):
    op = rng.choice(["dropout", "dropout_cast", "adapter_fwd", "adapter_fwd", "adapter_bwd"])
    p = rng.choice([0.0, 0.05, 0.1, 0.3, 0.5])
    if op == "dropout":
        return dict(op=op, rows=_spread(rng, 1, 8192, 1), cols=_spread(rng, 64, 8192, 8), p=p,
                    residual=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp32"]))
    if op == "dropout_cast":
        return dict(op=op, rows=_spread(rng, 16, 8192, 16), cols=_spread(rng, 64, 8192, 16), p=p,
                    residual=rng.random() < 0.5, fmt=rng.choice([E4M3, E5M2]),
                    dbias=rng.random() < 0.5)
    case = dict(op=op, rows=_spread(rng, 1, 16384, 1), k=_spread(rng, 64, 8192, 8),
                n=_spread(rng, 64, 8192, 8), rank=_spread(rng, 8, 128, 8),
                order=rng.choice(["scatter", "runs"]), none=rng.choice([0.0, 0.1, 0.5]))
    # Few adapters over many rows, many over few; at most 1024 ranks side by side.
    case["adapters"] = _spread(rng, 1, max(1, min(64, 1024 // case["rank"])), 1)
    while case["rows"] * (case["k"] + case["n"]) > 16384 * 8192:
        case["rows"] = case["rows"] * 2 // 3
    if op == "adapter_fwd":
        train = rng.random() < 0.4
        return dict(case, p=p if train else 0.0, keep_h=train)
    return dict(case, p=p, grads=rng.choice(["fp32", "bf16"]))


def _adapters_of_rows(case, g):
    """row_adapter [rows] int32: -1 for a share `none` of the rows or requests."""
    rows, count = case["rows"], case["adapters"]

    def ids(n):
        a = torch.randint(0, count, (n,), generator=g, device="cuda", dtype=torch.int32)
        off = torch.rand(n, generator=g, device="cuda") < case["none"]
        return torch.where(off, torch.full_like(a, -1), a)

    if case["order"] == "scatter":
        return ids(rows)
    # Requests of uneven lengths, one run of rows each; about one per adapter.
    cuts = torch.rand(count, generator=g, device="cuda")
    at = (cuts.sort().values * rows).to(torch.int64)
    request = torch.searchsorted(at, torch.arange(rows, device="cuda"), right=True)
    one_each = torch.arange(count + 1, device="cuda", dtype=torch.int32) % count
    off = torch.rand(count + 1, generator=g, device="cuda") < case["none"]
    return torch.where(off, torch.full_like(one_each, -1), one_each)[request]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = torch.bfloat16

    def normal(shape, std=1.0, dtype=bf):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case=case)
    s["rng"] = torch.randint(0, 2 ** 62, (2,), generator=g, device="cuda", dtype=torch.int64)
    if case["op"] in ("dropout", "dropout_cast"):
        shape = (case["rows"], case["cols"])
        cast = case["op"] == "dropout_cast"
        dtype = torch.float32 if case.get("dtype") == "fp32" else bf
        gradient = cast and case["fmt"] == E5M2
        s["x"] = normal(shape, 1e-3 if gradient else 1.0, dtype)
        s["residual"] = normal(shape, 1.0, dtype) if case["residual"] else None
        if cast:
            # The delayed scale that an amax of about five standard deviations leaves.
            top = 5e-3 if gradient and not case["residual"] else 6.0
            s["scale"] = torch.full((1,), FP8_MAX[case["fmt"]] / top, device="cuda")
        _own_dropout(s)
        return s
    rows, k, n, rank, count = (case[v] for v in ("rows", "k", "n", "rank", "adapters"))
    s["ids"] = _adapters_of_rows(case, g)
    s["a"] = normal((count, rank, k), k ** -0.5)
    s["b"] = normal((count, n, rank), 0.02)
    s["alpha"] = torch.rand(count, generator=g, device="cuda") + 1.0
    s["x"] = normal((rows, k))
    if case["op"] == "adapter_fwd":
        s["base"] = normal((rows, n))
    else:
        s["dy"] = normal((rows, n), 1e-3)
        s["base"] = normal((rows, k), 1e-3)
        s["h"] = torch.where((s["ids"] >= 0)[:, None],
                             normal((rows, rank), 1.5, torch.float32), 0.0)
    _own_adapters(s)
    return s


def _own_dropout(s):
    """The buffers that a user of the library keeps beside the inputs."""
    if own:
        import delayed_scaling_linear_amd as dsl
        c = s["case"]
        s["drop"] = dsl.Dropout(c["p"], s["rng"])
        # A gradient's or a plain dropout's cast needs the codes alone.
        s["y"] = torch.empty_like(s["x"]) if c["op"] == "dropout" or c["residual"] else None
        if c["op"] == "dropout_cast":
            s["out"] = dsl.Float8Tensor.empty(c["rows"], c["cols"], c["fmt"])
            s["amax"] = torch.zeros(1, device="cuda")
            s["dbias"] = s["ws"] = None
            if c["dbias"]:
                s["dbias"] = torch.empty(c["cols"], device="cuda")
                s["ws"] = torch.empty(dsl.fp8_cast_dbias_workspace_bytes(c["rows"], c["cols"]),
                                      dtype=torch.uint8, device="cuda")


def _own_adapters(s):
    """The adapters' handle, the batch's plan (built once, used by every
    layer of a step), the outputs and the workspace."""
    if own:
        import delayed_scaling_linear_amd as dsl
        c = s["case"]
        s["w"] = dsl.Adapters(s["a"], s["b"], s["alpha"])
        s["plan"] = dsl.AdapterPlan.empty(c["rows"], c["adapters"])
        dsl.fp8_adapter_plan(s["ids"], s["plan"])
        s["drop"] = dsl.Dropout(c["p"], s["rng"]) if c["p"] > 0 else None
        s["ws"] = torch.empty(dsl.fp8_adapter_workspace_bytes(c["rows"], c["adapters"], c["rank"],
                                                              c["k"], c["n"]),
                              dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty_like(s["base"])
        if c["op"] == "adapter_fwd":
            s["h"] = torch.empty(c["rows"], c["rank"], device="cuda") if c["keep_h"] else None
        else:
            dtype = torch.float32 if c["grads"] == "fp32" else torch.bfloat16
            s["da"] = torch.empty(s["a"].shape, dtype=dtype, device="cuda")
            s["db"] = torch.empty(s["b"].shape, dtype=dtype, device="cuda")


def _threshold(p):
    return int(round(p * 65536))


def _philox(e, rng):
    """Philox4x32-7 words [..., 4] for the 64-bit group indices e (int64)."""
    c = [e & MASK32, (e >> 32) & MASK32, rng[1] & MASK32, (rng[1] >> 32) & MASK32]
    k = [rng[0] & MASK32, (rng[0] >> 32) & MASK32]
    for _ in range(7):
        lo, hi = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((hi >> 32) & MASK32) ^ c[1] ^ k[0], hi & MASK32,
             ((lo >> 32) & MASK32) ^ c[3] ^ k[1], lo & MASK32]
        k = [(k[0] + 0x9E3779B9) & MASK32, (k[1] + 0xBB67AE85) & MASK32]
    return torch.stack(torch.broadcast_tensors(*c), -1)


def _keep(rows, cols, p, rng):
    """The mask [rows, cols] of the kept elements."""
    e = torch.arange(rows * cols // 8, device=rng.device, dtype=torch.int64)
    w = _philox(e, rng)
    u = torch.stack((w & 0xFFFF, w >> 16), -1)
    return (u >= _threshold(p)).view(rows, cols)


def _factor(p):
    return float(np.float32(65536.0 / (65536 - _threshold(p))))


def _dropped(x, p, rng):
    """fp32 dropout of x."""
    x = x.float()
    if p == 0.0:
        return x
    return torch.where(_keep(x.shape[0], x.shape[1], p, rng), x * _factor(p), 0.0)


def _plain_dropout(s):
    c = s["case"]
    y = _dropped(s["x"], c["p"], s["rng"])
    if c["residual"]:
        y = s["residual"].float() + y
    y = y.to(s["x"].dtype)
    if c["op"] == "dropout":
        return {"y": y}
    top = FP8_MAX[c["fmt"]]
    codes = (y.float() * s["scale"]).clamp(-top, top).to(FP8_TYPE[c["fmt"]])
    out = {"codes": codes, "codes_t": codes.t().contiguous(), "amax": y.abs().max().float(),
           "scale_inv": 1.0 / s["scale"]}
    if c["residual"]:
        out["y"] = y
    if c["dbias"]:
        out["dbias"] = y.float().sum(0)
    return out


def _side_by_side(s):
    """[rows, adapters] 1 where the row belongs to the adapter, times alpha."""
    count = s["case"]["adapters"]
    hit = s["ids"][:, None] == torch.arange(count, device="cuda", dtype=torch.int32)
    return hit[:, :, None].float(), s["alpha"][None, :, None]


def _plain_forward(s):
    c = s["case"]
    count, rank, rows = c["adapters"], c["rank"], c["rows"]
    mine, alpha = _side_by_side(s)
    xd = _dropped(s["x"], c["p"], s["rng"])
    # All adapters' ranks side by side, then each row's own kept.
    every = xd @ s["a"].float().reshape(count * rank, -1).t()
    every = every.view(rows, count, rank) * alpha * mine
    b = s["b"].float().permute(0, 2, 1).reshape(count * rank, -1)
    y = (s["base"].float() + every.reshape(rows, -1) @ b).to(torch.bfloat16)
    return {"y": y, "h": every.sum(1)} if c["keep_h"] else {"y": y}


def _plain_backward(s):
    c = s["case"]
    count, rank, rows = c["adapters"], c["rank"], c["rows"]
    mine, alpha = _side_by_side(s)
    dy, xd = s["dy"].float(), _dropped(s["x"], c["p"], s["rng"])
    a = s["a"].float().reshape(count * rank, -1)
    b = s["b"].float().permute(0, 2, 1).reshape(count * rank, -1)
    g = ((dy @ b.t()).view(rows, count, rank) * alpha * mine).reshape(rows, -1)
    h = (s["h"][:, None, :] * mine).reshape(rows, -1)
    dx = s["base"].float() + _dropped(g @ a, c["p"], s["rng"])
    dtype = torch.float32 if c["grads"] == "fp32" else torch.bfloat16
    db = (dy.t() @ h).view(-1, count, rank).permute(1, 0, 2).contiguous()
    return {"dx": dx.to(torch.bfloat16), "da": (g.t() @ xd).view(count, rank, -1).to(dtype),
            "db": db.to(dtype)}


def _own_run(s):
    import delayed_scaling_linear_amd as dsl
    c = s["case"]
    if c["op"] == "dropout":
        dsl.fp8_dropout(s["x"], s["drop"], s["y"], residual=s["residual"])
        return {"y": s["y"]}
    if c["op"] == "dropout_cast":
        out = s["out"]
        dsl.fp8_dropout_cast_transpose_amax(s["x"], s["drop"], s["scale"], out, s["amax"],
                                            residual=s["residual"], y=s["y"], dbias=s["dbias"],
                                            workspace=s["ws"])
        t = FP8_TYPE[c["fmt"]]
        r = {"codes": out.data.view(t), "codes_t": out.data_t.view(t), "amax": s["amax"][0],
             "scale_inv": out.scale_inv}
        if c["residual"]:
            r["y"] = s["y"]
        return dict(r, dbias=s["dbias"]) if c["dbias"] else r
    if c["op"] == "adapter_fwd":
        dsl.fp8_adapter_fwd(s["w"], s["plan"], s["x"], s["base"], s["out"], h=s["h"],
                            drop=s["drop"], workspace=s["ws"])
        return {"y": s["out"], "h": s["h"]} if c["keep_h"] else {"y": s["out"]}
    dsl.fp8_adapter_backward(s["w"], s["plan"], s["x"], s["dy"], s["h"], dx_base=s["base"],
                             dx=s["out"], da=s["da"], db=s["db"], drop=s["drop"],
                             workspace=s["ws"])
    return {"dx": s["out"], "da": s["da"], "db": s["db"]}


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op in ("dropout", "dropout_cast"):
        return _plain_dropout(state)
    return _plain_forward(state) if op == "adapter_fwd" else _plain_backward(state)


def work(case):
    if case["op"] in ("dropout", "dropout_cast"):
        e = case["rows"] * case["cols"]
        size = 4 if case.get("dtype") == "fp32" else 2
        moved = size * e * (3 if case["residual"] else 2)
        if case["op"] == "dropout_cast":
            moved = e * (8 if case["residual"] else 4) + (4 * case["cols"] if case["dbias"] else 0)
        return {"bytes": moved + 16, "flops": 2 * e}
    rows, k, n, rank = (case[v] for v in ("rows", "k", "n", "rank"))
    live = rows * (1.0 - case["none"])
    # Adapters that a row asks for: all of them where rows are many.
    used = case["adapters"]
    if case["order"] == "scatter":
        used *= 1.0 - (1.0 - 1.0 / case["adapters"]) ** live
    weights = 2 * used * rank * (k + n)
    if case["op"] == "adapter_fwd":
        moved = 2 * live * k + 4 * rows * n + weights + 4 * rows
        moved += 4 * rows * rank if case["keep_h"] else 0
        return {"bytes": int(moved), "flops": int(2 * live * rank * (k + n))}
    size = 4 if case["grads"] == "fp32" else 2
    moved = 2 * live * (k + n) + 4 * rows * k + 4 * live * rank + weights + 4 * rows
    moved += size * case["adapters"] * rank * (k + n)
    return {"bytes": int(moved), "flops": int(4 * live * rank * (k + n))}


# 64-bit results from the definitions, apart from the plain forms above: the
# random words by numpy's unsigned integers, each adapter's rows by themselves.

def _exact_mask(rows, cols, p, seed_offset):
    seed, offset = (int(v) & (2 ** 64 - 1) for v in seed_offset)
    u64, m = np.uint64, np.uint64(MASK32)
    e = np.arange(rows * cols // 8, dtype=u64)
    x0, x1 = e & m, e >> u64(32)
    x2, x3 = np.full_like(e, offset & MASK32), np.full_like(e, offset >> 32)
    key0, key1 = seed & MASK32, seed >> 32
    for _ in range(7):
        p0, p1 = x0 * u64(0xD2511F53), x2 * u64(0xCD9E8D57)
        x0, x1 = (p1 >> u64(32)) ^ x1 ^ u64(key0), p1 & m
        x2, x3 = (p0 >> u64(32)) ^ x3 ^ u64(key1), p0 & m
        key0, key1 = (key0 + 0x9E3779B9) & MASK32, (key1 + 0xBB67AE85) & MASK32
    words = np.stack([x0, x1, x2, x3], 1).astype("<u4")
    half = words.view("<u2").reshape(rows, cols)
    return torch.from_numpy(half.astype(np.int32) >= int(round(p * 65536))).cuda()


def _on_grid(v, fmt):
    """v rounded to the format's grid, ties to even (mantissa bits 3 and 2,
    least exponents -6 and -14)."""
    exponent = torch.frexp(v)[1] - 1
    step = torch.ldexp(torch.ones_like(v), exponent.clamp(min=(-6, -14)[fmt]) - (3, 2)[fmt])
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    rows, p = case["rows"], case["p"]
    cols = case["cols"] if "cols" in case else case["k"]
    mask = _exact_mask(rows, cols, p, s["rng"].cpu().tolist())
    factor = torch.tensor(65536.0 / (65536 - int(round(p * 65536)))).float().double().item()
    xd = s["x"].double() * factor
    xd[~mask] = 0.0
    if case["op"] in ("dropout", "dropout_cast"):
        y = xd if s["residual"] is None else s["residual"].double() + xd
        if case["op"] == "dropout":
            return {"y": y}
        # The codes, the amax and the bias gradient are those of y as stored:
        # an fp32 product, an fp32 sum, one rounding to bf16.
        stored = xd.float() if s["residual"] is None else s["residual"].float() + xd.float()
        stored = stored.to(torch.bfloat16).double()
        top = FP8_MAX[case["fmt"]]
        scale = s["scale"].double()
        codes = _on_grid((stored * scale).float().double().clamp(-top, top), case["fmt"])
        out = {"codes": codes, "codes_t": codes.t().contiguous(), "amax": stored.abs().max(),
               "scale_inv": 1.0 / scale}
        if case["residual"]:
            out["y"] = y
        if case["dbias"]:
            out["dbias"] = stored.sum(0)
        return out
    rank, count = case["rank"], case["adapters"]
    forward = case["op"] == "adapter_fwd"
    out = s["base"].double()
    h = torch.zeros(rows, rank, dtype=torch.float64, device="cuda")
    da, db = (torch.zeros(s[v].shape, dtype=torch.float64, device="cuda") for v in "ab")
    for i in range(count):
        at = torch.nonzero(s["ids"] == i)[:, 0]
        a, b, alpha = s["a"][i].double(), s["b"][i].double(), s["alpha"][i].double()
        if forward:
            h[at] = alpha * (xd[at] @ a.t())
            out[at] += h[at] @ b.t()
        else:
            dy = s["dy"][at].double()
            g = alpha * (dy @ b)
            da[i], db[i] = g.t() @ xd[at], dy.t() @ s["h"][at].double()
            out[at] += (g @ a) * mask[at] * factor
    if forward:
        return {"y": out, "h": h} if case["keep_h"] else {"y": out}
    return {"dx": out, "da": da, "db": db}
