"""GPU parity of fp8_grad_norm and fp8_adamw_step.

Moments, codes and scales are compared bit for bit: the definition rounds every
operation.  A parameter is compared with the float64 update from the same fp32
moments: the factor of the weight decay, its product and the last subtraction
are 3 roundings of 2^-24 of the parameter, and the update's factors, products,
root, sum and quotient are within 6 * 2^-24 + 2^-22 of it.  A bf16 parameter must
lie between the stochastic roundings of the ends of that interval: with one number u
the rounding never falls where its argument rises.  (Nearly always the ends agree;
where p0 and the update nearly cancel, the interval holds several bf16 values.)"""
import weakref

import numpy as np
import pytest
import torch

import delayed_scaling_linear_amd as dsl
from tests import adamw_reference as ref
from tests import op_reference as op
from tests.gpu_util import DEV, bf16_values, bits8, bits16, f32, f32_bits

pytestmark = pytest.mark.gpu

F = np.float32
LR, B1, B2, EPS, SEED = 3e-3, 0.9, 0.95, 1e-6, 0xFEDCBA9876543210


def _make(n, param, grad, bits, seed, copy=False, wd=0.1):
    r = np.random.default_rng(seed)
    t = lambda a: torch.from_numpy(a.astype(F))
    p, g = t(r.standard_normal(n)).to(param), t(r.standard_normal(n) * 1e-2).to(grad)
    m, v = (r.standard_normal(n) * 1e-2).astype(F), (r.random(n) * 1e-4).astype(F)
    item = dsl.AdamWTensor.zeros(
        p.to(DEV), g.to(DEV), bits,
        copy=torch.full((n,), -7.0, dtype=torch.bfloat16, device=DEV) if copy else None,
        weight_decay=wd)
    if bits == 8:
        for name, x in (("m", m), ("v", v)):
            codes, scales = ref.encode(x, np.full(n, 32768), name == "v")
            getattr(item, name).copy_(torch.from_numpy(codes))
            getattr(item, name + "_scale").copy_(torch.from_numpy(scales))
    else:
        item.m.copy_(torch.from_numpy(m))
        item.v.copy_(torch.from_numpy(v))
    return item


def _state_words(opt):
    """The steps taken; the counters behind them are zero between calls."""
    assert not opt.state[1:].any()
    return int(opt.state[0])


def _values(t):
    return bf16_values(bits16(t)).astype(np.float64) if t.dtype == torch.bfloat16 \
        else f32(t).astype(np.float64)


def _state(item):
    """What a step reads: float64 p, fp32 g, m, v."""
    if item.m_scale is None:
        m, v = f32(item.m), f32(item.v)
    else:
        m = ref.decode(bits8(item.m), f32(item.m_scale))
        v = ref.decode(bits8(item.v), f32(item.v_scale), square=True)
    return _values(item.param), _values(item.grad).astype(F), m, v


def _check(item, index, before, t, lr=LR, scale=None):
    p0, g, m, v = before
    n = p0.size
    m, v, p, update = ref.step(p0, g, m, v, t, float(F(lr)), float(F(item.weight_decay)), B1, B2, EPS,
                               scale)
    if item.m_scale is None:
        np.testing.assert_array_equal(f32_bits(item.m), m.view(np.uint32))
        np.testing.assert_array_equal(f32_bits(item.v), v.view(np.uint32))
    else:
        u = ref.words(n, 4, 2 * index, t, SEED)
        for codes, scales, x, half in ((item.m, item.m_scale, m, 0), (item.v, item.v_scale, v, 1)):
            want, want_scales = ref.encode(x, u[:, half].astype(np.int64), half == 1)
            np.testing.assert_array_equal(f32(scales), want_scales)
            np.testing.assert_array_equal(bits8(codes), want)
    slack = 2.0 ** -24 * 3 * np.maximum(np.abs(p0), np.abs(p)) + (2.0 ** -22 + 6 * 2.0 ** -24) * update
    if item.param.dtype == torch.float32:
        assert (np.abs(f32(item.param) - p) <= slack).all()
        if item.copy is not None:
            np.testing.assert_array_equal(bits16(item.copy), op.bf16_round(f32(item.param)))
    else:
        u = ref.words(n, 8, 2 * index + 1, t, SEED)[:, 0].astype(np.int64)
        got, lo, hi = (bf16_values(b) for b in (bits16(item.param),
                                                ref.stochastic_bf16(p - slack, u),
                                                ref.stochastic_bf16(p + slack, u)))
        assert ((lo <= got) & (got <= hi)).all()
        assert n == 0 or (lo == hi).mean() > 0.98            # so the ends tell something


TYPES = [(p, g, b) for p in (torch.float32, torch.bfloat16) for g in (torch.float32, torch.bfloat16)
         for b in (32, 8)]
SIZES = [0, 1, 2, 3, 4, 5, 7, 8, 9, 255, 256, 257, 1023, 2047, 2048, 2049, 5000, 20001]


def _adamw(items, lr=LR, t=0):
    opt = dsl.AdamW(items, lr=lr, betas=(B1, B2), eps=EPS, seed=SEED)
    opt.steps.fill_(t)
    return opt


@pytest.mark.parametrize("param, grad, bits", TYPES)
def test_sizes_in_one_call(param, grad, bits):
    """Every size, tails within a block and without a value among them."""
    items = [_make(n, param, grad, bits, n, copy=param == torch.float32 and n % 2 == 1)
             for n in SIZES]
    opt = _adamw(items, t=4)
    before = [_state(i) for i in items]
    opt.step()
    assert opt.steps.tolist() == [5]
    for index, (item, state) in enumerate(zip(items, before)):
        _check(item, index, state, 5)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_steps(bits):
    """From zeros on, three steps: the bias corrections of the first ones."""
    g = torch.Generator().manual_seed(1)
    item = dsl.AdamWTensor.zeros(torch.randn(777, generator=g).to(DEV),
                                 torch.randn(777, generator=g).to(DEV), bits, weight_decay=0.01)
    opt = _adamw([item])
    for t in (1, 2, 3):
        before = _state(item)
        opt.step()
        _check(item, 0, before, t)
        item.grad = torch.randn(777, generator=g).to(DEV)


def test_types_mixed_over_several_launches():
    """Over 48 tensors of every type: their place in the call feeds the rounding."""
    items = [_make(40 + 97 * i % 900, *TYPES[i % 8], seed=i, wd=0.01 * (i % 3))
             for i in range(117)]
    opt = _adamw(items, t=2 ** 33)
    before = [_state(i) for i in items]
    opt.step()
    assert _state_words(opt) == 2 ** 33 + 1
    for index, (item, state) in enumerate(zip(items, before)):
        _check(item, index, state, 2 ** 33 + 1)


def test_many_tiles():
    """More tiles than workgroups: each takes several, over tensors of two kinds."""
    items = [_make(1 << 22, torch.float32, torch.bfloat16, 8, 1, copy=True),
             _make((1 << 22) + 3, torch.bfloat16, torch.bfloat16, 32, 2),
             _make(2500001, torch.float32, torch.float32, 32, 3)]
    opt = _adamw(items, t=99)
    before = [_state(i) for i in items]
    opt.step()
    for index, (item, state) in enumerate(zip(items, before)):
        _check(item, index, state, 100)


@pytest.mark.parametrize("param, grad, bits", TYPES)
def test_longer_waves(param, grad, bits):
    """From a tile a compute unit on a wave takes four blocks at a time: whole ones, and
    ends of one value to four blocks."""
    sizes = [4096 * 300 + extra for extra in (0, 1, 255, 256, 1029, 2047, 4095)]
    items = [_make(n, param, grad, bits, i, copy=param == torch.float32 and i % 2 == 1)
             for i, n in enumerate(sizes)]
    opt = _adamw(items, t=7)
    before = [_state(i) for i in items]
    opt.step()
    for index, (item, state) in enumerate(zip(items, before)):
        _check(item, index, state, 8)


def test_no_tensors_count_a_step():
    opt = _adamw([], t=7)
    opt.step()
    opt.tensors = [_make(0, torch.float32, torch.float32, 32, 0)]
    opt.step()
    assert _state_words(opt) == 9


@pytest.mark.parametrize("bits", [32, 8])
def test_noop_and_gradient_scale(bits):
    item = _make(1000, torch.float32, torch.float32, bits, 5, copy=True)
    opt = _adamw([item], t=10)
    flag, scale = torch.ones(1, dtype=torch.int32, device=DEV), torch.tensor([0.3], device=DEV)
    tensors = [t for t in (item.param, item.m, item.v, item.m_scale, item.v_scale, item.copy)
               if t is not None]
    keep = [t.clone() for t in tensors]
    opt.step(grad_scale=scale, noop_flag=flag)
    assert all(torch.equal(a, b) for a, b in zip(tensors, keep)) and _state_words(opt) == 10
    flag.zero_()
    before = _state(item)
    opt.step(grad_scale=scale, noop_flag=flag)
    _check(item, 0, before, 11, scale=0.3)


@pytest.mark.parametrize("bits", [32, 8])
def test_special_gradients(bits):
    """NaN, infinities, the smallest and largest values: what is not finite stays
    within its element, and the rest of its block is stored as without it."""
    item = _make(600, torch.float32, torch.float32, bits, 6)
    item.grad[3], item.grad[300], item.grad[301] = float("nan"), float("inf"), float("-inf")
    item.grad[512:520] = torch.tensor([1e-45, -1e-45, 1e-30, 3e38, -3e38, 0.0, 1e-19, 1e19])
    opt = _adamw([item], t=20)
    for t in (21, 22):
        p0, g, m, v = _state(item)
        opt.step()
        m1, v1, p1, update = ref.step(p0, g, m, v, t, float(F(LR)), float(F(0.1)), B1, B2, EPS)
        got = f32(item.param)
        bad = np.isnan(p1)
        assert bad[3] and (np.isnan(got) == bad).all()
        assert not bad[515] and v1[515] == np.inf            # overflowed: held still
        if bits == 32:
            np.testing.assert_array_equal(f32(item.m), m1)
            np.testing.assert_array_equal(f32(item.v), v1)
        else:
            u = ref.words(600, 4, 0, t, SEED).astype(np.int64)
            for codes, scales, x, half in ((item.m, item.m_scale, m1, 0),
                                           (item.v, item.v_scale, v1, 1)):
                want, want_scales = ref.encode(x, u[:, half], half == 1)
                np.testing.assert_array_equal(f32(scales), want_scales)
                np.testing.assert_array_equal(bits8(codes), want)
        fine = ~bad
        slack = 2.0 ** -24 * 3 * np.maximum(np.abs(p0), np.abs(p1)) + \
            (2.0 ** -22 + 6 * 2.0 ** -24) * update
        assert (np.abs(got[fine] - p1[fine]) <= slack[fine]).all()


def test_bf16_parameters_at_their_ends():
    """NaN, infinities, zeros and the largest value are not carried past."""
    item = dsl.AdamWTensor.zeros(
        torch.tensor([float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 3.3895e38, 1e-40],
                     dtype=torch.bfloat16, device=DEV),
        torch.zeros(7, device=DEV), 32)
    before = bits16(item.param)
    opt = _adamw([item])
    for _ in range(5):
        opt.step()
    got = bits16(item.param)
    assert got[0] == 0x7FC0
    np.testing.assert_array_equal(got[1:], before[1:])       # a step of zero is exact


def test_small_steps_reach_bf16_parameters_and_8_bit_moments():
    """What rounding to nearest would lose arrives on average: v of a zero gradient
    falls by 1 - beta2 a step, a bf16 parameter takes updates of 2^-5 of its step."""
    n, steps = 1 << 16, 50
    item = dsl.AdamWTensor.zeros(torch.ones(n, dtype=torch.bfloat16, device=DEV),
                                 torch.full((n,), 1.0, device=DEV), 8)
    item.v.fill_(0x38)                                       # 1.0
    item.v_scale.fill_(1.0)
    opt = dsl.AdamW([item], lr=0.0, betas=(0.9, 0.999), seed=3)
    item.grad.zero_()
    for _ in range(steps):
        opt.step()
    v = (item.v.view(torch.float8_e4m3fn).float().view(-1, 256) * item.v_scale[:, None]).double()
    # Each step's rounding is unbiased with a deviation of at most half a neighbour's
    # distance, 2^-4: 50 of them over 65536 values move the mean by 2^-4 * sqrt(50) / 256
    # = 0.0017 (one deviation); the fall is 0.0488.
    assert abs(float(v.mean()) - 0.999 ** steps) < 5 * 0.0018
    p = dsl.AdamWTensor.zeros(torch.ones(n, dtype=torch.bfloat16, device=DEV),
                              torch.ones(n, device=DEV), 32)
    opt = dsl.AdamW([p], lr=2.0 ** -12, betas=(0.0, 0.0), eps=1e-12, seed=3)
    for _ in range(steps):
        opt.step()
    # Every update is 2^-12 against a distance of 2^-8 below 1: the mean's deviation is
    # at most 2^-9 * sqrt(50) / 256 = 5.4e-5, the fall 0.0122.
    assert abs(float(p.param.double().mean()) - (1 - steps * 2.0 ** -12)) < 5 * 5.5e-5


def test_past_32_bits_of_values():
    """The last values of a tensor of 2^32 + 1037 (bf16, states in 8 bits: 26 GB)."""
    n, tail = (1 << 32) + 1037, 5000
    like = dict(device=DEV, dtype=torch.bfloat16)
    item = dsl.AdamWTensor.zeros(torch.zeros(n, **like), torch.zeros(n, **like), 8)
    small = _make(tail, torch.bfloat16, torch.bfloat16, 32, 7)
    item.param[-tail:], item.grad[-tail:] = small.param, small.grad
    opt = _adamw([item])
    p0, g = _values(small.param), _values(small.grad).astype(F)
    opt.step()
    m, v, p, update = ref.step(p0, g, np.zeros(tail, F), np.zeros(tail, F), 1, float(F(LR)), 0.0, B1,
                               B2, EPS)
    slack = 2.0 ** -24 * 3 * np.maximum(np.abs(p0), np.abs(p)) + (2.0 ** -22 + 6 * 2.0 ** -24) * update
    group = (n - tail) // 8
    words = op.philox4x32([np.arange(group, (n + 7) // 8, dtype=np.uint64), 1, 1, 0],
                          (SEED & 0xFFFFFFFF, SEED >> 32), 7)
    u = np.stack(words, 1).astype("<u4").view("<u2").reshape(-1)[n - tail - 8 * group:][:tail]
    got = bf16_values(bits16(item.param[-tail:]))
    lo, hi = (bf16_values(ref.stochastic_bf16(p + s, u.astype(np.int64))) for s in (-slack, slack))
    assert ((lo <= got) & (got <= hi)).all()
    # Whole blocks of the end: from the last multiple of 256 within it.
    first = (n - tail + 255) // 256 * 256
    x = m[first - (n - tail):]
    np.testing.assert_array_equal(f32(item.m_scale[first // 256:]), ref.scales_of(x))
    assert int(item.m[:-tail].max()) == 0 and (item.param[:-tail] == 0).all()


# ---- the norm ------------------------------------------------------------------

def _norm(grads, most=float("inf")):
    out = [torch.full((1,), -7.0, device=DEV), torch.full((1,), -7.0, device=DEV),
           torch.full((1,), -7, dtype=torch.int32, device=DEV)]
    ws = torch.full((dsl.fp8_grad_norm_workspace_bytes(),), 0xFF, dtype=torch.uint8, device=DEV)
    dsl.fp8_grad_norm(grads, out[0], ws, most, factor=out[1], noop_flag=out[2])
    return float(out[0]), float(out[1]), int(out[2])


def _check_norm(norm, grads):
    """One rounding to fp32 of a 64-bit sum, whose own error 2^-50 covers."""
    want = np.sqrt(sum((_values(g) ** 2).sum() for g in grads))
    assert abs(norm - want) <= 2.0 ** -24 * want * (1 + 2.0 ** -20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 3, 4, 5, 255, 1037, 8191, 8192, 8193, 100003, (1 << 24) + 5])
def test_norm_sizes(n, dtype):
    g = torch.randn(n, generator=torch.Generator(DEV).manual_seed(n), device=DEV).to(dtype)
    norm, factor, flag = _norm([g], 0.5)
    _check_norm(norm, [g])
    assert flag == 0 and factor == (float(F(0.5) / F(norm)) if norm > 0.5 else 1.0)


@pytest.mark.parametrize("count", [0, 1, 99, 100, 101, 250])
def test_norm_of_many_tensors(count):
    """Sizes of one value to several tiles, empty tensors among them; the first
    launch small or large."""
    gen = torch.Generator(DEV).manual_seed(count)
    sizes = [0 if i % 7 == 3 else 1 + (i * 7919) % 30011 for i in range(count)]
    for order in (sizes, sizes[::-1]):
        grads = [torch.randn(n, generator=gen, device=DEV).to([torch.float32, torch.bfloat16][i % 2])
                 for i, n in enumerate(order)]
        norm, factor, flag = _norm(grads)
        _check_norm(norm, grads)
        assert (factor, flag) == (1.0, 0)
        assert _norm(grads)[0] == norm                       # the same bits


def test_norm_of_empty_tensors():
    assert _norm([torch.empty(0, device=DEV)] * 3) == (0.0, 1.0, 0)


def test_norm_at_the_ends():
    """Squares beyond fp32's range on both sides; what is not finite."""
    big, small = torch.full((1000,), 1e30, device=DEV), torch.full((1000,), 1e-30, device=DEV)
    for g in (big, small):
        norm, _, flag = _norm([g])
        _check_norm(norm, [g])
        assert flag == 0
    norm, factor, flag = _norm([big], 1.0)
    assert factor == float(F(1.0) / F(norm))
    over = torch.full((100,), 3e38, device=DEV)              # a norm that fp32 does not hold
    assert _norm([over], 1.0) == (float("inf"), 0.0, 1)
    big[17] = float("inf")
    assert _norm([small, big], 1.0)[::2] == (float("inf"), 1)
    big[18] = float("nan")
    norm, factor, flag = _norm([big, small], 1.0)
    assert np.isnan(norm) and factor == 1.0 and flag == 1


# ---- captured, on other streams ----------------------------------------------------

@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_steps_captured(bits):
    """Replays of a captured norm and step, with the program's own work, new gradients
    and a new learning rate between them, against eager steps on a copy: the same bits.
    An overflowed gradient leaves its step out."""
    def make():
        items = [_make(n, torch.float32, torch.float32, bits, n, copy=True)
                 for n in (5000, 33, 256 * 40)]
        lr = torch.full((1,), LR, device=DEV)
        opt = _adamw(items, lr=lr, t=3)
        own = [torch.zeros(1, device=DEV), torch.zeros(1, device=DEV),
               torch.zeros(1, dtype=torch.int32, device=DEV),
               torch.empty(dsl.fp8_grad_norm_workspace_bytes(), dtype=torch.uint8, device=DEV)]

        def run():
            dsl.fp8_grad_norm(opt.grads, own[0], own[3], 0.7, factor=own[1], noop_flag=own[2])
            opt.step(grad_scale=own[1], noop_flag=own[2])
        return opt, run, own

    def tensors(opt):
        return [t for i in opt.tensors for t in (i.param, i.m, i.v, i.m_scale, i.v_scale, i.copy)
                if t is not None] + [opt.state]

    (a, run_a, own_a), (b, run_b, own_b) = make(), make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_a()
    torch.cuda.current_stream().wait_stream(side)
    run_b()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        run_a()
    for i in range(5):
        gen = torch.Generator(DEV).manual_seed(i)
        for x, y in zip(a.tensors, b.tensors):
            x.grad.normal_(generator=gen)
            y.grad.copy_(x.grad)
        if i == 3:
            a.tensors[1].grad[7] = b.tensors[1].grad[7] = float("inf")
        a.lr.mul_(0.5)
        b.lr.mul_(0.5)
        torch.cuda.synchronize()
        graph.replay()
        run_b()
        torch.cuda.synchronize()
        for x, y in zip(tensors(a) + own_a[:3], tensors(b) + own_b[:3]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        assert int(own_a[2]) == (i == 3) and _state_words(a) == 3 + 1 + i + (i < 3)


def test_a_dropped_gradient_is_not_kept():
    """What a program frees between steps is free; the next gradient may lie in its place
    or elsewhere."""
    item = _make(3000, torch.float32, torch.float32, 8, 9)
    opt = _adamw([item], t=1)
    for t in (2, 3, 4):
        before = _state(item)
        opt.step()
        _check(item, 0, before, t)
        gone = weakref.ref(item.grad)
        item.grad = None
        assert gone() is None
        with pytest.raises(ValueError):
            opt.step()
        hold = torch.empty(3000 * t, device=DEV)
        item.grad = torch.randn(3000, generator=torch.Generator(DEV).manual_seed(t), device=DEV)
        del hold


def test_handles_see_what_changed():
    """A tensor of another shape or type in a handle is noticed at the next step."""
    item = _make(300, torch.float32, torch.float32, 8, 8)
    opt = _adamw([item])
    opt.step()
    item.grad = torch.zeros(299, device=DEV)
    with pytest.raises(ValueError):
        opt.step()
    item.grad = torch.zeros(600, device=DEV)[::2]
    with pytest.raises(ValueError):
        opt.step()
    item.grad = torch.zeros(300, dtype=torch.bfloat16, device=DEV)
    opt.step()
    item.m = item.m.float()
    with pytest.raises(TypeError):
        opt.step()
    assert _state_words(opt) == 2
    item.m = torch.zeros(300, dtype=torch.uint8, device=DEV)
    item.m_scale, item.v_scale = item.m_scale.cpu(), item.v_scale.cpu()
    with pytest.raises(ValueError):
        opt.step()
    odd = torch.zeros(304, device=DEV)[1:301]
    item = dsl.AdamWTensor.zeros(odd, torch.zeros(300, device=DEV))
    with pytest.raises(dsl.Fp8Error):                        # not 16-byte aligned
        _adamw([item]).step()
