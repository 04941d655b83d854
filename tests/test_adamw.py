"""The AdamW step over many tensors: refusals on the CPU, parity with the formula in 64 bits on the GPU,
and a run of forward, backward and step together."""
import ctypes
import math

import numpy as np
import pytest
import torch

import rank_gemm_lora_amd as rg
from tests import routed_ref as rr

OK, NULL, SHAPE, DTYPE, NONFIN, ALIGN, OVERLAP, WS, UNSUP, HIP = range(10)
F32, BF16 = rg.LORA_F32, rg.LORA_BF16
DEV = "cuda:0"
BASE = 0x10_0000_0000
U = 2.0 ** -24


def say(*a):
    print(*a, flush=True)


# ----------------------------------------------------------------------------- refusals (no GPU)

def tensor(i=0, n=1000, master=False, eight=False, **kw):
    a = {k: BASE * (8 * i + j + 1) for j, k in enumerate(("param", "master", "grad", "m", "v", "m_scale", "v_scale"))}
    if not master:
        a["master"] = None
    if not eight:
        a["m_scale"] = a["v_scale"] = None
    a.update(kw)
    return rg.LoraAdamWTensor(a["param"], a["master"], a["grad"], a["m"], a["v"], a["m_scale"], a["v_scale"], n)


def plan(ts, p=BF16, g=F32, bits=32, table=BASE * 1000, tb=1 << 20, out=None, null=False):
    arr = (rg.LoraAdamWTensor * max(1, len(ts)))(*ts)
    out = rg.LoraAdamWPlan() if out is None else out
    return rg._lib.lora_adamw_plan(None if null else arr, len(ts), p, g, bits, table, tb, ctypes.byref(out), None)


@pytest.mark.parametrize("ts,kw,code", [
    ([tensor()], dict(null=True), NULL), ([tensor(param=None)], {}, NULL), ([tensor(grad=None)], {}, NULL),
    ([tensor(m=None)], {}, NULL), ([tensor(v=None)], {}, NULL), ([tensor()], dict(bits=8), NULL),
    ([tensor(eight=True)], {}, NULL),
    ([tensor(n=-1)], {}, SHAPE), ([tensor(n=1 << 41)], {}, UNSUP), ([tensor(), tensor(1, n=1 << 40)], {}, UNSUP),
    ([tensor()], dict(p=2), DTYPE), ([tensor()], dict(g=-1), DTYPE), ([tensor(master=True)], dict(p=F32), DTYPE),
    ([tensor()], dict(bits=16), UNSUP),
    ([tensor(param=BASE + 1)], {}, ALIGN), ([tensor(grad=BASE * 3 + 2)], {}, ALIGN), ([tensor(m=BASE * 4 + 1)], {}, ALIGN),
    ([tensor(master=True, eight=True, m_scale=BASE * 6 + 2)], dict(bits=8), ALIGN),
    ([tensor()], dict(table=BASE * 1000 + 8), ALIGN),
    ([tensor()], dict(table=None), WS), ([tensor()], dict(tb=64), WS),
    ([tensor(grad=BASE + 1000)], {}, OVERLAP), ([tensor(v=BASE * 4 + 2000)], {}, OVERLAP),
    ([tensor(), tensor(1, param=BASE + 1998)], {}, OVERLAP), ([tensor()], dict(table=BASE * 4), OVERLAP),
    ([tensor(), tensor(1, m=BASE * 3)], {}, OVERLAP),
])
def test_plan_refusals(ts, kw, code):
    assert plan(ts, **kw) == code


def test_plan_of_nothing_and_table_size():
    p = rg.LoraAdamWPlan()
    assert plan([], table=None, tb=0, out=p) == OK and p.n_blocks == 0
    assert rg._lib.lora_adamw_step(ctypes.byref(p), 1e-3, 0.9, 0.99, 1e-8, 0.0, 1, None, 1.0, None) == OK
    assert rg.lora_adamw_table_size([]) == 0
    small, large = rg.lora_adamw_table_size([tensor(n=1)]), rg.lora_adamw_table_size([tensor(n=1 << 26)])
    assert 0 < small < large
    assert rg._lib.lora_adamw_plan(None, 0, BF16, F32, 32, None, 0, None, None) == NULL


@pytest.mark.parametrize("kw,code", [
    (dict(lr=math.nan), NONFIN), (dict(b1=math.inf), NONFIN), (dict(eps=math.nan), NONFIN), (dict(gs=math.inf), NONFIN),
    (dict(gs=1e300), NONFIN), (dict(lr=1e300), NONFIN), (dict(wd=-math.inf), NONFIN),
    (dict(b1=1.0), UNSUP), (dict(b1=-0.1), UNSUP), (dict(b2=1.5), UNSUP), (dict(eps=-1.0), UNSUP),
    (dict(wd=-1.0), UNSUP), (dict(lr=-1.0), UNSUP), (dict(step=0), UNSUP), (dict(dev=BASE + 4), ALIGN),
    (dict(table=None), NULL), (dict(bits=4), UNSUP), (dict(chunk=100), UNSUP), (dict(pd=5), DTYPE),
    (dict(res=1), SHAPE), (dict(blocks=-1), SHAPE),
])
def test_step_refusals(kw, code):
    a = dict(lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.01, step=1, dev=None, gs=1.0, table=BASE, blocks=1, chunk=2048,
             pd=BF16, bits=32, res=0)
    a.update(kw)
    p = rg.LoraAdamWPlan(a["table"], a["blocks"], 1, a["chunk"], a["pd"], F32, a["bits"], a["res"])
    assert rg._lib.lora_adamw_step(ctypes.byref(p), a["lr"], a["b1"], a["b2"], a["eps"], a["wd"], a["step"], a["dev"],
                                   a["gs"], None) == code
    assert rg._lib.lora_adamw_step(None, 1e-3, 0.9, 0.99, 1e-8, 0.0, 1, None, 1.0, None) == NULL


def test_helper_refuses():
    p, g = [torch.zeros(4, 4)], [torch.zeros(4, 4)]
    for args, kw, err in (((p, []), {}, ValueError), (([], []), {}, ValueError), ((p, g), dict(state_bits=4), ValueError),
                          ((p, [torch.zeros(4, 3)]), {}, ValueError), ((p, g), dict(master=[]), ValueError),
                          ((p, [torch.zeros(4, 4).t()[:, :2]]), {}, ValueError),
                          ((p + [torch.zeros(2).bfloat16()], g + [torch.zeros(2)]), {}, TypeError),
                          ((p, g), dict(state=dict(m=[torch.zeros(15)])), ValueError),
                          ((p, g), dict(lr_step=torch.zeros(2)), TypeError)):
        with pytest.raises(err):
            rg.LoraAdamW(*args, **kw)


# ----------------------------------------------------------------------------- parity (GPU)

def unpack(codes, scale):
    """The values of 8-bit moments, in 64 bits."""
    n = codes.numel()
    return codes.cpu().float().double() * scale.cpu().double().repeat_interleave(256)[:n]


def moments(opt, i):
    """m and sqrt(v) or v of tensor i as the step reads them, 64 bits: (m, v)."""
    if opt.state_bits == 32:
        return opt.m[i].cpu().double().clone(), opt.v[i].cpu().double().clone()
    return unpack(opt.m[i], opt.m_scale[i]), unpack(opt.v[i], opt.v_scale[i]) ** 2


def expect(p, g, m, v, opt, k, gs=1.0):
    """The formula in 64 bits from what the step reads, with what its roundings let through."""
    b1, b2 = opt.betas
    g = g * gs
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    # m: two products and a sum, constants rounded once, g and (8 bits) m scaled once: 5 roundings of the parts
    bm = 5 * U * ((b1 * m).abs() + ((1 - b1) * g).abs())
    bv = 7 * U * (b2 * v + (1 - b2) * g * g) + 2.0 ** -149
    root = v1.sqrt()
    den = root / math.sqrt(1 - b2 ** k) + opt.eps
    size = opt.lr / (1 - b1 ** k)
    upd = m1 / den * size
    # denominator: half of v's relative error, the root, its constant, product and sum; division, product
    bu = size * bm / den + (3.5 + 8) * U * upd.abs()
    p1 = p * (1 - opt.lr * opt.weight_decay) - upd
    bp = bu + 3 * U * p.abs() + 2 * U * p1.abs()
    return p1, bp, m1, bm, v1, bv


def check(got, want, bound, what):
    bad = ~((got.double().cpu() - want).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), got.double().cpu()[bad][:3], want[bad][:3])


def check_eight(codes, scale, x, bx, what, positive):
    """Stored values against x (within bx of what the kernel rounded): the nearest e4m3 of its block."""
    top = torch.stack([b.abs().max() for b in x.split(256)])
    btop = torch.stack([b.max() for b in bx.split(256)])
    assert ((scale.cpu().double() - top / 448).abs() <= btop / 448 + 2 * U * top / 448).all(), what
    sc = scale.cpu().double().repeat_interleave(256)[: x.numel()]
    got = unpack(codes, scale)
    half = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * sc) * (1 + 8 * U)
    if positive:
        half = torch.where((x > 0) & (x < 2.0 ** -9 * sc), 2.0 ** -9 * sc, half)
        assert (got[(x > bx)] > 0).all(), what
    check(got, x, half + 1.1 * bx + 8 * U * x.abs(), what)


SIZES = [(1,), (7,), (255,), (256,), (16, 17), (0,), (2048,), (3, 1001), (64, 200)]


def make(sizes, pdt, gdt, rng, offset=0):
    """Parameters and gradient buffers; with an offset, as views that no 16-byte boundary holds."""
    def put(shape, std, dt):
        n = math.prod(shape)
        buf = torch.zeros(n + offset, dtype=dt, device=DEV)
        buf[offset:] = torch.from_numpy(rng.standard_normal(n) * std).to(torch.float32).to(dt).to(DEV)
        return buf[offset:].view(shape)

    return [put(s, 0.05, pdt) for s in sizes], [put(s, 1e-3, gdt) for s in sizes]


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt,master", [("bf16", "f32", True), ("bf16", "bf16", False), ("f32", "f32", False),
                                            ("bf16", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", True)])
@pytest.mark.parametrize("offset", [0, 1])
def test_steps(bits, pdt, gdt, master, offset):
    say("adamw", bits, pdt, gdt, master, offset)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    rng = np.random.default_rng(bits + offset)
    params, grads = make(SIZES, dt[pdt], dt[gdt], rng, offset)
    opt = rg.LoraAdamW(params, grads, lr=3e-3, betas=(0.8, 0.95), eps=1e-7, weight_decay=0.1,
                       master=True if master else None, state_bits=bits)
    for k in (1, 2, 3):
        for g in grads:
            g.copy_(torch.from_numpy(rng.standard_normal(g.shape) * 10 ** rng.uniform(-6, 1)).to(DEV))
        before = [((opt.master[i] if master else p).double().cpu().view(-1), grads[i].double().cpu().view(-1),
                   *moments(opt, i)) for i, p in enumerate(params)]
        opt.step(grad_scale=0.5)
        for i, p in enumerate(params):
            if p.numel() == 0:
                continue
            p1, bp, m1, bm, v1, bv = expect(*before[i], opt, k, 0.5)
            if master:
                check(opt.master[i].view(-1), p1, bp, "master")
                assert torch.equal(p, opt.master[i].to(p.dtype))
            else:
                check(p.view(-1), p1, bp + (2.0 ** -8 * (p1.abs() + bp) if pdt == "bf16" else 0), "param")
            if bits == 32:
                check(opt.m[i], m1, bm, "m")
                check(opt.v[i], v1, bv, "v")
            else:
                check_eight(opt.m[i], opt.m_scale[i], m1, bm, "m", False)
                root = v1.sqrt()
                check_eight(opt.v[i], opt.v_scale[i], root, bv / root.clamp_min(1e-300) + U * root, "root", True)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_many_and_large_tensors(bits):
    """More tensors than one table upload takes, and a total that takes the larger share per workgroup."""
    say("adamw many", bits)
    rng = np.random.default_rng(1)
    sizes = [(i % 5 + 1, 37 * i + 1) for i in range(95)] + [(4099, 1001)]
    params, grads = make(sizes, torch.bfloat16, torch.float32, rng)
    opt = rg.LoraAdamW(params, grads, master=True, state_bits=bits)
    before = [(opt.master[i].double().cpu().view(-1), g.double().cpu().view(-1), *moments(opt, i))
              for i, g in enumerate(grads)]
    opt.step()
    for i in range(len(params)):
        p1, bp, m1, bm, v1, bv = expect(*before[i], opt, 1)
        check(opt.master[i].view(-1), p1, bp, "master")
        if bits == 32:
            check(opt.v[i], v1, bv, "v")
        else:
            check_eight(opt.m[i], opt.m_scale[i], m1, bm, "m", False)


@pytest.mark.gpu
def test_codes_are_the_nearest_e4m3():
    """With beta1 = 0 the first moment is the gradient: the codes of every e4m3 value, of the halves between
    neighbours (ties to even), of what lies below the smallest, and of a block's largest value itself."""
    say("adamw codes")
    values = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()  # 0 .. 448
    mid = (values[1:] + values[:-1]) / 2
    near = torch.cat([mid * (1 - 2 ** -20), mid * (1 + 2 ** -20)])
    pool = torch.cat([values, mid, near, -values, -mid])
    blocks = [torch.cat([torch.tensor([448.0]), c, torch.zeros(255 - c.numel())]) for c in pool.split(255)]
    g = torch.cat(blocks).to(DEV)
    opt = rg.LoraAdamW([torch.zeros_like(g)], [g], betas=(0.0, 0.0), state_bits=8)
    opt.step()
    want = g.cpu().to(torch.float8_e4m3fn)
    assert torch.equal(opt.m[0].cpu().view(torch.uint8)[g.cpu() != 0], want.view(torch.uint8)[g.cpu() != 0])
    assert bool((opt.m_scale[0] == 1).all())
    # the root of the second moment is |g|: rounded the same, but never to zero
    root = want.float().abs()
    root[(g.cpu() != 0) & (root == 0)] = 2.0 ** -9
    assert torch.equal(opt.v[0].cpu().float(), root) and bool((opt.v_scale[0] == 1).all())


@pytest.mark.gpu
def test_blocks_of_zeros_and_of_tiny_values():
    say("adamw tiny")
    g = torch.zeros(1024, device=DEV)
    g[256:512] = 1e-35           # below 2^-100
    g[512:768] = 1e-28
    g[512] = 1.0                 # (beside 1.0; the square of 1e-28, 1e-56, is zero in fp32, and so is its root)
    p = torch.ones(1024, device=DEV)
    opt = rg.LoraAdamW([p], [g], lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.0, state_bits=8)
    for _ in range(3):
        opt.step()
    assert bool(torch.isfinite(p).all()) and torch.equal(p[:256], torch.ones_like(p[:256]))
    assert not bool(opt.m_scale[0][:2].any()) and not bool(opt.v[0].float()[:512].any())
    assert not bool(opt.v[0].float()[513:].any())
    assert float((p[513:768] - 1).abs().max()) <= 3.1e-2  # at most lr a step


@pytest.mark.gpu
def test_small_roots_beside_a_large_one_stay_above_zero():
    """A gradient of 1e-15 beside 1.0 (squares and roots within fp32): its root takes the smallest code, its
    first moment is rounded to zero by the second step, and no update is larger than Adam's own."""
    say("adamw roots")
    g = torch.full((256,), 1e-15, device=DEV)
    g[0] = 1.0
    p = torch.ones(256, device=DEV)
    opt = rg.LoraAdamW([p], [g], lr=1e-2, betas=(0.9, 0.99), eps=1e-30, weight_decay=0.0, state_bits=8)
    for _ in range(3):
        opt.step()
        assert bool((opt.v[0].float()[1:] == 2.0 ** -9).all())
        assert bool(torch.isfinite(p).all()) and float((p - 1).abs().max()) <= 3.1e-2


@pytest.mark.gpu
@pytest.mark.parametrize("bits,block", [(32, 1), (8, 256)])
def test_a_gradient_that_is_not_finite_stays_in_its_block(bits, block):
    say("adamw nonfinite", bits)
    rng = np.random.default_rng(3)
    (p,), (g,) = make([(5000,)], torch.float32, torch.float32, rng)
    (q,), (h,) = [p.clone()], [g.clone()]
    h[700], h[3000] = float("inf"), float("nan")
    a, b = rg.LoraAdamW([p], [g], state_bits=bits), rg.LoraAdamW([q], [h], state_bits=bits)
    for _ in range(2):
        a.step(), b.step()
    keep = torch.ones(5000, dtype=torch.bool, device=DEV)
    for i in (700, 3000):
        keep[i // block * block: i // block * block + block] = False
    assert torch.equal(p[keep], q[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_follow_the_schedule(bits):
    """A captured step that reads {lr, step} from the device, replayed with new gradients: the bits of eager
    steps, on buffers whose ends stay untouched."""
    say("adamw graph", bits)
    rng = np.random.default_rng(4)
    sizes = [(300,), (16, 33), (1,)]
    p1, g1 = make(sizes, torch.bfloat16, torch.float32, rng)
    p2 = [p.clone() for p in p1]
    g2 = [g.clone() for g in g1]
    lr_step = torch.tensor([1e-3, 1.0], dtype=torch.float64, device=DEV)
    eager = rg.LoraAdamW(p1, g1, master=True, state_bits=bits)
    graphed = rg.LoraAdamW(p2, g2, master=True, state_bits=bits, lr_step=lr_step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for k in range(1, 5):
        for a, b in zip(g1, g2):
            a.normal_()
            b.copy_(a)
        eager.lr = 1e-3 * k
        lr_step.copy_(torch.tensor([1e-3 * k, float(k)], dtype=torch.float64))
        eager.step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(p1 + eager.master + eager.m + eager.v, p2 + graphed.master + graphed.m + graphed.v):
            assert torch.equal(a.view(torch.uint8) if a.dtype.itemsize == 1 else a,
                               b.view(torch.uint8) if b.dtype.itemsize == 1 else b)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_forward_backward_and_step_together(bits):
    """Two layers of one pool each trained for three steps: every step's outputs, gradients and parameters
    against the 64-bit forms of the same inputs (the forward's of the parameters that the last step left)."""
    say("routed training run", bits)
    T, dims, n, R = 200, [(64, 96), (96, 72)], 3, 16
    ds = [rr.case(T, K, N, n, R, 20 + i, "packed", tscale=False) for i, (K, N) in enumerate(dims)]
    gs = [{k: v.to(DEV) if torch.is_tensor(v) else v for k, v in d.items()} for d in ds]
    for d, g in zip(ds, gs):
        d["ids"] = ds[0]["ids"]
        g["ids"] = gs[0]["ids"]
    params = [g[k] for g in gs for k in ("A", "B")]
    grads = [torch.zeros(p.shape, device=DEV) for p in params]
    opt = rg.LoraAdamW(params, grads, lr=1e-2, master=True, state_bits=bits, weight_decay=0.0)
    target = torch.randn(T, dims[-1][1], device=DEV)

    def layer(i, x):
        g = gs[i]
        return rg.lora_linear_routed(x, g["W"], g["b"], g["A"], g["B"], g["scales"], g["ids"])

    for k in (1, 2, 3):
        h = layer(0, gs[0]["x"])
        y = layer(1, h)
        dy = (y.float() - target).to(torch.bfloat16)
        outs = [(gs[1], h, dy, y)]
        back = rg.lora_linear_routed_backward
        dh, _, _ = back(h, gs[1]["W"], gs[1]["A"], gs[1]["B"], dy, gs[1]["scales"], gs[1]["ids"], dA=grads[2], dB=grads[3])
        _, _, _ = back(gs[0]["x"], gs[0]["W"], gs[0]["A"], gs[0]["B"], dh, gs[0]["scales"], gs[0]["ids"], dA=grads[0],
                       dB=grads[1], want=("dA", "dB"))
        outs.append((gs[0], gs[0]["x"], dh, h))
        for j, (g, x, dout, out) in enumerate(outs):
            d = {kk: v.cpu() if torch.is_tensor(v) else v for kk, v in g.items()}
            d.update(x=x.cpu(), dy=dout.cpu(), token_scale=None, ranks=None)
            rr.check(out, *rr.forward(d), "y")
            (dx, dA, dB), bounds = rr.backward(d)
            rr.check(grads[2 - 2 * j], dA, bounds[1], "dA")
            rr.check(grads[3 - 2 * j], dB, bounds[2], "dB")
            if j == 0:
                rr.check(dh, dx, bounds[0], "dx")
        before = [(w.double().cpu().view(-1), g.double().cpu().view(-1), *moments(opt, i))
                  for i, (w, g) in enumerate(zip(opt.master, grads))]
        opt.step()
        for i, w in enumerate(opt.master):
            p1, bp, *_ = expect(*before[i], opt, k)
            check(w.view(-1), p1, bp, "master")
            assert torch.equal(params[i], w.to(torch.bfloat16))
