"""The AdamW step on the GPU: states bit for bit against NumPy, parameters within their
rounding of fp64."""

import itertools
import math

import numpy as np
import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests import adamw_ref as ref
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def host(t):
    return t.detach().float().cpu().numpy().reshape(-1)


class Problem:
    """A list of tensors on the GPU and what the definition makes of it."""

    def __init__(self, sizes, p="f32", g="f32", bits=32, copy=None, seed=0, shift=0, level=1e-2, fresh=False):
        rng = np.random.default_rng(seed)
        ps, gs = [[k] * len(sizes) if isinstance(k, str) else list(k) for k in (p, g)]

        def new(x, dtype):
            # (shift: a view that starts `shift` elements into its buffer, between others' values)
            buf = torch.full((x.size + 2 * shift,), 3.0, device=dev()).to(dtype)
            buf[shift:shift + x.size] = torch.from_numpy(x).to(dev()).to(dtype)
            return buf[shift:shift + x.size]
        self.bits = bits
        self.p = [new(rng.standard_normal(n) * 0.1, TYPES[k]) for n, k in zip(sizes, ps)]
        self.g = [new(rng.standard_normal(n) * level * np.exp(rng.uniform(-6, 2, n)), TYPES[k])
                  for n, k in zip(sizes, gs)]
        self.copies = None if copy is None else [
            None if k is None else new(np.zeros(n), TYPES[k]) for n, k in zip(sizes, itertools.cycle(copy))]
        m = [rng.standard_normal(n) * level * np.exp(rng.uniform(-8, 0, n)) * (not fresh) for n in sizes]
        r = [level * np.exp(rng.uniform(-9, 1, n)) * (not fresh) for n in sizes]
        if bits == 32:
            self.m, self.v = [new(x, torch.float32) for x in m], [new(x * x, torch.float32) for x in r]
            self.ms = self.vs = None
        else:
            both = [[ref.encode(x.astype(np.float32), np.zeros(len(x)), root) for x in xs]
                    for xs, root in ((m, False), (r, True))]
            (self.m, self.ms), (self.v, self.vs) = [
                ([new(c.astype(np.float64), torch.uint8) for c, _ in b], [new(s.astype(np.float64), torch.uint8)
                                                                          for _, s in b]) for b in both]
        self.list = fp8g.adamw_tensors(self.p, self.g, self.m, self.v, copies=self.copies, m_scales=self.ms,
                                       v_scales=self.vs)

    def run(self, step=3, lr=1e-2, b1=0.9, b2=0.95, eps=1e-8, decay=0.1, max_norm=None, seed=7, dev_args=False,
            lr_host=None):
        """One step on the GPU, checked."""
        before = [[host(t) for t in ts] for ts in (self.p, self.g)]
        lr_used = float(np.float32(lr)) if dev_args else lr
        kw, clip = {}, None
        if max_norm is not None:
            sumsq = sum(float((g.double() ** 2).sum()) for g in self.g)
            norm = torch.full((1,), -1.0, device=dev())
            kw = dict(sumsq=torch.tensor([sumsq], dtype=torch.float64, device=dev()), max_norm=max_norm, norm=norm)
            clip = ref.factor(sumsq, max_norm)
        want = []
        for i, (p, g) in enumerate(zip(*before)):
            if self.bits == 32:
                m, v = host(self.m[i]), host(self.v[i])
            else:
                m = ref.decode(self.m[i].cpu().numpy(), self.ms[i].cpu().numpy()).astype(np.float32)
                r = ref.decode(self.v[i].cpu().numpy(), self.vs[i].cpu().numpy()).astype(np.float32)
                with np.errstate(over="ignore"):
                    v = r * r
            m, v, r = ref.states(g, m, v, clip, b1, b2)
            want.append((m, v, r, *ref.params(p, m, r, step, lr_used, b1, b2, eps, decay)))
        s = torch.tensor([step], dtype=torch.int64, device=dev()) if dev_args else step
        rate = torch.tensor([lr], device=dev()) if dev_args else lr
        fp8g.adamw_step(self.list, s, rate, beta1=b1, beta2=b2, eps=eps, weight_decay=decay, seed=seed, **kw)
        torch.cuda.synchronize()
        if max_norm is not None:
            assert abs(float(norm) - math.sqrt(sumsq)) <= 2.0 ** -23 * math.sqrt(sumsq)
        for i, (m, v, r, p, u) in enumerate(want):
            assert np.array_equal(host(self.g[i]), before[1][i])
            if self.bits == 32:
                assert np.array_equal(host(self.m[i]), m) and np.array_equal(host(self.v[i]), v), i
            else:
                bits = ref.random_bits(seed, step, i, len(m))
                for codes, scales, x, cut, root in ((self.m, self.ms, m, bits & np.uint64(0xFFFF), False),
                                                    (self.v, self.vs, r, bits >> np.uint64(16), True)):
                    c, sc = ref.encode(x, cut.astype(np.float64), root)
                    assert np.array_equal(scales[i].cpu().numpy(), sc), i
                    assert np.array_equal(codes[i].cpu().numpy(), c), i
            # p (1 - lr wd): the factor's and the product's rounding; the update: size, inv, r inv,
            # + eps, the reciprocal (two half steps), two products; their difference; the type's
            got, e = host(self.p[i]).astype(np.float64), 2.0 ** -24
            tol = (np.abs(p) + u) * 2 * e + u * 8 * e + np.abs(p) * e
            for t, x in [(self.p[i], got)] + ([] if self.copies is None or self.copies[i] is None else [
                    (self.copies[i], host(self.copies[i]).astype(np.float64))]):
                fi = torch.finfo(t.dtype)
                with np.errstate(invalid="ignore"):
                    assert (np.abs(x - p) <= tol + (np.abs(p) + tol) * fi.eps / 2 + fi.smallest_normal * fi.eps / 2).all(), i


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[1], [0], [], [3, 0, 4, 5, 1], [127, 128, 129], [2047], [2048, 2049], [8192 + 7],
                                   [40000, 1, 300], [7] * 60, [130] * 250])
@pytest.mark.parametrize("p,g", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_sizes(sizes, bits, p, g):
    q = Problem(sizes, p, g, bits, seed=len(sizes))
    q.run()
    q.run(step=4, max_norm=0.05)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p,g", list(itertools.product(TYPES, TYPES)))
def test_types(p, g, bits):
    Problem([5000, 129], p, g, bits, copy=["bf16", "f16"]).run(max_norm=0.1)


@pytest.mark.parametrize("bits", [32, 8])
def test_mixed_list_with_some_copies(bits):
    kinds = [a for a, _ in itertools.product(TYPES, range(7))]
    sizes = [1 + 97 * i % 700 for i in range(len(kinds))]
    q = Problem(sizes, kinds, kinds[::-1], bits, copy=["bf16", None, "f16"])
    for step in (1, 2, 3):
        q.run(step=step, max_norm=0.2, seed=step)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [1, 2, 3, 4, 8])
def test_unaligned_views(bits, shift):
    q = Problem([1000, 129, 4096], "f32", "bf16", bits, copy=["bf16"], shift=shift)
    q.run()
    for ts in (q.p, q.g, q.m, q.v, q.copies):
        for t in ts:
            whole = torch.tensor([], dtype=t.dtype, device=dev()).set_(t.untyped_storage())
            assert (whole[:shift] == 3).all() and (whole[-shift:] == 3).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kw", [dict(step=1, b1=0.0, b2=0.0), dict(step=1, b1=0.9, b2=0.999), dict(step=10 ** 6),
                                dict(decay=0.0, eps=1e-3), dict(lr=0.0), dict(eps=0.0), dict(max_norm=1e9),
                                dict(max_norm=1e-6), dict(dev_args=True, max_norm=0.3), dict(dev_args=True, step=100000)])
def test_hyperparameters(bits, kw):
    Problem([3000], bits=bits).run(**kw)


def test_fresh_8_bit_states_and_many_steps():
    q = Problem([1500, 70], "f32", "bf16", 8, copy=["bf16"], fresh=True)
    for step in range(1, 9):
        q.run(step=step, seed=step * 1000003)
        for g in q.g:
            g.normal_(std=0.01)


@pytest.mark.parametrize("bits", [32, 8])
def test_large_list_takes_large_chunks(bits):
    """More than 2048 chunks of 8192 elements, and every element's own result."""
    n = 2048 * 8192 + 12345
    gen = torch.Generator(device=dev()).manual_seed(1)
    p = torch.randn(n, device=dev(), generator=gen)
    g = torch.randn(n, device=dev(), generator=gen)
    want = None
    for cut in (n, n // 3):                        # the same elements as one tensor and as the first of two
        pp = p.clone()
        state = ([torch.zeros(n, dtype=torch.uint8 if bits == 8 else torch.float32, device=dev()) for _ in range(2)])
        sc = [torch.zeros(-(-n // 128), dtype=torch.uint8, device=dev()) for _ in range(2)] if bits == 8 else None
        cut = cut // 2048 * 2048 if cut < n else n

        def split(t, unit=1):
            c = -(-cut // unit)
            return [t[:c]] + ([t[c:]] if cut < n else [])
        kw = dict(m_scales=split(sc[0], 128), v_scales=split(sc[1], 128)) if bits == 8 else {}
        lst = fp8g.adamw_tensors(split(pp), split(g), split(state[0]), split(state[1]), **kw)
        fp8g.adamw_step(lst, 1, 1e-2, weight_decay=0.0)
        if want is None:
            want = pp
    torch.cuda.synchronize()
    assert torch.equal(want, pp)
    # from fresh states the first step moves by lr g / (|g| + eps); ten roundings of that, one of p
    ref_p = p.double() - 1e-2 * g.double() / (g.double().abs() + 1e-8)
    assert bool(((want.double() - ref_p).abs() <= 2.0 ** -24 * ref_p.abs() + 1e-2 * 10 * 2.0 ** -24).all())


def test_rounding_of_8_bit_states_has_no_drift():
    """Without gradients sqrt(v) shrinks by sqrt(b2) a step, 0.05%: rounded to the nearest
    code it would stay; rounded as defined its mean follows, within five deviations of the
    mean of 65536 elements (a step's variance is at most a quarter of a code's step squared)."""
    n, steps, b2 = 65536, 300, 0.999
    p, g = torch.zeros(n, device=dev()), torch.zeros(n, device=dev())
    m = torch.zeros(n, dtype=torch.uint8, device=dev())
    code, scale = ref.encode(np.full(n, 300.0, np.float32), np.zeros(n), True)
    v, vs = torch.from_numpy(code).to(dev()), torch.from_numpy(scale).to(dev())
    lst = fp8g.adamw_tensors([p], [g], [m], [v], m_scales=[torch.zeros_like(vs)], v_scales=[vs])
    start = ref.decode(code, scale).mean()
    for step in range(1, steps + 1):
        fp8g.adamw_step(lst, step, 0.0, beta2=b2, weight_decay=0.0, seed=step)
    got = ref.decode(v.cpu().numpy(), vs.cpu().numpy()).mean()
    unit = 32.0                                    # of codes from 256 to 448
    assert abs(got - start * b2 ** (steps / 2)) < 5 * unit * math.sqrt(steps / 4 / n) + steps * unit * 2.0 ** -16


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_sum_that_is_not_finite_leaves_the_step_out(bits, bad):
    q = Problem([500, 3], "bf16", "f32", bits, copy=["f16"])
    held = [ts for ts in (q.p, q.g, q.m, q.v, q.ms, q.vs, q.copies) if ts is not None]
    before = [[t.clone() for t in ts] for ts in held]
    norm = torch.zeros(1, device=dev())
    fp8g.adamw_step(q.list, 1, 0.1, sumsq=torch.tensor([bad], dtype=torch.float64, device=dev()), max_norm=1.0,
                    norm=norm)
    assert all(torch.equal(a, b) for x, y in zip(held, before) for a, b in zip(x, y))
    assert str(float(norm)) == str(bad)


@pytest.mark.parametrize("bits", [32, 8])
def test_elements_that_are_not_finite_stay_alone(bits):
    q = Problem([400], bits=bits)
    clean = Problem([400], bits=bits)
    q.g[0][5], q.g[0][200], q.g[0][201] = float("nan"), float("inf"), float("-inf")
    for x in (q, clean):
        fp8g.adamw_step(x.list, 2, 1e-2)
    torch.cuda.synchronize()
    odd = np.zeros(400, bool)
    odd[[5, 200, 201]] = True
    assert not np.isfinite(host(q.p[0])[odd]).any()
    # (neighbours in the block of 128 keep their parameters; a block's scale goes by what is finite)
    assert np.array_equal(host(q.p[0])[~odd], host(clean.p[0])[~odd])
    if bits == 8:
        assert (q.m[0].cpu().numpy()[odd] & 127 == 127).all() and (q.v[0].cpu().numpy()[odd] == 127).all()
        assert (q.m[0].cpu().numpy()[~odd] & 127 != 127).all()
    else:
        assert not np.isfinite(host(q.m[0])[odd]).any() and np.isfinite(host(q.m[0])[~odd]).all()


def test_same_call_same_bits():
    a, b = (Problem([5000, 77], "f32", "bf16", 8, copy=["bf16"]) for _ in range(2))
    for q in (a, b):
        fp8g.adamw_step(q.list, 9, 1e-3, seed=123)
    assert all(torch.equal(x, y) for u, v in ((a.p, b.p), (a.m, b.m), (a.v, b.v), (a.ms, b.ms), (a.copies, b.copies))
               for x, y in zip(u, v))


def test_clipping_of_grad_clip():
    """The step with a sum of squares is grad_clip's gradients stepped without one."""
    a, b = (Problem([3000, 50], level=1.0) for _ in range(2))
    ws = torch.empty(max(8, fp8g.grad_norm_sq_workspace_size(a.g)), dtype=torch.uint8, device=dev())
    sumsq = torch.empty(1, dtype=torch.float64, device=dev())
    norm, norm2 = torch.empty(1, device=dev()), torch.empty(1, device=dev())
    fp8g.grad_norm_sq(a.g, sumsq, ws)
    fp8g.adamw_step(a.list, 2, 1e-2, sumsq=sumsq, max_norm=1.0, norm=norm)
    fp8g.grad_clip(b.g, b.g, sumsq, 1.0, norm2)
    fp8g.adamw_step(b.list, 2, 1e-2)
    assert torch.equal(norm, norm2) and float(norm) > 1.0
    assert all(torch.equal(x, y) for u, v in ((a.p, b.p), (a.m, b.m), (a.v, b.v)) for x, y in zip(u, v))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_and_replayed(bits):
    """A graph of norm and step: every replay takes the step's number and rate anew."""
    a, b = (Problem([2500, 130], "f32", "bf16", bits, copy=["bf16"]) for _ in range(2))
    step = torch.zeros(1, dtype=torch.int64, device=dev())
    lr = torch.zeros(1, device=dev())
    ws = torch.empty(max(8, fp8g.grad_norm_sq_workspace_size(a.g)), dtype=torch.uint8, device=dev())
    sumsq = torch.empty(1, dtype=torch.float64, device=dev())

    def call(q, s, rate):
        fp8g.grad_norm_sq(q.g, sumsq, ws)
        fp8g.adamw_step(q.list, s, rate, sumsq=sumsq, max_norm=0.1, seed=5)
    call(Problem([10], bits=bits), step, lr)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a, step, lr)
    gen = torch.Generator(device=dev()).manual_seed(3)
    for i in range(1, 5):
        step.fill_(i)
        lr.fill_(1e-2 / i)
        for x, y in zip(a.g, b.g):
            x.normal_(std=0.01 * i, generator=gen)
            y.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        call(b, i, float(lr))
        torch.cuda.synchronize()
        for u, v in ((a.p, b.p), (a.m, b.m), (a.v, b.v), (a.copies, b.copies)):
            assert all(torch.equal(x, y) for x, y in zip(u, v)), i


def test_another_stream():
    a, b = (Problem([3000]) for _ in range(2))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fp8g.adamw_step(a.list, 1, 1e-2)
    fp8g.adamw_step(b.list, 1, 1e-2, stream=side)
    side.synchronize()
    assert torch.equal(a.p[0], b.p[0]) and torch.equal(a.v[0], b.v[0])


def test_list_keeps_the_memory():
    q = Problem([1000])
    want = Problem([1000])
    lst = q.list
    old = q.p[0].data_ptr()
    del q
    torch.cuda.empty_cache()
    other = torch.full((1000,), 9.0, device=dev())
    fp8g.adamw_step(lst, 1, 1e-2)
    fp8g.adamw_step(want.list, 1, 1e-2)
    assert other.data_ptr() != old and (other == 9).all()
    assert torch.equal(torch.empty(0, device=dev()).set_(lst.held[0][0]), want.p[0])


def test_parameters_that_require_gradients():
    p = torch.nn.Parameter(torch.ones(64, device=dev()))
    (p * 2).sum().backward()
    m, v = torch.zeros(64, device=dev()), torch.zeros(64, device=dev())
    fp8g.adamw_step(fp8g.adamw_tensors([p], [p.grad], [m], [v]), 1, 0.5, weight_decay=0.0)
    assert torch.allclose(p.detach(), torch.full((64,), 0.5, device=dev()), rtol=0, atol=1e-6)


def test_binding_refuses():
    def z(n=8, dtype=torch.float32):
        return torch.zeros(n, dtype=dtype, device=dev())
    u8 = torch.uint8
    ok = dict(params=[z()], grads=[z()], exp_avgs=[z()], exp_avg_sqs=[z()])
    fp8g.adamw_tensors(**ok)
    eight = dict(ok, exp_avgs=[z(8, u8)], exp_avg_sqs=[z(8, u8)], m_scales=[z(1, u8)], v_scales=[z(1, u8)])
    fp8g.adamw_tensors(**eight)
    same = z()
    for bad in [dict(ok, grads=[z(7)]), dict(ok, grads=[]), dict(ok, params=[z().double()]), dict(ok, exp_avgs=[z(8, u8)]),
                dict(ok, exp_avg_sqs=[z().bfloat16()]), dict(ok, params=[torch.zeros(8)]), dict(ok, grads=[None]),
                dict(ok, params=[z(16)[::2]]), dict(ok, copies=[z()]), dict(ok, copies=[z(7).bfloat16()]),
                dict(eight, v_scales=None), dict(eight, m_scales=[z(2, u8)]), dict(eight, exp_avgs=[z()]),
                dict(ok, exp_avgs=[same], exp_avg_sqs=[same]), dict(ok, params=[same], grads=[same]),
                dict(params=[same, same], grads=[z(), z()], exp_avgs=[z(), z()], exp_avg_sqs=[z(), z()])]:
        with pytest.raises(ValueError):
            fp8g.adamw_tensors(**bad)
    lst = fp8g.adamw_tensors(**ok)
    for args, kw in [((0, 0.1), {}), ((1, float("nan")), {}), ((1, 0.1), dict(beta1=1.0)), ((1, 0.1), dict(beta2=-0.1)),
                     ((1, 0.1), dict(eps=-1.0)), ((1, 0.1), dict(norm=z(1))),
                     ((1, 0.1), dict(sumsq=z(1, torch.float64), max_norm=0.0))]:
        with pytest.raises(fp8g.Fp8GemmError):
            fp8g.adamw_step(lst, *args, **kw)
    for args, kw in [((z(1), 0.1), {}), ((1, z(1).double()), {}), ((z(2, torch.int64), 0.1), {}),
                     ((1, 0.1), dict(sumsq=z(1), max_norm=1.0))]:
        with pytest.raises(ValueError):
            fp8g.adamw_step(lst, *args, **kw)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("n", [52, 53, 64, 65, 129, 1000, 4097, 9000])
def test_long_lists(n, bits):
    """Lists that lie in device memory, empty tensors among them and at both ends."""
    rng = np.random.default_rng(n)
    sizes = list(rng.integers(0, 40, n))
    for i in rng.integers(0, n, 3):
        sizes[i] = 4500
    sizes[0] = sizes[-1] = 0
    q = Problem([int(k) for k in sizes], "f32", "bf16", bits, copy=["bf16"], seed=n)
    assert (q.list.table is not None) == (n > 52)
    q.run()
    q.run(step=4, max_norm=0.05)


@pytest.mark.parametrize("bits", [32, 8])
def test_long_list_by_value_and_by_table(bits):
    """A captured step takes the list by value, whatever becomes of the list's table: the same bits."""
    sizes = [1 + 37 * i % 400 for i in range(130)]
    a, b = (Problem(sizes, "bf16", "f32", bits, seed=3) for _ in range(2))
    lr, step = torch.full((1,), 1e-2, device=dev()), torch.ones(1, dtype=torch.int64, device=dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fp8g.adamw_step(a.list, step, lr, seed=5)
    table = a.list.table
    a.list = None
    table.fill_(0xFF)
    torch.cuda.synchronize()
    for t in (1, 2, 3):
        step.fill_(t)
        graph.replay()
        fp8g.adamw_step(b.list, t, 1e-2, seed=5)
        torch.cuda.synchronize()
        for x, y in zip([*a.p, *a.m, *a.v], [*b.p, *b.m, *b.v]):
            assert torch.equal(x, y)


def test_long_list_dropped_after_a_step_on_another_stream():
    sizes = [3000] * 200
    a, b = (Problem(sizes, seed=4) for _ in range(2))
    fp8g.adamw_step(b.list, 1, 1e-2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x = torch.randn(4096, 4096, device=dev())
        for _ in range(20):
            x = x @ x * 1e-4
        fp8g.adamw_step(a.list, 1, 1e-2)
    size = a.list.table.numel()
    a.list = None
    junk = [torch.full((size,), 0xFF, dtype=torch.uint8, device=dev()) for _ in range(8)]
    torch.cuda.synchronize()
    assert len(junk) == 8 and all(torch.equal(x, y) for x, y in zip(a.p + a.m, b.p + b.m))


def test_long_list_made_on_another_stream():
    """The list's table is there for a step on any stream, the default one too."""
    side = torch.cuda.Stream()
    a, b = (Problem([900] * 60, seed=6) for _ in range(2))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        a.list = fp8g.adamw_tensors(a.p, a.g, a.m, a.v)
    fp8g.adamw_step(a.list, 1, 1e-2)
    a.list = None
    fp8g.adamw_step(b.list, 1, 1e-2, stream=side)
    b.list = None
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.p + a.m, b.p + b.m))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_of_more_than_32_bits_elements(bits):
    """Elements past 2^32 step as a short tensor's do (parameters: the states' rounding goes by the
    element's number)."""
    n, tail = (1 << 32) + 5000, 4999
    kind = torch.bfloat16
    gen = torch.Generator(dev()).manual_seed(2)
    p, g = torch.zeros(n, device=dev(), dtype=kind), torch.zeros(n, device=dev(), dtype=kind)
    p[-tail:].normal_(generator=gen)
    g[-tail:].normal_(generator=gen)
    p[:5], g[:5] = p[-5:], g[-5:]
    state = torch.uint8 if bits == 8 else torch.float32
    zeros = lambda k, t: torch.zeros(k, device=dev(), dtype=t)  # noqa: E731
    scales = lambda k: dict(m_scales=[zeros(-(-k // 128), torch.uint8)],  # noqa: E731
                            v_scales=[zeros(-(-k // 128), torch.uint8)]) if bits == 8 else {}
    small = [p[-tail:].clone(), g[-tail:].clone()]
    big_m, big_v, m, v = zeros(n, state), zeros(n, state), zeros(tail, state), zeros(tail, state)
    fp8g.adamw_step(fp8g.adamw_tensors([p], [g], [big_m], [big_v], **scales(n)), 1, 1e-2)
    fp8g.adamw_step(fp8g.adamw_tensors([small[0]], [small[1]], [m], [v], **scales(tail)), 1, 1e-2)
    assert torch.equal(p[-tail:], small[0]) and torch.equal(p[:5], small[0][-5:])
    assert not p[5:-tail].any() and big_m[-tail:].any()
    if bits == 32:
        assert torch.equal(big_m[-tail:], m) and torch.equal(big_v[-tail:], v) and not big_m[5:-tail].any()
