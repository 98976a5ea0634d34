"""The AdamW step on the GPU where its documentation allows what the other tests do not do."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests import adamw_ref as ref
from tests.gpu_util import dev
from tests.test_gpu_adamw import Problem

pytestmark = pytest.mark.gpu


def eight_bit(n, m, r, m_byte, r_byte, seed=0):
    """Parameters, gradients and 8-bit states of one tensor: codes m and r (a number or an array), every
    scale m_byte and r_byte."""
    rng = np.random.default_rng(seed)

    def fill(k, x):
        return torch.from_numpy(np.broadcast_to(np.asarray(x, np.uint8), k).copy()).to(dev())
    p, g = [torch.from_numpy(rng.standard_normal(n).astype(np.float32) * k).to(dev()) for k in (0.1, 1e-2)]
    blocks = -(-n // 128)
    return p, g, fill(n, m), fill(n, r), fill(blocks, m_byte), fill(blocks, r_byte)


def step_one(p, g, m, r, ms, rs, step=1):
    lst = fp8g.adamw_tensors([p], [g], [m], [r], m_scales=[ms], v_scales=[rs])
    fp8g.adamw_step(lst, step, 1e-2, seed=3)
    torch.cuda.synchronize()


@pytest.mark.parametrize("n", [5, 128, 5000])
@pytest.mark.parametrize("m_byte,r_byte", [(255, 255), (255, 0), (0, 255), (254, 254), (1, 254)])
def test_codes_of_zeros_are_a_fresh_state_whatever_the_scales(n, m_byte, r_byte):
    want, got = eight_bit(n, 0, 0, 0, 0), eight_bit(n, 0, 0, m_byte, r_byte)
    step_one(*want)
    step_one(*got)
    assert bool(torch.isfinite(got[0]).all())
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_zeros_of_either_sign_among_unset_scales():
    """Some blocks' scales unset (every byte among them), m's codes zeros of both signs."""
    n = 256 * 128 + 37
    every = np.arange(257) % 256
    sign = np.random.default_rng(1).choice([0, 128], n)
    want, got = eight_bit(n, sign, 0, 0, 0), eight_bit(n, sign, 0, every, every[::-1])
    step_one(*want)
    step_one(*got)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_scale_byte_255_of_other_codes_is_nan():
    """As e8m0 says; codes of zeros beside them stay zeros, the other blocks are as without it."""
    n = 128 * 3
    codes = np.full(n, 40)
    codes[128:160] = 0
    scale = np.array([127, 255, 127])
    want, got = eight_bit(n, codes, codes, 127, 127), eight_bit(n, codes, codes, scale, scale)
    step_one(*want)
    step_one(*got)
    odd = np.zeros(n, bool)
    odd[160:256] = True
    p, q = want[0].cpu().numpy(), got[0].cpu().numpy()
    assert np.isnan(q[odd]).all() and np.array_equal(p[~odd], q[~odd])
    m, r = [t.cpu().numpy() for t in got[2:4]]
    assert (m[odd] & 127 == 127).all() and (r[odd] == 127).all()
    dec = ref.decode(m, got[4].cpu().numpy())
    assert np.isfinite(dec[~odd]).all()


def long_list(seed=0, n=60):
    """More tensors than one launch takes by value: parameters and the list."""
    gen = torch.Generator(device=dev()).manual_seed(seed)
    ps, gs = [[torch.randn(300 + i, device=dev(), generator=gen) for i in range(n)] for _ in range(2)]
    ms, vs = [[torch.zeros_like(p) for p in ps] for _ in range(2)]
    return ps, fp8g.adamw_tensors(ps, gs, ms, vs)


class Spy:
    """A list's table that writes down the streams it is recorded on."""

    def __init__(self, lst):
        self.table, self.on = lst.table, []
        lst.table = self

    def record_stream(self, stream):
        self.on.append(stream.cuda_stream)
        self.table.record_stream(stream)

    def data_ptr(self):
        return self.table.data_ptr()


class Handle:
    """A stream of someone else's."""

    def __init__(self, handle):
        self.cuda_stream = handle


def test_the_table_is_recorded_on_the_stream_of_the_step():
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    assert side.cuda_stream != 0 and other.cuda_stream != side.cuda_stream
    default = torch.cuda.default_stream().cuda_stream
    wants = []
    for made_on, kw, want in [(side, {}, [default]), (side, dict(stream=0), [default]),
                              (side, dict(stream=torch.cuda.default_stream()), [default]),
                              (side, dict(stream=other), [other.cuda_stream]), (side, dict(stream=side), []),
                              (side, dict(stream=side.cuda_stream), []), (None, {}, []), (None, dict(stream=0), []),
                              (None, dict(stream=side), [side.cuda_stream]),
                              # (handles that may be anyone's: the list goes by value)
                              (None, dict(stream=side.cuda_stream), []),
                              (None, dict(stream=torch.cuda.ExternalStream(side.cuda_stream)), []),
                              (None, dict(stream=Handle(side.cuda_stream)), [])]:
        want_p, ref_list = long_list()
        fp8g.adamw_step(ref_list, 1, 1e-2)
        torch.cuda.synchronize()
        with torch.cuda.stream(made_on):
            ps, lst = long_list()
        torch.cuda.synchronize()
        spy = Spy(lst)
        for step in (1, 2):                            # (once for each stream)
            fp8g.adamw_step(lst, step, 1e-2, **kw)
            if step == 1:
                torch.cuda.synchronize()
                wants.append(all(torch.equal(a, b) for a, b in zip(want_p, ps)))
        assert spy.on == want, kw
        torch.cuda.synchronize()
    assert all(wants)


def test_a_dropped_list_keeps_its_table_until_the_default_stream_is_done():
    """Made on a side stream, stepped on the default one: no allocation of the side stream gets the table's
    place while the step waits."""
    side = torch.cuda.Stream()
    want, ref_list = long_list()
    fp8g.adamw_step(ref_list, 1, 1e-2)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        ps, lst = long_list()
    torch.cuda.synchronize()
    x = torch.randn(4096, 4096, device=dev())
    for _ in range(60):
        x = x @ x * 1e-4
    fp8g.adamw_step(lst, 1, 1e-2)
    at, size = lst.table.data_ptr(), lst.table.numel()
    lst = None
    with torch.cuda.stream(side):
        new = [torch.empty(size, dtype=torch.uint8, device=dev()) for _ in range(8)]
    busy = not torch.cuda.default_stream().query()
    assert not busy or at not in [t.data_ptr() for t in new]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, ps))


@pytest.mark.parametrize("kinds", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("n", [3, 1000])
def test_subnormal_squares_without_eps(n, kinds):
    """eps = 0 and v down to the smallest subnormal: the step is m / sqrt(v), about lr, and finite."""
    types = {"f32": torch.float32, "bf16": torch.bfloat16}
    rng = np.random.default_rng(n)
    top = np.exp(np.linspace(np.log(1e-21), np.log(1e-17), n)) * rng.choice([-1, 1], n)
    p = torch.zeros(n, dtype=types[kinds[0]], device=dev())
    g = torch.from_numpy(top).float().to(dev()).to(types[kinds[1]])
    m, v = [torch.zeros(n, device=dev()) for _ in range(2)]
    b1, b2, lr = 0.9, 0.999, 1e-2
    fp8g.adamw_step(fp8g.adamw_tensors([p], [g], [m], [v]), 1, lr, beta1=b1, beta2=b2, eps=0.0, weight_decay=0.0)
    wm, wv, _ = ref.states(g.float().cpu().numpy(), np.zeros(n, np.float32), np.zeros(n, np.float32), None, b1, b2)
    assert np.array_equal(m.cpu().numpy(), wm) and np.array_equal(v.cpu().numpy(), wv)
    assert (wv > 0).all() and (wv < 2.0 ** -126).any()
    want = -lr / (1 - b1) * wm.astype(np.float64) / (np.sqrt(wv.astype(np.float64)) / np.sqrt(1 - b2))
    # half steps of fp32: lr's factor, the root's factor, the root 2, their product, the reciprocal 2, two
    # products; the difference with 0 is exact; then the type's
    tol = 8 * 2.0 ** -24 * np.abs(want)
    tol += torch.finfo(p.dtype).eps / 2 * (np.abs(want) + tol)
    assert (np.abs(p.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-37, 1e-38, 1e-40, 1e-45, 1e-60, 1e-300])
def test_an_eps_below_fp32s_normal_numbers(eps, bits):
    """Where gradient and states are 0 nothing moves, however small eps is; elsewhere it makes no difference."""
    n = 300
    p = torch.linspace(-1, 1, n, device=dev())
    g = torch.zeros(n, device=dev())
    g[::3] = 1e-3
    start = p.clone()

    def states():
        if bits == 32:
            return [[torch.zeros(n, device=dev())] for _ in range(2)], {}
        return ([[torch.zeros(n, dtype=torch.uint8, device=dev())] for _ in range(2)],
                {k: [torch.zeros(3, dtype=torch.uint8, device=dev())] for k in ("m_scales", "v_scales")})
    st, sc = states()
    fp8g.adamw_step(fp8g.adamw_tensors([p], [g], *st, **sc), 1, 1e-2, eps=eps, weight_decay=0.0)
    q, (st, sc) = start.clone(), states()
    fp8g.adamw_step(fp8g.adamw_tensors([q], [g], *st, **sc), 1, 1e-2, eps=1e-30, weight_decay=0.0)
    torch.cuda.synchronize()
    assert torch.equal(p, q)
    assert torch.equal(p[1::3], start[1::3]) and bool((p[::3] < start[::3]).all())


def test_overlapping_tensors_are_refused():
    def z(n, dtype=torch.float32):
        return torch.zeros(n, dtype=dtype, device=dev())
    flat, codes = z(1000), z(1000, torch.uint8)

    def lst(**kw):
        base = dict(params=[z(100), z(100)], grads=[z(100), z(100)], exp_avgs=[z(100), z(100)],
                    exp_avg_sqs=[z(100), z(100)])
        return fp8g.adamw_tensors(**dict(base, **kw))
    lst(params=[flat[:100], flat[100:200]], grads=[flat[200:300]] * 2, exp_avgs=[flat[300:400], flat[400:500]])
    # (shared gradients, empty tensors anywhere)
    lst(params=[flat[:100], flat[50:50]], grads=[z(100), flat[20:20]], exp_avgs=[z(100), z(0)], exp_avg_sqs=[z(100), z(0)])
    eight = dict(exp_avgs=[codes[:100], codes[100:200]], exp_avg_sqs=[codes[200:300], codes[300:400]],
                 m_scales=[codes[400:401], codes[401:402]], v_scales=[codes[402:403], codes[403:404]])
    lst(**eight)
    for bad in [dict(params=[flat[:100], flat[64:164]]), dict(params=[flat[:100], z(100)], exp_avgs=[flat[99:199], z(100)]),
                dict(params=[flat[64:164], z(100)], grads=[flat[:100], z(100)]),
                dict(params=[flat[64:164], z(100)], grads=[z(100), flat[100:200]]),
                dict(params=[flat[:100], z(100)], copies=[None, flat.view(torch.bfloat16)[199:299]]),
                dict(eight, v_scales=[codes[402:403], codes[399:400]]), dict(eight, m_scales=[codes[150:151], codes[401:402]]),
                dict(eight, grads=[codes[:400].view(torch.float32), z(100)])]:
        with pytest.raises(ValueError, match="overlaps"):
            lst(**bad)
    lst(params=[flat[:100], z(100)], copies=[None, flat.view(torch.bfloat16)[200:300]])


# 8-bit states, 2^24 elements and more, most of them of 16-bit parameters: chunks of 8192 elements rather than 2048
LARGE = 1 << 24


@pytest.mark.parametrize("sizes,p,copy", [
    ([LARGE + 4099], "bf16", None),
    ([70000, LARGE + 8192 * 3 + 1, 1, 8192, 8193, 0, 16384], "f16", None),
    # (a long list, fp32 parameters and copies among it)
    ([300000 + 137 * i for i in range(60)], ["f32" if i % 7 == 3 else "bf16" for i in range(60)], ["f16", None, "bf16"]),
])
def test_large_chunks_by_the_definition(sizes, p, copy):
    """Every parameter, code and scale byte against NumPy."""
    kinds = [p] * len(sizes) if isinstance(p, str) else p
    assert sum(sizes) >= LARGE and 2 * sum(n for n, k in zip(sizes, kinds) if k != "f32") > sum(sizes)
    q = Problem(sizes, p, "bf16", 8, copy=copy, seed=len(sizes))
    assert (q.list.table is not None) == (len(sizes) > 52)
    q.run(step=5, max_norm=30.0)


def test_large_chunks_and_small_ones_give_the_same_bits():
    """The same tensor first in a list of 16-bit parameters and in one that is mostly fp32."""
    n = LARGE + 12345
    gen = torch.Generator(device=dev()).manual_seed(4)
    p0 = torch.randn(n, device=dev(), generator=gen).bfloat16()
    g = torch.randn(n, device=dev(), generator=gen)
    results = []
    for more in (0, n + 1):
        ps = [p0.clone()] + [torch.zeros(more, device=dev())] * (more > 0)
        gs = [g] + [torch.zeros(more, device=dev())] * (more > 0)

        def state(k=1):
            return [torch.zeros(-(-p.numel() // k), dtype=torch.uint8, device=dev()) for p in ps]
        st = [state(), state(), state(128), state(128)]
        lst = fp8g.adamw_tensors(ps, gs, *st[:2], m_scales=st[2], v_scales=st[3])
        for step in (1, 2):
            fp8g.adamw_step(lst, step, 1e-2, seed=9)
        results.append([ps[0]] + [t[0] for t in st])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_large_chunks_by_table_and_by_value():
    """A long list of large chunks in one launch, and captured in launches of 52 tensors: the same bits."""
    sizes = [300000 + 31 * i for i in range(60)]
    kinds = ["f32" if i % 5 == 2 else "f16" for i in range(60)]
    a, b = (Problem(sizes, kinds, "f32", 8, copy=["bf16", None], seed=2) for _ in range(2))
    assert sum(sizes) >= LARGE and a.list.table is not None
    step, lr = torch.ones(1, dtype=torch.int64, device=dev()), torch.full((1,), 1e-2, device=dev())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8g.adamw_step(a.list, step, lr, seed=5)
    for t in (1, 2, 3):
        step.fill_(t)
        graph.replay()
        torch.cuda.synchronize()
        fp8g.adamw_step(b.list, t, float(lr), seed=5)
        torch.cuda.synchronize()
        for u, v in ((a.p, b.p), (a.m, b.m), (a.v, b.v), (a.ms, b.ms), (a.vs, b.vs)):
            assert all(torch.equal(x, y) for x, y in zip(u, v)), t
        assert all(x is None or torch.equal(x, y) for x, y in zip(a.copies, b.copies))
