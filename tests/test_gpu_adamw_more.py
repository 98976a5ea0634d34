"""The AdamW step on the GPU where its documentation allows what the other tests do not do."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_quantizer_amd as fp8g
from tests import adamw_ref as ref
from tests.gpu_util import dev

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
