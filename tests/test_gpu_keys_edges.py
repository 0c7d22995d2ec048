"""Key-set operators where single rows, values or sizes could go wrong (the
definitions and bounds of tests/keys_util.py)."""
import math

import pytest
import torch

from keys_util import Case, ref_mass
from token_locking_b200 import _abi as A
from token_locking_b200 import runtime as rt

pytestmark = pytest.mark.gpu

KERNELS = [("bf16", 128), ("bf16", 64), ("bf16", 96), ("f32", 64)]


def _within(got, want, bound):
    return float(((got.double() - want).abs() - bound).max()) <= 0


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("dtype,dh", KERNELS)
def test_rows_with_lse_of_minus_infinity_weigh_nothing(cuda_dev, dtype, dh, listed):
    """Whatever their queries hold: NaN and infinite scores of rows that the caller
    left out (lse = -inf) reach no weight.  The rows lie at the ends of blocks and
    sequences, and one sequence has no others."""
    c = Case(cuda_dev, dtype, [150, 3, 70], [300, 40, 129], 320, 6, 2, dh, listed=listed, seed=51)
    ka = c.key_attention()
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    dead = [0, 1, 41, 42, 63, 64, 127, 128, 149, 150, 151, 152, 153, 222]
    lse[dead] = -math.inf
    lse[200, 3:5] = -math.inf                            # two heads of a row whose query is fine
    values = [float("nan"), math.inf, -math.inf]
    for i, r in enumerate(dead):
        c.q[r] = values[i % 3]
    mass = torch.empty((3, 320), device=cuda_dev)
    ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len, keys=c.keys)
    c.q[dead] = 0.0                                      # the reference's products stay finite
    want, bound = ref_mass(c, lse)
    assert torch.isfinite(mass).all() and (mass[1] == 0).all()
    assert _within(mass, want, bound)


@pytest.mark.parametrize("dtype,dh", KERNELS)
def test_rows_with_lse_of_plus_infinity_follow_the_formula(cuda_dev, dtype, dh):
    """exp(z - inf) is 0 for a finite score z, and NaN for a score of NaN or +inf."""
    c = Case(cuda_dev, dtype, [40, 9], [100, 60], 130, 2, 1, dh, seed=52)
    ka = c.key_attention()
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    lse[7], lse[45] = math.inf, math.inf
    mass = torch.empty((2, 130), device=cuda_dev)
    ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len)
    want, bound = ref_mass(c, lse)
    assert torch.isfinite(mass).all() and _within(mass, want, bound)
    c.q[45] = float("nan")
    ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len)
    assert torch.isnan(mass[1, :60]).all() and (mass[1, 60:] == 0).all()
    assert _within(mass[:1], want[:1], bound[:1])


@pytest.mark.parametrize("keys,prefix", [(90, 0), (3000, 0), (70, 500)])
@pytest.mark.parametrize("dtype,dh", KERNELS)
def test_rows_of_minus_infinity_give_zero_whatever_v_holds(cuda_dev, dtype, dh, keys, prefix):
    """A row whose scores are all -inf gets o = 0 and lse = -inf, also where v is
    infinite or NaN, in whole units, in cut ones and over a joint prefix."""
    c = Case(cuda_dev, dtype, [20, 5], [keys, 33], keys, 2, 1, dh, prefix, seed=53)
    c.q.copy_((c.q.abs() + 0.1).to(c.dt))                # positive: the score's sign is the key's
    c.k[:keys] = -math.inf
    c.v[:keys:3], c.v[1:keys:3] = math.inf, float("nan")
    if prefix:                                           # then the other sequence sees no key either
        c.kp.fill_(-math.inf)
        c.vp.fill_(math.inf)
        c.k[keys:] = -math.inf
    ka = c.key_attention()
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    n = 25 if prefix else 20
    assert (o[:n] == 0).all() and (lse[:n] == -math.inf).all()
    assert torch.isfinite(o[20:]).all() and torch.isfinite(lse[n:]).all()


def test_budgets_beyond_32_bits(cuda_dev):
    """Any budget above the cache keeps everything, any negative one is refused."""
    m = torch.rand((2, 50), device=cuda_dev)
    for budget in (50, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 7, 10 ** 15):
        keys = torch.full((2, 50), -9, dtype=torch.int32, device=cuda_dev)
        n = torch.full((2,), -9, dtype=torch.int32, device=cuda_dev)
        rt.kv_evict(m, budget, keys, n)
        assert n.tolist() == [50, 50]
        assert torch.equal(keys.cpu(), torch.arange(50, dtype=torch.int32).repeat(2, 1))
    for budget in (-1, -(2 ** 31) - 1, -(2 ** 32), -(2 ** 32) + 7):
        with pytest.raises(A.SureLockError) as e:
            rt.kv_evict(m, budget, keys, n)
        assert e.value.status == A.SL_ERR_INVALID
