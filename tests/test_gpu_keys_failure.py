"""Bounded waits of the key-set kernels that run out, without a GPU fault: the wait
limit shortened to 20 ms and the copy of one key tile left out.  The kernel records
SL_ERR_TIMEOUT, ends by itself, and the same call right after is exact."""
import pytest
import torch

from keys_util import Case
from token_locking_b200 import _abi as A
from token_locking_b200 import runtime as rt

pytestmark = pytest.mark.gpu

# head_dim, listed, prefix, counts, lens, n_ctx: full tiles (bulk copies) and tiles
# copied row by row first; more key tiles than the ring has stages, and fewer; units
# that shares cut, whole ones, and a prefix for all rows together
CASES = [
    (128, False, 0, [300, 40], [1000, 700], 1000),
    (128, True, 0, [300, 40], [900, 700], 1000),
    (128, False, 0, [30], [50], 60),
    (128, False, 900, [20, 30, 1], [200, 0, 90], 200),
    (64, False, 0, [600], [3000], 3000),
    (64, True, 500, [150, 9], [300, 20], 400),
]


def _timeout(call):
    """`call` with its first key tile lost: it ends, and reports once."""
    rt.device_check(clear=True)
    try:
        rt.debug_set_wait_limit(20_000_000)              # 20 ms
        rt.debug_inject_lost_load()
        call()
        torch.cuda.synchronize()
        with pytest.raises(A.SureLockError) as e:
            rt.device_check(clear=True)
        assert e.value.status == A.SL_ERR_TIMEOUT
        rt.device_check(clear=True)                      # cleared: nothing recorded since
    finally:
        rt.debug_set_wait_limit(0)


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{'list' if c[1] else 'first'}-{c[2]}-{c[5]}")
def test_lost_key_tile_is_reported_and_the_next_call_exact(cuda_dev, case):
    dh, listed, prefix, counts, lens, n_ctx = case
    c = Case(cuda_dev, "bf16", counts, lens, n_ctx, 4, 2, dh, prefix, listed, seed=61)
    ka = c.key_attention()
    want, want_lse = c.outputs()
    c.attend(ka, want, want_lse)
    o, lse = c.outputs()
    _timeout(lambda: c.attend(ka, o, lse))
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)

    def weigh():
        m = torch.full((c.B, n_ctx), float("nan"), device=cuda_dev)
        ka.mass(c.q, c.k, lse, m, c.seq_off, key_len=c.key_len, keys=c.keys)
        return m

    want = weigh()
    _timeout(weigh)
    assert torch.equal(weigh(), want)
    rt.device_check(clear=True)


def test_a_bad_position_does_not_hide_a_timeout(cuda_dev):
    """The first report stays: a call that gave up, then one with a position outside
    the cache, before anyone asks."""
    c = Case(cuda_dev, "bf16", [9], [200], 256, 2, 2, 128, listed=True, seed=63)
    ka = c.key_attention()
    o, lse = c.outputs()

    def both():
        c.attend(ka, o, lse)                             # loses its first tile
        c.keys[0, 7] = 256
        c.attend(ka, o, lse)

    _timeout(both)
    c.attend(ka, o, lse)
    with pytest.raises(A.SureLockError) as e:
        rt.device_check(clear=True)
    assert e.value.status == A.SL_ERR_STATE
