"""Key-set operators where single rows, values or sizes could go wrong (the
definitions and bounds of tests/keys_util.py)."""
import math

import pytest
import torch

from keys_util import Case, ref_attend, ref_evict, ref_mass
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


# Work plans that the other shapes do not reach (on 148 SMs): shares long enough to be
# padded to each sequence's start, and a joint prefix whose units are dealt out whole.
PLANS = [
    ("bf16", [61, 102, 143, 218, 82], [539, 371, 71, 426, 189], 540, 6, 6, 128, 12414),
    ("bf16", [271, 259, 111, 108, 107], [217, 353, 212, 459, 420], 460, 6, 6, 64, 11142),
    ("bf16", [20, 20, 20], [240, 240, 240], 240, 37, 37, 128, 240),
    ("bf16", [20, 20, 20], [240, 240, 240], 240, 74, 74, 128, 240),
    ("f32", [8, 8, 8], [192, 192, 192], 192, 74, 74, 16, 192),
]


@pytest.mark.parametrize("shape", PLANS, ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
def test_padded_shares_and_whole_joint_units(cuda_dev, shape):
    dtype, counts, lens, n_ctx, H, Hk, dh, prefix = shape
    c = Case(cuda_dev, dtype, counts, lens, n_ctx, H, Hk, dh, prefix, seed=54, extra_rows=2)
    c.poison()
    ka = c.key_attention()
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    ro, bo, rl, bl = ref_attend(c)
    end = int(c.off[-1])
    assert (o[end:] == 7).all() and (lse[end:] == 7).all()
    assert _within(o[:end], ro[:end], bo[:end]) and _within(lse[:end], rl[:end], bl[:end])
    o2, lse2 = c.outputs()
    c.attend(ka, o2, lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_two_objects_at_the_same_time(cuda_dev):
    """Two objects, each on a stream of its own, nothing ordering them."""
    cs = [Case(cuda_dev, "bf16", [90, 300], [700, 300], 700, 4, 4, 128, prefix=p, listed=not p,
               seed=55) for p in (0, 333)]
    kas, want = [c.key_attention() for c in cs], []

    def both(c, ka, stream):
        with torch.cuda.stream(stream):
            o, lse = c.outputs()
            m = torch.empty((2, 700), device=cuda_dev)
            c.attend(ka, o, lse)
            ka.mass(c.q, c.k, lse, m, c.seq_off, key_len=c.key_len, keys=c.keys)
            return o, lse, m

    for c, ka in zip(cs, kas):
        want.append(both(c, ka, torch.cuda.current_stream()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [both(c, ka, s) for c, ka, s in zip(cs, kas, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(g, w))
    rt.device_check()


def _evicts(dev, mass, budget, protect, present):
    B, N = mass.shape
    keys = torch.full((B, N), -9, dtype=torch.int32, device=dev)
    n = torch.full((B,), -9, dtype=torch.int32, device=dev)
    out = torch.full((B, N), 9, dtype=torch.uint8, device=dev)
    rt.kv_evict(mass, budget, keys, n, protect=protect, present=present, present_out=out)
    for b, want in enumerate(ref_evict(mass.cpu().numpy(), budget, protect.cpu().numpy(),
                                       present.cpu().numpy())):
        flags = torch.zeros(N, dtype=torch.uint8)
        flags[want] = 1
        assert n[b] == len(want)
        assert keys[b, :len(want)].tolist() == want and (keys[b, len(want):] == -9).all()
        assert torch.equal(out[b].cpu(), flags)


@pytest.mark.parametrize("N", [4095, 4096, 4097, 8192, 8193, 12001, 16384, 16385, 393216, 393217])
def test_evict_at_the_borders_of_its_clusters(cuda_dev, N):
    """One, two, four and eight CTAs a sequence, entries kept in shared memory or read
    again, each side of every border."""
    g = torch.Generator(device=cuda_dev).manual_seed(N)
    B = 1 if N > 20000 else 2
    m = torch.exp(2 * torch.randn((B, N), device=cuda_dev, generator=g))
    ties = torch.randint(-1, 3, (B, N), device=cuda_dev, generator=g).float()
    protect = (torch.rand((B, N), device=cuda_dev, generator=g) < 0.1).to(torch.uint8)
    present = (torch.rand((B, N), device=cuda_dev, generator=g) < 0.8).to(torch.uint8)
    _evicts(cuda_dev, m, N // 2, protect, present)
    _evicts(cuda_dev, ties, N // 3, protect, present)


def test_captured_eviction_follows_new_weights(cuda_dev):
    B, N = 2, 9000
    m = torch.rand((B, N), device=cuda_dev)
    present = torch.ones((B, N), dtype=torch.uint8, device=cuda_dev)
    keys = torch.zeros((B, N), dtype=torch.int32, device=cuda_dev)
    n = torch.zeros(B, dtype=torch.int32, device=cuda_dev)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            rt.kv_evict(m, 1000, keys, n, present=present, present_out=present)
        for seed in range(3):
            g = torch.Generator(device=cuda_dev).manual_seed(seed)
            m.copy_(torch.randn((B, N), device=cuda_dev, generator=g))
            present.copy_((torch.rand((B, N), device=cuda_dev, generator=g) < 0.5).to(torch.uint8))
            was = present.cpu().numpy()
            graph.replay()
            st.synchronize()
            for b, want in enumerate(ref_evict(m.cpu().numpy(), 1000, None, was)):
                assert n[b] == len(want) and keys[b, :len(want)].tolist() == want
                assert present[b].nonzero()[:, 0].tolist() == want
