"""Key-set attention, attention weight per key and eviction against float64
definitions (tests/keys_util.py derives every tolerance)."""
import math

import numpy as np
import pytest
import torch

from keys_util import Case, ref_attend, ref_evict, ref_mass
from token_locking_b200 import _abi as A
from token_locking_b200 import runtime as rt

pytestmark = pytest.mark.gpu


def _check_attend(c, o, lse, fill=7.0):
    ro, bo, rl, bl = ref_attend(c)
    end = int(c.off[-1])
    assert torch.equal(o[end:].float(), torch.full_like(o[end:].float(), fill))
    assert torch.equal(lse[end:], torch.full_like(lse[end:], fill))
    got = o[:end].double()
    assert torch.isfinite(got).all()
    err = (got - ro[:end]).abs() - bo[:end]
    assert err.numel() == 0 or float(err.max()) <= 0, f"o off by {float(err.max())} above its bound"
    gl, wl = lse[:end].double(), rl[:end]
    empty = torch.isinf(wl)
    assert torch.equal(torch.isinf(gl) & (gl < 0), empty)
    err = torch.where(empty, torch.zeros_like(gl), (gl - wl).abs() - bl[:end])
    assert err.numel() == 0 or float(err.max()) <= 0, f"lse off by {float(err.max())} above its bound"


SHAPES = [
    # dtype, counts, lens, n_ctx, H, Hk, dh, prefix, listed
    ("bf16", [1], [1], 1, 1, 1, 128, 0, False),
    ("bf16", [1], [0], 5, 2, 1, 128, 0, False),
    ("bf16", [3], [127], 130, 2, 2, 128, 0, False),
    ("bf16", [129], [128], 128, 1, 1, 128, 0, False),
    ("bf16", [130, 0, 7], [129, 40, 0], 129, 4, 2, 128, 0, False),
    ("bf16", [300, 1, 64], [511, 200, 333], 600, 3, 3, 128, 0, True),
    ("bf16", [40, 40], [300, 0], 300, 4, 4, 128, 1, False),
    ("bf16", [5, 0, 77, 33, 1], [64, 10, 0, 333, 1], 333, 28, 4, 128, 1025, True),
    ("bf16", [1] * 8, [17] * 8, 40, 8, 2, 128, 700, False),
    ("bf16", [1] * 64, [3 * i % 50 for i in range(64)], 50, 4, 1, 128, 129, True),
    ("bf16", [260], [2000], 2000, 2, 2, 128, 0, False),
    ("bf16", [2, 500], [900, 1300], 1300, 3, 1, 64, 0, True),
    ("bf16", [33, 65], [100, 257], 257, 6, 2, 64, 300, False),
    ("bf16", [200], [400], 400, 5, 1, 64, 0, False),
    ("bf16", [9], [300], 300, 64, 1, 128, 55, False),
    ("bf16", [70, 3], [90, 200], 200, 4, 2, 96, 70, True),
    ("bf16", [17], [65], 65, 2, 2, 8, 0, False),
    ("f32", [1], [1], 1, 1, 1, 16, 0, False),
    ("f32", [64, 0, 5], [64, 3, 0], 65, 4, 4, 16, 0, False),
    ("f32", [33, 130], [200, 77], 200, 8, 2, 64, 0, True),
    ("f32", [1] * 6, [9] * 6, 12, 4, 2, 32, 333, False),
    ("f32", [100, 20], [128, 300], 300, 3, 1, 128, 65, True),
    ("f32", [10], [40], 40, 2, 1, 4, 0, False),
    # more units than CTAs, shares of whole ones; joint prefix over many rows, joined in fours
    ("bf16", [600, 550], [200, 170], 210, 32, 32, 128, 0, True),
    ("bf16", [300, 700], [96, 300], 300, 64, 64, 64, 0, False),
    ("bf16", [24, 5, 30, 1, 0, 41, 24, 24, 63, 24, 2, 50], [100] * 11 + [0], 120, 16, 16, 128, 900, False),
    ("bf16", [7, 40, 90], [64, 0, 500], 500, 48, 3, 64, 3001, True),
    ("f32", [200, 190, 64, 70], [100, 64, 129, 30], 130, 16, 16, 64, 70, True),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
def test_attend_and_mass_match_the_definition(cuda_dev, shape):
    dtype, counts, lens, n_ctx, H, Hk, dh, prefix, listed = shape
    c = Case(cuda_dev, dtype, counts, lens, n_ctx, H, Hk, dh, prefix, listed, seed=len(lens) + dh,
             extra_rows=3)
    c.poison()
    ka = c.key_attention()
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    _check_attend(c, o, lse)
    o2, lse2 = c.outputs(1.0)                    # the same bits again, whatever the workspace holds
    c.attend(ka, o2, lse2)
    end = int(c.off[-1])
    assert torch.equal(o[:end], o2[:end]) and torch.equal(lse[:end], lse2[:end])

    prev = torch.rand((c.B, n_ctx), device=cuda_dev)
    mass = torch.full_like(prev, float("nan"))
    ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len, keys=c.keys, mass_prev=prev,
            decay=0.5)
    want, bound = ref_mass(c, lse, prev, 0.5)
    assert float(((mass.double() - want).abs() - bound).max()) <= 0
    again = prev.clone()                         # in place
    ka.mass(c.q, c.k, lse, again, c.seq_off, key_len=c.key_len, keys=c.keys, mass_prev=again,
            decay=0.5)
    assert torch.equal(mass, again)
    fresh = torch.full_like(prev, float("nan"))  # decay 0 reads no earlier weights
    ka.mass(c.q, c.k, lse, fresh, c.seq_off, key_len=c.key_len, keys=c.keys)
    want, bound = ref_mass(c, lse)
    assert float(((fresh.double() - want).abs() - bound).max()) <= 0


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(cuda_dev, seed):
    rng = np.random.default_rng(1000 + seed)
    dtype = ["bf16", "bf16", "f32"][seed % 3]
    B = int(rng.integers(1, 9))
    n_ctx = int(rng.integers(1, 700))
    top = int(rng.choice([1, 8, 140, 400]))
    counts = rng.integers(0, top + 1, B)
    lens = rng.integers(0, n_ctx + 1, B)
    Hk, G = int(rng.integers(1, 4)), int(rng.integers(1, 10))
    dh = int(rng.choice([64, 128] if dtype == "bf16" else [16, 64]))
    prefix = int(rng.choice([0, rng.integers(1, 3000)]))
    c = Case(cuda_dev, dtype, counts, lens, n_ctx, Hk * G, Hk, dh, prefix,
             bool(rng.integers(0, 2)), seed=seed, extra_rows=int(rng.integers(0, 3)),
             pad=int(rng.choice([0, 8])), spread=float(rng.choice([1.0, 4.0])))
    c.poison(float(rng.choice([float("nan"), float("inf"), -float("inf")])))
    ka = c.key_attention()
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    _check_attend(c, o, lse)
    mass = torch.empty((B, n_ctx), device=cuda_dev)
    ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len, keys=c.keys)
    want, bound = ref_mass(c, lse)
    assert float(((mass.double() - want).abs() - bound).max()) <= 0


@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_no_lengths_and_another_scale(cuda_dev, dtype, dh):
    """key_len None means every cache entry; o and lse without an lse output agree."""
    c = Case(cuda_dev, dtype, [50, 90], [150, 150], 150, 4, 2, dh, seed=3, scale=0.02, pad=16)
    ka = c.key_attention()
    o, lse = c.outputs()
    ka.attend(c.q, c.k, c.v, o, c.seq_off, lse=lse)
    _check_attend(c, o, lse)
    o2, _ = c.outputs()
    ka.attend(c.q, c.k, c.v, o2, c.seq_off)
    assert torch.equal(o, o2)


KERNELS = [("bf16", 128), ("bf16", 64), ("bf16", 96), ("f32", 64)]


@pytest.mark.parametrize("dtype,dh", KERNELS)
def test_scores_far_apart(cuda_dev, dtype, dh):
    """Scores in the hundreds: the maximum rises by more than 2^8 between tiles
    and one key takes nearly all of a row's weight."""
    c = Case(cuda_dev, dtype, [70, 3], [400, 333], 400, 4, 2, dh, prefix=150, seed=31, spread=30.0)
    # later keys are longer, so that the running maximum keeps rising
    ramp = torch.linspace(0.1, 4.0, 400, device=cuda_dev).repeat(2)[:, None]
    c.k.copy_((c.k.float() * ramp).to(c.dt))
    ka = c.key_attention()
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    _check_attend(c, o, lse)
    mass = torch.empty((2, 400), device=cuda_dev)
    ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len)
    want, bound = ref_mass(c, lse)
    assert float(((mass.double() - want).abs() - bound).max()) <= 0


@pytest.mark.parametrize("dtype,dh", KERNELS)
def test_infinite_scores_and_nan_stay_in_their_rows(cuda_dev, dtype, dh):
    """Keys of -inf score weigh nothing, a row of them alone gives 0 and -inf, and a
    NaN query spoils its own row of attention only (and the weights it adds to)."""
    c = Case(cuda_dev, dtype, [40, 30], [130, 90], 200, 2, 1, dh, seed=33)
    H = c.H
    q = c.q.abs() + 0.1                                  # positive: the score's sign is the key's
    c.q.copy_(q.to(c.dt))
    c.k[5], c.k[77] = -math.inf, -math.inf               # two keys of sequence 0
    c.k[200:290] = -math.inf                             # all of sequence 1's
    c.q[3] = float("nan")
    ka = c.key_attention()
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    assert torch.isnan(o[3]).all() and torch.isnan(lse[3]).all()
    assert (o[40:70] == 0).all() and (lse[40:70] == -math.inf).all()
    clean = [r for r in range(40) if r != 3]
    assert torch.isfinite(o[clean]).all() and torch.isfinite(lse[clean]).all()
    live = [i for i in range(130) if i not in (5, 77)]
    s = 1.0 / math.sqrt(dh)
    for h in range(H):
        z = c.q[clean, h * dh:(h + 1) * dh].double() @ c.k[live].double().T * s
        assert torch.allclose(lse[clean, h].double(), torch.logsumexp(z, dim=1), atol=1e-4, rtol=1e-5)
    # without the NaN row the weights are finite, and zero for the -inf keys
    mass = torch.empty((2, 200), device=cuda_dev)
    ka.mass(c.q[4:], c.k, lse[4:].contiguous(), mass,
            torch.tensor([0, 36, 66], dtype=torch.int32, device=cuda_dev), key_len=c.key_len)
    assert torch.isfinite(mass).all() and (mass[0, [5, 77]] == 0).all() and (mass[1] == 0).all()
    ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len)
    assert torch.isnan(mass[0, live]).all() and (mass[1] == 0).all()


@pytest.mark.parametrize("dtype,dh", KERNELS)
def test_no_rows(cuda_dev, dtype, dh):
    """No rows at all: nothing attends, the weights only decay."""
    c = Case(cuda_dev, dtype, [0, 0], [9, 4], 12, 2, 1, dh, prefix=5, seed=35)
    ka = c.key_attention()
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    prev = torch.rand((2, 12), device=cuda_dev)
    mass = torch.full_like(prev, float("nan"))
    ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len, mass_prev=prev, decay=0.25)
    assert torch.equal(mass, prev * 0.25)
    ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len)
    assert (mass == 0).all()


@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_groups_up_to_sixty_four(cuda_dev, dtype, dh):
    for G in (3, 5, 31, 33, 64):
        c = Case(cuda_dev, dtype, [9, 1, 20], [70, 33, 128], 130, 2 * G, 2, dh, prefix=90, seed=G)
        c.poison()
        ka = c.key_attention()
        o, lse = c.outputs()
        c.attend(ka, o, lse)
        _check_attend(c, o, lse)
        mass = torch.empty((3, 130), device=cuda_dev)
        ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len)
        want, bound = ref_mass(c, lse)
        assert float(((mass.double() - want).abs() - bound).max()) <= 0


def test_alignment_of_sixteen_bytes(cuda_dev):
    """Operands and results on 16-byte boundaries that are no 32-byte ones."""
    c = Case(cuda_dev, "bf16", [150, 20], [200, 100], 200, 2, 2, 128, seed=37, pad=8)
    for n in ("q", "k", "v"):
        t = getattr(c, n)
        big = torch.full((t.shape[0], t.shape[1] + 24), float("nan"), dtype=t.dtype, device=cuda_dev)
        big[:, 8:8 + t.shape[1]] = t
        setattr(c, n, big[:, 8:8 + t.shape[1]])
    ka = c.key_attention()
    buf = torch.full((c.rows, 256 + 24), 7.0, dtype=c.dt, device=cuda_dev)
    o, lse = buf[:, 8:264], c.outputs()[1]
    c.attend(ka, o, lse)
    _check_attend(c, o, lse)
    assert (buf[:, :8] == 7).all() and (buf[:, 264:] == 7).all()


def test_streams_one_after_the_other(cuda_dev):
    """One object used from two streams that the caller orders, and its result read
    on a third."""
    c = Case(cuda_dev, "bf16", [90, 40], [700, 300], 700, 4, 4, 128, prefix=333, seed=39)
    ka = c.key_attention()
    outs = [c.outputs() for _ in range(4)]
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    last = None
    for i, (o, lse) in enumerate(outs):
        s = ss[i % 2]
        if last is not None:
            s.wait_event(last)
        c.attend(ka, o, lse, stream=s)
        last = torch.cuda.Event()
        last.record(s)
    torch.cuda.current_stream().wait_event(last)
    for o, lse in outs:
        _check_attend(c, o, lse)


@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("f32", 32)])
def test_duplicate_positions_count_twice(cuda_dev, dtype, dh):
    c = Case(cuda_dev, dtype, [20], [6], 300, 2, 1, dh, listed=True, seed=5)
    c.pos = [np.array([4, 4, 9, 250, 250, 250])]
    c.keys[0, :6] = torch.tensor(c.pos[0], dtype=torch.int32)
    ka = c.key_attention()
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    _check_attend(c, o, lse)
    mass = torch.empty((1, 300), device=cuda_dev)
    ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len, keys=c.keys)
    want, bound = ref_mass(c, lse)
    assert float(((mass.double() - want).abs() - bound).max()) <= 0


@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("f32", 32)])
def test_positions_out_of_range_are_zeros_and_reported(cuda_dev, dtype, dh):
    rt.device_check(clear=True)
    c = Case(cuda_dev, dtype, [9, 4], [200, 3], 256, 2, 2, dh, listed=True, seed=6)
    bad = [(0, 0, -1), (0, 100, 256), (0, 199, 2 ** 31 - 1), (1, 2, -(2 ** 31))]
    z = c.k.new_zeros((1, c.k.shape[1]))
    k, v = torch.cat([c.k, z]), torch.cat([c.v, z])        # row 512: zeros
    for b, i, n in bad:
        c.keys[b, i] = n
        c.pos[b] = c.pos[b].copy()
        c.pos[b][i] = 2 * 256 - b * 256                    # the reference reads row 512
    ka = c.key_attention()
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    real = c.k, c.v
    c.k, c.v = k, v
    _check_attend(c, o, lse)
    with pytest.raises(A.SureLockError) as e:
        rt.device_check(clear=True)
    assert e.value.status == A.SL_ERR_STATE
    c.k, c.v = real
    mass = torch.empty((2, 256), device=cuda_dev)
    ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len, keys=c.keys)
    with pytest.raises(A.SureLockError):
        rt.device_check(clear=True)
    for b, i, _ in bad:                                    # no position receives their weight
        c.pos[b] = np.delete(c.pos[b], [j for bb, j, _ in bad if bb == b]) if \
            len(c.pos[b]) == c.lens[b] else c.pos[b]
    want, bound = ref_mass(c, lse)
    assert float(((mass.double() - want).abs() - bound).max()) <= 0
    rt.device_check(clear=True)


@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("f32", 64)])
def test_bad_offsets_and_lengths_are_clamped(cuda_dev, dtype, dh):
    c = Case(cuda_dev, dtype, [10, 0, 30], [60, 60, 60], 60, 2, 2, dh, prefix=20, seed=8)
    ka = c.key_attention()
    c.seq_off.copy_(torch.tensor([-5, 10, 3, 1 << 30], dtype=torch.int32))
    c.key_len.copy_(torch.tensor([1 << 30, 60, 61], dtype=torch.int32))
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    _check_attend(c, o, lse)
    c.key_len.fill_(-3)
    c.lens, c.pos = [0, 0, 0], [np.arange(0)] * 3
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    _check_attend(c, o, lse)


@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("f32", 64)])
def test_captured_call_follows_new_offsets_on_another_stream(cuda_dev, dtype, dh):
    """A captured graph replays with new rows, offsets, lengths and lists in the
    same buffers; two graphs share the object on one stream."""
    n_ctx = 500
    a = Case(cuda_dev, dtype, [100, 3], [400, 50], n_ctx, 4, 2, dh, 260, True, seed=11, extra_rows=97)
    b = Case(cuda_dev, dtype, [1, 199], [500, 33], n_ctx, 4, 2, dh, 260, True, seed=12)
    ka = a.key_attention()
    st = torch.cuda.Stream()
    o, lse = a.outputs()
    mass = torch.zeros((2, n_ctx), device=cuda_dev)
    bufs = {n: getattr(a, n).clone() for n in ("q", "k", "v", "kp", "vp", "seq_off", "key_len", "keys")}

    def call():
        ka.attend(bufs["q"], bufs["k"], bufs["v"], o, bufs["seq_off"], key_len=bufs["key_len"],
                  keys=bufs["keys"], k_prefix=bufs["kp"], v_prefix=bufs["vp"], lse=lse)

    def weigh():
        ka.mass(bufs["q"], bufs["k"], lse, mass, bufs["seq_off"], key_len=bufs["key_len"],
                keys=bufs["keys"])

    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
        g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g1, stream=st):
            call()
        with torch.cuda.graph(g2, stream=st):
            weigh()
        for c in (a, b, a):
            for n in bufs:
                bufs[n].copy_(getattr(c, n))
            o.fill_(7.0)
            lse.fill_(7.0)
            g1.replay()
            g2.replay()
            st.synchronize()
            _check_attend(c, o, lse)
            want, bound = ref_mass(c, lse)
            assert float(((mass.double() - want).abs() - bound).max()) <= 0
        st.synchronize()


def test_cache_beyond_32_bit_offsets(cuda_dev):
    """Entries whose element offsets pass 2^31 (a cache of 5.2 GB)."""
    n_ctx, H, dh = 320_000, 16, 128
    B = 2
    k = torch.empty((B * n_ctx, H * dh), dtype=torch.bfloat16, device=cuda_dev)
    g = torch.Generator(device=cuda_dev).manual_seed(4)
    pos = np.array([0, 5, n_ctx // 2, n_ctx - 300, n_ctx - 1])
    rows = torch.from_numpy(np.concatenate([pos, pos + n_ctx])).to(cuda_dev)
    k[rows] = torch.randn((10, H * dh), device=cuda_dev, generator=g).to(torch.bfloat16)
    c = Case(cuda_dev, "bf16", [3, 2], [5, 5], 8, H, H, dh, seed=4)
    c.n_ctx, c.k, c.v, c.pos = n_ctx, k, k, [pos, pos]
    c.keys = torch.zeros((B, n_ctx), dtype=torch.int32, device=cuda_dev)
    c.keys[:, :5] = torch.from_numpy(pos.astype(np.int32)).to(cuda_dev)
    ka = c.key_attention()
    o, lse = c.outputs()
    c.attend(ka, o, lse)
    _check_attend(c, o, lse)
    mass = torch.empty((B, n_ctx), device=cuda_dev)
    ka.mass(c.q, c.k, lse, mass, c.seq_off, key_len=c.key_len, keys=c.keys)
    want, bound = ref_mass(c, lse)
    assert float(((mass.double() - want).abs() - bound).max()) <= 0


# ------------------------------------------------------------------ eviction --

def _evict(dev, mass, budget, protect=None, present=None, inplace=False):
    B, N = mass.shape
    t = torch.from_numpy(mass).to(dev)
    up = None if protect is None else torch.from_numpy(protect).to(dev)
    pr = None if present is None else torch.from_numpy(present).to(dev)
    keys = torch.full((B, N), -9, dtype=torch.int32, device=dev)
    n = torch.full((B,), -9, dtype=torch.int32, device=dev)
    out = pr if inplace else torch.full((B, N), 9, dtype=torch.uint8, device=dev)
    rt.kv_evict(t, budget, keys, n, protect=up, present=pr, present_out=out)
    return keys.cpu().numpy(), n.cpu().numpy(), out.cpu().numpy()


def _check_evict(got, want, N):
    keys, n, flags = got
    for b, w in enumerate(want):
        assert n[b] == len(w)
        np.testing.assert_array_equal(keys[b, :len(w)], w)
        assert (keys[b, len(w):] == -9).all()
        f = np.zeros(N, dtype=np.uint8)
        f[w] = 1
        np.testing.assert_array_equal(flags[b], f)


@pytest.mark.parametrize("B,N", [(1, 1), (2, 31), (3, 1024), (1, 1025), (64, 300), (2, 5000),
                                 (2, 40000), (1, 131073), (1, 500001)])
@pytest.mark.parametrize("kind", ["heavy", "ties", "zeros", "odd"])
def test_evict_matches_sorting(cuda_dev, B, N, kind):
    rng = np.random.default_rng(N + B)
    m = np.exp(2 * rng.standard_normal((B, N))).astype(np.float32)
    if kind == "ties":
        m = rng.integers(-2, 3, (B, N)).astype(np.float32)
    elif kind == "zeros":
        m = np.where(rng.random((B, N)) < 0.5, 0.0, -0.0).astype(np.float32)
    elif kind == "odd":
        pick = rng.random((B, N))
        m[pick < 0.2] = np.nan
        m[(pick >= 0.2) & (pick < 0.4)] = -np.inf
        m[(pick >= 0.4) & (pick < 0.5)] = np.inf
        m[(pick >= 0.5) & (pick < 0.6)] = -1e-40          # subnormal
        m[(pick >= 0.6) & (pick < 0.65)] = -np.float32(np.nan)
    protect = (rng.random((B, N)) < 0.1).astype(np.uint8)
    present = (rng.random((B, N)) < 0.7).astype(np.uint8) * rng.integers(1, 256, (B, N)).astype(np.uint8)
    for budget in sorted({0, 1, N // 3, N // 2 + 1, N, 3 * N}):
        _check_evict(_evict(cuda_dev, m, budget, protect, present),
                     ref_evict(m, budget, protect, present), N)
    b = N // 2
    _check_evict(_evict(cuda_dev, m, b), ref_evict(m, b), N)
    _check_evict(_evict(cuda_dev, m, b, None, present.copy(), inplace=True),
                 ref_evict(m, b, None, present), N)
    _check_evict(_evict(cuda_dev, m, b, protect), ref_evict(m, b, protect), N)
    _check_evict(_evict(cuda_dev, m, b, np.ones_like(protect), np.zeros_like(present)),
                 [[] for _ in range(B)], N)


# ------------------------------------------------------ together, and refusals --

@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("f32", 16)])
def test_steps_with_eviction(cuda_dev, dtype, dh):
    """As a decode uses them: attention over what is kept and a shared prompt,
    weights accumulated over steps and layers, eviction of the light locked
    entries, attention over the list that it leaves."""
    layers, n_ctx, P, budget = 2, 260, 150, 120
    c = [Case(cuda_dev, dtype, [30, 61, 7], [n_ctx] * 3, n_ctx, 4, 2, dh, P, seed=20 + l)
         for l in range(layers)]
    ka = c[0].key_attention()
    present = torch.ones((3, n_ctx), dtype=torch.uint8, device=cuda_dev)
    protect = torch.zeros_like(present)
    protect[:, 40:75] = 1
    keys = torch.zeros((3, n_ctx), dtype=torch.int32, device=cuda_dev)
    n = torch.full((3,), n_ctx, dtype=torch.int32, device=cuda_dev)
    mass = torch.zeros((3, n_ctx), device=cuda_dev)
    want = np.zeros((3, n_ctx))
    for step in range(3):
        for l, x in enumerate(c):
            if step > 0:
                x.keys, x.key_len = keys, n
                x.lens = n.tolist()
                x.pos = [keys[b, :x.lens[b]].cpu().numpy() for b in range(3)]
            o, lse = x.outputs()
            x.attend(ka, o, lse)
            _check_attend(x, o, lse)
            before = mass.clone()
            ka.mass(x.q, x.k, lse, mass, x.seq_off, key_len=x.key_len, keys=x.keys,
                    mass_prev=mass, decay=0.9)
            w, bound = ref_mass(x, lse, before, 0.9)
            assert float(((mass.double() - w).abs() - bound).max()) <= 0
        want = ref_evict(mass.cpu().numpy(), budget - 20 * step, protect.cpu().numpy(),
                         present.cpu().numpy())
        rt.kv_evict(mass, budget - 20 * step, keys, n, protect=protect, present=present,
                    present_out=present)
        assert n.tolist() == [len(x) for x in want]
        for b in range(3):
            np.testing.assert_array_equal(keys[b, :len(want[b])].cpu().numpy(), want[b])
        for x in c:                                       # what left the cache may hold anything
            gone = (present == 0).reshape(-1)
            x.k[gone] = float("nan")
            x.v[gone] = float("nan")


def test_binding_refusals(cuda_dev):
    c = Case(cuda_dev, "bf16", [4], [9], 16, 4, 2, 64, seed=1)
    ka = c.key_attention()
    o, lse = c.outputs()

    def call(**kw):
        a = dict(q=c.q, k=c.k, v=c.v, o=o, seq_off=c.seq_off, key_len=c.key_len, lse=lse)
        a.update(kw)
        ka.attend(**a)

    call()
    for bad in (dict(q=c.q.float()), dict(k=c.k[:5]), dict(v=c.v.cpu()), dict(o=o[:2]),
                dict(seq_off=c.seq_off.long()), dict(seq_off=c.seq_off[:1]),
                dict(key_len=c.key_len.float()), dict(lse=lse[:, :2]), dict(lse=lse.double()),
                dict(q=c.q[:, :64]), dict(k=c.k.t().contiguous().t()),
                dict(keys=torch.zeros((1, 15), dtype=torch.int32, device=cuda_dev)),
                dict(k_prefix=c.k)):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(A.SureLockError) as e:             # created without a prefix
        call(k_prefix=c.k, v_prefix=c.v)
    assert e.value.status == A.SL_ERR_INVALID and "prefix" in str(e.value)
    wide = torch.zeros((4, 4 * 64 + 4), dtype=torch.bfloat16, device=cuda_dev)
    with pytest.raises(A.SureLockError):                  # rows not 16-byte aligned
        call(q=wide[:, :256])
    with pytest.raises(A.SureLockError):
        call(q=wide[:, 4:])
    big = Case(cuda_dev, "bf16", [5], [9], 16, 4, 2, 64, seed=1)
    with pytest.raises(A.SureLockError) as e:             # more rows than max_rows
        call(q=big.q, o=big.outputs()[0], lse=None)
    assert "max_rows" in str(e.value)
    m = torch.zeros((1, 16), device=cuda_dev)
    with pytest.raises(A.SureLockError):                  # decay without earlier weights
        ka.mass(c.q, c.k, lse, m, c.seq_off, decay=1.0)
    keys = torch.zeros((1, 16), dtype=torch.int32, device=cuda_dev)
    n = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    with pytest.raises(A.SureLockError):
        rt.kv_evict(m, -1, keys, n)
    with pytest.raises(ValueError):
        rt.kv_evict(m, 4, keys.long(), n)
    with pytest.raises(ValueError):
        rt.kv_evict(m, 4, keys, n, protect=m)
    rt.device_check()
