"""GPU tests of the cache of states in 8 bits (gdn_state_store, gdn_state_load).  The codes and
scales are defined to the last bit (oracle/block.py), and so is what is read back, a float32
product: everything is compared for equality."""
import numpy as np
import pytest
import torch

from gated_delta_rule_19_gb300 import gdn
from oracle import block

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_19_gb300 import _build

    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _np(t):
    return t.detach().double().cpu().numpy()


def _cache(n, H, V, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randint(-127, 128, (n, H, V, K), generator=g, device="cuda", dtype=torch.int8),
            torch.rand(n, H, V, generator=g, device="cuda"))


def _states(B, H, V, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    return torch.randn(B, H, V, K, generator=g, device="cuda") * torch.exp(3 * torch.randn(B, H, V, 1, generator=g, device="cuda"))


def _slots(*s):
    return torch.tensor(s, dtype=torch.int32, device="cuda")


def _check(states, cache, scales, slots):
    codes, steps = block.park(_np(states))
    at = slots.long()
    np.testing.assert_array_equal(_np(scales[at]), steps)
    np.testing.assert_array_equal(_np(cache[at]), codes)


@pytest.mark.parametrize("B,H,V,K", [(1, 1, 16, 16), (1, 3, 32, 128), (5, 2, 64, 32), (3, 5, 128, 64), (4, 16, 128, 128), (7, 1, 16, 64),
                                     (2, 7, 128, 16)])
def test_store_and_load(B, H, V, K):
    n = B + 4
    cache, scales = _cache(n, H, V, K)
    kept_c, kept_s = cache.clone(), scales.clone()
    states = _states(B, H, V, K, seed=K)
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(B))[:B].to(torch.int32).cuda()
    before = cache._version, scales._version, states._version
    got = gdn.gdn_state_store(states, slots, cache, scales)
    assert got[0] is cache and got[1] is scales
    assert cache._version > before[0] and scales._version > before[1] and states._version == before[2]
    torch.cuda.synchronize()
    _check(states, cache, scales, slots)
    others = torch.ones(n, dtype=torch.bool, device="cuda")
    others[slots.long()] = False
    assert torch.equal(cache[others], kept_c[others]) and torch.equal(scales[others], kept_s[others])
    # any of them back, one twice, and new sequences
    back = _slots(n - 1, -1, int(slots[0]), n, int(slots[0]), 0, 2 ** 31 - 1, -2 ** 31)
    out = torch.full((8, H, V, K), float("nan"), device="cuda")
    res = gdn.gdn_state_load(cache, scales, back, states=out)
    torch.cuda.synchronize()
    assert res is out
    ref = cache.float() * scales[..., None]
    for i, s in enumerate(back.tolist()):
        assert torch.equal(out[i], ref[s] if 0 <= s < n else torch.zeros_like(out[i]))
    # what is read back is within half a step of what was parked
    mine = gdn.gdn_state_load(cache, scales, slots)
    assert ((mine - states).abs() <= scales[slots.long()][..., None] * 0.50001).all()


def test_sequences_outside_and_with_one_slot():
    B, H, V, K, n = 300, 2, 16, 32, 5
    cache, scales = _cache(n, H, V, K)
    kept = cache.clone(), scales.clone()
    states = _states(B, H, V, K)
    slots = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    slots[3], slots[299], slots[7], slots[8], slots[20], slots[21] = 2, 2, 4, 4, n, 2 ** 31 - 1
    gdn.gdn_state_store(states, slots, cache, scales)
    torch.cuda.synchronize()
    _check(states[[299, 8]], cache, scales, _slots(2, 4))
    for s in (0, 1, 3):
        assert torch.equal(cache[s], kept[0][s]) and torch.equal(scales[s], kept[1][s])


def test_ties_and_next_to_them():
    """Quotients at the middle between two whole numbers go to the even one, those next to it
    to the nearer one, for steps of any size."""
    K = 64
    rows = []
    for step in (1.0, 2.0 ** -3, np.float32(0.1), np.float32(1 / 3), np.float32(7.7e-20), np.float32(1.9e30)):
        s = np.float32(step)
        base = np.array([(i + 0.5) for i in range(-31, 31)], dtype=np.float64) * np.float64(s)
        for shift in (0, 1, -1):
            x = base.astype(np.float32)
            x = x if shift == 0 else np.nextafter(x, np.float32(np.inf if shift > 0 else -np.inf))
            rows.append(np.concatenate([[np.float32(np.float64(s) * 127)], x, [0.0]]).astype(np.float32))
    part = np.float32(1) / np.float32(127)
    r = np.random.default_rng(0)
    while len(rows) < 16 * 20:  # random steps, quotients next to a middle
        top = np.float32(np.exp(r.normal() * 20))
        s = top * part
        x = ((r.integers(-126, 126, 62) + 0.5) * np.float64(s)).astype(np.float32)
        x = np.where(r.random(62) < 0.5, np.nextafter(x, np.float32(np.inf)), x)
        rows.append(np.concatenate([[top], x, [-top]]).astype(np.float32))
    states = torch.from_numpy(np.stack(rows)[:320]).view(20, 1, 16, K).cuda()
    cache, scales = _cache(20, 1, 16, K)
    gdn.gdn_state_store(states, torch.arange(20, dtype=torch.int32, device="cuda"), cache, scales)
    torch.cuda.synchronize()
    _check(states, cache, scales, torch.arange(20, device="cuda"))


def test_rows_of_zeros_the_least_and_the_largest_numbers():
    states = torch.zeros(1, 1, 16, 32, device="cuda")
    states[0, 0, 1] = torch.linspace(-1, 1, 32, device="cuda") * 1e-40  # subnormal
    states[0, 0, 2] = torch.linspace(-1, 1, 32, device="cuda") * 3.4e38
    states[0, 0, 3, 5] = 1.5e-36  # a step next to the least
    states[0, 0, 4] = -0.0
    states[0, 0, 5, 0] = float("nan")
    states[0, 0, 6, 31] = float("inf")
    states[0, 0, 7, 31], states[0, 0, 7, 1] = -float("inf"), 5.0
    cache, scales = _cache(2, 1, 16, 32)
    gdn.gdn_state_store(states, _slots(1), cache, scales)
    back = gdn.gdn_state_load(cache, scales, _slots(1))
    torch.cuda.synchronize()
    fine = [0, 1, 2, 3, 4] + list(range(8, 16))
    codes, steps = block.park(_np(states[0, 0, fine]))
    np.testing.assert_array_equal(_np(scales[1, 0, fine]), steps)
    np.testing.assert_array_equal(_np(cache[1, 0, fine]), codes)
    assert back[0, 0, 5:8].isnan().all() and scales[1, 0, 5:8].isnan().all()
    assert back[0, 0, fine].isfinite().all()


def test_more_than_2_31_elements():
    """Slots past 2^31 bytes of cache, and states past 2^31 elements."""
    H, V, K = 16, 128, 128
    n = 2 ** 31 // (H * V * K) + 20
    cache = torch.zeros(n, H, V, K, dtype=torch.int8, device="cuda")
    scales = torch.zeros(n, H, V, device="cuda")
    states = _states(3, H, V, K)
    slots = _slots(n - 1, 4, n - 3)
    gdn.gdn_state_store(states, slots, cache, scales)
    back = gdn.gdn_state_load(cache, scales, torch.arange(n, dtype=torch.int32, device="cuda"))  # 8.6 GB
    torch.cuda.synchronize()
    _check(states, cache, scales, slots)
    ref = cache[slots.long()].float() * scales[slots.long()][..., None]
    assert torch.equal(back[slots.long()], ref) and int(back.flatten(1).any(1).sum()) == 3


def test_no_sequences_no_slots():
    cache, scales = _cache(0, 2, 16, 16)
    states = _states(2, 2, 16, 16)
    gdn.gdn_state_store(states, _slots(0, 1), cache, scales)  # nothing can be kept
    assert not gdn.gdn_state_load(cache, scales, _slots(0, 1)).any()
    cache, scales = _cache(3, 2, 16, 16)
    kept = cache.clone()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    gdn.gdn_state_store(states[:0], none, cache, scales)
    assert gdn.gdn_state_load(cache, scales, none).shape == (0, 2, 16, 16)
    torch.cuda.synchronize()
    assert torch.equal(cache, kept)


def test_other_stream_and_graph():
    cache, scales = _cache(9, 3, 32, 64)
    states, slots = _states(4, 3, 32, 64), _slots(7, 0, 3, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gdn.gdn_state_store(states, slots, cache, scales, stream=side)
    got = gdn.gdn_state_load(cache, scales, slots, stream=side)
    torch.cuda.synchronize()
    _check(states, cache, scales, slots)
    assert torch.equal(got, cache[slots.long()].float() * scales[slots.long()][..., None])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_state_store(states, slots, cache, scales)
        got = gdn.gdn_state_load(cache, scales, slots)
    states.mul_(-2.0)
    slots.copy_(_slots(1, 2, 4, 8))
    graph.replay()
    torch.cuda.synchronize()
    _check(states, cache, scales, slots)
    assert torch.equal(got, cache[slots.long()].float() * scales[slots.long()][..., None])


def test_refusals():
    cache, scales = _cache(9, 3, 32, 64)
    states, slots = _states(4, 3, 32, 64), _slots(7, 0, 3, 5)
    ok = dict(states=states, slots=slots, cache=cache, scales=scales)
    for over in (dict(states=states[:3]), dict(states=states.bfloat16()), dict(states=states.transpose(2, 3)), dict(states=None),
                 dict(slots=slots.long()), dict(slots=slots[:, None]), dict(slots=slots.cpu()), dict(cache=cache.float()),
                 dict(cache=cache[:, :2]), dict(cache=cache.transpose(2, 3)), dict(cache=cache[0]), dict(scales=scales[:5]),
                 dict(scales=scales.bfloat16()), dict(scales=scales[..., None]), dict(cache=cache[..., :24].contiguous(), states=states[..., :24].contiguous())):
        with pytest.raises(gdn.GdnError):
            gdn.gdn_state_store(**{**ok, **over})
        if "states" not in over:
            with pytest.raises(gdn.GdnError):
                gdn.gdn_state_load(**{n: t for n, t in {**ok, **over}.items()})
    with pytest.raises(gdn.GdnError):
        gdn.gdn_state_load(cache, scales, slots, states=states[:2])
    with pytest.raises(TypeError):
        gdn.gdn_state_store(3, slots, cache, scales)
    gdn.gdn_state_store(**ok)
    torch.cuda.synchronize()
