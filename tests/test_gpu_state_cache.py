"""States written to the 8-bit cache and read back: every code and scale
equal to the exact quotients' (64 bits)."""

import pytest
import torch

import gated_deltanet_linear_02_amd as gdn
import linattn_ref as ref
from gpu_util import note, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

I8, E4M3 = torch.int8, torch.float8_e4m3fn
BF, F32 = torch.bfloat16, torch.float32


def empty_cache(entries, hv, dv, dk, code):
    cache = torch.full((entries, hv, dv, dk), 0x55, dtype=torch.uint8, device="cuda").view(code)
    return cache, torch.full((entries, hv, dv), -7.0, device="cuda")


def values(cache):
    return cache.float().double()


def check_rows(cache, scales, entry, x, code):
    """Entry `entry` holds the states x."""
    codes, scale = ref.quantise(x, code)
    got = scales[entry]
    assert torch.equal(torch.isnan(got), torch.isnan(scale))
    assert torch.equal(got.nan_to_num(), scale.nan_to_num()), "scales differ"
    bad = (values(cache.view(torch.uint8)[entry].view(code)) != codes).nonzero()
    assert not len(bad), f"{len(bad)} codes differ, first at {bad[0].tolist()}"


def rows(shape, dtype, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    size = torch.exp(3.0 * torch.randn(*shape[:-1], 1, device="cuda", generator=gen))
    return (size * torch.randn(shape, device="cuda", generator=gen)).to(dtype)


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("hv,dv,dk", [(32, 128, 128), (1, 16, 16), (3, 16, 32), (5, 64, 16), (2, 32, 64), (7, 128, 32),
                                      (1, 16, 128)])
def test_write_and_read(hv, dv, dk, dtype, code):
    n, pool, entries = 5, 7, 9
    state = rows((pool, hv, dv, dk), dtype, hv + dk)
    cache, scales = empty_cache(entries, hv, dv, dk, code)
    slots = torch.tensor([6, 0, 3, 5, 3], dtype=torch.int32, device="cuda")  # one state twice
    to = torch.tensor([8, 1, 2, 0, 4], dtype=torch.int32, device="cuda")
    note(f"state_cache hv={hv} dv={dv} dk={dk} {dtype} {code}")
    gdn.state_cache_write(state, cache, scales, slots=slots, entries=to)
    torch.cuda.synchronize()
    for s, e in zip(slots.tolist(), to.tolist()):
        check_rows(cache, scales, e, state[s], code)
    for e in (3, 5, 6, 7):
        assert (scales[e] == -7).all() and (cache.view(torch.uint8)[e] == 0x55).all()
    back = torch.full((pool, hv, dv, dk), float("nan"), dtype=dtype, device="cuda")
    at = torch.tensor([5, 0, 2, 6], dtype=torch.int32, device="cuda")
    of = torch.tensor([1, 8, 8, 4], dtype=torch.int32, device="cuda")  # one entry twice
    gdn.state_cache_read(cache, scales, back, entries=of, slots=at)
    torch.cuda.synchronize()
    raw = cache.view(torch.uint8)[of.long()].view(code).float()
    assert torch.equal(back[at.long()], (raw * scales[of.long()][..., None]).to(dtype))
    assert torch.isnan(back[[1, 3, 4]].float()).all()


@pytest.mark.parametrize("code", [I8, E4M3])
def test_ties_and_their_neighbours(code):
    """Quotients on the middle between two codes, and one unit in the last
    place to either side of it, for scales that are powers of two (exact
    ties) and that are not."""
    top = 127.0 if code == I8 else 448.0
    vals = torch.arange(128.0) if code == I8 else torch.arange(127, dtype=torch.uint8).view(E4M3).float()
    mid = ((vals[1:] + vals[:-1]) / 2).cuda()
    out = []
    for unit in (1.0, 0.5, 2.0 ** -40, 0.1, 1.7, 3.3e-7, 12345.678, 2.0 ** -70 * 1.3, 1e-36, 2.0 ** 100 * 1.1):
        scale = torch.tensor(unit, device="cuda") * top / top
        amax = scale * top
        m = (mid.double() * (amax / top).double()).float()
        for x in (m, torch.nextafter(m, m.new_full((), float("inf"))), torch.nextafter(m, m.new_zeros(()))):
            x = torch.cat([x, -x])
            x = torch.cat([x, x.new_zeros(-len(x) % 127)]).view(-1, 127)
            out.append(torch.cat([amax.expand(len(x), 1), x], 1))
    state = torch.cat(out)
    state = torch.cat([state, state.new_zeros(-len(state) % 16, 128)]).view(1, -1, 16, 128).contiguous()
    hv = state.shape[1]
    cache, scales = empty_cache(1, hv, 16, 128, code)
    note(f"ties {code}")
    gdn.state_cache_write(state, cache, scales)
    torch.cuda.synchronize()
    check_rows(cache, scales, 0, state[0], code)


@pytest.mark.parametrize("code", [I8, E4M3])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_special_rows(dtype, code):
    state = rows((1, 2, 16, 64), dtype, 3)
    state[0, 0, 0] = 0
    state[0, 0, 1, 5] = float("nan")
    state[0, 0, 2, 63] = float("inf")
    state[0, 0, 3, 0] = float("-inf")
    state[0, 0, 4] *= 0
    state[0, 0, 4, 9] = torch.finfo(dtype).max
    state[0, 0, 5] = -state[0, 0, 5].abs()
    state[0, 0, 6] = -0.0
    tiny = rows((64,), F32, 4)
    state[0, 0, 7] = (tiny * 1e-30).to(dtype)
    state[0, 0, 8] = (tiny * 1e-36).to(dtype)
    state[0, 0, 9] = (tiny * 1e-38).to(dtype)
    state[0, 0, 10] = (tiny / tiny.abs().max() * 1e38).to(dtype)
    state[0, 0, 11] = 1e-45 if dtype == F32 else 1e-40
    cache, scales = empty_cache(1, 2, 16, 64, code)
    note(f"special rows {dtype} {code}")
    gdn.state_cache_write(state, cache, scales)
    back = torch.empty_like(state)
    gdn.state_cache_read(cache, scales, back)
    torch.cuda.synchronize()
    check_rows(cache, scales, 0, state[0], code)
    for r in (1, 2, 3):
        assert torch.isnan(back[0, 0, r].float()).all()
    assert (back[0, 0, 0] == 0).all() and (back[0, 0, 6] == 0).all()
    assert torch.isfinite(back[0, 1].float()).all() and torch.isfinite(back[0, 0, 4:].float()).all()


def test_items_outside_the_pools_are_skipped():
    state = rows((3, 2, 16, 32), F32, 5)
    cache, scales = empty_cache(3, 2, 16, 32, I8)
    slots = torch.tensor([0, -1, 3, 2, 1], dtype=torch.int32, device="cuda")
    entries = torch.tensor([2, 0, 1, 3, -2147483648], dtype=torch.int32, device="cuda")
    note("items outside the pools")
    gdn.state_cache_write(state, cache, scales, slots=slots, entries=entries)
    back = torch.full_like(state, float("nan"))
    gdn.state_cache_read(cache, scales, back, slots=slots, entries=entries)
    torch.cuda.synchronize()
    check_rows(cache, scales, 2, state[0], I8)
    assert (scales[:2] == -7).all() and (cache[:2] == 0x55).all()
    assert torch.isnan(back[1:]).all() and torch.isfinite(back[0]).all()


def test_many_items_and_a_pool_beyond_32_bits():
    """2,500 entries of 32 x 128 x 128 codes are 1.3 GB; their fp32 states
    (5.2 GB) lie beyond what 32 bits address."""
    hv, d, pool = 32, 128, 2500
    state = torch.zeros(pool, hv, d, d, device="cuda")
    state[pool - 1] = rows((hv, d, d), F32, 6)
    state[17] = rows((hv, d, d), F32, 7)
    cache = torch.zeros(pool, hv, d, d, dtype=torch.int8, device="cuda")
    scales = torch.full((pool, hv, d), -7.0, device="cuda")
    slots = torch.arange(pool - 1, -1, -1, dtype=torch.int32, device="cuda")
    note("large pools")
    gdn.state_cache_write(state, cache, scales, slots=slots)
    torch.cuda.synchronize()
    check_rows(cache, scales, 0, state[pool - 1], I8)
    check_rows(cache, scales, pool - 18, state[17], I8)
    assert int((scales != 0).sum()) == 2 * hv * d
    gdn.state_cache_read(cache, scales, state, slots=torch.arange(pool, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(state[pool - 18], cache[pool - 18].float() * scales[pool - 18][..., None])
    assert not state[pool - 1].any()


def test_graph_replays():
    state = rows((4, 4, 64, 64), F32, 8)
    cache, scales = empty_cache(4, 4, 64, 64, E4M3)
    back = torch.empty_like(state)
    order = torch.tensor([2, 0, 3, 1], dtype=torch.int32, device="cuda")

    def call(s, c, sc, b):
        gdn.state_cache_write(s, c, sc, entries=order)
        gdn.state_cache_read(c, sc, b, entries=order)

    note("state cache graph")
    call(state, cache, scales, back)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(state, cache, scales, back)
    for t in range(3):
        state.copy_(rows((4, 4, 64, 64), F32, 20 + t))
        note(f"replay {t}")
        graph.replay()
        torch.cuda.synchronize()
        c2, s2 = empty_cache(4, 4, 64, 64, E4M3)
        b2 = torch.empty_like(back)
        call(state, c2, s2, b2)
        torch.cuda.synchronize()
        assert torch.equal(back, b2) and torch.equal(scales, s2)
        assert torch.equal(cache.view(torch.uint8), c2.view(torch.uint8))


def test_states_of_the_delta_rule():
    """States of the gated delta rule go through the cache too."""
    T, hk, hv, d = 100, 2, 4, 64
    q, v = torch.randn(T, hk, d, device="cuda").to(BF), torch.randn(T, hv, d, device="cuda").to(BF)
    k = torch.nn.functional.normalize(torch.randn(T, hk, d, device="cuda"), dim=-1).to(BF)
    g, beta = -torch.rand(T, hv, device="cuda"), torch.rand(T, hv, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    _, state = gdn.prefill(q, k, v, g, beta, cu)
    cache, scales = empty_cache(1, hv, d, d, I8)
    gdn.state_cache_write(state, cache, scales)
    back = torch.empty_like(state)
    gdn.state_cache_read(cache, scales, back)
    # half a code of each row's scale, and the product's rounding
    assert ((back - state).abs() <= (0.5 + 2.0 ** -16) * scales[..., None]).all()
    out = gdn.decode_step(q[:1], k[:1], v[:1], g[:1], beta[:1], back)
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all()
