"""Linear attention with a decay per head against its 64-bit definition."""

import itertools

import pytest
import torch

import gated_deltanet_linear_02_amd as gdn
import linattn_ref as ref
from gpu_util import note, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

BF, F32 = torch.bfloat16, torch.float32


def make(lens, hk, hv, dk, dv, io, *, gate=F32, per_head=False, init=True, state=F32, seed=0, extra=0, g=None):
    """Inputs on the GPU; `extra` tokens stand before and behind the sequences."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000 + seed)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    T, N = sum(lens) + 2 * extra, len(lens)
    d = dict(
        q=torch.nn.functional.normalize(normal(T, hk, dk), dim=-1).to(io),
        k=torch.nn.functional.normalize(normal(T, hk, dk), dim=-1).to(io),
        v=normal(T, hv, dv).to(io),
        cu=(torch.tensor([0] + list(lens)).cumsum(0) + extra).to(torch.int32).cuda(),
        init=(0.5 * normal(N, hv, dv, dk)).to(state) if init else None)
    speed = torch.exp(-6.0 * torch.rand(hv, device="cuda", generator=gen))
    d["g"] = (-speed if per_head else -speed * torch.nn.functional.softplus(normal(T, hv))).to(gate)
    if g is not None:
        d["g"] = g(d["g"]).to(gate)
    return d


def run_checked(d, lens, *, scale=0.7, state=F32, what="", start=0, **kw):
    T, hv, dv = d["v"].shape
    io = d["q"].dtype
    out = torch.full((T, hv, dv), float("nan"), dtype=io, device="cuda")
    fin = torch.full((len(lens), hv, dv, d["q"].shape[2]), float("nan"), dtype=state, device="cuda")
    note(f"linattn_prefill {what} lens={list(lens)[:8]} q={tuple(d['q'].shape)} v={tuple(d['v'].shape)} {io} {state}")
    o, f = gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], d["cu"], scale=scale, initial_state=d["init"],
                               final_state=fin, out=out, **kw)
    torch.cuda.synchronize()
    w_o, w_S, mag, A = ref.scan(d["q"], d["k"], d["v"], d["g"], lens, scale=scale, init=d["init"], start=start)
    t_o, t_S = ref.prefill_bounds(w_o, w_S, mag, A, io, state, max(lens, default=0), d["q"].shape[2])
    inside = slice(start, start + sum(lens))
    ref.check(o[inside], w_o[inside], t_o[inside], f"{what} out")
    ref.check(f, w_S, t_S, f"{what} state")
    rest = torch.cat([o[:inside.start], o[inside.stop:]])
    assert torch.isnan(rest).all(), "tokens outside the sequences were written"
    return o, f


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("dk,dv", itertools.product([16, 32, 64, 128], repeat=2))
def test_prefill_head_sizes(dk, dv, io):
    lens = [130, 1, 0, 67]
    d = make(lens, 2, 4, dk, dv, io, seed=dk + dv)
    run_checked(d, lens, what="head sizes")


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63], [64], [65], [127], [128], [129], [0, 5, 0],
                                  [0], [300, 64, 0, 1], [1] * 70, [3, 200, 7] * 40], ids=lambda x: "x".join(map(str, x[:4])))
def test_prefill_lengths(lens, io):
    d = make(lens, 1, 2, 64, 64, io, seed=len(lens) + sum(lens))
    run_checked(d, lens, what="lengths")


@pytest.mark.parametrize("hk,hv", [(1, 1), (3, 3), (1, 5), (3, 6), (2, 16), (16, 32), (9, 9)])
@pytest.mark.parametrize("lens", [[333], [90, 260, 1]])
def test_prefill_head_layouts(hk, hv, lens):
    d = make(lens, hk, hv, 32, 64, BF, seed=hk + hv)
    run_checked(d, lens, what="head layouts")


@pytest.mark.parametrize("io,gate,state,per_head,init", [
    (io, gate, state, per_head, init)
    for io, state in ((BF, F32), (BF, BF), (F32, F32)) for gate in (BF, F32)
    for per_head in (False, True) for init in (False, True)])
def test_prefill_types(io, gate, state, per_head, init):
    lens = [150, 71]
    d = make(lens, 2, 4, 64, 128, io, gate=gate, per_head=per_head, init=init, state=state, seed=7)
    run_checked(d, lens, state=state, what="types")


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("lens,hk,hv,d", [([5000], 1, 2, 64), ([4096], 16, 32, 128), ([9001], 1, 1, 128),
                                          ([2500, 64, 0, 3001, 1], 2, 2, 128), ([20011], 2, 2, 16)])
@pytest.mark.parametrize("hint", [False, True])
def test_prefill_long(lens, hk, hv, d, io, hint):
    x = make(lens, hk, hv, d, d, io, seed=sum(lens))
    run_checked(x, lens, what="long", max_seqlen=max(lens) if hint else None)


@pytest.mark.parametrize("io,state", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("lens,hk,hv,dk,dv,kinds", [
    ([90], 2, 4, 64, 64, "out"),                               # whole
    ([300], 2, 4, 64, 64, "state out"),                        # segments, each sums those before it
    ([2048], 4, 16, 128, 128, "state [join] out"),             # (whichever the types make cheaper)
    ([700, 1, 1500], 2, 8, 64, 128, "state out"),
    ([16001], 2, 4, 64, 64, "state join out"),                 # segments joined by a kernel
    ([9000, 0, 7000, 63], 1, 2, 128, 128, "state join out"),
    ([7000], 8, 16, 128, 128, "state [join] out"),
])
def test_prefill_each_way_of_splitting(lens, hk, hv, dk, dv, kinds, io, state):
    d = make(lens, hk, hv, dk, dv, io, state=state, seed=hv + sum(lens))
    gdn.timing_start(8)
    run_checked(d, lens, state=state, what=kinds, max_seqlen=max(lens))
    ran = " ".join(k.removeprefix("linattn_") for k, r in gdn.timing_stop().items() if r["count"])
    assert ran in (kinds.replace("[join] ", ""), kinds.replace("[join]", "join"))


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("name", ["zero", "reset", "strong", "growing", "constant"])
def test_prefill_gates(name, io):
    """No decay at all, states forgotten (-inf) now and then, decays that
    underflow within a block, growth, and per-head decays of all speeds."""
    lens = [700, 130]
    change = {"zero": torch.zeros_like,
              "reset": lambda g: torch.where(torch.rand_like(g) < 0.1, float("-inf"), g),
              "strong": lambda g: 60.0 * g,
              "growing": lambda g: -0.02 * g,
              "constant": lambda g: g}[name]
    d = make(lens, 2, 4, 64, 64, io, seed=11, g=change, per_head=name == "constant")
    run_checked(d, lens, what=f"gates {name}")


def test_prefill_leaves_other_tokens_alone():
    lens = [100, 0, 77]
    for io in (BF, F32):
        d = make(lens, 2, 4, 64, 64, io, extra=40, seed=3)
        # what stands in the tokens of no sequence does not matter
        for x in ("q", "k", "v"):
            d[x][:40] = float("nan")
            d[x][40 + sum(lens):] = float("inf")
        d["g"][:40] = float("nan")
        run_checked(d, lens, what="padded", start=40)


@pytest.mark.parametrize("long", [False, True])
def test_prefill_non_finite_values_stay_in_their_sequence(long):
    lens = [3000, 2000, 2900] if long else [70, 90, 130]
    d = make(lens, 1, 2, 64, 64, BF, seed=5)
    lo, hi = lens[0], lens[0] + lens[1]
    clean, fin = gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["init"])
    for x in ("q", "k", "v"):
        d[x][lo + 66] = float("nan")
    note("non-finite values in the second of three sequences")
    out, f = gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["init"])
    torch.cuda.synchronize()
    for a, b in ((out[:lo], clean[:lo]), (out[hi:], clean[hi:]), (f[0], fin[0]), (f[2], fin[2]),
                 (out[lo:lo + 2], clean[lo:lo + 2])):
        assert torch.equal(a, b)
    assert torch.isnan(out[lo + 66:hi]).all() and torch.isnan(f[1]).any()


def test_prefill_malformed_offsets_are_made_monotone():
    """[0, 300, 100, 500, 9999] reads as [0, 300, 300, 500, T]."""
    d = make([600], 2, 2, 64, 64, BF, init=False, seed=6)
    bad = torch.tensor([-5, 300, 100, 500, 9999], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 300, 300, 500, 600], dtype=torch.int32, device="cuda")
    note("malformed cu_seqlens")
    a = gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], bad)
    b = gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], good)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("io", [BF, F32])
def test_prefill_widest_rows(io):
    """hv dv = 2^22, the limit: rows of a block 16 MB (fp32) apart."""
    d = make([40, 9], 1, 1 << 15, 16, 128, io, seed=8)
    run_checked(d, [40, 9], what="widest rows")


@pytest.mark.parametrize("lens", [[150, 131], [3000]])
def test_prefill_past_32_bits(lens):
    """The last tokens of tensors of more than 2^31 elements."""
    T, hk, hv, dk, dv = (1 << 31) // (32 * 128) + 4000, 1, 32, 16, 128
    n = sum(lens)
    d = make(lens, hk, hv, dk, dv, BF, seed=n)
    big = {x: torch.zeros((T, *d[x].shape[1:]), dtype=d[x].dtype, device="cuda") for x in ("q", "k", "v", "g")}
    for x in big:
        big[x][T - n:] = d[x]
    out = torch.zeros_like(big["v"])
    cu = d["cu"] + (T - n)
    note(f"linattn_prefill {tuple(out.shape)} lens={lens}")
    o, f = gdn.linattn_prefill(big["q"], big["k"], big["v"], big["g"], cu, scale=0.7, initial_state=d["init"], out=out,
                               max_seqlen=None)
    torch.cuda.synchronize()
    w_o, w_S, mag, A = ref.scan(d["q"], d["k"], d["v"], d["g"], lens, scale=0.7, init=d["init"])
    t_o, t_S = ref.prefill_bounds(w_o, w_S, mag, A, BF, F32, max(lens), dk)
    ref.check(o[T - n:], w_o, t_o, "out")
    ref.check(f, w_S, t_S, "state")
    assert not o[:T - n].any()


@pytest.mark.parametrize("lens,hk,hv,d,ordered", [
    ([i % 4 for i in range(5000)], 1, 1, 16, True),
    ([7] * 300 + [6000] + [0, 1, 64, 65] * 40, 1, 2, 64, True),
    ([0] * 399 + [500], 1, 2, 32, False),
    ([500] + [0] * 400, 1, 2, 32, True),
], ids=["short", "one_long", "at_the_limit", "past_the_limit"])
def test_prefill_many_sequences(lens, hk, hv, d, ordered):
    x = make(lens, hk, hv, d, d, BF, seed=len(lens), extra=5)
    gdn.timing_start(8)
    run_checked(x, lens, what="many sequences", max_seqlen=max(lens), start=5)
    ran = [k for k, r in gdn.timing_stop().items() if r["count"]]
    assert ("schedule" in ran) == ordered


@pytest.mark.parametrize("long", [0, 4000])
def test_prefill_malformed_offsets_of_many_sequences(long):
    """Offsets that jump ahead, fall back and leave [0, T], against the running
    maximum of what they are clamped to."""
    N, T = 700, 2100 + long
    gen = torch.Generator().manual_seed(long)
    bad = (torch.arange(N + 1) * 3 + torch.randint(-40, 40, (N + 1,), generator=gen)).to(torch.int32)
    bad[450:] += long
    bad[-5:] = torch.tensor([T + 7, 2 ** 31 - 1, -2 ** 31, 0, T])
    good = bad.clamp(0, T).cummax(0).values.to(torch.int32)
    d = make([T], 1, 2, 32, 64, BF, init=False, seed=9)
    note("malformed cu_seqlens of many sequences")
    a = gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], bad.cuda())
    b = gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], good.cuda())
    torch.cuda.synchronize()
    first = int(good[0])
    assert torch.equal(a[0][first:], b[0][first:]) and torch.equal(a[1], b[1])
    w_o, w_S, mag, A = ref.scan(d["q"], d["k"], d["v"], d["g"], good.diff().tolist(), start=first)
    t_o, t_S = ref.prefill_bounds(w_o, w_S, mag, A, BF, F32, T, 32)
    ref.check(a[0][first:], w_o[first:], t_o[first:], "out")
    ref.check(a[1], w_S, t_S, "state")


@pytest.mark.parametrize("io,state", [(BF, F32), (BF, BF), (F32, F32)])
def test_prefill_in_place_state_and_repeat(io, state):
    lens = [2500, 33]
    d = make(lens, 1, 2, 64, 64, io, state=state, seed=8)
    o1, f1 = gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["init"])
    s = d["init"].clone()
    o2, f2 = gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=s, final_state=s)
    torch.cuda.synchronize()
    assert f2 is s and torch.equal(o1, o2) and torch.equal(f1, s)
    o3, none = gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["init"],
                                   write_final_state=False)
    assert none is None and torch.equal(o1, o3)


@pytest.mark.parametrize("io", [BF, F32])
def test_prefill_in_fragments_then_tokens(io):
    """A prompt in three fragments and then token by token ends where one
    prefill of it all does."""
    T, cuts = 2600, (0, 1100, 2533, 2590)
    d = make([T], 2, 4, 64, 64, io, init=False, seed=9)
    state, outs = None, []
    for lo, hi in zip(cuts, cuts[1:]):
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        o, state = gdn.linattn_prefill(*(d[x][lo:hi] for x in ("q", "k", "v", "g")), cu, initial_state=state)
        outs.append(o)
    for t in range(cuts[-1], T):
        outs.append(gdn.linattn_decode_step(*(d[x][t:t + 1] for x in ("q", "k", "v", "g")), state))
    torch.cuda.synchronize()
    w_o, w_S, mag, A = ref.scan(d["q"], d["k"], d["v"], d["g"], [T])
    t_o, t_S = ref.prefill_bounds(w_o, w_S, mag, A, io, F32, T, 64)
    ref.check(torch.cat(outs), w_o, t_o, "fragments out")
    ref.check(state, w_S, t_S, "fragments state")


def test_prefill_hint_below_the_longest_only_steers():
    """The hint is not checked against the offsets: one that is too small
    changes the split, not the answer."""
    lens = [3000, 10, 10, 10]
    d = make(lens, 1, 2, 64, 64, BF, seed=10)
    run_checked(d, lens, what="hint", max_seqlen=800)


def test_prefill_workspace_of_the_caller():
    lens = [4000, 4500]
    d = make(lens, 1, 2, 128, 128, BF, seed=12)
    need = gdn.linattn_prefill_workspace_size(2, sum(lens), 1, 2, 128, 128, BF)
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns
    run_checked(d, lens, what="workspace", workspace=ws[:need])
    assert (ws[need:] == 255).all()
    d2 = make(lens, 1, 2, 128, 128, BF, seed=13)
    run_checked(d2, lens, what="workspace again", workspace=ws[:need])
    if need > 256:
        with pytest.raises(gdn.GdnError) as e:
            gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], d["cu"], workspace=ws[:need - 256])
        assert e.value.status == 4


@pytest.mark.parametrize("lens,hv", [([300, 77, 5], 4), ([6000, 1, 2000], 2)])
def test_prefill_graph_replays(lens, hv):
    """Captured once, replayed on new data between eager work, each replay
    equal to the eager call."""
    runs = [make(lens, hv // 2, hv, 128, 128, BF, seed=20 + t) for t in range(4)]
    static = {x: y.clone() for x, y in runs[0].items()}
    out, fin = torch.empty_like(static["v"]), torch.empty_like(static["init"])
    need = gdn.linattn_prefill_workspace_size(len(lens), sum(lens), hv // 2, hv, 128, 128, BF)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def call(s, o, f):
        return gdn.linattn_prefill(s["q"], s["k"], s["v"], s["g"], s["cu"], initial_state=s["init"], final_state=f,
                                   out=o, workspace=ws)

    note(f"linattn_prefill graph lens={lens}")
    call(static, out, fin)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(static, out, fin)
    for t in range(1, 4):
        for x in static:
            static[x].copy_(runs[t][x])
        note(f"replay {t}")
        graph.replay()
        torch.cuda.synchronize()
        o_g, f_g = out.clone(), fin.clone()
        o_e, f_e = call(runs[t], torch.empty_like(out), torch.empty_like(fin))
        torch.cuda.synchronize()
        assert torch.equal(o_g, o_e) and torch.equal(f_g, f_e)


def test_prefill_two_streams():
    """Two calls at once, each with its own workspace, on streams of their own."""
    lens = [5000]
    runs = [make(lens, 1, 2, 128, 128, BF, seed=30 + t) for t in range(2)]
    want = [gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["init"]) for d in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    note("two streams")
    got = [[gdn.linattn_prefill(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["init"], stream=s)
            for _ in range(5)] for d, s in zip(runs, streams)]
    torch.cuda.synchronize()
    for (o, f), g in zip(want, got):
        for o2, f2 in g:
            assert torch.equal(o, o2) and torch.equal(f, f2)


# ------------------------------------------------------------------ decode

def decode_inputs(B, hk, hv, dk, dv, io, gate, state, per_head, pool, seed):
    d = make([1] * B, hk, hv, dk, dv, io, gate=gate, per_head=per_head, init=False, seed=seed)
    d["state"] = (0.5 * torch.randn(pool, hv, dv, dk, device="cuda")).to(state)
    d["slots"] = torch.randperm(pool, device="cuda")[:B].to(torch.int32)
    return d


def decode_checked(d, slots, **kw):
    B, hv, dv = d["v"].shape
    dk = d["q"].shape[2]
    old = d["state"].clone()
    at = torch.arange(B, device="cuda") if slots is None else slots.long()
    there = (at >= 0) & (at < old.shape[0])
    io, state = d["q"].dtype, old.dtype
    w_o, w_S, mag, A = ref.scan(d["q"], d["k"], d["v"], d["g"], [1] * B, scale=0.7,
                                init=old[torch.where(there, at, 0)])
    t_o, t_S = ref.prefill_bounds(w_o, w_S, mag, A, io, state, 1, dk)
    out = torch.full((B, hv, dv), float("nan"), dtype=io, device="cuda")
    note(f"linattn_decode_step q={tuple(d['q'].shape)} v={tuple(d['v'].shape)} {io} {state} slots={slots is not None}")
    gdn.linattn_decode_step(d["q"], d["k"], d["v"], d["g"], d["state"], scale=0.7, state_slots=slots, out=out, **kw)
    torch.cuda.synchronize()
    new = kw.get("state_out", d["state"])
    ref.check(out[there], w_o[there], t_o[there], "decode out")
    assert (out[~there] == 0).all()
    ref.check(new[at[there]], w_S[there], t_S[there], "decode state")
    if new is not d["state"]:
        assert torch.equal(d["state"], old)
    else:
        kept = torch.ones(old.shape[0], dtype=torch.bool, device="cuda")
        kept[at[there]] = False
        assert torch.equal(new[kept], old[kept])
    return out


@pytest.mark.parametrize("io,state", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("dk,dv", itertools.product([16, 32, 64, 128], repeat=2))
def test_decode_head_sizes(dk, dv, io, state):
    d = decode_inputs(3, 2, 4, dk, dv, io, F32, state, False, 5, dk + dv)
    decode_checked(d, d["slots"])


@pytest.mark.parametrize("B,hk,hv,gate,per_head,use_slots", [
    (1, 16, 32, BF, False, False), (64, 16, 32, BF, False, True), (7, 1, 5, F32, True, True),
    (2, 3, 3, BF, True, False), (300, 1, 2, F32, False, True)])
@pytest.mark.parametrize("state", [F32, BF])
def test_decode_layouts(B, hk, hv, gate, per_head, use_slots, state):
    d = decode_inputs(B, hk, hv, 128, 128, BF, gate, state, per_head, B + 3, B)
    decode_checked(d, d["slots"] if use_slots else None)


@pytest.mark.parametrize("state", [F32, BF])
def test_decode_second_pool_and_skipped_slots(state):
    d = decode_inputs(6, 2, 4, 128, 64, BF, BF, state, False, 9, 1)
    slots = d["slots"].clone()
    slots[1], slots[4] = -1, 9  # no such slots
    second = torch.full_like(d["state"], float("nan"))
    out = decode_checked(d, slots, state_out=second)
    kept = torch.ones(9, dtype=torch.bool, device="cuda")
    kept[slots[[0, 2, 3, 5]].long()] = False
    assert torch.isnan(second[kept].float()).all(), "slots of no sequence were written"
    # in place: the same bits
    again = gdn.linattn_decode_step(d["q"], d["k"], d["v"], d["g"], d["state"], scale=0.7, state_slots=slots)
    used = slots[[0, 2, 3, 5]].long()
    assert torch.equal(again, out) and torch.equal(d["state"][used], second[used])


def test_decode_pool_beyond_32_bits():
    d = decode_inputs(3, 16, 32, 128, 128, BF, F32, BF, False, 4200, 5)
    decode_checked(d, torch.tensor([4199, 0, 4097], dtype=torch.int32, device="cuda"))


def test_decode_forgets_at_minus_infinity():
    d = decode_inputs(2, 1, 2, 64, 64, BF, F32, F32, False, 2, 2)
    d["g"][0] = float("-inf")
    decode_checked(d, None)


def test_decode_graph_replays():
    steps = [decode_inputs(8, 2, 4, 128, 128, BF, BF, F32, False, 10, 40 + t) for t in range(4)]
    static = {x: y.clone() for x, y in steps[0].items() if y is not None}
    eager = static["state"].clone()
    out = torch.empty_like(static["v"])
    note("linattn_decode_step graph")
    warm = static["state"].clone()
    gdn.linattn_decode_step(static["q"], static["k"], static["v"], static["g"], warm, state_slots=static["slots"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.linattn_decode_step(static["q"], static["k"], static["v"], static["g"], static["state"],
                                state_slots=static["slots"], out=out)
    for t in range(1, 4):
        for x in ("q", "k", "v", "g", "slots"):
            static[x].copy_(steps[t][x])
        note(f"replay {t}")
        graph.replay()
        s = steps[t]
        want = gdn.linattn_decode_step(s["q"], s["k"], s["v"], s["g"], eager, state_slots=s["slots"])
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(static["state"], eager)


# ----------------------------------------------------------- used together

@pytest.mark.parametrize("code", [torch.int8, torch.float8_e4m3fn])
def test_serving_run(code):
    """Prompts are prefilled, their states put into the 8-bit cache, taken up
    by other requests (one of them twice), continued by a prompt fragment and
    then decoded, against the same steps in 64 bits."""
    hk, hv, d, lens = 2, 4, 128, [700, 65]
    x = make(lens, hk, hv, d, d, BF, init=False, seed=50)
    note("serving run")
    _, fin = gdn.linattn_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"])
    cache = torch.zeros(8, hv, d, d, dtype=torch.uint8, device="cuda").view(code)
    scales = torch.zeros(8, hv, d, device="cuda")
    entries = torch.tensor([6, 2], dtype=torch.int32, device="cuda")
    gdn.state_cache_write(fin, cache, scales, entries=entries)
    pool = torch.full((5, hv, d, d), float("nan"), device="cuda")
    slots = torch.tensor([4, 0, 3], dtype=torch.int32, device="cuda")
    gdn.state_cache_read(cache, scales, pool, entries=torch.tensor([2, 6, 6], dtype=torch.int32, device="cuda"),
                         slots=slots)
    began = pool[slots.long()].clone()
    codes, scale = ref.quantise(fin[[1, 0, 0]], code)
    assert torch.equal(began, (codes.float() * scale[..., None]))
    frag = make([40, 3, 129], hk, hv, d, d, BF, init=False, seed=51)
    _, state = gdn.linattn_prefill(frag["q"], frag["k"], frag["v"], frag["g"], frag["cu"], initial_state=began)
    pool[slots.long()] = state
    w_o, w_S, _, A = ref.scan(frag["q"], frag["k"], frag["v"], frag["g"], [40, 3, 129], init=began)
    for t in range(5):
        y = make([1] * 3, hk, hv, d, d, BF, init=False, seed=60 + t)
        out = gdn.linattn_decode_step(y["q"], y["k"], y["v"], y["g"], pool, state_slots=slots)
        w_o, w_S, mag, _ = ref.scan(y["q"], y["k"], y["v"], y["g"], [1] * 3, init=w_S)
        A = y["g"].double().exp()[..., None, None] * A + \
            y["v"].double().abs()[..., None] * y["k"].double().abs().repeat_interleave(2, 1)[..., None, :]
        mag = (A * y["q"].double().abs().repeat_interleave(2, 1)[..., None, :]).sum(-1)
        t_o, t_S = ref.prefill_bounds(w_o, w_S, mag, A, BF, F32, 129 + 5, d)
        ref.check(out, w_o, t_o, f"decode {t}")
    ref.check(pool[slots.long()], w_S, t_S, "states at last")
