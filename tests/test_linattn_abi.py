"""Argument checks of the linear attention and the state cache (host only)."""

import pytest
import torch

import gated_deltanet_linear_02_amd as gdn
import linattn_ref as ref
from test_abi import (ALIAS, BAD_SHAPE, BAD_VALUE, BF16, F32, FAKE, MISALIGNED, NULL_ARG, OK, UNSUPPORTED,
                      WORKSPACE, lib, no_gpu)  # noqa: F401

G = 1 << 32


def _prefill(lib, **kw):
    a = dict(q=FAKE, k=FAKE + G, v=FAKE + 2 * G, g=FAKE + 3 * G, cu=FAKE + 4 * G, n=1, T=128, longest=0, hk=2, hv=4,
             dk=64, dv=128, scale=1.0, io=BF16, gate=F32, per_head=0, s0=None, sf=None, state=F32, out=FAKE + 5 * G,
             ws=FAKE + 6 * G, ws_bytes=1 << 32, stream=None)
    a.update(kw)
    return lib.gdn_linattn_prefill(*a.values())


@no_gpu
@pytest.mark.parametrize("want,kw", [
    (NULL_ARG, dict(q=None)), (NULL_ARG, dict(k=None)), (NULL_ARG, dict(v=None)), (NULL_ARG, dict(g=None)),
    (NULL_ARG, dict(cu=None)), (NULL_ARG, dict(out=None)),
    (BAD_SHAPE, dict(n=0)), (BAD_SHAPE, dict(T=-1)), (BAD_SHAPE, dict(T=1 << 31)), (BAD_SHAPE, dict(hk=3)),
    (BAD_SHAPE, dict(hk=0)), (BAD_SHAPE, dict(hv=0)),
    (UNSUPPORTED, dict(dk=96)), (UNSUPPORTED, dict(dv=256)), (UNSUPPORTED, dict(dk=0)), (UNSUPPORTED, dict(io=2)),
    (UNSUPPORTED, dict(gate=-1)), (UNSUPPORTED, dict(state=7)), (UNSUPPORTED, dict(io=F32, state=BF16)),
    (UNSUPPORTED, dict(n=1 << 23)),
    (BAD_VALUE, dict(per_head=2)), (BAD_VALUE, dict(longest=-1)), (BAD_VALUE, dict(longest=129)),
    (BAD_VALUE, dict(n=2, longest=63)),
    (MISALIGNED, dict(q=FAKE + 8)), (MISALIGNED, dict(k=FAKE + G + 2)), (MISALIGNED, dict(v=FAKE + 2 * G + 4)),
    (MISALIGNED, dict(out=FAKE + 5 * G + 8)), (MISALIGNED, dict(s0=FAKE + 7 * G + 4)),
    (MISALIGNED, dict(sf=FAKE + 7 * G + 4)),
    (ALIAS, dict(out=FAKE)), (ALIAS, dict(out=FAKE + 2 * G)), (ALIAS, dict(sf=FAKE + G)),
    (ALIAS, dict(out=FAKE + 3 * G)), (ALIAS, dict(sf=FAKE + 5 * G)), (ALIAS, dict(s0=FAKE + 5 * G)),
    (ALIAS, dict(s0=FAKE + 7 * G, sf=FAKE + 7 * G + 4096)),
], ids=str)
def test_prefill_refusals(lib, want, kw):  # noqa: F811
    assert _prefill(lib, **kw) == want


@no_gpu
def test_prefill_workspace_refusals(lib):  # noqa: F811
    size = lib.gdn_linattn_prefill_workspace_size
    assert size(1, 100000, 0, 2, 4, 128, 128, BF16) >= 256
    for bad in ((0, 10, 0, 2, 4, 64, 64, BF16), (1, -1, 0, 2, 4, 64, 64, BF16), (1, 10, 0, 3, 4, 64, 64, BF16),
                (1, 10, 0, 2, 4, 65, 64, BF16), (1, 10, 0, 2, 4, 64, 64, 3), (1, 10, 11, 2, 4, 64, 64, BF16)):
        assert size(*bad) == 0
    need = size(1, 100000, 0, 2, 4, 64, 128, BF16)
    if need > 256:
        assert _prefill(lib, T=100000, ws=None) == WORKSPACE
        assert _prefill(lib, T=100000, ws_bytes=need - 1) == WORKSPACE
        assert _prefill(lib, T=100000, ws=FAKE + 6 * G + 16) == WORKSPACE
        assert _prefill(lib, T=100000, ws=FAKE + 2 * G) == ALIAS
        assert _prefill(lib, T=100000, ws=FAKE + 5 * G) == ALIAS


@no_gpu
def test_size_limits(lib):  # noqa: F811
    """Rows, tokens and launches past what 32 bits address are refused, and
    nothing below the stated limits is."""
    size = lib.gdn_linattn_prefill_workspace_size
    top = (1 << 31) - 65
    assert size(1, top, 0, 1, 1, 16, 16, BF16) >= 256 and size(1, top + 1, 0, 1, 1, 16, 16, BF16) == 0
    assert size(1, 64, 0, 1, 1 << 15, 16, 128, BF16) >= 256 and size(1, 64, 0, 1, (1 << 15) + 1, 16, 128, BF16) == 0
    assert size(1, 64, 0, 1 << 15, 1 << 16, 128, 64, BF16) >= 256
    assert size(1, 64, 0, 1 << 16, 1 << 16, 128, 64, BF16) == 0
    for T in (0, 1, 1 << 20, 1 << 23, top):
        for hk, hv in ((1, 1), (1, 8), (16, 128)):
            for dk, dv in ((16, 16), (128, 128)):
                n = (1 << 23) // hv
                assert size(n, T, 0, hk, hv, dk, dv, BF16) >= 256
                assert size(4 * n, T, 0, hk, hv, dk, dv, F32) == 0
    assert _prefill(lib, T=top + 1) == UNSUPPORTED
    assert _decode(lib, batch=1 << 23) == UNSUPPORTED
    assert _decode(lib, batch=1 << 21, dk=128, sdt=BF16) == UNSUPPORTED
    assert _cache(lib, True, n=1 << 23) == UNSUPPORTED


def _decode(lib, **kw):
    a = dict(q=FAKE, k=FAKE + G, v=FAKE + 2 * G, g=FAKE + 3 * G, batch=4, hk=2, hv=4, dk=64, dv=128, scale=1.0,
             io=BF16, gate=F32, per_head=0, state=FAKE + 4 * G, state_out=None, sdt=F32, slots=FAKE + 5 * G, pool=8,
             out=FAKE + 6 * G, stream=None)
    a.update(kw)
    return lib.gdn_linattn_decode_step(*a.values())


@no_gpu
@pytest.mark.parametrize("want,kw", [
    (OK, dict(batch=0)), (NULL_ARG, dict(q=None)), (NULL_ARG, dict(g=None)), (NULL_ARG, dict(state=None)),
    (NULL_ARG, dict(out=None)), (BAD_SHAPE, dict(batch=-1)), (BAD_SHAPE, dict(hk=3)), (BAD_SHAPE, dict(pool=-1)),
    (BAD_SHAPE, dict(slots=None, pool=3)), (UNSUPPORTED, dict(dk=48)), (UNSUPPORTED, dict(dv=8)),
    (UNSUPPORTED, dict(io=F32, sdt=BF16)), (UNSUPPORTED, dict(sdt=2)), (BAD_VALUE, dict(per_head=-1)),
    (UNSUPPORTED, dict(batch=1 << 30)),
    (MISALIGNED, dict(state=FAKE + 4 * G + 8)), (MISALIGNED, dict(state_out=FAKE + 7 * G + 8)),
    (MISALIGNED, dict(v=FAKE + 2 * G + 2)),
    (ALIAS, dict(out=FAKE + 4 * G)), (ALIAS, dict(state=FAKE)), (ALIAS, dict(state_out=FAKE + 4 * G + 65536)),
    (ALIAS, dict(state_out=FAKE + 6 * G)), (ALIAS, dict(state_out=FAKE + 5 * G)), (ALIAS, dict(out=FAKE + 3 * G)),
], ids=str)
def test_decode_refusals(lib, want, kw):  # noqa: F811
    assert _decode(lib, **kw) == want


def _cache(lib, write, **kw):
    a = dict(state=FAKE, sdt=F32, slots=FAKE + G, pool=8, cache=FAKE + 2 * G, code=0, scales=FAKE + 3 * G,
             entries=FAKE + 4 * G, size=8, n=4, hv=4, dk=64, dv=128, stream=None)
    a.update(kw)
    tail = (a["n"], a["hv"], a["dk"], a["dv"], a["stream"])
    if write:
        return lib.gdn_state_cache_write(a["state"], a["sdt"], a["slots"], a["pool"], a["cache"], a["code"],
                                         a["scales"], a["entries"], a["size"], *tail)
    return lib.gdn_state_cache_read(a["cache"], a["code"], a["scales"], a["entries"], a["size"], a["state"],
                                    a["sdt"], a["slots"], a["pool"], *tail)


@no_gpu
@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("want,kw", [
    (OK, dict(n=0)), (NULL_ARG, dict(state=None)), (NULL_ARG, dict(cache=None)), (NULL_ARG, dict(scales=None)),
    (BAD_SHAPE, dict(n=-1)), (BAD_SHAPE, dict(pool=-1)), (BAD_SHAPE, dict(size=-1)), (BAD_SHAPE, dict(hv=0)),
    (BAD_SHAPE, dict(slots=None, pool=3)), (BAD_SHAPE, dict(entries=None, size=3)),
    (UNSUPPORTED, dict(dk=8)), (UNSUPPORTED, dict(dv=100)), (UNSUPPORTED, dict(sdt=2)), (UNSUPPORTED, dict(code=2)),
    (UNSUPPORTED, dict(hv=1 << 26)), (UNSUPPORTED, dict(n=1 << 30)),
    (MISALIGNED, dict(state=FAKE + 4)), (MISALIGNED, dict(cache=FAKE + 2 * G + 1)),
    (ALIAS, dict(cache=FAKE)), (ALIAS, dict(scales=FAKE)), (ALIAS, dict(scales=FAKE + 2 * G)),
], ids=str)
def test_cache_refusals(lib, write, want, kw):  # noqa: F811
    assert _cache(lib, write, **kw) == want


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refusals(lib):  # noqa: F811
    """Shapes, types and devices are checked before the library is called."""
    q, v, g = _t(4, 2, 64), _t(4, 4, 128), _t(4, 4, dtype=torch.float32)
    cu, st = torch.tensor([0, 4], dtype=torch.int32), _t(1, 4, 128, 64, dtype=torch.float32)
    prefill, decode = gdn.linattn_prefill, gdn.linattn_decode_step
    with pytest.raises(ValueError, match="k has shape"):
        prefill(q, q[:3], v, g, cu)
    with pytest.raises(ValueError, match="g has shape"):
        prefill(q, q, v, g[:, :2], cu)
    with pytest.raises(ValueError, match="g has shape"):
        prefill(q, q, v, g[0, :3], cu)
    with pytest.raises(TypeError, match="v is"):
        prefill(q, q, v.float(), g, cu)
    with pytest.raises(TypeError, match="cu_seqlens"):
        prefill(q, q, v, g, cu.long())
    with pytest.raises(TypeError, match="unsupported dtype"):
        prefill(q.half(), q.half(), v.half(), g, cu)
    with pytest.raises(ValueError, match="initial_state has shape"):
        prefill(q, q, v, g, cu, initial_state=st[:, :2])
    with pytest.raises(TypeError, match="one dtype"):
        prefill(q, q, v, g, cu, initial_state=st, final_state=st.bfloat16())
    with pytest.raises(ValueError, match="expected cpu|is on cpu"):
        prefill(q, q, v, g, cu)
    with pytest.raises(TypeError, match="state must be"):
        decode(q, q, v, g, st.half())
    with pytest.raises(ValueError, match="state has shape"):
        decode(q, q, v, g, st.transpose(2, 3))
    with pytest.raises(TypeError, match="state_out is"):
        decode(q, q, v, g, st, state_out=st.bfloat16())
    with pytest.raises(TypeError, match="state_slots must be int32"):
        decode(q, q, v, g, st, state_slots=torch.zeros(4, dtype=torch.long))
    with pytest.raises(ValueError, match="is on cpu"):
        decode(q, q, v, g, st)
    cache, scales = _t(2, 4, 128, 64, dtype=torch.int8), _t(2, 4, 128, dtype=torch.float32)
    for call in (lambda **k: gdn.state_cache_write(k["state"], k["cache"], k["scales"], **k["at"]),
                 lambda **k: gdn.state_cache_read(k["cache"], k["scales"], k["state"], **k["at"])):
        ok = dict(state=st, cache=cache, scales=scales, at={})
        for err, match, change in (
                (TypeError, "state must be", dict(state=st.half())), (TypeError, "cache must be", dict(cache=cache.float())),
                (ValueError, "cache has shape", dict(cache=cache[..., :32])),
                (ValueError, "scales has shape", dict(scales=scales[:1])),
                (TypeError, "scales is", dict(scales=scales.double())),
                (ValueError, "entries has shape", dict(at=dict(slots=cu, entries=cu[:1]))),
                (TypeError, "slots must be int32", dict(at=dict(slots=cu.long()))),
                (ValueError, "is on cpu", {})):
            with pytest.raises(err, match=match):
                call(**{**ok, **change})


def test_reference_codes():
    """The tests' own 64-bit rounding, on values worked by hand."""
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 3.49]])
    codes, scale = ref.quantise(x, torch.int8)
    assert scale.tolist() == [1.0] and codes.tolist() == [[127, 0, 2, 2, 0, -2, 126, 3]]
    x = torch.tensor([[448.0, 17.0, 19.0, 0.001, -2.0 ** -10, 3 * 2.0 ** -10, 432.0, 431.9]])
    codes, scale = ref.quantise(x, torch.float8_e4m3fn)
    assert scale.tolist() == [1.0]
    assert codes.tolist() == [[448, 16, 20, 2.0 ** -9, 0, 2.0 ** -8, 448, 416]]
    codes, scale = ref.quantise(torch.tensor([[0.0, 0.0], [1.0, float("nan")]]), torch.int8)
    assert codes.tolist() == [[0, 0], [0, 0]] and scale[0] == 0 and scale[1].isnan()


def test_reference_scan():
    """Two tokens of one head by hand."""
    q = torch.tensor([[[1.0, 2.0]], [[3.0, 1.0]]])
    k = torch.tensor([[[1.0, 0.0]], [[1.0, -1.0]]])
    v = torch.tensor([[[2.0]], [[4.0]]])
    g = torch.tensor([[0.0], [0.5]], dtype=torch.float64).log()
    out, S, mag, A = ref.scan(q, k, v, g, [2], scale=2.0, init=torch.tensor([[[[5.0, 7.0]]]]))
    assert out.flatten().tolist() == [4.0, 2 * (5 * 3 - 4)] and S.flatten().tolist() == [5.0, -4.0]
    assert mag.flatten().tolist() == [4.0, 2 * (5 * 3 + 4)] and A.flatten().tolist() == [5.0, 4.0]
