"""CPU checks of the mixture-of-experts operators: the header's symbols, structs and constants, and every refusal, which
comes before any device work."""

import ctypes
import os
import re
import struct

import pytest

from gemv_tq2_g128_amd import moe, tq2

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7F0000000000           # never dereferenced


def at(i):
    return BASE + (i << 44)


ROUTE = dict(x=at(1), weight=at(2), bias=at(3), weights=at(4), ids=at(5), tokens=4, hidden=64, experts=16, top_k=4,
             act_type=0, weight_type=2, scoring=0, renormalize=1, scale=1.0, workspace=at(6), workspace_bytes=1 << 40)
EXPERTS = dict(x=at(1), residual=at(2), out=at(3), ids=at(4), weights=at(5), gate_up=at(6), gate_up_scales=at(7),
               down=at(8), down_scales=at(9), tokens=4, top_k=2, experts=8, hidden=256, inter=384, act_type=0, format=0,
               group=64, workspace=at(10), workspace_bytes=1 << 40)


def text():
    with open(os.path.join(ROOT, "include", "tq2_moe.h")) as f:
        return re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)


def packed(layout, base, over):
    return layout.pack(*{**base, **over}.values())


def route(**over):
    return moe.route_ptr(packed(moe._ROUTE, ROUTE, over))


def experts(**over):
    return moe.experts_ptr(packed(moe._EXPERTS, EXPERTS, over))


def test_header_and_binding_agree():
    h = text()
    assert tuple(sorted(set(re.findall(r"\b(tq2_[a-z0-9_]+)\s*\(", h)))) == moe.EXPORTED_SYMBOLS
    handle = ctypes.CDLL(tq2.LIB_PATH)
    for name in moe.EXPORTED_SYMBOLS:
        assert hasattr(handle, name)
    for name, value in (("MAX_EXPERTS", moe.MAX_EXPERTS), ("MAX_TOP_K", moe.MAX_TOP_K), ("MAX_TOKENS", moe.MAX_TOKENS),
                        ("MAX_DIM", moe.MAX_DIM), ("SOFTMAX", moe.SCORING.index("softmax")),
                        ("SIGMOID", moe.SCORING.index("sigmoid"))):
        assert int(re.search(r"#define\s+TQ2_MOE_%s\s+(\d+)" % name, h).group(1)) == value
    assert "TQ2_MOE_MAX_ROUTE_TOKENS (1 << 20)" in h and moe.MAX_ROUTE_TOKENS == 1 << 20


@pytest.mark.parametrize("name,base,layout", [("route", ROUTE, moe._ROUTE), ("experts", EXPERTS, moe._EXPERTS)])
def test_structs(name, base, layout):
    body = re.search(r"typedef struct tq2_moe_%s_args \{(.*?)\}" % name, text(), flags=re.S).group(1)
    fields = [re.search(r"(\w+)$", d.strip()).group(1) for d in body.split(";") if d.strip()]
    assert fields == list(base)
    kinds = ["Q" if "*" in d else "d" if "double" in d else "q" for d in body.split(";") if d.strip()]
    assert struct.Struct("=" + "".join(kinds)).size == layout.size == 8 * len(fields)
    expanded = "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([Qqd])", layout.format))
    assert expanded == "".join(kinds)


def test_null_args():
    assert tq2.lib.tq2_moe_route(None, None) == tq2.TQ2_ERR_INVALID
    assert tq2.lib.tq2_moe_experts(None, None) == tq2.TQ2_ERR_INVALID
    assert tq2.lib.tq2_moe_route_workspace_bytes(None) == tq2.lib.tq2_moe_experts_workspace_bytes(None) == 0


@pytest.mark.parametrize("over", [dict(x=0), dict(weight=0), dict(weights=0), dict(ids=0), dict(workspace=0),
                                  dict(tokens=-1), dict(tokens=(1 << 20) + 1), dict(hidden=0), dict(hidden=-8),
                                  dict(hidden=16392), dict(experts=3), dict(experts=1025), dict(experts=0), dict(top_k=0),
                                  dict(top_k=17, experts=64), dict(top_k=-1), dict(act_type=3), dict(act_type=-1),
                                  dict(weight_type=3), dict(weight_type=4), dict(scoring=2), dict(scoring=-1),
                                  dict(scale=float("nan")), dict(scale=float("inf")), dict(workspace_bytes=0),
                                  dict(workspace_bytes=-1), dict(workspace_bytes=4 * 16 * 8 - 1)])
def test_route_invalid(over):
    assert route(**over) == tq2.TQ2_ERR_INVALID


def test_route_shape_align_alias():
    for hidden in (4, 63, 100):
        assert route(hidden=hidden) == tq2.TQ2_ERR_SHAPE
    for name in ("x", "weight", "workspace"):
        for off in (2, 4, 8):
            assert route(**{name: ROUTE[name] + off}) == tq2.TQ2_ERR_ALIGN
    for name in ("bias", "weights", "ids"):
        assert route(**{name: ROUTE[name] + 2}) == tq2.TQ2_ERR_ALIGN
    for out in ("weights", "ids", "workspace"):
        for other in ("x", "weight", "bias"):
            assert route(**{out: ROUTE[other]}) == tq2.TQ2_ERR_ALIAS
    assert route(ids=ROUTE["weights"] + 4 * 4 * 4 - 4) == tq2.TQ2_ERR_ALIAS
    assert route(workspace=ROUTE["weights"]) == tq2.TQ2_ERR_ALIAS
    assert route(workspace=ROUTE["ids"]) == tq2.TQ2_ERR_ALIAS


def test_route_no_tokens_is_a_no_op():
    assert route(tokens=0, x=0, weights=0, ids=0, workspace=0, workspace_bytes=0) == tq2.TQ2_OK
    assert moe.route_workspace_bytes_ptr(packed(moe._ROUTE, ROUTE, dict(tokens=0))) == 0


@pytest.mark.parametrize("over", [dict(x=0), dict(out=0), dict(ids=0), dict(weights=0), dict(gate_up=0),
                                  dict(gate_up_scales=0), dict(down=0), dict(down_scales=0), dict(workspace=0),
                                  dict(tokens=-1), dict(tokens=129), dict(top_k=0), dict(top_k=17), dict(experts=0),
                                  dict(experts=1025), dict(hidden=0), dict(hidden=16512), dict(inter=0),
                                  dict(inter=16512), dict(inter=-128), dict(act_type=3), dict(format=2), dict(format=-1),
                                  dict(group=16), dict(group=0), dict(group=256), dict(format=1),
                                  dict(format=1, group=128), dict(workspace_bytes=0), dict(workspace_bytes=-1)])
def test_experts_invalid(over):
    assert experts(**over) == tq2.TQ2_ERR_INVALID


def test_experts_shape_align_alias():
    for over in (dict(hidden=64), dict(hidden=200), dict(inter=64), dict(inter=320)):
        assert experts(**over) == tq2.TQ2_ERR_SHAPE
    for name in ("x", "residual", "out", "gate_up", "gate_up_scales", "down", "down_scales", "workspace"):
        for off in (2, 8):
            assert experts(**{name: EXPERTS[name] + off}) == tq2.TQ2_ERR_ALIGN
    for name in ("ids", "weights"):
        assert experts(**{name: EXPERTS[name] + 2}) == tq2.TQ2_ERR_ALIGN
    for out in ("out", "workspace"):
        for other in ("ids", "weights", "gate_up", "gate_up_scales", "down", "down_scales"):
            assert experts(**{out: EXPERTS[other]}) == tq2.TQ2_ERR_ALIAS
    last = 8 * 2 * 384 * 128 - 16                        # of gate_up's codes
    assert experts(out=EXPERTS["gate_up"] + last) == tq2.TQ2_ERR_ALIAS
    for name in ("x", "residual"):
        assert experts(out=EXPERTS[name] + 16) == tq2.TQ2_ERR_ALIAS
        assert experts(workspace=EXPERTS[name]) == tq2.TQ2_ERR_ALIAS
    assert experts(workspace=EXPERTS["out"]) == tq2.TQ2_ERR_ALIAS


def test_experts_workspace():
    size = moe.experts_workspace_bytes_ptr(packed(moe._EXPERTS, EXPERTS, {}))
    assert size >= 4 * 2 * 384 * 4
    assert experts(workspace_bytes=size - 1) == tq2.TQ2_ERR_INVALID
    for over in (dict(tokens=0), dict(hidden=64), dict(group=1)):
        assert moe.experts_workspace_bytes_ptr(packed(moe._EXPERTS, EXPERTS, over)) == 0
    assert experts(tokens=0, x=0, out=0, workspace=0, workspace_bytes=0) == tq2.TQ2_OK


def test_tensors_are_checked():
    x, w = torch.zeros(2, 64), torch.zeros(8, 64)
    with pytest.raises(ValueError, match="device tensor"):
        moe.route(x, w, 2)
    with pytest.raises(ValueError, match="hidden"):
        moe.route(x, torch.zeros(8, 72), 2)
    with pytest.raises(ValueError, match="scoring"):
        moe.route(x, w, 2, scoring="tanh")
    with pytest.raises(TypeError):
        moe.route(x, "w", 2)
    ids, share = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    with pytest.raises(ValueError, match="top_k"):
        moe.experts(x, (w, w), (w, w), ids, torch.zeros(2, 3))
    with pytest.raises(ValueError, match="one format"):
        moe.experts(x, (w, w), w, ids, share)
    with pytest.raises(ValueError, match="device tensor"):
        moe.experts(x, w, w, ids, share, experts=4)
