"""CPU checks of tq2_sample: the header's symbols, struct and constants, and every refusal, which comes before any device
work."""

import ctypes
import os
import re

import pytest

from gemv_tq2_g128_amd import sampling, tq2

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7F0000000000           # never dereferenced


def at(i):
    return BASE + (i << 44)


ARGS = dict(logits=at(1), u=at(2), ids=at(3), logprob=at(4), temperatures=at(5), top_ks=at(6), top_ps=at(7), min_ps=at(8),
            rows=4, vocab=1000, row_stride=1024, logits_type=0, top_k=0, temperature=1.0, top_p=1.0, min_p=0.0,
            workspace=at(9), workspace_bytes=1 << 40)
NAN = float("nan")


def packed(over):
    return sampling._ARGS.pack(*{**ARGS, **over}.values())


def call(**over):
    return sampling.sample_ptr(packed(over))


def test_header_and_binding_agree():
    with open(os.path.join(ROOT, "include", "tq2_sample.h")) as f:
        h = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    assert tuple(sorted(set(re.findall(r"\b(tq2_[a-z0-9_]+)\s*\(", h)))) == sampling.EXPORTED_SYMBOLS
    handle = ctypes.CDLL(tq2.LIB_PATH)
    for name in sampling.EXPORTED_SYMBOLS:
        assert hasattr(handle, name)
    assert int(re.search(r"TQ2_SAMPLE_MAX_ROWS\s+(\d+)", h).group(1)) == sampling.MAX_ROWS
    assert "TQ2_SAMPLE_MAX_VOCAB (1 << 20)" in h and sampling.MAX_VOCAB == 1 << 20
    body = re.search(r"typedef struct tq2_sample_args \{(.*?)\}", h, flags=re.S).group(1)
    fields = [d.strip() for d in body.split(";") if d.strip()]
    assert [re.search(r"(\w+)$", d).group(1) for d in fields] == list(ARGS)
    kinds = "".join("Q" if "*" in d else "d" if "double" in d else "q" for d in fields)
    assert kinds == "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([Qqd])", sampling._ARGS.format))


@pytest.mark.parametrize("over", [dict(logits=0), dict(u=0), dict(ids=0), dict(workspace=0), dict(rows=-1),
                                  dict(rows=4097), dict(vocab=0), dict(vocab=-5), dict(vocab=(1 << 20) + 1),
                                  dict(row_stride=-1), dict(row_stride=-1024), dict(row_stride=(1 << 40) + 1),
                                  dict(logits_type=3), dict(logits_type=-1), dict(workspace_bytes=0),
                                  dict(workspace_bytes=-1), dict(temperatures=0, temperature=-0.5),
                                  dict(temperatures=0, temperature=NAN), dict(top_ps=0, top_p=NAN),
                                  dict(min_ps=0, min_p=NAN)])
def test_invalid(over):
    assert call(**over) == tq2.TQ2_ERR_INVALID


def test_null_args():
    assert tq2.lib.tq2_sample(None, None) == tq2.TQ2_ERR_INVALID
    assert tq2.lib.tq2_sample_workspace_bytes(None) == 0


def test_alignment():
    for name in ("u", "ids", "logprob", "temperatures", "top_ks", "top_ps", "min_ps"):
        for off in (1, 2):
            assert call(**{name: ARGS[name] + off}) == tq2.TQ2_ERR_ALIGN
    assert call(logits=at(1) + 2) == tq2.TQ2_ERR_ALIGN
    assert call(logits=at(1) + 1, logits_type=1) == tq2.TQ2_ERR_ALIGN
    assert call(workspace=at(9) + 8) == tq2.TQ2_ERR_ALIGN


def test_aliasing():
    for out in ("ids", "logprob", "workspace"):
        for other in ("logits", "u", "temperatures", "top_ks", "top_ps", "min_ps"):
            assert call(**{out: ARGS[other]}) == tq2.TQ2_ERR_ALIAS
    assert call(ids=at(1) + 4 * (3 * 1024 + 999)) == tq2.TQ2_ERR_ALIAS
    assert call(ids=at(4) + 12) == tq2.TQ2_ERR_ALIAS
    assert call(workspace=at(3)) == tq2.TQ2_ERR_ALIAS
    assert call(workspace=at(4)) == tq2.TQ2_ERR_ALIAS


def test_workspace_and_no_rows():
    size = sampling.sample_workspace_bytes_ptr(packed({}))
    assert size > 0 and call(workspace_bytes=size - 1) == tq2.TQ2_ERR_INVALID
    for over in (dict(rows=0), dict(rows=5000), dict(vocab=0)):
        assert sampling.sample_workspace_bytes_ptr(packed(over)) == 0
    assert call(rows=0, logits=0, u=0, ids=0, workspace=0, workspace_bytes=0) == tq2.TQ2_OK


def test_tensors_are_checked():
    logits, u = torch.zeros(2, 10), torch.zeros(2)
    with pytest.raises(ValueError, match="device tensor"):
        sampling.sample(logits, u)
    with pytest.raises(ValueError, match="rows, vocab"):
        sampling.sample(u, u)
    with pytest.raises(TypeError):
        sampling.sample([1.0], u)
