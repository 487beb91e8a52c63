"""CPU checks of the paged-cache operators: refusals come before any device work, and the index arithmetic of the
kernels (csrc/tq2_pages.h) stays inside the cache for every table, length and offset."""

import ctypes
import os
import random
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")
from gemv_tq2_g128_amd import attn, tq2  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G = 1 << 36
A = 0x7F0000000000              # never dereferenced

CACHE = ["k", "v", "k_scale", "v_scale", "table", "kv_len", "cu_q", "batch", "tokens", "pages", "page", "table_cols",
         "table_stride", "kv_heads", "q_heads", "head_dim", "act_type", "cache_type", "k_page_stride", "k_head_stride",
         "k_token_stride", "v_page_stride", "v_head_stride", "v_token_stride"]
F32, F16, BF16, E4M3 = range(4)


def cache_fields(**over):
    c = dict(k=A, v=A + G, k_scale=0, v_scale=0, table=A + 2 * G, kv_len=A + 3 * G, cu_q=0, batch=3, tokens=3,
             pages=10, page=16, table_cols=4, table_stride=4, kv_heads=2, q_heads=4, head_dim=128, act_type=F32,
             cache_type=F16, k_page_stride=4096, k_head_stride=2048, k_token_stride=128, v_page_stride=4096,
             v_head_stride=2048, v_token_stride=128)
    c.update({n: x for n, x in over.items() if n in c})
    return c


def append(**over):
    c = cache_fields(**over)
    a = dict(q=A + 4 * G, k_new=A + 5 * G, v_new=A + 6 * G, q_out=A + 7 * G, q_ts=512, q_hs=128, k_ts=256, k_hs=128,
             v_ts=256, v_hs=128, o_ts=512, o_hs=128, freqs=A + 8 * G, positions=0, rot=128, axes=1, s0=64, s1=0, s2=0,
             interleaved=0, q_norm=0, k_norm=0, eps=1e-6)
    assert set(over) <= set(c) | set(a)
    a.update({n: x for n, x in over.items() if n in a})
    return attn.kv_append_ptr(attn._CACHE.pack(*(c[n] for n in CACHE)) + attn._APPEND.pack(*a.values()))


def attention(entry=attn.paged_attention_ptr, **over):
    c = cache_fields(**over)
    a = dict(q=A + 4 * G, out=A + 7 * G, q_ts=512, q_hs=128, o_ts=512, o_hs=128, max_q=1, max_kv=64, window=0,
             scale=0.1, workspace=0, workspace_bytes=0)
    assert set(over) <= set(c) | set(a)
    a.update({n: x for n, x in over.items() if n in a})
    return entry(attn._CACHE.pack(*(c[n] for n in CACHE)) + attn._ATTENTION.pack(*a.values()))


def test_header_and_binding_agree():
    with open(os.path.join(ROOT, "include", "tq2_attn.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    assert tuple(sorted(set(re.findall(r"\b(tq2_[a-z0-9_]+)\s*\(", text)))) == tuple(sorted(attn.EXPORTED_SYMBOLS))
    handle = ctypes.CDLL(tq2.LIB_PATH)
    for name in attn.EXPORTED_SYMBOLS:
        assert hasattr(handle, name)
    fields = re.search(r"typedef struct tq2_paged_cache \{(.*?)\}", text, flags=re.S).group(1)
    names = [n.strip(" *") for line in fields.split(";") if line.strip()
             for n in re.sub(r"^\s*(const\s+)?\w+\s*\*?", "", line.strip()).split(",")]
    assert names == CACHE and attn._CACHE.size == 8 * len(CACHE)


def test_valid_append_reaches_the_device_check():
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible; this check is for GPU-less hosts")
    for over in (dict(), dict(q=0, q_out=0), dict(act_type=BF16, cache_type=BF16), dict(act_type=F16, cache_type=F16),
                 dict(cache_type=E4M3, k_scale=A + 9 * G, v_scale=A + 10 * G), dict(rot=0, s0=0, freqs=0),
                 dict(q_out=A + 4 * G), dict(positions=A + 11 * G, axes=3, s0=30, s1=24, s2=10),
                 dict(cu_q=A + 12 * G, tokens=100), dict(page=1 << 20), dict(head_dim=64, rot=64, s0=32),
                 # q, k and v are columns of one array, q in place, keys and values of one page side by side
                 dict(q=A + 4 * G, k_new=A + 4 * G + 2048, v_new=A + 4 * G + 3072, q_ts=1024, k_ts=1024, v_ts=1024,
                      q_out=A + 4 * G, o_ts=1024),
                 dict(v=A + 8192, k_page_stride=8192, v_page_stride=8192)):
        assert append(**over) == tq2.TQ2_ERR_DEVICE, over


@pytest.mark.parametrize("over", [
    dict(k=0), dict(v=0), dict(table=0), dict(kv_len=0), dict(k_new=0), dict(v_new=0), dict(q=0), dict(q_out=0),
    dict(freqs=0), dict(batch=-1), dict(batch=1 << 17, tokens=1 << 17), dict(tokens=-1), dict(tokens=4),
    dict(cu_q=A + 12 * G, tokens=(1 << 30) + 1), dict(pages=-1), dict(pages=1 << 31), dict(table_cols=-1),
    dict(table_stride=-4), dict(kv_heads=0), dict(kv_heads=2000, q_heads=4000), dict(q_heads=0), dict(head_dim=32),
    dict(head_dim=80), dict(head_dim=512), dict(act_type=E4M3), dict(act_type=-1), dict(act_type=4),
    dict(cache_type=F32), dict(cache_type=BF16), dict(act_type=BF16), dict(act_type=F16, cache_type=BF16),
    dict(cache_type=E4M3), dict(cache_type=E4M3, k_scale=A + 9 * G), dict(k_scale=A + 9 * G, v_scale=A + 10 * G),
    dict(k_page_stride=-4096), dict(v_token_stride=1 << 41), dict(q_ts=-512), dict(rot=-8), dict(rot=136, s0=68),
    dict(axes=0), dict(axes=4, positions=A + 11 * G), dict(axes=2, s0=32, s1=32), dict(s0=63), dict(s0=65, s1=-1),
    dict(s0=32, s1=32), dict(eps=-1.0), dict(eps=float("nan"))])
def test_append_invalid(over):
    assert append(**over) == tq2.TQ2_ERR_INVALID


@pytest.mark.parametrize("over", [dict(page=0), dict(page=8), dict(page=24), dict(page=1 << 21), dict(kv_heads=3),
                                  dict(rot=4, s0=2), dict(rot=100, s0=50)])
def test_append_shape(over):
    assert append(**over) == tq2.TQ2_ERR_SHAPE


@pytest.mark.parametrize("over", [dict(k=A + 8), dict(v=A + G + 2), dict(table=A + 2 * G + 2), dict(q=A + 4 * G + 8),
                                  dict(k_new=A + 5 * G + 4), dict(q_out=A + 7 * G + 8), dict(k_token_stride=132),
                                  dict(v_head_stride=2052), dict(q_ts=514), dict(o_hs=130), dict(freqs=A + 4),
                                  dict(q_norm=A + 8), dict(cu_q=A + 1)])
def test_append_alignment(over):
    assert append(**over) == tq2.TQ2_ERR_ALIGN


@pytest.mark.parametrize("over", [
    dict(v=A), dict(q=A + 64), dict(k_new=A + 1024), dict(v_new=A + G), dict(q_out=A + 10 * 4096 * 2 - 16),
    dict(q_out=A + 4 * G + 16), dict(q_out=A + 4 * G, o_ts=1024), dict(q_out=A + 5 * G), dict(q_out=A + 6 * G + 16)])
def test_append_aliasing(over):
    assert append(**over) == tq2.TQ2_ERR_ALIAS


def test_append_without_tokens_is_a_no_op():
    assert append(tokens=0, batch=0, k=0, v=0, table=0, q=0, k_new=0, v_new=0) == tq2.TQ2_OK
    assert append(tokens=0, batch=0, page=24) == tq2.TQ2_ERR_SHAPE
    assert append(tokens=7, batch=0, cu_q=A + 12 * G, k=0, table=0) == tq2.TQ2_OK     # rows without a sequence
    assert attention(tokens=7, batch=0, cu_q=A + 12 * G, k=0, table=0) == tq2.TQ2_OK
    assert attention(attn.paged_attention_workspace_bytes_ptr, tokens=7, batch=0, cu_q=A, max_kv=5000) == 0


E8 = dict(cache_type=E4M3, k_scale=A + 9 * G, v_scale=A + 10 * G)


def test_valid_attention_reaches_the_device_check():
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible; this check is for GPU-less hosts")
    need = attention(attn.paged_attention_workspace_bytes_ptr, max_kv=5000)
    assert need > 0
    for over in (dict(), dict(act_type=BF16, cache_type=BF16), dict(act_type=F16, cache_type=F16), E8,
                 dict(out=A + 4 * G), dict(cu_q=A + 12 * G, tokens=100, max_q=90), dict(window=17), dict(max_q=0),
                 dict(max_kv=0), dict(pages=0, k=0, v=0),
                 dict(max_kv=5000, workspace=A + 13 * G, workspace_bytes=need)):
        assert attention(**over) == tq2.TQ2_ERR_DEVICE, over


@pytest.mark.parametrize("over", [
    dict(k=0), dict(v=0), dict(table=0), dict(kv_len=0), dict(q=0), dict(out=0), dict(batch=-1), dict(tokens=4),
    dict(tokens=-1), dict(kv_heads=0), dict(q_heads=0), dict(head_dim=80), dict(act_type=BF16), dict(cache_type=E4M3),
    dict(k_scale=A + 9 * G, v_scale=A + 10 * G), dict(q_ts=-512), dict(o_hs=1 << 41), dict(max_q=-1), dict(max_kv=-1),
    dict(max_kv=1 << 31), dict(window=-1), dict(window=1 << 31), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(workspace_bytes=-1), dict(max_kv=5000),
    dict(max_kv=5000, workspace=A + 13 * G, workspace_bytes=4096), dict(k_token_stride=1 << 27),
    dict(v_token_stride=1 << 27)])
def test_attention_invalid(over):
    assert attention(**over) == tq2.TQ2_ERR_INVALID


@pytest.mark.parametrize("over", [dict(page=0), dict(page=8), dict(page=48), dict(kv_heads=3)])
def test_attention_shape(over):
    assert attention(**over) == tq2.TQ2_ERR_SHAPE


@pytest.mark.parametrize("over", [dict(k=A + 8), dict(q=A + 4 * G + 8), dict(out=A + 7 * G + 4), dict(q_ts=514),
                                  dict(o_hs=130), dict(v_page_stride=4100), dict(workspace=A + 13 * G + 8)])
def test_attention_alignment(over):
    assert attention(**over) == tq2.TQ2_ERR_ALIGN


@pytest.mark.parametrize("over", [
    dict(v=A), dict(out=A + 4 * G + 16), dict(out=A + 4 * G, o_ts=1024), dict(out=A + 4096), dict(out=A + G),
    dict(max_kv=5000, workspace=A + 4 * G, workspace_bytes=1 << 30),
    dict(max_kv=5000, workspace=A + 7 * G, workspace_bytes=1 << 30),
    dict(max_kv=5000, workspace=A, workspace_bytes=1 << 30)])
def test_attention_aliasing(over):
    assert attention(**over) == tq2.TQ2_ERR_ALIAS


def test_attention_workspace():
    def need(**over):
        return attention(attn.paged_attention_workspace_bytes_ptr, **over)

    assert need(max_kv=0) == need(max_kv=1) == 0
    assert need(head_dim=80, max_kv=5000) == need(page=7, max_kv=5000) == need(tokens=0, batch=0, max_kv=5000) == 0
    assert 0 < need(max_kv=100000, window=500) < need(max_kv=100000)
    assert attention(tokens=0, batch=0, k=0, q=0, out=0, table=0) == tq2.TQ2_OK
    assert attention(tokens=0, batch=0, page=24) == tq2.TQ2_ERR_SHAPE


def test_front_end_checks():
    k = torch.zeros(2, 2, 64)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    lens, table = torch.ones(2, dtype=torch.int32), torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        attn.kv_append(k, k, cache, cache, lens, table)
    with pytest.raises(ValueError, match="kv_heads, head_dim"):
        attn.kv_append(k[0], k[0], cache, cache, lens, table)
    with pytest.raises(ValueError, match="device tensor"):
        attn.paged_attention(k, cache, cache, lens, table)
    with pytest.raises(ValueError, match="q_heads, head_dim"):
        attn.paged_attention(k[0], cache, cache, lens, table)


HARNESS = r"""
#include "tq2_pages.h"
extern "C" int64_t place_offset(const int32_t* table, const int32_t* kv_len, const int32_t* cu_q, int batch, int tokens,
                                int pages, int cols, int shift, int64_t table_stride, int b, int32_t n) {
  tq2::Pages p{};
  p.table = table; p.kv_len = kv_len; p.cu_q = cu_q; p.batch = batch; p.tokens = tokens; p.pages = pages;
  p.cols = cols; p.page_shift = shift; p.table_stride = table_stride;
  return tq2::page_of(p, b, n);
}
extern "C" void parts(int32_t first, int32_t keys, int32_t window, int32_t splits, int32_t split_keys, int32_t* out) {
  const tq2::Parts r = tq2::parts_of(tq2::Seq{0, 1, first, keys}, window, splits, split_keys);
  out[0] = r.base; out[1] = r.per; out[2] = r.count;
}
extern "C" void seq(const int32_t* kv_len, const int32_t* cu_q, int batch, int tokens, int cols, int shift, int b,
                    int32_t* out) {
  tq2::Pages p{};
  p.kv_len = kv_len; p.cu_q = cu_q; p.batch = batch; p.tokens = tokens; p.cols = cols; p.page_shift = shift;
  const tq2::Seq s = tq2::sequence(p, b);
  out[0] = s.q0; out[1] = s.q_len; out[2] = s.first; out[3] = s.keys;
}
"""


@pytest.fixture(scope="module")
def pages_lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("pages")
    (at / "pages.cc").write_text(HARNESS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "gemv_tq2_g128_amd", "csrc"), str(at / "pages.cc"), "-o", str(at / "pages.so")],
                   check=True)
    lib = ctypes.CDLL(str(at / "pages.so"))
    lib.place_offset.restype = ctypes.c_int64
    lib.place_offset.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int] * 5 + [ctypes.c_int64, ctypes.c_int,
                                                                              ctypes.c_int32]
    return lib


def test_page_lookups_stay_inside(pages_lib):
    table = torch.tensor([[3, -1, 10, 9], [2 ** 31 - 1, 0, -2 ** 31, 5]], dtype=torch.int32)

    def look(b, n):
        return pages_lib.place_offset(table.data_ptr(), None, None, 2, 2, 10, 4, 4, 4, b, n)

    assert [look(0, n) for n in (0, 15, 16, 31, 32, 48, 63)] == [3, 3, -1, -1, -1, 9, 9]
    assert [look(1, n) for n in (0, 16, 32, 63)] == [-1, 0, -1, 5]
    assert [look(0, n) for n in (-1, -2 ** 31, 64, 2 ** 31 - 1)] == [-1] * 4


def test_parts_cover_the_keys(pages_lib):
    """The parts of a sequence's keys: in order, no more than asked for, and every key a row can see is in one."""
    rng = random.Random(2)
    edge = [0, 1, 31, 32, 33, 100, 4096, 131071, 2 ** 31 - 1]
    for _ in range(4000):
        keys = rng.choice(edge) if rng.random() < 0.5 else rng.randrange(0, 1 << rng.randrange(1, 31))
        keys = min(keys, 0x7FFF0000)
        first = keys - rng.choice([0, 1, 5, 200, keys, keys + 7])
        window = rng.choice([0, 0, 1, 40, 1024, 2 ** 31 - 1])
        splits, split_keys = rng.choice([1, 2, 7, 512]), rng.choice([128, 1024])
        out = (ctypes.c_int32 * 3)()
        pages_lib.parts(first, keys, window, splits, split_keys, out)
        base, per, count = out
        assert base % 32 == 0 and per % 32 == 0 and per >= split_keys and 1 <= count <= splits
        assert 0 <= base <= keys and base + count * per >= keys and (count == 1 or base + (count - 1) * per < keys)
        assert base <= max(0, first - window + 1 if window else 0)


def test_sequences_are_cut_to_the_arrays(pages_lib):
    rng = random.Random(1)
    edge = [-2 ** 31, -7, -1, 0, 1, 5, 16, 17, 63, 64, 65, 1000, 2 ** 31 - 1]
    for _ in range(2000):
        kv = torch.tensor([rng.choice(edge) for _ in range(2)], dtype=torch.int32)
        cu = torch.tensor([rng.choice(edge) for _ in range(3)], dtype=torch.int32)
        out = (ctypes.c_int32 * 4)()
        pages_lib.seq(ctypes.c_void_p(kv.data_ptr()), ctypes.c_void_p(cu.data_ptr()), 2, 17, 4, 4, 1, out)
        q0, q_len, first, keys = out
        assert 0 <= q0 <= 17 and 0 <= q_len <= 17 - q0 and 0 <= keys <= 64 and keys <= max(0, int(kv[1]))
    kv, cu = torch.tensor([40, 9], dtype=torch.int32), torch.tensor([0, 3, 17], dtype=torch.int32)
    pages_lib.seq(ctypes.c_void_p(kv.data_ptr()), ctypes.c_void_p(cu.data_ptr()), 2, 17, 4, 4, 0, out)
    assert list(out) == [0, 3, 37, 40]
    pages_lib.seq(ctypes.c_void_p(kv.data_ptr()), ctypes.c_void_p(cu.data_ptr()), 2, 17, 4, 4, 1, out)
    assert list(out) == [3, 14, -5, 9]
    pages_lib.seq(ctypes.c_void_p(kv.data_ptr()), None, 2, 2, 4, 4, 1, out)
    assert list(out) == [1, 1, 8, 9]
