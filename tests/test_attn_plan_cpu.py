"""CPU checks of how an attention call is laid out (csrc/tq2_attn_plan.h, compiled for the host)."""

import ctypes
import os
import random
import subprocess

import pytest

pytest.importorskip("torch")
from gemv_tq2_g128_amd import attn  # noqa: E402
from tests.test_attn_cpu import A, BF16, CACHE, E4M3, F16, F32, G, ROOT, cache_fields  # noqa: E402

HARNESS = r"""
#include "tq2_attn_plan.h"
extern "C" void plan(const tq2_paged_attention_args* a, int64_t* out) {
  const tq2::AttnPlan p = tq2::plan_attention(*a);
  const int64_t all[] = {p.tiled, p.row_tiles, p.steps, p.splits, p.split_keys, int64_t(p.workspace)};
  for (int64_t v : all) *out++ = v;
}
extern "C" void tile_grid(int64_t splits, int64_t steps, int64_t kv_heads, int64_t batch, int64_t* out) {
  tq2::AttnPlan p{};
  p.splits = int32_t(splits), p.steps = int32_t(steps);
  const tq2::Grid g = tq2::tile_grid(p, kv_heads, batch);
  out[0] = g.x, out[1] = g.y, out[2] = g.z;
}
extern "C" void stream_grid(int64_t splits, int64_t steps, int64_t kv_heads, int64_t batch, int64_t* out) {
  tq2::AttnPlan p{};
  p.splits = int32_t(splits), p.steps = int32_t(steps);
  const tq2::Grid g = tq2::stream_grid(p, kv_heads, batch);
  out[0] = g.x, out[1] = g.y, out[2] = g.z;
}
extern "C" void append_grid(int64_t tokens, int64_t per_block, int64_t rounds, int64_t* out) {
  const tq2::Grid g = tq2::append_grid(tokens, per_block, rounds);
  out[0] = g.x, out[1] = g.y, out[2] = g.z;
}
extern "C" void row_grid(int64_t blocks, int64_t* out) {
  const tq2::Grid g = tq2::row_grid(blocks);
  out[0] = g.x, out[1] = g.y, out[2] = g.z;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cc").write_text(HARNESS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover", "-I", os.path.join(ROOT, "gemv_tq2_g128_amd", "csrc"),
                    str(at / "plan.cc"), "-o", str(at / "plan.so")], check=True)
    return ctypes.CDLL(str(at / "plan.so"))


class Plan:
    def __init__(self, host, max_q, max_kv, window=0, **over):
        e8 = dict(k_scale=A, v_scale=A) if over.get("cache_type") == E4M3 else {}
        self.cache = cache_fields(**{**e8, **over})
        tail = attn._ATTENTION.pack(A, A + G, 0, 0, 0, 0, max_q, max_kv, window, 0.1, 0, 0)
        args = attn._CACHE.pack(*(self.cache[n] for n in CACHE)) + tail
        out = (ctypes.c_int64 * 6)()
        host.plan(args, out)
        self.tiled, self.row_tiles, self.steps, self.splits, self.split_keys, self.workspace = out
        assert self.workspace == attn.paged_attention_workspace_bytes_ptr(args)


def grid(fn, *args):
    out = (ctypes.c_int64 * 3)()
    fn(*(ctypes.c_int64(a) for a in args), out)
    return tuple(out)


def launchable(g, threads=256):
    x, y, z = g
    return 1 <= x and x * threads < 1 << 32 and 1 <= y <= 65535 and 1 <= z <= 65535


@pytest.mark.parametrize("batch,each,heads", [(1024, 64, (32, 8)), (256, 512, (64, 8)), (512, 128, (64, 8)),
                                              (1024, 32, (64, 8)), (4096, 2, (64, 8)), (65535, 1, (64, 8)),
                                              (65535, 16384, (1024, 1024)), (1, 1 << 20, (1024, 1))])
def test_many_sequences_without_a_longest(host, batch, each, heads):
    """max_q left at all of q's rows: the grid can still be launched, and no more blocks start than are worth it."""
    p = Plan(host, batch * each, 4096, batch=batch, tokens=batch * each, cu_q=A, q_heads=heads[0], kv_heads=heads[1])
    assert p.tiled
    g = grid(host.tile_grid, p.splits, p.steps, heads[1], batch)
    assert launchable(g)
    assert g[0] * g[1] * g[2] <= max(1 << 19, batch * heads[1] * p.splits)


def test_plans_in_range(host):
    """Any sizes that a call accepts: the grid can be launched and the parts fit their fields."""
    rng = random.Random(3)

    def wide(most):
        return min(most, int(2 ** rng.uniform(0, most.bit_length())))

    for _ in range(4000):
        kv_heads = wide(1024)
        q_heads = kv_heads * rng.randrange(1, 1024 // kv_heads + 1)
        batch = wide(65535)
        act, cache = rng.choice([(F32, F16), (F32, E4M3), (F16, F16), (BF16, BF16), (BF16, E4M3)])
        tokens = min(wide(1 << 30), ((1 << 31) - 4097) // q_heads)
        max_kv = rng.choice([0, wide((1 << 31) - 1), (1 << 31) - 1])
        p = Plan(host, rng.choice([0, 1, wide(1 << 30), tokens]), max_kv, rng.choice([0, wide((1 << 31) - 1)]),
                 batch=batch, tokens=tokens, cu_q=A, q_heads=q_heads, kv_heads=kv_heads, act_type=act, cache_type=cache,
                 head_dim=rng.choice([64, 96, 128, 192, 256]))
        assert p.steps >= 1 and 1 <= p.splits <= 512 and p.split_keys >= 128 and p.split_keys % 32 == 0
        assert launchable(grid(host.tile_grid if p.tiled else host.stream_grid, p.splits, p.steps, kv_heads, batch))


@pytest.mark.parametrize("max_q", [1, 64, 5000])
def test_the_longest_cache(host, max_q):
    """Keys of a part stay in 31 bits where max_kv is the largest that is taken."""
    for max_kv in ((1 << 31) - 1, (1 << 31) - 200, 0x7FFF0000):
        p = Plan(host, max_q, max_kv, batch=60000, tokens=max_q * 60000, cu_q=A)
        assert 128 <= p.split_keys <= 0x7FFF0000 and (p.split_keys * p.splits >= 0x7FFF0000 or p.splits == 512)


@pytest.mark.parametrize("blocks", [1, 5, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, 1 << 24, (1 << 24) + 7, 99999989,
                                    (1 << 31) - 4097])
def test_row_grid(host, blocks):
    """Every block is there, less than a row is left over (16 rows of q each: below 2^32), and it can be launched."""
    g = grid(host.row_grid, blocks)
    assert launchable(g) and g[2] == 1
    assert 0 <= g[0] * g[1] - blocks < 1 << 20 and (g[1] == 1) == (blocks <= 1 << 20)


@pytest.mark.parametrize("per_block", [1, 4])
@pytest.mark.parametrize("tokens", [1, 7, 255, 4096, 1 << 22, (1 << 22) + 1, 1 << 26, (1 << 26) + 5, 1 << 30])
def test_append_grid(host, tokens, per_block):
    """Every token has a block, the kernel's token numbers stay in 31 bits, and the launch is one that can be made."""
    for rounds in (1, 3, 384):
        x, y, z = grid(host.append_grid, tokens, per_block, rounds)
        assert launchable((x, y, z)) and 1 <= y <= rounds
        assert tokens <= x * z * per_block < 1 << 31 and (z == 1 or x == 1 << 20)


@pytest.mark.parametrize("kv_heads", [1, 2, 8, 16])
@pytest.mark.parametrize("lengths", [[8] + [1] * 63, [128] + [8] * 3, [64] + [1] * 15, [16, 1] * 8, list(range(1, 65)),
                                     [32] * 4, [16] * 31, [512], [5, 4, 3, 2, 1]])
def test_parts_spread_over_the_card(host, kv_heads, lengths):
    """Blocks with work (part i of a sequence of more than i parts) are shared evenly by the places that a block's
    number gives it: 8 dies of 32 CUs, and 4 engines in each; or there is a CU for each."""
    splits, batch = max(lengths), len(lengths)
    x, y, z = grid(host.stream_grid, splits, 1, kv_heads, batch)
    assert (x, z) == (kv_heads, splits) and y >= batch
    for places in (8, 32):
        held = [0] * places
        for b, count in enumerate(lengths):
            for part in range(count):
                for head in range(kv_heads):
                    held[(head + x * (b + y * part)) % places] += 1
        mean = sum(held) / places
        assert max(held) <= max(1.35 * mean + 2, 256 / places), (places, held)


def test_neighbours_are_cut_alike(host):
    """No size is an exception: parts of a batch hardly longer, or of one sequence more, are hardly other parts."""
    for batch in (48, 63, 64, 65, 80, 128, 256):
        for keys in (4000, 6000, 8191, 8192, 8193, 12000, 16384, 40000):
            here = Plan(host, 1, keys, batch=batch, tokens=batch, q_heads=32, kv_heads=8, act_type=BF16, cache_type=BF16)
            for more, longer in ((1, 0), (0, 1), (-1, 0), (0, -1)):
                there = Plan(host, 1, keys + longer, batch=batch + more, tokens=batch + more, q_heads=32, kv_heads=8,
                             act_type=BF16, cache_type=BF16)
                assert abs(here.splits - there.splits) <= 1, (batch, keys, here.splits, there.splits)


@pytest.mark.parametrize("max_kv", [8192, 131072, 1 << 20])
@pytest.mark.parametrize("batch", [1, 16, 256, 1024, 4096, 65535])
def test_memory_of_the_parts(host, batch, max_kv):
    """However long the table says that sequences may be, a decode step's parts take no more than a dozen blocks'
    states for each of the card's 512 places (26 MB for 8 rows of 128 components)."""
    p = Plan(host, 1, max_kv, batch=batch, tokens=batch, q_heads=64, kv_heads=8, act_type=BF16, cache_type=BF16)
    assert p.workspace <= 12 * 512 * 8 * 132 * 4
    assert p.splits > 1 or batch * 8 * 2 > 12 * 512
