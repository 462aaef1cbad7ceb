"""The tests' copy of the rule for 4-bit products against the library's workspace
sizes, and that the sizes of tests/test_gpu_block_q4.py reach every kernel instance."""

import random

import pytest

import _q4_plan as P
import activation_sparse_ffn_gate_amd as tw

torch = pytest.importorskip("torch")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def test_workspace_sizes_agree():
    rng = random.Random(1)
    for _ in range(3000):
        M, N, K = (int(2 ** rng.uniform(0, hi)) for hi in (11, 14, 15))
        for x, dtype in TYPES.items():
            for gated in (False, True):
                want = P.workspace_bytes(x, gated, M, N, K)
                assert tw.q4_workspace_bytes(dtype, M, N, K, gated) == want, (x, gated, M, N, K)


def _reached(sizes, gated):
    reached = {}
    for M, N, K in sizes:
        for group in (32, 64, 128):
            for x in TYPES:
                name, loop = P.instance(x, gated, M, N, K, group)
                reached[name] = reached.get(name, False) or loop
    return reached


@pytest.mark.parametrize("gated", [False, True])
def test_sizes_reach_every_instance(gated):
    wide = _reached(P.WIDE_GATED if gated else P.WIDE, gated)
    want = [("wide", kind, group, rows, gated) for group in (32, 64, 128)
            for kind, tiles in (("rows", (32, 64, 128)), ("plane", (32, 64, 128)), ("planes", (32, 64))) for rows in tiles]
    missing = [w for w in want if not wide.get(w)]
    assert not missing
    tile = _reached(P.TILE_GATED if gated else P.TILE, gated)
    want = [("tile", x, group, waves, gated) for group in (32, 64, 128) for x in TYPES
            for waves in ((2,) if gated else (1, 2))]
    assert not [w for w in want if not tile.get(w)]


def test_ffn_sizes_reach_every_instance_of_the_down_product():
    reached = {}
    for M, d, F in P.FFN:
        for group in (32, 64, 128):
            name, loop = P.ffn_instance(M, d, F, group)
            reached[name] = reached.get(name, False) or loop
    want = [("tile", "planes", g, w, False) for g in (32, 64, 128) for w in (1, 2)]
    want += [("wide", "planes", g, rows, False) for g in (32, 64, 128) for rows in (32, 64)]
    assert not [w for w in want if not reached.get(w)]
