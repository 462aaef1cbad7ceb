"""The rule by which csrc/q4.hip picks a kernel for a 4-bit product, written out
again for the tests: which sizes reach which kernel. tests/test_q4_plan.py holds it
against the workspace sizes that the library gives."""

from __future__ import annotations

from dataclasses import dataclass

CHUNK = 128


def _up(a, b):
    return -(-a // b)


def pad8(K):
    return _up(K, 8) * 8


def plane_rows(M):
    return M if M <= 16 else 32 if M <= 32 else _up(M, 128) * 128


def parts(x):
    """Matrix operands of one value of x: bf16, f32, e4m3, or planes (the FFN's hidden values)."""
    return 3 if x in ("f32", "planes") else 1


def wide_rows(x, gated, M, N):
    if M <= 32 or (parts(x) == 3 and M <= 64):
        return 32
    return 128 if parts(x) == 1 and _up(N, 32 if gated else 64) * _up(M, 128) >= 384 else 64


def wide_waves(x, rows):
    return 8 if parts(x) == 3 and rows == 64 else 4


@dataclass(frozen=True)
class Plan:
    few: bool  # q4_tile_kernel, else q4_wide_kernel
    waves: int
    items: int
    splits: int
    split_chunks: int


def _cut(few, waves, items, want, piece, K):
    chunks, pieces = _up(K, CHUNK), _up(K, CHUNK * piece)
    want = max(1, min(want, 16))
    split_chunks = _up(pieces, want) * piece
    return Plan(few, waves, items, _up(chunks, split_chunks), split_chunks)


def plan_tile(x, gated, M, N, K):
    piece = 8 if parts(x) > 1 else 16
    for waves in (2,) if gated else (1, 2):
        units = 16 * waves // (2 if gated else 1)
        items = _up(N, units) * _up(M, 16)
        p = _cut(True, waves, items, min(512 // items, _up(K, CHUNK * piece) // 2), piece, K)
        if waves == 2 or p.items * p.splits <= 256:
            return p


def plan_wide(x, gated, M, N, K):
    rows = wide_rows(x, gated, M, N)
    waves, chunks = wide_waves(x, rows), _up(K, CHUNK)
    items = _up(N, 16 * waves // (2 if gated else 1)) * _up(M, rows)
    resident = 256 if waves == 8 else 512
    return _cut(False, waves, items, max(min(256 // items, chunks // 4), min(resident // items, chunks // 8)), 1, K)


def plan(x, gated, M, N, K, group):
    p = plan_tile(x, gated, M, N, K)
    work = p.items * p.splits * p.split_chunks
    if M <= 16 or p.items * p.splits <= 256:
        return p
    if (group == 128 and work <= 512 * 16) if parts(x) == 1 else work <= 768 * 8:
        return p
    return plan_wide(x, gated, M, N, K)


def _room(p, x, gated, M, N, K):
    planes = 0 if p.few or x == "planes" else _up(parts(x) * pad8(K) * plane_rows(M) * 2, 256) * 256
    part = p.splits * (2 if gated else 1) * M * N * 4 if p.splits > 1 else 0
    return planes + _up(part, 256) * 256


def workspace_bytes(x, gated, M, N, K):
    tile = _room(plan_tile(x, gated, M, N, K), x, gated, M, N, K)
    return tile if M <= 16 else max(tile, _room(plan_wide(x, gated, M, N, K), x, gated, M, N, K))


def instance(x, gated, M, N, K, group):
    """(kernel instance, whether its loop over whole pieces of K runs). x at an aligned address."""
    p = plan(x, gated, M, N, K, group)
    if p.few:
        piece = 8 if parts(x) > 1 else 16
        return ("tile", x, group, p.waves, gated), min(p.split_chunks, _up(K, CHUNK)) > piece
    rows = wide_rows(x, gated, M, N)
    ahead = 2 if parts(x) * rows // 16 <= 4 else 1
    row_major = x == "bf16" and K % 8 == 0
    return (("wide", "planes" if parts(x) == 3 else "rows" if row_major else "plane", group, rows, gated),
            min(p.split_chunks, K // CHUNK) >= 2 * ahead)


# Sizes M, N, K that between them reach every instance of q4_wide_kernel, its loop over
# whole chunks of K among them, for each group: 32, 64 and 128 rows a workgroup, K
# whole and cut, one or more splits.
WIDE = [(24, 8200, 1032), (24, 8200, 1027), (24, 8300, 2568), (90, 7500, 2328), (130, 7500, 1027), (259, 8200, 1032),
        (259, 8200, 1027)]
WIDE_GATED = [(24, 4200, 1224), (24, 4200, 1221), (108, 4600, 832), (108, 4600, 835), (162, 6600, 1096),
              (162, 6600, 1093)]

# And of q4_tile_kernel: 16 or 32 units a workgroup, one or more slices of K and rows
# of tiles, in splits.
TILE = [(5, 100, 2100), (16, 4201, 2503), (40, 500, 2100), (3, 64, 10241)]
TILE_GATED = [(5, 100, 2100), (33, 500, 2503), (3, 64, 10241)]

# M, d, F of the whole FFN, whose down product takes the hidden values (planes): both
# kernels, each with its tiles.
FFN = [(5, 200, 2100), (7, 4201, 1100), (40, 4100, 2100), (90, 4100, 2101)]


def ffn_instance(M, d, F, group):
    return instance("planes", False, M, d, F, group)
