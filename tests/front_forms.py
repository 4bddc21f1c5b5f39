"""Which compiled form of a kernel a call of the layer's front reaches.

The launch rules of ``csrc`` written down a second time, with the thresholds
read from the sources: a case says which form it is for, and stops being valid
when a threshold moves away from under it.  Also the cases of
``test_gpu_front_forms.py``, so that a CPU test can hold them against the forms
the library holds."""

from __future__ import annotations

import os
import re

import combine_ep_plan_amd as ep

CSRC = os.path.join(os.path.dirname(ep.__file__), "csrc")


def _source(name: str) -> str:
    with open(os.path.join(CSRC, name)) as fh:
        return fh.read()


def _numbers(name: str, pattern: str) -> list[int]:
    """The numbers a pattern's groups match, at its only place in a source."""
    found = re.findall(pattern, _source(name))
    assert len(found) == 1, (name, pattern, found)
    return [int(v) for v in (found[0] if isinstance(found[0], tuple) else found)]


def _constant(name: str, what: str) -> int:
    return _numbers(name, rf"constexpr int(?:32_t|64_t)? {what} = (\d+);")[0]


FEW_ROWS = _constant("norm.hip", "kFewRows")
STREAM_WAVES = _constant("gemm_int8.hip", "kStreamWaves")
FEW_PER_EXPERT = _constant("gemm_int8.hip", "kFewRowsPerExpert")
DIRECT_ROWS = _constant("gemm_int8.hip", "kDirectRows")
SHORT_ROWS = _constant("gemm_int8.hip", "kShortRows")
STREAM_IF_FILLS, STREAM_ELSE = _numbers("gemm_int8.hip", r"g\.n <= \(int64_t\)\(fills \? (\d+) : (\d+)\) \* g\.E")
MANY_FORWARD, MANY_BACKWARD = _numbers("score_route.hip", r"kManyForward = (\d+), kManyBackward = (\d+);")
WAVE_EXPERTS, WAVE_MANY, WAVE_FEW = _numbers(
    "score_route.hip", r"return E > (\d+) \|\| T <= \(E > many \? (\d+) : (\d+)\);")
STORE_LOW, STORE_HIGH = _numbers(
    "dispatch8.hip", r"bytes <= \(\(int64_t\)(\d+) << 20\) \|\| bytes \* g\.in_flight > \(\(int64_t\)(\d+) << 20\)")


def gemm_int8_form(layout: str, T: int, E: int, k: int, cap: int, K: int, N: int, glu: bool) -> tuple:
    """("stream", glu, few, split, table), ("tiles", glu) or ("wide", glu)."""
    n = T * k
    fills = N >= 256 and E * -(-N // 256) >= 256
    if n > (STREAM_IF_FILLS if fills else STREAM_ELSE) * E:
        return ("wide" if N >= 256 else "tiles", glu)
    most = cap if layout == "ll" and cap < T else T
    direct = most <= DIRECT_ROWS and n * K <= 2 ** 31 - 1
    split = min(n, E) * -(-N // 64) < STREAM_WAVES
    return ("stream", glu, n <= FEW_PER_EXPERT * E, split, not direct)


def row_form(rows: int, H: int) -> tuple:
    """(vectors a thread, a wave to a row, threads) of the norm and the INT8 quantiser."""
    V = H // 8
    if rows < FEW_ROWS and V <= 1024:
        return 1, False, -(-V // 64) * 64
    if V <= 256:
        return (1 if V <= 64 else 2 if V <= 128 else 4), True, 256
    threads = 256 if V <= 512 else 512 if V <= 1024 else 1024
    return (2 if V <= 2 * threads else 4), False, threads


def route_form(T: int, E: int, many: int) -> tuple:
    """(lanes a token, experts a lane) of the scored routing."""
    G = 64 if E > WAVE_EXPERTS or T <= (WAVE_MANY if E > many else WAVE_FEW) else 16
    per = -(-E // G)
    for p in ((1, 2, 4, 8) if G == 64 else (2, 4, 8)):
        if per <= p:
            return G, p
    return G, 16


def stores_form(k: int, rows: int, row_bytes: int, stores: str) -> tuple:
    """(k it is compiled for, non-temporal) of the dispatch of 8-bit rows."""
    size = rows * row_bytes
    nt = stores == "streaming" if stores != "auto" else size <= STORE_LOW << 20 or size > STORE_HIGH << 20
    return (k if k in (1, 2, 4, 8) else 0), nt


# Streaming GEMM: every mix of SwiGLU, ring, K split or not, table or not; layouts, slots, and a
# hot expert of more rows than one pass over the weights takes.
# (layout, R, cap, S, T, E, k, K, N, hot, form without glu)
STREAM_CASES = [
    ("ht", 1, 0, 0, 100, 64, 2, 64, 528, None, (True, False, False)),
    ("ht", 1, 0, 0, 100, 64, 2, 192, 528, 9, (True, False, False)),
    ("ht", 1, 0, 0, 128, 256, 1, 1088, 256, None, (True, False, False)),
    ("ll", 1, 70, 0, 200, 64, 1, 128, 528, 5, (True, False, False)),
    ("static", 4, 0, 2, 90, 64, 4, 320, 528, 7, (True, False, False)),
    ("ht", 1, 0, 0, 128, 64, 8, 64, 528, None, (False, False, False)),
    ("ht", 1, 0, 0, 128, 64, 8, 1088, 528, 3, (False, False, False)),
    ("ll", 1, 96, 0, 300, 64, 4, 192, 528, 11, (False, False, False)),
    ("static", 4, 0, 2, 128, 64, 8, 128, 528, 1, (False, False, False)),
    ("ht", 1, 0, 0, 200, 64, 1, 192, 528, None, (True, False, True)),
    ("ht", 1, 0, 0, 300, 64, 1, 1088, 528, 2, (True, False, True)),
    ("ll", 1, 160, 0, 340, 64, 1, 64, 528, 63, (True, False, True)),
    ("static", 4, 0, 2, 190, 64, 2, 256, 528, 0, (True, False, True)),
    ("ht", 1, 0, 0, 200, 64, 4, 64, 528, None, (False, False, True)),
    ("ht", 1, 0, 0, 250, 64, 8, 1088, 528, 4, (False, False, True)),
    ("static", 4, 0, 2, 250, 64, 8, 448, 528, 60, (False, False, True)),
    ("ht", 1, 0, 0, 1, 8, 1, 64, 16, None, (True, True, False)),
    ("ht", 1, 0, 0, 90, 32, 2, 1088, 48, 3, (True, True, False)),
    ("ht", 1, 0, 0, 120, 8, 3, 640, 272, 2, (False, True, False)),
    ("static", 4, 0, 2, 100, 8, 4, 192, 80, 5, (False, True, False)),
    ("ht", 1, 0, 0, 190, 40, 1, 192, 112, None, (True, True, True)),
    ("ht", 1, 0, 0, 230, 48, 1, 1088, 208, 17, (True, True, True)),
    ("static", 4, 0, 2, 140, 64, 2, 64, 144, 3, (True, True, True)),
    ("ht", 1, 0, 0, 200, 8, 2, 320, 144, 6, (False, True, True)),
]
# rows of every expert at and around each boundary of the large tiles' forms
WIDE_ROWS = [0, 1, 8, 9, 16, 17, 32, 33, 64, 65, 96, 97, 128, 129, 160, 161, 192, 193, 224, 225, 256, 257,
             320, 321, 385, 400, 512, 641]
WIDE_CASES = [(64, 256), (128, 272), (192, 512), (256, 528), (320, 256), (384, 304), (448, 272), (1088, 256)]
TILE_CASES = [(64, 16), (128, 144), (192, 240), (1088, 112)]
# rows, channels: rows to a wave, to workgroups of 256, 512 and 1024 threads
ROW_CASES = [(4096, 8), (4097, 512), (4099, 520), (4098, 1024), (4099, 1032), (4097, 2048), (4096, 2056),
             (4099, 4096), (4096, 4104), (4099, 7168), (4096, 8192), (4097, 8200), (4096, 16392),
             (4095, 2048), (300, 8192), (70, 8200), (40, 16392)]
# tokens, experts, k, groups, kept
ROUTE_CASES = [(70, 60, 6, 10, 3), (90, 100, 8, 4, 2), (300, 256, 8, 8, 4), (60, 384, 8, 8, 3), (33, 1024, 16, 64, 33),
               (2051, 20, 3, 4, 2), (2050, 32, 16, 1, 1), (2049, 33, 5, 11, 3), (2055, 64, 8, 8, 3),
               (4097, 65, 6, 13, 4), (4099, 100, 8, 20, 7), (4103, 128, 8, 1, 1), (4098, 130, 4, 2, 1),
               (4101, 256, 16, 16, 5)]
ROUTE_BWD_CASES = [(70, 60, 6), (90, 100, 8), (300, 256, 8), (60, 384, 8), (33, 1024, 16), (2051, 20, 3),
                   (2050, 32, 16), (2049, 33, 5), (2055, 64, 8), (2053, 100, 8), (2063, 128, 16), (4097, 130, 4),
                   (4101, 256, 16)]
# tokens, channels, k, stores
STORE_CASES = [(T, 512, k, s) for T, k in ((33, 1), (64, 2), (65, 4), (70, 8), (40, 3)) for s in ("cached", "streaming")] + \
    [(1200, 7168, 8, "auto"), (1000, 7168, 8, "auto"), (5000, 7168, 3, "auto"), (20, 16512, 16, "cached")]
