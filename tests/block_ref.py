"""Test-side model of the fp8b pool and its operators: the byte layout, the append
with the position rotation, and causal attention in 64 bits.  Written from the
descriptions in include/kvq.h; it shares no code with the CUDA path (E4M3 codes
come from the oracle's codec)."""
from __future__ import annotations

import numpy as np

import oracle

D, PAGE, BT = 256, 256, 64
TILE_BYTES, CODES, PAGE_BYTES = 32768, 131072, 131200


def k_off(t, d):
    return (d >> 7) * 8192 + (t >> 3) * 1024 + (t & 7) * 128 + ((((d >> 4) & 7) ^ (t & 7)) << 4) + (d & 15)


def v_off(t, d):
    return (d >> 3) * 512 + (d & 7) * 64 + (((t >> 4) ^ ((d >> 1) & 3)) << 4) + (t & 15)


_T, _DIM = np.arange(BT)[:, None], np.arange(D)[None]
K_MAP, V_MAP = k_off(_T, _DIM), 16384 + v_off(_T, _DIM)


class Cache:
    """One layer of an fp8b pool: codes [slots, heads, 2 (K, V), 256 tokens, 256] and scales [slots, heads, 4, 2]."""

    def __init__(self, n_slots, heads):
        self.codes = np.zeros((n_slots, heads, 2, PAGE, D), np.uint8)
        self.scales = np.zeros((n_slots, heads, 4, 2), np.float32)
        self.nonfinite = False

    def pack(self) -> np.ndarray:
        n, h = self.codes.shape[:2]
        out = np.zeros((n, h, PAGE_BYTES), np.uint8)
        for b in range(4):
            tile = out[:, :, b * TILE_BYTES:(b + 1) * TILE_BYTES]
            tile[:, :, K_MAP] = self.codes[:, :, 0, b * BT:(b + 1) * BT]
            tile[:, :, V_MAP] = self.codes[:, :, 1, b * BT:(b + 1) * BT]
        out[:, :, CODES:CODES + 32] = self.scales.reshape(n, h, 8).view(np.uint8)
        return out

    @staticmethod
    def unpack(raw: np.ndarray) -> "Cache":
        n, h = raw.shape[:2]
        c = Cache(n, h)
        for b in range(4):
            tile = raw[:, :, b * TILE_BYTES:(b + 1) * TILE_BYTES]
            c.codes[:, :, 0, b * BT:(b + 1) * BT] = tile[:, :, K_MAP]
            c.codes[:, :, 1, b * BT:(b + 1) * BT] = tile[:, :, V_MAP]
        c.scales = np.ascontiguousarray(raw[:, :, CODES:CODES + 32]).view(np.float32).reshape(n, h, 4, 2).copy()
        return c

    def append(self, table, pos0, k, v):
        """Rows k, v [n, heads, 256] fp32 (K already rotated) of one sequence at positions pos0 .. ."""
        n, pos = len(k), pos0
        while pos < pos0 + n:
            lo, blk = pos % BT, pos // BT
            hi = min(BT, lo + pos0 + n - pos)
            slot, b = table[blk // 4], blk % 4
            for side, x in ((0, k), (1, v)):
                x = x[pos - pos0:pos - pos0 + hi - lo].astype(np.float32)
                if not np.isfinite(x).all():
                    self.nonfinite = True
                    x = np.nan_to_num(x, nan=0.0)
                for h in range(x.shape[1]):
                    amax = float(np.abs(x[:, h]).max())
                    old = float(self.scales[slot, h, b, side]) if lo else 0.0
                    d = max(old, pow2_scale(amax))
                    rows = self.codes[slot, h, side, b * BT:(b + 1) * BT]
                    if d != old and lo:
                        rows[:lo] = oracle.f32_to_e4m3((oracle.e4m3_to_f32(rows[:lo].ravel()).astype(np.float64) *
                                                        (old / d)).astype(np.float32)).reshape(lo, D)
                    with np.errstate(over="ignore"):
                        y = x[:, h].astype(np.float64) / d if d else np.zeros((hi - lo, D))
                    rows[lo:hi] = oracle.f32_to_e4m3(np.clip(y, -448, 448).astype(np.float32).ravel()).reshape(hi - lo, D)
                    if d == 0:
                        rows[lo:hi] = 0
                    self.scales[slot, h, b, side] = d
            pos += hi - lo

    def values(self, table, n, head):
        """K and V of the first n tokens of a sequence, fp64 [n, 256] each."""
        pages = np.asarray(table[:(n + PAGE - 1) // PAGE])
        out = []
        for side in (0, 1):
            c = oracle.e4m3_to_f32(np.ascontiguousarray(self.codes[pages, head, side]).ravel()).astype(np.float64)
            c = c.reshape(len(pages), 4, BT, D) * self.scales[pages, head, :, side].astype(np.float64)[:, :, None, None]
            out.append(c.reshape(-1, D)[:n])
        return out


def pow2_scale(amax: float) -> float:
    if not amax > 0:
        return 0.0
    e = -120
    while e < 118 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rotate(x, pos, table, interleaved):
    """x [n, heads, 256] fp32 at positions pos; every product and sum rounded once in fp32."""
    x = x.astype(np.float32).copy()
    rot = table.shape[1]
    half = rot // 2
    c, s = table[pos][:, None, :half], table[pos][:, None, half:]
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia], x[..., ib]
    with np.errstate(all="ignore"):
        x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def rope_table(n_pos, rot, base=10000.0):
    half = rot // 2
    ang = np.arange(n_pos)[:, None] * base ** (-np.arange(half) / max(half, 1))[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def attend(q, k, v, limits):
    """q [rows, 256] fp64, row r over keys 0 .. limits[r] - 1.  Returns (out, the largest sum |q k| / 16 per row)."""
    s = q @ k.T / 16
    s[np.arange(k.shape[0])[None] >= np.asarray(limits)[:, None]] = -np.inf
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    a = (np.abs(q) @ np.abs(k).T / 16).max(1)
    return p @ v, a
