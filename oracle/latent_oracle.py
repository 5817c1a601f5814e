"""float64 oracle of the paged latent cache: rotary positions, e4m3 rows, append,
read-back and the dense / sparse latent attention. Test infrastructure only."""
from __future__ import annotations

import numpy as np

from .cache_append_oracle import encode_e4m3
from .indexcache_oracle import decode_e4m3

LATENT, ROW, ROW_BYTES, GROUP = 512, 576, 656, 128


def _f64(x):
    return np.asarray(x.detach().cpu().double().numpy() if hasattr(x, "detach") else x, dtype=np.float64)


def rope(x, pos, freq, rot_off=0, layout="interleaved", mscale=1.0, transpose=False):
    """x [T, H, D]; the rotated pair of dims (u, v) as the complex number u + iv times mscale e^{+-i pos freq}."""
    y = _f64(x).copy()
    freq = _f64(freq)
    n = len(freq)
    ang = np.asarray(pos, dtype=np.float64)[:, None] * freq[None, :]
    turn = mscale * np.exp((-1j if transpose else 1j) * ang)[:, None, :]
    u = np.arange(n) * (2 if layout == "interleaved" else 1) + rot_off
    v = u + (1 if layout == "interleaved" else n)
    z = (y[..., u] + 1j * y[..., v]) * turn
    y[..., u], y[..., v] = z.real, z.imag
    return y


def pow2_scale(y):
    """Least 2^e >= max|y| / 448 over the last axis (finite values), -100 <= e <= 119; 1 where all are zero."""
    y = _f64(y)
    amax = np.where(np.isfinite(y), np.abs(y), 0.0).max(axis=-1)
    s = np.ones_like(amax)
    for i in np.ndindex(amax.shape):
        if amax[i] > 0:
            e = -100
            while e < 119 and 448.0 * 2.0 ** e < amax[i]:
                e += 1
            s[i] = 2.0 ** e
    return s


def pack(rows):
    """Latent rows [R, 576] -> (codes uint8 [R, 512], scales [R, 4]) of the latent dims."""
    y = _f64(rows)[:, :LATENT].reshape(-1, LATENT // GROUP, GROUP)
    s = pow2_scale(y)
    return encode_e4m3(y / s[..., None]).reshape(-1, LATENT), s


def unpack(raw):
    """e4m3 row bytes [..., 656] -> float64 rows [..., 576]."""
    raw = np.asarray(raw.cpu().numpy() if hasattr(raw, "cpu") else raw, dtype=np.uint8)
    lead = raw.shape[:-1]
    raw = np.ascontiguousarray(raw.reshape(-1, ROW_BYTES))
    codes = decode_e4m3(raw[:, :LATENT]).astype(np.float64)
    s = np.ascontiguousarray(raw[:, LATENT:LATENT + 16]).view(np.float32).astype(np.float64)
    half = np.ascontiguousarray(raw[:, LATENT + 16:]).view(np.uint16).astype(np.uint32) << 16
    rot = half.view(np.float32).astype(np.float64)
    return np.concatenate([codes * np.repeat(s, GROUP, axis=1), rot], axis=1).reshape(*lead, ROW)


def cache_rows(cache):
    """A paged cache [P, page_size, 576 | 656] -> float64 rows [P * page_size, 576]."""
    rows = unpack(cache) if cache.shape[-1] == ROW_BYTES else _f64(cache)
    return rows.reshape(-1, ROW)


def attend(q, rows, sink=None, gate=None, sm_scale=ROW ** -0.5):
    """One token: q [H, 576], rows [n, 576], sink [H] (or None), gate [H, 512]. Returns (out, lse, mass, reach):
    mass[h, d] = sum_j p_j |v_jd| (gated), reach[h] = the largest sm_scale * sum_d |q_d k_jd|."""
    H, n = q.shape[0], rows.shape[0]
    s = np.full(H, -np.inf) if sink is None else _f64(sink)
    z = sm_scale * (q @ rows.T) if n else np.zeros((H, 0))
    m = np.maximum(z.max(axis=1), s) if n else s
    safe = np.where(np.isfinite(m), m, 0.0)
    p = np.exp(z - safe[:, None])
    den = p.sum(axis=1) + np.exp(s - safe)
    with np.errstate(divide="ignore"):
        lse = np.where(den > 0, safe + np.log(den), -np.inf)
    w = p / np.where(den > 0, den, 1.0)[:, None]
    out, mass = w @ rows[:, :LATENT], w @ np.abs(rows[:, :LATENT])
    if gate is not None:
        g = 1.0 / (1.0 + np.exp(-_f64(gate)))
        out, mass = out * g, mass * g
    reach = sm_scale * (np.abs(q) @ np.abs(rows).T).max(axis=1) if n else np.zeros(H)
    return out, lse, mass, reach


def decode(q, cache, block_table, lens, sink=None, gate=None, sm_scale=ROW ** -0.5, bad_pages=()):
    """q [B, Q, H, 576]: (out, lse, mass, reach) stacked over [B, Q]. Rows of pages in `bad_pages` are not seen."""
    rows, qf = cache_rows(cache), _f64(q)
    ps = cache.shape[1]
    table = np.asarray(block_table.cpu() if hasattr(block_table, "cpu") else block_table)
    got = []
    for b in range(qf.shape[0]):
        n = min(max(int(lens[b]), 0), table.shape[1] * ps)
        for j in range(qf.shape[1]):
            p = np.arange(max(0, n - (qf.shape[1] - 1 - j)))
            page = table[b, p // ps].astype(np.int64)
            keep = (page >= 0) & (page < cache.shape[0]) & ~np.isin(page, list(bad_pages))
            at = page[keep] * ps + (p % ps)[keep]
            got.append(attend(qf[b, j], rows[at], sink, None if gate is None else _f64(gate)[b, j], sm_scale))
    return tuple(np.stack([g[i] for g in got]).reshape(qf.shape[0], qf.shape[1], *got[0][i].shape) for i in range(4))


def sparse(q, cache, slots, sink=None, gate=None, sm_scale=ROW ** -0.5):
    """q [B, H, 576], slots [B, k] (-1 or out of range: skipped)."""
    rows, qf = cache_rows(cache), _f64(q)
    at = np.asarray(slots.cpu() if hasattr(slots, "cpu") else slots, dtype=np.int64)
    got = []
    for b in range(qf.shape[0]):
        keep = at[b][(at[b] >= 0) & (at[b] < rows.shape[0])]
        got.append(attend(qf[b], rows[keep], sink, None if gate is None else _f64(gate)[b], sm_scale))
    return tuple(np.stack([g[i] for g in got]) for i in range(4))
