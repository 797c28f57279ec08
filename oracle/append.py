"""Plain definition of appending tokens to paged caches - TEST INFRASTRUCTURE.

Token by token, in fp64 numpy, sharing no code with the CUDA library:

* token i of a sequence lives in slot i % 16 of page pages[i // 16] and carries
  rotary position pos0 + i; pair (j, j + d/2) of K (and of the query) is turned
  by the table's (cos, sin) of that position; V is stored as it is;
* when slot 0 of a page is written, the page's slots behind the call's last
  token become zero;
* in the 8-bit pool a page block (page, head) has one scale. need = the
  smallest power of two, 2^-24 at least (2^7 at most for V), whose 448-fold
  covers the call's new values in the block; the scale is need when slot 0 is
  written, else max(need, the scale before); held values are rounded again to
  the codes of a grown scale.

Values are returned unrounded (the held ones of an 8-bit block after their one
rounding): the tests allow the stored type's half step around them.
"""

from __future__ import annotations

import numpy as np

PAGE = 16


def rotate(x: np.ndarray, cs: np.ndarray) -> np.ndarray:
    """x [..., d], cs [d/2, 2] = (cos, sin)."""
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return np.concatenate([a * cs[:, 0] - b * cs[:, 1], b * cs[:, 0] + a * cs[:, 1]], -1)


def e4m3_values() -> np.ndarray:
    """The 127 non-negative finite e4m3 values, ascending (code = index)."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to the even code, saturated at 448."""
    v = e4m3_values()
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(v, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - v[lo], v[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(v[pick], x)


def block_scale(amax: float, top: int) -> float:
    e = -24
    while e < top and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(pool_k, pool_v, ks, vs, seqs, k, v, table):
    """pool_k, pool_v: fp64 [pages][H][16][d], values (of an 8-bit pool: codes'
    values without the scale), changed in place; ks, vs: fp64 [pages][H] scales
    or None. seqs: list of (pages, start, n_new, pos0). k, v: fp64 [T][H][d].
    table: fp64 [n_pos][d/2][2] or None."""
    t = 0
    for pages, start, n, pos0 in seqs:
        if n == 0:
            continue
        rows_k = [rotate(k[t + i], table[pos0 + start + i]) if table is not None else k[t + i] for i in range(n)]
        rows_v = [v[t + i] for i in range(n)]
        t += n
        for a in range(start // PAGE, (start + n - 1) // PAGE + 1):
            s0, s1 = max(start - a * PAGE, 0), min(start + n - a * PAGE, PAGE)
            page = pages[a]
            for pool, scale, rows, top in ((pool_k, ks, rows_k, 120), (pool_v, vs, rows_v, 7)):
                new = np.stack([rows[a * PAGE + s - start] for s in range(s0, s1)], 1)   # [H, n, d]
                if s0 == 0:
                    pool[page, :, s1:] = 0
                if scale is not None:
                    for h in range(new.shape[0]):
                        need = block_scale(np.abs(new[h]).max(), top)
                        now = need if s0 == 0 else max(need, scale[page, h])
                        if s0 > 0 and now != scale[page, h]:
                            pool[page, h, :s0] = to_e4m3(pool[page, h, :s0] * (scale[page, h] / now))
                        scale[page, h] = now
                        new[h] /= now
                pool[page, :, s0:s1] = new
