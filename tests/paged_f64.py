"""A paged KV cache in plain 64-bit numpy: what the tests hold the kernels to."""
import numpy as np


def rope_table(n, hd, theta=1e6):
    a = np.arange(n)[:, None] * theta ** (-2.0 * np.arange(hd // 2) / hd)
    return np.stack((np.cos(a), np.sin(a)), -1).astype(np.float32)


def places(starts, lens, table, page, n_pages, M):
    """Of each row: (sequence or -1, position, page or -1)."""
    out = []
    cut = np.clip(starts, 0, M)
    for row in range(M):
        b = int(np.searchsorted(starts, row, side="right")) - 1
        if b < 0 or b >= len(lens) or not cut[b] <= row < cut[b + 1]:
            out.append((-1, 0, -1))
            continue
        p = int(lens[b]) - int(cut[b + 1]) + row
        out.append((b, p, page_of(table[b], p, page, n_pages)))
    return out


def page_of(row, p, page, n_pages):
    if p < 0 or p // page >= len(row):
        return -1
    at = int(row[p // page])
    return at if 0 <= at < n_pages else -1


def turned(x, w, cs, eps):
    """x [heads, hd], w [hd] or None, cs [hd / 2, 2] -> normalised (f64) and rotated (f64)."""
    x, cs = np.asarray(x, np.float64), np.asarray(cs, np.float64)
    if w is not None:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + np.float64(np.float32(eps))) * np.asarray(w, np.float64)
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return x, np.concatenate((a * cs[:, 0] - b * cs[:, 1], b * cs[:, 0] + a * cs[:, 1]), -1)


def attend(q, data, starts, lens, table, window=0, sinks=0, scale=None, max_rows=None, max_len=None):
    """(out, err, seen) of q [M, nh, hd] over data [pages, 2, nkv, page, hd]: the
    exact output, a dict of what the tolerances are made of, and which rows the
    call writes. Everything in f64."""
    M, nh, hd = q.shape
    n_pages, _, nkv, page, _ = data.shape
    G = nh // nkv
    scale = hd ** -0.5 if scale is None else scale
    q = np.asarray(q, np.float64)
    out, pv, qk, vmax = (np.zeros(q.shape) for _ in range(4))
    n = np.zeros((M, 1, 1))
    written = np.zeros(M, bool)
    cut = np.clip(starts, 0, M)
    for b in range(len(lens)):
        a, z = int(cut[b]), int(cut[b + 1])
        held = min(int(lens[b]), max_len) if max_len is not None else int(lens[b])
        held = max(held, 0)
        rows = np.arange(a, z)
        pos = held - (z - a) + np.arange(z - a)
        if max_rows is not None:
            rows, pos = rows[:max_rows], pos[:max_rows]
        written[rows] = True
        if not len(rows) or held == 0:
            continue
        at = np.array([page_of(table[b], j, page, n_pages) for j in range(held)])
        ok = at >= 0
        j = np.arange(held)
        k = np.zeros((held, nkv, hd))
        v = np.zeros((held, nkv, hd))
        k[ok] = data[at[ok], 0, :, j[ok] % page]
        v[ok] = data[at[ok], 1, :, j[ok] % page]
        sees = ok & (j <= pos[:, None])
        if window:
            sees &= (j > pos[:, None] - window) | (j < sinks)
        for h in range(nh):
            g = h // G
            for r0 in range(0, len(rows), 512):
                rr, ss = rows[r0:r0 + 512], sees[r0:r0 + 512]
                any_ = ss.any(0)
                if not any_.any():
                    continue
                kk, vv, s2 = k[any_, g], v[any_, g], ss[:, any_]
                with np.errstate(all="ignore"):
                    s = np.where(s2, q[rr, h] @ kk.T * scale, -np.inf)
                    top = s.max(-1, keepdims=True)
                    e = np.where(s2, np.exp(s - np.where(np.isneginf(top), 0, top)), 0)
                    tot = e.sum(-1, keepdims=True)
                    p = e / np.where(tot == 0, 1, tot)
                    # (a place that a row does not see has no part in it, whatever it holds)
                    fine = np.where(np.isfinite(vv), vv, 0)
                    out[rr, h] = p @ fine
                    for jj, dd in zip(*np.nonzero(~np.isfinite(vv))):
                        out[rr, h, dd] = np.where(s2[:, jj], out[rr, h, dd] + vv[jj, dd], out[rr, h, dd])
                    pv[rr, h] = p @ np.abs(fine)
                    mag = np.abs(q[rr, h]) @ np.abs(np.where(np.isfinite(kk), kk, 0)).T * abs(scale)
                    qk[rr, h] = np.where(s2, mag, 0).max(-1, keepdims=True)
                    vmax[rr, h] = np.abs(np.where(s2[:, :, None].any(0), fine, 0)).max()
                    n[rr] = np.maximum(n[rr], s2.sum(-1)[:, None, None])
    return out, {"pv": pv, "qk": qk, "vmax": vmax, "n": n}, written


def bound(err, out, hd, f16):
    """How far an attention output may be off. A score is a sum of hd products in
    f32 over hd / 8 matrix steps (each sum truncated: 2^-23 of the magnitudes),
    with f32 activations of queries kept to 22 bits (2^-22): ds. An output moves
    by at most 2 ds sum p |v|. Weights: an exponential within 2^-22 of its value
    for an argument rounded at 2^-24 of up to 128, and 64 more roundings of 2^-23
    with what joins the parts of a row, and one for every 16 positions that the
    sum runs over. With f32 activations a weight's two parts end at 2^-24 beside
    a largest weight of 2^12 or more: n 2^-36 max |v|. With f16 activations a
    weight is rounded by half a step, 2^-11 of it, or 2^-25 beside a largest
    weight of 1 or more where it is subnormal, and the output once: half a step,
    2^-11 of it, or 2^-25."""
    ds = err["qk"] * ((0 if f16 else 2.0 ** -22) + (hd / 8 + 4) * 2.0 ** -23)
    b = (2 * ds + (64 + err["n"] / 16) * 2.0 ** -23 + (2.0 ** -11 if f16 else 0)) * err["pv"]
    if f16:
        return b + err["n"] * 2.0 ** -25 * err["vmax"] + 2.0 ** -11 * (np.abs(out) + b) + 2.0 ** -24
    return b + err["n"] * 2.0 ** -36 * err["vmax"]
