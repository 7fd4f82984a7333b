"""Float64 definitions of the 8-bit checkpoint and of the group norm on node rows (test side)."""
import numpy as np

BLOCK = 32


def keep64(x, fmt):
    """(values, codes as values, scale bytes) of the checkpoint of x [rows, cols] (float64 of the stored type)."""
    x = np.asarray(x, np.float64)
    top = 127.0 if fmt == "int8" else 448.0
    val, code = np.zeros_like(x), np.zeros_like(x)
    byte = np.zeros((x.shape[0], -(-x.shape[1] // BLOCK)), np.uint8)
    for r in range(x.shape[0]):
        for b in range(byte.shape[1]):
            v = x[r, b * BLOCK:(b + 1) * BLOCK]
            if not np.isfinite(v).all():
                byte[r, b] = 255
                val[r, b * BLOCK:(b + 1) * BLOCK] = np.nan
                continue
            amax = np.abs(v).max()
            e = max(-126, int(np.floor(np.log2(amax))) - 9) if amax > 0 else -126
            while amax > top * 2.0 ** e:
                e += 1
            t = v / 2.0 ** e
            if fmt == "int8":
                q = np.rint(t)
            else:
                step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** -6))) - 3)
                q = np.rint(t / step) * step
            byte[r, b] = e + 127
            code[r, b * BLOCK:(b + 1) * BLOCK] = q
            val[r, b * BLOCK:(b + 1) * BLOCK] = q * 2.0 ** e
    return val, code, byte


def _sigmoid(t):
    return 1.0 / (1.0 + np.exp(-t))


def norm64(x, w, b, lmax, groups, ptr, eps, act, grad=None, stats=None):
    """Forward (out, stats), or with grad the backward (dx, dw, db), from the formulas; stats given or computed."""
    x = np.asarray(x, np.float64)
    n, dim = x.shape
    k = (lmax + 1) ** 2
    c = dim // k
    x = x.reshape(n, k, c)
    w = np.ones((lmax + 1, c)) if w is None else np.asarray(w, np.float64)
    b = np.zeros(c) if b is None else np.asarray(b, np.float64)
    out = np.zeros_like(x)
    st = np.zeros((len(ptr) - 1, lmax + 2, groups))
    dw, db = np.zeros_like(w), np.zeros(c)
    ranks = [range(l * l, (l + 1) ** 2) for l in range(lmax + 1)]

    def spread(v):
        return np.repeat(v, c // groups)

    def group_mean(v):     # [rows, comps, c] -> [groups]
        return v.reshape(v.shape[0], v.shape[1], groups, -1).mean((0, 1, 3))
    for s in range(len(ptr) - 1):
        lo, hi = ptr[s], ptr[s + 1]
        if lo >= hi:
            continue
        v = x[lo:hi]
        if stats is None:
            st[s, 0] = group_mean(v[:, :1])
            for l in range(lmax + 1):
                d = v[:, ranks[l]] - (spread(st[s, 0]) if l == 0 else 0)
                st[s, 1 + l] = 1 / np.sqrt(group_mean(d * d) + eps)
        else:
            st[s] = np.asarray(stats[s], np.float64)
        hat, y = np.zeros_like(v), np.zeros_like(v)
        for l in range(lmax + 1):
            hat[:, ranks[l]] = (v[:, ranks[l]] - (spread(st[s, 0]) if l == 0 else 0)) * spread(st[s, 1 + l])
            y[:, ranks[l]] = hat[:, ranks[l]] * w[l] + (b if l == 0 else 0)
        f = _sigmoid(y[:, :1]) if act == "silu" else np.ones_like(y[:, :1])
        if grad is None:
            out[lo:hi] = y * f
            continue
        g = np.asarray(grad, np.float64).reshape(n, k, c)[lo:hi]
        dy = g * f
        if act == "silu":
            dy[:, 0] += (f * (1 - f))[:, 0] * (g * y).sum(1)
        db += dy[:, 0].sum(0)
        for l in range(lmax + 1):
            u, h = hat[:, ranks[l]], dy[:, ranks[l]] * w[l]
            dw[l] += (dy[:, ranks[l]] * u).sum((0, 1))
            d = h - u * spread(group_mean(h * u)) - (spread(group_mean(h)) if l == 0 else 0)
            out[lo:hi, ranks[l]] = d * spread(st[s, 1 + l])
    out = out.reshape(n, dim)
    return (out, st) if grad is None else (out, dw, db)


def norm_bounds(x, w, b, lmax, groups, ptr, act, stats, eps_type, grad=None, tiny=0.0):
    """Error bounds of a float32 evaluation whose result is rounded to a type of eps_type, element by
    element, from the formulas: out, or (dx, dw, db).

    u = 2^-24 is half a step of float32, relative. The statistics of a forward are off by at most 16 u
    (a row's at most 28 squares are added in float32, the square root halves that, then one rounding);
    those of a backward are given. A logistic function is off by (5 + 1.2 |y|) 2 u, by the bounds of
    CUDA's __expf and __fdividef. A sum of h xhat runs over at most `terms` float32 additions.
    """
    u = 2.0 ** -24
    x = np.asarray(x, np.float64)
    n, dim = x.shape
    k = (lmax + 1) ** 2
    c = dim // k
    terms = (-(-n // 148) + 8) * 7 + 256
    x = x.reshape(n, k, c)
    w = np.ones((lmax + 1, c)) if w is None else np.asarray(w, np.float64)
    b = np.zeros(c) if b is None else np.asarray(b, np.float64)
    rank = np.concatenate([[l] * (2 * l + 1) for l in range(lmax + 1)])
    wk = w[rank]
    out = np.zeros_like(x)
    dw, db = np.zeros_like(w), np.zeros(c)

    def spread(v):
        return np.repeat(v, c // groups, -1)
    for s in range(len(ptr) - 1):
        lo, hi = ptr[s], ptr[s + 1]
        if lo >= hi:
            continue
        st = np.asarray(stats[s], np.float64)
        r = spread(st[1:])[rank]
        mu = np.where(rank[:, None] == 0, spread(st[0])[None], 0.0)
        bk = np.where(rank[:, None] == 0, b[None], 0.0)
        hat = (x[lo:hi] - mu) * r
        ax = (np.abs(x[lo:hi]) + np.abs(mu)) * r
        y = hat * wk + bk
        d_hat = (20 if grad is None else 4) * u * ax
        d_y = np.abs(wk) * d_hat + 3 * u * (np.abs(wk) * ax + np.abs(bk))
        if act == "silu":
            f = _sigmoid(y[:, :1])
            # __fdividef gives 0 for divisors above 2^126: a logistic value below 2^-126 may become 0, which
            # is 2^-126 off at most, relative to f
            e_f = (1 - f) * d_y[:, :1] + 2 * u * (5 + 1.2 * np.abs(y[:, :1])) + 2.0 ** -126 / f
        else:
            f, e_f = np.ones_like(y[:, :1]), np.zeros_like(y[:, :1])
        if grad is None:
            o = np.abs(y * f)
            out[lo:hi] = d_y * f + o * (e_f + 3 * u + eps_type / 2) + tiny
            continue
        g = np.abs(np.asarray(grad, np.float64).reshape(n, k, c)[lo:hi])
        gs = np.asarray(grad, np.float64).reshape(n, k, c)[lo:hi]
        dy, d_dy = gs * f, g * f * (e_f + 3 * u)
        if act == "silu":
            fp = (f * (1 - f))[:, 0]
            t = (g * np.abs(y)).sum(1)
            d_t = (g * d_y).sum(1) + (k + 4) * u * t
            d_fp = (f * (1 - f) * e_f + f * (f * e_f + u))[:, 0]
            dy = dy.copy()
            dy[:, 0] += fp * (gs * y).sum(1)
            d_dy[:, 0] += d_fp * t + fp * d_t + 2 * u * fp * t
        cell = np.abs(dy * hat)
        d_cell = d_dy * np.abs(hat) + np.abs(dy) * d_hat
        db += d_dy[:, 0].sum(0) + terms * u * np.abs(dy[:, 0]).sum(0)
        h, d_h = dy * wk, np.abs(wk) * d_dy
        for l in range(lmax + 1):
            m = rank == l
            dw[l] += (d_cell[:, m] + terms * u * cell[:, m]).sum((0, 1))

            def group_mean(v):
                return spread(v.reshape(v.shape[0], v.shape[1], groups, -1).mean((0, 1, 3)))
            along = np.abs(group_mean(h[:, m] * hat[:, m]))
            d_along = group_mean(np.abs(w[l]) * (d_cell[:, m] + terms * u * cell[:, m]))
            level = np.abs(group_mean(h[:, m])) if l == 0 else 0.0
            d_level = group_mean(d_h[:, m] + terms * u * np.abs(h[:, m])) if l == 0 else 0.0
            ah = np.abs(hat[:, m])
            d = d_h[:, m] + d_hat[:, m] * along + ah * d_along + d_level
            d = d + 6 * u * (np.abs(h[:, m]) + ah * along + level)
            size = np.abs(h[:, m]) + ah * along + level
            out[lo:hi, m] = (d + eps_type / 2 * np.minimum(size, np.abs(
                h[:, m] - hat[:, m] * group_mean(h[:, m] * hat[:, m]) - (group_mean(h[:, m]) if l == 0 else 0)) + d)
                + 2 * u * size) * r[m] + tiny
    out = out.reshape(n, dim)
    return out if grad is None else (out, dw, db)
