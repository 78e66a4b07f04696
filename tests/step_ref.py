"""Plain 64-bit implementations of the serving-step operators (numpy) and the error bounds of
their GPU forms, for the tests.

Bounds.  u = torch.finfo(t).eps / 2 is the relative error of one rounding to type t.

norm + rotation: y = a c - b s of a normalised head.  fp32: the sum of D squares is off by at
most D 2^-24 relative, its inverse root by half of that and 2 more roundings, the products and
the sum by a few 2^-24 of |a| + |b|; then one rounding to t.  So
|err| <= u |y| + (D / 2 + 10) 2^-24 (|a| + |b|) + tiny, |a| + |b| <= 2 max_d |head|, tiny = half
the type's smallest subnormal.

attention: o = sum p v / sum p, A = sum p |v| / sum p.
 * scores: fp32 sums of W products, |ds| <= W 2^-23 scale sum |q| |k|; a weight is then off by
   exp(ds) - 1 <= 2 ds relative, numerator and denominator each: 4 ds A together;
 * weights rounded to t before the value product: u A; their exponential 2^-21 A;
 * the value sums of n terms, fp32: n 2^-23 A;
 * the result: u |o| + tiny.
expanded form: K and V are rounded to t: u A for V, ds grows by u scale sum |q| |k| for K; their
fp32 sums of R products add R 2^-23 sum |c| |w|.
"""
import numpy as np

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25, "f32": 2.0 ** -149}


def torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def step_tables(lens, new, seq_ptr, table, free, P):
    """(table, seq_ptr, lens, new_ptr, slots, positions, pages taken) as Python lists."""
    t_out, ptr, nptr, slots, pos, took = [], [0], [0], [], [], 0
    for s in range(len(lens)):
        pages = [int(x) for x in table[seq_ptr[s]:seq_ptr[s + 1]]]
        while len(pages) * P < lens[s] + new[s]:
            pages.append(int(free[took]))
            took += 1
        for i in range(int(lens[s]), int(lens[s] + new[s])):
            slots.append(pages[i // P] * P + i % P)
            pos.append(i)
        t_out += pages
        ptr.append(len(t_out))
        nptr.append(nptr[-1] + int(new[s]))
    return t_out, ptr, [int(a + b) for a, b in zip(lens, new)], nptr, slots, pos, took


def norm(x, w, eps):
    """x [..., D] in float64; w None: unchanged."""
    if w is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def rotate(x, cos, sin, inter):
    """x [T, H, D]; cos, sin [T, rot / 2]: the first rot dims turned."""
    y, half = x.copy(), cos.shape[1]
    if inter:
        a, b = np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)
    else:
        a, b = np.arange(half), np.arange(half, 2 * half)
    c, s = cos[:, None], sin[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def angles(table, pos, sections):
    """cos, sin [T, rot / 2] from the fp32 table [max_pos, rot] and positions [axes, T]."""
    half = table.shape[1] // 2
    axis = np.repeat(np.arange(len(sections)), sections)
    p = pos[axis].T
    return table[p, np.arange(half)].astype(np.float64), table[p, half + np.arange(half)].astype(np.float64)


def rope_bound(y, x, dtype):
    D = x.shape[-1]
    big = 2 * np.abs(x).max(-1, keepdims=True)
    return U[dtype] * np.abs(y) + (D / 2 + 10) * 2.0 ** -24 * big + TINY[dtype]


def cos_sin(max_pos, rot, theta=10000.0):
    ang = np.arange(max_pos)[:, None] * theta ** (-2 * np.arange(rot // 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def attention_row(q, k, v, scale, dtype, ds_extra=0.0, v_err=0.0):
    """One row: q [W], k [n, W], v [n, Dv]; (o, bound) with the bounds above."""
    n = len(k)
    if n == 0:
        return np.zeros(v.shape[1]), np.zeros(v.shape[1])
    s = k @ q * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    o, A = p @ v, p @ np.abs(v)
    ds = (np.abs(k) @ np.abs(q)).max() * abs(scale) * (len(q) * 2.0 ** -23 + ds_extra) + 2.0 ** -22 * np.abs(s).max()
    u = U[dtype]
    return o, u * np.abs(o) + (u + 4 * ds + 2.0 ** -21 + n * 2.0 ** -23) * A + v_err + TINY[dtype]
