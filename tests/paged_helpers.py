"""Plain fp64 forms of the paged operators, and the error bounds of the kernels against them."""
from __future__ import annotations

import numpy as np
import torch

from gpu_helpers import bf16_or_f32_to_np

BF16_ROWS = 0
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def plan_reference(cached, new, free, free_count, table, page, max_new, pool_pages):
    """The plan in plain Python: (table, seq_lens, q_start, slots, positions, free_count)."""
    table = [list(r) for r in table]
    cap = len(table[0]) * page
    cnt = min(max(free_count, 0), len(free))
    left, taken, total = cnt, 0, 0
    seq_lens, q_start, slots, positions = [], [0], [-1] * max_new, [0] * max_new
    for i, (a, f) in enumerate(zip(cached, new)):
        a, f = min(max(a, 0), cap), max(f, 0)
        kept = min(f, cap - a)
        for k in range(-(-a // page), -(-(a + kept) // page)):
            p = free[cnt - 1 - taken] if taken < cnt else -1
            table[i][k] = p if 0 <= p < pool_pages else -1
            taken += 1
        for k in range(f):
            if total + k >= max_new:
                break
            if k < kept:
                pos = a + k
                positions[total + k] = pos
                p = table[i][pos // page]
                slots[total + k] = p * page + pos % page if 0 <= p < pool_pages else -1
        total = total + f
        seq_lens.append(a + kept)
        q_start.append(min(total, max_new))
    left = max(0, cnt - taken)
    return table, seq_lens, q_start, slots, positions, left


def random_table(rng, lens, page, n_pages, width):
    """A block table [batch][width] with distinct random pages of the pool for every sequence."""
    need = [-(-n // page) for n in lens]
    order = rng.permutation(n_pages)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    assert at <= n_pages
    return table


def dequantised(oracle, c, kr, d, b, group):
    """float64 rows [tokens, d + d_rope] that the cache stands for, and the scale of each element
    (1 for bf16 rows)."""
    cn, kn = bf16_or_f32_to_np(c), bf16_or_f32_to_np(kr)
    if b == BF16_ROWS:
        v = torch.cat([c[:, :d].float(), kr.float()], 1).to(torch.bfloat16).double().numpy()
        return v, np.ones_like(v)
    if group:
        _, s, k = oracle.quantize_rows_grouped(cn, kn, d, b, group)
        s = np.repeat(s.view(np.float16).astype(np.float64).reshape(len(cn), -1), group, 1)
    else:
        _, s, k = oracle.quantize_rows(cn, kn, d, b)
        s = s.view(np.float16).astype(np.float64).reshape(len(cn), 1)
    v = k.astype(np.float64) * s
    return v, np.broadcast_to(s, v.shape)


def chunk_reference(rows, q, limits, d, sigma):
    """rows [T, n], q [R, n] in float64, limits [R] tokens seen by each row -> out [R, d], lse
    [R], and what the bounds need: sum p |v| [R, d], the largest score error unit max_t sum
    |q c| |sigma| [R], the largest weight [R]."""
    R, T = len(q), len(rows)
    seen = np.arange(T)[None, :] < np.asarray(limits)[:, None]
    with np.errstate(all="ignore"):
        z = np.where(seen, (q @ rows.T) * sigma, -np.inf)
        m = z.max(1, keepdims=True) if T else np.full((R, 1), -np.inf)
        p = np.where(seen, np.exp(z - np.where(np.isfinite(m), m, 0.0)), 0.0)
        l = p.sum(1, keepdims=True)
        p = np.where(l > 0, p / np.where(l > 0, l, 1), 0.0)
        out = p @ rows[:, :d]
        lse = np.where(l[:, 0] > 0, m[:, 0] + np.log(np.where(l[:, 0] > 0, l[:, 0], 1)), -np.inf)
    unit = np.where(seen, (np.abs(q) @ np.abs(rows).T) * abs(sigma), 0.0).max(1) if T else np.zeros(R)
    return out, lse, p @ np.abs(rows[:, :d]), unit, (p.max(1) if T else np.zeros(R))


def check_chunk(out, lse, ref, dtype, b, group, n, T, rows, scale, d, tensor, what=""):
    """Elementwise bounds, counted from the kernel's roundings.
    Scores: n + 4 fp32 products and sums of exact operands, relative 2^-24 each of sum |q c| sigma
    (dz); a score error of dz moves a weight by at most the factor e^(2 dz).
    Tensor-core kernel: P in 16 bits (f16 2^-11, bf16 rows 2^-8), the output operand (16-bit and
    group-scaled codes 2^-11), f16 subnormals of P (2^-25 of a weight whose largest is at least
    that of the row), 2^-20 for the exponential, the references and the fp32 sums' constants;
    T 2^-24 for the sum over tokens; half a step of the output type."""
    o_ref, l_ref, pv, unit, pmax = ref
    dz = (n + 4) * 2.0 ** -24 * unit
    rel = 2 * dz + 2 * T * 2.0 ** -24 + 2.0 ** -20
    sub = 0.0
    if tensor:
        rel = rel + (2.0 ** -8 if b == BF16_ROWS else 2.0 ** -11)
        if b == 16 or group:
            rel = rel + 2.0 ** -11
        if b != BF16_ROWS and T:
            ratio = scale.max() / max(scale[scale > 0].min(), 1e-30) if (scale > 0).any() else 1.0
            sub = 2.0 ** -25 * ratio * np.abs(rows[:, :d]).sum(0)[None, :] * pmax[:, None]
    tol = (rel[:, None] * pv + sub) * (1 + 2.0 ** -6) + np.abs(o_ref) * HALF_STEP[dtype] * 1.01 + 1e-30
    err = np.abs(out - o_ref)
    assert np.isfinite(out).all(), f"{what}: not finite"
    worst = (err / tol).max() if err.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} x the bound, err {err.max():.3e} at {np.unravel_index((err / tol).argmax(), err.shape)}"
    fin = np.isfinite(l_ref)
    assert np.array_equal(np.isfinite(lse), fin), f"{what}: lse"
    assert (lse[~fin] == -np.inf).all()
    if fin.any():
        tl = 2 * dz + 2 * T * 2.0 ** -24 + 1e-5
        e = np.abs(lse[fin] - l_ref[fin]) / tl[fin]
        assert e.max() <= 1.0, f"{what}: lse {e.max():.2f} x its bound"
    return worst
