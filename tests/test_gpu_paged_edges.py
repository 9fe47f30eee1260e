"""The paged operators at the edges of what their documentation allows: stops, overflowing steps,
counts updated in place by many CTAs, widely spread scales, long sums of small weights."""
import math
import time

import numpy as np
import pytest
import torch

from paged_helpers import (BF16_ROWS, check_chunk, chunk_reference, dequantised, plan_reference,
                           random_table)
from test_gpu_paged import Pool, _run, _values, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__
    __graft_entry__.build()
    import compressed_decode_attention_kvk_b200 as p
    assert torch.cuda.is_available()
    return p


@pytest.mark.parametrize("b,G,d", [(8, 0, 512), (16, 0, 512), (BF16_ROWS, 0, 512), (4, 32, 128),
                                   (8, 0, 128), (BF16_ROWS, 0, 192)])
def test_a_stop_at_any_moment_ends_soon(pkg, oracle_mod, b, G, d):
    """Wait limits that run out at different steps of the expanded-rows kernel: the two CTAs of a
    pair stop at different loads, the call ends without waiting for loads that never come (well
    under the two seconds that the kernel grants its own loads), and the next call is right."""
    q_lens, H = [40, 30], 40
    pool = Pool(pkg, oracle_mod, [1500, 700], d, 64, b, G, 64, 3)
    lay = pool.lay
    try:
        sigma = 1 / math.sqrt(d + 64)
        ql, qr = pool.queries(q_lens, H, torch.bfloat16, 1)
        _run(pool, pkg, pkg.KVK_PATH_TENSOR, q_lens, ql, qr, sigma, torch.bfloat16)
        stops = 0
        for limit in (1, 100, 300, 600, 1000, 1500, 2500, 4000, 8000, 16000):
            for _ in range(3):
                lay.set_wait_limit(limit)
                torch.cuda.synchronize()
                t0 = time.perf_counter()
                _run(pool, pkg, pkg.KVK_PATH_TENSOR, q_lens, ql, qr, sigma, torch.bfloat16)
                took = time.perf_counter() - t0
                status = lay.read_status(clear=True)
                assert status in (0, pkg.kvk.KVK_FLAG_TIMEOUT), limit
                stops += status != 0
                assert took < 1.0, f"limit {limit} ns: {took:.2f} s"
        assert stops >= 3
        lay.set_wait_limit(0)
        out, lse = _run(pool, pkg, pkg.KVK_PATH_TENSOR, q_lens, ql, qr, sigma, torch.bfloat16)
        pool.check(q_lens, ql, qr, out, lse, torch.bfloat16, sigma, True)
        assert lay.read_status() == 0
    finally:
        lay.close()


# ---------------------------------------------------------------------------------------
# steps that do not fit
# ---------------------------------------------------------------------------------------

def kept_plan(cached, new, free, count, table, page, max_new, pool_pages):
    """The plan of the tokens that are kept: the first max_new of the batch, and of those what fits
    the table row.  Returns (table, seq_lens, q_start, slots, positions, free count)."""
    table = [list(r) for r in table]
    cap = len(table[0]) * page
    cnt = min(max(count, 0), len(free))
    taken, row = 0, 0
    seq_lens, q_start, slots, positions = [], [0], [-1] * max_new, [0] * max_new
    for i, (a, f) in enumerate(zip(cached, new)):
        a, rows = min(max(a, 0), cap), min(max(f, 0), max_new - row)
        kept = min(rows, cap - a)
        for k in range(-(-a // page), -(-(a + kept) // page)):
            p = free[cnt - 1 - taken] if taken < cnt else -1
            table[i][k] = p if 0 <= p < pool_pages else -1
            taken += 1
        for k in range(kept):
            p = table[i][(a + k) // page]
            positions[row + k] = a + k
            slots[row + k] = p * page + (a + k) % page if 0 <= p < pool_pages else -1
        row += rows
        seq_lens.append(a + kept)
        q_start.append(row)
    return table, seq_lens, q_start, slots, positions, max(0, cnt - taken)


@pytest.mark.parametrize("batch,max_new", [(1, 0), (3, 5), (40, 100), (300, 1), (1000, 2500), (4096, 9000)])
def test_plan_keeps_the_first_max_new_tokens(pkg, batch, max_new):
    rng = np.random.default_rng(batch + max_new)
    page, width = 16, 6                              # rows of at most 96 tokens, some overflow
    cached = rng.integers(0, 90, batch).tolist()
    new = (rng.integers(0, 12, batch) * (rng.random(batch) < 0.8) + 1).astype(int).tolist()
    n_pages = batch * width + 3
    table = random_table(rng, cached, page, n_pages, width)
    held = set(table.ravel().tolist())
    free = [int(p) for p in rng.permutation(n_pages) if p not in held]
    lay = pkg.Layout([0], [64], [4], 64, 16, 1, n_pages * page)
    try:
        t = i32(table.tolist())
        p = lay.paged_plan(i32(cached), i32(new), i32(free), i32([len(free)]), t, page, max_new)
        ref = kept_plan(cached, new, free, len(free), table.tolist(), page, max_new, n_pages)
        got = (t.tolist(), p.seq_lens.tolist(), p.q_start.tolist(), p.slots.tolist(),
               p.positions.tolist(), p.free_count.item())
        for name, x, y in zip(("table", "seq_lens", "q_start", "slots", "positions", "free"), got, ref):
            assert x == y, name
        over = sum(new) > max_new or any(a + f > width * page for a, f in zip(cached, new))
        assert lay.read_status(clear=True) == (pkg.KVK_FLAG_SEQ_LEN if over else 0)
    finally:
        lay.close()


@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "apart"])
@pytest.mark.parametrize("batch,most,max_new", [(7, 2500, 9000), (200, 190, 40000), (4096, 9, 40000),
                                                (3, 100000, 300000)])
def test_plan_by_many_ctas(pkg, batch, most, max_new, in_place):
    """Plans that several CTAs share, the largest in grid strides (in place by a cluster of 8, else
    by 64 CTAs), with the free count updated in place or apart; the slots of one call after the
    other."""
    rng = np.random.default_rng(batch)
    page = 16
    cached = rng.integers(0, 70, batch).tolist()
    new = rng.integers(0, most, batch).tolist()
    assert sum(new) <= max_new and sum(new) > max_new // 4
    width = -(-(max(cached) + most) // page)
    n_pages = sum(-(-(a + f) // page) for a, f in zip(cached, new)) + 5
    table = random_table(rng, cached, page, n_pages, width)
    held = set(table.ravel().tolist())
    free = [int(p) for p in rng.permutation(n_pages) if p not in held]
    ref = plan_reference(cached, new, free, len(free), table.tolist(), page, max_new, n_pages)
    lay = pkg.Layout([0], [64], [4], 64, 16, 1, n_pages * page)
    try:
        c, f, fp = i32(cached), i32(new), i32(free)
        for rep in range(5):
            t, count = i32(table.tolist()), i32([len(free)])
            out = lay.new_paged_plan(batch, max_new)
            out = out._replace(free_count=count) if in_place else out
            for x in out:
                if x is not count:
                    x.fill_(-77)
            p = lay.paged_plan(c, f, fp, count, t, page, max_new, out=out)
            got = (t.tolist(), p.seq_lens.tolist(), p.q_start.tolist(), p.slots.tolist(),
                   p.positions.tolist(), p.free_count.item())
            for name, x, y in zip(("table", "seq_lens", "q_start", "slots", "positions", "free"), got, ref):
                assert x == y, (name, rep)
            assert in_place or int(count) == len(free)
        assert lay.read_status() == 0
    finally:
        lay.close()


@pytest.mark.parametrize("path", [1, 2], ids=["tensor", "cuda_core"])
@pytest.mark.parametrize("kind", ["max_new", "table_row"])
def test_an_overflowing_step_through_plan_write_and_attention(pkg, oracle_mod, kind, path):
    """More new tokens than max_new: the rows kept are those of their tokens' positions, nothing that
    was not written is read.  More than a table row holds: that sequence's rows are the last ones
    before the row's end, the other sequences are as ever."""
    d, dR, H, page, b = 128, 64, 6, 16, 8
    if kind == "max_new":
        cached, new, max_new, width = [20, 5, 40], [3, 6, 2], 7, 4
        lens, q_lens = [23, 9, 40], [3, 4, 0]
    else:
        cached, new, max_new, width = [20, 29, 7], [3, 6, 2], 11, 2
        lens, q_lens = [23, 32, 9], [3, 6, 2]
    B, N = 3, sum(new)
    g = torch.Generator().manual_seed(9)
    n_pages = 2 * B * width
    lay = pkg.Layout([0], [d], [b], d, dR, 1, n_pages * page)
    try:
        lay.set_decode_path(path)
        lay.arena[256:].random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(1))
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        free, count = i32(list(range(n_pages))), i32([n_pages])
        old = [_values(g, n, d, dR) for n in cached]
        plan = lay.paged_plan(i32([0] * B), i32(cached), free, count, table, page, sum(cached))
        lay.paged_write(0, torch.cat([c for c, _ in old]).cuda(), torch.cat([k for _, k in old]).cuda(),
                        plan.slots)
        assert lay.read_status() == 0
        fresh = [_values(g, n, d, dR) for n in new]
        plan = lay.paged_plan(i32(cached), i32(new), free, plan.free_count, table, page, max_new)
        assert lay.read_status(clear=True) == pkg.KVK_FLAG_SEQ_LEN
        # the caller's packed rows: all that it asked for; the map covers the first max_new
        c, kr = torch.cat([c for c, _ in fresh]).cuda(), torch.cat([k for _, k in fresh]).cuda()
        lay.paged_write(0, c[:max_new], kr[:max_new], plan.slots)
        ql = torch.randn(N, H, d, generator=g).to(torch.bfloat16)
        qr = torch.randn(N, H, dR, generator=g).to(torch.bfloat16)
        out = torch.full((N, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((N, H), 7.0, device="cuda")
        lay.mla_chunk(0, ql.cuda(), qr.cuda(), plan.q_start, plan.seq_lens, table, page, 0.07, out=out,
                      lse=lse)
        out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
        assert lay.read_status() == 0
        assert plan.seq_lens.tolist() == lens
        assert plan.q_start.tolist() == np.concatenate([[0], np.cumsum(q_lens)]).tolist()
        q = torch.cat([ql.double(), qr.double()], 2).numpy()
        row = 0
        for i, (n, m) in enumerate(zip(lens, q_lens)):
            if m == 0:
                continue
            rows, scale = dequantised(oracle_mod, torch.cat([old[i][0], fresh[i][0]])[:n],
                                      torch.cat([old[i][1], fresh[i][1]])[:n], d, b, 0)
            ref = chunk_reference(rows, q[row:row + m].reshape(m * H, -1),
                                  np.repeat(n - m + np.arange(m) + 1, H), d, 0.07)
            check_chunk(out[row:row + m].reshape(m * H, -1), lse[row:row + m].reshape(-1), ref,
                        torch.bfloat16, b, 0, d + dR, n, rows, scale, d, path == 1, f"seq {i}")
            row += m
        assert (out[row:] == 7.0).all() and (lse[row:] == 7.0).all()
    finally:
        lay.close()


@pytest.mark.parametrize("short", ["limit", "memory"])
def test_a_call_without_room_for_expanded_rows(pkg, oracle_mod, short):
    """No workspace given, and the expanded rows of the pool beyond the limit or refused by the
    allocator: the call converts the rows in the attention."""
    q_lens, H = [60, 50], 12
    pool = Pool(pkg, oracle_mod, [333, 200], 128, 64, 4, 0, 16, 8)
    lay = pool.lay
    try:
        N = sum(q_lens)
        base = lay.chunk_workspace_bytes(1, 0, 2, H)
        assert lay.chunk_workspace_bytes(1, N, 2, H) > base
        taken, make = [], lay._scratch

        def scratch(n):
            if n > base:
                raise torch.OutOfMemoryError("test")
            taken.append(n)
            return make(n)
        lay._scratch = scratch
        if short == "limit":
            lay._scratch_limit = lambda: base
        ql, qr = pool.queries(q_lens, H, torch.bfloat16, 4)
        lse = torch.empty(N, H, device="cuda")
        out = lay.mla_chunk(1, ql.cuda(), qr.cuda(), i32([0, 60, 110]), i32(pool.lens),
                            i32(pool.table.tolist()), pool.page, 0.07, lse=lse)
        pool.check(q_lens, ql, qr, out.cpu(), lse.cpu(), torch.bfloat16, 0.07, True)
        assert taken == [base] and lay.read_status() == 0
    finally:
        lay.close()


# ---------------------------------------------------------------------------------------
# weights of very different size
# ---------------------------------------------------------------------------------------

HALF16 = 2.0 ** -11


def _weighted_check(rows, scale, q, limits, d, sigma, out, lse, b, G, what):
    """Elementwise bound that counts the tensor-core kernel's roundings (see check_chunk), with f16's
    subnormals as they are: P_t is off by at most 2^-25, the largest P is at least 2^7, and P_t / l
    is s_t p_t (with group scales and bf16 rows p_t), so that a row's output is off by at most
    2^-32 max_t(s_t p_t) sum_t |code_t|."""
    n, T = rows.shape[1], len(rows)
    seen = np.arange(T)[None, :] < np.asarray(limits)[:, None]
    z = np.where(seen, (q @ rows.T) * sigma, -np.inf)
    m = z.max(1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(1, keepdims=True)
    p /= l
    ref = p @ rows[:, :d]
    unit = np.where(seen, (np.abs(q) @ np.abs(rows).T) * abs(sigma), 0.0).max(1, keepdims=True)
    rel = 2 * (n + 4) * 2.0 ** -24 * unit + 2 * T * 2.0 ** -24 + 2.0 ** -20 + HALF16
    if b == 16 or G:
        rel = rel + HALF16
    s = np.ones((T, 1)) if G else np.where(scale[:, :1] > 0, scale[:, :1], 1.0)
    # (in place of a scale of 0 the kernel takes 2^-24, f16's least)
    held = s if G else np.where(scale[:, :1] > 0, scale[:, :1], 2.0 ** -24)
    top = (p * held[:, 0]).max(1, keepdims=True)
    codes = np.abs(rows[:, :d]) / s
    sub = 2.0 ** -32 * top * (seen.astype(np.float64) @ codes)
    tol = (rel * (p @ np.abs(rows[:, :d])) + sub) * (1 + 2.0 ** -6) + np.abs(ref) * 2.0 ** -8 * 1.01 + 1e-30
    assert np.isfinite(out).all()
    worst = (np.abs(out - ref) / tol).max()
    assert worst <= 1.0, f"{what}: {worst:.2f} x the bound"
    le = (m + np.log(l))[:, 0]
    tl = (2 * (n + 4) * 2.0 ** -24 * unit + 2 * T * 2.0 ** -24 + 1e-5)[:, 0] + 2.0 ** -22 * np.abs(le)
    assert (np.abs(lse - le) <= tl).all(), f"{what}: lse"


def _attend(pkg, c, kr, d, b, G, ql, qr, sigma, path):
    T, N, H = len(c), ql.shape[0], ql.shape[1]
    lay = pkg.Layout([0], [d], [b], d, kr.shape[1], 1, -(-T // 64) * 64, scale_group=G)
    try:
        lay.paged_write(0, c.cuda(), kr.cuda(), torch.arange(T, dtype=torch.int32, device="cuda"))
        lay.set_decode_path(path)
        lse = torch.empty(N, H, device="cuda")
        out = lay.mla_chunk(0, ql.cuda(), qr.cuda(), i32([0, N]), i32([T]),
                            i32([list(range(-(-T // 64)))]), 64, sigma, lse=lse)
        assert lay.read_status() == 0
        return out.cpu().double().numpy().reshape(N * H, -1), lse.cpu().double().numpy().reshape(-1)
    finally:
        lay.close()


@pytest.mark.parametrize("q_len", [1, 16], ids=["one", "expanded"])
@pytest.mark.parametrize("gap", [12, 18, 24])
@pytest.mark.parametrize("b,G", [(8, 0), (16, 0), (4, 32), (2, 0)])
def test_many_small_weights_beside_a_large_one(pkg, oracle_mod, b, G, gap, q_len):
    """One token whose score is 2^gap times every other's weight and whose latents are zero: the
    output is made of the small weights alone, which must not vanish beside it."""
    d, dR, T, H, big = 128, 64, 5000, 20, 77
    g = torch.Generator().manual_seed(gap)
    c = (torch.rand(T, d, generator=g) + 0.5).to(torch.bfloat16)
    kr = torch.zeros(T, dR, dtype=torch.bfloat16)
    c[big] = 0
    kr[big, :32] = 2.0
    ql = torch.zeros(q_len, H, d, dtype=torch.bfloat16)
    qr = torch.zeros(q_len, H, dR, dtype=torch.bfloat16)
    qr[..., :32] = 1.0
    sigma = gap * math.log(2.0) / 64.0               # the large token's score: gap powers of two
    rows, scale = dequantised(oracle_mod, c, kr, d, b, G)
    q = torch.cat([ql.double(), qr.double()], 2).numpy().reshape(q_len * H, -1)
    lim = np.repeat(T - q_len + np.arange(q_len) + 1, H)
    out, lse = _attend(pkg, c, kr, d, b, G, ql, qr, sigma, pkg.KVK_PATH_TENSOR)
    _weighted_check(rows, scale, q, lim, d, sigma, out, lse, b, G, f"gap {gap}")


@pytest.mark.parametrize("q_len", [1, 3, 16])
@pytest.mark.parametrize("d", [64, 512])
@pytest.mark.parametrize("b", [2, 4, 8, 16])
def test_token_scales_far_apart_and_zero(pkg, oracle_mod, b, d, q_len):
    """Tokens of magnitudes from 2^-9 to 2^6 side by side, and tokens that are zero altogether (their
    score is 0, their scale too)."""
    dR, T, H = 64, 600, 20
    g = torch.Generator().manual_seed(b + d)
    mag = torch.exp2(torch.randint(-9, 7, (T, 1), generator=g).float())
    c = (torch.randn(T, d, generator=g) * mag).to(torch.bfloat16)
    kr = (torch.randn(T, dR, generator=g) * mag).to(torch.bfloat16)
    for t in (0, 5, 127, 128, 300, 598):
        c[t], kr[t] = 0, 0
    ql = torch.randn(q_len, H, d, generator=g).to(torch.bfloat16)
    qr = torch.randn(q_len, H, dR, generator=g).to(torch.bfloat16)
    sigma = 0.02 / math.sqrt(d / 64)
    rows, scale = dequantised(oracle_mod, c, kr, d, b, 0)
    assert (scale[:, 0] == 0).sum() == 6 and scale.max() / scale[scale > 0].min() > 2 ** 12
    q = torch.cat([ql.double(), qr.double()], 2).numpy().reshape(q_len * H, -1)
    lim = np.repeat(T - q_len + np.arange(q_len) + 1, H)
    for path in (pkg.KVK_PATH_TENSOR, pkg.KVK_PATH_CUDA_CORE):
        out, lse = _attend(pkg, c, kr, d, b, 0, ql, qr, sigma, path)
        _weighted_check(rows, scale, q, lim, d, sigma, out, lse, b, 0, f"path {path}")


@pytest.mark.parametrize("value", [0.0, 1.0])
def test_a_cache_of_equal_tokens(pkg, oracle_mod, value):
    """All tokens zero, or all the same: every weight is equal, lse is the logarithm of their count."""
    d, dR, T, H = 128, 64, 300, 8
    c, kr = torch.full((T, d), value), torch.full((T, dR), value)
    g = torch.Generator().manual_seed(1)
    for b, G in ((8, 0), (16, 0), (4, 32), (BF16_ROWS, 0)):
        for q_len in (1, 40):
            ql = torch.randn(q_len, H, d, generator=g).to(torch.bfloat16)
            qr = torch.randn(q_len, H, dR, generator=g).to(torch.bfloat16)
            for path in (pkg.KVK_PATH_TENSOR, pkg.KVK_PATH_CUDA_CORE):
                out, lse = _attend(pkg, c, kr, d, b, G, ql, qr, 0.05, path)
                rows, _ = dequantised(oracle_mod, c, kr, d, b, G)
                q = torch.cat([ql.double(), qr.double()], 2).numpy()
                z = (q @ rows[0]) * 0.05
                n = T - q_len + np.arange(q_len) + 1
                le = (z + np.log(n)[:, None]).reshape(-1)
                # the mean of equal values: the rows' high part, P (the same for all tokens), the
                # sums of T terms, the output's half step
                step = 2.0 ** -11 + 2.0 ** -8 + 2 * T * 2.0 ** -24 + 2.0 ** -8 * 1.01
                assert np.abs(out - rows[0, :d]).max() <= np.abs(rows[0, :d]).max() * step
                dz = (d + dR + 4) * 2.0 ** -24 * (np.abs(q) @ np.abs(rows[0])).max() * 0.05
                assert np.abs(lse - le).max() <= 2 * dz + 2 * T * 2.0 ** -24 + 1e-5


# ---------------------------------------------------------------------------------------
# group scales, and the contiguous calls beside the paged ones
# ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("q_lens", [[3, 1], [70, 90]], ids=["few", "expanded"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("b,G", [(16, 32), (8, 64), (4, 32), (2, 16)])
@pytest.mark.parametrize("d,dR", [(512, 64), (384, 64), (256, 64), (64, 32)])
def test_group_scales_at_every_rank(pkg, oracle_mod, d, dR, b, G, dtype, q_lens):
    """Group-scaled rows under bf16 and f16 queries at the ranks whose rings and stages differ."""
    if (d + dR) % G:
        pytest.skip("the group does not divide the row")
    lens, H = [333, 260], 9
    pool = Pool(pkg, oracle_mod, lens, d, dR, b, G, 32, d + b + G)
    try:
        assert pool.lay.chunk_path_for(0, dtype) == pkg.KVK_PATH_TENSOR
        sigma = 1 / math.sqrt(d + dR)
        ql, qr = pool.queries(q_lens, H, dtype, 7, gain=1.5)
        for path in (pkg.KVK_PATH_TENSOR, pkg.KVK_PATH_CUDA_CORE):
            out, lse = _run(pool, pkg, path, q_lens, ql, qr, sigma, dtype)
            q = torch.cat([ql.double(), qr.double()], 2).numpy()
            row = 0
            for i, (n, m) in enumerate(zip(lens, q_lens)):
                ref = chunk_reference(pool.rows[i], q[row:row + m].reshape(m * H, -1),
                                      np.repeat(n - m + np.arange(m) + 1, H), d, sigma)
                o = out[row:row + m].double().numpy().reshape(m * H, -1)
                if dtype == torch.float16:
                    # an f16 below 2^-14 has steps of 2^-24, whatever its value: its rounding is off by
                    # up to 2^-25 (a feature that only tokens of weight 3e-8 hold: -3.5e-8 rounds to
                    # -6.0e-8), which the half step relative to the value does not count
                    e = o - ref[0]
                    o = ref[0] + np.sign(e) * np.maximum(np.abs(e) - 2.0 ** -25, 0.0)
                check_chunk(o, lse[row:row + m].double().numpy().reshape(-1), ref, dtype, b, G, d + dR, n,
                            pool.rows[i], pool.scale[i], d, path == pkg.KVK_PATH_TENSOR,
                            f"path {path} seq {i}")
                row += m
        assert pool.lay.read_status() == 0
    finally:
        pool.lay.close()


@pytest.mark.parametrize("b,G", [(8, 0), (16, 0), (4, 32), (BF16_ROWS, 0)])
def test_decode_steps_beside_the_contiguous_calls(pkg, oracle_mod, b, G):
    """A prompt and then one-token steps, through plan, write and chunk attention and through
    kvk_quant_write and kvk_mla_decode over a contiguous cache: both within their bounds of the fp64
    form, and of one another."""
    d, dR, H, page, steps = 256, 64, 12, 16, 6
    prompt = [45, 130, 7]
    B, top = len(prompt), max(prompt) + steps
    g = torch.Generator().manual_seed(b + 6)
    c = [_values(g, n + steps, d, dR) for n in prompt]
    n_pages = sum(-(-(n + steps) // page) for n in prompt) + 2
    paged = pkg.Layout([0], [d], [b], d, dR, 1, n_pages * page, scale_group=G)
    flat = pkg.Layout([0], [d], [b], d, dR, B, top, scale_group=G)
    sigma = 1 / math.sqrt(d + dR)
    try:
        table = torch.full((B, -(-top // page)), -1, dtype=torch.int32, device="cuda")
        free, count = i32(list(range(n_pages))), i32([n_pages])
        cached, done = i32([0] * B), [0] * B
        for step in range(steps + 1):
            new = prompt if step == 0 else [1] * B
            N = sum(new)
            cs = [c[i][0][done[i]:done[i] + new[i]] for i in range(B)]
            ks = [c[i][1][done[i]:done[i] + new[i]] for i in range(B)]
            plan = paged.paged_plan(cached, i32(new), free, count, table, page, N)
            paged.paged_write(0, torch.cat(cs).cuda(), torch.cat(ks).cuda(), plan.slots)
            wide = max(new)                          # (rows behind a prompt's end lie past the cache)
            cf, kf = torch.zeros(B, wide, d, dtype=cs[0].dtype), torch.zeros(B, wide, dR, dtype=cs[0].dtype)
            for i in range(B):
                cf[i, :new[i]], kf[i, :new[i]] = cs[i], ks[i]
            flat.quant_write(0, cf.cuda(), kf.cuda(), cached)
            flat.read_status(clear=True)             # (and are flagged as such)
            done = [a + n for a, n in zip(done, new)]
            cached, count = plan.seq_lens, plan.free_count
            if step == 0:
                continue
            ql = torch.randn(B, H, d, generator=g).to(torch.bfloat16)
            qr = torch.randn(B, H, dR, generator=g).to(torch.bfloat16)
            lse, lse_flat = torch.empty(B, H, device="cuda"), torch.empty(B, H, device="cuda")
            out = paged.mla_chunk(0, ql.cuda(), qr.cuda(), plan.q_start, plan.seq_lens, table, page, sigma,
                                  lse=lse).cpu().double().numpy()
            out_flat = flat.mla_decode(0, ql.cuda(), qr.cuda(), plan.seq_lens, sigma,
                                       lse=lse_flat).cpu().double().numpy()
            lse, lse_flat = lse.cpu().double().numpy(), lse_flat.cpu().double().numpy()
            for i, n in enumerate(done):
                rows, scale = dequantised(oracle_mod, c[i][0][:n], c[i][1][:n], d, b, G)
                q = torch.cat([ql[i].double(), qr[i].double()], 1).numpy()
                ref = chunk_reference(rows, q, [n] * H, d, sigma)
                args = (b, G, d + dR, n, rows, scale, d, True)
                check_chunk(out[i], lse[i], ref, torch.bfloat16, *args, f"paged, step {step} seq {i}")
                check_chunk(out_flat[i], lse_flat[i], ref, torch.float32, *args, f"flat, step {step} seq {i}")
                dz = ((d + dR + 4) * 2.0 ** -24 * ref[3])[:, None]
                rel = 2 * dz + 2 * n * 2.0 ** -24 + 2.0 ** -20 + (2.0 ** -8 if b == BF16_ROWS else 2.0 ** -10)
                tol = 2 * rel * ref[2] * (1 + 2.0 ** -6) + np.abs(ref[0]) * 2.0 ** -8 * 1.02 + 1e-6
                assert (np.abs(out[i] - out_flat[i]) <= tol).all()
                assert (np.abs(lse[i] - lse_flat[i]) <= 4 * dz[:, 0] + 4 * n * 2.0 ** -24 + 2e-5).all()
        assert paged.read_status() == 0 and flat.read_status() == 0
    finally:
        paged.close()
        flat.close()


@pytest.mark.parametrize("b,G,d,H,q_lens", [(16, 0, 512, 40, [1] * 6), (8, 0, 512, 20, [90, 3, 1, 64, 0, 70]),
                                            (4, 32, 128, 40, [40] * 6), (BF16_ROWS, 0, 384, 24, [33] * 6)])
def test_calls_repeat_to_the_bit(pkg, oracle_mod, b, G, d, H, q_lens):
    """The work is split and joined by the lengths alone: the same call gives the same bits, also over
    a workspace that another call has used."""
    lens = [900, 300, 1, 640, 50, 2000]
    pool = Pool(pkg, oracle_mod, lens, d, 64, b, G, 64, 4)
    try:
        q_lens = [min(a, n) for a, n in zip(q_lens, lens)]
        N = sum(q_lens)
        ql, qr = pool.queries(q_lens, H, torch.bfloat16, 2)
        args = (ql.cuda(), qr.cuda(), i32(np.concatenate([[0], np.cumsum(q_lens)]).tolist()), i32(lens),
                i32(pool.table.tolist()), 64, 0.05)
        ws = pool.lay.new_chunk_workspace(0, N, len(lens), H)
        first = None
        for rep in range(8):
            if rep % 2:                              # the workspace's contents of a call of other sizes
                pool.lay.mla_chunk(0, args[0][:1], args[1][:1], i32([0] * 5 + [0, 1]), *args[3:], workspace=ws)
            lse = torch.empty(N, H, device="cuda")
            out = pool.lay.mla_chunk(0, *args, lse=lse, workspace=ws)
            if first is None:
                first = (out, lse)
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), rep
        pool.check(q_lens, ql, qr, first[0].cpu(), first[1].cpu(), torch.bfloat16, 0.05, True)
    finally:
        pool.lay.close()


@pytest.mark.parametrize("d,dR,b,G", [(528, 64, 8, 0), (1024, 64, 16, 0), (2032, 16, 4, 0), (1024, 64, 4, 32),
                                      (2048, 0, BF16_ROWS, 0), (128, 72, 8, 0), (128, 8, 2, 0), (48, 128, 16, 0),
                                      (512, 8, 4, 0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_widths_of_the_cuda_core_kernel_only(pkg, oracle_mod, d, dR, b, G, dtype):
    """Ranks beyond 512 and RoPE widths that the tensor-core kernel does not take, from one query token
    (a cluster splits the keys) to many."""
    lens, H = [150, 70], 9
    pool = Pool(pkg, oracle_mod, lens, d, dR, b, G, 16, d + b)
    try:
        assert pool.lay.chunk_path_for(0, dtype) == pkg.KVK_PATH_CUDA_CORE
        sigma = 1 / math.sqrt(d + dR)
        for q_lens in ([1, 0], [2, 1], [40, 30]):
            ql, qr = pool.queries(q_lens, H, dtype, 7, gain=1.5)
            out, lse = _run(pool, pkg, pkg.KVK_PATH_AUTO, q_lens, ql, qr, sigma, dtype)
            pool.check(q_lens, ql, qr, out, lse, dtype, sigma, False, f"{q_lens}")
        assert pool.lay.read_status() == 0
    finally:
        pool.lay.close()
