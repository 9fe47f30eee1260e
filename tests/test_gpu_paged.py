"""The paged cache: plan (block tables, slot map), write through the slot map, and the attention
of chunks of new tokens, each against its plain fp64 (or integer) form, and the three run
together as a serving step does."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import bf16_or_f32_to_np
from paged_helpers import (BF16_ROWS, check_chunk, chunk_reference, dequantised, plan_reference,
                           random_table)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__
    __graft_entry__.build()
    import compressed_decode_attention_kvk_b200 as p
    assert torch.cuda.is_available()
    return p


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------------------

PLANS = {   # cached, new, page
    "decode": ([5, 16, 0, 31, 100], [1, 1, 1, 1, 1], 16),
    "prefill": ([0, 0, 0], [37, 1, 300], 32),
    "mixed": ([63, 64, 65, 0, 7], [2, 0, 129, 0, 1], 64),
    "page_1": ([3, 0], [4, 9], 1),
    "none": ([9, 4], [0, 0], 8),
    "one": ([0], [1], 128),
}


@pytest.mark.parametrize("case", PLANS, ids=str)
def test_plan_matches_reference(pkg, case):
    cached, new, page = PLANS[case]
    rng = np.random.default_rng(7)
    width = max(-(-(a + f) // page) for a, f in zip(cached, new)) + 2
    n_pages = sum(-(-(a + f) // page) for a, f in zip(cached, new)) + 5
    table = random_table(rng, cached, page, n_pages, width)
    free = np.array([p for p in rng.permutation(n_pages) if p not in set(table.ravel())], np.int32)
    _check_plan(pkg, cached, new, free, len(free), table, page, sum(new) + 3, n_pages)


def _check_plan(pkg, cached, new, free, count, table, page, max_new, n_pages, flags=0):
    lay = pkg.Layout([0], [64], [4], 64, 16, 1, n_pages * page)
    try:
        t = i32(table.tolist())
        fc = i32([count])
        p = lay.paged_plan(i32(cached), i32(new), i32(free.tolist()), fc, t, page, max_new)
        ref = plan_reference(cached, new, free.tolist(), count, table.tolist(), page, max_new,
                             n_pages)
        got = (t.tolist(), p.seq_lens.tolist(), p.q_start.tolist(), p.slots.tolist(),
               p.positions.tolist(), p.free_count.item())
        for name, x, y in zip(("table", "seq_lens", "q_start", "slots", "positions", "free"), got,
                              ref):
            assert x == y, name
        assert fc.item() == count
        assert lay.read_status(clear=True) == flags
    finally:
        lay.close()


@pytest.mark.parametrize("batch", [1, 33, 1000, 4096])
def test_plan_many_sequences(pkg, batch):
    rng = np.random.default_rng(batch)
    page = 16
    cached = rng.integers(0, 70, batch).tolist()
    new = (rng.integers(0, 9, batch) * (rng.random(batch) < 0.7)).astype(int).tolist()
    width = 7
    n_pages = sum(-(-(a + f) // page) for a, f in zip(cached, new)) + 3
    table = random_table(rng, cached, page, n_pages, width)
    held = set(table.ravel().tolist())
    free = np.array([p for p in rng.permutation(n_pages) if p not in held], np.int32)
    _check_plan(pkg, cached, new, free, len(free), table, page, sum(new) + 1, n_pages)


def test_plan_short_free_list_and_bad_lengths(pkg):
    page, n_pages = 8, 12
    table = np.full((3, 4), -1, np.int32)
    table[0, 0] = 11
    free = np.array([1, 2, 3], np.int32)
    F = pkg.kvk
    # the third sequence gets no second page
    _check_plan(pkg, [3, 0, 0], [6, 8, 16], free, 3, table, page, 30, n_pages, F.KVK_FLAG_PAGE)
    # a free page and a held page outside the pool
    t2 = table.copy()
    t2[0, 0] = 12
    _check_plan(pkg, [3, 0, 0], [2, 8, 0], np.array([1, 99], np.int32), 2, t2, page, 10, n_pages,
                F.KVK_FLAG_PAGE)
    # negative lengths, a row that overflows, more tokens than max_new
    _check_plan(pkg, [-4, 0, 30], [2, -1, 9], free, 3, np.where(table < 0, 5, table), page, 6,
                n_pages, F.KVK_FLAG_SEQ_LEN)
    # a free count beyond the list counts as its length
    _check_plan(pkg, [0, 0, 0], [1, 1, 1], free, 3, table, page, 3, n_pages)


def test_plan_updates_the_free_count_in_place(pkg):
    lay = pkg.Layout([0], [64], [4], 64, 16, 1, 64 * 16)
    try:
        table = torch.full((2, 20), -1, dtype=torch.int32, device="cuda")
        free, count = i32(list(range(40))), i32([40])
        cached = i32([0, 0])
        out = lay.new_paged_plan(2, 64)._replace(free_count=count)
        for step in range(20):   # each step's lengths are the next step's cached ones
            p = lay.paged_plan(cached, i32([3, 17]), free, count, table, 16, 64, out=out)
            cached = p.seq_lens.clone()
        assert cached.tolist() == [60, 320]          # the table row ends at 320
        used = table[table >= 0].tolist()
        assert len(used) == len(set(used))
        assert int(count) == 40 - len(used)
    finally:
        lay.close()


# ---------------------------------------------------------------------------------------
# write
# ---------------------------------------------------------------------------------------

FORMATS = [(16, 0), (8, 0), (4, 0), (2, 0), (BF16_ROWS, 0), (16, 32), (8, 64), (4, 32), (2, 16)]


def _values(g, T, r, dR, dtype=torch.bfloat16):
    std = torch.empty(r).uniform_(0.5, 2.0, generator=g)
    return ((torch.randn(T, r, generator=g) * std).to(dtype),
            torch.randn(T, dR, generator=g).to(dtype))


def _row_refs(oracle, c, kr, d, b, G):
    cn, kn = bf16_or_f32_to_np(c), bf16_or_f32_to_np(kr)
    if b == BF16_ROWS:
        v = torch.cat([c[:, :d].float(), kr.float()], 1).to(torch.bfloat16)
        return v.view(torch.uint8).numpy(), np.full((len(cn), 1), 0x3C00, np.uint16)
    if G:
        rows, s, _ = oracle.quantize_rows_grouped(cn, kn, d, b, G)
    else:
        rows, s, _ = oracle.quantize_rows(cn, kn, d, b)
    return rows, s.view(np.uint16).reshape(len(cn), -1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,r,dR", [(512, 512, 64), (128, 512, 64), (32, 64, 16), (16, 16, 0)])
@pytest.mark.parametrize("b,G", FORMATS)
def test_write_bit_exact(pkg, oracle_mod, dtype, d, r, dR, b, G):
    if G and (d + dR) % G:
        pytest.skip("the group does not divide the row")
    T, pool = 61, 200
    g = torch.Generator().manual_seed(b * 31 + d + G)
    c, kr = _values(g, T, r, dR, dtype)
    c[3] = 0.0
    kr[3] = 0.0                                  # an all-zero token
    c[5] *= 1e-6
    kr[5] *= 1e-6
    slots = torch.randperm(pool, generator=g)[:T].to(torch.int32)
    slots[7] = -1                                # no token's
    lay = pkg.Layout([0, 0], [d, 0], [b, 0], r, dR, 2, pool // 2, scale_group=G)
    try:
        lay.arena[256:].fill_(0xA5)
        wide = torch.zeros(T, r + 8, dtype=dtype)
        wide[:, :r] = c
        cd = wide.cuda()[:, :r]                  # rows further apart than they are wide
        lay.paged_write(0, cd, kr.cuda(), slots.cuda())
        codes, scales = lay.cache_views(0)
        codes = codes.reshape(pool, -1).cpu().numpy()
        scales = scales.reshape(pool, -1).cpu().view(torch.int16).numpy().view(np.uint16)
        rows, s = _row_refs(oracle_mod, c, kr, d, b, G)
        keep = np.array([i for i in range(T) if i != 7])
        at = slots.numpy()[keep]
        assert np.array_equal(codes[at][:, :rows.shape[1]], rows[keep])
        assert not codes[at][:, rows.shape[1]:].any()
        assert np.array_equal(scales[at], s[keep])
        rest = np.setdiff1d(np.arange(pool), at)
        assert (codes[rest] == 0xA5).all() and (scales[rest] == 0xA5A5).all()
        assert lay.read_status() == 0
    finally:
        lay.close()


def test_write_refuses_slots_outside_the_pool(pkg):
    lay = pkg.Layout([0], [64], [8], 64, 16, 1, 32)
    try:
        c, kr = torch.ones(4, 64, device="cuda"), torch.ones(4, 16, device="cuda")
        lay.arena[256:].fill_(7)
        lay.paged_write(0, c, kr, i32([32, -5, 2147483647, 3]))
        assert lay.read_status(clear=True) == pkg.KVK_FLAG_WRITE_RANGE
        codes, _ = lay.cache_views(0)
        changed = (codes[0] != 7).any(1).nonzero().flatten().tolist()
        assert changed == [3]
        c[0, 5] = float("nan")
        lay.paged_write(0, c, kr, i32([1, 2, 4, 5]))
        assert lay.read_status(clear=True) == pkg.KVK_FLAG_NONFINITE
    finally:
        lay.close()


# ---------------------------------------------------------------------------------------
# chunk attention
# ---------------------------------------------------------------------------------------

class Pool:
    """A layout with every sequence's rows written to random pages, and their fp64 values."""

    def __init__(self, pkg, oracle, lens, d, dR, b, G, page, seed, r=None, spare=3, width=None):
        self.d, self.dR, self.b, self.G, self.page, self.lens = d, dR, b, G, page, lens
        r = r or d
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        n_pages = sum(-(-n // page) for n in lens) + spare
        self.n_pages = n_pages
        width = width or max(1, max(-(-n // page) for n in lens))
        self.table = random_table(rng, lens, page, n_pages, width)
        self.lay = pkg.Layout([0, 0], [d, 0], [b, 0], r, dR, 1, n_pages * page, scale_group=G)
        # slots that no token owns hold what a reused pool holds: anything
        self.lay.arena[256:].random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(seed))
        self.rows, self.scale = [], []
        for i, n in enumerate(lens):
            c, kr = _values(g, n, r, dR)
            if n:
                pos = np.arange(n)
                slots = self.table[i, pos // page] * page + pos % page
                self.lay.paged_write(0, c.cuda(), kr.cuda(), i32(slots.tolist()))
                v, s = dequantised(oracle, c, kr, d, b, G)
            else:
                v = s = np.zeros((0, d + dR))
            self.rows.append(v)
            self.scale.append(s)
        assert self.lay.read_status() == 0

    def queries(self, q_lens, H, dtype, seed, gain=1.0):
        g = torch.Generator().manual_seed(seed + 1)
        N = sum(q_lens)
        ql = (gain * torch.randn(N, H, self.d, generator=g)).to(dtype)
        qr = (gain * torch.randn(N, H, self.dR, generator=g)).to(dtype)
        return ql, qr

    def check(self, q_lens, ql, qr, out, lse, dtype, sigma, tensor, what=""):
        q = torch.cat([ql.double(), qr.double()], 2).numpy()
        H = q.shape[1]
        row0, worst = 0, 0.0
        for i, (n, m) in enumerate(zip(self.lens, q_lens)):
            if not m:
                continue
            lim = np.repeat(np.clip(n - m + np.arange(m) + 1, 0, n), H)
            ref = chunk_reference(self.rows[i], q[row0:row0 + m].reshape(m * H, -1), lim, self.d,
                                  sigma)
            o = out[row0:row0 + m].double().numpy().reshape(m * H, -1)
            w = check_chunk(o, lse[row0:row0 + m].double().numpy().reshape(-1), ref, dtype, self.b,
                            self.G, self.d + self.dR, n, self.rows[i], self.scale[i], self.d,
                            tensor, f"{what} seq {i}")
            worst = max(worst, w)
            row0 += m
        return worst


def _paths(pkg, lay, dtype):
    ps = [pkg.KVK_PATH_CUDA_CORE]
    if lay.chunk_path_for(0, dtype) == pkg.KVK_PATH_TENSOR:
        ps.append(pkg.KVK_PATH_TENSOR)
    return ps


def _run(pool, pkg, path, q_lens, ql, qr, sigma, dtype, **kw):
    lay = pool.lay
    lay.set_decode_path(path)
    N, H = ql.shape[:2]
    out = torch.full((N, H, pool.d), float("nan"), dtype=dtype, device="cuda")
    lse = torch.full((N, H), float("nan"), device="cuda")
    q_start = i32(np.concatenate([[0], np.cumsum(q_lens)]).tolist())
    lay.mla_chunk(kw.pop("layer", 1), ql.cuda(), qr.cuda(), q_start, i32(pool.lens),
                  i32(pool.table.tolist()), pool.page, sigma, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    lay.set_decode_path(pkg.KVK_PATH_AUTO)
    return out.cpu(), lse.cpu()


CHUNKS = {   # lens, q_lens, heads, page
    "one_token": ([1], [1], 8, 16),
    "decode": ([300, 1, 128, 129, 77], [1, 1, 1, 1, 1], 40, 64),
    "chunk": ([257], [33], 8, 16),
    "mixed": ([130, 5, 400, 64], [1, 5, 70, 0], 3, 32),
    "idle_first": ([9, 0, 200], [0, 0, 2], 28, 8),
    "beyond": ([3, 40], [6, 41], 5, 4),          # more queries than tokens: rows that see none
    "empty": ([0, 0], [2, 0], 4, 16),
    "many_heads": ([150], [3], 130, 1),
    "one_head": ([140], [140], 1, 256),
    # many row tiles a sequence: rows expanded once ahead of the attention
    "prefill": ([300, 129, 64], [300, 129, 64], 8, 16),
    "late_chunk": ([1000, 70], [130, 70], 12, 64),
    "small_pages": ([450], [100], 16, 8),
    "tiny_pages": ([450], [100], 16, 4),
}


@pytest.mark.parametrize("case", CHUNKS, ids=str)
@pytest.mark.parametrize("b,G", FORMATS)
@pytest.mark.parametrize("path", ["cuda_core", "tensor"])
def test_chunk_matches_reference(pkg, oracle_mod, path, case, b, G):
    lens, q_lens, H, page = CHUNKS[case]
    pool = Pool(pkg, oracle_mod, lens, 128, 64, b, G, page, 11 + b)
    try:
        p = pkg.KVK_PATH_TENSOR if path == "tensor" else pkg.KVK_PATH_CUDA_CORE
        sigma = 1 / math.sqrt(192)
        ql, qr = pool.queries(q_lens, H, torch.bfloat16, 5, gain=2.0)
        out, lse = _run(pool, pkg, p, q_lens, ql, qr, sigma, torch.bfloat16)
        pool.check(q_lens, ql, qr, out, lse, torch.bfloat16, sigma, path == "tensor", case)
        assert pool.lay.read_status() == 0
    finally:
        pool.lay.close()


SHAPES = [(512, 64), (384, 64), (256, 64), (16, 16), (192, 32), (512, 0), (80, 48)]


@pytest.mark.parametrize("q_lens", [[40, 1, 9], [100, 64, 120]], ids=["few", "many"])
@pytest.mark.parametrize("d,dR", SHAPES)
@pytest.mark.parametrize("dtype,b", [(torch.bfloat16, 16), (torch.bfloat16, 8), (torch.float16, 4),
                                     (torch.bfloat16, BF16_ROWS), (torch.float16, 16),
                                     (torch.float32, 16)])
def test_chunk_shapes_and_types(pkg, oracle_mod, d, dR, dtype, b, q_lens):
    lens, H = [333, 64, 700], 7
    pool = Pool(pkg, oracle_mod, lens, d, dR, b, 0, 32, d + b)
    try:
        sigma = 1 / math.sqrt(d + dR)
        ql, qr = pool.queries(q_lens, H, dtype, 9, gain=1.5)
        for path in _paths(pkg, pool.lay, dtype):
            out, lse = _run(pool, pkg, path, q_lens, ql, qr, sigma, dtype)
            pool.check(q_lens, ql, qr, out, lse, dtype, sigma, path == pkg.KVK_PATH_TENSOR,
                       f"path {path}")
        assert pool.lay.read_status() == 0
    finally:
        pool.lay.close()


def test_chunk_takes_the_tensor_kernel(pkg):
    for b, dtype, want in [(16, torch.bfloat16, 1), (8, torch.float16, 1), (4, torch.float32, 2),
                           (0, torch.bfloat16, 1), (0, torch.float16, 2)]:
        lay = pkg.Layout([0], [512], [b], 512, 64, 1, 64)
        assert lay.chunk_path_for(0, dtype) == want
        lay.close()
    lay = pkg.Layout([0], [528], [8], 528, 64, 1, 64)
    assert lay.chunk_path_for(0, torch.bfloat16) == pkg.KVK_PATH_CUDA_CORE
    lay.close()


@pytest.mark.parametrize("b", [2, 4, 8, 16])
def test_write_codes_next_to_rounding_borders(pkg, oracle_mod, b):
    """Values at and next to the borders (k + 1/2) s between two codes, where a quotient off by
    one unit in its last place would round the other way."""
    q = (1 << (b - 1)) - 1
    rng = np.random.default_rng(b)
    T, n = 512, 512
    s = np.exp(rng.uniform(np.log(2e-4), np.log(200.0), T)).astype(np.float16)
    k = rng.integers(-q, q, (T, n)).astype(np.float64)
    v = ((k + 0.5) * s[:, None].astype(np.float64)).astype(np.float32)
    v = (v.view(np.int32) + rng.integers(-3, 4, (T, n), dtype=np.int32)).view(np.float32)
    # the largest: just below q s (which binary32 may round up at 16 bits), so that its quotient by
    # q rounds up to the scale s exactly
    v[:, 0] = np.nextafter(np.float32(q) * s.astype(np.float32), np.float32(0))
    v = np.clip(v, -v[:, :1], v[:, :1])
    c = torch.from_numpy(v)
    kr = torch.zeros(T, 0)
    rows, sc, _ = oracle_mod.quantize_rows(v, np.zeros((T, 0), np.float32), n, b)
    assert np.array_equal(sc.view(np.uint16).reshape(-1), s.view(np.uint16))
    lay = pkg.Layout([0], [n], [b], n, 0, 1, T)
    try:
        lay.paged_write(0, c.cuda(), kr.cuda(), i32(list(range(T))))
        codes, _ = lay.cache_views(0)
        assert np.array_equal(codes[0].cpu().numpy()[:, :rows.shape[1]], rows)
    finally:
        lay.close()


def test_write_long_rows(pkg, oracle_mod):
    """Rows beyond the short form's 640 elements."""
    d, dR, T = 1024, 64, 9
    g = torch.Generator().manual_seed(3)
    c, kr = _values(g, T, d, dR)
    for b, G in [(8, 0), (4, 32), (0, 0)]:
        lay = pkg.Layout([0], [d], [b], d, dR, 1, 16, scale_group=G)
        try:
            slots = [3, 1, 15, 0, 7, -1, 9, 8, 4]
            lay.paged_write(0, c.cuda(), kr.cuda(), i32(slots))
            codes, scales = lay.cache_views(0)
            rows, s = _row_refs(oracle_mod, c, kr, d, b, G)
            keep = [i for i in range(T) if slots[i] >= 0]
            at = [slots[i] for i in keep]
            assert np.array_equal(codes[0].cpu().numpy()[at], rows[keep])
            assert np.array_equal(scales[0].reshape(16, -1).cpu().view(torch.int16).numpy()
                                  .view(np.uint16)[at], s[keep])
        finally:
            lay.close()
