"""The paged operators as a serving step uses them: run together, captured into a graph and
replayed, on other streams, with shared, missing and unfinished pages, with strided tensors, and
with what a caller gets wrong."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import bf16_or_f32_to_np
from paged_helpers import check_chunk, chunk_reference, dequantised
from test_gpu_paged import FORMATS, Pool, _run, _values, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__
    __graft_entry__.build()
    import compressed_decode_attention_kvk_b200 as p
    assert torch.cuda.is_available()
    return p


def test_serving_steps_match_the_contiguous_cache(pkg, oracle_mod):
    """Prefill in chunks, then decode steps: plan, write, chunk, against kvk_quant_write and
    kvk_mla_decode over a contiguous cache and against the fp64 form."""
    d, dR, H, page, b = 128, 64, 8, 16, 8
    lens = [45, 130, 7]
    g = torch.Generator().manual_seed(4)
    B, top = len(lens), max(lens)
    c = [_values(g, n, d, dR) for n in lens]
    n_pages = sum(-(-n // page) for n in lens) + 2
    paged = pkg.Layout([0, 0], [d, 0], [b, 0], d, dR, 1, n_pages * page)
    flat = pkg.Layout([0, 0], [d, 0], [b, 0], d, dR, B, top)
    sigma = 1 / math.sqrt(d + dR)
    try:
        table = torch.full((B, -(-top // page)), -1, dtype=torch.int32, device="cuda")
        free, count = i32(list(range(n_pages))[::-1]), i32([n_pages])
        cached = i32([0] * B)
        done = [0] * B
        step = 0
        while any(a < n for a, n in zip(done, lens)):
            # a chunk of up to 60 tokens, then one token a step; a sequence that is through idles
            new = [min(60 if n - a > 3 else 1, n - a) for a, n in zip(done, lens)]
            N = sum(new)
            out = paged.new_paged_plan(B, N)._replace(free_count=count)
            p = paged.paged_plan(cached, i32(new), free, count, table, page, N, out=out)
            cs = torch.cat([c[i][0][done[i]:done[i] + new[i]] for i in range(B)])
            ks = torch.cat([c[i][1][done[i]:done[i] + new[i]] for i in range(B)])
            paged.paged_write(0, cs.cuda(), ks.cuda(), p.slots)
            ql = torch.randn(N, H, d, generator=g).to(torch.bfloat16)
            qr = torch.randn(N, H, dR, generator=g).to(torch.bfloat16)
            lse = torch.empty(N, H, device="cuda")
            o = paged.mla_chunk(1, ql.cuda(), qr.cuda(), p.q_start, p.seq_lens, table, page, sigma,
                                lse=lse)
            o, lse = o.cpu(), lse.cpu()
            row = 0
            for i in range(B):
                if new[i]:
                    at = torch.zeros(B, dtype=torch.int32)
                    at[i] = done[i]
                    # the same tokens into the contiguous cache
                    flat.quant_write(0, c[i][0][done[i]:done[i] + new[i]].expand(B, -1, -1)
                                     .contiguous().cuda(),
                                     c[i][1][done[i]:done[i] + new[i]].expand(B, -1, -1)
                                     .contiguous().cuda(),
                                     torch.where(torch.arange(B) == i, at, top).int().cuda())
                n = done[i] + new[i]
                if new[i]:
                    rows, scale = dequantised(oracle_mod, c[i][0][:n], c[i][1][:n], d, b, 0)
                    q = torch.cat([ql[row:row + new[i]].double(), qr[row:row + new[i]].double()],
                                  2).numpy().reshape(new[i] * H, -1)
                    lim = np.repeat(done[i] + np.arange(new[i]) + 1, H)
                    ref = chunk_reference(rows, q, lim, d, sigma)
                    check_chunk(o[row:row + new[i]].double().numpy().reshape(new[i] * H, -1),
                                lse[row:row + new[i]].double().numpy().reshape(-1), ref,
                                torch.bfloat16, b, 0, d + dR, n, rows, scale, d, True,
                                f"step {step} seq {i}")
                row += new[i]
                done[i] = n
            cached = p.seq_lens.clone()
            step += 1
        assert paged.read_status() == 0
        assert cached.tolist() == lens
        # the pool's rows are the contiguous cache's, byte for byte
        pc, ps = paged.cache_views(0)
        fc, fs = flat.cache_views(0)
        t = table.cpu().numpy()
        for i, n in enumerate(lens):
            pos = np.arange(n)
            slot = torch.from_numpy(t[i, pos // page].astype(np.int64) * page + pos % page).cuda()
            assert torch.equal(pc[0][slot], fc[i, :n]) and torch.equal(ps[0][slot], fs[i, :n])
    finally:
        paged.close()
        flat.close()


@pytest.mark.parametrize("rows", ["decode", "chunk"])
def test_graph_replay_with_new_lengths(pkg, oracle_mod, rows):
    """plan + write + chunk captured once; replayed with other lengths, tokens and queries in the
    same buffers, padded to the captured sizes."""
    d, dR, H, page, b, B = 256, 64, 16, 32, 16, 3
    N, cap = (B, 600) if rows == "decode" else (140, 600)
    n_pages = 3 * (cap // page + 1) + 2
    lay = pkg.Layout([0], [d], [b], d, dR, 1, n_pages * page)
    sigma = 1 / math.sqrt(d + dR)
    width = cap // page + 1
    try:
        st = dict(cached=i32([0] * B), new=i32([0] * B), free=i32(list(range(n_pages))),
                  count=i32([n_pages]), table=torch.full((B, width), -1, dtype=torch.int32,
                                                         device="cuda"),
                  c=torch.zeros(N, d, dtype=torch.bfloat16, device="cuda"),
                  kr=torch.zeros(N, dR, dtype=torch.bfloat16, device="cuda"),
                  ql=torch.zeros(N, H, d, dtype=torch.bfloat16, device="cuda"),
                  qr=torch.zeros(N, H, dR, dtype=torch.bfloat16, device="cuda"),
                  out=torch.zeros(N, H, d, dtype=torch.bfloat16, device="cuda"),
                  lse=torch.zeros(N, H, device="cuda"))
        plan = lay.new_paged_plan(B, N)._replace(free_count=st["count"])
        ws = lay.new_chunk_workspace(0, N, B, H)

        def step():
            lay.paged_plan(st["cached"], st["new"], st["free"], st["count"], st["table"], page, N,
                           out=plan)
            lay.paged_write(0, st["c"], st["kr"], plan.slots)
            lay.mla_chunk(0, st["ql"], st["qr"], plan.q_start, plan.seq_lens, st["table"], page,
                          sigma, out=st["out"], lse=st["lse"], workspace=ws)

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()                                   # nothing to do: no new tokens
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
        torch.cuda.synchronize()
        assert int(st["count"]) == n_pages
        g = torch.Generator().manual_seed(2)
        hist = [(torch.zeros(0, d, dtype=torch.bfloat16), torch.zeros(0, dR, dtype=torch.bfloat16))
                for _ in range(B)]
        steps = [[1, 0, 1], [1, 1, 1], [0, 1, 0]] if rows == "decode" else \
            [[100, 3, 37], [1, 139, 0], [60, 1, 64]]
        if rows == "decode":                         # a prompt first, outside the graph
            first = [33, 200, 64]
            plan0 = lay.paged_plan(st["cached"], i32(first), st["free"], st["count"], st["table"],
                                   page, sum(first))
            cs = [_values(g, n, d, dR) for n in first]
            lay.paged_write(0, torch.cat([x[0] for x in cs]).cuda(),
                            torch.cat([x[1] for x in cs]).cuda(), plan0.slots)
            st["count"].copy_(plan0.free_count)
            st["cached"].copy_(plan0.seq_lens)
            hist = cs
        for new in steps:
            total = sum(new)
            c, kr = _values(g, N, d, dR)
            ql = torch.randn(N, H, d, generator=g).to(torch.bfloat16)
            qr = torch.randn(N, H, dR, generator=g).to(torch.bfloat16)
            st["new"].copy_(i32(new))
            for k, v in (("c", c), ("kr", kr), ("ql", ql), ("qr", qr)):
                st[k].copy_(v)
            st["out"].fill_(7.0)
            st["lse"].fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            out, lse = st["out"].cpu(), st["lse"].cpu()
            # rows behind the last sequence are as they were
            assert (out[total:] == 7.0).all() and (lse[total:] == 7.0).all()
            row = 0
            for i, m in enumerate(new):
                hist[i] = (torch.cat([hist[i][0], c[row:row + m]]),
                           torch.cat([hist[i][1], kr[row:row + m]]))
                if m:
                    n = len(hist[i][0])
                    rws, scale = dequantised(oracle_mod, hist[i][0], hist[i][1], d, b, 0)
                    q = torch.cat([ql[row:row + m].double(), qr[row:row + m].double()], 2).numpy()
                    ref = chunk_reference(rws, q.reshape(m * H, -1),
                                          np.repeat(n - m + np.arange(m) + 1, H), d, sigma)
                    check_chunk(out[row:row + m].double().numpy().reshape(m * H, -1),
                                lse[row:row + m].double().numpy().reshape(-1), ref, torch.bfloat16,
                                b, 0, d + dR, n, rws, scale, d, True, f"new {new} seq {i}")
                row += m
            st["cached"].copy_(plan.seq_lens)
        assert lay.read_status() == 0
        del graph
    finally:
        lay.close()


@pytest.mark.parametrize("q_lens", [[1, 1], [90, 70]], ids=["few", "many"])
def test_two_streams_with_a_workspace_each(pkg, oracle_mod, q_lens):
    lens, H, d = [400, 333], 16, 128
    pool = Pool(pkg, oracle_mod, lens, d, 64, 8, 0, 32, 21)
    try:
        sigma = 0.07
        q = [pool.queries(q_lens, H, torch.bfloat16, 30 + k) for k in range(2)]
        N = sum(q_lens)
        dev = [(a.cuda(), b.cuda()) for a, b in q]
        args = (i32(np.concatenate([[0], np.cumsum(q_lens)]).tolist()), i32(lens),
                i32(pool.table.tolist()), pool.page, sigma)
        ws = [pool.lay.new_chunk_workspace(0, N, 2, H) for _ in range(2)]
        out = [torch.empty(N, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        lse = [torch.empty(N, H, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for rep in range(3):
            for k in range(2):
                if rep % 2:                          # the stream as an argument, or as the current
                    pool.lay.mla_chunk(1, *dev[k], *args, out=out[k], lse=lse[k], workspace=ws[k],
                                       stream=streams[k])
                else:
                    with torch.cuda.stream(streams[k]):
                        pool.lay.mla_chunk(1, *dev[k], *args, out=out[k], lse=lse[k],
                                           workspace=ws[k])
        torch.cuda.synchronize()
        for k in range(2):
            pool.check(q_lens, *q[k], out[k].cpu(), lse[k].cpu(), torch.bfloat16, sigma, True)
    finally:
        pool.lay.close()


@pytest.mark.parametrize("q_lens", [[1, 2], [90, 70]], ids=["few", "many"])
def test_tensors_made_by_a_call_on_another_stream(pkg, oracle_mod, q_lens):
    """plan and chunk with a stream argument and no output or workspace given, again and again while
    the current stream allocates and writes: what a call allocates is its stream's."""
    lens, H = [300, 260], 8
    pool = Pool(pkg, oracle_mod, lens, 128, 64, 8, 0, 32, 25)
    try:
        ql, qr = pool.queries(q_lens, H, torch.bfloat16, 4)
        args = (ql.cuda(), qr.cuda(), i32(np.concatenate([[0], np.cumsum(q_lens)]).tolist()),
                i32(lens), i32(pool.table.tolist()), pool.page, 0.07)
        table, free, count = i32([[-1] * 12, [-1] * 12]), i32(list(range(20))), i32([20])
        new, zero = i32(lens), i32([0, 0])
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        outs, plans = [], []
        for _ in range(6):
            outs.append(pool.lay.mla_chunk(1, *args, stream=side))
            plans.append(pool.lay.paged_plan(zero, new, free, count, table, 32, 560, stream=side))
            for _ in range(4):
                torch.empty(4 << 20, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        lse = torch.empty(sum(q_lens), H, device="cuda")
        pool.lay.mla_chunk(1, *args, lse=lse)
        for o in outs:
            pool.check(q_lens, ql, qr, o.cpu(), lse.cpu(), torch.bfloat16, 0.07, True)
        for p in plans:
            assert p.seq_lens.tolist() == lens and p.q_start.tolist() == [0, 300, 560]
    finally:
        pool.lay.close()


@pytest.mark.parametrize("b,G", [(0, 0), (16, 0), (8, 0), (4, 32)])
def test_workspaces_small_and_full_of_garbage(pkg, oracle_mod, b, G):
    """With the whole workspace rows are expanded, with the base size converted in the kernel;
    whatever the memory held."""
    lens, q_lens, H = [333, 200], [100, 90], 12
    pool = Pool(pkg, oracle_mod, lens, 128, 64, b, G, 16, 31 + b)
    try:
        ql, qr = pool.queries(q_lens, H, torch.bfloat16, 4)
        N = sum(q_lens)
        args = (ql.cuda(), qr.cuda(), i32([0, 100, 190]), i32(lens), i32(pool.table.tolist()),
                pool.page, 0.07)
        base = pool.lay.chunk_workspace_bytes(1, 0, 2, H)
        full = pool.lay.chunk_workspace_bytes(1, N, 2, H)
        assert full > base
        for size in (full, full - 1, base):
            for fill in (0xFF, 0x7F, 0x01):
                ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
                lse = torch.empty(N, H, device="cuda")
                out = pool.lay.mla_chunk(1, *args, lse=lse, workspace=ws)
                pool.check(q_lens, ql, qr, out.cpu(), lse.cpu(), torch.bfloat16, 0.07, True)
        with pytest.raises(pkg.KvkError) as e:
            pool.lay.mla_chunk(1, *args, workspace=torch.empty(base - 1, dtype=torch.uint8,
                                                               device="cuda"))
        assert e.value.status == 5
        assert pool.lay.read_status() == 0
    finally:
        pool.lay.close()


@pytest.mark.parametrize("b", [0, 16])
def test_pool_of_more_than_2_gb(pkg, b):
    """Rows whose byte offsets (in the pool, and in the expanded rows) pass 2^31 and 2^32: the same
    bits as from a pool that is small."""
    d, dR, H, page, n = 512, 64, 16, 64, 200
    slots = 4 << 20                                  # 4.8 GB of codes
    g = torch.Generator().manual_seed(b)
    c, kr = _values(g, n, d, dR)
    q = [(torch.randn(m, H, d, generator=g).to(torch.bfloat16).cuda(),
          torch.randn(m, H, dR, generator=g).to(torch.bfloat16).cuda()) for m in (1, 40)]
    got = []
    for total, pages in ((256, [0, 1, 2, 3]),
                         (slots, [slots // page - 1, slots // page - 2, slots // page // 2, 7])):
        lay = pkg.Layout([0], [d], [b], d, dR, 1, total)
        try:
            table = i32([pages])
            pos = torch.arange(n, device="cuda")
            slot = (table[0][pos // page] * page + pos % page).int()
            lay.paged_write(0, c.cuda(), kr.cuda(), slot)
            outs = []
            for ql, qr in q:
                lse = torch.empty(len(ql), H, device="cuda")
                for path in (pkg.KVK_PATH_TENSOR, pkg.KVK_PATH_CUDA_CORE):
                    lay.set_decode_path(path)
                    outs.append((lay.mla_chunk(0, ql, qr, i32([0, len(ql)]), i32([n]), table, page,
                                               0.05, lse=lse).clone(), lse.clone()))
            assert lay.read_status() == 0
            got.append(outs)
        finally:
            lay.close()
            del lay
            torch.cuda.empty_cache()
    for (a, la), (e, le) in zip(*got):
        assert torch.isfinite(a.float()).all() and torch.equal(a, e) and torch.equal(la, le)


@pytest.mark.parametrize("b,G", [(8, 0), (0, 0), (4, 32), (16, 0)])
@pytest.mark.parametrize("q_len", [1, 60])
def test_missing_pages_are_skipped(pkg, oracle_mod, b, G, q_len):
    """Entries outside the pool: their tokens count as absent, on every path."""
    n, H, page = 300, 8, 16
    pool = Pool(pkg, oracle_mod, [n], 128, 64, b, G, page, 40 + b)
    try:
        sigma = 1 / math.sqrt(192)
        ql, qr = pool.queries([q_len], H, torch.bfloat16, 8)
        gone = [3, 11]
        pool.table[0, 3], pool.table[0, 11] = -1, pool.n_pages
        keep = np.array([t for t in range(n) if t // page not in gone])
        rows = pool.rows[0][keep]
        lim = np.repeat([(keep <= n - q_len + j).sum() for j in range(q_len)], H)
        q = torch.cat([ql.double(), qr.double()], 2).numpy().reshape(q_len * H, -1)
        ref = chunk_reference(rows, q, lim, 128, sigma)
        for path in (pkg.KVK_PATH_CUDA_CORE, pkg.KVK_PATH_TENSOR):
            out, lse = _run(pool, pkg, path, [q_len], ql, qr, sigma, torch.bfloat16)
            check_chunk(out.double().numpy().reshape(q_len * H, -1),
                        lse.double().numpy().reshape(-1), ref, torch.bfloat16, b, G, 192, n, rows,
                        pool.scale[0][keep], 128, path == pkg.KVK_PATH_TENSOR, f"path {path}")
            assert pool.lay.read_status(clear=True) == pkg.KVK_FLAG_PAGE
        # every page gone: rows that see nothing
        pool.table[:] = -5
        for path in (pkg.KVK_PATH_CUDA_CORE, pkg.KVK_PATH_TENSOR):
            out, lse = _run(pool, pkg, path, [q_len], ql, qr, sigma, torch.bfloat16)
            assert (out == 0).all() and (lse == -math.inf).all()
    finally:
        pool.lay.close()


@pytest.mark.parametrize("b,G", [(0, 0), (4, 32), (8, 0)])
@pytest.mark.parametrize("H", [4, 40])
def test_a_token_that_is_not_finite_stays_with_those_who_see_it(pkg, oracle_mod, b, G, H):
    """NaN and infinity in a row (or a scale) reach the queries at and behind its position, and no
    query before it in the same chunk."""
    n, q_len, bad = 200, 120, 150
    pool = Pool(pkg, oracle_mod, [n], 128, 64, b, G, 16, 60 + b)
    try:
        codes, scales = pool.lay.cache_views(0)
        slot = int(pool.table[0, bad // 16]) * 16 + bad % 16
        if b == 0:
            codes.view(-1, codes.shape[-1])[slot, 10:12] = torch.tensor([0x80, 0xFF], dtype=torch.uint8)
        else:
            scales.reshape(codes.shape[0] * codes.shape[1], -1)[slot, 0] = float("nan")
        sigma = 1 / math.sqrt(192)
        ql, qr = pool.queries([q_len], H, torch.bfloat16, 8)
        first = bad - (n - q_len)                    # the first query that sees it
        q = torch.cat([ql.double(), qr.double()], 2).numpy()[:first].reshape(first * H, -1)
        lim = np.repeat(n - q_len + np.arange(first) + 1, H)
        ref = chunk_reference(pool.rows[0], q, lim, 128, sigma)
        for path in (pkg.KVK_PATH_CUDA_CORE, pkg.KVK_PATH_TENSOR):
            out, lse = _run(pool, pkg, path, [q_len], ql, qr, sigma, torch.bfloat16)
            check_chunk(out[:first].double().numpy().reshape(first * H, -1),
                        lse[:first].double().numpy().reshape(-1), ref, torch.bfloat16, b, G, 192, n,
                        pool.rows[0], pool.scale[0], 128, path == pkg.KVK_PATH_TENSOR, f"{path}")
            assert torch.isnan(out[first:].float()).all() and torch.isnan(lse[first:]).all()
    finally:
        pool.lay.close()


@pytest.mark.parametrize("q_lens", [[3, 5], [80, 100]], ids=["few", "many"])
def test_strided_tensors_and_negative_scale(pkg, oracle_mod, q_lens):
    lens, H, d, dR = [150, 290], 6, 128, 64
    pool = Pool(pkg, oracle_mod, lens, d, dR, 8, 0, 64, 77)
    try:
        ql, qr = pool.queries(q_lens, H, torch.bfloat16, 3)
        N = sum(q_lens)
        both = torch.zeros(N, H + 2, d + dR + 8, dtype=torch.bfloat16)
        both[:, 1:H + 1, :d], both[:, 1:H + 1, d:d + dR] = ql, qr
        both = both.cuda()
        big = torch.full((N, H + 1, d + 16), 9.0, dtype=torch.bfloat16, device="cuda")
        wide = torch.full((2, 40), -1, dtype=torch.int32, device="cuda")
        wide[:, :pool.table.shape[1]] = i32(pool.table.tolist())
        lse = torch.empty(N, H, device="cuda")
        for sigma in (-0.05, 0.05):
            pool.lay.mla_chunk(0, both[:, 1:H + 1, :d], both[:, 1:H + 1, d:d + dR],
                               i32(np.concatenate([[0], np.cumsum(q_lens)]).tolist()), i32(lens),
                               wide[:, :pool.table.shape[1]], 64, sigma, out=big[:, :H, :d],
                               lse=lse)
            pool.check(q_lens, ql, qr, big[:, :H, :d].cpu(), lse.cpu(), torch.bfloat16, sigma, True)
        assert (big[:, H:] == 9.0).all() and (big[:, :, d:] == 9.0).all()
    finally:
        pool.lay.close()


@pytest.mark.parametrize("q_len", [1, 50])
def test_sequences_that_share_pages(pkg, oracle_mod, q_len):
    """Three sequences over the same pages, of different lengths that end within one page."""
    n, H, page = 260, 16, 64
    pool = Pool(pkg, oracle_mod, [n], 128, 64, 8, 0, page, 5)
    try:
        lens = [n, 200, 227]
        pool.table = np.repeat(pool.table, 3, 0)
        pool.rows = [pool.rows[0][:m] for m in lens]
        pool.scale = [pool.scale[0][:m] for m in lens]
        pool.lens = lens
        ql, qr = pool.queries([q_len] * 3, H, torch.bfloat16, 8)
        for path in (pkg.KVK_PATH_CUDA_CORE, pkg.KVK_PATH_TENSOR):
            out, lse = _run(pool, pkg, path, [q_len] * 3, ql, qr, 0.07, torch.bfloat16)
            pool.check([q_len] * 3, ql, qr, out, lse, torch.bfloat16, 0.07,
                       path == pkg.KVK_PATH_TENSOR, f"path {path}")
    finally:
        pool.lay.close()


def test_long_sequence_split_over_the_gpu(pkg, oracle_mod):
    """One sequence over every cluster, a few rows: partial tiles joined from many pieces."""
    n = 20000
    pool = Pool(pkg, oracle_mod, [n], 128, 64, 4, 0, 128, 9)
    try:
        for q_lens, H in (([1], 40), ([5], 40), ([1], 1)):
            ql, qr = pool.queries(q_lens, H, torch.bfloat16, 1, gain=3.0)
            out, lse = _run(pool, pkg, pkg.KVK_PATH_TENSOR, q_lens, ql, qr, 0.1, torch.bfloat16)
            pool.check(q_lens, ql, qr, out, lse, torch.bfloat16, 0.1, True, f"{q_lens} x {H}")
    finally:
        pool.lay.close()


def test_many_short_and_idle_sequences(pkg, oracle_mod):
    rng = np.random.default_rng(1)
    B, H = 700, 2
    lens = rng.integers(0, 20, B).tolist()
    q_lens = [int(x) for x in rng.integers(0, 3, B) * (rng.random(B) < 0.3)]
    pool = Pool(pkg, oracle_mod, lens, 16, 16, 8, 0, 8, 2)
    try:
        ql, qr = pool.queries(q_lens, H, torch.bfloat16, 1)
        for path in (pkg.KVK_PATH_CUDA_CORE, pkg.KVK_PATH_TENSOR):
            out, lse = _run(pool, pkg, path, q_lens, ql, qr, 0.2, torch.bfloat16)
            pool.check(q_lens, ql, qr, out, lse, torch.bfloat16, 0.2, path == pkg.KVK_PATH_TENSOR)
    finally:
        pool.lay.close()


@pytest.mark.parametrize("path", [1, 2], ids=["tensor", "cuda_core"])
def test_bad_offsets_and_lengths(pkg, oracle_mod, path):
    """Descending or overlong row offsets: flagged, nothing written.  Lengths beyond the table:
    clamped, flagged."""
    pool = Pool(pkg, oracle_mod, [64, 64], 128, 64, 8, 0, 32, 3)
    lay = pool.lay
    try:
        lay.set_decode_path(path)
        N, H = 6, 4
        ql, qr = pool.queries([3, 3], H, torch.bfloat16, 1)
        table = i32(pool.table.tolist())
        for starts in ([0, 4, 3], [0, 3, 7], [-1, 3, 6]):
            out = torch.full((N, H, 128), 5.0, dtype=torch.bfloat16, device="cuda")
            lay.mla_chunk(0, ql.cuda(), qr.cuda(), i32(starts), i32([64, 64]), table, 32, 0.07, out=out)
            torch.cuda.synchronize()
            assert (out == 5.0).all(), starts
            assert lay.read_status(clear=True) == pkg.KVK_FLAG_SEQ_LEN
        out = torch.empty(N, H, 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(N, H, device="cuda")
        lay.mla_chunk(0, ql.cuda(), qr.cuda(), i32([0, 3, 6]), i32([1000, 64]), table, 32, 0.07,
                      out=out, lse=lse)
        pool.check([3, 3], ql, qr, out.cpu(), lse.cpu(), torch.bfloat16, 0.07, path == 1)
        assert lay.read_status(clear=True) == pkg.KVK_FLAG_SEQ_LEN
    finally:
        lay.close()


def test_refusals(pkg):
    lay = pkg.Layout([0, 0], [64, 0], [8, 0], 64, 16, 1, 256)
    try:
        E = pkg.KvkError
        bf = dict(dtype=torch.bfloat16, device="cuda")
        ql, qr = torch.zeros(4, 2, 64, **bf), torch.zeros(4, 2, 16, **bf)
        start, lens, table = i32([0, 4]), i32([4]), i32([[0, 1]])
        ok = dict(q_start=start, seq_lens=lens, block_table=table, page_tokens=16, softmax_scale=1.0)

        def status(f, *a, **k):
            with pytest.raises(E) as e:
                f(*a, **k)
            return e.value.status

        lay.mla_chunk(0, ql, qr, **ok)
        assert status(lay.mla_chunk, 0, ql, qr, **{**ok, "page_tokens": 24}) == 1
        assert status(lay.mla_chunk, 0, ql, qr, **{**ok, "page_tokens": 0}) == 1
        assert status(lay.mla_chunk, 2, ql, qr, **ok) == 1
        assert status(lay.mla_chunk, 0, ql, qr, workspace=torch.empty(64, dtype=torch.uint8,
                                                                      device="cuda"), **ok) == 5
        shifted = torch.zeros(4 * 2 * 64 + 8, **bf)[1:4 * 2 * 64 + 1].view(4, 2, 64)
        assert status(lay.mla_chunk, 0, shifted, qr, **ok) == 6
        assert status(lay.mla_chunk, 0, torch.zeros(4, 2, 68, **bf)[:, :, :64], qr, **ok) == 6
        with pytest.raises(ValueError):
            lay.mla_chunk(0, ql.float(), qr, **ok)
        with pytest.raises(ValueError):
            lay.mla_chunk(0, ql[:, :, :32], qr, **ok)
        with pytest.raises(ValueError):
            lay.mla_chunk(0, ql, qr, out=torch.zeros(4, 2, 64, device="cuda"), **ok)
        with pytest.raises(ValueError):
            lay.mla_chunk(0, ql, qr, **{**ok, "seq_lens": lens.long()})
        assert status(lay.paged_write, 1, ql[:, 0], qr[:, 0], i32([0, 1, 2, 3])) == 4
        with pytest.raises(ValueError):
            lay.paged_write(0, ql[:, 0], qr[:, 0], i32([0, 1]))
        with pytest.raises(ValueError):
            lay.paged_write(0, ql[:, 0].half(), qr[:, 0].half(), i32([0, 1, 2, 3]))
        c1 = i32([0])
        assert status(lay.paged_plan, c1, i32([1]), i32([0]), i32([1]), table, 3, 4) == 1
        out = lay.new_paged_plan(1, 4)
        assert status(lay.paged_plan, c1, i32([1]), i32([0]), i32([1]), table, 16, 4,
                      out=out._replace(seq_lens=c1)) == 1
        both = i32([0, 0, 0])                        # results that overlap inputs or each other
        assert status(lay.paged_plan, both[1:2], i32([1]), i32([0]), i32([1]), table, 16, 4,
                      out=out._replace(q_start=both[:2])) == 1
        assert status(lay.paged_plan, c1, i32([1]), i32([0]), i32([1]), table, 16, 4,
                      out=out._replace(slots=out.positions)) == 1
        assert status(lay.paged_plan, c1, i32([1]), table[0], i32([1]), table, 16, 4, out=out) == 1
        with pytest.raises(ValueError):
            lay.paged_plan(c1, i32([1]), i32([0]), i32([1]), table, 16, 9, out=out)
        # no rows, no tokens: nothing to do
        lay.mla_chunk(0, ql[:0], qr[:0], **ok)
        lay.paged_write(0, ql[:0, 0], qr[:0, 0], i32([]))
        assert lay.read_status() == 0
    finally:
        lay.close()


def test_wait_limit_stops_the_kernel(pkg, oracle_mod):
    """A wait limit of nothing runs out: the kernel reports it and ends, and the context serves the
    next call."""
    pool = Pool(pkg, oracle_mod, [2000], 512, 64, 16, 0, 64, 3)
    lay = pool.lay
    try:
        for q_lens in ([1], [40]):
            ql, qr = pool.queries(q_lens, 40, torch.bfloat16, 1)
            lay.set_wait_limit(1)
            _run(pool, pkg, pkg.KVK_PATH_TENSOR, q_lens, ql, qr, 0.04, torch.bfloat16)
            assert lay.read_status(clear=True) & pkg.kvk.KVK_FLAG_TIMEOUT
            lay.set_wait_limit(0)
            out, lse = _run(pool, pkg, pkg.KVK_PATH_TENSOR, q_lens, ql, qr, 0.04, torch.bfloat16)
            pool.check(q_lens, ql, qr, out, lse, torch.bfloat16, 0.04, True)
            assert lay.read_status() == 0
    finally:
        lay.close()


@pytest.mark.parametrize("path", [1, 2], ids=["tensor", "cuda_core"])
def test_largest_batch_and_head_count(pkg, oracle_mod, path):
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 3, 4096).tolist()
    q_lens = [int(x) for x in rng.integers(0, 2, 4096)]
    pool = Pool(pkg, oracle_mod, lens, 16, 0, 8, 0, 2, 2)
    try:
        ql, qr = pool.queries(q_lens, 1, torch.bfloat16, 1)
        out, lse = _run(pool, pkg, path, q_lens, ql, qr, 0.2, torch.bfloat16)
        pool.check(q_lens, ql, qr, out, lse, torch.bfloat16, 0.2, path == 1)
    finally:
        pool.lay.close()
    pool = Pool(pkg, oracle_mod, [5, 70], 32, 16, 4, 0, 8, 2)
    try:
        ql, qr = pool.queries([1, 2], 4096, torch.bfloat16, 1)
        out, lse = _run(pool, pkg, path, [1, 2], ql, qr, 0.2, torch.bfloat16)
        pool.check([1, 2], ql, qr, out, lse, torch.bfloat16, 0.2, path == 1)
    finally:
        pool.lay.close()


@pytest.mark.parametrize("page", [1, 4, 65536])
@pytest.mark.parametrize("q_len", [2, 70])
def test_smallest_and_largest_pages(pkg, oracle_mod, page, q_len):
    pool = Pool(pkg, oracle_mod, [131, 300], 64, 32, 8, 0, page, 6)
    try:
        ql, qr = pool.queries([q_len, q_len], 10, torch.bfloat16, 1)
        for path in (pkg.KVK_PATH_CUDA_CORE, pkg.KVK_PATH_TENSOR):
            out, lse = _run(pool, pkg, path, [q_len, q_len], ql, qr, 0.1, torch.bfloat16)
            pool.check([q_len, q_len], ql, qr, out, lse, torch.bfloat16, 0.1,
                       path == pkg.KVK_PATH_TENSOR, f"path {path}")
    finally:
        pool.lay.close()
