"""Paged serving of the compressed MLA cache: what its operators compute, over which sizes.

Three operators, used one after the other in a serving step:

* plan   block tables, slot map, positions and sequence lengths built on the GPU from the
         requests' cached and new token counts and a list of free pages
* write  quantise-on-write of a packed batch of new tokens to the slots of that map
* chunk  causal attention of every sequence's new tokens (one, for a decode step, or a chunk
         of a prompt) over its paged cache, in the absorbed MLA form

A case is a dict of sizes; ``prepare`` makes its inputs, ``run`` one pass in the plain form
(``own`` false: elementary torch operations) or through the library (``own`` true), ``exact``
the same results from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

BF16_ROWS = 0       # bit width of an uncompressed anchor: rows of bfloat16


def listed():
    return [
        # the bookkeeping of one decode step of the 14B serving batch: latency
        dict(name="plan_step", op="plan", batch=32, tokens=8191, spread=0.5, chunk=1, qspread=0.0,
             page=64),
        # the bookkeeping of a prefill of ragged prompts, small pages
        dict(name="plan_prefill", op="plan", batch=32, tokens=0, spread=0.0, chunk=8192,
             qspread=0.9, page=16),
        # one decode step's new tokens of one layer: latency
        dict(name="write_step", op="write", batch=32, tokens=8192, spread=0.5, chunk=1,
             qspread=0.0, page=64, d=512, rope=64, bits=16, group=0, dtype="bf16"),
        # a prefill of ragged prompts into an 8-bit layer
        dict(name="write_prefill", op="write", batch=8, tokens=8192, spread=0.3, chunk=8192,
             qspread=0.3, page=16, d=512, rope=64, bits=8, group=0, dtype="bf16"),
        # fp32 latents into the rank-128 4-bit group-scaled layer of the 152x plan
        dict(name="write_group", op="write", batch=5, tokens=4099, spread=0.4, chunk=2053,
             qspread=0.4, page=32, d=128, rope=64, bits=4, group=32, dtype="f32"),
        # the smallest call: the tiny plan's 4-bit layer, fp32 queries
        dict(name="chunk_tiny", op="chunk", batch=1, tokens=256, spread=0.0, chunk=3, qspread=0.0,
             page=16, heads=8, d=64, rope=16, bits=4, group=0, dtype="f32"),
        # a decode step of the 14B serving batch, 16-bit codes (most layers of its 4x plan)
        dict(name="decode_14b", op="chunk", batch=32, tokens=8192, spread=0.0, chunk=1,
             qspread=0.0, page=64, heads=40, d=512, rope=64, bits=16, group=0, dtype="bf16"),
        # a decode step of the 7B batch with ragged lengths, 4-bit codes
        dict(name="decode_7b", op="chunk", batch=8, tokens=8191, spread=0.9, chunk=1, qspread=0.0,
             page=16, heads=28, d=512, rope=64, bits=4, group=0, dtype="f16"),
        # chunked prefill: 512 new tokens of four sequences near the end of an 8k context
        dict(name="chunk_8bit", op="chunk", batch=4, tokens=8192, spread=0.1, chunk=512,
             qspread=0.0, page=64, heads=40, d=512, rope=64, bits=8, group=0, dtype="bf16"),
        # decode and prefill in one batch, ragged on both sides, rank 384
        dict(name="chunk_mixed", op="chunk", batch=16, tokens=4097, spread=0.9, chunk=301,
             qspread=1.0, page=32, heads=40, d=384, rope=64, bits=16, group=0, dtype="bf16"),
        # a chunk over the rank-128 4-bit group-scaled layer of the 152x plan
        dict(name="chunk_group", op="chunk", batch=8, tokens=8192, spread=0.2, chunk=128,
             qspread=0.5, page=64, heads=40, d=128, rope=64, bits=4, group=32, dtype="bf16"),
        # a long context in an uncompressed bf16 layer: the largest
        dict(name="chunk_long", op="chunk", batch=1, tokens=32768, spread=0.0, chunk=1024,
             qspread=0.0, page=128, heads=40, d=512, rope=64, bits=BF16_ROWS, group=0,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "write", "chunk", "chunk", "chunk"])
    page = rng.choice([16, 32, 64, 128])
    batch = _log_int(rng, 1, 32)
    if op == "plan":
        return dict(op=op, batch=batch, tokens=_log_int(rng, 1, 8192), spread=rng.choice([0.0, 0.5, 0.9]),
                    chunk=rng.choice([1, _log_int(rng, 1, 8192)]), qspread=rng.choice([0.0, 0.5, 1.0]),
                    page=page)
    fmt = rng.choice([(16, 0), (8, 0), (4, 0), (2, 0), (BF16_ROWS, 0), (4, 32), (8, 64)])
    d = rng.choice([128, 256, 384, 512])
    if op == "write":
        tokens = _log_int(rng, 16, 8192)
        return dict(op=op, batch=min(batch, 8), tokens=tokens, spread=rng.choice([0.0, 0.5, 0.9]),
                    chunk=rng.choice([1, _log_int(rng, 1, tokens)]), qspread=rng.choice([0.0, 0.5, 1.0]),
                    page=page, d=d, rope=64, bits=fmt[0], group=fmt[1],
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    heads = rng.choice([8, 28, 40, _log_int(rng, 1, 64)])
    tokens = _log_int(rng, 64, 32768)
    # the cost of the plain form goes with batch x chunk x heads x tokens
    room = 1024 * 40 * 32768
    batch = max(1, min(batch, 262144 // tokens))
    most = max(1, min(tokens, room // (batch * heads * tokens), 1024))
    chunk = rng.choice([1, _log_int(rng, 1, most), _log_int(rng, 1, most)])
    dtype = "f16" if rng.random() < 0.25 and fmt[0] != BF16_ROWS else "bf16"
    return dict(op=op, batch=batch, tokens=tokens, spread=rng.choice([0.0, 0.3, 0.9]), chunk=chunk,
                qspread=rng.choice([0.0, 0.5, 1.0]), page=page, heads=heads, d=d, rope=64,
                bits=fmt[0], group=fmt[1], dtype=dtype)


# ---------------------------------------------------------------------------------------
# sizes that follow from a case
# ---------------------------------------------------------------------------------------

def _ragged(n, count, spread, phase):
    """count lengths between (1 - spread) n and n, spread evenly (the first is n)."""
    return [n - int(spread * n * ((i * 0.6180339887498949 + phase) % 1.0)) if i else n
            for i in range(count)]


def _lens(case):
    """(cached, new): token counts per sequence.  'tokens' counts the cached ones of a plan,
    and the cached and new ones together of a write or a chunk."""
    new = _ragged(case["chunk"], case["batch"], case["qspread"], 0.37)
    total = _ragged(case["tokens"], case["batch"], case["spread"], 0.0)
    if case["op"] == "plan":
        return total, new
    new = [min(a, b) for a, b in zip(new, total)]
    return [a - b for a, b in zip(total, new)], new


def _pages(tokens, page):
    return -(-tokens // page)


def _geometry(case):
    """Row geometry of the case's layer: elements, bytes of a packed row, scales per token."""
    n = case["d"] + case["rope"]
    bits = case["bits"] or 16
    return n, -(-(n * bits // 8) // 16) * 16, (n // case["group"] if case["group"] else 1)


# ---------------------------------------------------------------------------------------
# the plain quantiser: fp16 scale rounded up, half-to-even codes, offset binary, little endian
# ---------------------------------------------------------------------------------------

def _quantise(v, bits, group, row_bytes):
    """Rows of float32 values [tokens, n] -> (packed rows uint8 [tokens, row_bytes], scales
    float16 [tokens, scales per token])."""
    tokens, n = v.shape
    rows = torch.zeros(tokens, row_bytes, dtype=torch.uint8, device=v.device)
    if bits == BF16_ROWS:
        rows[:, :2 * n] = v.to(torch.bfloat16).view(torch.uint8)
        return rows, torch.ones(tokens, 1, dtype=torch.float16, device=v.device)
    q = (1 << (bits - 1)) - 1
    g = v.view(tokens, -1, group or n)
    top = g.abs().amax(2)
    s32 = top / torch.full_like(top, q)     # a division by a number would multiply by 1 / q
    s = s32.to(torch.float16)
    s = torch.where(s.float() < s32, (s.view(torch.int16) + 1).view(torch.float16), s)
    step = s.float().unsqueeze(2)
    codes = torch.where(step > 0, torch.round(g / step), torch.zeros_like(g)).clamp(-q, q)
    u = (codes.to(torch.int32) + (q + 1)).view(tokens, n)
    if bits == 16:
        rows[:, :2 * n] = torch.stack([u & 255, u >> 8], 2).view(tokens, 2 * n).to(torch.uint8)
    else:
        per = 8 // bits
        shift = torch.arange(per, device=v.device, dtype=torch.int32) * bits
        packed = (u.view(tokens, n // per, per) << shift).sum(2)
        rows[:, :n // per] = packed.to(torch.uint8)
    return rows, s


def _unpack(rows, scales, bits, group, n):
    """Packed rows [..., row_bytes] and their scales [..., scales per token] -> float32 values
    [..., n]."""
    if bits == BF16_ROWS:
        return rows[..., :2 * n].contiguous().view(torch.bfloat16).float()
    if bits == 16:
        u = rows[..., 0:2 * n:2].to(torch.int32) | (rows[..., 1:2 * n:2].to(torch.int32) << 8)
    else:
        per = 8 // bits
        shift = torch.arange(per, device=rows.device, dtype=torch.uint8) * bits
        u = (rows[..., :n // per].unsqueeze(-1) >> shift) & ((1 << bits) - 1)
        u = u.flatten(-2)
    codes = (u - (1 << (bits - 1))).float() if bits == 16 else u.float() - (1 << (bits - 1))
    s = scales.float()
    return codes * (s.repeat_interleave(group, -1) if group else s)


def _values(gen, tokens, d, rope):
    """Latents with per-channel standard deviations U(0.5, 2), and N(0, 1) RoPE keys."""
    dev = "cuda"
    std = torch.empty(d, device=dev).uniform_(0.5, 2.0, generator=gen)
    c = torch.randn(tokens, d, device=dev, generator=gen) * std
    return c, torch.randn(tokens, rope, device=dev, generator=gen)


_TYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    i32 = dict(dtype=torch.int32, device="cuda")
    cached, new = _lens(case)
    batch, page = case["batch"], case["page"]
    total = [a + b for a, b in zip(cached, new)]
    per_seq = max(1, max(_pages(t, page) for t in total))
    used = sum(_pages(t, page) for t in total)
    n_pages = used + batch + 1
    order = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32)
    have = [_pages(t, page) for t in (cached if case["op"] == "plan" else total)]
    table = torch.full((batch, per_seq), -1, **i32)
    at = torch.arange(per_seq, **i32).expand(batch, per_seq)
    first = torch.tensor([sum(have[:i]) for i in range(batch)], **i32).unsqueeze(1)
    held = at < torch.tensor(have, **i32).unsqueeze(1)
    table[held] = order[(first + at)[held].long()]
    st = dict(case=case, batch=batch, page=page, n_new=sum(new), qmax=max(new), tmax=max(total),
              table=table, cached=torch.tensor(cached, **i32), new=torch.tensor(new, **i32),
              lens=torch.tensor(total, **i32),
              q_start=torch.tensor([sum(new[:i]) for i in range(batch + 1)], **i32))
    if case["op"] == "plan":
        st["free"] = order[sum(have):].contiguous()
        st["free_count"] = torch.tensor([n_pages - sum(have)], **i32)
    if own:
        import compressed_decode_attention_kvk_b200 as kvk
    if case["op"] == "plan":
        if own:   # the pool's layout: any layer, the plan reads and writes no rows
            st["lay"] = kvk.Layout([0], [64], [4], 64, 16, 1, n_pages * page)
            st["out"] = st["lay"].new_paged_plan(batch, st["n_new"])
        return st
    d, rope, bits, group = case["d"], case["rope"], case["bits"], case["group"]
    n, row_bytes, sg = _geometry(case)
    slots = n_pages * page
    if own:
        lay = kvk.Layout([0], [d], [bits], d, rope, 1, slots, scale_group=group)
        codes, scales = lay.cache_views(0)
        st["lay"], st["codes"], st["scales"] = lay, codes.view(slots, row_bytes), scales.view(slots, sg)
    else:
        st["codes"] = torch.empty(slots, row_bytes, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty(slots, sg, dtype=torch.float16, device="cuda")
    st["codes"].zero_()
    st["scales"].zero_()
    if case["op"] == "write":
        c, kr = _values(gen, st["n_new"], d, rope)
        st["c"], st["kr"] = c.to(_TYPE[case["dtype"]]), kr.to(_TYPE[case["dtype"]])
        # the slots of the new tokens (a plan's result)
        seq = torch.repeat_interleave(torch.arange(batch, device="cuda"), st["new"].long())
        pos = torch.arange(st["n_new"], device="cuda") - st["q_start"][seq] + st["cached"][seq]
        st["slots"] = (table[seq, pos // page] * page + pos % page).to(torch.int32)
        return st
    for at0 in range(0, slots, 65536):       # every page holds a quantised cache
        m = min(65536, slots - at0)
        c, kr = _values(gen, m, d, rope)
        st["codes"][at0:at0 + m], st["scales"][at0:at0 + m] = _quantise(
            torch.cat([c, kr], 1), bits, group, row_bytes)
    st["sigma"] = 1.0 / math.sqrt(n)
    q = torch.randn(st["n_new"], case["heads"], n, device="cuda", generator=gen)
    q = q.to(_TYPE[case["dtype"]])
    st["q_lat"], st["q_rope"] = q[..., :d].contiguous(), q[..., d:].contiguous()
    if own:
        st["workspace"] = lay.new_chunk_workspace(0, st["n_new"], batch, case["heads"])
    return st


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    return _plan(st) if op == "plan" else _write(st) if op == "write" else _chunk(st)


def _plan(st):
    page, batch = st["page"], st["batch"]
    if own:
        p = st["lay"].paged_plan(st["cached"], st["new"], st["free"], st["free_count"], st["table"],
                                 page, st["n_new"], out=st["out"])
        return dict(table=st["table"], seq_lens=p.seq_lens, q_start=p.q_start, slots=p.slots,
                    positions=p.positions, free_count=p.free_count)
    cached, new = st["cached"].long(), st["new"].long()
    lens = cached + new
    q_start = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    have, need = (cached + page - 1) // page, (lens + page - 1) // page
    taken = (need - have).cumsum(0)
    before = taken - (need - have)
    # the k-th page taken in sequence order comes off the end of the free list
    at = torch.arange(st["table"].shape[1], device="cuda").unsqueeze(0)
    k = before.unsqueeze(1) + at - have.unsqueeze(1)
    fresh = (at >= have.unsqueeze(1)) & (at < need.unsqueeze(1))
    pick = (st["free_count"].long() - 1 - k).clamp(0, st["free"].numel() - 1)
    table = torch.where(fresh, st["free"][pick], st["table"])
    tok = torch.arange(st["n_new"], device="cuda")
    seq = torch.searchsorted(q_start[1:].contiguous(), tok, right=True)
    pos = tok - q_start[seq] + cached[seq]
    slots = table[seq, pos // page].long() * page + pos % page
    i32 = torch.int32
    return dict(table=table, seq_lens=lens.to(i32), q_start=q_start.to(i32), slots=slots.to(i32),
                positions=pos.to(i32), free_count=(st["free_count"].long() - taken[-1:]).to(i32))


def _write(st):
    case = st["case"]
    if own:
        st["lay"].paged_write(0, st["c"], st["kr"], st["slots"])
    else:
        v = torch.cat([st["c"], st["kr"]], 1).float()
        rows, scales = _quantise(v, case["bits"], case["group"], st["codes"].shape[1])
        at = st["slots"].long()
        st["codes"][at] = rows
        st["scales"][at] = scales
    return dict(codes=st["codes"], scales=st["scales"])


def _chunk(st):
    case = st["case"]
    if own:
        lse = torch.empty(st["n_new"], case["heads"], device="cuda")
        out = st["lay"].mla_chunk(0, st["q_lat"], st["q_rope"], st["q_start"], st["lens"],
                                  st["table"], st["page"], st["sigma"], lse=lse,
                                  workspace=st["workspace"])
        return dict(out=out, lse=lse)
    batch, page, d, heads = st["batch"], st["page"], case["d"], case["heads"]
    n, _, _ = _geometry(case)
    dev = st["table"].device
    # the cache of every sequence, padded to the longest
    t = torch.arange(st["tmax"], device=dev)
    slot = st["table"][:, t // page].clamp(min=0).long() * page + t % page
    kv = _unpack(st["codes"][slot], st["scales"][slot], case["bits"], case["group"], n)
    # the queries, padded to the longest chunk
    q_len = (st["q_start"][1:] - st["q_start"][:-1]).unsqueeze(1)
    j = torch.arange(st["qmax"], device=dev)
    at = (st["q_start"][:-1].unsqueeze(1) + j).clamp(max=st["n_new"] - 1).long()
    q = torch.cat([st["q_lat"], st["q_rope"]], 2).float()[at].view(batch, st["qmax"] * heads, n)
    z = torch.matmul(q, kv.transpose(1, 2)).mul_(st["sigma"]).view(batch, st["qmax"], heads, -1)
    pos = st["lens"].unsqueeze(1) - q_len + j
    z.masked_fill_((t > pos.unsqueeze(2)).unsqueeze(2), -math.inf)
    m = z.amax(3, keepdim=True).clamp(min=-3e38)
    p = z.sub_(m).exp_()
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p.view(batch, -1, st["tmax"]), kv[..., :d]).view(batch, st["qmax"], heads, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log()).squeeze(3)
    # back to the packed rows
    tok = torch.arange(st["n_new"], device=dev)
    seq = torch.searchsorted(st["q_start"][1:].contiguous(), tok.to(torch.int32), right=True)
    row = tok - st["q_start"][seq]
    return dict(out=o[seq, row].to(st["q_lat"].dtype), lse=lse[seq, row])


def work(case):
    cached, new = _lens(case)
    n_new = sum(new)
    page = case["page"]
    if case["op"] == "plan":
        total = [a + b for a, b in zip(cached, new)]
        fresh = sum(_pages(b, page) - _pages(a, page) for a, b in zip(cached, total))
        held = sum(1 for a, b in zip(cached, new) if b and a % page)
        # lengths in and out, offsets; the pages taken (read, written); slot and position
        return {"bytes": 4 * (4 * case["batch"] + 2 * fresh + held + 2 * n_new), "flops": 0}
    n, row_bytes, sg = _geometry(case)
    if case["op"] == "write":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": n_new * (n * size + row_bytes + 2 * sg + 4), "flops": 3 * n_new * n}
    heads, d = case["heads"], case["d"]
    size = 4 if case["dtype"] == "f32" else 2
    scale = 0 if case["bits"] == BF16_ROWS else 2 * sg
    read = sum((a + b) * (row_bytes + scale) for a, b in zip(cached, new) if b)
    pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(cached, new))
    return {"bytes": read + n_new * heads * ((n + d) * size + 4),
            "flops": 2 * heads * pairs * (n + d)}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits, one sequence at a time
# ---------------------------------------------------------------------------------------

def _field(rows, bits, n):
    """The n unsigned fields of packed rows (numpy uint8 [tokens, row_bytes])."""
    if bits >= 8:
        return rows.view("<u2" if bits == 16 else "u1")[:, :n].astype(np.int64)
    stream = np.unpackbits(rows, axis=1, bitorder="little")[:, :n * bits].reshape(-1, n, bits)
    return (stream.astype(np.int64) << np.arange(bits)).sum(2)


def exact(case, seed):
    st = prepare(case, seed)
    page = st["page"]
    cached, new = _lens(case)
    if case["op"] == "plan":
        free = st["free"].tolist()
        count = int(st["free_count"])
        table = st["table"].cpu().numpy().copy()
        slots, positions = [], []
        for i, (a, b) in enumerate(zip(cached, new)):
            for k in range(_pages(a, page), _pages(a + b, page)):
                count -= 1
                table[i, k] = free[count]
            pos = np.arange(a, a + b)
            positions.append(pos)
            slots.append(table[i, pos // page].astype(np.int64) * page + pos % page)
        i32 = np.int32
        return dict(table=table, seq_lens=np.array([a + b for a, b in zip(cached, new)], i32),
                    q_start=np.concatenate([[0], np.cumsum(new)]).astype(i32),
                    slots=np.concatenate(slots).astype(i32),
                    positions=np.concatenate(positions).astype(i32),
                    free_count=np.array([count], i32))
    bits, group, d = case["bits"], case["group"], case["d"]
    n, row_bytes, sg = _geometry(case)
    if case["op"] == "write":
        # every step of the quantiser is defined in binary32 (division) and binary16 (scale)
        if st["n_new"] * n > 1 << 22:
            return None
        v = torch.cat([st["c"], st["kr"]], 1).float().cpu().numpy()
        codes = st["codes"].cpu().numpy().copy()
        scales = st["scales"].cpu().numpy().copy()
        at = st["slots"].cpu().numpy()
        if bits == BF16_ROWS:
            w = v.view(np.uint32).astype(np.uint64)
            w = ((w + 0x7FFF + ((w >> 16) & 1)) >> 16).astype("<u2")
            rows, s = w.view(np.uint8).reshape(len(v), -1), np.ones((len(v), 1), np.float16)
        else:
            q = (1 << (bits - 1)) - 1
            g = v.reshape(len(v), -1, group or n)
            s32 = np.abs(g).max(2) / np.float32(q)
            s = s32.astype(np.float16)
            s = np.where(s.astype(np.float32) < s32, np.nextafter(s, np.float16(np.inf)), s)
            step = np.where(s > 0, s, 1).astype(np.float32)[..., None]
            c = np.clip(np.rint(np.where(s[..., None] > 0, g / step, 0)), -q, q)
            u = (c.astype(np.int64) + q + 1).reshape(len(v), n)
            bit = ((u[..., None] >> np.arange(bits)) & 1).astype(np.uint8).reshape(len(v), -1)
            rows = np.packbits(bit, axis=1, bitorder="little")
        full = np.zeros((len(v), row_bytes), np.uint8)
        full[:, :rows.shape[1]] = rows
        codes[at], scales[at] = full, s
        return dict(codes=codes, scales=scales)
    out = torch.zeros(st["n_new"], case["heads"], d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["n_new"], case["heads"], dtype=torch.float64, device="cuda")
    table = st["table"].cpu().numpy()
    row0 = 0
    for i, (a, b) in enumerate(zip(cached, new)):
        if not b:
            continue
        at = np.arange(a + b)
        slot = torch.from_numpy(table[i, at // page].astype(np.int64) * page + at % page).cuda()
        rows, s = st["codes"][slot], st["scales"][slot].double()
        if bits == BF16_ROWS:
            kv = rows[:, :2 * n].contiguous().view(torch.bfloat16).double()
        else:
            c = torch.from_numpy(_field(rows.cpu().numpy(), bits, n) - (1 << (bits - 1))).cuda()
            kv = (c.double().view(a + b, sg, -1) * s.unsqueeze(2)).view(a + b, n)
        q = torch.cat([st["q_lat"][row0:row0 + b], st["q_rope"][row0:row0 + b]], 2).double()
        for j0 in range(0, b, 64):          # 64 queries at a time
            j1 = min(b, j0 + 64)
            z = (q[j0:j1].reshape(-1, n) @ kv.T).view(j1 - j0, -1, a + b) * st["sigma"]
            seen = torch.arange(a + b, device="cuda") <= a + torch.arange(j0, j1, device="cuda")[:, None]
            z = z.masked_fill(~seen[:, None], -math.inf)
            l = torch.logsumexp(z, 2)
            lse[row0 + j0:row0 + j1] = l
            w = torch.exp(z - l.unsqueeze(2)).view(-1, a + b)
            out[row0 + j0:row0 + j1] = (w @ kv[:, :d]).view(j1 - j0, -1, d)
        row0 += b
    return dict(out=out, lse=lse)
