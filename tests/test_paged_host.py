"""Refusals of the paged entry points that need no GPU: every check that comes before a launch."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def kvk():
    import __graft_entry__
    __graft_entry__.build()
    from compressed_decode_attention_kvk_b200 import kvk
    return kvk


@pytest.fixture()
def lay(kvk):
    """A planning-only layout: everything before its missing arena can be checked."""
    handle, _, _ = kvk.kvk_create_layout([0, 0], [64, 0], [8, 0], 64, 16, 1, 256)
    yield handle
    kvk.kvk_destroy(handle)


def P(x):
    return ctypes.c_void_p(x)


def test_layout_without_arena_is_refused(kvk, lay):
    L = kvk._lib_handle()
    p = P(4096)
    assert L.kvk_paged_plan(lay, p, p, 1, p, p, 1, 16, p, 4, 4, 8, p, p, p, p, p, None) == 1
    assert L.kvk_paged_write(lay, 0, p, 1, 64, p, 16, 1, p, None) == 1
    assert L.kvk_mla_chunk(lay, 0, p, p, 1, 64, 64, 16, 16, 1, 1, 1, p, p, p, 4, 4, 16, 1.0, p, 64,
                           64, None, p, 1 << 30, None) == 1
    assert L.kvk_paged_plan(None, p, p, 1, p, p, 1, 16, p, 4, 4, 8, p, p, p, p, p, None) == 1


def test_write_needs_an_anchor_layer(kvk, lay):
    p = P(4096)
    assert kvk._lib_handle().kvk_paged_write(lay, 1, p, 1, 64, p, 16, 1, p, None) == 4
    assert kvk._lib_handle().kvk_paged_write(lay, 2, p, 1, 64, p, 16, 1, p, None) == 1


def test_workspace_and_path_queries(kvk, lay):
    assert kvk.kvk_chunk_workspace_bytes(lay, 0, 100, 4, 8) > 0
    assert kvk.kvk_chunk_workspace_bytes(lay, 1, 0, 4096, 1) > 0
    for bad in [(2, 1, 1, 1), (-1, 1, 1, 1), (0, -1, 1, 1), (0, 1, 0, 1), (0, 1, 4097, 1),
                (0, 1, 1, 0), (0, 1, 1, 4097)]:
        with pytest.raises(kvk.KvkError) as e:
            kvk.kvk_chunk_workspace_bytes(lay, *bad)
        assert e.value.status == 1
    assert kvk.kvk_chunk_path_for(lay, 0, torch.float32) == kvk.KVK_PATH_CUDA_CORE
    with pytest.raises(kvk.KvkError):
        kvk.kvk_chunk_path_for(lay, 0, 9)
    kvk.kvk_set_decode_path(lay, kvk.KVK_PATH_TENSOR)
    with pytest.raises(kvk.KvkError) as e:
        kvk.kvk_chunk_path_for(lay, 0, torch.float32)
    assert e.value.status == 8


def test_host_tensors_are_refused(kvk, lay):
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kvk.kvk_paged_plan(lay, t, t, t, t, t.view(2, 2), 16, 4, t, t, t, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        kvk.kvk_paged_write(lay, 0, torch.zeros(4, 64), torch.zeros(4, 16), t)
    q = torch.zeros(4, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        kvk.kvk_mla_chunk(lay, 0, q, q, t, t, t.view(2, 2), 16, 1.0, q, t)


def test_row_stride_of_single_rows(kvk):
    x = torch.zeros(3, 5, 64)
    assert kvk._row_stride(x) == 320 and kvk._row_stride(x, 1) == 64
    one = x[:1, :1]
    assert kvk._row_stride(one) % 8 == 0 and kvk._row_stride(one) >= 64
    assert kvk._row_stride(x[:, :, :0]) == 0
    assert kvk._row_stride(x.expand(3, 5, 64)[:, :1]) == 320


@pytest.mark.parametrize("through", ["function", "layout"])
@pytest.mark.parametrize("width,rope", [(63, 16), (32, 16), (0, 16), (64, 15), (64, 0), (8, 8)])
def test_write_refuses_rows_narrower_than_the_layer(kvk, lay, through, width, rope):
    """A row of fewer than d (or d_rope) elements would be read into the next one, the last past
    the tensor's end; the library sees strides only, so the binding has to refuse it."""
    c, kr = torch.zeros(4, width), torch.zeros(4, rope)
    slots = torch.zeros(4, dtype=torch.int32)
    if through == "function":
        def write(*a):
            kvk.kvk_paged_write(lay, 0, *a)
    else:
        L = object.__new__(kvk.Layout)   # the layout's widths without its arena
        L.anchor, L.d, L.d_rope, L.handle = [0, 0], [64, 0], 16, None

        def write(*a):
            L.paged_write(0, *a)
    with pytest.raises(ValueError, match="narrower"):
        write(c, kr, slots)
    # rows that are wide enough get as far as the check of their device
    with pytest.raises(ValueError, match="CUDA"):
        write(torch.zeros(4, 64), torch.zeros(4, 16), slots)
    with pytest.raises(ValueError, match="CUDA"):
        write(torch.zeros(4, 80), torch.zeros(4, 24), slots)


@pytest.mark.parametrize("d,dR,b,G", [(512, 64, 16, 0), (512, 64, 4, 0), (128, 64, 4, 32), (16, 16, 8, 0),
                                      (192, 0, 0, 0), (528, 64, 8, 0), (512, 72, 8, 0), (512, 128, 8, 0)])
def test_workspace_stays_within_its_documented_size(kvk, d, dR, b, G):
    slots, batch, H = 3000, 4, 40
    handle, _, _ = kvk.kvk_create_layout([0], [d], [b], d, dR, 1, slots, scale_group=G)
    try:
        base = kvk.kvk_chunk_workspace_bytes(handle, 0, 0, batch, H)
        tile = -(-128 * batch // H)                 # query tokens of one row tile a sequence
        small = kvk.kvk_chunk_workspace_bytes(handle, 0, tile - 1, batch, H)
        large = kvk.kvk_chunk_workspace_bytes(handle, 0, 2 * tile, batch, H)
        assert small == base
        row = 2 * (-(-d // 128) * 128 + -(-dR // 64) * 64) * (2 if b == 16 or G else 1) + 4
        tensor = d <= 512 and dR <= 64 and dR % 16 == 0
        assert large - base == 0 if not tensor else slots * row <= large - base <= slots * row + 3 * 256
    finally:
        kvk.kvk_destroy(handle)


@pytest.mark.parametrize("what,dtype,page,memory,want", [
    ("fits", torch.bfloat16, 64, 10 ** 9, "full"),
    ("fp32 queries", torch.float32, 64, 10 ** 9, "base"),
    ("unknown queries", torch.float64, 64, 10 ** 9, "base"),
    ("small pages", torch.bfloat16, 4, 10 ** 9, "base"),
    ("no memory", torch.bfloat16, 64, 20 * 10 ** 6, "base"),
    ("beyond the limit", torch.bfloat16, 64, 10 ** 12, "base"),
])
def test_a_call_without_workspace_takes_what_it_can_use(kvk, what, dtype, page, memory, want):
    """The scratch that Layout.mla_chunk allocates itself: the expanded rows of the pool only where
    the call expands rows, within the limit, and if the allocation succeeds."""
    slots = 10 ** 6
    lay = object.__new__(kvk.Layout)
    lay.handle, _, _ = kvk.kvk_create_layout([0], [64], [8], 64, 16, 1, slots)
    asked = []

    def scratch(n):
        asked.append(n)
        if n > memory:
            raise torch.OutOfMemoryError("test")
        return n
    lay._scratch = scratch
    lay._scratch_limit = lambda: 10 ** 8 if what == "beyond the limit" else 10 ** 11
    try:
        sizes = {"base": lay.chunk_workspace_bytes(0, 0, 2, 8), "full": lay.chunk_workspace_bytes(0, 100, 2, 8)}
        assert sizes["full"] - sizes["base"] > slots * 260
        assert lay._chunk_scratch(0, dtype, 100, 2, 8, page) == sizes[want]
        assert asked == ([sizes["full"], sizes["base"]] if what == "no memory" else [sizes[want]])
    finally:
        lay.close()
