"""Argument checks of the paged-cache calls: refused before any launch, on any machine."""

import ctypes

import pytest
import torch

import block_sparse_long_sm_b200 as spa
from block_sparse_long_sm_b200 import binding

A = 1 << 20            # an aligned stand-in address, never touched
ROWS = spa.SpaRows(A, 0, 4096, 128)


def paged(**kw):
    base = dict(page_size=16, num_pages=8, seqs=2, tokens=4, pages_per_seq=4)
    heads = (kw.pop("heads_q", 4), kw.pop("heads_kv", 2))
    base.update(kw)
    return spa.make_paged_params(*heads, **base)


def attn(p, q=ROWS, k=A, v=A, cu=A, kv=A, table=A, lists=None, counts=None, o=ROWS, lse=A, ws=A,
         nbytes=1 << 40, err=A):
    return spa.sparse_paged_attn(p, q, k, v, cu, kv, table, lists, counts, o, lse, ws, err,
                                 workspace_bytes=nbytes, stream=0)


def select(p, q=ROWS, summary=A, lists=A, counts=A, ws=A, nbytes=1 << 40, err=A):
    return spa.sparse_paged_select(p, q, summary, A, A, A, lists, counts, ws, err,
                                   workspace_bytes=nbytes, stream=0)


def append(p, r=None, q=None, k=ROWS, v=ROWS, qw=None, kw=None, table=A, qo=None, kc=A, vc=A,
           sm=None, err=A, cu=A):
    return spa.sparse_paged_append(p, r, q, k, v, qw, kw, table, cu, A, A, qo, kc, vc, sm, err,
                                   stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=64), spa.SPA_ERR_UNSUPPORTED), (dict(page_size=8), spa.SPA_ERR_UNSUPPORTED),
    (dict(page_size=48), spa.SPA_ERR_UNSUPPORTED), (dict(page_size=256), spa.SPA_ERR_UNSUPPORTED),
    (dict(page_size=0), spa.SPA_ERR_INVALID), (dict(num_pages=0), spa.SPA_ERR_INVALID),
    (dict(pages_per_seq=0), spa.SPA_ERR_INVALID), (dict(seqs=-1), spa.SPA_ERR_INVALID),
    (dict(tokens=-1), spa.SPA_ERR_INVALID), (dict(heads_q=3), spa.SPA_ERR_INVALID),
    (dict(heads_q=0), spa.SPA_ERR_INVALID), (dict(heads_kv=0), spa.SPA_ERR_INVALID),
    (dict(heads_q=258, heads_kv=2), spa.SPA_ERR_UNSUPPORTED),
    (dict(page_stride=100), spa.SPA_ERR_INVALID), (dict(page_stride=2048), spa.SPA_ERR_INVALID),
    (dict(page_stride=-128), spa.SPA_ERR_INVALID), (dict(softmax_scale=-1.0), spa.SPA_ERR_INVALID),
    (dict(softmax_scale=float("nan")), spa.SPA_ERR_INVALID),
    (dict(sink_pages=-1), spa.SPA_ERR_INVALID), (dict(local_pages=0), spa.SPA_ERR_INVALID),
    (dict(top_pages=-1), spa.SPA_ERR_INVALID),
    (dict(num_pages=1 << 27), spa.SPA_ERR_UNSUPPORTED),
    (dict(pages_per_seq=1 << 27), spa.SPA_ERR_UNSUPPORTED),
    (dict(top_pages=1 << 30), spa.SPA_ERR_UNSUPPORTED),
    (dict(tokens=1 << 30), spa.SPA_ERR_UNSUPPORTED)])
def test_params(kw, code):
    p = paged(**kw)
    assert spa.sparse_paged_workspace_bytes(p) == 0
    assert attn(p) == select(p) == append(p) == code


def test_workspace_is_closed_form_and_covers_its_parts():
    n = spa.sparse_paged_workspace_bytes(paged())
    assert n >= 2 * 148 * 256 * 130 * 4
    m = spa.sparse_paged_workspace_bytes(paged(tokens=1000, pages_per_seq=4096))
    assert m - n >= (1000 * 4096 - 4 * 4) * 2 * 4 - 256


def test_plain_attention_needs_no_room_for_scores():
    # a 16K chunk over 128K positions in pages of 16: the scores alone would be 1 GB per kv head
    small, large = paged(), paged(tokens=16384, pages_per_seq=8192)
    ranked = paged(tokens=16384, pages_per_seq=8192, top_pages=8)
    base = spa.sparse_paged_attn_workspace_bytes(small)
    assert base == spa.sparse_paged_attn_workspace_bytes(large)
    assert base == spa.sparse_paged_attn_workspace_bytes(ranked)
    assert 2 * 148 * 256 * 130 * 4 <= base < 40 << 20
    assert base <= spa.sparse_paged_workspace_bytes(small)
    assert spa.sparse_paged_attn_workspace_bytes(paged(head_dim=64)) == 0
    odd = spa.SpaRows(A, 0, 384, 256)      # refused behind the workspace's check
    for lists in (None, A):
        for p in (large, ranked):
            kw = dict(q=odd, lists=lists, counts=lists)
            assert attn(p, nbytes=base, **kw) == spa.SPA_ERR_UNSUPPORTED
            assert attn(p, nbytes=base - 1, **kw) == spa.SPA_ERR_WORKSPACE
    # the selection wants its scores' room when it ranks
    full = spa.sparse_paged_workspace_bytes(ranked)
    assert full - base >= 16384 * 2 * 8191 * 8
    assert select(ranked, nbytes=full, summary=0) == spa.SPA_ERR_INVALID
    assert select(ranked, nbytes=full - 1, summary=0) == spa.SPA_ERR_WORKSPACE
    assert select(large, nbytes=base, summary=0) == spa.SPA_ERR_INVALID
    assert select(large, nbytes=base - 1, summary=0) == spa.SPA_ERR_WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(ws=0), spa.SPA_ERR_INVALID), (dict(ws=A + 8), spa.SPA_ERR_INVALID),
    (dict(nbytes=100), spa.SPA_ERR_WORKSPACE), (dict(err=0), spa.SPA_ERR_INVALID),
    (dict(err=A + 2), spa.SPA_ERR_INVALID), (dict(q=None), spa.SPA_ERR_INVALID),
    (dict(q=spa.SpaRows(A + 8, 0, 128, 128)), spa.SPA_ERR_INVALID),
    (dict(q=spa.SpaRows(A, 0, 4, 128)), spa.SPA_ERR_INVALID),
    (dict(q=spa.SpaRows(A, 0, 128, 130)), spa.SPA_ERR_INVALID),
    (dict(q=spa.SpaRows(A, 0, -128, 128)), spa.SPA_ERR_UNSUPPORTED),
    (dict(q=spa.SpaRows(A, 0, 0, 128)), spa.SPA_ERR_UNSUPPORTED),
    (dict(q=spa.SpaRows(A, 0, 384, 256)), spa.SPA_ERR_UNSUPPORTED),
    (dict(q=spa.SpaRows(A, 0, 256, 384)), spa.SPA_ERR_UNSUPPORTED)])
def test_attn_and_select_arguments(kw, code):
    assert attn(paged(), **kw) == code
    if code != spa.SPA_ERR_UNSUPPORTED:
        assert select(paged(), **kw) == code


@pytest.mark.parametrize("kw", [dict(k=0), dict(v=A + 4), dict(cu=0), dict(kv=A + 1), dict(table=0),
                                dict(o=None), dict(lse=A + 2), dict(lists=A), dict(counts=A),
                                dict(lists=A + 1, counts=A)])
def test_attn_arguments(kw):
    assert attn(paged(), **kw) == spa.SPA_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(summary=0), dict(summary=A + 8), dict(lists=0), dict(counts=0)])
def test_select_arguments(kw):
    assert select(paged(), **kw) == spa.SPA_ERR_INVALID


def rope(**kw):
    base = dict(table_rows=64)
    base.update(kw)
    dims = [base.pop(n, d) for n, d in (("batch", 1), ("tokens", 4), ("heads_q", 4), ("heads_kv", 2))]
    return spa.make_rope_params(*dims, **base)


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(kc=0), dict(vc=A + 8), dict(err=0),
                                dict(cu=0), dict(q=ROWS), dict(qo=ROWS), dict(sm=A + 2),
                                dict(r=rope(batch=2)), dict(r=rope(tokens=5)),
                                dict(r=rope(heads_q=2)), dict(r=rope(), table=0),
                                dict(r=rope(), kw=A + 2), dict(r=rope(eps=-1.0)),
                                dict(k=spa.SpaRows(A, 0, 129, 128))])
def test_append_arguments(kw):
    assert append(paged(), **kw) == spa.SPA_ERR_INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=64), spa.SPA_ERR_UNSUPPORTED), (dict(rotary_dim=96), spa.SPA_ERR_UNSUPPORTED),
    (dict(rotary_dim=-2), spa.SPA_ERR_INVALID), (dict(rotary_dim=256), spa.SPA_ERR_INVALID),
    (dict(interleaved=2), spa.SPA_ERR_INVALID), (dict(table_rows=0), spa.SPA_ERR_INVALID),
    (dict(eps=float("inf")), spa.SPA_ERR_INVALID), (dict(batch=-1), spa.SPA_ERR_INVALID),
    (dict(heads_q=0), spa.SPA_ERR_INVALID),
    (dict(batch=1 << 16, tokens=1 << 16), spa.SPA_ERR_UNSUPPORTED)])
def test_rope_params(kw, code):
    r = rope(**kw)
    assert spa.sparse_qk_norm_rope(r, ROWS, ROWS, None, None, None, A, ROWS, ROWS, A,
                                   stream=0) == code


def test_rope_arguments():
    call = lambda q=ROWS, k=ROWS, qw=None, pos=None, table=A, qo=ROWS, ko=ROWS, err=A: \
        spa.sparse_qk_norm_rope(rope(), q, k, qw, None, pos, table, qo, ko, err, stream=0)
    for kw in (dict(q=None), dict(ko=None), dict(table=0), dict(table=A + 4), dict(err=0),
               dict(pos=A + 2), dict(qw=A + 2), dict(q=spa.SpaRows(A, 1, 128, 128)),
               dict(qo=spa.SpaRows(0, 0, 128, 128))):
        assert call(**kw) == spa.SPA_ERR_INVALID, kw


def test_empty_calls_launch_nothing():
    assert attn(paged(tokens=0), q=None, o=None, k=0, v=0) == spa.SPA_OK
    assert select(paged(seqs=0), q=None, summary=0) == spa.SPA_OK
    assert append(paged(tokens=0), k=None, v=None) == spa.SPA_OK
    assert spa.sparse_qk_norm_rope(rope(tokens=0), None, None, None, None, None, None, None, None, A,
                                   stream=0) == spa.SPA_OK
    assert spa.sparse_paged_status(0, stream=0) == spa.SPA_ERR_INVALID


def test_tensor_checks_of_the_binding():
    x = torch.zeros(4, 4, 128, dtype=torch.bfloat16)
    rows = binding.SpaRows.from_buffer_copy(binding._rows(x, 1, 4, 4, "q"))
    assert (rows.stride_batch, rows.stride_token, rows.stride_head) == (0, 512, 128)
    y = torch.zeros(2, 3, 5, 128, dtype=torch.bfloat16).transpose(1, 2)
    rows = binding.SpaRows.from_buffer_copy(binding._rows(y, 2, 5, 3, "q"))
    assert (rows.stride_batch, rows.stride_token, rows.stride_head) == (1920, 128, 640)
    for bad, exc in ((x.half(), TypeError), (x[:3], ValueError),
                     (x.transpose(1, 2).contiguous().transpose(1, 2), ValueError)):
        with pytest.raises(exc):
            binding._rows(bad, 1, 4, 4, "q")
    p = paged()
    cache = torch.zeros(8, 2, 16, 128, dtype=torch.bfloat16)
    assert binding._cache(p, cache, "k") == cache.data_ptr()
    for bad, exc in ((cache[:7], ValueError), (cache.float(), TypeError),
                     (cache.transpose(1, 2).contiguous().transpose(1, 2), ValueError),
                     (torch.zeros(8, 4, 16, 128, dtype=torch.bfloat16)[:, :2], ValueError)):
        with pytest.raises(exc):
            binding._cache(p, bad, "k")
    both = torch.zeros(8, 4, 16, 128, dtype=torch.bfloat16)
    assert binding._cache(paged(page_stride=4 * 16 * 128), both[:, 2:], "v") == both[:, 2:].data_ptr()
    with pytest.raises(ValueError):
        binding._flat(torch.zeros(3, dtype=torch.int32), torch.int32, 4, "cu_q")
    with pytest.raises(TypeError):
        binding._flat(torch.zeros(4, dtype=torch.int64), torch.int32, 4, "cu_q")
    with pytest.raises(ValueError):
        binding._flat(torch.zeros(4, 2, dtype=torch.int32)[:, 0], torch.int32, 4, "cu_q")
    with pytest.raises(ValueError):                    # host memory
        spa.sparse_paged_status(torch.zeros(1, dtype=torch.int32), stream=0)


def test_tensors_of_another_width_are_refused(monkeypatch):
    """A contiguous tensor with elements enough, but rows of another length, would be read with
    the wrong row stride.  Accepted ones reach the library, which refuses the head size."""
    monkeypatch.setattr(binding, "_device", lambda *x: -1)
    i32, f32, bf16 = torch.int32, torch.float32, torch.bfloat16
    z = lambda dtype, *shape: torch.zeros(*shape, dtype=dtype)
    p = paged(head_dim=64, sink_pages=1, local_pages=2, top_pages=3)     # 2 x 4 table, 4 x 2 x 6 lists
    r = rope(head_dim=64, batch=2)                                       # 64 x 128 table
    one = paged(head_dim=64, seqs=1, tokens=1, heads_kv=1)

    def on_attn(p, table=A, lists=A, counts=A, lse=A):
        return spa.sparse_paged_attn(p, ROWS, A, A, A, A, table, lists, counts, ROWS, lse, A, A,
                                     workspace_bytes=1 << 40, stream=0)

    def on_select(p, table=A, lists=A, counts=A, summary=A):
        return spa.sparse_paged_select(p, ROWS, summary, A, A, table, lists, counts, A, A,
                                       workspace_bytes=1 << 40, stream=0)

    def on_append(p, table=A, summary=A, angles=A, weight=None):
        return spa.sparse_paged_append(p, r, None, ROWS, ROWS, weight, weight, angles, A, A, table,
                                       None, A, A, summary, A, stream=0)

    def on_rope(r, positions=A, angles=A, weight=None):
        return spa.sparse_qk_norm_rope(r, ROWS, ROWS, weight, None, positions, angles, ROWS, ROWS, A,
                                       stream=0)

    for call, kw in ((on_attn, dict(table=z(i32, 2, 5))), (on_attn, dict(table=z(i32, 4, 2))),
                     (on_attn, dict(table=z(i32, 1, 8))), (on_select, dict(table=z(i32, 2, 5))),
                     (on_append, dict(table=z(i32, 2, 5))), (on_attn, dict(lists=z(i32, 4, 2, 7))),
                     (on_select, dict(lists=z(i32, 4, 2, 7))), (on_attn, dict(lists=z(i32, 4, 3, 6))),
                     (on_attn, dict(counts=z(i32, 4, 3))), (on_select, dict(counts=z(i32, 2, 4))),
                     (on_attn, dict(lse=z(f32, 4, 8))), (on_attn, dict(lse=z(f32, 3, 4))),
                     (on_select, dict(summary=z(bf16, 8, 4, 2, 128))),
                     (on_append, dict(summary=z(bf16, 8, 2, 4, 128))),
                     (on_append, dict(angles=z(f32, 64, 256))), (on_append, dict(angles=z(f32, 63, 128))),
                     (on_append, dict(weight=z(bf16, 4, 128))), (on_append, dict(table=z(i32, 7)))):
        with pytest.raises(ValueError, match="shape|elements"):
            call(p, **kw)
    for kw in (dict(positions=z(i32, 2, 5)), dict(angles=z(f32, 128, 64)), dict(weight=z(bf16, 2, 128))):
        with pytest.raises(ValueError, match="shape"):
            on_rope(r, **kw)
    # as wanted, with more rows, flat, or a single row that is longer
    for call, q, kw in ((on_attn, p, dict(table=z(i32, 2, 4), lists=z(i32, 4, 2, 6),
                                          counts=z(i32, 4, 2), lse=z(f32, 4, 4))),
                        (on_attn, p, dict(table=z(i32, 9, 4), lists=z(i32, 5, 2, 6),
                                          counts=z(i32, 5, 2), lse=z(f32, 6, 4))),
                        (on_attn, p, dict(table=z(i32, 8), lists=z(i32, 8, 6), counts=z(i32, 20))),
                        (on_attn, one, dict(table=z(i32, 1, 9), lists=z(i32, 1, 1, 7),
                                            counts=z(i32, 1, 1), lse=z(f32, 1, 4))),
                        (on_select, p, dict(summary=z(bf16, 8, 2, 2, 128))),
                        (on_select, p, dict(summary=z(bf16, 8, 2, 256))),
                        (on_append, p, dict(angles=z(f32, 80, 128), weight=z(bf16, 128))),
                        (on_append, p, dict(angles=z(f32, 1, 80, 128), table=z(i32, 1, 3, 4))),
                        (on_rope, r, dict(positions=z(i32, 2, 4), angles=z(f32, 64, 128),
                                          weight=z(bf16, 1, 128))),
                        (on_rope, r, dict(positions=z(i32, 8)))):
        assert call(q, **kw) == spa.SPA_ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        on_attn(p, table=z(torch.int64, 2, 4))
    with pytest.raises(ValueError, match="contiguous"):
        on_attn(p, table=z(i32, 2, 8)[:, :4])


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(spa.SpaRows) == 32
    assert ctypes.sizeof(spa.SpaRopeParams) == 36
    assert ctypes.sizeof(spa.SpaPagedParams) == 64
