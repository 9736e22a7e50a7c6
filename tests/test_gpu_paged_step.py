"""The paged-cache calls as a server uses them: in sequence, captured and replayed, on other
streams, with strided inputs and outputs, past 32-bit offsets, and with device values that are
out of range (reported, never followed)."""

import math

import numpy as np
import pytest
import torch

import block_sparse_long_sm_b200 as spa
from oracle import paged as op
from paged_common import (D, SENTINEL, Batch, attend, bits_of, check_attention, f64, to_f64, to_gpu)

pytestmark = pytest.mark.gpu


def close(o, ref, w, what):
    lim = 2.0 ** -8 * (w + np.abs(ref)) * (1 + 2.0 ** -5)      # as in check_attention
    assert np.all(np.abs(o - ref) <= lim), (what, float(np.max(np.abs(o - ref) / lim)))


def test_a_layer_from_the_prompt_to_the_answer():
    """Prompt: norm and rotation into the head-major layout, plan and attention over it, and the
    same keys into pages.  Answer: per token append, selection, attention -- against fp64 over
    what the cache really holds; and the prompt as a chunk over pages equals the dense prefill."""
    hq, hkv, page, L, steps = 8, 2, 32, 700, 5
    group, rng = hq // hkv, np.random.default_rng(0)
    cap = L + steps
    per_seq = (cap + page - 1) // page
    num_pages = per_seq + 3
    table = torch.from_numpy(rng.permutation(num_pages)[:per_seq][None].astype(np.int32)).cuda()
    rope = torch.from_numpy(op.rope_table(cap, 128)).cuda()
    wq, wk = (to_gpu(bits_of(1 + 0.2 * rng.standard_normal(D))) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((num_pages, hkv, page, D), float("nan"), device="cuda", dtype=torch.bfloat16)
              for _ in range(2))
    sm = torch.full((num_pages, hkv, 2, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")

    qkv = to_gpu(bits_of(rng.standard_normal((L, hq + 2 * hkv, D))))
    q_hm = torch.empty(1, hq, L, D, device="cuda", dtype=torch.bfloat16)
    k_hm = torch.empty(1, hkv, L, D, device="cuda", dtype=torch.bfloat16)
    r = spa.make_rope_params(1, L, hq, hkv, table_rows=cap)
    spa.check(spa.sparse_qk_norm_rope(r, qkv[None, :, :hq], qkv[None, :, hq:hq + hkv], wq, wk, None,
                                      rope, q_hm.transpose(1, 2), k_hm.transpose(1, 2), err))
    pp = spa.make_paged_params(hq, hkv, page_size=page, num_pages=num_pages, seqs=1, tokens=L,
                               pages_per_seq=per_seq)
    q_tok = torch.empty(L, hq, D, device="cuda", dtype=torch.bfloat16)
    spa.check(spa.sparse_paged_append(pp, r, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], wq,
                                      wk, rope, i32(0, L), i32(L), table, q_tok, kc, vc, sm, err))
    assert torch.equal(q_tok.transpose(0, 1), q_hm[0])
    phys = table[0].long()
    rows = lambda c, n: c[phys].transpose(1, 2).reshape(-1, hkv, D)[:n]
    assert torch.equal(rows(kc, L).transpose(0, 1), k_hm[0])
    assert torch.equal(rows(vc, L), qkv[:, hq + hkv:])

    v_hm = qkv[:, hq + hkv:].transpose(0, 1).contiguous()[None]
    dp = spa.make_params(1, hq, hkv, L, mode="dense")
    ws = torch.empty(spa.sparse_prefill_workspace_bytes(dp), dtype=torch.uint8, device="cuda")
    o_hm, lse_hm = torch.empty_like(q_hm), torch.empty(1, hq, L, device="cuda")
    spa.check(spa.sparse_prefill_plan(dp, q_hm, k_hm, ws))
    spa.check(spa.sparse_prefill_attn(dp, q_hm, k_hm, v_hm, ws, o_hm, lse_hm))
    pws = torch.empty(spa.sparse_paged_workspace_bytes(pp), dtype=torch.uint8, device="cuda")
    o = torch.empty(L, hq, D, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(L, hq, device="cuda")
    spa.check(spa.sparse_paged_attn(pp, q_tok, kc, vc, i32(0, L), i32(L), table, None, None, o, lse,
                                    pws, err))
    a, b = to_f64(o.transpose(0, 1)), to_f64(o_hm[0])
    va = np.abs(to_f64(v_hm[0])).max()
    assert np.max(np.abs(a - b)) <= 2 * 2.0 ** -8 * 2 * va      # both within their bound of the same
    assert np.max(np.abs(lse.T.cpu().numpy() - lse_hm[0].cpu().numpy())) <= 1e-4

    top = dict(sink_pages=1, local_pages=2, top_pages=4)
    for i in range(steps):
        x = to_gpu(bits_of(rng.standard_normal((1, hq + 2 * hkv, D))))
        n = L + i + 1
        p1 = spa.make_paged_params(hq, hkv, page_size=page, num_pages=num_pages, seqs=1, tokens=1,
                                   pages_per_seq=per_seq, **top)
        r1 = spa.make_rope_params(1, 1, hq, hkv, table_rows=cap)
        q1 = torch.empty(1, hq, D, device="cuda", dtype=torch.bfloat16)
        spa.check(spa.sparse_paged_append(p1, r1, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], wq,
                                          wk, rope, i32(0, 1), i32(n), table, q1, kc, vc, sm, err))
        w1 = torch.empty(spa.sparse_paged_workspace_bytes(p1), dtype=torch.uint8, device="cuda")
        lists = torch.empty(1, hkv, 7, dtype=torch.int32, device="cuda")
        counts = torch.empty(1, hkv, dtype=torch.int32, device="cuda")
        o1 = torch.empty(1, hq, D, device="cuda", dtype=torch.bfloat16)
        spa.check(spa.sparse_paged_select(p1, q1, sm, i32(0, 1), i32(n), table, lists, counts, w1, err))
        spa.check(spa.sparse_paged_attn(p1, q1, kc, vc, i32(0, 1), i32(n), table, lists, counts, o1,
                                        None, w1, err))
        kh, vh, qh, smh = to_f64(rows(kc, n)), to_f64(rows(vc, n)), to_f64(q1[0]), to_f64(sm[phys])
        for g in range(hkv):
            full = [kh[j * page:min(n, (j + 1) * page), g] for j in range((n - 1) // page + 1)]
            assert np.array_equal(smh[:len(full), g, 0], np.stack([f.min(0) for f in full]))
            assert np.array_equal(smh[:len(full), g, 1], np.stack([f.max(0) for f in full]))
            qg = qh[g * group:(g + 1) * group]
            want = op.select_pages(n - 1, page, 1, 2, 4,
                                   lambda a, z: op.page_bounds(qg, smh[a:z, g, 0], smh[a:z, g, 1]))
            assert lists[0, g, :want.size].tolist() == want.tolist()
            idx = (want[:, None] * page + np.arange(page)).reshape(-1)
            idx = idx[idx < n]
            for h in range(group):
                ref, _, w = op.attend(qg[h], kh[idx, g], vh[idx, g], 1 / math.sqrt(D))
                close(to_f64(o1[0, g * group + h]), ref, w, (i, g, h))
    spa.check(spa.sparse_paged_status(err))


def test_captured_steps_replay_on_changed_lengths():
    b = Batch(8, 2, 16, [(1, 300), (1, 90), (1, 1000)], seed=1)
    p = b.params(sink_pages=1, local_pages=2, top_pages=5)
    ws = b.workspace(p)
    sm = to_gpu(b.summary())
    lists = torch.zeros(b.T, 2, 8, dtype=torch.int32, device="cuda")
    counts = torch.zeros(b.T, 2, dtype=torch.int32, device="cuda")
    o, lse = torch.zeros(b.T, 8, D, device="cuda", dtype=torch.bfloat16), torch.zeros(b.T, 8, device="cuda")
    of, lsef = torch.zeros_like(o), torch.zeros_like(lse)

    def step(stream=None):
        spa.check(spa.sparse_paged_select(p, b.q, sm, b.cu_gpu, b.kv_gpu, b.table_gpu, lists, counts,
                                          ws, b.error, stream=stream))
        spa.check(spa.sparse_paged_attn(p, b.q, b.kc, b.vc, b.cu_gpu, b.kv_gpu, b.table_gpu, lists,
                                        counts, o, lse, ws, b.error, stream=stream))
        spa.check(spa.sparse_paged_attn(p, b.q, b.kc, b.vc, b.cu_gpu, b.kv_gpu, b.table_gpu, None,
                                        None, of, lsef, ws, b.error, stream=stream))
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for kv in ([300, 90, 1000], [17, 90, 16], [1, 64, 777]):
        b.kv_gpu.copy_(torch.tensor(kv, dtype=torch.int32))
        step()
        want = [x.clone() for x in (lists, counts, o, lse, of, lsef)]
        for x in (lists, counts, o, lse, of, lsef):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((lists, counts, o, lse, of, lsef), want):
            assert torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x,
                               y.view(torch.int16) if y.dtype == torch.bfloat16 else y)
        b.kv, save = kv, b.kv
        check_attention(b, of, lsef)
        b.kv = save
    b.ok()


def test_two_streams_with_workspaces_of_their_own():
    batches = [Batch(8, 2, 32, [(1, 3000), (150, 700)], seed=2), Batch(4, 1, 16, [(1, 2500), (40, 90)], seed=3)]
    alone = [attend(b) for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    out = []
    for rep in range(4):
        for b, s in zip(batches, streams):
            with torch.cuda.stream(s):
                out.append(attend(b))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(out):
        ref = alone[i % 2]
        assert torch.equal(o.view(torch.int16), ref[0].view(torch.int16)) and torch.equal(lse, ref[1])
    # a stream given by the caller, as an object and as a handle
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for given in (s, s.cuda_stream):
        o, lse = attend(batches[0], stream=given)
        s.synchronize()
    torch.cuda.synchronize()


def test_strided_queries_and_outputs():
    b = Batch(6, 2, 32, [(1, 500), (70, 130)], seed=4)
    wide = torch.full((b.T, 6, 2, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide[:, :, 1] = b.q
    buf = torch.full((6, b.T, 2 * D), SENTINEL, device="cuda", dtype=torch.bfloat16)
    o = buf[:, :, D:].transpose(0, 1)                  # head-major, rows twice as wide
    lse = torch.empty(b.T, 6, device="cuda")
    p = b.params()
    spa.check(spa.sparse_paged_attn(p, wide[:, :, 1], b.kc, b.vc, b.cu_gpu, b.kv_gpu, b.table_gpu, None,
                                    None, o, lse, b.workspace(p), b.error))
    check_attention(b, o, lse)
    assert bool((buf[:, :, :D] == SENTINEL).all())
    b.ok()


@pytest.mark.parametrize("hq,hkv,seqs", [(6, 2, [(1, 500), (70, 130), (200, 260)]), (1, 1, [(300, 400)]),
                                         (20, 1, [(9, 300), (1, 40)]), (4, 4, [(1, 99)])])
def test_head_major_queries(hq, hkv, seqs):
    b = Batch(hq, hkv, 32, seqs, seed=5)
    q = b.q.transpose(0, 1).contiguous().transpose(0, 1)      # as the prefill lays them out
    check_attention(b, *attend(b, q=q))
    b.ok()


def test_offsets_past_32_bits():
    # 24 pages 128 M elements apart: the last ones start past 2^31 elements (2^32 bytes)
    hq, hkv, page, n_pages, stride = 4, 2, 64, 24, 1 << 27
    big = torch.empty((n_pages - 1) * stride + 2 * hkv * page * D, device="cuda", dtype=torch.bfloat16)
    size, st = (n_pages, hkv, page, D), (stride, page * D, D, 1)
    b = Batch(hq, hkv, page, [(1, 300), (3, 200)], seed=5, filled="old")
    b.kc, b.vc = big.as_strided(size, st, 0), big.as_strided(size, st, hkv * page * D)
    b.num_pages, b.stride = n_pages, stride
    perm = np.random.default_rng(0).permutation(np.arange(12, 24))
    b.table[0, :5], b.table[1, :4] = perm[:5], perm[5:9]
    b.table[:, 5:] = 0
    b.table_gpu = torch.from_numpy(b.table).cuda()
    for s in range(2):
        for x in range(b.kv[s]):
            b.kc[int(b.table[s, x // page]), :, x % page] = to_gpu(b.k[s][x])
            b.vc[int(b.table[s, x // page]), :, x % page] = to_gpu(b.v[s][x])
    # the new rows once more, by the append (no norm, no rotation)
    qkv = b.qkv.copy()
    for t, s, pos in b.tokens():
        qkv[t, hq:hq + hkv], qkv[t, hq + hkv:] = b.k[s][pos], b.v[s][pos]
        b.kc[int(b.table[s, pos // page]), :, pos % page] = float("nan")
        b.vc[int(b.table[s, pos // page]), :, pos % page] = float("nan")
    g = to_gpu(qkv)
    p = b.params()
    spa.check(spa.sparse_paged_append(p, None, None, g[:, hq:hq + hkv], g[:, hq + hkv:], None, None,
                                      None, b.cu_gpu, b.kv_gpu, b.table_gpu, None, b.kc, b.vc, None,
                                      b.error))
    check_attention(b, *attend(b, p))
    b.ok()


@pytest.mark.parametrize("hq,hkv", [(32, 1), (40, 2), (128, 1)])
def test_lists_with_more_rows_than_a_few(hq, hkv):
    for seqs in ([(1, 500), (2, 90)], [(650, 700), (1, 50)]):
        b = Batch(hq, hkv, 16, seqs, seed=hq)
        p = b.params(sink_pages=1, local_pages=1, top_pages=6)
        rng = np.random.default_rng(0)
        lists = np.full((b.T, hkv, 8), -1, np.int32)
        counts = np.zeros((b.T, hkv), np.int32)
        want = {}
        for t, s, pos in b.tokens():
            for g in range(hkv):
                m = int(rng.integers(0, min(8, pos // 16 + 1) + 1))
                pg = np.sort(rng.permutation(pos // 16 + 1)[:m])
                lists[t, g, :m], counts[t, g], want[(t, g)] = pg, m, pg.astype(np.int64)
        o, lse = attend(b, p, torch.from_numpy(lists).cuda(), torch.from_numpy(counts).cuda())
        check_attention(b, o, lse, pages_of=lambda t, g: want[(t, g)],
                        rows=None if b.T < 9 else {0, 1, 333, 649, 650})
        b.ok()


def test_a_wait_that_runs_out_is_reported_and_leaves_the_context_usable():
    b = Batch(4, 2, 16, [(1, 300), (40, 200)], seed=6)
    p = b.params(debug_flags=spa.SPA_DEBUG_STALL_ATTN, wait_limit_us=2000)
    attend(b, p)
    assert spa.sparse_paged_status(b.error) == spa.SPA_ERR_TIMEOUT
    check_attention(b, *attend(b))
    b.ok()


def bad(b, field, value):
    t = getattr(b, field)
    t.copy_(torch.from_numpy(np.asarray(value, np.int32)).view(t.shape))


@pytest.mark.parametrize("field,value", [
    ("cu_gpu", [0, 2, 1, 4]), ("cu_gpu", [0, 1, 3, 400]), ("cu_gpu", [-5, 1, 3, 4]),
    ("kv_gpu", [100, -1, 30]), ("kv_gpu", [100, 10 ** 6, 30]), ("kv_gpu", [2 ** 31 - 1, 50, 30])])
def test_lengths_out_of_range_are_reported(field, value):
    b = Batch(4, 2, 16, [(1, 100), (2, 50), (1, 30)], seed=7)
    bad(b, field, value)
    attend(b)
    assert spa.sparse_paged_status(b.error) == spa.SPA_ERR_INVALID
    p = b.params(top_pages=2)
    sm = to_gpu(b.summary())
    lists = torch.zeros(b.T, 2, 3, dtype=torch.int32, device="cuda")
    counts = torch.zeros(b.T, 2, dtype=torch.int32, device="cuda")
    spa.check(spa.sparse_paged_select(p, b.q, sm, b.cu_gpu, b.kv_gpu, b.table_gpu, lists, counts,
                                      b.workspace(p), b.error))
    spa.check(spa.sparse_paged_append(p, None, None, b.qkv_gpu[:, 4:6], b.qkv_gpu[:, 6:], None, None,
                                      None, b.cu_gpu, b.kv_gpu, b.table_gpu, None, b.kc, b.vc, sm,
                                      b.error))
    assert spa.sparse_paged_status(b.error) == spa.SPA_ERR_INVALID
    torch.cuda.synchronize()


@pytest.mark.parametrize("entry", [-1, 10 ** 6, -2 ** 31])
def test_table_entries_out_of_range_are_reported(entry):
    b = Batch(4, 2, 16, [(1, 400), (30, 90)], seed=8)
    b.table_gpu[0, 3] = entry
    b.table_gpu[1, 5] = entry
    p = b.params(top_pages=2)
    sm = to_gpu(b.summary())
    lists = torch.zeros(b.T, 2, 3, dtype=torch.int32, device="cuda")
    counts = torch.zeros(b.T, 2, dtype=torch.int32, device="cuda")
    for call in range(3):
        if call == 0:
            attend(b)
        elif call == 1:
            spa.check(spa.sparse_paged_select(p, b.q, sm, b.cu_gpu, b.kv_gpu, b.table_gpu, lists,
                                              counts, b.workspace(p), b.error))
        else:
            spa.check(spa.sparse_paged_append(p, None, None, b.qkv_gpu[:, 4:6], b.qkv_gpu[:, 6:], None,
                                              None, None, b.cu_gpu, b.kv_gpu, b.table_gpu, None, b.kc,
                                              b.vc, sm, b.error))
        assert spa.sparse_paged_status(b.error) == spa.SPA_ERR_INVALID, call


@pytest.mark.parametrize("entries,count", [([3, 2, 5], 3), ([2, 2, 5], 3), ([-4, 2, 5], 3),
                                           ([0, 1, 7], 3), ([0, 1, 2], 9), ([0, 1, 2], -1)])
def test_lists_out_of_order_or_out_of_sight_are_reported(entries, count):
    b = Batch(4, 2, 16, [(1, 100)], seed=9)           # seven visible pages
    p = b.params(top_pages=2)
    lists = torch.tensor([entries, [0, 1, 6]], dtype=torch.int32, device="cuda").view(1, 2, 3)
    counts = torch.tensor([count, 3], dtype=torch.int32, device="cuda").view(1, 2)
    attend(b, p, lists, counts)
    assert spa.sparse_paged_status(b.error) == spa.SPA_ERR_INVALID


def test_captured_behind_copies_and_joined_streams():
    """Calls whose predecessors in a graph are copies, fills and kernels of two streams; each
    reads what those have just written."""
    b = Batch(8, 2, 16, [(1, 300), (4, 900), (1, 40)], seed=21)
    p = b.params(sink_pages=1, local_pages=2, top_pages=5)
    ws, sm = b.workspace(p), to_gpu(b.summary())
    r = spa.make_rope_params(1, b.T, 8, 2, table_rows=1024)
    table = torch.from_numpy(op.rope_table(1024, D)).cuda()
    pos = torch.tensor([pos for _, _, pos in b.tokens()], dtype=torch.int32, device="cuda")
    source, staged, turned = b.q.clone(), torch.zeros_like(b.q), torch.zeros_like(b.q)
    lens, kv = b.kv_gpu.clone(), torch.zeros_like(b.kv_gpu)
    lists = torch.zeros(b.T, 2, 8, dtype=torch.int32, device="cuda")
    counts = torch.zeros(b.T, 2, dtype=torch.int32, device="cuda")
    outs = [torch.zeros(b.T, 8, D, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    lses = [torch.zeros(b.T, 8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            kv.copy_(lens)
        staged.copy_(source)
        spa.check(spa.sparse_qk_norm_rope(r, staged, None, None, None, pos, table, turned, None,
                                          b.error))
        here.wait_stream(side)                                # a copy and a kernel before it
        spa.check(spa.sparse_paged_attn(p, turned, b.kc, b.vc, b.cu_gpu, kv, b.table_gpu, None, None,
                                        outs[0], lses[0], ws, b.error))
        lists.zero_()
        spa.check(spa.sparse_paged_select(p, turned, sm, b.cu_gpu, kv, b.table_gpu, lists, counts,
                                          ws, b.error))
        side.wait_stream(here)
        with torch.cuda.stream(side):
            outs[1].fill_(3.0)
        here.wait_stream(side)                                # two kernels before it
        spa.check(spa.sparse_paged_attn(p, turned, b.kc, b.vc, b.cu_gpu, kv, b.table_gpu, lists,
                                        counts, outs[1], lses[1], ws, b.error))
    step()
    torch.cuda.synchronize()
    tensors = [turned, lists, counts, *outs, *lses]
    want = [x.clone() for x in tensors]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for x in tensors + [staged, kv]:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(tensors, want):
            assert torch.equal(x, y)
    b.ok()


def test_the_stream_given_by_the_caller_is_the_one_used():
    """Every call's input is filled on that stream alone, behind a delay, so that a call on
    another stream would read what was there before; results are those of the current stream."""
    b = Batch(8, 2, 16, [(1, 300), (5, 700), (1, 40)], seed=22)
    p = b.params(sink_pages=1, local_pages=2, top_pages=5)
    ws, sm = b.workspace(p), to_gpu(b.summary())
    r = spa.make_rope_params(1, b.T, 8, 2, table_rows=1024)
    angles = torch.from_numpy(op.rope_table(1024, D)).cuda()
    pos = torch.tensor([pos for _, _, pos in b.tokens()], dtype=torch.int32, device="cuda")
    source, staged, turned = b.q.clone(), torch.zeros_like(b.q), torch.zeros_like(b.q)
    lens, kv = b.kv_gpu.clone(), torch.zeros_like(b.kv_gpu)
    kc, vc = torch.zeros_like(b.kc), torch.zeros_like(b.vc)
    lists = torch.zeros(b.T, 2, 8, dtype=torch.int32, device="cuda")
    counts = torch.zeros(b.T, 2, dtype=torch.int32, device="cuda")
    outs = [torch.zeros(b.T, 8, D, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    lses = [torch.zeros(b.T, 8, device="cuda") for _ in range(2)]
    made = [turned, kc, vc, lists, counts, *outs, *lses]

    def step(stream):
        spa.check(spa.sparse_qk_norm_rope(r, staged, None, None, None, pos, angles, turned, None,
                                          b.error, stream=stream))
        spa.check(spa.sparse_paged_append(p, None, None, b.qkv_gpu[:, 8:10], b.qkv_gpu[:, 10:], None,
                                          None, None, b.cu_gpu, kv, b.table_gpu, None, kc, vc, None,
                                          b.error, stream=stream))
        spa.check(spa.sparse_paged_select(p, turned, sm, b.cu_gpu, kv, b.table_gpu, lists, counts, ws,
                                          b.error, stream=stream))
        for i, (x, y) in enumerate(((None, None), (lists, counts))):
            spa.check(spa.sparse_paged_attn(p, turned, b.kc, b.vc, b.cu_gpu, kv, b.table_gpu, x, y,
                                            outs[i], lses[i], ws, b.error, stream=stream))

    staged.copy_(source)
    kv.copy_(lens)
    step(None)
    b.ok()
    want = [x.clone() for x in made]
    s = torch.cuda.Stream()
    for given in (s, s.cuda_stream):
        for x in [staged, kv, *made]:
            x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)          # some ten milliseconds
            staged.copy_(source)
            kv.copy_(lens)
        step(given)
        s.synchronize()
        for x, y in zip(made, want):
            assert torch.equal(x, y)
        spa.check(spa.sparse_paged_status(b.error, stream=given))
