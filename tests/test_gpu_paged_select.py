"""Page selection by upper bounds, and the attention over what it selects.

The lists are whole numbers and have to be equal to the oracle's, whose scores are exact sums
rounded once to fp32."""

import numpy as np
import pytest
import torch

import block_sparse_long_sm_b200 as spa
from oracle import paged as op
from paged_common import D, Batch, attend, bits_of, check_attention, f64, to_gpu

pytestmark = pytest.mark.gpu


def run_select(b, sink, local, top, summary=None, ws=None):
    p = b.params(sink_pages=sink, local_pages=local, top_pages=top)
    sm = b.summary() if summary is None else summary
    width = sink + local + top
    lists = torch.full((b.T, b.hkv, width), -7, dtype=torch.int32, device="cuda")
    counts = torch.full((b.T, b.hkv), -7, dtype=torch.int32, device="cuda")
    ws = b.workspace(p) if ws is None else ws
    spa.check(spa.sparse_paged_select(p, b.q, to_gpu(sm), b.cu_gpu, b.kv_gpu, b.table_gpu, lists,
                                      counts, ws, b.error), "select")
    return p, sm, lists, counts, ws


def expected(b, sm, sink, local, top):
    smf = f64(sm)
    out = {}
    for t, s, pos in b.tokens():
        for g in range(b.hkv):
            q = f64(b.qkv[t, g * b.group:(g + 1) * b.group])

            def score(first, last):
                ph = b.table[s, first:last]
                return op.page_bounds(q, smf[ph, g, 0], smf[ph, g, 1])
            out[(t, g)] = op.select_pages(pos, b.page, sink, local, top, score)
    return out


def check_lists(b, lists, counts, want):
    lh, ch = lists.cpu().numpy(), counts.cpu().numpy()
    rows = set()
    for (t, g), pg in want.items():
        rows.add(t)
        assert ch[t, g] == pg.size, (t, g, ch[t, g], pg)
        assert np.array_equal(lh[t, g, :pg.size], pg), (t, g, lh[t, g], pg)
        assert np.all(lh[t, g, pg.size:] == -1)
    for t in range(b.T):
        if t not in rows:
            assert np.all(lh[t] == -7) and np.all(ch[t] == -7)


@pytest.mark.parametrize("hq,hkv,page,seqs,sink,local,top", [
    (4, 2, 16, [(1, 700), (1, 33), (1, 1), (0, 20), (1, 0), (1, 160)], 1, 2, 5),
    (8, 1, 16, [(3, 2100), (1, 1500)], 0, 1, 17),
    (5, 1, 32, [(40, 900), (2, 2)], 2, 3, 4),
    (20, 2, 64, [(1, 6000)], 1, 1, 30),
    (2, 2, 128, [(1, 3000), (4, 130)], 0, 2, 1),
    (3, 1, 16, [(1, 800)], 3, 4, 0),
    (1, 1, 16, [(2, 5000)], 1, 1, 300),
    (4, 4, 16, [(6, 3)], 1, 1, 1)])
def test_select_and_attend(hq, hkv, page, seqs, sink, local, top):
    b = Batch(hq, hkv, page, seqs, seed=hq * 7 + page, lead_rows=1, pad_rows=2)
    p, sm, lists, counts, ws = run_select(b, sink, local, top)
    want = expected(b, sm, sink, local, top)
    check_lists(b, lists, counts, want)
    o, lse = attend(b, p, lists, counts, ws=ws)
    check_attention(b, o, lse, pages_of=lambda t, g: want[(t, g)])
    b.ok()


def test_ties_go_to_the_lowest_page():
    b = Batch(4, 1, 16, [(1, 1600)], seed=1)
    sm = b.summary()
    for j in range(100):                       # three kinds of pages only
        sm[b.table[0, j], 0, 0] = bits_of(np.full(D, -1.0 - j % 3))
        sm[b.table[0, j], 0, 1] = bits_of(np.full(D, 1.0 + j % 3))
    for top in (1, 20, 40, 70, 97):
        p, _, lists, counts, _ = run_select(b, 1, 2, top, summary=sm)
        check_lists(b, lists, counts, expected(b, sm, 1, 2, top))


def test_signs_zeros_and_large_scores():
    b = Batch(2, 1, 16, [(1, 3200)], seed=2)
    rng = np.random.default_rng(0)
    lo = rng.standard_normal((200, D)) * 10.0 ** rng.integers(-20, 15, size=(200, 1))
    lo[::7] = 0.0
    lo[3::7] = -0.0
    hi = np.maximum(lo, rng.standard_normal((200, D)))
    hi[::7] = 0.0
    sm = b.summary()
    sm[b.table[0, :200], 0, 0], sm[b.table[0, :200], 0, 1] = bits_of(lo), bits_of(hi)
    for top in (3, 60, 150):
        _, _, lists, counts, _ = run_select(b, 0, 1, top, summary=sm)
        check_lists(b, lists, counts, expected(b, sm, 0, 1, top))


def test_no_candidates_anywhere():
    b = Batch(4, 2, 16, [(1, 30), (2, 16)], seed=3)
    for sink, local, top in ((5, 5, 5), (0, 1, 0), (2, 1, 0)):
        _, sm, lists, counts, _ = run_select(b, sink, local, top)
        check_lists(b, lists, counts, expected(b, sm, sink, local, top))
    b.ok()


@pytest.mark.parametrize("top", [1, 700, 16000])
def test_more_candidates_than_fit_in_shared_memory(top):
    # 17000 pages of one sequence that share a few physical pages: many equal scores as well
    b = Batch(2, 1, 16, [(1, 16 * 20)], seed=6)
    n = 17000
    rng = np.random.default_rng(1)
    b.table = rng.integers(0, 20, size=(1, n)).astype(np.int32)
    b.per_seq = n
    b.table_gpu = torch.from_numpy(b.table).cuda()
    b.kv = [n * 16]
    b.kv_gpu = torch.tensor(b.kv, dtype=torch.int32).cuda()
    sm = bits_of(rng.standard_normal((b.num_pages, 1, 2, D)))
    sm[:, :, 1] = bits_of(np.maximum(f64(sm[:, :, 0]), f64(sm[:, :, 1])))
    _, _, lists, counts, _ = run_select(b, 1, 1, top, summary=sm)
    u = op.page_bounds(f64(b.qkv[0, :2]), f64(sm[:, 0, 0]), f64(sm[:, 0, 1]))
    want = op.select_pages(n * 16 - 1, 16, 1, 1, top, lambda a, z: u[b.table[0, a:z]])
    check_lists(b, lists, counts, {(0, 0): want})
    b.ok()


def test_many_tokens_take_whole_units_in_turn():
    b = Batch(4, 2, 16, [(500, 900), (3, 700), (120, 130)], seed=7, pad_rows=5)
    p, sm, lists, counts, ws = run_select(b, 1, 2, 9)
    pick = set(int(t) for t in np.random.default_rng(0).permutation(623)[:50]) | {0, 499, 500, 503, 622}
    want = expected(b, sm, 1, 2, 9)
    check_lists(b, lists, counts, want)
    o, lse = attend(b, p, lists, counts, ws=ws)
    check_attention(b, o, lse, pages_of=lambda t, g: want[(t, g)], rows=pick)
    b.ok()


@pytest.mark.parametrize("pages,top", [(256, 9), (515, 100), (516, 1), (516, 511), (515, 511),
                                       (1030, 700), (2051, 2047)])
def test_candidate_counts_around_the_kernels_limits(pages, top):
    b = Batch(8, 2, 16, [(1, 16 * pages - 3), (1, 40)], seed=pages)
    _, sm, lists, counts, _ = run_select(b, 1, 2, top)
    check_lists(b, lists, counts, expected(b, sm, 1, 2, top))
    b.ok()


@pytest.mark.parametrize("pages", [200, 900, 1900])
def test_ties_at_the_border_of_every_size(pages):
    b = Batch(2, 1, 16, [(1, 16 * pages)], seed=1)
    rng = np.random.default_rng(pages)
    kinds = bits_of(rng.standard_normal((4, 2, D)))
    kinds[:, 1] = bits_of(np.maximum(f64(kinds[:, 0]), f64(kinds[:, 1])))
    sm = b.summary()
    for j in range(pages):
        sm[b.table[0, j], 0] = kinds[rng.integers(0, 4)]
    for top in (pages // 7, pages // 2, pages - 3):
        _, _, lists, counts, _ = run_select(b, 1, 1, top, summary=sm)
        check_lists(b, lists, counts, expected(b, sm, 1, 1, top))


@pytest.mark.parametrize("pages", [2051, 2052, 5000])
def test_candidates_around_those_kept_in_registers(pages):
    b = Batch(4, 1, 16, [(1, 16 * pages - 5)], seed=pages)
    sm = b.summary()
    for top in (1, 333, 2047):
        _, _, lists, counts, _ = run_select(b, 1, 2, top, summary=sm)
        check_lists(b, lists, counts, expected(b, sm, 1, 2, top))
    b.ok()


def test_more_rankings_than_sms():
    b = Batch(4, 4, 16, [(12, 16 * 600), (30, 16 * 700 - 9)], seed=8, pad_rows=2)
    p, sm, lists, counts, ws = run_select(b, 1, 2, 50)
    want = expected(b, sm, 1, 2, 50)
    check_lists(b, lists, counts, want)
    o, lse = attend(b, p, lists, counts, ws=ws)
    check_attention(b, o, lse, pages_of=lambda t, g: want[(t, g)], rows={0, 11, 12, 41})
    b.ok()


@pytest.mark.parametrize("tokens", [127, 128, 131])
@pytest.mark.parametrize("pages,tops,kinds", [(40, (1, 30), 90), (135, (1, 26, 131), 600),
                                              (515, (1, 100, 511), 700), (515, (73, 257), 5),
                                              (200, (28, 100), 1), (516, (100,), 700)])
def test_many_selections_at_once(tokens, pages, tops, kinds):
    """Around a thousand tokens x kv heads, where whole warps take over from blocks, over tables
    that share physical pages (few kinds of them: many equal scores)."""
    hq, hkv, page = 16, 8, 16
    b = Batch(hq, hkv, page, [(1, 1)] * tokens, seed=tokens, free=max(0, kinds - tokens), extra_cols=0,
              pad_rows=1)
    rng = np.random.default_rng(pages + kinds)
    b.per_seq = pages
    b.table = rng.integers(0, min(kinds, b.num_pages), size=(tokens, pages)).astype(np.int32)
    b.table_gpu = torch.from_numpy(b.table).cuda()
    b.kv = [int(x) for x in rng.integers(1, pages * page + 1, size=tokens)]
    b.kv[0], b.kv[1], b.kv[-1] = pages * page, 3, pages * page - 7
    b.kv_gpu = torch.tensor(b.kv, dtype=torch.int32).cuda()
    raw = rng.standard_normal((b.num_pages, hkv, 2, D))
    sm = bits_of(np.stack([raw.min(2), raw.max(2)], 2))
    pick = [0, 1, 2, tokens // 2, tokens - 1]
    for top in tops:
        _, _, lists, counts, _ = run_select(b, 1, 2, top, summary=sm)
        lh, ch = lists.cpu().numpy(), counts.cpu().numpy()
        for t in pick:
            for g in (0, 5, hkv - 1):
                q = f64(b.qkv[t, 2 * g:2 * g + 2])
                smf = f64(sm[:, g])
                u = op.page_bounds(q, smf[:, 0], smf[:, 1])
                want = op.select_pages(b.kv[t] - 1, page, 1, 2, top, lambda a, z: u[b.table[t, a:z]])
                assert ch[t, g] == want.size
                assert np.array_equal(lh[t, g, :want.size], want), (t, g)
                assert np.all(lh[t, g, want.size:] == -1)
        assert np.all(lh[tokens] == -7) and np.all(ch[tokens] == -7)
    b.ok()
