"""Attention of new tokens over a paged cache, against fp64 (tolerances: paged_common)."""

import numpy as np
import pytest
import torch

import block_sparse_long_sm_b200 as spa
from paged_common import SENTINEL, Batch, attend, check_attention

pytestmark = pytest.mark.gpu

# (n, kv): lengths of one, tile and page borders and their neighbours, no new token, no keys,
# more new tokens than keys (the first ones see nothing)
EDGES = [(1, 1), (1, 127), (0, 40), (1, 128), (1, 129), (3, 3), (1, 0), (1, 17), (2, 257),
         (0, 0), (5, 2), (1, 700)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (8, 1)])
def test_single_tokens_and_edges(hq, hkv, page):
    b = Batch(hq, hkv, page, EDGES, seed=page + hq)
    check_attention(b, *attend(b))
    b.ok()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (3, 1), (10, 2), (7, 1), (16, 1), (33, 1), (64, 1),
                                    (100, 1), (128, 1)])
def test_group_sizes(hq, hkv):
    b = Batch(hq, hkv, 32, [(1, 300), (2, 65), (1, 1)], seed=hq)
    check_attention(b, *attend(b))
    b.ok()


@pytest.mark.parametrize("hq,hkv,page,seqs", [
    (4, 2, 16, [(200, 200)]), (4, 2, 64, [(131, 400), (300, 301)]), (2, 2, 128, [(257, 513)]),
    (5, 1, 32, [(60, 200), (77, 77)]), (8, 1, 16, [(33, 129), (64, 64), (1, 500)]),
    (3, 3, 64, [(129, 1000)]), (1, 1, 16, [(300, 290)]), (12, 2, 32, [(140, 143)])])
def test_chunks(hq, hkv, page, seqs):
    b = Batch(hq, hkv, page, seqs, seed=hq * 10 + page)
    check_attention(b, *attend(b))
    b.ok()


def test_one_long_sequence_is_split_over_every_sm():
    b = Batch(4, 1, 64, [(1, 30001)], seed=5)
    check_attention(b, *attend(b))
    b.ok()
    b = Batch(2, 1, 128, [(130, 9999)], seed=6)
    check_attention(b, *attend(b), rows={0, 1, 63, 64, 127, 128, 129})
    b.ok()


def test_many_sequences_more_than_a_block_scans_at_once():
    rng = np.random.default_rng(3)
    seqs = [(int(rng.integers(0, 3)), int(rng.integers(2, 90))) for _ in range(900)]
    b = Batch(2, 1, 16, seqs, seed=9)
    check_attention(b, *attend(b))
    b.ok()


def test_rows_outside_the_sequences_are_left_alone():
    b = Batch(4, 2, 16, [(2, 30), (1, 5), (0, 9)], seed=1, lead_rows=3, pad_rows=4)
    check_attention(b, *attend(b))        # NaN rows of q around, sentinels kept in o and lse
    b.ok()


@pytest.mark.parametrize("joint,gap", [(True, 0), (False, 3), (True, 5)])
def test_strided_pages(joint, gap):
    b = Batch(4, 2, 32, [(1, 100), (140, 200), (3, 64)], seed=2, joint=joint, gap=gap)
    check_attention(b, *attend(b))
    b.ok()


def test_softmax_scale_and_no_lse():
    b = Batch(4, 2, 16, [(1, 200), (4, 50)], seed=4)
    p = b.params(softmax_scale=0.2)
    o, lse = attend(b, p)
    check_attention(b, o, lse, scale=float(np.float32(0.2)))
    o2 = torch.full_like(o, SENTINEL)
    spa.check(spa.sparse_paged_attn(p, b.q, b.kc, b.vc, b.cu_gpu, b.kv_gpu, b.table_gpu, None, None,
                                    o2, None, b.workspace(p), b.error))
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16))


def test_empty_calls():
    b = Batch(4, 2, 16, [(0, 10), (0, 0)], seed=4, pad_rows=2)
    o, lse = attend(b)
    assert bool((o == SENTINEL).all()) and bool((lse == SENTINEL).all())
    b = Batch(4, 2, 16, [], seed=4)
    attend(b)
    b.ok()


@pytest.mark.parametrize("seqs", [[(1, 2000), (1, 77), (1, 500)], [(150, 800), (1, 40)]])
def test_repeats_are_bit_equal_on_a_dirty_workspace(seqs):
    b = Batch(8, 2, 32, seqs, seed=8)
    p = b.params()
    ws = b.workspace(p)
    o, lse = attend(b, p, ws=ws)
    for fill in (0x00, 0x7F):
        ws.fill_(fill)
        o2, lse2 = attend(b, p, ws=ws)
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
    check_attention(b, o, lse, rows={0, 1, 2, 149, 150})


def test_own_lists():
    # the caller's own ascending pages, with and without the token's own page, and none at all
    b = Batch(4, 2, 16, [(2, 100), (1, 33), (3, 2)], seed=11)
    p = b.params(sink_pages=1, local_pages=2, top_pages=3)
    lists = np.full((b.T, 2, 6), -1, np.int32)
    counts = np.zeros((b.T, 2), np.int32)
    want = {}
    rng = np.random.default_rng(0)
    for t, s, pos in b.tokens():
        for g in range(2):
            seen = max(0, pos + 1 + 15) // 16 if pos >= 0 else 0
            m = int(rng.integers(0, min(6, seen) + 1))
            pg = np.sort(rng.permutation(seen)[:m])
            lists[t, g, :m], counts[t, g] = pg, m
            want[(t, g)] = pg.astype(np.int64)
    o, lse = attend(b, p, torch.from_numpy(lists).cuda(), torch.from_numpy(counts).cuda())
    check_attention(b, o, lse, pages_of=lambda t, g: want[(t, g)])
    b.ok()


@pytest.mark.parametrize("hq,hkv,page,seed", [(4, 2, 16, 0), (20, 4, 32, 1), (8, 1, 64, 2),
                                              (6, 6, 128, 3), (32, 1, 16, 4), (12, 2, 16, 5)])
def test_batches_that_mix_tokens_and_chunks(hq, hkv, page, seed):
    # few rows, one row tile and two, with tails of all of them, in any order
    rng = np.random.default_rng(seed)
    seqs = []
    for _ in range(40):
        n = int(rng.choice([0, 1, 1, 1, 2, 3, 5, 17, 26, 40, 65, 130]))
        seqs.append((n, n + int(rng.choice([0, 0, 1, 100, 127, 128, 300, 700]))))
    b = Batch(hq, hkv, page, seqs, seed=seed)
    o, lse = attend(b)
    rows = set(int(t) for t in np.random.default_rng(seed).permutation(b.T)[:60])
    check_attention(b, o, lse, rows=rows | set(int(x) for x in b.cu[:-1]))
    b.ok()


@pytest.mark.parametrize("seqs", [[(1, 3000), (1, 77)], [(300, 2000), (1, 40)]])
def test_attention_stays_within_its_own_workspace(seqs):
    b = Batch(8, 2, 16, seqs, seed=12)
    p = b.params()
    n = spa.sparse_paged_attn_workspace_bytes(p)
    assert n < spa.sparse_paged_workspace_bytes(p)
    ws = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    o, lse = attend(b, p, ws=ws[:n])
    check_attention(b, o, lse, rows={0, 1, 127, 128, 299, 300})
    assert bool((ws[n:] == 0xFF).all())
    b.ok()
