"""Norm and rotation of the heads, and their append to a paged cache, against fp64.

Tolerance of a rotated element y = a c -+ b s: half a bf16 step (2^-8 |y|) for the one
rounding, and the fp32 arithmetic before: the norm's sum of 128 squares, root, division and
products (below 2^-17 relative in all) and the rotation's two products and sum (below 2^-22 of
|a| + |b|) -- 2^-16 (|a| + |b|) covers both.  Values and untouched rows are compared bit by bit.
"""

import numpy as np
import pytest
import torch

import block_sparse_long_sm_b200 as spa
from oracle import paged as op
from paged_common import D, SENTINEL, Batch, bits_of, f64, to_f64, to_gpu

pytestmark = pytest.mark.gpu


def weight_bits(rng):
    return bits_of(1.0 + 0.3 * rng.standard_normal(D))


def check_rows(got, x_bits, w_bits, angles, rot, pairs, eps=1e-6):
    x = f64(x_bits)
    w = None if w_bits is None else f64(w_bits)
    ref = op.norm_rope(x, w, eps, angles, rot, pairs)
    flat = op.norm_rope(x, w, eps, angles, 0, pairs)
    mag = np.abs(flat)
    both = mag.copy()
    for m in range(rot // 2):
        i, j = (2 * m, 2 * m + 1) if pairs else (m, m + rot // 2)
        both[..., i] = both[..., j] = mag[..., i] + mag[..., j]
    lim = 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * both + 1e-37
    d = np.abs(got - ref)
    assert np.all(d <= lim), float(np.max(d / lim))


@pytest.mark.parametrize("rot,pairs", [(128, 0), (128, 1), (64, 0), (64, 1), (32, 0), (32, 1),
                                       (16, 0), (16, 1), (0, 0)])
@pytest.mark.parametrize("norm", ["both", "q", "none"])
def test_rotations(rot, pairs, norm):
    rng = np.random.default_rng(rot * 4 + pairs)
    B, L, hq, hkv = 2, 5, 6, 3
    qkv = bits_of(rng.standard_normal((B, L, hq + 2 * hkv, D)))
    g = to_gpu(qkv)
    pos = rng.integers(0, 9000, size=(B, L)).astype(np.int32)
    table = op.rope_table(9000, max(rot, 16))[:, :max(rot, 1)]
    wq = weight_bits(rng) if norm != "none" else None
    wk = weight_bits(rng) if norm == "both" else None
    p = spa.make_rope_params(B, L, hq, hkv, table_rows=9000, rotary_dim=rot, interleaved=pairs)
    # head-major outputs, as the plan reads them
    qo = torch.full((B, hq, L, D), SENTINEL, device="cuda", dtype=torch.bfloat16)
    ko = torch.full((B, hkv, L, D), SENTINEL, device="cuda", dtype=torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tg = torch.from_numpy(np.ascontiguousarray(table)).cuda()
    spa.check(spa.sparse_qk_norm_rope(
        p, g[:, :, :hq], g[:, :, hq:hq + hkv], None if wq is None else to_gpu(wq),
        None if wk is None else to_gpu(wk), torch.from_numpy(pos).cuda(), tg,
        qo.transpose(1, 2), ko.transpose(1, 2), err))
    spa.check(spa.sparse_paged_status(err))
    ang = table[pos].astype(np.float64)
    check_rows(to_f64(qo.transpose(1, 2)), qkv[:, :, :hq], wq, ang, rot, pairs)
    check_rows(to_f64(ko.transpose(1, 2)), qkv[:, :, hq:hq + hkv], wk, ang, rot, pairs)


@pytest.mark.parametrize("L,hq,hkv", [(1, 1, 1), (1, 64, 8), (3, 28, 4), (700, 32, 8), (9000, 8, 2)])
def test_in_place_and_default_positions(L, hq, hkv):
    rng = np.random.default_rng(L)
    x = bits_of(rng.standard_normal((1, L, hq + hkv, D)))
    g = to_gpu(x)
    table = op.rope_table(L, 128)
    wq, wk = weight_bits(rng), weight_bits(rng)
    p = spa.make_rope_params(1, L, hq, hkv, table_rows=L)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    spa.check(spa.sparse_qk_norm_rope(p, g[:, :, :hq], g[:, :, hq:], to_gpu(wq), to_gpu(wk), None,
                                      torch.from_numpy(table).cuda(), g[:, :, :hq], g[:, :, hq:], err))
    spa.check(spa.sparse_paged_status(err))
    ang = table[None].astype(np.float64)
    got = to_f64(g)
    check_rows(got[:, :, :hq], x[:, :, :hq], wq, ang, 128, 0)
    check_rows(got[:, :, hq:], x[:, :, hq:], wk, ang, 128, 0)


def test_one_side_only_and_positions_outside_the_table():
    rng = np.random.default_rng(0)
    x = bits_of(rng.standard_normal((1, 4, 2, D)))
    g = to_gpu(x)
    out = torch.full((1, 4, 2, D), SENTINEL, device="cuda", dtype=torch.bfloat16)
    table = op.rope_table(8, 128)
    tg = torch.from_numpy(table).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = spa.make_rope_params(1, 4, 5, 2, table_rows=8)
    pos = torch.tensor([7, 8, -1, 0], dtype=torch.int32, device="cuda")
    spa.check(spa.sparse_qk_norm_rope(p, None, g, None, None, pos, tg, None, out, err))
    assert spa.sparse_paged_status(err) == spa.SPA_ERR_INVALID
    assert spa.sparse_paged_status(err) == spa.SPA_OK          # read and cleared
    got = to_f64(out)
    assert np.all(got[0, 1:3] == SENTINEL)
    ang = table[[7, 0]][None].astype(np.float64)
    check_rows(got[:, [0, 3]], x[:, [0, 3]], None, ang, 128, 0)


def extreme_rows():
    return np.stack([np.zeros(D), np.full(D, 1e-30), np.full(D, 3e4), np.eye(D)[5] * 1e-3])


def test_norm_of_zero_tiny_and_large_rows():
    x = bits_of(extreme_rows()[None, :, None])
    g = to_gpu(x)
    out = torch.empty((1, 4, 1, D), device="cuda", dtype=torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = bits_of(np.linspace(-2, 2, D))
    p = spa.make_rope_params(1, 4, 1, 1, table_rows=0, rotary_dim=0)
    spa.check(spa.sparse_qk_norm_rope(p, g, None, to_gpu(w), None, None, None, out, None, err))
    check_rows(to_f64(out), x, w, np.zeros((1, 4, 0)), 0, 0)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def run_append(b, *, rot=128, pairs=0, norm=True, queries=True, summary=True, rope=True, seed=0,
               table_rows=None):
    rng = np.random.default_rng(seed)
    rows = max([1] + b.kv) if table_rows is None else table_rows
    table = op.rope_table(rows, max(rot, 16))[:, :max(rot, 1)]
    wq = weight_bits(rng) if norm and rope else None
    wk = weight_bits(rng) if norm and rope else None
    p = b.params()
    r = spa.make_rope_params(1, b.T, b.hq, b.hkv, table_rows=rows, rotary_dim=rot,
                             interleaved=pairs) if rope else None
    sm = torch.full((b.num_pages, b.hkv, 2, D), SENTINEL, device="cuda", dtype=torch.bfloat16)
    qo = torch.full((b.T, b.hq, D), SENTINEL, device="cuda", dtype=torch.bfloat16)
    before = (b.kc.clone(), b.vc.clone())
    opt = lambda w: None if w is None else to_gpu(w)
    spa.check(spa.sparse_paged_append(
        p, r, b.q if queries else None, b.qkv_gpu[:, b.hq:b.hq + b.hkv],
        b.qkv_gpu[:, b.hq + b.hkv:], opt(wq), opt(wk),
        torch.from_numpy(np.ascontiguousarray(table)).cuda(), b.cu_gpu, b.kv_gpu, b.table_gpu,
        qo if queries else None, b.kc, b.vc, sm if summary else None, b.error))
    return dict(p=p, table=table, wq=wq, wk=wk, sm=sm, qo=qo, before=before, rot=rot if rope else 0,
                pairs=pairs, queries=queries, summary=summary)


def check_append(b, a, skip=()):
    kc, vc = b.kc.contiguous(), b.vc.contiguous()
    kh, k0 = to_f64(kc), to_f64(a["before"][0])
    vb, v0 = vc.view(torch.int16).cpu().numpy(), a["before"][1].contiguous().view(torch.int16).cpu().numpy()
    kb, kb0 = kc.view(torch.int16).cpu().numpy(), a["before"][0].contiguous().view(torch.int16).cpu().numpy()
    written = np.zeros((b.num_pages, b.page), bool)
    touched = {}
    qrows = np.zeros(b.T, bool)
    qo = to_f64(a["qo"])
    for t, s, pos in b.tokens():
        if s in skip:
            continue
        ph, r = b.table[s, pos // b.page], pos % b.page
        written[ph, r] = True
        touched[(s, pos // b.page)] = min(b.kv[s], (pos // b.page + 1) * b.page) - pos // b.page * b.page
        ang = a["table"][pos].astype(np.float64)
        check_rows(kh[ph, :, r], b.qkv[t, b.hq:b.hq + b.hkv], a["wk"], ang, a["rot"], a["pairs"])
        assert np.array_equal(vb[ph, :, r].view(np.uint16), b.qkv[t, b.hq + b.hkv:])
        qrows[t] = True
        if a["queries"]:
            check_rows(qo[t], b.qkv[t, :b.hq], a["wq"], ang, a["rot"], a["pairs"])
    assert np.array_equal(kb.transpose(0, 2, 1, 3)[~written], kb0.transpose(0, 2, 1, 3)[~written])
    assert np.array_equal(vb.transpose(0, 2, 1, 3)[~written], v0.transpose(0, 2, 1, 3)[~written])
    assert np.all(qo[~qrows] == SENTINEL)
    sm = to_f64(a["sm"])
    hit = np.zeros(b.num_pages, bool)
    if a["summary"]:
        for (s, j), rows in touched.items():
            ph = b.table[s, j]
            hit[ph] = True
            assert np.array_equal(sm[ph, :, 0], kh[ph, :, :rows].min(1))
            assert np.array_equal(sm[ph, :, 1], kh[ph, :, :rows].max(1))
    assert np.all(sm[~hit] == SENTINEL)


APPENDS = [(1, 1), (1, 16), (1, 17), (0, 40), (3, 3), (20, 30), (1, 200), (150, 333), (64, 128),
           (0, 0), (129, 129), (2, 66)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (5, 1)])
def test_append(hq, hkv, page):
    b = Batch(hq, hkv, page, APPENDS, seed=page, filled="old")
    check_append(b, run_append(b))
    b.ok()


@pytest.mark.parametrize("kw", [dict(rot=64), dict(pairs=1), dict(norm=False), dict(queries=False),
                                dict(summary=False), dict(rope=False), dict(rot=0),
                                dict(rot=32, pairs=1, norm=False, queries=False)])
def test_append_options(kw):
    b = Batch(6, 3, 32, APPENDS, seed=2, filled="old", joint=True, gap=2, lead_rows=2, pad_rows=3)
    check_append(b, run_append(b, **kw))
    b.ok()


@pytest.mark.parametrize("seqs", [[(1, 50)] * 70, [(1, 5 + i) for i in range(300)], [(2000, 2000)],
                                  [(0, 9)] * 5 + [(1, 9)] + [(0, 3)] * 4])
def test_append_batches(seqs):
    b = Batch(8, 2, 16, seqs, seed=3, filled="old")
    check_append(b, run_append(b))
    b.ok()


def test_append_is_repeatable_and_rewrites_after_a_step_back():
    # draft tokens that were rejected: the length goes back and other rows take their places
    b = Batch(4, 2, 16, [(5, 37)], seed=4, filled="old")
    a = run_append(b)
    first = (b.kc.clone(), a["sm"].clone())
    a = run_append(b)
    assert torch.equal(first[0].view(torch.int16), b.kc.view(torch.int16))
    assert torch.equal(first[1].view(torch.int16), a["sm"].view(torch.int16))
    b.n, b.kv = [2], [34]
    b.cu = np.array([0, 2], np.int32)
    b.cu_gpu, b.kv_gpu = torch.from_numpy(b.cu).cuda(), torch.tensor([34], dtype=torch.int32).cuda()
    b.qkv = b.qkv[::-1].copy()
    b.qkv_gpu = to_gpu(b.qkv)
    b.q = b.qkv_gpu[:, :b.hq]
    check_append(b, run_append(b, table_rows=40))
    b.ok()


def test_append_more_tokens_than_length_and_positions_past_the_table():
    b = Batch(4, 2, 16, [(1, 20), (5, 2), (1, 33)], seed=5, filled="old")
    a = run_append(b)
    check_append(b, a, skip=(1,))
    assert spa.sparse_paged_status(b.error) == spa.SPA_ERR_INVALID
    b = Batch(4, 2, 16, [(1, 20), (1, 41)], seed=5, filled="old")
    a = run_append(b, table_rows=40, summary=False)
    check_append(b, a, skip=(1,))
    assert spa.sparse_paged_status(b.error) == spa.SPA_ERR_INVALID
