"""A densely attended layer's cache at the ends of what its calls allow:
values that are infinite, NaN or huge, key weights past the largest number,
against the fp64 oracle (oracle/dense_cache.py); offsets on the device that
reach past what the host has named, behind guards; the longest sequence that a
description may name; and the choice by the groups' sum among weights whose sums are
denormal, past the largest number, NaN or next to nothing, in every launch form,
exactly."""
import numpy as np
import pytest
import torch

from oracle import dense_cache as C
import test_gpu_attn_weights as W
import test_gpu_evict as E
from test_gpu_dense_decode import SHAPES, _check, _f, _paged

pytestmark = pytest.mark.gpu

PAGE = 128


@pytest.fixture(scope="module")
def M():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from block_sparse_long_exp_b200 import build, msa
    build.build()
    msa.load_library()
    return msa


def _rows(table, b, n):
    j = torch.arange(n)
    return table[b].long()[j // PAGE] * PAGE + j % PAGE


def _decode(M, shape, lens, table, pages, q, k, v, w0=None):
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), max(lens), pages)
    w = None if w0 is None else w0.cuda()
    out, lse = M.msa_dense_attn_decode_paged(shape, pg, q.cuda(), k.cuda(), v.cuda(), weights=w)
    return out.cpu(), lse.cpu(), None if w is None else w.cpu()


# ------------------------------------------------------------------ values of the decode

@pytest.mark.parametrize("H,G,d", SHAPES)
@pytest.mark.parametrize("weights", [False, True])
def test_infinite_values_come_through(M, H, G, d, weights):
    # in group 0 alone: column 0 one +inf, 1 one -inf, 2 both signs (from two tokens on), 3 NaN, 9 +inf in every token,
    # d - 1 -inf in the middle; the other columns and groups stay what they are
    inf, lens = float("inf"), [1, 2, 17, 64, 129, 1000, 5003]
    k, v, table, pages, seqs = _paged(lens, G, d, 211)
    for b, n in enumerate(lens):
        x = seqs[b][1]
        x[0, 0, 0], x[n - 1, 0, 1], x[n // 3, 0, 3], x[n // 2, 0, d - 1] = inf, -inf, float("nan"), -inf
        x[0, 0, 2] = inf
        if n > 1:
            x[n - 1, 0, 2] = -inf
        x[:, 0, 9] = inf
        v[_rows(table, b, n)] = x
    q = (torch.randn(len(lens), H, d, generator=torch.Generator().manual_seed(212)) * 1.5).bfloat16()
    shape = M.make_shape(H, G, d, 64, 16)
    w0 = torch.rand(len(lens), G, table.shape[1] * PAGE, generator=torch.Generator().manual_seed(213)) if weights else None
    out, lse, w = _decode(M, shape, lens, table, pages, q, k, v, w0)
    for b, n in enumerate(lens):
        with np.errstate(invalid="ignore"):
            want, _, _, _ = C.decode_attention(_f(q[b]), _f(seqs[b][0]), _f(seqs[b][1]), shape.sm_scale)
        odd = ~np.isfinite(want)
        assert odd.any() and np.array_equal(odd[H // G:], np.zeros_like(odd[H // G:]))
        np.testing.assert_array_equal(_f(out[b])[odd], want[odd], err_msg=str(n))
    # and with zeros in their places every finite column, lse and weight is as near as ever
    cols = [0, 1, 2, 3, 9, d - 1]
    for b in range(len(lens)):
        seqs[b][1][:, 0, cols] = 0
        out[b, :H // G, cols] = 0
    _check(out, lse, w, q, seqs, shape.sm_scale, w0)


@pytest.mark.parametrize("H,G,d", [(8, 2, 64), (32, 2, 128)])
def test_values_of_heads_that_see_nothing_do_not_count(M, H, G, d):
    # every score of group 0 is -inf: zeros, though its values are infinite or NaN
    for n in (3, 200, 9000):
        k, v, table, pages, seqs = _paged([n], G, d, 221)
        at = _rows(table, 0, n)
        k[at, 0] = 0
        k[at, 0, 0] = float("-inf")
        v[at, 0, 1], v[at, 0, 5] = float("inf"), float("nan")
        q = torch.zeros(1, H, d).bfloat16()
        q[:, :, 0] = 1.0
        out, lse, _ = _decode(M, M.make_shape(H, G, d, 64, 16), [n], table, pages, q, k, v)
        assert torch.all(out[0, :H // G] == 0) and torch.all(lse[0, :H // G] == float("-inf"))
        assert torch.all(torch.isfinite(out[0, H // G:].float())) and torch.all(torch.isfinite(lse[0, H // G:]))


@pytest.mark.parametrize("H,G,d", [(8, 2, 64), (32, 2, 128)])
@pytest.mark.parametrize("n", [3, 17, 300, 9000])
def test_a_score_of_nan_leaves_nothing_but_nan(M, H, G, d, n):
    # a NaN or infinity among the keys of group 0, infinities among its values: every weight of the group is NaN
    for x in (float("nan"), float("inf")):
        k, v, table, pages, seqs = _paged([n, 5], G, d, 226)
        at = _rows(table, 0, n)
        k[at[n // 2], 0, 0] = x
        v[at, 0, 1], v[at[0], 0, 5] = float("inf"), float("-inf")
        q = (torch.rand(2, H, d, generator=torch.Generator().manual_seed(227)) + 0.5).bfloat16()
        shape = M.make_shape(H, G, d, 64, 16)
        w0 = torch.rand(2, G, table.shape[1] * PAGE)
        out, lse, w = _decode(M, shape, [n, 5], table, pages, q, k, v, w0)
        hg = H // G
        assert torch.all(torch.isnan(out[0, :hg].float())) and torch.all(torch.isnan(lse[0, :hg]))
        assert torch.all(torch.isnan(w[0, 0, :n])) and torch.equal(w[0, 0, n:], w0[0, 0, n:])
        _check(out[:, hg:2 * hg], lse[:, hg:2 * hg], w[:, 1:2], q[:, hg:2 * hg],
               [(a[:, 1:2].contiguous(), b[:, 1:2].contiguous()) for a, b in seqs], shape.sm_scale, w0[:, 1:2])


@pytest.mark.parametrize("H,G,d", [(8, 2, 64), (64, 4, 128), (16, 1, 64)])
def test_values_up_to_the_largest_allowed(M, H, G, d):
    # sizes from 2^80 to 2^88, of both signs
    lens = [1, 100, 4001]
    k, v, table, pages, seqs = _paged(lens, G, d, 231)
    gen = torch.Generator().manual_seed(233)
    for b, n in enumerate(lens):
        size = torch.exp2(80 + 8 * torch.rand(n, G, d, generator=gen))
        seqs[b][1].copy_((torch.sign(seqs[b][1].float()) * size).bfloat16())
        v[_rows(table, b, n)] = seqs[b][1]
    q = (torch.randn(len(lens), H, d, generator=torch.Generator().manual_seed(232)) * 1.5).bfloat16()
    shape = M.make_shape(H, G, d, 64, 16)
    out, lse, _ = _decode(M, shape, lens, table, pages, q, k, v)
    _check(out, lse, None, q, seqs, shape.sm_scale)


@pytest.mark.parametrize("scale", [2.0 ** -126, 2.3e38])
def test_scales_at_their_bounds(M, scale):
    # scores of 0: every key of a sequence weighs the same, whatever stands behind its end
    H, G, d, lens = 16, 2, 64, [1, 19, 300]
    k, v, table, pages, seqs = _paged(lens, G, d, 261)
    shape = M.make_shape(H, G, d, 64, 16, sm_scale=scale)
    w0 = torch.zeros(3, G, table.shape[1] * PAGE)
    q = torch.zeros(3, H, d).bfloat16()
    out, lse, w = _decode(M, shape, lens, table, pages, q, k, v, w0)
    _check(out, lse, w, q, seqs, scale, w0)
    kk = torch.cat([a for a, _ in seqs])
    ones = torch.log(torch.cat([torch.arange(1, n + 1) for n in lens]).float())[:, None].expand(-1, H).contiguous()
    got = M.msa_attn_weights(shape, W._varlen(M, lens, lens), torch.zeros(sum(lens), H, d).bfloat16().cuda(), kk.cuda(),
                             ones.cuda()).cpu()
    W._check(got, torch.zeros(sum(lens), H, d).bfloat16(), kk, ones, lens, lens, scale, torch.zeros(3, G, 300), 1.0)


# ------------------------------------------------------------------ key weights

@pytest.mark.parametrize("H,G,d", SHAPES)
@pytest.mark.parametrize("T", [40, 700, 3000])
def test_weights_past_the_largest_number_are_infinite(M, H, G, d, T):
    # scores of 0 and log-sum-exps of their own: query 5 gives 2^130, queries 20 .. 30 give 2^126 each, which
    # only together pass the largest number, the others 1; the keys up to the last of those queries get infinity
    shape = M.make_shape(H, G, d, 64, 16)
    q, k = torch.zeros(T, H, d).bfloat16(), torch.zeros(T, G, d).bfloat16()
    for heavy, last in (({5: 130.0}, 5), ({t: 126.0 for t in range(20, 31)}, 30), ({5: 130.0, T - 1: 130.0}, T - 1)):
        x = torch.zeros(T)
        for t, e in heavy.items():
            x[t] = e
        lse = (-x * np.log(2.0))[:, None].expand(T, H).contiguous()
        w = M.msa_attn_weights(shape, W._varlen(M, [T], [T]), q.cuda(), k.cuda(), lse.cuda(), decay=0.0).cpu()[0]
        want = (H // G) * torch.flip(torch.cumsum(torch.flip(torch.exp(-lse[:, 0].double()), [0]), 0), [0])
        inf = want > 2.0 ** 128 * 1.01
        assert bool((w[:, inf] == float("inf")).all()) and int(inf.sum()) >= 6
        # beyond `last` sums of ones: exact but for the exponential's 2^-22 (an argument of 0 has no error)
        rest = torch.arange(T) > last
        assert bool(((w[:, rest].double() - want[rest]).abs() <= want[rest] * 2.0 ** -21).all())


LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("cu_q,cu_k,bad", [
    ([0, 20, 70, 103], [0, 301, 430, 470], {0}),              # a key past the weights' width
    ([0, 20, 70, 103], [0, 300, 430, 471], {2}),              # past the keys
    ([0, 20, 70, 104], [0, 300, 430, 470], {2}),              # past the queries
    ([-1, 20, 70, 103], [0, 300, 430, 470], {0}), ([0, 20, 70, 103], [-1, 299, 430, 470], {0}),
    ([0, 20, 10, 103], [0, 300, 430, 470], {1, 2}),           # offsets that decrease; then more queries than keys
    ([0, 20, 70, 103], [0, 300, 200, 470], {1}), ([0, 20, 70, 103], [0, HIGH, 430, 470], {0, 1}),
    ([0, LOW, 70, 103], [0, 300, 430, 470], {0, 1}), ([0, HIGH, 70, 103], [0, 300, 430, 470], {0, 1}),
    ([0, 20, 70, HIGH], [0, 300, 430, HIGH], {2}), ([0, 20, 20, 103], [LOW, LOW, HIGH, 470], {0, 2}),
])
@pytest.mark.parametrize("captured", [False, True])
def test_key_weights_keep_to_what_the_host_has_named(M, cu_q, cu_k, bad, captured):
    # the device's offsets, changed after the description was made: a sequence that reaches past it is reported and left
    # alone, the others are done by the offsets that they have; guards on both sides of the weights
    T, S, G, guard = [20, 50, 33], [300, 130, 40], 2, 8192
    q, k = W._inputs(8, G, 64, T, S, 241)
    shape = M.make_shape(8, G, 64, 64, 16)
    lse = W._lse(q, k, T, S, shape.sm_scale) + 3.0
    seqs = W._varlen(M, T, S)
    around = torch.full((2 * guard + 3 * G * 300,), 7.0, device="cuda")
    w = around[guard:-guard].view(3, G, 300)
    w0 = torch.rand(3, G, 300, generator=torch.Generator().manual_seed(242))
    ws = torch.empty(M.msa_attn_weights_workspace_size(shape, seqs), dtype=torch.uint8, device="cuda")
    qd, kd, ld = q.cuda(), k.cuda(), lse.cuda()
    call = lambda check: M.msa_attn_weights(shape, seqs, qd, kd, ld, weights=w, decay=0.5, ws=ws, check=check)  # noqa: E731
    if captured:
        call(True)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(False)
    w.copy_(w0)
    seqs._keep[0].copy_(torch.tensor(cu_q, dtype=torch.int32))
    seqs._keep[1].copy_(torch.tensor(cu_k, dtype=torch.int32))
    if captured:
        graph.replay()
        with pytest.raises(M.MsaError, match="DEVICE_CHECK at site 251"):
            M._device_check(ws, None, "key weights")
    else:
        with pytest.raises(M.MsaError, match="DEVICE_CHECK at site 251"):
            call(True)
    got = w.cpu()
    for b in range(3):
        if b in bad or cu_q[b + 1] == cu_q[b]:
            assert torch.equal(got[b], w0[b]), b
            continue
        at, keys = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        W._check(got[b:b + 1], q[at], k[keys], lse[at], [cu_q[b + 1] - cu_q[b]], [cu_k[b + 1] - cu_k[b]], shape.sm_scale,
                 w0[b:b + 1], 0.5)
    assert bool((around[:guard] == 7.0).all()) and bool((around[-guard:] == 7.0).all())


# ------------------------------------------------------------------ the longest description

LONGEST = 16777213 * PAGE                                     # 2^31 - 384


def test_decode_under_the_longest_description(M):
    # a short cache whose description names the most that a call takes: 34 GB of scores, 8.6 GB of weights
    H, G, d, n = 4, 1, 64, 300
    k, v, table, pages, seqs = _paged([n], G, d, 251, extra_blocks=0)
    wide = torch.full((1, LONGEST // PAGE), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    q = torch.randn(1, H, d, generator=torch.Generator().manual_seed(252)).bfloat16()
    shape = M.make_shape(H, G, d, 64, 16)
    pg = M.make_paged(torch.tensor([n], dtype=torch.int32).cuda(), wide.cuda(), LONGEST, pages)
    w = torch.empty(1, G, LONGEST, device="cuda")
    w[:, :, n:n + 100] = 5.0
    w[:, :, -100:] = 5.0
    out, lse = M.msa_dense_attn_decode_paged(shape, pg, q.cuda(), k.cuda(), v.cuda(), weights=w, decay=0.0)
    head = w[:, :, :n].cpu()
    _check(out.cpu(), lse.cpu(), head, q, seqs, shape.sm_scale, torch.zeros(1, G, n))
    assert bool((w[:, :, n:n + 100] == 5.0).all()) and bool((w[:, :, -100:] == 5.0).all())
    del w
    torch.cuda.empty_cache()


def test_choice_under_the_longest_description(M):
    n, budget = 9000, 700
    shape = M.make_shape(4, 1, 64, 64, 16)
    table = torch.zeros(1, LONGEST // PAGE, dtype=torch.int32)
    pg = M.make_paged(torch.tensor([n], dtype=torch.int32).cuda(), table.cuda(), LONGEST, 1)
    w = torch.empty(1, 1, LONGEST, device="cuda")
    head = torch.rand(1, 1, n, generator=torch.Generator().manual_seed(253))
    w[:, :, :n] = head.cuda()
    w[:, :, n:n + 5000] = 9.0                                 # past the end: no candidates
    kept, new = M.msa_evict_select(shape, pg, w, budget, 3, 40)
    np.testing.assert_array_equal(kept[0].cpu().numpy(), C.evict_select(head[0].numpy(), budget, 3, 40, False))
    assert new.item() == budget
    del w
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ sums of the groups' weights

def _group_weights(B, G, blocks, kind, seed):
    g = torch.Generator().manual_seed(seed)
    shape = (B, G, blocks * PAGE)
    if kind in ("odd", "denormal"):
        return E._weights(B, G, blocks, seed, kind)
    if kind == "huge":                                        # sums past the largest number, of both signs, and just below it
        w = 3.4e38 * (0.02 + 0.98 * torch.rand(shape, generator=g))
        return torch.where(torch.rand(shape, generator=g) < 0.3, -w, w)
    if kind == "edge":                                        # sums that round to the largest number or to infinity, by a bit
        top = np.array(0x7f7fffff, np.int32).view(np.float32)
        w = torch.randint(0, 4, shape, generator=g).float() * 2.0 ** 103      # halves of the last place of the largest
        w[:, 0] = torch.where(torch.rand(shape[0], shape[2], generator=g) < 0.8, torch.tensor(top), w[:, 0])
        return w
    if kind == "halves":                                      # sums half way between two numbers: to the even one
        w = torch.randint(0, 5, shape, generator=g).float() * 0.5
        w[:, 0] = torch.randint(2 ** 24 - 3, 2 ** 24 + 3, (shape[0], shape[2]), generator=g).float()
        w[:, 0] *= torch.where(torch.rand(shape[0], shape[2], generator=g) < 0.2, -1.0, 1.0)
        return w
    assert kind == "cancel"                                   # sums far below their terms, denormal ones and zeros among them
    w = torch.exp2(torch.randint(-149, 128, shape, generator=g).double()).float() * (1 + torch.rand(shape, generator=g)).clamp(max=1.99)
    w[:, 1] = -w[:, 0] * (1 + 2.0 ** -23 * torch.randint(-2, 3, (shape[0], shape[2]), generator=g).float())
    if G > 2:
        w[:, 2:] *= (torch.rand(B, 1, shape[2], generator=g) < 0.3)
    return w


@pytest.mark.parametrize("G", [2, 4])
@pytest.mark.parametrize("kind", ["odd", "denormal", "huge", "edge", "halves", "cancel"])
@pytest.mark.parametrize("L,B", [(1000, 1), (4096, 2), (8000, 1), (20000, 1), (66000, 1), (9000, 49)])
def test_choice_by_the_sum_of_odd_weights(M, G, kind, L, B):
    # four or eight tokens a thread, a cluster, a CTA per part (long, and many rankings)
    lens = [L - 37 * b for b in range(B)]
    w = _group_weights(B, G, -(-L // PAGE), kind, 271 + G)
    score = w.double().sum(1).float()
    # budgets that end among infinities, in the middle, among NaN or the smallest ones
    for budget, sink, recent in ((L // 10, 0, 0), (L // 2, 5, 33), (L - L // 20, 0, 7)) if B == 1 else ((L // 3, 3, 9),):
        if B <= 2:
            with np.errstate(over="ignore", invalid="ignore"):
                E._select(M, w, lens, budget, sink, recent, False)
            continue
        kept, new = M.msa_evict_select(M.make_shape(4 * G, G, 64, 64, 16), E._pages(M, lens, blocks=w.shape[2] // PAGE),
                                       w.cuda(), budget, sink, recent)
        assert new.cpu().tolist() == [min(n, budget) for n in lens]
        for b, n in enumerate(lens):
            s = score[b, :n].numpy()
            # descending, NaN last, ties (zeros of both signs among them) to the lower position
            order = np.lexsort((np.arange(n), np.where(np.isnan(s), 0.0, -s.astype(np.float64)), np.isnan(s)))
            middle = order[(order >= sink) & (order < n - recent)][:budget - sink - recent]
            want = np.sort(np.concatenate([np.arange(sink), middle, np.arange(n - recent, n)]))
            np.testing.assert_array_equal(kept[b, 0].cpu().numpy()[:min(n, budget)], want if n > budget else np.arange(n))
