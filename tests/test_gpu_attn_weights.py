"""The attention weight that a prompt's queries give every key
(msa_attn_weights) against the formula in 64 bits: head shapes, lengths around
the kernel's blocks and tiles, windows of one query and more, sequences without
queries, junk outside the sequences, decay, wide rows, captured and side-stream
calls, offsets past 32 bits; and a prompt, decode steps and an eviction in a row.

Tolerances.  A score is a sum of d exact products in 32 bits, d / 16 steps of
the tensor cores, each off by at most 2^-22 of the sum of the terms' sizes, so
its error is at most D = sm_scale (d / 16 + 1) 2^-22 max sum_i |q_i k_ji|; the
scaled score, the log-sum-exp in units of log2 and their difference (at most X =
max |s| + |lse| in size) round by 4 X 2^-24 more.  An exponential is then off by
2 (D + 4 X 2^-24) + 2^-22 of its size.  A sum takes at most 32 additions in a
row, then compensated ones, then at most 147 of parts: below 180 x 2^-24 <
2^-16 of its size, the exponential's 2^-22 included."""
import numpy as np
import pytest
import torch

from oracle import dense_cache as C

pytestmark = pytest.mark.gpu

PAGE = 128


@pytest.fixture(scope="module")
def M():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from block_sparse_long_exp_b200 import build, msa
    build.build()
    msa.load_library()
    return msa


def _cu(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def _varlen(M, T, S):
    return M.make_varlen(torch.tensor(_cu(T), dtype=torch.int32).cuda(), torch.tensor(_cu(S), dtype=torch.int32).cuda(),
                         _cu(T), _cu(S))


def _inputs(H, G, d, T, S, seed, qscale=1.5):
    gen = torch.Generator().manual_seed(seed)
    q = (torch.randn(sum(T), H, d, generator=gen) * qscale).bfloat16()
    k = torch.randn(sum(S), G, d, generator=gen).bfloat16()
    return q, k


def _scores(q, k, scale):
    """[H, T, S] in 64 bits, -inf where the key is not seen; and the largest sum of the terms' sizes."""
    H, G, t, n = q.shape[1], k.shape[1], q.shape[0], k.shape[0]
    kk = k.double().repeat_interleave(H // G, 1).permute(1, 2, 0)
    x = torch.matmul(q.double().transpose(0, 1), kk) * scale
    terms = float(torch.matmul(q.double().abs().transpose(0, 1), kk.abs()).max()) if t else 0.0
    seen = torch.arange(n)[None, :] <= torch.arange(n - t, n)[:, None]
    return x.masked_fill(~seen, float("-inf")), terms


def _lse(q, k, T, S, scale):
    rows = []
    for b in range(len(T)):
        x, _ = _scores(q[_cu(T)[b]:_cu(T)[b + 1]], k[_cu(S)[b]:_cu(S)[b + 1]], scale)
        rows.append(torch.logsumexp(x, -1).transpose(0, 1).float())
    return torch.cat(rows).contiguous()


def _check(w, q, k, lse, T, S, scale, w0, decay):
    G = k.shape[1]
    for b in range(len(T)):
        t, n = T[b], S[b]
        if t == 0:
            assert torch.equal(w[b], w0[b])
            continue
        qs, ls = q[_cu(T)[b]:_cu(T)[b + 1]], lse[_cu(T)[b]:_cu(T)[b + 1]]
        x, terms = _scores(qs, k[_cu(S)[b]:_cu(S)[b + 1]], scale)
        p = torch.exp(x - ls.double().transpose(0, 1)[..., None])
        p = torch.where(torch.isneginf(ls).transpose(0, 1)[..., None], torch.zeros_like(p), p)
        want = p.sum(1).view(G, -1, n).sum(1)
        X = scale * terms + float(ls[torch.isfinite(ls)].abs().max())
        E = 2 * (scale * (q.shape[2] / 16 + 1) * 2.0 ** -22 * terms + 4 * X * 2.0 ** -24) + 2.0 ** -16
        old = decay * w0[b, :, :n].double()
        err = (w[b, :, :n].double() - (old + want)).abs()
        assert bool((err <= E * want + 2.0 ** -22 * (old.abs() + want)).all()), (b, t, n, float((err / want).max()), E)
        assert torch.equal(w[b, :, n:], w0[b, :, n:])


def _case(M, H, G, d, T, S, seed, decay=1.0, extra=5, qscale=1.5):
    q, k = _inputs(H, G, d, T, S, seed, qscale)
    shape = M.make_shape(H, G, d, 64, 16)
    lse = _lse(q, k, T, S, shape.sm_scale)
    w0 = torch.rand(len(T), G, max(S) + extra, generator=torch.Generator().manual_seed(seed + 1))
    w = w0.cuda()
    got = M.msa_attn_weights(shape, _varlen(M, T, S), q.cuda(), k.cuda(), lse.cuda(), weights=w, decay=decay)
    assert got is w
    _check(w.cpu(), q, k, lse, T, S, shape.sm_scale, w0, decay)


SHAPES = [(8, 2, 64), (64, 4, 128), (16, 1, 128), (4, 1, 64), (16, 4, 128), (32, 4, 64), (32, 2, 128), (8, 1, 128)]


@pytest.mark.parametrize("H,G,d", SHAPES)
def test_prompts_around_the_borders(M, H, G, d):
    S = [1, 2, 7, 8, 9, 31, 32, 33, 127, 128, 129, 255, 256, 257, 300]
    _case(M, H, G, d, S, S, 11, 0.75)


@pytest.mark.parametrize("H,G,d", SHAPES)
def test_windows(M, H, G, d):
    S = [1, 300, 129, 256, 257, 512, 513, 1000, 64, 1025]
    T = [1, 1, 0, 64, 63, 33, 8, 9, 64, 500]
    _case(M, H, G, d, T, S, 21, 0.5)


@pytest.mark.parametrize("H,G,d", [(64, 4, 128), (8, 2, 64), (16, 4, 64)])
@pytest.mark.parametrize("T,S", [(1, 1), (1, 5003), (64, 9001), (1000, 1000), (300, 2222)])
def test_one_sequence_over_many_ctas(M, H, G, d, T, S):
    _case(M, H, G, d, [T], [S], 31, 0.0)


def test_many_short_sequences(M):
    S = [(i * 37) % 150 for i in range(900)]
    T = [(n * 7) % (n + 1) if n else 0 for n in S]
    _case(M, 8, 2, 64, T, S, 41, 1.0)


def test_one_long_among_short(M):
    _case(M, 16, 2, 128, [3, 700, 1, 0, 70], [3, 4001, 1, 0, 70], 51, 0.25)


def test_no_queries_at_all(M):
    q, k = _inputs(8, 2, 64, [0, 0], [5, 7], 61)
    w0 = torch.rand(2, 2, 9)
    w = w0.cuda()
    M.msa_attn_weights(M.make_shape(8, 2, 64, 64, 16), _varlen(M, [0, 0], [5, 7]), q.cuda(), k.cuda(),
                       torch.zeros(0, 8).cuda(), weights=w, decay=0.5)
    assert torch.equal(w.cpu(), w0)


def test_default_weights_start_from_zero(M):
    T, S = [4, 6], [9, 6]
    q, k = _inputs(8, 2, 64, T, S, 71)
    shape = M.make_shape(8, 2, 64, 64, 16)
    lse = _lse(q, k, T, S, shape.sm_scale)
    w = M.msa_attn_weights(shape, _varlen(M, T, S), q.cuda(), k.cuda(), lse.cuda())
    assert w.shape == (2, 2, 9)
    _check(w.cpu(), q, k, lse, T, S, shape.sm_scale, torch.zeros(2, 2, 9), 1.0)


def test_peaked_scores_and_heads_that_see_nothing(M):
    _case(M, 16, 2, 128, [300, 64], [300, 1000], 81, 1.0, qscale=30.0)
    # group 0's keys score -inf for every query: lse -inf, weight 0
    H, G, d, n = 8, 2, 64, 200
    k = torch.randn(n, G, d, generator=torch.Generator().manual_seed(3))
    k[:, 0] = 0
    k[:, 0, 0] = float("-inf")
    q = torch.zeros(50, H, d)
    q[:, :, 0] = 1.0
    q, k = q.bfloat16(), k.bfloat16()
    shape = M.make_shape(H, G, d, 64, 16)
    lse = torch.full((50, H), float("-inf"))
    lse[:, 4:] = _lse(q[:, 4:].contiguous(), k[:, 1:].contiguous(), [50], [n], shape.sm_scale)
    w = M.msa_attn_weights(shape, _varlen(M, [50], [n]), q.cuda(), k.cuda(), lse.cuda()).cpu()
    assert torch.all(w[0, 0] == 0)
    _check(w[:, 1:], q[:, 4:], k[:, 1:], lse[:, 4:], [50], [n], shape.sm_scale, torch.zeros(1, 1, n), 1.0)
    # a finite score of a head that has seen nothing adds nothing either
    q, k = _inputs(H, G, d, [50], [n], 82)
    lse = _lse(q, k, [50], [n], shape.sm_scale)
    lse[7:20, 2] = float("-inf")
    w = M.msa_attn_weights(shape, _varlen(M, [50], [n]), q.cuda(), k.cuda(), lse.cuda()).cpu()
    _check(w, q, k, lse, [50], [n], shape.sm_scale, torch.zeros(1, G, n), 1.0)


def test_a_neighbour_full_of_nan_does_not_reach_over(M):
    T, S = [20, 130, 33], [300, 130, 40]
    H, G, d = 16, 2, 64
    q, k = _inputs(H, G, d, T, S, 91)
    shape = M.make_shape(H, G, d, 64, 16)
    lse = _lse(q, k, T, S, shape.sm_scale)
    w0 = torch.zeros(3, G, 300)
    clean = M.msa_attn_weights(shape, _varlen(M, T, S), q.cuda(), k.cuda(), lse.cuda()).cpu()
    _check(clean, q, k, lse, T, S, shape.sm_scale, w0, 1.0)
    q[20:150], k[300:430], lse[20:150] = float("nan"), float("inf"), float("nan")
    w = M.msa_attn_weights(shape, _varlen(M, T, S), q.cuda(), k.cuda(), lse.cuda()).cpu()
    assert torch.equal(w[0], clean[0]) and torch.equal(w[2], clean[2])
    # later keys that a query does not see may hold anything: all but the last query's own
    q, k = _inputs(H, G, d, [40], [40], 92)
    lse = _lse(q, k, [40], [40], shape.sm_scale)
    lse[30:] = float("inf")                                     # those queries give nothing
    a = M.msa_attn_weights(shape, _varlen(M, [40], [40]), q.cuda(), k.cuda(), lse.cuda()).cpu()
    k[35:] = float("nan")
    b = M.msa_attn_weights(shape, _varlen(M, [40], [40]), q.cuda(), k.cuda(), lse.cuda()).cpu()
    assert torch.equal(a[:, :, :35], b[:, :, :35]) and bool((a[:, :, 30:] == 0).all())


def test_more_queries_than_keys_is_reported(M):
    T, S = [20, 50, 33], [300, 130, 40]
    q, k = _inputs(8, 2, 64, T, S, 101)
    shape = M.make_shape(8, 2, 64, 64, 16)
    lse = _lse(q, k, T, S, shape.sm_scale)
    seqs = _varlen(M, T, S)
    seqs._keep[1].copy_(torch.tensor([0, 300, 320, 470], dtype=torch.int32))      # 50 queries, 20 keys
    w0 = torch.rand(3, 2, 300)
    w = w0.cuda()
    with pytest.raises(M.MsaError, match="DEVICE_CHECK at site 251"):
        M.msa_attn_weights(shape, seqs, q.cuda(), k.cuda(), lse.cuda(), weights=w)
    assert torch.equal(w[1].cpu(), w0[1]) and not torch.equal(w[0].cpu(), w0[0])


def test_same_from_run_to_run_on_side_streams_and_captured(M):
    T, S = [700, 64, 300], [700, 1500, 300]
    H, G, d = 32, 4, 64
    q, k = _inputs(H, G, d, T, S, 111)
    shape = M.make_shape(H, G, d, 64, 16)
    lse = _lse(q, k, T, S, shape.sm_scale)
    seqs = _varlen(M, T, S)
    qd, kd, ld = q.cuda(), k.cuda(), lse.cuda()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [M.msa_attn_weights(shape, seqs, qd, kd, ld, stream=s, check=False) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(x, got[0]) for x in got)
    _check(got[0].cpu(), q, k, lse, T, S, shape.sm_scale, torch.zeros(3, G, 1500), 1.0)

    w = torch.zeros(3, G, 1500, device="cuda")
    ws = torch.empty(M.msa_attn_weights_workspace_size(shape, seqs), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.msa_attn_weights(shape, seqs, qd, kd, ld, weights=w, decay=0.5, ws=ws, check=False)
    for seed in (112, 113):
        q, k = _inputs(H, G, d, T, S, seed)
        lse = _lse(q, k, T, S, shape.sm_scale)
        qd.copy_(q), kd.copy_(k), ld.copy_(lse)
        w0 = w.cpu()
        graph.replay()
        torch.cuda.synchronize()
        _check(w.cpu(), q, k, lse, T, S, shape.sm_scale, w0, 0.5)


def test_from_the_dense_attention_of_the_prompt(M):
    # every query's weights sum to one: a group's weights sum to its number of (query, head) pairs
    T = S = [513, 70]
    H, G, d = 16, 2, 128
    q, k = _inputs(H, G, d, T, S, 121)
    v = torch.randn(sum(S), G, d).bfloat16()
    shape = M.make_shape(H, G, d, 64, 16)
    seqs = _varlen(M, T, S)
    _, lse = M.msa_dense_attn(shape, seqs, q.cuda(), k.cuda(), v.cuda(), want_lse=True)
    w = M.msa_attn_weights(shape, seqs, q.cuda(), k.cuda(), lse).cpu().double()
    for b in range(2):
        assert torch.allclose(w[b].sum(-1), torch.full((G,), 8.0 * T[b], dtype=torch.float64), rtol=1e-3, atol=0)


def test_offsets_past_32_bits(M):
    # query rows past 2^31 elements, weight rows past 2^31 entries
    H, G, d = 16, 1, 128
    shape = M.make_shape(H, G, d, 64, 16)
    pad = 1100000                                              # queries of a first sequence: 2.25e9 elements of q
    T = [pad, 40]
    S = [pad, 300]
    seqs = _varlen(M, T, S)
    q = torch.empty(sum(T), H, d, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(sum(S), G, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(sum(T), H, device="cuda")
    tail_q, tail_k = _inputs(H, G, d, [40], [300], 131)
    tail_l = _lse(tail_q, tail_k, [40], [300], shape.sm_scale)
    q[pad:], k[pad:], lse[pad:] = tail_q.cuda(), tail_k.cuda(), tail_l.cuda()
    # on the device the first sequence has no queries (a call's offsets need not start at 0 there): no work for it
    seqs._keep[0].copy_(torch.tensor([pad, pad, pad + 40], dtype=torch.int32))
    wide = 2 ** 31 + 8
    w = torch.empty(2, G, wide, device="cuda")
    M.msa_attn_weights(shape, seqs, q, k, lse, weights=w, decay=0.0)
    _check(w[1:, :, :300].cpu(), tail_q, tail_k, tail_l, [40], [300], shape.sm_scale, torch.zeros(1, G, 300), 0.0)


@pytest.mark.parametrize("per_group", [False, True])
def test_prompt_decode_and_eviction_in_a_row(M, per_group):
    """A prompt's attention and weights, decode steps that go on from them, a cut
    to the budget and a step on the cut cache: as a serving loop runs them."""
    H, G, d, budget = 16, 2, 64, 100
    S, steps = [200, 90, 131], 3
    shape = M.make_shape(H, G, d, 64, 16)
    gen = torch.Generator().manual_seed(141)
    seqs = _varlen(M, S, S)
    q, k = _inputs(H, G, d, S, S, 142)
    v = torch.randn(sum(S), G, d, generator=gen).bfloat16()
    blocks, pages = 2, 9
    table = torch.tensor([[4, 0], [2, 7], [6, 1]], dtype=torch.int32)
    kp = torch.full((pages * PAGE, G, d), float("nan")).bfloat16().cuda()
    vp = kp.clone()
    hist_k, hist_v = [], []
    for b, n in enumerate(S):
        hist_k.append(k[_cu(S)[b]:_cu(S)[b + 1]])
        hist_v.append(v[_cu(S)[b]:_cu(S)[b + 1]])
        for j in range(n):
            row = int(table[b, j // PAGE]) * PAGE + j % PAGE
            kp[row], vp[row] = hist_k[b][j].cuda(), hist_v[b][j].cuda()
    _, lse = M.msa_dense_attn(shape, seqs, q.cuda(), k.cuda(), v.cuda(), want_lse=True)
    w = torch.zeros(3, G, blocks * PAGE, device="cuda")
    M.msa_attn_weights(shape, seqs, q.cuda(), k.cuda(), lse, weights=w, decay=0.0)
    want = [torch.from_numpy(C.key_weights(q[_cu(S)[b]:_cu(S)[b + 1]].double().numpy(), hist_k[b].double().numpy(),
                                           _lse(q, k, S, S, shape.sm_scale)[_cu(S)[b]:_cu(S)[b + 1]].numpy(),
                                           shape.sm_scale)) for b in range(3)]
    lens = list(S)
    decay = 0.9
    for _ in range(steps):
        qn = (torch.randn(3, H, d, generator=gen) * 1.5).bfloat16()
        for b in range(3):
            kn, vn = torch.randn(1, G, d, generator=gen).bfloat16(), torch.randn(1, G, d, generator=gen).bfloat16()
            row = int(table[b, lens[b] // PAGE]) * PAGE + lens[b] % PAGE
            kp[row], vp[row] = kn[0].cuda(), vn[0].cuda()
            hist_k[b], hist_v[b] = torch.cat([hist_k[b], kn]), torch.cat([hist_v[b], vn])
            lens[b] += 1
        pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), max(lens), pages)
        out, _ = M.msa_dense_attn_decode_paged(shape, pg, qn.cuda(), kp, vp, weights=w, decay=decay)
        for b in range(3):
            o, _, ww, mass = C.decode_attention(qn[b].double().numpy(), hist_k[b].double().numpy(),
                                                hist_v[b].double().numpy(), shape.sm_scale)
            want[b] = torch.cat([want[b], torch.zeros(G, 1)], 1) * decay + torch.from_numpy(ww)
            assert np.all(np.abs(out[b].double().cpu().numpy() - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -12 * mass)
    for b in range(3):
        # scores of size 10 here: D + 4 X 2^-24 is below 2^-15, some ten roundings of the sums and of lse with it
        assert torch.allclose(w[b, :, :lens[b]].double().cpu(), want[b], rtol=2.0 ** -11, atol=0)
    kept, new_lens = M.msa_evict_select(shape, pg, w, budget, 4, 16, per_group=per_group)
    new_table = torch.tensor([[3], [5], [8]], dtype=torch.int32)
    npg = M.make_paged(new_lens, new_table.cuda(), budget, pages)
    w2 = M.msa_evict_move(shape, pg, npg, kept, kp, vp, weights=w)
    nl = new_lens.cpu().tolist()
    assert nl == [100, 93, 100]
    kc = kept.cpu()
    qn = (torch.randn(3, H, d, generator=gen) * 1.5).bfloat16()
    before = w2.cpu().double()
    out, _ = M.msa_dense_attn_decode_paged(shape, npg, qn.cuda(), kp, vp, weights=w2, decay=decay)
    for b in range(3):
        chosen = C.evict_select(w[b, :, :lens[b]].cpu().numpy(), budget, 4, 16, per_group)
        cut_k, cut_v = torch.empty(nl[b], G, d).bfloat16(), torch.empty(nl[b], G, d).bfloat16()
        for g in range(G):
            row = kc[b, g if per_group else 0, :nl[b]].long()
            np.testing.assert_array_equal(row.numpy(), chosen[g if per_group else 0])
            cut_k[:, g], cut_v[:, g] = hist_k[b][row, g], hist_v[b][row, g]
            assert torch.equal(before[b, g, :nl[b]], w[b, g].cpu().double()[row])
        o, _, ww, mass = C.decode_attention(qn[b].double().numpy(), cut_k.double().numpy(), cut_v.double().numpy(),
                                            shape.sm_scale)
        assert np.all(np.abs(out[b].double().cpu().numpy() - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -12 * mass)
        assert torch.allclose(w2[b, :, :nl[b]].double().cpu(), before[b, :, :nl[b]] * decay + torch.from_numpy(ww),
                              rtol=2.0 ** -11, atol=0)


def test_workspace_with_anything_in_it_and_other_scales(M):
    T, S = [300, 0, 64], [300, 9, 900]
    H, G, d = 16, 2, 128
    q, k = _inputs(H, G, d, T, S, 151)
    seqs = _varlen(M, T, S)
    for scale in (1e-3, 0.7):
        shape = M.make_shape(H, G, d, 64, 16, sm_scale=scale)
        lse = _lse(q, k, T, S, scale)
        ws = torch.full((M.msa_attn_weights_workspace_size(shape, seqs),), 255, dtype=torch.uint8, device="cuda")
        w0 = torch.rand(3, G, 900)
        w = w0.cuda()
        M.msa_attn_weights(shape, seqs, q.cuda(), k.cuda(), lse.cuda(), weights=w, decay=0.3, ws=ws)
        _check(w.cpu(), q, k, lse, T, S, scale, w0, 0.3)


def test_exponentials_far_from_zero(M):
    # one score per query and a log-sum-exp of its own: exp(s - lse) from 2^-140 (0 in 32 bits) to 2^120
    H, G, d, T = 4, 1, 64, 400
    shape = M.make_shape(H, G, d, 64, 16)
    q, k = torch.zeros(T, H, d).bfloat16(), torch.zeros(T, G, d).bfloat16()
    x = torch.linspace(-140, 120, T)
    lse = (-x * np.log(2.0))[:, None].expand(T, H).contiguous()
    w = M.msa_attn_weights(shape, _varlen(M, [T], [T]), q.cuda(), k.cuda(), lse.cuda()).cpu().double()[0, 0]
    terms = H * torch.exp(-lse[:, 0].double())
    want = torch.flip(torch.cumsum(torch.flip(terms, [0]), 0), [0])          # key j is seen by the queries from j on
    # arguments of up to 140: two roundings and the difference are off by 140 x 3 x 2^-24 of the exponent, 2^-16 for the rest
    assert bool(((w - want).abs() <= want * (np.log(2.0) * 140 * 3 * 2.0 ** -24 + 2.0 ** -16)).all())
    # a query alone, from each end of the range: tiny results flush to 0, none comes out wrong
    for e in (-149.0, -130.0, -127.5, -127.0, -126.5, -126.0, -1.0, 0.0, 1.0, 100.0, 126.0):
        one = M.msa_attn_weights(shape, _varlen(M, [1], [1]), q[:1].cuda(), k[:1].cuda(),
                                 torch.full((1, H), float(-e * np.log(2.0)), dtype=torch.float32).cuda()).item()
        exact = H * 2.0 ** e
        if exact >= 2.0 ** 128:                                   # 4 x 2^126 is past the largest 32-bit number, 2^128 - 2^104
            assert one == float("inf")
            continue
        assert abs(one - exact) <= exact * 2.0 ** -14 + H * 2.0 ** -126, (e, one)
