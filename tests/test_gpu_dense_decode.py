"""Dense attention of one new token per sequence over a paged cache
(msa_dense_attn_decode_paged) against the fp64 oracle (oracle/dense_cache.py):
shapes, lengths around the tile and page borders, ragged and empty rows, junk
past a sequence's end, accumulated weights, bad pages and lengths, captured
and side-stream calls, offsets past 32 bits.

Tolerances.  A score is a sum of d exact products in 32 bits, d / 16 steps of
the tensor cores, each off by at most 2^-22 of the sum of the terms' sizes
(products aligned to the largest, then the accumulator's own rounding), so its
error is at most D = sm_scale (d / 16 + 1) 2^-22 max_j sum_i |q_i k_ji|, and the
scaled score and exponent (at most X = max |s| + |lse| in size) round by 4 X
2^-24 more.  A weight is then off by E = 2 (D + 4 X 2^-24) + 2^-16 of its size
(its own error, the sum's, and 2^-17 for its two bf16 terms with room for the
exponential's 2^-22 and the sums), out by 2^-8 |out| (its rounding to bf16) +
E sum_j p_j |v_j|, lse by E + 2^-22 |lse|, an accumulated weight by E + 2^-22 of
the sum of the parts' sizes."""
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


def _paged(lens, G, d, seed, spare=3, extra_blocks=1, junk=float("nan")):
    """K / V pages in a random order, rows outside the tokens full of junk."""
    gen = torch.Generator().manual_seed(seed)
    nblk = [-(-n // PAGE) for n in lens]
    pages = sum(nblk) + spare
    perm = torch.randperm(pages, generator=gen).tolist()
    k = torch.full((pages * PAGE, G, d), junk).bfloat16()
    v = torch.full((pages * PAGE, G, d), junk).bfloat16()
    table = torch.full((len(lens), max(max(nblk), 1) + extra_blocks), -1, dtype=torch.int32)
    seqs, i = [], 0
    for b, n in enumerate(lens):
        kb, vb = (torch.randn(n, G, d, generator=gen).bfloat16() for _ in range(2))
        seqs.append((kb, vb))
        for j in range(nblk[b]):
            table[b, j] = perm[i]
            rows = slice(perm[i] * PAGE, perm[i] * PAGE + min(PAGE, n - j * PAGE))
            k[rows], v[rows] = kb[j * PAGE:(j + 1) * PAGE], vb[j * PAGE:(j + 1) * PAGE]
            i += 1
    return k, v, table, pages, seqs


def _f(x):
    return x.double().cpu().numpy()


def _check(out, lse, w, q, seqs, scale, w0=None, decay=1.0, only=None):
    for b, (k, v) in enumerate(seqs):
        if only is not None and b not in only:
            continue
        n = k.shape[0]
        H, d = q.shape[1:]
        G = k.shape[1]
        if n == 0:
            assert torch.all(out[b] == 0) and torch.all(lse[b] == float("-inf"))
            if w is not None:
                assert torch.equal(w[b], w0[b])
            continue
        o_ref, l_ref, w_ref, mass = C.decode_attention(_f(q[b]), _f(k), _f(v), scale)
        hg = H // G
        terms = max(float((np.abs(_f(k[:, g])) @ np.abs(_f(q[b, g * hg:(g + 1) * hg])).T).max()) for g in range(G))
        D = scale * (d / 16 + 1) * 2.0 ** -22 * terms
        X = scale * terms + np.abs(l_ref).max()
        E = 2 * (D + 4 * X * 2.0 ** -24) + 2.0 ** -16
        got = _f(out[b])
        assert np.all(np.abs(got - o_ref) <= 2.0 ** -8 * np.abs(o_ref) + E * mass), (b, n, np.abs(got - o_ref).max())
        assert np.all(np.abs(_f(lse[b]) - l_ref) <= E + 2.0 ** -22 * np.abs(l_ref)), (b, n)
        if w is not None:
            old = decay * _f(w0[b, :, :n])
            want = old + w_ref
            assert np.all(np.abs(_f(w[b, :, :n]) - want) <= (E + 2.0 ** -22) * (np.abs(old) + w_ref)), (b, n)
            assert torch.equal(w[b, :, n:], w0[b, :, n:])


def _case(M, H, G, d, lens, seed, weights=False, decay=1.0, qscale=1.5):
    k, v, table, pages, seqs = _paged(lens, G, d, seed)
    q = (torch.randn(len(lens), H, d, generator=torch.Generator().manual_seed(seed + 1)) * qscale).bfloat16()
    shape = M.make_shape(H, G, d, 64, 16)
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), max(max(lens), 1), pages)
    w0 = w = None
    if weights:
        w0 = torch.rand(len(lens), G, table.shape[1] * PAGE, generator=torch.Generator().manual_seed(seed + 2))
        w = w0.cuda()
    out, lse = M.msa_dense_attn_decode_paged(shape, pg, q.cuda(), k.cuda(), v.cuda(), weights=w, decay=decay)
    _check(out.cpu(), lse.cpu(), None if w is None else w.cpu(), q, seqs, shape.sm_scale, w0, decay)


SHAPES = [(8, 2, 64), (64, 4, 128), (16, 1, 128), (4, 1, 64), (16, 4, 128), (32, 4, 64), (32, 2, 128), (8, 1, 128)]


@pytest.mark.parametrize("H,G,d", SHAPES)
@pytest.mark.parametrize("weights", [False, True])
def test_borders_and_ragged(M, H, G, d, weights):
    _case(M, H, G, d, [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 0, 255, 257, 1000, 0], 11, weights, 0.75)


@pytest.mark.parametrize("H,G,d", SHAPES)
@pytest.mark.parametrize("L", [1, 777, 5003])
def test_one_sequence_over_many_ctas(M, H, G, d, L):
    _case(M, H, G, d, [L], 21, True, 1.0)


@pytest.mark.parametrize("H,G,d", [(64, 4, 128), (16, 1, 64)])
def test_many_short_sequences(M, H, G, d):
    lens = [(i * 37) % 150 for i in range(421)]
    _case(M, H, G, d, lens, 31, True, 0.0)


def test_one_long_among_short(M):
    _case(M, 32, 2, 128, [3, 9001, 1, 0, 70], 41, True, 0.5)


def test_empty_batch_rows_only(M):
    _case(M, 16, 2, 64, [0, 0, 0], 51, True, 1.0)


def test_peaked_and_minus_infinite_scores(M):
    _case(M, 16, 2, 128, [300, 2000], 61, True, 1.0, qscale=60.0)
    # every score of group 0 is -inf: zeros and -inf; the first half of group 1's is
    H, G, d, n = 8, 2, 64, 200
    k = torch.zeros(2 * PAGE, G, d)
    k[:, 0, 0] = float("-inf")
    k[:100, 1, 0] = float("-inf")
    k[100:, 1, 0] = torch.randn(2 * PAGE - 100)
    v = torch.randn(2 * PAGE, G, d).bfloat16()
    q = torch.zeros(1, H, d)
    q[:, :, 0] = 1.0
    k, q = k.bfloat16(), q.bfloat16()
    shape = M.make_shape(H, G, d, 64, 16)
    pg = M.make_paged(torch.tensor([n], dtype=torch.int32).cuda(), torch.tensor([[0, 1]], dtype=torch.int32).cuda(), n, 2)
    w = torch.zeros(1, G, 2 * PAGE, device="cuda")
    out, lse = M.msa_dense_attn_decode_paged(shape, pg, q.cuda(), k.cuda(), v.cuda(), weights=w)
    assert torch.all(out[0, :4] == 0) and torch.all(lse[0, :4] == float("-inf")) and torch.all(w[0, 0] == 0)
    s = k[100:n, 1, 0].double() * shape.sm_scale
    p = torch.softmax(s, 0)
    want = p @ v[100:n, 1].double()
    assert torch.allclose(out[0, 4:].double().cpu(), want.expand(4, d), rtol=2 ** -8, atol=1e-4)
    assert torch.allclose(w[0, 1, 100:n].double().cpu(), 4 * p, rtol=1e-4, atol=0)
    assert torch.all(w[0, 1, :100] == 0)


def test_same_from_run_to_run_and_without_lse(M):
    lens = [4000, 1, 333]
    k, v, table, pages, _ = _paged(lens, 4, 128, 71)
    q = torch.randn(3, 64, 128).bfloat16().cuda()
    shape = M.make_shape(64, 4, 128, 64, 16)
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), 4096, pages)
    k, v = k.cuda(), v.cuda()
    o1, l1 = M.msa_dense_attn_decode_paged(shape, pg, q, k, v)
    o2, none = M.msa_dense_attn_decode_paged(shape, pg, q, k, v, want_lse=False)
    o3, l3 = M.msa_dense_attn_decode_paged(shape, pg, q, k, v, weights=torch.zeros(3, 4, table.shape[1] * PAGE).cuda())
    assert none is None and torch.equal(o1, o2) and torch.equal(o1, o3) and torch.equal(l1, l3)


def test_equals_the_sparse_call_that_selects_every_block(M):
    lens = [700, 2000]
    k, v, table, pages, _ = _paged(lens, 4, 128, 81, junk=3.0)
    q = torch.randn(2, 64, 128).bfloat16().cuda()
    shape = M.make_shape(64, 4, 128, 64, 16)
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), 2048, pages)
    sel = torch.full((2, 4, 16), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        sel[b, :, :-(-n // PAGE)] = torch.arange(-(-n // PAGE), dtype=torch.int32)
    a, la = M.msa_dense_attn_decode_paged(shape, pg, q, k.cuda(), v.cuda())
    s, ls = M.msa_sparse_attn_decode_paged(shape, pg, q, k.cuda(), v.cuda(), sel.cuda())
    assert float((a.float() - s.float()).abs().max()) <= 2e-2 and float((la - ls).abs().max()) <= 1e-3


def test_bad_pages_and_lengths_are_reported_not_read(M):
    lens = [700, 300, 50]
    H, G, d = 16, 2, 64
    k, v, table, pages, seqs = _paged(lens, G, d, 91)
    q = torch.randn(3, H, d).bfloat16()
    shape = M.make_shape(H, G, d, 64, 16)
    bad = table.clone()
    bad[0, 2], bad[0, 4] = pages + 5, -1
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), bad.cuda(), 700, pages)
    args = (q.cuda(), k.cuda(), v.cuda())
    with pytest.raises(M.MsaError, match="DEVICE_CHECK at site 241"):
        M.msa_dense_attn_decode_paged(shape, pg, *args)
    w = torch.zeros(3, G, table.shape[1] * PAGE, device="cuda")
    out, lse = M.msa_dense_attn_decode_paged(shape, pg, *args, weights=w, check=False)
    stay = torch.cat([torch.arange(0, 256), torch.arange(384, 512), torch.arange(640, 700)])
    stay = stay[stay < 512]                                          # blocks 2 and 4 are out
    stay = torch.cat([stay, torch.arange(640, 700)])
    part = [(seqs[0][0][stay], seqs[0][1][stay]), seqs[1], seqs[2]]
    _check(out.cpu(), lse.cpu(), None, q, part, shape.sm_scale)
    gone = torch.ones(700, dtype=torch.bool)
    gone[stay] = False
    assert torch.all(w[0, :, :700].cpu()[:, gone] == 0) and torch.all(w[0, :, :700].cpu()[:, stay] > 0)
    for wrong in (-1, 701, 2 ** 31 - 1):
        pg = M.make_paged(torch.tensor([700, wrong, 50], dtype=torch.int32).cuda(), table.cuda(), 700, pages)
        with pytest.raises(M.MsaError, match="DEVICE_CHECK at site 241"):
            M.msa_dense_attn_decode_paged(shape, pg, *args)
        out, lse = M.msa_dense_attn_decode_paged(shape, pg, *args, check=False)
        _check(out.cpu(), lse.cpu(), None, q, [seqs[0], (seqs[1][0][:0], seqs[1][1][:0]), seqs[2]], shape.sm_scale)


def test_shared_pages_have_weights_of_their_own(M):
    n = 300
    k, v, table, pages, seqs = _paged([n], 2, 64, 101)
    both = torch.cat([table, table])
    q = torch.randn(2, 8, 64).bfloat16()
    shape = M.make_shape(8, 2, 64, 64, 16)
    pg = M.make_paged(torch.tensor([n, 257], dtype=torch.int32).cuda(), both.cuda(), n, pages)
    w0 = torch.zeros(2, 2, table.shape[1] * PAGE)
    w = w0.cuda()
    out, lse = M.msa_dense_attn_decode_paged(shape, pg, q.cuda(), k.cuda(), v.cuda(), weights=w)
    part = [seqs[0], (seqs[0][0][:257], seqs[0][1][:257])]
    _check(out.cpu(), lse.cpu(), w.cpu(), q, part, shape.sm_scale, w0)


def test_captured_call_follows_its_inputs(M):
    lens = [500, 40, 0]
    H, G, d = 32, 4, 64
    k, v, table, pages, seqs = _paged([640, 640, 640], G, d, 111)
    shape = M.make_shape(H, G, d, 64, 16)
    lens_d = torch.tensor(lens, dtype=torch.int32).cuda()
    pg = M.make_paged(lens_d, table.cuda(), 640, pages)
    q = torch.randn(3, H, d).bfloat16()
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    w = torch.zeros(3, G, table.shape[1] * PAGE, device="cuda")
    ws = torch.empty(M.msa_dense_attn_decode_paged_workspace_size(shape, pg, True), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(3, H, d, dtype=torch.bfloat16, device="cuda"), torch.empty(3, H, device="cuda")
    call = lambda: M.msa_dense_attn_decode_paged(shape, pg, qd, kd, vd, out=out, lse=lse, weights=w, decay=0.5, ws=ws, check=False)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in (lens, [640, 1, 129], [0, 0, 640]):
        q2 = torch.randn(3, H, d).bfloat16()
        qd.copy_(q2)
        lens_d.copy_(torch.tensor(new, dtype=torch.int32))
        w0 = w.cpu()
        graph.replay()
        torch.cuda.synchronize()
        part = [(a[:n], c[:n]) for (a, c), n in zip(seqs, new)]
        _check(out.cpu(), lse.cpu(), w.cpu(), q2, part, shape.sm_scale, w0, 0.5)


def test_side_streams_and_two_calls_at_once(M):
    lens = [3000, 1200]
    k, v, table, pages, seqs = _paged(lens, 4, 128, 121)
    q = torch.randn(2, 64, 128).bfloat16()
    shape = M.make_shape(64, 4, 128, 64, 16)
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), 3000, pages)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [M.msa_dense_attn_decode_paged(shape, pg, qd, kd, vd, stream=s, check=False) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    _check(got[0][0].cpu(), got[0][1].cpu(), None, q, seqs, shape.sm_scale)


def test_offsets_past_32_bits(M):
    # pages past 4 GiB of the pool, weight rows past 2^31 entries
    H, G, d, lens = 16, 4, 128, [300, 129]
    k, v, table, pages, seqs = _paged(lens, G, d, 131, spare=0, extra_blocks=0)
    pool_pages = 40000
    big_k = torch.empty(pool_pages * PAGE, G, d, dtype=torch.bfloat16, device="cuda")
    big_v = torch.empty_like(big_k)
    big_k[-pages * PAGE:], big_v[-pages * PAGE:] = k.cuda(), v.cuda()
    wide = 2 ** 22 + 1
    table2 = torch.full((2, wide), -1, dtype=torch.int32)
    table2[:, :table.shape[1]] = torch.where(table >= 0, table + pool_pages - pages, table)
    q = torch.randn(2, H, d).bfloat16()
    shape = M.make_shape(H, G, d, 64, 16)
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table2.cuda(), 300, pool_pages)
    w = torch.empty(2, G, wide * PAGE, device="cuda")
    assert w[1].storage_offset() > 2 ** 31
    out, lse = M.msa_dense_attn_decode_paged(shape, pg, q.cuda(), big_k, big_v, weights=w, decay=0.0)
    w0 = torch.zeros(2, G, 3 * PAGE)
    head = w[:, :, :3 * PAGE].cpu()
    for b, n in enumerate(lens):
        head[b, :, n:] = 0
    _check(out.cpu(), lse.cpu(), head, q, seqs, shape.sm_scale, w0)


def test_more_rows_than_a_grid_dimension_holds(M):
    # 66000 padded or one-page rows over the same few pages
    H, G, d, B = 4, 1, 64, 66000
    k, v, table, pages, seqs = _paged([128, 128], G, d, 141)
    lens = torch.zeros(B, dtype=torch.int32)
    at = {0: 128, 1: 1, 77: 17, 65534: 100, 65535: 64, 65536: 65, 65999: 128}
    for b, n in at.items():
        lens[b] = n
    tab = table[torch.arange(B) % 2][:, :1].contiguous()
    q = torch.randn(B, H, d, generator=torch.Generator().manual_seed(5)).bfloat16()
    shape = M.make_shape(H, G, d, 64, 16)
    pg = M.make_paged(lens.cuda(), tab.cuda(), 128, pages)
    w0 = torch.rand(B, G, PAGE, generator=torch.Generator().manual_seed(6))
    w = w0.cuda()
    out, lse = M.msa_dense_attn_decode_paged(shape, pg, q.cuda(), k.cuda(), v.cuda(), weights=w, decay=0.5)
    out, lse, w = out.cpu(), lse.cpu(), w.cpu()
    rows = sorted(at)
    part = [(seqs[b % 2][0][:at[b]], seqs[b % 2][1][:at[b]]) for b in rows]
    _check(out[rows], lse[rows], w[rows], q[rows], part, shape.sm_scale, w0[rows], 0.5)
    empty = torch.ones(B, dtype=torch.bool)
    empty[rows] = False
    assert torch.all(out[empty] == 0) and torch.all(lse[empty] == float("-inf")) and torch.equal(w[empty], w0[empty])


@pytest.mark.parametrize("scale", [1e-3, 2.0])
def test_other_scales(M, scale):
    H, G, d, lens = 16, 2, 64, [300, 70]
    k, v, table, pages, seqs = _paged(lens, G, d, 151)
    q = torch.randn(2, H, d, generator=torch.Generator().manual_seed(7)).bfloat16()
    shape = M.make_shape(H, G, d, 64, 16, sm_scale=scale)
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), 300, pages)
    w0 = torch.zeros(2, G, table.shape[1] * PAGE)
    w = w0.cuda()
    out, lse = M.msa_dense_attn_decode_paged(shape, pg, q.cuda(), k.cuda(), v.cuda(), weights=w)
    _check(out.cpu(), lse.cpu(), w.cpu(), q, seqs, scale, w0)


def test_workspace_with_anything_in_it(M):
    lens = [500, 0, 9000]
    k, v, table, pages, seqs = _paged(lens, 2, 128, 161)
    q = torch.randn(3, 32, 128, generator=torch.Generator().manual_seed(8)).bfloat16()
    shape = M.make_shape(32, 2, 128, 64, 16)
    pg = M.make_paged(torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), 9000, pages)
    ws = torch.full((M.msa_dense_attn_decode_paged_workspace_size(shape, pg, True),), 255, dtype=torch.uint8, device="cuda")
    w0 = torch.zeros(3, 2, table.shape[1] * PAGE)
    w = w0.cuda()
    out, lse = M.msa_dense_attn_decode_paged(shape, pg, q.cuda(), k.cuda(), v.cuda(), weights=w, ws=ws)
    _check(out.cpu(), lse.cpu(), w.cpu(), q, seqs, shape.sm_scale, w0)
