"""A densely attended layer's cache at the ends of what its calls allow:
values that are infinite, NaN or huge, key weights past the largest number, against the fp64 oracle
(oracle/dense_cache.py)."""
import numpy as np
import pytest
import torch

from oracle import dense_cache as C
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


# ------------------------------------------------------------------ key weights

def _cu(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


def _varlen(M, T, S):
    return M.make_varlen(torch.tensor(_cu(T), dtype=torch.int32).cuda(), torch.tensor(_cu(S), dtype=torch.int32).cuda(),
                         _cu(T), _cu(S))


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
        w = M.msa_attn_weights(shape, _varlen(M, [T], [T]), q.cuda(), k.cuda(), lse.cuda(), decay=0.0).cpu()[0]
        want = (H // G) * torch.flip(torch.cumsum(torch.flip(torch.exp(-lse[:, 0].double()), [0]), 0), [0])
        inf = want > 2.0 ** 128 * 1.01
        assert bool((w[:, inf] == float("inf")).all()) and int(inf.sum()) >= 6
        # beyond `last` sums of ones: exact but for the exponential's 2^-22 (an argument of 0 has no error)
        rest = torch.arange(T) > last
        assert bool(((w[:, rest].double() - want[rest]).abs() <= want[rest] * 2.0 ** -21).all())
