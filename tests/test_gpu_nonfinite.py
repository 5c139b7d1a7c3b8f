"""Self-attention of values that are not finite: they reach the result where they count, and only there.

A NaN or +inf score makes the row's o and lse NaN; NaN of V reaches its channel.  (The definition gives the same:
the softmax of a row with a NaN or +inf score is NaN.)
"""
import pytest
import torch

import sequence_parallelism_st_b200 as st

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


def rand(seed, *shape, dtype=BF):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def run(fn, q, k, v, *args, o_fp32=0, **kw):
    B, T, S, H, D = q.shape
    o = torch.zeros(q.shape, dtype=F32 if o_fp32 else q.dtype, device="cuda")
    lse = torch.zeros(B, T, H, S, device="cuda")
    fn(q, k, v, o, lse, *args, o_fp32=o_fp32, **kw)
    assert st.st_check_device_status() == st.ST_OK
    return o, lse


def check_keys(call, q, k, v, places, what):
    """call(q, k, v) -> o, lse of all keys; head 0 of frame 0 gets the bad value."""
    for i in places:
        kn = k.clone()
        kn[0, 0, i, 0, 1] = NAN
        o, lse = call(q, kn, v)
        assert o[0, 0, :, 0].isnan().all() and lse[0, 0, 0].isnan().all(), f"{what}: K of key {i}"
        assert o[0, 0, :, 1].isfinite().all() and lse[0, 0, 1].isfinite().all()
        vn = v.clone()
        vn[0, 0, i, 0, 3] = NAN
        o, lse = call(q, k, vn)
        assert o[0, 0, :, 0, 3].isnan().all() and o[0, 0, :, 0, 4:].isfinite().all() and lse.isfinite().all(), what
        kn, qn = k.clone(), q.clone()
        kn[0, 0, i, 0], qn[0, 0, 7, 0] = torch.finfo(k.dtype).max / 4, 8.0
        kn[0, 0, i, 1], qn[0, 0, 7, 1] = torch.finfo(k.dtype).max / 4, -8.0      # a score of -inf: weight 0
        o, lse = call(qn, kn, v)
        assert o[0, 0, 7, 0].isnan().all() and lse[0, 0, 0, 7].isnan(), f"{what}: +inf at key {i}"
        assert o[0, 0, 7, 1].isfinite().all() and lse[0, 0, 1, 7].isfinite(), f"{what}: -inf at key {i}"
    qn = q.clone()
    qn[0, 0, 5, 0, 0] = NAN
    o, lse = call(qn, k, v)
    assert o[0, 0, 5, 0].isnan().all() and lse[0, 0, 0, 5].isnan(), f"{what}: Q"
    o[0, 0, 5, 0], lse[0, 0, 0, 5] = 0, 0
    assert o.isfinite().all() and lse.isfinite().all(), what


@pytest.mark.parametrize("D,S", [(32, 200), (64, 300), (72, 77), (72, 1600), (80, 260), (96, 390), (128, 300)])
def test_spatial(D, S):
    q, k, v = (rand(300 + i, 1, 2, S, 2, D) for i in range(3))
    places = list(range(16)) + [S - 1, S - 3, S // 2]
    check_keys(lambda *x: run(st.st_attn_spatial, *x), q, k, v, places, "spatial")
    check_keys(lambda *x: run(st.st_attn_ring, *x, 3), q, k, v, places[::5], "ring")
    def chained(q, k, v):
        o, lse = run(st.st_attn_spatial, q, k, v, o_fp32=1, kv_begin=0, kv_end=S // 2)
        out = torch.zeros_like(q)
        st.st_attn_spatial_merge(q, k, v, o, lse, out, lse, kv_begin=S // 2, kv_end=S)
        return out, lse
    check_keys(chained, q, k, v, places[::5] + places[-2:], "merge")


@pytest.mark.parametrize("n", [1, 4, 5])
def test_spatial_few_keys(n):
    """NaN in a query over at most four keys: its lse is NaN, not that of a row without keys."""
    q, k, v = (rand(310 + i, 1, 1, 40, 1, 72) for i in range(3))
    q[0, 0, 3, 0, 2] = NAN
    o, lse = run(st.st_attn_spatial, q, k, v, kv_begin=8, kv_end=8 + n)
    assert o[0, 0, 3].isnan().all() and lse[0, 0, 0, 3].isnan()
    assert lse.isnan().sum() == 1 and o.isnan().sum() == 72


def test_fp32():
    """The FMA kernel, plain, as ring and as a chain of two ranges; a first key whose score is -inf has weight 0."""
    S = 70
    q, k, v = (rand(320 + i, 1, 2, S, 2, 40, dtype=F32) for i in range(3))
    places = [0, 1, 33, S - 1]
    check_keys(lambda *x: run(st.st_attn_spatial, *x), q, k, v, places, "spatial")
    check_keys(lambda *x: run(st.st_attn_ring, *x, 3), q, k, v, places, "ring")

    def chained(q, k, v):
        o, lse = run(st.st_attn_spatial, q, k, v, kv_begin=0, kv_end=S // 2)
        out = torch.zeros_like(q)
        st.st_attn_spatial_merge(q, k, v, o, lse, out, lse, kv_begin=S // 2, kv_end=S)
        return out, lse
    check_keys(chained, q, k, v, places, "merge")
    # an accumulated row that is NaN stays NaN behind a range without keys and behind one with them
    acc, lacc = run(st.st_attn_spatial, q, k, v)
    acc[0, 0, 4, 1], lacc[0, 0, 1, 4] = NAN, NAN
    for end in (10, 20):
        out, lse = torch.zeros_like(q), torch.zeros_like(lacc)
        st.st_attn_spatial_merge(q, k, v, acc, lacc, out, lse, kv_begin=10, kv_end=end)
        assert out[0, 0, 4, 1].isnan().all() and lse[0, 0, 1, 4].isnan()
        assert out.isnan().sum() == 40 and lse.isnan().sum() == 1


def test_temporal():
    for dtype, D in ((F32, 40), (BF, 72)):
        q, k, v = (rand(330 + i, 1, 9, 6, 2, D, dtype=dtype) for i in range(3))
        for t in range(9):
            kn = k.clone()
            kn[0, t, 2, 0, 1] = NAN
            o, lse = torch.zeros_like(q), torch.zeros(1, 6, 2, 9, device="cuda")
            st.st_attn_temporal(q, kn, v, o, lse)
            assert o[0, :, 2, 0].isnan().all() and lse[0, 2, 0].isnan().all()
            assert o.isnan().sum() == 9 * D and lse.isnan().sum() == 9

@pytest.mark.parametrize("R", [1, 2, 3, 8])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_chunk_merge(R, dtype):
    """A partial that is NaN makes the merged row NaN, also where the other chunks hold no key of it."""
    U, S, H, D = 2, 33, 3, 72
    o = [rand(340 + c, U, S, H, D, dtype=F32) for c in range(R)]
    lse = [rand(350 + c, U, H, S, dtype=F32) for c in range(R)]
    for c in range(R):
        x, y = [t.clone() for t in o], [t.clone() for t in lse]
        x[c][0, 4, 1], y[c][0, 1, 4] = NAN, NAN
        x[c][1, 8, 2], y[c][1, 2, 8] = NAN, NAN
        for i in range(R):
            if i != c:
                y[i][1, 2, 8] = -INF
        out, lout = torch.zeros(U, S, H, D, dtype=dtype, device="cuda"), torch.zeros(U, H, S, device="cuda")
        st.attn_chunk_merge(x, y, U, S, H, D, out, lout)
        for u, s, h in ((0, 4, 1), (1, 8, 2)):
            assert out[u, s, h].isnan().all() and lout[u, h, s].isnan(), (c, u)
        assert out.isnan().sum() == 2 * D and lout.isnan().sum() == 2
