"""Host checks of the expert block's operators (gated feed-forward, 8-bit norm
rows and their dispatch, dropout): every refusal returns its status before anything is
launched, so fake addresses are enough and no GPU is needed."""
import pytest

eb = pytest.importorskip("recommender_embedding_tables_amd.embtab",
                         reason="libembtab.so not built")

A = 0x50000000  # a fake, aligned device address
INVALID, WS = eb.EMB_ERR_INVALID_ARG, eb.EMB_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


def test_add_norm_refusals():
    def call(x=A, block=A, w=A, n=10, d=64, t=eb.EMB_BF16, eps=1e-6, y=A, codes=A, scales=A):
        return eb.emb_add_norm_int8(x, block, w, n, d, t, eps, y, codes, scales, 0)

    for kw in (dict(x=None), dict(x=A + 1), dict(x=A + 2, t=eb.EMB_F32), dict(block=None),
               dict(block=A + 1), dict(w=None), dict(w=A + 2), dict(n=-1), dict(n=2**31),
               dict(d=7), dict(d=0), dict(d=8193), dict(t=3), dict(t=-1), dict(eps=-1e-6),
               dict(eps=NAN), dict(eps=INF), dict(y=None), dict(y=A + 1), dict(codes=None),
               dict(scales=None), dict(scales=A + 2)):
        assert call(**kw) == INVALID, kw
    assert call(n=0, x=None, block=None, y=None, codes=None, scales=None) == eb.EMB_OK
    assert call(n=0, w=None) == INVALID


def test_dispatch_int8_refusals():
    def call(codes=A, scales=A, pos=A, src=A, n=10, k=2, m=20, d=64, t=eb.EMB_BF16, xs=A):
        return eb.emb_expert_dispatch_int8(codes, scales, pos, src, n, k, m, d, t, xs, 0)

    for kw in (dict(codes=None), dict(scales=None), dict(scales=A + 2), dict(pos=None),
               dict(pos=A + 2), dict(src=None), dict(src=A + 1), dict(n=-1), dict(k=0),
               dict(k=65), dict(m=-1), dict(m=2**31), dict(d=7), dict(d=2**20 + 1), dict(t=3),
               dict(xs=None), dict(xs=A + 1), dict(xs=A + 2, t=eb.EMB_F32),
               dict(n=2**30, k=64)):
        assert call(**kw) == INVALID, kw
    assert call(n=0, m=0, codes=None, scales=None, pos=None, src=None, xs=None) == eb.EMB_OK


def test_dropout_refusals():
    def call(x=A, res=A, n=100, t=eb.EMB_BF16, p=0.1, rng=A, y=A):
        return eb.emb_dropout(x, res, n, t, p, rng, y, 0)

    for kw in (dict(x=None), dict(x=A + 1), dict(x=A + 2, t=eb.EMB_F32), dict(res=A + 1),
               dict(n=-1), dict(n=2**40), dict(t=3), dict(p=-0.01), dict(p=1.01), dict(p=NAN),
               dict(rng=None), dict(rng=A + 4), dict(y=None), dict(y=A + 1)):
        assert call(**kw) == INVALID, kw
    assert call(n=0, x=None, res=None, y=None) == eb.EMB_OK


def test_gated_ffn_refusals():
    bf = eb.EMB_BF16
    for bad in ((-1, 8, 64, 64, bf), (2**31, 8, 64, 64, bf), (10, 0, 64, 64, bf),
                (10, 1025, 64, 64, bf), (10, 8, 7, 64, bf), (10, 8, 64, 7, bf),
                (10, 8, 65537, 64, bf), (10, 8, 64, 65537, bf), (10, 8, 64, 64, 3),
                (2**30, 8, 1024, 64, bf), (2**30, 8, 64, 1024, bf)):
        assert eb.emb_gated_ffn_workspace_bytes(*bad) == 0, bad
    need = eb.emb_gated_ffn_workspace_bytes(100, 8, 64, 128, bf)
    assert need >= 100 * 2 * 128 * 2

    def forward(x=A, wi=A, wo=A, off=A, m=100, e=8, cap=0, d=64, f=128, t=bf, act=0, gu=A, a=A,
                y=A, ws=A, wb=need):
        return eb.emb_gated_ffn_forward(x, wi, wo, off, m, e, cap, d, f, t, act, gu, a, y, ws, wb,
                                        0)

    def backward(x=A, wi=A, wo=A, off=A, m=100, e=8, cap=0, d=64, f=128, t=bf, act=0, gu=A, a=A,
                 dy=A, dx=A, dwi=A, dwo=A, ws=A, wb=need):
        return eb.emb_gated_ffn_backward(x, gu, a, wi, wo, dy, off, m, e, cap, d, f, t, act, dx,
                                         dwi, dwo, ws, wb, 0)

    both = (dict(x=None), dict(x=A + 1), dict(wi=None), dict(wi=A + 1), dict(wo=None),
            dict(wo=A + 1), dict(off=A + 2), dict(off=None), dict(off=None, e=1, cap=100),
            dict(m=-1), dict(m=2**31), dict(e=0), dict(e=1025), dict(cap=-1), dict(cap=13),
            dict(cap=2**31), dict(d=7), dict(f=7), dict(d=65537), dict(f=65537), dict(t=3),
            dict(act=-1), dict(act=4), dict(gu=A + 1), dict(a=None), dict(a=A + 1),
            dict(x=A + 2, t=eb.EMB_F32))
    for kw in both + (dict(y=None), dict(y=A + 1)):
        assert forward(**kw) == INVALID, kw
    for kw in both + (dict(gu=None), dict(dy=None), dict(dy=A + 1), dict(dx=None), dict(dx=A + 1),
                      dict(dwi=None), dict(dwi=A + 1), dict(dwo=None), dict(dwo=A + 1)):
        assert backward(**kw) == INVALID, kw
    for kw in (dict(ws=None), dict(ws=A + 16), dict(wb=need - 1)):
        assert forward(**kw) == WS and backward(**kw) == WS, kw
    assert forward(m=0, x=None, gu=None, a=None, y=None, wb=need) == eb.EMB_OK
