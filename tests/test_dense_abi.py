"""The dense operators' host checks (gradient clip, table gradients in two
parts, expert routing, gated norm): every refusal returns its status before
anything is launched, so fake addresses are enough and no GPU is needed."""
import ctypes as C

import pytest

eb = pytest.importorskip("recommender_embedding_tables_amd.embtab",
                         reason="libembtab.so not built")

A = 0x50000000  # a fake, aligned device address
INVALID, WS = eb.EMB_ERR_INVALID_ARG, eb.EMB_ERR_WORKSPACE


class FakeList:
    """TensorList's layout over made-up (address, numel, dtype) entries."""

    def __init__(self, *items):
        self.array = (eb.emb_tensor_t * max(1, len(items)))()
        for a, (data, numel, dtype) in zip(self.array, items):
            a.data, a.numel, a.dtype = data, numel, dtype
        self.n, self.ptr = len(items), C.addressof(self.array)

    def __len__(self):
        return self.n


def clip(grads, out=None, extra=None, num_extra=0, max_norm=1.0, norm=A, ws=A, ws_bytes=1 << 20):
    return eb.emb_clip_grad_norm(grads, out, extra, num_extra, max_norm, norm, ws, ws_bytes, 0)


def test_clip_refusals():
    good = FakeList((A, 100, eb.EMB_F32), (A + 2, 7, eb.EMB_BF16))
    need = eb.emb_grad_workspace_bytes(good)
    assert need > 0 and need % 256 == 0
    for bad in (FakeList((None, 5, 0)), FakeList((A + 2, 5, 0)), FakeList((A, -1, 0)),
                FakeList((A, 5, 3)), FakeList((A + 1, 5, 1)), FakeList((A, 1 << 40, 0))):
        assert eb.emb_grad_workspace_bytes(bad) == 0
        assert clip(bad) == INVALID
    assert clip(good, out=FakeList((A, 100, 0))) == INVALID  # fewer tensors
    for out in (FakeList((A, 99, 0), (A, 7, 0)),               # another length
                FakeList((A, 100, 1), (A, 7, 1)),              # fp32 into bf16
                FakeList((A, 100, 0), (A, 7, 2)),              # bf16 into fp16
                FakeList((A, 100, 0), (A + 2, 7, 0))):         # in place, wider
        assert clip(good, out=out) == INVALID
    assert clip(good, num_extra=1) == INVALID
    assert clip(good, extra=A + 4, num_extra=1) == INVALID
    assert clip(good, num_extra=-1) == INVALID
    assert clip(good, max_norm=-1.0) == INVALID
    assert clip(good, max_norm=float("nan")) == INVALID
    assert clip(good, norm=None) == INVALID and clip(good, norm=A + 2) == INVALID
    assert clip(good, ws=None) == WS and clip(good, ws=A + 16) == WS
    assert clip(good, ws_bytes=need - 1) == WS


def test_tensor_list_refusals():
    import torch
    with pytest.raises(ValueError):
        eb.TensorList([torch.zeros(4, 6).t()])
    with pytest.raises(ValueError):
        eb.TensorList([torch.zeros(4, dtype=torch.float64)])
    assert len(eb.TensorList([])) == 0
    with pytest.raises(ValueError):
        eb.dtype_code(torch.int32)


def test_table_gradient_refusals():
    rows = (C.c_int64 * 2)(1000, 24)
    d = eb.emb_table_desc_t()
    d.num_tables, d.dim, d.rows_per_table = 2, 64, C.cast(rows, C.c_void_p)
    d.weights, d.accum, d.state, d.init_storage = A, 2 * A, 3 * A, 0
    st, h = eb.emb_table_create(d, 0)
    assert st == eb.EMB_OK
    try:
        need = eb.emb_workspace_bytes(h, 100, 300)

        def reduce(h=h, n=300, pool=0, g=A, sums=A, sq=A, ws=A, wb=need, batch=100):
            return eb.emb_bag_grad_reduce_prepared(h, batch, n, pool, g, sums, sq, ws, wb, 0)

        def step(h=h, n=300, sums=A, scale=A, lr=0.1, eps=1e-8, ws=A, wb=need):
            return eb.emb_bag_adagrad_reduced_prepared(h, 100, n, sums, scale, lr, eps, ws, wb, 0)

        for kw in (dict(h=None), dict(pool=2), dict(g=None), dict(g=A + 4), dict(sums=None),
                   dict(sums=A + 8), dict(sq=None), dict(sq=A + 4), dict(n=-1), dict(batch=-1)):
            assert reduce(**kw) == INVALID, kw
        for kw in (dict(ws=None), dict(ws=A + 16), dict(wb=need - 1)):
            assert reduce(**kw) == WS and step(**kw) == WS, kw
        assert reduce(n=2**33) == eb.EMB_ERR_UNSUPPORTED
        for kw in (dict(h=None), dict(sums=None), dict(sums=A + 4), dict(scale=A + 2),
                   dict(lr=float("nan")), dict(eps=-1.0), dict(n=-1)):
            assert step(**kw) == INVALID, kw
        assert step(n=0) == eb.EMB_OK  # nothing to do
    finally:
        eb.emb_table_destroy(h)


def test_expert_refusals():
    for bad in ((-1, 2, 8), (10, 0, 8), (10, 65, 8), (10, 2, 0), (10, 2, 1025), (2**31, 1, 8)):
        assert eb.emb_expert_workspace_bytes(*bad) == 0
    need = eb.emb_expert_workspace_bytes(1000, 2, 8)
    assert need > 0 and need % 256 == 0

    def sort(ids=A, n=1000, k=2, e=8, cap=0, off=A, src=A, pos=A, ws=A, wb=need):
        return eb.emb_expert_sort(ids, n, k, e, cap, off, src, pos, ws, wb, 0)

    for kw in (dict(ids=None), dict(ids=A + 4), dict(off=None), dict(src=None), dict(pos=None),
               dict(src=A + 2), dict(n=-1), dict(k=0), dict(k=65), dict(e=0), dict(e=1025),
               dict(cap=-1), dict(cap=2**30, e=8)):
        assert sort(**kw) == INVALID, kw
    for kw in (dict(ws=None), dict(ws=A + 16), dict(wb=need - 1)):
        assert sort(**kw) == WS, kw

    def rows(f, n=10, k=2, m=20, d=64, t=1, x=A, pos=A, src=A, w=A, out=A, dw=A):
        if f == "dispatch":
            return eb.emb_expert_dispatch(x, pos, src, n, k, m, d, t, out, 0)
        if f == "combine":
            return eb.emb_expert_combine(x, pos, w, n, k, m, d, t, out, 0)
        if f == "combine_backward":
            return eb.emb_expert_combine_backward(x, x, pos, src, w, n, k, m, d, t, out, dw, 0)
        return eb.emb_expert_dispatch_backward(x, pos, n, k, m, d, t, out, 0)

    for f in ("dispatch", "combine", "combine_backward", "dispatch_backward"):
        for kw in (dict(n=-1), dict(k=0), dict(k=65), dict(m=-1), dict(m=2**31), dict(d=7),
                   dict(d=(1 << 20) + 1), dict(t=3), dict(t=-1), dict(x=None), dict(x=A + 1),
                   dict(pos=None), dict(pos=A + 2), dict(out=None), dict(out=A + 1)):
            assert rows(f, **kw) == INVALID, (f, kw)
        if f in ("dispatch", "combine_backward"):
            assert rows(f, src=None) == INVALID
        if f == "combine_backward":
            assert rows(f, w=None) == INVALID and rows(f, dw=None) == INVALID
        assert rows(f, n=0, m=0) == eb.EMB_OK


def test_gated_norm_refusals():
    for bad in ((-1, 64), (10, 7), (10, 8193)):
        assert eb.emb_gated_norm_workspace_bytes(*bad) == 0
    need = eb.emb_gated_norm_workspace_bytes(10, 64)
    assert need > 0 and need % 256 == 0
    R, E, S = eb.EMB_GATE_ROW, eb.EMB_GATE_ELEMENT, eb.EMB_GATE_SIGMOID

    def fwd(x=A, block=A, gate=A, wp=A, sc=A, wn=A, n=10, d=64, t=1, kind=R, eps=1e-6, y=A, h=A):
        return eb.emb_gated_norm_forward(x, block, gate, wp, sc, wn, n, d, t, kind, eps, y, h, 0)

    def bwd(y=A, block=A, gate=A, wp=A, sc=A, wn=A, dy=A, dh=A, n=10, d=64, t=1, kind=R,
            eps=1e-6, dx=A, db=A, dg=A, dwp=A, dsc=A, dwn=A, ws=A, wb=need):
        return eb.emb_gated_norm_backward(y, block, gate, wp, sc, wn, dy, dh, n, d, t, kind, eps,
                                          dx, db, dg, dwp, dsc, dwn, ws, wb, 0)

    common = (dict(block=None), dict(gate=None), dict(sc=None), dict(wn=None), dict(wp=A + 2),
              dict(sc=A + 2), dict(n=-1), dict(d=7), dict(d=8193), dict(t=3), dict(kind=3),
              dict(kind=8), dict(kind=-1), dict(kind=eb.EMB_GATE_NONE), dict(kind=S, gate=None),
              dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
              dict(kind=E | S, gate=A + 1), dict(y=None), dict(block=A + 1))
    for kw in common:
        assert fwd(**kw) == INVALID, kw
        assert bwd(**kw) == INVALID, kw
    for kw in (dict(x=None), dict(h=None), dict(h=A + 1)):
        assert fwd(**kw) == INVALID, kw
    for kw in (dict(dy=None), dict(dh=None), dict(dx=None), dict(db=None), dict(dg=None),
               dict(dwp=None), dict(wp=None), dict(dsc=None), dict(dwn=A + 2),
               dict(kind=eb.EMB_GATE_NONE, gate=None)):
        assert bwd(**kw) == INVALID, kw
    for kw in (dict(ws=None), dict(ws=A + 16), dict(wb=need - 1)):
        assert bwd(**kw) == WS, kw
    assert fwd(n=0, x=None, block=None, gate=None, y=None, h=None) == eb.EMB_OK


class FakeTensor:
    """What TensorList reads of a tensor, on any device."""

    def __init__(self, device, shape=(4,), dtype="torch.float32", contiguous=True):
        import torch
        self.device, self.shape, self.dtype = torch.device(device), shape, dtype
        self.contiguous = contiguous

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return A

    def numel(self):
        return 4


def test_tensor_list_takes_tensors_of_one_gpu():
    import torch
    with pytest.raises(ValueError, match="cpu"):
        eb.TensorList([torch.zeros(4)])
    with pytest.raises(ValueError, match="meta"):
        eb.TensorList([torch.zeros(4, device="meta")])
    good = eb.TensorList([FakeTensor("cuda:1"), FakeTensor("cuda:1", dtype="torch.bfloat16")])
    assert [(a.data, a.numel, a.dtype) for a in good.array] == [(A, 4, 0), (A, 4, 1)]
    for bad in ([FakeTensor("cuda:0"), FakeTensor("cuda:1")],
                [FakeTensor("cuda:0"), FakeTensor("cpu")], [FakeTensor("cpu"), FakeTensor("cpu")]):
        with pytest.raises(ValueError, match="one GPU"):
            eb.TensorList(bad)
    for bad in (FakeTensor("cuda:0", contiguous=False),
                FakeTensor("cuda:0", dtype="torch.float64")):
        with pytest.raises(ValueError):
            eb.TensorList([bad])
