"""What the gated feed-forward asks its callers to hold: sizes alone, so no GPU is needed."""
import pytest

eb = pytest.importorskip("recommender_embedding_tables_amd.embtab",
                         reason="libembtab.so not built")


def weights_bytes(experts, dim, hidden):
    return 3 * experts * dim * hidden * 4


@pytest.mark.parametrize("rows,experts,dim,hidden", [
    (9, 32, 3328, 1664), (16, 32, 3328, 1664), (256, 32, 1664, 896), (256, 32, 1664, 640),
    (2048, 32, 1664, 896), (128, 16, 3327, 1663), (512, 1024, 64, 2000), (0, 4, 479, 640)])
def test_few_rows_do_not_cut_the_weights_of_every_expert(rows, experts, dim, hidden):
    """Cut weights are 6 bytes for each fp32 value of all experts, more than the weights
    themselves; here no row count would pay for making them."""
    need = eb.emb_gated_ffn_workspace_bytes(rows, experts, dim, hidden, eb.EMB_F32)
    rows_bytes = rows * 2 * hidden * 4  # the pre-activations' gradients
    assert rows_bytes <= need <= rows_bytes + weights_bytes(experts, dim, hidden) // 4


A = 0x50000000  # a fake, aligned device address
KINDS = (eb.EMB_F32, eb.EMB_BF16, eb.EMB_F16)


def forward(rows, experts, dim, hidden, kind, ws_bytes, gu=None, ws=A, **kw):
    v = dict(x=A, a=A, y=A, **kw) if rows else dict(x=None, a=None, y=None)
    return eb.emb_gated_ffn_forward(v["x"], A, A, A, rows, experts, 0, dim, hidden, kind,
                                    eb.EMB_ACT_SILU, gu, v["a"], v["y"], ws, ws_bytes, 0)


@pytest.mark.parametrize("rows,experts,dim,hidden", [
    (1, 1, 8, 8), (9, 32, 3328, 1664), (16, 8, 512, 1024), (64, 1, 3327, 1663),
    (4096, 1, 479, 1000), (10_240, 8, 479, 640), (32_768, 16, 3328, 1664), (0, 4, 64, 64)])
@pytest.mark.parametrize("kind", KINDS)
def test_a_forward_that_keeps_nothing_needs_its_own_workspace(rows, experts, dim, hidden, kind):
    shape = (rows, experts, dim, hidden, kind)
    own, both = eb.emb_gated_ffn_forward_workspace_bytes(*shape), \
        eb.emb_gated_ffn_workspace_bytes(*shape)
    assert 256 <= own <= both
    if kind != eb.EMB_F32 or rows <= 32 * experts:
        assert own == 256
    for ws, n in ((A, own - 1), (None, own), (A + 16, own)):
        assert forward(*shape, n, ws=ws) == eb.EMB_ERR_WORKSPACE
    if both > own:  # kept for a backward: the workspace of both
        assert forward(*shape, own, gu=A) == eb.EMB_ERR_WORKSPACE
    if rows == 0:  # nothing to launch
        assert forward(*shape, own) == eb.EMB_OK


def test_no_size_for_shapes_that_are_refused():
    for bad in ((-1, 8, 64, 64, eb.EMB_BF16), (10, 0, 64, 64, eb.EMB_BF16),
                (10, 1025, 64, 64, eb.EMB_F32), (10, 8, 7, 64, eb.EMB_F32),
                (10, 8, 64, 65_537, eb.EMB_F16), (10, 8, 64, 64, 3)):
        assert eb.emb_gated_ffn_forward_workspace_bytes(*bad) == 0, bad
