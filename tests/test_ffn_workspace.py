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
