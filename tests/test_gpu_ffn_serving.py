"""A gated feed-forward that keeps nothing for a backward, in the workspace that it asks
for and no more: the bits of one that keeps its pre-activations."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from recommender_embedding_tables_amd import embtab as eb  # noqa: E402
from tests.test_gpu_dense import DEV, TYPES, guarded  # noqa: E402
from tests.test_gpu_ffn import PATHS, SHAPES, Case  # noqa: E402

CASES = {**{f"shape{i}": s for i, s in enumerate(SHAPES)}, **PATHS,
         "planes_capacity": ([300, 41, 0, 299], 300, 0, 479, 96),
         "dense": ([4096], 0, 0, 479, 1000)}


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", list(CASES))
def test_forward_in_its_own_workspace(name, kind):
    c = Case(*CASES[name], kind, "gelu")
    _, a, y = c.forward()
    need = eb.emb_gated_ffn_forward_workspace_bytes(c.M, c.E, c.D, c.F, c.code)
    base = torch.full((256 + need + 4096,), 93, dtype=torch.uint8, device=DEV)
    (a2, check_a), (y2, check_y) = (guarded(v.shape, c.t) for v in (a, y))
    eb.check(eb.emb_gated_ffn_forward(c.x, c.w_in, c.w_out, c.offsets, *c.args, None, a2, y2,
                                      base[256:], need), "forward")
    torch.cuda.synchronize()
    check_a()
    check_y()
    assert torch.equal(a2, a) and torch.equal(y2, y)
    assert (base[:256] == 93).all() and (base[256 + need:] == 93).all(), "outside the workspace"
