"""The gated feed-forward captured into a graph and replayed on new inputs, with the
program's own eager work between the replays, and on two streams at once: every kernel
family, bit for bit what the eager call gives."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from recommender_embedding_tables_amd import embtab as eb  # noqa: E402
from tests.test_gpu_dense import DEV, gen, rand  # noqa: E402
from tests.test_gpu_ffn import Case, ragged  # noqa: E402

CASES = {
    "planes_and_parts_f32": ([2500], 0, 0, 40, 1200, "f32"),
    "planes_capacity_f32": ([300, 41, 0, 299], 300, 0, 479, 96, "f32"),
    "tiles_and_parts_f32": ([900 - 3 * i for i in range(8)], 0, 5, 136, 520, "f32"),
    "few_f32": ([3, 0, 19, 40], 0, 2, 479, 333, "f32"),
    "large_bf16": (ragged(20, 700, 1), 0, 3, 1032, 520, "bf16"),
    "odd_f16": ([200, 313], 0, 4, 351, 129, "f16"),
}


def run(c, out, ws, stream=None):
    gu, a, y, dx, dw_in, dw_out = out
    eb.check(eb.emb_gated_ffn_forward(c.x, c.w_in, c.w_out, c.offsets, *c.args, gu, a, y, ws,
                                      c.need, stream), "forward")
    eb.check(eb.emb_gated_ffn_backward(c.x, gu, a, c.w_in, c.w_out, c.dy, c.offsets, *c.args, dx,
                                       dw_in, dw_out, ws, c.need, stream), "backward")


def outputs(c):
    def empty(*shape):
        return torch.full(shape, 77, dtype=c.t, device=DEV)

    return [empty(c.M, 2 * c.F), empty(c.M, c.F), empty(c.M, c.D), empty(c.M, c.D),
            empty(*c.w_in.shape), empty(*c.w_out.shape)]


def same(got, want, what):
    for v, w, name in zip(got, want, ("gu", "a", "y", "dx", "dw_in", "dw_out")):
        assert torch.equal(v, w), f"{what}: {name}"


@pytest.mark.parametrize("name", list(CASES))
def test_replays_on_new_inputs(name):
    c = Case(*CASES[name], "silu")
    out, ws = outputs(c), torch.empty_like(c.ws)
    run(c, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c, out, ws)
    work = rand(gen(3), 512, 512)
    want_work = (work @ work).sum(0)
    for i in range(4):
        g = gen(20 + i)
        for v in (c.x, c.dy):
            v[c.live] = rand(g, int(c.live.sum()), c.D).to(c.t)
        for v in (c.w_in, c.w_out):
            v.copy_(rand(g, *v.shape, scale=v.shape[-1] ** -0.5))
        want = outputs(c)
        run(c, want, torch.empty_like(c.ws).fill_(i))
        for v in out:
            v.fill_(77)
        ws.fill_(255 - i)
        assert torch.equal((work @ work).sum(0), want_work)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same(out, want, f"replay {i}")
        assert all(torch.isfinite(v[c.live] if v.shape[0] == c.M else v).all() for v in out)


@pytest.mark.parametrize("name", list(CASES))
def test_two_calls_at_once(name):
    """The same inputs on two streams, each with its own workspace and outputs."""
    c = Case(*CASES[name], "gelu")
    want = outputs(c)
    run(c, want, c.ws)
    both = [(outputs(c), torch.empty_like(c.ws), torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for out, ws, stream in both:
            run(c, out, ws, stream)
    torch.cuda.synchronize()
    for i, (out, _, _) in enumerate(both):
        same(out, want, f"stream {i}")
