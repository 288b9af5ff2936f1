"""Linear attention with one decay per head: calls as a program makes them around a step of
its own: workspaces with old contents or shared by graphs, outputs inside larger buffers,
one tensor in several places, calls that overlap."""
import pytest
import torch

from gated_delta_rule_108_b200 import kda
from test_gpu_linear import DTYPES, case, dev, ids

pytestmark = pytest.mark.gpu

# B, T, H, lengths: uncut, few segments, summed in pieces, many segments, one after another, packed and cut
SHAPES = [(2, 200, 2, None), (1, 1024, 30, None), (1, 1500, 60, None), (1, 3000, 1, None), (5, 2000, 32, None),
          (1, 1700, 20, (1600, 0, 100))]


def sizes(B, T, H, lens, dtype):
    args = (B, T, H, 64, 64, B if lens is None else len(lens), lens is not None, dtype)
    return kda.linear_chunk_fwd_workspace_size(*args), kda.linear_chunk_bwd_workspace_size(*args)


def inside(t, room=512):
    """A copy of t's shape inside a larger buffer of sevens, and what tells whether the rest still is."""
    buf = torch.full((t.numel() + 2 * room,), 7, dtype=t.dtype, device=t.device)
    return buf[room:room + t.numel()].view(t.shape), lambda: bool((buf[:room] == 7).all() and (buf[-room:] == 7).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_old_contents_and_neighbours(cuda_device, shape, dtype):
    """What the workspace held does not matter, and nothing outside workspace and outputs is written."""
    B, T, H, lens = shape
    x, back = (dev(t) for t in case(B, T, H, 64, 64, dtype, lens=lens, seed=70))
    o, S = kda.linear_chunk_fwd(**x, check=True)
    g = kda.linear_chunk_bwd(**x, **back, check=True)
    fwd, bwd = sizes(B, T, H, lens, dtype)
    for fill in (255, 1):
        ws = torch.full((fwd + 4096,), fill, dtype=torch.uint8, device="cuda")
        (o2, o_kept), (S2, S_kept) = inside(o), inside(S)
        kda.linear_chunk_fwd(**x, o=o2, final_state=S2, workspace=ws[:fwd], check=True)
        assert torch.equal(o, o2) and torch.equal(S, S2)
        assert o_kept() and S_kept() and bool((ws[fwd:] == fill).all())
        ws = torch.full((bwd + 4096,), fill, dtype=torch.uint8, device="cuda")
        r = kda.linear_chunk_bwd(**x, **back, workspace=ws[:bwd], check=True)
        assert all(torch.equal(g[n], r[n]) for n in g) and bool((ws[bwd:] == fill).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_graphs_that_share_a_workspace(cuda_device, dtype):
    """Captured calls of every kind over one workspace, replayed on one stream in any order."""
    work, ws = [], torch.empty(max(max(sizes(*s, dtype)) for s in SHAPES), dtype=torch.uint8, device="cuda")
    for shape in SHAPES:
        B, T, H, lens = shape
        x, back = (dev(t) for t in case(B, T, H, 64, 64, dtype, lens=lens, seed=71))
        expected = kda.linear_chunk_fwd(**x), kda.linear_chunk_bwd(**x, **back)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = kda.linear_chunk_fwd(**x, workspace=ws), kda.linear_chunk_bwd(**x, **back, workspace=ws)
        work.append((graph, expected, got, x, back))
    for i in (0, 4, 3, 5, 1, 4, 2, 3, 0, 4, 5, 2):
        graph, ((o, S), g), ((o2, S2), g2), _, _ = work[i]
        for t in (o2, S2, *g2.values()):
            t.zero_()
        graph.replay()
        assert kda.workspace_status(ws) == 0
        assert torch.equal(o, o2) and torch.equal(S, S2) and all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_one_tensor_in_every_place(cuda_device, shape, dtype):
    B, T, H, lens = shape
    x, back = (dev(t) for t in case(B, T, H, 64, 64, dtype, lens=lens, seed=72))
    same = {**x, "q": x["k"], "v": x["k"]}
    copies = {**same, "q": x["k"].clone(), "v": x["k"].clone()}
    for a, b in zip(kda.linear_chunk_fwd(**same), kda.linear_chunk_fwd(**copies)):
        assert torch.equal(a, b)
    a = kda.linear_chunk_bwd(**same, d_o=x["k"], d_final_state=x["initial_state"])
    b = kda.linear_chunk_bwd(**copies, d_o=x["k"].clone(), d_final_state=x["initial_state"].clone())
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_calls_of_following_segments_that_overlap(cuda_device, dtype):
    """Two such calls at once, and a third kernel between their blocks: each ends, with its own results."""
    ins = [tuple(dev(t) for t in case(5, 2000, 32, 64, 64, dtype, seed=80 + i)) for i in range(3)]
    ref = [(kda.linear_chunk_fwd(**x), kda.linear_chunk_bwd(**x, **b)) for x, b in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = []
    for _ in range(4):
        for s, (x, b) in zip(streams, ins):
            got.append((kda.linear_chunk_fwd(**x, stream=s), kda.linear_chunk_bwd(**x, **b, stream=s)))
    torch.cuda.synchronize()
    for i, ((o, S), g) in enumerate(got):
        (ro, rS), rg = ref[i % 3]
        assert torch.equal(o, ro) and torch.equal(S, rS) and all(torch.equal(g[n], rg[n]) for n in g)


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_states_in_place_at_every_shape(cuda_device, shape, dtype):
    """Sums in pieces are joined in another order when the state is updated in place.  A state
    element takes one rounding for each of at most 24 chunks and 8 joins, in either order: 64 times
    2^-24 of the largest.  o reads states with unit rows of q (sum of magnitudes 8, times 1/8): that
    difference, 2^-16 where two parts of the state round apart, and one step of its type."""
    B, T, H, lens = shape
    x, _ = (dev(t) for t in case(B, T, H, 64, 64, dtype, lens=lens, seed=73))
    o, S = kda.linear_chunk_fwd(**x)
    S0 = x["initial_state"].clone()
    o2, S2 = kda.linear_chunk_fwd(**{**x, "initial_state": S0}, final_state=S0, check=True)
    assert S2.data_ptr() == S0.data_ptr()
    size = S.abs().amax()
    assert float((S - S2).abs().max()) <= 64 * 2.0 ** -24 * float(size)
    off = (o.double() - o2.double()).abs()
    assert bool((off <= torch.finfo(dtype).eps * o.double().abs() + (64 + 256) * 2.0 ** -24 * float(size)).all())
