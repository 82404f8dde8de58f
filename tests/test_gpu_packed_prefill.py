"""Packed prefill in the settings of a server: captured graphs, several
streams, and inputs at which the pieces of a long sequence meet."""
import pytest
import torch

from test_gpu_mixer import BF16, _gen, _layer, _lens_case, _scan_inputs, rs  # noqa: F401

pytestmark = pytest.mark.gpu


def _slow(ins):
    """Slow decays, so that earlier pieces of a sequence reach into later ones."""
    ins[3] = (ins[3].float() * 0.02).to(ins[3].dtype)
    return ins


def test_captured_prefill_beside_larger_eager_calls(rs):  # noqa: F811
    """A prefill captured after an eager one of its size, then a larger eager one on the same layer and tensors that
    may take any memory freed since: every replay gives the eager result bit for bit and writes nothing else."""
    lens, H, G = [1500, 3, 900], 4, 1
    g, n, slots, cu, _ = _lens_case(lens, 71, 0)
    cu = cu.cuda()
    ins = _slow([t.cuda() for t in _scan_inputs(g, sum(lens), H, G, BF16)])
    ls, *_ = _layer(rs, n, H, G, BF16, 73)
    start = ls.snapshot()
    want = rs.prefill_packed(ls, *ins, cu)
    after = ls.snapshot()
    y = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rs.prefill_packed(ls, *ins, cu, y=y)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rs.prefill_packed(ls, *ins, cu, y=y)
    big = [3000, 700, 4100]
    more = _slow([t.cuda() for t in _scan_inputs(g, sum(big), H, G, BF16)])
    rs.prefill_packed(ls, *more, torch.tensor([0, *big]).cumsum(0).to(torch.int32).cuda())
    torch.cuda.synchronize()
    guards = [torch.full((k,), 7.0, device="cuda") for k in (1 << 10, 1 << 14, 1 << 17, 1 << 18, 1 << 19, 1 << 20) * 4]
    for i in range(5):
        ls.restore(start)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
        for k, v in after.items():
            assert torch.equal(ls.tensors()[k], v), (i, k)
        rs.prefill_packed(ls, *more, torch.tensor([0, *big]).cumsum(0).to(torch.int32).cuda())
        assert all(bool((t == 7).all()) for t in guards), i
    rs.check_device_errors(ls)


def test_prefills_of_one_layer_on_two_streams(rs):  # noqa: F811
    """Calls that overlap on disjoint slots of a layer give what they give one after the other."""
    H, G, halves = 4, 1, ([2000, 1100], [900, 2500])
    g = _gen(81)
    jobs = []
    for lens, slots in zip(halves, ([0, 3], [2, 1])):
        ins = _slow([t.cuda() for t in _scan_inputs(g, sum(lens), H, G, BF16)])
        jobs.append((ins, torch.tensor([0, *lens]).cumsum(0).to(torch.int32).cuda(),
                     torch.tensor(slots, dtype=torch.int32, device="cuda")))
    one, *_ = _layer(rs, 4, H, G, BF16, 83)
    two, *_ = _layer(rs, 4, H, G, BF16, 83)
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for i in range(4):
        want = [rs.prefill_packed(one, *ins, cu, slots=sl) for ins, cu, sl in jobs]
        got = [rs.prefill_packed(two, *ins, cu, slots=sl, stream=s) for (ins, cu, sl), s in zip(jobs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        assert torch.equal(one.ckpt, two.ckpt), i
    rs.check_device_errors(two)
