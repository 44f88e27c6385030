"""The gate's and the experts' calls in a chain where each reads what the one
before it wrote: back to back, on a side stream, in two streams at once and
replayed from a graph, with inputs that change between runs.  Results are
compared, bit for bit, with a run that waits for the device after every call, in
buffers filled with another value before each run: a call that did not run, ran
too early or ran elsewhere shows."""
import pytest
import torch

from combine_ep_get_03_gb300 import ep
from combine_ep_get_03_gb300 import moe
from test_gpu_experts import DEV, gen, quantize

pytestmark = pytest.mark.gpu
ROWS, H, F, T, E, k = 416, 256, 384, 640, 32, 4
GROUPS = 3


def make_inputs(seed):
    """Rows, weights, groups and logits of one run."""
    g = gen(seed)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    xq, xs = quantize(rand(ROWS, H))
    w1, w1s = moe.quantize_blocks(rand(GROUPS, 2 * F, H) / H ** 0.5)
    w2, w2s = moe.quantize_blocks(rand(GROUPS, H, F) / F ** 0.5)
    count = torch.randint(60, 130, (GROUPS,), generator=g, device=DEV).int()
    offset = torch.tensor([0, 130, 260], device=DEV).int() + torch.randint(0, 20, (1,), generator=g, device=DEV).int()
    return dict(xq=xq.view(torch.uint8), xs=xs.t().contiguous(), w1=w1.view(torch.uint8), w1s=w1s,
                w1t=w1.view(torch.uint8).transpose(1, 2).contiguous(), w1ts=w1s.transpose(1, 2).contiguous(),
                w2=w2.view(torch.uint8), w2s=w2s, w2t=w2.view(torch.uint8).transpose(1, 2).contiguous(),
                w2ts=w2s.transpose(1, 2).contiguous(), count=count, offset=offset, rw=rand(ROWS), logits=rand(T, E),
                go=rand(T, k))


class Chain:
    """Buffers of one chain, and its calls."""

    def __init__(self):
        e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
        f8, bf = torch.uint8, torch.bfloat16
        self.i = {n: torch.empty_like(t) for n, t in make_inputs(0).items()}
        self.o = dict(act=e(ROWS, F, dt=f8), acts=e(F // 128, ROWS), pre=e(ROWS, 2 * F, dt=f8),
                      pres=e(2 * F // 128, ROWS), y=e(ROWS, H, dt=bf), gy=e(ROWS, F, dt=bf), gp=e(ROWS, 2 * F, dt=f8),
                      gps=e(2 * F // 128, ROWS), grw=e(ROWS), dw1=e(GROUPS, 2 * F, H, dt=bf), gx=e(ROWS, H, dt=bf),
                      idx=e(T, k, dt=torch.int64), w=e(T, k), cnt=e(E + 1, dt=torch.int32), prob=e(E), loss=e(1),
                      gl=e(T, E))
        self.ws = torch.zeros(ep.ep_gate_workspace_bytes(E), dtype=torch.uint8, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def take(self, inputs):
        for n, t in inputs.items():
            self.i[n].copy_(t)

    def poison(self):
        for t in self.o.values():
            t.view(torch.uint8).fill_(0x2A)

    def run(self, after=lambda: None):
        i, o = self.i, self.o
        at = dict(group_count=i["count"], group_offset=i["offset"], device_status=self.status)
        ep.ep_gate_forward(i["logits"], o["idx"], o["w"], o["cnt"], o["prob"], o["loss"], self.ws, loss_coef=0.5)
        after()
        ep.ep_gate_backward(i["logits"], o["idx"], o["cnt"], i["go"], o["loss"], o["gl"], loss_coef=0.5)
        after()
        ep.ep_grouped_matmul_swiglu(i["xq"], i["xs"], i["w1"], i["w1s"], o["act"], o["acts"], row_weights=i["rw"],
                                    pre=o["pre"], pre_scales=o["pres"], **at)
        after()
        ep.ep_grouped_matmul(o["act"], o["acts"], i["w2"], i["w2s"], o["y"], **at)
        after()
        # the rows themselves stand in for the output's gradient
        ep.ep_grouped_matmul(i["xq"], i["xs"], i["w2t"], i["w2ts"], o["gy"], **at)
        after()
        ep.ep_grouped_swiglu_backward(o["gy"], o["pre"], o["pres"], o["gp"], o["gps"], row_weights=i["rw"],
                                      grad_row_weights=o["grw"], **at)
        after()
        ep.ep_grouped_weight_grad(o["gp"], o["gps"], i["xq"], i["xs"], o["dw1"], **at)
        after()
        ep.ep_grouped_matmul(o["gp"], o["gps"], i["w1t"], i["w1ts"], o["gx"], **at)
        after()

    def results(self):
        return {n: t.clone() for n, t in self.o.items()}


def one_by_one(inputs):
    c = Chain()
    c.take(inputs)
    c.poison()
    torch.cuda.synchronize()
    c.run(after=torch.cuda.synchronize)
    assert int(c.status) == ep.EP_OK
    return c.results()


def same(got, want):
    for n in want:
        assert torch.equal(got[n].view(torch.uint8), want[n].view(torch.uint8)), n


@pytest.fixture(scope="module")
def sets():
    made = [make_inputs(s) for s in (101, 102, 103)]
    want = [one_by_one(m) for m in made]
    for n in want[0]:  # every result depends on the inputs
        assert not torch.equal(want[0][n].view(torch.uint8), want[1][n].view(torch.uint8)), n
    return made, want


def test_back_to_back(sets):
    """No wait anywhere, buffers used again at once by other inputs."""
    made, want = sets
    c = Chain()
    got = []
    for i in range(12):
        c.take(made[i % 3])
        c.poison()
        c.run()
        got.append(c.results())
    torch.cuda.synchronize()
    for i in range(12):
        same(got[i], want[i % 3])
    assert int(c.status) == ep.EP_OK and not c.ws.any()


def test_given_stream_and_current_stream(sets):
    """The current stream is the one that torch says, whatever ran before."""
    made, want = sets
    c = Chain()
    side = torch.cuda.Stream()
    for i in range(3):
        c.take(made[i])
        c.poison()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.run()
            got = c.results()
        side.synchronize()
        same(got, want[i])
        torch.cuda.current_stream().wait_stream(side)


def test_two_streams_at_once(sets):
    made, want = sets
    chains = [Chain(), Chain()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    torch.cuda.synchronize()
    for i in range(8):
        for j in (0, 1):
            with torch.cuda.stream(streams[j]):
                chains[j].take(made[(i + j) % 3])
                chains[j].poison()
                chains[j].run()
                got[j].append(chains[j].results())
    torch.cuda.synchronize()
    for j in (0, 1):
        for i in range(8):
            same(got[j][i], want[(i + j) % 3])
        assert int(chains[j].status) == ep.EP_OK


def test_replayed_from_a_graph(sets):
    """The captured chain reads what its buffers hold when it is replayed."""
    made, want = sets
    c = Chain()
    c.take(made[0])
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    got = []
    for i in range(6):
        c.take(made[i % 3])
        c.poison()
        graph.replay()
        got.append(c.results())
    torch.cuda.synchronize()
    for i in range(6):
        same(got[i], want[i % 3])
    assert int(c.status) == ep.EP_OK
