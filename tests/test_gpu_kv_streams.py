"""KV-cache calls at once: two streams, each with caches, weights and workspaces of its own, give what the calls one
after the other give, eagerly and as two captured graphs replayed together."""
import pytest
import torch

from full_attention_gated_b200 import binding as hb

pytestmark = pytest.mark.gpu


class Loop:
    """append -> decode with weights -> choice -> compaction on one stream; d = 256 and 128 by turns."""

    def __init__(self, seed, B, T, Hq, H, d, n_keep):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.k, self.v = (torch.randn((B, T, H, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
        self.q = torch.randn((B, Hq, d), generator=gen, device="cuda").bfloat16()
        self.lens = torch.randint(1, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        self.cache = [torch.zeros(s, dtype=t, device="cuda") for s, t in 2 * [((B, T, H, d // 2), torch.uint8),
                                                                             ((B, T, H, d // 32), torch.float16)]]
        self.acc = torch.zeros((B, H, T), device="cuda")
        self.o = torch.empty_like(self.q)
        self.keep = torch.empty((B, H, n_keep), dtype=torch.int32, device="cuda")
        self.n_keep = n_keep
        self.ws = torch.empty(hb.gqa_attn_decode_q4_0_workspace_size(B, Hq, H, d, T, True), dtype=torch.uint8,
                              device="cuda")

    def reset(self):
        for t in self.cache + [self.acc]:
            t.zero_()

    def run(self, stream=None):
        hb.kv_append_q4_0(self.k, self.v, *self.cache, stream=stream)
        for _ in range(3):
            hb.gqa_attn_decode_q4_0(self.q, *self.cache, cache_len=self.lens, o=self.o, acc_in=self.acc,
                                    acc_out=self.acc, workspace=self.ws, stream=stream)
        hb.kv_evict_select(self.acc, self.n_keep, 8, cache_len=self.lens, keep=self.keep, stream=stream)
        hb.kv_compact(self.keep, self.cache, acc=self.acc, stream=stream)

    def results(self):
        return [t.clone() for t in self.cache + [self.acc, self.o, self.keep]]


@pytest.fixture
def loops():
    both = [Loop(1, 6, 2000, 12, 4, 256, 300), Loop(2, 9, 1500, 8, 2, 128, 1499)]
    want = []
    for x in both:
        x.reset()
        x.run()
        torch.cuda.synchronize()
        want.append(x.results())
    return both, want


def _same(both, want):
    for x, w in zip(both, want):
        for got, ref in zip(x.results(), w):
            assert torch.equal(got, ref)


def test_two_streams_at_once(loops):
    both, want = loops
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(5):
        for x in both:
            x.reset()
        torch.cuda.synchronize()
        for x, s in zip(both, streams):
            x.run(stream=s)
        torch.cuda.synchronize()
        _same(both, want)
    hb.hh_device_status()


def test_two_graphs_at_once(loops):
    both, want = loops
    graphs, streams = [], [torch.cuda.Stream() for _ in both]
    for x in both:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    for _ in range(3):
        for x in both:
            x.reset()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        _same(both, want)
    hb.hh_device_status()
