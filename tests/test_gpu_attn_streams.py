"""GPU: attention calls on several streams at once, queued behind one another, eager, prepared and captured."""
import pytest
import torch

from bit_quantized_decode_amd import binding as B
from helpers import device
from test_gpu_attn_decode import FORMATS, Batch

pytestmark = pytest.mark.gpu

WAIT = 2_000_000      # clock ticks, about a millisecond: what follows on that stream is queued behind it


def test_every_round_of_overlapping_streams():
    """Ten rounds on three streams, nothing waited for in between; each round's outputs are checked."""
    dev = device()
    xs = [Batch(dev, f, [3000, 100], 10, 2, 128, 64, seed=s) for s, f in enumerate(FORMATS)]
    qs = [x.q.to(dev) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[] for _ in xs]
    for _ in range(10):
        for x, q, s, g in zip(xs, qs, streams, got):
            g.append(B.attn_decode(q, x.cache, x.table, x.seq, lse=True, stream=s))
    torch.cuda.synchronize()
    for x, g in zip(xs, got):
        x.check(*g[0])
        for out, lse in g[1:]:
            assert torch.equal(out, g[0][0]) and torch.equal(lse, g[0][1])


def test_a_larger_workspace_while_calls_are_queued():
    """Calls that need more and more of their stream's workspace, all queued before the first one runs."""
    dev = device()
    xs = [Batch(dev, B.NVFP4_KV_NVFP4, [3000, 100], 2, 2, 64, 64, seed=1),
          Batch(dev, B.NVFP4_KV_E4M3, [5000] * 4, 10, 2, 128, 64, seed=2),
          Batch(dev, B.NVFP4_KV_BF16, [6000, 900], 32, 2, 256, 64, seed=3)]
    qs = [x.q.to(dev) for x in xs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, sizes = [], []
    with torch.cuda.stream(s):
        torch.cuda._sleep(WAIT)
        for x, q in zip(xs, qs):
            got.append(B.attn_decode(q, x.cache, x.table, x.seq, lse=True))
            sizes += [w.numel() for key, w in B._workspaces.items() if key[-1] == s.cuda_stream]
            filler = torch.full((4 << 20,), 0xff, dtype=torch.uint8, device=dev)   # takes memory that the old one gave back
        for x, q in zip(xs, qs):
            got.append(B.attn_decode(q, x.cache, x.table, x.seq, lse=True))
    torch.cuda.synchronize()
    del filler
    assert sizes[0] < sizes[1] < sizes[2]
    for x, a, b in zip(xs, got[:3], got[3:]):
        x.check(*a)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_prepared_calls_at_once():
    """Two prepared calls over one cache on two streams, and a third that shares the second's stream."""
    dev = device()
    x = Batch(dev, B.NVFP4_KV_NVFP4, [4000, 0, 700], 10, 2, 128, 64, seed=4)
    q = x.q.to(dev)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    calls = [B.attn_decode_prepared(q, x.cache, x.table, x.seq, lse=True, stream=s) for s in (a, b, b)]
    kept = []
    for _ in range(8):
        for s in (a, b):
            with torch.cuda.stream(s):
                torch.cuda._sleep(WAIT // 20)
        outs = [call() for call in calls]
        torch.cuda.synchronize()
        kept.append([[t.clone() for t in out] for out in outs])
    x.check(*kept[0][0])
    for outs in kept:
        for out, lse in outs:
            assert torch.equal(out, kept[0][0][0]) and torch.equal(lse, kept[0][0][1])


def test_capture_by_a_call_told_its_stream():
    """A call told the capturing stream, while another is current: its graph has a workspace of its own, whatever the stream's eager
    one holds (here counters that no call has left so, put back afterwards)."""
    dev = device()
    x = Batch(dev, B.NVFP4_KV_NVFP4, [4000, 0, 700], 10, 2, 128, 64, seed=5)
    q = x.q.to(dev)
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    want = B.attn_decode(q, x.cache, x.table, x.seq, lse=True)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        B.attn_decode(q, x.cache, x.table, x.seq)             # the stream has an eager workspace
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        with torch.cuda.stream(other):
            out, lse = B.attn_decode(q, x.cache, x.table, x.seq, lse=True, stream=s)
    torch.cuda.synchronize()
    eager = [w for key, w in B._workspaces.items() if key[-1] == s.cuda_stream][0]
    for step in range(3):
        out.fill_(7.0)
        lse.fill_(7.0)
        eager[:1024] = 255
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager[:1024] = 0
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), step
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            again = B.attn_decode(q, x.cache, x.table, x.seq, lse=True)
        torch.cuda.synchronize()
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_prepared_under_capture():
    """A call prepared inside a capture, called there, before that graph ever ran, in a second graph, and among replays."""
    dev = device()
    x = Batch(dev, B.NVFP4_KV_BF16, [4000, 0, 700], 10, 2, 128, 64, seed=6)
    q = x.q.to(dev)
    want = B.attn_decode(q, x.cache, x.table, x.seq, lse=True)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        call = B.attn_decode_prepared(q, x.cache, x.table, x.seq, lse=True)
        call()
    with torch.cuda.graph(second):
        out, lse = call()
    torch.cuda.synchronize()
    ws = call.keep[-1]
    for step in range(3):
        for run in (call, second.replay, first.replay, call):
            out.fill_(7.0)
            lse.fill_(7.0)
            if step == 0 and run is not first.replay:
                ws[:1024] = 255                 # as memory may be that nothing has written yet
            run()
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), (step, run)
    assert not ws[:1024].any()


def test_inputs_let_go_while_a_call_is_queued():
    """Calls told another stream than the current one; every input is dropped, and its memory asked for again, before they run."""
    dev = device()
    x = Batch(dev, B.NVFP4_KV_E4M3, [400, 37], 4, 2, 64, 64, seed=7)
    table = B.rope_table(64, device=dev)
    pos = torch.tensor([399, 36], dtype=torch.int32, device=dev)
    slots = torch.stack([x.table[i, p // 64].long() * 64 + p % 64 for i, p in enumerate((399, 36))])
    kv = torch.randn(2, 2, 64, device=dev).to(torch.bfloat16)
    q = x.q.to(dev)
    k, v = (t.clone() for t in B.kv_read(x.cache, slots))

    def chain(stream, *inputs):
        pool, table_pages, seq, turns, p, at, new, query = inputs
        cache = B.KvCache(x.cache.pages, 64, 2, 64, x.fmt, device=dev, pool=pool)
        rope = B.RopeTable(turns, 64, table.layout, table.magnitude)
        turned = B.kv_append(cache, new, new, at, positions=p, table=rope, q=query, stream=stream)
        return (B.rope(new, p, rope, stream=stream), turned, *B.kv_read(cache, at, stream=stream),
                *B.attn_decode(turned, cache, table_pages, seq, lse=True, stream=stream))

    inputs = [x.cache.pool, x.table, x.seq, table.freqs, pos, slots, kv, q]
    want = chain(None, *(t.clone() for t in inputs))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    copies = [t.clone() for t in inputs]
    sizes = [t.numel() * t.element_size() for t in copies]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20 * WAIT)
    got = chain(s, *copies)
    del copies
    taken = [torch.full((n,), 0, dtype=torch.uint8, device=dev) for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    del taken
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert not torch.equal(want[2], k) and not torch.equal(want[3], v)


def test_a_stream_of_another_device():
    """Refused, by every call that can be told its stream, before anything is made there or launched."""
    dev = device()

    class Elsewhere:
        device, cuda_stream = torch.device("cuda", torch.cuda.device_count()), 0

    s, table = Elsewhere(), B.rope_table(64, device=dev)
    cache = B.KvCache(2, 16, 1, 64, B.NVFP4_KV_BF16, device=dev)
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device=dev)
    ints, slots = torch.ones(2, dtype=torch.int32, device=dev), torch.zeros(2, dtype=torch.int64, device=dev)
    for call in (lambda: B.rope(x, ints, table, stream=s), lambda: B.kv_append(cache, x, x, slots, stream=s),
                 lambda: B.kv_read(cache, slots, stream=s),
                 lambda: B.attn_decode(x, cache, ints[:, None], ints, stream=s),
                 lambda: B.attn_decode_prepared(x, cache, ints[:, None], ints, stream=s)):
        with pytest.raises(ValueError, match="stream is on"):
            call()


def test_prepared_under_capture_in_inference_mode():
    """As a serving program does (torch wants graphs of that mode captured and replayed there); called outside it too."""
    dev = device()
    x = Batch(dev, B.NVFP4_KV_NVFP4, [4000, 0, 700], 10, 2, 128, 64, seed=8)
    q = x.q.to(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.inference_mode():
        want = B.attn_decode(q, x.cache, x.table, x.seq, lse=True)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            call = B.attn_decode_prepared(q, x.cache, x.table, x.seq, lse=True)
            out, lse = call()

    def replay():
        with torch.inference_mode():
            graph.replay()

    for run in (call, replay, replay, call, replay):
        with torch.inference_mode():
            out.fill_(7.0)
            lse.fill_(7.0)
        run()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), run


def test_a_prepared_call_let_go_while_it_is_queued():
    """Prepared on one stream and called on another; the callable, and with it its workspace, is dropped before the call has
    run, and its memory asked for again: neither the outputs nor what is made there meanwhile is touched."""
    dev = device()
    x = Batch(dev, B.NVFP4_KV_NVFP4, [9000, 0, 700], 10, 2, 128, 64, seed=9)
    q = x.q.to(dev)
    want = B.attn_decode(q, x.cache, x.table, x.seq, lse=True)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = B.attn_decode_prepared(q, x.cache, x.table, x.seq, lse=True)
    need = call.keep[-1].numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20 * WAIT)
        out, lse = call()
    del call
    taken = [torch.full((need,), 3, dtype=torch.uint8, device=dev) for _ in range(4)]
    torch.cuda.synchronize()
    assert all((t == 3).all() for t in taken)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
