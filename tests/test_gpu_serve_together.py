"""The 8-bit operators as a layer uses them together: weights and rows
quantised, the rows dispatched as 8-bit rows and multiplied in the receive
windows, SwiGLU rows quantised for the down product into the staging windows,
combined; and the layer for a few tokens on the same weights, behind the norm
and the router."""
import pytest
import torch

from tests import ops_ref, serve_ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def _r(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def _weights(cco, E, H, I):
    """(w13, s13, w2, s2): bf16 weights quantised by rows, which are the
    products' columns."""
    w13, w2 = _r((E, 2 * I, H), 6, 0.05), _r((E, H, I), 7, 0.05)
    q13, s13 = cco.quant_rows(w13.view(-1, H))
    q2, s2 = cco.quant_rows(w2.view(-1, I))
    return q13.view(w13.shape), s13.view(E, 2 * I), q2.view(w2.shape), s2.view(E, H)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_an_8_bit_layer_in_the_windows(cco, T):
    H, K, E, S, I = 256, 2, 8, 4, 128
    say("case: 8-bit layer T=%d" % T)
    w13, s13, w2, s2 = _weights(cco, E, H, I)
    x = _r((T, H), 1)
    idx, w = cco.route(_r((T, E), 2, 1.0, torch.float32), K, renorm=True)
    q, s = cco.quant_rows(x)
    heap = cco.SymHeap(S, cco.required_slot_bytes(T, H, K, E, I, S))
    moe = cco.MoE(heap, T, H, K, E, I)
    with heap:
        with pytest.raises(ValueError):
            moe.window8(0, 0)
        moe.plan(idx)
        moe.dispatch_fp8(q, s[:, None], w)
        total = moe.status()[1]
        eps = moe.eps
        for slot in range(S):
            rows = int(total[slot])
            first, count = moe.expert_groups(slot)
            xq, xs = moe.window8(slot, rows)
            assert rows == 0 or xq.data_ptr() == moe.dispatch_view(slot)  # in place
            mine = slice(slot * eps, (slot + 1) * eps)
            gu = cco.group_product_i8(first, count, xq, xs[:, 0], w13[mine], s13[mine],
                                      dtype=torch.float32)
            hq, hs = cco.quant_swiglu(gu)
            cco.group_product_i8(first, count, hq, hs, w2[mine], s2[mine],
                                 out=moe.window("out_tok", slot, rows))
            # each product exactly, from the operands it was given
            f, c = first.tolist(), count.tolist()
            want = serve_ref.product_i8(f, c, xq.cpu(), xs[:, 0].cpu(), w13[mine].cpu(),
                                        s13[mine].cpu(), torch.zeros(rows, 2 * I).double())
            ops_ref.assert_within(gu, want, serve_ref.product_i8_bound(want, torch.float32), "gu")
            want = serve_ref.product_i8(f, c, hq.cpu(), hs.cpu(), w2[mine].cpu(), s2[mine].cpu(),
                                        torch.zeros(rows, H).double())
            ops_ref.assert_within(moe.window("out_tok", slot, rows), want,
                                  serve_ref.product_i8_bound(want, BF), "y")
        out, _ = moe.combine(w)
    # the whole against the layer of the same weights on the unquantised rows:
    # a row's error is half a step of 1/127 of its largest value, twice
    y, err = serve_ref.layer(x.cpu(), idx.cpu(), w.cpu(), w13.cpu(), w2.cpu(), s13.cpu(), s2.cpu())
    assert float((out.cpu().double() - y).abs().max()) <= 0.05 * float(y.abs().max())
    if T <= 64:
        few = cco.moe_few(x, idx, w, w13, w2, s13=s13, s2=s2)
        ops_ref.assert_within(few, y, serve_ref.layer_bound(y, err, BF), "few")


@pytest.mark.parametrize("T", [1, 7, 64])
def test_a_served_block_of_a_few_tokens(cco, T):
    H, K, E, I = 512, 3, 16, 256
    x = _r((T, H), 1)
    pre, post, nxt = (1 + _r(H, s, 0.1, torch.float32) for s in (2, 3, 4))
    wr, w13, w2 = _r((1, E, H), 5, 0.05), _r((E, 2 * I, H), 6, 0.05), _r((E, H, I), 7, 0.05)
    first, count = (torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, T))
    heap = cco.SymHeap(4, cco.required_slot_bytes(T, H, K, E, I, 4))
    moe = cco.MoE(heap, T, H, K, E, I)

    def block():
        _, u = cco.block_norm(x, pre=pre)
        idx, w = cco.route(cco.group_product(first, count, u, wr), K, score="sigmoid", renorm=True)
        y = cco.moe_few(u, idx, w, w13, w2)
        return (u, idx, w, y) + tuple(cco.block_norm(x, y, post=post, pre=nxt, scale=0.5))

    with heap:
        u, idx, w, y, out, un = block()
        y64, err = serve_ref.layer(u.cpu(), idx.cpu(), w.cpu(), w13.cpu(), w2.cpu(), None, None)
        ops_ref.assert_within(y, y64, serve_ref.layer_bound(y64, err, BF), "y")
        # the path's own layer rounds h and each expert's row to bf16
        moe.plan(idx)
        moe.dispatch(u, w)
        moe.expert(w13, w2)
        path, _ = moe.combine(w)
        assert float((path.float() - y.float()).abs().max()) <= 2e-2 * float(y64.abs().max())
    # captured, replayed between eager calls
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block()
    for seed in range(3):
        x.copy_(_r((T, H), 30 + seed))
        eager = block()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)


def test_two_layers_at_once(cco):
    # two streams, each with its own workspace
    c = [(_r((16, 1024), s), _r((8, 2048, 1024), s + 1, 0.05), _r((8, 1024, 1024), s + 2, 0.05))
         for s in (1, 10)]
    idx, w = cco.route(_r((16, 8), 20, 1.0, torch.float32), 2)
    want = [cco.moe_few(x, idx, w, a, b) for x, a, b in c]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in c]
    got = []
    for _ in range(4):
        got.append([cco.moe_few(x, idx, w, a, b, stream=s) for (x, a, b), s in zip(c, streams)])
    torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])
