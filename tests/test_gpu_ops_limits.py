"""The operators around the path at the ends of their ranges: more tokens than
one launch has threads for and than an int32 counts, windows that hold 8-bit
rows, and general products of more tiles than workgroups."""
import itertools

import numpy as np
import pytest
import torch

from tests import ops_ref as ref
from tests.gpu_util import make_moe, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def test_more_tokens_than_a_launch_has_threads(cco):
    # 64 lanes a token: from 2^26 tokens on one launch would need 2^32 threads
    T, E = 2 ** 26 + 77, 2
    say("case: route T=%d" % T)
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randint(-2, 3, (T, E), generator=g, device="cuda", dtype=torch.int8).to(BF)
    idx, w = cco.route(logits, 1, renorm=True)
    assert torch.equal(idx[:, 0] == 1, logits[:, 1] > logits[:, 0])  # equal: the lower id
    assert bool((w == 1.0).all())
    del w
    dw = torch.ones((T, 1), device="cuda")
    got = cco.route_grad(logits, idx, dw, score="sigmoid")
    # five distinct logits: sigmoid' of the chosen one, 0 for the other
    chosen = torch.gather(logits, 1, idx.long()).double()
    s = torch.sigmoid(chosen)
    want = s * (1 - s)
    # exp and two quotients in 32 bits, rounded once to bf16
    bound = want * (ref.half_step(BF) + 32 * ref.U)
    assert bool(((torch.gather(got, 1, idx.long()).double() - want).abs() <= bound).all())
    assert not bool(torch.gather(got, 1, 1 - idx.long()).any())


def test_tokens_past_the_counts_type_are_refused(cco):
    # 2^32 + 5 rows are not 5 rows
    x = torch.empty((2 ** 32 + 5, 1), dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        cco.route(x, 1)
    with pytest.raises(ValueError):
        cco.block_norm(x, pre=torch.ones(1, device="cuda"))


def test_window_of_8_bit_rows_is_refused(cco):
    from synth import get_config
    from synth.gen import activations, quantized_activations, routing
    cfg = get_config("tiny")
    idx, w = (torch.from_numpy(np.ascontiguousarray(v, t)).cuda()
              for v, t in zip(routing(cfg), (np.int32, np.float32)))
    x8, sc = (torch.from_numpy(v).cuda() for v in quantized_activations(cfg, None, block=64))
    x = activations(cfg).cuda()
    heap, moe = make_moe(cfg)
    with heap:
        moe.plan(idx)
        moe.dispatch(x, w)
        moe.window("disp_x", 0, 4)
        moe.dispatch_fp8(x8, sc, w)
        with pytest.raises(ValueError):
            moe.window("disp_x", 0, 4)
        with pytest.raises(ValueError):
            moe.window("disp_x", 1, 0)
        moe.window("out_tok", 0, 4)
        moe.window("hbuf", 0, 4)
        moe.dispatch(x, w)
        first, count = moe.expert_groups(0)
        rows = int(moe.status()[1][0])
        xs = moe.window("disp_x", 0, rows)
        tok = moe.read_rows("meta", 0, 0, rows)["src"] // cfg.K  # src is t * K + j
        assert torch.equal(xs.cpu(), x.cpu()[torch.from_numpy(tok.astype(np.int64))])


@pytest.mark.parametrize("counts,n,k,what", [
    ([3000, 0, 1, 2777, 130, 2100], 8501, 33, ("product",)),
    ([3000, 0, 1, 2777, 130, 2100], 33, 8501, ("dx",)),
    ([3000, 0, 1, 2777, 130, 2100], 8501, 5, ("product",)),
    ([70, 0, 1, 130, 64, 65, 3, 90, 127, 1], 2701, 2703, ("dw", "dw32")),
    ([70, 0, 1, 130, 64, 65, 3, 90, 127, 1, 0, 300], 7, 60001, ("dw", "dw32"))])
def test_general_products_of_more_tiles_than_workgroups(cco, counts, n, k, what):
    # rows that are no whole 16 bytes, over 4096 tiles of 128 x 128: a
    # workgroup's next tile takes the LDS its last results lay in
    ct = {"product": n, "dx": k}
    rows, G = sum(counts), len(counts)
    tiles = sum(-(-c // 128) for c in counts) * -(-ct.get(what[0], 1) // 128) \
        if what[0] in ct else G * -(-n // 128) * -(-k // 128)
    assert tiles > 4096
    first = [0] + list(itertools.accumulate(counts))[:-1]
    f, c = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (first, counts))
    gen = torch.Generator(device="cuda").manual_seed(n + k)

    def r(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(BF)

    say("case: general %s G=%d rows=%d n=%d k=%d tiles=%d" % (what, G, rows, n, k, tiles))
    x, dy = r(rows, k), r(rows, n)
    w = None if what[0] == "dw" else r(G, n, k)
    for name in what:
        if name == "product":
            def run(): return cco.group_product(f, c, x, w)
        elif name == "dx":
            def run(): return cco.group_product_dx(f, c, dy, w)
        else:
            dt = F32 if name == "dw32" else BF
            buf = torch.empty((G, n, k), dtype=dt, device="cuda")

            def run(): return cco.group_product_dw(f, c, dy, x, out=buf.fill_(float("nan")))
        got = run().clone()
        for g in range(G):
            lo, hi = first[g], first[g] + counts[g]
            if name == "product":
                a, b, t, o = x[lo:hi], w[g].t(), k, got[lo:hi]
            elif name == "dx":
                a, b, t, o = dy[lo:hi], w[g], n, got[lo:hi]
            else:
                a, b, t, o = dy[lo:hi].t(), x[lo:hi], hi - lo, got[g]
            v, s = ref.product(a.cpu(), b.cpu())
            ref.assert_within(o, v, ref.product_bound(v, s, t, got.dtype),
                              "%s group %d" % (name, g))
        for _ in range(3):
            assert torch.equal(run(), got)
