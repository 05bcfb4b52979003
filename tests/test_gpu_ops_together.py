"""The operators as a layer uses them together: norm, router, the path with
the layer's experts, the fused combine with the norms around the next block;
and a training step of the same layer, its experts' products, their gradients
and the router's and norms' gradients against 64-bit differentiation."""
import numpy as np
import pytest
import torch

from tests import ops_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def _r(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def _layer(cco, T, H, K, E, S, I):
    heap = cco.SymHeap(S, cco.required_slot_bytes(T, H, K, E, I, S))
    return heap, cco.MoE(heap, T, H, K, E, I)


@pytest.mark.parametrize("T", [1, 7, 200])
def test_a_served_block(cco, T):
    H, K, E, S, I = 512, 3, 16, 4, 256
    heap, moe = _layer(cco, T, H, K, E, S, I)
    with heap:
        say("case: served block T=%d" % T)
        x = _r((T, H), 1)
        pre, post, nxt = (1 + _r(H, s, 0.1, torch.float32) for s in (2, 3, 4))
        wr = _r((1, E, H), 5, 0.05)
        w13, w2 = _r((E, 2 * I, H), 6, 0.05), _r((E, H, I), 7, 0.05)
        first, count = (torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, T))
        _, u = cco.block_norm(x, pre=pre)
        logits = cco.group_product(first, count, u, wr)  # one group: a dense product
        idx, w = cco.route(logits, K, score="sigmoid", renorm=True)
        moe.plan(idx)
        moe.dispatch(u, w)
        moe.expert(w13, w2)
        out, un, y = cco.combine_norm(moe, x, w, post=post, pre=nxt, scale=0.5, keep_y=True)
        assert moe.status()[0] == cco.CCO_OK
        # each stage from what the one before left, in 64 bits
        _, u64 = ref.block(x.cpu().double(), None, None, None, pre.cpu().double(), 1.0, EPS)
        assert bool(((u.cpu().double() - u64).abs() <=
                     (2.0 ** -8 + 1e-5) * u64.abs() + 1e-30).all())
        lv, ls = ref.product(u.cpu(), wr[0].cpu().t())
        ref.assert_within(logits, lv, ref.product_bound(lv, ls, H, BF), "logits")
        assert idx.cpu().tolist() == ref.choose(logits.cpu(), K, "sigmoid", None, 1, 1)
        y64 = torch.zeros(T, H, dtype=torch.float64)
        for t in range(T):
            for j in range(K):
                e = int(idx[t, j])
                gu = w13[e].cpu().double() @ u[t].cpu().double()
                h = torch.nn.functional.silu(gu[:I]) * gu[I:]
                y64[t] += float(w[t, j]) * (w2[e].cpu().double() @ h)
        err = (y.cpu().double() - y64).abs().max()
        # the layer's own tolerance (bf16 intermediate rows)
        assert float(err) <= 2e-2 * float(y64.abs().max())
        want = cco.block_norm(x, y, post=post, pre=nxt, scale=0.5)
        assert torch.equal(out, want[0]) and torch.equal(un, want[1])


def test_products_on_the_layers_windows(cco):
    # the routing state is the groups: a slot's experts on its receive rows
    T, H, K, E, S, I = 300, 256, 4, 12, 3, 128
    heap, moe = _layer(cco, T, H, K, E, S, I)
    with heap:
        logits = _r((T, E), 1, 1.0, torch.float32)
        idx, w = cco.route(logits, K)
        x = _r((T, H), 2)
        w13, w2 = _r((E, 2 * I, H), 3, 0.05), _r((E, H, I), 4, 0.05)
        moe.plan(idx)
        moe.dispatch(x, w)
        moe.expert(w13, w2)
        for s in range(S):
            say("case: slot %d" % s)
            first, count = moe.expert_groups(s)
            rows = int(moe.status()[1][s])
            xs, hs, ys = (moe.window(n, s, rows) for n in ("disp_x", "hbuf", "out_tok"))
            assert xs.data_ptr() == moe.dispatch_view(s)
            eps = moe.eps
            gu = cco.group_product(first, count, xs, w13[s * eps:(s + 1) * eps])
            g, u = gu.float().chunk(2, 1)
            h = torch.nn.functional.silu(g) * u
            assert float((hs.float() - h).abs().max()) <= 2e-2 * float(h.abs().max())
            y = cco.group_product(first, count, hs, w2[s * eps:(s + 1) * eps])
            # the same sums of the same rows: one step of bf16 at most
            d = (y.float() - ys.float()).abs()
            assert bool((d <= 2.0 ** -7 * ys.float().abs() + 1e-3 * ys.float().abs().max()).all())


def test_a_training_step(cco):
    """Forward and backward of norm -> router -> experts (SwiGLU) -> combine
    -> norm, with gate and residual, the rows sorted by expert; gradients of
    every parameter against 64-bit differentiation of the same block at the
    rows the kernels were given."""
    T, H, K, E, I = 150, 256, 2, 6, 128
    x = _r((T, H), 1)
    pre, post, gate = (1 + _r(H, s, 0.1, torch.float32) for s in (2, 3, 4))
    wr = _r((1, E, H), 5, 0.08)
    w13, w2 = _r((E, 2 * I, H), 6, 0.08), _r((E, H, I), 7, 0.08)
    dout = _r((T, H), 8)
    one_f, one_c = (torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, T))
    # ---- forward
    _, u = cco.block_norm(x, pre=pre)
    logits = cco.group_product(one_f, one_c, u, wr)
    idx, w = cco.route(logits, K, score="softmax", renorm=True, scale=1.5)
    order = torch.argsort(idx.flatten().long(), stable=True)
    count = torch.bincount(idx.flatten().long(), minlength=E).to(torch.int32)
    first = (torch.cumsum(count, 0) - count).to(torch.int32)
    tok = order // K
    xs = u[tok].contiguous()
    gu = cco.group_product(first, count, xs, w13)
    g, up = gu.float().chunk(2, 1)
    h = (torch.nn.functional.silu(g) * up).to(BF)
    ys = cco.group_product(first, count, h, w2)
    wrow = w.flatten()[order]
    y = torch.zeros(T, H, device="cuda").index_add_(0, tok, ys.float() * wrow[:, None]).to(BF)
    out, _ = cco.block_norm(x, y, post=post, gate=gate, scale=0.5)
    # ---- backward
    dx, dy, dpost, dgate, _ = cco.block_norm_grad(x, y, dout, None, post=post, gate=gate, scale=0.5)
    dyrow = dy[tok].float()
    dw = torch.empty(T * K, device="cuda")
    dw[order] = (dyrow * ys.float()).sum(1)
    dys = (dyrow * wrow[:, None]).to(BF)
    dh = cco.group_product_dx(first, count, dys, w2).float()
    dw2 = cco.group_product_dw(first, count, dys, h, out=torch.empty(E, H, I, device="cuda"))
    sg = torch.sigmoid(g)
    dgu = torch.cat([dh * up * sg * (1 + g * (1 - sg)), dh * g * sg], 1).to(BF)
    dw13 = cco.group_product_dw(first, count, dgu, xs, out=torch.empty(E, 2 * I, H, device="cuda"))
    dxs = cco.group_product_dx(first, count, dgu, w13).float()
    dlogits = cco.route_grad(logits, idx, dw.view(T, K), score="softmax", renorm=True, scale=1.5)
    dwr = cco.group_product_dw(one_f, one_c, dlogits, u, out=torch.empty(1, E, H, device="cuda"))
    du = torch.zeros(T, H, device="cuda").index_add_(0, tok, dxs)
    du = (du + cco.group_product_dx(one_f, one_c, dlogits, wr).float()).to(BF)
    dx2, _, _, _, dpre = cco.block_norm_grad(x, None, None, du, pre=pre)
    dx = dx.float() + dx2.float()
    # ---- 64 bits, the same choice of experts
    v = {n: t.cpu().double().requires_grad_(True) for n, t in
         dict(x=x, pre=pre, post=post, gate=gate, wr=wr[0], w13=w13, w2=w2).items()}
    _, u64 = ref.block(v["x"], None, None, None, v["pre"], 1.0, EPS)
    ids = idx.cpu().long()
    w64 = ref.weights(u64 @ v["wr"].t(), ids, "softmax", True, 1.5)
    y64 = torch.zeros(T, H, dtype=torch.float64)
    rows = []
    for t in range(T):
        acc = 0
        for j in range(K):
            e = int(ids[t, j])
            gu64 = v["w13"][e] @ u64[t]
            hh = torch.nn.functional.silu(gu64[:I]) * gu64[I:]
            acc = acc + w64[t, j] * (v["w2"][e] @ hh)
        rows.append(acc)
    y64 = torch.stack(rows)
    o64, _ = ref.block(v["x"], y64, v["post"], v["gate"], None, 0.5, EPS)
    names = list(v)
    want = dict(zip(names, torch.autograd.grad(o64, [v[n] for n in names], dout.cpu().double())))
    got = dict(x=dx, pre=dpre, post=dpost, gate=dgate, wr=dwr[0], w13=dw13, w2=dw2)
    # Eight roundings to bf16 (2^-8 each) lie between the rows and a
    # gradient: u, logits, gu, h, ys, y, dy and dys (or dgu).  Each changes a
    # gradient by up to 2^-8 of its size, and they add up like independent
    # errors in the norm of a tensor: sqrt(8) 2^-8 = 0.011, doubled for the
    # products in which two rounded factors meet.
    for n in names:
        err = float((got[n].cpu().double() - want[n]).norm() / want[n].norm())
        say("  %s: relative error %.2e" % (n, err))
        assert err <= 0.023, (n, err)


def test_the_whole_block_in_a_graph(cco):
    T, H, K, E, S, I = 64, 256, 2, 8, 4, 128
    heap, moe = _layer(cco, T, H, K, E, S, I)
    with heap:
        x = _r((T, H), 1)
        pre, nxt = (1 + _r(H, s, 0.1, torch.float32) for s in (2, 3))
        wr = _r((1, E, H), 5, 0.05)
        w13, w2 = _r((E, 2 * I, H), 6, 0.05), _r((E, H, I), 7, 0.05)
        f, c = (torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, T))

        def block():
            _, u = cco.block_norm(x, pre=pre)
            logits = cco.group_product(f, c, u, wr)
            idx, w = cco.route(logits, K, renorm=True)
            moe.plan(idx)
            moe.dispatch(u, w)
            moe.expert(w13, w2)
            return cco.combine_norm(moe, x, w, pre=nxt)[:2]

        block()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, un = block()
        for i in range(3):
            x.copy_(_r((T, H), 20 + i))
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone(), un.clone()
            want = block()
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_binding_refusals_on_the_device(cco):
    x = _r((4, 16), 1)
    f = torch.zeros(2, dtype=torch.int32, device="cuda")
    w = _r((2, 8, 16), 2)
    bad = [lambda: cco.group_product(f, f[:1], x, w),
           lambda: cco.group_product(f, f, x, w[:1]),
           lambda: cco.group_product(f, f, x, w.half()),
           lambda: cco.group_product(f, f, x.float(), w.float()),
           lambda: cco.group_product(f.long(), f, x, w),
           lambda: cco.group_product(f, f, x.t(), w),
           lambda: cco.group_product(f, f, x[:1].expand(4, 16), w),
           lambda: cco.group_product(f, f, x, w, out=x),
           lambda: cco.group_product_dw(f, f, x, x, accumulate=True),
           lambda: cco.group_product_dw(f, f, x, x[:2]),
           lambda: cco.route(x, 2, score="top"),
           lambda: cco.route(x, 2, bias=torch.zeros(3, device="cuda")),
           lambda: cco.route(x.long(), 2),
           lambda: cco.block_norm(x, x, post=torch.ones(8, device="cuda")),
           lambda: cco.block_norm(x, x[:2]),
           lambda: cco.block_norm(x, x, gate=torch.ones(16, device="cuda"),
                                  token_gate=torch.ones(4, device="cuda")),
           lambda: cco.block_norm(x, x, post=torch.ones(16, device="cuda"),
                                  pre=torch.ones(16, device="cuda", dtype=BF)),
           lambda: cco.block_norm(x, x, pre=torch.ones(16, device="cuda", dtype=torch.float16)),
           lambda: cco.block_norm(x.t(), x.t())]
    for i, fn in enumerate(bad):
        with pytest.raises(ValueError):
            fn()
            pytest.fail("call %d was accepted" % i)
    for fn in (lambda: cco.route(x, 17), lambda: cco.route(x, 0),
               lambda: cco.route(x, 2, groups=3), lambda: cco.block_norm(x),
               lambda: cco.block_norm_grad(x, x, None, None)):
        with pytest.raises(cco.CcoError):
            fn()
