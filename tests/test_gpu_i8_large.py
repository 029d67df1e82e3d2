"""The 8-bit layer's operators where an offset passes 32 bits, where calls overlap
in time, and where they replay in one graph.  Tolerances as in each operator's
own tests."""
import numpy as np
import pytest
import torch

import i8_oracle as ora

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def test_norm_rows_beyond_32_bits():
    from token_dynamic_expert_b200 import ace
    T, d = 2 ** 18 + 3, 16384                       # 4.3e9 elements
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(5, d, device="cuda").bfloat16()
    x.zero_()
    x[-5:] = tail
    q, qs = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    gamma = torch.rand(d, device="cuda") + 0.5
    ace.ace_add_rmsnorm(x, gamma, q=q, q_scale=qs, y=x)
    y, rq, rs = ora.norm(ora.f64(tail), ora.f64(gamma), 1e-6)
    assert np.array_equal(q[-5:].cpu().numpy(), rq)
    assert ora.close(ora.f64(qs[-5:]), rs, 24 * ora.U32) <= 1
    assert ora.close(ora.f64(x[-5:]), y, ora.HALF["bf16"] + 24 * ora.U32, 1e-38) <= 1
    assert not q[:-5].any() and not qs[:-5].any()


def test_swiglu_stride_beyond_32_bits():
    from token_dynamic_expert_b200 import ace
    ld = 2 ** 31 + 8
    buf = torch.empty(2 * ld + 128, dtype=torch.bfloat16, device="cuda")
    gu = buf.as_strided((3, 128), (ld, 1))
    gu.copy_(torch.randn(3, 128, device="cuda"))
    q, qs = torch.empty(3, 64, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    ace.ace_swiglu(gu, q=q, q_scale=qs)
    _, rq, rs = ora.swiglu(ora.f64(gu))
    assert np.array_equal(q.cpu().numpy(), rq) and ora.close(ora.f64(qs), rs, 13 * ora.U32) <= 1


def test_gate_stride_beyond_32_bits():
    from token_dynamic_expert_b200 import ace
    ld = 2 ** 30 + 4
    buf = torch.empty(4 * ld + 64, device="cuda")
    x = buf.as_strided((5, 64), (ld, 1))
    x.copy_(torch.randn(5, 64, device="cuda"))
    idx, w = torch.empty(5, 8, dtype=torch.int32, device="cuda"), torch.empty(5, 8, device="cuda")
    ace.ace_gate_topk(x, idx, w, score="sigmoid", n_groups=4, topk_groups=2)
    ri, _ = ora.gate(ora.f64(x), 8, score="sigmoid", n_groups=4, topk_groups=2)
    assert np.array_equal(idx.cpu().numpy(), ri)


def test_product_weights_and_outputs_beyond_32_bits():
    from token_dynamic_expert_b200 import ace
    g = torch.Generator(device="cuda").manual_seed(1)
    E, N, K = 512, 4112, 2176                       # 4.6e9 bytes of weights
    wq = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
    wq[-1] = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    wsc = torch.rand(E, N, generator=g, device="cuda")
    xq = torch.randint(-128, 128, (9, K), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = torch.rand(9, generator=g, device="cuda"), ace.alloc_workspace(256)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = 9
    y = torch.empty(9, N, device="cuda")
    ace.ace_matmul_i8(xq, xs, wq, wsc, y, ws, offsets=off)
    assert ace.ace_read_status(ws) == (ace.ACE_OK, 0)
    ref = ora.matmul(ora.f64(xq), ora.f64(xs), ora.f64(wq[-1]), ora.f64(wsc[-1]))
    assert ora.close(ora.f64(y), ref, 5 * ora.U32) <= 1
    del wq
    S = 1050000                                     # 4.3e9 outputs
    wq, wsc = torch.randint(-128, 128, (N, 64), generator=g, device="cuda", dtype=torch.int8), wsc[0].contiguous()
    xq = torch.randint(-128, 128, (S, 64), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(S, generator=g, device="cuda")
    y = torch.empty(S, N, dtype=torch.bfloat16, device="cuda")
    ace.ace_matmul_i8(xq, xs, wq, wsc, y, ws)
    assert ace.ace_read_status(ws) == (ace.ACE_OK, 0)
    for sl in (slice(0, 7), slice(S // 2, S // 2 + 7), slice(S - 7, S)):
        ref = ora.matmul(ora.f64(xq[sl]), ora.f64(xs[sl]), ora.f64(wq), ora.f64(wsc))
        assert ora.close(ora.f64(y[sl]), ref, ora.HALF["bf16"] + 4 * ora.U32) <= 1


def test_group_many_tokens():
    from token_dynamic_expert_b200 import ace
    T, k, E = 400000, 5, 77
    idx = torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32)
    off, so = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    ace.ace_moe_group(idx, E, off, so)
    roff, rso, _ = ora.group(idx.cpu().numpy(), None, E)
    assert np.array_equal(off.cpu().numpy(), roff) and np.array_equal(so.cpu().numpy(), rso)


def test_calls_that_overlap_on_two_streams():
    """Two products, two gates and two groupings at once, each on its own buffers."""
    from token_dynamic_expert_b200 import ace
    g = torch.Generator(device="cuda").manual_seed(2)
    sets = []
    for i in range(2):
        xq = torch.randint(-128, 128, (3000, 512), generator=g, device="cuda", dtype=torch.int8)
        wq = torch.randint(-128, 128, (16, 1024, 512), generator=g, device="cuda", dtype=torch.int8)
        xs, wsc = torch.rand(3000, generator=g, device="cuda"), torch.rand(16, 1024, generator=g, device="cuda")
        off = torch.linspace(0, 3000, 17, device="cuda").to(torch.int32)
        row = torch.randint(0, 3000, (3000,), generator=g, device="cuda", dtype=torch.int32)
        logits = torch.randn(3000, 64, generator=g, device="cuda")
        sets.append(dict(a=(xq, xs, wq, wsc), kw=dict(offsets=off, row_of=row), ws=ace.alloc_workspace(256),
                         logits=logits, bias=torch.rand(64, device="cuda")))
    torch.cuda.synchronize()

    def run(s):
        y = torch.empty(3000, 1024, device="cuda")
        idx, w = torch.empty(3000, 4, dtype=torch.int32, device="cuda"), torch.empty(3000, 4, device="cuda")
        off, so = torch.empty(65, dtype=torch.int32, device="cuda"), torch.empty(3000, 4, dtype=torch.int32, device="cuda")
        for _ in range(8):
            ace.ace_matmul_i8(*s["a"], y, s["ws"], **s["kw"])
            ace.ace_gate_topk(s["logits"], idx, w, bias=s["bias"], score="sigmoid")
            ace.ace_moe_group(idx, 64, off, so)
        return y, idx, w, off, so

    alone = [run(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    both = []
    for s, st in zip(sets, streams):
        with torch.cuda.stream(st):
            both.append(run(s))
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_captured_products_share_a_workspace():
    """The workspace holds only the status word: graphs that share it replay one
    after the other with the same results."""
    from token_dynamic_expert_b200 import ace
    g = torch.Generator(device="cuda").manual_seed(3)
    ws, graphs, outs, refs = ace.alloc_workspace(256), [], [], []
    for S, N, K in ((300, 384, 256), (5, 1000, 512)):
        xq = torch.randint(-128, 128, (S, K), generator=g, device="cuda", dtype=torch.int8)
        wq = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
        xs, wsc, y = torch.rand(S, device="cuda"), torch.rand(N, device="cuda"), torch.zeros(S, N, device="cuda")
        ace.ace_matmul_i8(xq, xs, wq, wsc, y, ws)
        refs.append(y.clone())
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            ace.ace_matmul_i8(xq, xs, wq, wsc, y, ws)
        y.zero_()
        graphs.append((gr, xq, wq, xs, wsc))
        outs.append(y)
    for _ in range(3):
        for gr, *_ in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, refs))
    assert ace.ace_read_status(ws) == (ace.ACE_OK, 0)
