"""ace_matmul_i8 against 64-bit products.  The integer sum is exact; its fp32
conversion, the product of the scales (2 roundings) and the scaling take 4 half
steps of fp32, then one rounding to the output type."""
import numpy as np
import pytest
import torch

import i8_oracle as ora

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _q(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def _offsets(g, S, E, used=None):
    cut = torch.sort(torch.randint(0, (S if used is None else used) + 1, (E - 1,), generator=g, device="cuda")).values
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:E] = cut.to(torch.int32)
    off[E] = S if used is None else used
    return off


def _check(S, N, K, E=0, out="bf16", rows=None, gate=False, used=None, seed=0, offsets=None, row_of=None):
    from token_dynamic_expert_b200 import ace
    g = torch.Generator(device="cuda").manual_seed(seed + S + N + K)
    R = rows or S
    xq, wq = _q(g, R, K), _q(g, max(E, 1), N, K)
    xs, wsc = torch.rand(R, generator=g, device="cuda") + 0.1, torch.rand(max(E, 1), N, generator=g, device="cuda")
    if not E:
        wq, wsc = wq[0], wsc[0]
    off = (offsets if offsets is not None else _offsets(g, S, E, used)) if E else None
    if row_of is None and rows:
        row_of = torch.randint(0, R, (S,), generator=g, device="cuda", dtype=torch.int32)
    ss = torch.randn(S, generator=g, device="cuda") if gate else None
    y = torch.full((S, N), 7, dtype=DT[out], device="cuda")
    ws = torch.full((256,), 0xAB, dtype=torch.uint8, device="cuda")
    ace.ace_matmul_i8(xq, xs, wq, wsc, y, ws, offsets=off, row_of=row_of, slot_scale=ss)
    assert ace.ace_read_status(ws) == (ace.ACE_OK, 0)
    ref = ora.matmul(ora.f64(xq), ora.f64(xs), ora.f64(wq), ora.f64(wsc), None if off is None else off.tolist(),
                     None if row_of is None else row_of.cpu().numpy(), None if ss is None else ora.f64(ss), S=S)
    n = S if off is None else int(off[-1])
    assert ora.close(ora.f64(y)[:n], ref[:n], ora.HALF[out] + 4 * ora.U32) <= 1
    assert (y[n:] == 7).all()


@pytest.mark.parametrize("S,N,K", [(1, 1, 16), (1, 128, 128), (2, 129, 144), (8, 2048, 2048), (15, 100, 48),
                                   (16, 257, 512), (17, 64, 4096), (33, 1000, 320), (100, 130, 272),
                                   (257, 513, 400), (1000, 2000, 1040), (3001, 384, 656)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_dense(S, N, K, out):
    _check(S, N, K, out=out)


def test_dense_large_odd():
    _check(4099, 4097, 272, out="f32")


@pytest.mark.parametrize("S,N,K", [(4100, 4000, 1056), (4096, 4096, 1024), (4000, 4097, 1168)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_dense_large(S, N, K, out):
    _check(S, N, K, out=out)


@pytest.mark.parametrize("S,N,K,E", [(33000, 1030, 1040, 100), (40000, 768, 1024, 37), (70000, 300, 1152, 7),
                                     (30000, 1024, 3200, 256)])
@pytest.mark.parametrize("rows,gate", [(None, True), (900, False)])
def test_grouped_large(S, N, K, E, rows, gate):
    _check(S, N, K, E, rows=rows, gate=gate, used=S - 5)


@pytest.mark.parametrize("S,N,K,E", [(1, 128, 128, 4), (64, 1536, 512, 128), (61, 100, 144, 7), (500, 257, 256, 3),
                                     (3000, 384, 336, 64), (777, 96, 64, 512), (5000, 512, 128, 2)])
@pytest.mark.parametrize("rows,gate", [(None, False), (None, True), (97, False), (1, True)])
def test_grouped(S, N, K, E, rows, gate):
    _check(S, N, K, E, rows=rows, gate=gate)


def test_grouped_f32_with_rows_behind_the_last_slot():
    for used in (0, 1, 300, 511):
        _check(512, 200, 128, 9, out="f32", used=used)


def test_one_group_holds_everything_or_nothing():
    for off in ([0, 0, 0, 400], [0, 400, 400, 400], [0, 0, 399, 400]):
        _check(400, 192, 256, 3, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))


def test_row_map_repeats_and_leaves_the_range():
    r = torch.tensor([0, 0, 0, 5, -1, 6, 7, -2 ** 31, 2 ** 31 - 1, 2], dtype=torch.int32, device="cuda")
    _check(10, 130, 128, rows=6, row_of=r)


def test_extreme_values_do_not_wrap():
    """Every product 127^2 or -128 x -128 at the largest K that is allowed."""
    from token_dynamic_expert_b200 import ace
    K = 65536
    for a, b in ((127, 127), (-128, -128), (-128, 127)):
        xq = torch.full((3, K), a, dtype=torch.int8, device="cuda")
        wq = torch.full((5, K), b, dtype=torch.int8, device="cuda")
        y, ws = torch.empty(3, 5, device="cuda"), ace.alloc_workspace(256)
        ace.ace_matmul_i8(xq, torch.ones(3, device="cuda"), wq, torch.ones(5, device="cuda"), y, ws)
        assert (y == float(a * b * K)).all()  # a multiple of 2^16 below 2^31: exact in fp32


def test_bad_offsets_raise_the_flag_and_write_nothing():
    from token_dynamic_expert_b200 import ace
    xq, xs = torch.ones(40, 64, dtype=torch.int8, device="cuda"), torch.ones(40, device="cuda")
    wq, wsc = torch.ones(3, 96, 64, dtype=torch.int8, device="cuda"), torch.ones(3, 96, device="cuda")
    ws = ace.alloc_workspace(256)
    for off in ([0, 20, 10, 40], [1, 10, 20, 40], [0, 10, 20, 41], [0, -1, 20, 40], [0, 50, 20, 40], [0, 0, 0, -5]):
        y = torch.full((40, 96), 7.0, device="cuda")
        ace.ace_matmul_i8(xq, xs, wq, wsc, y, ws, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        assert ace.ace_read_status(ws) == (ace.ACE_ERR_DEVICE_FAULT, ace.ACE_FLAG_BAD_INDEX)
        assert (y == 7).all()
    y = torch.full((40, 96), 7.0, device="cuda")
    ace.ace_matmul_i8(xq, xs, wq, wsc, y, ws, offsets=torch.tensor([0, 3, 9, 40], dtype=torch.int32, device="cuda"))
    assert ace.ace_read_status(ws) == (ace.ACE_OK, 0) and (y == 64).all()


def test_strides_of_inputs_and_output():
    from token_dynamic_expert_b200 import ace
    g = torch.Generator(device="cuda").manual_seed(5)
    xbig, wq = _q(g, 70, 320), _q(g, 200, 256)
    xq = xbig[:, 32:288]
    xs, wsc = torch.rand(70, device="cuda"), torch.rand(200, device="cuda")
    ybig, ws = torch.full((70, 260), 7.0, device="cuda"), ace.alloc_workspace(256)
    ace.ace_matmul_i8(xq, xs, wq, wsc, ybig[:, 11:211], ws)
    ref = ora.matmul(ora.f64(xq), ora.f64(xs), ora.f64(wq), ora.f64(wsc))
    assert ora.close(ora.f64(ybig[:, 11:211]), ref, 5 * ora.U32) <= 1
    assert (ybig[:, :11] == 7).all() and (ybig[:, 211:] == 7).all()


def test_same_bits_again_and_in_a_graph():
    from token_dynamic_expert_b200 import ace
    g = torch.Generator(device="cuda").manual_seed(6)
    xq, wq = _q(g, 600, 256), _q(g, 8, 320, 256)
    xs, wsc = torch.rand(600, device="cuda"), torch.rand(8, 320, device="cuda")
    off, ws = _offsets(g, 600, 8), ace.alloc_workspace(256)
    a, b = torch.empty(600, 320, device="cuda"), torch.zeros(600, 320, device="cuda")
    ace.ace_matmul_i8(xq, xs, wq, wsc, a, ws, offsets=off)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        ace.ace_matmul_i8(xq, xs, wq, wsc, b, ws, offsets=off)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b)
