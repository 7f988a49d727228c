"""Products grouped by expert against products in 64 bits. Whole numbers of few digits make every sum
exact in fp32, so that the result is the exact one rounded once, whatever the order of the sum: those
are compared for equality. For real values an fp32 sum of K terms in steps of 16, each of which may
lose four units in the last place of what it holds (aligned and cut by the tensor cores), is at most
(K / 16 + 16) 2^-22 of the sum of the magnitudes off, and half a step of the type more."""
import pytest
import torch

from moe_expert_router_gb300 import binding as B

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def whole(gen, shape, dtype, top=2):
    return torch.randint(-top, top + 1, shape, generator=gen, device=DEV).to(dtype)


def offsets_of(counts, start=0):
    o = [start]
    for n in counts:
        o.append(o[-1] + n)
    return torch.tensor(o, dtype=torch.int32, device=DEV), o


def wide(t, pad):
    """The same values with rows `pad` elements further apart, NaN between them."""
    out = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
    out[:, :t.shape[1]] = t
    return out[:, :t.shape[1]]


COUNTS = [[1], [5], [0, 3, 0, 0, 1], [127, 128, 129], [255, 0, 256, 257], [1] * 37, [600, 2, 33], [0, 0], [64, 65, 63, 1],
          [31, 32, 33, 200, 0, 7], [513]]
SIZES = [(8, 8), (64, 256), (72, 264), (264, 520), (136, 40), (512, 128), (1408, 300 * 8)]


def run(x, w, offsets, out, transposed=False, **kw):
    ws = B.grouped_workspace(w.shape[0])
    B.moe_grouped_mm(x, w, offsets, out, ws, transposed=transposed, **kw)
    assert B.moe_get_device_error(ws) == 0
    return out


@pytest.mark.parametrize("K,N", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_products_and_gradients_of_whole_numbers(K, N, dtype):
    gen = torch.Generator(DEV).manual_seed(K + N)
    for i, counts in enumerate(COUNTS):
        start, tail, pad = (0, 0, 0) if i % 2 == 0 else (3, 5, 8)
        G = len(counts)
        offsets, o = offsets_of(counts, start)
        R = o[-1] + tail
        x, dy = whole(gen, (R, K), dtype), whole(gen, (R, N), dtype)
        if start:                                           # rows of no group hold anything
            x[:start], x[o[-1]:] = float("nan"), float("inf")
            dy[:start], dy[o[-1]:] = float("inf"), float("nan")
        w = whole(gen, (G, N, K), dtype)
        x, dy = wide(x, pad), wide(dy, pad)
        want = torch.full((R, N), 77.0, dtype=dtype, device=DEV)
        want_dx = torch.full((R, K), 77.0, dtype=dtype, device=DEV)
        want_dw = torch.zeros((G, N, K), dtype=dtype, device=DEV)
        for g in range(G):
            a, b = o[g], o[g + 1]
            want[a:b] = (x[a:b].double() @ w[g].double().t()).to(dtype)
            want_dx[a:b] = (dy[a:b].double() @ w[g].double()).to(dtype)
            want_dw[g] = (dy[a:b].double().t() @ x[a:b].double()).to(dtype)
        w_t = w.transpose(1, 2).contiguous()
        for t, matrix in ((False, w), (True, w_t)):
            out = wide(torch.full((R, N), 77.0, dtype=dtype, device=DEV), pad)
            assert torch.equal(run(x, matrix, offsets, out, t), want), (counts, t)
            dx = wide(torch.full((R, K), 77.0, dtype=dtype, device=DEV), pad)
            assert torch.equal(run(dy, matrix, offsets, dx, not t), want_dx), (counts, t)
            if pad:                                         # nothing is written between the rows
                assert torch.isnan(out.as_strided((R, pad), (N + pad, 1), N)).all()
        ws = B.grouped_workspace(G)
        dw = torch.full((G, N, K), 77.0, dtype=dtype, device=DEV)
        B.moe_grouped_wgrad(dy, x, offsets, dw, ws)
        assert torch.equal(dw, want_dw), counts
        dw = torch.full((G, K, N), 77.0, dtype=dtype, device=DEV)
        B.moe_grouped_wgrad(x, dy, offsets, dw, ws)
        assert torch.equal(dw, want_dw.transpose(1, 2)), counts
        assert B.moe_get_device_error(ws) == 0


@pytest.mark.parametrize("R,G", [(1, 1), (8, 32), (5, 64), (2, 3), (16, 8), (17, 8), (32, 256), (33, 300), (40, 2)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_few_rows(R, G, dtype):
    """Single tokens: a few rows spread over many groups, or in one."""
    gen = torch.Generator(DEV).manual_seed(R * G)
    for K, N in ((8, 8), (520, 72), (2048, 264), (1400, 136)):
        for spread in (True, False):
            counts = [0] * G
            for r in range(R):
                counts[(r * 7919) % G if spread else G // 2] += 1
            offsets, o = offsets_of(counts)
            x, w = whole(gen, (R, K), dtype), whole(gen, (G, N, K), dtype)
            want = torch.empty((R, N), dtype=dtype, device=DEV)
            for g in range(G):
                want[o[g]:o[g + 1]] = (x[o[g]:o[g + 1]].double() @ w[g].double().t()).to(dtype)
            for t, matrix in ((False, w), (True, w.transpose(1, 2).contiguous())):
                out = torch.full((R, N), 77.0, dtype=dtype, device=DEV)
                assert torch.equal(run(x, matrix, offsets, out, t), want), (K, N, spread, t)


@pytest.mark.parametrize("counts", [[64], [0, 17, 0, 30], [9, 8, 7, 0, 16, 1], [1] * 100 + [56] + [0] * 27, [2] * 128, [16, 48]])
def test_few_rows_of_groups_of_several(counts):
    """Around the borders of the few-row kernel: groups that take several of its blocks, rows of no group,
    NaN in those and between rows, bad offsets."""
    gen = torch.Generator(DEV).manual_seed(len(counts))
    for start, pad, K, N in ((0, 0, 264, 40), (3, 8, 72, 1032)):
        offsets, o = offsets_of(counts, start)
        R, G = o[-1] + 2, len(counts)
        x = whole(gen, (R, K), BF16)
        x[:start], x[o[-1]:] = float("nan"), float("inf")
        x, w = wide(x, pad), whole(gen, (G, N, K), BF16)
        want = torch.full((R, N), 77.0, dtype=BF16, device=DEV)
        for g in range(G):
            want[o[g]:o[g + 1]] = (x[o[g]:o[g + 1]].double() @ w[g].double().t()).to(BF16)
        out = wide(torch.full((R, N), 77.0, dtype=BF16, device=DEV), pad)
        assert torch.equal(run(x, w, offsets, out), want)
        bad = offsets.clone()
        bad[-1] = R + 1
        out.fill_(77.0)
        ws = B.grouped_workspace(G)
        B.moe_grouped_mm(x, w, bad, out, ws)
        assert B.moe_get_device_error(ws) == B.DEVERR_BAD_OFFSETS and (out == 77).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_real_values(dtype):
    gen = torch.Generator(DEV).manual_seed(1)
    for counts, K, N in (([300, 0, 41, 700], 1032, 776), ([1, 3, 0, 2], 4096, 520)):
        offsets, o = offsets_of(counts)
        R, G = o[-1], len(counts)
        x, dy = torch.randn((R, K), generator=gen, device=DEV).to(dtype), torch.randn((R, N), generator=gen, device=DEV).to(dtype)
        w = torch.randn((G, N, K), generator=gen, device=DEV).to(dtype)
        out = run(x, w, offsets, torch.empty((R, N), dtype=dtype, device=DEV))
        dx = run(dy, w, offsets, torch.empty((R, K), dtype=dtype, device=DEV), True)
        dw = torch.empty_like(w)
        B.moe_grouped_wgrad(dy, x, offsets, dw, B.grouped_workspace(G))
        for g in range(G):
            a, b = o[g], o[g + 1]
            X, D, W = x[a:b].double(), dy[a:b].double(), w[g].double()
            for got, l, r in ((out[a:b], X, W.t()), (dx[a:b], D, W), (dw[g], D.t(), X)):
                want, size = l @ r, l.abs() @ r.abs()
                bound = torch.finfo(dtype).eps / 2 * want.abs() + (l.shape[1] / 16 + 16) * 2.0 ** -22 * size
                assert ((got.double() - want).abs() <= bound + 1e-7).all()


def quantized(v):
    rows, cols = v.reshape(-1, v.shape[-1]).shape
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
    scales = B.mx_scales_empty((rows, cols), DEV)
    B.moe_mx_quantize(v.reshape(rows, cols).contiguous(), codes, scales)
    return codes.view(v.shape), scales


@pytest.mark.parametrize("K,N", [(128, 8), (256, 520), (1408, 224), (512, 232), (128, 448)])
def test_mxfp8_of_whole_numbers(K, N):
    """Numbers up to 8 times powers of two for each block are exact in MXFP8."""
    gen = torch.Generator(DEV).manual_seed(K + N)
    for i, counts in enumerate(COUNTS):
        start, tail = (0, 0) if i % 2 == 0 else (3, 5)
        offsets, o = offsets_of(counts, start)
        R, G = o[-1] + tail, len(counts)
        x, w = whole(gen, (R, K), BF16, 8), whole(gen, (G, N, K), BF16, 8)
        x.mul_(torch.exp2(torch.randint(-2, 3, (R, K // 32, 1), generator=gen, device=DEV).float()).expand(-1, -1, 32).reshape(R, K).to(BF16))
        w[0] *= 4
        xc, xs = quantized(x)
        wc, wss = quantized(w)
        if start:
            xc[:start], xc[o[-1]:] = 0x7f, 0xff             # NaN in rows of no group
        want = torch.full((R, N), 77.0, dtype=BF16, device=DEV)
        for g in range(G):
            want[o[g]:o[g + 1]] = (x[o[g]:o[g + 1]].double() @ w[g].double().t()).float().to(BF16)
        out = wide(torch.full((R, N), 77.0, dtype=BF16, device=DEV), 8 if start else 0)
        ws = B.grouped_workspace(G)
        B.moe_grouped_mm_mx(xc, xs, wc, wss, offsets, out, ws)
        assert B.moe_get_device_error(ws) == 0
        assert torch.equal(out, want), counts


@pytest.mark.parametrize("bad", [[0, 5, 3, 10], [0, 5, 7, 11], [-1, 5, 7, 10], [0, 2**31 - 1, 0, 10]])
def test_bad_offsets_compute_nothing(bad):
    x, w = torch.ones((10, 64), dtype=BF16, device=DEV), torch.ones((3, 72, 64), dtype=BF16, device=DEV)
    offsets = torch.tensor(bad, dtype=torch.int32, device=DEV)
    out, ws = torch.full((10, 72), 77.0, dtype=BF16, device=DEV), B.grouped_workspace(3)
    B.moe_grouped_mm(x, w, offsets, out, ws)
    assert B.moe_get_device_error(ws) == B.DEVERR_BAD_OFFSETS and (out == 77).all()
    dw = torch.full_like(w, 77.0)
    B.moe_grouped_wgrad(out, x, offsets, dw, ws)
    assert B.moe_get_device_error(ws) == B.DEVERR_BAD_OFFSETS and (dw == 0).all()
    good = torch.tensor([0, 5, 7, 10], dtype=torch.int32, device=DEV)
    out.fill_(77)
    B.moe_grouped_mm(x, w.transpose(1, 2).contiguous(), offsets, out, ws, transposed=True)
    assert B.moe_get_device_error(ws) == B.DEVERR_BAD_OFFSETS and (out == 77).all()
    w.fill_(1)
    B.moe_grouped_mm(x, w, good, out, ws)
    assert B.moe_get_device_error(ws) == 0 and (out == 64).all()
    xc, xs = quantized(torch.ones((10, 128), dtype=BF16, device=DEV))
    wc, wss = quantized(torch.ones((3, 72, 128), dtype=BF16, device=DEV))
    out.fill_(77)
    B.moe_grouped_mm_mx(xc, xs, wc, wss, offsets, out, ws)
    assert B.moe_get_device_error(ws) == B.DEVERR_BAD_OFFSETS and (out == 77).all()
    B.moe_grouped_mm_mx(xc, xs, wc, wss, good, out, ws)
    assert B.moe_get_device_error(ws) == 0 and (out == 128).all()


@pytest.mark.parametrize("rows", [50, 900, 3000])
def test_the_most_groups(rows):
    gen = torch.Generator(DEV).manual_seed(rows)
    G, K, N = 1024, 136, 72
    counts = torch.bincount(torch.randint(0, G, (rows,), generator=gen, device=DEV) ** 2 // G, minlength=G)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    group = torch.repeat_interleave(torch.arange(G, device=DEV), counts)
    x, dy, w = whole(gen, (rows, K), BF16), whole(gen, (rows, N), BF16), whole(gen, (G, N, K), BF16)
    want = torch.einsum("rk,rnk->rn", x.float(), w.float()[group]).to(BF16)
    dx = torch.einsum("rn,rnk->rk", dy.float(), w.float()[group]).to(BF16)
    assert torch.equal(run(x, w, offsets, torch.empty_like(dy)), want)
    assert torch.equal(run(dy, w, offsets, torch.empty_like(x), True), dx)
    dw, ws = torch.empty_like(w), B.grouped_workspace(G)
    B.moe_grouped_wgrad(dy, x, offsets, dw, ws)
    want = torch.zeros((G, N, K), device=DEV).index_add_(0, group, dy.float()[:, :, None] * x.float()[:, None])
    assert torch.equal(dw, want.to(BF16)) and B.moe_get_device_error(ws) == 0
    K = 128
    x, w = x[:, :K].contiguous(), w[:, :, :K].contiguous()
    out = torch.empty_like(dy)
    B.moe_grouped_mm_mx(*quantized(x), *quantized(w), offsets, out, ws)
    assert torch.equal(out, torch.einsum("rk,rnk->rn", x.float(), w.float()[group]).to(BF16))


def test_operands_beyond_32_bits():
    """More than 2^32 bytes, and 2^31 elements, of matrices and of rows: the last group's values."""
    gen = torch.Generator(DEV).manual_seed(7)
    G, N, K = 5, 20480, 22000                               # 2.25e9 elements
    w = torch.zeros((G, N, K), dtype=BF16, device=DEV)
    w[-1] = whole(gen, (N, K), BF16, 1)
    for R in (6, 700):
        counts = [0, 1, 0, 1, R - 2]
        offsets, o = offsets_of(counts)
        x, dy = whole(gen, (R, K), BF16, 1), whole(gen, (R, N), BF16, 1)
        out = run(x, w, offsets, torch.full((R, N), 77.0, dtype=BF16, device=DEV))
        assert (out[:2] == 0).all() and torch.equal(out[2:], (x[2:].float() @ w[-1].float().t()).to(BF16))
        dx = run(dy, w, offsets, torch.full((R, K), 77.0, dtype=BF16, device=DEV), True)
        assert (dx[:2] == 0).all() and torch.equal(dx[2:], (dy[2:].float() @ w[-1].float()).to(BF16))
    dw = torch.full_like(w, 77.0)
    B.moe_grouped_wgrad(dy, x, offsets, dw, B.grouped_workspace(G))
    assert (dw[0] == 0).all() and (dw[2] == 0).all()
    assert torch.equal(dw[-1], (dy[2:].float().t() @ x[2:].float()).to(BF16))
    del w, dw
    R, K, N = 140_000, 16384, 8                             # 2.3e9 elements of x
    x = torch.zeros((R, K), dtype=BF16, device=DEV)
    x[-1000:] = whole(gen, (1000, K), BF16, 1)
    w = whole(gen, (2, N, K), BF16, 1)
    offsets, _ = offsets_of([R - 1000, 1000])
    out = run(x, w, offsets, torch.full((R, N), 77.0, dtype=BF16, device=DEV))
    assert (out[:-1000] == 0).all() and torch.equal(out[-1000:], (x[-1000:].float() @ w[1].float().t()).to(BF16))


def test_no_rows():
    x, w = torch.empty((0, 64), dtype=BF16, device=DEV), torch.ones((3, 72, 64), dtype=BF16, device=DEV)
    offsets, ws = torch.zeros((4,), dtype=torch.int32, device=DEV), B.grouped_workspace(3)
    out = torch.empty((0, 72), dtype=BF16, device=DEV)
    B.moe_grouped_mm(x, w, offsets, out, ws)
    B.moe_grouped_wgrad(out, x, offsets, w, ws)
    assert (w == 0).all()


def test_columns_of_one_tensor():
    """x and out as neighbouring columns of one wide tensor."""
    gen = torch.Generator(DEV).manual_seed(5)
    buf, w = whole(gen, (300, 64 + 128), BF16), whole(gen, (2, 128, 64), BF16)
    offsets, _ = offsets_of([100, 200])
    x = buf[:, :64].clone()
    run(buf[:, :64], w, offsets, buf[:, 64:])
    assert torch.equal(buf[:, :64], x)
    assert torch.equal(buf[:100, 64:], (x[:100].double() @ w[0].double().t()).to(BF16))


def test_captured_replayed_and_on_another_stream():
    gen = torch.Generator(DEV).manual_seed(6)
    x, dy, w = whole(gen, (700, 136), BF16), whole(gen, (700, 264), BF16), whole(gen, (4, 264, 136), BF16)
    offsets, _ = offsets_of([300, 0, 111, 289])
    out, dx, dw = torch.empty((700, 264), dtype=BF16, device=DEV), torch.empty_like(x), torch.empty_like(w)
    ws = B.grouped_workspace(4)

    def step():
        B.moe_grouped_mm(x, w, offsets, out, ws)
        B.moe_grouped_mm(dy, w, offsets, dx, ws, transposed=True)
        B.moe_grouped_wgrad(dy, x, offsets, dw, ws)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            step()
    # other group sizes in the captured call
    offsets.copy_(torch.tensor([0, 1, 400, 400, 700], dtype=torch.int32))
    for t in (out, dx, dw):
        t.fill_(77)
    graph.replay()
    torch.cuda.synchronize()
    o = [0, 1, 400, 400, 700]
    for g in range(4):
        a, b = o[g], o[g + 1]
        assert torch.equal(out[a:b], (x[a:b].double() @ w[g].double().t()).to(BF16))
        assert torch.equal(dx[a:b], (dy[a:b].double() @ w[g].double()).to(BF16))
        assert torch.equal(dw[g], (dy[a:b].double().t() @ x[a:b].double()).to(BF16))
    assert B.moe_get_device_error(ws) == 0


@pytest.mark.parametrize("counts,K,N", [([700, 0, 1031, 224, 449], 1664, 776), ([225, 31, 190, 97], 2048, 520), ([7, 0, 13] * 30, 2944, 1032)])
def test_mxfp8_of_many_blocks(counts, K, N):
    """Several tiles a group, and more k-blocks than are held at a time: whole numbers whose sums stay below
    2^24 units are exact."""
    gen = torch.Generator(DEV).manual_seed(K)
    offsets, o = offsets_of(counts, 2)
    R, G = o[-1] + 3, len(counts)
    x, w = whole(gen, (R, K), BF16, 8), whole(gen, (G, N, K), BF16, 8)
    xc, xs = quantized(x)
    wc, wss = quantized(w)
    xc[:2], xc[o[-1]:] = 0x7f, 0xff                         # NaN in rows of no group
    want = torch.full((R, N), 77.0, dtype=BF16, device=DEV)
    for g in range(G):
        want[o[g]:o[g + 1]] = (x[o[g]:o[g + 1]].double() @ w[g].double().t()).float().to(BF16)
    out, ws = torch.full((R, N), 77.0, dtype=BF16, device=DEV), B.grouped_workspace(G)
    for _ in range(3):
        B.moe_grouped_mm_mx(xc, xs, wc, wss, offsets, out, ws)
        assert B.moe_get_device_error(ws) == 0
        assert torch.equal(out, want)
        out.fill_(77.0)


def test_mxfp8_on_two_streams_and_replayed():
    """Two calls at a time, each with a workspace of its own, and a captured one replayed on new operands."""
    gen = torch.Generator(DEV).manual_seed(11)
    counts, K, N = [130, 0, 300, 5], 640, 520
    offsets, o = offsets_of(counts)
    sets = []
    for _ in range(3):
        x, w = whole(gen, (o[-1], K), BF16, 8), whole(gen, (len(counts), N, K), BF16, 8)
        want = torch.cat([(x[a:b].double() @ m.double().t()).float().to(BF16) for a, b, m in zip(o, o[1:], w)])
        sets.append((*quantized(x), *quantized(w), want, torch.empty_like(want), B.grouped_workspace(len(counts))))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, (xc, xs, wc, wss, _, out, ws) in zip(streams, sets):
            with torch.cuda.stream(s):
                B.moe_grouped_mm_mx(xc, xs, wc, wss, offsets, out, ws)
    torch.cuda.synchronize()
    for _, _, _, _, want, out, ws in sets[:2]:
        assert B.moe_get_device_error(ws) == 0 and torch.equal(out, want)
    xc, xs, wc, wss, _, out, ws = sets[2]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_grouped_mm_mx(xc, xs, wc, wss, offsets, out, ws)
    for other in sets[:2]:
        for dst, src in zip((xc, xs, wc, wss), other):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, other[4])
