"""mla_linear against its 64-bit form.

Bound of one value: the storage rounding (half a step of the result), K + 4
additions whose partial sums stay below S = |x| |w|^T + |bias| (2^-24 each), and
the float activation: SiLU and GELU have slopes below 1.13, __expf and the fast
division are off by less than 2^-20 of the value (|x| <= 88 enters exp with an
error of 2^-24 |x| more, which is below 2^-17 of a value that is at most x), erff
and the products by less than 2^-20 |x|.
"""
import pytest
import torch

from head_latent_attention_02_b200 import mla
from tests import chunk_reference as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HALF = {BF: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from head_latent_attention_02_b200 import build
    build.build()
    mla.lib()
    assert mla.get_status() == 0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ws(x, w, fill=0xff):
    """A workspace of NaN bits: nothing may rely on its contents."""
    return torch.full((max(mla.linear_workspace_size(x, w), 256),), fill, dtype=torch.uint8, device="cuda")


def _check(got, x, w, bias, act, residual, what=""):
    want = R.linear(x, w, bias, act, residual)
    size = x.double().abs() @ w.double().abs().T
    if bias is not None:
        size = size + bias.double().abs()
    pre = R.linear(x, w, bias).abs()
    tol = HALF[got.dtype] * want.abs() + 1.13 * (x.shape[1] + 4) * 2.0 ** -24 * size + 2.0 ** -23 * want.abs()
    if act != "none":
        tol = tol + 2.0 ** -17 * pre
    if residual is not None:
        tol = tol + 2.0 ** -24 * residual.double().abs()
    off = (got.double() - want).abs()
    assert off.le(tol).all(), f"{what}: {float((off - tol).max())}"


def _run(dt, M, N, K, bias, act, res, seed=0):
    g = _gen(M * 7 + N * 3 + K + seed)
    x = torch.randn(M, K, device="cuda", generator=g).to(dt)
    w = (torch.randn(N, K, device="cuda", generator=g) / K ** 0.5).to(dt)
    b = torch.randn(N, device="cuda", generator=g) if bias else None
    r = torch.randn(M, N, device="cuda", generator=g).to(dt) if res else None
    out = torch.full((M, N), float("nan"), device="cuda", dtype=dt)
    mla.linear(x, w, out, bias=b, act=act, residual=r, workspace=_ws(x, w))
    assert mla.get_status() == 0
    _check(out, x, w, b, act, r, (M, N, K))


@pytest.mark.parametrize("M", [1, 2, 16, 33, 128, 129, 256, 300, 1000])
@pytest.mark.parametrize("N,K", [(8, 64), (257, 1000), (1000, 72), (2056, 2048)])
@pytest.mark.parametrize("bias,act,res", [(False, "none", False), (True, "silu", True), (True, "gelu", False)])
def test_bf16(M, N, K, bias, act, res):
    _run(BF, M, N, K, bias, act, res)


@pytest.mark.parametrize("M,N,K", [
    (16, 7168, 4096),      # split along K, W on the tile's rows
    (4, 300, 16384),       # few tiles, long K: many partial sums a tile
    (700, 520, 8192),      # split, x on the tile's rows
    (3000, 5120, 640),     # full rounds of tiles and tiles left over
    (2600, 4700, 1288),    # two column blocks a tile, ragged edges
])
def test_bf16_splits_and_rounds(M, N, K):
    _run(BF, M, N, K, True, "none", True)


@pytest.mark.parametrize("M,N,K", [(3, 5, 7), (1, 1, 1), (40, 70, 33), (130, 9, 17), (1, 200, 8), (20, 64, 12)])
def test_bf16_rows_that_take_no_tma(M, N, K):
    for act, bias, res in [("none", False, False), ("silu", True, True)]:
        _run(BF, M, N, K, bias, act, res)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 70, 129), (100, 64, 1000), (513, 65, 40), (600, 130, 33)])
@pytest.mark.parametrize("bias,act,res", [(False, "none", False), (True, "silu", True), (True, "gelu", True)])
def test_f32(M, N, K, bias, act, res):
    _run(torch.float32, M, N, K, bias, act, res)


@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("M", [5, 300])
def test_strided_operands_leave_the_rest_alone(dt, M):
    g = _gen(5)
    N, K = 200, 256
    for pad in (8, 3):              # 3: rows that are not 16-byte aligned
        x = torch.randn(M, K + pad, device="cuda", generator=g).to(dt)[:, :K]
        w = (torch.randn(N, 2 * K + pad, device="cuda", generator=g) / 16).to(dt)[:, :K]
        r = torch.randn(M, N + pad, device="cuda", generator=g).to(dt)[:, pad:]
        whole = torch.full((M + 2, N + 2 * pad), float("nan"), device="cuda", dtype=dt)
        out = whole[1:M + 1, pad:pad + N]
        mla.linear(x, w, out, residual=r, workspace=_ws(x, w))
        _check(out, x, w, None, "none", r, pad)
        keep = torch.ones_like(whole, dtype=torch.bool)
        keep[1:M + 1, pad:pad + N] = False
        assert torch.isnan(whole[keep]).all()


@pytest.mark.parametrize("M,N,K", [(16, 1024, 8192), (300, 512, 512)])
def test_residual_in_place(M, N, K):
    g = _gen(6)
    x = torch.randn(M, K, device="cuda", generator=g).to(BF)
    w = (torch.randn(N, K, device="cuda", generator=g) / K ** 0.5).to(BF)
    r = torch.randn(M, N, device="cuda", generator=g).to(BF)
    out = r.clone()
    mla.linear(x, w, out, residual=out, workspace=_ws(x, w))
    _check(out, x, w, None, "none", r)


@pytest.mark.parametrize("M", [7, 400])
def test_infinities_and_nan_stay_in_their_row_or_column(M):
    g = _gen(8)
    N, K = 264, 520
    x = torch.randn(M, K, device="cuda", generator=g).to(BF)
    w = torch.randn(N, K, device="cuda", generator=g).to(BF)
    x[3, 5] = float("nan")
    w[77, 9] = float("inf")
    out = torch.zeros(M, N, device="cuda", dtype=BF)
    mla.linear(x, w, out, workspace=_ws(x, w))
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[3], bad[:, 77] = True, True
    assert torch.isfinite(out[~bad]).all() and not torch.isfinite(out[bad]).any()
    assert torch.isnan(out[3]).all()


@pytest.mark.parametrize("M,N,K", [(16, 7168, 4096), (700, 520, 8192)])
def test_split_sums_do_not_depend_on_timing(M, N, K):
    g = _gen(9)
    x = torch.randn(M, K, device="cuda", generator=g).to(BF)
    w = torch.randn(N, K, device="cuda", generator=g).to(BF)
    assert mla.linear_workspace_size(x, w) > 0
    outs = []
    for i in range(3):
        out = torch.empty(M, N, device="cuda", dtype=BF)
        mla.linear(x, w, out, workspace=_ws(x, w, fill=i))
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_workspace_is_asked_for():
    x = torch.randn(16, 8192, device="cuda").to(BF)
    w = torch.randn(7168, 8192, device="cuda").to(BF)
    out = torch.full((16, 7168), float("nan"), device="cuda", dtype=BF)
    need = mla.linear_workspace_size(x, w)
    assert need > 0
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device="cuda")):
        with pytest.raises(mla.MLAError) as e:
            mla.linear(x, w, out, workspace=ws)
        assert e.value.code == 3
    with pytest.raises(mla.MLAError) as e:
        mla.linear(x, w, out, workspace=torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:])
    assert e.value.code == 1
    assert torch.isnan(out).all()


def test_two_streams_and_a_replayed_graph():
    g = _gen(10)
    xs = [torch.randn(16, 4096, device="cuda", generator=g).to(BF) for _ in range(2)]
    w = (torch.randn(2048, 4096, device="cuda", generator=g) / 64).to(BF)
    outs = [torch.empty(16, 2048, device="cuda", dtype=BF) for _ in range(2)]
    wss = [_ws(xs[0], w) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for i, s in enumerate(streams):
            mla.linear(xs[i], w, outs[i], workspace=wss[i], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        _check(outs[i], xs[i], w, None, "none", None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        mla.linear(xs[0], w, outs[0], workspace=wss[0])
        mla.linear(xs[1], w, outs[1], workspace=wss[0])       # one workspace, in order
    xs[0].normal_(generator=g)
    xs[1].normal_(generator=g)
    graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        _check(outs[i], xs[i], w, None, "none", None)


def _passed_on(dt, M, N, K, values, act):
    """act of given values, each the whole of a sum: x holds them in its first column, w ones."""
    v = torch.tensor(values, dtype=torch.float64, device="cuda").to(dt)
    x = torch.zeros(M, K, device="cuda", dtype=dt)
    x[:, 0] = v[torch.arange(M, device="cuda") % len(values)]
    w = torch.zeros(N, K, device="cuda", dtype=dt)
    w[:, 0] = 1
    out = torch.full((M, N), float("nan"), device="cuda", dtype=dt)
    mla.linear(x, w, out, act=act, workspace=_ws(x, w))
    assert mla.get_status() == 0
    return x[:, :1].double(), out.double()


SHAPES = [(BF, 4, 300, 16384), (BF, 100, 264, 512), (BF, 300, 520, 512), (BF, 5, 9, 7), (torch.float32, 40, 70, 33)]


@pytest.mark.parametrize("dt,M,N,K", SHAPES)
def test_gelu_of_negative_values(dt, M, N, K):
    """Relative to the result, which is small there: v / sqrt 2 is off by 1.5 * 2^-24, which erfc makes
    v^2 + 1 times larger, erfc itself by 4 of its last places (2^-21), two products by 2^-24 each.  (The
    tensor-core kernel's form: half of v^2, twice rounded, enters an exponential that is off by 2^-22; its
    polynomial by less than 2^-21.  No more than that.)"""
    values = [-12, -9.5, -8, -7, -6, -5.5, -5, -4, -3, -1, -0.25, 0.0, 0.5, 2, 5, 30]
    v, got = _passed_on(dt, M, N, K, values, "gelu")
    want = 0.5 * v * torch.special.erfc(-v / 2 ** 0.5)
    tol = (HALF[dt] + (1.5 * (v * v + 1) + 10) * 2.0 ** -24) * want.abs()
    tol = torch.where(v > 0, (HALF[dt] + 2.0 ** -20) * want.abs(), tol)
    assert (got - want).abs().le(tol * (1 + HALF[dt])).all()


@pytest.mark.parametrize("dt,M,N,K", SHAPES)
def test_silu_of_far_negative_values(dt, M, N, K):
    """Relative to the result, down to 3e-37: __expf(v) is off by 2 + 1.17 |v| of its last places, what
    follows by four more; below 2^-126 an exponential has a step of 2^-149."""
    values = [-89.5, -89, -88.5, -88, -87.5, -80, -20, -3, -0.5, 0.0, 1, 40, 90]
    v, got = _passed_on(dt, M, N, K, values, "silu")
    want = v / (1 + torch.exp(-v))
    tol = (HALF[dt] + (6 + 1.17 * v.abs()) * 2.0 ** -23) * want.abs() + v.abs() * 2.0 ** -149
    assert (got - want).abs().le(tol * (1 + HALF[dt])).all()
