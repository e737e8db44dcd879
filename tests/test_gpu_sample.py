"""Sampling against its 64-bit form, row by row: every filter alone and together, vocabularies from one token to more
than shared memory holds, ties, masked rows, infinities, NaN, extreme temperatures, strides, both logit types.

Tokens have to be equal: each weight is right to 2^-27 of itself and the sums are exact, so a token could differ only
where u, top_p or min_p falls within 2^-27 of a border (less than 1e-6 a row), which these seeds do not meet.
Log-probabilities: the ratio of a weight and a sum, each right to 2^-27 (2^-26 absolute in the logarithm), and the fp32
rounding of the result (2^-24 relative)."""
import math

import pytest
import torch

import nvfp4_weight_only_flint_b200 as fm
import paged_ref as R

pytestmark = pytest.mark.gpu


def _logits(seed, rows, V, dtype=torch.float32, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, V), generator=g) * spread
    hot = torch.randint(0, V, (rows, min(V, 60)), generator=g)
    x.scatter_add_(1, hot, 4.0 + 6.0 * torch.rand(hot.shape, generator=g))
    return x.to(dtype)


def _run(x, t=None, k=None, p=None, m=None, u=None, status=None, stride=None, lp=True):
    rows, V = x.shape
    dev = lambda v, dt: None if v is None else torch.tensor(v, dtype=dt).cuda()  # noqa: E731
    stride = V if stride is None else stride
    buf = torch.full((rows * stride,), math.nan, dtype=x.dtype)
    for r in range(rows):
        buf[r * stride:r * stride + V] = x[r]
    buf = buf.cuda()
    tok = torch.full((rows,), -99, dtype=torch.int32, device="cuda")
    logp = torch.full((rows,), math.nan, device="cuda") if lp else None
    fm.flint_sample(buf, rows, V, stride, fm.FLINT_LOGITS_F32 if x.dtype == torch.float32 else fm.FLINT_LOGITS_BF16,
                    dev(t, torch.float32), dev(k, torch.int32), dev(p, torch.float32), dev(m, torch.float32),
                    dev(u, torch.float32), tok, logp, status)
    torch.cuda.synchronize()
    return tok.cpu(), logp.cpu() if lp else None


def _check(x, t=None, k=None, p=None, m=None, u=None, **kw):
    rows = x.shape[0]
    tok, logp = _run(x, t, k, p, m, u, **kw)
    f32 = lambda v, i, d: d if v is None else float(torch.tensor(v[i], dtype=torch.float32))  # noqa: E731
    for r in range(rows):
        want, lw = R.sample(x[r].double(), f32(t, r, 1.0), 0 if k is None else k[r], f32(p, r, 1.0), f32(m, r, 0.0),
                            f32(u, r, 0.0))
        assert int(tok[r]) == want, (r, int(tok[r]), want)
        assert abs(float(logp[r]) - lw) <= 2 ** -23 * abs(lw) + 2 ** -26, (r, float(logp[r]), lw)


def _u(seed, rows):
    return torch.rand(rows, generator=torch.Generator().manual_seed(seed)).tolist()


@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4096, 4097, 9999, 32768, 150144])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_filters(V, dtype):
    kinds = [(1.0, 0, 1.0, 0.0), (0.8, 50, 0.9, 0.0), (0.7, 40, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.3, 0, 0.99, 0.0),
             (1.2, 0, 1.0, 0.05), (0.0, 0, 1.0, 0.0), (0.9, 1000, 0.95, 0.02), (1.0, 1, 1.0, 0.0), (2.0, V - 1, 0.5, 0.0),
             (5.0, 0, 0.9999, 0.0), (1.0, V, 1.0, 0.0)]
    x = _logits(V, len(kinds), V, dtype)
    _check(x, *[[q[i] for q in kinds] for i in range(4)], _u(V, len(kinds)))


def test_sample_larger_than_shared_memory():
    V = 900_001  # above what eight CTAs hold
    kinds = [(1.0, 0, 1.0, 0.0), (0.8, 50, 0.9, 0.0), (1.0, 0, 0.95, 0.0), (1.0, 0, 1.0, 0.1)]
    _check(_logits(7, 4, V), *[[q[i] for q in kinds] for i in range(4)], _u(8, 4))


@pytest.mark.parametrize("rows,V", [(37, 65_600), (60, 70_001), (2, 376_832), (2, 376_833), (3, 400_003)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_shares_held_and_read_again(rows, V, dtype):
    # up to 376,832 tokens (8 CTAs of 47,104) the row is held in shared memory
    kinds = [(1.0, 0, 1.0, 0.0), (0.8, 50, 0.9, 0.0), (1.0, 0, 0.95, 0.0), (1.0, 0, 1.0, 0.1), (0.0, 0, 1.0, 0.0)]
    _check(_logits(rows, rows, V, dtype), *[[kinds[r % 5][i] for r in range(rows)] for i in range(4)], _u(9, rows))


def test_sample_defaults_and_no_logprobs():
    x = _logits(3, 5, 2000)
    _check(x, u=_u(3, 5))
    a, _ = _run(x, u=_u(3, 5))
    b, none = _run(x, u=_u(3, 5), lp=False)
    assert none is None and torch.equal(a, b)


@pytest.mark.parametrize("stride", [1001, 1002, 1004, 1500])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_strided_rows(stride, dtype):
    _check(_logits(stride, 6, 1001, dtype), t=[0.9] * 6, k=[20, 0, 7, 0, 0, 100], p=[0.9, 0.8, 1.0, 1.0, 0.3, 0.95],
           m=[0.0, 0.0, 0.0, 0.2, 0.0, 0.01], u=_u(stride, 6), stride=stride)


def test_sample_ties_go_to_the_lowest_index():
    V = 10_000
    x = torch.zeros((6, V))
    x[1, 5000:] = 1.0
    x[2] = torch.arange(V) % 3
    x[3, ::2] = -0.0  # equals +0
    x[4] = -math.inf
    x[4, 17::100] = 3.5
    # the exactly halved mass: of V equal tokens, V / 2 hold half
    _check(x, [1.0] * 6, [5, 3000, 4000, 7, 30, 0], [1.0, 0.5, 0.75, 1.0, 0.5, 0.5], [0.0] * 6,
           [0.999, 0.5, 0.25, 0.875, 0.0, 0.9999])
    _check(x, [0.0] * 6, u=[0.5] * 6)


def test_sample_every_u_of_a_small_row():
    x = torch.tensor([[0.0, 1.0, -math.inf, 0.5]]).repeat(65, 1)
    _check(x, u=[min(i / 64, 1 - 2 ** -24) for i in range(65)])
    w = torch.tensor([[0.0] * 4]).repeat(8, 1)  # exact borders: u = 1/4 is the second token's first
    tok, _ = _run(w, u=[0.0, 0.25, 0.5, 0.75, 0.2499, 0.4999, 0.7499, 0.9999])
    assert tok.tolist() == [0, 1, 2, 3, 0, 1, 2, 3]


def test_sample_masked_rows_and_infinities():
    V = 5000
    x = _logits(11, 7, V)
    x[0] = -math.inf                 # nothing to sample
    x[1] = -math.inf
    x[1, 4321] = -5.0                # one token left
    x[2, 100], x[2, 200] = math.inf, math.inf   # two infinite ones share the mass
    x[3, ::2] = math.nan             # NaN counts as masked
    x[4] = torch.finfo(torch.float32).min       # the type's lowest value everywhere
    x[5, 1:] = torch.finfo(torch.float32).min
    x[6] = math.nan
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    u = _u(12, 7)
    for k, p, m in (([0] * 7, [1.0] * 7, [0.0] * 7), ([10] * 7, [0.9] * 7, [0.05] * 7), ([4999] * 7, [0.999] * 7, [0.0] * 7)):
        st.zero_()
        tok, lp = _run(x, [0.9] * 7, k, p, m, u, status=st)
        assert int(st.item()) == fm.FLINT_DEVCHECK_NONFINITE
        assert int(tok[0]) == -1 and int(tok[6]) == -1 and float(lp[0]) == -math.inf
        for r in range(1, 6):
            f = lambda v: float(torch.tensor(v[r], dtype=torch.float32))  # noqa: E731
            want, lw = R.sample(x[r].double(), f([0.9] * 7), k[r], f(p), f(m), f(u))
            assert int(tok[r]) == want, r
            assert abs(float(lp[r]) - lw) <= 2 ** -23 * abs(lw) + 2 ** -26
    assert _run(x, [0.0] * 7, u=u)[0].tolist()[1:3] == [4321, 100]
    # the same where the row is not held in shared memory
    long = x[2:3].repeat(8, 80)  # 400,000 tokens
    tok, lp = _run(long, [0.9] * 8, [0] * 8, [1.0] * 8, [0.0] * 8, _u(13, 8))
    want = {100 + V * i for i in range(80)} | {200 + V * i for i in range(80)}
    assert set(tok.tolist()) <= want and abs(float(lp[0]) + math.log(160)) < 1e-6


@pytest.mark.parametrize("t", [1e-44, 1e-30, 1e-3, 0.05, 20.0, 1e6, math.inf])
def test_sample_extreme_temperatures(t):
    x = _logits(21, 4, 20_000)
    _check(x, [t] * 4, [0, 500, 0, 0], [1.0, 0.9, 0.9, 1.0], [0.0, 0.0, 0.0, 0.3], _u(22, 4))


def test_sample_infinite_temperature_with_min_p():
    # every weight is 1: min-p of 1 keeps them all
    x = _logits(23, 4, 5000)
    _check(x, [math.inf] * 4, [0, 0, 700, 20], [1.0, 0.9, 1.0, 1.0], [1.0, 1.0, 2.0, 0.5], _u(24, 4))


@pytest.mark.parametrize("k", [255, 256, 257, 511, 512, 513, 1024, 1025, 3000])
def test_sample_prefix_sizes(k):
    # prefixes on both sides of every form's limit: counted ranks, sorted, narrowed
    x = _logits(k, 6, 20_000, spread=3.0)
    _check(x, [1.0] * 6, [k] * 6, [1.0, 0.9, 0.999, 1.0, 0.5, 1.0], [0.0, 0.0, 0.0, 0.01, 0.0, 1e-6], _u(k, 6))


@pytest.mark.parametrize("spread", [0.01, 0.5, 6.0, 40.0])
def test_sample_flat_and_steep_rows(spread):
    # top-p ends within the near bins, below them, among one bin's many tokens
    x = torch.randn((8, 30_000), generator=torch.Generator().manual_seed(5)) * spread
    _check(x, [1.0] * 8, [0, 0, 0, 0, 700, 300, 50, 29_999], [0.1, 0.5, 0.9, 0.9999999, 0.9, 0.5, 0.99, 0.3], [0.0] * 8,
           _u(6, 8))


def test_sample_top_k_of_crowded_bins():
    # thousands of tokens within a bin of the k-th: the gather is given up
    x = torch.full((4, 50_000), -1.0) + torch.rand((4, 50_000), generator=torch.Generator().manual_seed(9)) * 0.01
    _check(x, [1.0] * 4, [50, 500, 5, 100], [1.0, 0.9, 0.5, 1.0], [0.0] * 4, _u(10, 4))


def test_sample_filters_at_their_ends():
    x = _logits(31, 8, 3000)
    _check(x, [1.0] * 8, [0, -3, 3000, 5000, 1, 2, 0, 0], [0.0, -1.0, 1e-9, 2.0, 0.5, 1.0, 1.0, 1 - 2 ** -24],
           [0.0, 0.0, 0.0, -1.0, 0.0, 1.0, 7.0, 0.0], _u(32, 8))


def test_sample_many_rows_are_the_single_ones():
    x = _logits(41, 300, 700)
    g = torch.Generator().manual_seed(42)
    k = torch.randint(-1, 800, (300,), generator=g).tolist()
    p = torch.rand(300, generator=g).tolist()
    m = (torch.rand(300, generator=g) * 0.1).tolist()
    t = (torch.rand(300, generator=g) * 2).tolist()
    _check(x, t, k, p, m, _u(43, 300))


def test_sample_bad_parameters_give_no_token():
    x = _logits(51, 6, 500)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = [1.0, -1.0, math.nan, 1.0, 1.0, 1.0]
    u = [0.5, 0.5, 0.5, 1.0, -0.1, math.nan]
    tok, lp = _run(x, t, u=u, status=st)
    assert int(st.item()) == fm.FLINT_DEVCHECK_INDEX
    assert tok.tolist()[1:] == [-1] * 5 and int(tok[0]) >= 0 and float(lp[1]) == -math.inf


def test_sample_repeats_and_replays():
    x = _logits(61, 16, 150144).cuda()
    f = lambda v: torch.full((16,), v, device="cuda")  # noqa: E731
    t, p, m = f(1.1), f(0.97), f(0.0)
    k = torch.zeros(16, dtype=torch.int32, device="cuda")
    u = torch.tensor(_u(62, 16)).cuda()
    tok, lp = torch.zeros(16, dtype=torch.int32, device="cuda"), f(0.0)
    call = lambda: fm.flint_sample(x, 16, 150144, 150144, fm.FLINT_LOGITS_F32, t, k, p, m, u, tok, lp)  # noqa: E731
    call()
    torch.cuda.synchronize()
    first = tok.clone(), lp.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(5):
        tok.zero_(), lp.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(tok, first[0]) and torch.equal(lp, first[1])
    side = torch.cuda.Stream()  # two calls at once
    tok2 = torch.zeros_like(tok)
    side.wait_stream(torch.cuda.current_stream())
    call()
    with torch.cuda.stream(side):
        fm.flint_sample(x, 16, 150144, 150144, fm.FLINT_LOGITS_F32, t, k, p, m, u, tok2, None)
    torch.cuda.synchronize()
    assert torch.equal(tok, first[0]) and torch.equal(tok2, first[0])


def test_sample_refuses_tensors_it_would_read_wrongly():
    x = torch.zeros((4, 200), device="cuda")
    u, tok = torch.zeros(4, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    call = lambda **k: fm.flint_sample(**{**dict(logits=x, rows=4, vocab=200, row_stride=200,  # noqa: E731
                                                 logits_dtype=fm.FLINT_LOGITS_F32, temperature=None, top_k=None,
                                                 top_p=None, min_p=None, u=u, tokens=tok), **k})
    call()
    for bad in (dict(logits=x[:, ::2]), dict(logits=x[:2]), dict(u=u[:3]), dict(tokens=tok.cpu()), dict(row_stride=300),
                dict(logits=x.to_sparse()), dict(top_k=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(fm.FlintError) as e:
            call(**bad)
        assert e.value.code == -1


@pytest.mark.parametrize("V", [1000, 20_001, 150_144, 400_000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_log_probability_of_a_light_token(V, dtype):
    # u = 0 draws the first token, of a few units of mass only; every form of the draw (ranks counted, sorted, whole row)
    x = torch.full((7, V), -math.inf)
    x[:, 0] = torch.tensor([-29.0, -30.0, -29.5, -28.7, -25.0, -20.0, -29.25])
    x[:, V // 2:V // 2 + 40] = torch.linspace(-1, 0, 40)
    x[2, V // 4:V // 4 + 200] = torch.linspace(-3, -2, 200)
    x[3, V // 4:V // 4 + 240] = torch.linspace(-3, -2, 240)
    x[5, :V // 8] = -20.0
    x[6] = x[6].clamp_min(-29.25)
    _check(x.to(dtype), [1.0] * 7, [0, 60, 500, 300, 700, 0, 0], [1.0] * 7, [0.0] * 7, [0.0] * 7)
